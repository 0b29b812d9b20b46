"""The operators between the embedding lookup and the head loss, with the C
ABI's names: attention over packed sequences, the norms around a block fused
with its gate and residual scale, and gradient clipping over many tensors.
PyTorch provides device memory and the current stream; the arithmetic is all
in liblce.so.

With `stream` given, the call's outputs and scratch are allocated for that
stream; as for the library's other calls, inputs made on another stream have
to be ready there (and stay alive until that stream is done with them)."""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _abi

_DT = {torch.bfloat16: _abi.LCE_BF16, torch.float32: _abi.LCE_FP32}
_NOTHING = contextlib.nullcontext()


def _on(stream):
    """Allocations inside belong to `stream` (None: the current one)."""
    return _NOTHING if stream is None else torch.cuda.stream(stream)


def _stream(stream, device) -> int:
    return int((torch.cuda.current_stream(device) if stream is None else stream).cuda_stream)


def _scratch(given, need: int, device):
    """(address, bytes, tensor to keep) of a call's scratch."""
    if need == 0:
        return None, 0, None
    if given is None:
        given = torch.empty(need, dtype=torch.uint8, device=device)
    elif not given.is_cuda or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return given.data_ptr(), given.numel() * given.element_size(), given


# ------------------------------------------------------------------ attention

def _check_heads(name, t, ref, shape=None):
    if not t.is_cuda or t.device != ref.device:
        raise ValueError(f"{name} must be a CUDA tensor on q's device (there is no CPU path)")
    if t.dtype != ref.dtype:
        raise ValueError(f"{name} must have q's dtype")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")


def _tokens(name, t):
    """A [B, L, heads, D] tensor as [B*L, heads, D], without a copy."""
    if t.dim() == 3:
        return t
    B, L, H, D = t.shape
    if B > 1 and L > 0 and t.stride(0) != L * t.stride(1):
        raise ValueError(f"{name}: the rows of a [B, L, heads, D] tensor must be evenly spaced over B and L")
    return t.as_strided((B * L, H, D), (t.stride(1), t.stride(2), t.stride(3)))


def _strides(t):
    """Token and head strides; a dimension of one entry has none of its own."""
    T, H, D = t.shape
    return (t.stride(0) if T > 1 else H * D), (t.stride(1) if H > 1 else D)


def _attn_args(q, k, v, cu_q, cu_k, causal, scale):
    if q.dtype not in _DT or not q.is_cuda:
        raise ValueError("q must be a bfloat16 or float32 CUDA tensor (there is no CPU path)")
    if q.dim() not in (3, 4) or k.dim() != q.dim() or v.shape != k.shape:
        raise ValueError("q must be [Tq, heads, D] and k, v [Tk, kv_heads, D] (or all [B, L, heads, D])")
    if k.shape[-1] != q.shape[-1] or (q.dim() == 4 and k.shape[0] != q.shape[0]):
        raise ValueError("shape mismatch between q, k and v")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_heads(name, t, q)
    batch = q.shape[0] if q.dim() == 4 else 1
    q, k, v = _tokens("q", q), _tokens("k", k), _tokens("v", v)
    a = _abi.LceAttn()
    if cu_q is not None or cu_k is not None:
        if batch != 1:
            raise ValueError("sequence offsets go with [T, heads, D] tensors")
        cu_q = cu_k if cu_q is None else cu_q
        cu_k = cu_q if cu_k is None else cu_k
        for name, c in (("cu_seqlens_q", cu_q), ("cu_seqlens_k", cu_k)):
            if c.dtype != torch.int32 or c.dim() != 1 or c.device != q.device or not c.is_contiguous() or c.numel() < 2:
                raise ValueError(f"{name} must be a contiguous int32 tensor of at least two offsets on q's device")
        if cu_q.numel() != cu_k.numel():
            raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
        batch = cu_q.numel() - 1
        a.cu_q, a.cu_k = cu_q.data_ptr(), cu_k.data_ptr()
    Tq, Hq, D = q.shape
    Tk, Hk, _ = k.shape
    if Hq < 1 or Hk < 1 or Hq % Hk:
        raise ValueError("the number of query heads must be a multiple of the number of key heads")
    a.dtype, a.causal, a.scale = _DT[q.dtype], 1 if causal else 0, D ** -0.5 if scale is None else scale
    a.B, a.Tq, a.Tk, a.Hq, a.Hk, a.D = max(batch, 1), Tq, Tk, Hq, Hk, D
    a.q, a.k, a.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    a.q_ts, a.q_hs = _strides(q)
    a.k_ts, a.k_hs = _strides(k)
    a.v_ts, a.v_hs = _strides(v)
    return a


def attention_workspace_size(Tq: int, Tk: int, Hq: int, Hk: int, D: int, batch: int = 1, dtype=torch.bfloat16) -> int:
    """Bytes of scratch attention_backward needs (`batch`: the number of sequences)."""
    a = _abi.LceAttn()
    # equal lengths are not asked for here: a stand-in for the offsets
    a.cu_q = a.cu_k = 16
    a.dtype, a.B, a.Tq, a.Tk, a.Hq, a.Hk, a.D = _DT[dtype], batch, Tq, Tk, Hq, Hk, D
    return int(_abi.lib().lce_attention_workspace_size(ctypes.byref(a)))


def attention_forward(q, k, v, cu_seqlens_q=None, cu_seqlens_k=None, *, causal: bool = True, scale=None, out=None,
                      stream=None):
    """(o, lse) of softmax attention over packed sequences: q [Tq, heads, D],
    k and v [Tk, kv_heads, D] with int32 token offsets of the sequences (one
    sequence without them), or [B, L, heads, D] tensors of equal lengths. o has
    q's shape and dtype, lse is fp32 [heads, tokens]; rows that see no key get
    o = 0 and lse = -inf. `scale` is D**-0.5 if not given; `out` receives o."""
    a = _attn_args(q, k, v, cu_seqlens_q, cu_seqlens_k, causal, scale)
    with _on(stream):
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        else:
            _check_heads("out", out, q, q.shape)
        lse = torch.empty((a.Hq, a.Tq), dtype=torch.float32, device=q.device)
        o = _tokens("out", out)
        a.o, (a.o_ts, a.o_hs) = o.data_ptr(), _strides(o)
        a.lse = lse.data_ptr()
        a.stream = _stream(stream, q.device)
        _abi.check(_abi.lib().lce_attention_forward(ctypes.byref(a)), "lce_attention_forward")
    return out, lse


def attention_backward(do, q, k, v, o, lse, cu_seqlens_q=None, cu_seqlens_k=None, *, causal: bool = True, scale=None,
                       dq=None, dk=None, dv=None, workspace=None, stream=None):
    """(dq, dk, dv) from the forward's inputs, its o and lse, and the gradient
    `do` of o; the probabilities are recomputed. dq, dk and dv may be given
    (strided slices of one gradient, say). `workspace`: a uint8 CUDA tensor of
    at least attention_workspace_size bytes."""
    a = _attn_args(q, k, v, cu_seqlens_q, cu_seqlens_k, causal, scale)
    _check_heads("do", do, q, q.shape)
    _check_heads("o", o, q, q.shape)
    if lse.dtype != torch.float32 or lse.shape != (a.Hq, a.Tq) or not lse.is_contiguous() or lse.device != q.device:
        raise ValueError("lse must be the forward's contiguous fp32 [heads, tokens] tensor")
    with _on(stream):
        grads = []
        for name, g, ref in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            if g is None:
                g = torch.empty(ref.shape, dtype=ref.dtype, device=ref.device)
            else:
                _check_heads(name, g, q, ref.shape)
            grads.append(g)
        d, p = _tokens("do", do), _tokens("o", o)
        a.dO, (a.dO_ts, a.dO_hs) = d.data_ptr(), _strides(d)
        a.o, (a.o_ts, a.o_hs) = p.data_ptr(), _strides(p)
        a.lse = lse.data_ptr()
        x, y, z = (_tokens(n, g) for n, g in zip(("dq", "dk", "dv"), grads))
        a.dq, (a.dq_ts, a.dq_hs) = x.data_ptr(), _strides(x)
        a.dk, (a.dk_ts, a.dk_hs) = y.data_ptr(), _strides(y)
        a.dv, (a.dv_ts, a.dv_hs) = z.data_ptr(), _strides(z)
        lib = _abi.lib()
        a.workspace, a.workspace_bytes, keep = _scratch(workspace, lib.lce_attention_workspace_size(ctypes.byref(a)),
                                                        q.device)
        a.stream = _stream(stream, q.device)
        _abi.check(lib.lce_attention_backward(ctypes.byref(a)), "lce_attention_backward")
        del keep
    return tuple(grads)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k, causal, scale):
        o, lse = attention_forward(q, k, v, cu_q, cu_k, causal=causal, scale=scale)
        ctx.save_for_backward(q, k, v, o, lse, cu_q, cu_k)
        ctx.causal, ctx.scale = causal, scale
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, cu_q, cu_k = ctx.saved_tensors
        # autograd may hand over an expanded or permuted gradient, whose rows the kernels cannot read
        dq, dk, dv = attention_backward(do.contiguous(), q, k, v, o, lse, cu_q, cu_k, causal=ctx.causal, scale=ctx.scale)
        need = ctx.needs_input_grad
        return dq if need[0] else None, dk if need[1] else None, dv if need[2] else None, None, None, None, None


def attention(q, k, v, cu_seqlens_q=None, cu_seqlens_k=None, *, causal: bool = True, scale=None):
    """Autograd form of attention_forward (returns o)."""
    return _Attention.apply(q, k, v, cu_seqlens_q, cu_seqlens_k, causal, scale)


# ---------------------------------------------------------------- block norms

def _rows(name, t, ref):
    """Row stride of a [N, d] tensor whose rows are contiguous."""
    if t.device != ref.device or t.dtype != ref.dtype or t.shape != ref.shape:
        raise ValueError(f"{name} must be a {tuple(ref.shape)} tensor of the same dtype and device")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _at(t):
    """A tensor's address; without elements some other than NULL, which would mean no tensor (it is not read)."""
    return t.data_ptr() or 16


def _norm_args(ref, b, w_post, gate, w_pre, scale, eps):
    if ref.dtype not in _DT or not ref.is_cuda or ref.dim() != 2:
        raise ValueError("the stream must be a bfloat16 or float32 CUDA tensor [N, d] (there is no CPU path)")
    a = _abi.LceNorm()
    a.dtype, (a.N, a.d), a.scale, a.eps = _DT[ref.dtype], ref.shape, scale, eps
    for name, w in (("w_post", w_post), ("w_pre", w_pre)):
        if w is not None:
            if w.device != ref.device or w.dtype != ref.dtype or w.shape != (ref.shape[1],) or not w.is_contiguous():
                raise ValueError(f"{name} must be a contiguous [d] tensor of the stream's dtype")
            setattr(a, name, w.data_ptr())
    if b is None:
        if w_post is not None or gate is not None or w_pre is None:
            raise ValueError("without b there is only the norm by w_pre")
    else:
        a.b, a.ld_b = _at(b), _rows("b", b, ref)
    if gate is not None:
        if gate.dim() == 2:
            a.gate_full, a.ld_gate = 1, _rows("gate", gate, ref)
        elif gate.device != ref.device or gate.dtype != ref.dtype or gate.shape != (ref.shape[1],) or not gate.is_contiguous():
            raise ValueError("gate must be [d] (contiguous) or [N, d], of the stream's dtype")
        a.gate = _at(gate)
    return a


def block_norm_workspace_size(N: int, d: int) -> int:
    """Bytes of scratch block_norm_backward needs."""
    a = _abi.LceNorm()
    a.N, a.d = N, d
    return int(_abi.lib().lce_block_norm_workspace_size(ctypes.byref(a)))


def block_norm_forward(x, b=None, *, w_post=None, gate=None, w_pre=None, scale: float = 1.0, eps: float = 1e-6,
                       out_r=None, stream=None):
    """(r, n, rstd_post, rstd_pre) for the residual stream x [N, d] and a
    block's output b [N, d]:
        r = x + scale * gate * rms_norm(b) * w_post,   n = rms_norm(r) * w_pre
    with gate [d] or [N, d]; any of w_post, gate and w_pre may be None (n and
    the matching rstd are None then). Without b, r is x itself. `out_r`
    receives r and may be x (the stream updated in place)."""
    a = _norm_args(x, b, w_post, gate, w_pre, scale, eps)
    a.x, a.ld_x = x.data_ptr(), _rows("x", x, x)
    N = x.shape[0]
    with _on(stream):
        r, n, rstd_post, rstd_pre = x, None, None, None
        if b is not None:
            if out_r is None:
                r = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            else:
                r = out_r
                if r.shape != x.shape or r.dtype != x.dtype or r.device != x.device or not r.is_contiguous():
                    raise ValueError("out_r must be a contiguous tensor like x")
            a.r = r.data_ptr()
            if w_post is not None:
                rstd_post = torch.empty(N, dtype=torch.float32, device=x.device)
                a.rstd_post = rstd_post.data_ptr()
        if w_pre is not None:
            n = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            rstd_pre = torch.empty(N, dtype=torch.float32, device=x.device)
            a.n, a.rstd_pre = n.data_ptr(), rstd_pre.data_ptr()
        a.stream = _stream(stream, x.device)
        _abi.check(_abi.lib().lce_block_norm_forward(ctypes.byref(a)), "lce_block_norm_forward")
    return r, n, rstd_post, rstd_pre


def block_norm_backward(dr, dn, r, b=None, *, w_post=None, gate=None, w_pre=None, scale: float = 1.0, rstd_post=None,
                        rstd_pre=None, workspace=None, stream=None):
    """(dx, db, dw_post, dgate, dw_pre) from the gradients dr of r (None: zero)
    and dn of n, the forward's r, b and rstd; None where the forward had no
    such input. `workspace`: a uint8 CUDA tensor of at least
    block_norm_workspace_size(N, d) bytes."""
    ref = r if r is not None else b
    a = _norm_args(ref, b, w_post, gate, w_pre, scale, 0.0)
    N, d = ref.shape
    if dr is not None:
        a.dr, a.ld_dr = dr.data_ptr(), _rows("dr", dr, ref)
    if w_pre is not None:
        if dn is None or r is None:
            raise ValueError("with w_pre the backward needs dn and r")
        a.dn, a.ld_dn = dn.data_ptr(), _rows("dn", dn, ref)
        a.r, a.ld_r = r.data_ptr(), _rows("r", r, ref)
    for name, w, t in (("rstd_post", w_post, rstd_post), ("rstd_pre", w_pre, rstd_pre)):
        if w is not None:
            if t is None or t.dtype != torch.float32 or t.shape != (N,) or t.device != ref.device or not t.is_contiguous():
                raise ValueError(f"{name} must be the forward's contiguous fp32 [N] tensor")
            setattr(a, name, t.data_ptr())
    with _on(stream):
        new = lambda like: torch.empty(like.shape, dtype=like.dtype, device=like.device)  # noqa: E731
        dx, db, dw_post, dgate, dw_pre = new(ref), None, None, None, None
        a.dx = dx.data_ptr()
        if b is not None:
            db = new(b)
            a.db = db.data_ptr()
        if w_post is not None:
            dw_post = new(w_post)
            a.dw_post = dw_post.data_ptr()
        if gate is not None:
            dgate = new(gate)
            a.dgate = dgate.data_ptr()
        if w_pre is not None:
            dw_pre = new(w_pre)
            a.dw_pre = dw_pre.data_ptr()
        lib = _abi.lib()
        a.workspace, a.workspace_bytes, keep = _scratch(workspace, lib.lce_block_norm_workspace_size(ctypes.byref(a)),
                                                        ref.device)
        a.stream = _stream(stream, ref.device)
        _abi.check(lib.lce_block_norm_backward(ctypes.byref(a)), "lce_block_norm_backward")
        del keep
    return dx, db, dw_post, dgate, dw_pre


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, b, w_post, gate, w_pre, scale, eps):
        r, n, rstd_post, rstd_pre = block_norm_forward(x, b, w_post=w_post, gate=gate, w_pre=w_pre, scale=scale, eps=eps)
        ctx.save_for_backward(r if w_pre is not None else None, b, w_post, gate, w_pre, rstd_post, rstd_pre)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return r, n

    @staticmethod
    def backward(ctx, dr, dn):
        r, b, w_post, gate, w_pre, rstd_post, rstd_pre = ctx.saved_tensors
        ref = r if r is not None else b
        if w_pre is not None and dn is None:
            dn = torch.zeros_like(ref)
        if dr is None and w_pre is None:
            dr = torch.zeros_like(ref)
        rows = lambda t: None if t is None else t.contiguous()  # noqa: E731
        dx, db, dw_post, dgate, dw_pre = block_norm_backward(
            rows(dr), rows(dn), r, b, w_post=w_post, gate=gate, w_pre=w_pre, scale=ctx.scale, rstd_post=rstd_post,
            rstd_pre=rstd_pre)
        need = ctx.needs_input_grad
        return tuple(g if n else None for g, n in zip((dx, db, dw_post, dgate, dw_pre), need)) + (None, None)


def block_norm(x, b=None, *, w_post=None, gate=None, w_pre=None, scale: float = 1.0, eps: float = 1e-6):
    """Autograd form of block_norm_forward: (r, n); n is None without w_pre,
    and without b the first output is x passed through."""
    if b is None:
        return _Norm.apply(x, w_pre, eps)
    return _BlockNorm.apply(x, b, w_post, gate, w_pre, scale, eps)


class _Norm(torch.autograd.Function):
    """The norm alone: (x, n), with the gradient that reaches x past the norm
    joined inside the kernel."""

    @staticmethod
    def forward(ctx, x, w_pre, eps):
        _, n, _, rstd = block_norm_forward(x, w_pre=w_pre, eps=eps)
        ctx.save_for_backward(x, w_pre, rstd)
        ctx.set_materialize_grads(False)
        return x.view_as(x), n

    @staticmethod
    def backward(ctx, dr, dn):
        x, w_pre, rstd = ctx.saved_tensors
        if dn is None:
            dn = torch.zeros_like(x)
        dx, _, _, _, dw = block_norm_backward(None if dr is None else dr.contiguous(), dn.contiguous(), x, w_pre=w_pre,
                                              rstd_pre=rstd)
        return dx if ctx.needs_input_grad[0] else None, dw if ctx.needs_input_grad[1] else None, None


# ------------------------------------------------------------------- clipping

def clip_workspace_size(count: int) -> int:
    """Bytes of scratch grad_norm and clip_grad_norm need for `count` tensors."""
    return int(_abi.lib().lce_clip_workspace_size(int(count)))


def _table(grads, out):
    n = len(grads)
    if n == 0:
        raise ValueError("no gradients given")
    device = grads[0].device
    dtypes = [_DT.get(t.dtype, -1) for t in grads]
    if device.type != "cuda" or any(t.device != device for t in grads):
        raise ValueError("gradients must be CUDA tensors on one device (there is no CPU path)")
    if -1 in dtypes:
        raise ValueError("gradients must be bfloat16 or float32")
    if not all(t.is_contiguous() for t in grads):
        raise ValueError("gradients must be contiguous")
    sizes = [t.numel() for t in grads]
    ptrs = [t.data_ptr() for t in grads]
    outs = None
    if out is not None:
        if len(out) != n or any(o.dtype != t.dtype or o.device != device or o.shape != t.shape for o, t in zip(out, grads)):
            raise ValueError("out must hold a tensor like each gradient")
        if not all(o.is_contiguous() for o in out):
            raise ValueError("out tensors must be contiguous")
        outs = (ctypes.c_void_p * n)(*[o.data_ptr() for o in out])
    return device, n, (ctypes.c_void_p * n)(*ptrs), outs, (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*dtypes)


def grad_norm(grads, *, workspace=None, stream=None):
    """The 2-norm of all tensors together (bf16 and fp32 may be mixed), a
    0-d fp32 CUDA tensor; the host does not wait for it."""
    grads = list(grads)
    device, n, ptrs, _, sizes, dtypes = _table(grads, None)
    with _on(stream):
        norm = torch.empty((), dtype=torch.float32, device=device)
        lib = _abi.lib()
        at, size, keep = _scratch(workspace, lib.lce_clip_workspace_size(n), device)
        _abi.check(lib.lce_grad_norm(n, ptrs, sizes, dtypes, norm.data_ptr(), at, size, _stream(stream, device)),
                   "lce_grad_norm")
        del keep
    return norm


def clip_grad_norm(grads, max_norm: float, *, out=None, eps: float = 1e-6, return_factor: bool = False, workspace=None,
                   stream=None):
    """Scale all tensors by min(1, max_norm / (norm + eps)), norm being their
    2-norm together, and return the norm from before (0-d fp32 CUDA tensor;
    with return_factor (norm, factor)). In place, or into the tensors `out`."""
    grads = list(grads)
    device, n, ptrs, outs, sizes, dtypes = _table(grads, out)
    with _on(stream):
        res = torch.empty(2, dtype=torch.float32, device=device)
        lib = _abi.lib()
        at, size, keep = _scratch(workspace, lib.lce_clip_workspace_size(n), device)
        base = res.data_ptr()
        _abi.check(lib.lce_clip_grads(n, ptrs, outs, sizes, dtypes, max_norm, eps, base, base + 4, at, size,
                                      _stream(stream, device)), "lce_clip_grads")
        del keep
    return (res[0], res[1]) if return_factor else res[0]
