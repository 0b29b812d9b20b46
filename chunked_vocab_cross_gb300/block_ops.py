"""The operators between the embedding lookup and the head loss, with the C
ABI's names: attention over packed sequences, the norms around a block fused
with its gate and residual scale, and gradient clipping over many tensors.
PyTorch provides device memory and the current stream; the arithmetic is all
in liblce.so.

With `stream` given, the call's outputs and scratch are allocated for that
stream; as for the library's other calls, inputs made on another stream have
to be ready there (and stay alive until that stream is done with them)."""
from __future__ import annotations

import array
import functools
import operator

import torch
from torch.autograd.function import once_differentiable

from . import _abi

_DT = {torch.bfloat16: _abi.LCE_BF16, torch.float32: _abi.LCE_FP32}
_ATTN, _NORM = _abi.packer(_abi.LceAttn), _abi.packer(_abi.LceNorm)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)   # CUDA is up: the tensors are there


def _on_stream(call):
    """With `stream` given, the call runs with that stream as the current one:
    its allocations belong to it and its launches go there."""
    @functools.wraps(call)
    def wrapped(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return wrapped


def _stream(index: int) -> int:
    """The current stream of device `index`, which the tensors are on. The library
    runs on the current device, whatever the stream."""
    if index != _current_device():
        raise ValueError(f"the tensors are on cuda:{index}, which is not the current device")
    return _current_stream(index) if _current_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _scratch(given, need: int, device):
    """A call's scratch: (address, bytes, tensor to keep until it is enqueued)."""
    if given is None:
        given = torch.empty(need, dtype=torch.uint8, device=device)
        return given.data_ptr(), need, given
    if given.device != device or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
    return given.data_ptr(), given.numel() * given.element_size(), given


# Autograd learns of tensors that a caller gives to be written: one that it keeps for a backward pass is then an error
# there. (0.2 us for one tensor, 0.9 for 28; clipping 28 gradients that were just made takes 3 us longer, 38 instead of 35.)
_written = torch.autograd.graph.increment_version


def _like(t):
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _whole(t):
    """A gradient from autograd as the kernels can read it: it may be expanded,
    permuted, or contiguous at an address off 16 bytes (a slice of another)."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


# ------------------------------------------------------------------ attention

def _tokens(name, t, device, dtype, shape=None):
    """(address, token stride, head stride) of a [T, heads, D] tensor, or of a
    [B, L, heads, D] one as [B*L, heads, D]. A dimension of one entry has no
    stride of its own."""
    sh = t.shape
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor with q's device and dtype (there is no CPU path)")
    if shape is not None and sh != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(sh)}")
    st = t.stride()
    H, D = sh[-2], sh[-1]
    if st[-1] != 1 and D > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    hs = st[-2] if H > 1 else D
    if len(sh) == 4:
        B, L = sh[0], sh[1]
        if B > 1 and L > 1 and st[0] != L * st[1]:
            raise ValueError(f"{name}: the rows of a [B, L, heads, D] tensor must be evenly spaced over B and L")
        ts = st[1] if L > 1 else st[0] if B > 1 else H * D
    else:
        ts = st[0] if sh[0] > 1 else H * D
    return t.data_ptr(), ts, hs


def _sequences(q, k, v, cu_q, cu_k):
    """(B, Tq, Tk, Hq, Hk, D, address of cu_q, address of cu_k)."""
    sq, sk = q.shape, k.shape
    if q.dtype not in _DT or not q.is_cuda:
        raise ValueError("q must be a bfloat16 or float32 CUDA tensor (there is no CPU path)")
    n = len(sq)
    if n not in (3, 4) or len(sk) != n or v.shape != sk:
        raise ValueError("q must be [Tq, heads, D] and k, v [Tk, kv_heads, D] (or all [B, L, heads, D])")
    if sk[-1] != sq[-1] or (n == 4 and sk[0] != sq[0]):
        raise ValueError("shape mismatch between q, k and v")
    Hq, Hk = sq[-2], sk[-2]
    if Hq < 1 or Hk < 1 or Hq % Hk:
        raise ValueError("the number of query heads must be a multiple of the number of key heads")
    if cu_q is None and cu_k is None:
        if n == 4:
            return max(sq[0], 1), sq[0] * sq[1], sk[0] * sk[1], Hq, Hk, sq[3], 0, 0
        return 1, sq[0], sk[0], Hq, Hk, sq[2], 0, 0
    if n == 4:
        raise ValueError("sequence offsets go with [T, heads, D] tensors")
    cu_q = cu_k if cu_q is None else cu_q
    cu_k = cu_q if cu_k is None else cu_k
    for name, c in (("cu_seqlens_q", cu_q), ("cu_seqlens_k", cu_k)) if cu_q is not cu_k else (("cu_seqlens", cu_q),):
        if c.dtype != torch.int32 or c.dim() != 1 or c.device != q.device or not c.is_contiguous() or c.numel() < 2:
            raise ValueError(f"{name} must be a contiguous int32 tensor of at least two offsets on q's device")
    if cu_q.numel() != cu_k.numel():
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    return cu_q.numel() - 1, sq[0], sk[0], Hq, Hk, sq[2], cu_q.data_ptr(), cu_k.data_ptr()


@functools.lru_cache(maxsize=256)
def attention_workspace_size(Tq: int, Tk: int, Hq: int, Hk: int, D: int, batch: int = 1, dtype=torch.bfloat16) -> int:
    """Bytes of scratch attention_backward needs (`batch`: the number of sequences)."""
    a = _abi.LceAttn()
    # equal lengths are not asked for here: a stand-in for the offsets
    a.cu_q = a.cu_k = 16
    a.dtype, a.B, a.Tq, a.Tk, a.Hq, a.Hk, a.D = _DT[dtype], batch, Tq, Tk, Hq, Hk, D
    return int(_abi.lib().lce_attention_workspace_size(_abi.ctypes.byref(a)))


@functools.lru_cache(maxsize=256)
def attention_forward_workspace_size(Tq: int, Tk: int, Hq: int, Hk: int, D: int, batch: int = 1, dtype=torch.bfloat16,
                                     causal: bool = True) -> int:
    """Bytes of scratch attention_forward needs: 0 but for few rows over long keys."""
    a = _abi.LceAttn()
    a.cu_q = a.cu_k = 16
    a.dtype, a.B, a.Tq, a.Tk, a.Hq, a.Hk, a.D, a.causal = _DT[dtype], batch, Tq, Tk, Hq, Hk, D, 1 if causal else 0
    return int(_abi.lib().lce_attention_forward_workspace_size(_abi.ctypes.byref(a)))


@_on_stream
def attention_forward(q, k, v, cu_seqlens_q=None, cu_seqlens_k=None, *, causal: bool = True, scale=None, out=None,
                      workspace=None):
    """(o, lse) of softmax attention over packed sequences: q [Tq, heads, D],
    k and v [Tk, kv_heads, D] with int32 token offsets of the sequences (one
    sequence without them), or [B, L, heads, D] tensors of equal lengths. o has
    q's shape and dtype, lse is fp32 [heads, tokens]; rows that see no key get
    o = 0 and lse = -inf. `scale` is D**-0.5 if not given; `out` receives o;
    `workspace`: a uint8 CUDA tensor of at least
    attention_forward_workspace_size bytes; `stream`: the stream to run on (the
    current one if not given)."""
    B, Tq, Tk, Hq, Hk, D, pcq, pck = _sequences(q, k, v, cu_seqlens_q, cu_seqlens_k)
    device, dtype = q.device, q.dtype
    pq, pk, pv = _tokens("q", q, device, dtype), _tokens("k", k, device, dtype), _tokens("v", v, device, dtype)
    given = out is not None
    if given:
        po, ots, ohs = _tokens("out", out, device, dtype, q.shape)
    else:
        out = torch.empty(q.shape, dtype=dtype, device=device)
        po, ots, ohs = out.data_ptr(), Hq * D, D
    lse = torch.empty((Hq, Tq), dtype=torch.float32, device=device)
    ws, size, keep = 0, 0, None
    need = attention_forward_workspace_size(Tq, Tk, Hq, Hk, D, B, dtype, causal)
    if need:
        ws, size, keep = _scratch(workspace, need, device)
    args = _ATTN.pack(_DT[dtype], 1 if causal else 0, D ** -0.5 if scale is None else scale, B, Tq, Tk, Hq, Hk, D,
                      pcq, pck, pq[0], pk[0], pv[0], pq[1], pq[2], pk[1], pk[2], pv[1], pv[2], po, ots, ohs,
                      lse.data_ptr(), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, ws, size, _stream(device.index))
    _abi.check(_abi.lib().lce_attention_forward(args), "lce_attention_forward")
    del keep
    if given:
        _written(out)
    return out, lse


@_on_stream
def attention_backward(do, q, k, v, o, lse, cu_seqlens_q=None, cu_seqlens_k=None, *, causal: bool = True, scale=None,
                       dq=None, dk=None, dv=None, workspace=None):
    """(dq, dk, dv) from the forward's inputs, its o and lse, and the gradient
    `do` of o; the probabilities are recomputed. dq, dk and dv may be given
    (strided slices of one gradient, say). `workspace`: a uint8 CUDA tensor of
    at least attention_workspace_size bytes; `stream`: the stream to run on."""
    B, Tq, Tk, Hq, Hk, D, pcq, pck = _sequences(q, k, v, cu_seqlens_q, cu_seqlens_k)
    device, dtype = q.device, q.dtype
    pq, pk, pv = _tokens("q", q, device, dtype), _tokens("k", k, device, dtype), _tokens("v", v, device, dtype)
    pg, po = _tokens("do", do, device, dtype, q.shape), _tokens("o", o, device, dtype, q.shape)
    if lse.dtype != torch.float32 or lse.shape != (Hq, Tq) or not lse.is_contiguous() or lse.device != device:
        raise ValueError("lse must be the forward's contiguous fp32 [heads, tokens] tensor")
    given = [t for t in (dq, dk, dv) if t is not None]
    if dq is None:
        dq = torch.empty(q.shape, dtype=dtype, device=device)
        px = dq.data_ptr(), Hq * D, D
    else:
        px = _tokens("dq", dq, device, dtype, q.shape)
    if dk is None:
        dk = torch.empty(k.shape, dtype=dtype, device=device)
        py = dk.data_ptr(), Hk * D, D
    else:
        py = _tokens("dk", dk, device, dtype, k.shape)
    if dv is None:
        dv = torch.empty(k.shape, dtype=dtype, device=device)
        pz = dv.data_ptr(), Hk * D, D
    else:
        pz = _tokens("dv", dv, device, dtype, k.shape)
    ws, size, keep = _scratch(workspace, attention_workspace_size(Tq, Tk, Hq, Hk, D, B, dtype), device)
    args = _ATTN.pack(_DT[dtype], 1 if causal else 0, D ** -0.5 if scale is None else scale, B, Tq, Tk, Hq, Hk, D,
                      pcq, pck, pq[0], pk[0], pv[0], pq[1], pq[2], pk[1], pk[2], pv[1], pv[2], po[0], po[1], po[2],
                      lse.data_ptr(), pg[0], pg[1], pg[2], px[0], py[0], pz[0], px[1], px[2], py[1], py[2], pz[1],
                      pz[2], ws, size, _stream(device.index))
    _abi.check(_abi.lib().lce_attention_backward(args), "lce_attention_backward")
    del keep
    if given:
        _written(given)
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k, causal, scale):
        o, lse = attention_forward(q, k, v, cu_q, cu_k, causal=causal, scale=scale)
        ctx.save_for_backward(q, k, v, o, lse, cu_q, cu_k)
        ctx.causal, ctx.scale = causal, scale
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, cu_q, cu_k = ctx.saved_tensors
        dq, dk, dv = attention_backward(_whole(do), q, k, v, o, lse, cu_q, cu_k, causal=ctx.causal, scale=ctx.scale)
        need = ctx.needs_input_grad
        return dq if need[0] else None, dk if need[1] else None, dv if need[2] else None, None, None, None, None


def attention(q, k, v, cu_seqlens_q=None, cu_seqlens_k=None, *, causal: bool = True, scale=None):
    """Autograd form of attention_forward (returns o)."""
    return _Attention.apply(q, k, v, cu_seqlens_q, cu_seqlens_k, causal, scale)


# ---------------------------------------------------------------- block norms

_ONLY_W_PRE = "without b there is only the norm by w_pre"


class _Expanded(Exception):
    """All rows of a tensor are one row of memory. The library has no such
    stride: 0 stands for d there."""


def _spread(t):
    return t.contiguous() if t is not None and t.dim() == 2 and t.stride(0) == 0 else t


def _rows(name, t, ref):
    """(address, row stride) of a [N, d] tensor whose rows are contiguous. The
    address of a tensor without rows is not read; it must not be NULL, which
    would mean no tensor."""
    sh = t.shape
    if sh != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
        raise ValueError(f"{name} must be a {tuple(ref.shape)} tensor of the same dtype and device")
    st = t.stride()
    if st[1] != 1 and sh[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if sh[0] < 2:
        return t.data_ptr() or 16, sh[1]
    if st[0] == 0:
        raise _Expanded
    return t.data_ptr(), st[0]


def _vector(name, t, ref):
    if t.shape != ref.shape[1:] or t.dtype != ref.dtype or t.device != ref.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [d] tensor of the stream's dtype")
    return t.data_ptr()


def _norm_inputs(ref, b, w_post, gate, w_pre):
    """(dtype, N, d, (b, ld), w_post, (gate, ld), w_pre, gate_full)."""
    dtype = _DT.get(ref.dtype)
    if dtype is None or not ref.is_cuda or ref.dim() != 2:
        raise ValueError("the stream must be a bfloat16 or float32 CUDA tensor [N, d] (there is no CPU path)")
    if b is None and (w_post is not None or gate is not None or w_pre is None):
        raise ValueError(_ONLY_W_PRE)
    pg, full = (0, 0), 0
    if gate is not None:
        full = 1 if gate.dim() == 2 else 0
        pg = _rows("gate", gate, ref) if full else (_vector("gate", gate, ref), 0)
    N, d = ref.shape
    return (dtype, N, d, (0, 0) if b is None else _rows("b", b, ref), 0 if w_post is None else _vector("w_post", w_post, ref),
            pg, 0 if w_pre is None else _vector("w_pre", w_pre, ref), full)


@functools.lru_cache(maxsize=256)
def block_norm_workspace_size(N: int, d: int) -> int:
    """Bytes of scratch block_norm_backward needs."""
    a = _abi.LceNorm()
    a.N, a.d = N, d
    return int(_abi.lib().lce_block_norm_workspace_size(_abi.ctypes.byref(a)))


@_on_stream
def block_norm_forward(x, b=None, *, w_post=None, gate=None, w_pre=None, scale: float = 1.0, eps: float = 1e-6,
                       out_r=None):
    """(r, n, rstd_post, rstd_pre) for the residual stream x [N, d] and a
    block's output b [N, d]:
        r = x + scale * gate * rms_norm(b) * w_post,   n = rms_norm(r) * w_pre
    with gate [d] or [N, d]; any of w_post, gate and w_pre may be None (n and
    the matching rstd are None then). Without b, r is x itself. `out_r`
    receives r and may be x (the stream updated in place); `stream`: the stream
    to run on (the current one if not given). Expanded rows are copied first."""
    try:
        dtype, N, d, pb, p_post, pg, p_pre, full = _norm_inputs(x, b, w_post, gate, w_pre)
        px = _rows("x", x, x)
    except _Expanded:
        r, *rest = block_norm_forward(_spread(x), _spread(b), w_post=w_post, gate=_spread(gate), w_pre=w_pre, scale=scale,
                                      eps=eps, out_r=out_r)
        return x if b is None else r, *rest
    device = x.device
    r, n, rstd_post, rstd_pre = x, None, None, None
    pr = pn = ps_post = ps_pre = 0
    if b is not None:
        if out_r is None:
            r = _like(x)
        else:
            r = out_r
            if r.shape != x.shape or r.dtype != x.dtype or r.device != device or not r.is_contiguous():
                raise ValueError("out_r must be a contiguous tensor like x")
        pr = r.data_ptr()
    if p_post:
        rstd_post = torch.empty(N, dtype=torch.float32, device=device)
        ps_post = rstd_post.data_ptr()
    if p_pre:
        n = _like(x)
        rstd_pre = torch.empty(N, dtype=torch.float32, device=device)
        pn, ps_pre = n.data_ptr(), rstd_pre.data_ptr()
    args = _NORM.pack(dtype, N, d, scale, eps, px[0], pb[0], p_post, pg[0], p_pre, full, px[1], pb[1], pg[1], pr, pn,
                      ps_post, ps_pre, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, _stream(device.index))
    _abi.check(_abi.lib().lce_block_norm_forward(args), "lce_block_norm_forward")
    if b is not None and out_r is not None:
        _written(out_r)
    return r, n, rstd_post, rstd_pre


@_on_stream
def block_norm_backward(dr, dn, r, b=None, *, w_post=None, gate=None, w_pre=None, scale: float = 1.0, rstd_post=None,
                        rstd_pre=None, workspace=None):
    """(dx, db, dw_post, dgate, dw_pre) from the gradients dr of r (None: zero)
    and dn of n, the forward's r, b and rstd; None where the forward had no
    such input. `workspace`: a uint8 CUDA tensor of at least
    block_norm_workspace_size(N, d) bytes; `stream`: the stream to run on."""
    ref = r if r is not None else b
    try:
        dtype, N, d, pb, p_post, pg, p_pre, full = _norm_inputs(ref, b, w_post, gate, w_pre)
        pdr = (0, 0) if dr is None else _rows("dr", dr, ref)
        pdn = pr = (0, 0)
        if w_pre is not None:
            if dn is None or r is None:
                raise ValueError("with w_pre the backward needs dn and r")
            pdn, pr = _rows("dn", dn, ref), _rows("r", r, ref)
    except _Expanded:
        return block_norm_backward(_spread(dr), _spread(dn), _spread(r), _spread(b), w_post=w_post, gate=_spread(gate),
                                   w_pre=w_pre, scale=scale, rstd_post=rstd_post, rstd_pre=rstd_pre, workspace=workspace)
    device = ref.device
    stats = [0, 0]
    for i, (name, w, t) in enumerate((("rstd_post", w_post, rstd_post), ("rstd_pre", w_pre, rstd_pre))):
        if w is not None:
            if t is None or t.dtype != torch.float32 or t.shape != (N,) or t.device != device or not t.is_contiguous():
                raise ValueError(f"{name} must be the forward's contiguous fp32 [N] tensor")
            stats[i] = t.data_ptr()
    dx = _like(ref)
    db = None if b is None else _like(b)
    dw_post = None if w_post is None else torch.empty_like(w_post)
    dgate = None if gate is None else _like(gate)
    dw_pre = None if w_pre is None else torch.empty_like(w_pre)
    at = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    ws, size, keep = _scratch(workspace, block_norm_workspace_size(N, d), device)
    args = _NORM.pack(dtype, N, d, scale, 0.0, 0, pb[0], p_post, pg[0], p_pre, full, 0, pb[1], pg[1], pr[0], 0,
                      stats[0], stats[1], pdr[0], pdn[0], pr[1], pdr[1], pdn[1], at(dx), at(db), at(dw_post),
                      at(dgate), at(dw_pre), ws, size, _stream(device.index))
    _abi.check(_abi.lib().lce_block_norm_backward(args), "lce_block_norm_backward")
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
    @once_differentiable
    def backward(ctx, dr, dn):
        r, b, w_post, gate, w_pre, rstd_post, rstd_pre = ctx.saved_tensors
        ref = r if r is not None else b
        if w_pre is not None and dn is None:
            dn = torch.zeros_like(ref)
        if dr is None and w_pre is None:
            dr = torch.zeros_like(ref)
        dx, db, dw_post, dgate, dw_pre = block_norm_backward(
            _whole(dr), _whole(dn), r, b, w_post=w_post, gate=gate, w_pre=w_pre, scale=ctx.scale, rstd_post=rstd_post,
            rstd_pre=rstd_pre)
        need = ctx.needs_input_grad
        return tuple(g if n else None for g, n in zip((dx, db, dw_post, dgate, dw_pre), need)) + (None, None)


def block_norm(x, b=None, *, w_post=None, gate=None, w_pre=None, scale: float = 1.0, eps: float = 1e-6):
    """Autograd form of block_norm_forward: (r, n); n is None without w_pre,
    and without b the first output is x passed through."""
    if b is None:
        if w_post is not None or gate is not None or w_pre is None:
            raise ValueError(_ONLY_W_PRE)
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
    @once_differentiable
    def backward(ctx, dr, dn):
        x, w_pre, rstd = ctx.saved_tensors
        if dn is None:
            dn = torch.zeros_like(x)
        dx, _, _, _, dw = block_norm_backward(_whole(dr), _whole(dn), x, w_pre=w_pre, rstd_pre=rstd)
        return dx if ctx.needs_input_grad[0] else None, dw if ctx.needs_input_grad[1] else None, None


# ------------------------------------------------------------------- clipping

@functools.lru_cache(maxsize=256)
def clip_workspace_size(count: int) -> int:
    """Bytes of scratch grad_norm and clip_grad_norm need for `count` tensors."""
    return int(_abi.lib().lce_clip_workspace_size(int(count)))


_ptr, _numel, _index, _dense = (torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.get_device,
                                torch.Tensor.is_contiguous)
_dtype = operator.attrgetter("dtype")


def _table(grads, out):
    """Host arrays of the tensors' addresses, sizes and types: one pass of C
    calls for each, since there may be hundreds of tensors."""
    if not grads:
        raise ValueError("no gradients given")
    index = grads[0].get_device()
    if index < 0 or set(map(_index, grads)) != {index}:
        raise ValueError("gradients must be CUDA tensors on one device (there is no CPU path)")
    kinds = list(map(_dtype, grads))
    try:
        dtypes = array.array("i", map(_DT.__getitem__, kinds))
    except KeyError:
        raise ValueError("gradients must be bfloat16 or float32") from None
    if not all(map(_dense, grads)):
        raise ValueError("gradients must be contiguous")
    sizes = array.array("q", map(_numel, grads))
    outs = None
    if out is not None:
        if (len(out) != len(grads) or set(map(_index, out)) != {index} or list(map(_dtype, out)) != kinds
                or array.array("q", map(_numel, out)) != sizes):
            raise ValueError("out must hold a tensor like each gradient")
        if not all(map(_dense, out)):
            raise ValueError("out tensors must be contiguous")
        outs = array.array("Q", map(_ptr, out))
    return index, array.array("Q", map(_ptr, grads)), outs, sizes, dtypes


def _buffer(a):
    return None if a is None else a.buffer_info()[0]


def _clip_scratch(workspace, n, sizes, device):
    # up to 1 MB, each tensor rounded up to 4 KB, the library needs no scratch (beyond, it would allocate it itself)
    if workspace is None and 4 * sum(sizes) + 4096 * n <= 256 * 4096 and n <= 240:
        return None, 0, None
    return _scratch(workspace, clip_workspace_size(n), device)


@_on_stream
def grad_norm(grads, *, workspace=None):
    """The 2-norm of all tensors together (bf16 and fp32 may be mixed), a
    0-d fp32 CUDA tensor; the host does not wait for it. `stream`: the stream
    to run on (the current one if not given)."""
    grads = list(grads)
    index, ptrs, _, sizes, dtypes = _table(grads, None)
    n, device = len(grads), grads[0].device
    norm = torch.empty((), dtype=torch.float32, device=device)
    at, size, keep = _clip_scratch(workspace, n, sizes, device)
    _abi.check(_abi.lib().lce_grad_norm(n, _buffer(ptrs), _buffer(sizes), _buffer(dtypes), norm.data_ptr(), at, size,
                                        _stream(index)), "lce_grad_norm")
    del keep
    return norm


@_on_stream
def clip_grad_norm(grads, max_norm: float, *, out=None, eps: float = 1e-6, return_factor: bool = False, workspace=None):
    """Scale all tensors by min(1, max_norm / (norm + eps)), norm being their
    2-norm together, and return the norm from before (0-d fp32 CUDA tensor;
    with return_factor (norm, factor)). In place, or into the tensors `out`
    (each of its gradient's dtype and number of elements). `stream`: the stream
    to run on."""
    grads = list(grads)
    out = out if out is None else list(out)
    index, ptrs, outs, sizes, dtypes = _table(grads, out)
    n, device = len(grads), grads[0].device
    norm = torch.empty((), dtype=torch.float32, device=device)
    factor = torch.empty((), dtype=torch.float32, device=device) if return_factor else None
    at, size, keep = _clip_scratch(workspace, n, sizes, device)
    _abi.check(_abi.lib().lce_clip_grads(n, _buffer(ptrs), _buffer(outs), _buffer(sizes), _buffer(dtypes), max_norm, eps,
                                         norm.data_ptr(), factor.data_ptr() if return_factor else None, at, size,
                                         _stream(index)), "lce_clip_grads")
    del keep
    _written(grads if out is None else out)
    return (norm, factor) if return_factor else norm
