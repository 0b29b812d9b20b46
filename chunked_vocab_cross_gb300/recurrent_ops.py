"""The operators of a recurrent block that keeps its activations in 8 bits, with
the C ABI's names: the layer norm with the residual sum before it, activations
packed to 8 bits and the weight gradient taken from them, and the gated
recurrence over packed sequences. Memory, streams and checks are as in
block_ops; the arithmetic is in liblce.so, but for linear_keep8's two plain
matrix products."""
from __future__ import annotations

import functools

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from .block_ops import _DT, _Expanded, _like, _on_stream, _rows, _scratch, _spread, _stream, _vector, _whole, _written

_LN, _WGRAD, _SCAN = _abi.packer(_abi.LceLayerNorm), _abi.packer(_abi.LceWgrad), _abi.packer(_abi.LceRecurrence)
_at = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731


# ------------------------------------------------------- activations in 8 bits

class PackedActivation:
    """Rows of channels in 8 bits: `codes`, uint8 [N, d], the bytes of e4m3
    values, and `exps`, int8 [ceil(d / 128), N], an exponent for every 128
    channels of a row; a code stands for its value times 2**exponent (-128: the
    block held an infinity or NaN and stands for NaNs). Both have rows on
    16-byte strides, and are copied to such where they have not (brought back
    from host memory, say). Their bytes have to be those that pack_activation
    leaves, which is not checked: exponents of -128 or -100 to 119, and the codes
    of NaN (0x7f, 0xff) only under -128. `dtype`: of the tensor that was
    packed."""
    __slots__ = ("shape", "dtype", "device", "_codes", "_exps", "_fields")

    def __init__(self, codes, exps, dtype):
        if codes.dtype != torch.uint8 or exps.dtype != torch.int8 or codes.dim() != 2 or exps.dim() != 2 or dtype not in _DT:
            raise ValueError("codes must be uint8 [N, d], exps int8 [ceil(d / 128), N] and dtype bfloat16 or float32")
        if exps.shape != ((codes.shape[1] + 127) // 128, codes.shape[0]) or exps.device != codes.device or not codes.is_cuda:
            raise ValueError("exps must be [ceil(d / 128), N] for codes [N, d], both on one CUDA device (there is no CPU path)")
        if (codes.stride(1) != 1 and codes.shape[1] > 1) or (exps.stride(1) != 1 and exps.shape[1] > 1):
            raise ValueError("the rows of codes and exps must be contiguous")
        codes, exps = _on_16(codes), _on_16(exps)
        self.shape, self.dtype, self.device, self._codes, self._exps = codes.shape, dtype, codes.device, codes, exps
        (n, d), blocks = codes.shape, exps.shape[0]
        # addresses and row strides; a single row has no stride of its own
        self._fields = (codes.data_ptr(), exps.data_ptr(), codes.stride(0) if n > 1 else _up16(d),
                        exps.stride(0) if blocks > 1 else _up16(n))

    @property
    def codes(self):
        return self._codes[:, :self.shape[1]]

    @property
    def exps(self):
        return self._exps[:, :self.shape[0]]


def _up16(n: int) -> int:
    return (n + 15) // 16 * 16


def _on_16(t):
    """t [rows, n] of bytes with its rows on 16-byte strides that do not overlap
    and, since the kernels read whole 16 bytes, the last of them inside its
    memory."""
    rows, n = t.shape
    if rows == 0:
        return t
    last = (rows - 1) * t.stride(0)
    if (t.data_ptr() % 16 == 0 and (rows < 2 or (t.stride(0) % 16 == 0 and t.stride(0) >= n))
            and t.storage_offset() + last + _up16(n) <= t.untyped_storage().nbytes()):
        return t
    room = torch.empty((rows, _up16(n)), dtype=t.dtype, device=t.device)[:, :n]
    return room.copy_(t)


def _packed_like(x) -> PackedActivation:
    """Room for the rows of x [N, d]."""
    n, d = x.shape
    ld, le, device = _up16(d), _up16(n), x.device
    p = PackedActivation.__new__(PackedActivation)
    p.shape, p.dtype, p.device = x.shape, x.dtype, device
    p._codes = codes = torch.empty((n, ld), dtype=torch.uint8, device=device)
    p._exps = exps = torch.empty(((d + 127) // 128, le), dtype=torch.int8, device=device)
    p._fields = codes.data_ptr(), exps.data_ptr(), ld, le
    return p


def _matrix(name, t):
    """(address, row stride) of a [N, d] tensor whose rows are contiguous."""
    if t.dtype not in _DT or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a bfloat16 or float32 CUDA tensor [N, d] (there is no CPU path)")
    return _rows(name, t, t)


@_on_stream
def pack_activation(x) -> PackedActivation:
    """x [N, d] in 8 bits (about half of bf16's memory), for what a backward pass
    needs of it: e4m3 codes with one power of two for every 128 channels of a
    row. A value comes back within 2**-4 of itself, or 2**-10 of its block's
    scale where that is more. `stream`: the stream to run on."""
    try:
        px, ld = _matrix("x", x)
    except _Expanded:
        return pack_activation(_spread(x))
    n, d = x.shape
    p = _packed_like(x)
    codes, exps, ldc, lde = p._fields
    _abi.check(_abi.lib().lce_pack8(_DT[x.dtype], px, ld, n, d, codes, ldc, exps, lde, _stream(x.device.index)), "lce_pack8")
    return p


@_on_stream
def unpack_activation(p: PackedActivation, *, dtype=None, out=None):
    """What a packed activation stands for, [N, d], in the dtype that was packed
    or `dtype` (exact in either), or in `out`, whose dtype then counts.
    `stream`: the stream to run on."""
    n, d = p.shape
    given = out is not None
    if given:
        if out.shape != p.shape or out.device != p.device or (dtype is not None and out.dtype != dtype):
            raise ValueError(f"out must be a {tuple(p.shape)} tensor on the packed activation's device, of dtype if that is given")
        if n > 1 and out.stride(0) < d:
            raise ValueError("the rows of out must not overlap")
    else:
        dtype = p.dtype if dtype is None else dtype
        if dtype not in _DT:
            raise ValueError("dtype must be bfloat16 or float32")
        out = torch.empty((n, d), dtype=dtype, device=p.device)
    po, ld = _matrix("out", out)
    codes, exps, ldc, lde = p._fields
    _abi.check(_abi.lib().lce_unpack8(_DT[out.dtype], codes, ldc, exps, lde, n, d, po, ld, _stream(p.device.index)),
               "lce_unpack8")
    if given:
        _written(out)
    return out


@functools.lru_cache(maxsize=256)
def packed_weight_grad_workspace_size(T: int, n: int, k: int, dtype=torch.bfloat16, out_dtype=None) -> int:
    """Bytes of scratch packed_weight_grad needs for a dy [T, n] of `dtype` and k
    packed channels."""
    a = _abi.LceWgrad()
    a.dtype, a.dw_dtype, a.T, a.n, a.k = _DT[dtype], _DT[dtype if out_dtype is None else out_dtype], T, n, k
    return int(_abi.lib().lce_packed_wgrad_workspace_size(_abi.ctypes.byref(a)))


@_on_stream
def packed_weight_grad(dy, x: PackedActivation, *, out=None, out_dtype=None, workspace=None):
    """dw [n, k] = dy^T x: a linear layer's weight gradient from the gradient dy
    [T, n] of its output and its packed input x [T, k]. In dy's dtype, or fp32
    with out_dtype=torch.float32; `out` receives it. `workspace`: a uint8 CUDA
    tensor of at least packed_weight_grad_workspace_size bytes; `stream`: the
    stream to run on."""
    try:
        py, ld = _matrix("dy", dy)
    except _Expanded:
        return packed_weight_grad(_spread(dy), x, out=out, out_dtype=out_dtype, workspace=workspace)
    T, n = dy.shape
    if x.shape[0] != T or x.device != dy.device:
        raise ValueError("dy and x must have the same number of rows and one device")
    k = x.shape[1]
    given = out is not None
    if given:
        if out.shape != (n, k) or out.device != dy.device or not out.is_contiguous() or out_dtype not in (None, out.dtype):
            raise ValueError(f"out must be a contiguous ({n}, {k}) tensor on dy's device, of out_dtype if that is given")
        out_dtype = out.dtype
    else:
        out_dtype = dy.dtype if out_dtype is None else out_dtype
    if out_dtype not in (dy.dtype, torch.float32):
        raise ValueError("the gradient is of dy's dtype or float32")
    if not given:
        out = torch.empty((n, k), dtype=out_dtype, device=dy.device)
    ws, size, keep = 0, 0, None
    need = packed_weight_grad_workspace_size(T, n, k, dy.dtype, out_dtype)
    if need:
        ws, size, keep = _scratch(workspace, need, dy.device)
    codes, exps, ldc, lde = x._fields
    args = _WGRAD.pack(_DT[dy.dtype], _DT[out_dtype], T, n, k, py, ld, codes, exps, ldc, lde, out.data_ptr(), ws, size,
                       _stream(dy.device.index))
    _abi.check(_abi.lib().lce_packed_wgrad(args), "lce_packed_wgrad")
    del keep
    if given:
        _written(out)
    return out


def _recorded(*tensors) -> bool:
    """Whether a backward pass can follow a call on these. (ctx.needs_input_grad
    tells of the inputs alone: parameters have it where no gradient is recorded
    as well.)"""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _readable(t):
    """t [..., d] as [N, d] rows that the kernels can read: itself, or a copy where
    its elements, its address or its rows' distance are not theirs."""
    t = t.reshape(-1, t.shape[-1])
    if (t.stride(1) == 1 and t.data_ptr() % 16 == 0
            and (t.shape[0] < 2 or (t.stride(0) >= t.shape[1] and t.stride(0) * t.element_size() % 16 == 0))):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _LinearKeep8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        if ctx.needs_input_grad[1]:
            p = pack_activation(_readable(x))
            ctx.save_for_backward(w, p.codes, p.exps)
        else:
            ctx.save_for_backward(w, None, None)
        ctx.dtype = x.dtype
        return torch.nn.functional.linear(x, w)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w, codes, exps = ctx.saved_tensors
        dx = dy @ w if ctx.needs_input_grad[0] else None
        dw = None
        if ctx.needs_input_grad[1]:
            dw = packed_weight_grad(_readable(dy), PackedActivation(codes, exps, ctx.dtype))
        return dx, dw


def linear_keep8(x, w):
    """x w^T for x [..., k] and w [n, k], differentiable (once); of x only its
    8-bit form is kept for w's gradient, for which n and k must be multiples of
    8. Under autocast both are cast to its dtype first, as for PyTorch's own
    linear. The two other products are PyTorch's."""
    if torch.is_autocast_enabled("cuda"):
        dtype = torch.get_autocast_dtype("cuda")
        cast = lambda t: t.to(dtype) if t.dtype in (torch.float32, torch.bfloat16, torch.float16) else t  # noqa: E731
        with torch.autocast("cuda", enabled=False):
            return linear_keep8(cast(x), cast(w))
    if x.dtype not in _DT or not x.is_cuda or x.dtype != w.dtype or w.dim() != 2 or x.shape[-1] != w.shape[1] or x.device != w.device:
        raise ValueError("x [..., k] and w [n, k] must be bfloat16 or float32 tensors of one dtype on one CUDA device")
    if not _recorded(x, w):
        return torch.nn.functional.linear(x, w)
    if w.requires_grad and (w.shape[0] % 8 or w.shape[1] % 8 or not w.numel()):
        raise ValueError(f"w's gradient needs n and k that are multiples of 8, got {tuple(w.shape)}")
    return _LinearKeep8.apply(x, w)


# ------------------------------------------------------------------ layer norm

@functools.lru_cache(maxsize=256)
def layer_norm_workspace_size(N: int, d: int) -> int:
    """Bytes of scratch layer_norm_backward needs."""
    a = _abi.LceLayerNorm()
    a.N, a.d = N, d
    return int(_abi.lib().lce_layer_norm_workspace_size(_abi.ctypes.byref(a)))


@_on_stream
def layer_norm_forward(x, b=None, *, weight, bias=None, eps: float = 1e-5, keep8: bool = False, out_r=None):
    """(r, n, mean, rstd, kept) for the residual stream x [N, d] and a block's
    output b [N, d] (r is x itself without it):
        r = x + b,   n = (r - mean(r)) / sqrt(var(r) + eps) * weight + bias
    with weight and bias [d] (bias may be None), the statistics over d. `kept`
    is r as a PackedActivation with keep8, packed in the same pass, else None;
    layer_norm_backward takes it in r's place. `out_r` receives r and may be x
    or b; `stream`: the stream to run on. Expanded rows are copied first."""
    if x.dtype not in _DT or not x.is_cuda or x.dim() != 2:
        raise ValueError("the stream must be a bfloat16 or float32 CUDA tensor [N, d] (there is no CPU path)")
    pb = ldb = 0
    try:
        px, ldx = _rows("x", x, x)
        if b is not None:
            pb, ldb = _rows("b", b, x)
    except _Expanded:
        r, *rest = layer_norm_forward(_spread(x), _spread(b), weight=weight, bias=bias, eps=eps, keep8=keep8, out_r=out_r)
        return x if b is None else r, *rest
    w = _vector("weight", weight, x)
    c = 0 if bias is None else _vector("bias", bias, x)
    (N, d), device = x.shape, x.device
    r, pr = x, 0
    if b is not None:
        if out_r is None:
            r = _like(x)
        else:
            r = out_r
            if r.shape != x.shape or r.dtype != x.dtype or r.device != device or not r.is_contiguous():
                raise ValueError("out_r must be a contiguous tensor like x")
        pr = r.data_ptr()
    elif out_r is not None:
        raise ValueError("without b, r is x itself: there is nothing to write to out_r")
    n = _like(x)
    mean = torch.empty(N, dtype=torch.float32, device=device)
    rstd = torch.empty_like(mean)
    kept, packed = None, (0, 0, 0, 0)
    if keep8:
        kept = _packed_like(x)
        packed = kept._fields
    args = _LN.pack(_DT[x.dtype], N, d, eps, px, pb, w, c, ldx, ldb, pr, n.data_ptr(), mean.data_ptr(), rstd.data_ptr(), *packed,
                    0, 0, 0, 0, 0, 0, 0, 0, 0, 0, _stream(device.index))
    _abi.check(_abi.lib().lce_layer_norm_forward(args), "lce_layer_norm_forward")
    if out_r is not None:
        _written(out_r)
    return r, n, mean, rstd, kept


@_on_stream
def layer_norm_backward(dr, dn, r, *, weight, mean, rstd, bias: bool = True, workspace=None):
    """(dx, dweight, dbias) from the gradients dr of r (None: zero) and dn of n,
    the forward's r, or its 8-bit form, and statistics. dx is the gradient of x
    and of b; dbias is None with bias=False. `workspace`: a uint8 CUDA tensor of
    at least layer_norm_workspace_size(N, d) bytes; `stream`: the stream to run
    on."""
    if dn.dtype not in _DT or not dn.is_cuda or dn.dim() != 2:
        raise ValueError("dn must be a bfloat16 or float32 CUDA tensor [N, d] (there is no CPU path)")
    kept = isinstance(r, PackedActivation)
    pd = ldd = pr = ldr = 0
    packed = (0, 0, 0, 0)
    try:
        pn, ldn = _rows("dn", dn, dn)
        if dr is not None:
            pd, ldd = _rows("dr", dr, dn)
        if not kept:
            pr, ldr = _rows("r", r, dn)
    except _Expanded:
        return layer_norm_backward(_spread(dr), _spread(dn), r if kept else _spread(r), weight=weight, mean=mean, rstd=rstd,
                                   bias=bias, workspace=workspace)
    if kept:
        if r.shape != dn.shape or r.device != dn.device:
            raise ValueError(f"the packed r must be {tuple(dn.shape)} on dn's device")
        packed = r._fields
    w = _vector("weight", weight, dn)
    (N, d), device = dn.shape, dn.device
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.shape != (N,) or t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} must be the forward's contiguous fp32 [N] tensor")
    dx, dw = _like(dn), torch.empty_like(weight)
    dc = torch.empty_like(weight) if bias else None
    ws, size, keep = _scratch(workspace, layer_norm_workspace_size(N, d), device)
    args = _LN.pack(_DT[dn.dtype], N, d, 0.0, 0, 0, w, 0, 0, 0, pr, 0, mean.data_ptr(), rstd.data_ptr(), *packed, pd, pn, ldr, ldd,
                    ldn, dx.data_ptr(), dw.data_ptr(), _at(dc), ws, size, _stream(device.index))
    _abi.check(_abi.lib().lce_layer_norm_backward(args), "lce_layer_norm_backward")
    del keep
    return dx, dw, dc


class _LayerNorm(torch.autograd.Function):
    """(r, n); without b, r is x passed through, and the gradient that reaches
    it past the norm is joined inside the kernel."""

    @staticmethod
    def forward(ctx, x, b, weight, bias, eps, keep8):
        r, n, mean, rstd, kept = layer_norm_forward(x, b, weight=weight, bias=bias, eps=eps, keep8=keep8)
        if keep8:
            ctx.save_for_backward(kept.codes, kept.exps, weight, mean, rstd)
        else:
            ctx.save_for_backward(r, None, weight, mean, rstd)
        ctx.bias = bias is not None
        ctx.set_materialize_grads(False)
        return x.view_as(x) if b is None else r, n

    @staticmethod
    @once_differentiable
    def backward(ctx, dr, dn):
        r, exps, weight, mean, rstd = ctx.saved_tensors
        if exps is not None:
            r = PackedActivation(r, exps, weight.dtype)
        dn = torch.zeros(r.shape, dtype=weight.dtype, device=weight.device) if dn is None else _whole(dn)
        dx, dw, dc = layer_norm_backward(_whole(dr), dn, r, weight=weight, mean=mean, rstd=rstd, bias=ctx.bias)
        need = ctx.needs_input_grad
        return tuple(g if n else None for g, n in zip((dx, dx, dw, dc), need)) + (None, None)


def layer_norm(x, b=None, *, weight, bias=None, eps: float = 1e-5, keep8: bool = False):
    """Autograd form of layer_norm_forward: (r, n). With keep8 the backward pass
    keeps r's 8-bit form instead of r."""
    if not _recorded(x, b, weight, bias):
        return layer_norm_forward(x, b, weight=weight, bias=bias, eps=eps)[:2]
    return _LayerNorm.apply(x, b, weight, bias, eps, keep8)


# ----------------------------------------------------------- gated recurrence

_EVERY = 128   # tokens between the states that the forward keeps


def _tokens(name, t, like):
    """(address, token stride) of a [T, d] tensor, or of a [B, L, d] one as
    [B*L, d]. A dimension of one entry has no stride of its own."""
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be a {tuple(like.shape)} tensor of x's dtype and device")
    sh, st = t.shape, t.stride()
    d = sh[-1]
    if st[-1] != 1 and d > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if len(sh) == 3:
        B, L = sh[0], sh[1]
        if B > 1 and L > 1 and st[0] != L * st[1]:
            raise ValueError(f"{name}: the rows of a [B, L, d] tensor must be evenly spaced over B and L")
        ld, rows = (st[1] if L > 1 else st[0] if B > 1 else d), B * L
    else:
        ld, rows = st[0], sh[0]
    if rows < 2:
        ld = d
    elif ld < d:
        raise ValueError(f"the rows of {name} must not overlap")
    return t.data_ptr(), ld


def _recurrent(x, cu):
    """(B, T, d, address of cu)."""
    if x.dtype not in _DT or not x.is_cuda:
        raise ValueError("x must be a bfloat16 or float32 CUDA tensor (there is no CPU path)")
    if x.dim() not in (2, 3):
        raise ValueError("x must be [T, d] or [B, L, d]")
    if cu is None:
        return (x.shape[0], x.shape[0] * x.shape[1], x.shape[2], 0) if x.dim() == 3 else (1, x.shape[0], x.shape[1], 0)
    if x.dim() == 3:
        raise ValueError("sequence offsets go with [T, d] tensors")
    if cu.dtype != torch.int32 or cu.dim() != 1 or cu.device != x.device or not cu.is_contiguous() or cu.numel() < 2:
        raise ValueError("cu_seqlens must be a contiguous int32 tensor of at least two offsets on x's device")
    return cu.numel() - 1, x.shape[0], x.shape[1], cu.data_ptr()


def _states(name, t, B, d, device):
    if t is None:
        return 0
    if t.dtype != torch.float32 or t.shape != (B, d) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 [{B}, {d}] tensor on x's device")
    return t.data_ptr()


@_on_stream
def gated_recurrence_forward(x, g, cu_seqlens=None, *, state=None, out=None, out_state=None, keep: bool = False):
    """(h, final, kept) of the recurrence
        a_t = sigmoid(g_t),   h_t = a_t * h_{t-1} + (1 - a_t) * x_t
    over packed sequences: x and g (the gates' logits) [T, d] with int32 token
    offsets of the sequences (one sequence without them), or [B, L, d] tensors
    of equal lengths; L = 1 is one step of B sequences. `state` (fp32 [B, d];
    zeros if not given) is h before the first tokens and `final` h after the
    last ones, fp32; `out` receives h, `out_state` receives final and may be
    `state` (the backward then needs a copy of that as it was); else outputs
    must not overlap inputs or one another. Tokens behind the last sequence get
    h = 0. `kept` is what gated_recurrence_backward needs (with keep=True): fp32
    states, one for 128 tokens. `stream`: the stream to run on."""
    B, T, d, pc = _recurrent(x, cu_seqlens)
    device = x.device
    px, pg = _tokens("x", x, x), _tokens("g", g, x)
    ps = _states("state", state, B, d, device)
    given = [t for t in (out, out_state) if t is not None]
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=device)
    ph = _tokens("out", out, x)
    if out_state is None:
        out_state = torch.empty((B, d), dtype=torch.float32, device=device)
    pf = _states("out_state", out_state, B, d, device)
    kept = torch.empty(((T + _EVERY - 1) // _EVERY, d), dtype=torch.float32, device=device) if keep else None
    args = _SCAN.pack(_DT[x.dtype], max(B, 1), T, d, pc, px[0], pg[0], px[1], pg[1], ps, _at(kept), ph[0], ph[1], pf, 0, 0, 0, 0, 0, 0, 0, 0,
                      _stream(device.index))
    _abi.check(_abi.lib().lce_recurrence_forward(args), "lce_recurrence_forward")
    if given:
        _written(given)
    return out, out_state, kept


@_on_stream
def gated_recurrence_backward(dh, x, g, kept, cu_seqlens=None, *, state=None, dfinal=None, dx=None, dg=None):
    """(dx, dg, dstate) from the gradients dh of h and dfinal of the final states
    (fp32 [B, d]; None: zero), the forward's x, g and state, and the states it
    kept; h is formed again from those. dstate is None without a state. dx and
    dg may be given (strided slices of one gradient, say; not overlapping an
    input). `stream`: the stream to run on."""
    B, T, d, pc = _recurrent(x, cu_seqlens)
    device = x.device
    px, pg, pd = _tokens("x", x, x), _tokens("g", g, x), _tokens("dh", dh, x)
    ps, pf = _states("state", state, B, d, device), _states("dfinal", dfinal, B, d, device)
    chunks = (T + _EVERY - 1) // _EVERY
    if kept is None or kept.dtype != torch.float32 or kept.shape != (chunks, d) or kept.device != device or not kept.is_contiguous():
        raise ValueError(f"kept must be the forward's contiguous fp32 [{chunks}, {d}] states (keep=True)")
    given = [t for t in (dx, dg) if t is not None]
    dx = torch.empty(x.shape, dtype=x.dtype, device=device) if dx is None else dx
    dg = torch.empty(x.shape, dtype=x.dtype, device=device) if dg is None else dg
    pdx, pdg = _tokens("dx", dx, x), _tokens("dg", dg, x)
    dstate = None if state is None else torch.empty((B, d), dtype=torch.float32, device=device)
    args = _SCAN.pack(_DT[x.dtype], max(B, 1), T, d, pc, px[0], pg[0], px[1], pg[1], ps, kept.data_ptr(), 0, 0, 0, pd[0], pd[1], pf, pdx[0],
                      pdg[0], pdx[1], pdg[1], _at(dstate), _stream(device.index))
    _abi.check(_abi.lib().lce_recurrence_backward(args), "lce_recurrence_backward")
    if given:
        _written(given)
    return dx, dg, dstate


class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, cu, state):
        h, final, kept = gated_recurrence_forward(x, g, cu, state=state, keep=True)
        ctx.save_for_backward(x, g, cu, state, kept)
        ctx.set_materialize_grads(False)
        return h, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dfinal):
        x, g, cu, state, kept = ctx.saved_tensors
        dh = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dh is None else _whole(dh)
        dx, dg, dstate = gated_recurrence_backward(dh, x, g, kept, cu, state=state, dfinal=_whole(dfinal))
        need = ctx.needs_input_grad
        return dx if need[0] else None, dg if need[1] else None, None, dstate if need[3] else None


def gated_recurrence(x, g, cu_seqlens=None, *, state=None):
    """Autograd form of gated_recurrence_forward: (h, final)."""
    if not _recorded(x, g, state):
        return gated_recurrence_forward(x, g, cu_seqlens, state=state)[:2]
    return _GatedRecurrence.apply(x, g, cu_seqlens, state)
