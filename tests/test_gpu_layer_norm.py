"""Layer norm with the residual sum before it, forward and backward, with the
stream or its 8-bit form kept, against the fp64 reference.

Tolerances, elementwise: an output is rounded once to its type (u = half a
step: 2^-8 for bf16, 2^-24 for fp32); the fp32 arithmetic before it acts on the
absolute terms of each formula with F = 2^-24 * (64 + d / 8): a thread adds at
most d/threads values in a row, the threads' sums are joined in a tree, and each
formula is a handful of operations long. The mean is off by F mean|r|, a centred
value by that and a rounding, so the variance by F (1 + 2 mean|r| rstd) of
itself. Column sums add the roundings of N terms: 2^-24 * (64 + N) more."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402
from oracle import recurrent_oracle as ro  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    lce.device_status()
    yield


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(N, d, dtype, add, seed=0, wide=0, shift=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s, mean=0.0, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std + mean).to(DT[dtype])

    rows = lambda std=1.0, mean=0.0: r(N, d + wide, std=std, mean=mean)[:, :d]  # noqa: E731
    return dict(x=rows(2.0, shift), b=rows() if add else None, w=r(d, mean=1.0, std=0.3), c=r(d), dn=rows(), dr=rows())


def close(name, got, want, u, slack):
    err = np.abs(f64(got) - want)
    tol = u * np.abs(want) + slack
    assert np.all(err <= tol), (name, float(err.max()), float((err - tol).max()))


def check(N, d, dtype, add=True, bias=True, more=True, keep8=False, seed=0, wide=0, eps=1e-5, shift=0.5):
    t = make(N, d, dtype, add, seed, wide, shift)
    w, c, dr = t["w"], t["c"] if bias else None, t["dr"] if more else None
    r, n, mean, rstd, kept = lce.layer_norm_forward(t["x"], t["b"], weight=w, bias=c, eps=eps, keep8=keep8)
    assert (kept is not None) == keep8 and (add or r is t["x"])
    store = lambda v: f64(torch.from_numpy(v).to(DT[dtype]))  # noqa: E731
    R, Nn, M, S = ro.layer_norm_forward(f64(t["x"]), f64(t["b"]), f64(w), f64(c), eps, store)
    u, F = U[dtype], 2.0 ** -24 * (64 + d / 8)
    close("r", r, R, u, 2.0 ** -24 * np.abs(R))
    Rs = f64(r)
    if add:
        R_, Nn, M, S = ro.layer_norm_forward(Rs, None, f64(w), f64(c), eps)
    A = np.abs(Rs).mean(1)
    rel = F * (1 + 2 * A * S)
    close("mean", mean, M, 0, F * A)
    close("rstd", rstd, S, 0, rel * S)
    W, C = np.abs(f64(w)), 0 if c is None else np.abs(f64(c))
    hat = np.abs(Rs - M[:, None]) * S[:, None]
    close("n", n, Nn, u, 2 * (rel[:, None] * hat * W + F * (A * S)[:, None] * W + F * C))
    # backward, from the statistics as they were left
    source = Rs
    if keep8:
        codes, exps = ro.pack(Rs)
        assert np.array_equal(kept.codes.cpu().numpy(), codes) and np.array_equal(kept.exps.cpu().numpy(), exps)
        source = ro.unpack(codes, exps)
    M, S = f64(mean), f64(rstd)
    held = kept if keep8 else r
    got = lce.layer_norm_backward(dr, t["dn"], held, weight=w, mean=mean, rstd=rstd, bias=bias)
    again = lce.layer_norm_backward(dr, t["dn"], held, weight=w, mean=mean, rstd=rstd, bias=bias)
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, again))
    want = ro.layer_norm_backward(f64(dr), f64(t["dn"]), source, f64(w), M, S)
    H, D = (np.abs(source) + np.abs(M)[:, None]) * S[:, None], np.abs(f64(t["dn"]))
    ut = W * D
    terms = S[:, None] * (ut + ut.mean(1, keepdims=True) + H * (ut * H).mean(1, keepdims=True)) + (0 if dr is None else np.abs(f64(dr)))
    Fc = 2.0 ** -24 * (64 + N) + 4 * F
    close("dx", got[0], want[0], u, 4 * F * terms)
    close("dweight", got[1], want[1], u, Fc * (D * H).sum(0))
    if bias:
        close("dbias", got[2], want[2], u, Fc * D.sum(0))
    else:
        assert got[2] is None
    return r, n, mean, rstd, kept, got


SHAPES = [(1, 8), (3, 64), (7, 264), (1, 4096), (33, 1000), (5, 2048), (400, 520), (3, 4104), (2, 8192), (9, 12288), (2, 16384),
          (1000, 128), (4099, 128), (2500, 1032)]


@pytest.mark.parametrize("keep8", [False, True], ids=["", "keep8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_shapes(shape, dtype, keep8):
    check(*shape, dtype, keep8=keep8)
    assert lce.device_status() == 0


@pytest.mark.parametrize("keep8", [False, True], ids=["", "keep8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("add,bias,more", [(False, True, True), (True, False, True), (True, True, False), (False, False, False)])
def test_options(add, bias, more, dtype, keep8):
    for N, d, wide in ((37, 320, 0), (37, 320, 24), (3000, 776, 8), (700, 4104, 0)):
        check(N, d, dtype, add, bias, more, keep8, seed=2, wide=wide)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_mean_far_above_the_spread(dtype):
    """The variance is taken around the mean: sums of squares would lose it in fp32."""
    check(40, 512, dtype, shift=1000.0, add=False)


def test_rows_that_are_constant_or_zero():
    x = torch.zeros(3, 256, device="cuda")
    x[1] = 7.0
    w, c = torch.ones(256, device="cuda"), torch.full((256,), 0.25, device="cuda")
    r, n, mean, rstd, kept = lce.layer_norm_forward(x, weight=w, bias=c, keep8=True)
    assert torch.equal(n, torch.full_like(n, 0.25)) and mean.tolist() == [0.0, 7.0, 0.0]
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    assert torch.equal(lce.unpack_activation(kept), x)


def test_infinities_stay_in_their_row():
    x = torch.randn(600, 256, device="cuda").bfloat16()
    x[5, 7], x[9, 0], x[599, 255] = float("inf"), float("nan"), float("-inf")
    w = torch.ones(256, device="cuda").bfloat16()
    _, n, mean, rstd, kept = lce.layer_norm_forward(x, weight=w, keep8=True)
    bad = torch.zeros(600, dtype=torch.bool, device="cuda")
    bad[[5, 9, 599]] = True
    assert bool(n.float().isnan().any(1)[bad].all()) and not bool((~n.float().isfinite()).any(1)[~bad].any())
    dx, _, _ = lce.layer_norm_backward(None, torch.ones_like(x), kept, weight=w, mean=mean, rstd=rstd)
    assert not bool((~dx.float().isfinite()).any(1)[~bad].any())


def test_no_rows():
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    for keep8 in (False, True):
        r, n, mean, rstd, kept = lce.layer_norm_forward(x, x, weight=w, keep8=keep8)
        dx, dw, dc = lce.layer_norm_backward(None, x, kept if keep8 else r, weight=w, mean=mean, rstd=rstd)
        assert n.shape == dx.shape == (0, 64) and not dw.any() and not dc.any()


def test_in_place_on_another_stream_and_in_a_graph():
    t = make(500, 640, "bf16", True, seed=3)
    w, c = t["w"], t["c"]
    r, n, mean, rstd, kept = lce.layer_norm_forward(t["x"], t["b"], weight=w, bias=c, keep8=True)
    grads = lce.layer_norm_backward(t["dr"], t["dn"], kept, weight=w, mean=mean, rstd=rstd)
    for into in ("x", "b"):
        x, b = t["x"].clone(), t["b"].clone()
        out = x if into == "x" else b
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = lce.layer_norm_forward(x, b, weight=w, bias=c, out_r=out, stream=s)
        torch.cuda.synchronize()
        assert got[0] is out and torch.equal(out, r) and torch.equal(got[1], n)
    need = lce.layer_norm_workspace_size(500, 640)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g_r, g_n, g_mean, g_rstd, g_kept = lce.layer_norm_forward(t["x"], t["b"], weight=w, bias=c, keep8=True)
        g_grads = lce.layer_norm_backward(t["dr"], t["dn"], g_kept, weight=w, mean=g_mean, rstd=g_rstd, workspace=ws[:need])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g_r, r) and torch.equal(g_n, n) and all(torch.equal(a, b) for a, b in zip(g_grads, grads))
    assert torch.equal(g_kept.codes, kept.codes) and torch.equal(g_kept.exps, kept.exps) and bool((ws[need:] == 77).all())


def test_expanded_rows_are_copied_and_given_tensors_count_as_written():
    w = torch.randn(64, device="cuda")
    x, b = torch.randn(1, 64, device="cuda").expand(50, 64), torch.randn(50, 64, device="cuda")
    r, n, *_ = lce.layer_norm_forward(x, b, weight=w)
    r2, n2, *_ = lce.layer_norm_forward(x.contiguous(), b, weight=w)
    assert torch.equal(r, r2) and torch.equal(n, n2)
    out, before = torch.empty_like(b), b._version
    lce.layer_norm_forward(x, b, weight=w, out_r=out)
    assert out._version > 0 and b._version == before


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("add", [False, True])
def test_autograd(add, keep8):
    t = make(30, 136, "fp32", add)
    leaves = [t[k].clone().requires_grad_(True) for k in (("x", "b", "w", "c") if add else ("x", "w", "c"))]
    x, b, w, c = leaves if add else (leaves[0], None, *leaves[1:])
    r, n = lce.layer_norm(x, b, weight=w, bias=c, keep8=keep8)
    grads = torch.autograd.grad((r * t["dr"]).sum() + (n * t["dn"]).sum(), leaves)
    _, _, mean, rstd, kept = lce.layer_norm_forward(t["x"], t["b"], weight=t["w"], bias=t["c"], keep8=True)
    dx, dw, dc = lce.layer_norm_backward(t["dr"], t["dn"], kept if keep8 else r.detach(), weight=t["w"], mean=mean, rstd=rstd)
    assert all(torch.equal(g, v) for g, v in zip(grads, (dx, dx, dw, dc) if add else (dx, dw, dc)))
    # n alone, r alone, and no second derivative
    r, n = lce.layer_norm(x, b, weight=w, bias=c, keep8=keep8)
    (gx,) = torch.autograd.grad(n.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        gx.sum().backward()
    r, n = lce.layer_norm(x, b, weight=w, bias=c, keep8=keep8)
    (gx,) = torch.autograd.grad(r.sum(), x)
    assert torch.equal(gx, torch.ones_like(gx))


def test_keep8_keeps_a_byte_a_value():
    x = torch.randn(4096, 1024, device="cuda").bfloat16().requires_grad_(True)
    w = torch.ones(1024, device="cuda").bfloat16().requires_grad_(True)
    held = {}
    for keep8 in (False, True):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        y = x * 1.0
        r, n = lce.layer_norm(y, weight=w, keep8=keep8)
        del y, r
        held[keep8] = torch.cuda.memory_allocated() - before - n.numel() * 2
        del n
    assert held[False] > 2 * x.numel() and held[True] < 1.1 * x.numel()
