"""The norms around a block with its gate and residual scale, forward and
backward, against the fp64 reference.

Tolerances, elementwise: an output is rounded once to its type (u = 2^-8 for
bf16, twice the largest relative rounding; 2^-23 for fp32); the fp32
arithmetic before it acts on the absolute terms of each formula with
F = 2^-24 * (64 + d / 8): a thread adds at most d/threads squares or products
in a row and the threads' sums are joined in a tree, and each formula is a
handful of operations long. Column sums add the roundings of N terms in
groups: F_cols = 2^-24 * (64 + N)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402
from oracle import block_oracle as bo  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    yield


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(N, d, dtype, post, gate, pre, seed=0, wide=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s, mean=0.0, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std + mean).to(DT[dtype])

    rows = lambda std=1.0, mean=0.0: r(N, d + wide, std=std, mean=mean)[:, :d]  # noqa: E731
    return dict(x=rows(2.0), b=rows(), w_post=r(d, mean=1.0, std=0.2) if post else None,
                gate={"none": None, "channel": r(d), "full": rows()}[gate], w_pre=r(d, mean=1.0, std=0.2) if pre else None,
                dr=rows(), dn=rows() if pre else None)


def check(N, d, dtype, post, gate, pre, scale=0.5, eps=1e-6, seed=0, wide=0, no_dr=False):
    t = make(N, d, dtype, post, gate, pre, seed, wide)
    kw = dict(w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"], scale=scale)
    r, n, po, pr = lce.block_norm_forward(t["x"], t["b"], eps=eps, **kw)
    R, Nn, Po, Pr = bo.block_norm_forward(*(f64(t[k]) for k in ("x", "b", "w_post", "gate", "w_pre")), scale, eps)
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    F = 2.0 ** -24 * (64 + d / 8)
    X = np.abs(f64(t["x"])) + np.abs(R - f64(t["x"]))     # absolute terms of r
    assert np.all(np.abs(f64(r) - R) <= u * np.abs(R) + F * X)
    if post:
        assert np.all(np.abs(f64(po) - Po) <= F * Po)
    if pre:
        # r enters with its terms' rounding, relative to the row's size
        rel = F * (1 + (X * X).mean(1) * Pr ** 2)
        assert np.all(np.abs(f64(pr) - Pr) <= rel * Pr)
        A = np.abs(f64(t["w_pre"])) * Pr[:, None] * X
        assert np.all(np.abs(f64(n) - Nn) <= u * np.abs(Nn) + 4 * rel[:, None] * A)
    else:
        assert n is None and pr is None
    dr = None if no_dr else t["dr"]
    got = lce.block_norm_backward(dr, t["dn"], r, t["b"], rstd_post=po, rstd_pre=pr, **kw)
    got2 = lce.block_norm_backward(dr, t["dn"], r, t["b"], rstd_post=po, rstd_pre=pr, **kw)
    torch.cuda.synchronize()
    for a, b in zip(got, got2):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    args = [f64(z) for z in (dr, t["dn"], r, t["b"], t["w_post"], t["gate"], t["w_pre"])]
    want = bo.block_norm_backward(*args, scale, f64(po), f64(pr))
    # absolute terms: the same formulas with every factor taken absolutely
    dx_t = np.zeros((N, d)) if dr is None else np.abs(f64(dr))
    hat_r = np.abs(f64(r) * f64(pr)[:, None]) if pre else None
    if pre:
        ut = np.abs(f64(t["w_pre"]) * f64(t["dn"]))
        dx_t = dx_t + f64(pr)[:, None] * (ut + hat_r * (ut * hat_r).mean(1, keepdims=True))
    hat_b = np.abs(f64(t["b"])) * (f64(po)[:, None] if post else 1.0)
    wp = np.abs(f64(t["w_post"])) if post else 1.0
    gt = np.abs(f64(t["gate"])) if gate != "none" else 1.0
    dy_t = abs(scale) * gt * dx_t
    db_t = f64(po)[:, None] * (wp * dy_t + hat_b * (wp * dy_t * hat_b).mean(1, keepdims=True)) if post else dy_t
    Fc = 2.0 ** -24 * (64 + N) + 4 * F
    dg_t = abs(scale) * dx_t * hat_b * wp
    terms = (dx_t, db_t, (dy_t * hat_b).sum(0) if post else None,
             None if gate == "none" else dg_t if gate == "full" else dg_t.sum(0),
             (np.abs(f64(t["dn"])) * hat_r).sum(0) if pre else None)
    for i, (a, w, s) in enumerate(zip(got, want, terms)):
        if w is None:
            assert a is None
            continue
        err = np.abs(f64(a) - w)
        tol = u * np.abs(w) + (4 * F if i < 2 else Fc) * s
        assert np.all(err <= tol), (i, err.max(), float((err - tol).max()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 8), (3, 64), (7, 264), (1, 4096), (33, 1000), (5, 2048), (400, 520), (3, 4104),
                                   (2, 8192), (9, 12288), (2, 16384), (1000, 128)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_shapes(shape, dtype):
    check(*shape, dtype, True, "channel", True)
    check(*shape, dtype, True, "full", True, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("post", [False, True], ids=["", "post"])
@pytest.mark.parametrize("gate", ["none", "channel", "full"])
@pytest.mark.parametrize("pre", [False, True], ids=["", "pre"])
def test_options(post, gate, pre, dtype):
    check(37, 320, dtype, post, gate, pre, scale=1.0)
    check(37, 320, dtype, post, gate, pre, scale=-0.3, seed=2, wide=24, no_dr=pre)


@pytest.mark.parametrize("dtype,d", [("bf16", 264), ("bf16", 4608), ("fp32", 2560), ("fp32", 5128)])
@pytest.mark.parametrize("post,gate,pre,no_dr", [(True, "channel", True, False), (True, "channel", True, True), (False, "full", True, False),
                                                 (True, "full", True, True), (True, "channel", False, False), (True, "full", False, False)])
def test_options_in_the_backward_of_rows_of_all_widths(dtype, d, post, gate, pre, no_dr):
    check(45, d, dtype, post, gate, pre, scale=0.7, seed=3, no_dr=no_dr)


@pytest.mark.parametrize("dtype,d", [("bf16", 264), ("bf16", 4608), ("bf16", 8712), ("fp32", 2560), ("fp32", 5128)])
@pytest.mark.parametrize("with_dr", [False, True])
def test_norm_alone_at_all_widths(dtype, d, with_dr):
    """Only w_pre. The bound is a rounding of the result and, for sums of d
    or 45 products of values of order one, d + 45 fp32 roundings of the largest."""
    t = make(45, d, dtype, False, "none", True)
    x = t["x"].contiguous()
    _, n, _, pr = lce.block_norm_forward(x, w_pre=t["w_pre"])
    dr = t["dr"] if with_dr else None
    dx, _, _, _, dw = lce.block_norm_backward(dr, t["dn"], x, w_pre=t["w_pre"], rstd_pre=pr)
    want = bo.block_norm_backward(f64(dr) if with_dr else None, f64(t["dn"]), f64(x), w_pre=f64(t["w_pre"]), rstd_pre=f64(pr))
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for got, w in ((dx, want[0]), (dw, want[4])):
        assert np.all(np.abs(f64(got) - w) <= u * np.abs(w) + (d + 45) * 2.0 ** -24 * np.abs(w).max())


def test_norm_alone_and_in_place():
    t = make(50, 512, "bf16", True, "channel", True)
    x = t["x"].contiguous()
    r, n, po, pr = lce.block_norm_forward(x, w_pre=t["w_pre"])
    assert r is x and po is None
    _, Nn, _, Pr = bo.block_norm_forward(f64(x), w_pre=f64(t["w_pre"]))
    assert np.all(np.abs(f64(n) - Nn) <= 2.0 ** -8 * np.abs(Nn) + 1e-6)
    dx, db, dwp, dg, dw = lce.block_norm_backward(None, t["dn"], x, w_pre=t["w_pre"], rstd_pre=pr)
    want = bo.block_norm_backward(None, f64(t["dn"]), f64(x), w_pre=f64(t["w_pre"]), rstd_pre=f64(pr))
    assert db is None and dwp is None and dg is None
    assert np.abs(f64(dx) - want[0]).max() <= 2.0 ** -8 * np.abs(want[0]).max()
    assert np.abs(f64(dw) - want[4]).max() <= 2.0 ** -8 * np.abs(want[4]).max()
    kw = dict(w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"])
    a = lce.block_norm_forward(x.clone(), t["b"], **kw)
    y = x.clone()
    b = lce.block_norm_forward(y, t["b"], out_r=y, **kw)
    assert b[0] is y and all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_no_rows(dtype):
    t = make(0, 64, dtype, True, "channel", True)
    kw = dict(w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"])
    r, n, po, pr = lce.block_norm_forward(t["x"], t["b"], **kw)
    assert r.shape == (0, 64)
    out = lce.block_norm_backward(t["dr"], t["dn"], r, t["b"], rstd_post=po, rstd_pre=pr, **kw)
    torch.cuda.synchronize()
    assert all(bool((w == 0).all()) for w in out[2:])


def test_rows_of_zeros_and_not_finite():
    """A row of zeros is normed by 1/sqrt(eps); a row that is not finite stays within itself."""
    t = make(6, 256, "fp32", True, "none", True)
    t["x"][2] = 0
    t["b"][2] = 0
    kw = dict(w_post=t["w_post"], w_pre=t["w_pre"])
    r, n, po, pr = lce.block_norm_forward(t["x"], t["b"], **kw)
    assert bool((r[2] == 0).all()) and bool((n[2] == 0).all()) and abs(po[2].item() - 1e3) < 1e-2
    t["b"][4, 7] = float("nan")
    r2, n2, po2, _ = lce.block_norm_forward(t["x"], t["b"], **kw)
    keep = [0, 1, 2, 3, 5]
    assert torch.equal(r2[keep], r[keep]) and torch.equal(n2[keep], n[keep]) and bool(n2[4].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [1, 7, 33])
def test_infinities_of_the_last_row_stay_infinities_in_the_column_sums(rows, dtype):
    """An infinite gradient in the last row is an infinity in its own column's sums and nothing in the others'."""
    t = make(rows, 256, dtype, True, "channel", True)
    kw = dict(w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"])
    r, _, po, pr = lce.block_norm_forward(t["x"], t["b"], **kw)
    t["dr"][rows - 1, 9] = float("inf")
    dx, _, dw_post, dgate, dw_pre = lce.block_norm_backward(t["dr"], t["dn"], r, t["b"], rstd_post=po, rstd_pre=pr, **kw)
    for got in (dx[rows - 1], dw_post, dgate):
        assert torch.nonzero(~got.isfinite()).flatten().tolist() == [9] and bool(got[9].isinf())
    assert bool(dw_pre.isfinite().all())
    t["dr"][rows - 1, 9] = 0.0
    t["dn"][rows - 1, 5] = float("-inf")
    dw_pre = lce.block_norm_backward(t["dr"], t["dn"], r, t["b"], rstd_post=po, rstd_pre=pr, **kw)[4]
    assert torch.nonzero(~dw_pre.isfinite()).flatten().tolist() == [5] and bool(dw_pre[5].isinf())


def test_autograd_and_differences():
    """Central differences of the fp32 forward (h = 2^-7): truncation of order
    h^2, rounding of order 2^-24 |f| / h; the bound is 1e-2 of |grad||z|/sqrt(n)."""
    t = make(20, 192, "fp32", True, "full", True)
    names = ("x", "b", "w_post", "gate", "w_pre")
    leaves = {k: t[k].clone().requires_grad_(True) for k in names}
    call = lambda d: lce.block_norm(d["x"], d["b"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"], scale=0.7)  # noqa: E731
    f = lambda d: sum((o.double() * w.double()).sum() for o, w in zip(call(d), (t["dr"], t["dn"])))  # noqa: E731
    f(leaves).backward()
    g = torch.Generator(device="cuda").manual_seed(9)
    for k in names:
        z = torch.randn(t[k].shape, generator=g, device="cuda")
        hi, lo = dict(t), dict(t)
        hi[k], lo[k] = t[k] + z * 2.0 ** -7, t[k] - z * 2.0 ** -7
        with torch.no_grad():
            num = (f(hi) - f(lo)).item() * 2.0 ** 6
        want = (leaves[k].grad.double() * z.double()).sum().item()
        assert abs(num - want) <= 1e-2 * float(leaves[k].grad.norm()), k
    # the norm alone, with a gradient past it
    x, w = t["x"].clone().requires_grad_(True), t["w_pre"].clone().requires_grad_(True)
    r, n = lce.block_norm(x, w_pre=w)
    ((r * t["dr"]).sum() + (n * t["dn"]).sum()).backward()
    x2, w2 = t["x"].clone().requires_grad_(True), t["w_pre"].clone().requires_grad_(True)
    m = x2 * (x2.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt() * w2
    ((x2 * t["dr"]).sum() + (m * t["dn"]).sum()).backward()
    assert torch.allclose(x.grad, x2.grad, atol=1e-4) and torch.allclose(w.grad, w2.grad, atol=1e-3)


def test_another_stream_and_long_rows_apart():
    """A row stride that takes offsets past 2^31 elements, on another stream."""
    N, d, wide = 3, 512, 1 << 30
    buf = torch.empty(N * wide, device="cuda", dtype=torch.bfloat16).view(N, wide)
    t = make(N, d, "bf16", True, "channel", True)
    x = buf[:, 64:64 + d]
    x.copy_(t["x"])
    kw = dict(w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"])
    want = lce.block_norm_forward(t["x"].contiguous(), t["b"], **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lce.block_norm_forward(x, t["b"], stream=s, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    t = make(4, 64, "bf16", True, "channel", True)
    f = lce.block_norm_forward
    for bad in (lambda: f(t["x"].cpu(), t["b"]), lambda: f(t["x"].half(), t["b"].half()), lambda: f(t["x"], t["b"].float()),
                lambda: f(t["x"], t["b"][:2]), lambda: f(t["x"], t["b"], w_post=t["w_post"][:8]),
                lambda: f(t["x"]), lambda: f(t["x"], w_post=t["w_post"], w_pre=t["w_pre"]),
                lambda: f(t["x"], t["b"], gate=t["b"][:2]), lambda: f(t["x"][0], t["b"][0]),
                lambda: f(t["x"].t(), t["b"].t()), lambda: f(t["x"], t["b"], out_r=t["x"][:2]),
                lambda: lce.block_norm_backward(t["dr"], None, t["x"], t["b"], w_pre=t["w_pre"]),
                lambda: lce.block_norm_backward(t["dr"], t["dn"], t["x"], t["b"], w_pre=t["w_pre"])):
        with pytest.raises(ValueError):
            bad()
    wide = lambda d: torch.zeros(2, d, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    for d in (12, 16392):
        with pytest.raises(lce.LceError):
            f(wide(d), wide(d))
    with pytest.raises(lce.LceError):
        f(t["x"], t["b"], scale=float("inf"))
    with pytest.raises(lce.LceError):
        f(t["x"], t["b"], eps=-1.0)
    odd = torch.zeros(4 * 64 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(4, 64)
    with pytest.raises(lce.LceError):
        f(odd, t["b"])
    assert lce.block_norm_workspace_size(4, 64) > 0
