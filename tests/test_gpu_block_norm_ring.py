"""Block norms of enough rows that every block takes more rounds than its ring
has stages, forward and backward, at widths of every number of packs a thread,
with rows apart and numbers of rows that no group divides; and the backward of
rows too wide for the ring, several rows a block. Against the fp64 reference,
evaluated on the GPU (these tensors hold up to 10 million elements).

Tolerances: those of the smaller shapes. An output is rounded once to its type
(u = 2^-8 bf16, 2^-23 fp32); fp32 arithmetic acts on the absolute terms of each
formula with F = 2^-24 * (64 + d / 8); column sums add N terms in groups,
F_cols = 2^-24 * (64 + N) + 4 F."""
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    yield
    assert lce.device_status() == 0


def make(N, d, dtype, post, gate, pre, wide=0):
    g = torch.Generator(device="cuda").manual_seed(N + d)
    r = lambda *s, mean=0.0, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std + mean).to(DT[dtype])  # noqa: E731
    rows = lambda std=1.0: r(N, d + wide, std=std)[:, :d]  # noqa: E731
    return dict(x=rows(2.0), b=rows(), w_post=r(d, mean=1.0, std=0.2) if post else None,
                gate={"none": None, "channel": r(d), "full": rows()}[gate], w_pre=r(d, mean=1.0, std=0.2) if pre else None,
                dr=rows(), dn=rows() if pre else None)


def f64(t):
    return None if t is None else t.double()


def within(name, got, want, tol):
    assert bool(((f64(got) - want).abs() <= tol).all()), (name, float(((f64(got) - want).abs() - tol).max()))


def check(N, d, dtype, post, gate, pre, scale=0.5, eps=1e-6, wide=0, no_dr=False, no_b=False):
    t = make(N, d, dtype, post, gate, pre, wide)
    x, b, wo, gt, wi = (f64(t[k]) for k in ("x", "b", "w_post", "gate", "w_pre"))
    kw = dict(w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"])
    if no_b:
        r, n, po, pr = lce.block_norm_forward(t["x"], w_pre=t["w_pre"], eps=eps)
        t["b"] = b = None
    else:
        r, n, po, pr = lce.block_norm_forward(t["x"], t["b"], scale=scale, eps=eps, **kw)
        kw["scale"] = scale
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    F = 2.0 ** -24 * (64 + d / 8)
    R, X = x, x.abs()
    if not no_b:
        y = b
        if post:
            Po = (b.square().mean(1) + eps).rsqrt()
            within("rstd_post", po, Po, F * Po)
            y = b * Po[:, None] * wo
        add = scale * (y if gt is None else y * gt)
        R, X = x + add, x.abs() + add.abs()
        within("r", r, R, u * R.abs() + F * X)
        del y, add
    if pre:
        Pr = (R.square().mean(1) + eps).rsqrt()
        rel = F * (1 + X.square().mean(1) * Pr ** 2)
        within("rstd_pre", pr, Pr, rel * Pr)
        Nn = R * Pr[:, None] * wi
        within("n", n, Nn, u * Nn.abs() + 4 * rel[:, None] * wi.abs() * Pr[:, None] * X)
        del Nn
    del x, R, X
    dr = None if no_dr else t["dr"]
    stats = dict(rstd_post=po, rstd_pre=pr)
    got = lce.block_norm_backward(dr, t["dn"], r, t["b"], **stats, **kw)
    again = lce.block_norm_backward(dr, t["dn"], r, t["b"], **stats, **kw)
    for p, q in zip(got, again):
        assert (p is None) == (q is None) and (p is None or torch.equal(p, q))
    del again
    # the formulas, and beside each the sum of its terms' absolute values
    po, pr = f64(po), f64(pr)
    dx = torch.zeros(N, d, device="cuda", dtype=torch.float64) if no_dr else f64(dr)
    dx_t = dx.abs()
    Fc = 2.0 ** -24 * (64 + N) + 4 * F
    if pre:
        hat, dn = f64(r) * pr[:, None], f64(t["dn"])
        within("dw_pre", got[4], (dn * hat).sum(0), u * (dn * hat).sum(0).abs() + Fc * (dn * hat).abs().sum(0))
        z = wi * dn
        dx = dx + pr[:, None] * (z - hat * (z * hat).mean(1, keepdim=True))
        dx_t = dx_t + pr[:, None] * (z.abs() + hat.abs() * (z * hat).abs().mean(1, keepdim=True))
        del z, hat, dn
    within("dx", got[0], dx, u * dx.abs() + 4 * F * dx_t)
    if no_b:
        assert got[1] is None and got[2] is None and got[3] is None
        return
    bh = b * po[:, None] if post else b
    dy, dy_t = scale * dx, abs(scale) * dx_t
    if gt is not None:
        g, s = dy * bh * (wo if post else 1.0), dy_t * bh.abs() * (wo.abs() if post else 1.0)
        if gate == "channel":
            g, s = g.sum(0), s.sum(0)
        within("dgate", got[3], g, u * g.abs() + Fc * s)
        dy, dy_t = dy * gt, dy_t * gt.abs()
        del g, s
    if post:
        g, s = (dy * bh).sum(0), (dy_t * bh.abs()).sum(0)
        within("dw_post", got[2], g, u * g.abs() + Fc * s)
        z, z_t = wo * dy, wo.abs() * dy_t
        dy = po[:, None] * (z - bh * (z * bh).mean(1, keepdim=True))
        dy_t = po[:, None] * (z_t + bh.abs() * (z_t * bh.abs()).mean(1, keepdim=True))
    within("db", got[1], dy, u * dy.abs() + 4 * F * dy_t)


# (dtype, d, N): by packs a thread 1, 2, 4 (8 in fp32) in the forward; of 16 bytes, 1, 2 and more in the backward.
# N rows give a block of 152 more rounds than stages in both directions.
ROWS = [("bf16", 128, 100_003), ("bf16", 512, 20_011), ("bf16", 1000, 10_007), ("bf16", 2048, 5003), ("bf16", 4096, 2503),
        ("bf16", 4608, 1511), ("bf16", 8192, 1009),
        ("fp32", 128, 50_021), ("fp32", 256, 30_011), ("fp32", 520, 12_007), ("fp32", 1024, 8009), ("fp32", 2048, 4003), ("fp32", 2560, 2011),
        ("fp32", 4096, 1013)]


@pytest.mark.parametrize("dtype,d,N", ROWS, ids=lambda v: str(v))
@pytest.mark.parametrize("post,gate,pre", [(True, "channel", True), (True, "full", True)], ids=["channel", "full"])
def test_many_rows(dtype, d, N, post, gate, pre):
    check(N, d, dtype, post, gate, pre)


@pytest.mark.parametrize("dtype,d,N", [r for r in ROWS if r[1] in (512, 1000, 4608, 520, 2560)], ids=lambda v: str(v))
@pytest.mark.parametrize("post,gate,pre,no_dr", [(False, "none", True, False), (True, "none", False, False), (False, "channel", True, True),
                                                 (True, "full", False, False), (False, "none", False, False), (True, "full", True, True)])
def test_many_rows_options(dtype, d, N, post, gate, pre, no_dr):
    check(N, d, dtype, post, gate, pre, scale=-0.3, wide=24, no_dr=no_dr)


@pytest.mark.parametrize("dtype,d,N", [r for r in ROWS if r[1] in (512, 4096, 520, 2560)], ids=lambda v: str(v))
def test_many_rows_alone_and_in_place(dtype, d, N):
    check(N, d, dtype, False, "none", True, no_b=True)
    check(N, d, dtype, False, "none", True, no_b=True, wide=8, no_dr=True)
    t = make(N, d, dtype, True, "channel", True)
    kw = dict(w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"], scale=0.5)
    want = lce.block_norm_forward(t["x"], t["b"], **kw)
    got = lce.block_norm_forward(t["x"], t["b"], out_r=t["x"], **kw)
    assert got[0] is t["x"] and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype,d,N", [("bf16", 8712, 701), ("bf16", 12288, 700), ("fp32", 5128, 903), ("fp32", 16384, 611)], ids=lambda v: str(v))
@pytest.mark.parametrize("post,gate,pre,no_dr", [(True, "channel", True, False), (True, "full", True, True), (False, "none", True, False)])
def test_wide_rows(dtype, d, N, post, gate, pre, no_dr):
    check(N, d, dtype, post, gate, pre, no_dr=no_dr)


@pytest.mark.parametrize("dtype,d,N", [("bf16", 8, 400_009), ("bf16", 24, 150_001), ("fp32", 8, 200_003), ("fp32", 40, 40_009)], ids=lambda v: str(v))
@pytest.mark.parametrize("gate", ["channel", "full"])
def test_narrow_rows(dtype, d, N, gate):
    check(N, d, dtype, True, gate, True)
