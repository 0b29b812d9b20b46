"""Block norms of tensors whose rows share memory (expanded over the tokens):
the results are, bit for bit, those of the same values laid out row by row, so
no tolerance is needed."""
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SHAPES = [(7, 264), (2, 8), (305, 1000), (5001, 520), (3, 12288)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    yield


def make(N, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(N + d)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(DT[dtype])  # noqa: E731
    t = {k: r(N, d) for k in ("x", "b", "gate", "dr", "dn")}
    t.update({k + "_row": r(1, d) for k in ("x", "b", "gate", "dr", "dn")})
    t.update(w_post=r(d), w_pre=r(d))
    return t


def both(t, names, N):
    """The tensors with `names` expanded from one row, and the same laid out in full."""
    spread = {k: t[k + "_row"].expand(N, -1) if k in names else t[k] for k in ("x", "b", "gate", "dr", "dn")}
    assert all(spread[k].stride(0) == 0 for k in names)
    return spread, {k: v.contiguous() for k, v in spread.items()}


def same(xs, ys):
    assert len(xs) == len(ys)
    for x, y in zip(xs, ys):
        assert (x is None) == (y is None) and (x is None or torch.equal(x, y))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
@pytest.mark.parametrize("names", [("x",), ("b",), ("gate",), ("dr",), ("dn",), ("x", "b", "gate", "dr", "dn")], ids=lambda n: "+".join(n))
def test_expanded_rows(names, shape, dtype):
    N, d = shape
    t = make(N, d, dtype)
    got, want = [], []
    for v, out in zip(both(t, names, N), (got, want)):
        kw = dict(w_post=t["w_post"], gate=v["gate"], w_pre=t["w_pre"], scale=0.5)
        r, n, po, pr = lce.block_norm_forward(v["x"], v["b"], **kw)
        out += [r, n, po, pr, *lce.block_norm_backward(v["dr"], v["dn"], r, v["b"], rstd_post=po, rstd_pre=pr, **kw)]
        # the norm alone, whose stream is the input itself
        x, n, _, pr = lce.block_norm_forward(v["x"], w_pre=t["w_pre"])
        assert x is v["x"]
        out += [n, pr, *lce.block_norm_backward(v["dr"], v["dn"], x, w_pre=t["w_pre"], rstd_pre=pr)]
    same(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_expanded_rows_through_autograd(dtype):
    """A gate and a block output of one row each, broadcast by the caller: their gradients are sums over the rows."""
    N, d = 37, 320
    t = make(N, d, dtype)
    full = both(t, ("b", "gate"), N)[1]
    leaf = lambda v: v.clone().requires_grad_(True)  # noqa: E731
    x, b, gate = leaf(t["x"]), leaf(t["b_row"]), leaf(t["gate_row"])
    x2, b2, gate2 = leaf(t["x"]), leaf(full["b"]), leaf(full["gate"])
    for args in ((x, b.expand(N, -1), gate.expand(N, -1)), (x2, b2, gate2)):
        out = lce.block_norm(args[0], args[1], w_post=t["w_post"], gate=args[2], w_pre=t["w_pre"])
        torch.autograd.backward(out, (t["dr"], t["dn"]))
    assert torch.equal(x.grad, x2.grad)
    # both are sums of the same N terms, added in fp32 in some order and rounded once to their type
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for a, b in ((b.grad, b2.grad), (gate.grad, gate2.grad)):
        want, terms = b.double().sum(0), b.double().abs().sum(0)
        assert bool(((a.double()[0] - want).abs() <= u * want.abs() + N * 2.0 ** -24 * terms).all())
