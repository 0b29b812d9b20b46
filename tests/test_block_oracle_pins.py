"""The fp64 reference of the block operators against torch autograd in fp64
(an independent derivative) and against differences."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import block_oracle as bo  # noqa: E402

CASES = [([5], [5], 2, 1, True), ([3, 0, 7, 1], [3, 0, 7, 1], 4, 2, True), ([4, 6, 2], [9, 3, 0], 2, 2, True),
         ([4, 6, 2], [9, 3, 0], 6, 2, False), ([1, 1], [1, 6], 1, 1, True)]


def _inputs(lq, lk, H, Hk, seed=0, D=8):
    g = np.random.default_rng(seed)
    t = lambda n, h: g.standard_normal((n, h, D))  # noqa: E731
    return t(sum(lq) + 2, H), t(sum(lk) + 2, Hk), t(sum(lk) + 2, Hk), t(sum(lq) + 2, H)


def _torch_attention(q, k, v, lq, lk, causal, scale):
    """Whole-matrix softmax with a block mask (rows that see nothing give 0)."""
    Tq, Tk, H = q.shape[0], k.shape[0], q.shape[1]
    ok = torch.zeros(Tq, Tk, dtype=torch.bool)
    a = c = 0
    for x, y in zip(lq, lk):
        for i in range(x):
            ok[a + i, c:c + (max(0, min(y, i + 1 + y - x)) if causal else y)] = True
        a, c = a + x, c + y
    kk, vv = (t.repeat_interleave(H // k.shape[1], 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, kk) * scale
    s = s.masked_fill(~ok, -1e300)
    p = torch.softmax(s, -1) * ok
    return torch.einsum("hij,jhd->ihd", p, vv)


@pytest.mark.parametrize("lq,lk,H,Hk,causal", CASES)
def test_attention_reference_against_autograd(lq, lk, H, Hk, causal):
    q, k, v, do = _inputs(lq, lk, H, Hk)
    o, lse, _, _ = bo.attention_forward(q, k, v, lq, lk, causal, 0.4)
    tq, tk, tv = (torch.tensor(t, requires_grad=True) for t in (q, k, v))
    to = _torch_attention(tq, tk, tv, lq, lk, causal, 0.4)
    np.testing.assert_allclose(o, to.detach().numpy(), atol=1e-12)
    to.backward(torch.tensor(do))
    ref = bo.attention_backward(do, q, k, v, o, lse, lq, lk, causal, 0.4)
    for name, t in (("dq", tq), ("dk", tk), ("dv", tv)):
        np.testing.assert_allclose(ref[name][0], t.grad.numpy(), atol=1e-12, err_msg=name)
        assert np.all(ref[name][1] + 1e-12 >= np.abs(ref[name][0]))


def test_attention_reference_against_differences():
    lq, lk = [4, 3], [4, 5]
    q, k, v, do = _inputs(lq, lk, 2, 1, seed=3)
    f = lambda q, k, v: (bo.attention_forward(q, k, v, lq, lk, True, 0.3)[0] * do).sum()  # noqa: E731
    o, lse, _, _ = bo.attention_forward(q, k, v, lq, lk, True, 0.3)
    ref = bo.attention_backward(do, q, k, v, o, lse, lq, lk, True, 0.3)
    g = np.random.default_rng(1)
    for name, at in (("dq", 0), ("dk", 1), ("dv", 2)):
        z = g.standard_normal(ref[name][0].shape)
        hi, lo = [q, k, v], [q, k, v]
        hi[at], lo[at] = hi[at] + 1e-5 * z, lo[at] - 1e-5 * z
        # central difference: error of order h^2 = 1e-10 times the third derivative, and eps/h = 1e-11
        assert abs((f(*hi) - f(*lo)) / 2e-5 - (ref[name][0] * z).sum()) < 1e-7


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "full"])
@pytest.mark.parametrize("pre", [False, True])
def test_norm_reference_against_autograd(post, gate, pre):
    g = np.random.default_rng(5)
    N, d = 6, 16
    t = lambda *s: torch.tensor(g.standard_normal(s), requires_grad=True)  # noqa: E731
    x, b = t(N, d), t(N, d)
    wp, wn = (t(d) if post else None), (t(d) if pre else None)
    gt = {"none": None, "channel": t(d) if gate == "channel" else None, "full": t(N, d) if gate == "full" else None}[gate]
    rms = lambda z: z * (z.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    y = rms(b) * wp if post else b
    r = x + 0.7 * (y if gt is None else gt * y)
    r.retain_grad()
    a, c = torch.tensor(g.standard_normal((N, d))), torch.tensor(g.standard_normal((N, d)))
    n = rms(r) * wn if pre else None
    ((r * a).sum() + ((n * c).sum() if pre else 0.0)).backward()
    num = lambda z: None if z is None else z.detach().numpy()  # noqa: E731
    R, Nn, po, pr = bo.block_norm_forward(num(x), num(b), num(wp), num(gt), num(wn), 0.7)
    np.testing.assert_allclose(R, num(r), atol=1e-12)
    out = bo.block_norm_backward(num(a), num(c) if pre else None, R, num(b), num(wp), num(gt), num(wn), 0.7, po, pr)
    for got, want in zip(out, (x, b, wp, gt, wn)):
        if want is None:
            assert got is None
        else:
            np.testing.assert_allclose(got, want.grad.numpy(), atol=1e-11)
    if pre:
        np.testing.assert_allclose(Nn, num(n), atol=1e-12)


def test_clip_reference():
    norm, c, out = bo.clip([np.array([3.0]), np.array([[4.0, 0.0]])], 1.0, eps=0.0)
    assert norm == 5.0 and c == 0.2
    np.testing.assert_allclose(np.concatenate([o.ravel() for o in out]), [0.6, 0.8, 0.0])
    assert bo.clip([np.array([3.0])], 10.0)[1] == 1.0
