"""The fp64 reference of the recurrent block's operators, pinned to torch: the
8-bit form to torch's own e4m3 conversion, the gradients to torch's autograd and
to differences."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import recurrent_oracle as ro  # noqa: E402

RNG = np.random.default_rng(0)


def test_e4m3_values_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t[:127], ro.E4M3) and np.array_equal(-t[128:255], ro.E4M3) and np.isnan(t[[127, 255]]).all()


@pytest.mark.parametrize("d", [8, 128, 200])
def test_pack_is_torchs_rounding_at_the_least_scale(d):
    x = RNG.standard_normal((40, d)) * np.exp(3 * RNG.standard_normal((40, d)))
    x = x.astype(np.float32).astype(np.float64)
    x[0] = 0.0
    x[1, :8] = [448.0, 449.0, 1.75, 1.7500001, 0.0, -0.0, 2.0 ** -9, 2.0 ** -10]
    codes, exps = ro.pack(x)
    for n in range(40):
        for k in range((d + 127) // 128):
            y, e = x[n, 128 * k:128 * k + 128], int(exps[k, n])
            assert np.abs(y).max() <= 448 * 2.0 ** e and (e == -100 or np.abs(y).max() > 448 * 2.0 ** (e - 1))
            want = torch.from_numpy(y * 2.0 ** -e).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            assert np.array_equal(codes[n, 128 * k:128 * k + 128], want)
    back = ro.unpack(codes, exps)
    scale = 2.0 ** np.repeat(exps.astype(np.float64).T, 128, 1)[:, :d]
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale))


def test_pack_of_values_that_are_not_finite_and_of_the_largest():
    x = np.zeros((3, 256))
    x[0, 5], x[1, 130], x[2, 0] = np.inf, np.nan, 3.4e38
    codes, exps = ro.pack(x)
    back = ro.unpack(codes, exps)
    assert np.isnan(back[0, :128]).all() and np.isnan(back[1, 128:]).all() and not np.isnan(back[0, 128:]).any()
    assert back[2, 0] == 448 * 2.0 ** 119 and exps[0, 2] == 119


def test_layer_norm_is_torchs():
    x, b, dn, dr = (torch.from_numpy(RNG.standard_normal((7, 40)) + 0.3) for _ in range(4))
    w, c = torch.from_numpy(RNG.standard_normal(40)), torch.from_numpy(RNG.standard_normal(40))
    leaves = [t.requires_grad_(True) for t in (x, b, w, c)]
    r = x + b
    n = torch.nn.functional.layer_norm(r, (40,), w, c, 1e-5)
    grads = torch.autograd.grad((r * dr).sum() + (n * dn).sum(), leaves)
    R, N, mean, rstd = ro.layer_norm_forward(*(t.detach().numpy() for t in (x, b, w, c)))
    assert np.allclose(N, n.detach().numpy(), rtol=1e-12, atol=1e-12) and np.allclose(R, r.detach().numpy())
    dx, dw, dc = ro.layer_norm_backward(dr.numpy(), dn.numpy(), R, w.detach().numpy(), mean, rstd)
    for got, want in zip((dx, dx, dw, dc), grads):
        assert np.allclose(got, want.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("with_state", [False, True])
def test_recurrence_is_autograds(with_state):
    lens, d = [5, 0, 1, 140], 3
    T = sum(lens) + 2
    x, g, dh = (torch.from_numpy(RNG.standard_normal((T, d))) for _ in range(3))
    s, df = (torch.from_numpy(RNG.standard_normal((4, d))) for _ in range(2))
    leaves = [t.requires_grad_(True) for t in (x, g, s)]
    a, t, hs, finals = torch.sigmoid(g), 0, [], []
    for i, n in enumerate(lens):
        h = s[i] if with_state else torch.zeros(d, dtype=torch.float64)
        for _ in range(n):
            h = a[t] * h + (1 - a[t]) * x[t]
            hs.append(h)
            t += 1
        finals.append(h)
    H, F = torch.stack(hs), torch.stack(finals)
    grads = torch.autograd.grad((H * dh[:t]).sum() + (F * df).sum(), leaves, allow_unused=True)
    args = [z.detach().numpy() for z in (x, g)]
    state = s.detach().numpy() if with_state else None
    h, final, eh, _, kept = ro.recurrence_forward(*args, lens, state)
    assert np.allclose(h[:t], H.detach().numpy(), rtol=1e-13, atol=1e-14) and not h[t:].any()
    assert np.allclose(final, F.detach().numpy()) and np.all(eh >= np.abs(h)) and np.array_equal(kept[1], h[127])
    out = ro.recurrence_backward(dh.numpy(), *args, lens, state, df.numpy())
    for name, want in zip(("dx", "dg", "dstate"), grads):
        if want is not None and (with_state or name != "dstate"):
            assert np.allclose(out[name][0], want.numpy(), rtol=1e-10, atol=1e-13), name
            assert np.all(out[name][1] >= np.abs(out[name][0]) * (1 - 1e-12))


def test_gradients_are_differences():
    lens, d = [4, 3], 2
    x, g, dh, s = RNG.standard_normal((7, d)), RNG.standard_normal((7, d)), RNG.standard_normal((7, d)), RNG.standard_normal((2, d))
    out = ro.recurrence_backward(dh, x, g, lens, s)
    loss = lambda: (ro.recurrence_forward(x, g, lens, s)[0] * dh).sum()  # noqa: E731
    for name, t in (("dx", x), ("dg", g), ("dstate", s)):
        for i in range(t.shape[0]):
            keep = t[i, 1]
            t[i, 1] = keep + 1e-6
            up = loss()
            t[i, 1] = keep - 1e-6
            down = loss()
            t[i, 1] = keep
            assert abs((up - down) / 2e-6 - out[name][0][i, 1]) < 1e-8
