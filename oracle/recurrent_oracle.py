"""fp64 reference of the operators of a recurrent block, written out from their
definitions: the layer norm with its gradients, what activations kept in 8 bits
stand for, and the gated recurrence, one sequence and one token at a time, with
its gradients. The recurrence also returns, for every output element, what the
rounding errors of all steps before it amount to, from which tolerances are
derived."""
import numpy as np

BLOCK, LOW, HIGH, MOST = 128, -100, 119, 448.0
# the magnitudes that an e4m3 code can stand for: 8 steps in each power of two from 2^-6 to 2^8 (480 is not one), and
# the eighths of 2^-6 below
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1])


def pack(x):
    """(codes, exponents [ceil(d/128), N]) of x [N, d], fp64."""
    x = np.asarray(x, dtype=np.float64)
    N, d = x.shape
    blocks = (d + BLOCK - 1) // BLOCK
    codes, exps = np.zeros((N, d), dtype=np.uint8), np.zeros((blocks, N), dtype=np.int8)
    for k in range(blocks):
        y = x[:, k * BLOCK:(k + 1) * BLOCK]
        good = np.isfinite(y).all(1)
        y = np.where(good[:, None], y, 0.0)
        top = np.abs(y).max(1)
        e = np.full(N, LOW)
        for c in range(LOW, HIGH):                      # the least exponent that holds the largest value
            e = np.where(top > MOST * 2.0 ** c, c + 1, e)
        z = y * 2.0 ** -e[:, None].astype(np.float64)
        mag = np.minimum(np.abs(z), MOST)
        i = np.searchsorted(E4M3, mag)                  # E4M3[i - 1] < mag <= E4M3[i]
        low = np.maximum(i - 1, 0)
        up, down = E4M3[i] - mag, mag - E4M3[low]
        pick = np.where(up < down, i, np.where(up > down, low, np.where(i % 2 == 0, i, low)))
        c = pick | np.where(np.signbit(z), 0x80, 0)
        codes[:, k * BLOCK:(k + 1) * BLOCK] = np.where(good[:, None], c, 0x7F)
        exps[k] = np.where(good, e, -128)
    return codes, exps


def unpack(codes, exps):
    codes = np.asarray(codes)
    e = np.repeat(np.asarray(exps).astype(np.float64).T, BLOCK, 1)[:, :codes.shape[1]]
    value = np.concatenate([E4M3, [np.nan]])[codes & 0x7F] * np.where(codes & 0x80, -1.0, 1.0)
    return np.where(e == -128, np.nan, value * 2.0 ** np.where(e == -128, 0, e))


def layer_norm_forward(x, b=None, weight=None, bias=None, eps=1e-5, store=lambda r: r):
    """(r, n, mean, rstd); `store` rounds r to its type, which n and the
    statistics are taken from."""
    f = lambda t: None if t is None else np.asarray(t, dtype=np.float64)  # noqa: E731
    x, b, weight, bias = map(f, (x, b, weight, bias))
    r = x if b is None else x + b
    s = r if b is None else store(r)
    mean = s.mean(1)
    c = s - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    n = c * rstd[:, None] * weight
    return r, n if bias is None else n + bias, mean, rstd


def layer_norm_backward(dr, dn, r, weight, mean, rstd):
    """(dx, dweight, dbias) from the chain rule, with the given statistics."""
    dn, r, weight, mean, rstd = (np.asarray(t, dtype=np.float64) for t in (dn, r, weight, mean, rstd))
    hat = (r - mean[:, None]) * rstd[:, None]
    u = weight * dn
    dx = rstd[:, None] * (u - u.mean(1, keepdims=True) - hat * (u * hat).mean(1, keepdims=True))
    if dr is not None:
        dx = dx + np.asarray(dr, dtype=np.float64)
    return dx, (dn * hat).sum(0), dn.sum(0)


def _gates(g):
    with np.errstate(over="ignore"):
        e = np.exp(-np.asarray(g, dtype=np.float64))
    return 1.0 / (1.0 + e), 1.0 / (1.0 + np.exp(np.minimum(np.asarray(g, dtype=np.float64), 700.0)))


def recurrence_forward(x, g, lens, state=None):
    """(h, final, err_h, err_final, kept). A step that is off by a share of the
    absolute values of its terms, every step before it as well, is off by that
    share of err_*: e_t = a_t e_{t-1} + abs_t, abs_t being h_t with every term
    taken absolutely. kept[c] = h of token 128 c - 1 (zeros for c = 0)."""
    x = np.asarray(x, dtype=np.float64)
    T, d = x.shape
    a, rest = _gates(g)
    h, eh = np.zeros_like(x), np.zeros_like(x)
    final, efinal, t = [], [], 0
    for i, n in enumerate(lens):
        s = np.zeros(d) if state is None else np.asarray(state[i], dtype=np.float64)
        z = np.abs(s)
        e = z
        for _ in range(n):
            s, z = a[t] * s + rest[t] * x[t], a[t] * z + rest[t] * np.abs(x[t])
            e = a[t] * e + z
            h[t], eh[t] = s, e
            t += 1
        final.append(s), efinal.append(e)
    kept = np.zeros(((T + 127) // 128, d))
    if T > 128:
        kept[1:] = h[127:T - 1:128][:len(kept) - 1]
    return h, np.array(final), eh, np.array(efinal), kept


def recurrence_backward(dh, x, g, lens, state=None, dfinal=None):
    """{name: (gradient, err)} for dx, dg, dstate, err as above."""
    dh, x = np.asarray(dh, dtype=np.float64), np.asarray(x, dtype=np.float64)
    T, d = x.shape
    a, rest = _gates(g)
    h, _, eh, _, _ = recurrence_forward(x, g, lens, state)
    dx, dg, ex, eg = (np.zeros_like(x) for _ in range(4))
    ds, es, begin = [], [], 0
    for i, n in enumerate(lens):
        m = np.zeros(d) if dfinal is None else np.asarray(dfinal[i], dtype=np.float64)
        e = z = np.abs(m)
        for t in range(begin + n - 1, begin - 1, -1):
            first = t == begin
            hp = (np.zeros(d) if state is None else np.asarray(state[i], dtype=np.float64)) if first else h[t - 1]
            ep = np.abs(hp) if first else eh[t - 1]
            m, z = dh[t] + m, np.abs(dh[t]) + z
            e = e + z
            dx[t], ex[t] = rest[t] * m, rest[t] * e
            dg[t], eg[t] = m * (hp - x[t]) * a[t] * rest[t], e * (ep + np.abs(x[t])) * a[t] * rest[t]
            m, z, e = a[t] * m, a[t] * z, a[t] * e
        ds.append(m), es.append(e)
        begin += n
    return {"dx": (dx, ex), "dg": (dg, eg), "dstate": (np.array(ds), np.array(es))}
