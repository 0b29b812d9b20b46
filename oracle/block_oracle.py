"""fp64 reference of the operators between the embedding lookup and the head
loss, written out from their definitions one sequence and one head at a time:
packed attention with its gradients, the block norms with theirs, and the
clipping of gradients by their global norm. The attention functions also
return, for every output element, the sum of the absolute values of the terms
it is made of, from which rounding tolerances are derived."""
import numpy as np


def _sequences(lens_q, lens_k):
    a = c = 0
    for lq, lk in zip(lens_q, lens_k):
        yield a, a + lq, c, c + lk
        a, c = a + lq, c + lk


def _allowed(lq, lk, causal):
    if not causal:
        return np.ones((lq, lk), dtype=bool)
    return np.arange(lk)[None, :] <= np.arange(lq)[:, None] + (lk - lq)


def attention_forward(q, k, v, lens_q, lens_k, causal, scale):
    """(o, lse, abs_o, err): abs_o = sum_j p |v|; err = the largest
    scale * sum |q||k| + |lse|, which bounds the rounding of an exponent."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    T, H, _ = q.shape
    grp = H // k.shape[1]
    o, abs_o = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((H, T), -np.inf)
    err = 0.0
    for a, b, c, e in _sequences(lens_q, lens_k):
        if a == b or c == e:
            continue
        ok = _allowed(b - a, e - c, causal)
        rows = ok.any(1)
        for h in range(H):
            kk, vv = k[c:e, h // grp], v[c:e, h // grp]
            s = np.where(ok, scale * (q[a:b, h] @ kk.T), -np.inf)
            m = np.where(rows, s.max(1), 0.0)
            p = np.exp(s - m[:, None])
            tot = p.sum(1)
            p = p / np.where(rows, tot, 1.0)[:, None]
            o[a:b, h], abs_o[a:b, h] = p @ vv, p @ np.abs(vv)
            with np.errstate(divide="ignore"):
                lse[h, a:b] = np.where(rows, m + np.log(tot), -np.inf)
            big = np.where(ok, abs(scale) * (np.abs(q[a:b, h]) @ np.abs(kk).T), 0.0).max()
            err = max(err, big + np.abs(lse[h, a:b][rows]).max(initial=0.0))
    return o, lse, abs_o, err


def attention_backward(do, q, k, v, o, lse, lens_q, lens_k, causal, scale):
    """{name: (gradient, terms, parts)} for dq, dk, dv: `terms` sums |ds||k|
    (or |ds||q|, p|do|), what a rounding of ds and p to an operand type acts
    on; `parts` sums p (|do||v| + |do||o|) |k|, what fp32 arithmetic on ds
    acts on."""
    do, q, k, v, o, lse = (np.asarray(t, dtype=np.float64) for t in (do, q, k, v, o, lse))
    H = q.shape[1]
    grp = H // k.shape[1]
    zero = lambda t: [np.zeros_like(t) for _ in range(3)]  # noqa: E731
    dq, dk, dv = zero(q), zero(k), zero(v)
    for a, b, c, e in _sequences(lens_q, lens_k):
        if a == b or c == e:
            continue
        ok = _allowed(b - a, e - c, causal)
        for h in range(H):
            g = h // grp
            qq, kk, vv, dd = q[a:b, h], k[c:e, g], v[c:e, g], do[a:b, h]
            s = np.where(ok, scale * (qq @ kk.T), -np.inf)
            low = np.where(ok.any(1), lse[h, a:b], 0.0)
            p = np.exp(s - low[:, None])
            ds = np.where(ok, p * (dd @ vv.T - (dd * o[a:b, h]).sum(1, keepdims=True)), 0.0)
            part = p * (np.abs(dd) @ np.abs(vv).T + (np.abs(dd) * np.abs(o[a:b, h])).sum(1, keepdims=True))
            z = abs(scale)
            for acc, x, y in zip(dq, (scale * ds @ kk, z * np.abs(ds) @ np.abs(kk), z * part @ np.abs(kk)), range(3)):
                acc[a:b, h] = x
            for acc, x in zip(dk, (scale * ds.T @ qq, z * np.abs(ds).T @ np.abs(qq), z * part.T @ np.abs(qq))):
                acc[c:e, g] += x
            for acc, x in zip(dv, (p.T @ dd, p.T @ np.abs(dd), p.T @ np.abs(dd))):
                acc[c:e, g] += x
    return {"dq": tuple(dq), "dk": tuple(dk), "dv": tuple(dv)}


def block_norm_forward(x, b=None, w_post=None, gate=None, w_pre=None, scale=1.0, eps=1e-6):
    """(r, n, rstd_post, rstd_pre)."""
    f = lambda t: None if t is None else np.asarray(t, dtype=np.float64)  # noqa: E731
    x, b, w_post, gate, w_pre = map(f, (x, b, w_post, gate, w_pre))
    rstd = lambda t: 1.0 / np.sqrt((t * t).mean(1) + eps)  # noqa: E731
    post = pre = n = None
    r = x
    if b is not None:
        y = b
        if w_post is not None:
            post = rstd(b)
            y = b * post[:, None] * w_post
        r = x + scale * (y if gate is None else gate * y)
    if w_pre is not None:
        pre = rstd(r)
        n = r * pre[:, None] * w_pre
    return r, n, post, pre


def block_norm_backward(dr, dn, r, b=None, w_post=None, gate=None, w_pre=None, scale=1.0, rstd_post=None, rstd_pre=None):
    """(dx, db, dw_post, dgate, dw_pre) from the chain rule, with the given
    1/rms values."""
    f = lambda t: None if t is None else np.asarray(t, dtype=np.float64)  # noqa: E731
    dr, dn, r, b, w_post, gate, w_pre, rstd_post, rstd_pre = map(
        f, (dr, dn, r, b, w_post, gate, w_pre, rstd_post, rstd_pre))
    ref = r if r is not None else b

    def through(t, w, rstd, grad):
        hat = t * rstd[:, None]
        u = grad * w
        return rstd[:, None] * (u - hat * (u * hat).mean(1, keepdims=True)), (grad * hat).sum(0)

    dx = np.zeros_like(ref) if dr is None else dr.copy()
    db = dw_post = dgate = dw_pre = None
    if w_pre is not None:
        more, dw_pre = through(r, w_pre, rstd_pre, dn)
        dx = dx + more
    if b is not None:
        y = b if w_post is None else b * rstd_post[:, None] * w_post
        dy = scale * dx
        if gate is not None:
            dgate = scale * dx * y
            dgate = dgate.sum(0) if gate.ndim == 1 else dgate
            dy = dy * gate
        db = dy
        if w_post is not None:
            db, dw_post = through(b, w_post, rstd_post, dy)
    return dx, db, dw_post, dgate, dw_pre


def clip(grads, max_norm, eps=1e-6):
    """(norm, factor, clipped tensors)."""
    grads = [np.asarray(g, dtype=np.float64) for g in grads]
    norm = np.sqrt(sum((g * g).sum() for g in grads))
    factor = min(1.0, max_norm / (norm + eps))
    return norm, factor, [g * factor for g in grads]
