"""The operators of a training step between the embedding lookup and the head
loss, as cases to be timed: attention forward and backward over packed
sequences, the norms around a block fused with its gate and residual scale
(forward and backward), and the global gradient norm with clipping.

`run` computes each in elementary torch operations in 32 bits (own = False) or
through this package's entry points (own = True). Sequence lengths are part of
a case (a text of numbers), so that the work of a case is known from it alone."""
import math

import torch

own = False
DEV = "cuda"
EPS = 1e-6          # norm epsilon
CLIP_EPS = 1e-6     # added to the gradient norm in the clip factor


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a short prompt of a small model: latency only
        dict(name="attn fwd short prompt", op="attn_fwd", lens_q="37", lens_k="37", tail=0, heads=8, kv_heads=2, dim=64,
             causal=True, dtype="bf16"),
        # documents packed into one 8192-token row, lengths ~ N(850, 300): the framework's llama8b width (4096 = 32 x 128)
        dict(name="attn fwd packed documents", op="attn_fwd", lens_q="1012,433,761,1290,850,517,64,1103,905,288,969",
             lens_k="1012,433,761,1290,850,517,64,1103,905,288,969", tail=0, heads=32, kv_heads=8, dim=128, causal=True,
             dtype="bf16"),
        # one long document at the same width: the arithmetic-bound end
        dict(name="attn bwd long document", op="attn_bwd", lens_q="8192", lens_k="8192", tail=0, heads=32, kv_heads=8,
             dim=128, causal=True, dtype="bf16"),
        # the gpt1b width (2048 = 32 x 64), no shared heads, ragged rows and a padded end (3482 of 4096 valid)
        dict(name="attn bwd ragged rows", op="attn_bwd", lens_q="1024,771,1,640,333,713", lens_k="1024,771,1,640,333,713",
             tail=614, heads=32, kv_heads=32, dim=64, causal=True, dtype="bf16"),
        # queries over other keys (an encoder's states), a head size between the powers of two, one side empty in places
        dict(name="attn bwd cross", op="attn_bwd", lens_q="300,0,511,97,200", lens_k="1500,320,777,0,1", tail=0, heads=16,
             kv_heads=4, dim=80, causal=False, dtype="bf16"),
        # the tiny fp32 configuration (256 tokens, width 64)
        dict(name="attn bwd tiny fp32", op="attn_bwd", lens_q="131,125", lens_k="131,125", tail=0, heads=2, kv_heads=2,
             dim=32, causal=True, dtype="fp32"),
        # one generated token: latency only
        dict(name="norm fwd one token", op="norm_fwd", rows=1, d=4096, post=True, gate="none", pre=True, scale=1.0,
             dtype="bf16"),
        # a training batch at the llama8b width: norms on both sides of a block and a learned gate per channel
        dict(name="norm fwd batch", op="norm_fwd", rows=16384, d=4096, post=True, gate="channel", pre=True, scale=0.5,
             dtype="bf16"),
        # its backward pass
        dict(name="norm bwd batch", op="norm_bwd", rows=16384, d=4096, post=True, gate="channel", pre=True, scale=0.5,
             dtype="bf16"),
        # the same in fp32 at the gpt1b width, an odd number of rows, a gate of its own for every element
        dict(name="norm bwd fp32 full gate", op="norm_bwd", rows=3482, d=2048, post=True, gate="full", pre=True, scale=1.0,
             dtype="fp32"),
        # a small model's gradients: many little tensors, latency only
        dict(name="clip small model", op="clip", sizes="64000," + "4096,4096,4096,4096,64,16384,16384,64," * 3 + "64,63,1",
             fp32_every=1, max_norm=1.0),
        # the gpt1b width: fp32 gradient of the vocabulary matrix (50304 x 2048) and eight blocks in bf16
        dict(name="clip large model", op="clip",
             sizes="103022592," + "4194304,4194304,4194304,4194304,16777216,16777216,2048," * 8 + "2048",
             fp32_every=57, max_norm=1.0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attn_fwd", "attn_bwd", "attn_bwd", "norm_fwd", "norm_bwd", "clip"])
    dtype = "bf16" if rng.random() < 0.8 else "fp32"
    if op.startswith("attn"):
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 7])
        dim = rng.choice([8, 32, 64, 64, 72, 80, 96, 128, 128, 128])
        most = 32768 if dtype == "bf16" else 1024
        most = min(most, int(math.sqrt(8192.0 * 8192.0 * 32 * 128 / (heads * max(dim, 64))) * (0.7 if op == "attn_bwd" else 1.0)))
        total = log(1, most)
        cross = rng.random() < 0.3
        n = min(total, log(1, 24))
        cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
        lens_q = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        lens_k = [rng.choice([0, 1, x, x + rng.randrange(1, 200), x // 2]) for x in lens_q] if cross else lens_q
        if op == "attn_bwd" or sum(lens_k) == 0:
            # one sequence of some length: over a single key the gradients of q and k are nothing but zeros
            lens_q[-1] += 17
            lens_k = lens_q if not cross else lens_k[:-1] + [lens_k[-1] + 17]
        return dict(op=op, lens_q=",".join(map(str, lens_q)), lens_k=",".join(map(str, lens_k)),
                    tail=rng.choice([0, 0, rng.randrange(1, 300)]), heads=heads, kv_heads=kv, dim=dim,
                    causal=rng.random() < 0.75, dtype=dtype)
    if op.startswith("norm"):
        d = 8 * log(8, 1024)
        return dict(op=op, rows=log(1, min(16384, 16384 * 4096 // d // (2 if dtype == "fp32" else 1))), d=d,
                    post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "full"]), pre=rng.random() < 0.85,
                    scale=rng.choice([1.0, 0.5, 0.22]), dtype=dtype)
    n = log(1, 60)
    sizes = [log(1, 4_000_000) for _ in range(n)]
    return dict(op="clip", sizes=",".join(map(str, sizes)), fp32_every=rng.choice([1, 2, 5, 1000]),
                max_norm=rng.choice([0.1, 1.0, 1e6]))


def _ints(text):
    return [int(x) for x in str(text).split(",") if x != ""]


def _pairs(case):
    """Allowed (query, key) pairs."""
    n = 0
    for lq, lk in zip(_ints(case["lens_q"]), _ints(case["lens_k"])):
        if not case["causal"]:
            n += lq * lk
        else:
            # row i sees clamp(i + 1 + lk - lq, 0, lk) keys
            first = max(0, lq - lk)              # rows before it see nothing
            m = lq - first
            n += m * (1 + lk - lq + first) + m * (m - 1) // 2 if m > 0 and lk > 0 else 0
    return n


def work(case):
    es = 2 if case.get("dtype") == "bf16" else 4
    if case["op"].startswith("attn"):
        tq = sum(_ints(case["lens_q"])) + case["tail"]
        tk = sum(_ints(case["lens_k"])) + case["tail"]
        q, kv = tq * case["heads"] * case["dim"] * es, tk * case["kv_heads"] * case["dim"] * es
        lse = tq * case["heads"] * 4
        pairs = _pairs(case) * case["heads"] * case["dim"]
        if case["op"] == "attn_fwd":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * pairs}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * pairs}
    if case["op"].startswith("norm"):
        nd = case["rows"] * case["d"]
        full = 1 if case["gate"] == "full" else 0
        if case["op"] == "norm_fwd":
            return {"bytes": nd * es * (3 + full + (1 if case["pre"] else 0)), "flops": nd * 10}
        return {"bytes": nd * es * (4 + 2 * full + (2 if case["pre"] else 0) - (0 if case["pre"] or case["post"] or case["gate"] != "none" else 1)),
                "flops": nd * 25}
    nbytes = sum(n * (4 if i % case["fp32_every"] == 0 else 2) for i, n in enumerate(_ints(case["sizes"])))
    return {"bytes": 2 * nbytes, "flops": 3 * sum(_ints(case["sizes"]))}


# ----------------------------------------------------------------- the inputs

def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def _attn_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    lq, lk = _ints(case["lens_q"]), _ints(case["lens_k"])
    tq, tk = sum(lq) + case["tail"], sum(lk) + case["tail"]
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if lq == lk:
        # self-attention: q, k and v are slices of one projection's output
        qkv = torch.randn(tq, h + 2 * hk, d, generator=g, device=DEV).to(dt)
        q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        cu_q = _cu(lq)
        cu_k = cu_q
    else:
        q = torch.randn(tq, h, d, generator=g, device=DEV).to(dt)
        kv = torch.randn(tk, 2 * hk, d, generator=g, device=DEV).to(dt)
        k, v = kv[:, :hk], kv[:, hk:]
        cu_q, cu_k = _cu(lq), _cu(lk)
    do = torch.randn(tq, h, d, generator=g, device=DEV).to(dt)
    return q, k, v, do, cu_q, cu_k


def _norm_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    n, d = case["rows"], case["d"]

    def rand(*shape, mean=0.0, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dt)

    s = {"x": rand(n, d, std=2.0), "b": rand(n, d), "scale": case["scale"],
         "w_post": rand(d, mean=1.0, std=0.1) if case["post"] else None,
         "w_pre": rand(d, mean=1.0, std=0.1) if case["pre"] else None,
         "gate": {"none": None, "channel": rand(d, mean=0.5, std=0.2), "full": rand(n, d, mean=0.5, std=0.2)}[case["gate"]]}
    if case["op"] == "norm_bwd":
        s["dr"] = rand(n, d)
        s["dn"] = rand(n, d) if case["pre"] else None
    return s


def prepare(case, seed):
    s = {"op": case["op"]}
    if case["op"].startswith("attn"):
        q, k, v, do, cu_q, cu_k = _attn_inputs(case, seed)
        s.update(q=q, k=k, v=v, cu_q=cu_q, cu_k=cu_k, causal=case["causal"], scale=case["dim"] ** -0.5)
        if case["op"] == "attn_bwd":
            # what the forward pass left: its output, rounded once, and each row's log-sum-exp
            o, lse = _attention_forward(q, k, v, cu_q, cu_k, case["causal"], s["scale"])
            s.update(do=do, o=o, lse=lse)
    elif case["op"].startswith("norm"):
        s.update(_norm_inputs(case, seed))
        if case["op"] == "norm_bwd":
            # what the forward pass left: the stream after the block and the rows' 1/rms
            r, _, s["rstd_post"], s["rstd_pre"] = _norm_forward(s["x"], s["b"], s["w_post"], s["gate"], s["w_pre"], s["scale"])
            s["r"] = r
            del s["x"]
    else:
        g = torch.Generator(device=DEV).manual_seed(seed)
        s["grads"] = [(torch.randn(n, generator=g, device=DEV) * 0.02).to(torch.float32 if i % case["fp32_every"] == 0 else torch.bfloat16)
                      for i, n in enumerate(_ints(case["sizes"]))]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        s["max_norm"] = case["max_norm"]
    return s


# ------------------------------------------------------------- the plain forms

def _allowed(cu_q, cu_k, tq, tk, causal):
    iq, ik = torch.arange(tq, device=DEV), torch.arange(tk, device=DEV)
    cq, ck = cu_q.long(), cu_k.long()
    sq, sk = torch.bucketize(iq, cq[1:], right=True), torch.bucketize(ik, ck[1:], right=True)
    n = cq.numel() - 1
    ok = (sq[:, None] == sk[None, :]) & (sq[:, None] < n)
    if causal:
        at = sq.clamp(max=n - 1)
        end = iq - cq[at] + (ck[at + 1] - ck[at]) - (cq[at + 1] - cq[at])   # last key position a row sees
        ok &= (ik - ck[sk.clamp(max=n - 1)])[None, :] <= end[:, None]
    return ok


def _scores(q, k, cu_q, cu_k, causal, scale):
    """Masked scores [kv heads, group, queries, keys] and q, k in 32 bits by head."""
    hk = k.shape[1]
    qf = q.float().transpose(0, 1).reshape(hk, q.shape[1] // hk, q.shape[0], q.shape[2])
    kf = k.float().transpose(0, 1).unsqueeze(1)
    s = torch.matmul(qf, kf.transpose(-1, -2))
    s *= scale
    s.masked_fill_(~_allowed(cu_q, cu_k, q.shape[0], k.shape[0], causal), -math.inf)
    return s, qf, kf


def _attention_forward(q, k, v, cu_q, cu_k, causal, scale):
    s, _, _ = _scores(q, k, cu_q, cu_k, causal, scale)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.float().transpose(0, 1).unsqueeze(1))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log()).squeeze(-1)
    return o.flatten(0, 1).transpose(0, 1).contiguous().to(q.dtype), lse.flatten(0, 1)


def _attention_backward(do, q, k, v, o, lse, cu_q, cu_k, causal, scale):
    p, qf, kf = _scores(q, k, cu_q, cu_k, causal, scale)
    hk, grp = qf.shape[:2]
    low = lse.view(hk, grp, -1, 1)
    p = p.sub_(torch.where(low == -math.inf, torch.zeros_like(low), low)).exp_()
    dof = do.float().transpose(0, 1).reshape(qf.shape)
    vf = v.float().transpose(0, 1).unsqueeze(1)
    dv = torch.matmul(p.transpose(-1, -2), dof).sum(1)
    delta = (do.float() * o.float()).sum(-1).transpose(0, 1).reshape(hk, grp, -1, 1)
    ds = torch.matmul(dof, vf.transpose(-1, -2)).sub_(delta).mul_(p)
    dq = torch.matmul(ds, kf) * scale
    dk = torch.matmul(ds.transpose(-1, -2), qf).sum(1) * scale
    rows = lambda t: t.transpose(0, 1).contiguous().to(q.dtype)  # noqa: E731
    return rows(dq.flatten(0, 1)), rows(dk), rows(dv)


def _norm_forward(x, b, w_post, gate, w_pre, scale):
    y, rstd_post, rstd_pre, n = b.float(), None, None, None
    if w_post is not None:
        rstd_post = torch.rsqrt((y * y).mean(-1) + EPS)
        y = y * rstd_post[:, None] * w_post.float()
    if gate is not None:
        y = y * gate.float()
    r = x.float() + scale * y
    if w_pre is not None:
        rstd_pre = torch.rsqrt((r * r).mean(-1) + EPS)
        n = (r * rstd_pre[:, None] * w_pre.float()).to(x.dtype)
    return r.to(x.dtype), n, rstd_post, rstd_pre


def _norm_backward(dr, dn, r, b, w_post, gate, w_pre, scale, rstd_post, rstd_pre):
    dt, dw_pre, dw_post, dgate = b.dtype, None, None, None
    g = dr.float()
    if w_pre is not None:
        hat = r.float() * rstd_pre[:, None]
        u = dn.float()
        dw_pre = (u * hat).sum(0).to(dt)
        u = u * w_pre.float()
        g = g + rstd_pre[:, None] * (u - hat * (u * hat).mean(-1, keepdim=True))
    bf = b.float()
    hat = bf * rstd_post[:, None] if w_post is not None else bf
    y = hat * w_post.float() if w_post is not None else bf
    db = scale * g
    if gate is not None:
        dgate = db * y
        dgate = (dgate if gate.dim() == 2 else dgate.sum(0)).to(dt)
        db = db * gate.float()
    if w_post is not None:
        dw_post = (db * hat).sum(0).to(dt)
        u = db * w_post.float()
        db = rstd_post[:, None] * (u - hat * (u * hat).mean(-1, keepdim=True))
    return g.to(dt), db.to(dt), dw_post, dgate, dw_pre


def _clip(grads, max_norm, out):
    squares = torch.stack([t.float().square().sum() for t in grads])
    norm = squares.sum().sqrt()
    c = (max_norm / (norm + CLIP_EPS)).clamp(max=1.0)
    return norm, [o.copy_(t.float() * c) for t, o in zip(grads, out)]


def run(s):
    op = s["op"]
    if own:
        import chunked_vocab_cross_gb300 as lce
        if op == "attn_fwd":
            return lce.attention_forward(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["causal"], scale=s["scale"])
        if op == "attn_bwd":
            return lce.attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu_q"], s["cu_k"],
                                          causal=s["causal"], scale=s["scale"])
        if op == "norm_fwd":
            return lce.block_norm_forward(s["x"], s["b"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"],
                                          scale=s["scale"], eps=EPS)
        if op == "norm_bwd":
            return lce.block_norm_backward(s["dr"], s["dn"], s["r"], s["b"], w_post=s["w_post"], gate=s["gate"],
                                           w_pre=s["w_pre"], scale=s["scale"], rstd_post=s["rstd_post"],
                                           rstd_pre=s["rstd_pre"])
        norm = lce.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"], eps=CLIP_EPS)
        return norm, s["out"]
    if op == "attn_fwd":
        return _attention_forward(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["causal"], s["scale"])
    if op == "attn_bwd":
        return _attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu_q"], s["cu_k"], s["causal"],
                                   s["scale"])
    if op == "norm_fwd":
        return _norm_forward(s["x"], s["b"], s["w_post"], s["gate"], s["w_pre"], s["scale"])
    if op == "norm_bwd":
        return _norm_backward(s["dr"], s["dn"], s["r"], s["b"], s["w_post"], s["gate"], s["w_pre"], s["scale"],
                              s["rstd_post"], s["rstd_pre"])
    return _clip(s["grads"], s["max_norm"], s["out"])


# --------------------------------------------- the definitions, in 64 bits

def _exact_attention(case, seed):
    """One sequence and one head at a time, straight from the definition."""
    st = prepare(case, seed)
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    scale, grp = st["scale"], case["heads"] // case["kv_heads"]
    back = case["op"] == "attn_bwd"
    if back:
        do, o_in, lse_in = st["do"].double(), st["o"].double(), st["lse"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    else:
        o = torch.zeros_like(q)
        lse = torch.full((case["heads"], q.shape[0]), -math.inf, dtype=torch.float64, device=DEV)
    a = c = 0
    for lq, lk in zip(_ints(case["lens_q"]), _ints(case["lens_k"])):
        b, e = a + lq, c + lk
        if lq and lk:
            hidden = torch.ones(lq, lk, dtype=torch.bool, device=DEV).triu(lk - lq + 1) if case["causal"] else None
            for h in range(case["heads"]):
                kk, vv = k[c:e, h // grp], v[c:e, h // grp]
                z = scale * (q[a:b, h] @ kk.T)
                if hidden is not None:
                    z.masked_fill_(hidden, -math.inf)
                if back:
                    w = torch.exp(z - lse_in[h, a:b, None])
                    w[z == -math.inf] = 0.0
                    dz = w * (do[a:b, h] @ vv.T - (do[a:b, h] * o_in[a:b, h]).sum(1, keepdim=True))
                    dq[a:b, h] = scale * (dz @ kk)
                    dk[c:e, h // grp] += scale * (dz.T @ q[a:b, h])
                    dv[c:e, h // grp] += w.T @ do[a:b, h]
                else:
                    lse[h, a:b] = torch.logsumexp(z, 1)
                    w = torch.exp(z - lse[h, a:b, None])
                    w[z == -math.inf] = 0.0
                    o[a:b, h] = w @ vv
        a, c = b, e
    return (dq, dk, dv) if back else (o, lse)


def _exact_norm(case, seed):
    """Forward from the definition; backward as autograd's derivative of it with
    the given 1/rms values in the place of the computed ones."""
    s = {n: t.double() if torch.is_tensor(t) else t for n, t in prepare(case, seed).items()}
    one = lambda t: 1.0 if t is None else t  # noqa: E731
    if case["op"] == "norm_fwd":
        rms = lambda t: (t.pow(2).sum(-1) / case["d"] + EPS).pow(-0.5)  # noqa: E731
        post = rms(s["b"]) if case["post"] else None
        y = s["b"] * (post[:, None] * s["w_post"] if case["post"] else 1.0)
        r = s["x"] + case["scale"] * one(s["gate"]) * y
        pre = rms(r) if case["pre"] else None
        return r, r * pre[:, None] * s["w_pre"] if case["pre"] else None, post, pre

    def through(t, w, rstd, grad):
        """Gradients of n = t * rstd(t) * w, where d rstd / dt = -rstd^3 t / d."""
        inner = (grad * w * t).sum(-1, keepdim=True)
        return rstd[:, None] * grad * w - rstd[:, None].pow(3) * t * inner / case["d"], (grad * t * rstd[:, None]).sum(0)

    dx, dw_pre, dw_post, dgate = s["dr"], None, None, None
    if case["pre"]:
        more, dw_pre = through(s["r"], s["w_pre"], s["rstd_pre"], s["dn"])
        dx = dx + more
    dy = case["scale"] * one(s["gate"]) * dx
    if case["gate"] != "none":
        dgate = case["scale"] * dx * s["b"] * (s["rstd_post"][:, None] * s["w_post"] if case["post"] else 1.0)
        dgate = dgate if case["gate"] == "full" else dgate.sum(0)
    db = dy
    if case["post"]:
        db, dw_post = through(s["b"], s["w_post"], s["rstd_post"], dy)
    return dx, db, dw_post, dgate, dw_pre


def exact(case, seed):
    if case["op"].startswith("attn"):
        return _exact_attention(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, seed)
    s = prepare(case, seed)
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(t.double()).pow(2)) for t in s["grads"]))
    c = min(1.0, case["max_norm"] / (norm + CLIP_EPS))
    return torch.tensor(norm, dtype=torch.float64), [t.double() * c for t in s["grads"]]
