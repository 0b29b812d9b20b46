"""The operators of a recurrent block that keeps its activations in 8 bits, as
cases to be timed: the layer norm with the residual sum before it (forward,
backward, and both with the stream kept in 8 bits between them), activations
packed to 8 bits and unpacked, a weight's gradient taken from packed
activations, and the gated recurrence (forward and backward) over packed
sequences and for single tokens.

`run` computes each in elementary torch operations in 32 bits (own = False) or
through this package's entry points (own = True). Sequence lengths are part of
a case (a text of numbers), so that the work of a case is known from it alone."""
import math

import torch

own = False
DEV = "cuda"
EPS = 1e-5            # layer norm epsilon
BLOCK = 128           # channels that share a scale in 8 bits
LOW, HIGH = -100, 119  # exponents of the scales
EVERY = 128           # tokens between the states that a recurrence keeps for its backward pass


# ------------------------------------------------------------------ the cases

def listed():
    documents = "1012,433,761,1290,850,517,64,1103,905,288,969"
    return [
        # one generated token: latency only
        dict(name="layer norm fwd one token", op="ln_fwd", rows=1, d=4096, add=True, bias=True, dtype="bf16"),
        # a training batch at the llama8b width: a block's output added, then the next block's norm
        dict(name="layer norm fwd batch", op="ln_fwd", rows=16384, d=4096, add=True, bias=True, dtype="bf16"),
        # its backward pass, joined with the gradient that passes by on the stream
        dict(name="layer norm bwd batch", op="ln_bwd", rows=16384, d=4096, more=True, bias=True, dtype="bf16"),
        # forward and backward of a norm that keeps its stream in 8 bits, the gpt1b width, an odd number of rows
        dict(name="layer norm kept in 8 bits", op="ln_kept", rows=3482, d=2048, add=True, bias=True, dtype="bf16"),
        # an activation set aside in 8 bits and brought back for the backward pass: an MLP's inner width
        dict(name="activation to 8 bits and back", op="keep", rows=8192, d=8192, dtype="bf16"),
        # a small fp32 model's, rows that end inside a block
        dict(name="activation to 8 bits and back, small fp32", op="keep", rows=613, d=1000, dtype="fp32"),
        # the gradient of an MLP's first matrix from 7373 valid tokens of a llama8b batch (16384 = 4 x 4096)
        dict(name="weight gradient large", op="wgrad", tokens=7373, n=16384, k=4096, dtype="bf16"),
        # a small model's: few tiles, a short and odd number of tokens
        dict(name="weight gradient small", op="wgrad", tokens=1213, n=256, k=200, dtype="bf16"),
        # one step of 16 sequences that are being generated, with their states: latency
        dict(name="recurrence fwd single tokens", op="rec_fwd", lens=",".join(["1"] * 16), tail=0, equal=True, d=4096,
             state=True, dtype="bf16"),
        # documents packed into one 8192-token row, lengths ~ N(850, 300), at the llama8b width
        dict(name="recurrence fwd packed documents", op="rec_fwd", lens=documents, tail=0, equal=False, d=4096, state=False,
             dtype="bf16"),
        # the backward pass of one long document at the same width
        dict(name="recurrence bwd long document", op="rec_bwd", lens="16384", tail=0, equal=False, d=4096, state=False,
             dtype="bf16"),
        # fp32 over ragged rows with states, an empty one among them, and a padded end: the smoke width 128
        dict(name="recurrence bwd ragged fp32", op="rec_bwd", lens="1024,771,1,0,640,333,713", tail=614, equal=False, d=128,
             state=True, dtype="fp32"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ln_fwd", "ln_bwd", "ln_kept", "keep", "wgrad", "wgrad", "rec_fwd", "rec_fwd", "rec_bwd", "rec_bwd"])
    dtype = "bf16" if rng.random() < 0.75 else "fp32"
    if op == "wgrad":
        tokens, n, k = log(1, 16384), 8 * log(1, 2048), 8 * log(1, 1024)
        most = 7373 * 16384 * 4096 // (1 if dtype == "bf16" else 6)
        while tokens * n * k > most:
            tokens, n, k = max(1, tokens // 2), max(8, n // 16 * 8), k
        return dict(op=op, tokens=tokens, n=n, k=k, dtype=dtype)
    if op.startswith("rec"):
        d = 8 * log(1, 512)
        most = 16384 * 4096 // (2 if dtype == "fp32" else 1) // (2 if op == "rec_fwd" else 1)
        total = log(1, min(65536, most // d))
        state = rng.random() < 0.5
        if rng.random() < 0.3:
            length = rng.choice([1, 1, log(1, total)])
            return dict(op=op, lens=",".join([str(length)] * max(1, min(total // length, 512))), tail=0, equal=True, d=d, state=state,
                        dtype=dtype)
        n = min(total, log(1, 40))
        cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return dict(op=op, lens=",".join(map(str, lens)), tail=rng.choice([0, 0, rng.randrange(1, 300)]), equal=False, d=d,
                    state=state, dtype=dtype)
    d = 8 * log(1, 1024)
    most = 16384 * 4096 // (2 if dtype == "fp32" else 1) // (2 if op in ("ln_kept", "keep") else 1)
    case = dict(op=op, rows=log(1, min(32768, most // d)), d=d, dtype=dtype)
    if op.startswith("ln"):
        case["bias"] = rng.random() < 0.7
        if op != "ln_bwd":
            case["add"] = rng.random() < 0.7
        else:
            case["more"] = rng.random() < 0.7
    return case


def _ints(text):
    return [int(x) for x in str(text).split(",") if x != ""]


def _scales(rows, d):
    return rows * ((d + BLOCK - 1) // BLOCK)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "wgrad":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": t * n * es + t * k + _scales(t, k) + n * k * es, "flops": 2 * t * n * k}
    if op.startswith("rec"):
        lens = _ints(case["lens"])
        tokens, d = sum(lens) + case["tail"], case["d"]
        states = len(lens) * d * 4
        if op == "rec_fwd":
            return {"bytes": 3 * tokens * d * es + states * (2 if case["state"] else 1), "flops": 8 * tokens * d}
        return {"bytes": 5 * tokens * d * es + states * (3 if case["state"] else 1), "flops": 16 * tokens * d}
    rows, d = case["rows"], case["d"]
    nd = rows * d
    if op == "keep":
        return {"bytes": 2 * (nd * es + nd + _scales(rows, d)), "flops": 4 * nd}
    vectors = d * es * (2 if case["bias"] else 1)
    if op == "ln_fwd":
        return {"bytes": nd * es * (4 if case["add"] else 2) + 8 * rows + vectors, "flops": 9 * nd}
    if op == "ln_bwd":
        return {"bytes": nd * es * (4 if case["more"] else 3) + 8 * rows + 2 * vectors, "flops": 14 * nd}
    # forward (writing 8 bits as well) and backward from them
    return {"bytes": nd * es * ((4 if case["add"] else 2) + 3) + 2 * (nd + _scales(rows, d)) + 16 * rows + 3 * vectors,
            "flops": 26 * nd}


# ----------------------------------------------------------------- the inputs

def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _activations(g, rows, d):
    """Values as they come out of a layer: some channels much larger than others, one in ten exactly zero."""
    size = torch.exp(torch.randn(d, generator=g, device=DEV))
    x = torch.randn(rows, d, generator=g, device=DEV) * size
    return x * (torch.rand(rows, d, generator=g, device=DEV) > 0.1)


def _pack_plain(x):
    """(codes, exponents): e4m3 values as their bytes, and one exponent for each block of a row's channels."""
    rows, d = x.shape
    blocks = (d + BLOCK - 1) // BLOCK
    y = torch.zeros(rows, blocks * BLOCK, device=x.device)
    y[:, :d] = x.float()
    y = y.view(rows, blocks, BLOCK)
    m, p = torch.frexp(y.abs().amax(-1))          # m in [0.5, 1): 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, p - 9, p - 8)
    e = torch.where(m == 0, torch.full_like(e, LOW), e.clamp(LOW, HIGH))
    y = torch.ldexp(y, -e[..., None]).clamp(-448.0, 448.0)
    codes = y.to(torch.float8_e4m3fn).view(torch.uint8).view(rows, blocks * BLOCK)[:, :d]
    return codes, e.to(torch.int8)


def _unpack_plain(codes, exponents):
    """The values that the codes stand for, in 32 bits."""
    rows, d = codes.shape
    value = codes.contiguous().view(torch.float8_e4m3fn).float()
    e = exponents.int().repeat_interleave(BLOCK, 1)[:, :d]
    return torch.ldexp(value, e)


def _layout(case):
    """(offsets of the sequences, for every token: its sequence or -1, whether it is the sequence's first, its last)."""
    lens = _ints(case["lens"])
    ends = torch.tensor(lens, dtype=torch.int64).cumsum(0)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), ends])
    total = int(cu[-1])
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens, dtype=torch.int64))
    at = torch.arange(total)
    first, last = at == cu[seq], at == cu[seq + 1] - 1
    seq = torch.cat([seq, torch.full((case["tail"],), -1, dtype=torch.int64)])
    no = torch.zeros(case["tail"], dtype=torch.bool)
    return cu.to(torch.int32).to(DEV), seq.to(DEV), torch.cat([first, no]).to(DEV), torch.cat([last, no]).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, op = _dt(case), case["op"]

    def rand(*shape, mean=0.0, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dt)

    s = {"op": op, "dtype": dt}
    if op == "wgrad":
        s["dy"] = rand(case["tokens"], case["n"], std=0.02)
        x = _activations(g, case["tokens"], case["k"]).to(dt)
        s["codes"], s["exponents"] = _pack_plain(x)
        if own:
            import chunked_vocab_cross_gb300 as lce
            s["kept"] = lce.pack_activation(x)          # what the forward pass left
    elif op.startswith("rec"):
        cu, s["seq"], s["first"], s["last"] = _layout(case)
        lens, d = _ints(case["lens"]), case["d"]
        tokens = sum(lens) + case["tail"]
        # both are slices of one projection's output; the gates mostly remember
        xg = torch.cat([rand(tokens, d), rand(tokens, d, mean=2.0, std=1.5)], 1)
        x, gate = xg[:, :d], xg[:, d:]
        s["cu"] = None if case["equal"] else cu
        s["shape"] = (len(lens), lens[0], d) if case["equal"] else (tokens, d)
        s["x"], s["g"] = x.unflatten(0, s["shape"][:-1]), gate.unflatten(0, s["shape"][:-1])
        s["state"] = torch.randn(len(lens), d, generator=g, device=DEV) if case["state"] else None
        s["sequences"] = len(lens)
        if op == "rec_bwd":
            s["dh"] = rand(tokens, d).unflatten(0, s["shape"][:-1])
            s["dfinal"] = torch.randn(len(lens), d, generator=g, device=DEV) if case["state"] else None
            # what the forward pass left: the state before every 128th token, in 32 bits
            h, _, _ = _recurrence(s)
            kept = torch.zeros((tokens + EVERY - 1) // EVERY, d, device=DEV)
            if tokens > EVERY:
                kept[1:] = h[EVERY - 1:-1:EVERY][:kept.shape[0] - 1]
            s["kept"] = kept
    elif op == "keep":
        s["x"] = _activations(g, case["rows"], case["d"]).to(dt)
    else:
        rows, d = case["rows"], case["d"]
        s["w"] = rand(d, mean=1.0, std=0.1)
        s["c"] = rand(d, std=0.1) if case["bias"] else None
        s["x"] = rand(rows, d, mean=0.5, std=2.0)
        s["b"] = rand(rows, d) if case.get("add") else None
        if op != "ln_fwd":
            s["dn"] = rand(rows, d)
            s["dr"] = rand(rows, d) if case.get("more", True) else None
        if op == "ln_bwd":
            # what the forward pass left: the stream and its rows' statistics
            s["r"] = s.pop("x")
            s["mean"], s["rstd"] = _statistics(s["r"].float())
    return s


# ------------------------------------------------------------- the plain forms

def _statistics(r):
    mean = r.mean(1)
    rstd = ((r - mean[:, None]).square().mean(1) + EPS).rsqrt()
    return mean, rstd


def _ln_forward(s):
    r = s["x"] if s["b"] is None else (s["x"].float() + s["b"].float()).to(s["dtype"])
    mean, rstd = _statistics(r.float())
    n = (r.float() - mean[:, None]) * rstd[:, None] * s["w"].float()
    if s["c"] is not None:
        n = n + s["c"].float()
    return r, n.to(s["dtype"]), mean, rstd


def _ln_backward(s, r, mean, rstd):
    dt = s["dtype"]
    hat = (r - mean[:, None]) * rstd[:, None]
    dn = s["dn"].float()
    u = dn * s["w"].float()
    dx = rstd[:, None] * (u - u.mean(1, keepdim=True) - hat * (u * hat).mean(1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    return dx.to(dt), (dn * hat).sum(0).to(dt), dn.sum(0).to(dt) if s["c"] is not None else None


def _scan(a, v):
    """h_t = a_t h_{t-1} + v_t, by doubling the distance that has been covered."""
    step = 1
    while step < a.shape[0]:
        v = torch.cat([v[:step], v[step:] + a[step:] * v[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return v


def _recurrence(s):
    """(h, the state before each token, gates) in 32 bits."""
    x, g = s["x"].flatten(0, -2).float(), s["g"].flatten(0, -2).float()
    seq, first = s["seq"], s["first"]
    live = (seq >= 0)[:, None]
    a = torch.where(live, torch.sigmoid(g), 0.0)
    v = torch.where(live, torch.sigmoid(-g) * x, 0.0)
    begin = torch.zeros_like(x)
    if s["state"] is not None:
        begin = torch.where(first[:, None], s["state"][seq.clamp(min=0)], 0.0)
    h = _scan(torch.where(first[:, None], 0.0, a), v + a * begin)
    before = torch.where(first[:, None], begin, torch.cat([torch.zeros_like(h[:1]), h[:-1]]))
    return h, before, a


def _rec_forward(s):
    h, _, _ = _recurrence(s)
    final = torch.zeros(s["sequences"], h.shape[1], device=DEV) if s["state"] is None else s["state"].clone()
    final[s["seq"][s["last"]]] = h[s["last"]]
    return h.to(s["dtype"]).view(s["shape"]), final


def _rec_backward(s):
    dt = s["dtype"]
    _, before, a = _recurrence(s)
    x, g, dh = (s[k].flatten(0, -2).float() for k in ("x", "g", "dh"))
    seq, first, last = s["seq"], s["first"], s["last"]
    if s["dfinal"] is not None:
        dh = dh + torch.where(last[:, None], s["dfinal"][seq.clamp(min=0)], 0.0)
    live = (seq >= 0)[:, None]
    dh = torch.where(live, dh, 0.0)
    m = _scan(torch.where(last[:, None], 0.0, a).flip(0), (a * dh).flip(0)).flip(0)
    grad = dh + torch.where(last[:, None], 0.0, torch.cat([m[1:], torch.zeros_like(m[:1])]))
    rest = torch.sigmoid(-g)
    dx = torch.where(live, rest * grad, 0.0)
    dg = torch.where(live, grad * (before - x) * a * rest, 0.0)
    dstate = None
    if s["state"] is not None:
        dstate = s["dfinal"].clone()
        dstate[seq[first]] = m[first]
    return dx.to(dt).view(s["shape"]), dg.to(dt).view(s["shape"]), dstate


def _run_plain(s):
    op, dt = s["op"], s["dtype"]
    if op == "ln_fwd":
        return _ln_forward(s)
    if op == "ln_bwd":
        return _ln_backward(s, s["r"].float(), s["mean"], s["rstd"])
    if op == "ln_kept":
        r, n, mean, rstd = _ln_forward(s)
        return (r, n) + _ln_backward(s, _unpack_plain(*_pack_plain(r)), mean, rstd)
    if op == "keep":
        return _unpack_plain(*_pack_plain(s["x"])).to(dt)
    if op == "wgrad":
        return torch.matmul(s["dy"].float().t(), _unpack_plain(s["codes"], s["exponents"])).to(dt)
    return _rec_forward(s) if op == "rec_fwd" else _rec_backward(s)


def _run_own(s):
    import chunked_vocab_cross_gb300 as lce
    op = s["op"]
    if op == "ln_fwd":
        return lce.layer_norm_forward(s["x"], s["b"], weight=s["w"], bias=s["c"], eps=EPS)[:4]
    if op == "ln_bwd":
        return lce.layer_norm_backward(s["dr"], s["dn"], s["r"], weight=s["w"], mean=s["mean"], rstd=s["rstd"],
                                       bias=s["c"] is not None)
    if op == "ln_kept":
        r, n, mean, rstd, kept = lce.layer_norm_forward(s["x"], s["b"], weight=s["w"], bias=s["c"], eps=EPS, keep8=True)
        return (r, n) + lce.layer_norm_backward(s["dr"], s["dn"], kept, weight=s["w"], mean=mean, rstd=rstd,
                                                bias=s["c"] is not None)
    if op == "keep":
        return lce.unpack_activation(lce.pack_activation(s["x"]))
    if op == "wgrad":
        return lce.packed_weight_grad(s["dy"], s["kept"])
    if op == "rec_fwd":
        return lce.gated_recurrence_forward(s["x"], s["g"], s["cu"], state=s["state"])[:2]
    return lce.gated_recurrence_backward(s["dh"], s["x"], s["g"], s["kept"], s["cu"], state=s["state"], dfinal=s["dfinal"])


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ------------------------------------------------------------ the exact values

def _nearest(x):
    """Every value of x (fp64, [rows, d]) as its 8-bit form stands for it: the nearest value of 4 significant bits
    (ties to even) at its block's scale."""
    rows, d = x.shape
    out = torch.zeros_like(x)
    for lo in range(0, d, BLOCK):
        y = x[:, lo:lo + BLOCK]
        top = y.abs().amax(1, keepdim=True)
        e = torch.full_like(top, float(LOW))
        some = top > 0
        e[some] = torch.ceil(torch.log2(top[some] / 448.0)).clamp(LOW, HIGH)
        e = torch.where(some & (top > 448.0 * torch.exp2(e)) & (e < HIGH), e + 1, e)
        e = torch.where(some & (top <= 448.0 * torch.exp2(e - 1)) & (e > LOW), e - 1, e)
        z = (y * torch.exp2(-e)).clamp(-448.0, 448.0)
        size = torch.where(z == 0, torch.ones_like(z), z.abs())
        place = torch.floor(torch.log2(size))
        place = torch.where(torch.exp2(place) > size, place - 1, place)
        place = torch.where(torch.exp2(place + 1) <= size, place + 1, place)
        unit = torch.exp2(place.clamp(min=-6.0) - 3.0)
        out[:, lo:lo + BLOCK] = torch.round(z / unit) * unit * torch.exp2(e)
    return out


def _exact_ln(case, s):
    d64 = lambda t: None if t is None else t.double()  # noqa: E731
    w, c = d64(s["w"]), d64(s["c"])
    outs = ()
    if case["op"] == "ln_bwd":
        used, mean, rstd = s["r"].double(), s["mean"].double(), s["rstd"].double()
    else:
        total = s["x"].double() if s["b"] is None else s["x"].double() + s["b"].double()
        used = total.to(s["dtype"]).double()
        mean = used.sum(1) / case["d"]
        centred = used - mean[:, None]
        rstd = 1.0 / torch.sqrt((centred * centred).sum(1) / case["d"] + EPS)
        n = centred * rstd[:, None] * w
        n = n if c is None else n + c
        if case["op"] == "ln_fwd":
            return total, n, mean, rstd
        outs, used = (total, n), _nearest(used)
    xhat = (used - mean[:, None]) * rstd[:, None]
    dn = s["dn"].double()
    u = dn * w
    inner = u - (u.sum(1, keepdim=True) + xhat * (u * xhat).sum(1, keepdim=True)) / case["d"]
    dx = inner * rstd[:, None]
    dx = dx if s["dr"] is None else dx + s["dr"].double()
    return outs + (dx, (dn * xhat).sum(0), None if c is None else dn.sum(0))


def _exact_recurrence(case, s):
    x, g = s["x"].flatten(0, -2).double(), s["g"].flatten(0, -2).double()
    lens, d = _ints(case["lens"]), case["d"]
    a = 1.0 / (1.0 + torch.exp(-g))
    rest = torch.exp(-g) / (1.0 + torch.exp(-g))
    v = rest * x
    h = torch.zeros_like(x)
    zero = torch.zeros(d, dtype=torch.float64, device=DEV)
    begin = [zero if s["state"] is None else s["state"][i].double() for i in range(len(lens))]
    before = torch.zeros_like(x)
    final, at = [], 0
    for i, n in enumerate(lens):
        last = begin[i]
        for t in range(at, at + n):
            last = torch.addcmul(v[t], a[t], last, out=h[t])
        if n:
            before[at] = begin[i]
            before[at + 1:at + n] = h[at:at + n - 1]
        final.append(last.clone())
        at += n
    if case["op"] == "rec_fwd":
        return h.view(s["shape"]), torch.stack(final)
    dh = s["dh"].flatten(0, -2).double()
    grad = torch.zeros_like(x)
    dstate, at = [], 0
    for i, n in enumerate(lens):
        carry = zero if s["dfinal"] is None else s["dfinal"][i].double()
        for t in range(at + n - 1, at - 1, -1):
            torch.add(dh[t], carry, out=grad[t])
            carry = a[t] * grad[t]
        dstate.append(carry)
        at += n
    dx, dg = grad * rest, grad * (before - x) * a * rest
    dg[at:] = 0.0
    return dx.view(s["shape"]), dg.view(s["shape"]), None if s["state"] is None else torch.stack(dstate)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("ln"):
        return _exact_ln(case, s)
    if case["op"].startswith("rec"):
        return _exact_recurrence(case, s)
    if case["op"] == "keep":
        return _nearest(s["x"].double())
    value = s["codes"].contiguous().view(torch.float8_e4m3fn).double()
    scale = torch.exp2(s["exponents"].double()).repeat_interleave(BLOCK, 1)[:, :case["k"]]
    return s["dy"].double().t() @ (value * scale)
