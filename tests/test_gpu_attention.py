"""Attention over packed sequences and its backward pass, through the public
entry points, against the fp64 reference.

Tolerances, elementwise, from the arithmetic (u = 2^-8 is bf16's unit
roundoff, e = 2^-24 fp32's):
  forward   |err| <= u (|o| + sum p|v|) + F sum p|v|
  gradients |err| <= u (|g| + terms) + F parts
where `terms` are the absolute terms the rounded operands (p, ds) enter with,
`parts` what fp32 errors of ds enter with, and
  F = 4 e (D + keys + queries*group) (1 + E),  E = max |exponent| terms,
bounds the accumulated fp32 roundings: of a score (D terms), of its exponent
(relative to its size E) and of the sums over keys or queries. fp32 inputs
have u = e. Below the types' normal range nothing holds relatively: a
probability under 2^-126 may be lost, so every bound adds TINY = 2^-126 *
(keys + queries*group) * max |operand|^3 (ds is a product of two operands, and
its partner one more)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402
from oracle import block_oracle as bo  # noqa: E402

pytestmark = pytest.mark.gpu
EPS32 = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    lce.device_status()
    yield


def f64(t):
    return t.detach().double().cpu().numpy()


def cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def make(lq, lk, H, Hk, D, dtype, seed=0, tail=0, mult=1.0):
    """q, k, v as slices of one buffer (self-attention lengths) or of two."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * mult).to(DT[dtype])  # noqa: E731
    if list(lq) == list(lk):
        x = r(sum(lq) + tail, H + 2 * Hk, D)
        q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    else:
        q, kv = r(sum(lq) + tail, H, D), r(sum(lk) + tail, 2 * Hk, D)
        k, v = kv[:, :Hk], kv[:, Hk:]
    return q, k, v, r(sum(lq) + tail, H, D)


def check(lq, lk, H, Hk, D, causal, dtype, tail=0, seed=0, scale=None, mult=1.0):
    q, k, v, do = make(lq, lk, H, Hk, D, dtype, seed, tail, mult)
    scale = D ** -0.5 if scale is None else scale
    cq, ck = cu(lq), cu(lk)
    o, lse = lce.attention_forward(q, k, v, cq, ck, causal=causal, scale=scale)
    grads = lce.attention_backward(do, q, k, v, o, lse, cq, ck, causal=causal, scale=scale)
    torch.cuda.synchronize()
    assert lce.device_status() == 0
    ro, rl, abs_o, E = bo.attention_forward(f64(q), f64(k), f64(v), lq, lk, causal, scale)
    u = 2.0 ** -8 if dtype == "bf16" else EPS32
    F = 4 * EPS32 * (D + max(lk) + max(lq) * (H // Hk)) * (1 + E)
    got = f64(lse)
    assert np.array_equal(np.isinf(got), np.isinf(rl)) and np.all(got[np.isinf(rl)] == -np.inf)
    fin = np.isfinite(rl)
    assert np.all(np.abs(got[fin] - rl[fin]) <= F + EPS32 * 4 * np.abs(rl[fin]))
    biggest = max([1.0] + [float(t.float().abs().max()) for t in (q, k, v, do) if t.numel()])
    tiny = 2.0 ** -126 * (max(lk) + max(lq) * (H // Hk)) * biggest ** 3
    err = np.abs(f64(o) - ro)
    assert np.all(err <= u * (np.abs(ro) + abs_o) + F * abs_o + tiny), (err.max(), "o")
    ref = bo.attention_backward(f64(do), f64(q), f64(k), f64(v), f64(o), f64(lse), lq, lk, causal, scale)
    for name, t in zip(("dq", "dk", "dv"), grads):
        want, terms, parts = ref[name]
        err, tol = np.abs(f64(t) - want), u * (np.abs(want) + terms) + F * parts + tiny
        assert np.all(err <= tol), (name, err.max(), float((err - tol).max()))
    return q, k, v, do, o, lse, grads


LENS = {
    "one": ([1], [1]), "two": ([2], [2]), "tile": ([128], [128]), "over": ([129], [129]), "under": ([127], [127]),
    "64": ([64], [64]), "ragged": ([300, 1, 0, 77, 200], [300, 1, 0, 77, 200]), "long": ([700], [700]),
    "many": ([3] * 40 + [17, 0, 0, 130], [3] * 40 + [17, 0, 0, 130]),
    "cross": ([130, 5, 0, 64, 257], [300, 0, 40, 63, 1]), "prefix": ([33, 150], [290, 150 + 128]),
    "more queries": ([300, 140], [100, 1]), "one query": ([1, 1, 1], [1000, 129, 1]),
}


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("lens", list(LENS), ids=lambda s: s.replace(" ", "_"))
@pytest.mark.parametrize("D", [64, 128])
def test_bf16_lengths(lens, causal, D):
    lq, lk = LENS[lens]
    check(lq, lk, 4, 2, D, causal, "bf16", tail=0 if lens == "one" else 3)


def longer(lens):
    """Tokens after the last sequence that make the call one of long rows, whose P and dS go in as one bf16 operand."""
    return 513 * len(lens)


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("lens", list(LENS), ids=lambda s: s.replace(" ", "_"))
@pytest.mark.parametrize("D", [64, 128])
def test_bf16_lengths_one_part(lens, causal, D):
    lq, lk = LENS[lens]
    check(lq, lk, 4, 2, D, causal, "bf16", tail=longer(lq), seed=1)


@pytest.mark.parametrize("D", [8, 24, 72, 80, 96, 104])
def test_bf16_head_sizes_one_part(D):
    check([150, 40], [150, 40], 2, 1, D, True, "bf16", tail=longer([150, 40]), seed=D)


@pytest.mark.parametrize("heads", [(1, 1), (7, 1), (6, 3), (8, 8), (12, 4)], ids=lambda h: f"{h[0]}_{h[1]}")
def test_bf16_head_layouts_one_part(heads):
    check([200, 57], [200, 57], *heads, 64, True, "bf16", tail=longer([200, 57]), seed=2)
    check([200, 57], [90, 157], *heads, 128, False, "bf16", tail=longer([200, 57]), seed=3)


@pytest.mark.parametrize("heads,D", [((4, 1), 128), ((1, 1), 64), ((6, 2), 80)], ids=lambda h: f"{h[0]}_{h[1]}" if isinstance(h, tuple) else str(h))
@pytest.mark.parametrize("lens", [([1], [3000]), ([130], [2600]), ([1, 0, 3], [2500, 700, 3000]), ([1500], [1500]), ([40, 200], [2300, 90])],
                         ids=lambda n: f"{n[0]}_{n[1]}".replace(" ", ""))
def test_few_rows_over_long_keys(lens, heads, D):
    """Rows whose keys are taken in ranges: the last range ragged, empty for
    short sequences, or beyond what a causal row sees; rows without keys, and
    tokens after the last sequence."""
    lq, lk = lens
    for causal in (True, False):
        q, k, v, do, o, lse, _ = check(lq, lk, *heads, D, causal, "bf16", tail=3, seed=D)
        o2, lse2 = lce.attention_forward(q, k, v, cu(lq), cu(lk), causal=causal)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        need = lce.attention_forward_workspace_size(q.shape[0], k.shape[0], *heads, D, len(lq), causal=causal)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            o3, _ = lce.attention_forward(q, k, v, cu(lq), cu(lk), causal=causal, workspace=ws)
            assert torch.equal(o, o3)
            with pytest.raises(lce.LceError):
                lce.attention_forward(q, k, v, cu(lq), cu(lk), causal=causal, workspace=ws[:need - 1])
        assert bool((o[sum(lq):] == 0).all()) and bool((lse[:, sum(lq):] == -float("inf")).all())


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("heads,D", [((14, 2), 96), ((16, 1), 64), ((6, 1), 128), ((8, 2), 80), ((28, 4), 8)],
                         ids=lambda h: f"{h[0]}_{h[1]}" if isinstance(h, tuple) else str(h))
def test_key_heads_whose_query_heads_are_shared_out(heads, D, causal):
    """Few key tiles with many query heads each: dK and dV come as sums of
    shares. Sequences without queries or keys, and tokens after the last."""
    for lq, lk, tail in (([700], [700], 0), ([300, 0, 129, 1], [200, 77, 0, 300], 5), ([513, 200], [513, 200], 2100)):
        q, k, v, do, o, lse, grads = check(lq, lk, *heads, D, causal, "bf16", tail=tail, seed=D)
        again = lce.attention_backward(do, q, k, v, o, lse, cu(lq), cu(lk), causal=causal)
        assert all(torch.equal(x, y) for x, y in zip(grads, again))
        if lq == lk:
            dx = torch.zeros(q.shape[0], heads[0] + 2 * heads[1], D, device="cuda", dtype=torch.bfloat16)
            outs = dx.split((heads[0], heads[1], heads[1]), dim=1)
            lce.attention_backward(do, q, k, v, o, lse, cu(lq), cu(lk), causal=causal, dq=outs[0], dk=outs[1], dv=outs[2])
            assert all(torch.equal(x, y) for x, y in zip(grads, outs))
        assert all(bool((t[sum(n):] == 0).all()) for t, n in zip(grads, (lq, lk, lk)))


@pytest.mark.parametrize("heads,D", [((8, 8), 64), ((4, 1), 128)], ids=["8x64", "4of1x128"])
def test_small_calls_lose_little_more_than_the_rounding_of_the_result(heads, D):
    """Rounding values of any size to bf16 costs 2^-8 / sqrt(3) * sqrt(mean
    1/m^2) = 0.00166 of their norm for significands m spread evenly over their
    logarithm; a second rounding, of P or dS, would make it 0.00235. Small
    calls keep the first: 0.0020 leaves a fifth for the sizes that come up."""
    lens = [256]
    q, k, v, do = make(lens, lens, *heads, D, "bf16", seed=11)
    o, lse = lce.attention_forward(q, k, v)
    grads = lce.attention_backward(do, q, k, v, o, lse)
    want = [bo.attention_forward(f64(q), f64(k), f64(v), lens, lens, True, D ** -0.5)[0]]
    ref = bo.attention_backward(f64(do), f64(q), f64(k), f64(v), f64(o), f64(lse), lens, lens, True, D ** -0.5)
    want += [ref[n][0] for n in ("dq", "dk", "dv")]
    for t, w in zip((o, *grads), want):
        assert np.linalg.norm(f64(t) - w) <= 0.0020 * np.linalg.norm(w)


@pytest.mark.parametrize("D", [8, 16, 24, 40, 56, 72, 80, 96, 104, 120])
def test_bf16_head_sizes(D):
    check([150, 40], [150, 40], 2, 1, D, True, "bf16", seed=D)


@pytest.mark.parametrize("heads", [(1, 1), (7, 1), (6, 3), (8, 8), (12, 4)], ids=lambda h: f"{h[0]}_{h[1]}")
def test_bf16_head_layouts(heads):
    check([200, 57], [200, 57], *heads, 64, True, "bf16", seed=2)
    check([200, 57], [90, 157], *heads, 128, False, "bf16", seed=3)


@pytest.mark.parametrize("lens", ["one", "over", "ragged", "cross", "more queries"], ids=lambda s: s.replace(" ", "_"))
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("D", [8, 32, 72, 128])
def test_fp32(lens, causal, D):
    lq, lk = LENS[lens]
    check(lq, lk, 4, 2, D, causal, "fp32", tail=2, seed=D)


@pytest.mark.parametrize("mult,scale", [(6.0, None), (1.0, 3.0), (1.0, -0.2), (1.0, 0.0), (0.01, 1.0)])
def test_score_ranges(mult, scale):
    """Peaked rows (a maximum that grows by hundreds along the keys), flat rows, a negative scale."""
    check([260, 140], [260, 140], 2, 2, 64, True, "bf16", seed=5, mult=mult, scale=scale)
    check([150], [400], 2, 1, 128, False, "bf16", seed=6, mult=mult, scale=scale)


def test_growing_maximum():
    """Scores that rise by more than any fixed margin from tile to tile, and fall."""
    T, D = 1024, 64
    for sign in (1.0, -1.0):
        q = torch.ones(T, 1, D, device="cuda", dtype=torch.bfloat16)
        ramp = sign * torch.arange(T, device="cuda").float()[:, None, None] * 0.05
        k = (ramp + torch.randn(T, 1, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 0.1).bfloat16()
        v = torch.randn(T, 1, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).bfloat16()
        o, lse = lce.attention_forward(q, k, v, causal=False, scale=1.0)
        ro, rl, abs_o, E = bo.attention_forward(f64(q), f64(k), f64(v), [T], [T], False, 1.0)
        F = 4 * EPS32 * (D + T) * (1 + E)
        assert np.all(np.abs(f64(lse) - rl) <= F * 1.0 + 4 * EPS32 * np.abs(rl))
        assert np.all(np.abs(f64(o) - ro) <= 2.0 ** -8 * (np.abs(ro) + abs_o) + F * abs_o)


@pytest.mark.parametrize("heads", [4, 16])
def test_sequences_do_not_reach_each_other(heads):
    """NaN and infinities in one sequence and in the tokens after the last: the
    others' results are those without them, bit for bit."""
    for dtype in ("bf16", "fp32"):
        lens = [100, 60, 131, 9]
        q, k, v, do = make(lens, lens, heads, 2, 64, dtype, tail=20)
        run = lambda: lce.attention_forward(q, k, v, cu(lens))  # noqa: E731
        o, lse = run()
        grads = lce.attention_backward(do, q, k, v, o, lse, cu(lens))
        bad = list(range(100, 160)) + list(range(300, 320))
        good = [i for i in range(320) if i not in bad]
        for t, val in ((q, np.nan), (k, np.inf), (v, np.nan), (do, -np.inf)):
            t[bad] = val
        o2, lse2 = run()
        for t in (o2, o):
            t[bad] = float("nan") if t is o2 else t[bad]
        lse2[:, bad] = float("nan")
        lse2[:, 300:] = -float("inf")
        grads2 = lce.attention_backward(do, q, k, v, o2, lse2, cu(lens))
        torch.cuda.synchronize()
        assert torch.equal(o2[good], o[good]) and torch.equal(lse2[:, good], lse[:, good])
        for x, y in zip(grads2, grads):
            assert torch.equal(x[good], y[good])
            assert bool((x[300:] == 0).all())
        lce.device_status()


@pytest.mark.parametrize("heads", [2, 24])
def test_masked_keys_that_are_not_finite_do_not_change_earlier_scores(heads):
    """Causal: a key of NaN or infinity beyond a row's reach leaves the row's lse as it is."""
    q, k, v, _ = make([200], [200], heads, 2, 64, "bf16")
    _, lse = lce.attention_forward(q, k, v)
    k[150:] = float("nan")
    _, lse2 = lce.attention_forward(q, k, v)
    assert torch.equal(lse2[:, :150], lse[:, :150])
    assert bool(lse2[:, 150:].isnan().all())


def test_deterministic_and_on_another_stream():
    lens = [513, 200]
    q, k, v, do = make(lens, lens, 8, 2, 128, "bf16")
    first = None
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, None, s):
        o, lse = lce.attention_forward(q, k, v, cu(lens), stream=stream)
        torch.cuda.synchronize()
        out = (o, lse) + lce.attention_backward(do, q, k, v, o, lse, cu(lens), stream=stream)
        torch.cuda.synchronize()
        if first is None:
            first = out
        assert all(torch.equal(x, y) for x, y in zip(out, first))


def test_batched_tensors_and_given_outputs():
    """[B, L, heads, D] tensors are B sequences of L tokens; gradients into slices of one buffer."""
    B, L, H, Hk, D = 3, 70, 4, 2, 64
    x = torch.randn(B, L, H + 2 * Hk, D, device="cuda").bfloat16()
    q, k, v = x[:, :, :H], x[:, :, H:H + Hk], x[:, :, H + Hk:]
    do = torch.randn(B, L, H, D, device="cuda").bfloat16()
    dx = torch.full((B, L, H + 2 * Hk + 1, D), 7.0, device="cuda", dtype=torch.bfloat16)
    o, lse = lce.attention_forward(q, k, v)
    lce.attention_backward(do, q, k, v, o, lse, dq=dx[:, :, :H], dk=dx[:, :, H:H + Hk], dv=dx[:, :, H + Hk:-1])
    flat = lambda t: t.reshape(B * L, *t.shape[2:])  # noqa: E731
    o3, lse3 = lce.attention_forward(flat(q), flat(k), flat(v), cu([L] * B))
    g3 = lce.attention_backward(flat(do), flat(q), flat(k), flat(v), o3, lse3, cu([L] * B))
    assert torch.equal(flat(o), o3) and torch.equal(lse, lse3)
    for x3, got in zip(g3, (dx[:, :, :H], dx[:, :, H:H + Hk], dx[:, :, H + Hk:-1])):
        assert torch.equal(flat(got), x3)
    assert bool((dx[:, :, -1] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_empty_sides(dtype):
    for lq, lk in (([0], [5]), ([5], [0]), ([0], [0])):
        q, k, v, do = make(lq, lk, 2, 1, 64, dtype)
        o, lse = lce.attention_forward(q, k, v, cu(lq), cu(lk))
        dq, dk, dv = lce.attention_backward(do, q, k, v, o, lse, cu(lq), cu(lk))
        torch.cuda.synchronize()
        assert bool((lse == -float("inf")).all())
        assert all(bool((t == 0).all()) for t in (o, dq, dk, dv))
    assert lce.device_status() == 0


def test_offsets_past_32_bits():
    """Token strides that take element offsets past 2^31."""
    T, wide = 300, 8 * 1024 * 1024
    buf = torch.empty(T, wide, device="cuda", dtype=torch.bfloat16)
    small = torch.randn(T, 3, 64, device="cuda").bfloat16()
    x = buf[:, wide - 192:].unflatten(1, (3, 64))
    x.copy_(small)
    q, k, v = x[:, :1], x[:, 1:2], x[:, 2:]
    do = torch.randn(T, 1, 64, device="cuda").bfloat16()
    o, lse = lce.attention_forward(q, k, v)
    dx = buf[:, :192].unflatten(1, (3, 64))
    lce.attention_backward(do, q, k, v, o, lse, dq=dx[:, :1], dk=dx[:, 1:2], dv=dx[:, 2:])
    a, b, c = small[:, :1], small[:, 1:2], small[:, 2:]
    o2, lse2 = lce.attention_forward(a, b, c)
    g2 = lce.attention_backward(do, a, b, c, o2, lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(dx[:, i:i + 1], g) for i, g in enumerate(g2))


def test_many_sequences_of_one_token():
    """More sequences than one round of the search covers."""
    n = 3000
    lens = [1, 0, 2] * (n // 3)
    q, k, v, do = make(lens, lens, 1, 1, 64, "bf16")
    o, lse = lce.attention_forward(q, k, v, cu(lens))
    ro, rl, abs_o, _ = bo.attention_forward(f64(q), f64(k), f64(v), lens, lens, True, 0.125)
    assert np.all(np.abs(f64(o) - ro) <= 2.0 ** -7 * (abs_o + 1e-30))
    dq, dk, dv = lce.attention_backward(do, q, k, v, o, lse, cu(lens))
    ref = bo.attention_backward(f64(do), f64(q), f64(k), f64(v), f64(o), f64(lse), lens, lens, True, 0.125)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        want, terms, parts = ref[name]
        assert np.all(np.abs(f64(t) - want) <= 2.0 ** -8 * (np.abs(want) + terms) + 2.0 ** -12 * parts), name


def test_invalid_offsets_are_reported():
    q, k, v, do = make([100], [100], 2, 2, 64, "bf16")
    for bad in ([0, 60, 40, 100], [0, 50, 100, 101], [1, 20, 30, 100], [0, -5, 30, 100]):
        c = torch.tensor(bad, dtype=torch.int32, device="cuda")
        lce.device_status()
        lce.attention_forward(q, k, v, c)
        assert lce.device_status() == 4, bad
        o, lse = torch.zeros_like(q), torch.zeros(2, 100, device="cuda")
        lce.attention_backward(do, q, k, v, o, lse, c)
        assert lce.device_status() == 4, bad


def test_autograd_and_differences():
    """The gradient of a smooth function of o against central differences of
    the fp32 forward: the step h = 2^-6 leaves a truncation error of order
    h^2 and a rounding error of order 2^-24 |f| / h, both below 1e-3 |g|."""
    lens = [40, 23]
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, w = (torch.randn(63, 2, 32, generator=g, device="cuda") for _ in range(4))
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    (lce.attention(*leaves, cu(lens)) * w).sum().backward()
    f = lambda *t: (lce.attention_forward(*t, cu(lens))[0].double() * w.double()).sum().item()  # noqa: E731
    for i, leaf in enumerate(leaves):
        z = torch.randn(q.shape, generator=g, device="cuda")
        hi, lo = [q, k, v], [q, k, v]
        hi[i], lo[i] = hi[i] + z * 2.0 ** -6, lo[i] - z * 2.0 ** -6
        want = (leaf.grad.double() * z.double()).sum().item()
        size = float(leaf.grad.norm()) * 1.0
        assert abs((f(*hi) - f(*lo)) * 2.0 ** 5 - want) <= 2e-2 * size


@pytest.mark.parametrize("D", [64, 128])
def test_many_passes_back_to_back(D):
    """Hand-overs between warps under load: no wait gives up, and every pass
    gives the same bits."""
    lens = [700, 300, 1000, 48]
    q, k, v, do = make(lens, lens, 8, 4, D, "bf16", tail=30)
    c = cu(lens)
    lce.device_status()
    want = None
    for _ in range(150):
        o, lse = lce.attention_forward(q, k, v, c)
        got = (o, lse) + lce.attention_backward(do, q, k, v, o, lse, c)
        if want is None:
            want = got
            same = torch.ones((), dtype=torch.bool, device="cuda")
        for x, y in zip(got, want):
            same &= (x == y).all()
    assert bool(same) and lce.device_status() == 0


def test_graph_capture():
    lens = [200, 56]
    q, k, v, do = make(lens, lens, 4, 2, 64, "bf16")
    c = cu(lens)
    o, lse = lce.attention_forward(q, k, v, c)
    want = (o, lse) + lce.attention_backward(do, q, k, v, o, lse, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = lce.attention_forward(q, k, v, c)
        got = (o2, lse2) + lce.attention_backward(do, q, k, v, o2, lse2, c)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_refusals():
    q, k, v, do = make([8], [8], 2, 1, 64, "bf16")
    o, lse = lce.attention_forward(q, k, v)
    fwd = lce.attention_forward
    for args in ((q.cpu(), k, v), (q, k.float(), v), (q.half(), k.half(), v.half()), (q, k, v[:4]),
                 (q, k[..., :32], v[..., :32]), (q[:, :, ::2], k[:, :, ::2], v[:, :, ::2]), (q[0], k[0], v[0])):
        with pytest.raises(ValueError):
            fwd(*args)
    with pytest.raises(ValueError):
        fwd(torch.cat([q, q, q], 1)[:, :5], torch.cat([k, k], 1), torch.cat([v, v], 1))   # 5 heads over 2
    for c in (cu([8]).long(), cu([8])[:1], cu([8]).cpu(), torch.cat([cu([8])] * 2)[::2]):
        with pytest.raises(ValueError):
            fwd(q, k, v, c)
    with pytest.raises(ValueError):
        fwd(q, k, v, cu([8]), cu([4, 4]))
    with pytest.raises(lce.LceError):   # 264 channels; 12 channels; a scale that is not a number
        fwd(*(torch.zeros(4, 1, 264, device="cuda", dtype=torch.bfloat16),) * 3)
    with pytest.raises(lce.LceError):
        fwd(*(torch.zeros(4, 1, 12, device="cuda", dtype=torch.bfloat16),) * 3)
    with pytest.raises(lce.LceError):
        fwd(q, k, v, scale=float("nan"))
    odd = torch.zeros(8 * 64 * 2 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(8, 2, 64)
    with pytest.raises(lce.LceError):
        fwd(odd, k, v)
    with pytest.raises(ValueError):
        lce.attention_backward(do, q, k, v, o, lse[:1])
    with pytest.raises(ValueError):
        lce.attention_backward(do[:4], q, k, v, o, lse)
    with pytest.raises(lce.LceError):
        lce.attention_backward(do, q, k, v, o, lse, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lce.LceError):   # gradients of several rows in one place
        lce.attention_backward(do, q, k, v, o, lse, dq=torch.zeros(1, 2, 64, device="cuda", dtype=torch.bfloat16).expand(8, 2, 64))
    assert lce.attention_workspace_size(8, 8, 2, 1, 64) > 0
