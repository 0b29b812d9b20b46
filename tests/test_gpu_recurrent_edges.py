"""The recurrent block's operators where they can go wrong: long sums, values at
the ends of their types, geometries that only large calls reach, layouts that
autograd hands over. Tolerances count half steps of the output's type (2^-8 for
bf16, 2^-24 for fp32) and are derived beside each test."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    lce.device_status()
    yield


def rand(*shape, seed=0, dtype=torch.float32, positive=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand if positive else torch.randn)(*shape, generator=g, device="cuda").to(dtype)


def packed_grad64(dy, p, rows):
    """The first `rows` rows of dy^T x in fp64."""
    return dy[:, :rows].double().T @ lce.unpack_activation(p, dtype=torch.float32).double()


# ------------------------------------------------------------ weight gradient

@pytest.mark.parametrize("T,n,k", [(4097, 1024, 4096), (16384, 4096, 2568), (20000, 256, 256)])
def test_fp32_gradient_of_a_bf16_dy_of_many_tokens_that_all_add_up(T, n, k):
    """Each addition of 16 products is truncated twice, by less than a step each, 2^-23 of a sum that is half filled on average. A
    run of 1024 tokens has 64 additions, so it is off by at most 2^-17 of itself, and by half of that on average; the runs are
    added up with roundings of 2^-24 of what there is by then."""
    dy, p = rand(T, n, seed=3, dtype=torch.bfloat16, positive=True), lce.pack_activation(rand(T, k, seed=4, positive=True))
    got = lce.packed_weight_grad(dy, p, out_dtype=torch.float32)
    want = packed_grad64(dy, p, 256)
    off = (got[:256].double() - want) / want
    runs = (T + 1023) // 1024 + 152   # and splits
    assert off.abs().max().item() <= 2.0 ** -17 + runs * 2.0 ** -24
    assert abs(off.mean().item()) <= 2.0 ** -18 + 2.0 ** -24 * runs ** 0.5
    assert off.norm().item() / off.numel() ** 0.5 <= 1e-6   # what a product of plain fp32 is off by
    assert torch.equal(lce.packed_weight_grad(dy, p, out_dtype=torch.float32), got)


def test_bf16_gradient_of_very_many_tokens_that_all_add_up():
    """A run of 32768 tokens has 2048 additions, truncated twice, by half a step each on average: one step of 2^-23 of a sum that
    is half filled, 2^-13 of it together, give or take 6 times sqrt(4096 / 12) steps, less than a sixteenth of that. Rounding
    to bf16 keeps the order, so the result lies between the roundings of the sum less that and of the sum (1 + 2^-22: the runs'
    joins)."""
    T, n, k = 262144, 4096, 2432
    dy, p = rand(T, n, seed=5, dtype=torch.bfloat16, positive=True), lce.pack_activation(rand(T, k, seed=6, positive=True))
    got = lce.packed_weight_grad(dy, p)
    want = packed_grad64(dy, p, 64)
    assert bool((got[:64] >= (want * (1 - 2.0 ** -13 * 1.0625)).bfloat16()).all())
    assert bool((got[:64] <= (want * (1 + 2.0 ** -22)).bfloat16()).all())
    need = lce.packed_weight_grad_workspace_size(T, n, k)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    assert torch.equal(lce.packed_weight_grad(dy, p, workspace=ws[:need]), got) and bool((ws[need:] == 77).all())
    with pytest.raises(RuntimeError):
        lce.packed_weight_grad(dy, p, workspace=ws[:need - 1])
    assert lce.device_status() == 0


def test_a_large_gradient_repeats_itself_beside_other_work():
    """7373 tokens of a 4096 to 16384 layer: the same bits whatever runs beside it, and its error that of rounding to bf16."""
    dy, p = rand(7373, 16384, seed=7, dtype=torch.bfloat16), lce.pack_activation(rand(7373, 4096, seed=8, dtype=torch.bfloat16))
    got, junk, side = lce.packed_weight_grad(dy, p), torch.zeros(1 << 28, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    for i in range(30):
        if i % 2:
            with torch.cuda.stream(side):
                junk.add_(1)
        assert torch.equal(lce.packed_weight_grad(dy, p), got)
    want = packed_grad64(dy, p, 512)
    off, rounding = (got[:512].double() - want).norm().item(), (want.bfloat16().double() - want).norm().item()
    # the sums' own error, 1e-5 of the norm at most, is independent of the rounding's, 1.6e-3 of it
    assert off <= rounding * (1 + 1e-4)
    torch.cuda.synchronize()


def test_fp32_dy_up_to_the_largest_value():
    """Values that bf16 would round to infinity: the lowest value of a mask among them, beside codes of zero and of one."""
    most = torch.finfo(torch.float32).max
    dy, x = torch.zeros(70, 64, device="cuda"), torch.zeros(70, 256, device="cuda")
    dy[0, 0], dy[1, 1], dy[2, 2], dy[3, 3], dy[65, 4] = most, -most, 3.395e38, 3.39e38, float("inf")
    x[:4, 0], x[65, 0] = 1.0, 1.0
    x[:4, 1] = 0.5
    got, want = lce.packed_weight_grad(dy, lce.pack_activation(x)), (dy.double().T @ x.double()).float()
    assert torch.equal(got[:4], want[:4]) and got[0, 0] == most and got[1, 0] == -most and not got[:4, 2:].any()
    assert got[4, 0] == float("inf") and got[4, 1:].isnan().all() and not got[5:].any()


# --------------------------------------------------------------- linear_keep8

def test_linear_keep8_refuses_at_the_call_what_its_gradient_cannot_take():
    x = rand(40, 64, dtype=torch.bfloat16)
    for shape in ((12, 64), (0, 64)):
        with pytest.raises(ValueError, match="multiples of 8"):
            lce.linear_keep8(x, rand(*shape, dtype=torch.bfloat16).requires_grad_(True))
    with pytest.raises(ValueError, match="multiples of 8"):
        lce.linear_keep8(rand(40, 20), rand(16, 20).requires_grad_(True))
    with torch.no_grad():
        lce.linear_keep8(x, rand(12, 64, dtype=torch.bfloat16).requires_grad_(True))
    # a frozen weight has no such gradient
    w = rand(12, 64, dtype=torch.bfloat16)
    y = lce.linear_keep8(x.requires_grad_(True), w)
    assert torch.equal(y, torch.nn.functional.linear(x, w))
    assert torch.equal(torch.autograd.grad(y, x, torch.ones_like(y))[0], torch.ones_like(y) @ w)


@pytest.mark.parametrize("x_dtype,w_dtype", [("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_linear_keep8_under_autocast(x_dtype, w_dtype):
    """The gradients of the casts and of the bf16 operator, bit for bit; the products outside it are autocast's as before."""
    x = rand(3, 30, 136, dtype=DT[x_dtype]).requires_grad_(True)
    w, dy = rand(72, 136, seed=1, dtype=DT[w_dtype]).requires_grad_(True), rand(3, 30, 72, seed=2, dtype=torch.bfloat16)
    with torch.autocast("cuda", dtype=torch.bfloat16):
        y = lce.linear_keep8(x, w)
        assert (x @ w.T).dtype == torch.bfloat16
    xb, wb = x.detach().bfloat16(), w.detach().bfloat16()
    assert y.dtype == torch.bfloat16 and torch.equal(y, torch.nn.functional.linear(xb, wb))
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    want = lce.packed_weight_grad(dy.view(90, 72), lce.pack_activation(xb.view(90, 136)))
    assert dx.dtype == x.dtype and dw.dtype == w.dtype and torch.equal(dx, (dy @ wb).to(x.dtype)) and torch.equal(dw, want.to(w.dtype))
    with torch.autocast("cuda", dtype=torch.float16), pytest.raises(ValueError, match="bfloat16 or float32"):
        lce.linear_keep8(x, w)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_keep8_takes_x_in_any_layout(dtype):
    """Transposed, expanded, off 16 bytes, with odd rows: what PyTorch's linear takes, and the gradient of a plain copy."""
    base = rand(41 * 137, dtype=DT[dtype])
    w, dy = rand(72, 136, seed=1, dtype=DT[dtype]).requires_grad_(True), rand(40, 72, seed=2, dtype=DT[dtype])
    layouts = (rand(136, 40, seed=3, dtype=DT[dtype]).t(), base[1:1 + 40 * 136].view(40, 136), base[:40 * 137].view(40, 137)[:, :136],
               base[:136].expand(40, 136), base[:40].view(40, 1).expand(40, 136), rand(40, 272, dtype=DT[dtype])[:, ::2])
    for x in layouts:
        y = lce.linear_keep8(x, w)
        (dw,) = torch.autograd.grad(y, w, dy)
        want = lce.packed_weight_grad(dy, lce.pack_activation(x.clone(memory_format=torch.contiguous_format)))
        assert torch.equal(y, torch.nn.functional.linear(x, w)) and torch.equal(dw, want)


def test_nothing_is_kept_where_no_gradient_is_recorded():
    """Parameters ask for gradients under no_grad as well; what a call leaves and takes there is its result alone."""
    N, d = 4096, 1024
    x, g = rand(N, d, dtype=torch.bfloat16).requires_grad_(True), rand(N, d, seed=1, dtype=torch.bfloat16).requires_grad_(True)
    w, s = rand(d, d, seed=2, dtype=torch.bfloat16).requires_grad_(True), torch.zeros(1, d, device="cuda")
    v = torch.ones(d, dtype=torch.bfloat16, device="cuda").requires_grad_(True)
    calls = ((lambda: lce.linear_keep8(x, w), 0, N * d * 2), (lambda: lce.layer_norm(x, weight=v, keep8=True), 1, N * d * 2 + N * 8),
             (lambda: lce.layer_norm(x, g, weight=v, bias=v, keep8=True), 1, N * d * 4 + N * 8),
             (lambda: lce.gated_recurrence(x, g), 1, N * d * 2 + d * 4))
    for call, launches, size in calls:
        recorded = call()
        for grad_off in (torch.no_grad, torch.inference_mode):
            with grad_off():
                torch.cuda.synchronize()
                before, held = lce.launch_count(), torch.cuda.memory_allocated()
                torch.cuda.reset_peak_memory_stats()
                got = call()
                assert lce.launch_count() - before == launches and torch.cuda.max_memory_allocated() - held <= size + (1 << 14)
            pairs = [(got, recorded)] if torch.is_tensor(got) else zip(got, recorded)
            assert all(torch.equal(a, b) and not a.requires_grad for a, b in pairs if a is not x)
    # nor with gradients recorded, where no input asks for one
    before = lce.launch_count()
    lce.linear_keep8(x.detach(), w.detach())
    assert lce.launch_count() == before


# ----------------------------------------------------------------- layer norm

@pytest.mark.parametrize("N,d,dtype", [(16001, 1032, "bf16"), (30011, 64, "bf16"), (4099, 4104, "bf16"), (9001, 1032, "fp32"),
                                       (1501, 4096, "fp32")])
@pytest.mark.parametrize("keep8", [False, True], ids=["", "keep8"])
def test_layer_norm_in_place_through_the_ring(N, d, dtype, keep8):
    """r written over x or over b while later rows are still on their way, the last row copied in place of rows past it: the bits
    of a call with an r of its own, at sizes whose blocks refill their ring and end inside a stage."""
    x, b, w, c = rand(N, d, dtype=DT[dtype]), rand(N, d, seed=1, dtype=DT[dtype]), rand(d, seed=2, dtype=DT[dtype]), rand(d, seed=3, dtype=DT[dtype])
    r, n, mean, rstd, kept = lce.layer_norm_forward(x, b, weight=w, bias=c, keep8=keep8)
    assert torch.equal(r, (x.float() + b.float()).to(DT[dtype]))
    for into in (0, 1):
        pair = [x.clone(), b.clone()]
        r2, n2, mean2, rstd2, kept2 = lce.layer_norm_forward(*pair, weight=w, bias=c, keep8=keep8, out_r=pair[into])
        assert r2 is pair[into] and torch.equal(r2, r) and torch.equal(pair[1 - into], (x, b)[1 - into])
        assert torch.equal(n2, n) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
        assert not keep8 or (torch.equal(kept2.codes, kept.codes) and torch.equal(kept2.exps, kept.exps))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,d", [(3, 1000), (5000, 1000), (5000, 1032), (3000, 2600), (1200, 5000)])
def test_layer_norm_of_rows_of_one_value(N, d, dtype):
    """Rows of whole numbers whose sums fp32 holds: the mean is the value itself, so nothing is left to be scaled up by the square
    root of 1 / eps."""
    x = (torch.arange(N, device="cuda") - N // 2).remainder(256).sub(128).mul(8.0)[:, None].expand(N, d).to(DT[dtype]).contiguous()
    w, c = rand(d, dtype=DT[dtype]), rand(d, seed=1, dtype=DT[dtype])
    _, n, mean, rstd, _ = lce.layer_norm_forward(x, weight=w, bias=c)
    assert torch.equal(mean, x[:, 0].float()) and torch.equal(n, c.expand(N, d))


# ------------------------------------------------------------------- autograd

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_at_addresses_off_16_bytes(dtype):
    """A slice of another gradient, as an output that was flattened behind a few other values gets it, is contiguous and starts
    anywhere: the same bits as from a gradient of its own."""
    r = lambda *s, seed=0: rand(*s, seed=seed, dtype=DT[dtype]).requires_grad_(True)  # noqa: E731
    x, b, w, c, m = r(40, 64), r(40, 64, seed=1), r(64, seed=2), r(64, seed=3), r(24, 64, seed=4)
    s, q, k = rand(1, 64, seed=5).requires_grad_(True), r(40, 2, 64, seed=6), r(40, 1, 64, seed=7)
    calls = ((lambda: lce.linear_keep8(x, m), (x, m)), (lambda: lce.layer_norm(x, b, weight=w, bias=c), (x, b, w, c)),
             (lambda: lce.layer_norm(x, weight=w, bias=c, keep8=True), (x, w, c)), (lambda: lce.gated_recurrence(x, b, state=s), (x, b, s)),
             (lambda: lce.attention(q, k, k), (q, k)), (lambda: lce.block_norm(x, b, w_post=w, w_pre=c), (x, b, w, c)),
             (lambda: lce.block_norm(x, w_pre=w), (x, w)))
    for call, leaves in calls:
        outs = call()
        outs = (outs,) if torch.is_tensor(outs) else outs
        grads = [rand(*o.shape, seed=9 + i, dtype=o.dtype) for i, o in enumerate(outs)]
        odd = []
        for g in grads:
            room = torch.empty(g.numel() + 3, dtype=g.dtype, device="cuda")
            odd.append(room[3:].view(g.shape).copy_(g))
            assert odd[-1].is_contiguous() and odd[-1].data_ptr() % 16
        want = torch.autograd.grad(outs, leaves, grads, retain_graph=True)
        got = torch.autograd.grad(outs, leaves, odd)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ----------------------------------------------------------------- recurrence

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gates_and_their_complements_to_their_own_precision(dtype):
    """Seen one at a time: from zero states and x = 1 a token's state is 1 - a, from a gradient of 1 of that state alone the
    state's own is a. In units of 2^-24: the exponential is off by 4 (two steps of the approximation) and a rounding, the sum
    with 1 and the product by a rounding each, the reciprocal by 2 (a step): 9. bf16 logits add |z| / 2 for z = g log2(e),
    times ln 2: |g| / 2 and the same for what fp32 leaves of log2(e)."""
    for lo, hi in ((-4, 4), (4, 8), (8, 16), (16, 30), (30, 60), (60, 87), (-8, -4), (-30, -8), (-87, -30)):
        g = (rand(4096, 64, seed=lo + 100, positive=True) * (hi - lo) + lo).to(DT[dtype])
        one, zero, ones = torch.ones_like(g), torch.zeros(4096, 64, device="cuda"), torch.ones(4096, 64, device="cuda")
        cu = torch.arange(4097, dtype=torch.int32, device="cuda")
        _, rest, kept = lce.gated_recurrence_forward(one, g, cu, state=zero, keep=True)
        _, rest1, _ = lce.gated_recurrence_forward(one.unsqueeze(1), g.unsqueeze(1), state=zero)
        dx, _, a = lce.gated_recurrence_backward(torch.zeros_like(g), one, g, kept, cu, state=zero, dfinal=ones)
        G, units = g.double(), 9 + (g.abs().max().item() if dtype == "bf16" else 0)
        for got, want in ((rest, 1 / (1 + torch.exp(G))), (rest1, 1 / (1 + torch.exp(G))), (a, 1 / (1 + torch.exp(-G)))):
            assert ((got.double() - want).abs() / want).max().item() <= units * 2.0 ** -24, (lo, hi)
        want = 1 / (1 + torch.exp(G))
        assert ((dx.double() - want).abs() / want).max().item() <= (units + 1) * 2.0 ** -24 + (U["bf16"] if dtype == "bf16" else 0)


@pytest.mark.parametrize("B,L", [(0, 5), (0, 1), (0, 0), (3, 0)])
def test_batches_without_sequences_or_tokens(B, L):
    x = torch.empty(B, L, 64, device="cuda")
    state, dfinal = rand(B, 64), rand(B, 64, seed=1)
    for s in (state, None):
        h, final, kept = lce.gated_recurrence_forward(x, x, state=s, keep=True, out_state=torch.full((B, 64), 7.0, device="cuda"))
        assert h.shape == x.shape and torch.equal(final, state if s is not None else torch.zeros(B, 64, device="cuda"))
        dx, dg, dstate = lce.gated_recurrence_backward(x, x, x, kept, state=s, dfinal=dfinal)
        assert dx.shape == dg.shape == x.shape and (dstate is None if s is None else torch.equal(dstate, dfinal))
    leaf, s = x.clone().requires_grad_(True), state.clone().requires_grad_(True)
    h, final = lce.gated_recurrence(leaf, leaf, state=s)
    (ds,) = torch.autograd.grad(final, s, dfinal)
    assert torch.equal(ds, dfinal)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("where", [0, 5, 140, 700])
def test_an_infinity_stays_one_through_gates_that_forget(where, dtype):
    """A gate is never zero, so no token after an infinite one (or before an infinite gradient) has a finite state or a NaN,
    however small the product of the gates between them: here e^-20 each."""
    T, d = 1400, 64
    x, g, dh = rand(T, d, dtype=DT[dtype]), torch.full((T, d), -20.0, dtype=DT[dtype], device="cuda"), rand(T, d, seed=1, dtype=DT[dtype])
    x[where, ::2], x[where, 1::2] = float("inf"), float("-inf")
    sign = torch.tensor([1.0, -1.0], device="cuda").repeat(d // 2)
    h, final, kept = lce.gated_recurrence_forward(x, g, keep=True)
    assert bool((h[where:].float() == sign * float("inf")).all()) and bool(h[:where].isfinite().all())
    assert torch.equal(final[0], sign * float("inf"))
    dh[T - 1 - where, ::2], dh[T - 1 - where, 1::2] = float("inf"), float("-inf")
    x = rand(T, d, dtype=DT[dtype])
    _, _, kept = lce.gated_recurrence_forward(x, g, keep=True)
    state = torch.ones(1, d, device="cuda")
    dx, _, dstate = lce.gated_recurrence_backward(dh, x, g, kept, state=state)
    assert bool((dx[:T - where].float() == sign * float("inf")).all()) and bool(dx[T - where:].isfinite().all())
    assert torch.equal(dstate[0], sign * float("inf"))
    # an infinite state, and one sequence among others
    lens = [300, 500, 600]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    state = torch.ones(3, d, device="cuda")
    state[1] = sign * float("inf")
    h, final, _ = lce.gated_recurrence_forward(x, g, cu, state=state)
    assert bool((h[300:800].float() == sign * float("inf")).all()) and torch.equal(final[1], state[1])
    assert bool(h[:300].isfinite().all()) and bool(h[800:].isfinite().all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_millions_of_empty_sequences(dtype):
    """Before, between and behind sequences, in a tile and at its border: the results are those without them, bit for bit, and
    their states pass through."""
    lens, d, many = [200, 56, 300, 84], 16, 700_000
    x, g, dh = (rand(700, d, seed=i, dtype=DT[dtype]) for i in range(3))   # the last 60 tokens belong to no sequence
    ends = torch.tensor([0] + lens).cumsum(0)
    some = torch.tensor([0, 1, 2, 3]) + many * torch.tensor([1, 2, 3, 4])   # their numbers with `many` empty ones before each
    cu = torch.cat([ends[i].repeat(many + 1) for i in range(4)] + [ends[4].repeat(many)])
    cu = torch.cat([cu, ends[4:]]).to(torch.int32).cuda()
    B = cu.numel() - 1
    state, dfinal = rand(B, d, seed=4), rand(B, d, seed=5)
    few, less, dless = ends.to(torch.int32).cuda(), state[some].contiguous(), dfinal[some].contiguous()
    h, final, kept = lce.gated_recurrence_forward(x, g, cu, state=state, keep=True)
    h2, final2, kept2 = lce.gated_recurrence_forward(x, g, few, state=less, keep=True)
    assert torch.equal(h, h2) and torch.equal(final[some], final2) and torch.equal(kept, kept2)
    got = lce.gated_recurrence_backward(dh, x, g, kept, cu, state=state, dfinal=dfinal)
    want = lce.gated_recurrence_backward(dh, x, g, kept2, few, state=less, dfinal=dless)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2][some], want[2])
    rest = torch.ones(B, dtype=torch.bool)
    rest[some] = False
    assert torch.equal(final[rest], state[rest]) and torch.equal(got[2][rest], dfinal[rest])
    assert lce.device_status() == 0


def recurrence64(x, g, dh, lens, state, dfinal):
    """The recurrence and its gradients in fp64, a token at a time, each with the absolute sums of the terms of all steps before
    it: {name: (value, terms)}. A step that is off by a share of its terms, every step before it as well, is off by that share."""
    x, g, dh, state, dfinal = (t.double() for t in (x, g, dh, state, dfinal))
    T, d = x.shape
    a, rest = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    h, eh, dx, ex, dg, eg = (torch.zeros_like(x) for _ in range(6))
    final, ef, ds, es = (torch.zeros_like(state) for _ in range(4))
    begin = 0
    for i, n in enumerate(lens):
        s, z, e = state[i], state[i].abs(), state[i].abs()
        before = []
        for t in range(begin, begin + n):
            before.append((s, e))
            s, z = a[t] * s + rest[t] * x[t], a[t] * z + rest[t] * x[t].abs()
            e = a[t] * e + z
            h[t], eh[t] = s, e
        final[i], ef[i] = s, e
        m, z, e = dfinal[i], dfinal[i].abs(), dfinal[i].abs()
        for t in range(begin + n - 1, begin - 1, -1):
            hp, ep = before[t - begin]
            m, z = dh[t] + m, dh[t].abs() + z
            e = e + z
            dx[t], ex[t] = rest[t] * m, rest[t] * e
            dg[t], eg[t] = m * (hp - x[t]) * a[t] * rest[t], e * (ep + x[t].abs()) * a[t] * rest[t]
            m, z, e = a[t] * m, a[t] * z, a[t] * e
        ds[i], es[i] = m, e
        begin += n
    return {"h": (h, eh), "final": (final, ef), "dx": (dx, ex), "dg": (dg, eg), "dstate": (ds, es)}


@pytest.mark.parametrize("d,lens,tail,dtype", [
    (4096, [1012, 433, 0, 761, 1290, 64, 1], 300, "bf16"), (4096, [2900], 0, "bf16"), (8192, [700, 1250], 90, "bf16"),
    (2048, [3100, 5, 900], 30, "bf16"), (2560, [1999, 1300], 0, "bf16"), (10000, [900, 640], 10, "bf16"), (10000, [1500], 0, "bf16"),
    (2048, [1012, 433, 0, 761, 1290, 64, 1], 300, "fp32"), (4096, [2000, 300], 0, "fp32"), (5000, [900, 640], 10, "fp32"),
    (1024, [3500, 600], 0, "fp32"), (1024, [2600, 2, 1500], 20, "bf16"), (256, [4000, 1500], 0, "bf16")], ids=lambda v: str(v).replace(" ", ""))
def test_wide_models_over_many_tiles(d, lens, tail, dtype):
    """Widths whose channels leave each slice clusters of 1 to 16 CTAs over thousands of tokens: the rings of tiles, of their
    sequences' ends and of the cluster's steps go round many times. The tolerances are those of the narrow models: a rounding to
    the type, and before it F = 2^-24 (16 + 2 max|g|) of the terms, twice that for products of two sums; below fp32's normal
    range 2^-74."""
    T, B = sum(lens) + tail, len(lens)
    xg = torch.cat([rand(T, d, seed=1), rand(T, d, seed=2) * 1.5 + 2], 1).to(DT[dtype])
    x, g, dh = xg[:, :d], xg[:, d:], rand(T, d, seed=3, dtype=DT[dtype])
    state, dfinal = rand(B, d, seed=4), rand(B, d, seed=5)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    h, final, kept = lce.gated_recurrence_forward(x, g, cu, state=state, keep=True)
    dx, dg, dstate = lce.gated_recurrence_backward(dh, x, g, kept, cu, state=state, dfinal=dfinal)
    for _ in range(3):
        assert torch.equal(lce.gated_recurrence_forward(x, g, cu, state=state)[0], h)
        assert all(torch.equal(p, q) for p, q in zip(lce.gated_recurrence_backward(dh, x, g, kept, cu, state=state, dfinal=dfinal),
                                                     (dx, dg, dstate)))
    want, F = recurrence64(x, g, dh, lens, state, dfinal), 2.0 ** -24 * (16 + 2 * g.abs().max().item())
    for name, got, u, share in (("h", h, U[dtype], F), ("final", final, U["fp32"], F), ("dx", dx, U[dtype], 2 * F),
                                ("dg", dg, U[dtype], 2 * F), ("dstate", dstate, U["fp32"], 2 * F)):
        value, terms = want[name]
        over = (got.double() - value).abs() - (u * value.abs() + share * terms + 2.0 ** -74)
        assert over.max().item() <= 0, (name, over.max().item())
    assert lce.device_status() == 0
