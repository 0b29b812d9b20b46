"""The gated recurrence over packed sequences, forward and backward, against the
fp64 reference.

Tolerances, elementwise: an output is rounded once to its type (u = half a
step: 2^-8 for bf16, 2^-24 for fp32 and the states); before it every step is off
by a share F = 2^-24 * (16 + 2 max|g|) of its absolute terms, since the gate's
exponent is off by |g| / ln 2 roundings and a step and its place in the scan are
a dozen operations; the reference sums up what all steps before amount to. The
backward's products of two such sums take twice that share. Below fp32's normal
range a gate is off by 2^-126 at most (logits below -87 count as -87, subnormals
have fewer bits); what multiplies it are sums of at most 2^13 products of two
values below 2^4, less than 2^26 (dg: a product of two such sums, 2^52 times
smaller gates still): 2^-74 absolutely."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402
from oracle import recurrent_oracle as ro  # noqa: E402

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


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def cu(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


def make(lens, d, dtype, tail=0, state=True, seed=0, slices=True, gates=(2.0, 1.5)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, B = sum(lens) + tail, len(lens)
    r = lambda *s, mean=0.0, std=1.0: torch.randn(*s, generator=g, device="cuda") * std + mean  # noqa: E731
    xg = torch.cat([r(T, d), r(T, d, mean=gates[0], std=gates[1])], 1).to(DT[dtype])
    x, gate = xg[:, :d], xg[:, d:]
    if not slices:
        x, gate = x.contiguous(), gate.contiguous()
    return dict(x=x, g=gate, dh=r(T, d).to(DT[dtype]), state=r(B, d) if state else None, dfinal=r(B, d) if state else None)


def close(name, got, want, u, slack):
    err = np.abs(f64(got) - want)
    tol = u * np.abs(want) + slack + 2.0 ** -74
    assert np.all(err <= tol), (name, float(err.max()), float((err - tol).max()))


def check(lens, d, dtype, tail=0, state=True, equal=False, seed=0, slices=True, gates=(2.0, 1.5)):
    t = make(lens, d, dtype, tail, state, seed, slices, gates)
    B, T = len(lens), sum(lens) + tail
    shape = (lambda z: z.unflatten(0, (B, lens[0]))) if equal else (lambda z: z)
    x, g, dh, offsets = shape(t["x"]), shape(t["g"]), shape(t["dh"]), None if equal else cu(lens)
    h, final, kept = lce.gated_recurrence_forward(x, g, offsets, state=t["state"], keep=True)
    grads = lce.gated_recurrence_backward(dh, x, g, kept, offsets, state=t["state"], dfinal=t["dfinal"])
    h2, final2, none = lce.gated_recurrence_forward(x, g, offsets, state=t["state"])
    grads2 = lce.gated_recurrence_backward(dh, x, g, kept, offsets, state=t["state"], dfinal=t["dfinal"])
    assert none is None and torch.equal(h, h2) and torch.equal(final, final2) and h.shape == x.shape
    assert all(a is b or torch.equal(a, b) for a, b in zip(grads, grads2))
    H, Fi, eh, ef, K = ro.recurrence_forward(f64(t["x"]), f64(t["g"]), lens, f64(t["state"]))
    ek = np.zeros_like(K)
    if T > 128:
        ek[1:] = eh[127:T - 1:128][:len(K) - 1]
    gmax = np.abs(f64(t["g"])).max() if T else 0.0
    u, F = U[dtype], 2.0 ** -24 * (16 + 2 * gmax)
    close("h", h.reshape(T, d), H, u, F * eh)
    close("final", final, Fi, 2.0 ** -24, F * ef)
    close("kept", kept, K, 2.0 ** -24, F * ek)
    want = ro.recurrence_backward(f64(t["dh"]), f64(t["x"]), f64(t["g"]), lens, f64(t["state"]), f64(t["dfinal"]))
    for name, got in zip(("dx", "dg", "dstate"), grads):
        if name == "dstate" and not state:
            assert got is None
            continue
        v, e = want[name]
        close(name, got.reshape(v.shape), v, U["fp32"] if name == "dstate" else u, 2 * F * e)
    assert lce.device_status() == 0
    return t, h, final, kept, grads


LENS = [[1], [2], [127], [128], [129], [300], [1, 1, 1], [5, 0, 7, 0], [0], [0, 0, 3], [64, 64, 64], [128, 128], [1000, 1, 24],
        [700, 3, 0, 0, 1, 500, 129, 0]]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", LENS, ids=lambda s: "-".join(map(str, s)))
def test_lengths(lens, dtype):
    check(lens, 72, dtype, state=True)
    check(lens, 72, dtype, state=False, tail=37)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [8, 16, 24, 64, 72, 128, 136, 200, 520, 1032])
def test_widths(d, dtype):
    check([130, 0, 45, 261], d, dtype, tail=5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(5000, 8), (2100, 64), (4097, 40), (1300, 264)])
def test_long_sequences(T, d, dtype):
    check([T], d, dtype)
    check([T - 600, 600], d, dtype, tail=300, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,L,d", [(1, 1, 8), (16, 1, 128), (5, 1, 1000), (300, 1, 64), (3, 2, 64), (4, 130, 72), (2, 700, 16)])
def test_equal_lengths_and_single_tokens(B, L, d, dtype):
    check([L] * B, d, dtype, equal=True)
    check([L] * B, d, dtype, equal=True, state=False, slices=False, seed=1)


def test_many_short_sequences():
    check([1] * 700, 64, "bf16")
    check([0, 3, 1, 0, 0, 2, 5] * 90, 24, "fp32", tail=9)
    check([0] * 500 + [10] + [0] * 500, 16, "fp32")


@pytest.mark.parametrize("gates", [(0.0, 1.0), (-8.0, 6.0), (12.0, 6.0), (0.0, 60.0)])
def test_gates_that_remember_everything_or_nothing(gates):
    check([600, 77], 64, "fp32", gates=gates)
    check([600, 77], 64, "bf16", gates=gates)


def test_logits_at_the_ends_of_their_type():
    x = torch.ones(6, 8, device="cuda")
    g = torch.tensor([-3.4e38, 3.4e38, 0.0, float("inf"), float("-inf"), -100.0], device="cuda")[:, None].repeat(1, 8)
    h, final, kept = lce.gated_recurrence_forward(x, g, keep=True)
    assert torch.allclose(h[:, 0].cpu(), torch.ones(6), atol=1e-7)
    dx, dg, _ = lce.gated_recurrence_backward(torch.ones_like(x), x, g, kept)
    assert dx.isfinite().all() and dg.isfinite().all()
    g[2, 3] = float("nan")
    h, *_ = lce.gated_recurrence_forward(x, g)
    assert h[2:4, 3].isnan().all() and not h[:, :3].isnan().any() and not h[:2].isnan().any()


def test_nothing_reaches_another_sequence():
    """Infinities and NaN in one sequence, its state, its gradients and the tail; the others' results bit for bit."""
    lens, d, tail = [40, 300, 1, 200], 72, 50
    for dtype in ("bf16", "fp32"):
        t = make(lens, d, dtype, tail)
        run = lambda: (lce.gated_recurrence_forward(t["x"], t["g"], cu(lens), state=t["state"], keep=True))  # noqa: E731
        h, final, kept = run()
        grads = lce.gated_recurrence_backward(t["dh"], t["x"], t["g"], kept, cu(lens), state=t["state"], dfinal=t["dfinal"])
        for name in ("x", "g", "dh"):
            t[name] = t[name].clone()
            t[name][40:340] = float("nan")
            t[name][45] = float("inf")
            t[name][541:] = float("nan")
        for name in ("state", "dfinal"):
            t[name][1] = float("inf")
        h2, final2, kept = run()
        grads2 = lce.gated_recurrence_backward(t["dh"], t["x"], t["g"], kept, cu(lens), state=t["state"], dfinal=t["dfinal"])
        rows = torch.ones(sum(lens) + tail, dtype=torch.bool)
        rows[40:340] = False
        seqs = torch.tensor([True, False, True, True])
        assert torch.equal(h[rows], h2[rows]) and torch.equal(final[seqs], final2[seqs])
        assert torch.equal(grads[0][rows], grads2[0][rows]) and torch.equal(grads[1][rows], grads2[1][rows])
        assert torch.equal(grads[2][seqs], grads2[2][seqs]) and not h2[541:].any() and not grads2[0][541:].any()


def test_state_updated_in_place():
    for lens, equal in (([1] * 9, True), ([5, 0, 300, 1], False)):
        t = make(lens, 136, "bf16")
        shape = (lambda z: z.unflatten(0, (len(lens), 1))) if equal else (lambda z: z)
        offsets = None if equal else cu(lens)
        h, final, _ = lce.gated_recurrence_forward(shape(t["x"]), shape(t["g"]), offsets, state=t["state"])
        state = t["state"].clone()
        h2, f2, _ = lce.gated_recurrence_forward(shape(t["x"]), shape(t["g"]), offsets, state=state, out_state=state)
        assert f2 is state and torch.equal(state, final) and torch.equal(h, h2) and state._version > 0


def test_token_by_token_is_the_whole_sequence():
    t = make([50, 50, 50], 64, "fp32", state=False, slices=False)
    x, g = (t[k].unflatten(0, (3, 50)) for k in ("x", "g"))
    h, final, _ = lce.gated_recurrence_forward(x, g)
    state = torch.zeros(3, 64, device="cuda")
    for i in range(50):
        step, _, _ = lce.gated_recurrence_forward(x[:, i:i + 1], g[:, i:i + 1], state=state, out_state=state)
        assert (step[:, 0] - h[:, i]).abs().max() <= 50 * 2.0 ** -22
    assert (state - final).abs().max() <= 50 * 2.0 ** -22


def test_given_outputs_strides_streams_and_graphs():
    lens, d = [200, 0, 333], 136
    t = make(lens, d, "bf16", tail=11)
    args = (t["x"], t["g"], cu(lens))
    h, final, kept = lce.gated_recurrence_forward(*args, state=t["state"], keep=True)
    grads = lce.gated_recurrence_backward(t["dh"], t["x"], t["g"], kept, cu(lens), state=t["state"], dfinal=t["dfinal"])
    T = sum(lens) + 11
    wide = torch.full((T, 3 * d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, f2 = wide[:, :d], torch.empty_like(final)
    lce.gated_recurrence_forward(*args, state=t["state"], out=out, out_state=f2, stream=s)
    dx, dg = wide[:, d:2 * d], wide[:, 2 * d:3 * d]
    lce.gated_recurrence_backward(t["dh"], t["x"], t["g"], kept, cu(lens), state=t["state"], dfinal=t["dfinal"], dx=dx, dg=dg, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, h) and torch.equal(f2, final) and torch.equal(dx, grads[0]) and torch.equal(dg, grads[1])
    assert bool((wide[:, 3 * d:] == 3).all()) and wide._version > 0
    offsets = cu(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g_h, g_f, g_k = lce.gated_recurrence_forward(t["x"], t["g"], offsets, state=t["state"], keep=True)
        g_grads = lce.gated_recurrence_backward(t["dh"], t["x"], t["g"], g_k, offsets, state=t["state"], dfinal=t["dfinal"])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g_h, h) and torch.equal(g_f, final) and torch.equal(g_k, kept)
    assert all(torch.equal(a, b) for a, b in zip(g_grads, grads))


def test_offsets_that_do_not_ascend_are_reported():
    t = make([60, 40], 64, "bf16", state=False)
    for bad in ([0, 70, 60], [0, 50, 101], [1, 50, 100], [0, -5, 100]):
        lce.gated_recurrence_forward(t["x"], t["g"], torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert lce.device_status() == 4
    lce.gated_recurrence_forward(t["x"], t["g"], cu([60, 40]))
    assert lce.device_status() == 0


def test_autograd():
    lens = [70, 0, 200]
    t = make(lens, 72, "fp32")
    x, g, s = (t[k].clone().requires_grad_(True) for k in ("x", "g", "state"))
    h, final = lce.gated_recurrence(x, g, cu(lens), state=s)
    grads = torch.autograd.grad((h * t["dh"]).sum() + (final * t["dfinal"]).sum(), (x, g, s))
    _, _, kept = lce.gated_recurrence_forward(t["x"], t["g"], cu(lens), state=t["state"], keep=True)
    want = lce.gated_recurrence_backward(t["dh"], t["x"], t["g"], kept, cu(lens), state=t["state"], dfinal=t["dfinal"])
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    # the final state alone (no gradient reaches h), a state without a gradient, expanded gradients
    h, final = lce.gated_recurrence(x, g, cu(lens), state=t["state"])
    (gx,) = torch.autograd.grad(final.sum(), x)
    ones = torch.ones_like(final)
    want = lce.gated_recurrence_backward(torch.zeros_like(t["dh"]), t["x"], t["g"], kept, cu(lens), state=t["state"], dfinal=ones)
    assert torch.equal(gx, want[0])
    h, final = lce.gated_recurrence(x, g, cu(lens))
    (gx,) = torch.autograd.grad(h.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        gx.sum().backward()


def test_the_gradient_is_a_difference():
    lens = [140, 9]
    t = make(lens, 8, "fp32", slices=False)
    loss = lambda: (lce.gated_recurrence_forward(t["x"], t["g"], cu(lens), state=t["state"])[0].double() * t["dh"].double()).sum().item()  # noqa: E731
    _, _, kept = lce.gated_recurrence_forward(t["x"], t["g"], cu(lens), state=t["state"], keep=True)
    grads = lce.gated_recurrence_backward(t["dh"], t["x"], t["g"], kept, cu(lens), state=t["state"])
    for name, grad, i in (("x", grads[0], 3), ("g", grads[1], 130), ("g", grads[1], 141), ("state", grads[2], 1)):
        keep, eps = t[name][i, 5].item(), 1e-2
        t[name][i, 5] = keep + eps
        up = loss()
        t[name][i, 5] = keep - eps
        down = loss()
        t[name][i, 5] = keep
        # third derivatives (below 1 here) times eps^2 and the roundings of h over 2 eps
        assert abs((up - down) / (2 * eps) - grad[i, 5].item()) < 1e-3
