"""Global gradient norm and clipping against the fp64 reference.

Tolerances: squares are summed in fp32 over at most 64 elements and in fp64
from there, so the norm's relative error is below (64 * 2^-24) / 2 plus its
own rounding: 2^-18. A clipped element is rounded once more (2^-8 covers bf16
twice over, 2^-23 fp32) and carries the factor's error, 2^-18."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402
from oracle import block_oracle as bo  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    yield


def f64(t):
    return t.detach().double().cpu().numpy()


def make(sizes, kinds, seed=0, std=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(torch.bfloat16 if k == "b" else torch.float32)
            for n, k in zip(sizes, kinds * len(sizes))]


def check(grads, max_norm, eps=1e-6):
    norm, c, want = bo.clip([f64(t) for t in grads], max_norm, eps)
    out = [torch.full_like(t, 3.0) for t in grads]
    got, factor = lce.clip_grad_norm(grads, max_norm, out=out, eps=eps, return_factor=True)
    assert abs(got.item() - norm) <= 2.0 ** -18 * norm
    assert abs(factor.item() - c) <= 2.0 ** -18 * c
    assert lce.grad_norm(grads).item() == got.item()
    here = [t.clone() for t in grads]
    assert lce.clip_grad_norm(here, max_norm, eps=eps).item() == got.item()
    for o, h, w, t in zip(out, here, want, grads):
        u = 2.0 ** -8 if t.dtype == torch.bfloat16 else 2.0 ** -23
        assert np.all(np.abs(f64(o) - w) <= (u + 2.0 ** -18) * np.abs(w) + 1e-38)
        assert torch.equal(o, h)
    return factor.item()


SIZES = [[1], [7], [4096], [100003], [1, 2, 3, 0, 5, 8, 13], [16384, 16385, 16383, 40000, 1, 0], [3_000_001, 17],
         [33] * 241, [5] * 700]


@pytest.mark.parametrize("kinds", ["b", "f", "bf"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip(sizes, kinds):
    grads = make(sizes, kinds)
    assert check(grads, 0.05) < 1.0
    assert check(grads, 1e9) == 1.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_slices_of_a_flat_buffer(dtype):
    """Gradients that start anywhere, outputs that start elsewhere, and what lies between them."""
    flat = torch.randn(200_000, device="cuda").to(dtype)
    out = torch.full((200_000,), 9.0, device="cuda", dtype=dtype)
    cuts = [(1, 6), (9, 9), (10, 30), (33, 20_001), (20_003, 90_000), (90_001, 150_007)]
    grads = [flat[a:b] for a, b in cuts]
    for shift in (0, 1, 3, 8):
        out.fill_(9.0)
        outs = [out[a + shift:b + shift] for a, b in cuts]
        # slices of one buffer must not overlap: write only every second one
        use = [i for i in range(len(cuts)) if i % 2 == 1]
        norm = lce.clip_grad_norm([grads[i] for i in use], 0.5, out=[outs[i] for i in use])
        ref, c, want = bo.clip([f64(grads[i]) for i in use], 0.5)
        assert abs(norm.item() - ref) <= 2.0 ** -18 * ref
        untouched = torch.ones_like(out, dtype=torch.bool)
        u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
        for i, w in zip(use, want):
            assert np.all(np.abs(f64(outs[i]) - w) <= (u + 2.0 ** -18) * np.abs(w))
            untouched[cuts[i][0] + shift:cuts[i][1] + shift] = False
        assert bool((out[untouched] == 9.0).all())


def test_not_finite():
    grads = make([1000, 50], "bf")
    grads[0][3] = float("inf")
    norm, factor = lce.clip_grad_norm([t.clone() for t in grads], 1.0, return_factor=True)
    assert norm.item() == float("inf") and factor.item() == 0.0
    grads[1][2] = float("nan")
    norm, factor = lce.clip_grad_norm(grads, 1.0, return_factor=True)
    assert norm.isnan() and factor.isnan() and bool(grads[1].isnan().all())


def test_zero_gradients_and_large_values():
    z = [torch.zeros(100, device="cuda")]
    norm, factor = lce.clip_grad_norm(z, 1.0, return_factor=True)
    assert norm.item() == 0.0 and factor.item() == 1.0
    big = [torch.full((1 << 20,), 1e18, device="cuda")]
    assert abs(lce.grad_norm(big).item() / 1.024e21 - 1) < 1e-5


def test_more_than_32_bits_of_elements():
    n = (1 << 31) + 12345
    t = torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16)
    norm = lce.clip_grad_norm([t], 1.0)
    assert abs(norm.item() / (0.5 * n ** 0.5) - 1) < 2.0 ** -18
    want = torch.tensor(0.5 * (1.0 / (0.5 * n ** 0.5))).bfloat16()
    assert torch.equal(t[-5:].cpu(), want.expand(5)) and torch.equal(t[:5].cpu(), want.expand(5))
    assert bool((t == t[0]).all())


def test_deterministic_stream_and_graph():
    grads = make([300_000, 77, 1_000_000], "bf")
    out = [torch.empty_like(t) for t in grads]
    a = lce.clip_grad_norm(grads, 0.1, out=out)
    first = [t.clone() for t in out]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = lce.clip_grad_norm(grads, 0.1, out=out, stream=s)
    torch.cuda.synchronize()
    assert a.item() == b.item() and all(torch.equal(x, y) for x, y in zip(first, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = lce.clip_grad_norm(grads, 0.1, out=out)
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert c.item() == a.item() and all(torch.equal(x, y) for x, y in zip(first, out))


def test_refusals():
    g = make([10, 20], "bf")
    for bad in (lambda: lce.grad_norm([]), lambda: lce.grad_norm([g[0].cpu()]), lambda: lce.grad_norm([g[0].half()]),
                lambda: lce.grad_norm([torch.zeros(4, 4, device="cuda").t()[:, ::2]]),
                lambda: lce.clip_grad_norm(g, 1.0, out=g[:1]), lambda: lce.clip_grad_norm(g, 1.0, out=[g[1], g[0]])):
        with pytest.raises(ValueError):
            bad()
    for m, eps in ((-1.0, 1e-6), (float("nan"), 1e-6), (1.0, -1.0)):
        with pytest.raises(lce.LceError):
            lce.clip_grad_norm(g, m, eps=eps)
    with pytest.raises(lce.LceError):
        lce.grad_norm(g, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert lce.clip_workspace_size(2) > 0
