"""Seeded random calls of the recurrent block's operators against the fp64
references, with the tolerances of their own tests, and calls that run at once
on several streams."""
import random

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402
import test_gpu_layer_norm as norms  # noqa: E402
import test_gpu_packed as packed  # noqa: E402
import test_gpu_recurrence as recurrence  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    lce.device_status()
    yield


def log(rng, lo, hi):
    return int(round(2 ** rng.uniform(np.log2(lo), np.log2(hi))))


@pytest.mark.parametrize("seed", range(40))
def test_layer_norm(seed):
    rng = random.Random(seed)
    d = 8 * log(rng, 1, 2048 if rng.random() < 0.3 else 640)
    N = log(rng, 1, min(30000, 6_000_000 // d))
    norms.check(N, d, rng.choice(["bf16", "fp32"]), add=rng.random() < 0.6, bias=rng.random() < 0.7, more=rng.random() < 0.7,
                keep8=rng.random() < 0.5, seed=seed, wide=rng.choice([0, 0, 8, 40]), shift=rng.choice([0.0, 0.5, 30.0]))
    assert lce.device_status() == 0


@pytest.mark.parametrize("seed", range(30))
def test_pack(seed):
    rng = random.Random(100 + seed)
    d = 8 * log(rng, 1, 1500)
    packed.check_pack(packed.values(log(rng, 1, min(4000, 2_000_000 // d)), d, rng.choice(["bf16", "fp32"]), seed=seed,
                                    wide=rng.choice([0, 0, 8, 56])))


@pytest.mark.parametrize("seed", range(40))
def test_weight_gradient(seed):
    rng = random.Random(200 + seed)
    T, n, k = log(rng, 1, 8000), 8 * log(rng, 1, 300), 8 * log(rng, 1, 300)
    while T * n * k > 4e9:
        T = max(1, T // 2)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    dy, p, got = packed.check_wgrad(T, n, k, dtype, rng.choice([dtype, "fp32"]), seed=seed, wide=rng.choice([0, 0, 8, 64]))
    need = lce.packed_weight_grad_workspace_size(T, n, k, dy.dtype, got.dtype)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    again = lce.packed_weight_grad(dy, p, out_dtype=got.dtype, workspace=ws[:need] if need else None)
    assert torch.equal(again, got) and bool((ws[need:] == 77).all())


@pytest.mark.parametrize("seed", range(50))
def test_recurrence(seed):
    rng = random.Random(300 + seed)
    d = 8 * log(rng, 1, 150)
    most = max(2, min(6000, 600_000 // d))
    if rng.random() < 0.25:
        L = rng.choice([1, 1, 2, log(rng, 1, most)])
        lens, equal, tail = [L] * max(1, min(most // L, log(rng, 1, 300))), True, 0
    else:
        lens = [rng.choice([0, 1, log(rng, 1, most), log(rng, 1, 200)]) for _ in range(log(rng, 1, 60))]
        while sum(lens) > 2 * most:
            lens.pop()
        lens, equal, tail = lens or [0], False, rng.choice([0, 0, 1, 200])
    recurrence.check(lens, d, rng.choice(["bf16", "fp32"]), tail=tail, state=rng.random() < 0.5, equal=equal, seed=seed,
                     slices=rng.random() < 0.7, gates=rng.choice([(2.0, 1.5), (0.0, 1.0), (-3.0, 3.0), (6.0, 2.0)]))


def test_calls_at_once_on_several_streams():
    """The same calls one after the other and side by side: the same bits."""
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    sets = [(r(3000, 512), r(3000, 512), r(512), r(3000, 1024), r(3000, 256)) for _ in range(4)]
    cu = torch.tensor([0, 700, 700, 2950], dtype=torch.int32, device="cuda")

    def calls(x, dn, w, xg, dy):
        _, n, mean, rstd, kept = lce.layer_norm_forward(x, weight=w, keep8=True)
        dx, dw, dc = lce.layer_norm_backward(None, dn, kept, weight=w, mean=mean, rstd=rstd)
        h, final, states = lce.gated_recurrence_forward(xg[:, :512], xg[:, 512:], cu, keep=True)
        a, b, _ = lce.gated_recurrence_backward(x, xg[:, :512], xg[:, 512:], states, cu)
        return n, dx, dw, dc, h, final, a, b, lce.packed_weight_grad(dy, kept)

    want = [calls(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, stream in zip(sets, streams):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                got.append(calls(*s))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, b in zip(got, want) for x, y in zip(a, b))
    assert lce.device_status() == 0
