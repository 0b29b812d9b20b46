"""Gradient norms of large values: every finite value whose norm fp32 can hold,
whichever way a list is summed (up to 1 MB one cluster takes it, beyond that
blocks of 64 KB), whole or starting between 16-byte boundaries.

Tolerances: fp32 sums of at most 130 squares, and of a warp's 32 lanes, before
fp64: below (130 + 5) * 2^-24 / 2 < 2^-17 relative in the norm, its own rounding
included; a factor of max_norm / norm has it once more with a division (2^-16),
and below 2^-126 its spacing is 2^-149. A clipped element is rounded once (2^-8
bf16, 2^-23 fp32)."""
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
FMAX = 3.4028234663852886e38


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    yield


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 40, 1000, 100_000, 600_001, 3_000_001])
@pytest.mark.parametrize("value", [1e17, 1e18, 1.5e19, 1e25, 1e34])
@pytest.mark.parametrize("start", [0, 3])
def test_large_values(value, n, dtype, start):
    t = torch.full((n + start,), value, device="cuda").to(DT[dtype])[start:]
    norm = t.double().square().sum().sqrt().item()
    assert norm < FMAX
    got, factor = lce.clip_grad_norm([t], 2.0, out=[out := torch.empty_like(t)], return_factor=True)
    assert abs(got.item() - norm) <= 2.0 ** -17 * norm
    assert abs(factor.item() - 2.0 / norm) <= 2.0 ** -16 * (2.0 / norm) + 2.0 ** -149
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    want = t.double() * factor.double()
    assert bool(((out.double() - want).abs() <= u * want.abs()).all())
    assert lce.grad_norm([t]).item() == got.item()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1000, 1_000_001])
def test_one_large_value_among_small_ones(n, dtype):
    t = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda").to(DT[dtype])
    t[n // 3] = 3e30
    norm = t.double().square().sum().sqrt().item()
    assert abs(lce.grad_norm([t]).item() - norm) <= 2.0 ** -17 * norm
    both = [t, torch.full((5,), 2.0, device="cuda"), torch.zeros(3, device="cuda")]
    assert abs(lce.grad_norm(both).item() - norm) <= 2.0 ** -17 * norm


@pytest.mark.parametrize("n", [64, 1_000_000])
def test_a_norm_beyond_fp32_is_infinite(n):
    t = torch.full((n,), 3e38, device="cuda")
    norm, factor = lce.clip_grad_norm([t], 1.0, return_factor=True)
    assert norm.item() == float("inf") and factor.item() == 0.0 and bool((t == 0).all())
    t = torch.full((n,), 1.0, device="cuda")
    for bad in (float("inf"), float("nan")):
        t[n // 2] = bad
        got = lce.grad_norm([t]).item()
        assert got == bad or got != got
    assert got != got
