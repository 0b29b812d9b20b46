"""Attention where a whole side has no tokens, with and without offsets, over
the head sizes and layouts that choose each compiled form: zeros, lse = -inf,
zero gradients, and a clear status word. No arithmetic, so no tolerance."""
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    lce.device_status()
    yield


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,D", [((2, 1), 64), ((14, 2), 96), ((3, 3), 80), ((32, 8), 128)], ids=lambda v: str(v))
@pytest.mark.parametrize("B,lq,lk", [(1, 5, 0), (1, 0, 5), (3, 700, 0), (3, 0, 700), (2, 0, 0)])
@pytest.mark.parametrize("offsets", [False, True], ids=["batch", "packed"])
def test_one_side_empty(B, lq, lk, heads, D, dtype, offsets):
    H, Hk = heads
    r = lambda L, h: torch.randn(B, L, h, D, device="cuda").to(DT[dtype])  # noqa: E731
    q, k, v, do = r(lq, H), r(lk, Hk), r(lk, Hk), r(lq, H)
    cu = ()
    if offsets:
        q, k, v, do = (t.flatten(0, 1) for t in (q, k, v, do))
        cu = tuple(torch.arange(B + 1, device="cuda", dtype=torch.int32) * n for n in (lq, lk))
    for causal in (True, False):
        o, lse = lce.attention_forward(q, k, v, *cu, causal=causal)
        grads = lce.attention_backward(do, q, k, v, o, lse, *cu, causal=causal)
        torch.cuda.synchronize()
        assert lse.shape == (H, B * lq) and bool((lse == -float("inf")).all())
        assert all(bool((t == 0).all()) for t in (o, *grads))
        assert [t.shape for t in grads] == [q.shape, k.shape, v.shape]
    assert lce.device_status() == 0
