"""Every entry point refuses tensors that are not on the current device. One GPU
shows it by another answer to which device is current: nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402
from chunked_vocab_cross_gb300 import block_ops  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    yield


def entries():
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    q, k, v, do, lse = r(9, 2, 32), r(9, 1, 32), r(9, 1, 32), r(9, 2, 32), r(2, 9)
    x, b, w, rstd = r(6, 64), r(6, 64), r(64), r(6)
    H, W, t, rows = r(6, 64), r(100, 64), torch.arange(6, device="cuda"), r(6)
    return {
        "attention_forward": lambda: lce.attention_forward(q, k, v),
        "attention_backward": lambda: lce.attention_backward(do, q, k, v, q, lse),
        "block_norm_forward": lambda: lce.block_norm_forward(x, b, w_pre=w),
        "block_norm_backward": lambda: lce.block_norm_backward(x, b, x, b, w_pre=w, rstd_pre=rstd),
        "grad_norm": lambda: lce.grad_norm([x, w]),
        "clip_grad_norm": lambda: lce.clip_grad_norm([x.clone()], 1.0),
        "lce_forward": lambda: lce.lce_forward(H, W, t),
        "lce_forward_backward": lambda: lce.lce_forward_backward(H, W, t),
        "lce_backward": lambda: lce.lce_backward(H, W, t, rows),
        "lce_compact": lambda: lce.lce_compact(t),
        "embedding_forward": lambda: lce.embedding_forward(W, t),
        "embedding_backward": lambda: lce.embedding_backward(H, t, 0, 100),
        "step": lambda: lce.FusedOptimizer(W.clone()).step(H, t),
    }


@pytest.mark.parametrize("name", ["attention_forward", "attention_backward", "block_norm_forward", "block_norm_backward", "grad_norm",
                                  "clip_grad_norm", "lce_forward", "lce_forward_backward", "lce_backward", "lce_compact",
                                  "embedding_forward", "embedding_backward", "step"])
def test_refused_unless_current(name, monkeypatch):
    call = entries()[name]
    call()
    torch.cuda.synchronize()
    launches = lce.launch_count()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(block_ops, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        call()
    assert lce.launch_count() == launches
