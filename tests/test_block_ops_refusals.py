"""Refusals of the block operators that are decided on the host, without a GPU."""
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402


@pytest.mark.parametrize("given", ["w_post", "gate", "both"])
def test_block_norm_without_a_block_output_has_no_gate_and_no_norm_of_it(given):
    """The autograd form refuses what block_norm_forward refuses, with the same words."""
    x, w = torch.zeros(4, 64), torch.ones(64)
    kw = {k: w for k in ("w_post", "gate") if given in (k, "both")}
    for call in (lce.block_norm, lambda x, **kw: lce.block_norm(x, None, **kw)):
        with pytest.raises(ValueError, match="without b there is only the norm by w_pre"):
            call(x, w_pre=w, **kw)
    with pytest.raises(ValueError, match="without b there is only the norm by w_pre"):
        lce.block_norm(x)


def test_tensors_of_another_device_than_the_current_one(monkeypatch):
    """Without a GPU: the lookup of the stream refuses before it asks for one."""
    from chunked_vocab_cross_gb300 import block_ops, ops

    class Stream:
        cuda_stream, device = 7, torch.device("cuda", 0)

    class Tensor:
        device = torch.device("cuda", 1)
        get_device = lambda self: 1  # noqa: E731

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(block_ops, "_current_device", lambda: 0)
    monkeypatch.setattr(block_ops, "_current_stream", lambda index: 7)
    assert block_ops._stream(0) == 7
    with pytest.raises(ValueError, match="current device"):
        block_ops._stream(1)
    for stream in (None, Stream()):
        with pytest.raises(ValueError, match="current one"):
            ops._stream(stream, Tensor())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current one"):   # a stream of the other device
        ops._stream(Stream(), Tensor())


def test_workspace_of_another_device():
    from chunked_vocab_cross_gb300 import block_ops

    class Workspace:
        device, is_cuda = torch.device("cuda", 1), True
        is_contiguous = lambda self: True  # noqa: E731
        data_ptr = lambda self: 4096  # noqa: E731
        numel = lambda self: 1 << 20  # noqa: E731
        element_size = lambda self: 1  # noqa: E731

    with pytest.raises(ValueError, match="workspace"):
        block_ops._scratch(Workspace(), 16, torch.device("cuda", 0))
    assert block_ops._scratch(Workspace(), 16, torch.device("cuda", 1))[:2] == (4096, 1 << 20)
