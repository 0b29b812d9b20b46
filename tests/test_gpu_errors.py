"""An error that a call returns is that call's alone: neither the library's next
call nor the program's own next use of CUDA meets it again."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402
from chunked_vocab_cross_gb300 import _abi  # noqa: E402

pytestmark = pytest.mark.gpu
LCE_ERR_CUDA, OUT_OF_MEMORY = 5, 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    yield


def attention_args(t):
    """Row statistics of more bytes than any memory has: the call ends where its scratch is refused, before a launch."""
    a = _abi.LceAttn()
    a.causal, a.scale = 1, 0.125
    a.B, a.Tq, a.Tk, a.Hq, a.Hk, a.D = 1, (1 << 30) - 1, 1, 4096, 1, 64
    for n in ("q", "k", "v", "o", "dO", "dq", "dk", "dv"):
        setattr(a, n, t.data_ptr())
        setattr(a, n + "_ts", 4096 * 64)
        setattr(a, n + "_hs", 64)
    a.lse = t.data_ptr()
    return a


def loss_args(t):
    a = _abi.LceArgs()
    a.H = a.W = a.targets = a.loss = a.dH = a.dW = t.data_ptr()
    a.ignore_index = -100
    a.N, a.d, a.V = (1 << 30), 16384, 1 << 20
    return a


@pytest.mark.parametrize("entry", ["lce_attention_backward", "lce_run"])
def test_scratch_that_cannot_be_had(entry):
    t = torch.zeros(1 << 20, device="cuda")
    args = attention_args(t) if entry == "lce_attention_backward" else loss_args(t)
    size = _abi.lib().lce_attention_workspace_size if entry == "lce_attention_backward" else _abi.lib().lce_workspace_size_args
    if size(ctypes.byref(args)) < 1 << 42:
        pytest.fail("not more than any memory has")
    launches = lce.launch_count()
    assert getattr(_abi.lib(), entry)(ctypes.byref(args)) == LCE_ERR_CUDA
    assert _abi.lib().lce_last_cuda_error() == OUT_OF_MEMORY and lce.launch_count() == launches
    # the next calls are whole
    assert lce.grad_norm([torch.ones(16, device="cuda")]).item() == 4.0
    assert float((torch.ones(8, device="cuda") + 1).sum()) == 16.0
    torch.cuda.synchronize()
