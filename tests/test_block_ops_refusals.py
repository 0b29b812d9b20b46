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
