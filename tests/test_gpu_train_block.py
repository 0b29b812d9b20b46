"""The example decoder: its operators together, against the same model in plain
torch, and training."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import chunked_vocab_cross_gb300 as lce  # noqa: E402
import train_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    yield


def _plain(model, tokens, cu, targets):
    """The decoder in elementary fp64 torch operations."""
    p64 = {k: v.detach().double().requires_grad_(True) for k, v in model.named_parameters()}
    W = p64["W"]
    x = torch.where((tokens != train_block.PAD)[:, None], W[tokens], torch.zeros((), dtype=torch.float64, device=W.device))
    rms = lambda t, w: t * (t.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt() * w  # noqa: E731
    n = rms(x, p64["first"])
    T = tokens.numel()
    seq = torch.bucketize(torch.arange(T, device=W.device), cu[1:].long(), right=True)
    i = torch.arange(T, device=W.device)
    ok = (seq[:, None] == seq[None, :]) & (i[:, None] >= i[None, :]) & (seq[:, None] < cu.numel() - 1)
    for l in range(len(model.layers)):
        p = lambda name: p64[f"layers.{l}.{name}"]  # noqa: E731,B023
        h, hk, d = model.heads, model.kv_heads, model.head_dim
        qkv = (n @ p("qkv").T).unflatten(1, (-1, d))
        q, k, v = qkv.split([h, hk, hk], 1)
        k, v = (t.repeat_interleave(h // hk, 1) for t in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        a = torch.softmax(s.masked_fill(~ok, -1e300), -1) * ok
        b = torch.einsum("hij,jhd->ihd", a, v).flatten(1) @ p("o").T
        x = x + p("gate1") * rms(b, p("post1"))
        n = rms(x, p("pre1"))
        b = torch.nn.functional.gelu(n @ p("up").T) @ p("down").T
        x = x + p("gate2") * rms(b, p("post2"))
        n = rms(x, p("pre2"))
    loss = torch.nn.functional.cross_entropy(n @ W.T, targets, ignore_index=train_block.IGNORE)
    loss.backward()
    return loss.item(), {k: v.grad for k, v in p64.items()}


def test_gradients_against_plain_torch():
    """fp32 model, one batch: the loss and every gradient. The head's split-bf16
    products are good to about 2^-16 of a logit, the rest to fp32's rounding
    over sums of at most a few thousand terms; 1e-3 of each gradient's norm
    leaves a factor of ten over either."""
    g = torch.Generator().manual_seed(5)
    model = train_block.Decoder(300, dtype=torch.float32)
    data = train_block.batch(g, 300, tokens=700)
    loss = model(*data)
    loss.backward()
    want, grads = _plain(model, *data)
    assert abs(loss.item() - want) <= 1e-3
    for name, p in model.named_parameters():
        err = (p.grad.double() - grads[name]).norm() / grads[name].norm()
        assert err <= 1e-3, (name, err.item())
    assert lce.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_training_lowers_the_loss(dtype):
    losses, norms = train_block.train(40, dtype)
    assert all(map(math.isfinite, losses + norms)) and min(norms) > 0
    assert abs(losses[0] - math.log(1000)) < 1.5
    assert sum(losses[-5:]) / 5 < losses[0] - 1.0
    assert lce.device_status() == 0
