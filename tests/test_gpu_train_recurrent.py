"""The recurrent example: its operators together, against the same model in
plain torch, with and without activations in 8 bits, and token by token."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import chunked_vocab_cross_gb300 as lce  # noqa: E402
import train_block  # noqa: E402
import train_recurrent  # noqa: E402

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
    W, d = p64["W"], model.d
    x = torch.where((tokens != train_block.PAD)[:, None], W[tokens], torch.zeros((), dtype=torch.float64, device=W.device))

    def norm(t, w, c):
        t = t - t.mean(1, keepdim=True)
        return t * (t.pow(2).mean(1, keepdim=True) + 1e-5).rsqrt() * w + c

    n = norm(x, p64["w0"], p64["c0"])
    offsets = cu.tolist()
    for l in range(len(model.layers)):
        p = lambda name: p64[f"layers.{l}.{name}"]  # noqa: E731,B023
        xg = n @ p("xg").T
        a, v = torch.sigmoid(xg[:, d:]), torch.sigmoid(-xg[:, d:]) * xg[:, :d]
        rows = []
        for lo, hi in zip(offsets, offsets[1:]):
            h = torch.zeros(d, dtype=torch.float64, device=W.device)
            for t in range(lo, hi):
                h = a[t] * h + v[t]
                rows.append(h)
        h = torch.cat([torch.stack(rows), torch.zeros(tokens.numel() - offsets[-1], d, dtype=torch.float64, device=W.device)])
        x = x + h @ p("o").T
        n = norm(x, p("w1"), p("c1"))
        x = x + torch.nn.functional.gelu(n @ p("up").T) @ p("down").T
        n = norm(x, p("w2"), p("c2"))
    loss = torch.nn.functional.cross_entropy(n @ W.T, targets, ignore_index=train_block.IGNORE)
    loss.backward()
    return loss.item(), {k: v.grad for k, v in p64.items()}


def _grads(keep8, data, dtype=torch.float32):
    model = train_recurrent.Decoder(300, dtype=dtype, keep8=keep8)
    loss = model(*data)
    loss.backward()
    return model, loss, {k: p.grad.double() for k, p in model.named_parameters()}


def test_gradients_against_plain_torch():
    """fp32 model, one batch: the loss and every gradient. The head's split-bf16
    products are good to about 2^-16 of a logit, the rest to fp32's rounding over
    sums of at most a few thousand terms; 1e-3 of each gradient's norm leaves a
    factor of ten over either. With activations in 8 bits the forward is the same
    bit for bit; a value kept is off by half a step of four bits, 2^-4 / sqrt(3)
    of itself in the root mean square at most, independently of the others, and
    so is a sum of products with them; 0.15 of a gradient's norm leaves a factor
    of four for sums whose terms partly cancel."""
    data = train_block.batch(torch.Generator().manual_seed(5), 300, tokens=700)
    model, loss, got = _grads(False, data)
    want, grads = _plain(model, *data)
    assert abs(loss.item() - want) <= 1e-3
    for name, g in got.items():
        err = (g - grads[name]).norm() / grads[name].norm()
        assert err <= 1e-3, (name, err.item())
    _, loss8, got8 = _grads(True, data)
    assert loss8.item() == loss.item()
    for name, g in got8.items():
        err = (g - got[name]).norm() / got[name].norm()
        assert err <= 0.15, (name, err.item())
    assert lce.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_training_runs(dtype):
    model, losses, norms = train_recurrent.train(4, dtype)
    assert all(map(math.isfinite, losses + norms)) and min(norms) > 0
    out = train_recurrent.generate(model, torch.tensor([[7, 42], [9, 3]], device="cuda"), 5)
    assert out.shape == (2, 5) and int(out.min()) >= 0 and int(out.max()) < 1000
    assert lce.device_status() == 0


def test_single_tokens_follow_the_sequence():
    """fp32: states handed from step to step give the head's input of the whole sequence."""
    model = train_recurrent.Decoder(300, dtype=torch.float32)
    tokens = torch.randint(1, 300, (3, 140), generator=torch.Generator().manual_seed(2)).cuda()
    with torch.no_grad():
        whole, last = model.hidden(tokens)
        n, states = model.hidden(tokens[:, :100])
        for i in range(100, 140):
            n, states = model.hidden(tokens[:, i:i + 1], states=states)
    # rounding differs by the order of sums alone: a few hundred fp32 roundings of values of order one to ten
    assert (n - whole.view(3, 140, -1)[:, -1]).abs().max() <= 1e-4
    assert all((a - b).abs().max() <= 1e-4 for a, b in zip(states, last))


def test_a_step_captured_in_a_graph():
    """Forward and backward of the recurrent block in one graph, replayed on new inputs."""
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda")).bfloat16()  # noqa: E731
    x, wx, wo, w = r(600, 256), r(512, 256) / 16, r(256, 256) / 16, r(256)
    cu = torch.tensor([0, 250, 250, 590], dtype=torch.int32, device="cuda")

    def step(x):
        res, n, mean, rstd, kept = lce.layer_norm_forward(x, weight=w, keep8=True)
        xg, p = n @ wx.T, lce.pack_activation(n)
        h, _, states = lce.gated_recurrence_forward(xg[:, :256], xg[:, 256:], cu, keep=True)
        y = h @ wo.T
        dh = y @ wo
        dxg = torch.empty_like(xg)
        lce.gated_recurrence_backward(dh, xg[:, :256], xg[:, 256:], states, cu, dx=dxg[:, :256], dg=dxg[:, 256:])
        dwx = lce.packed_weight_grad(dxg, p)
        dx, dw, dc = lce.layer_norm_backward(y, dxg @ wx, kept, weight=w, mean=mean, rstd=rstd)
        return y, dwx, dx, dw, dc

    step(x)
    static, graph = x.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(static)
    for seed in (1, 2):
        new = torch.randn(600, 256, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, step(new)))
    assert lce.device_status() == 0
