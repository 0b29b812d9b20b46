"""Seeded random calls of the block operators against the fp64 references, with
the tolerances of their own tests: attention over sequences of any lengths and
head layouts (the lengths make every splitting rule choose both ways), norms of
any shape and options, lists of tensors for the norm of gradients."""
import random

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402
import test_gpu_attention as attention  # noqa: E402
import test_gpu_block_norm_ring as norms  # noqa: E402
import test_gpu_clip as clip  # noqa: E402

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


def attention_case(seed):
    rng = random.Random(seed)
    dtype = "bf16" if rng.random() < 0.8 else "fp32"
    Hk = rng.choice([1, 1, 2, 3, 5])
    H = Hk * rng.choice([1, 2, 3, 4, 7, 8] if Hk < 3 else [1, 2, 3])
    D = 8 * rng.randint(1, 16)
    n = log(rng, 1, 40)
    kind = rng.choice(["self", "self", "cross", "decode", "prefix", "empty"])
    most = 1200 // (1 + H // 4) if dtype == "bf16" else 300
    lq = [rng.choice([0, 1, log(rng, 1, most), log(rng, 1, most)]) for _ in range(max(1, n // 4) if n < 20 else n)]
    if len(lq) > 8:
        lq = [min(x, 60) for x in lq]
    lk = lq
    if kind == "cross":
        lk = [rng.choice([0, 1, x, x // 2, x + rng.randint(1, 300)]) for x in lq]
    elif kind == "decode":
        lq = [rng.choice([0, 1, 1, 1, 2]) for _ in lq]
        lk = [rng.choice([0, 1, log(rng, 1, 16000 // len(lq) + 2)]) for _ in lq]
    elif kind == "prefix":
        lk = [x + rng.choice([0, 64, 128, 1000]) for x in lq]
    elif kind == "empty":
        lk = [0 if rng.random() < 0.7 else x for x in lq]
    return dict(lq=lq, lk=lk, H=H, Hk=Hk, D=D, causal=rng.random() < 0.6, dtype=dtype, tail=rng.choice([0, 0, 3, 700]), seed=seed)


@pytest.mark.parametrize("seed", range(60))
def test_attention(seed):
    c = attention_case(seed)
    q, k, v, do, o, lse, grads = attention.check(**c)
    # the same again with scratch of the stated sizes, on another stream
    H, Hk, D, B = c["H"], c["Hk"], c["D"], len(c["lq"])
    cq, ck, dt = attention.cu(c["lq"]), attention.cu(c["lk"]), attention.DT[c["dtype"]]
    f = lce.attention_forward_workspace_size(len(q), len(k), H, Hk, D, B, dt, c["causal"])
    b = lce.attention_workspace_size(len(q), len(k), H, Hk, D, B, dt)
    guard = 4096
    ws = [torch.full((n + guard,), 77, dtype=torch.uint8, device="cuda") for n in (f, b)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, lse2 = lce.attention_forward(q, k, v, cq, ck, causal=c["causal"], workspace=ws[0][:f] if f else None, stream=s)
    grads2 = lce.attention_backward(do, q, k, v, o2, lse2, cq, ck, causal=c["causal"], workspace=ws[1][:b], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((o, lse, *grads), (o2, lse2, *grads2)))
    assert all(bool((w[n:] == 77).all()) for w, n in zip(ws, (f, b)))
    assert lce.device_status() == 0


def norm_case(seed):
    rng = random.Random(1000 + seed)
    dtype = rng.choice(["bf16", "fp32"])
    d = 8 * log(rng, 1, 2048 if rng.random() < 0.3 else 640)
    N = log(rng, 1, min(30000, 6_000_000 // d))
    post, gate, pre = rng.random() < 0.7, rng.choice(["none", "channel", "full"]), rng.random() < 0.8
    no_b = pre and rng.random() < 0.15
    return dict(N=N, d=d, dtype=dtype, post=post and not no_b, gate="none" if no_b else gate, pre=pre, scale=rng.choice([1.0, 0.3, -0.7]),
                wide=rng.choice([0, 0, 8, 40]), no_dr=pre and rng.random() < 0.3, no_b=no_b)


@pytest.mark.parametrize("seed", range(60))
def test_block_norm(seed):
    norms.check(**norm_case(seed))
    assert lce.device_status() == 0


@pytest.mark.parametrize("seed", range(30))
def test_clip(seed):
    rng = random.Random(2000 + seed)
    sizes = [rng.choice([0, 1, log(rng, 1, 300_000), log(rng, 1, 5000)]) for _ in range(log(rng, 1, 300))]
    grads = clip.make(sizes, rng.choice(["b", "f", "bf", "ffb"]), seed=seed, std=10.0 ** rng.uniform(-6, 6))
    if sum(sizes) == 0:
        return
    size = float(torch.stack([t.double().square().sum() for t in grads]).sum().sqrt())
    clip.check(grads, size * rng.choice([0.01, 0.5, 2.0]), eps=rng.choice([0.0, 1e-6]))
