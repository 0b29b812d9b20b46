"""Attention of tensors in other memory orders than the ones it makes itself:
head by head, q, k and v interleaved by head, rows apart. The results are, bit
for bit, those of the same values token by token, so no tolerance is needed."""
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


def head_major(t):
    T, H, D = t.shape
    return torch.full((H, T, D), 7.0, device="cuda", dtype=t.dtype).transpose(0, 1)


def interleaved(t):
    T, H, D = t.shape
    return torch.full((T, H, 3, D), 7.0, device="cuda", dtype=t.dtype)[:, :, 1]


def apart(t):
    T, H, D = t.shape
    return torch.full((T, 2 * H + 1, D + 8), 7.0, device="cuda", dtype=t.dtype)[:, 1::2, 8:][:, :H]


def gaps(t):
    """Heads in the gaps that the tokens leave: token stride 2 rows, the next head an odd number of rows on."""
    T, H, D = t.shape
    if H > 2:
        return head_major(t)
    flat = torch.full(((4 * T + 4) * D,), 7.0, device="cuda", dtype=t.dtype)
    return flat.as_strided((T, H, D), (2 * D, (2 * T - 1) * D if T > 1 else D, 1))


LAYOUTS = {"head major": head_major, "interleaved": interleaved, "apart": apart, "gaps": gaps}


@pytest.mark.parametrize("layout", list(LAYOUTS), ids=lambda s: s.replace(" ", "_"))
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,D", [((2, 1), 64), ((8, 2), 128), ((3, 3), 72)], ids=lambda v: str(v))
@pytest.mark.parametrize("lq,lk", [([130, 1, 60], [130, 1, 60]), ([40, 200], [300, 90]), ([2], [3000]), ([1500], [1500])], ids=lambda v: "_".join(map(str, v)))
def test_layouts(layout, dtype, heads, D, lq, lk):
    if dtype == "fp32" and max(lk) > 1000:
        return
    H, Hk = heads
    place = LAYOUTS[layout]
    g = torch.Generator(device="cuda").manual_seed(len(lq) + D)
    plain = [torch.randn(sum(n), h, D, generator=g, device="cuda").to(DT[dtype]) for n, h in ((lq, H), (lk, Hk), (lk, Hk), (lq, H))]
    other = []
    for t in plain:
        other.append(place(t))
        other[-1].copy_(t)
    cu = [torch.tensor([0] + n, device="cuda").cumsum(0).to(torch.int32) for n in (lq, lk)]
    q, k, v, do = plain
    o, lse = lce.attention_forward(q, k, v, *cu)
    grads = lce.attention_backward(do, q, k, v, o, lse, *cu)
    q2, k2, v2, do2 = other
    out = place(q)
    o2, lse2 = lce.attention_forward(q2, k2, v2, *cu, out=out)
    assert o2 is out and torch.equal(o, o2) and torch.equal(lse, lse2)
    outs = [place(t) for t in (q, k, v)]
    lce.attention_backward(do2, q2, k2, v2, o2, lse2, *cu, dq=outs[0], dk=outs[1], dv=outs[2])
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))
    # what lies between the rows stays
    for t in (out, *outs):
        whole = torch.empty(0, dtype=t.dtype, device="cuda").set_(t.untyped_storage())
        mask = torch.zeros(whole.numel(), dtype=torch.bool, device="cuda")
        mask.as_strided(t.shape, t.stride(), t.storage_offset()).fill_(True)
        assert bool((whole[~mask] == 7.0).all())
    assert lce.device_status() == 0


def test_transposed_batch():
    """[B, heads, L, D] seen as [B, L, heads, D]: one sequence is taken as it lies; several are not evenly spaced and refused."""
    x = torch.randn(2, 4, 100, 64, device="cuda").bfloat16()
    one = x[:1].transpose(1, 2)
    a, b = lce.attention_forward(one, one, one), lce.attention_forward(*(one.contiguous(),) * 3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError, match="evenly spaced"):
        lce.attention_forward(*(x.transpose(1, 2),) * 3)
