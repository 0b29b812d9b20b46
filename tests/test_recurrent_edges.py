"""The recurrent block's operators without a GPU: layouts and refusals that no
kernel is needed for."""
import pytest

torch = pytest.importorskip("torch")

from chunked_vocab_cross_gb300 import recurrent_ops  # noqa: E402


@pytest.mark.parametrize("rows,n", [(1, 5), (1, 16), (1, 24), (2, 24), (3, 16), (3, 40), (0, 24)])
def test_rows_of_packed_activations_have_whole_16_bytes(rows, n):
    """Rows that the kernels read in pieces of 16 bytes lie inside their memory, wherever they came from."""
    wide = (n + 15) // 16 * 16
    exact = torch.arange(rows * n, dtype=torch.uint8).view(rows, n).clone()
    short = torch.empty(max(rows - 1, 0) * wide + n, dtype=torch.uint8).as_strided((rows, n), (wide, 1))   # the last row ends early
    short.copy_(exact)
    room = torch.zeros(rows, wide, dtype=torch.uint8)[:, :n]
    for t in (exact, short, room):
        got = recurrent_ops._on_16(t)
        assert torch.equal(got, t) and got.data_ptr() % 16 == 0
        assert rows < 2 or got.stride(0) % 16 == 0
        if rows:
            assert got.storage_offset() + (rows - 1) * got.stride(0) + wide <= got.untyped_storage().nbytes()
    assert recurrent_ops._on_16(room) is room


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_that_the_kernels_cannot_read_are_copied(dtype):
    base = torch.arange(4096).to(dtype)
    good = (base[:640].view(10, 64), base.view(16, 256)[:10, :64], base[:640].view(2, 5, 64), base[:64].view(1, 64), base[:0].view(0, 64))
    bad = (base[1:641].view(10, 64), base[:650].view(10, 65)[:, :64], base[:640].view(64, 10).t(), base[:64].expand(10, 64),
           base[:10].view(10, 1).expand(10, 64), base[:1280].view(10, 128)[:, ::2], base.as_strided((10, 64), (16, 1)), base[1:65].view(1, 64))
    for t in good:
        assert recurrent_ops._readable(t).data_ptr() == t.data_ptr()
    for t in bad:
        got = recurrent_ops._readable(t)
        assert got.is_contiguous() and got.data_ptr() != t.data_ptr() and got.data_ptr() % 16 == 0
    for t in good + bad:
        assert torch.equal(recurrent_ops._readable(t), t.reshape(-1, 64))
