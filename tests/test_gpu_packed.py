"""Activations in 8 bits and the weight gradient from them, against the fp64
reference: codes, exponents and what they stand for bit for bit; the gradient
within a rounding of its type (u = half a step: 2^-8 for bf16, 2^-24 for fp32)
and, for fp32 sums of T products taken in any order, T + 64 roundings of 2^-23
of the absolute sum (a tensor core's sums are truncated, so a whole step)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402
from oracle import recurrent_oracle as ro  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    lce.device_status()
    yield


def f64(t):
    return t.detach().double().cpu().numpy()


def values(N, d, dtype, seed=0, wide=0):
    """Channels of very different sizes, zeros, and rows of one block only."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, d + wide, generator=g, device="cuda") * torch.exp(3 * torch.randn(d + wide, generator=g, device="cuda"))
    x = x * (torch.rand(N, d + wide, generator=g, device="cuda") > 0.1)
    return x.to(DT[dtype])[:, :d]


def check_pack(x):
    p = lce.pack_activation(x)
    codes, exps = ro.pack(f64(x))
    assert p.shape == x.shape and p.dtype == x.dtype
    assert np.array_equal(p.exps.cpu().numpy(), exps)
    want = ro.unpack(codes, exps)
    bad = np.isnan(want)
    assert np.array_equal(p.codes.cpu().numpy()[~bad], codes[~bad])
    for dt in DT.values():
        back = f64(lce.unpack_activation(p, dtype=dt))
        assert np.array_equal(back, want, equal_nan=True)
    assert lce.unpack_activation(p).dtype == x.dtype
    return p


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 8), (1, 4096), (3, 128), (5, 136), (17, 264), (64, 1000), (33, 2048), (2, 20000), (3001, 120)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_pack_and_back(shape, dtype):
    check_pack(values(*shape, dtype))
    check_pack(values(*shape, dtype, seed=1, wide=24))


def test_edges_of_the_format():
    x = torch.zeros(16, 256, device="cuda")
    x[0, 0], x[0, 1] = 448.0, 1.0                       # the largest value fits at scale 1
    x[1, 0], x[1, 1] = 448.0001, 464.0                  # just does not: the next scale
    x[2, :3] = torch.tensor([1.0, 1.0625, 1.1875])      # ties to even
    x[3, :3] = torch.tensor([448.0, 2.0 ** -10, 3 * 2.0 ** -10])   # half of the smallest code, and a tie above it
    x[4, 0], x[5, 200], x[6, 3] = float("inf"), float("nan"), float("-inf")
    x[7, 0], x[7, 130] = 3.4028234e38, -3.4028234e38    # saturate
    x[8, 0] = 1e-45                                      # below the smallest scale
    x[9, 0], x[9, 1] = 448 * 2.0 ** -100, 1e-33
    x[10] = -0.0
    x[11, 0], x[11, 1] = 2.0 ** -126, 2.0 ** -110
    check_pack(x)
    back = lce.unpack_activation(check_pack(x))
    assert back[4, :128].isnan().all() and not back[4, 128:].isnan().any() and back[7, 0] == 448 * 2.0 ** 119


def test_rows_and_outputs_that_are_slices():
    x = values(50, 296, "bf16", wide=40)
    p = check_pack(x)
    out = torch.full((50, 320), 7.0, dtype=torch.bfloat16, device="cuda")
    got = lce.unpack_activation(p, out=out[:, :296])
    assert torch.equal(got, lce.unpack_activation(p)) and bool((out[:, 296:] == 7).all()) and out._version > 0
    codes = torch.full((50, 304), 1, dtype=torch.uint8, device="cuda")
    codes[:, :296] = p.codes
    q = lce.PackedActivation(codes[:, :296], p.exps.clone(memory_format=torch.preserve_format), p.dtype)
    assert torch.equal(lce.unpack_activation(q), got)
    assert lce.unpack_activation(lce.pack_activation(x[:0])).shape == (0, 296)
    e = torch.randn(1, 64, device="cuda").expand(9, 64)
    assert torch.equal(lce.unpack_activation(lce.pack_activation(e)), lce.unpack_activation(lce.pack_activation(e.contiguous())))


def check_wgrad(T, n, k, dtype, out_dtype=None, seed=0, wide=0, exact=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dy = torch.randn(T, n + wide, generator=g, device="cuda").to(DT[dtype])[:, :n]
    x = values(T, k, dtype, seed=seed + 1)
    p = lce.pack_activation(x)
    out_dtype = dtype if out_dtype is None else out_dtype
    got = lce.packed_weight_grad(dy, p, out_dtype=DT[out_dtype])
    again = lce.packed_weight_grad(dy, p, out_dtype=DT[out_dtype])
    assert got.dtype == DT[out_dtype] and torch.equal(got, again)
    xh, y = f64(lce.unpack_activation(p, dtype=torch.float32)), f64(dy)
    want, terms = y.T @ xh, np.abs(y).T @ np.abs(xh)
    err, tol = np.abs(f64(got) - want), U[out_dtype] * np.abs(want) + (T + 64) * 2.0 ** -23 * terms
    assert np.all(err <= tol), (float(err.max()), float((err - tol).max()))
    # the sums' errors together, as roundings that do not conspire: far below a step of the largest terms
    rms = np.sqrt(np.mean(np.where(terms > 0, err - U[out_dtype] * np.abs(want), 0).clip(0) ** 2)) / max(np.sqrt(np.mean(terms ** 2)), 1e-30)
    assert rms <= 2.0 ** -19, rms
    assert lce.device_status() == 0
    return dy, p, got


SIZES = [(1, 8, 8), (2, 16, 128), (63, 128, 128), (64, 256, 256), (65, 264, 136), (200, 8, 1000), (129, 520, 72), (1000, 384, 264),
         (1213, 256, 200), (4097, 136, 392), (300, 1032, 1160), (9000, 64, 64)]


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_weight_gradient(size, dtype, out_dtype):
    check_wgrad(*size, dtype, out_dtype)


@pytest.mark.parametrize("size", [(512, 4096, 4096), (769, 4104, 2568), (2048, 2304, 4096)], ids=lambda s: "x".join(map(str, s)))
def test_weight_gradient_of_more_tiles_than_run_at_once(size):
    """A tile's output beside the next one's steps, again and again: the same bits each time."""
    dy, p, got = check_wgrad(*size, "bf16", "fp32")
    for _ in range(20):
        assert torch.equal(lce.packed_weight_grad(dy, p, out_dtype=torch.float32), got)
    if size[0] < 1000:
        check_wgrad(*size, "fp32")


def test_fp32_weight_gradient_of_many_tokens_that_all_add_up():
    """Where every term is positive, each truncated addition of the tensor cores loses in one direction. A run of 512 tokens has
    32 additions of 16 products, each off by at most two steps of 2^-23 of a sum that is half filled on average: 2^-18. The
    16 runs are added up with roundings of 2^-24 of what there is by then."""
    T, n, k = 8192, 1024, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    dy, p = torch.rand(T, n, generator=g, device="cuda"), lce.pack_activation(torch.rand(T, k, generator=g, device="cuda"))
    want = dy.double().T @ lce.unpack_activation(p, dtype=torch.float32).double()
    got = lce.packed_weight_grad(dy, p)
    assert ((got.double() - want).abs() / want).max().item() <= 2.0 ** -18 + 16 * 2.0 ** -24
    assert torch.equal(lce.packed_weight_grad(dy, p), got)


def test_weight_gradient_of_slices_of_no_rows_and_into_a_given_tensor():
    dy, p, got = check_wgrad(500, 120, 264, "bf16", wide=40)
    out = torch.full((120 * 264 + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    view = out[:120 * 264].view(120, 264)
    assert lce.packed_weight_grad(dy, p, out=view) is view and torch.equal(view, got)
    assert bool((out[120 * 264:] == 5).all()) and out._version > 0
    zero = lce.packed_weight_grad(dy[:0], lce.pack_activation(torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")))
    assert zero.shape == (120, 264) and not zero.any()


def test_nothing_reaches_another_channel():
    """What is not finite stays in its rows of dw (dy) and in its block's columns (x)."""
    dy, x = torch.randn(300, 264, device="cuda").bfloat16(), torch.randn(300, 520, device="cuda").bfloat16()
    dy[7, 3], x[299, 130] = float("inf"), float("nan")
    got = lce.packed_weight_grad(dy, lce.pack_activation(x)).float()
    bad = torch.zeros(264, 520, dtype=torch.bool, device="cuda")
    bad[3], bad[:, 128:256] = True, True
    assert not bool((~got.isfinite())[~bad].any()) and bool(got[:, 128:256].isnan().all())


def test_scratch_streams_and_graphs():
    dy, x = torch.randn(3000, 256, device="cuda").bfloat16(), values(3000, 200, "bf16")
    p = lce.pack_activation(x)
    want = lce.packed_weight_grad(dy, p)
    need = lce.packed_weight_grad_workspace_size(3000, 256, 200)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = lce.packed_weight_grad(dy, p, workspace=ws[:need], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool((ws[need:] == 77).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = lce.pack_activation(x)
        got = lce.packed_weight_grad(dy, q)
        back = lce.unpack_activation(q)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(back, lce.unpack_activation(p))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_keep8(dtype):
    x = values(90, 136, dtype).contiguous().view(3, 30, 136).requires_grad_(True)
    w = torch.randn(72, 136, device="cuda").to(DT[dtype]).requires_grad_(True)
    y = lce.linear_keep8(x, w)
    assert torch.equal(y, torch.nn.functional.linear(x, w))
    dy = torch.randn(3, 30, 72, device="cuda").to(DT[dtype])
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert torch.equal(dx, dy @ w)
    p = lce.pack_activation(x.detach().view(90, 136))
    assert torch.equal(dw, lce.packed_weight_grad(dy.view(90, 72), p))
    y = lce.linear_keep8(x, w)
    (dw,) = torch.autograd.grad(y.sum(), w)   # an expanded gradient
    assert torch.equal(dw, lce.packed_weight_grad(torch.ones(90, 72, dtype=DT[dtype], device="cuda"), p))
    (dw,) = torch.autograd.grad(lce.linear_keep8(x, w).square().sum(), w, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dw.sum().backward()
