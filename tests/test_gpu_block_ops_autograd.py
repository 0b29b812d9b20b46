"""What autograd is told of the block operators: tensors that they write in
place, and gradients that cannot be differentiated again."""
import pytest

torch = pytest.importorskip("torch")

import chunked_vocab_cross_gb300 as lce  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from chunked_vocab_cross_gb300.build import build
    build()
    yield


def rand(*s):
    return torch.randn(*s, device="cuda")


def test_given_outputs_count_as_written():
    """Every tensor that a caller hands in to be written has its version raised; inputs keep theirs."""
    x, b, w = rand(6, 64), rand(6, 64), rand(64)
    before = [t._version for t in (x, b, w)]
    out = torch.empty_like(x)
    lce.block_norm_forward(x, b, w_pre=w, out_r=out)
    assert out._version > 0 and [t._version for t in (x, b, w)] == before
    lce.block_norm_forward(x, b, w_pre=w, out_r=x)
    assert x._version > before[0] and b._version == before[1]

    q, k, v, do = rand(9, 2, 32), rand(9, 1, 32), rand(9, 1, 32), rand(9, 2, 32)
    out, grads = torch.empty_like(q), [torch.empty_like(t) for t in (q, k, v)]
    o, lse = lce.attention_forward(q, k, v, out=out)
    assert o is out and out._version > 0
    lce.attention_backward(do, q, k, v, o, lse, dq=grads[0], dk=grads[1], dv=grads[2])
    assert all(t._version > 0 for t in grads) and all(t._version == 0 for t in (q, k, v, do, lse))

    g = [rand(100), rand(7)]
    outs = [torch.empty_like(t) for t in g]
    lce.clip_grad_norm(g, 0.1, out=outs)
    lce.grad_norm(g)
    assert all(t._version == 0 for t in g) and all(t._version > 0 for t in outs)
    lce.clip_grad_norm(g, 0.1)
    assert all(t._version > 0 for t in g)
    with torch.inference_mode():   # tensors without versions
        z = rand(6, 64)
        lce.block_norm_forward(z, rand(6, 64), w_pre=rand(64), out_r=z)
        lce.clip_grad_norm([rand(5)], 0.1)


def test_a_saved_tensor_that_was_overwritten_is_an_error():
    x, w = rand(6, 64), rand(6, 64).requires_grad_(True)
    y = (x * w).sum()             # keeps x for the gradient of w
    lce.block_norm_forward(x, rand(6, 64), w_pre=rand(64), out_r=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    g = rand(50)
    y = (g * rand(50).requires_grad_(True)).sum()
    lce.clip_grad_norm([g], 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def calls():
    q, k, v = (rand(20, 2, 32).requires_grad_(True) for _ in range(3))
    W = rand(100, 64).requires_grad_(True)
    x, b, w = rand(6, 64).requires_grad_(True), rand(6, 64).requires_grad_(True), rand(64).requires_grad_(True)
    return {"attention": (q, lambda: lce.attention(q, k, v)), "block_norm": (b, lambda: lce.block_norm(x, b, w_post=w, w_pre=w)[1]),
            "norm alone": (x, lambda: lce.block_norm(x, w_pre=w)[1]),
            "linear_cross_entropy": (x, lambda: lce.linear_cross_entropy(x, W, torch.arange(6, device="cuda"))),
            "embedding": (W, lambda: lce.embedding(W, torch.arange(6, device="cuda")))}


@pytest.mark.parametrize("name", ["attention", "block_norm", "norm alone", "linear_cross_entropy", "embedding"])
def test_gradients_are_not_differentiated_again_without_a_word(name):
    """A penalty on a gradient: an error, not a gradient that lacks the penalty's terms."""
    leaf, call = calls()[name]
    (first,) = torch.autograd.grad(call().square().sum(), leaf)
    (grad,) = torch.autograd.grad(call().square().sum(), leaf, create_graph=True)
    assert grad.requires_grad
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.square().sum().backward()
    assert first.shape == grad.shape
