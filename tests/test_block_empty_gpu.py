"""Batches without rows, through the operators from the last block to the loss and their gradients."""
import pytest

from test_vocab_gpu import V  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_norm(V):  # noqa: F811
    x, r = torch.empty((0, 40), device="cuda"), torch.empty((0, 40), device="cuda")
    y, total, rstd = V.rms_norm_forward(x, residual=r)
    assert total is not x and total is not r and y.shape == total.shape == (0, 40) and rstd.shape == (0,)
    assert V.rms_norm_forward(x)[1] is x
    into = torch.empty_like(x)
    assert V.rms_norm_forward(x, residual=r, sum_out=into)[1] is into
    x.requires_grad_()
    w = torch.ones(40, device="cuda", requires_grad=True)
    y, s = V.rms_norm(x, w, residual=r)
    (y.sum() + s.sum()).backward()
    assert x.grad.shape == (0, 40) and w.grad.shape == (40,) and not w.grad.any()


def test_dropout(V):  # noqa: F811
    x, r = (torch.empty((0, 40), device="cuda", requires_grad=True) for _ in range(2))
    V.dropout(x, 0.5, 1, residual=r).sum().backward()
    assert x.grad.shape == r.grad.shape == (0, 40)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_cross_entropy(V, dtype):  # noqa: F811
    h = torch.empty((0, 64), device="cuda", dtype=dtype, requires_grad=True)
    t = torch.randn((50, 64), device="cuda").to(dtype).requires_grad_()
    at, lse = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    for table in (t, t.detach()):  # both gradients, the hidden states' alone
        loss = V.cross_entropy_loss(h, table, at)
        assert loss.shape == (0,)
        h.grad = None
        loss.sum().backward()
        assert h.grad.shape == (0, 64)
    assert not t.grad.any()
    V.cross_entropy_loss(h.detach(), t, at).sum().backward()  # the table's alone
    assert not t.grad.any()
    dh, dt = V.cross_entropy_backward(h.detach(), t.detach(), at, lse, want_table=False)
    assert dh.shape == (0, 64) and dt is None
    with pytest.raises(ValueError):
        V.cross_entropy_backward(h.detach(), t.detach(), at, torch.empty(1, device="cuda"), want_table=False)


def test_broadcast_gradients_of_no_rows(V):  # noqa: F811
    """An expanded tensor without elements counts as contiguous and keeps its strides of zero."""
    none = torch.zeros((), device="cuda").expand(0, 40)
    assert none.contiguous().stride() == (0, 0)
    x, w = torch.empty((0, 40), device="cuda"), torch.ones(40, device="cuda")
    dx, dw = V.rms_norm_backward(none, x, w, torch.empty(0, device="cuda"), grad_sum=none)
    assert dx.shape == (0, 40) and not dw.any()
    assert V.dropout(none, 0.5, 1).shape == V.rms_norm_forward(none)[0].shape == (0, 40)
