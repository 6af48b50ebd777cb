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
