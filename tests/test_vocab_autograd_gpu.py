"""The vocabulary operators beside autograd: what it cannot differentiate or see is refused."""
import pytest

from test_vocab_gpu import V  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def rows(N=4, n_vocab=500, K=6):
    g = torch.Generator(device="cuda").manual_seed(2)
    z = torch.randn((N, n_vocab), generator=g, device="cuda")
    ids = torch.argsort(torch.rand((N, n_vocab), generator=g, device="cuda"), -1)[:, :K].contiguous()
    return z, ids, torch.randn((N, K), generator=g, device="cuda")


def test_second_derivatives_of_the_loss_are_refused(V):
    z, ids, t = rows()
    x = z.clone().requires_grad_()
    (g,) = torch.autograd.grad(V.distill_loss(x, ids, t).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        ((g * g).sum() + x.sum()).backward()
    x.grad = None
    V.distill_loss(x, ids, t).sum().backward()
    assert torch.equal(x.grad, g.detach())
