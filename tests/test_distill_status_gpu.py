"""Error bits of the differentiable distillation loss."""
import pytest

from test_vocab_gpu import V  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_ids_beyond_the_vocabulary(V):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn((6, 200), generator=g, device="cuda").requires_grad_()
    teacher = torch.randn((6, 5), generator=g, device="cuda")
    ids = torch.stack([torch.randperm(200, generator=g, device="cuda")[:5] for _ in range(6)])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss = V.distill_loss(z, ids, teacher, status=status)
    loss.sum().backward()
    assert status.item() == 0 and torch.equal(loss, V.distill_loss(z, ids, teacher))
    ids[2, 3] = 200
    loss = V.distill_loss(z, ids, teacher, temperature=2.0, status=status)
    assert status.item() == 1
    status.zero_()
    (got,) = torch.autograd.grad(loss.sum(), z)
    assert status.item() == 1
    assert torch.equal(got, V.distill_step(z.detach(), ids, teacher, temperature=2.0)[1])
