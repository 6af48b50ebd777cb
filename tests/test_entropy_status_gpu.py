"""Error bits of the differentiable cross entropy: targets beyond the table are reported, in the forward and the backward."""
import pytest

from test_vocab_gpu import V  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("N,n_vocab,D", [(5, 100, 64), (70, 300, 72), (300, 1000, 33)])
def test_targets_beyond_the_table(V, N, n_vocab, D):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(N)
    h = torch.randn((N, D), generator=g, device="cuda").half().requires_grad_()
    t = torch.randn((n_vocab, D), generator=g, device="cuda").half().requires_grad_()
    at = torch.randint(0, n_vocab, (N,), generator=g, device="cuda")
    at[1] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss = V.cross_entropy_loss(h, t, at, status=status)
    good = torch.autograd.grad(loss.sum(), (h, t))
    assert status.item() == 0 and torch.equal(loss, V.cross_entropy_loss(h, t, at))
    bad = at.clone()
    bad[0], bad[N - 1] = n_vocab, 1 << 40
    silent = at.clone()
    silent[0] = silent[N - 1] = -1
    loss = V.cross_entropy_loss(h, t, bad, status=status)
    assert status.item() == 1 and loss[0] == 0 and loss[N - 1] == 0
    status.zero_()  # between the two: the backward reports for itself, and the loss's history stands
    got = torch.autograd.grad(loss.sum(), (h, t))
    assert status.item() == 1
    want = torch.autograd.grad(V.cross_entropy_loss(h, t, silent).sum(), (h, t))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not torch.equal(got[0], good[0])
    with pytest.raises(ValueError):
        V.cross_entropy_loss(h, t, at, status=torch.zeros(2, dtype=torch.int32, device="cuda"))
