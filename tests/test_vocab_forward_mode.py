"""Forward-mode derivatives of the vocabulary operators: dropout carries tangents, the other differentiable calls
refuse them. On the CPU with a stand-in for the compiled entry, and on the GPU."""
import pytest

torch = pytest.importorskip("torch")
fwAD = torch.autograd.forward_ad

from sparse_embedding_bag_gb300 import vocab  # noqa: E402


class Entry:
    """The compiled entry's dropout for tensors on the host: the mask is every third element."""

    def dropout(self, x, p, seed, call, residual, out):
        held = int(call)
        keep = (torch.arange(x.numel()).reshape(x.shape) + seed + held) % 3 > 0
        y = torch.where(keep, x.detach() / (1 - p), torch.zeros(()))
        return y if residual is None else y + residual.detach()


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def device(request, monkeypatch):
    if request.param == "cpu":
        monkeypatch.setattr(vocab, "_entry", Entry())
    return request.param


@pytest.mark.parametrize("held", [False, True])
def test_tangents_of_dropout(device, held):
    x, dx, r, dr = (torch.randn(5, 36, device=device) for _ in range(4))
    call = torch.tensor([4], device=device) if held else 4
    want = vocab.dropout(dx, 0.25, 7, call)
    for grad in (True, False):
        with torch.set_grad_enabled(grad), fwAD.dual_level():
            y = fwAD.unpack_dual(vocab.dropout(fwAD.make_dual(x, dx), 0.25, 7, call))
            assert torch.equal(y.primal, vocab.dropout(x, 0.25, 7, call)) and torch.equal(y.tangent, want)
            y = fwAD.unpack_dual(vocab.dropout(fwAD.make_dual(x, dx), 0.25, 7, call, residual=fwAD.make_dual(r, dr)))
            assert torch.equal(y.primal, vocab.dropout(x, 0.25, 7, call, residual=r))
            assert torch.equal(y.tangent, vocab.dropout(dx, 0.25, 7, call, residual=dr))
            y = fwAD.unpack_dual(vocab.dropout(x, 0.25, 7, call, residual=fwAD.make_dual(r, dr)))
            assert torch.equal(y.tangent, dr)
            y = fwAD.unpack_dual(vocab.dropout(fwAD.make_dual(x, dx), 0.25, 7, call, residual=r))
            assert torch.equal(y.tangent, want)
            # a tangent whose rows are the same memory; no tangent at all
            y = fwAD.unpack_dual(vocab.dropout(fwAD.make_dual(x, torch.ones(1, 36, device=device).expand(5, 36)), 0.25, 7, call))
            assert torch.equal(y.tangent, vocab.dropout(torch.ones(5, 36, device=device), 0.25, 7, call))
            assert fwAD.unpack_dual(vocab.dropout(x, 0.25, 7, call)).tangent is None


def test_forward_over_backward(device):
    x, dx, c = (torch.randn(5, 36, device=device) for _ in range(3))
    leaf = x.clone().requires_grad_()
    with fwAD.dual_level():
        y = vocab.dropout(fwAD.make_dual(leaf, dx), 0.25, 7)
        (g,) = torch.autograd.grad(y, leaf, fwAD.make_dual(c, dx))
        g = fwAD.unpack_dual(g)
    assert torch.equal(g.primal, vocab.dropout(c, 0.25, 7)) and torch.equal(g.tangent, vocab.dropout(dx, 0.25, 7))


@pytest.mark.gpu
def test_the_others_refuse_tangents():
    x = torch.randn(5, 64, device="cuda")
    h, t, at = x.half(), torch.randn(100, 64, device="cuda").half(), torch.arange(5, device="cuda")
    ids = torch.arange(4, device="cuda").repeat(5, 1)
    with fwAD.dual_level():
        for f in (lambda: vocab.rms_norm(fwAD.make_dual(x, x)),
                  lambda: vocab.cross_entropy_loss(fwAD.make_dual(h, h), t, at),
                  lambda: vocab.cross_entropy_loss(h, fwAD.make_dual(t, t), at),
                  lambda: vocab.distill_loss(fwAD.make_dual(x, x), ids, x[:, :4].contiguous())):
            with pytest.raises((RuntimeError, NotImplementedError)):
                f()
