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


def in_place(V):
    z, ids, t = rows()
    ones = torch.ones(4, device="cuda")
    _, stats = V.distill_forward(z, ids, t)
    one = (ids[:, 0].contiguous(), torch.arange(5, device="cuda"))
    m = V.micro_quantize(z)
    return {
        "process_logits": lambda out: V.process_logits(z, output=one, frequency=ones, out=out),
        "distill_step": lambda out: V.distill_step(z, ids, t, out=out),
        "distill_backward": lambda out: V.distill_backward(z, ids, t, stats, out=out),
        "micro_lookup": lambda out: V.micro_lookup(m, out=out),
        "micro_matmul": lambda out: V.micro_matmul(m, V.micro_quantize(torch.ones(500, 500, device="cuda")), out=out),
    }


@pytest.mark.parametrize("name", ["process_logits", "distill_step", "distill_backward", "micro_lookup", "micro_matmul"])
def test_autograd_sees_what_a_call_overwrites(V, name):
    call = in_place(V)[name]
    z, ids, t = rows()
    w = torch.empty_like(z)
    before = w._version
    call(w)
    assert w._version > before
    # a tensor saved for a backward
    x = z.clone().requires_grad_()
    y = x * 1.0
    loss = V.distill_loss(y, ids, t)
    with torch.no_grad():
        call(y)
    with pytest.raises(RuntimeError):
        loss.sum().backward()
    # a leaf that takes a gradient
    with pytest.raises(ValueError):
        call(x)
    assert torch.equal(x.detach(), z)
    with torch.no_grad():
        call(x)
    with torch.inference_mode():
        w = torch.empty_like(z)
        call(w)
    call(w)  # no versions there


def test_quantising_into_a_matrix_is_seen(V):
    z = rows()[0]
    m = V.micro_quantize(z)
    before = m.codes._version, m.scales._version
    V.micro_quantize(z, out=m)
    assert m.codes._version > before[0] and m.scales._version > before[1]
