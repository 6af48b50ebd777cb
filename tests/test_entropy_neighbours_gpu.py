"""A row's loss does not depend on which other rows of the batch take part, to the last bit."""
import pytest

from test_vocab_gpu import V  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,n_vocab,D", [(7, 500, 1000), (100, 500, 1000), (130, 700, 264), (400, 300, 2056), (700, 300, 1031),
                                         (1300, 300, 1000), (9000, 100, 264)])
def test_losses(V, dtype, N, n_vocab, D):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(N)
    h = torch.randn((N, D), generator=g, device="cuda").to(dtype)
    t = (torch.randn((n_vocab, D), generator=g, device="cuda") * D ** -0.5).to(dtype)
    at = torch.randint(0, n_vocab, (N,), generator=g, device="cuda")
    loss, lse = V.cross_entropy_forward(h, t, at)
    step = V.cross_entropy_step(h, t, at)[0]
    for silent in (slice(0, 1), slice(1, None, 2), slice(0, None, 3), slice(3, N - 2)):
        some = at.clone()
        some[silent] = -1
        part = some >= 0
        a, b = V.cross_entropy_forward(h, t, some)
        c = V.cross_entropy_step(h, t, some)[0]
        assert torch.equal(a[part], loss[part]) and torch.equal(b[part], lse[part]) and torch.equal(c[part], step[part])
