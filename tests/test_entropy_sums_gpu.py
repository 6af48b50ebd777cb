"""Long sums of the cross entropy's gradients on the GPU. The tensor cores cut an accumulator towards zero at every 16
elements, by half a unit of its last place in the mean: at most 2^-24 of a sum that grows. Over n elements in one
accumulator a gradient therefore comes out up to n / 16 * 2^-24 too small. Rounding errors of single elements have no
direction; what all of a gradient lacks in common shows in its projection on the true one."""
import pytest

import _block_ref as R
from test_vocab_gpu import V  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

EIGHTH = {torch.float16: 2.0 ** -14, torch.bfloat16: 2.0 ** -11}  # of the type's half step


def lacking(got, want):
    return 1 - ((got.double() * want).sum() / (want * want).sum()).item()


def noise(want, dtype, factors=None):
    """Six deviations of the projection's error from independent roundings of the outputs, and of G's elements, whose
    parts of the projection are `factors` (uniform within half a step: deviation below 0.58 half steps)."""
    total = (want ** 4).sum() + ((factors ** 2).sum() if factors is not None else 0)
    return 6 * 0.58 * R.HALF_STEP[dtype] * (total.sqrt() / (want * want).sum()).item()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_table_gradient_of_many_tokens(V, dtype):  # noqa: F811
    """Tokens of the table that are nobody's target: sums of positive products, which only grow."""
    N, n_vocab, D = 600000, 64, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    h = (1 + 0.25 * torch.randn((N, D), generator=g, device="cuda")).to(dtype)
    t = (torch.randn((n_vocab, D), generator=g, device="cuda") * 0.1).to(dtype)
    at = torch.randint(0, 8, (N,), generator=g, device="cuda")
    p = torch.softmax(h.double() @ t.double().T, -1)[:, 8:]
    want = p.T @ h.double()
    _, lse = V.cross_entropy_forward(h, t, at)
    both = V.cross_entropy_backward(h, t, at, lse)[1]
    alone = V.cross_entropy_backward(h, t, at, lse, want_hidden=False)[1]
    step = V.cross_entropy_step(h, t, at)[2]
    tol = EIGHTH[dtype] + noise(want, dtype, p * (h.double() @ want.T))
    for got in (both, alone, step):
        assert abs(lacking(got[8:], want)) <= tol
    assert torch.equal(both, alone)
    # a strided table, and rows that take no part between the others
    wide = torch.zeros((n_vocab, D + 3), device="cuda").to(dtype)
    V.cross_entropy_backward(h, t, at, lse, out_table=wide[:, 1:D + 1])
    assert torch.equal(wide[:, 1:D + 1], both) and not wide[:, 0].any() and not wide[:, D + 1:].any()
    at[::3] = -1
    part = at >= 0
    want = p[part].T @ h[part].double()
    got = V.cross_entropy_backward(h, t, at, lse)[1]
    assert abs(lacking(got[8:], want)) <= EIGHTH[dtype] + noise(want, dtype, p[part] * (h[part].double() @ want.T))


@pytest.mark.parametrize("N", [8, 130])
def test_hidden_gradient_over_a_long_vocabulary(V, N):  # noqa: F811
    """Rows of the table around a positive mean, the targets' rows zero: sums that only grow."""
    dtype, n_vocab, D = torch.float16, 150000, 8192
    g = torch.Generator(device="cuda").manual_seed(2)
    t = torch.empty((n_vocab, D), dtype=dtype, device="cuda").normal_(1.0, 0.25, generator=g)
    t[:4] = 0
    h = (torch.randn((N, D), generator=g, device="cuda") * 0.01).to(dtype)
    at = torch.randint(0, 4, (N,), generator=g, device="cuda")
    z = torch.cat([h.double() @ x.double().T for x in t.split(10000)], 1)
    p = torch.softmax(z, -1)
    want = sum(q @ x.double() for q, x in zip(p.split(10000, 1), t.split(10000)))
    _, lse = V.cross_entropy_forward(h, t, at)
    both = V.cross_entropy_backward(h, t, at, lse)[0]
    alone = V.cross_entropy_backward(h, t, at, lse, want_table=False)[0]
    dots = torch.cat([want @ x.double().T for x in t.split(10000)], 1)
    # fp16 has steps of 2^-24 under the scale that brings a weight of one to 2^14: 2^-38 of a probability
    small = (2.0 ** -39 * dots.abs()).sum().item() / (want * want).sum().item() / n_vocab ** 0.5 * 6
    tol = EIGHTH[dtype] + noise(want, dtype, p * dots) + small
    for got in (both, alone):
        assert abs(lacking(got, want)) <= tol


@pytest.mark.parametrize("N", [30, 300])
def test_logits_of_wide_rows(V, N):  # noqa: F811
    """Logits of 15 that are not the targets': what G takes of them is off by what their sums lack."""
    dtype, n_vocab, D = torch.float16, 2000, 32768
    g = torch.Generator(device="cuda").manual_seed(3)
    t = (torch.randn((n_vocab, D), generator=g, device="cuda") * 1.3 / D ** 0.5).to(dtype)
    at, other = (torch.randint(0, n_vocab, (N,), generator=g, device="cuda") for _ in range(2))
    h = (torch.randn((N, D), generator=g, device="cuda") + 15 / 1.69 * t[other].float()).to(dtype)
    z = h.double() @ t.double().T
    p = torch.softmax(z, -1)
    G = p.scatter_add(1, at[:, None], -torch.ones_like(p[:, :1]))
    lse = torch.logsumexp(z, -1).float()
    for w in (None, torch.rand(N, generator=g, device="cuda") + 0.5):
        dh, dt = V.cross_entropy_backward(h, t, at, lse, w)
        u = G if w is None else G * w.double()[:, None]
        a, b = u @ t.double(), u.T @ h.double()
        # sums of 2048 elements, 128 steps: at most 128 * 2^-24 of a logit of 15
        common = 128 * 2.0 ** -24 * 16 * 1.01
        assert abs(lacking(dh, a)) <= common + noise(a, dtype, u * (a @ t.double().T))
        assert abs(lacking(dt, b)) <= common + noise(b, dtype, u * (h.double() @ b.T))
