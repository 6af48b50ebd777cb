"""Long sums of the cross entropy's gradients on the GPU. The tensor cores cut an accumulator towards zero at every 16
elements, by half a unit of its last place in the mean: at most 2^-24 of a sum that grows. Over n elements in one
accumulator a gradient therefore comes out up to n / 16 * 2^-24 too small. Rounding errors of single elements have no
direction; what all of a gradient lacks in common shows in its projection on the true one."""
import ctypes

import pytest

import _block_ref as R
from sparse_embedding_bag_gb300 import embbwd as E
from test_entropy_gpu import impatient  # noqa: F401 (a fixture)
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


@pytest.mark.parametrize("N,n_vocab,D", [(9000, 1200, 264), (300, 3000, 8256), (30, 5000, 8264)])
def test_long_sums_that_give_up(V, impatient, N, n_vocab, D):  # noqa: F811
    """As for short sums: an error bit, NaN where nothing was computed, and a GPU that carries on."""
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    f = impatient.emb_cross_entropy_step
    f.argtypes = [i32, vp, i32, i64, i64, vp, i64, i32, i32, vp, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp]
    g = torch.Generator(device="cuda").manual_seed(N)
    h = torch.randn((N, D), generator=g, device="cuda").half()
    t = (torch.randn((n_vocab, D), generator=g, device="cuda") * D ** -0.5).half()
    at = torch.randint(-1, n_vocab, (N,), generator=g, device="cuda")
    want = V.cross_entropy_step(h, t, at)
    need = E.emb_cross_entropy_workspace(0, N, n_vocab, D, t, D, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    gave_up = 0
    for _ in range(3):
        loss, dh, dt = torch.full((N,), 7.0, device="cuda"), torch.full_like(h, 7.0), torch.full_like(t, 7.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert f(0, h.data_ptr(), E.EMB_F16, D, N, t.data_ptr(), D, n_vocab, D, at.data_ptr(), None, loss.data_ptr(),
                 dh.data_ptr(), D, dt.data_ptr(), D, ws.data_ptr(), need, status.data_ptr(),
                 torch.cuda.current_stream().cuda_stream) == 0
        missing = 0
        for got, right in zip((loss, dh, dt), want):
            nan = got.isnan()
            missing += nan.sum().item()
            assert torch.equal(torch.where(nan, right, got), right)
        assert status.item() in (0, 4) and (missing > 0) <= (status.item() == 4)
        gave_up += status.item() == 4
    assert gave_up
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(V.cross_entropy_step(h, t, at, status=status), want)) and status.item() == 0
