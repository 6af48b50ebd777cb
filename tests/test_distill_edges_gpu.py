"""Distillation where the student gives next to nothing off the teacher's list: the mass there is far
below what fp32 holds relative to the largest logit, or zero. Against the 64-bit reference, with its
bounds; exponentials below 2^-126 are 0, of which a coefficient of at most 2^16 makes 2^-110."""
import numpy as np
import pytest

import _vocab_ref as R
from test_vocab_gpu import DTYPES, V, close, dev, f64  # noqa: F401 (V is a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def lists(rng, N, n_vocab, K, tau, rest):
    """Teachers with `rest` of their mass off the list: ids, logits, log-sum-exp of the whole."""
    ids = np.stack([rng.choice(n_vocab, K, replace=False) for _ in range(N)])
    t = rng.normal(0, 1, (N, K)).astype(np.float32)
    lse = (np.log(np.exp(t.astype(float) / tau).sum(-1)) - np.log1p(-rest)).astype(np.float32)
    return ids, t, lse


def coefficient(st, ref, tol):
    """stats[:, 2] is the coefficient, or the binary logarithm of r / u where that is above 2^64."""
    for got, want, d in zip(st, ref, tol):
        if got > 1:
            lg = np.log2(-want)
            assert want < -2.0 ** 63.9 and abs(got - lg) <= 1.4427 * d / -want * 1.01 + 4 * R.U * lg, (got, want, d)
        else:
            assert want > -2.0 ** 64.1 and abs(got - want) <= d, (got, want, d)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap,tau", [(20, 1.0), (60, 1.0), (90, 1.0), (100, 1.0), (200, 1.0), (600, 1.0), (14, 0.1),
                                     (30, 0.25), (600, 5.0)])
@pytest.mark.parametrize("N,n_vocab,K", [(3, 2000, 16), (2, 50021, 40)])
def test_student_far_surer_of_the_list(V, dtype, gap, tau, N, n_vocab, K):
    rng = np.random.default_rng(gap + n_vocab)
    ids, t, lse = lists(rng, N, n_vocab, K, tau, 0.01)
    # off the list down to a tenth of the gap's scale; the largest off-list logit of a row varies
    x = rng.normal(0, 1, (N, n_vocab)) * tau
    x[np.arange(N)[:, None], ids] = gap + 0.25 * t
    z = dev(x, dtype)
    weight = rng.uniform(0.5, 2, N).astype(np.float32)
    ref = R.distill(f64(z), ids, t.astype(float), tau, lse.astype(float), weight.astype(float))
    assert np.isfinite(ref["loss"]).all()
    i_dev, t_dev, w_dev = dev(ids), dev(t), dev(weight)
    kw = dict(temperature=tau, teacher_lse=dev(lse))
    loss, stats = V.distill_forward(z, i_dev, t_dev, **kw)
    close(f64(loss), ref["loss"], ref["loss_tol"])
    coefficient(f64(stats)[:, 2], ref["stats"][:, 2], ref["coef_tol"])
    tol = ref["grad_tol"] + R.rounding(ref["grad"], dtype) * 1.01 + (weight * tau * 2.0 ** -108)[:, None]
    loss2, g = V.distill_step(z, i_dev, t_dev, w_dev, **kw)
    close(f64(loss2), ref["loss"], ref["loss_tol"])
    close(f64(g), ref["grad"], tol)
    g = V.distill_backward(z, i_dev, t_dev, stats, w_dev, temperature=tau)
    close(f64(g), ref["grad"], tol)
    w = z.clone()
    assert torch.equal(V.distill_backward(w, i_dev, t_dev, stats, w_dev, temperature=tau, out=w), g)


@pytest.mark.parametrize("shape", ["listed", "masked"])
def test_nothing_finite_off_the_list_and_no_more_mass_there_than_rounding(V, shape):
    # The teacher's whole mass is on the list: 1 - (its sum) is a residue of rounding. Off the list is
    # nothing (the list holds the whole vocabulary), or nothing finite (the student masks it).
    rng = np.random.default_rng(7)
    K = 40
    n_vocab = K if shape == "listed" else 3001
    for tau in (1.0, 0.3, 2.0):
        ids = np.stack([rng.permutation(K) for _ in range(64)])
        t = rng.normal(5, 3, (64, K)).astype(np.float32)
        z = rng.normal(0, 2, (64, n_vocab))
        z[:, K:] = -np.inf
        z = dev(z, "float32")
        lse = np.log(np.exp(t.astype(float) / tau).sum(-1)).astype(np.float32)
        ones = np.ones(64, np.float32)
        ref = R.distill(f64(z), ids, t.astype(float), tau, None, ones.astype(float))
        kw = dict(temperature=tau, teacher_lse=dev(lse))
        loss, stats = V.distill_forward(z, dev(ids), dev(t), **kw)
        close(f64(loss), ref["loss"], ref["loss_tol"])
        assert (f64(stats)[:, 2] == 1).all()
        loss, g = V.distill_step(z, dev(ids), dev(t), **kw)
        close(f64(loss), ref["loss"], ref["loss_tol"])
        close(f64(g), ref["grad"], ref["grad_tol"] + R.rounding(ref["grad"], "float32"))
        g = V.distill_backward(z, dev(ids), dev(t), stats, temperature=tau)
        close(f64(g), ref["grad"], ref["grad_tol"] + R.rounding(ref["grad"], "float32"))


def test_teacher_mass_where_the_student_has_none(V):
    # the loss is infinite, the gradient is not: p - q on the list, 0 off it
    rng = np.random.default_rng(8)
    N, n_vocab, K = 5, 2000, 12
    ids, t, lse = lists(rng, N, n_vocab, K, 1.0, 0.1)
    x = np.full((N, n_vocab), -np.inf)
    x[np.arange(N)[:, None], ids] = rng.normal(0, 2, (N, K))
    z = dev(x, "float32")
    q = np.exp(t.astype(float) - lse.astype(float)[:, None])
    p = np.exp(np.take_along_axis(f64(z), ids, 1))
    want = np.zeros((N, n_vocab))
    np.put_along_axis(want, ids, p / p.sum(-1, keepdims=True) - q, 1)
    loss, stats = V.distill_forward(z, dev(ids), dev(t), teacher_lse=dev(lse))
    loss2, g = V.distill_step(z, dev(ids), dev(t), teacher_lse=dev(lse))
    assert (loss == float("inf")).all() and (loss2 == float("inf")).all()
    close(f64(g), want, 1e-5)
    close(f64(V.distill_backward(z, dev(ids), dev(t), stats)), want, 1e-5)
