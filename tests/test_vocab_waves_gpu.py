"""Launch shapes of real tables and batches: product CTAs that take several tiles, and the gradient's
largest pieces."""
import numpy as np
import pytest

import _vocab_ref as R
from test_vocab_gpu import V, close, codes_of, dev, f64  # noqa: F401 (V is a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(1, 66001, 300), (16, 80000, 96), (33, 66001, 520), (64, 70001, 1056), (100, 66001, 300),
                                   (128, 80000, 64), (129, 66001, 520), (300, 66001, 288)])
def test_product_of_several_tiles_a_cta(V, fmt, M, N, K):
    # at least three tiles for each of 152 CTAs of 128 table rows, or 76 pairs of 256: both
    # accumulators, the columns they share, and stages that run on from tile to tile
    rng = np.random.default_rng(M + N + K)
    gx, gw = (1.0, 1.0) if fmt == "mx" else (float(np.float32(6.5 / 2688)), float(np.float32(0.13 / 2688)))
    x = V.micro_quantize(dev(rng.normal(0, 1, (M, K)), "float32"), fmt, gx)
    w = V.micro_quantize(dev(rng.normal(0, 0.02, (N, K)), "float32"), fmt, gw)
    xv, wv = R.decode(*codes_of(x), M, K, fmt, gx)[0], R.decode(*codes_of(w), N, K, fmt, gw)[0]
    want, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    for out in ("float32", "bfloat16"):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = V.micro_matmul(x, w, dtype=getattr(torch, out), status=status)
        close(f64(got), want, (2 * K + 8) * R.U * mag + R.rounding(want, out) * 1.01)
        assert status.item() == 0
        for _ in range(3):
            assert torch.equal(V.micro_matmul(x, w, dtype=getattr(torch, out)), got)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("pad", [0, 8])
def test_gradient_in_the_largest_pieces(V, dtype, tail, pad):
    # pieces of 32768 elements: two a row
    rng = np.random.default_rng(21)
    N, n_vocab, K, tau = 800, 33001, 24, 1.5
    ids = rng.integers(0, n_vocab, (N, K))
    ids[:, -1] = rng.integers(32768, n_vocab, N)
    ids[3::7, K // 2:] = -1
    ids[5] = -1
    t = rng.normal(3, 2, (N, K)).astype(np.float32)
    z = torch.randn(N, n_vocab + pad, device="cuda").mul_(2).to(getattr(torch, dtype))[:, :n_vocab]
    weight = rng.uniform(0.5, 2, N).astype(np.float32)
    lse = None
    if tail:
        lse = (np.log(np.exp(np.where(ids >= 0, t / tau, -np.inf)).sum(-1) + 1e-9) + 0.2).astype(np.float32)
    kw = dict(temperature=tau)
    loss, stats = V.distill_forward(z, dev(ids), dev(t), teacher_lse=None if lse is None else dev(lse), **kw)
    g = V.distill_backward(z, dev(ids), dev(t), stats, dev(weight), **kw)
    loss2, g2 = V.distill_step(z, dev(ids), dev(t), dev(weight), teacher_lse=None if lse is None else dev(lse), **kw)
    rows = np.r_[0:8, 400, 401, 797:800]
    ref = R.distill(f64(z[rows]), ids[rows], t[rows].astype(float), tau, None if lse is None else lse[rows].astype(float),
                    weight[rows].astype(float))
    tol = ref["grad_tol"] + R.rounding(ref["grad"], dtype) * 1.01
    for x in (loss, loss2):
        close(f64(x[rows]), ref["loss"], ref["loss_tol"])
    for x in (g, g2):
        close(f64(x[rows]), ref["grad"], tol)
