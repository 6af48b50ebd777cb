"""Gradients of logits that are views with far-apart rows: as large as the logits, not as their buffer."""
import numpy as np
import pytest

import _vocab_ref as R
from test_vocab_gpu import V, close, f64, teacher_lists, dev  # noqa: F401 (V is a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,n_vocab", [(64, 5000), (63, 5001), (64, 4098), (3, 20000)])
def test_gradient_of_a_slice_of_a_sequence(V, dtype, T, n_vocab):
    B, K = 4, 7
    rng = np.random.default_rng(T + n_vocab)
    ids, t = teacher_lists(rng, B, n_vocab, K)
    size = torch.finfo(dtype).bits // 8
    for at in (0, T - 1):
        z = torch.randn(B, T, n_vocab, device="cuda").to(dtype)[:, at]
        ref = R.distill(f64(z), ids, t.astype(float), 1.0, None, np.ones(B))
        tol = ref["grad_tol"] + R.rounding(ref["grad"], str(dtype)[6:]) * 1.01
        stats = V.distill_forward(z, dev(ids), dev(t))[1]
        x = z.detach().requires_grad_()
        V.distill_loss(x, dev(ids), dev(t)).sum().backward()
        for g in (V.distill_step(z, dev(ids), dev(t))[1], V.distill_backward(z, dev(ids), dev(t), stats), x.grad):
            assert g.untyped_storage().nbytes() <= B * (n_vocab * size + 16)
            close(f64(g), ref["grad"], tol)
    one = torch.randn(2, 9, n_vocab, device="cuda")[:1, 3]
    g = V.distill_step(one, dev(ids[:1]), dev(t[:1]))[1]
    assert g.is_contiguous() and g.untyped_storage().nbytes() == n_vocab * 4
