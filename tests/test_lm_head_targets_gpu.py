"""Training of the example with targets beyond the table: not counted in the mean, and an error after the steps."""
import pytest

from test_block_together_gpu import model
from test_vocab_gpu import V  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_targets_beyond_the_table(V):  # noqa: F811
    from sparse_embedding_bag_gb300 import lm_head
    table, layer, norm, tokens, targets = model(torch.float16)
    bad, silent = targets.clone(), targets.clone()
    bad[1:20:4], silent[1:20:4] = table.shape[0], -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(p=0.25, seed=9, call=2)
    loss, got = lm_head.gradients(table, layer, norm, tokens, bad, **args, status=status)
    want_loss, want = lm_head.gradients(table, layer, norm, tokens, silent, **args)
    assert status.item() == 1 and torch.equal(loss, want_loss)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(RuntimeError, match="error bits 1"):
        lm_head.train(table.clone(), layer.clone(), norm.clone(), tokens, bad, lr=0.5, steps=2)
    assert len(lm_head.train(table, layer, norm, tokens, silent, lr=0.5, steps=2)) == 2
