"""The example's serving loop: hidden states of zeros, and no wait for the GPU within a step."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("format", ["nv", "mx"])
def test_serves_hidden_states_of_zeros(format):
    from sparse_embedding_bag_gb300 import lm_head
    g = torch.Generator(device="cuda").manual_seed(4)
    table = torch.randn((300, 64), generator=g, device="cuda").bfloat16()
    layer = torch.randn((64, 64), generator=g, device="cuda").bfloat16()
    # equal logits: the lowest token not yet penalised by a bias
    bias = (torch.tensor([0, 1], device="cuda"), torch.tensor([0, 2, 2], device="cuda"), torch.full((2,), -5.0, device="cuda"))
    for t, w in ((table, torch.zeros_like(layer)), (torch.zeros_like(table), layer)):
        out = lm_head.serve(t, w, [[5, 6], [7]], 3, format=format, repetition=1.0, frequency=1.0, bias=bias)
        assert out == [[2, 3, 4], [0, 1, 2]]


def test_serving_steps_do_not_wait_for_the_gpu():
    from sparse_embedding_bag_gb300 import lm_head, vocab
    g = torch.Generator(device="cuda").manual_seed(5)
    table = (torch.randn((500, 64), generator=g, device="cuda") * 0.1).bfloat16()
    layer = torch.randn((64, 64), generator=g, device="cuda").bfloat16()
    want = lm_head.serve(table, layer, [[1, 2], [3]], 4, format="nv")
    process, calls = vocab.process_logits, []

    def watched(*a, **kw):  # from the first step's last call on
        torch.cuda.set_sync_debug_mode("error")
        calls.append(1)
        return process(*a, **kw)
    vocab.process_logits = watched
    stopped = None
    try:
        lm_head.serve(table, layer, [[1, 2], [3]], 4, format="nv")
    except RuntimeError as e:  # reading the status at the end does wait
        stopped = e
    finally:
        torch.cuda.set_sync_debug_mode("default")
        vocab.process_logits = process
    assert stopped is not None and len(calls) == 4
    assert lm_head.serve(table, layer, [[1, 2], [3]], 4, format="nv") == want
