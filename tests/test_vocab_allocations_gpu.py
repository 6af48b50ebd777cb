"""What the vocabulary operators allocate, PyTorch's dispatcher sees: each call's new tensors under a dispatch mode."""
import pytest

from test_vocab_gpu import V  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from torch.utils._python_dispatch import TorchDispatchMode  # noqa: E402


class Allocations(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in str(func):
            self.seen.append(tuple(out.shape))
        return out


def test_dispatch_modes_see_allocations(V):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((40, 96), generator=g, device="cuda").half()
    t = torch.randn((200, 96), generator=g, device="cuda").half()
    w, at = torch.ones(96, device="cuda"), torch.arange(40, device="cuda")
    z, ids = torch.randn((4, 300), generator=g, device="cuda"), torch.arange(5, device="cuda").repeat(4, 1)
    m = V.micro_quantize(t, "mx8")
    lse = V.cross_entropy_forward(x, t, at)[1]
    codes, scales = tuple(m.codes.shape), tuple(m.scales.shape)
    for call, shapes in (
            (lambda: V.process_logits(z), [(4, 300)]),
            (lambda: V.distill_step(z, ids, z[:, :5].contiguous()), [(4,), (4, 300)]),
            (lambda: V.micro_quantize(t, "mx8"), [codes, scales]),
            (lambda: V.micro_lookup(m), [(200, 96)]),
            (lambda: V.micro_matmul(m, m), [(200, 200)]),
            (lambda: V.rms_norm_forward(x, w, residual=x), [(40, 96), (40,), (40, 96)]),
            (lambda: V.rms_norm_backward(x, x, w, w[:40].contiguous()), [(40, 96), (96,)]),
            (lambda: V.dropout(x, 0.5, 1), [(40, 96)]),
            (lambda: V.cross_entropy_forward(x, t, at), [(40,), (40,)]),
            (lambda: V.cross_entropy_backward(x, t, at, lse), [(40, 96), (200, 96)]),
            (lambda: V.cross_entropy_step(x, t, at), [(40,), (40, 96), (200, 96)])):
        with Allocations() as mode:
            call()
        for shape in shapes:
            assert shape in mode.seen
            mode.seen.remove(shape)


def test_results_where_memory_is_filled(V):  # noqa: F811
    """PyTorch fills new memory with NaN here: no call's results depend on what its memory held."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x, t = (torch.randn((n, 131), generator=g, device="cuda").bfloat16() for n in (70, 500))
    w, at = torch.rand(131, generator=g, device="cuda"), torch.randint(-1, 500, (70,), generator=g, device="cuda")

    def run():
        y, s, rstd = V.rms_norm_forward(x, w, residual=x)
        m, _, _ = V.rms_norm_forward(x, w, format="mx8")
        return [y, s, rstd, *V.rms_norm_backward(x, s, w, rstd), V.dropout(x, 0.3, 5), *V.cross_entropy_step(y, t, at),
                V.micro_matmul(m, V.micro_quantize(t, "mx8"))]
    want = run()
    try:
        torch.use_deterministic_algorithms(True)
        got = run()
    finally:
        torch.use_deterministic_algorithms(False)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_profiles_and_fills_see_allocations(V):  # noqa: F811
    x = torch.randn(8, 64, device="cuda")

    def ops():
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as p:
            V.dropout(x, 0.5, 1)
        return [e.name for e in p.events()]
    V.dropout(x, 0.5, 1)
    seen = ops()
    assert "aten::empty" in seen and "aten::fill_" not in seen
    try:
        torch.use_deterministic_algorithms(True)
        assert "aten::fill_" in ops()
        torch.utils.deterministic.fill_uninitialized_memory = False
        assert "aten::fill_" not in ops()
    finally:
        torch.utils.deterministic.fill_uninitialized_memory = True
        torch.use_deterministic_algorithms(False)
