"""The norm in place without a residual: what it returns as the sum is what the gradient may take, or nothing."""
import pytest

from test_vocab_gpu import V  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,D", [(1, 64), (5, 100), (7, 1031), (40, 4096)])
def test_in_place_without_a_residual(V, dtype, N, D):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(D)
    x, dy = (torch.randn((N, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    w = torch.rand(D, generator=g, device="cuda")
    y, total, rstd = V.rms_norm_forward(x, w)
    assert total is x
    want = V.rms_norm_backward(dy, total, w, rstd)
    # y takes x's place: no sum is left that a gradient could take
    a = x.clone()
    into, none, rstd_in = V.rms_norm_forward(a, w, out=a)
    assert into is a and none is None and torch.equal(a, y) and torch.equal(rstd_in, rstd)
    with pytest.raises(ValueError):
        V.rms_norm_backward(dy, none, w, rstd_in)
    a = x.clone()
    assert V.rms_norm_forward(a, w, out=a[:])[1] is None  # another tensor of the same memory
    # a sum_out keeps x's values, also x itself where y goes elsewhere
    a, kept = x.clone(), torch.empty_like(x)
    _, total, rstd_in = V.rms_norm_forward(a, w, out=a, sum_out=kept)
    assert total is kept and torch.equal(kept, x) and torch.equal(a, y)
    for got, right in zip(V.rms_norm_backward(dy, total, w, rstd_in), want):
        assert torch.equal(got, right)
    a = x.clone()
    _, total, _ = V.rms_norm_forward(a, w, sum_out=a)
    assert total is a and torch.equal(a, x)
    # another tensor for y: the sum is x
    assert V.rms_norm_forward(x, w, out=torch.empty_like(x))[1] is x
    assert V.rms_norm_forward(x, w, format="mx8")[1] is x


def test_in_place_with_a_residual(V):  # noqa: F811
    x, r = torch.randn(4, 96, device="cuda"), torch.randn(4, 96, device="cuda")
    for into in (0, 1):
        a = [x.clone(), r.clone()]
        y, total, _ = V.rms_norm_forward(a[0], residual=a[1], out=a[into])
        assert y is a[into] and torch.equal(total, x + r) and total.data_ptr() not in (a[0].data_ptr(), a[1].data_ptr())
