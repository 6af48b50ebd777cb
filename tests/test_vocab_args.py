"""What the vocabulary operators refuse, on the host before any CUDA call (no GPU needed): every
malformed argument of a call that would otherwise do nothing (no rows)."""
import pytest

from sparse_embedding_bag_gb300 import build as B
from sparse_embedding_bag_gb300 import embbwd as E

torch = pytest.importorskip("torch")

P = 1 << 20  # stands for an aligned device pointer; no call here reaches the device


@pytest.fixture(scope="module")
def lib():
    B.build()
    return E.load()


def call(lib, name, defaults, **kw):
    assert set(kw) <= set(defaults)
    return getattr(lib, name)(*{**defaults, **kw}.values())


LOGITS = dict(device=0, logits=P, dtype=0, stride=100, B=0, V=100, p=P, po=P, pn=4, o=P, oo=P, on=4, rep=P, freq=P,
              pres=P, b=P, bo=P, bv=P, bn=4, mask=P, mask_stride=4, out=P + 64, out_dtype=0, out_stride=100, status=P,
              stream=None)
DISTILL = dict(device=0, logits=P, dtype=0, stride=100, N=0, V=100, ids=P, t=P, t_dtype=0, t_stride=8, K=8)
FORWARD = dict(DISTILL, lse=P, tau=1.0, loss=P, stats=P, status=P, stream=None)
BACKWARD = dict(DISTILL, stats=P, weight=P, tau=1.0, out=P, out_stride=100, status=P, stream=None)
STEP = dict(DISTILL, lse=P, weight=P, tau=1.0, loss=P, out=P, out_stride=100, status=P, stream=None)
QUANT = dict(device=0, x=P, dtype=0, stride=64, R=0, K=64, fmt=0, g=1.0, codes=P, scales=P, stream=None)
LOOKUP = dict(device=0, codes=P, scales=P, R=10, K=64, fmt=0, g=1.0, ids=P, n=0, out=P, dtype=0, stride=64, status=P,
              stream=None)
MATMUL = dict(device=0, x=P, xs=P, gx=1.0, M=0, w=P, ws=P, gw=1.0, N=10, K=64, fmt=0, out=P, dtype=0, stride=10,
              status=P, stream=None)


@pytest.mark.parametrize("name,defaults", [
    ("emb_logits_process", LOGITS), ("emb_distill_forward", FORWARD), ("emb_distill_backward", BACKWARD),
    ("emb_distill_step", STEP), ("emb_micro_quantize", QUANT), ("emb_micro_lookup", LOOKUP),
    ("emb_micro_matmul", MATMUL)])
def test_calls_without_rows_do_nothing(lib, name, defaults):
    assert call(lib, name, defaults) == E.EMB_OK


@pytest.mark.parametrize("kw", [
    dict(device=-1), dict(B=-1), dict(B=65536), dict(V=0), dict(V=(1 << 20) + 1), dict(dtype=3), dict(out_dtype=-1),
    dict(pn=-1), dict(po=None), dict(oo=None), dict(bo=None), dict(bv=None), dict(p=P + 4), dict(oo=P + 4),
    dict(rep=P + 2), dict(mask=P + 1), dict(status=P + 2),
    # with rows to work on
    dict(B=2, logits=None), dict(B=2, out=None), dict(B=2, logits=P + 2), dict(B=2, stride=99), dict(B=2, out_stride=99),
    dict(B=2, mask_stride=3), dict(B=2, out=P, out_dtype=1), dict(B=2, out=P, out_stride=101)])
def test_logits_refuses(lib, kw):
    assert call(lib, "emb_logits_process", LOGITS, **kw) == E.EMB_ERR_INVALID_ARG


COMMON = [dict(device=-1), dict(N=-1), dict(V=0), dict(V=(1 << 20) + 1), dict(K=-1), dict(K=1025), dict(dtype=3),
          dict(t_dtype=-1), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("inf")), dict(tau=float("nan")),
          dict(ids=P + 4), dict(t=P + 2), dict(status=P + 1), dict(N=2, logits=None), dict(N=2, logits=P + 2),
          dict(N=2, ids=None), dict(N=2, t=None), dict(N=2, stride=99), dict(N=2, t_stride=7)]


@pytest.mark.parametrize("kw", COMMON + [dict(loss=P + 1), dict(stats=P + 8), dict(lse=P + 2), dict(N=2, loss=None),
                                         dict(N=2, stats=None)])
def test_distill_forward_refuses(lib, kw):
    assert call(lib, "emb_distill_forward", FORWARD, **kw) == E.EMB_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", COMMON + [dict(weight=P + 1), dict(stats=P + 4), dict(N=2, stats=None), dict(N=2, out=None),
                                         dict(N=2, out_stride=99), dict(N=2, out=P, out_stride=101),
                                         dict(N=2, out=P + 2)])
def test_distill_backward_refuses(lib, kw):
    assert call(lib, "emb_distill_backward", BACKWARD, **kw) == E.EMB_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", COMMON + [dict(weight=P + 1), dict(lse=P + 1), dict(N=2, loss=None), dict(N=2, out=None),
                                         dict(N=2, out=P, out_stride=101)])
def test_distill_step_refuses(lib, kw):
    assert call(lib, "emb_distill_step", STEP, **kw) == E.EMB_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(device=-1), dict(R=-1), dict(K=0), dict(K=(1 << 20) + 1), dict(dtype=3), dict(fmt=2), dict(g=2.0),
    dict(fmt=1, g=0.0), dict(fmt=1, g=-1.0), dict(fmt=1, g=float("nan")), dict(fmt=1, g=1e20), dict(R=2, x=None),
    dict(R=2, codes=None), dict(R=2, scales=P + 8), dict(R=2, codes=P + 8), dict(R=2, stride=63), dict(R=2, x=P + 2)])
def test_quantize_refuses(lib, kw):
    assert call(lib, "emb_micro_quantize", QUANT, **kw) == E.EMB_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(device=-1), dict(R=-1), dict(n=-1), dict(K=0), dict(dtype=3), dict(fmt=-1), dict(g=0.5), dict(n=2, out=None),
    dict(n=2, stride=63), dict(n=2, codes=None), dict(n=2, scales=P + 4), dict(n=2, ids=P + 4), dict(n=11, ids=None),
    dict(n=2, status=P + 1)])
def test_lookup_refuses(lib, kw):
    assert call(lib, "emb_micro_lookup", LOOKUP, **kw) == E.EMB_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(device=-1), dict(M=-1), dict(N=-1), dict(K=0), dict(M=(1 << 21) + 1), dict(dtype=3), dict(fmt=2), dict(gx=2.0),
    dict(fmt=1, gw=0.0), dict(M=2, x=None), dict(M=2, xs=P + 8), dict(M=2, w=P + 8), dict(M=2, ws=None),
    dict(M=2, out=None), dict(M=2, out=P + 2), dict(M=2, stride=9), dict(M=2, status=P + 1)])
def test_matmul_refuses(lib, kw):
    assert call(lib, "emb_micro_matmul", MATMUL, **kw) == E.EMB_ERR_INVALID_ARG


def test_bindings_refuse_tensors_on_the_host():
    from sparse_embedding_bag_gb300 import vocab
    z = torch.zeros(2, 10)
    i = torch.zeros(2, 3, dtype=torch.int64)
    t = torch.zeros(2, 3)
    m = vocab.MicroMatrix(torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 2, 10, "mx")
    for f in (lambda: vocab.process_logits(z), lambda: vocab.distill_step(z, i, t),
              lambda: vocab.distill_forward(z, i, t), lambda: vocab.micro_quantize(z), lambda: vocab.micro_lookup(m),
              lambda: vocab.micro_matmul(m, m)):
        with pytest.raises(ValueError):
            f()


def test_layout_sizes_match_the_header():
    from sparse_embedding_bag_gb300 import vocab
    assert [vocab._row_bytes(k) for k in (1, 32, 33, 4096)] == [16, 16, 32, 2048]
    assert [vocab._tiles(k, "mx") for k in (1, 128, 129, 4096)] == [1, 1, 2, 32]
    assert [vocab._tiles(k, "nv") for k in (1, 64, 65, 4096)] == [1, 1, 2, 64]
    assert vocab._scale_bytes(129, 129, "mx") == 2 * 2 * 512
    assert E.EMB_MICRO_MX == 0 and E.EMB_MICRO_NV == 1
