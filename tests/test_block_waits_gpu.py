"""The calls return before the GPU has done their work: each is made behind a kernel that keeps the stream busy for some
20 ms, and that kernel is still running when the call returns. (PyTorch's own check for synchronisations does not see
those of a library.)"""
import pytest

from test_vocab_gpu import V  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BUSY = 40_000_000  # cycles


def calls(V):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(1)

    def rows(N, D, dtype=torch.bfloat16):
        return torch.randn((N, D), generator=g, device="cuda").to(dtype)
    out = {}
    for D in (264, 1031):  # on 16-byte boundaries, and off them
        for dtype in (torch.float32, torch.bfloat16):
            x, r, w = rows(300, D, dtype), rows(300, D, dtype), torch.ones(D, device="cuda")
            rstd = torch.ones(300, device="cuda")
            name = f"{D} {dtype}"
            out["norm " + name] = lambda x=x, r=r, w=w: V.rms_norm_forward(x, w, residual=r)
            out["norm to 8 bits " + name] = lambda x=x, w=w: V.rms_norm_forward(x, w, format="mx8")
            out["norm backward " + name] = lambda x=x, r=r, w=w, s=rstd: V.rms_norm_backward(x, r, w, s, grad_sum=r)
            out["dropout " + name] = lambda x=x, r=r: V.dropout(x, 0.1, 5, residual=r)
        for N in (20, 100, 400):  # few tokens, a tile, several
            h, t = rows(N, D), rows(3001, D) * 0.1
            at = torch.randint(-1, 3001, (N,), generator=g, device="cuda")
            lse = V.cross_entropy_forward(h, t, at)[1]
            name = f"{N} x {D}"
            out["loss " + name] = lambda h=h, t=t, at=at: V.cross_entropy_forward(h, t, at)
            out["gradients " + name] = lambda h=h, t=t, at=at, lse=lse: V.cross_entropy_backward(h, t, at, lse)
            out["hidden gradient " + name] = lambda h=h, t=t, at=at, lse=lse: V.cross_entropy_backward(h, t, at, lse, want_table=False)
            out["table gradient " + name] = lambda h=h, t=t, at=at, lse=lse: V.cross_entropy_backward(h, t, at, lse, want_hidden=False)
            out["step " + name] = lambda h=h, t=t, at=at: V.cross_entropy_step(h, t, at)
    m = V.micro_quantize(rows(500, 264), "mx8")
    out["quantise"] = lambda x=rows(500, 264): V.micro_quantize(x, "mx8")
    out["look up"] = lambda ids=torch.arange(40, device="cuda"): V.micro_lookup(m, ids)
    out["product"] = lambda: V.micro_matmul(m, m)
    held = torch.zeros(1, dtype=torch.int64, device="cuda")
    out["dropout of a held call"] = lambda x=rows(64, 64): V.dropout(x, 0.1, 5, held)
    return out


def test_calls_return_before_their_work_is_done(V):  # noqa: F811
    run = calls(V)
    for f in run.values():  # kernels loaded, memory in the allocator's hands
        f()
    torch.cuda.synchronize()
    waited = []
    for name, f in run.items():
        done = torch.cuda.Event()
        torch.cuda._sleep(BUSY)
        done.record()
        f()
        if done.query():
            waited.append(name)
        torch.cuda.synchronize()
        assert done.query()
    assert not waited
