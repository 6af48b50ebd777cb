"""The vocabulary operators on the GPU against 64-bit references, at the sizes, masks, strides and
lists where they can go wrong. Tolerances are the references' bounds of fp32 arithmetic plus one
rounding to the output's type."""
import numpy as np
import pytest

import _vocab_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

N_ALIGN = 8  # elements of 16 bits in 16 bytes
DTYPES = ["float32", "float16", "bfloat16"]


@pytest.fixture(scope="module")
def V():
    from sparse_embedding_bag_gb300 import build, vocab
    build.build()
    assert torch.cuda.is_available()
    return vocab


def dev(a, dtype=None, pad=0, shift=0):
    """A device tensor of `a`; 2-D ones inside rows `pad` wider, `shift` elements into the buffer."""
    t = torch.as_tensor(np.asarray(a), device="cuda")
    t = t.to(getattr(torch, dtype)) if dtype else t
    if t.dim() == 2 and (pad or shift):
        flat = torch.full((t.shape[0] * (t.shape[1] + pad) + shift,), 7.0, device="cuda").to(t.dtype)
        wide = flat[shift:].view(t.shape[0], -1)[:, :t.shape[1]]
        wide.copy_(t)
        return wide
    return t


def f64(t):
    return t.detach().double().cpu().numpy()


def csr(lists, dtype=np.int64):
    off = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int64)
    ids = np.concatenate([np.asarray(x, np.int64) for x in lists] or [np.zeros(0, np.int64)])
    return dev(ids.astype(np.int64)), dev(off)


def close(got, want, tol):
    got, want = np.asarray(got), np.asarray(want)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    ok = same | (np.abs(np.where(same, 0, got - want)) <= tol)
    assert ok.all(), (np.argwhere(~ok)[:5], got[~ok][:5], want[~ok][:5], np.broadcast_to(tol, ok.shape)[~ok][:5])


# ---- logits

@pytest.mark.parametrize("dtype,out", [("float32", "float32"), ("bfloat16", "float32"), ("float16", "float16"),
                                       ("bfloat16", "bfloat16"), ("float32", "bfloat16"), ("float16", "float32")])
@pytest.mark.parametrize("B,n_vocab,pad,shift", [(1, 1, 0, 0), (3, 33, 0, 1), (5, 1023, 0, 0), (4, 8192, 64, 0),
                                                 (3, 20001, 3, 3), (2, 70000, 0, 5)])
def test_logits(V, dtype, out, B, n_vocab, pad, shift):
    rng = np.random.default_rng(B * n_vocab + pad)
    z = dev(rng.normal(0, 3, (B, n_vocab)), dtype, pad, shift)
    prompt = [list((rng.random(rng.integers(0, 300)) ** 3 * n_vocab).astype(int)) for _ in range(B)]
    output = [list((rng.random(rng.integers(0, 200)) ** 3 * n_vocab).astype(int)) for _ in range(B)]
    prompt[0], output[-1] = [], []
    output[0] = [n_vocab - 1] * 70 + output[0]
    bias = [[(int(v), float(np.float32(x))) for v, x in zip(rng.integers(0, n_vocab, 40), rng.normal(0, 4, 40))]
            for _ in range(B)]  # ids repeat
    bias[B // 2] = []
    rep, freq, pres = (rng.uniform(*r, B).astype(np.float32) for r in ((0.8, 1.6), (-0.5, 0.5), (-1, 1)))
    mask = rng.integers(0, 1 << 32, (B, (n_vocab + 31) // 32 + 2), dtype=np.uint64).astype(np.uint32).view(np.int32)
    mask[0] = -1
    if B > 2:
        mask[1] = 0  # nothing left
    y, tol = R.process_logits(f64(z), prompt, output, rep.astype(float), freq.astype(float), pres.astype(float), bias,
                              mask)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, off = csr([[v for v, _ in b] for b in bias])
    values = dev(np.array([x for b in bias for _, x in b], np.float32))
    got = V.process_logits(z, prompt=csr(prompt), output=csr(output), repetition=dev(rep), frequency=dev(freq),
                           presence=dev(pres), bias=(ids, off, values), mask=dev(mask), dtype=getattr(torch, out),
                           status=status)
    close(f64(got), y, tol + R.rounding(np.where(np.isfinite(y), y, 0), out) * 1.01)
    assert status.item() == 0
    # each part alone, and in place
    none = [[] for _ in range(B)]
    one = np.ones(B)
    only = V.process_logits(z, output=csr(output), frequency=dev(freq), dtype=torch.float32)
    y, tol = R.process_logits(f64(z), none, output, one, freq.astype(float), 0 * one, none, None)
    close(f64(only), y, tol)
    w = z.clone(memory_format=torch.preserve_format) if not (pad or shift) else z
    y, tol = R.process_logits(f64(w), prompt, none, rep.astype(float), 0 * one, 0 * one, none, mask)
    got = V.process_logits(w, prompt=csr(prompt), repetition=dev(rep), mask=dev(mask), out=w)
    assert got is w
    close(f64(w), y, tol + R.rounding(np.where(np.isfinite(y), y, 0), dtype) * 1.01)


def test_logits_long_history_and_special_values(V):
    n_vocab = 50021
    rng = np.random.default_rng(2)
    z = rng.normal(0, 3, (3, n_vocab)).astype(np.float32)
    z[0, :7] = [np.inf, -np.inf, 0.0, -0.0, np.nan, 3.4e38, -3.4e38]
    prompt = [list(rng.integers(0, n_vocab, 40000)), [], [0]]
    output = [[0, 1, 2, 3], list(np.full(70001, 17)), []]
    rep, freq, pres = np.array([1.25, 1, 2]), np.array([0.5, 0.25, 1]), np.array([0.0, 1, 1])
    with np.errstate(over="ignore", invalid="ignore"):
        y, tol = R.process_logits(z.astype(float), prompt, output, rep, freq, pres, [[], [], []], None)
    y = np.where(y > 3.5e38, np.inf, np.where(y < -3.5e38, -np.inf, y))
    got = f64(V.process_logits(dev(z), prompt=csr(prompt), output=csr(output), repetition=dev(rep.astype(np.float32)),
                               frequency=dev(freq.astype(np.float32)), presence=dev(pres.astype(np.float32))))
    close(got, y, tol + R.rounding(np.where(np.isfinite(y), y, 0), "float32"))


def test_logits_reports_bad_ids_and_offsets(V):
    z = torch.randn(3, 500, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rep = torch.full((3,), 2.0, device="cuda")
    got = V.process_logits(z, prompt=csr([[5, 500, -1], [], [7]]), repetition=rep, status=status)
    assert status.item() == 1
    want = z.clone()
    for b, v in ((0, 5), (2, 7)):
        want[b, v] = want[b, v] / 2 if want[b, v] > 0 else want[b, v] * 2
    assert torch.equal(got, want)
    status.zero_()
    ids, off = csr([[1, 2], [3], [4]])
    for bad in ([0, 3, 2, 4], [0, 2, 3, 5], [-1, 2, 3, 4]):
        got = V.process_logits(z, output=(ids, dev(np.array(bad))), frequency=rep, status=status)
        assert status.item() == 2
        status.zero_()
        assert torch.isfinite(got).all()
    V.process_logits(z, bias=(dev(np.array([9, 600])), dev(np.array([0, 2, 2, 2])), torch.ones(2, device="cuda")),
                     status=status)
    assert status.item() == 1
    assert V.process_logits(z[:0]).shape == (0, 500)


# ---- distillation

def teacher_lists(rng, N, n_vocab, K, repeat=False):
    ids = np.stack([rng.choice(n_vocab, K, replace=repeat or K > n_vocab) for _ in range(N)]) if K else \
        np.zeros((N, 0), int)
    t = np.sort(rng.normal(3, 2, (N, K)))[:, ::-1].astype(np.float32).copy()
    for n in range(N):
        if n % 4 == 3:
            ids[n, K // 2:] = -1
    return ids.astype(np.int64), t


def check_distill(V, z, ids, t, tau, lse, weight, dtype, teacher="float32"):
    t_dev = dev(t, teacher)
    ref = R.distill(f64(z), ids, f64(t_dev), tau, None if lse is None else lse.astype(float), weight.astype(float))
    kw = dict(temperature=tau, teacher_lse=None if lse is None else dev(lse))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i_dev, w_dev = dev(ids), dev(weight)
    loss, stats = V.distill_forward(z, i_dev, t_dev, status=status, **kw)
    close(f64(loss), ref["loss"], ref["loss_tol"])
    st = f64(stats)
    close(st[:, 0], ref["stats"][:, 0], 0)
    close(st[:, 1], ref["stats"][:, 1], 1e-4 * ref["stats"][:, 1])
    close(st[:, 2], ref["stats"][:, 2], ref["coef_tol"])
    # the step sums over another split of the row than the forward
    loss2, g2 = V.distill_step(z, i_dev, t_dev, w_dev, status=status, **kw)
    close(f64(loss2), ref["loss"], ref["loss_tol"])
    tol = ref["grad_tol"] + R.rounding(np.nan_to_num(ref["grad"]), dtype) * 1.01
    close(f64(g2), ref["grad"], tol)
    g = V.distill_backward(z, i_dev, t_dev, stats, w_dev, temperature=tau, status=status)
    close(f64(g), ref["grad"], tol)
    assert g.dtype == z.dtype and g2.dtype == z.dtype and status.item() == 0
    # in place, on rows at the same places in 16 bytes (the order of the sums goes by them)
    flat = torch.empty(z.numel() + N_ALIGN + z.shape[0] * z.stride(0), dtype=z.dtype, device="cuda")
    at = (z.data_ptr() // z.element_size() - flat.data_ptr() // z.element_size()) % N_ALIGN
    w = flat.as_strided(z.shape, z.stride(), at).copy_(z)
    loss3, g3 = V.distill_step(w, i_dev, t_dev, w_dev, out=w, **kw)
    assert g3 is w
    assert torch.equal(loss3, loss2) and torch.equal(g3, g2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("N,n_vocab,K,tau,pad,shift", [(1, 2, 1, 1.0, 0, 0), (5, 37, 5, 2.0, 0, 1), (9, 1000, 8, 0.7, 8, 0),
                                                       (4, 4097, 64, 1.0, 0, 3), (6, 32001, 100, 2.0, 0, 0),
                                                       (3, 50001, 1024, 1.0, 7, 5), (2, 128256, 32, 1.0, 0, 0)])
def test_distill(V, dtype, tail, N, n_vocab, K, tau, pad, shift):
    rng = np.random.default_rng(n_vocab + K)
    ids, t = teacher_lists(rng, N, n_vocab, K)
    x = rng.normal(0, 2, (N, n_vocab))
    for n in range(N):
        on = ids[n] >= 0
        x[n, ids[n][on]] = t[n][on] + 2 * rng.normal(size=on.sum())
    lse = None
    if tail:
        lt = np.where(ids >= 0, t / tau, -np.inf)
        lse = (np.log(np.exp(lt).sum(-1)) + rng.uniform(0.001, 0.7, N)).astype(np.float32)
    weight = rng.uniform(0.2, 2, N).astype(np.float32)
    check_distill(V, dev(x, dtype, pad, shift), ids, t, tau, lse, weight, dtype)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_empty_rows_repeated_ids_and_padding(V, tail):
    rng = np.random.default_rng(3)
    N, n_vocab, K = 7, 3001, 24
    ids, t = teacher_lists(rng, N, n_vocab, K, repeat=True)
    ids[0, 1::2] = ids[0, 0]  # one id many times
    ids[1] = -1               # no entry
    ids[2, :23] = -1          # one entry
    t[3, :5] = -np.inf        # entries without mass
    lse = None
    if tail:
        lt = np.where(ids >= 0, t, -np.inf)
        with np.errstate(divide="ignore"):
            lse = (np.log(np.exp(lt).sum(-1)) + 0.1).astype(np.float32)
        lse[1] = 0
        lse[5] = -np.inf      # a teacher without mass
    else:
        t[4] = -np.inf        # a teacher that says nothing
    for teacher in DTYPES:
        check_distill(V, dev(rng.normal(0, 2, (N, n_vocab)), "float32"), ids, t, 1.0, lse,
                      np.ones(N, np.float32), "float32", teacher)


def test_distill_whole_vocabulary_on_the_list_and_masked_logits(V):
    rng = np.random.default_rng(4)
    ids = np.tile(np.arange(40), (3, 1)).astype(np.int64)
    t = rng.normal(0, 2, (3, 40)).astype(np.float32)
    z = rng.normal(0, 2, (3, 40))
    check_distill(V, dev(z, "float32"), ids, t, 1.0, None, np.ones(3, np.float32), "float32")
    z = rng.normal(0, 2, (3, 5000))
    z[0, 40:] = -np.inf       # the student gives nothing off the list
    z[1, 100:4000] = -3.4e38
    check_distill(V, dev(z, "float32"), ids, t, 1.0, None, np.ones(3, np.float32), "float32")
    z[2, 3] = -np.inf         # nor to a token of the teacher: infinite loss, finite gradient
    loss, g = V.distill_step(dev(z, "float32"), dev(ids), dev(t))
    assert torch.isinf(loss[2]) and loss[2] > 0 and torch.isfinite(g).all() and torch.isfinite(loss[:2]).all()
    z[1, 17] = np.nan
    loss, g = V.distill_step(dev(z, "float32"), dev(ids), dev(t))
    assert torch.isnan(loss[1]) and torch.isnan(g[1]).all() and torch.isfinite(g[0]).all()
    z[0] = -np.inf            # nothing left at all: as 0 / 0
    loss, g = V.distill_step(dev(z, "float32"), dev(ids), dev(t))
    assert torch.isnan(loss[0]) and torch.isnan(g[0]).all()


def test_distill_rows_at_the_lowest_value_of_their_type(V):
    # masked throughout with finfo.min: as uniform as a row of equal logits
    for dtype in DTYPES:
        low = torch.finfo(getattr(torch, dtype)).min
        ids, t = np.array([[1, 7, 300]]), np.array([[1.0, 0.5, 0.0]], np.float32)
        lse = np.array([1.9], np.float32)
        for tail in (None, dev(lse)):
            got = V.distill_step(torch.full((1, 900), low, device="cuda", dtype=getattr(torch, dtype)), dev(ids), dev(t),
                                 teacher_lse=tail)
            want = V.distill_step(torch.zeros(1, 900, device="cuda", dtype=getattr(torch, dtype)), dev(ids), dev(t),
                                  teacher_lse=tail)
            assert torch.isfinite(got[0]).all() and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_beyond_32_bit_offsets(V):
    # three rows 2^31 elements apart
    n_vocab, stride = 5003, 1 << 31
    rng = np.random.default_rng(12)
    flat = torch.empty(2 * stride + n_vocab, dtype=torch.bfloat16, device="cuda")
    z = flat.as_strided((3, n_vocab), (stride, 1))
    z.copy_(dev(rng.normal(0, 2, (3, n_vocab)), "bfloat16"))
    near = z.clone(memory_format=torch.contiguous_format)
    hist, rep = csr([[1, 2], [5, 5, 5], [5002]]), torch.full((3,), 1.5, device="cuda")
    want = V.process_logits(near, output=hist, repetition=rep)
    assert torch.equal(V.process_logits(z, output=hist, repetition=rep), want)
    ids, t = teacher_lists(rng, 3, n_vocab, 9)
    loss, g = V.distill_step(near, dev(ids), dev(t))
    loss2, g2 = V.distill_step(z, dev(ids), dev(t), out=z)
    close(f64(loss2), f64(loss), 1e-5 * np.abs(f64(loss)))
    close(f64(g2), f64(g), 2.0 ** -7 * np.abs(f64(g)) + 1e-7)
    z.copy_(near)
    m = V.micro_quantize(z)
    assert torch.equal(m.codes, V.micro_quantize(near).codes)
    V.micro_lookup(m, out=z)
    assert torch.equal(z, V.micro_lookup(m, dtype=torch.bfloat16))
    y = V.micro_matmul(m, m)
    wide = flat.as_strided((3, 3), (stride, 1))
    V.micro_matmul(m, m, out=wide)
    assert torch.equal(wide, y)


def test_distill_student_sure_of_the_list(V):
    # the student's mass off the list is about 1e-12: u must not come from 1 - (mass on the list)
    rng = np.random.default_rng(5)
    N, n_vocab, K = 2, 20000, 16
    ids, t = teacher_lists(rng, N, n_vocab, K)
    x = rng.normal(0, 1, (N, n_vocab))
    x[np.arange(N)[:, None], ids] = 40 + t
    lse = (np.log(np.exp(t.astype(float)).sum(-1)) + 1e-3).astype(np.float32)
    check_distill(V, dev(x, "float32"), ids, t, 1.0, lse, np.ones(N, np.float32), "float32")


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_against_differences(V, tail):
    rng = np.random.default_rng(6)
    N, n_vocab, K, tau = 3, 23, 5, 1.5
    ids, t = teacher_lists(rng, N, n_vocab, K)
    z = rng.normal(0, 2, (N, n_vocab)).astype(np.float32)
    lse = (np.log(np.exp(np.where(ids >= 0, t / tau, -np.inf)).sum(-1)) + 0.2).astype(np.float32) if tail else None
    x = dev(z).requires_grad_()
    loss = V.distill_loss(x, dev(ids), dev(t), temperature=tau, teacher_lse=None if lse is None else dev(lse))
    weight = rng.uniform(0.5, 2, N).astype(np.float32)
    (loss * dev(weight)).sum().backward()
    ref = lambda y: R.distill(y, ids, t.astype(float), tau, None if lse is None else lse.astype(float),
                              weight.astype(float))
    bound = ref(z.astype(float))
    h = 1e-4  # central differences: h^2 / 6 times a third derivative below 10, and 1e-15 / h of rounding
    for n in range(N):
        for v in range(n_vocab):
            up, down = z.astype(float).copy(), z.astype(float).copy()
            up[n, v] += h
            down[n, v] -= h
            d = (ref(up)["loss"][n] - ref(down)["loss"][n]) / (2 * h) * weight[n]
            assert abs(f64(x.grad)[n, v] - d) <= bound["grad_tol"][n, v] + 1e-6 + 2 * R.U * abs(d)


def test_distill_reports_bad_ids(V):
    z = torch.randn(3, 300, device="cuda")
    ids = torch.tensor([[1, 2, -1], [300, 4, 5], [-2, 7, 8]], device="cuda")
    t = torch.randn(3, 3, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, g = V.distill_step(z, ids, t, status=status)
    assert status.item() == 1
    good = torch.where((ids < 0) | (ids >= 300), -1, ids)
    loss2, g2 = V.distill_step(z, good, t)
    assert torch.equal(loss, loss2) and torch.equal(g, g2)
    loss, g = V.distill_step(z, ids[:, :0], t[:, :0])
    assert not loss.any() and not g.any()
    assert V.distill_step(z[:0], ids[:0], t[:0])[1].shape == (0, 300)


def test_distill_wide_rows(V):
    # the widest rows
    rng = np.random.default_rng(8)
    N, n_vocab, K = 2, 1 << 20, 16
    ids, t = teacher_lists(rng, N, n_vocab, K)
    lse = (np.log(np.exp(t.astype(float)).sum(-1)) + 0.1).astype(np.float32)
    check_distill(V, dev(rng.normal(0, 2, (N, n_vocab)), "float32"), ids, t, 1.0, lse, np.ones(N, np.float32),
                  "float32")


# ---- microscaled 4 bits

def codes_of(m):
    return m.codes.cpu().numpy(), m.scales.cpu().numpy()


@pytest.mark.parametrize("fmt,g", [("mx", 1.0), ("nv", 2.0 ** -9), ("nv", 0.13 / 2688)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (3, 31, 0, 1), (17, 100, 8, 0), (130, 96, 0, 0),
                                                 (5, 4100, 3, 5), (257, 520, 0, 0)])
def test_micro_rows(V, fmt, g, dtype, rows, cols, pad, shift):
    g = float(np.float32(g))
    rng = np.random.default_rng(rows * cols)
    x = rng.normal(0, 1, (rows, cols)) * np.exp(rng.normal(0, 1.5, (rows, 1)))
    x[rows // 2, : cols // 2] = 0
    if dtype != "float16":
        x[0] *= 1e-20
    x = dev(x, dtype, pad, shift)
    m = V.micro_quantize(x, fmt, g)
    v, code, s = R.decode(*codes_of(m), rows, cols, fmt, g)
    xs = f64(x)
    n = 32 if fmt == "mx" else 16
    for r in range(rows):
        for j in range(-(-cols // n)):
            b = xs[r, j * n:(j + 1) * n]
            sb = s[r, j * n]
            big = np.abs(b).max()
            if fmt == "mx":
                assert sb == (2.0 ** max(np.floor(np.log2(big)) - 2, -127) if big > 0 else 2.0 ** -127)
            else:
                t = big / (6 * g)
                assert sb == R.e4m3(t) or abs(sb - t) <= abs(R.e4m3(t) - t) * (1 + 2.0 ** -18)
    d = s * g
    ok = d >= 2.0 ** -126 if fmt == "nv" else np.ones_like(d, bool)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(ok, np.abs(xs) / d, 0.0)
    mag = R.GRID[code & 7]
    best = np.abs(R.GRID[None, None] - np.minimum(y, 6.0)[..., None]).min(-1)
    assert (np.abs(mag - np.minimum(y, 6.0)) <= best + (0 if fmt == "mx" else 2.0 ** -21) * np.minimum(y, 6.0)).all()
    assert (np.where(code >= 8, -1, 1) * np.sign(xs) >= 0).all()
    # halves of the exact format go to the code with an even mantissa
    tie = np.ptp(np.sort(np.abs(R.GRID[None, None] - y[..., None]), -1)[..., :2], axis=-1) == 0
    if fmt == "mx":
        assert ((code[tie & (y < 6)] & 1) == 0).all()
    # all of the buffers is written: codes past the row and scales past the blocks and rows are zero
    full = np.zeros((rows, m.codes.shape[1] * 2), np.uint8)
    full[:, :cols] = code
    packed = codes_of(m)[0]
    assert np.array_equal((full[:, 0::2] | (full[:, 1::2] << 4)), packed)
    rows_p, blocks = -(-rows // 128) * 128, m.scales.shape[1] * 4
    t = codes_of(m)[1].transpose(0, 3, 2, 1, 4).reshape(rows_p, blocks)
    used = -(-cols // 32) * (32 // n)
    assert not t[rows:].any() and not t[:, used:].any()
    # read back
    for out in DTYPES:
        got = f64(V.micro_lookup(m, dtype=getattr(torch, out)))
        close(got, v, 2 * R.U * np.abs(v) + R.rounding(v, out) * 1.01)
    ids = torch.from_numpy(rng.integers(0, rows, 11)).cuda()
    assert torch.equal(V.micro_lookup(m, ids), V.micro_lookup(m)[ids])
    wide = torch.zeros(11, cols + 5, device="cuda")
    V.micro_lookup(m, ids, out=wide[:, 1:cols + 1])
    assert torch.equal(wide[:, 1:cols + 1], V.micro_lookup(m)[ids]) and not wide[:, cols + 1:].any()
    again = V.micro_quantize(x, fmt, g, out=V.MicroMatrix(torch.full_like(m.codes, 255), torch.full_like(m.scales, 255),
                                                          rows, cols, fmt, g))
    assert torch.equal(again.codes, m.codes) and torch.equal(again.scales, m.scales)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_micro_special_values(V, fmt):
    n = 32 if fmt == "mx" else 16
    x = torch.ones(1, 6 * n + 3, device="cuda")
    x[0, 1] = float("nan")
    x[0, n + 2] = float("inf")
    x[0, 2 * n + 3] = -float("inf")
    x[0, 3 * n:4 * n] = 0
    x[0, 4 * n:5 * n] = 3.4e38
    x[0, 5 * n:6 * n] = 1e-42  # subnormal
    v = V.micro_lookup(V.micro_quantize(x, fmt, 1.0 if fmt == "mx" else 0.5))[0]
    assert torch.isnan(v[:3 * n]).all() and not v[3 * n:4 * n].any()
    if fmt == "mx":
        assert (v[4 * n:5 * n] == 6 * 2.0 ** 125).all()   # 3.4e38 / 2^125 is just below 8: saturates
        assert not v[5 * n:6 * n].any()                    # below half the smallest magnitude, 0.25 * 2^-127
    else:
        assert (v[4 * n:5 * n] == 448 * 6 * 0.5).all()     # the block scale saturates
        assert not v[5 * n:6 * n].any()
    assert (v[6 * n:] - 1).abs().max() <= (0 if fmt == "mx" else 1 / 16)


def test_micro_lookup_reports_bad_ids(V):
    m = V.micro_quantize(torch.randn(5, 64, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = V.micro_lookup(m, torch.tensor([4, 5, -1, 0], device="cuda"), status=status)
    assert status.item() == 1 and not got[1:3].any()
    assert torch.equal(got[[0, 3]], V.micro_lookup(m)[[4, 0]])
    assert V.micro_lookup(m, torch.zeros(0, dtype=torch.int64, device="cuda")).shape == (0, 64)
    assert V.micro_quantize(torch.zeros(0, 64, device="cuda")).rows == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 300, 64), (2, 128, 256), (7, 129, 100), (16, 257, 520), (17, 1000, 2056),
                                   (33, 127, 8192), (64, 640, 1000), (100, 384, 2048), (129, 511, 300), (130, 50, 4096),
                                   (256, 1024, 512), (300, 2000, 96), (513, 257, 1056)])
def test_micro_matmul(V, fmt, M, N, K):
    rng = np.random.default_rng(M * N + K)
    gx, gw = (1.0, 1.0) if fmt == "mx" else (float(np.float32(6.5 / 2688)), float(np.float32(0.13 / 2688)))
    x = V.micro_quantize(dev(rng.normal(0, 1, (M, K)) * np.exp(rng.normal(0, 1, (M, 1))), "float32"), fmt, gx)
    w = V.micro_quantize(dev(rng.normal(0, 0.02, (N, K)), "float32"), fmt, gw)
    xv, wv = R.decode(*codes_of(x), M, K, fmt, gx)[0], R.decode(*codes_of(w), N, K, fmt, gw)[0]
    want, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    for out in DTYPES:
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = V.micro_matmul(x, w, dtype=getattr(torch, out), status=status)
        # K additions, each rounding or cutting at most 2 u of the sum of magnitudes
        close(f64(got), want, (2 * K + 8) * R.U * mag + R.rounding(want, out) * 1.01)
        assert status.item() == 0
        again = V.micro_matmul(x, w, dtype=getattr(torch, out))
        assert torch.equal(again, got)
    for pad, shift in ((3, 1), (8, 0)):
        flat = torch.full((M * (N + pad) + shift,), 5.0, dtype=torch.bfloat16, device="cuda")
        wide = flat[shift:].view(M, N + pad)
        V.micro_matmul(x, w, out=wide[:, :N])
        assert torch.equal(wide[:, :N], V.micro_matmul(x, w)) and (wide[:, N:] == 5).all() and (flat[:shift] == 5).all()


def test_micro_matmul_nan_scale_stays_in_its_row(V):
    x, w = torch.randn(40, 512, device="cuda"), torch.randn(300, 512, device="cuda")
    x[3, 100] = float("nan")
    w[200, 7] = float("inf")
    for fmt, g in (("mx", 1.0), ("nv", 2.0 ** -8)):
        y = V.micro_matmul(V.micro_quantize(x, fmt, g), V.micro_quantize(w, fmt, g), dtype=torch.float32)
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[3], bad[:, 200] = True, True
        assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()
    assert V.micro_matmul(V.micro_quantize(x[:0]), V.micro_quantize(w)).shape == (0, 300)


# ---- how they are called

def test_other_stream_and_graph(V):
    z = torch.randn(64, 5001, device="cuda")
    ids = torch.randint(0, 5001, (64, 9), device="cuda")
    t = torch.randn(64, 9, device="cuda")
    hist = (torch.randint(0, 5001, (640,), device="cuda"), torch.arange(0, 641, 10, device="cuda"))
    rep = torch.full((64,), 1.3, device="cuda")
    w = V.micro_quantize(torch.randn(500, 256, device="cuda"))
    h = torch.randn(64, 256, device="cuda")

    def calls():
        return (V.process_logits(z, output=hist, repetition=rep), *V.distill_step(z, ids, t),
                V.micro_matmul(V.micro_quantize(h), w))
    want = calls()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = calls()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = calls()
    for x in got:
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_repeated_calls_give_the_same_bits(V):
    rng = np.random.default_rng(9)
    z = dev(rng.normal(0, 2, (40, 32001)), "bfloat16")
    ids, t = teacher_lists(rng, 40, 32001, 50, repeat=True)
    hist = csr([list((rng.random(3000) ** 3 * 32001).astype(int)) for _ in range(40)])
    freq = torch.rand(40, device="cuda")
    bias = (hist[0], hist[1], torch.randn(hist[0].numel(), device="cuda"))
    first = (V.process_logits(z, output=hist, frequency=freq, bias=bias), *V.distill_step(z, dev(ids), dev(t)))
    for _ in range(5):
        again = (V.process_logits(z, output=hist, frequency=freq, bias=bias), *V.distill_step(z, dev(ids), dev(t)))
        assert all(torch.equal(a, b) for a, b in zip(again, first))


def test_the_bindings_of_the_c_abi_give_the_same(V):
    from sparse_embedding_bag_gb300 import embbwd as E
    z = torch.randn(3, 400, device="cuda")
    ids, t = torch.randint(0, 400, (3, 5), device="cuda"), torch.randn(3, 5, device="cuda")
    hist, off = csr([[1, 2, 2], [], [399]])
    rep, w = torch.full((3,), 1.5, device="cuda"), torch.rand(3, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, loss, stats = torch.empty_like(z), torch.empty(3, device="cuda"), torch.empty(3, 4, device="cuda")
    E.emb_logits_process(0, z, 0, 400, 3, 400, None, None, 0, hist, off, 4, rep, None, None, None, None, None, 0, None, 0,
                         out, 0, 400, status)
    assert torch.equal(out, V.process_logits(z, output=(hist, off), repetition=rep))
    E.emb_distill_forward(0, z, 0, 400, 3, 400, ids, t, 0, 5, 5, None, 2.0, loss, stats, status)
    want = V.distill_forward(z, ids, t, temperature=2.0)
    assert torch.equal(loss, want[0]) and torch.equal(stats, want[1])
    E.emb_distill_backward(0, z, 0, 400, 3, 400, ids, t, 0, 5, 5, stats, w, 2.0, out, 400, status)
    assert torch.equal(out, V.distill_backward(z, ids, t, stats, w, temperature=2.0))
    E.emb_distill_step(0, z, 0, 400, 3, 400, ids, t, 0, 5, 5, None, w, 2.0, loss, out, 400, status)
    want = V.distill_step(z, ids, t, w, temperature=2.0)
    assert torch.equal(loss, want[0]) and torch.equal(out, want[1])
    m = V.micro_quantize(z, "nv", 0.01)
    codes, scales = torch.empty_like(m.codes), torch.empty_like(m.scales)
    E.emb_micro_quantize(0, z, 0, 400, 3, 400, E.EMB_MICRO_NV, 0.01, codes, scales)
    assert torch.equal(codes, m.codes) and torch.equal(scales, m.scales)
    E.emb_micro_lookup(0, codes, scales, 3, 400, E.EMB_MICRO_NV, 0.01, None, 3, out, 0, 400, status)
    assert torch.equal(out, V.micro_lookup(m))
    y = torch.empty(3, 3, device="cuda")
    E.emb_micro_matmul(0, codes, scales, 0.01, 3, codes, scales, 0.01, 3, 400, E.EMB_MICRO_NV, y, 0, 3, status)
    assert torch.equal(y, V.micro_matmul(m, m, dtype=torch.float32)) and status.item() == 0
    with pytest.raises(E.EmbError):
        E.emb_micro_matmul(0, codes, scales, -1.0, 3, codes, scales, 0.01, 3, 400, E.EMB_MICRO_NV, y, 0, 3, status)
    with pytest.raises(E.EmbError):
        V.distill_step(z, ids, t, temperature=0.0)


def test_bindings_refuse_what_does_not_fit(V):
    z, ids, t = torch.randn(3, 400, device="cuda"), torch.zeros(3, 5, dtype=torch.int64, device="cuda"), \
        torch.randn(3, 5, device="cuda")
    m = V.micro_quantize(z)
    bad = [
        lambda: V.process_logits(z.double()), lambda: V.process_logits(z[0]), lambda: V.process_logits(z.t()),
        lambda: V.process_logits(z, repetition=torch.ones(2, device="cuda")),
        lambda: V.process_logits(z, repetition=torch.ones(3)),
        lambda: V.process_logits(z, prompt=(ids[0], ids[0])),
        lambda: V.process_logits(z, prompt=(ids[0].int(), ids[0, :4])),
        lambda: V.process_logits(z, bias=(ids[0], ids[0, :4])),
        lambda: V.process_logits(z, mask=torch.zeros(3, 12, dtype=torch.int32, device="cuda")),
        lambda: V.process_logits(z, mask=torch.zeros(3, 13, device="cuda")),
        lambda: V.process_logits(z, out=z[:, :399]), lambda: V.process_logits(z, dtype=torch.float64),
        lambda: V.process_logits(z, out=z, dtype=torch.bfloat16), lambda: V.process_logits(z, status=t),
        lambda: V.distill_step(z, ids.int(), t), lambda: V.distill_step(z, ids[:2], t[:2]),
        lambda: V.distill_step(z, ids, t[:, :4]), lambda: V.distill_step(z, ids, t.double()),
        lambda: V.distill_step(z, ids, t, out=z.bfloat16()), lambda: V.distill_step(z, ids, t, torch.ones(4, device="cuda")),
        lambda: V.distill_step(z, ids, t, teacher_lse=torch.ones(3)), lambda: V.distill_backward(z, ids, t, t),
        lambda: V.micro_quantize(z, "fp4"), lambda: V.micro_quantize(z.long()),
        lambda: V.micro_quantize(z, "nv", 0.1, out=m), lambda: V.micro_quantize(z[:2], out=m),
        lambda: V.micro_lookup(m, ids[0].int()), lambda: V.micro_lookup(m, out=z[:2]),
        lambda: V.micro_lookup(m, dtype=torch.int32), lambda: V.micro_matmul(m, V.micro_quantize(z, "nv", 0.1)),
        lambda: V.micro_matmul(m, V.micro_quantize(z[:, :64])), lambda: V.micro_matmul(m, m, out=z),
        lambda: V.micro_matmul(m, V.MicroMatrix(m.codes, m.scales, 4, 400, "mx")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")


def test_lm_head_serves_and_learns(V):
    from sparse_embedding_bag_gb300 import lm_head
    g = torch.Generator(device="cuda").manual_seed(3)
    n_vocab, dim, N, K = 1003, 64, 48, 8
    table = torch.randn((n_vocab, dim), generator=g, device="cuda") * 0.1
    layer = torch.randn((dim, dim), generator=g, device="cuda") * dim ** -0.5
    allowed = np.zeros((2, (n_vocab + 31) // 32 * 32), bool)
    allowed[0, 500:520], allowed[1, [7, 1002]] = True, True
    mask = torch.from_numpy(np.packbits(allowed, axis=1, bitorder="little").view(np.int32)).cuda()
    for fmt in ("mx", "nv"):
        out = lm_head.serve(table.bfloat16(), layer.bfloat16(), [[1, 2, 3], [4]], 5, format=fmt, mask=mask)
        assert all(500 <= v < 520 for v in out[0]) and all(v in (7, 1002) for v in out[1])
    tokens = torch.randint(0, n_vocab, (N,), generator=g, device="cuda")
    ids = torch.stack([torch.randperm(n_vocab, generator=g, device="cuda")[:K] for _ in range(N)])
    teacher = torch.randn((N, K), generator=g, device="cuda") * 2
    ref_table = table.clone().requires_grad_()
    losses = lm_head.distill(table, layer, tokens, ids, teacher, lr=5.0, steps=12)
    assert losses[-1] < 0.8 * losses[0] and all(b < a for a, b in zip(losses, losses[1:]))
    # the first loss, and through autograd the direction of the table's whole gradient
    hidden = torch.tanh(ref_table[tokens] @ layer)
    loss = V.distill_loss(hidden @ ref_table.t(), ids, teacher, temperature=2.0).mean()
    assert abs(loss.item() - losses[0]) <= 1e-4 * losses[0]
    loss.backward()
    assert ((table - ref_table.detach()) * ref_table.grad).sum() < 0
