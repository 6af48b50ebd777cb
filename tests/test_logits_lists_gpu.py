"""Logits processing with long lists and wide slices: biases beyond a block's threads, tokens that
repeat among them, outputs too long for 16-bit counts, in place, in slices of one round of loads and of
several. Against the 64-bit reference with its bounds."""
import numpy as np
import pytest

import _vocab_ref as R
from test_vocab_gpu import DTYPES, V, close, csr, dev, f64  # noqa: F401 (V is a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def check(V, rng, z, out, prompt, output, bias, mask, inplace=False):
    """bias: (ids, values) of each row."""
    B = z.shape[0]
    rep, freq, pres = (rng.uniform(*r, B).astype(np.float32) for r in ((0.8, 1.6), (-0.5, 0.5), (-1, 1)))
    pairs = [list(zip(i.tolist(), x.astype(float).tolist())) for i, x in bias]
    y, tol = R.process_logits(f64(z), prompt, output, rep.astype(float), freq.astype(float), pres.astype(float), pairs,
                              mask)
    ids, off = csr([i for i, _ in bias])
    values = dev(np.concatenate([x for _, x in bias]))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = V.process_logits(z, prompt=csr(prompt), output=csr(output), repetition=dev(rep), frequency=dev(freq),
                           presence=dev(pres), bias=(ids, off, values), mask=None if mask is None else dev(mask),
                           status=status, **(dict(out=z) if inplace else dict(dtype=getattr(torch, out))))
    close(f64(got), y, tol + R.rounding(np.where(np.isfinite(y), y, 0), out) * 1.01)
    assert status.item() == 0


def biases(rng, B, n_vocab, n, repeats):
    """n biases a row, a share `repeats` of them of tokens named before."""
    out = []
    for b in range(B):
        ids = rng.permutation(n_vocab)[:n] if n <= n_vocab else rng.integers(0, n_vocab, n)
        again = rng.random(n) < repeats
        ids[again] = ids[rng.integers(0, n, again.sum())]
        out.append((ids.astype(np.int64), rng.normal(0, 4, n).astype(np.float32)))
    return out


def words(rng, B, n_vocab):
    return rng.integers(0, 1 << 32, (B, (n_vocab + 31) // 32), dtype=np.uint64).astype(np.uint32).view(np.int32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("n_vocab,n,repeats", [(1500, 700, 0.0), (1500, 700, 0.02), (5003, 4000, 0.5), (90, 3000, 0.9),
                                               (40001, 9000, 0.001)])
def test_biases_beyond_a_block_of_threads(V, dtype, inplace, n_vocab, n, repeats):
    rng = np.random.default_rng(n_vocab + n)
    B = 3
    z = dev(rng.normal(0, 3, (B, n_vocab)), dtype)
    lists = [[list(rng.integers(0, n_vocab, 200)) for _ in range(B)] for _ in range(2)]
    check(V, rng, z, dtype, *lists, biases(rng, B, n_vocab, n, repeats), words(rng, B, n_vocab), inplace)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inplace", [False, True])
def test_long_outputs_with_biases_and_masks(V, dtype, inplace):
    rng = np.random.default_rng(11)
    B, n_vocab = 4, 20011
    z = dev(rng.normal(0, 3, (B, n_vocab)), dtype)
    output = [list((rng.random(n) ** 3 * n_vocab).astype(int)) for n in (16383, 16384, 40000, 0)]
    prompt = [list(rng.integers(0, n_vocab, 3000)) for _ in range(B)]
    check(V, rng, z, dtype, prompt, output, biases(rng, B, n_vocab, 600, 0.1), words(rng, B, n_vocab), inplace)


@pytest.mark.parametrize("dtype,out", [("float32", "float32"), ("bfloat16", "bfloat16"), ("bfloat16", "float32")])
@pytest.mark.parametrize("B,n_vocab", [(64, 128256), (114, 131071)])
def test_slices_of_a_serving_batch(V, dtype, out, B, n_vocab):
    # slices of 18432 and 32768 tokens: several rounds of a block's loads; some outputs take the
    # wide counts, in pieces of half a slice
    rng = np.random.default_rng(B)
    z = dev(rng.normal(0, 3, (B, n_vocab)), dtype, 0 if n_vocab % 8 == 0 else 1)
    prompt = [list((rng.random(rng.integers(0, 800)) ** 3 * n_vocab).astype(int)) for _ in range(B)]
    output = [list((rng.random(20000 if b % 40 == 5 else rng.integers(0, 300)) ** 3 * n_vocab).astype(int))
              for b in range(B)]
    check(V, rng, z, out, prompt, output, biases(rng, B, n_vocab, 20, 0.05), words(rng, B, n_vocab))


def test_a_repeated_bias_does_not_make_a_long_list_quadratic(V):
    # one token twice in a list of 30000: 256 threads that each went over the whole list for each of
    # their entries would take over ten times as long as for a list without the repeated token
    n_vocab, n = 30000, 30000
    z = torch.randn(1, n_vocab, device="cuda")
    ids = torch.randperm(n_vocab, device="cuda")
    off, x = torch.tensor([0, n], device="cuda"), torch.randn(n, device="cuda")
    twice = ids.clone()
    twice[-1] = twice[0]

    def ms(ids):
        call = lambda: V.process_logits(z, bias=(ids, off, x))  # noqa: E731
        for _ in range(3):
            call()
        best = []
        for _ in range(10):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            b.synchronize()
            best.append(a.elapsed_time(b))
        return min(best)
    plain, repeated = ms(ids), ms(twice)
    print(f"distinct {plain * 1e3:.0f} us, one repeated {repeated * 1e3:.0f} us")
    assert repeated < 10 * plain


def test_an_output_list_too_long_to_count(V):
    # 2^30 times one token would run into the flags beside its count
    n = (1 << 30) + 5
    ids, z = torch.full((n + 3,), 2, dtype=torch.int64, device="cuda"), torch.randn(2, 100, device="cuda")
    ids[-3:] = 7
    ones, status = torch.ones(2, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = V.process_logits(z, output=(ids, torch.tensor([0, n, n + 3], device="cuda")), frequency=ones, presence=ones,
                           status=status)
    want = z.clone()
    want[1, 7] = want[1, 7] - 3 - 1
    assert status.item() == 2
    torch.testing.assert_close(got, want, rtol=1e-6, atol=1e-6)
