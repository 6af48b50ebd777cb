"""The vocabulary operators of a language model, as cases to measure and in their plain form.

``logits``   penalties for repeated tokens, biases and grammar masks on logits (serving)
``distill``  distillation from a teacher's top logits: forward, backward, and both in one step
``micro``    rows quantised to microscaled 4-bit floating point and read back
``product``  hidden states times a microscaled 4-bit table: quantise the rows, multiply

With ``own`` false every operator is computed by elementary torch operations in 32 bits; with
``own`` true by the calls of ``sparse_embedding_bag_gb300.vocab``.
"""
import math

import numpy as np
import torch

own = False

F16, BF16, F32 = "float16", "bfloat16", "float32"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the codes 0..7; bit 3 is the sign
MX, NV = "mx", "nv"
BLOCK = {MX: 32, NV: 16}  # elements that share a scale
X_MAX, W_MAX = 6.5, 0.13  # calibrated magnitudes of activations and of a table, for the NV tensor scales


def listed():
    return [
        # one request of an assistant, long prompt, constrained by a grammar: latency between two tokens
        dict(name="logits one request", op="logits", B=1, V=128256, dtype=BF16, out=F32, prompt=2000, output=300,
             bias=0, mask=True, pad=0),
        # a serving batch with per-request biases, logits from an fp32 head
        dict(name="logits batch", op="logits", B=64, V=128256, dtype=F32, out=F32, prompt=1500, output=500, bias=20,
             mask=True, pad=0),
        # the largest batch: long conversations, no grammar, an odd vocabulary
        dict(name="logits large", op="logits", B=512, V=131071, dtype=BF16, out=BF16, prompt=3000, output=1000, bias=0,
             mask=False, pad=0),
        # a micro-batch of a small model with an odd vocabulary, teacher renormalised over its top 8
        dict(name="distill step small", op="distill", dir="step", N=16, V=32001, K=8, dtype=F32, tail=False, tau=2.0,
             pad=0),
        # the training step over a full batch of tokens, with the teacher's remaining mass
        dict(name="distill step", op="distill", dir="step", N=4096, V=128256, K=64, dtype=BF16, tail=True, tau=1.0,
             pad=0),
        # validation loss, fp32 logits
        dict(name="distill forward", op="distill", dir="forward", N=1024, V=128256, K=32, dtype=F32, tail=True, tau=1.0,
             pad=0),
        # a backward of its own (the gradient of the loss arrives later), odd vocabulary, fp16
        dict(name="distill backward", op="distill", dir="backward", N=2048, V=50001, K=100, dtype=F16, tail=False,
             tau=2.0, pad=0),
        # the token table laid out in 4 bits and read back whole
        dict(name="micro table", op="micro", R=128256, K=4096, dtype=BF16, fmt=MX, pad=0),
        # the activations of a few tokens, an odd width
        dict(name="micro rows", op="micro", R=17, K=4100, dtype=F32, fmt=NV, pad=0),
        # next-token logits of one request against the 4-bit token table
        dict(name="product one token", op="product", M=1, N=128256, K=4096, dtype=BF16, out=BF16, fmt=MX),
        # a decoding batch of odd size, odd vocabulary and width
        dict(name="product batch", op="product", M=97, N=50001, K=2056, dtype=BF16, out=F16, fmt=NV),
        # logits of a whole prompt
        dict(name="product prompt", op="product", M=2048, N=128256, K=4096, dtype=BF16, out=BF16, fmt=NV),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logits", "distill", "micro", "product"])
    if op == "logits":
        V = _log_int(rng, 1000, 200000)
        B = _log_int(rng, 1, min(512, 512 * 131071 // V))
        return dict(op=op, B=B, V=V, dtype=rng.choice([F32, F16, BF16]), out=rng.choice([F32, F32, BF16, F16]),
                    prompt=rng.choice([0, _log_int(rng, 1, 4000)]), output=rng.choice([0, _log_int(rng, 1, 2000)]),
                    bias=rng.choice([0, _log_int(rng, 1, 300)]), mask=rng.random() < 0.6, pad=rng.choice([0, 0, 64]))
    if op == "distill":
        V = _log_int(rng, 1000, 200000)
        N = _log_int(rng, 1, min(4096, 4096 * 128256 // (2 * V)))
        return dict(op=op, dir=rng.choice(["forward", "backward", "step"]), N=N, V=V, K=_log_int(rng, 1, 256),
                    dtype=rng.choice([F32, F16, BF16]), tail=rng.random() < 0.5, tau=rng.choice([1.0, 2.0, 0.7]),
                    pad=rng.choice([0, 0, 64]))
    K = _log_int(rng, 64, 8192)
    if op == "micro":
        R = _log_int(rng, 1, min(128256, 128256 * 4096 // K))
        return dict(op=op, R=R, K=K, dtype=rng.choice([F32, F16, BF16]), fmt=rng.choice([MX, NV]),
                    pad=rng.choice([0, 0, 64]))
    N = _log_int(rng, 100, min(128256, 128256 * 4096 // K))
    M = _log_int(rng, 1, 2048)
    return dict(op=op, M=M, N=N, K=K, dtype=rng.choice([F32, F16, BF16]), out=rng.choice([F16, BF16]),
                fmt=rng.choice([MX, NV]))


# ---------------------------------------------------------------- inputs

def _gen(seed, *words):
    s = np.random.SeedSequence([int(seed) & 0xffffffff, *words]).generate_state(1, np.uint64)[0]
    return torch.Generator(device="cuda").manual_seed(int(s) & (2 ** 63 - 1))


def _rows(t, pad):
    """The rows of `t` inside a wider buffer: a row stride of its own."""
    if not pad:
        return t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _lengths(B, mean, seed):
    """Ragged lengths from none to twice the mean, the last row at the mean: the same total for every seed."""
    if B == 1 or mean == 0:
        return np.full(B, mean, np.int64)
    n = np.round(np.linspace(0, 2 * mean, B)).astype(np.int64)
    return np.random.default_rng(seed).permutation(n)


def _history(g, B, V, mean, seed):
    """CSR lists of token ids, skewed to low ids so that tokens repeat: (ids, offsets)."""
    n = _lengths(B, mean, seed)
    off = np.concatenate([[0], np.cumsum(n)])
    u = torch.rand(int(off[-1]), generator=g, device="cuda", dtype=torch.float64)
    return (u.pow(3) * V).long().clamp_(max=V - 1), torch.from_numpy(off).cuda()


def _distinct(g, rows, count, V):
    """`count` distinct ids in each row."""
    step = 7919
    while V % step == 0 or count > V:
        step += 2
    a = torch.randint(0, V, (rows, 1), generator=g, device="cuda")
    return (a + torch.arange(count, device="cuda") * step) % V


def prepare(case, seed):
    g = _gen(seed, 1)
    op = case["op"]
    s = dict(case)
    if op == "logits":
        B, V = case["B"], case["V"]
        z = torch.randn((B, V), generator=g, device="cuda") * 3.0
        s["logits"] = _rows(z.to(getattr(torch, case["dtype"])), case["pad"])
        s["prompt_csr"] = _history(g, B, V, case["prompt"], seed + 1) if case["prompt"] else None
        s["output_csr"] = _history(g, B, V, case["output"], seed + 2) if case["output"] else None
        u = torch.rand((3, B), generator=g, device="cuda")
        s["repetition"], s["frequency"], s["presence"] = 1.0 + 0.5 * u[0], u[1] - 0.25, u[2].clone()
        s["bias_csr"] = None
        if case["bias"]:
            n = torch.full((B,), min(case["bias"], V), dtype=torch.int64, device="cuda")
            ids = _distinct(g, B, int(min(case["bias"], V)), V).reshape(-1)
            off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), n.cumsum(0)])
            val = torch.randn(ids.numel(), generator=g, device="cuda") * 5.0
            s["bias_csr"] = (ids, off, val)
        s["mask"] = None
        if case["mask"]:  # most rows free, some strict (few tokens left), one where nothing is left
            words = -(-V // 32)
            keep = torch.rand((B, words * 32), generator=g, device="cuda")
            row = torch.arange(B, device="cuda")
            limit = torch.where(row % 3 == 0, 0.02, torch.where(row % 3 == 1, 2.0, 0.5))
            limit = torch.where(row == 7, -1.0, limit)
            bits = (keep < limit[:, None]).reshape(B, words, 32).long() << torch.arange(32, device="cuda")
            s["mask"] = bits.sum(-1).to(torch.int32)  # bit v % 32 of word v // 32: token v allowed
        return s
    if op == "distill":
        N, V, K = case["N"], case["V"], min(case["K"], case["V"])
        z = torch.empty((N, V), device="cuda", dtype=getattr(torch, case["dtype"])).normal_(0, 1.5, generator=g)
        ids = _distinct(g, N, K, V)
        k = torch.arange(K, device="cuda")
        t = 9.0 - 6.0 * torch.log1p(k.float())[None] + torch.randn((N, K), generator=g, device="cuda")
        near = t + torch.randn((N, K), generator=g, device="cuda") + 4.0  # the student agrees with the teacher roughly
        z.scatter_(1, ids, near.to(z.dtype))
        row = torch.arange(N, device="cuda")
        short = (row % 8 == 3)[:, None] & (k[None] >= (K + 1) // 2)  # lists cut short, padded with -1
        none = (row % 32 == 31)[:, None].expand(N, K)                # rows that take no part (prompt tokens)
        s["ids"] = torch.where(short | none, -1, ids)
        s["teacher"] = t
        s["lse"] = None
        if case["tail"]:
            lt = torch.where(s["ids"] >= 0, t / case["tau"], -math.inf)
            rest = 0.01 + 0.2 * torch.rand(N, generator=g, device="cuda")
            s["lse"] = torch.logsumexp(lt, -1) - torch.log1p(-rest)
            s["lse"] = torch.where(row % 32 == 31, 0.0, s["lse"])
        w = torch.rand(N, generator=g, device="cuda") + 0.5
        s["weight"] = w if case["dtype"] == F16 else w / N  # fp16 gradients are trained under a loss scale
        s["logits"] = _rows(z, case["pad"])
        if case["dir"] == "backward":
            s["stats"] = _distill_forward(s)[1]
        return s
    if op == "micro":
        x = torch.randn((case["R"], case["K"]), generator=g, device="cuda")
        x *= 0.02 * torch.exp(0.5 * torch.randn((case["R"], 1), generator=g, device="cuda"))
        s["x"] = _rows(x.to(getattr(torch, case["dtype"])), case["pad"])
        s["scale"] = _tensor_scale(case["fmt"], W_MAX)
        return s
    x = torch.randn((case["M"], case["K"]), generator=g, device="cuda").clamp_(-X_MAX, X_MAX)
    s["x"] = x.to(getattr(torch, case["dtype"]))
    s["x_scale"], s["w_scale"] = _tensor_scale(case["fmt"], X_MAX), _tensor_scale(case["fmt"], W_MAX)
    codes, scales = [], []
    for r in range(0, case["N"], 16384):  # the table is laid out in 4 bits once, when it is loaded
        w = torch.randn((min(16384, case["N"] - r), case["K"]), generator=g, device="cuda") * 0.02
        c, b = _micro_quantize(w, case["fmt"], s["w_scale"])
        codes.append(c)
        scales.append(b)
    s["w_codes"], s["w_scales"] = _pack(torch.cat(codes)), _tile(torch.cat(scales))
    return s


# ---------------------------------------------------------------- 4-bit layout and plain forms

def _tensor_scale(fmt, amax):
    """The fp32 scale of the whole tensor: NV spreads `amax` over the range of its block scales; MX has none."""
    return float(np.float32(amax / (6.0 * 448.0))) if fmt == NV else 1.0


def _micro_quantize(x, fmt, scale):
    """Codes [R, Kp] (uint8, 0..15) and block scales [R, Kp / block] (their bytes), Kp = K rounded up to 32."""
    R, K = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -K % 32)).reshape(R, -1, BLOCK[fmt])
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    if fmt == MX:  # the power of two that brings the largest magnitude to [4, 8)
        e = ((amax.view(torch.int32) >> 23) - 129).clamp(-127, 125)
        byte = torch.where(bad, 255, e + 127).to(torch.uint8)
        inv = ((127 - e) << 23).view(torch.float32)
    else:
        s8 = (amax / (6.0 * torch.tensor(scale, device=x.device))).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte = torch.where(bad, torch.full_like(s8.view(torch.uint8), 0x7f), s8.view(torch.uint8))
        d = s8.float() * scale
        inv = torch.where(d >= 2.0 ** -126, 1.0 / d, 0.0)
    y = x * inv[..., None]
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = torch.where(bad[..., None], 0, code + 8 * torch.signbit(y).to(torch.uint8))
    return code.to(torch.uint8).reshape(R, -1), byte


def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _tile(byte):
    """Block scales in tiles of 128 rows x 4 blocks, 512 bytes each: byte (r % 32) * 16 + (r % 128 // 32) * 4 + j % 4."""
    R, J = byte.shape
    byte = torch.nn.functional.pad(byte, (0, -J % 4, 0, -R % 128))
    t = byte.reshape(byte.shape[0] // 128, 4, 32, byte.shape[1] // 4, 4)
    return t.permute(0, 3, 2, 1, 4).contiguous()


def _values(code, byte, fmt, scale):
    """What the codes [R, Kp] and scale bytes [R, Kp / block] stand for, in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    v = table[code.int()].reshape(code.shape[0], -1, BLOCK[fmt])
    if fmt == MX:
        bits = torch.where(byte == 0, 1 << 22, byte.int() << 23)  # 2^(byte - 127); 2^-127 is subnormal
        s = torch.where(byte == 255, math.nan, bits.to(torch.int32).view(torch.float32))
        return (v * s[..., None]).reshape(code.shape)
    return (v * byte.view(torch.float8_e4m3fn).float()[..., None] * scale).reshape(code.shape)


def _unpack(codes, scales, fmt, R):
    code = torch.stack([codes & 15, codes >> 4], -1).reshape(R, -1)
    t = scales.permute(0, 3, 2, 1, 4)
    byte = t.reshape(t.shape[0] * 128, -1)[:R, :code.shape[1] // BLOCK[fmt]]
    return code, byte.contiguous()


def _counts(csr, B, V):
    ids, off = csr
    row = torch.repeat_interleave(torch.arange(B, device="cuda"), off[1:] - off[:-1], output_size=ids.numel())
    return torch.zeros(B * V, device="cuda").scatter_add_(0, row * V + ids, torch.ones_like(ids, dtype=torch.float32)).view(B, V)


def _process_logits(s):
    B, V = s["B"], s["V"]
    y = s["logits"].float()
    count = _counts(s["output_csr"], B, V) if s["output_csr"] else torch.zeros((B, V), device="cuda")
    seen = count > 0
    if s["prompt_csr"]:
        seen = seen | (_counts(s["prompt_csr"], B, V) > 0)
    rep = s["repetition"][:, None]
    y = torch.where(seen, torch.where(y > 0, y / rep, y * rep), y)
    y = y - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias_csr"]:
        ids, off, val = s["bias_csr"]
        row = torch.repeat_interleave(torch.arange(B, device="cuda"), off[1:] - off[:-1], output_size=ids.numel())
        y = y.reshape(-1).scatter_add(0, row * V + ids, val).view(B, V)
    if s["mask"] is not None:
        bit = (s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        y = torch.where(bit.reshape(B, -1)[:, :V] != 0, y, -math.inf)
    return y.to(getattr(torch, s["out"]))


def _distill_terms(s):
    z, ids, tau = s["logits"].float(), s["ids"], s["tau"]
    valid = ids >= 0
    lt = torch.where(valid, s["teacher"].float() / tau, -math.inf)
    if s["lse"] is None:
        big = lt.amax(-1, keepdim=True)
        big = torch.where(torch.isfinite(big), big, 0.0)
        tl = (big + (lt - big).exp().sum(-1, keepdim=True).log()).squeeze(-1)
    else:
        tl = s["lse"]
    return z, ids, tau, valid, lt, torch.where(valid.any(-1), tl, 0.0)


def _distill_forward(s):
    """(loss [N], stats [N, 4] = largest logit, sum of exp((z - largest) / tau), coefficient off the list, teacher's lse)."""
    z, ids, tau, valid, lt, tl = _distill_terms(s)
    N, V = z.shape
    top = torch.zeros((N, V + 1), dtype=torch.bool, device="cuda").scatter_(1, torch.where(valid, ids, V), True)[:, :V]
    m = z.amax(-1, keepdim=True)
    e = ((z - m) / tau).exp()
    rest = torch.where(top, 0.0, e).sum(-1)
    total = rest + torch.where(top, e, 0.0).sum(-1)
    logq = lt - tl[:, None]
    q = logq.exp()
    logp = (z.gather(1, ids.clamp(min=0)) - m) / tau - total.log()[:, None]
    loss = torch.where(q > 0, q * (logq - logp), 0.0).sum(-1)
    coef = torch.ones_like(loss)
    if s["lse"] is not None:
        r = (1.0 - q.sum(-1)).clamp(min=0.0)
        u = rest / total
        loss = loss + torch.where(r > 0, r * (r.log() - u.log()), 0.0)
        coef = torch.where(r > 0, 1.0 - r / u, 1.0)
    part = valid.any(-1)
    stats = torch.stack([m.squeeze(-1), total, coef, tl], -1)
    empty = torch.tensor([0.0, 1.0, 0.0, 0.0], device="cuda")
    return torch.where(part, tau * tau * loss, 0.0), torch.where(part[:, None], stats, empty)


def _distill_backward(s, stats):
    z, ids, tau, valid, lt, tl = _distill_terms(dict(s, lse=stats[:, 3]))
    N, V = z.shape
    p = ((z - stats[:, :1]) / tau).exp() / stats[:, 1:2]
    at = torch.where(valid, ids, V)
    top = torch.zeros((N, V + 1), dtype=torch.bool, device="cuda").scatter_(1, at, True)[:, :V]
    q = torch.zeros((N, V + 1), device="cuda").scatter_add_(1, at, (lt - tl[:, None]).exp())[:, :V]
    grad = s["weight"][:, None] * tau * (torch.where(top, p, stats[:, 2:3] * p) - q)
    return torch.where(valid.any(-1)[:, None], grad, 0.0).to(s["logits"].dtype)


def run(state):
    s, op = state, state["op"]
    if own:
        from sparse_embedding_bag_gb300 import vocab
        if op == "logits":
            return vocab.process_logits(s["logits"], prompt=s["prompt_csr"], output=s["output_csr"],
                                        repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                                        bias=s["bias_csr"], mask=s["mask"], dtype=getattr(torch, s["out"]))
        if op == "distill":
            if s["dir"] == "forward":
                return vocab.distill_forward(s["logits"], s["ids"], s["teacher"], temperature=s["tau"],
                                             teacher_lse=s["lse"])
            if s["dir"] == "backward":
                return vocab.distill_backward(s["logits"], s["ids"], s["teacher"], s["stats"], s["weight"],
                                              temperature=s["tau"])
            return vocab.distill_step(s["logits"], s["ids"], s["teacher"], s["weight"], temperature=s["tau"],
                                      teacher_lse=s["lse"])
        if op == "micro":
            m = vocab.micro_quantize(s["x"], s["fmt"], s["scale"])
            return vocab.micro_lookup(m, dtype=torch.float32 if s["fmt"] == NV else torch.bfloat16)
        w = vocab.MicroMatrix(s["w_codes"], s["w_scales"], s["N"], s["K"], s["fmt"], s["w_scale"])
        x = vocab.micro_quantize(s["x"], s["fmt"], s["x_scale"])
        return vocab.micro_matmul(x, w, dtype=getattr(torch, s["out"]))
    if op == "logits":
        return _process_logits(s)
    if op == "distill":
        if s["dir"] == "backward":
            return _distill_backward(s, s["stats"])
        loss, stats = _distill_forward(s)
        return (loss, stats) if s["dir"] == "forward" else (loss, _distill_backward(s, stats))
    if op == "micro":
        code, byte = _micro_quantize(s["x"], s["fmt"], s["scale"])
        out = torch.float32 if s["fmt"] == NV else torch.bfloat16
        return _values(code, byte, s["fmt"], s["scale"])[:, :s["K"]].to(out)
    code, byte = _micro_quantize(s["x"], s["fmt"], s["x_scale"])
    x = _values(code, byte, s["fmt"], s["x_scale"])
    w = _values(*_unpack(s["w_codes"], s["w_scales"], s["fmt"], s["N"]), s["fmt"], s["w_scale"])
    return (x @ w.t()).to(getattr(torch, s["out"]))


# ---------------------------------------------------------------- what a pass cannot do without

def _size(dtype):
    return 4 if dtype == F32 else 2


def _packed_bytes(rows, K, fmt):
    return rows * K / 2 + rows * K / BLOCK[fmt]


def work(case):
    op = case["op"]
    if op == "logits":
        B, V = case["B"], case["V"]
        ids = B * (case["prompt"] + case["output"])
        by = B * V * (_size(case["dtype"]) + _size(case["out"])) + 8 * ids + 12 * B * case["bias"] + 12 * B
        return {"bytes": by + (B * V / 8 if case["mask"] else 0), "flops": B * V + 4 * ids}
    if op == "distill":
        N, V, K = case["N"], case["V"], min(case["K"], case["V"])
        part = N - N // 32  # rows with a list; of the others only the gradient is written
        size = _size(case["dtype"])
        by = part * V * size + 12 * N * K + 8 * N + (4 * N if case["tail"] else 0)
        by += 16 * N if case["dir"] != "step" else 0
        by += N * V * size if case["dir"] != "forward" else 0
        return {"bytes": by, "flops": part * V * {"forward": 4, "backward": 4, "step": 8}[case["dir"]]}
    if op == "micro":
        R, K = case["R"], case["K"]
        values = R * K * (4 if case["fmt"] == NV else 2)
        return {"bytes": R * K * _size(case["dtype"]) + 2 * _packed_bytes(R, K, case["fmt"]) + values, "flops": 5 * R * K}
    M, N, K = case["M"], case["N"], case["K"]
    by = M * K * _size(case["dtype"]) + _packed_bytes(N, K, case["fmt"]) + 2 * M * N
    return {"bytes": by, "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the definitions in 64 bits

def _nearest(v, step):
    return torch.round(v / step) * step  # halves go to the even multiple


def _exact_micro(x, fmt, scale):
    """x [R, K] in 64 bits as its microscaled values."""
    R, K = x.shape
    n = BLOCK[fmt]
    x = torch.cat([x, x.new_zeros((R, -K % n))], 1).view(R, -1, n)
    big = x.abs().max(-1).values
    power = lambda v: torch.where(v > 0, v / torch.frexp(v).mantissa, 0.0)  # the power of two above v, exactly  # noqa: E731
    if fmt == MX:
        d = (power(big) / 8).clamp(min=2.0 ** -127)
    else:
        t = big / (6.0 * scale)
        d = _nearest(t, power(t).clamp(min=2.0 ** -5) / 16).clamp(max=448.0) * scale
    y = torch.where(d[..., None] > 0, x.abs() / d[..., None], 0.0)
    grid = torch.where(y < 2, _nearest(y, 0.5), torch.where(y < 4, _nearest(y, 1.0), _nearest(y, 2.0))).clamp(max=6.0)
    return (torch.sign(x) * grid * d[..., None]).view(R, -1)[:, :K]


def _exact_table(s, lo, hi):
    """Rows lo..hi of the packed table in 64 bits, each scale fetched from its place in the tiles."""
    K, fmt = s["K"], s["fmt"]
    byte = s["w_codes"][lo:hi].long()
    r, k = torch.arange(lo, hi, device="cuda")[:, None], torch.arange(K, device="cuda")[None]
    code = (byte[:, (k[0] // 2)] >> (4 * (k % 2))) & 15
    m = code & 7
    mag = torch.where(m < 2, m * 0.5, (1 + 0.5 * (m & 1)) * torch.exp2((m >> 1).double() - 1))
    j = torch.arange(-(-K // BLOCK[fmt]), device="cuda")[None]
    at = ((r // 128) * s["w_scales"].shape[1] + j // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + j % 4
    b = s["w_scales"].reshape(-1)[at].long()
    if fmt == MX:
        d = torch.exp2(b.double() - 127)
    else:
        e, f = (b >> 3) & 15, (b & 7).double()
        d = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.double() - 7), f * 2.0 ** -9) * s["w_scale"]
    return torch.where(code >= 8, -mag, mag) * d.repeat_interleave(BLOCK[fmt], 1)[:, :K]


def _exact_logits(s):
    B, V = s["B"], s["V"]
    out = s["logits"].double().clone()
    lists = {}
    for name in ("prompt_csr", "output_csr", "bias_csr"):
        lists[name] = s[name] and [x.cpu() if i == 1 else x for i, x in enumerate(s[name])]
    for b in range(B):
        part = lambda name: (lists[name][0][lists[name][1][b]:lists[name][1][b + 1]] if lists[name] else torch.empty(0, dtype=torch.int64, device="cuda"))  # noqa: E731
        rep, freq, pres = (s[n][b].double() for n in ("repetition", "frequency", "presence"))
        said, times = torch.unique(part("output_csr"), return_counts=True)
        ever = torch.unique(torch.cat([said, part("prompt_csr")]))
        v = out[b, ever]
        out[b, ever] = torch.where(v > 0, v / rep, v * rep)
        out[b, said] -= freq * times + pres
        if lists["bias_csr"]:
            lo, hi = lists["bias_csr"][1][b], lists["bias_csr"][1][b + 1]
            out[b, part("bias_csr")] += s["bias_csr"][2][lo:hi].double()
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        allowed = (s["mask"].long()[:, v // 32] >> (v % 32)) % 2 == 1
        out[~allowed] = -math.inf
    return out


def _exact_distill(s):
    z, tau = s["logits"], s["tau"]
    N, V = z.shape
    loss = torch.zeros(N, dtype=torch.float64, device="cuda")
    stats = torch.zeros((N, 4), dtype=torch.float64, device="cuda")
    stats[:, 1] = 1.0
    grad = torch.zeros((N, V), dtype=torch.float64 if N * V < 3e8 else torch.float32, device="cuda")
    for lo in range(0, N, 256):
        ids = s["ids"][lo:lo + 256]
        some = (ids >= 0).any(-1).nonzero().squeeze(-1)
        if not len(some):
            continue
        ids = ids[some]
        n = lo + some
        x = z[n].double() / tau
        t = torch.where(ids >= 0, s["teacher"][n].double() / tau, -math.inf)
        norm = torch.logsumexp(t, -1) if s["lse"] is None else s["lse"][n].double()
        q = (t - norm[:, None]).exp()
        logp = x - torch.logsumexp(x, -1, keepdim=True)
        wide = torch.zeros((len(n), V + 1), dtype=torch.float64, device="cuda")
        spot = torch.where(ids >= 0, ids, V)
        on = wide.scatter(1, spot, 1.0)[:, :V]
        target = wide.scatter_add(1, spot, q)[:, :V]
        there = logp.gather(1, ids.clamp(min=0))
        ls = torch.where(q > 0, q * (q.clamp(min=1e-300).log() - there), 0.0).sum(-1)
        coef = torch.ones_like(ls)
        if s["lse"] is not None:
            r = 1.0 - q.sum(-1)
            u = (logp.exp() * (1 - on)).sum(-1)
            ls = ls + r * (r / u).log()
            coef = 1.0 - r / u
        loss[n] = tau * tau * ls
        peak = z[n].double().amax(-1)
        stats[n] = torch.stack([peak, ((z[n].double() - peak[:, None]) / tau).exp().sum(-1), coef, norm], -1)
        if s["dir"] != "forward":
            if s["dir"] == "backward":
                coef = s["stats"][n, 2].double()
            grad[n] = (s["weight"][n].double()[:, None] * tau * (logp.exp() * (on + (1 - on) * coef[:, None]) - target)).to(grad.dtype)
    return (loss, stats) if s["dir"] == "forward" else grad if s["dir"] == "backward" else (loss, grad)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "logits":
        return _exact_logits(s)
    if op == "distill":
        return _exact_distill(s)
    if op == "micro":
        out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for r in range(0, case["R"], 8192):
            out[r:r + 8192] = _exact_micro(s["x"][r:r + 8192].double(), case["fmt"], s["scale"])
        return out
    x = _exact_micro(s["x"].double(), case["fmt"], s["x_scale"])
    out = torch.empty((case["M"], case["N"]), dtype=torch.float64, device="cuda")
    for r in range(0, case["N"], 8192):
        out[:, r:r + 8192] = x @ _exact_table(s, r, min(r + 8192, case["N"])).t()
    return out
