"""The vocabulary operators together, as a language model with a tied token table uses them.

    python -m sparse_embedding_bag_gb300.lm_head [--vocab 32001] [--dim 512] [--tokens 256] [--steps 8]

Serving: the token table is laid out in 4 bits once; a step looks the last tokens up in it,
multiplies the hidden states with it, applies each request's penalties, biases and grammar mask to
the logits, and takes the largest. Training: the student's logits come from the full-precision
table, ``distill_step`` gives the loss against a teacher's top logits and the logits' gradient, and
the table is updated through both of its sides: the output side by a dense SGD step, the looked-up
rows by ``emb_nobag_bwd_sgd``. The model between lookup and head is one linear layer.
"""
from __future__ import annotations

import argparse

import numpy as np
import torch

from . import embbwd as E
from . import vocab


def csr(lists, device):
    """(ids, offsets) of a list of token lists."""
    offsets = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int64)
    ids = np.concatenate([np.asarray(x, np.int64) for x in lists]) if lists else np.zeros(0, np.int64)
    return torch.from_numpy(ids.astype(np.int64)).to(device), torch.from_numpy(offsets).to(device)


def serve(table, layer, prompts, steps, *, format="nv", mask=None, repetition=1.2, frequency=0.1, bias=None):
    """Greedy continuations of ``prompts`` (lists of token ids, none empty): a list of ``steps`` ids each.

    table [V, D] bf16, layer [D, D] bf16; mask int32 [B, ceil(V / 32)]; bias (ids, offsets, values).
    """
    device, B = table.device, len(prompts)
    # tensor scales that spread the largest magnitude over the block scales: the table's, and 1 for
    # hidden states, which tanh bounds (so that no step waits for its own); a table of zeros takes any
    scale = float(table.abs().max()) / (6 * 448) or 1.0 if format == "nv" else 1.0
    x_scale = 1 / (6 * 448) if format == "nv" else 1.0
    packed = vocab.micro_quantize(table, format, scale)
    prompt = csr(prompts, device)
    rep = torch.full((B,), repetition, device=device)
    freq = torch.full((B,), frequency, device=device)
    last = torch.tensor([p[-1] for p in prompts], device=device)
    said = torch.empty((B, 0), dtype=torch.int64, device=device)
    status = torch.zeros(1, dtype=torch.int32, device=device)
    for step in range(steps):
        hidden = torch.tanh(vocab.micro_lookup(packed, last, dtype=table.dtype, status=status) @ layer)
        logits = vocab.micro_matmul(vocab.micro_quantize(hidden, format, x_scale), packed, dtype=torch.float32,
                                    status=status)
        output = (said.reshape(-1), torch.arange(0, B * step + 1, step, device=device)) if step else None
        vocab.process_logits(logits, prompt=prompt, output=output, repetition=rep, frequency=freq, bias=bias, mask=mask,
                             out=logits, status=status)
        last = logits.argmax(-1)
        said = torch.cat([said, last[:, None]], 1)
    if status.item():
        raise RuntimeError(f"device error bits {status.item()}")
    return said.tolist()


def distill(table, layer, tokens, teacher_ids, teacher_logits, *, lr=1.0, steps=1, temperature=2.0):
    """``steps`` steps of distillation on one batch of ``tokens`` [N]; returns the mean loss of each.

    table [V, D] fp32, updated in place; teacher_ids, teacher_logits [N, K].
    """
    V, D = table.shape
    N = tokens.numel()
    plan = E.emb_bwd_plan(table.device.index, 1, [0, V], [0, D], [0], None, E.EMB_F32, E.EMB_F32, N, 1)
    offsets = torch.tensor([0, N], device=table.device)
    weight = torch.full((N,), 1.0 / N, device=table.device)
    losses = []
    try:
        for _ in range(steps):
            rows = table[tokens]
            hidden = torch.tanh(rows @ layer)
            logits = hidden @ table.t()
            loss, grad = vocab.distill_step(logits, teacher_ids, teacher_logits, weight, temperature=temperature,
                                            out=logits)
            losses.append(loss.mean())
            grad_rows = ((grad @ table) * (1 - hidden * hidden)) @ layer.t()
            table.addmm_(grad.t(), hidden, alpha=-lr)
            E.emb_nobag_bwd_sgd(plan, table, tokens, offsets, N, 1, grad_rows.contiguous(), lr, E.EMB_NOBAG_SORTED)
        st = E.emb_plan_status(plan)
        if st != E.EMB_OK:
            raise E.EmbError(st, "emb_nobag_bwd_sgd")
    finally:
        E.emb_plan_destroy(plan)
    return [x.item() for x in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--vocab", type=int, default=32001)
    ap.add_argument("--dim", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randn((a.vocab, a.dim), generator=g, device="cuda") * 0.05
    layer = torch.randn((a.dim, a.dim), generator=g, device="cuda") * a.dim ** -0.5
    prompts = [list(range(1 + i, 6 + 3 * i)) for i in range(4)]
    for p, out in zip(prompts, serve(table.bfloat16(), layer.bfloat16(), prompts, a.steps)):
        print(f"prompt of {len(p)} tokens: {out}")
    tokens = torch.randint(0, a.vocab, (a.tokens,), generator=g, device="cuda")
    teacher = torch.randn((a.tokens, 16), generator=g, device="cuda").sort(-1, descending=True).values * 3
    ids = torch.stack([torch.randperm(a.vocab, generator=g, device="cuda")[:16] for _ in range(a.tokens)])
    losses = distill(table, layer, tokens, ids, teacher, lr=20.0, steps=a.steps)
    print("distillation loss:", " ".join(f"{x:.3f}" for x in losses))


if __name__ == "__main__":
    main()
