"""Vocabulary operators of a language model on PyTorch tensors.

``process_logits``    penalties for repeated tokens, biases and grammar masks
``distill_forward``, ``distill_backward``, ``distill_step``, ``distill_loss``
                      distillation from a teacher's top logits (``distill_loss`` is
                      differentiable by autograd)
``micro_quantize``, ``micro_lookup``, ``micro_matmul``
                      a matrix in microscaled 4-bit floating point: laid out, read by row, and
                      multiplied

Marshalling only, as in ``device``: arguments are checked, outputs allocated, and the library's
kernels called on the current stream of the tensors' device, by the compiled entry ``_vocab``
(one call's host work counts beside a kernel of a few microseconds). Formulas and layouts are in
the C header. Malformed arguments raise ValueError, a status of the library EmbError. ``status`` is
an int32 tensor of one element that collects device error bits (1: an id out of range, 2:
malformed offsets, 4: a bounded wait of a product ran out, and what was not finished is NaN); the
caller clears it.

Of these only ``distill_loss`` takes part in autograd: the other calls take tensors that require
gradients as values, and what they return has no history. An ``out`` counts as changed in place.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import embbwd as E

_FORMAT = {"mx": E.EMB_MICRO_MX, "nv": E.EMB_MICRO_NV}
_BLOCK = {"mx": 32, "nv": 16}
_entry = None


def _native():
    """The compiled entry, given the library's functions (raises if either has not been built)."""
    global _entry
    if _entry is None:
        lib = E.load()
        from . import _vocab
        _vocab.bind(E.EmbError, *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "emb_logits_process", "emb_distill_forward", "emb_distill_backward", "emb_distill_step",
            "emb_micro_quantize", "emb_micro_lookup", "emb_micro_matmul")))
        _entry = _vocab
    return _entry


def _format(name):
    code = _FORMAT.get(name)
    if code is None:
        raise ValueError(f"format must be 'mx' or 'nv', got {name!r}")
    return code


def process_logits(logits, *, prompt=None, output=None, repetition=None, frequency=None, presence=None, bias=None,
                   mask=None, out=None, dtype=None, status=None):
    """Penalised, biased and masked logits [B, V], as ``dtype`` (``logits``' own if not given) or into ``out``.

    prompt, output   (ids, offsets): int64 CSR lists of each request's token ids
    repetition, frequency, presence   fp32 [B]
    bias             (ids, offsets, values): CSR lists with fp32 values
    mask             int32 [B, ceil(V / 32)]: bit v % 32 of word v // 32 allows token v
    ``out`` may be ``logits``.
    """
    return (_entry or _native()).process_logits(logits, prompt, output, repetition, frequency, presence, bias, mask, out,
                                                dtype, status)


def distill_forward(logits, teacher_ids, teacher_logits, *, temperature=1.0, teacher_lse=None, status=None):
    """(loss fp32 [N], stats fp32 [N, 4]) of student ``logits`` [N, V] against a teacher's lists [N, K].

    teacher_ids int64 (-1: no entry); teacher_lse fp32 [N]: log of the teacher's whole sum of
    exp(logit / temperature), to count its mass off the list; without it the list is renormalised.
    """
    return (_entry or _native()).distill_forward(logits, teacher_ids, teacher_logits, temperature, teacher_lse, status)


def distill_backward(logits, teacher_ids, teacher_logits, stats, row_weight=None, *, temperature=1.0, out=None,
                     status=None):
    """row_weight[n] * dloss[n] / dlogits from the forward's ``stats``; ``out`` may be ``logits``."""
    return (_entry or _native()).distill_backward(logits, teacher_ids, teacher_logits, stats, row_weight, temperature,
                                                  out, status)


def distill_step(logits, teacher_ids, teacher_logits, row_weight=None, *, temperature=1.0, teacher_lse=None, out=None,
                 status=None):
    """(loss [N], row_weight[n] * dloss[n] / dlogits) in one call; ``out`` may be ``logits``."""
    return (_entry or _native()).distill_step(logits, teacher_ids, teacher_logits, row_weight, temperature, teacher_lse,
                                              out, status)


class _DistillGradient(torch.autograd.Function):
    """The loss's gradient; its own derivatives are not built, and asking for them is an error."""

    @staticmethod
    def forward(ctx, logits, grad, teacher_ids, teacher_logits, stats, temperature):
        return distill_backward(logits, teacher_ids, teacher_logits, stats, grad, temperature=temperature)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError("distill_loss can be differentiated only once")


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_ids, teacher_logits, temperature, teacher_lse):
        loss, stats = distill_forward(logits, teacher_ids, teacher_logits, temperature=temperature,
                                      teacher_lse=teacher_lse)
        ctx.save_for_backward(logits, teacher_ids, teacher_logits, stats)
        ctx.temperature = temperature
        return loss

    @staticmethod
    def backward(ctx, grad):
        logits, ids, teacher, stats = ctx.saved_tensors
        return (_DistillGradient.apply(logits, grad.float().contiguous(), ids, teacher, stats, ctx.temperature), None,
                None, None, None)


def distill_loss(logits, teacher_ids, teacher_logits, *, temperature=1.0, teacher_lse=None):
    """Differentiable loss [N] of ``logits`` (once; the teacher takes no gradient)."""
    return _DistillLoss.apply(logits, teacher_ids, teacher_logits, temperature, teacher_lse)


@dataclasses.dataclass
class MicroMatrix:
    """A [rows, cols] matrix in microscaled 4-bit floating point (layout in the C header)."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int
    format: str  # "mx" or "nv"
    tensor_scale: float = 1.0

    def _parts(self):
        return self.codes, self.scales, self.rows, self.cols, _format(self.format), self.tensor_scale


def _row_bytes(cols):
    return (cols + 31) // 32 * 16


def _tiles(cols, format):
    return ((cols + 31) // 32 * (32 // _BLOCK[format]) + 3) // 4


def _scale_bytes(rows, cols, format):
    return (rows + 127) // 128 * _tiles(cols, format) * 512


def micro_quantize(x, format="mx", tensor_scale=1.0, *, out=None):
    """``x`` [rows, cols] as a MicroMatrix (``out``: an existing one of that shape, overwritten).

    For "nv", tensor_scale spreads the tensor's range over the block scales: amax / (6 * 448) of
    calibrated data.
    """
    entry = _entry or _native()
    if out is None:
        codes, scales = entry.micro_quantize(x, _format(format), tensor_scale, None, None)
        return MicroMatrix(codes, scales, x.shape[0], x.shape[1], format, tensor_scale)
    if (out.rows, out.cols, out.format) != (*x.shape, format):
        raise ValueError("out has another shape or format")
    entry.micro_quantize(x, _format(format), tensor_scale, out.codes, out.scales)
    out.tensor_scale = tensor_scale
    return out


def micro_lookup(table, ids=None, *, dtype=torch.float32, out=None, status=None):
    """Rows ``ids`` (int64; all rows if not given) of ``table`` as values [n, cols]."""
    return (_entry or _native()).micro_lookup(*table._parts(), ids, dtype, out, status)


def micro_matmul(x, w, *, dtype=torch.bfloat16, out=None, status=None):
    """x [M, K] times the transpose of w [N, K], both MicroMatrix of one format: [M, N] as ``dtype``."""
    return (_entry or _native()).micro_matmul(*x._parts(), *w._parts(), dtype, out, status)
