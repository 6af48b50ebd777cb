"""Vocabulary operators of a language model on PyTorch tensors.

``process_logits``    penalties for repeated tokens, biases and grammar masks
``distill_forward``, ``distill_backward``, ``distill_step``, ``distill_loss``
                      distillation from a teacher's top logits (``distill_loss`` is
                      differentiable by autograd)
``micro_quantize``, ``micro_lookup``, ``micro_matmul``
                      a matrix in microscaled 4-bit or 8-bit floating point: laid out, read by
                      row, and multiplied
``rms_norm_forward``, ``rms_norm_backward``, ``rms_norm``
                      root-mean-square norm with the residual's addition, to the rows' type or to
                      a microscaled 8-bit matrix (``rms_norm`` is differentiable)
``dropout``           dropout from a counter-based generator, with the residual's addition
                      (differentiable)
``cross_entropy_forward``, ``cross_entropy_backward``, ``cross_entropy_step``, ``cross_entropy_loss``
                      softmax cross entropy of hidden states against the token table, without the
                      logits in memory (``cross_entropy_loss`` is differentiable)

Marshalling only, as in ``device``: arguments are checked, outputs allocated, and the library's
kernels called on the current stream of the tensors' device, by the compiled entry ``_vocab``
(one call's host work counts beside a kernel of a few microseconds). Formulas and layouts are in
the C header. Malformed arguments raise ValueError, a status of the library EmbError. ``status`` is
an int32 tensor of one element that collects device error bits (1: an id out of range, 2:
malformed offsets, 4: a bounded wait of a product ran out, and what was not finished is NaN); the
caller clears it.

Of these ``distill_loss``, ``rms_norm``, ``dropout`` and ``cross_entropy_loss`` take part in autograd, all but
``dropout`` once (second derivatives are refused) and in backward mode alone (tangents are refused). The other
calls take tensors that require gradients, or carry tangents, as values, and what they return has no history. An
``out`` counts as changed in place, and shares no memory with another tensor of the call but where that says so.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch
from torch.autograd import forward_ad

from . import embbwd as E

_FORMAT = {"mx": E.EMB_MICRO_MX, "nv": E.EMB_MICRO_NV, "mx8": E.EMB_MICRO_MX8}
_BLOCK = {"mx": 32, "nv": 16, "mx8": 32}
_entry = None


def _native():
    """The compiled entry, given the library's functions (raises if either has not been built)."""
    global _entry
    if _entry is None:
        lib = E.load()
        from . import _vocab
        _vocab.bind(E.EmbError, *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "emb_logits_process", "emb_distill_forward", "emb_distill_backward", "emb_distill_step",
            "emb_micro_quantize", "emb_micro_lookup", "emb_micro_matmul", "emb_rms_norm_forward", "emb_rms_norm_workspace",
            "emb_rms_norm_backward", "emb_dropout", "emb_cross_entropy_workspace", "emb_cross_entropy_forward",
            "emb_cross_entropy_backward", "emb_cross_entropy_step")))
        _entry = _vocab
    return _entry


def _format(name):
    code = _FORMAT.get(name)
    if code is None:
        raise ValueError(f"format must be 'mx', 'nv' or 'mx8', got {name!r}")
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
    def forward(ctx, logits, grad, teacher_ids, teacher_logits, stats, temperature, status):
        return distill_backward(logits, teacher_ids, teacher_logits, stats, grad, temperature=temperature, status=status)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError("distill_loss can be differentiated only once")


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_ids, teacher_logits, temperature, teacher_lse, status):
        loss, stats = distill_forward(logits, teacher_ids, teacher_logits, temperature=temperature,
                                      teacher_lse=teacher_lse, status=status)
        ctx.save_for_backward(logits, teacher_ids, teacher_logits, stats)
        ctx.temperature, ctx.status = temperature, status
        return loss

    @staticmethod
    def backward(ctx, grad):
        logits, ids, teacher, stats = ctx.saved_tensors
        return (_DistillGradient.apply(logits, grad.float().contiguous(), ids, teacher, stats, ctx.temperature,
                                       ctx.status), None, None, None, None, None)


def distill_loss(logits, teacher_ids, teacher_logits, *, temperature=1.0, teacher_lse=None, status=None):
    """Differentiable loss [N] of ``logits`` (once; the teacher takes no gradient). ``status`` collects the error
    bits of the forward and of the backward."""
    return _DistillLoss.apply(logits, teacher_ids, teacher_logits, temperature, teacher_lse, status)


@dataclasses.dataclass
class MicroMatrix:
    """A [rows, cols] matrix in microscaled floating point (layout in the C header)."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int
    format: str  # "mx" or "nv" (4 bits), "mx8" (8 bits)
    tensor_scale: float = 1.0

    def _parts(self):
        return self.codes, self.scales, self.rows, self.cols, _format(self.format), self.tensor_scale


def _row_bytes(cols, format="mx"):
    return (cols + 31) // 32 * (32 if format == "mx8" else 16)


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


def rms_norm_forward(x, weight=None, *, residual=None, eps=1e-6, format=None, out=None, sum_out=None):
    """(y, sum, rstd fp32 [N]) of rows x [N, D]: y = sum * rstd * weight, sum = x + residual.

    weight [D] of any of the three types; residual [N, D] of x's type (without it ``sum`` is x itself, or
    ``sum_out`` with its values; None where ``out`` is x and no ``sum_out`` keeps them). With format "mx8" y is a
    MicroMatrix and rstd None. ``out`` and ``sum_out`` may be x or residual.
    """
    if format not in (None, "mx8"):
        raise ValueError(f"format must be None or 'mx8', got {format!r}")
    y, total, rstd = (_entry or _native()).rms_norm_forward(x, weight, residual, eps, format is not None, out, sum_out)
    if format is not None:
        y = MicroMatrix(*y, x.shape[0], x.shape[1], format)
    return y, total, rstd


def rms_norm_backward(grad, sum, weight, rstd, *, grad_sum=None, want_weight=True, out=None):
    """(gradient of x and residual, gradient of weight or None) from the gradient of y and the forward's
    ``sum`` and ``rstd``; grad_sum: the gradient that arrives at the sum by other ways."""
    return (_entry or _native()).rms_norm_backward(grad, sum, weight, rstd, grad_sum, want_weight, out)


def _rows(t):
    """A gradient as the library takes it: rows contiguous, none of them the same memory."""
    return t if t.stride(-1) == 1 and (t.shape[0] < 2 or t.stride(0) >= t.shape[1]) else t.contiguous()


class _RmsNormGradient(torch.autograd.Function):
    """The norm's gradient; its own derivatives are not built, and asking for them is an error."""

    @staticmethod
    def forward(ctx, grad, total, weight, rstd, grad_sum, want_weight):
        return rms_norm_backward(grad, total, weight, rstd, grad_sum=grad_sum, want_weight=want_weight)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("rms_norm can be differentiated only once")


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        y, total, rstd = rms_norm_forward(x, weight, residual=residual, eps=eps)
        ctx.save_for_backward(total, weight, rstd)
        ctx.summed = residual is not None
        return (y, total) if ctx.summed else y

    @staticmethod
    def backward(ctx, grad, grad_sum=None):
        total, weight, rstd = ctx.saved_tensors
        if grad is None:  # only the sum was used
            return grad_sum, None, grad_sum, None
        dx, dw = _RmsNormGradient.apply(_rows(grad), total, weight, rstd, None if grad_sum is None else _rows(grad_sum),
                                        ctx.needs_input_grad[1])
        return dx, dw, dx if ctx.summed else None, None


def rms_norm(x, weight=None, *, residual=None, eps=1e-6):
    """Differentiable norm of rows x [N, D]: y, or (y, x + residual) with a residual."""
    return _RmsNorm.apply(x, weight, residual, eps)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, call, residual):
        ctx.p, ctx.seed = p, seed
        if isinstance(call, torch.Tensor):
            ctx.save_for_backward(call)  # advanced before the backward: an error
            ctx.save_for_forward(call)
            ctx.call = None
        else:
            ctx.call = call
        ctx.summed = residual is not None
        return _native().dropout(x, p, seed, call, residual, None)

    @staticmethod
    def backward(ctx, grad):
        call = ctx.saved_tensors[0] if ctx.call is None else ctx.call
        dx = dropout(_rows(grad), ctx.p, ctx.seed, call) if ctx.needs_input_grad[0] else None
        return dx, None, None, None, grad if ctx.summed else None

    @staticmethod
    def jvp(ctx, dx, _p, _seed, _call, dres):
        call = ctx.saved_tensors[0] if ctx.call is None else ctx.call
        if dx is None:
            return dres.clone()
        return dropout(_rows(dx), ctx.p, ctx.seed, call, residual=None if dres is None else _rows(dres))


def dropout(x, p, seed, call=0, *, residual=None, out=None):
    """x [N, D] with each element kept and divided by 1 - p, or zero with probability p, plus residual.

    The elements kept depend on ``seed`` (0 to 2^64 - 1) and ``call``: an int, or an int64 CUDA tensor of one
    element that is read when the call runs, for captured graphs. Equal pairs keep equal elements, so a
    program counts its calls. Differentiable, in forward mode too, unless ``out`` is given (which may be x or
    residual).
    """
    # tensors carry tangents while a dual level is open, which `requires_grad` does not tell
    if out is None and (forward_ad._current_level >= 0 or torch.is_grad_enabled() and (
            getattr(x, "requires_grad", False) or getattr(residual, "requires_grad", False))):
        return _Dropout.apply(x, p, seed, call, residual)
    return (_entry or _native()).dropout(x, p, seed, call, residual, out)


def cross_entropy_forward(hidden, table, targets, *, status=None):
    """(loss fp32 [N], lse fp32 [N]) of the logits hidden [N, D] times the transpose of table [V, D].

    hidden and table both float16 or both bfloat16; targets int64 [N], negative: the row takes no part.
    """
    return (_entry or _native()).cross_entropy_forward(hidden, table, targets, status)


def cross_entropy_backward(hidden, table, targets, lse, row_weight=None, *, want_hidden=True, want_table=True,
                           out_hidden=None, out_table=None, status=None):
    """Gradients of sum(row_weight * loss) for (hidden, table) from the forward's ``lse``; None for one not wanted."""
    return (_entry or _native()).cross_entropy_backward(hidden, table, targets, lse, row_weight, want_hidden, want_table,
                                                        out_hidden, out_table, status)


def cross_entropy_step(hidden, table, targets, row_weight=None, *, out_hidden=None, out_table=None, status=None):
    """(loss [N], gradient of hidden, gradient of table) of sum(row_weight * loss) in one call."""
    return (_entry or _native()).cross_entropy_step(hidden, table, targets, row_weight, out_hidden, out_table, status)


class _EntropyGradient(torch.autograd.Function):
    """The loss's gradients; their own derivatives are not built, and asking for them is an error."""

    @staticmethod
    def forward(ctx, hidden, table, grad, targets, lse, want_hidden, want_table, status):
        return cross_entropy_backward(hidden, table, targets, lse, grad, want_hidden=want_hidden, want_table=want_table,
                                      status=status)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("cross_entropy_loss can be differentiated only once")


class _EntropyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, table, targets, status):
        loss, lse = cross_entropy_forward(hidden, table, targets, status=status)
        ctx.save_for_backward(hidden, table, targets, lse)
        ctx.status = status  # collects bits, and may be cleared at any time: not a saved value
        return loss

    @staticmethod
    def backward(ctx, grad):
        hidden, table, targets, lse = ctx.saved_tensors
        want = ctx.needs_input_grad
        return (*_EntropyGradient.apply(hidden, table, grad.float().contiguous(), targets, lse, want[0], want[1],
                                        ctx.status), None, None)


def cross_entropy_loss(hidden, table, targets, *, status=None):
    """Differentiable loss [N] of hidden states against the table (once). ``status`` collects the error bits of the
    forward and of the backward: a target beyond the table takes no part, and is only reported there."""
    return _EntropyLoss.apply(hidden, table, targets, status)
