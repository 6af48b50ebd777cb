"""Vocabulary operators of a language model on PyTorch tensors.

``process_logits``    penalties for repeated tokens, biases and grammar masks
``distill_forward``, ``distill_backward``, ``distill_step``, ``distill_loss``
                      distillation from a teacher's top logits (``distill_loss`` is
                      differentiable by autograd)
``micro_quantize``, ``micro_lookup``, ``micro_matmul``
                      a matrix in microscaled 4-bit floating point: laid out, read by row, and
                      multiplied

Marshalling only, as in ``device``: arguments are checked, outputs allocated, and the library's
kernels called on the current stream of the tensors' device. Formulas and layouts are in the C header.
``status`` is an int32 tensor of one element that collects device error bits (1: an id out of
range, 2: malformed offsets, 4: a bounded wait ran out); the caller clears it.
"""
from __future__ import annotations

import dataclasses

import torch

from . import embbwd as E

_DTYPE = {torch.float32: E.EMB_F32, torch.float16: E.EMB_F16, torch.bfloat16: E.EMB_BF16}
_FORMAT = {"mx": E.EMB_MICRO_MX, "nv": E.EMB_MICRO_NV}
_BLOCK = {"mx": 32, "nv": 16}


def _matrix(x, name):
    """(dtype code, row stride) of a 2-D CUDA tensor whose rows are contiguous."""
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    code = _DTYPE.get(x.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {x.dtype}")
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return code, x.stride(0)


def _vector(x, like, dtype, n, name):
    if x is not None and (x.dtype != dtype or x.device != like.device or x.dim() != 1
                          or x.numel() != n or not x.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {like.device}")
    return x


def _status(status, like):
    if status is not None and (status.dtype not in (torch.int32, torch.uint32) or status.numel() != 1
                               or status.device != like.device):
        raise ValueError(f"status must be an int32 tensor of one element on {like.device}")
    return status


def _stream(x):
    return torch.cuda.current_stream(x.device).cuda_stream


def _csr(lists, like, B, name):
    """(ids, offsets, number of ids) of a CSR list, or nothing."""
    if lists is None:
        return None, None, 0
    ids, offsets = lists[0], lists[1]
    _vector(ids, like, torch.int64, ids.numel(), f"{name} ids")
    _vector(offsets, like, torch.int64, B + 1, f"{name} offsets")
    return ids, offsets, ids.numel()


def _out_like(out, like, rows, cols, dtype, name="out"):
    if out.shape != (rows, cols) or out.device != like.device or (dtype and out.dtype != dtype):
        raise ValueError(f"{name} must be a [{rows}, {cols}] tensor{f' of {dtype}' if dtype else ''} on {like.device}")
    return out


def process_logits(logits, *, prompt=None, output=None, repetition=None, frequency=None, presence=None, bias=None,
                   mask=None, out=None, dtype=None, status=None):
    """Penalised, biased and masked logits [B, V], as ``dtype`` (``logits``' own if not given) or into ``out``.

    prompt, output   (ids, offsets): int64 CSR lists of each request's token ids
    repetition, frequency, presence   fp32 [B]
    bias             (ids, offsets, values): CSR lists with fp32 values
    mask             int32 [B, ceil(V / 32)]: bit v % 32 of word v // 32 allows token v
    ``out`` may be ``logits``.
    """
    zc, zs = _matrix(logits, "logits")
    B, V = logits.shape
    p, po, pn = _csr(prompt, logits, B, "prompt")
    o, oo, on = _csr(output, logits, B, "output")
    b, bo, bn = _csr(bias, logits, B, "bias")
    values = None if bias is None else _vector(bias[2], logits, torch.float32, bn, "bias values")
    _vector(repetition, logits, torch.float32, B, "repetition")
    _vector(frequency, logits, torch.float32, B, "frequency")
    _vector(presence, logits, torch.float32, B, "presence")
    ms = 0
    if mask is not None:
        if (mask.dim() != 2 or mask.dtype not in (torch.int32, torch.uint32) or mask.device != logits.device
                or mask.shape[0] != B or mask.shape[1] < (V + 31) // 32 or mask.stride(1) != 1):
            raise ValueError(f"mask must be an int32 [{B}, {(V + 31) // 32}] tensor on {logits.device}")
        ms = mask.stride(0)
    if out is None:
        out = torch.empty((B, V), dtype=dtype or logits.dtype, device=logits.device)
    else:
        _out_like(out, logits, B, V, dtype)
    yc, ys = _matrix(out, "out")
    E.emb_logits_process(logits.device.index, logits, zc, zs, B, V, p, po, pn, o, oo, on, repetition, frequency,
                         presence, b, bo, values, bn, mask, ms, out, yc, ys, _status(status, logits), _stream(logits))
    return out


def _teacher(logits, ids, teacher):
    N, V = logits.shape
    tc, ts = _matrix(teacher, "teacher_logits")
    if ids.dtype != torch.int64 or ids.shape != teacher.shape or ids.shape[0] != N or ids.device != logits.device:
        raise ValueError(f"teacher_ids must be an int64 tensor shaped as teacher_logits, of {N} rows")
    if ids.shape[1] > 1 and ids.stride(1) != 1 or N > 1 and ids.stride(0) != ts:
        raise ValueError("teacher_ids and teacher_logits must have contiguous rows and the same row stride")
    return tc, ts


def _like_rows(x):
    """A new tensor shaped as x, its rows as far apart as x's."""
    N, V = x.shape
    stride = max(x.stride(0), V)
    return torch.empty_strided((N, V), (stride, 1), dtype=x.dtype, device=x.device)


def distill_forward(logits, teacher_ids, teacher_logits, *, temperature=1.0, teacher_lse=None, status=None):
    """(loss fp32 [N], stats fp32 [N, 4]) of student ``logits`` [N, V] against a teacher's lists [N, K].

    teacher_ids int64 (-1: no entry); teacher_lse fp32 [N]: log of the teacher's whole sum of
    exp(logit / temperature), to count its mass off the list; without it the list is renormalised.
    """
    zc, zs = _matrix(logits, "logits")
    N, V = logits.shape
    tc, ts = _teacher(logits, teacher_ids, teacher_logits)
    _vector(teacher_lse, logits, torch.float32, N, "teacher_lse")
    loss = torch.empty(N, dtype=torch.float32, device=logits.device)
    stats = torch.empty((N, 4), dtype=torch.float32, device=logits.device)
    E.emb_distill_forward(logits.device.index, logits, zc, zs, N, V, teacher_ids, teacher_logits, tc, ts,
                          teacher_ids.shape[1], teacher_lse, temperature, loss, stats, _status(status, logits), _stream(logits))
    return loss, stats


def distill_backward(logits, teacher_ids, teacher_logits, stats, row_weight=None, *, temperature=1.0, out=None,
                     status=None):
    """row_weight[n] * dloss[n] / dlogits from the forward's ``stats``; ``out`` may be ``logits``."""
    zc, zs = _matrix(logits, "logits")
    N, V = logits.shape
    tc, ts = _teacher(logits, teacher_ids, teacher_logits)
    if stats.dtype != torch.float32 or stats.shape != (N, 4) or not stats.is_contiguous():
        raise ValueError(f"stats must be a contiguous float32 [{N}, 4] tensor")
    _vector(row_weight, logits, torch.float32, N, "row_weight")
    out = _like_rows(logits) if out is None else _out_like(out, logits, N, V, logits.dtype)
    E.emb_distill_backward(logits.device.index, logits, zc, zs, N, V, teacher_ids, teacher_logits, tc, ts,
                           teacher_ids.shape[1], stats, row_weight, temperature, out, _matrix(out, "out")[1],
                           _status(status, logits), _stream(logits))
    return out


def distill_step(logits, teacher_ids, teacher_logits, row_weight=None, *, temperature=1.0, teacher_lse=None, out=None,
                 status=None):
    """(loss [N], row_weight[n] * dloss[n] / dlogits) in one call; ``out`` may be ``logits``."""
    zc, zs = _matrix(logits, "logits")
    N, V = logits.shape
    tc, ts = _teacher(logits, teacher_ids, teacher_logits)
    _vector(teacher_lse, logits, torch.float32, N, "teacher_lse")
    _vector(row_weight, logits, torch.float32, N, "row_weight")
    loss = torch.empty(N, dtype=torch.float32, device=logits.device)
    out = _like_rows(logits) if out is None else _out_like(out, logits, N, V, logits.dtype)
    E.emb_distill_step(logits.device.index, logits, zc, zs, N, V, teacher_ids, teacher_logits, tc, ts,
                       teacher_ids.shape[1], teacher_lse, row_weight, temperature, loss, out,
                       _matrix(out, "out")[1], _status(status, logits), _stream(logits))
    return loss, out


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
        return (distill_backward(logits, ids, teacher, stats, grad.float().contiguous(),
                                 temperature=ctx.temperature), None, None, None, None)


def distill_loss(logits, teacher_ids, teacher_logits, *, temperature=1.0, teacher_lse=None):
    """Differentiable loss [N] of ``logits`` (the teacher takes no gradient)."""
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

    def _check(self, name):
        if self.format not in _FORMAT:
            raise ValueError(f"the format of {name} must be 'mx' or 'nv', got {self.format!r}")
        if self.codes.numel() != self.rows * _row_bytes(self.cols) or \
                self.scales.numel() != _scale_bytes(self.rows, self.cols, self.format):
            raise ValueError(f"the codes or scales of {name} do not fit its shape")
        if self.codes.dtype != torch.uint8 or self.scales.dtype != torch.uint8 or not self.codes.is_cuda or \
                not self.codes.is_contiguous() or not self.scales.is_contiguous() or \
                self.codes.device != self.scales.device:
            raise ValueError(f"codes and scales of {name} must be contiguous uint8 CUDA tensors")
        return _FORMAT[self.format]


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
    xc, xs = _matrix(x, "x")
    R, K = x.shape
    if format not in _FORMAT:
        raise ValueError(f"format must be 'mx' or 'nv', got {format!r}")
    if out is None:
        codes = torch.empty((R, _row_bytes(K)), dtype=torch.uint8, device=x.device)
        scales = torch.empty(((R + 127) // 128, _tiles(K, format), 32, 4, 4), dtype=torch.uint8, device=x.device)
        out = MicroMatrix(codes, scales, R, K, format, tensor_scale)
    else:
        out._check("out")
        if (out.rows, out.cols, out.format, out.codes.device) != (R, K, format, x.device):
            raise ValueError("out has another shape, format or device")
        out.tensor_scale = tensor_scale
    E.emb_micro_quantize(x.device.index, x, xc, xs, R, K, _FORMAT[format], tensor_scale, out.codes, out.scales,
                         _stream(x))
    return out


def micro_lookup(table, ids=None, *, dtype=torch.float32, out=None, status=None):
    """Rows ``ids`` (int64; all rows if not given) of ``table`` as values [n, cols]."""
    fmt = table._check("table")
    if ids is not None:
        _vector(ids, table.codes, torch.int64, ids.numel(), "ids")
    n = table.rows if ids is None else ids.numel()
    if out is None:
        out = torch.empty((n, table.cols), dtype=dtype, device=table.codes.device)
    else:
        _out_like(out, table.codes, n, table.cols, None)
    oc, os_ = _matrix(out, "out")
    E.emb_micro_lookup(out.device.index, table.codes, table.scales, table.rows, table.cols, fmt, table.tensor_scale,
                       ids, n, out, oc, os_, _status(status, out), _stream(out))
    return out


def micro_matmul(x, w, *, dtype=torch.bfloat16, out=None, status=None):
    """x [M, K] times the transpose of w [N, K], both MicroMatrix of one format: [M, N] as ``dtype``."""
    fmt = x._check("x")
    if w._check("w") != fmt or w.cols != x.cols or w.codes.device != x.codes.device:
        raise ValueError("x and w must have the same format, columns and device")
    if out is None:
        out = torch.empty((x.rows, w.rows), dtype=dtype, device=x.codes.device)
    else:
        _out_like(out, x.codes, x.rows, w.rows, None)
    oc, os_ = _matrix(out, "out")
    E.emb_micro_matmul(out.device.index, x.codes, x.scales, x.tensor_scale, x.rows, w.codes, w.scales,
                       w.tensor_scale, w.rows, x.cols, fmt, out, oc, os_, _status(status, out), _stream(out))
    return out
