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

One call's host work counts beside a kernel of a few microseconds: the checks below look at each
tensor once, and the library is called with pointers, past the binding's per-argument helpers.
"""
from __future__ import annotations

import dataclasses

import torch

from . import embbwd as E

_DTYPE = {torch.float32: E.EMB_F32, torch.float16: E.EMB_F16, torch.bfloat16: E.EMB_BF16}
_FORMAT = {"mx": E.EMB_MICRO_MX, "nv": E.EMB_MICRO_NV}
_BLOCK = {"mx": 32, "nv": 16}
_F32, _I64 = torch.float32, torch.int64
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda index: torch.cuda.current_stream(index).cuda_stream


def _matrix(x, name):
    """(device index, dtype code, row stride) of a 2-D CUDA tensor whose rows are contiguous."""
    dev, code = x.get_device(), _DTYPE.get(x.dtype)
    if dev < 0 or x.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {x.dtype}")
    row, col = x.stride()
    if col != 1 and x.shape[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return dev, code, row


def _vector(x, dev, dtype, n, name):
    """The pointer of a contiguous tensor of n elements, or None."""
    if x is None:
        return None
    if x.dtype is not dtype or x.get_device() != dev or x.numel() != n or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on cuda:{dev}")
    return x.data_ptr()


def _status(status, dev):
    if status is None:
        return None
    if status.dtype not in (torch.int32, torch.uint32):
        raise ValueError(f"status must be an int32 tensor of one element on cuda:{dev}")
    return _vector(status, dev, status.dtype, 1, "status")


def _csr(lists, dev, B, name):
    """(ids, offsets, number of ids) of a CSR list, or nothing."""
    if lists is None:
        return None, None, 0
    n = lists[0].numel()
    return _vector(lists[0], dev, _I64, n, f"{name} ids"), _vector(lists[1], dev, _I64, B + 1, f"{name} offsets"), n


def _out_like(out, dev, rows, cols, dtype, name="out"):
    """(dtype code, row stride) of a given output."""
    at, code, stride = _matrix(out, name)
    if out.shape != (rows, cols) or at != dev or (dtype and out.dtype != dtype):
        raise ValueError(f"{name} must be a [{rows}, {cols}] tensor{f' of {dtype}' if dtype else ''} on cuda:{dev}")
    return code, stride


_functions = {}  # of the library, by name


def _call(name, *args):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(E.load(), name)
    st = f(*args)
    if st:
        raise E.EmbError(st, name)


def process_logits(logits, *, prompt=None, output=None, repetition=None, frequency=None, presence=None, bias=None,
                   mask=None, out=None, dtype=None, status=None):
    """Penalised, biased and masked logits [B, V], as ``dtype`` (``logits``' own if not given) or into ``out``.

    prompt, output   (ids, offsets): int64 CSR lists of each request's token ids
    repetition, frequency, presence   fp32 [B]
    bias             (ids, offsets, values): CSR lists with fp32 values
    mask             int32 [B, ceil(V / 32)]: bit v % 32 of word v // 32 allows token v
    ``out`` may be ``logits``.
    """
    dev, zc, zs = _matrix(logits, "logits")
    B, V = logits.shape
    p, po, pn = _csr(prompt, dev, B, "prompt")
    o, oo, on = _csr(output, dev, B, "output")
    b, bo, bn = _csr(bias, dev, B, "bias")
    bv = None if bias is None else _vector(bias[2], dev, _F32, bn, "bias values")
    mp, ms = None, 0
    if mask is not None:
        if (mask.dim() != 2 or mask.dtype not in (torch.int32, torch.uint32) or mask.get_device() != dev
                or mask.shape[0] != B or mask.shape[1] < (V + 31) // 32 or (mask.shape[1] > 1 and mask.stride(1) != 1)):
            raise ValueError(f"mask must be an int32 [{B}, {(V + 31) // 32}] tensor on cuda:{dev}")
        mp, ms = mask.data_ptr(), mask.stride(0)
    if out is None:
        out = torch.empty((B, V), dtype=dtype or logits.dtype, device=logits.device)
        yc, ys = _DTYPE.get(out.dtype, -1), V
    else:
        yc, ys = _out_like(out, dev, B, V, dtype)
    _call("emb_logits_process", dev, logits.data_ptr(), zc, zs, B, V, p, po, pn, o, oo, on,
          _vector(repetition, dev, _F32, B, "repetition"), _vector(frequency, dev, _F32, B, "frequency"),
          _vector(presence, dev, _F32, B, "presence"), b, bo, bv, bn, mp, ms, out.data_ptr(), yc, ys,
          _status(status, dev), _raw_stream(dev))
    return out


def _rows_and_lists(logits, ids, teacher):
    """What the distillation calls share: device, dtype and the arguments from logits to list length."""
    dev, zc, zs = _matrix(logits, "logits")
    N, V = logits.shape
    at, tc, ts = _matrix(teacher, "teacher_logits")
    if at != dev or ids.dtype is not _I64 or ids.get_device() != dev or ids.shape != teacher.shape or ids.shape[0] != N:
        raise ValueError(f"teacher_ids (int64) and teacher_logits must be [{N}, K] tensors on cuda:{dev}")
    if (ids.shape[1] > 1 and ids.stride(1) != 1) or (N > 1 and ids.stride(0) != ts):
        raise ValueError("teacher_ids and teacher_logits must have contiguous rows and the same row stride")
    return dev, N, V, (dev, logits.data_ptr(), zc, zs, N, V, ids.data_ptr(), teacher.data_ptr(), tc, ts, ids.shape[1])


def _gradient(logits, out, dev, N, V):
    """The gradient's tensor and row stride: `out`, or a new one with its rows as far apart as those of logits."""
    if out is not None:
        return out, _out_like(out, dev, N, V, logits.dtype)[1]
    stride = max(logits.stride(0), V)
    return torch.empty_strided((N, V), (stride, 1), dtype=logits.dtype, device=logits.device), stride


def distill_forward(logits, teacher_ids, teacher_logits, *, temperature=1.0, teacher_lse=None, status=None):
    """(loss fp32 [N], stats fp32 [N, 4]) of student ``logits`` [N, V] against a teacher's lists [N, K].

    teacher_ids int64 (-1: no entry); teacher_lse fp32 [N]: log of the teacher's whole sum of
    exp(logit / temperature), to count its mass off the list; without it the list is renormalised.
    """
    dev, N, V, rows = _rows_and_lists(logits, teacher_ids, teacher_logits)
    loss = torch.empty(N, dtype=_F32, device=logits.device)
    stats = torch.empty((N, 4), dtype=_F32, device=logits.device)
    _call("emb_distill_forward", *rows, _vector(teacher_lse, dev, _F32, N, "teacher_lse"), temperature,
          loss.data_ptr(), stats.data_ptr(), _status(status, dev), _raw_stream(dev))
    return loss, stats


def distill_backward(logits, teacher_ids, teacher_logits, stats, row_weight=None, *, temperature=1.0, out=None,
                     status=None):
    """row_weight[n] * dloss[n] / dlogits from the forward's ``stats``; ``out`` may be ``logits``."""
    dev, N, V, rows = _rows_and_lists(logits, teacher_ids, teacher_logits)
    out, stride = _gradient(logits, out, dev, N, V)
    _call("emb_distill_backward", *rows, _vector(stats, dev, _F32, 4 * N, "stats"),
          _vector(row_weight, dev, _F32, N, "row_weight"), temperature, out.data_ptr(), stride, _status(status, dev),
          _raw_stream(dev))
    return out


def distill_step(logits, teacher_ids, teacher_logits, row_weight=None, *, temperature=1.0, teacher_lse=None, out=None,
                 status=None):
    """(loss [N], row_weight[n] * dloss[n] / dlogits) in one call; ``out`` may be ``logits``."""
    dev, N, V, rows = _rows_and_lists(logits, teacher_ids, teacher_logits)
    loss = torch.empty(N, dtype=_F32, device=logits.device)
    out, stride = _gradient(logits, out, dev, N, V)
    _call("emb_distill_step", *rows, _vector(teacher_lse, dev, _F32, N, "teacher_lse"),
          _vector(row_weight, dev, _F32, N, "row_weight"), temperature, loss.data_ptr(), out.data_ptr(), stride,
          _status(status, dev), _raw_stream(dev))
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
        """(device index, format code, pointers of codes and scales)."""
        codes, scales, dev = self.codes, self.scales, self.codes.get_device()
        fmt = _FORMAT.get(self.format)
        if fmt is None:
            raise ValueError(f"the format of {name} must be 'mx' or 'nv', got {self.format!r}")
        if codes.numel() != self.rows * _row_bytes(self.cols) or \
                scales.numel() != _scale_bytes(self.rows, self.cols, self.format):
            raise ValueError(f"the codes or scales of {name} do not fit its shape")
        if dev < 0 or scales.get_device() != dev or codes.dtype is not torch.uint8 or \
                scales.dtype is not torch.uint8 or not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError(f"codes and scales of {name} must be contiguous uint8 CUDA tensors on one device")
        return dev, fmt, codes.data_ptr(), scales.data_ptr()


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
    dev, xc, xs = _matrix(x, "x")
    R, K = x.shape
    fmt = _FORMAT.get(format)
    if fmt is None:
        raise ValueError(f"format must be 'mx' or 'nv', got {format!r}")
    if out is None:
        codes = torch.empty((R, _row_bytes(K)), dtype=torch.uint8, device=x.device)
        scales = torch.empty(((R + 127) // 128, _tiles(K, format), 32, 4, 4), dtype=torch.uint8, device=x.device)
        out = MicroMatrix(codes, scales, R, K, format, tensor_scale)
    else:
        if (out.rows, out.cols, out.format, out._check("out")[0]) != (R, K, format, dev):
            raise ValueError("out has another shape, format or device")
        out.tensor_scale = tensor_scale
    _call("emb_micro_quantize", dev, x.data_ptr(), xc, xs, R, K, fmt, tensor_scale, out.codes.data_ptr(),
          out.scales.data_ptr(), _raw_stream(dev))
    return out


def micro_lookup(table, ids=None, *, dtype=torch.float32, out=None, status=None):
    """Rows ``ids`` (int64; all rows if not given) of ``table`` as values [n, cols]."""
    dev, fmt, codes, scales = table._check("table")
    n = table.rows if ids is None else ids.numel()
    if out is None:
        out = torch.empty((n, table.cols), dtype=dtype, device=table.codes.device)
        oc, stride = _DTYPE.get(dtype, -1), table.cols
    else:
        oc, stride = _out_like(out, dev, n, table.cols, None)
    _call("emb_micro_lookup", dev, codes, scales, table.rows, table.cols, fmt, table.tensor_scale,
          _vector(ids, dev, _I64, n, "ids"), n, out.data_ptr(), oc, stride, _status(status, dev), _raw_stream(dev))
    return out


def micro_matmul(x, w, *, dtype=torch.bfloat16, out=None, status=None):
    """x [M, K] times the transpose of w [N, K], both MicroMatrix of one format: [M, N] as ``dtype``."""
    dev, fmt, xc, xs = x._check("x")
    at, wfmt, wc, ws = w._check("w")
    if wfmt != fmt or w.cols != x.cols or at != dev:
        raise ValueError("x and w must have the same format, columns and device")
    M, N = x.rows, w.rows
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=x.codes.device)
        oc, stride = _DTYPE.get(dtype, -1), N
    else:
        oc, stride = _out_like(out, dev, M, N, None)
    _call("emb_micro_matmul", dev, xc, xs, x.tensor_scale, M, wc, ws, w.tensor_scale, N, x.cols, fmt, out.data_ptr(), oc,
          stride, _status(status, dev), _raw_stream(dev))
    return out
