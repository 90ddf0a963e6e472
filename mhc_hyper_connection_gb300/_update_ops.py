"""Orthogonalised updates of weight matrices on torch tensors.

Argument checks and marshalling only, in the manner of _layer_ops; the
computation is in the CUDA library (include/mhc_orth.h).
"""
from __future__ import annotations

import ctypes
from ctypes import byref, c_size_t
from functools import lru_cache

import torch

from ._binding import MHC_DTYPE_FP32, MhcOrthArgs
from ._layer_ops import _DTYPES, _at, _bf16, _check, _lib, _on, _stream, _u8

# (a, b, c) of each step, X <- a X + (b A + c A A) X with A = X X^T: five steps that take
# singular values from a few thousandths up into [0.7, 1.2] (the coefficients in common
# use for this iteration).
NEWTON_SCHULZ = ((3.4445, -4.7750, 2.0315),) * 5

_IN = {**_DTYPES, torch.float32: MHC_DTYPE_FP32}


@lru_cache(maxsize=64)
def _coefficients(steps):
    if any(len(step) != 3 for step in steps):
        raise ValueError("steps must be (a, b, c) triples")
    flat = [float(v) for step in steps for v in step]
    return (ctypes.c_float * len(flat))(*flat)


@lru_cache(maxsize=256)
def _scratch_bytes(batch, rows, cols) -> int:
    n = c_size_t(0)
    _check(_lib.mhc_orth_workspace_size(batch, rows, cols, byref(n)), "mhc_orth_workspace_size")
    return n.value


def _sizes(shape):
    if len(shape) < 2:
        raise ValueError("update must have at least two dimensions")
    batch = 1
    for n in shape[:-2]:
        batch *= n
    return batch, shape[-2], shape[-1]


def orthogonalise_workspace(shape, device):
    """Scratch (uint8) that orthogonalise takes for an update of this shape: for callers
    that keep one buffer over calls or want to read its status afterwards."""
    ws = torch.empty((max(_scratch_bytes(*_sizes(tuple(shape))), 256),), dtype=_u8, device=device)
    ws[:256].zero_()
    return ws


def orthogonalise_status(workspace, stream=None) -> int:
    """Waits for `stream` (default: torch's current stream), then the device status of
    the last call that used `workspace`: MHC_ERR_RUNTIME if one of its waits gave up."""
    return _lib.mhc_orth_status(_at(workspace, "workspace", _u8, workspace.shape, workspace.device),
                                _stream(stream, workspace.device))


def orthogonalise(update, steps=NEWTON_SCHULZ, eps=1e-7, out=None, workspace=None, stream=None):
    """The matrices of update (fp32, bf16 or fp16 [..., rows, cols]) divided by their norm
    + eps and brought near the closest ones with orthonormal rows (or columns, the
    shorter side) by Newton-Schulz steps (a, b, c): X <- a X + (b A + c A A) X, A = X X^T
    (include/mhc_orth.h, which states the precision).  Returns bf16 of the same shape, or
    `out` (bf16 or fp16).  Products run on fp16 operands with fp32 sums.  A device wait
    that gave up is reported by orthogonalise_status on a given workspace only."""
    shape, dev = update.shape, update.device
    dt = _IN.get(update.dtype)
    if dt is None:
        raise ValueError(f"update must be fp32, bf16 or fp16 (got {update.dtype})")
    batch, rows, cols = _sizes(shape)
    coefficients = _coefficients(tuple(tuple(s) for s in steps))
    xp = _at(update, "update", update.dtype, shape, dev)
    raw, made = _stream(stream, dev), []
    if out is None:
        out = torch.empty(shape, dtype=_bf16, device=dev)
        made.append(out)
        od, op = _DTYPES[_bf16], out.data_ptr()
    else:
        od = _DTYPES.get(out.dtype)
        if od is None:
            raise ValueError(f"out must be bf16 or fp16 (got {out.dtype})")
        op = _at(out, "out", out.dtype, shape, dev)
    if workspace is None:
        n = _scratch_bytes(batch, rows, cols)
        workspace = torch.empty((n,), dtype=_u8, device=dev)
        made.append(workspace)
        wp = workspace.data_ptr()
    else:
        wp, n = _at(workspace, "workspace", _u8, workspace.shape, dev), workspace.numel()
    if stream is not None and made:
        _on(raw, stream, dev, *made)
    a = MhcOrthArgs(batch, rows, cols, dt, od, len(coefficients) // 3, eps, coefficients, xp, op, wp, n)
    _check(_lib.mhc_orth_run(byref(a), raw), "mhc_orth_run")
    return out
