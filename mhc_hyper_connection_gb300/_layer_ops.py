"""The layer operators on torch tensors: 8-bit checkpoints, the post-mapping
with a checkpoint and its backward, the gated feed-forward block.

Argument checks and marshalling only; the computation is in the CUDA library
(include/mhc_ckpt.h, mhc_post_backward.h, mhc_ffn.h).  A call of these is as
short as a launch or two, so the checks are one comparison each and torch's
current stream is read as a raw handle.  Contiguous CUDA tensors on the current
device only.

Outputs given to a call must overlap neither its inputs nor one another (MhcError).
Nothing is recorded for automatic differentiation: the backward calls are made by
hand, as examples/train_layer.py does.

A call runs on `stream` (torch's current one if None).  If that is another
stream, it waits for the current one only where the call allocates something;
what the inputs still wait for is the caller's to order.
"""
from __future__ import annotations

from ctypes import byref, c_size_t
from typing import NamedTuple

import torch

from ._binding import (CKPT_BLOCK, MHC_DTYPE_BF16, MHC_DTYPE_FP16, MHC_FFN_GELU, MHC_FFN_SILU, MHC_OK, MhcError,
                       MhcFfnArgs, MhcFfnBwdArgs, MhcPostBwdArgs, last_error, library)

_lib = library()
_bf16, _f32, _u8 = torch.bfloat16, torch.float32, torch.uint8
_DTYPES = {torch.bfloat16: MHC_DTYPE_BF16, torch.float16: MHC_DTYPE_FP16}
_ACTS = {"silu": MHC_FFN_SILU, "gelu": MHC_FFN_GELU}
_current_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


class Ckpt8(NamedTuple):
    """An 8-bit checkpoint of a 16-bit tensor [..., D]: codes uint8 [..., D] and
    scales uint8 [..., ceil(D / 128)] (block exponent + 127)."""
    codes: torch.Tensor
    scales: torch.Tensor


def _stream(stream, device) -> int:
    """Raw handle of a torch stream, an integer, or torch's current stream.
    The library launches on the current device, so the tensors' device has to
    be that one."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device (got {device})")
    if device.index != _current_device():
        raise ValueError(f"tensors are on {device}, but the current CUDA device is cuda:{_current_device()} "
                         "(make theirs current for the call: torch.cuda.device)")
    if stream is None:
        return _current_raw_stream(device.index)
    return int(getattr(stream, "cuda_stream", stream))


def _on(raw, stream, device, *made):
    """Tensors that a call allocated come from torch's current stream.  If the
    call runs on another one (`stream` given), that one first waits for what
    the current stream may still do with their memory, and the allocator is
    told that it uses them."""
    if stream is not None and raw != _current_raw_stream(device.index):
        ext = torch.cuda.ExternalStream(raw, device=device)
        ext.wait_stream(torch.cuda.current_stream(device))
        for t in made:
            t.record_stream(ext)


def _at(t, name, dtype, shape, device) -> int:
    """Address of a contiguous tensor that must have this dtype, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} {tuple(shape)} on {device} (got {t.dtype} "
                     f"{tuple(t.shape)}{'' if t.is_contiguous() else ', not contiguous,'} on {t.device})")


def _x16(x, name="x") -> int:
    """Type code of a 16-bit tensor."""
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise ValueError(f"{name} must be bf16 or fp16 (got {x.dtype})")
    return dt


def _tokens(lead) -> int:
    """Token count of the leading dims: (T,) or (B, S)."""
    if len(lead) == 1:
        return lead[0]
    if len(lead) == 2:
        return lead[0] * lead[1]
    raise ValueError("leading dims must be (T,) or (B, S)")


def _lead(shape):
    """(T, leading dims, n, D) of streams [T, n, D] or [B, S, n, D]."""
    if len(shape) == 3:
        T, n, D = shape
        return T, (T,), n, D
    *lead, n, D = shape if len(shape) > 1 else (0, 0)
    lead = tuple(lead)
    return _tokens(lead), lead, n, D


def _check(st, where):
    if st != MHC_OK:
        raise MhcError(st, where, last_error())


def _scales_shape(shape):
    *lead, D = shape
    return (*lead, (D + CKPT_BLOCK - 1) // CKPT_BLOCK)


def _ckpt_new(shape, device) -> Ckpt8:
    return Ckpt8(torch.empty(shape, dtype=_u8, device=device),
                 torch.empty(_scales_shape(shape), dtype=_u8, device=device))


def _ckpt_at(ckpt, shape, device):
    return _at(ckpt.codes, "codes", _u8, shape, device), _at(ckpt.scales, "scales", _u8, _scales_shape(shape), device)


def _ckpt_out(ckpt, shape, device):
    """A checkpoint to write into, given or new, and its addresses."""
    if ckpt is None:
        ckpt = _ckpt_new(shape, device)
        return ckpt, ckpt.codes.data_ptr(), ckpt.scales.data_ptr()
    return (ckpt,) + _ckpt_at(ckpt, shape, device)


def _out(t, name, like):
    """A tensor to write into, given or new, of another's type and shape, and its address."""
    if t is None:
        t = torch.empty_like(like)
        return t, t.data_ptr()
    return t, _at(t, name, like.dtype, like.shape, like.device)


def ckpt8_pack(x, out=None, stream=None) -> Ckpt8:
    """The 8-bit checkpoint of x (bf16 or fp16 [..., D], D a multiple of 8):
    e4m3 codes with one power-of-two scale per 128 columns.  `out` is a Ckpt8
    to write into.  Raises MhcError on a host-side rejection."""
    dt, shape, dev = _x16(x), x.shape, x.device
    if not shape:
        raise ValueError("x must have at least one dimension")
    D = shape[-1]
    xp = _at(x, "x", x.dtype, shape, dev)
    raw, given = _stream(stream, dev), out
    out, codes, scales = _ckpt_out(out, shape, dev)
    if stream is not None and given is None:
        _on(raw, stream, dev, *out)
    _check(_lib.mhc_ckpt8_pack_run(x.numel() // D if D else 0, D, dt, xp, codes, scales, raw), "mhc_ckpt8_pack_run")
    return out


def ckpt8_restore(ckpt, dtype=None, out=None, stream=None):
    """The 16-bit tensor a checkpoint stands for (exact; dtype: the type it was
    packed from, default bf16).  A Ckpt8 does not hold that type: a bf16
    checkpoint read as fp16 is rounded as a cast would."""
    codes = ckpt.codes
    shape, dev = codes.shape, codes.device
    cp, sp = _ckpt_at(ckpt, shape, dev)
    raw = _stream(stream, dev)
    if out is None:
        out = torch.empty(shape, dtype=dtype or _bf16, device=dev)
        op = out.data_ptr()
        if stream is not None:
            _on(raw, stream, dev, out)
    else:
        op = _at(out, "out", dtype or out.dtype, shape, dev)
    D = shape[-1]
    _check(_lib.mhc_ckpt8_restore_run(codes.numel() // D if D else 0, D, _x16(out, "out"), cp, sp, op, raw),
           "mhc_ckpt8_restore_run")
    return out


def hc_post_ckpt(x, residual, post, comb, out=None, ckpt=None, stream=None):
    """hc_post that also writes the 8-bit checkpoint of its output in the same
    pass; returns (out, Ckpt8).  Same tensors and layouts as hc_post."""
    shape, dev = residual.shape, residual.device
    T, lead, n, D = _lead(shape)
    rp = _at(residual, "residual", _bf16, shape, dev)
    xp = _at(x, "x", _bf16, lead + (D,), dev)
    pp = _at(post, "post", _f32, lead + (n,), dev)
    cp = _at(comb, "comb", _f32, lead + (n, n), dev)
    raw = _stream(stream, dev)
    made = () if stream is None else (out is None, ckpt is None)
    out, op = _out(out, "out", residual)
    ckpt, codes, scales = _ckpt_out(ckpt, shape, dev)
    if any(made):
        _on(raw, stream, dev, *((out,) if made[0] else ()), *(ckpt if made[1] else ()))
    _check(_lib.mhc_post_ckpt_run(T, n, D, xp, rp, pp, cp, op, codes, scales, raw), "mhc_post_ckpt_run")
    return out, ckpt


def hc_post_backward(grad_out, x, residual, post, comb, grads=None, stream=None):
    """Backward of hc_post (include/mhc_post_backward.h): grad_out bf16
    [T, n, D] (or BSND), the forward's x, post and comb, and its residual as
    bf16 or as a Ckpt8.  Returns {"grad_x", "grad_residual" (bf16),
    "grad_post", "grad_comb" (fp32)}, written into `grads` when given."""
    shape, dev = grad_out.shape, grad_out.device
    T, lead, n, D = _lead(shape)
    gp = _at(grad_out, "grad_out", _bf16, shape, dev)
    xp = _at(x, "x", _bf16, lead + (D,), dev)
    pp = _at(post, "post", _f32, lead + (n,), dev)
    cp = _at(comb, "comb", _f32, lead + (n, n), dev)
    rp = codes = scales = None
    if isinstance(residual, Ckpt8):
        codes, scales = _ckpt_at(residual, shape, dev)
    else:
        rp = _at(residual, "residual", _bf16, shape, dev)
    raw = _stream(stream, dev)
    if grads is None:
        grads = {"grad_x": torch.empty_like(x), "grad_residual": torch.empty_like(grad_out),
                 "grad_post": torch.empty_like(post), "grad_comb": torch.empty_like(comb)}
        out = [t.data_ptr() for t in grads.values()]
        if stream is not None:
            _on(raw, stream, dev, *grads.values())
    else:
        out = [_at(grads["grad_x"], "grad_x", _bf16, x.shape, dev),
               _at(grads["grad_residual"], "grad_residual", _bf16, shape, dev),
               _at(grads["grad_post"], "grad_post", _f32, post.shape, dev),
               _at(grads["grad_comb"], "grad_comb", _f32, comb.shape, dev)]
    a = MhcPostBwdArgs(T, n, D, gp, xp, rp, codes, scales, pp, cp, *out)
    _check(_lib.mhc_post_backward_run(byref(a), raw), "mhc_post_backward_run")
    return grads


# ------------------------------------------------------- gated feed-forward block

def _scratch_bytes(T, D, F, backward) -> int:
    n = c_size_t(0)
    if backward:
        _check(_lib.mhc_ffn_backward_workspace_size(T, D, F, byref(n)), "mhc_ffn_backward_workspace_size")
    else:
        _check(_lib.mhc_ffn_workspace_size(T, D, F, byref(n)), "mhc_ffn_workspace_size")
    return n.value


def gated_ffn_workspace(T: int, D: int, F: int, device, backward: bool = False):
    """Scratch (uint8) that gated_ffn, or with backward=True
    gated_ffn_backward, takes for T tokens: for callers that keep one buffer
    over calls or want to read its status afterwards."""
    ws = torch.empty((max(_scratch_bytes(T, D, F, backward), 256),), dtype=_u8, device=device)
    ws[:256].zero_()
    return ws


def gated_ffn_status(workspace=None, stream=None) -> int:
    """Waits for `stream` (default: torch's current stream), then the device
    status of the last call that used `workspace`: MHC_ERR_RUNTIME if one of its
    waits gave up.  Without a workspace only the stream's own errors are seen:
    the status of a call lies in its workspace."""
    if workspace is None:
        raw = _current_raw_stream(_current_device()) if stream is None else int(getattr(stream, "cuda_stream", stream))
        return _lib.mhc_ffn_status(None, raw or None)
    return _lib.mhc_ffn_status(_at(workspace, "workspace", _u8, workspace.shape, workspace.device),
                               _stream(stream, workspace.device))


def _scratch(workspace, T, D, F, backward, device, made):
    """Workspace of one call: the tensor, its address, its bytes; a new one is
    added to `made`."""
    if workspace is None:
        n = _scratch_bytes(T, D, F, backward)
        workspace = torch.empty((n,), dtype=_u8, device=device)
        made.append(workspace)
        return workspace, workspace.data_ptr(), n
    return workspace, _at(workspace, "workspace", _u8, workspace.shape, device), workspace.numel()


def _ffn_inputs(x, w_gate_up, w_down, act):
    """Checked inputs: (type code, act code, T, D, F, shape of the kept sums,
    addresses of x, w_gate_up, w_down)."""
    dt, dev, xt = _x16(x), x.device, x.dtype
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)} (got {act!r})")
    ws = w_gate_up.shape
    if len(ws) != 3 or ws[0] != 2:
        raise ValueError("w_gate_up must be [2, F, D]")
    *lead, D = x.shape
    lead, F = tuple(lead), ws[1]
    return (dt, _ACTS[act], _tokens(lead), D, F, lead + (2, F), _at(x, "x", xt, x.shape, dev),
            _at(w_gate_up, "w_gate_up", xt, (2, F, D), dev), _at(w_down, "w_down", xt, (D, F), dev))


def gated_ffn(x, w_gate_up, w_down, act="silu", save=None, y=None, kept=None, workspace=None, stream=None):
    """y = (act(x Wg^T) (.) x Wu^T) Wd^T (include/mhc_ffn.h): x bf16 or fp16
    [T, D] (or [B, S, D]), w_gate_up [2, F, D] (Wg, Wu), w_down [D, F], act
    "silu" or "gelu" (tanh form).  save keeps both projections for the
    backward: "16bit" as a tensor [T, 2, F], "8bit" as a Ckpt8 of that shape.
    Returns (y, kept); kept is None without save.  y, kept and workspace are
    allocated unless given; a device wait that gave up (outputs are then
    incomplete) is reported by gated_ffn_status on a given workspace only."""
    dt, ac, T, D, F, shape, xp, gp, wp = _ffn_inputs(x, w_gate_up, w_down, act)
    dev = x.device
    kp = codes = scales = None
    raw, made = _stream(stream, dev), []
    if save is None:
        if kept is not None:
            raise ValueError("kept goes with save")
    elif save == "16bit":
        if kept is None:
            kept = torch.empty(shape, dtype=x.dtype, device=dev)
            made.append(kept)
        kp = _at(kept, "kept", x.dtype, shape, dev)
    elif save == "8bit":
        if kept is None:
            kept = _ckpt_new(shape, dev)
            made.extend(kept)
        codes, scales = _ckpt_at(kept, shape, dev)
    else:
        raise ValueError(f'save must be None, "16bit" or "8bit" (got {save!r})')
    if y is None:
        y = torch.empty_like(x)
        made.append(y)
    yp = _at(y, "y", x.dtype, x.shape, dev)
    workspace, p, n = _scratch(workspace, T, D, F, False, dev, made)
    if stream is not None and made:
        _on(raw, stream, dev, *made)
    a = MhcFfnArgs(T, D, F, dt, ac, xp, gp, wp, yp, kp, codes, scales, p, n)
    _check(_lib.mhc_ffn_run(byref(a), raw), "mhc_ffn_run")
    return y, kept


def gated_ffn_backward(grad_y, x, w_gate_up, w_down, kept, act="silu", grads=None, workspace=None, stream=None):
    """Backward of gated_ffn from what it kept (a tensor or a Ckpt8): returns
    {"grad_x", "grad_w_gate_up", "grad_w_down"} in x's type, written into
    `grads` when given.  Status as for gated_ffn."""
    dt, ac, T, D, F, shape, xp, gp, wp = _ffn_inputs(x, w_gate_up, w_down, act)
    dev, xt = x.device, x.dtype
    yp = _at(grad_y, "grad_y", xt, x.shape, dev)
    kp = codes = scales = None
    if isinstance(kept, Ckpt8):
        codes, scales = _ckpt_at(kept, shape, dev)
    else:
        kp = _at(kept, "kept", xt, shape, dev)
    raw, made = _stream(stream, dev), []
    if grads is None:
        grads = {"grad_x": torch.empty_like(x), "grad_w_gate_up": torch.empty_like(w_gate_up),
                 "grad_w_down": torch.empty_like(w_down)}
        out = [t.data_ptr() for t in grads.values()]
        made.extend(grads.values())
    else:
        out = [_at(grads["grad_x"], "grad_x", xt, x.shape, dev),
               _at(grads["grad_w_gate_up"], "grad_w_gate_up", xt, w_gate_up.shape, dev),
               _at(grads["grad_w_down"], "grad_w_down", xt, w_down.shape, dev)]
    workspace, p, n = _scratch(workspace, T, D, F, True, dev, made)
    if stream is not None and made:
        _on(raw, stream, dev, *made)
    a = MhcFfnBwdArgs(T, D, F, dt, ac, yp, xp, gp, wp, kp, codes, scales, *out, p, n)
    _check(_lib.mhc_ffn_backward_run(byref(a), raw), "mhc_ffn_backward_run")
    return grads
