"""Routed experts on torch tensors: the router and its gradient, the plan of the
routed tokens, the experts' gated feed-forward blocks and their backward.

Argument checks and marshalling only, in the manner of _layer_ops; the
computation is in the CUDA library (include/mhc_route.h, mhc_experts.h).
Contiguous CUDA tensors on the current device only; outputs given to a call must
overlap neither its inputs nor one another (MhcError).  Nothing is recorded for
automatic differentiation.

    routes = route_experts(logits, k, ...)                      # experts, weights
    plan = expert_plan(routes.experts, E)
    y, kept = experts_ffn(x, routes.weights, plan, w_gate_up, w_down, save="16bit")
    g = experts_ffn_backward(grad_y, x, routes.weights, plan, w_gate_up, w_down, kept)
    grad_logits = route_experts_backward(g["grad_weights"], logits, routes.experts, ...)
"""
from __future__ import annotations

from ctypes import byref, c_int64, c_size_t
from functools import lru_cache
from typing import NamedTuple

import torch

from ._binding import (MHC_DTYPE_FP32, MHC_GROUP_MAX, MHC_GROUP_TOP2, MHC_SCORE_SIGMOID, MHC_SCORE_SOFTMAX,
                       MhcExpertsArgs, MhcExpertsBwdArgs, MhcRouteArgs, MhcRouteBwdArgs)
from ._layer_ops import _ACTS, _DTYPES, _at, _check, _f32, _lib, _on, _stream, _tokens, _u8, _x16

_i32 = torch.int32
_LOGITS = {**_DTYPES, torch.float32: MHC_DTYPE_FP32}
_SCORES = {"softmax": MHC_SCORE_SOFTMAX, "sigmoid": MHC_SCORE_SIGMOID}
_GROUP_SCORES = {"max": MHC_GROUP_MAX, "top2": MHC_GROUP_TOP2}


class Routes(NamedTuple):
    """experts int32 [T, k] (-1: none) and weights fp32 [T, k]; leading dims (T,) or
    (B, S)."""
    experts: torch.Tensor
    weights: torch.Tensor


class ExpertPlan(NamedTuple):
    """The slots of experts [T, k] in the order in which the experts take them
    (include/mhc_route.h): an opaque buffer and the sizes it was made for."""
    buffer: torch.Tensor
    lead: tuple
    k: int
    num_experts: int
    rows: int

    @property
    def counts(self):
        """Slots of each expert, int32 [E] (a view)."""
        return self.buffer[256:256 + 4 * self.num_experts].view(_i32)


def _kind(logits, score):
    dt = _LOGITS.get(logits.dtype)
    if dt is None:
        raise ValueError(f"logits must be fp32, bf16 or fp16 (got {logits.dtype})")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)} (got {score!r})")
    if logits.dim() not in (2, 3):
        raise ValueError("logits must be [T, E] or [B, S, E]")
    return dt, _SCORES[score]


def route_experts(logits, top_k, score="softmax", bias=None, groups=1, top_groups=None, group_score="top2",
                  renormalise=True, scale=1.0, out=None, stream=None) -> Routes:
    """The top_k experts of every token and their weights (include/mhc_route.h).

    logits fp32, bf16 or fp16 [T, E] (or [B, S, E]); score "softmax" over the row or
    "sigmoid"; bias fp32 [E] is added to the scores for the choice alone; with
    groups > 1 only experts of the top_groups best of so many runs of E / groups are
    taken, a group counting for its largest ("max") or two largest ("top2") scores.
    Weights are the scores, divided by their sum with renormalise, times scale.  A
    logit of -inf takes its expert out; slots without an expert hold -1 and 0.  Ties
    go to the lower index, -0 and +0 being one.  `out` is a Routes to write into.
    Logits begin at an address of four elements where E is a multiple of four, of two
    where it is even (every tensor that is no view does; else MhcError)."""
    dt, sc = _kind(logits, score)
    if group_score not in _GROUP_SCORES:
        raise ValueError(f"group_score must be one of {sorted(_GROUP_SCORES)} (got {group_score!r})")
    *lead, E = logits.shape
    lead, dev, k = tuple(lead), logits.device, int(top_k)
    lp = _at(logits, "logits", logits.dtype, logits.shape, dev)
    bp = None if bias is None else _at(bias, "bias", _f32, (E,), dev)
    raw = _stream(stream, dev)
    shape = lead + (k,)
    if out is None:
        if k < 1:
            raise ValueError(f"top_k must be at least 1 (got {k})")
        out = Routes(torch.empty(shape, dtype=_i32, device=dev), torch.empty(shape, dtype=_f32, device=dev))
        ep, wp = out.experts.data_ptr(), out.weights.data_ptr()
        if stream is not None:
            _on(raw, stream, dev, *out)
    else:
        ep, wp = _at(out.experts, "experts", _i32, shape, dev), _at(out.weights, "weights", _f32, shape, dev)
    a = MhcRouteArgs(_tokens(lead), E, k, dt, sc, groups, groups if top_groups is None else top_groups,
                     _GROUP_SCORES[group_score], 1 if renormalise else 0, scale, lp, bp, ep, wp)
    _check(_lib.mhc_route_run(byref(a), raw), "mhc_route_run")
    return out


def route_experts_backward(grad_weights, logits, experts, score="softmax", renormalise=True, scale=1.0,
                           grad_logits=None, stream=None):
    """The gradient of logits from that of the weights (fp32 [T, k]), for the experts
    that route_experts chose with the same score, renormalise and scale.  Returns
    grad_logits in the logits' type, written into the one given (aligned as the logits
    of route_experts)."""
    dt, sc = _kind(logits, score)
    *lead, E = logits.shape
    lead, dev = tuple(lead), logits.device
    k = experts.shape[-1] if experts.dim() else 0
    shape = lead + (k,)
    lp = _at(logits, "logits", logits.dtype, logits.shape, dev)
    ep = _at(experts, "experts", _i32, shape, dev)
    gp = _at(grad_weights, "grad_weights", _f32, shape, dev)
    raw = _stream(stream, dev)
    if grad_logits is None:
        grad_logits = torch.empty_like(logits)
        op = grad_logits.data_ptr()
        if stream is not None:
            _on(raw, stream, dev, grad_logits)
    else:
        op = _at(grad_logits, "grad_logits", logits.dtype, logits.shape, dev)
    a = MhcRouteBwdArgs(_tokens(lead), E, k, dt, sc, 1 if renormalise else 0, scale, lp, ep, gp, op)
    _check(_lib.mhc_route_backward_run(byref(a), raw), "mhc_route_backward_run")
    return grad_logits


@lru_cache(maxsize=256)
def _plan_sizes(T, k, E):
    n, rows = c_size_t(0), c_int64(0)
    _check(_lib.mhc_expert_plan_size(T, k, E, byref(n)), "mhc_expert_plan_size")
    _check(_lib.mhc_expert_plan_rows(T, k, E, byref(rows)), "mhc_expert_plan_rows")
    return n.value, rows.value


def expert_plan(experts, num_experts, buffer=None, stream=None) -> ExpertPlan:
    """The plan of experts (int32 [T, k] or [B, S, k]): what experts_ffn and its
    backward read.  Slots with an expert outside [0, num_experts) take no part.
    `buffer` is the buffer of an earlier plan of the same sizes to write into."""
    if experts.dim() not in (2, 3):
        raise ValueError("experts must be [T, k] or [B, S, k]")
    *lead, k = experts.shape
    lead, dev, E = tuple(lead), experts.device, int(num_experts)
    T = _tokens(lead)
    xp = _at(experts, "experts", _i32, experts.shape, dev)
    raw = _stream(stream, dev)
    n, rows = _plan_sizes(T, k, E)
    if buffer is None:
        buffer = torch.empty((n,), dtype=_u8, device=dev)
        bp = buffer.data_ptr()
        if stream is not None:
            _on(raw, stream, dev, buffer)
    else:
        bp = _at(buffer, "buffer", _u8, (n,), dev)
    _check(_lib.mhc_expert_plan_run(T, k, E, xp, bp, n, raw), "mhc_expert_plan_run")
    return ExpertPlan(buffer, lead, k, E, rows)


@lru_cache(maxsize=256)
def _scratch_bytes(T, E, k, D, F, backward) -> int:
    n = c_size_t(0)
    if backward:
        _check(_lib.mhc_experts_backward_workspace_size(T, E, k, D, F, byref(n)), "mhc_experts_backward_workspace_size")
    else:
        _check(_lib.mhc_experts_workspace_size(T, E, k, D, F, byref(n)), "mhc_experts_workspace_size")
    return n.value


def experts_ffn_workspace(T: int, num_experts: int, top_k: int, D: int, F: int, device, backward: bool = False):
    """Scratch (uint8) that experts_ffn, or with backward=True experts_ffn_backward,
    takes: for callers that keep one buffer over calls or want to read its status
    afterwards."""
    ws = torch.empty((max(_scratch_bytes(T, num_experts, top_k, D, F, backward), 256),), dtype=_u8, device=device)
    ws[:256].zero_()
    return ws


def experts_ffn_status(workspace, stream=None) -> int:
    """Waits for `stream` (default: torch's current stream), then the device status of
    the last call that used `workspace`: MHC_ERR_RUNTIME if one of its waits gave up."""
    return _lib.mhc_experts_status(_at(workspace, "workspace", _u8, workspace.shape, workspace.device),
                                   _stream(stream, workspace.device))


def _scratch(workspace, T, E, k, D, F, backward, device, made):
    if workspace is None:
        n = _scratch_bytes(T, E, k, D, F, backward)
        workspace = torch.empty((n,), dtype=_u8, device=device)
        made.append(workspace)
        return workspace, workspace.data_ptr(), n
    return workspace, _at(workspace, "workspace", _u8, workspace.shape, device), workspace.numel()


def _inputs(x, weights, plan, w_gate_up, w_down, act):
    """Checked inputs: (type code, act code, T, E, k, D, F, addresses of x, weights, the
    plan, w_gate_up, w_down)."""
    dt, dev, xt = _x16(x), x.device, x.dtype
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)} (got {act!r})")
    if not isinstance(plan, ExpertPlan):
        raise ValueError("plan must be an ExpertPlan (expert_plan)")
    ws = w_gate_up.shape
    if len(ws) != 4 or ws[1] != 2 or ws[0] != plan.num_experts:
        raise ValueError(f"w_gate_up must be [{plan.num_experts}, 2, F, D], as many experts as the plan has")
    *lead, D = x.shape
    lead, E, F = tuple(lead), ws[0], ws[2]
    if lead != plan.lead:
        raise ValueError(f"the plan is of tokens {plan.lead}, x of {lead}")
    T = _tokens(lead)
    n = _plan_sizes(T, plan.k, E)[0]
    return (dt, _ACTS[act], T, E, plan.k, D, F, _at(x, "x", xt, x.shape, dev),
            _at(weights, "weights", _f32, lead + (plan.k,), dev), _at(plan.buffer, "plan", _u8, (n,), dev),
            _at(w_gate_up, "w_gate_up", xt, (E, 2, F, D), dev), _at(w_down, "w_down", xt, (E, D, F), dev))


def experts_ffn(x, weights, plan, w_gate_up, w_down, act="silu", save=None, y=None, kept=None, workspace=None,
                stream=None):
    """y_t = sum_j weights_tj gated_ffn_e(x_t), e = experts_tj (include/mhc_experts.h): x
    bf16 or fp16 [T, D] (or [B, S, D]), weights fp32 [T, k], plan of the experts,
    w_gate_up [E, 2, F, D] (Wg, Wu), w_down [E, D, F], act "silu" or "gelu" (tanh form).
    save="16bit" keeps both projections for the backward, [plan.rows, 2, F] in the
    plan's order.  Returns (y, kept); kept is None without save.  y, kept and workspace
    are allocated unless given; a device wait that gave up (outputs are then
    incomplete) is reported by experts_ffn_status on a given workspace only."""
    dt, ac, T, E, k, D, F, xp, tp, pp, gp, wp = _inputs(x, weights, plan, w_gate_up, w_down, act)
    dev = x.device
    raw, made, kp = _stream(stream, dev), [], None
    if save is None:
        if kept is not None:
            raise ValueError("kept goes with save")
    elif save == "16bit":
        if kept is None:
            kept = torch.empty((plan.rows, 2, F), dtype=x.dtype, device=dev)
            made.append(kept)
        kp = _at(kept, "kept", x.dtype, (plan.rows, 2, F), dev)
    else:
        raise ValueError(f'save must be None or "16bit" (got {save!r})')
    if y is None:
        y = torch.empty_like(x)
        made.append(y)
    yp = _at(y, "y", x.dtype, x.shape, dev)
    workspace, p, n = _scratch(workspace, T, E, k, D, F, False, dev, made)
    if stream is not None and made:
        _on(raw, stream, dev, *made)
    a = MhcExpertsArgs(T, E, k, D, F, dt, ac, xp, tp, pp, gp, wp, yp, kp, p, n)
    _check(_lib.mhc_experts_run(byref(a), raw), "mhc_experts_run")
    return y, kept


def experts_ffn_backward(grad_y, x, weights, plan, w_gate_up, w_down, kept, act="silu", grads=None, workspace=None,
                         stream=None):
    """Backward of experts_ffn from what it kept: returns {"grad_x", "grad_w_gate_up",
    "grad_w_down"} in x's type and "grad_weights" in fp32, written into `grads` when
    given.  Status as for experts_ffn."""
    dt, ac, T, E, k, D, F, xp, tp, pp, gp, wp = _inputs(x, weights, plan, w_gate_up, w_down, act)
    dev, xt = x.device, x.dtype
    yp = _at(grad_y, "grad_y", xt, x.shape, dev)
    kp = _at(kept, "kept", xt, (plan.rows, 2, F), dev)
    raw, made = _stream(stream, dev), []
    if grads is None:
        grads = {"grad_x": torch.empty_like(x), "grad_weights": torch.empty_like(weights),
                 "grad_w_gate_up": torch.empty_like(w_gate_up), "grad_w_down": torch.empty_like(w_down)}
        out = [t.data_ptr() for t in grads.values()]
        made.extend(grads.values())
    else:
        out = [_at(grads["grad_x"], "grad_x", xt, x.shape, dev),
               _at(grads["grad_weights"], "grad_weights", _f32, weights.shape, dev),
               _at(grads["grad_w_gate_up"], "grad_w_gate_up", xt, w_gate_up.shape, dev),
               _at(grads["grad_w_down"], "grad_w_down", xt, w_down.shape, dev)]
    workspace, p, n = _scratch(workspace, T, E, k, D, F, True, dev, made)
    if stream is not None and made:
        _on(raw, stream, dev, *made)
    a = MhcExpertsBwdArgs(T, E, k, D, F, dt, ac, yp, xp, tp, pp, gp, wp, kp, *out, p, n)
    _check(_lib.mhc_experts_backward_run(byref(a), raw), "mhc_experts_backward_run")
    return grads
