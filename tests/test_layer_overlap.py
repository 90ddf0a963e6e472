"""Outputs of the layer operators that share memory with inputs or with one
another: refused on the host before any CUDA call (a kernel reads its inputs
while it writes).  Addresses only; nothing is launched."""
import itertools

import pytest

import mhc_hyper_connection_gb300 as mp
from mhc_hyper_connection_gb300 import build as mbuild

T, N, D, F = 300, 4, 64, 136            # F: two blocks of scales, the second short
GAP = 1 << 24


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mp.library()


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


def _struct(cls, run, kw):
    def call(at):
        a = cls(**kw)
        for k, v in at.items():
            setattr(a, k, v)
        return run(a)
    return call


def _cases():
    """(name, call of {tensor: address}, outputs, inputs): tensors as {name: bytes}."""
    nb = N * D
    st, w = T * nb * 2, F * D * 2
    yield ("pack", lambda at: mp.mhc_ckpt8_pack_run(T, D, 0, at["x"], at["codes"], at["scales"]),
           {"codes": T * D, "scales": T}, {"x": T * D * 2})
    yield ("restore", lambda at: mp.mhc_ckpt8_restore_run(T, D, 0, at["codes"], at["scales"], at["x"]),
           {"x": T * D * 2}, {"codes": T * D, "scales": T})
    yield ("post_ckpt", lambda at: mp.mhc_post_ckpt_run(T, N, D, *(at[k] for k in ("x", "residual", "post", "comb", "out",
                                                                                  "codes", "scales"))),
           {"out": st, "codes": st // 2, "scales": T * N},
           {"x": T * D * 2, "residual": st, "post": T * N * 4, "comb": T * N * N * 4})
    outs = {"grad_x": T * D * 2, "grad_residual": st, "grad_post": T * N * 4, "grad_comb": T * N * N * 4}
    ins = {"grad_out": st, "x": T * D * 2, "post": T * N * 4, "comb": T * N * N * 4}
    run = _struct(mp.MhcPostBwdArgs, mp.mhc_post_backward_run, dict(T=T, n=N, D=D))
    yield "post_backward", run, outs, dict(ins, residual=st)
    yield "post_backward from codes", run, outs, dict(ins, codes=st // 2, scales=T * N)
    for kept in ({}, {"gate_up": T * 2 * F * 2}, {"codes": T * 2 * F, "scales": T * 2 * 2}):
        ws = mp.mhc_ffn_workspace_size(T, D, F)[1]
        yield ("ffn", _struct(mp.MhcFfnArgs, mp.mhc_ffn_run, dict(T=T, D=D, F=F, workspace_bytes=ws)),
               dict(kept, y=T * D * 2, workspace=ws), {"x": T * D * 2, "w_gate_up": 2 * w, "w_down": w})
        if kept:
            ws = mp.mhc_ffn_backward_workspace_size(T, D, F)[1]
            yield ("ffn_backward", _struct(mp.MhcFfnBwdArgs, mp.mhc_ffn_backward_run, dict(T=T, D=D, F=F, workspace_bytes=ws)),
                   {"grad_x": T * D * 2, "grad_w_gate_up": 2 * w, "grad_w_down": w, "workspace": ws},
                   dict(kept, grad_y=T * D * 2, x=T * D * 2, w_gate_up=2 * w, w_down=w))


def test_overlaps_are_refused(lib):
    for name, call, outs, ins in _cases():
        size = {**outs, **ins}
        apart = {k: GAP * (i + 1) for i, k in enumerate(size)}
        for a, b in list(itertools.product(outs, ins)) + list(itertools.permutations(outs, 2)):
            # the same start; b begins in a's last 256 bytes, and a in b's
            for at in ({b: apart[a]}, {b: apart[a] + (size[a] - 1) // 256 * 256}, {a: apart[b] + (size[b] - 1) // 256 * 256}):
                assert call({**apart, **at}) == mp.MHC_ERR_PARAM_INVALID, (name, a, b, at)
                assert "overlaps" in mp.last_error(), (name, a, b, mp.last_error())


def test_tensors_side_by_side_are_not(lib):
    """Rows that follow one another without a gap, and inputs that share memory,
    pass the checks: without a GPU the call then fails where it needs one."""
    if not _no_gpu():
        pytest.skip("a GPU is present")
    for name, call, outs, ins in _cases():
        at, here = {}, GAP
        for k, v in {**outs, **ins}.items():
            at[k], here = here, here + (v + 255) // 256 * 256
        assert call(at) == mp.MHC_ERR_RUNTIME, (name, mp.last_error())
        first = next(iter(ins))
        assert call({**at, **{k: at[first] for k in ins}}) == mp.MHC_ERR_RUNTIME, (name, mp.last_error())
