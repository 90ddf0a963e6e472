"""The layer operators' C ABI without a GPU: every function that their headers
declare is exported, struct layouts match, and bad arguments are refused on
the host before any CUDA call."""
import ctypes
import os
import re

import pytest

import mhc_hyper_connection_gb300 as mp
from mhc_hyper_connection_gb300 import build as mbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096     # a non-NULL, well aligned address that no call here reaches


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mp.library()


@pytest.mark.parametrize("header", ["mhc_ckpt.h", "mhc_post_backward.h", "mhc_ffn.h"])
def test_library_exports_every_declared_symbol(lib, header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = re.findall(r"MHC_API[^;(]*?\b(mhc_[a-z0-9_]+)\s*\(", text)
    assert names
    for name in names:
        assert hasattr(lib, name), f"{name} declared in {header} but not exported"


def test_ckpt_refusals(lib):
    pack, restore = mp.mhc_ckpt8_pack_run, mp.mhc_ckpt8_restore_run
    for f in (lambda rows, D, dt, x, c, s: pack(rows, D, dt, x, c, s),
              lambda rows, D, dt, x, c, s: restore(rows, D, dt, c, s, x)):
        assert f(0, 64, 0, 0, 0, 0) == mp.MHC_OK
        for bad in ((-1, 64, 0, P, P, P), (1, 0, 0, P, P, P), (1, 60, 0, P, P, P), (1, (1 << 20) + 8, 0, P, P, P),
                    (1, 64, 2, P, P, P), (1, 64, 0, P + 2, P, P), (1, 64, 0, P, P + 1, P), (1 << 40, 64, 0, P, P, P)):
            assert f(*bad) == mp.MHC_ERR_PARAM_INVALID, bad
            assert mp.last_error()
        for bad in ((1, 64, 0, 0, P, P), (1, 64, 0, P, 0, P), (1, 64, 0, P, P, 0)):
            assert f(*bad) == mp.MHC_ERR_NULLPTR, bad


def test_post_ckpt_refusals(lib):
    f = mp.mhc_post_ckpt_run
    ok = [1, 4, 64] + [P] * 7
    assert f(0, 4, 64, *[0] * 7) == mp.MHC_OK
    for k, v in ((0, -1), (1, 0), (1, 9), (2, 0), (2, 12), (3, P + 8), (4, P + 2), (5, P + 2), (6, P + 1), (7, P + 4),
                 (8, P + 4)):
        a = list(ok)
        a[k] = v
        assert f(*a) == mp.MHC_ERR_PARAM_INVALID, (k, v)
    for k in range(3, 10):
        a = list(ok)
        a[k] = 0
        assert f(*a) == mp.MHC_ERR_NULLPTR, k


def _post_bwd(**kw):
    a = mp.MhcPostBwdArgs()
    a.T, a.n, a.D = 1, 4, 64
    for k in ("grad_out", "x", "residual", "post", "comb", "grad_x", "grad_residual", "grad_post", "grad_comb"):
        setattr(a, k, P)
    for k, v in kw.items():
        setattr(a, k, v)
    return mp.mhc_post_backward_run(a)


def test_post_backward_refusals(lib):
    assert ctypes.sizeof(mp.MhcPostBwdArgs) == 14 * 8
    assert lib.mhc_post_backward_run(None, None) == mp.MHC_ERR_NULLPTR
    assert _post_bwd(T=0, x=None) == mp.MHC_OK
    for kw in ({"T": -1}, {"n": 0}, {"n": 9}, {"D": 0}, {"D": 36}, {"x": P + 8}, {"grad_out": P + 2},
               {"grad_residual": P + 8}, {"post": P + 2}, {"codes": P, "scales": P}, {"codes": P},
               {"residual": None, "codes": P}, {"residual": None, "codes": P + 4, "scales": P}):
        assert _post_bwd(**kw) == mp.MHC_ERR_PARAM_INVALID, kw
        assert mp.last_error()
    for k in ("grad_out", "x", "residual", "post", "comb", "grad_x", "grad_residual", "grad_post", "grad_comb"):
        assert _post_bwd(**{k: None}) == mp.MHC_ERR_NULLPTR, k


def _ffn(backward=False, **kw):
    a = mp.MhcFfnBwdArgs() if backward else mp.MhcFfnArgs()
    a.T, a.D, a.F = 4, 64, 128
    names = ("grad_y", "x", "w_gate_up", "w_down", "gate_up", "grad_x", "grad_w_gate_up", "grad_w_down") if backward \
        else ("x", "w_gate_up", "w_down", "y")
    for k in names + ("workspace",):
        setattr(a, k, P)
    a.workspace_bytes = 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return (mp.mhc_ffn_backward_run if backward else mp.mhc_ffn_run)(a)


def test_ffn_workspace_sizes(lib):
    assert mp.mhc_ffn_workspace_size(0, 64, 128) == (mp.MHC_OK, 0)
    assert mp.mhc_ffn_workspace_size(3, 64, 128) == (mp.MHC_OK, 256 + 768)
    assert mp.mhc_ffn_backward_workspace_size(3, 64, 128) == (mp.MHC_OK, 256 + 1536 + 768)
    for bad in ((-1, 64, 128), (1, 0, 128), (1, 60, 128), (1, 64, 0), (1, 64, 132), ((1 << 24) + 1, 64, 128),
                (1, (1 << 20) + 8, 8)):
        assert mp.mhc_ffn_workspace_size(*bad)[0] == mp.MHC_ERR_PARAM_INVALID
        assert mp.mhc_ffn_backward_workspace_size(*bad)[0] == mp.MHC_ERR_PARAM_INVALID
    assert lib.mhc_ffn_workspace_size(1, 8, 8, None) == mp.MHC_ERR_NULLPTR


@pytest.mark.parametrize("backward", [False, True])
def test_ffn_refusals(lib, backward):
    assert lib.mhc_ffn_run(None, None) == lib.mhc_ffn_backward_run(None, None) == mp.MHC_ERR_NULLPTR
    assert ctypes.sizeof(mp.MhcFfnArgs) == 3 * 8 + 8 + 9 * 8 + 8
    assert ctypes.sizeof(mp.MhcFfnBwdArgs) == 3 * 8 + 8 + 12 * 8 + 8
    if not backward:
        assert _ffn(T=0, x=None) == mp.MHC_OK
    for kw in ({"T": -1}, {"D": 0}, {"D": 60}, {"F": 4}, {"dtype": 2}, {"act": 2}, {"act": -1}, {"x": P + 8},
               {"w_down": P + 2}, {"workspace": P + 16}, {"workspace_bytes": 100}, {"codes": P}, {"scales": P},
               {"gate_up": P, "codes": P, "scales": P}, {"wait_limit_us": 10000001}, {"withhold_copy": 2}):
        assert _ffn(backward, **kw) == mp.MHC_ERR_PARAM_INVALID, kw
        assert mp.last_error()
    for k in ("x", "w_gate_up", "w_down", "workspace") + (("grad_y", "gate_up", "grad_x", "grad_w_gate_up", "grad_w_down")
                                                          if backward else ("y",)):
        assert _ffn(backward, **{k: None}) == mp.MHC_ERR_NULLPTR, k
