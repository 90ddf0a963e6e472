"""The C ABI of the routed experts and of the orthogonalised updates without a GPU:
every declared function is exported, struct layouts match, bad arguments and overlapping
tensors are refused on the host before any CUDA call; and the torch side's own checks."""
import ctypes
import itertools
import os
import re

import pytest
import torch

import mhc_hyper_connection_gb300 as mp
from mhc_hyper_connection_gb300 import build as mbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 40                               # well aligned addresses that no call here reaches, far apart
STEP = 1 << 36


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mp.library()


@pytest.mark.parametrize("header", ["mhc_route.h", "mhc_experts.h", "mhc_orth.h"])
def test_library_exports_every_declared_symbol(lib, header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = re.findall(r"MHC_API[^;(]*?\b(mhc_[a-z0-9_]+)\s*\(", text)
    assert names
    for name in names:
        assert hasattr(lib, name), f"{name} declared in {header} but not exported"


def test_struct_layouts(lib):
    assert ctypes.sizeof(mp.MhcRouteArgs) == 3 * 8 + 7 * 4 + 4 + 4 * 8
    assert ctypes.sizeof(mp.MhcRouteBwdArgs) == 3 * 8 + 4 * 4 + 4 * 8
    assert ctypes.sizeof(mp.MhcExpertsArgs) == 5 * 8 + 8 + 8 * 8 + 8 + 8
    assert ctypes.sizeof(mp.MhcExpertsBwdArgs) == 5 * 8 + 8 + 12 * 8 + 8 + 8
    assert ctypes.sizeof(mp.MhcOrthArgs) == 3 * 8 + 4 * 4 + 4 * 8 + 8 + 8


SPECS = {
    "route": (mp.MhcRouteArgs, mp.mhc_route_run,
              dict(T=100, E=64, k=4, dtype=2, score=0, groups=4, top_groups=2, group_score=1, renormalise=1, scale=1.0),
              {"experts": 1600, "weights": 1600}, {"logits": 25600, "bias": 256}),
    "route_backward": (mp.MhcRouteBwdArgs, mp.mhc_route_backward_run,
                       dict(T=100, E=64, k=4, dtype=2, score=1, renormalise=1, scale=1.0),
                       {"grad_logits": 25600}, {"logits": 25600, "experts": 1600, "grad_weights": 1600}),
    "experts": (mp.MhcExpertsArgs, mp.mhc_experts_run, dict(T=100, E=8, k=2, D=64, F=136, dtype=0, act=0),
                {"y": 12800, "gate_up": 170000, "workspace": None},
                {"x": 12800, "weights": 800, "plan": None, "w_gate_up": 278528, "w_down": 139264}),
    "experts_backward": (mp.MhcExpertsBwdArgs, mp.mhc_experts_backward_run, dict(T=100, E=8, k=2, D=64, F=136, dtype=1, act=1),
                         {"grad_x": 12800, "grad_weights": 800, "grad_w_gate_up": 278528, "grad_w_down": 139264, "workspace": None},
                         {"grad_y": 12800, "x": 12800, "weights": 800, "plan": None, "w_gate_up": 278528, "w_down": 139264,
                          "gate_up": 170000}),
    "orth": (mp.MhcOrthArgs, mp.mhc_orth_run, dict(batch=3, rows=40, cols=72, dtype=2, out_dtype=0, steps=2, eps=1e-7),
             {"out": 17280, "workspace": None}, {"x": 34560}),
}
COEF = (ctypes.c_float * 6)(1.5, -0.5, 0.0, 1.5, -0.5, 0.0)


def _sizes(name):
    outs, ins = dict(SPECS[name][3]), dict(SPECS[name][4])
    if name.startswith("experts"):
        f = mp.mhc_experts_workspace_size if name == "experts" else mp.mhc_experts_backward_workspace_size
        outs["workspace"] = f(100, 8, 2, 64, 136)[1]
        ins["plan"] = mp.mhc_expert_plan_size(100, 2, 8)[1]
    if name == "orth":
        outs["workspace"] = mp.mhc_orth_workspace_size(3, 40, 72)[1]
    return outs, ins


def _call(name, **kw):
    cls, run, sizes, _, _ = SPECS[name]
    outs, ins = _sizes(name)
    a = cls(**sizes)
    for i, k in enumerate({**outs, **ins}):
        setattr(a, k, P + i * STEP)
    if hasattr(a, "workspace_bytes"):
        a.workspace_bytes = outs["workspace"]
    if name == "orth":
        a.coefficients = COEF
    for k, v in kw.items():
        setattr(a, k, v)
    return run(a)


BAD = {
    "route": [dict(T=-1), dict(T=(1 << 20) + 1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33, E=64, groups=1, top_groups=1), dict(k=65),
              dict(T=1 << 20, k=8), dict(dtype=3), dict(score=2), dict(groups=0), dict(groups=3), dict(groups=64), dict(top_groups=0),
              dict(top_groups=5), dict(k=20, top_groups=1), dict(group_score=2), dict(renormalise=2), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(logits=P + 4), dict(logits=P + 2, dtype=0), dict(E=63, groups=1, top_groups=1, logits=P + 2),
              dict(bias=P + 2), dict(experts=P + 2), dict(weights=P + 1)],
    "route_backward": [dict(T=-1), dict(E=0), dict(k=0), dict(k=33), dict(dtype=-1), dict(score=5), dict(renormalise=-1),
                       dict(scale=float("inf")), dict(logits=P + 2), dict(grad_logits=P + 8), dict(experts=P + 2), dict(grad_weights=P + 2)],
    "experts": [dict(T=-1), dict(E=0), dict(k=9), dict(D=60), dict(D=0), dict(D=16392), dict(F=4), dict(F=16392), dict(dtype=2), dict(act=2),
                dict(x=P + 8), dict(y=P + 2), dict(weights=P + 2), dict(gate_up=P + 8), dict(w_down=P + 8), dict(plan=P + 128),
                dict(workspace=P + 16), dict(workspace_bytes=1000), dict(wait_limit_us=10000001), dict(withhold_copy=2)],
    "experts_backward": [dict(T=-1), dict(E=1025), dict(k=0), dict(D=12), dict(F=0), dict(dtype=3), dict(act=-1), dict(grad_y=P + 8),
                         dict(grad_weights=P + 2), dict(grad_w_gate_up=P + 8), dict(plan=P + 4), dict(workspace=P + 128),
                         dict(workspace_bytes=0), dict(wait_limit_us=10000001), dict(withhold_copy=-1)],
    "orth": [dict(batch=-1), dict(batch=65536), dict(rows=0), dict(cols=32769), dict(dtype=3), dict(out_dtype=2), dict(steps=0),
             dict(steps=33), dict(eps=-1.0), dict(eps=float("nan")), dict(x=P + 2), dict(out=P + 1), dict(workspace=P + 64),
             dict(workspace_bytes=100), dict(wait_limit_us=10000001), dict(withhold_copy=2),
             dict(coefficients=(ctypes.c_float * 6)(1, 2, float("nan"), 0, 0, 0)), dict(coefficients=(ctypes.c_float * 6)(1, 2000, 0, 0, 0, 0)),
             dict(batch=65535, rows=32768, cols=32768, workspace_bytes=1 << 62)],
}


@pytest.mark.parametrize("name", list(SPECS))
def test_refusals(lib, name):
    assert getattr(lib, SPECS[name][1].__name__)(None, None) == mp.MHC_ERR_NULLPTR
    for kw in BAD[name]:
        assert _call(name, **kw) == mp.MHC_ERR_PARAM_INVALID, kw
        assert mp.last_error()
    outs, ins = _sizes(name)
    optional = {"bias"} | ({"gate_up"} if name == "experts" else set())
    for k in list(outs) + list(ins):
        if k not in optional:
            assert _call(name, **{k: None}) == mp.MHC_ERR_NULLPTR, k
    if name == "orth":
        assert _call(name, coefficients=None) == mp.MHC_ERR_NULLPTR


@pytest.mark.parametrize("name", ["route", "route_backward", "experts", "orth"])
def test_nothing_to_do(lib, name):
    outs, ins = _sizes(name)
    nothing = {k: None for k in list(outs) + list(ins)}
    assert _call(name, **nothing, **({"batch": 0} if name == "orth" else {"T": 0})) == mp.MHC_OK


@pytest.mark.parametrize("name", list(SPECS))
def test_overlaps_are_refused(lib, name):
    outs, ins = _sizes(name)
    size = {**outs, **ins}
    at = {k: P + i * STEP for i, k in enumerate(size)}
    for a, b in list(itertools.product(outs, ins)) + list(itertools.permutations(outs, 2)):
        for move in ({b: at[a]}, {b: at[a] + (size[a] - 1) // 256 * 256}, {a: at[b] + (size[b] - 1) // 256 * 256}):
            assert _call(name, **move) == mp.MHC_ERR_PARAM_INVALID, (a, b)
            assert "overlaps" in mp.last_error(), (a, b, mp.last_error())
    if not torch.cuda.is_available():
        assert _call(name) == mp.MHC_ERR_RUNTIME          # nothing else is wrong with the call


def test_plan_sizes_and_refusals(lib):
    assert mp.mhc_expert_plan_rows(0, 1, 8) == (mp.MHC_OK, 0)
    assert mp.mhc_expert_plan_rows(10, 2, 8) == (mp.MHC_OK, 20 + 8 * 15)
    assert mp.mhc_expert_plan_rows(2, 2, 8) == (mp.MHC_OK, 4 + 4 * 15)
    st, n = mp.mhc_expert_plan_size(10, 2, 8)
    assert st == mp.MHC_OK and n % 256 == 0
    for bad in ((-1, 1, 8), (1, 0, 8), (1, 9, 8), (1, 1, 0), (1, 1, 1025), (1 << 20, 8, 8), (1, 33, 64)):
        assert mp.mhc_expert_plan_size(*bad)[0] == mp.mhc_expert_plan_rows(*bad)[0] == mp.MHC_ERR_PARAM_INVALID
    assert lib.mhc_expert_plan_size(1, 1, 1, None) == lib.mhc_expert_plan_rows(1, 1, 1, None) == mp.MHC_ERR_NULLPTR
    run = mp.mhc_expert_plan_run
    assert run(10, 2, 8, 0, P, n) == run(10, 2, 8, P, 0, n) == run(0, 2, 8, 0, 0, n) == mp.MHC_ERR_NULLPTR
    for bad in ((10, 2, 8, P + 2, 2 * P, n), (10, 2, 8, P, 2 * P + 128, n), (10, 2, 8, P, 2 * P, n - 1), (10, 2, 8, P, P, n),
                (10, 2, 8, P + n - 64, P, n), (10, 9, 8, P, 2 * P, n)):
        assert run(*bad) == mp.MHC_ERR_PARAM_INVALID, bad


def test_workspace_sizes(lib):
    for f in (mp.mhc_experts_workspace_size, mp.mhc_experts_backward_workspace_size):
        assert f(0, 8, 2, 64, 128) == (mp.MHC_OK, 0)
        assert f(10, 8, 2, 64, 128)[0] == mp.MHC_OK
        for bad in ((-1, 8, 2, 64, 128), (1, 0, 1, 64, 128), (1, 8, 9, 64, 128), (1, 8, 2, 60, 128), (1, 8, 2, 64, 16392)):
            assert f(*bad)[0] == mp.MHC_ERR_PARAM_INVALID
    assert mp.mhc_orth_workspace_size(0, 4, 4) == (mp.MHC_OK, 0)
    for bad in ((-1, 4, 4), (1, 0, 4), (1, 4, 0), (1, 32769, 4)):
        assert mp.mhc_orth_workspace_size(*bad)[0] == mp.MHC_ERR_PARAM_INVALID


def test_torch_side_refusals(lib):
    """Types, shapes and host tensors are refused before the library is called."""
    t = torch.zeros
    l, i32, f32 = t(4, 8), torch.int32, torch.float32
    e, w = t(4, 2, dtype=i32), t(4, 2)
    plan = mp.ExpertPlan(t(16, dtype=torch.uint8), (4,), 2, 8, 100)
    x, wg, wd = t(4, 64, dtype=torch.bfloat16), t(8, 2, 64, 64, dtype=torch.bfloat16), t(8, 64, 64, dtype=torch.bfloat16)
    calls = [
        lambda: mp.route_experts(l, 2), lambda: mp.route_experts(l.double(), 2), lambda: mp.route_experts(l, 2, score="relu"),
        lambda: mp.route_experts(l, 2, group_score="sum"), lambda: mp.route_experts(l[0], 2), lambda: mp.route_experts(l, 0),
        lambda: mp.route_experts(l, 2, bias=t(7)), lambda: mp.route_experts_backward(w, l, e), lambda: mp.route_experts_backward(w, l, w),
        lambda: mp.expert_plan(e, 8), lambda: mp.expert_plan(w, 8), lambda: mp.expert_plan(e[0], 8),
        lambda: mp.experts_ffn(x, w, plan, wg, wd), lambda: mp.experts_ffn(x, w, (1, 2), wg, wd),
        lambda: mp.experts_ffn(x, w, plan, wg[:7], wd), lambda: mp.experts_ffn(x[:3], w, plan, wg, wd),
        lambda: mp.experts_ffn(x.float(), w, plan, wg, wd), lambda: mp.experts_ffn(x, w, plan, wg, wd, act="relu"),
        lambda: mp.experts_ffn(x, w, plan, wg, wd, save="8bit"), lambda: mp.orthogonalise(l), lambda: mp.orthogonalise(l[0]),
        lambda: mp.orthogonalise(e), lambda: mp.orthogonalise(l, steps=((1, 2),))]
    for c in calls:
        with pytest.raises(ValueError):
            c()


def test_streams_and_devices(lib, monkeypatch):
    """The stream that the library gets; tensors of another device never reach it."""
    import test_layer_calls as tl
    from mhc_hyper_connection_gb300 import _expert_ops, _layer_ops, _update_ops
    sizes = {(f, a): getattr(_expert_ops, f)(*a) for f, a in (("_plan_sizes", (3, 2, 8)), ("_scratch_bytes", (3, 8, 2, 64, 72, False)))}
    assert all(sizes.values()) and _update_ops._scratch_bytes(1, 64, 72)
    record = tl.Library()
    for m in (_expert_ops, _layer_ops, _update_ops):
        monkeypatch.setattr(m, "_lib", record)
    monkeypatch.setattr(_layer_ops, "_current_device", lambda: tl.CURRENT)
    monkeypatch.setattr(_layer_ops, "_current_raw_stream", lambda index: tl.STREAM + index)

    def calls(device):
        def t(*s, d=torch.bfloat16):
            v = tl.Tensor(s, d, device)
            v.dim = lambda: len(s)
            return v
        f, i, u = torch.float32, torch.int32, torch.uint8
        l, e, w, x = t(3, 8, d=f), t(3, 2, d=i), t(3, 2, d=f), t(3, 64)
        plan = mp.ExpertPlan(t(_expert_ops._plan_sizes(3, 2, 8)[0], d=u), (3,), 2, 8, 100)
        wg, wd, ws = t(8, 2, 72, 64), t(8, 64, 72), t(1 << 20, d=u)
        grads = {"grad_x": x, "grad_weights": w, "grad_w_gate_up": wg, "grad_w_down": wd}
        return [("mhc_route_run", lambda s: mp.route_experts(l, 2, out=mp.Routes(e, w), stream=s)),
                ("mhc_route_backward_run", lambda s: mp.route_experts_backward(w, l, e, grad_logits=l, stream=s)),
                ("mhc_expert_plan_run", lambda s: mp.expert_plan(e, 8, buffer=plan.buffer, stream=s)),
                ("mhc_experts_run", lambda s: mp.experts_ffn(x, w, plan, wg, wd, y=x, workspace=ws, stream=s)),
                ("mhc_experts_backward_run", lambda s: mp.experts_ffn_backward(x, x, w, plan, wg, wd, t(100, 2, 72), grads=grads,
                                                                               workspace=ws, stream=s)),
                ("mhc_orth_run", lambda s: mp.orthogonalise(t(64, 72), out=t(64, 72), workspace=ws, stream=s))]
    for k in range(6):
        name, call = calls("cuda:0")[k]
        for stream, want in ((None, tl.STREAM), (77, 77), (type("S", (), {"cuda_stream": 99})(), 99)):
            call(stream)
            assert record.calls[name][-1] == want
        record.calls.clear()
        for device in ("cpu", "cuda:1"):
            for stream in (None, 77):
                with pytest.raises(ValueError):
                    calls(device)[k][1](stream)
        assert not record.calls
