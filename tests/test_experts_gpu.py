"""Routed experts (include/mhc_experts.h) against their formulas in 64 bits, forward and
backward; bounds as expert_refs derives them."""
import numpy as np
import pytest
import torch

import expert_refs as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _f64(t):
    return t.double().cpu().numpy()


def _case(device, T, E, k, D, F, kind, seed, skew=1.0, dropped=0.1):
    gen = torch.Generator(device=device).manual_seed(seed)
    rn = lambda *shape, m=1.0: torch.randn(shape, generator=gen, device=device) * m  # noqa: E731
    l = rn(T, E) + skew * rn(E)
    idx = l.topk(k, -1).indices.int()
    idx[torch.rand((T, k), generator=gen, device=device) < dropped] = -1
    return dict(x=rn(T, D).to(DT[kind]), w=rn(E, 2, F, D, m=D ** -0.5).to(DT[kind]), wd=rn(E, D, F, m=F ** -0.5).to(DT[kind]),
                gy=rn(T, D, m=0.25).to(DT[kind]), idx=idx.contiguous(), wt=rn(T, k))


def _near(got, want, tol, what):
    got = _f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - want)):.3g}"


def _run(c, act, save="16bit"):
    from mhc_hyper_connection_gb300 import expert_plan, experts_ffn, experts_ffn_status, experts_ffn_workspace
    E, _, F, D = c["w"].shape
    T, k = c["idx"].shape
    plan = expert_plan(c["idx"], E)
    ws = experts_ffn_workspace(T, E, k, D, F, c["x"].device)
    y, kept = experts_ffn(c["x"], c["wt"], plan, c["w"], c["wd"], act=act, save=save, workspace=ws)
    assert experts_ffn_status(ws) == 0
    return plan, y, kept


def _slots(c, kept):
    """Kept sums by slot [T, k, 2, F], zeros where there is no expert."""
    idx = c["idx"].cpu().numpy()
    places = ref.plan(idx, c["w"].shape[0])[1]
    v = _f64(kept)[np.maximum(places, 0)]
    return np.where((places >= 0)[..., None, None], v, 0.0), places


def _check_forward(c, kind, act, y, kept=None):
    idx = c["idx"].cpu().numpy()
    want, tol, sums, esums = ref.experts(*(_f64(c[n]) for n in ("x", "wt")), idx, _f64(c["w"]), _f64(c["wd"]), act, kind)
    _near(y, want, tol, "y")
    if kept is not None:
        got, places = _slots(c, kept)
        bad = np.abs(got - sums) > ref.U[kind] * np.abs(sums) + 2 * esums + ref.TINY
        assert not bad[places >= 0].any()


def _check_backward(c, kind, act, plan, kept, workspace=None):
    from mhc_hyper_connection_gb300 import experts_ffn_backward, experts_ffn_status, experts_ffn_workspace
    E, _, F, D = c["w"].shape
    T, k = c["idx"].shape
    ws = experts_ffn_workspace(T, E, k, D, F, c["x"].device, backward=True)
    got = experts_ffn_backward(c["gy"], c["x"], c["wt"], plan, c["w"], c["wd"], kept, act=act, workspace=ws)
    assert experts_ffn_status(ws) == 0
    want = ref.experts_backward(_f64(c["gy"]), _f64(c["x"]), _f64(c["wt"]), c["idx"].cpu().numpy(), _f64(c["w"]), _f64(c["wd"]),
                                _slots(c, kept)[0], act, kind)
    for name, (v, tol) in want.items():
        _near(got[name], v, tol, name)
    return got


SHAPES = [(1, 1, 1, 8, 8), (1, 4, 2, 64, 128), (3, 8, 3, 72, 136), (17, 16, 4, 136, 72), (40, 3, 2, 264, 200), (64, 64, 6, 128, 64),
          (130, 5, 2, 520, 264), (300, 2, 1, 200, 392), (333, 12, 3, 264, 520), (700, 4, 2, 136, 264)]


@pytest.mark.parametrize("kind,act", [("bf16", "silu"), ("fp16", "gelu")])
@pytest.mark.parametrize("T,E,k,D,F", SHAPES)
def test_forward(cuda_device, T, E, k, D, F, kind, act):
    c = _case(cuda_device, T, E, k, D, F, kind, T + D)
    for save in (None, "16bit"):
        _, y, kept = _run(c, act, save)
        _check_forward(c, kind, act, y, kept)


@pytest.mark.parametrize("kind,act", [("bf16", "gelu"), ("fp16", "silu")])
@pytest.mark.parametrize("T,E,k,D,F", SHAPES)
def test_backward(cuda_device, T, E, k, D, F, kind, act):
    c = _case(cuda_device, T, E, k, D, F, kind, T + F)
    plan, _, kept = _run(c, act)
    _check_backward(c, kind, act, plan, kept)
