"""Routed experts and updates beyond 32-bit offsets, sums over very many rows, and device
waits that give up."""
import numpy as np
import pytest
import torch

import expert_refs as ref
import test_experts_gpu as te

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def test_sums_over_very_many_rows(cuda_device):
    """An expert with 100000 rows, terms of one sign: its weight gradients are formed in
    parts of 32768 rows joined in fp32, each off by at most (32768 / 16) 2^-23 of itself
    (the tensor core truncates as it adds), 2.4e-4; three roundings to bf16 (gradients of
    gate and up or w a, grad_y exact, the result) come on top."""
    from mhc_hyper_connection_gb300 import expert_plan, experts_ffn, experts_ffn_backward
    T, E, D, F = 100000, 3, 64, 64
    gen = torch.Generator(device=cuda_device).manual_seed(1)
    pos = lambda *s: (0.5 + torch.rand(s, generator=gen, device=cuda_device)).bfloat16()  # noqa: E731
    x, w, wd, gy = pos(T, D), pos(E, 2, F, D) / 64, pos(E, D, F), pos(T, D)
    idx = torch.ones((T, 1), dtype=torch.int32, device=cuda_device)
    idx[:50] = 0
    idx[70000:70010] = 2
    wt = (0.5 + torch.rand((T, 1), generator=gen, device=cuda_device))
    plan = expert_plan(idx, E)
    y, kept = experts_ffn(x, wt, plan, w, wd, save="16bit")
    got = experts_ffn_backward(gy, x, wt, plan, w, wd, kept)
    for _ in range(2):
        again = experts_ffn_backward(gy, x, wt, plan, w, wd, kept)
        assert all(torch.equal(got[k], again[k]) for k in got)
    for e in range(E):
        t = torch.nonzero(idx[:, 0] == e)[:, 0]
        xe, we, wde, ge, wte = x[t].double(), w[e].double(), wd[e].double(), gy[t].double(), wt[t].double()
        g, u = xe @ we[0].t(), xe @ we[1].t()
        s = torch.sigmoid(g)
        a, ga = g * s * u, wte * (ge @ wde)
        want = {"grad_w_gate_up": torch.stack([(ga * u * s * (1 + g * (1 - s))).t() @ xe, (ga * g * s).t() @ xe]),
                "grad_w_down": ge.t() @ (wte * a)}
        for k, v in want.items():
            # kept sums, their gradient and the result are rounded once each
            assert ((got[k][e].double() - v).abs() <= (2.4e-4 + 3 * 2.0 ** -8) * v.abs()).all(), (e, k)
            assert float((got[k][e].double() - v).norm()) <= 2.0 ** -8 * float(v.norm()), (e, k)


def test_offsets_beyond_32_bits(cuda_device):
    """Kept sums of 2.6e9 elements and rows of 5.2e9 bytes, checked on tokens from both ends."""
    from mhc_hyper_connection_gb300 import expert_plan, experts_ffn, experts_ffn_backward
    T, E, k, D, F = 20000, 8, 8, 64, 8192
    c = te._case(cuda_device, T, E, k, D, F, "bf16", 3, dropped=0.0)
    plan = expert_plan(c["idx"], E)
    y, kept = experts_ffn(c["x"], c["wt"], plan, c["w"], c["wd"], save="16bit")
    assert kept.numel() > 1 << 31
    got = experts_ffn_backward(c["gy"], c["x"], c["wt"], plan, c["w"], c["wd"], kept)
    pick = torch.tensor([0, 1, 9999, 13000, 16384, 19998, 19999], device=cuda_device)
    d = {n: c[n][pick].contiguous() for n in ("x", "gy", "idx", "wt")}
    d.update(w=c["w"], wd=c["wd"])
    te._check_forward(d, "bf16", "silu", y[pick])
    places = ref.plan(c["idx"].cpu().numpy(), E)[1][pick.cpu().numpy()]
    sums = te._f64(kept[torch.as_tensor(places.reshape(-1), device=cuda_device)]).reshape(len(pick), k, 2, F)
    want = ref.experts_backward(te._f64(d["gy"]), te._f64(d["x"]), te._f64(d["wt"]), d["idx"].cpu().numpy(), te._f64(c["w"]),
                                te._f64(c["wd"]), sums, "silu", "bf16")
    te._near(got["grad_x"][pick], *want["grad_x"], "grad_x")
    te._near(got["grad_weights"][pick], *want["grad_weights"], "grad_weights")


def test_update_beyond_32_bits(cuda_device):
    """Ninety matrices of 8192 x 3000: 2.2e9 elements, the last one as it is alone."""
    from mhc_hyper_connection_gb300 import orthogonalise
    g = torch.empty((90, 8192, 3000), dtype=torch.bfloat16, device=cuda_device)
    for i in range(90):
        g[i].normal_()
    out = orthogonalise(g)
    for i in (0, 87, 88, 89):
        assert torch.equal(out[i], orthogonalise(g[i].contiguous()))


def _fwd(mp, c, plan, y, kept, ws, **kw):
    a = mp.MhcExpertsArgs()
    a.T, a.D = c["x"].shape
    a.E, _, a.F, _ = c["w"].shape
    a.k = c["idx"].shape[1]
    a.x, a.weights, a.plan, a.w_gate_up, a.w_down, a.y, a.gate_up, a.workspace = (
        t.data_ptr() for t in (c["x"], c["wt"], plan.buffer, c["w"], c["wd"], y, kept, ws))
    a.workspace_bytes = ws.numel()
    for k, v in kw.items():
        setattr(a, k, v)
    return mp.mhc_experts_run(a, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("T,E,k,D,F", [(900, 4, 2, 1024, 1152), (20, 30, 3, 2048, 512), (300, 3, 2, 136, 264)])
def test_waits_that_give_up(cuda_device, T, E, k, D, F):
    """A withheld copy: the waits on it give up after 20 ms, the status says so, no wait for a
    copy in flight runs out (100 ms each), and the next call on the same buffers is whole."""
    import mhc_hyper_connection_gb300 as mp
    c = te._case(cuda_device, T, E, k, D, F, "bf16", T)
    plan = mp.expert_plan(c["idx"], E)
    ws = mp.experts_ffn_workspace(T, E, k, D, F, cuda_device)
    wb = mp.experts_ffn_workspace(T, E, k, D, F, cuda_device, backward=True)
    y, kept = mp.experts_ffn(c["x"], c["wt"], plan, c["w"], c["wd"], save="16bit", workspace=ws)
    grads = mp.experts_ffn_backward(c["gy"], c["x"], c["wt"], plan, c["w"], c["wd"], kept, workspace=wb)
    y2, kept2 = torch.zeros_like(y), torch.zeros_like(kept)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(2):
        a.record()
        assert _fwd(mp, c, plan, y2, kept2, ws, wait_limit_us=20000, withhold_copy=1) == mp.MHC_OK
        b.record()
        assert mp.experts_ffn_status(ws) == mp.MHC_ERR_RUNTIME and "gave up" in mp.last_error()
        assert a.elapsed_time(b) < 95
        assert _fwd(mp, c, plan, y2, kept2, ws) == mp.MHC_OK
        assert mp.experts_ffn_status(ws) == mp.MHC_OK and torch.equal(y, y2)
    out = {n: torch.zeros_like(v) for n, v in grads.items()}
    d = mp.MhcExpertsBwdArgs()
    d.T, d.D = c["x"].shape
    d.E, d.k, d.F = E, k, F
    d.grad_y, d.x, d.weights, d.plan, d.w_gate_up, d.w_down, d.gate_up, d.workspace = (
        t.data_ptr() for t in (c["gy"], c["x"], c["wt"], plan.buffer, c["w"], c["wd"], kept, wb))
    for n, v in out.items():
        setattr(d, n, v.data_ptr())
    d.workspace_bytes, d.wait_limit_us, d.withhold_copy = wb.numel(), 20000, 1
    raw = torch.cuda.current_stream().cuda_stream
    a.record()
    assert mp.mhc_experts_backward_run(d, raw) == mp.MHC_OK
    b.record()
    assert mp.experts_ffn_status(wb) == mp.MHC_ERR_RUNTIME
    assert a.elapsed_time(b) < 95
    d.wait_limit_us = d.withhold_copy = 0
    assert mp.mhc_experts_backward_run(d, raw) == mp.MHC_OK
    assert mp.experts_ffn_status(wb) == mp.MHC_OK and all(torch.equal(out[n], grads[n]) for n in grads)


@pytest.mark.parametrize("m,n", [(700, 1100), (1100, 700), (100, 100)])
def test_update_whose_waits_give_up(cuda_device, m, n):
    import ctypes
    import mhc_hyper_connection_gb300 as mp
    g = torch.randn((m, n), generator=torch.Generator(device=cuda_device).manual_seed(1), device=cuda_device)
    ws = mp.orthogonalise_workspace(g.shape, cuda_device)
    want = mp.orthogonalise(g, workspace=ws)
    out = torch.zeros_like(want)
    co = (ctypes.c_float * 15)(*[v for s in mp.NEWTON_SCHULZ for v in s])
    a = mp.MhcOrthArgs(1, m, n, mp.MHC_DTYPE_FP32, mp.MHC_DTYPE_BF16, 5, 1e-7, co, g.data_ptr(), out.data_ptr(), ws.data_ptr(),
                       ws.numel(), 20000, 1)
    raw = torch.cuda.current_stream().cuda_stream
    s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(2):
        a.wait_limit_us, a.withhold_copy = 20000, 1
        s.record()
        assert mp.mhc_orth_run(a, raw) == mp.MHC_OK
        e.record()
        assert mp.orthogonalise_status(ws) == mp.MHC_ERR_RUNTIME
        assert s.elapsed_time(e) < 95
        a.wait_limit_us = a.withhold_copy = 0
        assert mp.mhc_orth_run(a, raw) == mp.MHC_OK
        assert mp.orthogonalise_status(ws) == mp.MHC_OK and torch.equal(out, want)
