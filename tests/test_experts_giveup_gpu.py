"""Device waits that give up in launches of more tiles than a pair's slots hold: the
scheduler then still has tiles to hand out, and its own wait gives up too."""
import pytest
import torch

import test_experts_gpu as te
from test_experts_large_gpu import _fwd, built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,D,F", [(2000, 8, 3, 16384, 136), (500, 64, 4, 8192, 64)])
def test_waits_that_give_up_with_tiles_left(cuda_device, T, E, k, D, F):
    """More than a thousand tiles in the launches whose copy is withheld (down, rows of
    grad_x), six or more of them a pair: the waits give up after 20 ms, no wait for what is
    still in flight runs out (100 ms each), and the next calls on the same buffers are whole."""
    import mhc_hyper_connection_gb300 as mp
    c = te._case(cuda_device, T, E, k, D, F, "bf16", T)
    plan = mp.expert_plan(c["idx"], E)
    tiles = int(plan.buffer.view(torch.int32)[2]) * D // 256
    assert tiles > 1000
    ws = mp.experts_ffn_workspace(T, E, k, D, F, cuda_device)
    wb = mp.experts_ffn_workspace(T, E, k, D, F, cuda_device, backward=True)
    y, kept = mp.experts_ffn(c["x"], c["wt"], plan, c["w"], c["wd"], save="16bit", workspace=ws)
    grads = mp.experts_ffn_backward(c["gy"], c["x"], c["wt"], plan, c["w"], c["wd"], kept, workspace=wb)
    y2, kept2, out = torch.zeros_like(y), torch.zeros_like(kept), {n: torch.zeros_like(v) for n, v in grads.items()}
    d = mp.MhcExpertsBwdArgs()
    d.T, d.D, d.E, d.k, d.F = T, D, E, k, F
    d.grad_y, d.x, d.weights, d.plan, d.w_gate_up, d.w_down, d.gate_up, d.workspace = (
        t.data_ptr() for t in (c["gy"], c["x"], c["wt"], plan.buffer, c["w"], c["wd"], kept, wb))
    for n, v in out.items():
        setattr(d, n, v.data_ptr())
    d.workspace_bytes = wb.numel()
    raw = torch.cuda.current_stream().cuda_stream
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        a.record()
        assert _fwd(mp, c, plan, y2, kept2, ws, wait_limit_us=20000, withhold_copy=1) == mp.MHC_OK
        b.record()
        assert mp.experts_ffn_status(ws) == mp.MHC_ERR_RUNTIME and "gave up" in mp.last_error()
        assert a.elapsed_time(b) < 95
        assert _fwd(mp, c, plan, y2, kept2, ws) == mp.MHC_OK
        assert mp.experts_ffn_status(ws) == mp.MHC_OK and torch.equal(y, y2)
        d.wait_limit_us, d.withhold_copy = 20000, 1
        a.record()
        assert mp.mhc_experts_backward_run(d, raw) == mp.MHC_OK
        b.record()
        assert mp.experts_ffn_status(wb) == mp.MHC_ERR_RUNTIME
        assert a.elapsed_time(b) < 95
        d.wait_limit_us = d.withhold_copy = 0
        assert mp.mhc_experts_backward_run(d, raw) == mp.MHC_OK
        assert mp.experts_ffn_status(wb) == mp.MHC_OK and all(torch.equal(out[n], grads[n]) for n in grads)
