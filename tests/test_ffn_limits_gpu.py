"""The feed-forward block's device waits: what their limit counts, and how a
call ends whose waits give up."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _args(mp, x, w, wd, y, ws, **kw):
    a = mp.MhcFfnArgs()
    (a.T, a.D), a.F = x.shape, w.shape[1]
    a.x, a.w_gate_up, a.w_down, a.y = (t.data_ptr() for t in (x, w, wd, y))
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_limit_does_not_count_the_product_before(cuda_device):
    """Four tokens against 5 GB of weights: the second product's blocks start
    while the first product runs.  A block's own share of a product takes at
    most 136 us here; waits that also count the rest of the first product
    take 314.  A limit of 220 us is sound."""
    import mhc_hyper_connection_gb300 as mp
    T, D, F = 4, 20480, 40960
    gen = torch.Generator(device=cuda_device).manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=gen, device=cuda_device, dtype=torch.bfloat16)  # noqa: E731
    x, w, wd = rn(T, D), rn(2, F, D).mul_(D ** -0.5), rn(D, F).mul_(F ** -0.5)
    ws = mp.gated_ffn_workspace(T, D, F, cuda_device)
    want, _ = mp.gated_ffn(x, w, wd, workspace=ws)
    assert mp.gated_ffn_status(ws) == mp.MHC_OK
    for _ in range(5):
        y = torch.zeros_like(want)
        a = _args(mp, x, w, wd, y, ws, wait_limit_us=220)
        assert mp.mhc_ffn_run(a, torch.cuda.current_stream().cuda_stream) == mp.MHC_OK
        assert mp.gated_ffn_status(ws) == mp.MHC_OK
        assert torch.equal(y, want)


@pytest.mark.parametrize("T,D,F", [(1500, 2048, 2304), (300, 512, 8192), (700, 264, 1000), (300, 10040, 136)])
def test_copies_of_a_pair_are_counted_when_its_waits_give_up(cuda_device, T, D, F):
    """Copies withheld unevenly: of the first pair the odd CTA stops a stage
    before the even one, of the second the even one before the odd.  Every copy
    that was issued is still counted before the pair leaves: no wait for one
    runs out (100 ms each; the waits' limit is 20), and the next call on the
    same buffers is whole."""
    import mhc_hyper_connection_gb300 as mp
    gen = torch.Generator(device=cuda_device).manual_seed(T)
    rn = lambda *s, k=1.0: (torch.randn(s, generator=gen, device=cuda_device) * k).bfloat16()  # noqa: E731
    x, w, wd, gy = rn(T, D), rn(2, F, D, k=D ** -0.5), rn(D, F, k=F ** -0.5), rn(T, D)
    ws = mp.gated_ffn_workspace(T, D, F, cuda_device)
    wb = mp.gated_ffn_workspace(T, D, F, cuda_device, backward=True)
    y, kept = mp.gated_ffn(x, w, wd, save="16bit", workspace=ws)
    grads = mp.gated_ffn_backward(gy, x, w, wd, kept, workspace=wb)
    out, g2 = torch.empty_like(y), {k: torch.empty_like(v) for k, v in grads.items()}
    stream = torch.cuda.current_stream().cuda_stream

    def forward(withhold):
        return mp.mhc_ffn_run(_args(mp, x, w, wd, out, ws, wait_limit_us=20000, withhold_copy=withhold), stream)

    def backward(withhold):
        b = mp.MhcFfnBwdArgs()
        b.T, b.D, b.F = T, D, F
        b.grad_y, b.x, b.w_gate_up, b.w_down, b.gate_up = (t.data_ptr() for t in (gy, x, w, wd, kept))
        b.grad_x, b.grad_w_gate_up, b.grad_w_down = (g2[k].data_ptr() for k in ("grad_x", "grad_w_gate_up", "grad_w_down"))
        b.workspace, b.workspace_bytes, b.wait_limit_us, b.withhold_copy = wb.data_ptr(), wb.numel(), 20000, withhold
        return mp.mhc_ffn_backward_run(b, stream)
    for call, space in ((forward, ws), (backward, wb)):
        for withhold in (1, 0, 1, 0):
            t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            t0.record()
            assert call(withhold) == mp.MHC_OK
            t1.record()
            assert mp.gated_ffn_status(space) == (mp.MHC_ERR_RUNTIME if withhold else mp.MHC_OK)
            assert t0.elapsed_time(t1) < 90.0
    assert torch.equal(out, y) and all(torch.equal(g2[k], grads[k]) for k in grads)
