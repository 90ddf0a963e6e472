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
