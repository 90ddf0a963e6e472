"""The feed-forward block beside memory that is not finite, in clusters of every
size with their status read, and its weight gradients past 32-bit offsets.  The
tolerances are those of the operator's other tests."""
import pytest
import torch

import test_ffn_gpu as tf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _within(t, fill, rows=384):
    """A copy of t in a larger buffer, `fill` before and after it."""
    room = torch.full((t.numel() + 2 * rows * 128,), fill, dtype=t.dtype, device=t.device)
    part = room[rows * 128:rows * 128 + t.numel()].view(t.shape)
    part.copy_(t)
    return part


@pytest.mark.parametrize("T,D,F", [(5, 72, 136), (100, 520, 264), (200, 72, 136), (300, 264, 1000)])
@pytest.mark.parametrize("fill", [float("inf"), float("nan")])
def test_memory_beside_the_tensors_is_not_multiplied_in(cuda_device, T, D, F, fill):
    """Infinities or NaN right before and after every input, and in the outputs
    and the workspace beforehand, change no bit."""
    from mhc_hyper_connection_gb300 import ckpt8_pack, gated_ffn, gated_ffn_backward, gated_ffn_workspace
    c = tf._case(cuda_device, T, D, F, "bf16", 2)
    want = {s: gated_ffn(c["x"], c["w"], c["wd"], save=s) for s in (None, "16bit", "8bit")}
    gu8 = ckpt8_pack(c["gu"])
    want_b = [gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], k) for k in (c["gu"], gu8)]
    d = {k: _within(v, fill) for k, v in c.items()}

    def space(backward):
        ws = gated_ffn_workspace(T, D, F, cuda_device, backward=backward)
        ws[256:].fill_(0xFF)                     # NaN in 16 and in 32 bits
        return ws
    for save, (y, kept) in want.items():
        y2, kept2 = gated_ffn(d["x"], d["w"], d["wd"], save=save, y=torch.full_like(y, fill), workspace=space(False))
        assert torch.equal(y2, y)
        if save == "16bit":
            assert torch.equal(kept2, kept)
        if save == "8bit":
            assert torch.equal(kept2.codes, kept.codes) and torch.equal(kept2.scales, kept.scales)
    for k, w in zip((d["gu"], gu8), want_b):
        grads = {n: torch.full_like(v, fill) for n, v in w.items()}
        got = gated_ffn_backward(d["gy"], d["x"], d["w"], d["wd"], k, grads=grads, workspace=space(True))
        assert all(torch.equal(got[n], w[n]) for n in w)


@pytest.mark.parametrize("T", [1, 16, 33, 64, 65, 80, 100, 128])
@pytest.mark.parametrize("D,F", [(512, 768), (768, 1280), (1024, 1280), (1280, 1536), (1792, 768), (2048, 1024)])
def test_clusters_report_no_wait(cuda_device, T, D, F):
    """Depths of 8 to 32 chunks: blocks in clusters of 2 to 8, forward and
    backward, whose error words stay clear."""
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward, gated_ffn_status, gated_ffn_workspace
    c = tf._case(cuda_device, T, D, F, "fp16", T + D)
    ws = gated_ffn_workspace(T, D, F, cuda_device)
    y, kept = gated_ffn(c["x"], c["w"], c["wd"], act="gelu", save="8bit", workspace=ws)
    assert gated_ffn_status(ws) == 0
    tf._check_forward(c, "fp16", "gelu", y, kept)
    wb = gated_ffn_workspace(T, D, F, cuda_device, backward=True)
    got = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, act="gelu", workspace=wb)
    assert gated_ffn_status(wb) == 0
    tf._check_backward(c, "fp16", "gelu", got, kept)


@pytest.mark.parametrize("save", ["16bit", "8bit"])
def test_weight_gradients_past_32_bit_offsets(cuda_device, save):
    """70001 tokens at F = 16384: [gg, gu] and the kept sums pass 2^31 elements.
    Each row of a weight gradient against its sum in 64 bits (a, gg, gu and the
    result are rounded to bf16: 2 2^-8 of a row's norm at most)."""
    from mhc_hyper_connection_gb300 import ckpt8_restore, gated_ffn, gated_ffn_backward
    T, D, F = 70001, 64, 16384
    c = tf._case(cuda_device, T, D, F, "bf16", 7)
    _, kept = gated_ffn(c["x"], c["w"], c["wd"], save=save)
    got = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept)
    sums = kept if save == "16bit" else ckpt8_restore(kept)
    want_gu = torch.zeros((2, F, D), dtype=torch.float64, device=cuda_device)
    want_down = torch.zeros((D, F), dtype=torch.float64, device=cuda_device)
    w, wd = c["w"].double(), c["wd"].double()
    for t0 in range(0, T, 4096):
        at = slice(t0, t0 + 4096)
        g, u = sums[at, 0].double(), sums[at, 1].double()
        s = torch.sigmoid(g)
        ga = c["gy"][at].double() @ wd
        gg, gu = ga * u * s * (1 + g * (1 - s)), ga * g * s
        want_gu[0] += gg.t() @ c["x"][at].double()
        want_gu[1] += gu.t() @ c["x"][at].double()
        want_down += c["gy"][at].double().t() @ (g * s * u)
        # grad_x of these tokens, each row by itself
        want_x = gg @ w[0] + gu @ w[1]
        off = (got["grad_x"][at].double() - want_x).norm(dim=1) / want_x.norm(dim=1)
        assert float(off.max()) <= 2.0 ** -7, (t0, float(off.max()))
    for k, want in (("grad_w_gate_up", want_gu), ("grad_w_down", want_down)):
        off = (got[k].double() - want).norm(dim=-1) / want.norm(dim=-1)
        assert float(off.max()) <= 2.0 ** -7, (k, float(off.max()))
