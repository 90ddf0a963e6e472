"""The layer operators on tensors of more than 2^31 (checkpoints: 2^32)
elements, checked on rows from both ends and around the 32-bit offsets.  The
tolerances are those of the operators' own tests."""
import numpy as np
import pytest
import torch

import layer_refs as ref
import test_ffn_gpu as tf
import test_post_bwd_gpu as tp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _rows(T, per_row, count=6):
    """Row numbers at the ends and on both sides of 2^31 and 2^32 elements."""
    picks = {0, 1, T - 2, T - 1}
    for edge in (1 << 31, 1 << 32):
        r = edge // per_row
        picks.update(v for v in (r - 1, r, r + 1) if 0 <= v < T)
    return sorted(picks)


def test_checkpoint_beyond_32_bits(cuda_device):
    from mhc_hyper_connection_gb300 import Ckpt8, ckpt8_pack, ckpt8_restore
    for D in (4096, 4104):                       # blocks that fill the row, and a last one of eight columns
        T = (1 << 32) // D + 37
        x = torch.empty((T, D), dtype=torch.bfloat16, device=cuda_device)
        for t0 in range(0, T, 1 << 18):
            x[t0:t0 + (1 << 18)].normal_()
        ck = ckpt8_pack(x)
        back = ckpt8_restore(ck)
        rows = torch.as_tensor(_rows(T, D), device=cuda_device)
        small = ckpt8_pack(x[rows].contiguous())
        assert torch.equal(ck.codes[rows], small.codes) and torch.equal(ck.scales[rows], small.scales)
        assert torch.equal(back[rows], ckpt8_restore(Ckpt8(small.codes, small.scales)))
        del x, ck, back


def test_post_backward_and_post_ckpt_beyond_32_bits(cuda_device):
    from mhc_hyper_connection_gb300 import ckpt8_pack, hc_post, hc_post_backward, hc_post_ckpt
    n, D = 8, 4096
    T = (1 << 31) // (n * D) + 1003
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=gen, device=cuda_device, dtype=torch.bfloat16)  # noqa: E731
    x, res, g = rn(T, D), rn(T, n, D), rn(T, n, D)
    post = torch.rand((T, n), generator=gen, device=cuda_device)
    comb = torch.rand((T, n, n), generator=gen, device=cuda_device)
    rows = _rows(T, n * D)
    at = torch.as_tensor(rows, device=cuda_device)
    out, ck = hc_post_ckpt(x, res, post, comb)
    small = hc_post(x[at].contiguous(), res[at].contiguous(), post[at].contiguous(), comb[at].contiguous())
    assert torch.equal(out[at], small)
    two = ckpt8_pack(small)
    assert torch.equal(ck.codes[at], two.codes) and torch.equal(ck.scales[at], two.scales)
    from mhc_synth import make_post_case
    case = make_post_case(device=cuda_device, T=1, n=n, D=8)
    case.T, case.D, case.x, case.residual, case.post, case.comb = T, D, x, res, post, comb
    tp._check(case, g, hc_post_backward(g, x, res, post, comb), tokens=rows)
    got = hc_post_backward(g, x, ck, post, comb)
    sub = [t[at] for t in ck]
    want, mag = ref.post_backward(tp._f64(g[at]), tp._f64(x[at]), ref.restore(*(t.cpu().numpy() for t in sub)),
                                  tp._f64(post[at]), tp._f64(comb[at]))
    d = np.abs(tp._f64(got["grad_comb"][at]) - want["grad_comb"])
    assert (d <= (D / 32 + 24) * 2.0 ** -23 * mag["grad_comb"]).all()


def test_ffn_beyond_32_bits(cuda_device):
    """70001 tokens at F = 16384: the kept sums and [gg, gu] pass 2^31 elements."""
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward
    T, D, F = 70001, 64, 16384
    c = tf._case(cuda_device, T, D, F, "bf16", 6)
    rows = _rows(T, 2 * F)
    at = torch.as_tensor(rows, device=cuda_device)
    sub = dict(c, x=c["x"][at], gy=c["gy"][at])
    for save in ("16bit", "8bit"):
        y, kept = gated_ffn(c["x"], c["w"], c["wd"], save=save)
        part = kept[at] if save == "16bit" else type(kept)(kept.codes[at], kept.scales[at])
        tf._check_forward(sub, "bf16", "silu", y[at], part)
        got = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept)
        # grad_x of those rows: from their own call, which sums in the same order
        own = gated_ffn_backward(sub["gy"].contiguous(), sub["x"].contiguous(), c["w"], c["wd"],
                                 part if save == "8bit" else part.contiguous())
        tf._check_backward(sub, "bf16", "silu", own, part)
        assert float((got["grad_x"][at].double() - own["grad_x"].double()).norm()) <= 2.0 ** -7 * float(own["grad_x"].double().norm())
        # weight gradients: sums over all tokens against 64 bits, in pieces of tokens
        if save == "16bit":
            wd64, want = c["wd"].double(), torch.zeros((D, F), dtype=torch.float64, device=cuda_device)
            for t0 in range(0, T, 4096):
                g, u = kept[t0:t0 + 4096, 0].double(), kept[t0:t0 + 4096, 1].double()
                want += c["gy"][t0:t0 + 4096].double().t() @ (g * torch.sigmoid(g) * u)
            off = float((got["grad_w_down"].double() - want).norm() / want.norm())
            assert off <= 2.0 ** -7, off        # a and the result are rounded to bf16: 2 2^-8 at most
        del y, kept, got
