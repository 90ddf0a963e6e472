"""Long sums of the feed-forward block: over a million tokens (weight gradients)
and over F = 131072 (y, grad_x).

The tensor core truncates as it adds, so a chain of K terms of one sign ends low
by a share that grows with K: at most s(K) = (K / 16 + 16) 2^-22, the bound of
the other feed-forward tests.  Chains are at most 32768 long here and joined in
fp32, whatever the depth.  With terms of one sign every output is low by about
the same share, while the roundings to fp16 (2^-11 each, of the operands and of
the result) go both ways and leave less than 2^-15 in a mean over 4096 outputs
and more.  So the mean relative error is at most s(32768) + 2^-15 = 5.2e-4; in
one chain it was 6.7e-3 at a million."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BOUND = (32768 / 16 + 16) * 2.0 ** -22 + 2.0 ** -15


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _positive(device, seed):
    gen = torch.Generator(device=device).manual_seed(seed)
    return lambda *s, k=1.0: ((torch.rand(s, generator=gen, device=device) + 0.5) * k).half()


def _gates(gy, wd, kept):
    """gg, gu and a of silu in 64 bits."""
    g, u = kept[:, 0].double(), kept[:, 1].double()
    s = torch.sigmoid(g)
    ga = gy.double() @ wd.double()
    return ga * u * s * (1 + g * (1 - s)), ga * g * s, g * s * u


def _mean_error(got, want):
    return float(((got.double() - want) / want).mean())


@pytest.mark.parametrize("form", ["16bit", "8bit"])
@pytest.mark.parametrize("T", [32769, 1048573])
def test_weight_gradients_over_many_tokens(cuda_device, T, form):
    from mhc_hyper_connection_gb300 import ckpt8_pack, ckpt8_restore, gated_ffn_backward, gated_ffn_status, gated_ffn_workspace
    D, F = 64, 72
    pos = _positive(cuda_device, 1)
    x, w, wd, gy, kept = pos(T, D), pos(2, F, D), pos(D, F, k=0.125), pos(T, D, k=2.0 ** -9), pos(T, 2, F)
    ws = gated_ffn_workspace(T, D, F, cuda_device, backward=True)
    if form == "8bit":
        given = ckpt8_pack(kept)
        kept = ckpt8_restore(given, dtype=torch.float16)
    else:
        given = kept
    got = gated_ffn_backward(gy, x, w, wd, given, workspace=ws)
    assert gated_ffn_status(ws) == 0
    want_gu = torch.zeros((2, F, D), dtype=torch.float64, device=cuda_device)
    want_down = torch.zeros((D, F), dtype=torch.float64, device=cuda_device)
    for t0 in range(0, T, 1 << 16):
        at = slice(t0, t0 + (1 << 16))
        gg, gu, a = _gates(gy[at], wd, kept[at])
        want_gu[0] += gg.t() @ x[at].double()
        want_gu[1] += gu.t() @ x[at].double()
        want_down += gy[at].double().t() @ a
    for h in (0, 1):
        assert abs(_mean_error(got["grad_w_gate_up"][h], want_gu[h])) <= BOUND
    assert abs(_mean_error(got["grad_w_down"], want_down)) <= BOUND
    again = gated_ffn_backward(gy, x, w, wd, given, workspace=ws)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_sums_over_a_wide_block(cuda_device):
    """Two whole rounds of tiles, which nothing but the depth cuts."""
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward, gated_ffn_status, gated_ffn_workspace
    T, D, F = 4864, 2048, 131072
    pos = _positive(cuda_device, 2)
    x, w, wd, gy = pos(T, D), pos(2, F, D, k=1 / D), pos(D, F, k=2.0 ** -11), pos(T, D, k=2.0 ** -4)
    at = torch.tensor([0, 1, 255, 256, 1000, 4095, 4862, 4863], device=cuda_device)
    ws = gated_ffn_workspace(T, D, F, cuda_device, backward=True)
    y, kept = gated_ffn(x, w, wd, save="16bit", workspace=ws)
    assert gated_ffn_status(ws) == 0
    g, u = (x[at].double() @ w[h].double().t() for h in (0, 1))
    want = (g * torch.sigmoid(g) * u) @ wd.double().t()
    # g and u are sums over D = 2048 themselves
    assert abs(_mean_error(y[at], want)) <= BOUND + 3 * (D / 16 + 16) * 2.0 ** -22
    got = gated_ffn_backward(gy, x, w, wd, kept, workspace=ws)
    assert gated_ffn_status(ws) == 0
    gg, gu, _ = _gates(gy[at], wd, kept[at])
    want = gg @ w[0].double() + gu @ w[1].double()
    assert abs(_mean_error(got["grad_x"][at], want)) <= BOUND + (D / 16 + 16) * 2.0 ** -22
