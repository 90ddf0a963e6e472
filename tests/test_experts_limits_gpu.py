"""Routed experts and updates at the ends of their ranges: the widest D and F, as many choices
as there may be, the most tokens, the largest batch of matrices; each against 64 bits."""
import pytest
import torch

import test_experts_gpu as te
import test_orth_gpu as to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


@pytest.mark.parametrize("kind,act", [("bf16", "gelu"), ("fp16", "silu")])
@pytest.mark.parametrize("T,E,k", [(9, 40, 32), (70, 64, 21), (33, 32, 32), (300, 40, 13)])
def test_many_choices(cuda_device, T, E, k, kind, act):
    c = te._case(cuda_device, T, E, k, 72, 64, kind, T + k)
    plan, y, kept = te._run(c, act)
    te._check_forward(c, kind, act, y, kept)
    te._check_backward(c, kind, act, plan, kept)


def _off(got, want):
    return float((got.double() - want).norm()) / float(want.norm())


def _check_norms(c, y, got):
    """Silu, as norms: y has its own rounding and that of a, at most 2^-8 each; a gradient at
    most eight in line between it and an input (kept sums, gate gradients, w a, itself), and
    sums over N rows that the tensor core cuts, off by N / 16 2^-23 of their terms' sum at most
    (32768 at a time: 2^-12)."""
    E, T = c["w"].shape[0], c["x"].shape[0]
    y64, gx = torch.zeros_like(c["x"], dtype=torch.float64), torch.zeros_like(c["x"], dtype=torch.float64)
    gw, gwg, gwd = torch.zeros_like(c["wt"], dtype=torch.float64), [], []
    for e in range(E):
        t, j = torch.nonzero(c["idx"] == e, as_tuple=True)
        x, gy, w, wd, wt = c["x"][t].double(), c["gy"][t].double(), c["w"][e].double(), c["wd"][e].double(), c["wt"][t, j].double()[:, None]
        g, u = x @ w[0].t(), x @ w[1].t()
        s = torch.sigmoid(g)
        a, ga = g * s * u, gy @ wd
        y64.index_add_(0, t, wt * (a @ wd.t()))
        gw[t, j] = (a * ga).sum(1)
        gg, gu = wt * ga * u * s * (1 + g * (1 - s)), wt * ga * g * s
        gx.index_add_(0, t, gg @ w[0] + gu @ w[1])
        gwg.append(torch.stack([gg.t() @ x, gu.t() @ x]))
        gwd.append(gy.t() @ (wt * a))
    assert _off(y, y64) <= 2.0 ** -7
    for n, v in (("grad_x", gx), ("grad_weights", gw), ("grad_w_gate_up", torch.stack(gwg)), ("grad_w_down", torch.stack(gwd))):
        assert _off(got[n], v) <= 2.0 ** -5, n


@pytest.mark.parametrize("T,E,k,D,F", [(5, 2, 2, 16384, 16384), (40, 3, 2, 16384, 16376), (1 << 20, 16, 4, 8, 8), (1 << 17, 1024, 32, 8, 16)])
def test_widest_and_most(cuda_device, T, E, k, D, F):
    from mhc_hyper_connection_gb300 import experts_ffn_backward
    c = te._case(cuda_device, T, E, k, D, F, "bf16", 1)
    plan, y, kept = te._run(c, "silu")
    got = experts_ffn_backward(c["gy"], c["x"], c["wt"], plan, c["w"], c["wd"], kept)
    _check_norms(c, y, got)


def test_largest_batch_of_matrices(cuda_device):
    """65535 of 2 x 8: some against 64 bits and as they are alone, all of them near an
    orthogonal matrix as the steps leave one."""
    from mhc_hyper_connection_gb300 import orthogonalise
    g = to._noise(cuda_device, (65535, 2, 8), torch.float32, 1)
    out = orthogonalise(g)
    for i in (0, 1, 30000, 65533, 65534):
        to._check(g[i], out[i])
        assert torch.equal(out[i], orthogonalise(g[i].contiguous()))
    want = to._exact(g)
    assert _off(out, want) <= 2.0 ** -7
