"""Backward of the post-mapping (include/mhc_post_backward.h) against its
formulas in 64 bits and against differences of the forward.

Tolerances, from the arithmetic: grad_x and grad_residual are n products
added in fp32 and rounded once to bf16, so off by at most 2^-8 |ref| (half a
bf16 step, 2^-9, and the same again for a rounding that the fp32 error tips)
plus n 2^-23 times the sum of the terms' magnitudes.  grad_post and grad_comb
are fp32 dot products; a lane adds at most ceil(D / 256) vectors of eight
products one after another, then five joins over lanes and at most eight over
warps: (D / 32 + 24) 2^-23 times the sum of the magnitudes."""
import numpy as np
import pytest
import torch

import layer_refs as ref
from mhc_synth import make_post_case, sample_tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _case(device, T, n, D, seed):
    case = make_post_case(device=device, T=T, n=n, D=D, seed=seed)
    gen = torch.Generator(device=device).manual_seed(seed)
    g = (torch.randn((T, n, D), generator=gen, device=device) * 0.05).bfloat16()
    return case, g


def _f64(t):
    return t.double().cpu().numpy()


def _check(case, g, got, residual=None, tokens=None):
    sel = (lambda a: a) if tokens is None else (lambda a: a[torch.as_tensor(tokens, device=a.device)])
    res = _f64(sel(case.residual)) if residual is None else residual
    want, mag = ref.post_backward(_f64(sel(g)), _f64(sel(case.x)), res, _f64(sel(case.post)), _f64(sel(case.comb)))
    n, D = case.n, case.D
    for k in ("grad_x", "grad_residual", "grad_post", "grad_comb"):
        v = _f64(sel(got[k]))
        if k in ("grad_x", "grad_residual"):
            tol = 2.0 ** -8 * np.abs(want[k]) + n * 2.0 ** -23 * mag[k]
        else:
            tol = (D / 32 + 24) * 2.0 ** -23 * mag[k]
        bad = ~(np.abs(v - want[k]) <= tol + 1e-38)
        assert not bad.any(), f"{k}: {bad.sum()} outside, worst {np.abs(v - want[k]).max():.3g}"


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("T,D", [(1, 8), (3, 264), (37, 256), (9, 1032), (2, 16384)])
def test_shapes(cuda_device, n, T, D):
    from mhc_hyper_connection_gb300 import hc_post_backward
    case, g = _case(cuda_device, T, n, D, n * 7 + D)
    got = hc_post_backward(g, case.x, case.residual, case.post, case.comb)
    _check(case, g, got)


@pytest.mark.parametrize("n", [1, 3, 4, 8])
@pytest.mark.parametrize("T,D", [(1, 8), (33, 136), (5, 2056), (300, 512)])
def test_from_checkpoint(cuda_device, n, T, D):
    """The residual's values are those the codes stand for, exactly."""
    from mhc_hyper_connection_gb300 import ckpt8_pack, hc_post_backward
    case, g = _case(cuda_device, T, n, D, n * 5 + D)
    ck = ckpt8_pack(case.residual)
    got = hc_post_backward(g, case.x, ck, case.post, case.comb)
    res = ref.restore(ck.codes.cpu().numpy(), ck.scales.cpu().numpy())
    _check(case, g, got, residual=res)


@pytest.mark.parametrize("T", [200, 620, 1300, 2500, 5000])
def test_every_split(cuda_device, T):
    """Token counts on both sides of each step of the warps-per-token rule."""
    from mhc_hyper_connection_gb300 import hc_post_backward
    case, g = _case(cuda_device, T, 4, 2048, T)
    got = hc_post_backward(g, case.x, case.residual, case.post, case.comb)
    _check(case, g, got, tokens=sample_tokens(T, 64, seed=T))


def test_prefill_shape_sampled(cuda_device):
    from mhc_hyper_connection_gb300 import hc_post_backward
    T, n, D = 32768, 4, 7168
    gen = torch.Generator(device=cuda_device).manual_seed(4)
    rn = lambda *s: torch.randn(s, generator=gen, device=cuda_device, dtype=torch.bfloat16)  # noqa: E731
    case = make_post_case(device=cuda_device, T=4, n=n, D=8, seed=0)
    case.T, case.D, case.x, case.residual = T, D, rn(T, D), rn(T, n, D)
    case.post = torch.rand((T, n), generator=gen, device=cuda_device)
    case.comb = torch.rand((T, n, n), generator=gen, device=cuda_device)
    g = rn(T, n, D)
    got = hc_post_backward(g, case.x, case.residual, case.post, case.comb)
    _check(case, g, got, tokens=sample_tokens(T, 48, seed=3))


def test_against_differences(cuda_device):
    """Central differences of <g, post-mapping> in 64 bits.  The forward is
    linear in each input, so a difference is exact up to 64-bit rounding and
    only the tolerance of the formulas' test remains (here 2^-8 of the largest
    gradient, which covers it: every bound there is below that)."""
    from mhc_hyper_connection_gb300 import hc_post_backward
    case, g = _case(cuda_device, 3, 4, 40, 77)
    got = hc_post_backward(g, case.x, case.residual, case.post, case.comb)
    v = {"grad_x": _f64(case.x), "grad_residual": _f64(case.residual), "grad_post": _f64(case.post),
         "grad_comb": _f64(case.comb)}
    gg = _f64(g)

    def loss():
        return float((gg * ref.post(v["grad_x"], v["grad_residual"], v["grad_post"], v["grad_comb"])).sum())
    rng = np.random.RandomState(0)
    for k, a in v.items():
        flat, out = a.reshape(-1), _f64(got[k]).reshape(-1)
        for i in rng.choice(flat.size, min(12, flat.size), replace=False):
            keep = flat[i]
            flat[i] = keep + 0.5
            up = loss()
            flat[i] = keep - 0.5
            down = loss()
            flat[i] = keep
            assert abs((up - down) - out[i]) <= 2.0 ** -8 * np.abs(out).max(), (k, i)


def test_exact_where_the_mathematics_is(cuda_device):
    """Unit gates, identity mix: grad_residual is g, and zero g gives zeros."""
    from mhc_hyper_connection_gb300 import hc_post_backward
    case, g = _case(cuda_device, 50, 4, 1024, 5)
    case.post.zero_()
    case.post[:, 2] = 1
    case.comb.copy_(torch.eye(4, device=cuda_device).expand(50, 4, 4))
    got = hc_post_backward(g, case.x, case.residual, case.post, case.comb)
    assert torch.equal(got["grad_residual"], g) and torch.equal(got["grad_x"], g[:, 2])
    got = hc_post_backward(torch.zeros_like(g), case.x, case.residual, case.post, case.comb)
    assert all(not v.any() for v in got.values())


def test_nonfinite_stays_in_its_token(cuda_device):
    from mhc_hyper_connection_gb300 import hc_post_backward
    case, g = _case(cuda_device, 20, 4, 512, 6)
    clean = hc_post_backward(g, case.x, case.residual, case.post, case.comb)
    g2 = g.clone()
    g2[7, 1, 3] = float("nan")
    got = hc_post_backward(g2, case.x, case.residual, case.post, case.comb)
    keep = [t for t in range(20) if t != 7]
    for k in clean:
        assert torch.equal(got[k][keep], clean[k][keep])
    assert torch.isnan(got["grad_x"][7, 3]) and torch.isnan(got["grad_post"][7, 1])
    assert torch.isnan(got["grad_comb"][7, :, 1]).all() and not torch.isnan(got["grad_comb"][7, :, 0]).any()


def test_stream_bsnd_given_outputs_and_repeats(cuda_device):
    from mhc_hyper_connection_gb300 import hc_post_backward
    case, g = _case(cuda_device, 300, 6, 2048, 11)
    a = hc_post_backward(g, case.x, case.residual, case.post, case.comb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lead = lambda t: t.reshape((3, 100) + t.shape[1:])  # noqa: E731
    grads = {k: lead(torch.empty_like(v)) for k, v in a.items()}
    b = hc_post_backward(lead(g), lead(case.x), lead(case.residual), lead(case.post), lead(case.comb), grads=grads,
                         stream=s)
    torch.cuda.synchronize()
    assert b is grads
    for k in a:
        assert torch.equal(a[k].reshape(-1), b[k].reshape(-1))
    _check(case, g, a)


def test_empty(cuda_device):
    from mhc_hyper_connection_gb300 import hc_post_backward
    e = lambda *s, d=torch.bfloat16: torch.empty(s, dtype=d, device=cuda_device)  # noqa: E731
    got = hc_post_backward(e(0, 4, 64), e(0, 64), e(0, 4, 64), e(0, 4, d=torch.float32), e(0, 4, 4, d=torch.float32))
    assert got["grad_residual"].shape == (0, 4, 64)


def test_refusals(cuda_device):
    from mhc_hyper_connection_gb300 import ckpt8_pack, hc_post_backward
    case, g = _case(cuda_device, 4, 4, 64, 1)
    ok = (g, case.x, case.residual, case.post, case.comb)
    for k, bad in ((0, g.float()), (1, case.x[:, :32]), (2, case.residual.half()), (3, case.post.bfloat16()),
                   (4, case.comb[:, :2]), (2, ckpt8_pack(case.residual[:2].contiguous())), (2, case.residual.cpu())):
        args = list(ok)
        args[k] = bad
        with pytest.raises(ValueError):
            hc_post_backward(*args)
    with pytest.raises(ValueError):
        hc_post_backward(g.transpose(1, 2).contiguous().transpose(1, 2), *ok[1:])
