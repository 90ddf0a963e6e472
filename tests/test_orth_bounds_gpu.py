"""Updates of unusual magnitudes and steps, within the bound that test_orth_gpu derives."""
import pytest
import torch

import test_orth_gpu as to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


@pytest.mark.parametrize("m,n", [(96, 160), (300, 70), (5, 1000)])
def test_magnitudes(cuda_device, m, n):
    """Times a power of two the exact result is the same.  Where the norm is eps X is half as
    large."""
    from mhc_hyper_connection_gb300 import orthogonalise
    g = to._noise(cuda_device, (m, n), torch.float32, m + n)
    g[0, 0] = 1.0
    for k in (2.0 ** 120, 2.0 ** 60, 1.0, 2.0 ** -60, 2.0 ** -115):
        to._check(g, orthogonalise(g * k, eps=0.0))
    small = g * (1e-7 / float(g.norm()))
    want = to._exact(small)
    err = orthogonalise(small).double() - want
    e, many = to._bound(small, to.STEPS)
    u = to.U[torch.bfloat16]
    assert float(err.norm()) <= e + (u / 3 ** 0.5 if many else u) * float(want.norm()) + 2.0 ** -25


def test_many_steps(cuda_device):
    from mhc_hyper_connection_gb300 import orthogonalise
    q, _ = torch.linalg.qr(to._noise(cuda_device, (200, 200), torch.float32, 4))
    s = torch.linspace(0.3, 1.0, 96, device=cuda_device)
    g = (q[:96] * s[:, None]) @ torch.linalg.qr(to._noise(cuda_device, (200, 200), torch.float32, 5))[0]
    for steps in (((1.5, -0.5, 0.0),) * 24, ((1.5, -0.5, 0.0),) * 32, ((15 / 8, -10 / 8, 3 / 8),) * 8, ((3.4445, -4.775, 2.0315),)):
        to._check(g, orthogonalise(g, steps=steps), steps)
