"""Orthogonalised updates (include/mhc_orth.h) against the iteration in 64 bits.

Tolerance.  A step p(X) = a X + B X, B = b A + c A A, rounds X, A and B once each to fp16,
by u = 2^-11 of an entry at most and 2^-12 rms, and forms its products in fp32 (off by s(K)
as everywhere).  In the singular directions of X (values s_i) an error d of X becomes, entry
by entry, d_ij times a divided difference of p: (p(s_i) - p(s_j)) / (s_i - s_j) for its
symmetric part, (p(s_i) + p(s_j)) / (s_i + s_j) for the other; an error of A enters B as (b +
c (s_i^2 + s_j^2)) d_ij; an error of B enters X as d_ij s_j.  So in norm, step by step,
    e' = G e + v ( |X'| + |B| |s| + |A| |(b + c (s_i^2 + s_j^2)) s_j| )
with v = u and the largest factor of each kind: a bound that holds for every matrix.  On a
matrix with both sides from 64 up the roundings are many and independent: they spread over
all directions alike, so each factor is the rms one instead of the largest, v = 2^-12, and
the terms add as squares; this is granted a factor of 2.  One rounding of the result comes
on top (u at most, u / sqrt(3) rms); an entry of such a matrix is granted 8 times the
rms error (a sum of thousands of roundings: 8 sigma)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
STEPS = ((3.4445, -4.7750, 2.0315),) * 5


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _exact(g, steps=STEPS, eps=1e-7):
    x = g.double()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    if x.shape[-2] > x.shape[-1]:
        return _exact(g.mT, steps, eps).mT
    for a, b, c in steps:
        p = x @ x.mT
        x = a * x + (b * p + c * p @ p) @ x
    return x


def _bound(g, steps, eps=1e-7):
    """Bound of the result's error in norm, before its last rounding."""
    x = g.double()
    x = x / (x.square().sum().sqrt() + eps)
    if x.shape[0] > x.shape[1]:
        x = x.T
    many = x.shape[0] >= 64
    v = (2.0 ** -12 if many else 2.0 ** -11) + (x.shape[1] / 16 + 16) * 2.0 ** -22
    size = (lambda t: t.square().mean().sqrt()) if many else (lambda t: t.abs().max())
    add = (lambda *t: sum(q * q for q in t) ** 0.5) if many else (lambda *t: sum(t))
    e = v * x.norm()
    for a, b, c in steps:
        p = x @ x.T
        q = b * p + c * p @ p
        s = torch.linalg.eigvalsh(p.cpu()).clamp_min(0.0).sqrt().to(x.device)
        f = a * s + b * s ** 3 + c * s ** 5
        i, j, fi, fj = s[:, None], s[None], f[:, None], f[None]
        slope = (a + 3 * b * s ** 2 + 5 * c * s ** 4)[:, None].expand(len(s), len(s))
        close = (i - j).abs() < 1e-6
        minus = torch.where(close, slope, (fi - fj) / torch.where(close, 1.0, i - j))
        plus = (fi + fj) / (i + j).clamp_min(1e-300)
        grow = torch.cat([minus, plus]) if many else torch.maximum(minus.abs(), plus.abs())
        via_a = (b + c * (i ** 2 + j ** 2)) * j
        x = a * x + q @ x
        e = add(size(grow) * e, v * x.norm(), v * q.norm() * size(s), v * p.norm() * size(via_a))
    return float(e) * (2 if many else 1), many


def _check(g, out, steps=STEPS):
    want = _exact(g, steps)
    err = out.double() - want
    e, many = _bound(g, steps)
    u = U[out.dtype]
    tol = e + (u / 3 ** 0.5 if many else u) * float(want.norm()) + 2.0 ** -25
    assert float(err.norm()) <= tol
    if many:
        assert (err.abs() <= 8 * tol / want.numel() ** 0.5 + u * want.abs() + 2.0 ** -25).all()


def _noise(device, shape, kind, seed, scale=1.0):
    gen = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=device) * scale).to(kind)


SHAPES = [(1, 1), (1, 7), (5, 1), (2, 2), (3, 200), (64, 64), (65, 63), (127, 300), (259, 515), (515, 259), (256, 256), (257, 256),
          (300, 1000), (1000, 300), (768, 2051), (1031, 520)]


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n", SHAPES)
def test_single(cuda_device, m, n, kind):
    from mhc_hyper_connection_gb300 import orthogonalise, orthogonalise_status, orthogonalise_workspace
    g = _noise(cuda_device, (m, n), kind, m + n)
    ws = orthogonalise_workspace(g.shape, cuda_device)
    out = orthogonalise(g, workspace=ws)
    assert orthogonalise_status(ws) == 0 and out.dtype == torch.bfloat16
    _check(g, out)
    half = torch.empty(g.shape, dtype=torch.float16, device=cuda_device)
    _check(g, orthogonalise(g, out=half))


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n", [(1, 100), (100, 1), (2, 2500), (4, 1000), (1000, 4), (23, 3078), (3078, 23), (130, 6000)])
def test_few_rows(cuda_device, m, n, kind):
    """Rows that are nearly orthogonal to start with: A is nearly a multiple of 1, and what its
    and B's diagonals lost to fp16 would grow up to tenfold (3.9 x 1.4 x 1.6 over the last
    steps for singular values of 0.2).  These are carried beside, so what stays is random: five
    roundings of X, 2^-12 rms each, of which nearly all lies across X's rows and keeps its
    size, granted a factor of 2; the off-diagonals, 1 / sqrt(n) of that; the result's own, u /
    sqrt(3)."""
    from mhc_hyper_connection_gb300 import orthogonalise
    g = _noise(cuda_device, (m, n), torch.float32, 3 * m + n)
    want = _exact(g)
    out = orthogonalise(g, out=torch.empty(g.shape, dtype=kind, device=cuda_device)).double()
    tol = ((2 * 5 ** 0.5 * 2.0 ** -12) ** 2 + U[kind] ** 2 / 3) ** 0.5
    assert float((out - want).norm()) <= tol * float(want.norm())


@pytest.mark.parametrize("shape", [(520, 4100), (4100, 520), (3, 300, 5000), (2, 5001, 257), (1025, 9000), (70, 32768), (32768, 70)])
def test_deep(cuda_device, shape):
    """X X^T of few tiles is summed in parts of its depth: the bound of every shape, the same
    bits every time, nothing behind the workspace that was asked for."""
    from mhc_hyper_connection_gb300 import orthogonalise, orthogonalise_status, orthogonalise_workspace
    g = _noise(cuda_device, shape, torch.float32, sum(shape))
    n = orthogonalise_workspace(shape, cuda_device).numel()
    room = torch.full((n + 4096,), 0x7F, dtype=torch.uint8, device=cuda_device)
    room[:256] = 0
    out = orthogonalise(g, workspace=room[:n])
    assert orthogonalise_status(room[:n]) == 0 and bool((room[n:] == 0x7F).all())
    for x, y in zip(g.reshape(-1, *shape[-2:]), out.reshape(-1, *shape[-2:])):
        _check(x, y)
    assert torch.equal(out, orthogonalise(g, workspace=room[:n]))


@pytest.mark.parametrize("shape", [(3, 40, 72), (2, 2, 300, 264), (17, 264, 130), (5, 513, 770)])
def test_batches(cuda_device, shape):
    """Every matrix of a batch has its own norm, and gives the bits that it gives alone."""
    from mhc_hyper_connection_gb300 import orthogonalise
    g = _noise(cuda_device, shape, torch.float32, 1)
    g *= torch.logspace(-6, 6, g[..., 0, 0].numel(), device=cuda_device).reshape(*shape[:-2], 1, 1)
    out = orthogonalise(g, eps=0.0)
    flat, got = g.reshape(-1, *shape[-2:]), out.reshape(-1, *shape[-2:])
    for i in range(flat.shape[0]):
        _check(flat[i] * (1.0 / flat[i].abs().max()), got[i])
        if shape[-1] % 8 == 0:
            assert torch.equal(got[i], orthogonalise(flat[i].contiguous(), eps=0.0))


def test_magnitudes(cuda_device):
    """The norm neither overflows nor underflows; eps counts where the norm is as small; a
    zero matrix gives zeros, one that is not finite NaN, its neighbours untouched."""
    from mhc_hyper_connection_gb300 import orthogonalise
    g = _noise(cuda_device, (96, 160), torch.float32, 3)
    want = _exact(g)
    for k in (2.0 ** 120, 2.0 ** 60, 2.0 ** -60, 2.0 ** -120):
        out = orthogonalise(g * k, eps=0.0)
        assert (out.double() - want).abs().max() <= 2.0 ** -6
    tiny = (g * 2.0 ** -140)                                # subnormal: few bits of each entry are left
    _check(tiny.double() * 2.0 ** 140, orthogonalise(tiny, eps=0.0))
    small = g * (1e-7 / float(g.norm()))                    # norm = eps: X half as large
    assert (orthogonalise(small).double() - _exact(small)).abs().max() <= 2.0 ** -7
    b = torch.stack([g, torch.zeros_like(g), g, g])
    b[2, 5, 7] = float("nan")
    b[3, 50, 0] = float("inf")
    out = orthogonalise(b)
    assert torch.equal(out[0], orthogonalise(g)) and (out[1] == 0).all() and out[2:].isnan().all()
    assert (orthogonalise(torch.zeros((8, 8), device=cuda_device), eps=0.0) == 0).all()


def test_other_steps(cuda_device):
    """Steps of other coefficients, none with a fifth power too; after many steps of 1.5 x -
    0.5 x^3 the result is orthogonal."""
    from mhc_hyper_connection_gb300 import orthogonalise
    q, _ = torch.linalg.qr(_noise(cuda_device, (200, 200), torch.float32, 4))
    s = torch.linspace(0.3, 1.0, 96, device=cuda_device)
    g = (q[:96] * s[:, None]) @ torch.linalg.qr(_noise(cuda_device, (200, 200), torch.float32, 5))[0]
    cubic = ((1.5, -0.5, 0.0),) * 24
    out = orthogonalise(g, steps=cubic)
    assert (out.double() @ out.double().mT - torch.eye(96, device=cuda_device)).abs().max() <= 2.0 ** -6
    quintic = ((15 / 8, -10 / 8, 3 / 8),) * 3
    _check(g, orthogonalise(g, steps=quintic), quintic)
    _check(g, orthogonalise(g, steps=((3.4445, -4.775, 2.0315), (2.0, -1.5, 0.5))), ((3.4445, -4.775, 2.0315), (2.0, -1.5, 0.5)))


def test_strong_directions(cuda_device):
    """A few directions ten times as strong as the rest."""
    from mhc_hyper_connection_gb300 import orthogonalise
    m, n = 384, 640
    g = _noise(cuda_device, (m, n), torch.float32, 6)
    g = g + _noise(cuda_device, (m, 4), torch.float32, 7) @ _noise(cuda_device, (4, n), torch.float32, 8) * 0.5
    _check(g, orthogonalise(g))


def test_streams_graph_and_repeats(cuda_device):
    from mhc_hyper_connection_gb300 import orthogonalise, orthogonalise_workspace
    g = _noise(cuda_device, (4, 300, 520), torch.bfloat16, 9)
    want = orthogonalise(g)
    for _ in range(5):
        assert torch.equal(orthogonalise(g), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = orthogonalise(g, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    ws, out = orthogonalise_workspace(g.shape, cuda_device), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orthogonalise(g, out=out, workspace=ws)
    other = _noise(cuda_device, (4, 300, 520), torch.bfloat16, 10)
    for src in (other, g):
        g2 = src.clone()
        g.copy_(g2)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, orthogonalise(g))
