"""The rows of outputs and of grad_x as they wait for a token's sum (include/mhc_experts.h):
16 significant bits rounded to nearest, fp32's range.

The data make everything before such a row exact: x is one-hot, the gate 64 (whose
sigmoid is 1 in fp32), so a and gu are powers of two, and a row's values are sums of two or
three 16-bit numbers with at most 20 significant bits.  A token takes one such row and, with
weight -1, another expert's whose values are the first ones' nearest of 16 bits: what
is left is the difference, off by half a step of 16 bits (2^-16 of the power of two below the
value) and one rounding of the result, which is small itself."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
BITS = {"bf16": 8, "fp16": 11}


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _pieces(v, bits, n):
    """v (fp64) as n numbers of so many bits, largest first; their sum is v."""
    out = []
    for _ in range(n):
        m, e = np.frexp(v)
        p = np.ldexp(np.trunc(m * 2.0 ** bits), e - bits)
        out.append(p)
        v = v - p
    assert (v == 0).all()
    return out


def _values(n, seed):
    """(v, its nearest of 16 bits): v has 20 significant bits, both signs, several powers of two."""
    rng = np.random.default_rng(seed)
    m = rng.integers(1 << 19, 1 << 20, n) | 1                     # odd: never midway between two of 16 bits
    m = np.where(m % 16 == 8, m + 1, m)
    v = np.ldexp(m.astype(np.float64), -20) * 2.0 ** rng.integers(0, 3, n) * rng.choice([-1.0, 1.0], n)
    f, e = np.frexp(v)
    return v, np.ldexp(np.rint(f * 2.0 ** 16), e - 16)


def _tensor(a, kind, device):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(device).to(DT[kind])
    assert (t.double().cpu().numpy() == a).all()                  # the data are of the type
    return t


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D", [(1, 256), (70, 520), (300, 2048)])
def test_output_rows(cuda_device, T, D, kind):
    from mhc_hyper_connection_gb300 import expert_plan, experts_ffn
    F = 8
    v, near = _values(D, D)
    w, wd = np.zeros((2, 2, F, D)), np.zeros((2, D, F))
    w[:, 0, :, 0], w[:, 1, :, 0] = 64.0, 2.0 ** -6                # a = 1
    for e, x in ((0, v), (1, near)):
        for f, p in enumerate(_pieces(x, BITS[kind], 3)):
            wd[e, :, f] = p
    x = np.zeros((T, D))
    x[:, 0] = 1.0
    idx = torch.tensor([[0, 1]], dtype=torch.int32, device=cuda_device).expand(T, 2).contiguous()
    wt = torch.tensor([[1.0, -1.0]], device=cuda_device).expand(T, 2).contiguous()
    y, _ = experts_ffn(_tensor(x, kind, cuda_device), wt, expert_plan(idx, 2), _tensor(w, kind, cuda_device), _tensor(wd, kind, cuda_device))
    _check(y, v, near, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D", [(1, 256), (70, 520), (300, 2048)])
def test_rows_of_grad_x(cuda_device, T, D, kind):
    """up = 0, so gg = 0 and gu = w ga 64 with ga = 2^-6: a row is the sum of Wu's."""
    from mhc_hyper_connection_gb300 import expert_plan, experts_ffn, experts_ffn_backward
    F = 8
    v, near = _values(D, D + 1)
    v[0] = near[0] = 0.0
    w, wd = np.zeros((2, 2, F, D)), np.zeros((2, D, F))
    w[:, 0, :, 0] = 64.0
    wd[:, 0, :] = 2.0 ** -6
    for e, x in ((0, v), (1, near)):
        for f, p in enumerate(_pieces(x, BITS[kind], 3)):
            w[e, 1, f] = p
    x, gy = np.zeros((T, D)), np.zeros((T, D))
    x[:, 0] = gy[:, 0] = 1.0
    idx = torch.tensor([[0, 1]], dtype=torch.int32, device=cuda_device).expand(T, 2).contiguous()
    wt = torch.tensor([[1.0, -1.0]], device=cuda_device).expand(T, 2).contiguous()
    x, gy, w, wd = (_tensor(a, kind, cuda_device) for a in (x, gy, w, wd))
    plan = expert_plan(idx, 2)
    y, kept = experts_ffn(x, wt, plan, w, wd, save="16bit")
    assert (y == 0).all()
    _check(experts_ffn_backward(gy, x, wt, plan, w, wd, kept)["grad_x"], v, near, kind)


def _check(got, v, near, kind):
    got = got.double().cpu().numpy()
    want = v - near
    half = np.ldexp(1.0, np.frexp(v)[1] - 1) * 2.0 ** -16 * (v != 0)      # half a step of 16 bits
    # the result is a difference of rows of 16 bits: at most a step, rounded once (fp16: 2^-25 at least)
    tol = half + 2.0 ** -BITS[kind] * (np.abs(want) + half) + (2.0 ** -25 if kind == "fp16" else 0.0)
    bad = np.abs(got - want) > tol
    assert not bad.any(), (bad.sum(), bad.size, np.abs(got - want).max())


def test_rows_keep_the_range_of_fp32(cuda_device):
    """Rows beyond fp16's range whose weighted sum is inside it; infinities, NaN and the largest
    finite sums stay what they are."""
    from mhc_hyper_connection_gb300 import expert_plan, experts_ffn
    D, F = 64, 8
    for kind in ("fp16", "bf16"):
        w, wd = np.zeros((2, 2, F, D)), np.zeros((2, D, F))
        w[:, 0, :, 0], w[:, 1, :, 0] = 64.0, 2.0                  # a = 128
        wd[0, :, 0], wd[1, :, 0] = 1024.0, 1008.0
        wd[0, 1, 0], wd[0, 2, 0] = np.inf, np.nan
        w, wd = (torch.from_numpy(a).to(cuda_device).to(DT[kind]) for a in (w, wd))
        x = torch.zeros((40, D), device=cuda_device, dtype=DT[kind])
        x[:, 0] = 1
        idx = torch.tensor([[0, 1]], dtype=torch.int32, device=cuda_device).expand(40, 2).contiguous()
        wt = torch.tensor([[1.0, -1.0]], device=cuda_device).expand(40, 2).contiguous()
        y = experts_ffn(x, wt, expert_plan(idx, 2), w, wd)[0].float()
        assert (y[:, 1] == np.inf).all() and y[:, 2].isnan().all() and (y[:, 3:] == 2048.0).all()
    # a row of 2^128 - 2^112 (sixteen ones, the largest of 16 bits), and one step of fp32 less than 2^128
    w = torch.zeros((1, 2, F, D), device=cuda_device, dtype=torch.bfloat16)
    w[0, 0, :, 0], w[0, 1, :, 0] = 64.0, 2.0 ** -6
    wd = torch.zeros((1, D, F), device=cuda_device, dtype=torch.bfloat16)
    wd[0, :, 0] = (2.0 - 2.0 ** -7) * 2.0 ** 127
    wd[0, :, 1] = (2.0 - 2.0 ** -7) * 2.0 ** 119
    wd[0, ::2, 2] = (2.0 - 2.0 ** -7) * 2.0 ** 111
    x = torch.zeros((3, D), device=cuda_device, dtype=torch.bfloat16)
    x[:, 0] = 1
    wt = torch.full((3, 1), 2.0 ** -8, device=cuda_device)
    y = experts_ffn(x, wt, expert_plan(torch.zeros((3, 1), dtype=torch.int32, device=cuda_device), 1), w, wd)[0]
    assert (y.double() == 2.0 ** 120).all()
