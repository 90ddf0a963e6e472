"""8-bit activation checkpoints (include/mhc_ckpt.h) against the 64-bit form
of their definition.  Everything here is exact: a code is the nearest value of
the grid, and a restored value is code 2^e without rounding, so codes, scales
and values have to be equal."""
import numpy as np
import pytest
import torch

import layer_refs as ref
from mhc_synth import make_post_case

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _check(x, kind):
    from mhc_hyper_connection_gb300 import ckpt8_pack, ckpt8_restore
    ck = ckpt8_pack(x)
    back = ckpt8_restore(ck, dtype=DT[kind])
    torch.cuda.synchronize()
    D = x.shape[-1]
    codes, scales = ref.pack(x.double().cpu().numpy().reshape(-1, D), kind)
    got_c = ck.codes.cpu().numpy().reshape(-1, D)
    assert np.array_equal(ck.scales.cpu().numpy().reshape(codes.shape[0], -1), scales)
    assert np.array_equal(got_c, codes)
    want = ref.restore(codes, scales)
    assert np.array_equal(back.double().cpu().numpy().reshape(-1, D), want, equal_nan=True)
    return ck, back


def _data(shape, kind, seed, device, spread=True):
    gen = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.randn(shape, generator=gen)
    if spread:      # magnitudes over many binades, per element
        x = x * torch.exp2(torch.randint(-9, 9, shape, generator=gen).float())
    return x.to(DT[kind]).to(device)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [8, 120, 128, 136, 256, 520, 1024, 2056])
def test_codes_and_values(cuda_device, kind, D):
    _check(_data((37, D), kind, D, cuda_device), kind)


@pytest.mark.parametrize("rows", [1, 2, 63, 64, 65, 513])
def test_ragged_rows(cuda_device, rows):
    _check(_data((rows, 128), "bf16", rows, cuda_device), "bf16")
    _check(_data((rows, 72), "fp16", rows, cuda_device), "fp16")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_every_finite_value(cuda_device, kind):
    """All 65536 bit patterns, in blocks of one binade and shuffled over blocks:
    infinities and NaN become NaN, extremes saturate inside the type's range."""
    bits = np.arange(65536, dtype=np.uint16)
    for order in (bits, np.random.RandomState(1).permutation(bits)):
        x = torch.from_numpy(order.view(np.int16).copy()).to(cuda_device).view(DT[kind]).reshape(512, 128)
        ck, back = _check(x, kind)
        fine = torch.isfinite(x)
        assert torch.equal(torch.isfinite(back), fine)
        assert not torch.isinf(back).any()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_block_exponent_edges(cuda_device, kind):
    """amax just at, below and above 448 2^e, zero blocks, blocks with nothing finite."""
    rows = []
    for base in (448.0, 447.0, 449.0, 450.0, 256.0, 1.0, 1.75, 1.7578125, 0.0, 6e-8, 65504.0):
        r = np.zeros(128)
        r[5], r[77] = base, -base / 3
        rows.append(r)
    for fill in (np.nan, np.inf, -np.inf):
        rows.append(np.full(128, fill))
        r = np.linspace(-2, 3, 128)
        r[::7] = fill
        rows.append(r)
    _check(torch.from_numpy(np.stack(rows)).to(cuda_device).to(DT[kind]), kind)


def test_restored_values_are_fixed_points(cuda_device):
    """Packing what a checkpoint stands for gives the same values again."""
    from mhc_hyper_connection_gb300 import ckpt8_pack, ckpt8_restore
    a = ckpt8_restore(ckpt8_pack(_data((64, 1000), "bf16", 3, cuda_device)))
    assert torch.equal(a, ckpt8_restore(ckpt8_pack(a)))


def test_layouts_streams_and_given_outputs(cuda_device):
    from mhc_hyper_connection_gb300 import Ckpt8, ckpt8_pack, ckpt8_restore
    x = _data((3, 5, 4, 264), "bf16", 9, cuda_device)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = Ckpt8(torch.empty((3, 5, 4, 264), dtype=torch.uint8, device=cuda_device),
                torch.empty((3, 5, 4, 3), dtype=torch.uint8, device=cuda_device))
    ck = ckpt8_pack(x, out=out, stream=s)
    assert ck is out
    y = torch.empty_like(x)
    ckpt8_restore(ck, out=y, stream=s)
    torch.cuda.synchronize()
    ck2, back = _check(x, "bf16")
    assert torch.equal(ck.codes, ck2.codes) and torch.equal(y, back)


def test_empty(cuda_device):
    from mhc_hyper_connection_gb300 import ckpt8_pack, ckpt8_restore
    ck = ckpt8_pack(torch.empty((0, 4, 64), dtype=torch.bfloat16, device=cuda_device))
    assert ck.codes.shape == (0, 4, 64) and ck.scales.shape == (0, 4, 1)
    assert ckpt8_restore(ck).shape == (0, 4, 64)


def test_refusals(cuda_device):
    from mhc_hyper_connection_gb300 import Ckpt8, MhcError, ckpt8_pack, ckpt8_restore
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=cuda_device)
    with pytest.raises(ValueError):
        ckpt8_pack(x.float())
    with pytest.raises(ValueError):
        ckpt8_pack(x.t())
    with pytest.raises(MhcError):
        ckpt8_pack(x[:, :60].contiguous())
    with pytest.raises(MhcError):                       # base not 16-byte aligned
        ckpt8_pack(torch.zeros(65, dtype=torch.bfloat16, device=cuda_device)[1:].reshape(1, 64))
    ck = ckpt8_pack(x)
    with pytest.raises(ValueError):
        ckpt8_restore(Ckpt8(ck.codes, ck.scales[:2]))
    with pytest.raises(ValueError):
        ckpt8_restore(ck, dtype=torch.float16, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        ckpt8_pack(x, out=Ckpt8(ck.codes[:, :32], ck.scales))


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("T,D", [(1, 8), (37, 136), (64, 256), (5, 2056)])
def test_post_ckpt_is_post_then_pack(cuda_device, n, T, D):
    from mhc_hyper_connection_gb300 import ckpt8_pack, hc_post, hc_post_ckpt
    case = make_post_case(device=cuda_device, T=T, n=n, D=D, seed=n * 31 + D)
    out, ck = hc_post_ckpt(case.x, case.residual, case.post, case.comb)
    want = hc_post(case.x, case.residual, case.post, case.comb)
    assert torch.equal(out, want)
    two = ckpt8_pack(want)
    assert torch.equal(ck.codes, two.codes) and torch.equal(ck.scales, two.scales)


def test_post_ckpt_large_and_nonfinite(cuda_device):
    from mhc_hyper_connection_gb300 import ckpt8_pack, hc_post, hc_post_ckpt
    case = make_post_case(device=cuda_device, T=3001, n=4, D=4104, seed=2)
    case.x[7, 100] = float("inf")
    case.residual[9, 2, 4103] = float("nan")
    case.post[11, 3] = float("nan")
    out, ck = hc_post_ckpt(case.x, case.residual, case.post, case.comb)
    want = hc_post(case.x, case.residual, case.post, case.comb)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    two = ckpt8_pack(want)
    assert torch.equal(ck.codes, two.codes) and torch.equal(ck.scales, two.scales)


def test_post_ckpt_refusals(cuda_device):
    from mhc_hyper_connection_gb300 import hc_post_ckpt
    case = make_post_case(device=cuda_device, T=4, n=4, D=64, seed=2)
    with pytest.raises(ValueError):
        hc_post_ckpt(case.x.half(), case.residual, case.post, case.comb)
    with pytest.raises(ValueError):
        hc_post_ckpt(case.x, case.residual, case.post, case.comb[:2])
