"""Checkpoints read back in another type than the one they were taken from."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def test_checkpoint_read_in_another_type(cuda_device):
    """A bf16 checkpoint read as fp16 is the cast of what it stands for; an fp16
    one is exact in both types."""
    from mhc_hyper_connection_gb300 import ckpt8_pack, ckpt8_restore
    gen = torch.Generator(device=cuda_device).manual_seed(1)
    x = torch.randn((40, 520), generator=gen, device=cuda_device)
    x = x * torch.exp2(torch.randint(-30, 30, (40, 520), generator=gen, device=cuda_device).float())
    ck = ckpt8_pack(x.bfloat16())
    half = ckpt8_restore(ck, dtype=torch.float16)
    assert torch.isinf(half).any() and torch.equal(half, ckpt8_restore(ck).half())
    ck = ckpt8_pack(x.clamp(-60000, 60000).half())
    assert torch.equal(ckpt8_restore(ck).double(), ckpt8_restore(ck, dtype=torch.float16).double())
