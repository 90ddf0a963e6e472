"""The bytes that examples/train_layer.py states a layer keeps, against what its body returns."""
import pytest
import torch

from test_train_layer_gpu import example  # noqa: F401


def test_sums_of_experts_are_counted(example):  # noqa: F811
    """Every chosen row's two sums in 16 bits, whatever keep says of the streams."""
    for T, D, F, E, k in ((4096, 2048, 1408, 16, 2), (100, 256, 136, 6, 3), (1, 64, 64, 8, 8)):
        for keep in ("8bit", "16bit"):
            plain = example.kept_bytes(T, D, F, keep)
            streams = example.kept_bytes(T, D, 0, keep)
            assert plain - streams == pytest.approx(T * 2 * F * (129 / 128 if keep == "8bit" else 2))
            experts = example.kept_bytes(T, D, F, keep, E, k) - streams
            assert experts >= T * k * 2 * F * 2
            assert experts == example.kept_bytes(T, D, F, "16bit", E, k) - example.kept_bytes(T, D, 0, "16bit")


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(200, 6, 2), (3, 16, 4), (1500, 4, 3)])
def test_against_what_a_body_keeps(example, cuda_device, T, E, k):  # noqa: F811
    D, F = 256, 136
    y = torch.randn((T, D), generator=torch.Generator(device=cuda_device).manual_seed(1), device=cuda_device).bfloat16()
    size = lambda *ts: sum(t.numel() * t.element_size() for t in ts)  # noqa: E731
    for keep in ("8bit", "16bit"):
        z, (logits, routes, plan, sums) = example.ExpertLayer(D, F, cuda_device, 1, experts=E, choices=k).body(y, keep)
        got = size(logits, *routes, plan.buffer, sums)
        assert example.kept_bytes(T, D, F, keep, E, k) == pytest.approx(example.kept_bytes(T, D, 0, keep) + got)
