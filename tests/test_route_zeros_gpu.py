"""Logits that are zeros of either sign: equal numbers, so the lower expert comes first
(include/mhc_route.h).  The choice is compared exactly, the weights as in test_route_gpu."""
import numpy as np
import pytest
import torch

import expert_refs as ref
from test_route_gpu import DT, _check, _f64, built  # noqa: F401

pytestmark = pytest.mark.gpu


def _zeros(device, T, E, kind, seed, others):
    """Zeros of random sign; `others` of each row's logits are -0.5 or less, or -inf."""
    gen = torch.Generator(device=device).manual_seed(seed)
    at = lambda p: torch.rand((T, E), generator=gen, device=device) < p  # noqa: E731
    l = torch.where(at(0.5), 0.0, -0.0).to(device)
    l = torch.where(at(others), -0.5 - torch.rand((T, E), generator=gen, device=device), l)
    return l.masked_fill(at(others / 2), -np.inf).to(DT[kind])


def test_two_zeros(cuda_device):
    """The least case of each width: -0 before +0."""
    from mhc_hyper_connection_gb300 import route_experts
    for kind in DT:
        for E in (2, 40, 70, 130, 200, 256, 300, 700):
            l = torch.full((3, E), -1.0, device=cuda_device, dtype=DT[kind])
            l[:, 0], l[:, E - 1] = -0.0, 0.0
            for score in ("softmax", "sigmoid"):
                r = route_experts(l, 2, score=score)
                assert r.experts.tolist() == [[0, E - 1]] * 3, (kind, E, score)
                assert route_experts(l, 1, score=score).experts.tolist() == [[0]] * 3, (kind, E, score)


@pytest.mark.parametrize("kind", list(DT))
@pytest.mark.parametrize("E,groups,top", [(2, 1, 1), (31, 1, 1), (64, 8, 3), (72, 6, 2), (96, 3, 2), (160, 8, 3), (160, 5, 2), (192, 16, 5),
                                          (256, 8, 4), (384, 3, 2), (512, 16, 6), (1000, 10, 4), (1024, 32, 9)])
def test_zeros_of_either_sign(cuda_device, E, groups, top, kind):
    """Rows of zeros alone, and with other logits so that zeros of both signs stand at the
    border of what is chosen; with and without groups and bias (whose own zeros have signs)."""
    from mhc_hyper_connection_gb300 import route_experts
    for others in (0.0, 0.9):
        l = _zeros(cuda_device, 60, E, kind, E + groups, others)
        bias = torch.where(torch.arange(E, device=cuda_device) % 3 == 0, -0.0, 0.0)
        for k in {1, min(2, E), min(8, E // groups * top)}:
            for score in ("softmax", "sigmoid"):
                for g, t, mark in {(1, 1, "max"), (groups, top, "top2"), (groups, top, "max")}:
                    for b in (None, bias):
                        how = dict(score=score, groups=g, top_groups=t, group_score=mark, renormalise=True, scale=1.0)
                        _check(route_experts(l, k, bias=b, **how), l, b, k, **how)


def test_masked_by_multiplication(cuda_device):
    """Scores times 0 or 1, and small negative ones that fp16 rounds to -0: the gradient too
    follows the experts that the definition chooses."""
    from mhc_hyper_connection_gb300 import route_experts, route_experts_backward
    gen = torch.Generator(device=cuda_device).manual_seed(5)
    l = torch.randn((200, 64), generator=gen, device=cuda_device) * (torch.rand((200, 64), generator=gen, device=cuda_device) < 0.05)
    small = (torch.randn((200, 64), generator=gen, device=cuda_device) * 2.0 ** -30).half()
    d = torch.randn((200, 6), generator=gen, device=cuda_device)
    for x in (l, l.bfloat16(), small):
        for score in ("softmax", "sigmoid"):
            how = dict(score=score, renormalise=True, scale=1.0)
            r = route_experts(x, 6, **how)
            _check(r, x, None, 6, **how)
            e, _ = ref.route(_f64(x), 6, **how)
            want = route_experts_backward(d, x, torch.from_numpy(e).to(cuda_device), score=score)
            assert torch.equal(route_experts_backward(d, x, r.experts, score=score), want)
