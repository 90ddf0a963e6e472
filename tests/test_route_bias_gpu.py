"""Choice of groups under biases of unlike sign (include/mhc_route.h: the order is that of the
exact keys).  A group's mark is then the small sum of two large keys, each rounded by more
than marks differ: fp32 cannot order them."""
import pytest
import torch

from test_route_gpu import _check, built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [1.0, 100.0, 1.0e4])
@pytest.mark.parametrize("E,groups,top", [(64, 8, 3), (256, 8, 4), (72, 6, 2), (160, 5, 2), (192, 16, 5), (512, 8, 4), (1000, 10, 4)])
def test_groups_of_keys_that_cancel(cuda_device, E, groups, top, size):
    """Of each group one expert is pushed up and one down by as much, differently from group to
    group: keys lie far apart and marks close together.  Also one up and all others down, alike."""
    from mhc_hyper_connection_gb300 import route_experts
    gen = torch.Generator(device=cuda_device).manual_seed(E + groups)
    l = torch.randn((300, E), generator=gen, device=cuda_device) * 0.05
    per = E // groups
    apart = torch.full((E,), -4.0 * size, device=cuda_device)
    by = size * (1.0 + torch.arange(groups, device=cuda_device) / groups)
    apart[::per], apart[1::per] = by, -by
    alike = torch.full((E,), -size, device=cuda_device)
    alike[::per] = size
    for bias, k in ((apart, top), (apart, 2 * top), (alike, 6)):
        for score in ("sigmoid", "softmax"):
            for mark in ("top2", "max"):
                how = dict(score=score, groups=groups, top_groups=top, group_score=mark, renormalise=True, scale=1.0)
                _check(route_experts(l, k, bias=bias, **how), l, bias, k, **how)


def test_groups_pushed_out(cuda_device):
    """Experts and whole groups left out by a very negative bias, one forced in: as the exact
    keys say."""
    from mhc_hyper_connection_gb300 import route_experts
    gen = torch.Generator(device=cuda_device).manual_seed(2)
    for E in (64, 160, 512):
        l = torch.randn((300, E), generator=gen, device=cuda_device)
        bias = 0.1 * torch.randn((E,), generator=gen, device=cuda_device)
        bias[: E // 8] = -1.0e9
        bias[E // 8 + 1: E // 4] = -1.0e9
        bias[E // 2] = 1.0e6
        for score in ("sigmoid", "softmax"):
            for mark in ("top2", "max"):
                how = dict(score=score, groups=8, top_groups=4, group_score=mark, renormalise=True, scale=1.0)
                _check(route_experts(l, 6, bias=bias, **how), l, bias, 6, **how)


@pytest.mark.parametrize("size", [1.0e4, 1.0e5])
@pytest.mark.parametrize("E,groups,top", [(64, 8, 3), (256, 8, 4), (72, 6, 2), (160, 5, 2), (192, 16, 5), (512, 8, 4), (1000, 10, 4)])
def test_one_group_that_cancels(cuda_device, E, groups, top, size):
    """One group's mark is a sum of keys that cancel, the others' are plain sums: the mark that
    fp32 has wrong need be neither the last one taken nor the first left out.  Also every
    second group's."""
    from mhc_hyper_connection_gb300 import route_experts
    gen = torch.Generator(device=cuda_device).manual_seed(E)
    l = torch.randn((300, E), generator=gen, device=cuda_device) * 0.05
    per = E // groups
    one, some = torch.zeros((groups,), device=cuda_device), size * (1.0 + torch.arange(groups, device=cuda_device) / groups)
    one[groups // 2] = size
    some[::2] = 0.0
    for by in (one, some):
        bias = torch.full((E,), -4.0 * size, device=cuda_device)
        bias[::per], bias[1::per] = by, -by
        for k in (top, 2 * top):
            for score in ("sigmoid", "softmax"):
                how = dict(score=score, groups=groups, top_groups=top, group_score="top2", renormalise=True, scale=1.0)
                _check(route_experts(l, k, bias=bias, **how), l, bias, k, **how)
