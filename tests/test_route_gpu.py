"""Routing to experts (include/mhc_route.h) against its definition in 64 bits: choice
and plan exactly, weights and gradients within fp32's rounding.

Tolerances: scores are formed with expf (2 ulp), a few roundings and a sum over E terms
in pairs: a relative error below 2^-19 of a weight (24 bits, at most 16 units).  A
gradient is a sum of products of such factors: 2^-18 of the sum of their magnitudes,
and one rounding to its type (u) with half the smallest step of fp16."""
import numpy as np
import pytest
import torch

import expert_refs as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _f64(t):
    return t.double().cpu().numpy()


def _logits(device, T, E, kind, seed, masked=0.1, padded=0.1):
    gen = torch.Generator(device=device).manual_seed(seed)
    l = torch.randn((T, E), generator=gen, device=device) * 2
    l[torch.rand((T, E), generator=gen, device=device) < masked] = -np.inf
    l[torch.rand((T,), generator=gen, device=device) < padded] = -np.inf
    return l.to(DT[kind]), torch.randn((E,), generator=gen, device=device) * 0.1


def _check(routes, l, bias, k, **how):
    e, w = ref.route(_f64(l).reshape(-1, l.shape[-1]), k, bias=None if bias is None else _f64(bias), **how)
    np.testing.assert_array_equal(routes.experts.cpu().numpy().reshape(-1, k), e)
    got = _f64(routes.weights).reshape(-1, k)
    assert np.all(np.abs(got - w) <= 2.0 ** -19 * np.abs(w) + 1e-37)


SIZES = [(1, 1, 1, 1), (1, 2, 2, 1), (3, 8, 8, 1), (7, 31, 3, 1), (33, 60, 4, 2), (65, 64, 8, 8), (5, 72, 6, 8), (130, 128, 8, 4),
         (17, 160, 6, 32), (257, 256, 8, 8), (9, 384, 32, 3), (31, 512, 1, 16), (12, 1000, 7, 10), (6, 1024, 32, 32), (4, 96, 5, 32)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups", SIZES)
def test_choice_and_weights(cuda_device, T, E, k, groups, score):
    from mhc_hyper_connection_gb300 import route_experts
    for i, kind in enumerate(("fp32", "bf16", "fp16")):
        l, bias = _logits(cuda_device, T, E, kind, 10 * T + i)
        for b in (None, bias):
            for renorm, mark in ((True, "top2"), (False, "max")):
                need = -(-k // (E // groups))
                for g, top in ((1, 1), (groups, max(need, (groups + 1) // 2))):
                    how = dict(score=score, groups=g, top_groups=top, group_score=mark, renormalise=renorm, scale=2.5)
                    _check(route_experts(l, k, bias=b, **how), l, b, k, **how)


def test_many_rows_near_ties(cuda_device):
    """Thousands of rows whose keys fp32 cannot always order: scores on a fine grid and a
    bias, so that exact ties, ties of rounded keys and distinct keys closer than 2^-24
    all occur; 16-bit logits, whose equal values tie exactly."""
    from mhc_hyper_connection_gb300 import route_experts
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    for score in ("sigmoid", "softmax"):
        for kind in ("fp32", "bf16"):
            l = (torch.randint(0, 40, (1500, 64), generator=gen, device=cuda_device) / 8 - 2.5).to(DT[kind])
            near = torch.randint(-2, 3, (1500, 64), generator=gen, device=cuda_device) * 2.0 ** -22
            if kind == "fp32":
                l = l + near * l.abs()
            bias = torch.randint(0, 2, (64,), generator=gen, device=cuda_device) * 2.0 ** -12
            for g, top in ((1, 1), (8, 3)):
                how = dict(score=score, groups=g, top_groups=top, group_score="top2", renormalise=True, scale=1.0)
                _check(route_experts(l, 6, bias=bias, **how), l, bias, 6, **how)
                _check(route_experts(l, 6, **how), l, None, 6, **how)


@pytest.mark.parametrize("equals", [1, 2, 3, 6])
def test_equals_before_a_larger_key(cuda_device, equals):
    """Behind experts with the same logit and bias one whose key is larger by less than
    fp32 shows, at the border of what is chosen."""
    from mhc_hyper_connection_gb300 import route_experts
    base = torch.linspace(1.0, 6.0, 400, device=cuda_device)
    l = torch.full((400, 40), -4.0, device=cuda_device)
    l[:, 1:1 + equals] = base[:, None]
    l[:, 30] = torch.nextafter(base, base + 1)
    l[:, 35] = base + 1
    bias = torch.full((40,), 2.0 ** -12, device=cuda_device)
    for score in ("sigmoid", "softmax"):
        for k in range(1, equals + 3):
            how = dict(score=score, renormalise=True, scale=1.0)
            _check(route_experts(l, k, bias=bias, **how), l, bias, k, **how)


@pytest.mark.parametrize("E,groups,top", [(72, 6, 2), (80, 5, 2), (96, 8, 3), (160, 8, 3), (160, 5, 2), (192, 8, 4), (192, 16, 5), (96, 32, 9)])
def test_rows_of_three_five_and_six_scores_a_lane(cuda_device, E, groups, top):
    """Widths between the powers of two: ordinary rows, and rows of the grid above."""
    from mhc_hyper_connection_gb300 import route_experts
    gen = torch.Generator(device=cuda_device).manual_seed(E + groups)
    fine = torch.randint(0, 40, (400, E), generator=gen, device=cuda_device) / 8 - 2.5
    fine = fine + torch.randint(-2, 3, (400, E), generator=gen, device=cuda_device) * 2.0 ** -22 * fine.abs()
    for kind in ("fp32", "bf16"):
        l, bias = _logits(cuda_device, 400, E, kind, E)
        for x, b in ((l, bias), (fine.to(DT[kind]), torch.randint(0, 2, (E,), generator=gen, device=cuda_device) * 2.0 ** -12)):
            for score in ("softmax", "sigmoid"):
                for g, t, mark in ((1, 1, "max"), (groups, top, "top2"), (groups, top, "max")):
                    how = dict(score=score, groups=g, top_groups=t, group_score=mark, renormalise=True, scale=1.0)
                    _check(route_experts(x, 6, bias=b, **how), x, b, 6, **how)
                    _check(route_experts(x, 6, **how), x, None, 6, **how)


def test_signed_nan(cuda_device):
    """A NaN of either sign, of a logit or of the bias, is chosen first."""
    from mhc_hyper_connection_gb300 import route_experts
    for bits in (0x7FC00000, -0x400000, 0x7F800001, -0x7FFFFF):
        nan = torch.tensor([bits], dtype=torch.int32, device=cuda_device).view(torch.float32)[0]
        assert bool(nan.isnan())
        for E in (40, 256):
            l, bias = torch.randn((3, E), device=cuda_device), torch.zeros((E,), device=cuda_device)
            bad = l.clone()
            bad[:, 33] = nan
            worse = bias.clone()
            worse[33] = nan
            for x, b in ((bad, None), (bad, bias), (l, worse)):
                r = route_experts(x, 4, score="sigmoid", bias=b)
                assert (r.experts[:, 0] == 33).all() and (r.experts[:, 1:] != 33).all()


def test_saturated_and_tiny_scores(cuda_device):
    """Logits at which fp32 scores are all 1 or all underflow still have their order and
    their shares."""
    from mhc_hyper_connection_gb300 import route_experts, route_experts_backward
    base = torch.arange(16, device=cuda_device, dtype=torch.float32)
    for shift in (20.0, 90.0, -90.0, -120.0, -300.0):
        l = (base * 0.25 + shift).expand(4, 16).contiguous()
        for score in ("softmax", "sigmoid"):
            how = dict(score=score, renormalise=True, scale=1.0)
            r = route_experts(l, 5, **how)
            np.testing.assert_array_equal(r.experts.cpu().numpy(), np.tile(np.arange(15, 10, -1), (4, 1)))
            _, w = ref.route(_f64(l), 5, **how)
            assert np.all(np.abs(_f64(r.weights) - w) <= 2.0 ** -19 * w)
            d = torch.randn((4, 5), device=cuda_device)
            g, mag = ref.route_backward(_f64(d), _f64(l), r.experts.cpu().numpy(), score, True, 1.0)
            got = _f64(route_experts_backward(d, l, r.experts, **how))
            assert np.all(np.abs(got - g) <= 2.0 ** -18 * mag + 1e-37)


def test_values_that_are_not_finite(cuda_device):
    """A NaN is chosen first and seen in every weight that it takes part in; +inf is
    chosen first; a row of -inf alone chooses nothing."""
    from mhc_hyper_connection_gb300 import route_experts
    l = torch.zeros((4, 40), device=cuda_device)
    l[0, 17] = np.nan
    l[1, 23] = np.inf
    l[2] = -np.inf
    l[3, :39] = -np.inf
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros((40,), device=cuda_device)):
            r = route_experts(l, 3, score=score, bias=bias)
            e, w = r.experts.cpu().numpy(), r.weights.cpu().numpy()
            assert np.isnan(w[0]).all()
            if bias is None or score == "sigmoid":
                assert e[0, 0] == 17 and e[1, 0] == 23
            assert np.isnan(w[1]).all() if score == "softmax" else np.isfinite(w[1]).all()
            assert (e[2] == -1).all() and (w[2] == 0).all()
            assert e[3].tolist() == [39, -1, -1] and w[3].tolist() == [1, 0, 0]


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k,groups", SIZES)
def test_backward(cuda_device, T, E, k, groups, score, renorm):
    from mhc_hyper_connection_gb300 import route_experts, route_experts_backward
    for i, kind in enumerate(("fp32", "bf16", "fp16")):
        l, _ = _logits(cuda_device, T, E, kind, 7 * T + i)
        r = route_experts(l, k, score=score, renormalise=renorm, scale=1.5)
        d = torch.randn((T, k), device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(T))
        d[r.experts < 0] = np.nan                                 # slots without an expert are not read into anything
        got = route_experts_backward(d, l, r.experts, score=score, renormalise=renorm, scale=1.5)
        assert got.dtype == l.dtype
        g, mag = ref.route_backward(np.nan_to_num(_f64(d)), _f64(l), r.experts.cpu().numpy(), score, renorm, 1.5)
        got = _f64(got)
        assert np.all(np.abs(got - g) <= 2.0 ** -18 * mag + U[kind] * np.abs(g) + (0 if kind == "fp32" else 2.0 ** -25) + 1e-37)


def test_backward_against_differences(cuda_device):
    """Central differences of sum d w in 64 bits, the choice held."""
    from mhc_hyper_connection_gb300 import route_experts, route_experts_backward
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            l, _ = _logits(cuda_device, 5, 12, "fp32", 1, masked=0.0, padded=0.0)
            how = dict(score=score, renormalise=renorm, scale=2.0)
            r = route_experts(l, 3, **how)
            d = torch.randn((5, 3), device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(1))
            got, e, dn = _f64(route_experts_backward(d, l, r.experts, **how)), r.experts.cpu().numpy(), _f64(d)

            def loss(ln):
                s = np.take_along_axis(ref.scores(ln, score), e, 1)
                return float((dn * 2.0 * (s / s.sum(-1, keepdims=True) if renorm else s)).sum())
            ln = _f64(l)
            for t in range(5):
                for i in range(12):
                    up, dn_ = ln.copy(), ln.copy()
                    up[t, i] += 1e-5
                    dn_[t, i] -= 1e-5
                    # the step's own error is below 1e-9, fp32's below 2^-18 of the terms (at most 8)
                    assert abs((loss(up) - loss(dn_)) / 2e-5 - got[t, i]) <= 2.0 ** -18 * 8 + 1e-8


def test_backward_with_given_experts(cuda_device):
    """Experts that no routing chose: one twice, some outside the range, one masked."""
    from mhc_hyper_connection_gb300 import route_experts_backward
    l, _ = _logits(cuda_device, 6, 20, "fp32", 4, masked=0.0, padded=0.0)
    l[:, 3] = -np.inf
    e = torch.tensor([[1, 1, 2, 5], [-1, 7, 20, 7], [3, 3, 3, 3], [-1, -1, -1, -1], [3, 4, 1000, 4], [0, 1, 2, 19]],
                     device=cuda_device, dtype=torch.int32)
    d = torch.randn((6, 4), device=cuda_device, generator=torch.Generator(device=cuda_device).manual_seed(2))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = _f64(route_experts_backward(d, l, e, score=score, renormalise=renorm))
            g, mag = ref.route_backward(_f64(d), _f64(l), e.cpu().numpy(), score, renorm, 1.0)
            assert np.all(np.abs(got - g) <= 2.0 ** -18 * mag + 1e-37)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (5, 2, 3), (100, 8, 64), (1000, 8, 40), (1024, 8, 1024), (1025, 8, 9), (4099, 6, 300),
                                   (2500, 32, 1024), (20000, 4, 5)])
def test_plan(cuda_device, T, k, E):
    """Counts and order, by the rows that experts_ffn reads: a plan's rows are checked
    through its buffer (places and rows lie behind the table, as mhc_experts.cuh says)."""
    from mhc_hyper_connection_gb300 import expert_plan
    gen = torch.Generator(device=cuda_device).manual_seed(T)
    e = torch.randint(-2, E + 2, (T, k), generator=gen, device=cuda_device, dtype=torch.int32)
    if T == 1000:
        e[:700] = 5                                               # one expert with most slots, many times a token
    for _ in range(2):
        p = expert_plan(e, E)
        counts, places, rows = ref.plan(e.cpu().numpy(), E)
        np.testing.assert_array_equal(p.counts.cpu().numpy(), counts)
        words = p.buffer.view(torch.int32).cpu().numpy()
        up = lambda n: (n + 63) // 64 * 64  # noqa: E731
        slots, active = T * k, min(E, T * k)
        width = min(256, max(32, up2(-(-4 * slots // E))))
        tiles = slots // width + active
        at = 64 + up(E) + up(E + 1) + up(8 * tiles)
        np.testing.assert_array_equal(words[at:at + slots], places.reshape(-1))
        at += up(slots)
        assert words[1] == len(rows) <= p.rows
        np.testing.assert_array_equal(words[at:at + len(rows)], rows)
        # tiles cover each expert's rows once
        table = words[64 + up(E) + up(E + 1):][:8 * words[2]].reshape(-1, 8)
        seen = np.zeros(len(rows), int)
        for i, (x, first, n, row, n_rows, w, wide, _) in enumerate(table):
            j = i - first
            assert 0 <= j < n <= 8 and w % 32 == 0 and w + (32 if wide else 0) <= width
            off = j * w + 32 * min(j, wide)
            b, m = row + off, min(w + (32 if j < wide else 0), n_rows - off)
            assert m > 0
            seen[b:b + m] += 1
            assert (e.cpu().numpy().reshape(-1)[rows[b:b + m]] == x).all()
        np.testing.assert_array_equal(seen, rows >= 0)


def test_plan_of_very_many_slots(cuda_device):
    """2^22 slots: the order against a stable sort."""
    from mhc_hyper_connection_gb300 import expert_plan
    T, k, E = 1 << 20, 4, 1000
    e = torch.randint(-1, E, (T, k), generator=torch.Generator(device=cuda_device).manual_seed(1), device=cuda_device, dtype=torch.int32)
    p = expert_plan(e, E)
    flat = e.reshape(-1).long()
    counts = torch.bincount(flat + 1, minlength=E + 1)[1:]
    assert torch.equal(p.counts.long(), counts)
    padded = (counts + 15) // 16 * 16
    start = padded.cumsum(0) - padded
    order = torch.sort(flat, stable=True).indices[flat.numel() - int(counts.sum()):]        # slots by expert, -1 first
    rank = torch.arange(order.numel(), device=cuda_device) - (counts.cumsum(0) - counts)[flat[order]]
    want = torch.full_like(flat, -1)
    want[order] = start[flat[order]] + rank
    up = lambda n: (n + 63) // 64 * 64  # noqa: E731
    tiles = T * k // 256 + E
    at = 64 + up(E) + up(E + 1) + up(8 * tiles)
    words = p.buffer.view(torch.int32)
    assert torch.equal(words[at:at + T * k].long(), want)
    rows = words[at + up(T * k):][:int(padded.sum())].long()
    assert torch.equal(rows[want[order]], order) and int((rows < 0).sum()) == int((padded - counts).sum())


def up2(n):
    return (n + 31) // 32 * 32


def test_given_outputs_streams_and_shapes(cuda_device):
    from mhc_hyper_connection_gb300 import Routes, expert_plan, route_experts, route_experts_backward
    l, bias = _logits(cuda_device, 60, 48, "fp32", 9)
    want = route_experts(l, 4, bias=bias)
    l3 = l.reshape(6, 10, 48)
    out = Routes(torch.empty((6, 10, 4), dtype=torch.int32, device=cuda_device), torch.empty((6, 10, 4), device=cuda_device))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = route_experts(l3, 4, bias=bias, out=out, stream=side)
    assert got.experts is out.experts
    d = torch.randn((6, 10, 4), device=cuda_device)
    side.wait_stream(torch.cuda.current_stream())
    gl = route_experts_backward(d, l3, got.experts, stream=side)
    plan = expert_plan(got.experts, 48, stream=side)
    side.synchronize()
    assert torch.equal(got.experts.reshape(60, 4), want.experts) and torch.equal(got.weights.reshape(60, 4), want.weights)
    assert torch.equal(gl.reshape(60, 48), route_experts_backward(d.reshape(60, 4), l, want.experts))
    assert torch.equal(plan.counts, expert_plan(want.experts, 48).counts)
    empty = route_experts(l[:0], 4)
    assert empty.experts.shape == (0, 4) and expert_plan(empty.experts, 48).counts.tolist() == [0] * 48
    assert route_experts_backward(empty.weights, l[:0], empty.experts).shape == (0, 48)
