"""Routed experts (include/mhc_experts.h) against their formulas in 64 bits, forward and
backward; bounds as expert_refs derives them."""
import numpy as np
import pytest
import torch

import expert_refs as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def _f64(t):
    return t.double().cpu().numpy()


def _case(device, T, E, k, D, F, kind, seed, skew=1.0, dropped=0.1):
    gen = torch.Generator(device=device).manual_seed(seed)
    rn = lambda *shape, m=1.0: torch.randn(shape, generator=gen, device=device) * m  # noqa: E731
    l = rn(T, E) + skew * rn(E)
    idx = l.topk(k, -1).indices.int()
    idx[torch.rand((T, k), generator=gen, device=device) < dropped] = -1
    return dict(x=rn(T, D).to(DT[kind]), w=rn(E, 2, F, D, m=D ** -0.5).to(DT[kind]), wd=rn(E, D, F, m=F ** -0.5).to(DT[kind]),
                gy=rn(T, D, m=0.25).to(DT[kind]), idx=idx.contiguous(), wt=rn(T, k))


def _near(got, want, tol, what):
    got = _f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - want)):.3g}"


def _run(c, act, save="16bit"):
    from mhc_hyper_connection_gb300 import expert_plan, experts_ffn, experts_ffn_status, experts_ffn_workspace
    E, _, F, D = c["w"].shape
    T, k = c["idx"].shape
    plan = expert_plan(c["idx"], E)
    ws = experts_ffn_workspace(T, E, k, D, F, c["x"].device)
    y, kept = experts_ffn(c["x"], c["wt"], plan, c["w"], c["wd"], act=act, save=save, workspace=ws)
    assert experts_ffn_status(ws) == 0
    return plan, y, kept


def _slots(c, kept):
    """Kept sums by slot [T, k, 2, F], zeros where there is no expert."""
    idx = c["idx"].cpu().numpy()
    places = ref.plan(idx, c["w"].shape[0])[1]
    v = _f64(kept)[np.maximum(places, 0)]
    return np.where((places >= 0)[..., None, None], v, 0.0), places


def _check_forward(c, kind, act, y, kept=None):
    idx = c["idx"].cpu().numpy()
    want, tol, sums, esums = ref.experts(*(_f64(c[n]) for n in ("x", "wt")), idx, _f64(c["w"]), _f64(c["wd"]), act, kind)
    _near(y, want, tol, "y")
    if kept is not None:
        got, places = _slots(c, kept)
        bad = np.abs(got - sums) > ref.U[kind] * np.abs(sums) + 2 * esums + ref.TINY
        assert not bad[places >= 0].any()


def _check_backward(c, kind, act, plan, kept, workspace=None):
    from mhc_hyper_connection_gb300 import experts_ffn_backward, experts_ffn_status, experts_ffn_workspace
    E, _, F, D = c["w"].shape
    T, k = c["idx"].shape
    ws = experts_ffn_workspace(T, E, k, D, F, c["x"].device, backward=True)
    got = experts_ffn_backward(c["gy"], c["x"], c["wt"], plan, c["w"], c["wd"], kept, act=act, workspace=ws)
    assert experts_ffn_status(ws) == 0
    want = ref.experts_backward(_f64(c["gy"]), _f64(c["x"]), _f64(c["wt"]), c["idx"].cpu().numpy(), _f64(c["w"]), _f64(c["wd"]),
                                _slots(c, kept)[0], act, kind)
    for name, (v, tol) in want.items():
        _near(got[name], v, tol, name)
    return got


SHAPES = [(1, 1, 1, 8, 8), (1, 4, 2, 64, 128), (3, 8, 3, 72, 136), (17, 16, 4, 136, 72), (40, 3, 2, 264, 200), (64, 64, 6, 128, 64),
          (130, 5, 2, 520, 264), (300, 2, 1, 200, 392), (333, 12, 3, 264, 520), (700, 4, 2, 136, 264)]


@pytest.mark.parametrize("kind,act", [("bf16", "silu"), ("fp16", "gelu")])
@pytest.mark.parametrize("T,E,k,D,F", SHAPES)
def test_forward(cuda_device, T, E, k, D, F, kind, act):
    c = _case(cuda_device, T, E, k, D, F, kind, T + D)
    for save in (None, "16bit"):
        _, y, kept = _run(c, act, save)
        _check_forward(c, kind, act, y, kept)


@pytest.mark.parametrize("kind,act", [("bf16", "gelu"), ("fp16", "silu")])
@pytest.mark.parametrize("T,E,k,D,F", SHAPES)
def test_backward(cuda_device, T, E, k, D, F, kind, act):
    c = _case(cuda_device, T, E, k, D, F, kind, T + F)
    plan, _, kept = _run(c, act)
    _check_backward(c, kind, act, plan, kept)


def _torch64(c, act):
    """The layer body in 64 bits for automatic differentiation: (y, leaves)."""
    x, w, wd, wt = (c[n].double().requires_grad_() for n in ("x", "w", "wd", "wt"))
    y = torch.zeros_like(x)
    for e in range(w.shape[0]):
        for j in range(c["idx"].shape[1]):
            t = torch.nonzero(c["idx"][:, j] == e)[:, 0]
            if len(t):
                g, u = x[t] @ w[e, 0].t(), x[t] @ w[e, 1].t()
                h = g * torch.sigmoid(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
                y = y.index_add(0, t, wt[t, j, None] * ((h * u) @ wd[e].t()))
    return y, dict(grad_x=x, grad_w_gate_up=w, grad_w_down=wd, grad_weights=wt)


def test_one_expert_takes_everything(cuda_device):
    """All slots, many of them a token's twice, in one of several experts: more tiles than
    one band of an expert, no rows elsewhere."""
    c = _case(cuda_device, 1300, 3, 2, 264, 136, "bf16", 1)
    c["idx"][:] = 1
    plan, y, kept = _run(c, "silu")
    assert plan.counts.tolist() == [0, 2600, 0]
    _check_forward(c, "bf16", "silu", y, kept)
    got = _check_backward(c, "bf16", "silu", plan, kept)
    assert (got["grad_w_gate_up"][0] == 0).all() and (got["grad_w_down"][2] == 0).all()


def test_no_slot_has_an_expert(cuda_device):
    from mhc_hyper_connection_gb300 import experts_ffn_backward
    c = _case(cuda_device, 50, 4, 2, 64, 72, "fp16", 2)
    for v in (-1, 4, 1000):
        c["idx"][:] = v
        plan, y, kept = _run(c, "gelu")
        assert (y == 0).all()
        got = experts_ffn_backward(c["gy"], c["x"], c["wt"], plan, c["w"], c["wd"], kept, act="gelu")
        assert all((v == 0).all() for v in got.values())


def test_no_tokens(cuda_device):
    from mhc_hyper_connection_gb300 import expert_plan, experts_ffn, experts_ffn_backward
    c = _case(cuda_device, 3, 4, 2, 64, 72, "bf16", 2)
    plan = expert_plan(c["idx"][:0], 4)
    y, kept = experts_ffn(c["x"][:0], c["wt"][:0], plan, c["w"], c["wd"], save="16bit")
    assert y.shape == (0, 64) and kept.shape == (0, 2, 72)
    grads = {"grad_x": y, "grad_weights": c["wt"][:0], "grad_w_gate_up": torch.ones_like(c["w"]), "grad_w_down": torch.ones_like(c["wd"])}
    got = experts_ffn_backward(y, c["x"][:0], c["wt"][:0], plan, c["w"], c["wd"], kept, grads=grads)
    assert (got["grad_w_gate_up"] == 0).all() and (got["grad_w_down"] == 0).all()


@pytest.mark.parametrize("T,E,k,D,F", [(2000, 8, 3, 1032, 520), (5000, 40, 6, 520, 264), (600, 1, 1, 2056, 1288)])
def test_large(cuda_device, T, E, k, D, F):
    """More tiles than pairs of SMs in every product, a ragged edge on each axis, the plan in
    several blocks."""
    c = _case(cuda_device, T, E, k, D, F, "bf16", 5)
    plan, y, kept = _run(c, "silu")
    _check_forward(c, "bf16", "silu", y, kept)
    _check_backward(c, "bf16", "silu", plan, kept)


def test_values_that_are_not_finite(cuda_device):
    """An expert's NaN reaches the tokens that take it and its own gradients, a token's
    infinity its own row and the gradients of its experts: everything else keeps its bits,
    the experts whose rows share a copy among them."""
    from mhc_hyper_connection_gb300 import experts_ffn_backward
    c = _case(cuda_device, 200, 6, 2, 136, 264, "bf16", 6, skew=0.0)
    plan, y, kept = _run(c, "silu")
    got = experts_ffn_backward(c["gy"], c["x"], c["wt"], plan, c["w"], c["wd"], kept)
    idx, places = c["idx"].cpu().numpy(), _slots(c, kept)[1]
    for what in ("expert", "token", "grad"):
        d = {k: v.clone() for k, v in c.items()}
        if what == "expert":
            d["w"][3, 0, 5, 7] = float("nan")
            d["wd"][3, 100] = float("inf")
            rows = (idx == 3).any(1)
            experts = {3}
        else:
            (d["x"] if what == "token" else d["gy"])[11] = float("inf") if what == "token" else float("nan")
            rows = np.arange(200) == 11
            experts = set(idx[11][idx[11] >= 0].tolist())
        _, y2, kept2 = _run(d, "silu")
        got2 = experts_ffn_backward(d["gy"], d["x"], d["wt"], plan, d["w"], d["wd"], kept2)
        clean = torch.as_tensor(~rows, device=cuda_device)
        assert torch.equal(y2[clean], y[clean]) and torch.equal(got2["grad_x"][clean], got["grad_x"][clean])
        if what != "grad":
            assert not torch.isfinite(y2[~clean].float()).all(1).any()
        same = torch.as_tensor((idx < 0) | ~np.isin(idx, list(experts)) | (~rows[:, None] & (what != "expert")), device=cuda_device)
        assert torch.equal(got2["grad_weights"][same], got["grad_weights"][same])
        for e in range(6):
            for k in ("grad_w_gate_up", "grad_w_down"):
                if e in experts:
                    assert not torch.isfinite(got2[k][e].float()).all()
                else:
                    assert torch.equal(got2[k][e], got[k][e]), (what, e, k)


def test_padding_of_the_kept_sums_is_left_alone(cuda_device):
    from mhc_hyper_connection_gb300 import expert_plan, experts_ffn
    c = _case(cuda_device, 70, 5, 2, 64, 136, "bf16", 7)
    plan = expert_plan(c["idx"], 5)
    kept = torch.full((plan.rows, 2, 136), 7.0, dtype=torch.bfloat16, device=cuda_device)
    experts_ffn(c["x"], c["wt"], plan, c["w"], c["wd"], save="16bit", kept=kept)
    rows = ref.plan(c["idx"].cpu().numpy(), 5)[2]
    pad = np.ones(plan.rows, bool)
    pad[:len(rows)] = rows < 0
    assert pad.any() and (kept[torch.as_tensor(pad, device=cuda_device)] == 7.0).all()


def test_against_automatic_differentiation_and_differences(cuda_device):
    """All gradients against automatic differentiation in 64 bits, as norms: the kernels
    round g, u, a, gg, gu, w a to fp16 (2^-11 each at most) and each result once: 2^-8 of a
    gradient's norm covers seven of them in line."""
    from mhc_hyper_connection_gb300 import experts_ffn_backward
    for act in ("silu", "gelu"):
        c = _case(cuda_device, 60, 5, 3, 72, 136, "fp16", 8)
        plan, y, kept = _run(c, act)
        got = experts_ffn_backward(c["gy"], c["x"], c["wt"], plan, c["w"], c["wd"], kept, act=act)
        want, leaves = _torch64(c, act)
        (want * c["gy"].double()).sum().backward()
        for k, v in leaves.items():
            assert float((got[k].double() - v.grad).norm()) <= 2.0 ** -8 * float(v.grad.norm()), (act, k)
        loss = lambda: float((_torch64(c, act)[0].detach() * c["gy"].double()).sum())  # noqa: E731
        out = got["grad_weights"].double()
        for t, j in ((0, 0), (7, 1), (31, 2), (59, 0)):
            if c["idx"][t, j] >= 0:                  # the loss is linear in a weight
                keep = c["wt"][t, j].clone()
                c["wt"][t, j] = keep + 0.5
                up = loss()
                c["wt"][t, j] = keep - 0.5
                assert abs(up - loss() - float(out[t, j])) <= 2.0 ** -8 * float(out.abs().max())
                c["wt"][t, j] = keep


def test_repeats_streams_and_shapes(cuda_device):
    from mhc_hyper_connection_gb300 import expert_plan, experts_ffn, experts_ffn_backward
    c = _case(cuda_device, 600, 9, 3, 264, 200, "bf16", 9)
    plan, y, kept = _run(c, "silu")
    got = experts_ffn_backward(c["gy"], c["x"], c["wt"], plan, c["w"], c["wd"], kept)
    for _ in range(5):
        plan2, y2, kept2 = _run(c, "silu")
        again = experts_ffn_backward(c["gy"], c["x"], c["wt"], plan2, c["w"], c["wd"], kept2)
        assert torch.equal(y, y2) and all(torch.equal(got[k], again[k]) for k in got)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = {k: v.reshape(30, 20, -1) for k, v in c.items() if k in ("x", "gy", "idx", "wt")}
    p3 = expert_plan(b["idx"], 9, stream=side)
    y3, kept3 = experts_ffn(b["x"], b["wt"], p3, c["w"], c["wd"], save="16bit", stream=side)
    g3 = experts_ffn_backward(b["gy"], b["x"], b["wt"], p3, c["w"], c["wd"], kept3, stream=side)
    side.synchronize()
    assert y3.shape == (30, 20, 264) and torch.equal(y3.reshape(y.shape), y)
    assert all(torch.equal(g3[k].reshape(got[k].shape), got[k]) for k in got)


def test_two_calls_at_once(cuda_device):
    """Calls of one plan on two streams with workspaces of their own."""
    from mhc_hyper_connection_gb300 import experts_ffn
    c = _case(cuda_device, 900, 9, 3, 264, 520, "bf16", 10)
    d = _case(cuda_device, 900, 9, 3, 264, 520, "bf16", 11)
    plan, y, _ = _run(c, "silu")
    want = experts_ffn(d["x"], d["wt"], plan, d["w"], d["wd"])[0]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(10):
        for s, v, o in zip(streams, (c, d), outs):
            o.append(experts_ffn(v["x"], v["wt"], plan, v["w"], v["wd"], stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o in outs[0]) and all(torch.equal(o, want) for o in outs[1])


def _step(mhc, c, logits, ws, out):
    """A whole training step of the body on given buffers."""
    r = mhc.route_experts(logits, 3, score="sigmoid", bias=out["bias"], groups=3, top_groups=2, out=out["routes"])
    plan = mhc.expert_plan(r.experts, 9, buffer=out["plan"])
    mhc.experts_ffn(c["x"], r.weights, plan, c["w"], c["wd"], save="16bit", y=out["y"], kept=out["kept"], workspace=ws[0])
    g = mhc.experts_ffn_backward(c["gy"], c["x"], r.weights, plan, c["w"], c["wd"], out["kept"], grads=out["grads"], workspace=ws[1])
    mhc.route_experts_backward(g["grad_weights"], logits, r.experts, score="sigmoid", grad_logits=out["grad_logits"])
    mhc.orthogonalise(g["grad_w_down"], out=out["update"], workspace=ws[2])


def test_whole_step_captured(cuda_device):
    """Routing, plan, experts, gradients and the weights' update captured into two graphs that
    share workspaces, replayed on other inputs than they were captured with."""
    import mhc_hyper_connection_gb300 as mhc
    T, E, k, D, F = 333, 9, 3, 136, 264
    c = _case(cuda_device, T, E, k, D, F, "bf16", 12)
    gen = torch.Generator(device=cuda_device).manual_seed(1)
    logits = torch.randn((T, E), generator=gen, device=cuda_device)
    ws = (mhc.experts_ffn_workspace(T, E, k, D, F, cuda_device), mhc.experts_ffn_workspace(T, E, k, D, F, cuda_device, backward=True),
          mhc.orthogonalise_workspace((E, D, F), cuda_device))
    rows = mhc.expert_plan(c["idx"], E).rows

    def buffers():
        e = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device=cuda_device)  # noqa: E731
        return dict(bias=0.1 * torch.arange(E, device=cuda_device, dtype=torch.float32),
                    routes=mhc.Routes(e(T, k, d=torch.int32), e(T, k, d=torch.float32)), plan=torch.empty_like(mhc.expert_plan(c["idx"], E).buffer),
                    y=e(T, D), kept=e(rows, 2, F), grad_logits=e(T, E, d=torch.float32), update=e(E, D, F),
                    grads=dict(grad_x=e(T, D), grad_weights=e(T, k, d=torch.float32), grad_w_gate_up=e(E, 2, F, D), grad_w_down=e(E, D, F)))

    def results(o):
        return [o["y"], o["grad_logits"], o["update"], *o["routes"], *o["grads"].values()]

    eager, a, b = buffers(), buffers(), buffers()
    _step(mhc, c, logits, ws, eager)
    graphs = []
    for o in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _step(mhc, c, logits, ws, o)
        graphs.append(graph)
    other = _case(cuda_device, T, E, k, D, F, "bf16", 13)
    for data in (other, c, other):
        for n in ("x", "gy"):
            c[n].copy_(data[n].clone())
        logits.add_(0.3 * torch.randn((T, E), generator=gen, device=cuda_device))
        _step(mhc, c, logits, ws, eager)
        for graph, o in zip(graphs, (a, b)):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(results(o), results(eager)))
    assert all(mhc.experts_ffn_status(w) == 0 for w in ws[:2]) and mhc.orthogonalise_status(ws[2]) == 0


def test_layer_body_against_automatic_differentiation(cuda_device):
    """Routing, experts and both backward passes together, in 64 bits with the choice held: y
    and every gradient as norms.  About eight roundings of at most 2^-8 lie between an input
    and a gradient: 2^-5."""
    import mhc_hyper_connection_gb300 as mhc
    for score, renorm, act in (("softmax", True, "silu"), ("sigmoid", True, "gelu"), ("softmax", False, "silu"), ("sigmoid", False, "silu")):
        c = _case(cuda_device, 150, 12, 3, 72, 136, "bf16", 14)
        logits = torch.randn((150, 12), generator=torch.Generator(device=cuda_device).manual_seed(3), device=cuda_device)
        bias = 0.2 * torch.randn((12,), generator=torch.Generator(device=cuda_device).manual_seed(4), device=cuda_device)
        how = dict(score=score, renormalise=renorm, scale=1.5)
        r = mhc.route_experts(logits, 3, bias=bias, groups=4, top_groups=2, **how)
        plan = mhc.expert_plan(r.experts, 12)
        y, kept = mhc.experts_ffn(c["x"], r.weights, plan, c["w"], c["wd"], act=act, save="16bit")
        got = mhc.experts_ffn_backward(c["gy"], c["x"], r.weights, plan, c["w"], c["wd"], kept, act=act)
        got["grad_logits"] = mhc.route_experts_backward(got["grad_weights"], logits, r.experts, **how)
        l64 = logits.double().requires_grad_()
        s = torch.softmax(l64, -1) if score == "softmax" else torch.sigmoid(l64)
        w = s.gather(1, r.experts.long())
        w = 1.5 * (w / w.sum(-1, keepdim=True) if renorm else w)
        want, leaves = _torch64(dict(c, idx=r.experts, wt=w.detach()), act)
        (want * c["gy"].double()).sum().backward()
        w.backward(leaves["grad_weights"].grad)
        leaves["grad_logits"] = l64
        assert float((y.double() - want).norm()) <= 2.0 ** -7 * float(want.norm())
        for k, v in leaves.items():
            assert float((got[k].double() - v.grad).norm()) <= 2.0 ** -5 * float(v.grad.norm()), (score, renorm, k)
