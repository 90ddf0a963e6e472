"""The gated feed-forward block (include/mhc_ffn.h) against its formulas in 64
bits, forward and backward.

Tolerances, from the arithmetic (u = 2^-8 bf16, 2^-11 fp16: one rounding;
tiny = half the smallest step of fp16, 2^-25):
  * a product of depth K is summed in fp32, sixteen products at a time: off by
    at most s(K) = (K / 16 + 16) 2^-22 times the sum of the magnitudes;
  * act and act' carry a few fast-math errors of 2^-22: 2^-18 of their scale;
  * a, gg and gu are rounded to 16 bits (u and tiny), outputs once more.
These are propagated through the formulas with magnitudes (|act'| <= 1.13)."""
import numpy as np
import pytest
import torch

import layer_refs as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = 2.0 ** -25
FAST = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


def s(K):
    return (K / 16 + 16) * 2.0 ** -22


def _f64(t):
    return t.double().cpu().numpy()


def _case(device, T, D, F, kind, seed):
    gen = torch.Generator(device=device).manual_seed(seed)
    rn = lambda *shape, k=1.0: (torch.randn(shape, generator=gen, device=device) * k).to(DT[kind])  # noqa: E731
    return dict(x=rn(T, D), w=rn(2, F, D, k=D ** -0.5), wd=rn(D, F, k=F ** -0.5), gy=rn(T, D, k=0.25),
                gu=rn(T, 2, F))


def _near(got, want, tol, what):
    got = _f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.abs(got - want).max():.3g}"


def _check_forward(c, kind, act, y, kept=None):
    x, w, wd = _f64(c["x"]), _f64(c["w"]), _f64(c["wd"])
    u = U[kind]
    D, F = w.shape[2], w.shape[1]
    yr, g, up = ref.ffn(x, w, wd, act)
    eg, eu = (s(D) * (np.abs(x) @ np.abs(w[h]).T) for h in (0, 1))
    h = ref.act(g, act)[0]
    a = h * up
    ea = (1.13 * eg + FAST * np.abs(g)) * (np.abs(up) + eu) + (np.abs(h) + FAST * np.abs(g)) * eu + u * np.abs(a)
    ea = ea * (1 + u) + TINY
    _near(y, yr, (ea + s(F) * np.abs(a)) @ np.abs(wd).T + 1.01 * u * np.abs(yr) + u * (ea @ np.abs(wd).T) + TINY, "y")
    if kept is None:
        return
    if isinstance(kept, torch.Tensor):
        for k, (v, e) in enumerate(((g, eg), (up, eu))):
            _near(kept[:, k], v, u * np.abs(v) + 2 * e + TINY, "kept")
    else:
        codes, scales = kept.codes.cpu().numpy(), kept.scales.cpu().numpy()
        for k, (v, e) in enumerate(((g, eg), (up, eu))):
            got = ref.restore(codes[:, k], scales[:, k])
            # half a step: 2^-4 of the value, or half the smallest step of a
            # scale that may be one power above the exact one
            sc = np.repeat(2.0 ** (ref.pack(v, kind)[1].astype(float) - 127), 128, -1)[:, :F]
            bad = ~(np.abs(got - v) <= 2.0 ** -4 * np.abs(v) + 2.0 ** -9 * sc + 2 * e)
            assert not bad.any(), f"kept codes: {bad.sum()} outside"


def _check_backward(c, kind, act, got, kept):
    x, w, wd, gy = _f64(c["x"]), _f64(c["w"]), _f64(c["wd"]), _f64(c["gy"])
    if isinstance(kept, torch.Tensor):
        g, up = _f64(kept[:, 0]), _f64(kept[:, 1])
    else:
        g, up = (ref.restore(kept.codes.cpu().numpy()[:, k], kept.scales.cpu().numpy()[:, k]) for k in (0, 1))
    u = U[kind]
    D, F, T = w.shape[2], w.shape[1], x.shape[0]
    want = ref.ffn_backward(gy, x, w, wd, g, up, act)
    h, dh = ref.act(g, act)
    ga = gy @ wd
    ega = s(D) * (np.abs(gy) @ np.abs(wd))
    gg, gu, a = ga * up * dh, ga * h, h * up
    fast = FAST * (1 + np.abs(g)) * (1 + (0 if act == "silu" else 1) * g * g)
    egg = (np.abs(up) * (1.13 * ega + np.abs(ga) * fast) + u * np.abs(gg)) * (1 + u) + TINY
    egu = (np.abs(h) * ega + np.abs(ga) * FAST * (1 + np.abs(g)) + u * np.abs(gu)) * (1 + u) + TINY
    ea = (np.abs(up) * FAST * (1 + np.abs(g)) + u * np.abs(a)) * (1 + u) + TINY
    out = lambda e, v: e * (1 + u) + u * np.abs(v) + TINY  # noqa: E731
    e = (egg + s(2 * F) * np.abs(gg)) @ np.abs(w[0]) + (egu + s(2 * F) * np.abs(gu)) @ np.abs(w[1])
    _near(got["grad_x"], want["grad_x"], out(e, want["grad_x"]), "grad_x")
    e = np.stack([(d + s(T) * np.abs(v)).T @ np.abs(x) for d, v in ((egg, gg), (egu, gu))])
    _near(got["grad_w_gate_up"], want["grad_w_gate_up"], out(e, want["grad_w_gate_up"]), "grad_w_gate_up")
    e = np.abs(gy).T @ (ea + s(T) * np.abs(a))
    _near(got["grad_w_down"], want["grad_w_down"], out(e, want["grad_w_down"]), "grad_w_down")


SHAPES = [(1, 8, 8), (3, 64, 128), (5, 72, 136), (17, 256, 264), (64, 136, 1032), (65, 520, 256), (127, 64, 504),
          (128, 128, 128), (129, 264, 520), (300, 512, 392), (513, 256, 1000)]


@pytest.mark.parametrize("kind,act", [("bf16", "silu"), ("fp16", "gelu")])
@pytest.mark.parametrize("T,D,F", SHAPES)
def test_forward(cuda_device, T, D, F, kind, act):
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_status, gated_ffn_workspace
    c = _case(cuda_device, T, D, F, kind, T + D)
    ws = gated_ffn_workspace(T, D, F, cuda_device)
    for save in (None, "16bit", "8bit"):
        y, kept = gated_ffn(c["x"], c["w"], c["wd"], act=act, save=save, workspace=ws)
        assert gated_ffn_status(ws) == 0
        _check_forward(c, kind, act, y, kept)


@pytest.mark.parametrize("kind,act", [("bf16", "gelu"), ("fp16", "silu")])
@pytest.mark.parametrize("T,D,F", SHAPES)
def test_backward(cuda_device, T, D, F, kind, act):
    from mhc_hyper_connection_gb300 import ckpt8_pack, gated_ffn_backward, gated_ffn_status, gated_ffn_workspace
    c = _case(cuda_device, T, D, F, kind, T + F)
    ws = gated_ffn_workspace(T, D, F, cuda_device, backward=True)
    for kept in (c["gu"], ckpt8_pack(c["gu"])):
        got = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, act=act, workspace=ws)
        assert gated_ffn_status(ws) == 0
        _check_backward(c, kind, act, got, kept)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 96, 111, 128])
def test_few_tokens(cuda_device, T):
    """Few tokens, forward and backward: a depth and a width that do not divide
    evenly over the blocks that share them, and ones that do."""
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward
    for kind, act, D, F in (("bf16", "silu", 1544, 2056), ("fp16", "gelu", 2048, 1024)):
        c = _case(cuda_device, T, D, F, kind, T)
        for save in (None, "16bit", "8bit"):
            y, kept = gated_ffn(c["x"], c["w"], c["wd"], act=act, save=save)
            _check_forward(c, kind, act, y, kept)
            if save:
                _check_backward(c, kind, act, gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, act=act), kept)


def test_large_and_deep(cuda_device):
    """More tiles than SMs in every product, a ragged edge on each axis."""
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward
    c = _case(cuda_device, 1501, 2056, 2568, "bf16", 5)
    y, kept = gated_ffn(c["x"], c["w"], c["wd"], save="16bit")
    _check_forward(c, "bf16", "silu", y, kept)
    _check_backward(c, "bf16", "silu", gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept), kept)


@pytest.mark.parametrize("T,D,F", [(200, 136, 8584), (257, 1032, 6152), (700, 64, 12288)])
def test_deep_and_narrow(cuda_device, T, D, F):
    """Few output tiles over a deep product: the depth is cut into slices whose
    sums are joined; repeated runs agree bit for bit."""
    import mhc_hyper_connection_gb300 as mp
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    assert mp.mhc_ffn_workspace_size(T, D, F)[1] > 256 + up(2 * T * F)      # room for the slices' sums
    assert mp.mhc_ffn_backward_workspace_size(T, D, F)[1] > 256 + up(4 * T * F) + up(2 * T * F)
    for kind, act in (("bf16", "silu"), ("fp16", "gelu")):
        c = _case(cuda_device, T, D, F, kind, T)
        y, kept = gated_ffn(c["x"], c["w"], c["wd"], act=act, save="16bit")
        _check_forward(c, kind, act, y, kept)
        got = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, act=act)
        _check_backward(c, kind, act, got, kept)
        for _ in range(5):
            y2, _ = gated_ffn(c["x"], c["w"], c["wd"], act=act, save="16bit")
            again = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, act=act)
            assert torch.equal(y, y2) and all(torch.equal(got[k], again[k]) for k in got)


def test_against_differences(cuda_device):
    """Central differences of <grad_y, y> in 64 bits, from the kept sums of the
    same inputs.  The kept sums are rounded to fp16 (u = 2^-11), which moves a
    gradient by about its curvature times u, and the kernels round three times
    more: 2^-7 of the largest gradient of each kind covers these and the
    difference's own step error (1e-4 squared)."""
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward
    for act in ("silu", "gelu"):
        c = _case(cuda_device, 6, 16, 24, "fp16", 3)
        _, kept = gated_ffn(c["x"], c["w"], c["wd"], act=act, save="16bit")
        got = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, act=act)
        v = {"grad_x": _f64(c["x"]), "grad_w_gate_up": _f64(c["w"]), "grad_w_down": _f64(c["wd"])}
        gy = _f64(c["gy"])
        loss = lambda: float((gy * ref.ffn(v["grad_x"], v["grad_w_gate_up"], v["grad_w_down"], act)[0]).sum())  # noqa: E731
        rng = np.random.RandomState(1)
        for k, a in v.items():
            flat, out = a.reshape(-1), _f64(got[k]).reshape(-1)
            for i in rng.choice(flat.size, 16, replace=False):
                keep = flat[i]
                flat[i] = keep + 1e-4
                up = loss()
                flat[i] = keep - 1e-4
                down = loss()
                flat[i] = keep
                assert abs((up - down) / 2e-4 - out[i]) <= 2.0 ** -7 * np.abs(out).max(), (act, k, i)


def test_no_tokens(cuda_device):
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward
    c = _case(cuda_device, 0, 64, 128, "bf16", 1)
    y, kept = gated_ffn(c["x"], c["w"], c["wd"], save="16bit")
    assert y.shape == (0, 64) and kept.shape == (0, 2, 128)
    grads = {"grad_x": torch.empty_like(c["x"]), "grad_w_gate_up": torch.ones_like(c["w"]),
             "grad_w_down": torch.ones_like(c["wd"])}
    gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, grads=grads)
    assert not grads["grad_w_gate_up"].any() and not grads["grad_w_down"].any()


@pytest.mark.parametrize("T", [5, 200])
def test_nonfinite_stays_in_its_token(cuda_device, T):
    """A NaN in one token's input reaches that token's y only, and an infinity
    beyond the matrix edges nothing (padding is not multiplied in)."""
    from mhc_hyper_connection_gb300 import gated_ffn
    c = _case(cuda_device, T, 72, 136, "bf16", 2)
    clean, _ = gated_ffn(c["x"], c["w"], c["wd"])
    c["x"][3, 71] = float("nan")
    y, kept = gated_ffn(c["x"], c["w"], c["wd"], save="8bit")
    keep = [t for t in range(T) if t != 3]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[3]).all()
    assert (kept.codes[3] == 0x7F).all()


def test_extreme_gates(cuda_device):
    """Gates far out on both sides: act tends to z and to 0 without NaN."""
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward
    for act in ("silu", "gelu"):
        c = _case(cuda_device, 4, 8, 8, "bf16", 4)
        c["x"].fill_(8.0)
        c["w"][0] = torch.linspace(-30, 30, 8, device=cuda_device)[:, None].expand(8, 8).bfloat16()
        y, kept = gated_ffn(c["x"], c["w"], c["wd"], act=act, save="16bit")
        assert torch.isfinite(y).all()
        got = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, act=act)
        assert all(torch.isfinite(v).all() for v in got.values())
        _check_backward(c, "bf16", act, got, kept)


@pytest.mark.parametrize("T", [9, 700])
def test_stream_layouts_given_outputs_and_repeats(cuda_device, T):
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward
    c = _case(cuda_device, T - T % 3, 256, 520, "fp16", 8)
    T -= T % 3
    y, kept = gated_ffn(c["x"], c["w"], c["wd"], act="gelu", save="8bit")
    g1 = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, act="gelu")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    lead = lambda t: t.reshape((3, T // 3) + t.shape[1:])  # noqa: E731
    y2 = torch.empty_like(lead(y))
    for _ in range(3):
        out, kept2 = gated_ffn(lead(c["x"]), c["w"], c["wd"], act="gelu", save="8bit", y=y2, stream=st)
        g2 = gated_ffn_backward(lead(c["gy"]), lead(c["x"]), c["w"], c["wd"], kept2, act="gelu", stream=st)
        torch.cuda.synchronize()
        assert out is y2 and torch.equal(y2.reshape(y.shape), y)
        assert torch.equal(kept2.codes.reshape(kept.codes.shape), kept.codes)
        for k in g1:
            assert torch.equal(g1[k].reshape(-1), g2[k].reshape(-1)), k


def test_graph_replay(cuda_device):
    """Capture into a CUDA graph and replay on new inputs: bit for bit an eager run."""
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward
    for T in (4, 300):
        c = _case(cuda_device, T, 256, 520, "bf16", 9)

        def step():
            y, kept = gated_ffn(c["x"], c["w"], c["wd"], save="8bit")
            return y, gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step()
        torch.cuda.current_stream().wait_stream(st)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, g = step()
        c["x"].copy_(torch.randn_like(c["x"]))
        graph.replay()
        torch.cuda.synchronize()
        y, g = y.clone(), {k: v.clone() for k, v in g.items()}
        ye, ge = step()
        assert torch.equal(y, ye) and all(torch.equal(g[k], ge[k]) for k in g)


@pytest.mark.parametrize("T", [4, 300])
def test_wait_that_gives_up_is_reported(cuda_device, T):
    """A withheld copy: the waits on it run out, the status says so, and the
    next call on the same buffers is whole again."""
    import mhc_hyper_connection_gb300 as mp
    c = _case(cuda_device, T, 256, 520, "bf16", 10)
    ws = mp.gated_ffn_workspace(T, 256, 520, cuda_device, backward=True)
    y, kept = mp.gated_ffn(c["x"], c["w"], c["wd"], save="16bit")
    grads = mp.gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, workspace=ws)
    for withhold in (1, 0):
        a = mp.MhcFfnArgs()
        a.T, a.D, a.F = T, 256, 520
        out = torch.zeros_like(y)
        a.x, a.w_gate_up, a.w_down, a.y = (t.data_ptr() for t in (c["x"], c["w"], c["wd"], out))
        a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
        a.wait_limit_us, a.withhold_copy = 20000, withhold
        assert mp.mhc_ffn_run(a, torch.cuda.current_stream().cuda_stream) == mp.MHC_OK
        assert mp.gated_ffn_status(ws) == (mp.MHC_ERR_RUNTIME if withhold else mp.MHC_OK)
        b = mp.MhcFfnBwdArgs()
        b.T, b.D, b.F = T, 256, 520
        b.grad_y, b.x, b.w_gate_up, b.w_down, b.gate_up = (t.data_ptr() for t in (c["gy"], c["x"], c["w"], c["wd"], kept))
        g2 = {k: torch.zeros_like(v) for k, v in grads.items()}
        b.grad_x, b.grad_w_gate_up, b.grad_w_down = (g2[k].data_ptr() for k in ("grad_x", "grad_w_gate_up", "grad_w_down"))
        b.workspace, b.workspace_bytes, b.wait_limit_us, b.withhold_copy = ws.data_ptr(), ws.numel(), 20000, withhold
        assert mp.mhc_ffn_backward_run(b, torch.cuda.current_stream().cuda_stream) == mp.MHC_OK
        assert mp.gated_ffn_status(ws) == (mp.MHC_ERR_RUNTIME if withhold else mp.MHC_OK)
    assert torch.equal(out, y) and all(torch.equal(g2[k], grads[k]) for k in grads)


def test_refusals(cuda_device):
    from mhc_hyper_connection_gb300 import MhcError, gated_ffn, gated_ffn_backward
    c = _case(cuda_device, 4, 64, 128, "bf16", 1)
    x, w, wd, gy, gu = c["x"], c["w"], c["wd"], c["gy"], c["gu"]
    for args in ((x.float(), w, wd), (x, w.half(), wd), (x, w, wd.half()), (x, w[:1], wd), (x, w, wd.t().contiguous()),
                 (x[:, :32].contiguous(), w, wd), (x.t(), w, wd), (x, w.cpu(), wd)):
        with pytest.raises(ValueError):
            gated_ffn(*args)
    for kw in ({"act": "relu"}, {"save": "4bit"}, {"kept": gu}, {"y": x.half()}):
        with pytest.raises(ValueError):
            gated_ffn(x, w, wd, **kw)
    with pytest.raises(MhcError):
        gated_ffn(x, w, wd, workspace=torch.zeros(256, dtype=torch.uint8, device=cuda_device))
    with pytest.raises(MhcError):
        gated_ffn(x[:, :60].contiguous(), w[:, :, :60].contiguous(), wd[:60].contiguous())
    for args in ((gy.half(), x, w, wd, gu), (gy, x, w, wd, gu[:, :1]), (gy, x, w, wd, gu.half()), (gy[:2], x, w, wd, gu)):
        with pytest.raises(ValueError):
            gated_ffn_backward(*args)


def test_new_outputs_on_another_stream_wait_for_their_memory(cuda_device):
    """A call on another stream than torch's current one gets memory that the
    current stream was still writing: its results must not be overwritten."""
    from mhc_hyper_connection_gb300 import gated_ffn, hc_post_backward
    from mhc_synth import make_post_case
    c = _case(cuda_device, 64, 256, 520, "bf16", 12)
    want, _ = gated_ffn(c["x"], c["w"], c["wd"])
    pc = make_post_case(device=cuda_device, T=64, n=4, D=256, seed=2)
    g = pc.residual.clone()
    want_b = hc_post_backward(g, pc.x, pc.residual, pc.post, pc.comb)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    big = torch.empty((1 << 28,), device=cuda_device)
    for _ in range(4):
        for _ in range(10):
            big.fill_(1.0)                       # the current stream is behind by a millisecond
        del_me = [torch.empty_like(want) for _ in range(4)] + [torch.empty_like(g), torch.empty_like(pc.post)]
        for t in del_me:
            t.fill_(float("nan"))                # queued writes to memory that is now freed
        del t, del_me
        y, _ = gated_ffn(c["x"], c["w"], c["wd"], stream=st)
        b = hc_post_backward(g, pc.x, pc.residual, pc.post, pc.comb, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and all(torch.equal(b[k], want_b[k]) for k in b)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [1, 130])
def test_gates_whose_square_overflows(cuda_device, T, act):
    """Gates up to the type's largest values: the derivative is 1 and 0 there,
    not 0 times an overflowed square.  One value of grad_y is not zero, so ga is
    one exact product; gg and the gradient are then rounded to bf16 once each."""
    from mhc_hyper_connection_gb300 import gated_ffn_backward
    c = _case(cuda_device, T, 8, 8, "bf16", 5)
    z = torch.tensor([1e10, -1e10, 2e19, -2e19, 1e25, -1e25, 3e38, -3e38], device=cuda_device).bfloat16()
    kept = torch.empty((T, 2, 8), device=cuda_device, dtype=torch.bfloat16)
    kept[:, 0] = z
    kept[:, 1] = 0.5
    c["gy"].zero_()
    c["gy"][0, 3] = 1.0
    c["wd"][3] = 2.0 ** -20                      # ga z and grad_x stay finite
    got = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, act=act)
    assert all(torch.isfinite(v).all() for v in got.values())
    gg = np.where(_f64(z) > 0, 0.5 * 2.0 ** -20, 0.0)
    want = gg[:, None] * _f64(c["x"])[0]
    _near(got["grad_w_gate_up"][0], want, 1.01 * 2.0 ** -8 * np.abs(want), "grad_w_gate_up")


@pytest.mark.parametrize("T", [1, 16, 33, 64, 65, 80, 100, 128])
@pytest.mark.parametrize("D,F", [(768, 1280), (1280, 1536), (1792, 768)])
def test_few_tokens_in_clusters_of_every_size(cuda_device, T, D, F):
    """Depths of 12, 20, 24 and 28 chunks: blocks in clusters of 3, 5, 6 and 7,
    whose shares of the tokens are not equal."""
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward, gated_ffn_status
    c = _case(cuda_device, T, D, F, "bf16", T + D)
    y, kept = gated_ffn(c["x"], c["w"], c["wd"], save="8bit")
    _check_forward(c, "bf16", "silu", y, kept)
    got = gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept)
    assert gated_ffn_status() == 0
    _check_backward(c, "bf16", "silu", got, kept)


@pytest.mark.parametrize("T,D,F", [(300, 64, 10240), (300, 10040, 72), (769, 72, 4104), (420, 7112, 136)])
def test_tiles_of_three_quarters(cuda_device, T, D, F):
    """Sizes at which tiles 192 wide take the fewest rounds: many columns, few
    rows, in the gate gradients (wide F) or in the down product (wide D)."""
    from mhc_hyper_connection_gb300 import gated_ffn, gated_ffn_backward
    for kind, act in (("bf16", "silu"), ("fp16", "gelu")):
        c = _case(cuda_device, T, D, F, kind, T + 1)
        for save in ("16bit", "8bit"):
            y, kept = gated_ffn(c["x"], c["w"], c["wd"], act=act, save=save)
            _check_forward(c, kind, act, y, kept)
            _check_backward(c, kind, act, gated_ffn_backward(c["gy"], c["x"], c["w"], c["wd"], kept, act=act), kept)


def test_slices_of_three_quarter_tiles(cuda_device):
    """A deep down product whose slices are 192 wide."""
    from mhc_hyper_connection_gb300 import gated_ffn
    c = _case(cuda_device, 824, 136, 15104, "bf16", 3)
    y, kept = gated_ffn(c["x"], c["w"], c["wd"])
    _check_forward(c, "bf16", "silu", y, kept)
