"""Measured cases of the operators that train and serve one hyper-connection layer.

A layer maps its n residual streams to one input (the pre-mapping), runs a
gated feed-forward block on it and maps the result back into the streams (the
post-mapping).  The operators here are what training that layer takes next to
the pre-mapping, and what serving it takes for a few tokens:

  ckpt       the 8-bit checkpoint of 16-bit activations, written and read back
  post_ckpt  the post-mapping that writes the checkpoint of its output streams
             in the same pass, and the reading back
  post_bwd   the post-mapping's backward, its residual streams kept in 16 bits
             or in a checkpoint
  ffn_fwd    the gated feed-forward block, gate and up sums kept or not
  ffn_bwd    its backward from the kept sums
  ffn_step   forward and backward with the sums kept in 8 bits

8-bit form: each row is cut into blocks of 128 columns (the last may be
shorter); a block has one exponent e, the smallest with amax <= 448 2^e inside
the range that makes every value exact in the 16-bit type again, and holds
e4m3 codes of x 2^-e, ties to even, capped at 448.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ERANGE = {"bf16": (-100, 119), "fp16": (-15, 7)}   # exponents of a block's scale
BLOCK = 128


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode batch of streams parked in 8 bits: latency counts
        dict(name="ckpt_decode", op="ckpt", T=64, n=4, D=7168, dtype="bf16"),
        # the streams entering one layer of a long training batch
        dict(name="ckpt_streams", op="ckpt", T=8192, n=4, D=7168, dtype="bf16"),
        # post-mapping of a training batch whose output the next layer checkpoints
        dict(name="post_ckpt_train", op="post_ckpt", T=4096, n=4, D=4096),
        # ragged token count, eight streams, a last block of eight columns
        dict(name="post_ckpt_ragged", op="post_ckpt", T=1021, n=8, D=2056),
        # backward of the post-mapping at the largest batch
        dict(name="post_bwd_large", op="post_bwd", T=32768, n=4, D=7168, ckpt=False),
        # the same from a checkpoint, eight streams
        dict(name="post_bwd_ckpt", op="post_bwd", T=16384, n=8, D=2048, ckpt=True),
        # a smallest training call: launch and latency
        dict(name="post_bwd_tiny", op="post_bwd", T=64, n=4, D=256, ckpt=False),
        # serving one token: the weights are read once
        dict(name="ffn_token", op="ffn_fwd", T=1, D=7168, F=8192, act="silu", dtype="bf16", save=False),
        # serving a batch of tokens
        dict(name="ffn_decode", op="ffn_fwd", T=24, D=4096, F=8192, act="gelu", dtype="fp16", save=False),
        # training forward that keeps gate and up in 16 bits
        dict(name="ffn_forward", op="ffn_fwd", T=4096, D=4096, F=8192, act="silu", dtype="bf16", save=True),
        # backward on a ragged batch and a width that fills no tile
        dict(name="ffn_bwd_ragged", op="ffn_bwd", T=1021, D=2048, F=5512, act="gelu", dtype="fp16"),
        # one training step of the block, gate and up kept in 8 bits: the largest work
        dict(name="ffn_step_8bit", op="ffn_step", T=4096, D=4096, F=8192, act="silu", dtype="bf16"),
    ]


MOST_STREAMS = 32768 * 4 * 7168          # elements of the largest stream tensor
MOST_FFN = 4096 * 4096 * 8192            # T D F of the largest block


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], spread over its logarithm, a multiple of step."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        v = max(step, v // step * step)
        if v != 3072:
            return v


def draw(rng):
    op = rng.choice(["ckpt", "post_ckpt", "post_bwd", "ffn_fwd", "ffn_bwd", "ffn_step"])
    if op in ("ckpt", "post_ckpt", "post_bwd"):
        n = rng.choice([1, 2, 4, 4, 6, 8])
        D = _log(rng, 64, 8192, 8)
        T = _log(rng, 1, min(32768, MOST_STREAMS // (n * D)))
        c = dict(op=op, T=T, n=n, D=D)
        if op == "ckpt":
            c["dtype"] = rng.choice(["bf16", "fp16"])
        if op == "post_bwd":
            c["ckpt"] = rng.random() < 0.5
        return c
    D = _log(rng, 128, 8192, 8)
    F = _log(rng, 128, 16384, 8)
    T = _log(rng, 1, max(1, min(8192, MOST_FFN // (D * F))))
    c = dict(op=op, T=T, D=D, F=F, act=rng.choice(["silu", "gelu"]), dtype=rng.choice(["bf16", "fp16"]))
    if op == "ffn_fwd":
        c["save"] = rng.random() < 0.5
    return c


def work(case):
    c, op, T, D = case, case["op"], case["T"], case["D"]
    if op == "ckpt":
        rows, blocks = T * c["n"], -(-D // BLOCK)
        return {"bytes": rows * (6 * D + 2 * blocks), "flops": 6 * rows * D}
    if op == "post_ckpt":
        n, blocks = c["n"], -(-D // BLOCK)
        coef = 4 * T * (n + n * n)
        # x, streams in; streams out; the checkpoint written and read; the streams restored
        return {"bytes": 2 * T * D * (1 + 2 * n) + coef + T * n * (2 * D + 2 * blocks + 2 * D),
                "flops": 2 * T * D * (n + n * n)}
    if op == "post_bwd":
        n = c["n"]
        res = T * n * (D + -(-D // BLOCK)) if c["ckpt"] else 2 * T * n * D
        return {"bytes": 2 * T * n * D + 2 * T * D + res + 2 * T * D + 2 * T * n * D + 8 * T * (n + n * n),
                "flops": 4 * T * D * (n + n * n)}
    F = c["F"]
    weights = 2 * 3 * D * F
    kept = 2 * T * 2 * F
    if op == "ffn_fwd":
        return {"bytes": weights + 4 * T * D + (kept if c["save"] else 0), "flops": 6 * T * D * F}
    if op == "ffn_bwd":
        return {"bytes": 2 * weights + 6 * T * D + kept, "flops": 12 * T * D * F}
    return {"bytes": 2 * weights + 8 * T * D, "flops": 18 * T * D * F}


# ----------------------------------------------------------------- the inputs

def _streams(gen, shape, dtype):
    """Residual streams: unit scale, one column in a hundred twenty times larger."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    big = torch.rand(shape[-1], generator=gen, device="cuda") < 0.01
    return x.mul_(torch.where(big, 20.0, 1.0).to(dtype))


def _mixes(gen, T, n):
    """Post-mapping weights: gates in (0, 2), a mix whose rows sum to one."""
    post = 2 * torch.sigmoid(torch.randn((T, n), generator=gen, device="cuda"))
    comb = torch.softmax(torch.randn((T, n, n), generator=gen, device="cuda"), -1)
    return post, comb.contiguous()


def prepare(case, seed):
    c, op, T, D = case, case["op"], case["T"], case["D"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[c.get("dtype", "bf16")]
    rn = lambda *shape, scale=1.0: torch.randn(shape, generator=gen, device="cuda", dtype=dt).mul_(scale)  # noqa: E731
    s = dict(case=dict(c))
    if op == "ckpt":
        s["x"] = _streams(gen, (T, c["n"], D), dt)
        return s
    if op in ("post_ckpt", "post_bwd"):
        n = c["n"]
        s["x"], s["residual"] = rn(T, D), _streams(gen, (T, n, D), dt)
        s["post"], s["comb"] = _mixes(gen, T, n)
        if op == "post_bwd":
            s["grad_out"] = rn(T, n, D, scale=2.0 ** -6)
            if c["ckpt"]:
                s["codes"], s["scales"] = _pack(s.pop("residual"), "bf16")
        return s
    F = c["F"]
    s["x"] = rn(T, D)
    s["w_gate_up"] = rn(2, F, D, scale=D ** -0.5)
    s["w_down"] = rn(D, F, scale=F ** -0.5)
    if op != "ffn_fwd":
        s["grad_y"] = rn(T, D, scale=2.0 ** -3)
    if op == "ffn_bwd":
        s["gate_up"] = rn(T, 2, F)
    return s


# ------------------------------------------------------------ the plain forms

def _pow2(e):
    """2^e in 32 bits from whole exponents in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _blocks(x):
    """[..., D] as [..., blocks, 128], filled up with zeros."""
    D = x.shape[-1]
    pad = -D % BLOCK
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[:-1] + (pad,))], -1)
    return x.reshape(x.shape[:-1] + (-1, BLOCK))


def _pack(x, kind):
    """(codes uint8 [..., D], scales uint8 [..., blocks]: exponent + 127) of 32-bit or 16-bit x."""
    lo, hi = ERANGE[kind]
    b = _blocks(x.float())
    fine = torch.isfinite(b)
    amax = torch.where(fine, b.abs(), torch.zeros_like(b)).amax(-1)
    m, k = torch.frexp(amax)                             # amax = m 2^k, m in [1/2, 1)
    e = torch.where(m <= 0.875, k - 9, k - 8)            # 448 = 0.875 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, lo)).clamp(lo, hi)
    q = (b * _pow2(-e)[..., None]).clamp(-448.0, 448.0)
    codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where(fine, codes, torch.full_like(codes, 0x7F))
    D = x.shape[-1]
    codes = codes.reshape(codes.shape[:-2] + (-1,))[..., :D].contiguous()
    return codes, (e + 127).to(torch.uint8)


def _unpack(codes, scales):
    """The 32-bit values that codes and scales stand for."""
    D = codes.shape[-1]
    v = codes.view(torch.float8_e4m3fn).float()
    s = _pow2(scales.to(torch.int32) - 127).repeat_interleave(BLOCK, -1)[..., :D]
    return v * s


def _post(s):
    """The post-mapping in 32 bits."""
    return s["post"][..., None] * s["x"].float()[:, None] + torch.matmul(s["comb"].transpose(1, 2), s["residual"].float())


def _post_bwd(s):
    g, x = s["grad_out"].float(), s["x"].float()
    res = _unpack(s["codes"], s["scales"]) if "codes" in s else s["residual"].float()
    return {"grad_x": (s["post"][..., None] * g).sum(1).bfloat16(),
            "grad_residual": torch.matmul(s["comb"], g).bfloat16(),
            "grad_post": (g * x[:, None]).sum(-1),
            "grad_comb": torch.matmul(res, g.transpose(1, 2))}


C0 = math.sqrt(2.0 / math.pi)


def _act(z, act):
    """The activation and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    t = torch.tanh(C0 * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * C0 * (1.0 + 3 * 0.044715 * z * z)


def _ffn_sums(s):
    x, w = s["x"].float(), s["w_gate_up"].float()
    return torch.matmul(x, w[0].t()), torch.matmul(x, w[1].t())


def _ffn_bwd(s, g, u, dt):
    x, w, wd, gy = s["x"].float(), s["w_gate_up"].float(), s["w_down"].float(), s["grad_y"].float()
    h, dh = _act(g, s["case"]["act"])
    a = h * u
    ga = torch.matmul(gy, wd)
    gg, gu = ga * u * dh, ga * h
    return {"grad_x": (torch.matmul(gg, w[0]) + torch.matmul(gu, w[1])).to(dt),
            "grad_w_gate_up": torch.stack([torch.matmul(gg.t(), x), torch.matmul(gu.t(), x)]).to(dt),
            "grad_w_down": torch.matmul(gy.t(), a).to(dt)}


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    dt = DTYPES[c.get("dtype", "bf16")]
    if op == "ckpt":
        return {"restored": _unpack(*_pack(s["x"], c["dtype"])).to(dt)}
    if op == "post_ckpt":
        out = _post(s).bfloat16()
        return {"out": out, "restored": _unpack(*_pack(out, "bf16")).bfloat16()}
    if op == "post_bwd":
        return _post_bwd(s)
    if op == "ffn_bwd":
        return _ffn_bwd(s, s["gate_up"][:, 0].float(), s["gate_up"][:, 1].float(), dt)
    g, u = _ffn_sums(s)
    y = torch.matmul(_act(g, c["act"])[0] * u, s["w_down"].float().t()).to(dt)
    if op == "ffn_fwd":
        return {"y": y, "gate_up": torch.stack([g, u], 1).to(dt)} if c["save"] else {"y": y}
    kept = torch.stack([_unpack(*_pack(v, c["dtype"])) for v in (g, u)])
    return {"y": y, **_ffn_bwd(s, kept[0], kept[1], dt)}


# --------------------------------------------------------- the user's program

def _own(s):
    import mhc_hyper_connection_gb300 as mhc
    c, op = s["case"], s["case"]["op"]
    if op == "ckpt":
        return {"restored": mhc.ckpt8_restore(mhc.ckpt8_pack(s["x"]), dtype=s["x"].dtype)}
    if op == "post_ckpt":
        out, ckpt = mhc.hc_post_ckpt(s["x"], s["residual"], s["post"], s["comb"])
        return {"out": out, "restored": mhc.ckpt8_restore(ckpt, dtype=out.dtype)}
    if op == "post_bwd":
        residual = mhc.Ckpt8(s["codes"], s["scales"]) if c["ckpt"] else s["residual"]
        return mhc.hc_post_backward(s["grad_out"], s["x"], residual, s["post"], s["comb"])
    if op == "ffn_bwd":
        return mhc.gated_ffn_backward(s["grad_y"], s["x"], s["w_gate_up"], s["w_down"], s["gate_up"], act=c["act"])
    if op == "ffn_fwd":
        y, kept = mhc.gated_ffn(s["x"], s["w_gate_up"], s["w_down"], act=c["act"], save="16bit" if c["save"] else None)
        return {"y": y, "gate_up": kept} if c["save"] else {"y": y}
    y, kept = mhc.gated_ffn(s["x"], s["w_gate_up"], s["w_down"], act=c["act"], save="8bit")
    return {"y": y, **mhc.gated_ffn_backward(s["grad_y"], s["x"], s["w_gate_up"], s["w_down"], kept, act=c["act"])}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------- in 64 bits

def _exact_8bit(v, kind):
    """What the 8-bit form of v holds, from its definition: a grid of step
    2^(floor(log2 |v 2^-e|) - 3), at least 2^-9, ties to even."""
    lo, hi = ERANGE[kind]
    D = v.shape[-1]
    out = torch.empty_like(v)
    for b0 in range(0, D, BLOCK):
        w = v[..., b0:b0 + BLOCK]
        ok = torch.isfinite(w)
        top = torch.where(ok, w.abs(), 0.0).amax(-1, keepdim=True)
        e = torch.ceil(torch.log2((top / 448.0).clamp_min(2.0 ** -200)))
        e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)      # the logarithm's own rounding
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e).clamp(lo, hi)
        q = (w / torch.exp2(e)).clamp(-448.0, 448.0)
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
        out[..., b0:b0 + BLOCK] = torch.where(ok, torch.round(q / step) * step * torch.exp2(e), math.nan)
    return out


def _exact_post(c, s):
    T, n = c["T"], c["n"]
    x, post, comb = s["x"].double(), s["post"].double(), s["comb"].double()
    if c["op"] == "post_ckpt":
        out = torch.stack([sum((comb[:, i, j, None] * s["residual"][:, i].double() for i in range(n)),
                               post[:, j, None] * x) for j in range(n)], 1)
        return {"out": out, "restored": _exact_8bit(out.bfloat16().double(), "bf16")}
    got = {"grad_x": torch.zeros_like(x), "grad_residual": torch.zeros((T, n, c["D"]), dtype=torch.float64, device="cuda"),
           "grad_post": torch.empty_like(post), "grad_comb": torch.empty_like(comb)}
    for i in range(n):
        if c["ckpt"]:
            v = s["codes"][:, i].to(torch.int32)
            p, m = (v >> 3) & 15, (v & 7).double()
            mag = torch.where(p > 0, torch.exp2(p.double() - 7) * (1 + m / 8), m * 2.0 ** -9)
            mag = torch.where((v & 127) == 127, math.nan, mag) * torch.where(v > 127, -1.0, 1.0)
            sc = torch.exp2(s["scales"][:, i].double() - 127)
            res = mag * sc[:, torch.arange(c["D"], device="cuda") // BLOCK]
        else:
            res = s["residual"][:, i].double()
        for j in range(n):
            g = s["grad_out"][:, j].double()
            got["grad_residual"][:, i] += comb[:, i, j, None] * g
            got["grad_comb"][:, i, j] = (res * g).sum(-1)
            if i == 0:
                got["grad_x"] += post[:, j, None] * g
                got["grad_post"][:, j] = (x * g).sum(-1)
    return got


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "ckpt":
        return {"restored": _exact_8bit(s["x"].double(), c["dtype"])}
    if op in ("post_ckpt", "post_bwd"):
        return _exact_post(c, s)
    x, wg, wu, wd = s["x"].double(), s["w_gate_up"][0].double(), s["w_gate_up"][1].double(), s["w_down"].double()

    def act(z):
        return z / (1 + torch.exp(-z)) if c["act"] == "silu" else z / (1 + torch.exp(-2 * C0 * z * (1 + 0.044715 * z ** 2)))

    got = {}
    if op == "ffn_bwd":
        g, u = s["gate_up"][:, 0].double(), s["gate_up"][:, 1].double()
    else:
        g, u = x @ wg.T, x @ wu.T
        got["y"] = (act(g) * u) @ wd.T
        if op == "ffn_fwd":
            if c["save"]:
                got["gate_up"] = torch.stack([g, u], 1)
            return got
        g, u = _exact_8bit(g, c["dtype"]), _exact_8bit(u, c["dtype"])
    if c["act"] == "silu":
        slope = 1 / (1 + torch.exp(-g)) + g * torch.exp(-g.abs()) / (1 + torch.exp(-g.abs())) ** 2
    else:
        r = 2 * C0 * g * (1 + 0.044715 * g ** 2)          # gelu(z) = z sigmoid(r(z))
        slope = 1 / (1 + torch.exp(-r)) + g * torch.exp(-r.abs()) / (1 + torch.exp(-r.abs())) ** 2 * 2 * C0 * (1 + 3 * 0.044715 * g ** 2)
    gy = s["grad_y"].double()
    ga = gy @ wd
    gg, gu = ga * u * slope, ga * act(g)
    got["grad_x"] = gg @ wg + gu @ wu
    got["grad_w_gate_up"] = torch.stack([gg.T @ x, gu.T @ x])
    got["grad_w_down"] = gy.T @ (act(g) * u)
    return got
