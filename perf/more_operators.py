"""Measured cases of the operators that give a layer routed experts.

A layer's body may be several feed-forward blocks ("experts") of which every
token takes a few.  Training and serving such a body takes, next to the
mappings and the single block:

  route         experts and weights of every token from its router scores:
                softmax or sigmoid, a bias that only steers the choice, groups,
                top-k, renormalised weights
  route_bwd     the gradient of the weights carried back to the scores
  experts       the chosen experts' gated feed-forward blocks and the weighted
                sum of their outputs
  experts_step  a training step of the body: routing, experts, all gradients
  orthogonalise the weight matrices' update made orthogonal by Newton-Schulz
                products, one matrix or as many as there are experts

A score of -inf takes an expert out of a token's choice; a token all of whose
scores are -inf (a padded row) takes none: its slots hold expert -1, weight 0,
and its output row is 0.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
STEPS = ((3.4445, -4.7750, 2.0315),) * 5           # (a, b, c): X <- a X + (b A + c A A) X, A = X X^T
EPS = 1e-7
C0 = math.sqrt(2.0 / math.pi)


# ------------------------------------------------------------------ the cases

def listed():
    sig = dict(score="sigmoid", bias=True, groups=8, top_groups=4, renorm=True, scale=2.5)
    soft = dict(score="softmax", bias=False, groups=1, top_groups=1, renorm=True, scale=1.0)
    return [
        # one decode batch through a router with groups: latency counts
        dict(name="route_decode", op="route", T=8, E=256, k=8, dtype="fp32", pad=0.0, **sig),
        # the prompts of a serving batch, an eighth of it padding
        dict(name="route_prefill", op="route", T=16384, E=256, k=8, dtype="fp32", pad=0.125, **sig),
        # the router's gradient on a training batch, weights renormalised
        dict(name="route_bwd_train", op="route_bwd", T=8192, E=128, k=8, dtype="fp32", pad=0.0, **soft),
        # sixteen-bit scores, an odd number of experts and tokens, plain softmax weights
        dict(name="route_bwd_ragged", op="route_bwd", T=1021, E=60, k=4, dtype="bf16", pad=0.1,
             score="softmax", bias=False, groups=1, top_groups=1, renorm=False, scale=1.0),
        # serving one token: the weights of its experts are read once
        dict(name="experts_token", op="experts", T=1, E=64, k=8, D=4096, F=2048, act="silu", dtype="bf16", pad=0.0),
        # serving a batch of tokens: most experts have a few of them
        dict(name="experts_decode", op="experts", T=64, E=64, k=6, D=2048, F=1408, act="gelu", dtype="fp16", pad=0.0),
        # the prompts of a serving batch
        dict(name="experts_prefill", op="experts", T=4096, E=64, k=8, D=4096, F=2048, act="silu", dtype="bf16", pad=0.0),
        # training step on a ragged batch with padding, widths that fill no tile
        dict(name="experts_step_ragged", op="experts_step", T=1021, E=12, k=3, D=1032, F=1160, act="gelu", dtype="fp16",
             pad=0.1, **soft),
        # training step of a large batch: the largest work
        dict(name="experts_step_train", op="experts_step", T=8192, E=32, k=4, D=4096, F=2048, act="silu", dtype="bf16",
             pad=0.0, **dict(sig, groups=4, top_groups=2)),
        # a small matrix of odd sizes
        dict(name="orthogonalise_small", op="orthogonalise", B=1, m=515, n=259, dtype="fp32"),
        # the momenta of one weight of every expert, taller than wide
        dict(name="orthogonalise_experts", op="orthogonalise", B=32, m=2816, n=1024, dtype="bf16"),
        # the momentum of a large block's weight
        dict(name="orthogonalise_block", op="orthogonalise", B=1, m=4096, n=8192, dtype="fp32"),
    ]


MOST_SCORES = 16384 * 256                # T E of the largest routing
MOST_ROWS = 8192 * 4 * 4096 * 2048       # T k D F of the largest experts
MOST_WEIGHTS = 64 * 4096 * 2048          # E D F of the most weights
MOST_ORTH = 4096 * 4096 * 8192           # B min(m, n)^2 max(m, n) of the largest orthogonalisation


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], spread over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))
    return max(step, v // step * step)


def _router(rng, E):
    groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
    return dict(score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                top_groups=rng.randint(max(1, groups // 2), groups), renorm=rng.random() < 0.7,
                scale=rng.choice([1.0, 2.5]))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "experts", "experts_step", "orthogonalise"])
    if op in ("route", "route_bwd"):
        E = rng.choice([8, 16, 24, 60, 64, 72, 128, 160, 256, 384, 512])
        r = _router(rng, E)
        k = rng.randint(1, min(8, E // r["groups"] * r["top_groups"]))
        r["renorm"] = r["renorm"] and k > 1                      # one renormalised weight has no gradient
        T = _log(rng, 1, MOST_SCORES // max(E, 128))
        return dict(op=op, T=T, E=E, k=k, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    pad=rng.choice([0.0, 0.1]), **r)
    if op == "orthogonalise":
        m, n = _log(rng, 16, 8192), _log(rng, 16, 8192)
        while min(m, n) ** 2 * max(m, n) > MOST_ORTH:
            m, n = _log(rng, 16, 8192), _log(rng, 16, 8192)
        B = _log(rng, 1, max(1, min(32, MOST_ORTH // (min(m, n) ** 2 * max(m, n)))))
        return dict(op=op, B=B, m=m, n=n, dtype=rng.choice(["fp32", "bf16"]))
    E = rng.choice([4, 8, 12, 16, 32, 60, 64, 128])
    D, F = _log(rng, 128, 4096, 8), _log(rng, 128, 4096, 8)
    while E * D * F > MOST_WEIGHTS:
        D, F = _log(rng, 128, 4096, 8), _log(rng, 128, 4096, 8)
    r = _router(rng, E)
    k = rng.randint(1, min(8, E // r["groups"] * r["top_groups"]))
    r["renorm"] = r["renorm"] and k > 1
    T = _log(rng, 1, max(1, min(8192, MOST_ROWS // (k * D * F))))
    c = dict(op=op, T=T, E=E, k=k, D=D, F=F, act=rng.choice(["silu", "gelu"]), dtype=rng.choice(["bf16", "fp16"]),
             pad=rng.choice([0.0, 0.1]))
    return dict(c, **r) if op == "experts_step" else c


def work(case):
    c, op = case, case["op"]
    if op == "orthogonalise":
        m, n = min(c["m"], c["n"]), max(c["m"], c["n"])
        # A and A A are symmetric: half of each is enough
        flops = len(STEPS) * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)
        return {"bytes": c["B"] * m * n * (DTYPES[c["dtype"]].itemsize + 2), "flops": c["B"] * flops}
    T, E, k = c["T"], c["E"], c["k"]
    if op in ("route", "route_bwd"):
        scores = T * E * DTYPES[c["dtype"]].itemsize
        return {"bytes": scores + 8 * T * k if op == "route" else 2 * scores + 8 * T * k, "flops": 8 * T * E}
    D, F = c["D"], c["F"]
    active = E * (1.0 - (1.0 - k / E) ** T)          # experts that some token takes, if all are taken alike
    weights = int(active * 3 * D * F * 2)
    if op == "experts":
        return {"bytes": weights + 4 * T * D + 8 * T * k, "flops": 6 * T * k * D * F}
    return {"bytes": weights + 6 * E * D * F + 8 * T * D + 4 * T * E, "flops": 18 * T * k * D * F}


# ----------------------------------------------------------------- the inputs

def _scores(gen, c):
    """Router scores: unit scale, some experts liked more; padded rows -inf."""
    T, E = c["T"], c["E"]
    l = torch.randn((T, E), generator=gen, device="cuda") + 0.5 * torch.randn((E,), generator=gen, device="cuda")
    if c["pad"]:
        l[torch.rand((T,), generator=gen, device="cuda") < c["pad"]] = -math.inf
    return l


def prepare(case, seed):
    c, op = case, case["op"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case=dict(c))
    if op == "orthogonalise":
        # a momentum: noise and a few strong directions
        B, m, n = c["B"], c["m"], c["n"]
        r = min(8, m, n)
        u = torch.randn((B, m, r), generator=gen, device="cuda")
        v = torch.randn((B, r, n), generator=gen, device="cuda")
        g = torch.randn((B, m, n), generator=gen, device="cuda")
        s["update"] = ((g + torch.matmul(u, v) * r ** -0.5) * 2.0 ** -8).to(DTYPES[c["dtype"]])
        return s
    if op in ("route", "route_bwd"):
        s["logits"] = _scores(gen, c).to(DTYPES[c["dtype"]])
        s["bias"] = 0.05 * torch.randn((c["E"],), generator=gen, device="cuda") if c["bias"] else None
        if op == "route_bwd":
            s["experts"] = _route(s["logits"], s["bias"], c)[0]
            s["grad_weights"] = torch.randn((c["T"], c["k"]), generator=gen, device="cuda")
        return s
    T, E, D, F, dt = c["T"], c["E"], c["D"], c["F"], DTYPES[c["dtype"]]
    rn = lambda *shape, scale=1.0: torch.randn(shape, generator=gen, device="cuda", dtype=dt).mul_(scale)  # noqa: E731
    s["x"] = rn(T, D)
    s["w_gate_up"] = rn(E, 2, F, D, scale=D ** -0.5)
    s["w_down"] = rn(E, D, F, scale=F ** -0.5)
    logits = _scores(gen, c)
    if op == "experts":
        router = dict(c, score="softmax", groups=1, top_groups=1, renorm=True, scale=1.0)
        s["experts"], s["weights"] = _route(logits, None, router)
    else:
        s["logits"] = logits.to(dt)                  # a 16-bit product's
        s["bias"] = 0.05 * torch.randn((E,), generator=gen, device="cuda") if c["bias"] else None
        s["grad_y"] = rn(T, D, scale=2.0 ** -3)
    return s


# ------------------------------------------------------------ the plain forms

def _route(logits, bias, c):
    """(experts int32 [T, k], weights fp32 [T, k]).  Comparisons in 64 bits."""
    l = logits.double()
    T, E = l.shape
    k, groups = c["k"], c["groups"]
    out = l == -math.inf
    if c["score"] == "softmax":
        top = l.amax(-1, keepdim=True)
        p = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
        score = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    # without a bias the scores' order is that of the logits
    key = l if bias is None else score + bias.double()
    key = torch.where(out, torch.full_like(key, -math.inf), key)
    if groups > 1:
        # a group counts for the sum of its two best, a lone one for itself
        by = torch.where(out, torch.full_like(key, -math.inf), score if bias is None else key)
        best = by.reshape(T, groups, E // groups).topk(2, -1).values
        mark = torch.where(best[..., 1] == -math.inf, best[..., 0], best[..., 0] + best[..., 1])
        order = torch.sort(mark, dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros((T, groups), dtype=torch.bool, device=l.device).scatter_(1, order, True)
        key = torch.where(kept.repeat_interleave(E // groups, 1), key, torch.full_like(key, -math.inf))
    val, idx = torch.sort(key, dim=-1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    none = val == -math.inf
    w = torch.where(none, torch.zeros_like(val), score.gather(1, idx))
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
    experts = torch.where(none, torch.full_like(idx, -1), idx).int()
    return experts, (w * c["scale"]).float()


def _route_bwd(grad_weights, logits, experts, c):
    """The gradient of the scores from that of the weights, in 32 bits."""
    l, gw = logits.float(), grad_weights.float()
    none = experts < 0
    idx = experts.long().clamp_min(0)
    if c["score"] == "softmax":
        top = l.amax(-1, keepdim=True)
        p = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
        score = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    u = torch.where(none, torch.zeros_like(gw), score.gather(1, idx))
    gw = torch.where(none, torch.zeros_like(gw), gw) * c["scale"]
    slope = torch.ones_like(u) if c["score"] == "softmax" else 1.0 - u
    g = torch.zeros_like(l)
    if c["renorm"]:
        w = u / u.sum(-1, keepdim=True).clamp_min(1e-30)
        return g.scatter_add_(1, idx, w * (gw - (gw * w).sum(-1, keepdim=True)) * slope).to(logits.dtype)
    g.scatter_add_(1, idx, gw * u * slope)
    if c["score"] == "softmax":
        g = g - score * (gw * u).sum(-1, keepdim=True)
    return g.to(logits.dtype)


def _act(z, act):
    """The activation and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    t = torch.tanh(C0 * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * C0 * (1.0 + 3 * 0.044715 * z * z)


def _experts(s, experts, weights, grad_y=None):
    """The experts' outputs and, with grad_y, all gradients but the scores'; the
    backward takes the gate and up sums as they are kept, in 16 bits."""
    c, dt = s["case"], s["x"].dtype
    x = s["x"].float()
    y = torch.zeros_like(x)
    if grad_y is not None:
        gy, gx, gwt = grad_y.float(), torch.zeros_like(x), torch.zeros_like(weights)
        gwgu, gwd = torch.zeros_like(s["w_gate_up"]), torch.zeros_like(s["w_down"])
    for e in range(c["E"]):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        if not t.numel():
            continue
        w, xe = weights[t, j][:, None], x[t]
        wg, wu, wd = s["w_gate_up"][e, 0].float(), s["w_gate_up"][e, 1].float(), s["w_down"][e].float()
        g, u = torch.matmul(xe, wg.t()), torch.matmul(xe, wu.t())
        y.index_add_(0, t, w * torch.matmul(_act(g, c["act"])[0] * u, wd.t()))
        if grad_y is None:
            continue
        g, u = g.to(dt).float(), u.to(dt).float()
        h, dh = _act(g, c["act"])
        a, ga = h * u, torch.matmul(gy[t], wd)
        gwt[t, j] = (a * ga).sum(-1)
        ga = ga * w
        gg, gu = ga * u * dh, ga * h
        gx.index_add_(0, t, torch.matmul(gg, wg) + torch.matmul(gu, wu))
        gwgu[e, 0], gwgu[e, 1] = torch.matmul(gg.t(), xe).to(dt), torch.matmul(gu.t(), xe).to(dt)
        gwd[e] = torch.matmul((w * gy[t]).t(), a).to(dt)
    if grad_y is None:
        return {"y": y.to(dt)}
    return {"y": y.to(dt), "grad_x": gx.to(dt), "grad_weights": gwt, "grad_w_gate_up": gwgu, "grad_w_down": gwd}


def _orthogonalise(g):
    x = g.float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-2, -1)
    x = x / (x.double().square().sum((-2, -1), keepdim=True).sqrt().float() + EPS)
    for a, b, c in STEPS:
        p = torch.matmul(x, x.transpose(-2, -1))
        x = a * x + torch.matmul(b * p + c * torch.matmul(p, p), x)
    return (x.transpose(-2, -1) if tall else x).to(torch.bfloat16)


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "route":
        experts, weights = _route(s["logits"], s["bias"], c)
        return {"experts": experts, "weights": weights}
    if op == "route_bwd":
        return {"grad_logits": _route_bwd(s["grad_weights"], s["logits"], s["experts"], c)}
    if op == "experts":
        return _experts(s, s["experts"], s["weights"])
    if op == "experts_step":
        experts, weights = _route(s["logits"], s["bias"], c)
        got = _experts(s, experts, weights, s["grad_y"])
        got["grad_logits"] = _route_bwd(got.pop("grad_weights"), s["logits"], experts, c)
        return got
    return {"update": _orthogonalise(s["update"])}


# --------------------------------------------------------- the user's program

def _own(s):
    import mhc_hyper_connection_gb300 as mhc
    c, op = s["case"], s["case"]["op"]
    if op == "orthogonalise":
        return {"update": mhc.orthogonalise(s["update"], steps=STEPS, eps=EPS)}
    if op == "experts":
        plan = mhc.expert_plan(s["experts"], c["E"])
        return {"y": mhc.experts_ffn(s["x"], s["weights"], plan, s["w_gate_up"], s["w_down"], act=c["act"])[0]}
    how = dict(score=c["score"], renormalise=c["renorm"], scale=c["scale"])
    if op == "route_bwd":
        return {"grad_logits": mhc.route_experts_backward(s["grad_weights"], s["logits"], s["experts"], **how)}
    experts, weights = mhc.route_experts(s["logits"], c["k"], bias=s["bias"], groups=c["groups"],
                                         top_groups=c["top_groups"], group_score="top2", **how)
    if op == "route":
        return {"experts": experts, "weights": weights}
    plan = mhc.expert_plan(experts, c["E"])
    y, kept = mhc.experts_ffn(s["x"], weights, plan, s["w_gate_up"], s["w_down"], act=c["act"], save="16bit")
    got = mhc.experts_ffn_backward(s["grad_y"], s["x"], weights, plan, s["w_gate_up"], s["w_down"], kept, act=c["act"])
    grad_logits = mhc.route_experts_backward(got["grad_weights"], s["logits"], experts, **how)
    return {"y": y, "grad_x": got["grad_x"], "grad_w_gate_up": got["grad_w_gate_up"], "grad_w_down": got["grad_w_down"],
            "grad_logits": grad_logits}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------- in 64 bits

def _exact_choice(l, bias, c):
    """(score, experts, weights) of 64-bit logits: one slot after the other."""
    T, E = l.shape
    per = E // c["groups"]
    ok = ~torch.isinf(l)
    if c["score"] == "softmax":
        z = torch.where(ok, l, torch.full_like(l, -1e6))
        z = torch.logsumexp(z, -1, keepdim=True)
        score = torch.where(ok, torch.exp(l - z), 0.0)
    else:
        score = torch.where(ok, torch.sigmoid(l), 0.0)
    steer = score if bias is None else score + bias.double()
    if c["groups"] > 1:
        mark = torch.full((T, c["groups"]), -math.inf, dtype=torch.float64, device=l.device)
        for g in range(c["groups"]):
            v = torch.where(ok, steer, -math.inf)[:, g * per:(g + 1) * per]
            first, at = v.max(-1)
            rest = v.scatter(1, at[:, None], -math.inf).amax(-1)
            mark[:, g] = torch.where(torch.isinf(rest), first, first + rest)
        # a group stays if fewer than top_groups are ahead of it
        a, b = mark[:, :, None], mark[:, None, :]
        ids = torch.arange(c["groups"], device=l.device)
        ahead = (b > a) | ((b == a) & (ids[None, None, :] < ids[None, :, None]))
        ok = ok & (ahead.sum(-1) < c["top_groups"]).repeat_interleave(per, 1)
    steer = torch.where(ok, l if bias is None else steer, -math.inf)
    experts = torch.full((T, c["k"]), -1, dtype=torch.int32, device=l.device)
    weights = torch.zeros((T, c["k"]), dtype=torch.float64, device=l.device)
    ids = torch.arange(E, device=l.device)
    for j in range(c["k"]):
        best = steer.amax(-1, keepdim=True)
        at = torch.where(steer == best, ids, E).amin(-1)
        any_ = ~torch.isinf(best[:, 0])
        experts[:, j] = torch.where(any_, at, -1).int()
        weights[:, j] = torch.where(any_, score.gather(1, at[:, None])[:, 0], 0.0)
        steer = steer.scatter(1, at[:, None], -math.inf)
    if c["renorm"]:
        total = weights.sum(-1, keepdim=True)
        weights = torch.where(total > 0, weights / torch.where(total > 0, total, 1.0), 0.0)
    return score, experts, c["scale"] * weights


def _exact_route_bwd(gw, score, experts, c):
    T, E = score.shape
    d = torch.zeros((T, E), dtype=torch.float64, device=score.device)       # by the scores
    rows = torch.arange(T, device=score.device)
    total = torch.zeros((T,), dtype=torch.float64, device=score.device)
    dot = torch.zeros_like(total)
    for j in range(c["k"]):
        on, e = experts[:, j] >= 0, experts[:, j].long().clamp_min(0)
        p = torch.where(on, score[rows, e], 0.0)
        total += p
        dot += p * gw[:, j].double()
    safe = torch.where(total > 0, total, 1.0)
    for j in range(c["k"]):
        on, e = experts[:, j] >= 0, experts[:, j].long().clamp_min(0)
        v = gw[:, j].double()
        if c["renorm"]:
            v = (v - dot / safe) / safe
        d[rows, e] += torch.where(on, c["scale"] * v, 0.0)
    if c["score"] == "sigmoid":
        return d * score * (1.0 - score)
    return score * (d - (0.0 if c["renorm"] else (d * score).sum(-1, keepdim=True)))


def _exact_experts(s, experts, weights, grad_y=None):
    c, dt = s["case"], s["x"].dtype

    def act(z):
        return z / (1 + torch.exp(-z)) if c["act"] == "silu" else z / (1 + torch.exp(-2 * C0 * z * (1 + 0.044715 * z ** 2)))

    flat = experts.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat + 1, minlength=c["E"] + 1).tolist()
    parts = torch.split(order, counts)[1:]
    f64 = dict(dtype=torch.float64, device="cuda")
    T, D = s["x"].shape
    y = torch.zeros((T, c["k"], D), **f64)
    if grad_y is not None:
        gx, gw = torch.zeros((T, c["k"], D), **f64), torch.zeros((T * c["k"],), **f64)
        gwgu, gwd = torch.zeros(s["w_gate_up"].shape, **f64), torch.zeros(s["w_down"].shape, **f64)
    for e, part in enumerate(parts):
        if not len(part):
            continue
        x = s["x"].double()[part // c["k"]]
        w = weights.reshape(-1)[part].double()
        wgu, wd = s["w_gate_up"][e].double(), s["w_down"][e].double()
        g, u = x @ wgu[0].T, x @ wgu[1].T
        y.view(-1, D)[part] = (w[:, None] * (act(g) * u)) @ wd.T
        if grad_y is None:
            continue
        g, u = g.to(dt).double(), u.to(dt).double()
        if c["act"] == "silu":
            r, dr = g, 1.0
        else:
            r, dr = 2 * C0 * g * (1 + 0.044715 * g ** 2), 2 * C0 * (1 + 3 * 0.044715 * g ** 2)
        q = torch.exp(-r.abs())
        slope = 1 / (1 + torch.exp(-r)) + g * q / (1 + q) ** 2 * dr
        gy = grad_y.double()[part // c["k"]]
        ga = gy @ wd
        gw[part] = (ga * act(g) * u).sum(-1)
        gu_, gg = w[:, None] * ga * act(g), w[:, None] * ga * u * slope
        gx.view(-1, D)[part] = gg @ wgu[0] + gu_ @ wgu[1]
        gwgu[e, 0], gwgu[e, 1] = gg.T @ x, gu_.T @ x
        gwd[e] = gy.T @ (w[:, None] * act(g) * u)
    if grad_y is None:
        return {"y": y.sum(1)}, None
    return {"y": y.sum(1), "grad_x": gx.sum(1), "grad_w_gate_up": gwgu, "grad_w_down": gwd}, gw.reshape(T, c["k"])


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "orthogonalise":
        x = s["update"].double()
        x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + EPS)
        for a, b, q in STEPS:
            if c["m"] <= c["n"]:
                p = x @ x.mT
                x = a * x + (b * p + q * p @ p) @ x
            else:
                p = x.mT @ x
                x = a * x + x @ (b * p + q * p @ p)
        return {"update": x}
    if op == "experts":
        return _exact_experts(s, s["experts"], s["weights"])[0]
    score, experts, weights = _exact_choice(s["logits"].double(), s["bias"], c)
    if op == "route":
        return {"experts": experts, "weights": weights}
    if op == "route_bwd":
        return {"grad_logits": _exact_route_bwd(s["grad_weights"], score, s["experts"], c)}
    got, gw = _exact_experts(s, experts, weights, s["grad_y"])
    got["grad_logits"] = _exact_route_bwd(gw, score, experts, c)
    return got
