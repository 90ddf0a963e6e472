"""Plain 64-bit statements of the routed experts' operators, for their tests.  numpy
only; nothing of the library is imported."""
import numpy as np

import layer_refs as ref


def scores(l, score):
    """Scores of logits l [T, E]; a row of -inf alone has zeros."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        top = l.max(-1, keepdims=True)
        p = np.exp(l - np.where(top == -np.inf, 0.0, top))
        total = p.sum(-1, keepdims=True)
        return np.where(total == 0.0, 0.0, p / np.where(total == 0.0, 1.0, total))


def route(l, k, score="softmax", bias=None, groups=1, top_groups=None, group_score="top2", renormalise=True, scale=1.0):
    """(experts, weights), one token and one slot after the other."""
    T, E = l.shape
    per = E // groups
    top_groups = groups if top_groups is None else top_groups
    s = scores(l, score)
    key = s if bias is None else s + bias
    experts, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        able = [e for e in range(E) if l[t, e] > -np.inf and key[t, e] > -np.inf]
        if groups > 1:
            marks = []
            for g in range(groups):
                v = sorted((key[t, e] for e in able if e // per == g), reverse=True)
                marks.append(-np.inf if not v else v[0] if group_score == "max" or len(v) == 1 else v[0] + v[1])
            stay = sorted(range(groups), key=lambda g: (-marks[g], g))[:top_groups]
            able = [e for e in able if e // per in stay]
        by = l[t] if bias is None else key[t]
        best = sorted(able, key=lambda e: (-by[e], e))[:k]
        w = np.array([s[t, e] for e in best])
        if renormalise and len(w):
            if score == "softmax":
                w = np.exp(l[t, best] - l[t, best].max())
            w = w / w.sum()
        experts[t, :len(best)] = best
        weights[t, :len(best)] = w * scale
    return experts, weights


def route_backward(gw, l, experts, score, renormalise, scale):
    """(grad_logits, the sums of magnitudes that bound its rounding)."""
    T, E = l.shape
    s = scores(l, score)
    got, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = [j for j in range(experts.shape[1]) if 0 <= experts[t, j] < E]
        e = [experts[t, j] for j in on]
        d = scale * gw[t, on]
        u = s[t, e]
        if renormalise:
            if score == "softmax" and len(e) and l[t, e].max() > -np.inf:
                u = np.exp(l[t, e] - l[t, e].max())
            total = u.sum()
            w = u / total if total > 0 else np.zeros_like(u)
            h = 1.0 - s[t, e] if score == "sigmoid" else np.ones_like(u)
            for i, j in enumerate(e):
                got[t, j] += w[i] * (d[i] - (d * w).sum()) * h[i]
                mag[t, j] += w[i] * (abs(d[i]) + (np.abs(d) * w).sum()) * h[i]
        elif score == "sigmoid":
            for i, j in enumerate(e):
                got[t, j] += d[i] * u[i] * (1.0 - u[i])
                mag[t, j] += abs(d[i]) * u[i] * (1.0 - u[i])
        else:
            for i, j in enumerate(e):
                got[t, j] += d[i] * u[i]
                mag[t, j] += abs(d[i]) * u[i]
            got[t] -= s[t] * (d * u).sum()
            mag[t] += s[t] * (np.abs(d) * u).sum()
    return got, mag


def plan(experts, E):
    """(counts, place of each slot or -1, slot of each row or -1): slots sorted by expert,
    in their order within one, runs from multiples of 16."""
    flat = experts.reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(E)])
    places, rows, start = np.full(flat.shape, -1), [], 0
    for e in range(E):
        slots = np.nonzero(flat == e)[0]
        places[slots] = start + np.arange(len(slots))
        pad = -len(slots) % 16
        rows.extend(list(slots) + [-1] * pad)
        start += len(slots) + pad
    return counts, places.reshape(experts.shape), np.array(rows, int)


# Rounding bounds, from the arithmetic (u: one rounding to 16 bits, tiny: half the
# smallest step of fp16):
#   * a product of depth K is summed in fp32, sixteen products at a time: off by at
#     most s(K) = (K / 16 + 16) 2^-22 times the sum of the magnitudes;
#   * act and act' carry a few fast-math errors of 2^-22: 2^-18 of their scale;
#   * a, gg, gu, w a, an expert's rows and the outputs are each rounded to 16 bits once.
# They are propagated through the formulas with magnitudes (|act'| <= 1.13).
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = 2.0 ** -25
FAST = 2.0 ** -18


def s(K):
    return (K / 16 + 16) * 2.0 ** -22


def experts(x, weights, idx, w_gate_up, w_down, name, kind):
    """(y, its bound, gate and up sums of every slot [T, k, 2, F], their bounds)."""
    T, k = idx.shape
    E, _, F, D = w_gate_up.shape
    u = U[kind]
    y, ey = np.zeros((T, D)), np.zeros((T, D))
    kept, ekept = np.zeros((T, k, 2, F)), np.zeros((T, k, 2, F))
    for e in range(E):
        t, j = np.nonzero(idx == e)
        if not len(t):
            continue
        xe, w, wd = x[t], w_gate_up[e], w_down[e]
        row, g, up = ref.ffn(xe, w, wd, name)
        eg, eu = (s(D) * (np.abs(xe) @ np.abs(w[h]).T) for h in (0, 1))
        h = ref.act(g, name)[0]
        a = h * up
        ea = (1.13 * eg + FAST * np.abs(g)) * (np.abs(up) + eu) + (np.abs(h) + FAST * np.abs(g)) * eu + u * np.abs(a)
        ea = ea * (1 + u) + TINY
        er = (ea + s(F) * np.abs(a)) @ np.abs(wd).T
        er = er * (1 + u) + u * np.abs(row) + TINY
        wt = weights[t, j][:, None]
        np.add.at(y, t, wt * row)
        np.add.at(ey, t, np.abs(wt) * (er + 2.0 ** -22 * np.abs(row)))
        kept[t, j] = np.stack([g, up], 1)
        ekept[t, j] = np.stack([eg, eu], 1)
    return y, ey * (1 + u) + u * np.abs(y) + TINY, kept, ekept


def experts_backward(gy, x, weights, idx, w_gate_up, w_down, kept, name, kind):
    """{name: (gradient, bound)} from the kept sums [T, k, 2, F]."""
    T, k = idx.shape
    E, _, F, D = w_gate_up.shape
    u = U[kind]
    z = lambda *s_: (np.zeros(s_), np.zeros(s_))  # noqa: E731
    got = {"grad_x": z(T, D), "grad_weights": z(T, k), "grad_w_gate_up": z(E, 2, F, D), "grad_w_down": z(E, D, F)}
    for e in range(E):
        t, j = np.nonzero(idx == e)
        if not len(t):
            continue
        xe, ge, wt, w, wd = x[t], gy[t], weights[t, j][:, None], w_gate_up[e], w_down[e]
        g, up = kept[t, j, 0], kept[t, j, 1]
        h, dh = ref.act(g, name)
        a, ga = h * up, ge @ wd
        ega = s(D) * (np.abs(ge) @ np.abs(wd))
        efast = FAST * (1 + np.abs(g))
        got["grad_weights"][0][t, j] = (a * ga).sum(-1)
        got["grad_weights"][1][t, j] = (np.abs(a) * ega + np.abs(up * ga) * efast + s(F) * np.abs(a * ga)).sum(-1) + 1e-30
        aw = np.abs(wt)
        gg, gu, wa = wt * ga * up * dh, wt * ga * h, wt * a
        fast = efast * (1 + (0 if name == "silu" else 1) * g * g)
        egg = (aw * np.abs(up) * (1.13 * ega + np.abs(ga) * fast) + u * np.abs(gg)) * (1 + u) + TINY
        egu = (aw * (np.abs(h) * ega + np.abs(ga) * efast) + u * np.abs(gu)) * (1 + u) + TINY
        ea = (aw * np.abs(up) * efast + u * np.abs(wa)) * (1 + u) + TINY
        row = gg @ w[0] + gu @ w[1]
        er = (egg + s(2 * F) * np.abs(gg)) @ np.abs(w[0]) + (egu + s(2 * F) * np.abs(gu)) @ np.abs(w[1])
        np.add.at(got["grad_x"][0], t, row)
        np.add.at(got["grad_x"][1], t, er * (1 + u) + u * np.abs(row) + TINY)
        R = len(t)
        out = lambda err, v: err * (1 + u) + u * np.abs(v) + TINY  # noqa: E731
        for i, (d, v) in enumerate(((egg, gg), (egu, gu))):
            got["grad_w_gate_up"][0][e, i] = v.T @ xe
            got["grad_w_gate_up"][1][e, i] = out((d + s(R) * np.abs(v)).T @ np.abs(xe), v.T @ xe)
        got["grad_w_down"][0][e] = ge.T @ wa
        got["grad_w_down"][1][e] = out(np.abs(ge).T @ (ea + s(R) * np.abs(wa)), ge.T @ wa)
    v, b = got["grad_x"]
    got["grad_x"] = (v, b * (1 + u) + u * np.abs(v) + TINY)
    return got
