"""Plain 64-bit statements of the layer operators, for their tests: the 8-bit
checkpoint form, the post-mapping's backward and the gated feed-forward block.
numpy only; nothing of the library is imported."""
import numpy as np

E_RANGE = {"bf16": (-100, 119), "fp16": (-15, 7)}
BLOCK = 128


def e4m3_values():
    """The 256 values of e4m3: sign, four exponent bits of bias 7, three
    mantissa bits, no infinities, 0x7F and 0xFF NaN."""
    v = np.empty(256)
    for c in range(256):
        p, m = (c >> 3) & 15, c & 7
        mag = np.nan if (c & 127) == 127 else (2.0 ** (p - 7) * (1 + m / 8) if p else m * 2.0 ** -9)
        v[c] = -mag if c > 127 else mag
    return v


VALUES = e4m3_values()


def pack(x, kind):
    """(codes, scales) of x [rows, D] (float64 holding 16-bit values), searched
    from the definition: the exponent by trial, each code as the nearest value
    with ties to the even code."""
    lo, hi = E_RANGE[kind]
    rows, D = x.shape
    nb = -(-D // BLOCK)
    codes = np.zeros((rows, D), np.uint8)
    scales = np.zeros((rows, nb), np.uint8)
    pos = VALUES[:127]                       # 0 .. 448 ascending
    mid = (pos[1:] + pos[:-1]) / 2
    for r in range(rows):
        for b in range(nb):
            w = x[r, b * BLOCK:(b + 1) * BLOCK]
            fine = np.isfinite(w)
            amax = np.abs(w[fine]).max() if fine.any() else 0.0
            e = lo
            while e < hi and amax > 448.0 * 2.0 ** e:
                e += 1
            scales[r, b] = e + 127
            q = np.minimum(np.abs(np.where(fine, w, 0.0)) / 2.0 ** e, 448.0)
            i = np.searchsorted(mid, q, side="left")           # value nearest to q; a tie picks the lower one
            tie = (i < len(mid)) & (q == mid[np.minimum(i, len(mid) - 1)]) & (i % 2 == 1)
            i = np.where(tie, i + 1, i)
            c = i.astype(np.uint8) | np.where(np.signbit(w), 128, 0).astype(np.uint8)
            codes[r, b * BLOCK:(b + 1) * BLOCK] = np.where(fine, c, 127)
    return codes, scales


def restore(codes, scales):
    D = codes.shape[-1]
    s = 2.0 ** (scales.astype(np.float64) - 127)
    return VALUES[codes] * np.repeat(s, BLOCK, -1)[..., :D]


def post(x, res, post_w, comb):
    return post_w[..., None] * x[:, None] + np.einsum("tij,tid->tjd", comb, res)


def post_backward(g, x, res, post_w, comb):
    """(gradients, the sums of magnitudes that bound their rounding)."""
    def form(g, x, res, p, c):
        return {"grad_x": np.einsum("tj,tjd->td", p, g), "grad_residual": np.einsum("tij,tjd->tid", c, g),
                "grad_post": np.einsum("tjd,td->tj", g, x), "grad_comb": np.einsum("tid,tjd->tij", res, g)}
    return form(g, x, res, post_w, comb), form(*(np.abs(v) for v in (g, x, res, post_w, comb)))


GELU_C = np.sqrt(2.0 / np.pi)


def act(z, name):
    """The activation and its derivative."""
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    t = np.tanh(GELU_C * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * z ** 2)


def ffn(x, w_gate_up, w_down, name):
    """(y, gate, up) of the gated feed-forward block."""
    g, u = x @ w_gate_up[0].T, x @ w_gate_up[1].T
    return (act(g, name)[0] * u) @ w_down.T, g, u


def ffn_backward(grad_y, x, w_gate_up, w_down, g, u, name):
    h, dh = act(g, name)
    ga = grad_y @ w_down
    gg, gu = ga * u * dh, ga * h
    return {"grad_x": gg @ w_gate_up[0] + gu @ w_gate_up[1],
            "grad_w_gate_up": np.stack([gg.T @ x, gu.T @ x]),
            "grad_w_down": grad_y.T @ (h * u)}
