"""Training hyper-connection layers with checkpointed activations.

A stack of layers, each

    y, h_post, comb = pre-mapping(X)        X: n = 4 residual streams [T, 4, D]
    z               = gated feed-forward(y)
    X'              = post-mapping(z, X, h_post, comb)

is trained on random targets for the mean of its output streams.  With
keep="8bit" the residual streams and the feed-forward sums wait for the backward
pass in 8 bits: the post-mapping writes the checkpoint of the streams it
produces, its backward reads it directly, and the pre-mapping's backward gets it
restored.  With keep="16bit" everything is kept as it was.

    python examples/train_layer.py [--tokens T] [--width D] [--hidden F] [--layers L] [--steps K] [--keep 8bit|16bit]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mhc_hyper_connection_gb300 as mhc  # noqa: E402

N = 4


class Layer:
    def __init__(self, D, F, device, seed, act="silu"):
        gen = torch.Generator(device=device).manual_seed(seed)
        rn = lambda *s, k: torch.randn(s, generator=gen, device=device) * k  # noqa: E731
        self.op = mhc.MhcPre(N, D, need_backward=True)
        self.act = act
        self.phi = rn(N * N + 2 * N, N * D, k=(N * D) ** -0.5)
        self.alpha = torch.full((3,), 0.5, device=device)
        self.bias = rn(N * N + 2 * N, k=0.1)
        self.w_gate_up = rn(2, F, D, k=D ** -0.5).bfloat16()
        self.w_down = rn(D, F, k=0.1 * F ** -0.5).bfloat16()

    def params(self):
        return {"phi": self.phi, "alpha": self.alpha, "bias": self.bias, "w_gate_up": self.w_gate_up,
                "w_down": self.w_down}

    def forward(self, X, X_ckpt, keep):
        """Streams X and, with keep="8bit", their checkpoint; returns the next
        layer's pair and what the backward needs."""
        pre = self.op.allocate(X.shape[0], X.device)
        self.op.run(X, self.phi, self.alpha, self.bias, pre)
        z, sums = mhc.gated_ffn(pre["y"], self.w_gate_up, self.w_down, act=self.act, save=keep)
        if keep == "8bit":
            out, out_ckpt = mhc.hc_post_ckpt(z, X, pre["h_post"], pre["h_res"])
            return out, out_ckpt, (X_ckpt, pre, z, sums)
        return mhc.hc_post(z, X, pre["h_post"], pre["h_res"]), None, (X, pre, z, sums)

    def backward(self, g, saved):
        """Gradient of the output streams in; that of the input streams and of
        the parameters out."""
        X, pre, z, sums = saved
        post = mhc.hc_post_backward(g, z, X, pre["h_post"], pre["h_res"])
        ffn = mhc.gated_ffn_backward(post["grad_x"], pre["y"], self.w_gate_up, self.w_down, sums, act=self.act)
        if isinstance(X, mhc.Ckpt8):
            X = mhc.ckpt8_restore(X)
        grads = self.op.allocate_backward(g.shape[0], g.device)
        self.op.backward(X, self.phi, self.alpha, None, ffn["grad_x"], post["grad_post"], post["grad_comb"], pre, grads,
                         grad_x_post=post["grad_residual"])
        return grads["grad_x"], {"phi": grads["grad_phi"], "alpha": grads["grad_alpha"], "bias": grads["grad_bias"],
                                 "w_gate_up": ffn["grad_w_gate_up"], "w_down": ffn["grad_w_down"]}


def forward_backward(layers, X, target, keep):
    """Loss 0.5 sum (mean over streams - target)^2 / T, and the gradients of
    every layer's parameters and of X."""
    ckpt = mhc.ckpt8_pack(X) if keep == "8bit" else None
    saved = []
    for layer in layers:
        X, ckpt, s = layer.forward(X, ckpt, keep)
        saved.append(s)
    err = X.float().mean(1) - target
    loss = 0.5 * (err * err).sum() / X.shape[0]
    g = (err / (N * X.shape[0])).bfloat16()[:, None].expand(-1, N, -1).contiguous()
    grads = [None] * len(layers)
    for i in reversed(range(len(layers))):
        g, grads[i] = layers[i].backward(g, saved[i])
    return loss, grads, g


def kept_bytes(tokens, width, hidden, keep):
    """Bytes of activations that a layer keeps: streams, y, z, feed-forward sums."""
    streams, sums = tokens * N * width, tokens * 2 * hidden
    return (streams + sums) * (129 / 128 if keep == "8bit" else 2) + 4 * tokens * width


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--layers", type=int, default=3)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--lr", type=float, default=0.5)
    ap.add_argument("--keep", choices=("8bit", "16bit"), default="8bit")
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(0)
    X = torch.randn((a.tokens, 1, a.width), generator=gen, device=dev).expand(-1, N, -1).contiguous().bfloat16()
    target = torch.randn((a.tokens, a.width), generator=gen, device=dev)
    layers = [Layer(a.width, a.hidden, dev, seed=i + 1) for i in range(a.layers)]
    print(f"{a.layers} layers, {a.tokens} tokens, width {a.width}, hidden {a.hidden}: "
          f"{kept_bytes(a.tokens, a.width, a.hidden, a.keep) / 2 ** 20:.1f} MiB kept per layer ({a.keep})")
    for step in range(a.steps):
        loss, grads, _ = forward_backward(layers, X, target, a.keep)
        norm = sum(float(g.float().square().sum()) for d in grads for g in d.values()) ** 0.5
        lr = a.lr / max(1.0, norm)                        # steps of a length of at most a.lr
        for layer, g in zip(layers, grads):
            for k, p in layer.params().items():
                p.sub_((lr * g[k].float()).to(p.dtype))
        print(f"step {step}: loss {loss.item():.4f}", flush=True)


if __name__ == "__main__":
    main()
