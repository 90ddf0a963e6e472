"""The example that runs the layer operators together (examples/train_layer.py):
its gradients against automatic differentiation of the same layers in 64 bits,
and its 8-bit route against its 16-bit one.

Tolerances, as 2-norms: the 16-bit route rounds y, z, the streams and each
gradient on the way to bf16, about ten roundings of at most 2^-8 per layer that
add up like random errors or, at worst, in line: 10 2^-8 = 2^-4.7 of a
gradient's norm, 2^-4 allowed for two layers' parameters.  The 8-bit route holds
streams and sums to half a step, 2^-4 of a value at most and 2^-4 / sqrt(3) on
average over a step; an input that is off by that share moves a gradient by
about as much, and a gradient sees at most three of them (g, u, and the
streams): 3 2^-4 / sqrt(3) = 2^-3.2, 2^-3 allowed."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from mhc_hyper_connection_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("train_layer", os.path.join(ROOT, "examples", "train_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _layer64(p, X, act, n=4, iters=20, eps=1e-6):
    """One layer in 64 bits, from the formulas of the three operators."""
    T, _, D = X.shape
    flat = X.reshape(T, n * D)
    mix = (flat @ p["phi"].t()) * (flat.square().mean(1, keepdim=True) + eps).rsqrt()
    b, a = p["bias"], p["alpha"]
    h_pre = torch.sigmoid(a[0] * mix[:, :n] + b[:n]) + eps
    h_post = 2 * torch.sigmoid(a[1] * mix[:, n:2 * n] + b[n:2 * n])
    H = (a[2] * mix[:, 2 * n:] + b[2 * n:]).reshape(T, n, n)
    M = torch.softmax(H, -1) + eps
    M = M / (M.sum(1, keepdim=True) + eps)
    for _ in range(iters - 1):
        M = M / (M.sum(2, keepdim=True) + eps)
        M = M / (M.sum(1, keepdim=True) + eps)
    y = (h_pre[..., None] * X).sum(1)
    g, u = y @ p["w_gate_up"][0].t(), y @ p["w_gate_up"][1].t()
    z = (g * torch.sigmoid(g) * u) @ p["w_down"].t()
    return h_post[..., None] * z[:, None] + torch.einsum("tij,tid->tjd", M, X)


def _setup(example, device, T=300, D=256, F=520, layers=2):
    gen = torch.Generator(device=device).manual_seed(5)
    X = torch.randn((T, 4, D), generator=gen, device=device).bfloat16()
    target = torch.randn((T, D), generator=gen, device=device)
    return [example.Layer(D, F, device, seed=i) for i in range(layers)], X, target


def _off(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_gradients_against_automatic_differentiation(example, cuda_device):
    layers, X, target = _setup(example, cuda_device)
    loss, grads, gX = example.forward_backward(layers, X, target, "16bit")
    ps = [{k: v.double().requires_grad_() for k, v in layer.params().items()} for layer in layers]
    X64 = X.double().requires_grad_()
    Y = X64
    for p in ps:
        Y = _layer64(p, Y, "silu")
    want = 0.5 * (Y.mean(1) - target.double()).square().sum() / X.shape[0]
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 2.0 ** -7 * float(want.detach())
    assert _off(gX, X64.grad) <= 2.0 ** -4
    for g, p in zip(grads, ps):
        for k in ("w_gate_up", "w_down", "phi", "bias"):
            assert _off(g[k], p[k].grad) <= 2.0 ** -4, k


def test_8bit_route_follows_the_16bit_one(example, cuda_device):
    layers, X, target = _setup(example, cuda_device)
    l16, g16, x16 = example.forward_backward(layers, X, target, "16bit")
    l8, g8, x8 = example.forward_backward(layers, X, target, "8bit")
    assert float(l8) == float(l16)            # the forward is the same, bit for bit
    assert _off(x8, x16) <= 2.0 ** -3
    for a, b in zip(g8, g16):
        for k in ("w_gate_up", "w_down", "phi", "bias"):
            assert _off(a[k], b[k]) <= 2.0 ** -3, k


@pytest.mark.parametrize("keep", ["8bit", "16bit"])
def test_loss_falls(example, cuda_device, keep):
    layers, X, target = _setup(example, cuda_device, T=256, D=128, F=256)
    losses = []
    for _ in range(6):
        loss, grads, _ = example.forward_backward(layers, X, target, keep)
        losses.append(float(loss))
        for layer, g in zip(layers, grads):
            for k, p in layer.params().items():
                p.sub_((0.02 * g[k].float()).to(p.dtype))
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
