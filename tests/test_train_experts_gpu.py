"""The example with routed experts and orthogonalised updates (examples/train_layer.py): its
gradients against automatic differentiation of the same layers in 64 bits with the choice
held, and that its steps run.

Tolerance, as 2-norms: as for the plain layers (tests/test_train_layer_gpu.py), ten roundings
of at most 2^-8 per layer, 2^-4 allowed for two layers' parameters."""
import pytest
import torch

from test_train_layer_gpu import _layer64, _off, example  # noqa: F401

pytestmark = pytest.mark.gpu


def _setup(example, device, T=200, D=256, F=136, layers=2):  # noqa: F811
    gen = torch.Generator(device=device).manual_seed(6)
    X = torch.randn((T, 4, D), generator=gen, device=device).bfloat16()
    target = torch.randn((T, D), generator=gen, device=device)
    return [example.ExpertLayer(D, F, device, seed=i, experts=6, choices=2) for i in range(layers)], X, target


def _body64(p, experts):
    def body(y):
        s = torch.sigmoid(y @ p["router"].t()).gather(1, experts)
        w = s / s.sum(-1, keepdim=True)
        z = torch.zeros_like(y)
        for j in range(experts.shape[1]):
            for e in range(p["router"].shape[0]):
                t = torch.nonzero(experts[:, j] == e)[:, 0]
                g, u = y[t] @ p["w_gate_up"][e, 0].t(), y[t] @ p["w_gate_up"][e, 1].t()
                z = z.index_add(0, t, w[t, j, None] * ((g * torch.sigmoid(g) * u) @ p["w_down"][e].t()))
        return z
    return body


@pytest.mark.parametrize("keep", ["16bit", "8bit"])
def test_gradients_against_automatic_differentiation(example, cuda_device, keep, monkeypatch):  # noqa: F811
    layers, X, target = _setup(example, cuda_device)
    chosen = []
    real = example.mhc.expert_plan
    monkeypatch.setattr(example.mhc, "expert_plan", lambda e, n: chosen.append(e.long()) or real(e, n))
    loss, grads, gX = example.forward_backward(layers, X, target, keep)
    ps = [{k: v.double().requires_grad_() for k, v in layer.params().items()} for layer in layers]
    X64 = X.double().requires_grad_()
    Y = X64
    for p, e in zip(ps, chosen):
        # the plain layer's formulas with its feed-forward block replaced by the experts
        flat = dict(p, w_gate_up=torch.zeros((2, 8, 256), dtype=torch.float64, device=cuda_device),
                    w_down=torch.zeros((256, 8), dtype=torch.float64, device=cuda_device))
        base = _layer64(flat, Y, "silu")                     # without the body: comb's part alone
        T, n, D = Y.shape
        mix = (Y.reshape(T, n * D) @ p["phi"].t()) * (Y.reshape(T, n * D).square().mean(1, keepdim=True) + 1e-6).rsqrt()
        h_pre = torch.sigmoid(p["alpha"][0] * mix[:, :n] + p["bias"][:n]) + 1e-6
        h_post = 2 * torch.sigmoid(p["alpha"][1] * mix[:, n:2 * n] + p["bias"][n:2 * n])
        Y = base + h_post[..., None] * _body64(p, e)((h_pre[..., None] * Y).sum(1))[:, None]
    want = 0.5 * (Y.mean(1) - target.double()).square().sum() / X.shape[0]
    want.backward()
    tol = 2.0 ** -4 if keep == "16bit" else 2.0 ** -3        # streams kept to half a step of 8 bits
    assert abs(float(loss) - float(want.detach())) <= 2.0 ** -7 * float(want.detach())
    assert _off(gX, X64.grad) <= tol
    for g, p in zip(grads, ps):
        for k in ("w_gate_up", "w_down", "router", "phi", "bias"):
            assert _off(g[k], p[k].grad) <= tol, k


def test_steps_run(example, cuda_device):  # noqa: F811
    """Steps along gradients and along orthogonalised momenta change every parameter, stay
    finite, and the balance follows the load."""
    layers, X, target = _setup(example, cuda_device)
    momentum = example.Momentum(layers)
    before = [{k: v.clone() for k, v in layer.params().items()} for layer in layers]
    for _ in range(3):
        loss, grads, _ = example.forward_backward(layers, X, target, "8bit")
        assert torch.isfinite(loss)
        for layer, g in zip(layers, grads):
            for k in ("phi", "alpha", "bias", "router"):
                layer.params()[k].sub_(0.02 * g[k].float())
            assert int(layer.load.sum()) == 2 * X.shape[0]
            layer.follow_load()
        momentum.step(layers, grads, 0.02)
    for layer, b in zip(layers, before):
        assert all(torch.isfinite(v.float()).all() and not torch.equal(v, b[k]) for k, v in layer.params().items())
        assert layer.balance.abs().max() > 0
