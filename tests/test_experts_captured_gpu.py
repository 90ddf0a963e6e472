"""Routed experts and updates captured into graphs in the forms that take several dependent
launches: a plan of many slots, more experts than a kernel's default shared memory, X X^T in
parts of its depth; replayed on other data, beside eager calls, and two graphs at once."""
import pytest
import torch

import mhc_hyper_connection_gb300 as mhc
import test_experts_gpu as te

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mhc_hyper_connection_gb300 import build
    build.build()


class Step:
    """A step of the body on buffers of its own."""

    def __init__(self, device, T, E, k, D, F, seed):
        self.c = te._case(device, T, E, k, D, F, "bf16", seed)
        self.k, self.E, self.deep = k, E, torch.randn((2, 96, 9000), device=device, generator=torch.Generator(device=device).manual_seed(seed))
        self.logits = torch.randn((T, E), generator=torch.Generator(device=device).manual_seed(seed), device=device)
        e = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device=device)  # noqa: E731
        plan = mhc.expert_plan(self.c["idx"], E)
        self.plan, self.routes = torch.empty_like(plan.buffer), mhc.Routes(e(T, k, d=torch.int32), e(T, k, d=torch.float32))
        self.y, self.kept, self.gl = e(T, D), e(plan.rows, 2, F), e(T, E, d=torch.float32)
        self.grads = dict(grad_x=e(T, D), grad_weights=e(T, k, d=torch.float32), grad_w_gate_up=e(E, 2, F, D), grad_w_down=e(E, D, F))
        self.update = e(2, 96, 9000)
        self.ws = (mhc.experts_ffn_workspace(T, E, k, D, F, device), mhc.experts_ffn_workspace(T, E, k, D, F, device, backward=True),
                   mhc.orthogonalise_workspace(self.deep.shape, device))

    def run(self):
        c = self.c
        r = mhc.route_experts(self.logits, self.k, out=self.routes)
        p = mhc.expert_plan(r.experts, self.E, buffer=self.plan)
        mhc.experts_ffn(c["x"], r.weights, p, c["w"], c["wd"], save="16bit", y=self.y, kept=self.kept, workspace=self.ws[0])
        g = mhc.experts_ffn_backward(c["gy"], c["x"], r.weights, p, c["w"], c["wd"], self.kept, grads=self.grads, workspace=self.ws[1])
        mhc.route_experts_backward(g["grad_weights"], self.logits, r.experts, grad_logits=self.gl)
        mhc.orthogonalise(self.deep, out=self.update, workspace=self.ws[2])

    def results(self):
        return [*self.routes, self.y, self.gl, self.update, *self.grads.values()]

    def change(self, seed):
        gen = torch.Generator(device=self.y.device).manual_seed(seed)
        self.logits.normal_(generator=gen)
        self.deep.normal_(generator=gen)
        self.c["x"].copy_(torch.randn(self.c["x"].shape, generator=gen, device=self.y.device))

    def clear(self):
        for t in self.results():
            t.zero_()

    def sound(self):
        return all(mhc.experts_ffn_status(w) == 0 for w in self.ws[:2]) and mhc.orthogonalise_status(self.ws[2]) == 0


@pytest.mark.parametrize("T,E,k,D,F", [(2500, 1024, 3, 64, 72), (3000, 12, 4, 264, 136), (5, 300, 8, 520, 264)])
def test_captured_steps(cuda_device, T, E, k, D, F):
    s, t = Step(cuda_device, T, E, k, D, F, 1), Step(cuda_device, T, E, k, D, F, 2)
    graphs = []
    for one in (s, t):
        one.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            one.run()
        graphs.append(graph)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in (3, 4, 5):
        want = []
        for one in (s, t):
            one.change(seed)
            one.clear()
            one.run()
            want.append([v.clone() for v in one.results()])
            one.clear()
        for graph, one, w in zip(graphs, (s, t), want):          # one after the other
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(one.results(), w))
            one.clear()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, side):                   # at once
            with torch.cuda.stream(stream):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for one, w in zip((s, t), want):
            assert all(torch.equal(a, b) for a, b in zip(one.results(), w)) and one.sound()
