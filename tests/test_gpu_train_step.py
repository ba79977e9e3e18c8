"""Dense products around the expert layer and the update of all their weights,
as a training step uses them: forward, backward, update, eager and as a replayed
graph.

Each stage is held to the float64 oracle given the stage's stored inputs, at the
tolerances of the stage's own tests (the expert layer has its own parity tests;
here its gradients are the update's inputs)."""

import numpy as np
import pytest
import torch

from oracle import dense_ref as ref

from helpers import say
from test_gpu_dense import DT, HALF, U, _check, _f64, g_of
from test_gpu_muon import _check_one
from token_routing_grouped_amd import inputs

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
T, D, E, K, H = 264, 128, 8, 2, 64
LR, MU, DECAY = 0.02, 0.9, 0.5


class Step:
    """gelu projection with bias, experts, projection back onto the first one's output."""

    def __init__(self, dt):
        from token_routing_grouped_amd.layer import LinearGPU, MoELayerGPU, MuonGPU

        g = np.random.default_rng(31)
        t = lambda *n, sc=1.0: (torch.from_numpy(g.standard_normal(n)) * sc).to(DEV).to(DT[dt])
        self.x, self.dy, self.bias = t(T, D), t(T, D), t(D)
        self.wr = t(E, D, sc=D ** -0.5)
        self.w = [t(D, D, sc=D ** -0.5), t(E, H, D, sc=D ** -0.5), t(E, H, D, sc=D ** -0.5), t(E, D, H, sc=H ** -0.5),
                  t(D, D, sc=D ** -0.5)]
        self.forced = torch.from_numpy(inputs.forced_routing("uniform", T, E, K, 3)).to(DEV)
        self.scale = torch.ones((), device=DEV)
        self.up, self.down = LinearGPU(T, D, D, DT[dt], act="gelu"), LinearGPU(T, D, D, DT[dt])
        self.moe = MoELayerGPU(T, D, E, K, H, DT[dt], DEV)
        self.opt = MuonGPU(self.w, lr=LR, momentum=MU, weight_decay=DECAY, lr_scale=self.scale)

    def grads(self):
        return [self.up.dw, self.moe.dw1, self.moe.dw3, self.moe.dw2, self.down.dw]

    def run(self):
        w0, w1, w3, w2, w4 = self.w
        u = self.up.forward(self.x, w0, bias=self.bias)
        m = self.moe.forward(u, self.wr, w1, w3, w2, forced_idx=self.forced)
        self.down.forward(m, w4, res=u)
        dm = self.down.backward(self.dy, m, w4)
        du = self.moe.backward(dm, u, self.wr, w1, w3, w2)
        du.add_(self.dy)  # the residual's share
        self.up.backward(du, self.x, w0)
        self.opt.step(self.grads())

    def state(self):
        return [*self.w, *self.opt.bufs, *(m for m in self.opt.masters if m is not None), self.up.dbias, self.down.y]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_every_stage(dt):
    say(f"train step {dt}")
    s = Step(dt)
    w = [t.clone() for t in s.w]
    s.run()
    torch.cuda.synchronize()
    x, dy, u, m = _f64(s.x), _f64(s.dy), _f64(s.up.y), _f64(s.moe.y)
    ry, rz = ref.linear(x, _f64(w[0]), _f64(s.bias), None, "gelu")
    bz = g_of(D) * (np.abs(x) @ np.abs(_f64(w[0])).T) + 2 * U * np.abs(rz)
    _check("up", s.up.y, ry, 1.13 * bz + 16 * U * (1 + np.abs(rz)) + 2 * U * np.abs(ry), HALF[dt])
    ry, _ = ref.linear(m, _f64(w[4]), None, u)
    _check("down", s.down.y, ry, g_of(D) * (np.abs(m) @ np.abs(_f64(w[4])).T) + 4 * U * np.abs(ry), HALF[dt])
    rx, rw, _, _ = ref.linear_bwd(dy, m, _f64(w[4]), None, "none")
    _check("down dx", s.down.dx, rx, g_of(D) * (np.abs(dy) @ np.abs(_f64(w[4]))), HALF[dt])
    _check("down dw", s.down.dw, rw, g_of(T) * (np.abs(dy).T @ np.abs(m)), HALF[dt])
    du = _f64(s.moe.dx)
    _, rw, rb, rz = ref.linear_bwd(du, x, _f64(w[0]), _f64(s.up.z), "gelu")
    ez = 16 * U * np.abs(du) * (1 + np.abs(_f64(s.up.z)))
    e = HALF[dt] * np.abs(rz) + ez * (1 + HALF[dt])
    _check("up dw", s.up.dw, rw, g_of(T) * ((np.abs(rz) + e).T @ np.abs(x)) + e.T @ np.abs(x), HALF[dt])
    _check("up db", s.up.dbias, rb, g_of(T) * (np.abs(rz) + e).sum(0) + ez.sum(0), HALF[dt])
    mu = float(np.float32(MU))
    for i, (before, after, g) in enumerate(zip(w, s.w, s.grads())):
        r, c = before.shape[-2:]
        step = LR * max(1.0, r / c) ** 0.5
        after = s.opt.masters[i] if dt == "bf16" else after
        for b, a, gb in zip(*(_f64(t).reshape(-1, r, c) for t in (before, after, g))):
            # the buffer starts at zero: u = g + mu g
            _check_one(a, gb * (1 + mu), "f32", scale=-step, base=b * (1 - LR * DECAY))
        if dt == "bf16":
            assert torch.equal(s.opt.masters[i].bfloat16(), s.w[i])


def test_captured_and_replayed():
    """A whole step in one graph against eager steps from the same state."""
    a, b = Step("bf16"), Step("bf16")
    for s in (a, b):
        s.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            a.run()
    torch.cuda.current_stream().wait_stream(side)
    for rep in range(4):
        g = torch.Generator(device=DEV).manual_seed(rep)
        new = torch.randn(T, D, device=DEV, generator=g).bfloat16()
        for s in (a, b):
            s.scale.fill_(1.0 / (rep + 1))
            s.x.copy_(new)
        b.run()
        graph.replay()
        torch.cuda.synchronize()
        for k, (p, q) in enumerate(zip(a.state(), b.state())):
            assert torch.equal(p, q), (rep, k)


def test_nothing_moves_when_a_gradient_does_not_fit():
    from token_routing_grouped_amd import _abi
    from token_routing_grouped_amd.layer import MuonGPU

    w = [torch.ones(2, 16, 24, device=DEV), torch.ones(16, 32, device=DEV)]
    opt = MuonGPU(w)
    for bad in (torch.ones(32, 16, device=DEV), torch.ones(16, 32, device=DEV).bfloat16(), torch.ones(16, 32),
                torch.ones(32, 16, device=DEV).t()):
        with pytest.raises(_abi.MoeError, match="gradient 1 must be"):
            opt.step([torch.ones(2, 16, 24, device=DEV), bad])
    with pytest.raises(_abi.MoeError, match="2 gradients expected"):
        opt.step([w[0]])
    assert all((v == 1).all() for v in w) and all((v == 0).all() for v in opt.bufs)
    with pytest.raises(_abi.MoeError, match="given twice"):
        MuonGPU([w[0], w[0]])
