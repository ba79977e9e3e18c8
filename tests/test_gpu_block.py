"""MoEBlockGPU (norm and layer, forward and backward) over the layer's own
modes (lean and two streams are bf16 only).

The block is the calls of moe_rmsnorm_fwd, MoELayerGPU and moe_rmsnorm_bwd in
turn, so its results are theirs bit for bit (norm and layer have their own
parity tests); and the layer inside is held to the float64 oracle at its
parity bounds (bf16: helpers.py; fp32: rel-L2 1e-4, largest 1e-3), given the
normed rows that the block stored.
"""

import numpy as np
import pytest
import torch

from oracle import moe_ref, norm_ref

from helpers import assert_close, say, to_np
from token_routing_grouped_amd import inputs

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
T, D, E, K, H = 264, 256, 8, 2, 128
EPS = 1e-5
OUT = ("y", "dw1", "dw3", "dw2", "dwr", "topk_idx")


def _abi():
    from token_routing_grouped_amd import _abi as a

    return a


def _inputs(dt):
    g = np.random.default_rng(21)
    t = lambda *n, sc=1.0: (torch.from_numpy(g.standard_normal(n)) * sc).to(DEV).to(dt)
    w = [t(E, D, sc=D ** -0.5), t(E, H, D, sc=D ** -0.5), t(E, H, D, sc=D ** -0.5), t(E, D, H, sc=H ** -0.5)]
    return dict(x=t(T, D), res=t(T, D), dy=t(T, D), ds=t(T, D), nw=(1 + 0.1 * t(D).float()).to(dt), w=w)


def _layer(dt, **flags):
    from token_routing_grouped_amd.layer import MoELayerGPU

    return MoELayerGPU(T, D, E, K, H, dt, DEV, **flags)


def _forced(mode):
    return torch.from_numpy(inputs.forced_routing(mode, T, E, K, 3)).to(DEV) if mode else None


def _block_step(i, dt, flags, forced, steps=1):
    from token_routing_grouped_amd.layer import MoEBlockGPU

    b = MoEBlockGPU(_layer(dt, **flags), eps=EPS)
    for _ in range(steps):
        b.forward(i["x"], i["nw"], *i["w"], res=i["res"], forced_idx=forced)
        b.backward(i["dy"], i["nw"], *i["w"], ds=i["ds"])
    torch.cuda.synchronize()
    return b


MODES = [("bf16", {}, None), ("bf16", {}, "uniform"), ("bf16", dict(aux_alpha=0.5), "zipf"), ("bf16", dict(lean=True), None),
         ("bf16", dict(overlap=True), None), ("bf16", dict(lean=True, overlap=True, aux_alpha=0.5), None),
         ("f32", {}, None), ("f32", dict(aux_alpha=0.5), "uniform"),
         ("bf16", dict(mx=True), None), ("bf16", dict(mx=True, overlap=True, aux_alpha=0.5), "zipf"),
         ("bf16", dict(mx=True, lean=True, wq_overlap=False), None)]


@pytest.mark.parametrize("dt,flags,mode", MODES, ids=[f"{d}-{'-'.join(f) or 'plain'}-{m or 'router'}" for d, f, m in MODES])
def test_block_is_its_calls_in_turn(dt, flags, mode):
    say(f"block {dt} {flags} {mode}")
    abi = _abi()
    dt = torch.bfloat16 if dt == "bf16" else torch.float32
    i, forced = _inputs(dt), _forced(mode)
    b = _block_step(i, dt, flags, forced, steps=2)  # the second step reuses the streams' events
    la = _layer(dt, **flags)
    xn, s, dx, dnw = (torch.empty_like(i[n]) for n in ("x", "x", "x", "nw"))
    rstd = torch.empty(T, device=DEV)
    abi.moe_rmsnorm_fwd(i["x"], i["nw"], EPS, xn, res=i["res"], s=s, rstd=rstd)
    la.forward(xn, *i["w"], forced_idx=forced)
    dxn = la.backward(i["dy"], xn, *i["w"])
    abi.moe_rmsnorm_bwd(dxn, s, i["nw"], rstd, dx, dnw, abi.workspace(abi.moe_rmsnorm_bwd_workspace_size(T, D), DEV),
                        ds=i["ds"])
    torch.cuda.synchronize()
    for n in OUT:
        assert torch.equal(getattr(b.layer, n), getattr(la, n)), n
    for n, got, want in (("s", b.s, s), ("xn", b.xn, xn), ("dx", b.dx, dx), ("dnorm_w", b.dnorm_w, dnw)):
        assert torch.equal(got, want), n
    if mode:
        assert torch.equal(b.layer.topk_idx, forced)


@pytest.mark.parametrize("dt,alpha,mode", [("f32", 0.0, "zipf"), ("f32", 0.5, "uniform"), ("bf16", 0.5, "zipf")])
def test_block_with_a_given_routing_against_the_oracle(dt, alpha, mode):
    say(f"block oracle {dt} alpha={alpha} {mode}")
    rel, frac = (1e-4, 1e-3) if dt == "f32" else (1e-2, 2e-2)
    dt = torch.bfloat16 if dt == "bf16" else torch.float32
    i, forced = _inputs(dt), _forced(mode)
    b = _block_step(i, dt, dict(aux_alpha=alpha), forced)
    f64 = lambda a: to_np(a).astype(np.float64)
    rxn, rs, _ = norm_ref.forward(f64(i["x"]), f64(i["nw"]), EPS, f64(i["res"]))
    assert_close("s", to_np(b.s), rs, rel=rel, max_frac=frac)
    assert_close("xn", to_np(b.xn), rxn, rel=rel, max_frac=frac)
    xn, w = f64(b.xn), [f64(a) for a in i["w"]]
    f = moe_ref.layer_forward(xn, *w, K, forced_idx=to_np(forced))
    g = moe_ref.layer_backward(f, f64(i["dy"]), xn, *w, aux_alpha=alpha)
    for n, got, want in (("y", b.layer.y, f["y"]), ("dxn", b.layer.dx, g["dx"]), ("dw1", b.layer.dw1, g["dw1"]),
                         ("dw3", b.layer.dw3, g["dw3"]), ("dw2", b.layer.dw2, g["dw2"]), ("dwr", b.layer.dwr, g["dwr"])):
        assert_close(n, to_np(got), want, rel=rel, max_frac=frac)
    rdx, rdw = norm_ref.backward(f64(b.layer.dx), f64(b.s), f64(i["nw"]), f64(b.rstd), f64(i["ds"]))
    assert_close("dx", to_np(b.dx), rdx, rel=rel, max_frac=frac)
    assert_close("dnorm_w", to_np(b.dnorm_w), rdw, rel=rel, max_frac=frac)
