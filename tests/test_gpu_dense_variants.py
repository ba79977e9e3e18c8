"""Every launch variant of the dense products and of the orthogonalised update, at
dense_variants.py's shapes, against the float64 oracle at test_gpu_dense.py's and
test_gpu_muon.py's tolerances."""

import numpy as np
import pytest
import torch

from oracle import dense_ref as ref

import dense_variants as dv
from helpers import say
from test_gpu_dense import ACTS, DEV, DT, HALF, U, _abi, _check, _f64, _inputs, _ws, g_of
from test_gpu_muon import FAR, _gradients, _model, evaluation

pytestmark = pytest.mark.gpu


def _check_forward(i, y, z, act, dt):
    x, w, b, r = (_f64(i[k]) for k in ("x", "w", "b", "r"))
    ry, rz = ref.linear(x, w, b, r, act)
    bz = g_of(x.shape[1]) * (np.abs(x) @ np.abs(w).T) + 2 * U * np.abs(rz)
    _check("z", z, rz, bz, HALF[dt])
    _check("y", y, ry, 1.13 * bz + 16 * U * (1 + np.abs(rz)) + 2 * U * np.abs(ry), HALF[dt])


@pytest.mark.parametrize("dt,T,n,K,tiles", [(dt, *s) for dt in dv.FEW for s in dv.FEW[dt]])
def test_few_tokens(dt, T, n, K, tiles):
    assert dv.forward(T, n, K, dt).row_tiles == tiles
    say(f"few tokens {dt} {T} {n} {K} {tiles}")
    abi, i, act = _abi(), _inputs(T, n, K, dt, 70), ACTS[(T + n // 8 + K // 8) % 4]
    y, z = torch.full_like(i["r"], np.nan), torch.full_like(i["r"], np.nan)
    ws = _ws(abi, abi.moe_linear_workspace_size, T, n, K, DT[dt])
    abi.moe_linear_fwd(i["x"], i["w"], y, ws, bias=i["b"], res=i["r"], act=act, z=z)
    _check_forward(i, y, z, act, dt)
    y2 = i["r"].clone()  # the residual in place
    abi.moe_linear_fwd(i["x"], i["w"], y2, ws, bias=i["b"], res=y2, act=act)
    assert torch.equal(y, y2)


def _full(like):
    return torch.full_like(like, np.nan)


@pytest.mark.parametrize("dt,T,n,K", [(dt, *s) for dt, layout in dv.PRODUCTS if layout == "fwd"
                                      for s in dv.PRODUCTS[dt, layout]])
def test_forward_tiles(dt, T, n, K):
    say(f"forward tiles {dt} {T} {n} {K} {dv.variant(dv.forward(T, n, K, dt))}")
    abi, i = _abi(), _inputs(T, n, K, dt, 71)
    ws = _ws(abi, abi.moe_linear_workspace_size, T, n, K, DT[dt])
    x, w, b, r = (_f64(i[k]) for k in ("x", "w", "b", "r"))
    rz = x @ w.T + b
    bz = g_of(K) * (np.abs(x) @ np.abs(w).T) + 2 * U * np.abs(rz)
    for act in ACTS:
        y, z = _full(i["r"]), _full(i["r"])
        abi.moe_linear_fwd(i["x"], i["w"], y, ws.fill_(0xFF), bias=i["b"], res=i["r"], act=act, z=z)
        _check(f"{act} z", z, rz, bz, HALF[dt])
        ry = ref.act(rz, act) + r
        _check(f"{act} y", y, ry, 1.13 * bz + 16 * U * (1 + np.abs(rz)) + 2 * U * np.abs(ry), HALF[dt])
        y2 = i["r"].clone()
        abi.moe_linear_fwd(i["x"], i["w"], y2, ws, bias=i["b"], res=y2, act=act)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("dt,layout,T,n,K", [(*k, *s) for k in dv.PRODUCTS if k[1] != "fwd" for s in dv.PRODUCTS[k]])
def test_gradient_tiles(dt, layout, T, n, K):
    say(f"{layout} tiles {dt} {T} {n} {K} {dv.variant(dv.gradient(T, n, K, dt, layout == 'dw'))}")
    abi, i = _abi(), _inputs(T, n, K, dt, 72)
    ws = _ws(abi, abi.moe_linear_bwd_workspace_size, T, n, K, DT[dt])
    dy, other = _f64(i["dy"]), _f64(i["w" if layout == "dx" else "x"])
    if layout == "dx":
        got = _full(i["x"])
        abi.moe_linear_bwd(i["dy"], i["x"], i["w"], ws, dx=got)
        a = dy
    else:
        got = _full(i["w"])
        abi.moe_linear_bwd(i["dy"], i["x"], i["w"], ws, dw=got)
        a = dy.T
    _check(layout, got, a @ other, g_of(a.shape[1]) * (np.abs(a) @ np.abs(other)), HALF[dt])


class Orthogonal:
    """What a matrix's result may be, as test_gpu_muon.py's _check_one has it."""

    def __init__(self, u, planes):
        name = "f32" if planes == 2 else "bf16"
        self.exact = ref.orthogonalize(u)
        self.e = ref.iterate(u, **_model(name)) - self.exact
        self.far, self.ev = FAR[name], evaluation(u, 5, 1e-7, planes == 2)

    def check(self, got, half, scale=1.0, base=0.0):
        want, s = base + scale * self.exact, abs(scale)
        err, norm = np.abs(got - want), np.linalg.norm
        out = half * norm(want) + 2.0 ** -23 * (norm(base) + s * norm(self.exact))
        assert norm(err) <= s * (self.far * norm(self.e) + self.ev) + out, (norm(err), s * norm(self.e))
        one = half * np.abs(want) + 2.0 ** -23 * (np.abs(base) + s * np.abs(self.exact)).max()
        assert (err <= s * (4 * np.abs(self.e).max() + self.ev) + one + 1e-30).all()


@pytest.mark.parametrize("B,rows,cols,dt,master", dv.MATRICES)
def test_matrix_tiles(B, rows, cols, dt, master):
    """Three matrices at most, over and over: the oracle looks at each once (of more
    than 2^21 values: at the last), and every copy has its bits."""
    plan = dv.ortho(B, rows, cols, dt, master)
    say(f"matrix tiles {B} {rows} {cols} {dt} {master}", *(dv.variant(getattr(plan, n)) for n in ("gram", "square", "update")))
    abi, k = _abi(), min(B, 3)
    g3 = _gradients(k, rows, cols, dt, 73)
    w3 = torch.randn(k, rows, cols, device=DEV, generator=torch.Generator(device=DEV).manual_seed(74)).mul_(0.05)
    again = lambda t: t[torch.arange(B, device=DEV) % k].contiguous()
    g, w32 = again(g3), again(w3)
    w, buf = w32.to(DT[dt]), torch.zeros_like(w32)
    outs = dict(w_out=_full(w), buf_out=_full(buf), master_out=_full(w32) if master else None)
    ws = _ws(abi, abi.moe_orthogonalize_workspace_size, B, rows, cols, DT[dt])
    # momentum 0: what is orthogonalised is g
    abi.moe_muon_step(w, g, buf, ws, step=0.5, decay=0.25, momentum=0.0, nesterov=False, master=w32 if master else None, **outs)
    assert torch.equal(outs["buf_out"], g.float())
    if not master:
        outs["o"] = _full(g)
        abi.moe_orthogonalize(g, outs["o"], ws.fill_(0xFF))
    for name in ("w_out", "master_out", "o"):
        t = outs.get(name)
        assert t is None or torch.equal(t, again(t[:k])), name
    for b in range(k - 1 if rows * cols > 1 << 21 else 0, k):
        ortho = Orthogonal(_f64(g[b]), plan.planes)
        base = 0.75 * _f64((w32 if master else w)[b])
        ortho.check(_f64(outs["w_out"][b]), HALF[dt], -0.5, base)
        if master:
            ortho.check(_f64(outs["master_out"][b]), HALF["f32"], -0.5, base)
            assert torch.equal(outs["master_out"][b].to(w.dtype), outs["w_out"][b])
        else:
            ortho.check(_f64(outs["o"][b]), HALF[dt])


@pytest.mark.parametrize("layout,T,n,K", [("fwd", 267, 11248, 288), ("fwd", 131, 11536, 528), ("fwd", 8236, 1496, 280),
                                          ("dx", 11042, 264, 304), ("dx", 10934, 280, 1048),
                                          ("dw", 281, 11408, 272), ("dw", 269, 13184, 920)])
def test_what_lies_around_wide_tiles(layout, T, n, K):
    """Operands with NaNs before and behind them, the result in a guarded buffer."""
    say(f"around {layout} {T} {n} {K} {dv.variant(dv.product(layout, T, n, K, 'bf16')[0])}")
    abi, i, pad = _abi(), _inputs(T, n, K, "bf16", 75), 1 << 16

    def inside(t, fill):
        big = torch.full((t.numel() + 2 * pad,), fill, dtype=t.dtype, device=DEV)
        v = big[pad:pad + t.numel()].view(t.shape)
        v.copy_(t)
        return big, v

    def call(v, out):
        if layout == "fwd":
            ws = _ws(abi, abi.moe_linear_workspace_size, T, n, K, out.dtype)
            abi.moe_linear_fwd(v["x"], v["w"], out, ws, bias=v["b"], res=v["r"], act="silu")
        else:
            ws = _ws(abi, abi.moe_linear_bwd_workspace_size, T, n, K, out.dtype)
            abi.moe_linear_bwd(v["dy"], v["x"], v["w"], ws, **{layout: out})

    want = torch.empty_like(i[{"fwd": "r", "dx": "x", "dw": "w"}[layout]])
    call(i, want)
    big, out = inside(torch.zeros_like(want), 7.0)
    call({k: inside(t, np.nan)[1] for k, t in i.items()}, out)
    assert torch.isfinite(want).all() and torch.equal(out, want)
    assert (big[:pad] == 7).all() and (big[pad + want.numel():] == 7).all()
