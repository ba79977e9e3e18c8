"""moe_linear_fwd / _bwd against the float64 oracle.

Tolerances.  Products of bf16 values are exact in fp32; a sum of N products is
within g(N) = (N + 64) 2^-23 of the sum of their magnitudes (a whole step each:
the matrix instructions' inner sums may truncate).  z adds the bias: one more
term.  An activation has a slope under 1.13 and its fp32 evaluation is within
16 2^-24 (1 + |z|).  dz is rounded once to its type (HALF, relative) before the
two products.  Each output is rounded once.
"""

import numpy as np
import pytest
import torch

from oracle import dense_ref as ref

from helpers import say, to_np

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
ACTS = ("none", "relu", "gelu", "silu")
TINY = 1e-37


def g_of(n):
    return (n + 64) * 2.0 ** -23


def _abi():
    from token_routing_grouped_amd import _abi as a

    return a


def _f64(t):
    return to_np(t).astype(np.float64)


def _inputs(T, n, K, dt, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 131 * T + 17 * n + K)
    mk = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV).mul_(std).to(DT[dt])
    return dict(x=mk(T, K), w=mk(n, K, std=0.1), b=mk(n), r=mk(T, n, std=2.0), dy=mk(T, n), z=mk(T, n))


def _ws(abi, f, *size):
    return abi.workspace(f(*size), DEV).fill_(0xFF)


def _check(name, got, want, bound, half):
    got = _f64(got)
    lim = half * np.abs(want) + bound * (1 + half) + TINY
    bad = ~(np.abs(got - want) <= lim)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.abs(got - want).max()))


# one row, one tile's edges, ragged in each direction, several K steps, parts of K
SHAPES = [(1, 8, 8), (1, 136, 264), (3, 64, 72), (16, 16, 512), (17, 48, 2048), (64, 256, 128), (65, 264, 520),
          (127, 120, 64), (128, 128, 128), (129, 136, 200), (255, 72, 1032), (300, 520, 136), (513, 1032, 72),
          (33, 2056, 24)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,n,K", SHAPES)
@pytest.mark.parametrize("act,bias,res", [("none", False, False), ("relu", True, False), ("gelu", True, True),
                                          ("silu", False, True)])
def test_forward(T, n, K, dt, act, bias, res):
    if dt == "f32":
        n, K = n - 4, K - 4  # rows of an odd number of 16-byte pieces
    say(f"linear fwd {T} {n} {K} {dt} {act}")
    abi, i = _abi(), _inputs(T, n, K, dt)
    b, r = i["b"] if bias else None, i["r"] if res else None
    y, z = torch.full_like(i["r"], np.nan), torch.full_like(i["r"], np.nan)
    ws = _ws(abi, abi.moe_linear_workspace_size, T, n, K, DT[dt])
    abi.moe_linear_fwd(i["x"], i["w"], y, ws, bias=b, res=r, act=act, z=z)
    x, w = _f64(i["x"]), _f64(i["w"])
    ry, rz = ref.linear(x, w, None if b is None else _f64(b), None if r is None else _f64(r), act)
    bz = g_of(K) * (np.abs(x) @ np.abs(w).T) + (2 * U * np.abs(rz) if bias else 0)
    by = 1.13 * bz + 16 * U * (1 + np.abs(rz)) + 2 * U * np.abs(ry)
    _check("z", z, rz, bz, HALF[dt])
    _check("y", y, ry, by, HALF[dt])
    y2 = torch.empty_like(y)  # y does not change with whether z is kept; the residual in place
    if r is not None:
        y2.copy_(r)
        r = y2
    abi.moe_linear_fwd(i["x"], i["w"], y2, ws, bias=b, res=r, act=act)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,n,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_backward(T, n, K, dt, act):
    if dt == "f32":
        n, K = n - 4, K - 4
    say(f"linear bwd {T} {n} {K} {dt} {act}")
    abi, i = _abi(), _inputs(T, n, K, dt, 5)
    z = None if act == "none" else i["z"]
    dx, dw, db = (torch.full_like(v, np.nan) for v in (i["x"], i["w"], i["b"]))
    ws = _ws(abi, abi.moe_linear_bwd_workspace_size, T, n, K, DT[dt])
    abi.moe_linear_bwd(i["dy"], i["x"], i["w"], ws, act=act, z=z, dx=dx, dw=dw, dbias=db)
    dy, x, w = _f64(i["dy"]), _f64(i["x"]), _f64(i["w"])
    rx, rw, rb, rz = ref.linear_bwd(dy, x, w, _f64(i["z"]), act)
    ez = 0 if act == "none" else 16 * U * np.abs(dy) * (1 + np.abs(_f64(i["z"])))
    e = 0 if act == "none" else HALF[dt] * np.abs(rz) + ez * (1 + HALF[dt])
    mag = np.abs(rz) + e
    _check("dx", dx, rx, g_of(n) * (mag @ np.abs(w)) + (e @ np.abs(w) if act != "none" else 0), HALF[dt])
    _check("dw", dw, rw, g_of(T) * (mag.T @ np.abs(x)) + (e.T @ np.abs(x) if act != "none" else 0), HALF[dt])
    _check("db", db, rb, g_of(T) * mag.sum(0) + (np.sum(ez, axis=0) if act != "none" else 0), HALF[dt])
    # each by itself gives the same bits
    for name, full in (("dx", dx), ("dw", dw), ("dbias", db)):
        one = torch.full_like(full, np.nan)
        abi.moe_linear_bwd(i["dy"], i["x"], i["w"], ws.fill_(0xFF), act=act, z=z, **{name: one})
        assert torch.equal(one, full), name


@pytest.mark.parametrize("T,n,K", [(4104, 4104, 72), (2056, 8200, 40)])
def test_many_tiles(T, n, K):
    """Enough output for the largest tiles, ragged at each edge, all layouts."""
    say(f"linear many tiles {T} {n} {K}")
    abi, i = _abi(), _inputs(T, n, K, "bf16", 9)
    y = torch.full_like(i["r"], np.nan)
    abi.moe_linear_fwd(i["x"], i["w"], y, _ws(abi, abi.moe_linear_workspace_size, T, n, K, y.dtype))
    x, w = _f64(i["x"]), _f64(i["w"])
    _check("y", y, x @ w.T, g_of(K) * (np.abs(x) @ np.abs(w).T), HALF["bf16"])
    # the same sizes as gradients: dx of [T, K'] sums over few columns, dw over few rows
    i = _inputs(T, K, n, "bf16", 10)
    dx = torch.full_like(i["x"], np.nan)
    abi.moe_linear_bwd(i["dy"], i["x"], i["w"], _ws(abi, abi.moe_linear_bwd_workspace_size, T, K, n, y.dtype), dx=dx)
    dy, w = _f64(i["dy"]), _f64(i["w"])
    _check("dx", dx, dy @ w, g_of(K) * (np.abs(dy) @ np.abs(w)), HALF["bf16"])
    i = _inputs(K, T, n, "bf16", 11)
    dw = torch.full_like(i["w"], np.nan)
    abi.moe_linear_bwd(i["dy"], i["x"], i["w"], _ws(abi, abi.moe_linear_bwd_workspace_size, K, T, n, y.dtype), dw=dw)
    dy, x = _f64(i["dy"]), _f64(i["x"])
    _check("dw", dw, dy.T @ x, g_of(K) * (np.abs(dy).T @ np.abs(x)), HALF["bf16"])


def test_no_rows():
    abi = _abi()
    for dt in DT.values():
        x, w = torch.empty(0, 64, dtype=dt, device=DEV), torch.ones(48, 64, dtype=dt, device=DEV)
        y = torch.empty(0, 48, dtype=dt, device=DEV)
        abi.moe_linear_fwd(x, w, y, _ws(abi, abi.moe_linear_workspace_size, 0, 48, 64, dt))
        dw, db = torch.full_like(w, np.nan), torch.full_like(w[:, 0], np.nan)
        abi.moe_linear_bwd(y, x, w, _ws(abi, abi.moe_linear_bwd_workspace_size, 0, 48, 64, dt), act="gelu", z=y,
                           dx=x, dw=dw, dbias=db)
        assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T", [2, 70])
def test_what_lies_around_is_not_read_or_written(T):
    """Operands with NaNs before and behind them, outputs inside guarded
    buffers: every K tail reads as zero and no edge is crossed."""
    abi, n, K, pad = _abi(), 40, 88, 256
    i = _inputs(T, n, K, "bf16", 3)

    def inside(t, fill=np.nan):
        big = torch.full((t.numel() + 2 * pad,), fill, dtype=t.dtype, device=DEV)
        v = big[pad:pad + t.numel()].view(t.shape)
        v.copy_(t)
        return big, v

    held = {k: inside(v) for k, v in i.items()}
    v = {k: h[1] for k, h in held.items()}
    out = {k: inside(torch.zeros_like(s), 7.0) for k, s in (("y", i["r"]), ("z", i["r"]), ("dx", i["x"]),
                                                            ("dw", i["w"]), ("db", i["b"]))}
    o = {k: h[1] for k, h in out.items()}
    wsf = _ws(abi, abi.moe_linear_workspace_size, T, n, K, torch.bfloat16)
    wsb = _ws(abi, abi.moe_linear_bwd_workspace_size, T, n, K, torch.bfloat16)
    abi.moe_linear_fwd(v["x"], v["w"], o["y"], wsf, bias=v["b"], res=v["r"], act="silu", z=o["z"])
    abi.moe_linear_bwd(v["dy"], v["x"], v["w"], wsb, act="silu", z=v["z"], dx=o["dx"], dw=o["dw"], dbias=o["db"])
    for k, (big, t) in out.items():
        assert torch.isfinite(t).all(), k
        assert (big[:pad] == 7).all() and (big[pad + t.numel():] == 7).all(), k
    y = torch.empty_like(o["y"])
    abi.moe_linear_fwd(i["x"], i["w"], y, wsf, bias=i["b"], res=i["r"], act="silu")
    assert torch.equal(y, o["y"])


def test_one_bad_token_stays_its_own():
    """NaN and infinity in a token's row reach that row of z and y alone."""
    abi, T, n, K = _abi(), 130, 72, 96
    i = _inputs(T, n, K, "bf16", 4)
    ws = _ws(abi, abi.moe_linear_workspace_size, T, n, K, torch.bfloat16)
    clean, y = torch.empty_like(i["r"]), torch.empty_like(i["r"])
    for act in ACTS:
        abi.moe_linear_fwd(i["x"], i["w"], clean, ws, act=act)
        x = i["x"].clone()
        x[5, 3], x[129, 95] = float("nan"), float("inf")
        abi.moe_linear_fwd(x, i["w"], y, ws, act=act)
        keep = torch.ones(T, dtype=torch.bool, device=DEV)
        keep[[5, 129]] = False
        assert torch.equal(y[keep], clean[keep]) and y[5].isnan().all()


def test_gradient_by_differences():
    """The loss's change along a direction, forward differences of the GPU's own
    fp32 forward: step 2^-6, so curvature adds at most about 1e-2 of the slope
    and rounding 1e-4."""
    abi, T, n, K = _abi(), 37, 44, 52
    for act in ACTS:
        i = _inputs(T, n, K, "f32", 6)
        ws = _ws(abi, abi.moe_linear_workspace_size, T, n, K, torch.float32)
        wsb = _ws(abi, abi.moe_linear_bwd_workspace_size, T, n, K, torch.float32)

        def loss(x, w, b):
            y = torch.empty_like(i["r"])
            abi.moe_linear_fwd(x, w, y, ws, bias=b, act=act, z=i["z"])
            return (y.double() * i["dy"].double()).sum().item()

        dx, dw, db = (torch.empty_like(v) for v in (i["x"], i["w"], i["b"]))
        loss(i["x"], i["w"], i["b"])
        abi.moe_linear_bwd(i["dy"], i["x"], i["w"], wsb, act=act, z=i["z"], dx=dx, dw=dw, dbias=db)
        h = 2.0 ** -6
        for name, grad in (("x", dx), ("w", dw), ("b", db)):
            d = grad / grad.double().norm().float()  # along the gradient itself: slope = its norm
            args = lambda s: [i[k] + s * d if k == name else i[k] for k in ("x", "w", "b")]
            got = (loss(*args(h)) - loss(*args(-h))) / (2 * h)
            want = grad.double().norm().item()
            assert abs(got - want) <= 1e-2 * want, (act, name, got, want)


def test_captured_and_replayed():
    """Forward and backward in one graph, replayed with new inputs in the same
    buffers, eager work of the same calls between the replays."""
    abi, T, n, K = _abi(), 150, 264, 512
    i = _inputs(T, n, K, "bf16", 12)
    mk = lambda: [torch.empty_like(v) for v in (i["r"], i["r"], i["x"], i["w"], i["b"])]
    ws = [_ws(abi, abi.moe_linear_workspace_size, T, n, K, torch.bfloat16) for _ in range(2)]
    wsb = [_ws(abi, abi.moe_linear_bwd_workspace_size, T, n, K, torch.bfloat16) for _ in range(2)]

    def step(o, k):
        y, z, dx, dw, db = o
        abi.moe_linear_fwd(i["x"], i["w"], y, ws[k], bias=i["b"], res=i["r"], act="gelu", z=z)
        abi.moe_linear_bwd(i["dy"], i["x"], i["w"], wsb[k], act="gelu", z=z, dx=dx, dw=dw, dbias=db)

    a, b = mk(), mk()
    step(a, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step(a, 0)
    torch.cuda.current_stream().wait_stream(s)
    for rep in range(4):
        for k, v in _inputs(T, n, K, "bf16", 20 + rep).items():
            i[k].copy_(v)
        step(b, 1)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(a, b):
            assert torch.equal(p, q), rep


def test_two_streams_at_once():
    abi, T, n, K = _abi(), 200, 520, 1024
    i = _inputs(T, n, K, "bf16", 30)
    ws = _ws(abi, abi.moe_linear_workspace_size, T, n, K, torch.bfloat16)
    want = torch.empty_like(i["r"])
    abi.moe_linear_fwd(i["x"], i["w"], want, ws, act="silu")
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(want) for _ in range(2)]
    wss = [_ws(abi, abi.moe_linear_workspace_size, T, n, K, torch.bfloat16) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, wk in zip(streams, outs, wss):
            with torch.cuda.stream(s):
                abi.moe_linear_fwd(i["x"], i["w"], o, wk, act="silu")
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
