"""moe_rmsnorm_fwd / _bwd against the float64 oracle.

Tolerances.  u = 2^-24 (half a step of fp32, relative).  A row's sum of squares
adds non-negative terms in at most 64 + 6 + 16 additions a lane, wave and
workgroup, so rstd is within (86 / 2 + 4) u of the exact one; with the
addition, the products and the conversions every y is within N u, N = 128, of
its exact value, relatively, before its own rounding (half a step of its type).
dx adds terms that may cancel, so its bound goes with the terms' magnitudes;
dw adds T terms, so its bound is (T + 64) u times the sum of their magnitudes.
"""

import numpy as np
import pytest
import torch

from oracle import mx_ref, norm_ref

from helpers import mx_scales_to_rows, say, to_np

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U, N = 2.0 ** -24, 128
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 1e-6

# T, d: one row, ragged rows, one piece, every waves-a-row / pieces-a-lane class
SHAPES = [(1, 8), (1, 2048), (3, 40), (5, 512), (7, 1000), (4, 2048), (2, 2056), (9, 4096), (3, 6144), (2, 8200),
          (2, 16384), (2, 16392), (1, 32768), (37, 136), (1030, 256)]


def _abi():
    from token_routing_grouped_amd import _abi as a

    return a


def _dev(a, dt):
    return torch.from_numpy(np.asarray(a, np.float32)).to(DEV).to(dt)


def _f64(t):
    return to_np(t).astype(np.float64)


def _inputs(T, d, dt, seed=0):
    g = np.random.default_rng(seed + 131 * T + d)
    x, res, dy, ds = (_dev(g.standard_normal((T, d)), dt) for _ in range(4))
    return x, res, _dev(1 + 0.2 * g.standard_normal(d), dt), dy, ds


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("with_res", [False, True])
def test_norm_forward(T, d, dt, with_res):
    say(f"norm fwd T={T} d={d} {dt} res={with_res}")
    abi = _abi()
    x, res, w, _, _ = _inputs(T, d, DT[dt])
    res = res if with_res else None
    y, s, rstd = torch.full_like(x, np.nan), torch.full_like(x, np.nan), torch.full((T,), np.nan, device=DEV)
    abi.moe_rmsnorm_fwd(x, w, EPS, y, res=res, s=s, rstd=rstd)
    ry, _, rr = norm_ref.forward(_f64(x), _f64(w), EPS, None if res is None else _f64(res))
    one = x.float() if res is None else x.float() + res.float()
    assert torch.equal(s, one.to(x.dtype))  # one fp32 addition, one rounding
    assert (np.abs(_f64(rstd) - rr) <= N * U * rr).all()
    assert (np.abs(_f64(y) - ry) <= (HALF[dt] + N * U) * np.abs(ry) + 1e-38).all()
    # neither output changes with which others are asked for
    y2 = torch.empty_like(x)
    abi.moe_rmsnorm_fwd(x, w, EPS, y2, res=res)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 32), (3, 96), (5, 128), (2, 160), (33, 2048), (130, 512), (3, 4128), (2, 6144),
                                 (2, 16416)])
def test_norm_mx_copy(T, d, dt):
    """The 8-bit copy: each scale from the block's largest y, each element
    within half an E4M3 step (2^-4 relative; 2^-10 of the scale below the
    smallest normal) of y, saturating at 448."""
    say(f"norm mx T={T} d={d} {dt}")
    abi = _abi()
    x, res, w, _, _ = _inputs(T, d, DT[dt], 7)
    x[0, :32] = 0
    res[0, :32] = 0  # an all-zero block
    y = torch.empty_like(x)
    q = torch.full((T, d), 0xEE, dtype=torch.uint8, device=DEV)
    qs = torch.full((abi.mx_scale_bytes(T, d),), 0xEE, dtype=torch.uint8, device=DEV)
    abi.moe_rmsnorm_fwd(x, w, EPS, y, res=res, q=q, qs=qs)
    ry, _, _ = norm_ref.forward(_f64(x), _f64(w), EPS, _f64(res))
    raw = to_np(qs).reshape(-1, T, 4)
    sb = mx_scales_to_rows(to_np(qs), T, d).astype(np.int64)
    # places past the row's last block hold 0
    assert not raw.transpose(1, 0, 2).reshape(T, -1)[:, d // 32:].any()
    b = ry.reshape(T, d // 32, 32)
    amax = np.abs(b).max(axis=2)
    want = mx_ref.block_scale_exp(amax) + 127
    m = np.frexp(amax)[0]  # in [0.5, 1): near either end the fp32 amax may sit across the power of two
    edge = (amax > 0) & ((m < 0.5 * (1 + 2 * N * U)) | (m > 1 - 2 * N * U))
    assert (np.abs(sb - want)[edge] <= 1).all() and (sb == want)[~edge].all()
    v = b / np.ldexp(1.0, sb - 127)[:, :, None]
    code = mx_ref.e4m3_decode(to_np(q)).reshape(v.shape)
    near = np.abs(code - np.clip(v, -448, 448)) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) * (1 + 2 * N * U)
    assert near.all()
    y2 = torch.empty_like(x)
    abi.moe_rmsnorm_fwd(x, w, EPS, y2, res=res)
    assert torch.equal(y, y2)
    q2, qs2 = torch.empty_like(q), torch.empty_like(qs)
    abi.moe_rmsnorm_fwd(x, w, EPS, None, res=res, q=q2, qs=qs2)
    assert torch.equal(q, q2) and torch.equal(qs, qs2)
    if dt == "f32":  # the same values through the quantiser
        abi.mx_quantize(y, T, q2, qs2.fill_(0), seg_rows=T)
        assert torch.equal(q, q2) and torch.equal(qs, qs2)


def test_norm_mx_copy_of_non_finite_rows():
    """A NaN in a row makes the whole row's y NaN: so do its codes; other rows
    are untouched.  An infinite value: its own y is NaN, the others' 0."""
    abi = _abi()
    x, _, w, _, _ = _inputs(4, 128, torch.bfloat16)
    clean = x.clone()
    x[1, 5], x[2, 9] = float("nan"), float("inf")
    out = []
    for v in (clean, x):
        y = torch.empty_like(x)
        q = torch.empty(4, 128, dtype=torch.uint8, device=DEV)
        qs = torch.empty(abi.mx_scale_bytes(4, 128), dtype=torch.uint8, device=DEV)
        abi.moe_rmsnorm_fwd(v, w, EPS, y, q=q, qs=qs)
        out.append((y, q, qs.view(1, 4, 4)))
    (y0, q0, s0), (y, q, s) = out
    for r in (0, 3):
        assert torch.equal(y[r], y0[r]) and torch.equal(q[r], q0[r]) and torch.equal(s[:, r], s0[:, r])
    assert y[1].isnan().all() and ((q[1] & 0x7F) == 0x7F).all()
    assert torch.equal(y[2].isnan(), torch.arange(128, device=DEV) == 9) and (q[2, 9] & 0x7F) == 0x7F
    keep = torch.arange(128, device=DEV) != 9
    assert ((q[2] & 0x7F)[keep] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_extreme_rows(dt):
    """Zero rows, rows of the smallest and of large values."""
    abi = _abi()
    d = 264
    x = torch.zeros(5, d, dtype=DT[dt], device=DEV)
    x[1], x[2], x[3, 7], x[4] = 1e-30, 1e15, -3.0, 1e-3
    w = torch.ones(d, dtype=DT[dt], device=DEV)
    y, rstd = torch.empty_like(x), torch.empty(5, device=DEV)
    abi.moe_rmsnorm_fwd(x, w, EPS, y, rstd=rstd)
    ry, _, rr = norm_ref.forward(_f64(x), _f64(w), EPS)
    assert (np.abs(_f64(y) - ry) <= (HALF[dt] + N * U) * np.abs(ry) + 1e-38).all()
    assert (np.abs(_f64(rstd) - rr) <= N * U * rr).all()
    dy = torch.ones_like(x)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = abi.workspace(abi.moe_rmsnorm_bwd_workspace_size(5, d), DEV)
    abi.moe_rmsnorm_bwd(dy, x, w, rstd, dx, dw, ws)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("alias", ["s_is_x", "s_is_res", "y_is_x"])
def test_norm_in_place(alias):
    abi = _abi()
    x, res, w, _, _ = _inputs(6, 2056, torch.bfloat16)
    y, s = torch.empty_like(x), torch.empty_like(x)
    abi.moe_rmsnorm_fwd(x, w, EPS, y, res=res, s=s)
    x2, res2, y2 = x.clone(), res.clone(), torch.empty_like(x)
    if alias == "y_is_x":
        s2 = torch.empty_like(x)
        abi.moe_rmsnorm_fwd(x2, w, EPS, x2, res=res2, s=s2)
        y2 = x2
    else:
        s2 = x2 if alias == "s_is_x" else res2
        abi.moe_rmsnorm_fwd(x2, w, EPS, y2, res=res2, s=s2)
    assert torch.equal(y, y2) and torch.equal(s, s2)


def _bwd_bounds(dy, s, w, rstd, ds, T, half):
    g, xh = dy * w, s * rstd[:, None]
    terms = rstd[:, None] * (np.abs(g) + np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True))
    if ds is not None:
        terms = terms + np.abs(ds)
    return N * U * terms, (T + 64) * U * np.sum(np.abs(dy * xh), axis=0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("with_ds", [False, True])
def test_norm_backward(T, d, dt, with_ds):
    say(f"norm bwd T={T} d={d} {dt} ds={with_ds}")
    abi = _abi()
    s, _, w, dy, ds = _inputs(T, d, DT[dt], 3)
    ds = ds if with_ds else None
    rstd = torch.from_numpy((1 / np.sqrt((_f64(s) ** 2).mean(axis=1) + EPS)).astype(np.float32)).to(DEV)
    dx, dw = torch.full_like(s, np.nan), torch.full_like(w, np.nan)
    ws = abi.workspace(abi.moe_rmsnorm_bwd_workspace_size(T, d), DEV).fill_(0xFF)
    abi.moe_rmsnorm_bwd(dy, s, w, rstd, dx, dw, ws, ds=ds)
    d64 = None if ds is None else _f64(ds)
    rx, rw = norm_ref.backward(_f64(dy), _f64(s), _f64(w), _f64(rstd), d64)
    bx, bw = _bwd_bounds(_f64(dy), _f64(s), _f64(w), _f64(rstd), d64, T, HALF[dt])
    assert (np.abs(_f64(dx) - rx) <= HALF[dt] * np.abs(rx) + bx * (1 + HALF[dt])).all()
    assert (np.abs(_f64(dw) - rw) <= HALF[dt] * np.abs(rw) + bw * (1 + HALF[dt])).all()
    # repeatable, and in place of either incoming gradient
    for target in [dy.clone()] + ([ds.clone()] if with_ds else []):
        dw2 = torch.empty_like(dw)
        if with_ds and target.data_ptr() != dy.data_ptr() and torch.equal(target, ds):
            abi.moe_rmsnorm_bwd(dy, s, w, rstd, target, dw2, ws, ds=target)
        else:
            abi.moe_rmsnorm_bwd(target, s, w, rstd, target, dw2, ws, ds=ds)
        assert torch.equal(target, dx) and torch.equal(dw2, dw)


def test_norm_backward_of_no_rows():
    abi = _abi()
    for dt in DT.values():
        e, w = torch.empty(0, 96, dtype=dt, device=DEV), torch.ones(96, dtype=dt, device=DEV)
        dw = torch.full_like(w, np.nan)
        ws = abi.workspace(abi.moe_rmsnorm_bwd_workspace_size(0, 96), DEV).fill_(0xFF)
        abi.moe_rmsnorm_bwd(e, e, w, torch.empty(0, device=DEV), e, dw, ws)
        abi.moe_rmsnorm_fwd(e, w, EPS, e)
        assert (dw == 0).all()


def test_norm_gradient_by_differences_on_the_gpu():
    """<dy, y(s + h u)> - <dy, y(s - h u)> over 2h against <dx, u>, all in fp32.
    The difference quotient's truncation is taken from the oracle's own; its
    rounding is at most 2 sum |dy y| N u / 2h."""
    abi = _abi()
    T, d, h = 6, 264, 2.0 ** -6
    s, direction, w, dy, _ = _inputs(T, d, torch.float32, 11)
    rstd = torch.empty(T, device=DEV)
    y = torch.empty_like(s)
    abi.moe_rmsnorm_fwd(s, w, EPS, y, rstd=rstd)
    dx, dw = torch.empty_like(s), torch.empty_like(w)
    abi.moe_rmsnorm_bwd(dy, s, w, rstd, dx, dw, abi.workspace(abi.moe_rmsnorm_bwd_workspace_size(T, d), DEV))
    ends, ref = [], []
    for sign in (1, -1):
        at = s + sign * h * direction
        abi.moe_rmsnorm_fwd(at, w, EPS, y)
        ends.append(np.sum(_f64(dy) * _f64(y)))
        ref.append(np.sum(_f64(dy) * norm_ref.forward(_f64(at), _f64(w), EPS)[0]))
    size = np.sum(np.abs(_f64(dy) * _f64(y)))
    exact_dir = np.sum(norm_ref.backward(_f64(dy), _f64(s), _f64(w), _f64(rstd))[0] * _f64(direction))
    truncation = abs((ref[0] - ref[1]) / (2 * h) - exact_dir)
    got = np.sum(_f64(dx) * _f64(direction))
    bound = truncation + 2 * size * N * U / (2 * h) + np.sum(np.abs(_f64(direction)) * 4) * N * U
    assert abs((ends[0] - ends[1]) / (2 * h) - got) <= bound
    assert truncation < 0.05 * abs(exact_dir)  # the quotient says something


@pytest.mark.parametrize("mx", [False, True])
def test_norm_captured_and_on_another_stream(mx):
    abi = _abi()
    T, d = 37, 2048
    x, res, w, dy, ds = _inputs(T, d, torch.bfloat16, 5)
    o = dict(y=torch.empty_like(x), s=torch.empty_like(x), rstd=torch.empty(T, device=DEV), dx=torch.empty_like(x),
             dw=torch.empty_like(w), q=torch.empty(T, d, dtype=torch.uint8, device=DEV),
             qs=torch.empty(abi.mx_scale_bytes(T, d), dtype=torch.uint8, device=DEV))
    ws = abi.workspace(abi.moe_rmsnorm_bwd_workspace_size(T, d), DEV)

    def step():
        abi.moe_rmsnorm_fwd(x, w, EPS, o["y"], res=res, s=o["s"], q=o["q"] if mx else None,
                            qs=o["qs"] if mx else None, rstd=o["rstd"])
        abi.moe_rmsnorm_bwd(dy, o["s"], w, o["rstd"], o["dx"], o["dw"], ws, ds=ds)

    names = [n for n in o if mx or n not in ("q", "qs")]
    step()
    torch.cuda.synchronize()
    want = {n: o[n].clone() for n in names}

    def wiped():
        for n in names:
            o[n].zero_()

    side = torch.cuda.Stream()
    wiped()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(o[n], want[n]) for n in names)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        wiped()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[n], want[n]) for n in names)
