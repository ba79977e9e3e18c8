"""The dense and update calls at the sizes where their launches change: every form
of the few-token product, more matrices than one launch counts, and tensors of
more than 2^31 elements (sampled rows and matrices).  Tolerances as in
test_gpu_dense.py and test_gpu_muon.py."""

import numpy as np
import pytest
import torch

from oracle import dense_ref as ref

from helpers import say
from test_gpu_dense import ACTS, DT, HALF, U, _abi, _check, _f64, _inputs, _ws, g_of
from test_gpu_muon import DEV, _check_one

pytestmark = pytest.mark.gpu


def _check_forward(i, y, z, act, rows):
    x, w, b, r = _f64(i["x"][rows]), _f64(i["w"]), _f64(i["b"]), _f64(i["r"][rows])
    dt = "f32" if y.dtype == torch.float32 else "bf16"
    ry, rz = ref.linear(x, w, b, r, act)
    bz = g_of(x.shape[1]) * (np.abs(x) @ np.abs(w).T) + 2 * U * np.abs(rz)
    _check("z", z[rows], rz, bz, HALF[dt])
    _check("y", y[rows], ry, 1.13 * bz + 16 * U * (1 + np.abs(rz)) + 2 * U * np.abs(ry), HALF[dt])


# one or two row tiles a workgroup, one or two token tiles, their last rows ragged
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,n,K", [(4, 6152, 136), (5, 6136, 136), (5, 6144, 1032), (16, 6168, 200), (17, 6152, 520),
                                   (32, 6168, 264), (32, 40, 1024), (31, 6136, 72), (33, 6152, 72), (20, 72, 4104)])
def test_few_tokens(T, n, K, dt):
    say(f"few tokens {T} {n} {K} {dt}")
    abi, i, act = _abi(), _inputs(T, n, K, dt, 60), ACTS[(T + n) % 4]
    y, z = torch.full_like(i["r"], np.nan), torch.full_like(i["r"], np.nan)
    ws = _ws(abi, abi.moe_linear_workspace_size, T, n, K, DT[dt])
    abi.moe_linear_fwd(i["x"], i["w"], y, ws, bias=i["b"], res=i["r"], act=act, z=z)
    _check_forward(i, y, z, act, slice(None))
    y2 = i["r"].clone()  # the residual in place
    abi.moe_linear_fwd(i["x"], i["w"], y2, ws, bias=i["b"], res=y2, act=act)
    assert torch.equal(y, y2)


def test_more_than_2_31_outputs():
    T, n, K = 270001, 8200, 64
    say(f"linear {T} {n} {K}")
    abi = _abi()
    g = torch.Generator(device=DEV).manual_seed(61)
    mk = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.bfloat16)
    i = dict(x=mk(T, K), w=mk(n, K).mul_(0.1), b=mk(n), r=mk(T, n))
    y, z = torch.empty_like(i["r"]), torch.empty_like(i["r"])
    abi.moe_linear_fwd(i["x"], i["w"], y, _ws(abi, abi.moe_linear_workspace_size, T, n, K, y.dtype), bias=i["b"],
                       res=i["r"], act="silu", z=z)
    # around 2^31 elements, and the ends
    edge = 2 ** 31 // n
    rows = torch.tensor([0, 1, edge - 1, edge, edge + 1, T - 200, T - 1], device=DEV)
    _check_forward(i, y, z, "silu", rows)
    # its gradients, from dy = y
    dx, dw, db = torch.empty_like(i["x"]), torch.empty_like(i["w"]), torch.empty_like(i["b"])
    abi.moe_linear_bwd(y, i["x"], i["w"], _ws(abi, abi.moe_linear_bwd_workspace_size, T, n, K, y.dtype), act="silu", z=z,
                       dx=dx, dw=dw, dbias=db)
    dy, w, zz = _f64(y[rows]), _f64(i["w"]), _f64(z[rows])
    rx, _, _, rz = ref.linear_bwd(dy, _f64(i["x"][rows]), w, zz, "silu")
    e = HALF["bf16"] * np.abs(rz) + 16 * U * np.abs(dy) * (1 + np.abs(zz)) * (1 + HALF["bf16"])
    _check("dx", dx[rows], rx, g_of(n) * ((np.abs(rz) + e) @ np.abs(w)) + e @ np.abs(w), HALF["bf16"])
    cols = torch.tensor([0, 4099, n - 1], device=DEV)  # three of dW's rows, over every token
    dy, x, zz = _f64(y[:, cols]), _f64(i["x"]), _f64(z[:, cols])
    _, rw, rb, rz = ref.linear_bwd(dy, x, w[cols.cpu().numpy()], zz, "silu")
    ez = 16 * U * np.abs(dy) * (1 + np.abs(zz))
    e = HALF["bf16"] * np.abs(rz) + ez * (1 + HALF["bf16"])
    mag = np.abs(rz) + e
    _check("dw", dw[cols], rw, g_of(T) * (mag.T @ np.abs(x)) + e.T @ np.abs(x), HALF["bf16"])
    _check("db", db[cols], rb, g_of(T) * mag.sum(0) + ez.sum(0), HALF["bf16"])


def test_more_matrices_than_a_launch_counts():
    B, rows, cols = 33001, 3, 8
    say(f"orthogonalize {B} {rows} {cols}")
    abi = _abi()
    g = torch.randn(B, rows, cols, device=DEV, generator=torch.Generator(device=DEV).manual_seed(62)).bfloat16()
    out = torch.full_like(g, np.nan)
    abi.moe_orthogonalize(g, out, _ws(abi, abi.moe_orthogonalize_workspace_size, B, rows, cols, g.dtype))
    assert torch.isfinite(out).all()
    for b in (0, 1, 32767, 32768, 32769, B - 1):
        _check_one(_f64(out[b]), _f64(g[b]), "f32", half=HALF["bf16"])


def test_more_than_2_31_values_of_matrices():
    B, rows, cols = 8400, 64, 4096
    say(f"muon {B} {rows} {cols}")
    abi = _abi()
    gen = torch.Generator(device=DEV).manual_seed(63)
    g = torch.randn(B, rows, cols, device=DEV, generator=gen, dtype=torch.bfloat16)
    w = torch.randn(B, rows, cols, device=DEV, generator=gen, dtype=torch.bfloat16).mul_(0.02)
    buf = torch.zeros(B, rows, cols, device=DEV)
    at = (0, 2015, 2016, 8191, 8192, B - 1)  # (chunks of the batch, and 2^31 values)
    w0 = {b: _f64(w[b]) for b in at}
    abi.moe_muon_step(w, g, buf, _ws(abi, abi.moe_orthogonalize_workspace_size, B, rows, cols, g.dtype), step=0.5,
                      momentum=0.0)
    for b in at:
        assert torch.equal(buf[b], g[b].float())
        _check_one(_f64(w[b]), _f64(g[b]), "bf16", scale=-0.5, base=w0[b])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,n", [(1, 8), (63, 72), (64, 64), (256, 136), (257, 520), (319, 56), (320, 264), (321, 200), (513, 72)])
def test_bias_gradient(T, n, dt):
    """In one launch with dz up to 320 rows, from partial sums above."""
    K, act = 64, ACTS[(T + n // 8) % 4]
    if dt == "f32":
        n -= 4
    say(f"bias gradient {T} {n} {dt} {act}")
    abi, i = _abi(), _inputs(T, n, K, dt, 64)
    ws = _ws(abi, abi.moe_linear_bwd_workspace_size, T, n, K, DT[dt])
    db, dx, alone = torch.full_like(i["b"], np.nan), torch.full_like(i["x"], np.nan), torch.full_like(i["x"], np.nan)
    z = None if act == "none" else i["z"]
    abi.moe_linear_bwd(i["dy"], i["x"], i["w"], ws, act=act, z=z, dbias=db, dx=dx)
    abi.moe_linear_bwd(i["dy"], i["x"], i["w"], ws.fill_(0xFF), act=act, z=z, dx=alone)
    assert torch.equal(dx, alone)
    dy, zz = _f64(i["dy"]), _f64(i["z"])
    _, _, rb, rz = ref.linear_bwd(dy, _f64(i["x"]), _f64(i["w"]), zz, act)
    ez = 0 * dy if act == "none" else 16 * U * np.abs(dy) * (1 + np.abs(zz))
    _check("db", db, rb, g_of(T) * (np.abs(rz) + ez).sum(0) + ez.sum(0), HALF[dt])
