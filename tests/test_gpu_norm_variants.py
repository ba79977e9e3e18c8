"""The norm's row shapes and row loops that its smaller tests do not reach:
backward workgroups of 4 and 16 waves a row that take several rows each, more
than 256 partial weight gradients, and the widest rows.

Tolerances: u = 2^-24.  y and dx as in the smaller tests, N u = 128 u of the
terms' magnitudes before their own rounding (a lane adds at most 64 products,
then come 6 + 16 additions).  dw adds T terms, (T + 64) u of the sum of their
magnitudes, then its rounding.
"""

import numpy as np
import pytest
import torch

from oracle import norm_ref

from helpers import say, to_np

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U, N = 2.0 ** -24, 128
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _abi():
    from token_routing_grouped_amd import _abi as a

    return a


def _f64(t):
    return to_np(t).astype(np.float64)


def _dev(g, *n, dt, std=1.0, mean=0.0):
    return (torch.from_numpy(mean + std * g.standard_normal(n, dtype=np.float32))).to(DEV).to(dt)


# rows a workgroup: 3 and more on 256 workgroups, 2 and 3 (four at once), 8 and 9 on 512; the last unequal
@pytest.mark.parametrize("T,d,dt", [
    (771, 2056, "f32"), (1021, 1032, "f32"), (771, 4104, "bf16"), (515, 2056, "bf16"),  # 4 waves a row
    (773, 6144, "f32"), (771, 16392, "bf16"), (517, 4104, "f32"),                       # 16 waves
    (259, 32776, "bf16"), (258, 32768, "f32"),                                         # 16 waves, 8 pieces a lane
    (1100, 40, "bf16"), (4099, 40, "bf16"), (4099, 1032, "f32"), (4099, 2056, "bf16"), (8195, 264, "f32")])
def test_norm_backward_over_several_rows(T, d, dt):
    say(f"norm bwd T={T} d={d} {dt}")
    abi, g = _abi(), np.random.default_rng(T + d)
    s, dy, ds = (_dev(g, T, d, dt=DT[dt], std=sd) for sd in (2.0, 1.0, 1.0))
    w = _dev(g, d, dt=DT[dt], std=0.2, mean=1.0)
    rstd = torch.from_numpy((1 / np.sqrt((_f64(s) ** 2).mean(axis=1) + 1e-6)).astype(np.float32)).to(DEV)
    ws = abi.workspace(abi.moe_rmsnorm_bwd_workspace_size(T, d), DEV)
    first = None
    for fill in (0xFF, 0x3C):  # whatever the workspace and the outputs held
        ws.fill_(fill)
        dx, dw = torch.full_like(s, np.nan), torch.full_like(w, np.nan)
        abi.moe_rmsnorm_bwd(dy, s, w, rstd, dx, dw, ws, ds=ds)
        first = first or (dx, dw)
        assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])
    rw, mw = np.zeros(d), np.zeros(d)
    w64 = _f64(w)
    for r in range(0, T, 512):  # a part of the rows at a time, for the host's memory
        part = slice(r, min(r + 512, T))
        dy64, s64, ds64, r64 = _f64(dy[part]), _f64(s[part]), _f64(ds[part]), _f64(rstd[part])
        rx, pw = norm_ref.backward(dy64, s64, w64, r64, ds64)
        gg, xh = np.abs(dy64 * w64), np.abs(s64 * r64[:, None])
        terms = r64[:, None] * (gg + xh * np.mean(gg * xh, axis=1, keepdims=True)) + np.abs(ds64)
        assert (np.abs(_f64(dx[part]) - rx) <= HALF[dt] * np.abs(rx) + N * U * terms * (1 + HALF[dt])).all()
        rw += pw
        mw += np.sum(np.abs(dy64) * xh, axis=0)
    assert (np.abs(_f64(dw) - rw) <= HALF[dt] * np.abs(rw) + (T + 64) * U * mw * (1 + HALF[dt])).all()


@pytest.mark.parametrize("T,d,dt", [(3, 32800, "bf16"), (2, 65536, "bf16"), (2, 32768, "f32"), (70, 40960, "bf16")])
def test_norm_forward_of_the_widest_rows(T, d, dt):
    say(f"norm fwd T={T} d={d} {dt}")
    abi, g = _abi(), np.random.default_rng(T + d)
    x, res = _dev(g, T, d, dt=DT[dt]), _dev(g, T, d, dt=DT[dt])
    w = _dev(g, d, dt=DT[dt], std=0.2, mean=1.0)
    y, s, rstd = torch.full_like(x, np.nan), torch.full_like(x, np.nan), torch.full((T,), np.nan, device=DEV)
    q = torch.empty(T, d, dtype=torch.uint8, device=DEV)
    qs = torch.empty(abi.mx_scale_bytes(T, d), dtype=torch.uint8, device=DEV)
    abi.moe_rmsnorm_fwd(x, w, 1e-6, y, res=res, s=s, q=q, qs=qs, rstd=rstd)
    ry, _, rr = norm_ref.forward(_f64(x), _f64(w), 1e-6, _f64(res))
    assert torch.equal(s, (x.float() + res.float()).to(x.dtype))
    assert (np.abs(_f64(rstd) - rr) <= N * U * rr).all()
    assert (np.abs(_f64(y) - ry) <= (HALF[dt] + N * U) * np.abs(ry) + 1e-38).all()
    if dt == "f32":  # the 8-bit copy is the quantiser's of these very values
        q2, qs2 = torch.empty_like(q), torch.zeros_like(qs)
        abi.mx_quantize(y, T, q2, qs2, seg_rows=T)
        assert torch.equal(q, q2) and torch.equal(qs, qs2)


def test_norm_output_over_its_residual():
    abi, g = _abi(), np.random.default_rng(1)
    for T, d in ((6, 2056), (5, 512), (3, 16392)):
        x, res, w = _dev(g, T, d, dt=DT["bf16"]), _dev(g, T, d, dt=DT["bf16"]), _dev(g, d, dt=DT["bf16"])
        y, s, s2 = (torch.empty_like(x) for _ in range(3))
        abi.moe_rmsnorm_fwd(x, w, 1e-6, y, res=res, s=s)
        abi.moe_rmsnorm_fwd(x, w, 1e-6, res, res=res, s=s2)
        assert torch.equal(res, y) and torch.equal(s, s2)


def test_residual_stream_in_place_and_behind_the_live_tokens():
    """A decode layer's residual stream kept in its own buffer: forward(x,
    res=layer.s) adds x into all of the rows that x has, while y's rows behind
    the live tokens stay as they were."""
    from token_routing_grouped_amd.layer import MoEDecodeGPU

    g, bf = np.random.default_rng(2), torch.bfloat16
    T, d, E, h = 12, 256, 8, 64
    wr, w1, w3, w2 = (_dev(g, *n, dt=bf, std=n[-1] ** -0.5) for n in ((E, d), (E, h, d), (E, h, d), (E, d, h)))
    nw = _dev(g, d, dt=bf, std=0.1, mean=1.0)
    m, one = (MoEDecodeGPU(T, 2, wr, w1, w3, w2, norm_w=nw) for _ in range(2))
    x = _dev(g, T, d, dt=bf)
    m.forward(x)
    stream = x.clone()
    for live in (12, 5, 0, 7):
        step = _dev(g, T, d, dt=bf)
        m.y.fill_(9)
        n = torch.tensor([live], dtype=torch.int32, device=DEV)
        m.forward(step, res=m.s, n_live=n)
        one.forward(step, res=stream)
        stream = (step.float() + stream.float()).to(bf)
        assert torch.equal(m.s, stream)
        assert torch.equal(m.y[:live], one.y[:live]) and (m.y[live:] == 9).all()
