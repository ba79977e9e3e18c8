"""Where bf16 matrices are iterated in two fp16 planes: with fp32 master weights,
and with a side of at most 32.  Then the result is as exact as an fp32 matrix's,
at test_gpu_muon.py's tolerances for those, and is rounded once to what it is
stored in."""

import numpy as np
import pytest
import torch

from oracle import dense_ref as ref

from helpers import say
from test_gpu_muon import DEV, HALF, _abi, _check_one, _f64, _gradients, _ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,rows,cols", [(3, 16, 24), (2, 40, 64), (2, 136, 72), (1, 100, 600)])
def test_master_weights(B, rows, cols):
    say(f"muon planes {B} {rows} {cols}")
    abi = _abi()
    g, buf = _gradients(B, rows, cols, "bf16", 50), _gradients(B, rows, cols, "f32", 51)
    m = torch.randn(B, rows, cols, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).mul_(0.02)
    w, mo, wo, bo = m.bfloat16(), torch.full_like(m, np.nan), torch.full_like(g, np.nan), torch.empty_like(buf)
    abi.moe_muon_step(w, g, buf, _ws(abi, g), step=0.002, decay=3e-5, master=m, w_out=wo, buf_out=bo, master_out=mo)
    for b in range(B):
        # (the momentum 0.95 and the decay as the fp32 values that the call takes)
        mu, keep = float(np.float32(0.95)), 1.0 - float(np.float32(3e-5))
        _, rb = ref.muon(_f64(m[b]), _f64(g[b]), _f64(buf[b]), 0, 0, mu, True)
        _check_one(_f64(mo[b]), _f64(g[b]) + mu * rb, "f32", scale=-float(np.float32(0.002)), base=_f64(m[b]) * keep)
    assert torch.equal(mo.bfloat16(), wo)


@pytest.mark.parametrize("B,rows,cols", [(2, 16, 16), (2, 32, 200), (1, 1000, 24)])
def test_short_sides(B, rows, cols):
    say(f"orthogonalize planes {B} {rows} {cols}")
    abi = _abi()
    g = _gradients(B, rows, cols, "bf16", 52)
    out = torch.full_like(g, np.nan)
    abi.moe_orthogonalize(g, out, _ws(abi, g))
    for b in range(B):
        _check_one(_f64(out[b]), _f64(g[b]), "f32", half=HALF["bf16"])


def test_chunked_and_one_plane_fit_the_same_workspace():
    """The size that is asked for covers both forms of a call."""
    abi = _abi()
    for B, rows, cols in ((1, 64, 64), (128, 40, 4096), (3, 4096, 40), (600, 512, 512), (1, 33, 40)):
        one = abi.moe_orthogonalize_workspace_size(B, rows, cols, torch.bfloat16)
        assert one >= abi.moe_orthogonalize_workspace_size(B, rows, cols, torch.float32)


@pytest.mark.parametrize("master", [True, False])
def test_two_streams_at_once(master):
    """Two updates under way together, each with its own state and workspace."""
    say(f"muon two streams {master}")
    abi = _abi()
    g = _gradients(3, 200, 264, "bf16", 53)
    w0 = torch.randn(3, 200, 264, device=DEV, generator=torch.Generator(device=DEV).manual_seed(4)).mul_(0.05)

    def state():
        return [w0.bfloat16(), torch.zeros_like(w0), w0.clone(), _ws(abi, g)]

    def step(t):
        abi.moe_muon_step(t[0], g, t[1], t[3], step=0.1, decay=0.01, master=t[2] if master else None)

    want, both = state(), [state(), state()]
    for _ in range(4):
        step(want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, t in zip(streams, both):
            with torch.cuda.stream(s):
                step(t)
    torch.cuda.synchronize()
    for t in both:
        assert all(torch.equal(p, q) for p, q in zip(t[:3], want[:3]))
