"""gelu and silu far from zero, where their values are small but not nothing:
relative to the value, forward and slope, through each way a product takes.

The weights are the identity, so z is x exactly (sums of one value and zeros).
Tolerances, in U = 2^-24 relative to the value (for a slope: to the magnitudes
of its two terms), besides the output's rounding:
  gelu  Phi(z) = erfc(-z / sqrt 2) / 2.  The argument is off by two roundings, and
        erfc's condition number is at most 2 x^2 + 1 = z^2 + 1: 2 (z^2 + 1) U; the
        function itself by at most 16 ulp = 32 U (bf16: the fit's 5.3e-7 = 9 U, the
        exponential's argument 1.25 z^2 U, a few roundings); three products and sums.
        The density's exponential: z^2 U from its argument, 4 U of its own.
        Together under (48 + 3 z^2) U.  Where z^2 passes 200, Phi is 0 or 1.
  silu  the exponential's argument is off by three roundings (|z| log2 e in bf16's):
        under 4 |z| U; the function, the sum and the reciprocal under 16 U; a slope's
        1 - s by U absolutely, times |z| s.
What is under 1e-37 may be zero."""

import numpy as np
import pytest
import torch

from oracle import dense_ref as ref

from helpers import say
from test_gpu_dense import DEV, DT, HALF, TINY, U, _abi, _f64, _ws

pytestmark = pytest.mark.gpu

N = 64


def _points(T, dt, far):
    z = np.linspace(-far, far, T * N).astype(np.float32)
    if far < 20:
        z[:8] = [-1e30, -1e4, -100, -15, 15, 100, 1e4, 1e30]
    return torch.from_numpy(np.random.default_rng(T).permutation(z)).view(T, N).to(DEV).to(DT[dt])


# a few tokens; tiles
@pytest.mark.parametrize("T", [16, 96])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act,far", [("gelu", 13.0), ("silu", 80.0)])
def test_values_and_slopes(act, far, dt, T):
    say(f"tails {act} {dt} {T}")
    abi, x = _abi(), _points(T, dt, far)
    w = torch.eye(N, device=DEV, dtype=x.dtype)
    y, z, dx = (torch.full_like(x, np.nan) for _ in range(3))
    abi.moe_linear_fwd(x, w, y, _ws(abi, abi.moe_linear_workspace_size, T, N, N, x.dtype), act=act, z=z)
    assert torch.equal(z, x)
    abi.moe_linear_bwd(torch.ones_like(x), x, w, _ws(abi, abi.moe_linear_bwd_workspace_size, T, N, N, x.dtype), act=act,
                       z=z, dx=dx)
    v = _f64(x)
    a = np.abs(v)
    if act == "gelu":
        rel = (48 + 3 * np.minimum(v * v, 200.0)) * U
        p = ref.act(v, act) / v
        terms, extra = p + a * np.exp(-np.minimum(v * v, 1e3) / 2) / np.sqrt(2 * np.pi), 0.0
    else:
        rel = (32 + 4 * a) * U
        s = ref.act(v, act) / v
        terms, extra = s + a * s * (1 - s), 4 * U * a * s
    with np.errstate(over="ignore"):
        for name, got, want, mag in (("y", y, ref.act(v, act), a * (terms * 0 + ref.act(v, act) / v)),
                                     ("slope", dx, ref.slope(v, act), terms)):
            lim = HALF[dt] * np.abs(want) + (1 + HALF[dt]) * (rel * mag + (extra if name == "slope" else 0)) + TINY
            bad = ~(np.abs(_f64(got) - want) <= lim)
            at = np.argwhere(bad)[:4]
            assert not bad.any(), (name, int(bad.sum()), [(v[tuple(i)], _f64(got)[tuple(i)], want[tuple(i)]) for i in at])
