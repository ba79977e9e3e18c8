"""Every launch variant of the dense products, at dense_variants.py's shapes, against
the float64 oracle at test_gpu_dense.py's tolerances."""

import numpy as np
import pytest
import torch

from oracle import dense_ref as ref

import dense_variants as dv
from helpers import say
from test_gpu_dense import ACTS, DT, HALF, U, _abi, _check, _f64, _inputs, _ws, g_of

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
