"""Sizes that the dense calls refuse because something that counts them would
wrap (no GPU needed; calls that pass are not made here)."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "token_routing_grouped_amd", "libtrg_moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")

P = [ctypes.c_void_p(1 << 20 | i << 12) for i in range(12)]
UNSUPPORTED = 2
BIG = 1 << 40


def _lib():
    from token_routing_grouped_amd import _abi

    return _abi.lib()


def _refused(status):
    msg = _lib().moe_last_error_string().decode()
    assert status == UNSUPPORTED and "too large" in msg, (status, msg)


@pytest.mark.parametrize("dt", [0, 1])
def test_tokens_whose_next_rows_pass_32_bits(dt):
    """A gradient's pass over its rows steps past the last one."""
    lib = _lib()
    for T in ((1 << 30) + 1, (1 << 31) - 64, (1 << 31) - 8, (1 << 31) - 1):
        assert lib.moe_linear_workspace_size(T, 8, 8, dt) == 0
        assert lib.moe_linear_bwd_workspace_size(T, 8, 8, dt) == 0
        _refused(lib.moe_linear_bwd(P[0], P[1], P[2], P[3], T, 8, 8, 2, dt, P[4], P[5], P[6], P[7], BIG, None))
        _refused(lib.moe_linear_fwd(P[0], P[1], None, None, T, 8, 8, 0, dt, None, P[2], P[3], BIG, None))
    assert lib.moe_linear_workspace_size(1 << 30, 8, 8, dt) > 0
    assert lib.moe_linear_bwd_workspace_size(1 << 30, 8, 8, dt) > 0


def test_sizes_past_32_bits_are_not_cut_down():
    """2^32 + 5 rows are not 5: refused by the binding (host views of one row)."""
    import torch

    from token_routing_grouped_amd import _abi

    bf, n = torch.bfloat16, (1 << 32) + 5
    x, w, ws = torch.zeros(1, 8, dtype=bf).expand(n, 8), torch.zeros(8, 8, dtype=bf), torch.zeros(64, dtype=torch.uint8)
    g = torch.zeros(1, 1, 8).expand(n, 1, 8)
    for call in (lambda: _abi.moe_linear_fwd(x, w, x, ws), lambda: _abi.moe_linear_fwd(w, x, w, ws),
                 lambda: _abi.moe_linear_bwd(x, x, w, ws, dx=x), lambda: _abi.moe_orthogonalize(g, g, ws),
                 lambda: _abi.moe_muon_step(g, g, g, ws, step=0.1),
                 lambda: _abi.moe_linear_workspace_size(n, 8, 8, bf), lambda: _abi.moe_linear_workspace_size(8, 8, n + 3, bf),
                 lambda: _abi.moe_linear_bwd_workspace_size(n, 8, 8, bf),
                 lambda: _abi.moe_orthogonalize_workspace_size(n, 8, 8, bf)):
        with pytest.raises(_abi.MoeError, match="can be counted"):
            call()
    assert _abi.moe_linear_workspace_size(1 << 30, 8, 8, bf) > 0
