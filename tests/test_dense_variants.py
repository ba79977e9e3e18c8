"""dense_variants.py's shapes reach the variants that they say (host only; they
run in test_gpu_dense_variants.py)."""

import os

import pytest

import dense_variants as dv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "token_routing_grouped_amd", "libtrg_moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")


@pytest.mark.parametrize("dt", list(dv.DT))
def test_few_tokens(dt):
    got = {}
    for T, n, K, want in dv.FEW[dt]:
        p = dv.forward(T, n, K, dt)
        assert p.row_tiles == want, (dt, T, n, K, p.row_tiles)
        got.setdefault((T > 16, want), []).append((n, K))
    assert set(got) == {(False, 0), (False, 1), (False, 2), (True, 0), (True, 1), (True, 2)}
    # a workgroup's last rows, and lines that leave some of its 8 waves without one
    for (_, tiles), sizes in got.items():
        if tiles:
            assert any(n % (16 * tiles) for n, _ in sizes)
    for T in (0, 33, 64):
        assert dv.forward(T, 2048, 2048, dt).row_tiles == 0


@pytest.mark.parametrize("dt", list(dv.DT))
def test_row_tiles_follow_the_fullest_cu(dt):
    """Two row tiles a workgroup pay where one leaves some CUs with two workgroups
    and others with one, and not while every CU has one at most."""
    for K in (512, 1024, 2048, 4096):
        for T in range(1, 33):
            for n in range(16, 4097, 16):
                assert dv.forward(T, n, K, dt).row_tiles != 2, (T, n, K)
    assert all(dv.forward(T, 5120, 512, dt).row_tiles == 2 for T in (16, 17, 32))
    assert dv.forward(1, 5120, 2048, dt).row_tiles == 1


def test_workspace_follows_the_choice():
    from token_routing_grouped_amd import _abi

    size = _abi.lib().moe_linear_workspace_size
    for dt, code in dv.DT.items():
        for T, n, K, tiles in dv.FEW[dt]:
            p = dv.forward(T, n, K, dt)
            parts = p.parts * T * -(-n // 8) * 8 * 4 if not tiles and p.parts > 1 else 0
            assert size(T, n, K, code) == parts + 16
