"""dense_variants.py's shapes reach the variants that they say (host only; they
run in test_gpu_dense_variants.py)."""

import math
import os
import random

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


def _sizes(lo, hi, step, seed):
    """Sizes spread evenly over their logarithm."""
    rng = random.Random(seed)
    while True:
        yield max(step, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step)


@pytest.mark.parametrize("dt,layout", list(dv.PRODUCTS))
def test_products(dt, layout):
    al, es = (4, 4) if dt == "f32" else (8, 2)
    rows, cols = _sizes(1, 16384, 1, 1), _sizes(al, 16384, al, 2)
    reach = set()
    for _ in range(30000):
        T, n, K = next(rows), next(cols), next(cols)
        p, *_ = dv.product(layout, T, n, K, dt)
        if not p.row_tiles:
            reach.add(dv.variant(p))
    got = set()
    for T, n, K in dv.PRODUCTS[dt, layout]:
        p, M, N, S = dv.product(layout, T, n, K, dt)
        assert not p.row_tiles and dv.ragged(p, M, N, S, es), (T, n, K)
        got.add(dv.variant(p))
    tiles = (64, 128, 256) if dt == "bf16" else (64, 128)
    assert {t for t, *_ in got} == set(tiles) and got >= reach, reach - got
    assert (128, 4, False) in got and (128, 2, False) in got


def test_matrices():
    reach = set()
    many, rows, cols = _sizes(1, 160, 1, 3), _sizes(2, 6000, 1, 4), _sizes(8, 6400, 8, 5)
    for i in range(30000):
        B, r, c = next(many), next(rows), next(cols)
        if B * r * c <= 1 << 26:
            for dt, master in (("f32", False), ("bf16", True), ("bf16", False)):
                reach |= {k for k, _ in dv.step_products(B, r, c, dt, master)}
    got = set()
    for case in dv.MATRICES:
        got |= {k for k, full in dv.step_products(*case) if full}
    assert got >= reach, reach - got
    for planes in (1, 2):
        for tall in (True, False):
            assert {(t, s) for p, a, n, t, s, _ in got if (p, a, n) == (planes, tall, "update")} \
                == {(64, 4), (128, 4), (128, 2), (256, 2)}
