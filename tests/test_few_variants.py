"""The shapes of few_variants.py reach every launch variant that any size
reaches (host only; test_gpu_few_variants.py runs them)."""

import itertools
import os

import pytest

import few_variants as fv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "token_routing_grouped_amd", "libtrg_moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")


def _reachable(wt):
    """Plans of a grid of sizes that spans each rule's borders."""
    dims = (32, 64, 128, 256, 512, 1024, 2048, 4096, 8192, 16384)
    for T, E, k in itertools.product((1, 4, 5, 8, 9, 16, 17, 32, 33, 64), (1, 8, 16, 17, 64, 65, 128, 129, 512, 513, 1024),
                                     (1, 4, 32)):
        if k <= E:
            for d, h in itertools.product(dims, dims):
                yield T, fv.plan(T, d, E, k, h, wt)


@pytest.mark.parametrize("wt", list(fv.WT))
def test_every_variant_of_the_layer_has_a_shape(wt):
    host = {"route": set(), "up": set(), "down": set()}
    got = {"route": set(), "up": set(), "down": set()}

    def add(s, T, p):
        s["route"].add((p.pro, p.router, p.epl, p.pro and T <= 4) if p.pro else (0, 0, p.epl))
        if not p.pro:
            s["up"].add((p.up_rows, p.up_waves))
            s["down"].add((p.down_rows, p.down_waves))

    for T, p in _reachable(wt):
        add(host, T, p)
    columns = {"up": set(), "down": set(), "pro": set()}
    for case in fv.FEW + fv.PRO:
        if case[0] != wt:
            continue
        _, T, d, E, k, h = case
        p, c = fv.plan(T, d, E, k, h, wt), fv.counts(T, d, E, k)
        assert bool(p.pro) == (case in fv.PRO), case
        add(got, T, p)
        if p.pro:
            columns["pro"] |= fv.up_classes(c, wt, True)
        else:
            # 4 bits: with the waves, on which a lane's staging and lines depend
            w = (lambda n: (n,)) if wt == "e2m1" else (lambda n: ())
            columns["up"] |= {(p.up_rows, *w(p.up_waves), n) for n in fv.up_classes(c, wt, False)}
            columns["down"] |= {(p.down_rows, *w(p.down_waves), n) for n in fv.down_classes(c, wt)}
    assert got["up"] >= host["up"] and got["down"] >= host["down"], (host["up"] - got["up"], host["down"] - got["down"])
    assert {r for r in got["route"] if r[0]} >= {r for r in host["route"] if r[0]}
    if wt == "e2m1":
        assert columns["pro"] == {2, 8}
        assert {n for _, _, n in columns["up"]} == {4, 16, 64}
        assert {(r, n) for r, _, n in columns["down"]} >= {(r, n) for r in (2, 4) for n in (2, 8, 16, 64)} - {(2, 2)}
        assert {(w, n) for r, w, n in columns["down"] if r == 4} >= {(w, n) for w in (1, 2) for n in (2, 8, 16, 64)}
    else:
        want = {(r, n) for r in (1, 2) for n in (16, 32, 48, 64)}
        assert columns["up"] >= want, want - columns["up"]
        want = {(r, n) for r in (2, 4) for n in (16, 32, 48, 64)}
        assert columns["down"] >= want, want - columns["down"]


def test_routing_launches_of_every_width_have_a_shape():
    widths = {fv.plan(T, d, E, k, h, wt).epl for wt, T, d, E, k, h in fv.FEW}
    assert widths == {1, 2, 8, 16}


def test_every_row_and_column_tile_count_of_the_dense_product_has_a_shape():
    rows = {}
    for T in fv.LINEAR_T:
        cols = 4 if T <= 4 else 16 if T <= 16 else 32 if T <= 32 else 64
        for n in fv.LINEAR_N:
            m = fv.linear_row_tiles(T, n)
            if n % (16 * m):
                rows.setdefault(cols, set()).add(m)
    reach = {T: {fv.linear_row_tiles(T, n) for n in range(1, 70000, 16)} for T in (1, 13, 17, 64)}
    assert rows == {4: reach[1], 16: reach[13], 32: reach[17], 64: reach[64]}
    assert rows[4] == rows[16] == rows[32] == {1, 2, 3, 4}


def test_no_four_row_tiles_with_four_column_tiles():
    """Their accumulators and operands do not fit into the registers."""
    assert {fv.linear_row_tiles(T, n) for T in (33, 48, 64) for n in range(16, 1 << 18, 16)} == {1, 2, 3}
