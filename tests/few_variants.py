"""Shapes that reach every launch variant of the few-token layer and of the
4-bit dense product, and the library's own choice for a shape (no GPU needed).

A variant is picked on the host from the sizes (row tiles a wave, waves a row
tile, where the routing happens, ...) and on the device from an expert's number
of tokens (column classes).  The router's inputs are whole numbers times a
power of two, so that every logit is exact in fp32, the chosen experts are
known on the host and equal logits occur (they go to the lower expert).
"""

from __future__ import annotations

import ctypes

import numpy as np

F32, BF16, E2M1 = 0, 1, 4
WT = {"f32": F32, "bf16": BF16, "e2m1": E2M1}


class Plan(ctypes.Structure):
    """trg::FewPlan (csrc/kernels.h)."""
    _fields_ = [(n, ctypes.c_int) for n in ("pro", "router", "logit_tiles", "epl", "up_rows", "up_waves", "down_rows",
                                            "down_waves")]


def _lib():
    from token_routing_grouped_amd import _abi

    lib = _abi.lib()
    lib._ZN3trg8few_planEiiiiii.restype = Plan
    lib._ZN3trg8few_planEiiiiii.argtypes = [ctypes.c_int] * 6
    lib._ZN3trg16linear_row_tilesEii.restype = ctypes.c_int
    lib._ZN3trg16linear_row_tilesEii.argtypes = [ctypes.c_int] * 2
    return lib


def plan(T, d, E, k, h, wt):
    return _lib()._ZN3trg8few_planEiiiiii(T, d, E, k, h, WT[wt])


def linear_row_tiles(T, n):
    return _lib()._ZN3trg16linear_row_tilesEii(T, n)


def router_inputs(T, d, E):
    """x [T,d] and wr [E,d] whose logits are exact, with a spread of about 1.5."""
    g = np.random.default_rng(T + 7 * d + 31 * E)
    m = int(np.round(np.log2(2.1 * np.sqrt(d) / 1.5)))
    return (g.integers(-4, 5, (T, d)).astype(np.float64),
            g.integers(-1, 2, (E, d)).astype(np.float64) * 2.0 ** -m)


def choose(x, wr, k):
    """Logits and the k chosen experts of every token, best first."""
    L = x @ wr.T
    return L, np.argsort(-L, axis=1, kind="stable")[:, :k]


def counts(T, d, E, k):
    _, idx = choose(*router_inputs(T, d, E), k)
    return np.bincount(idx.reshape(-1), minlength=E)


def _class(n, ends):
    return next(e for e in ends if n <= e)


def up_classes(c, wt, pro):
    ends = (2, 8) if pro else (4, 16, 64)
    return {_class(n, ends if wt == "e2m1" else (16, 32, 48, 64)) for n in c if n}


def down_classes(c, wt):
    return {_class(n, (2, 8, 16, 64) if wt == "e2m1" else (16, 32, 48, 64)) for n in c if n}


# (T, d, E, k, h); rows and lines of every one end ragged
FEW = [
    # bf16 rows up to 256, 512 and over 4096 bytes where row tiles are many
    ("bf16", 64, 248, 1000, 20, 72), ("bf16", 64, 488, 1000, 20, 72), ("bf16", 40, 2056, 128, 4, 136),
    # 8 waves and two row tiles, 17 to 48 tokens an expert; and all 64
    ("bf16", 64, 2056, 64, 32, 264), ("bf16", 64, 2056, 32, 32, 520), ("bf16", 64, 2056, 3, 3, 72),
    # hidden rows of 512, over 512 and over 4096 bytes, many and few row tiles
    ("bf16", 64, 264, 256, 8, 392), ("bf16", 64, 264, 256, 4, 520), ("bf16", 64, 264, 256, 4, 2056),
    ("bf16", 9, 72, 4, 2, 2056), ("bf16", 40, 72, 4, 4, 2056),
    # every expert has all the tokens: one row tile a wave up, four down; and in few row tiles
    ("bf16", 50, 2056, 32, 32, 72), ("bf16", 24, 72, 4, 4, 136),
    # 8 tokens an expert, 4 waves and two row tiles
    ("bf16", 64, 264, 100, 12, 200),
    ("f32", 64, 120, 1000, 20, 72), ("f32", 64, 248, 1000, 20, 72), ("f32", 40, 1032, 128, 4, 136),
    ("f32", 64, 1032, 64, 32, 264), ("f32", 64, 1032, 64, 32, 72), ("f32", 64, 264, 32, 32, 520),
    ("f32", 64, 1032, 3, 3, 72), ("f32", 64, 264, 256, 8, 200), ("f32", 64, 264, 256, 4, 264),
    ("f32", 64, 264, 256, 4, 1032), ("f32", 9, 72, 4, 2, 1032), ("f32", 40, 72, 4, 4, 1032),
    ("f32", 50, 2056, 32, 32, 72), ("f32", 24, 72, 4, 4, 136),
    # 4-bit rows up to 512, up to 1024, over 1024 and over 4096 bytes: one to two, two, about six, sixteen tokens
    ("e2m1", 64, 480, 1000, 20, 96), ("e2m1", 64, 1056, 1000, 32, 96), ("e2m1", 64, 2080, 1000, 20, 96),
    ("e2m1", 20, 8224, 16, 4, 96), ("e2m1", 64, 480, 340, 32, 224), ("e2m1", 64, 544, 128, 32, 544),
    ("e2m1", 64, 1056, 128, 32, 1056), ("e2m1", 64, 160, 512, 16, 1056), ("e2m1", 64, 160, 512, 10, 2080),
    ("e2m1", 64, 160, 512, 8, 8224), ("e2m1", 20, 96, 16, 4, 8224), ("e2m1", 64, 96, 4, 4, 96),
    ("e2m1", 12, 96, 4, 4, 96),
]
# routed in the up projection, on both sides of 4 tokens: 16 experts (the logits too), to 128, to 512, more
PRO = [(wt, T, d, E, k, h) for wt in WT for T, d, E, k, h in
       [(1, 160, 130, 4, 160), (7, 288, 300, 8, 96), (3, 96, 600, 5, 96), (8, 160, 1000, 8, 96), (4, 160, 512, 8, 224),
        (5, 288, 513, 6, 224), (8, 160, 16, 3, 160), (3, 160, 9, 4, 96), (3, 2080, 16, 4, 96), (6, 160, 40, 5, 96), (2, 96, 128, 12, 288)]]

# n for 1, 2, 3 and 4 (to 32 tokens) row tiles a wave, none a multiple of 16 of them
LINEAR_T = (1, 4, 5, 13, 17, 32, 33, 64)
LINEAR_N = (4090, 4117, 6140, 8209, 10007, 12310, 16391, 20491, 24571, 40933)
