"""The library's own choice of launch variants for a dense product (no GPU
needed), and shapes that reach every variant of the few-token kernel.

The choice is the host's, by estimates from the sizes alone: 16 or 32 weight rows
a workgroup for a few tokens, else tiles of 64, 128 or 256 and parts of K."""

from __future__ import annotations

import ctypes

F32, BF16 = 0, 1
DT = {"f32": F32, "bf16": BF16}


class Plan(ctypes.Structure):
    """trg::DensePlan (csrc/kernels.h)."""
    _fields_ = [(n, ctypes.c_int) for n in ("row_tiles", "tile", "stages", "parts")]


class Ortho(ctypes.Structure):
    """trg::OrthoPlan."""
    _fields_ = [("planes", ctypes.c_int), ("chunk", ctypes.c_int), ("gram", Plan), ("square", Plan), ("update", Plan)]


def _call(name, res, *args):
    from token_routing_grouped_amd import _abi

    f = getattr(_abi.lib(), name)
    f.restype, f.argtypes = res, [ctypes.c_bool if isinstance(a, bool) else ctypes.c_int for a in args]
    return f(*args)


def forward(T, n, K, dt):
    return _call("_ZN3trg11linear_planEiiii", Plan, T, n, K, DT[dt])


def gradient(T, n, K, dt, dw):
    """dx [T, K], or dw [n, K]."""
    return _call("_ZN3trg15linear_bwd_planEiiiib", Plan, T, n, K, DT[dt], bool(dw))


def ortho(B, rows, cols, dt, master=False):
    return _call("_ZN3trg10ortho_planEiiiib", Ortho, B, rows, cols, DT[dt], bool(master))


# (T, n, K, row tiles, 0: the other kernels' tiles); rows, columns and lines end ragged
FEW = {
    "bf16": [(1, 6152, 2056, 1), (13, 4088, 520, 1), (16, 8, 8, 1), (17, 2056, 1032, 1), (32, 72, 264, 1),
             (16, 5144, 1544, 2), (16, 5128, 520, 2), (32, 5128, 520, 2), (31, 5144, 264, 2),
             (16, 12296, 2056, 0), (16, 520, 16392, 0), (32, 2056, 6152, 0), (24, 24584, 264, 0), (17, 24, 16392, 0)],
    "f32": [(1, 6148, 2052, 1), (13, 4084, 516, 1), (16, 4, 4, 1), (17, 2052, 1028, 1), (32, 68, 260, 1),
            (16, 5124, 1028, 2), (16, 6140, 260, 2), (32, 5124, 1028, 2), (31, 8196, 260, 2),
            (16, 516, 16388, 0), (32, 2052, 4100, 0), (24, 24580, 1028, 0), (17, 20, 16388, 0)],
}

# (T, n, K) of products with two tiles or more each way, all ragged, of a sum with a
# last step that ends inside 128 bytes and enough steps for the unrolled ones
PRODUCTS = {
    ("bf16", "fwd"): [(75, 72, 520), (82, 72, 8744), (267, 11248, 288), (5805, 160, 5984), (131, 11536, 528),
                      (130, 5496, 2712), (8236, 1496, 280), (387, 4384, 11640)],
    ("bf16", "dx"): [(72, 688, 72), (69, 10008, 80), (11042, 264, 304), (131, 4664, 9328), (193, 608, 8432),
                     (6026, 2864, 136), (10934, 280, 1048), (797, 5720, 4712)],
    ("bf16", "dw"): [(542, 72, 72), (8421, 72, 72), (281, 11408, 272), (5928, 6288, 136), (518, 144, 12904),
                     (2707, 5536, 144), (269, 13184, 920), (5616, 5504, 704)],
    ("f32", "fwd"): [(65, 72, 304), (70, 68, 5628), (12020, 516, 132), (1663, 584, 3708), (215, 12412, 292),
                     (195, 4188, 1204)],
    ("f32", "dx"): [(79, 276, 68), (79, 4220, 76), (485, 136, 12944), (209, 3788, 4368), (409, 264, 7188),
                    (197, 1368, 4420)],
    ("f32", "dw"): [(273, 88, 68), (4122, 80, 76), (137, 456, 12396), (3789, 2136, 460), (292, 12848, 200),
                    (1348, 524, 1800)],
}

# (B, rows, cols, type, with master weights), the same of every product of a step
MATRICES = [
    (1, 129, 132, "f32", False), (1, 137, 136, "f32", False), (143, 129, 136, "f32", False),
    (145, 153, 136, "bf16", True), (57, 202, 196, "f32", False), (59, 196, 240, "bf16", True),
    (1, 65, 536, "bf16", False), (1, 546, 72, "bf16", False), (157, 266, 280, "bf16", False),
    (126, 295, 264, "bf16", False), (1, 65, 2056, "f32", False), (1, 2061, 68, "f32", False),
    (18, 65, 2680, "bf16", False), (20, 2674, 72, "bf16", False), (159, 387, 416, "f32", False),
    (49, 131, 1008, "f32", False), (55, 465, 388, "f32", False), (53, 1030, 136, "f32", False),
    (67, 195, 608, "bf16", False), (1, 519, 608, "bf16", False), (1, 606, 520, "bf16", False),
    (85, 560, 400, "bf16", False), (26, 656, 200, "f32", False), (73, 523, 224, "bf16", False),
    (80, 394, 680, "bf16", False), (28, 210, 740, "f32", False), (47, 133, 3040, "bf16", False),
    (43, 3159, 136, "bf16", False), (27, 2137, 200, "bf16", False), (35, 195, 2608, "bf16", False),
    (16, 546, 528, "bf16", False), (9, 536, 536, "bf16", False), (15, 524, 584, "bf16", False),
    (7, 638, 520, "bf16", False), (28, 404, 1300, "f32", False), (27, 1665, 408, "f32", False),
    (1, 1182, 840, "f32", False), (1, 880, 1176, "bf16", True), (28, 3765, 400, "bf16", False),
    (28, 388, 4200, "bf16", False), (2, 1016, 984, "f32", False), (2, 1019, 1028, "f32", False),
    (1, 1927, 2200, "bf16", True), (1, 1984, 1928, "bf16", True), (1, 2223, 1896, "f32", False),
    (2, 1963, 1972, "f32", False), (2, 2128, 1944, "bf16", True),
]


def product(layout, T, n, K, dt):
    """(its plan, its rows, columns and the length of its sums)"""
    if layout == "fwd":
        return forward(T, n, K, dt), T, n, K
    return gradient(T, n, K, dt, layout == "dw"), *((n, K, T) if layout == "dw" else (T, K, n))


def variant(p):
    return p.tile, p.stages, p.parts > 1


def ragged(p, M, N, S, es, runs=1):
    """Two tiles or more each way, none a multiple of them, a sum that ends inside a
    step and is long enough for the unrolled steps."""
    steps = -(-(-(-S * es // 128)) // p.parts) * runs
    return M > p.tile and N > p.tile and M % p.tile and N % p.tile and S * es % 128 and steps > 2 * p.stages


def step_products(B, rows, cols, dt, master):
    """(variant of a product, whether it is ragged) for the three of a step."""
    o, m, n = ortho(B, rows, cols, dt, master), min(rows, cols), max(rows, cols)
    for name, M, N, S in (("gram", m, m, n), ("square", m, m, m), ("update", rows, cols, m)):
        p = getattr(o, name)
        yield (o.planes, rows > cols, name, *variant(p)), bool(ragged(p, M, N, S, 2, 3 if o.planes == 2 else 1))
