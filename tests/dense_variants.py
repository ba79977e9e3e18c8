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
    _fields_ = [(n, ctypes.c_int) for n in ("row_tiles", "tile", "parts")]


def _call(name, res, *args):
    from token_routing_grouped_amd import _abi

    f = getattr(_abi.lib(), name)
    f.restype, f.argtypes = res, [ctypes.c_int] * len(args)
    return f(*args)


def forward(T, n, K, dt):
    return _call("_ZN3trg11linear_planEiiii", Plan, T, n, K, DT[dt])


def gradient(T, n, K, dt, dw):
    """dx [T, K], or dw [n, K]."""
    return _call("_ZN3trg15linear_bwd_planEiiiib", Plan, T, n, K, DT[dt], int(dw))


# (T, n, K, row tiles, 0: the other kernels' tiles); rows, columns and lines end ragged
FEW = {
    "bf16": [(1, 6152, 2056, 1), (13, 4088, 520, 1), (16, 8, 8, 1), (17, 2056, 1032, 1), (32, 72, 264, 1),
             (16, 5144, 1544, 2), (16, 5128, 520, 2), (32, 5128, 520, 2), (31, 5144, 264, 2),
             (16, 12296, 2056, 0), (16, 520, 16392, 0), (32, 2056, 6152, 0), (24, 24584, 264, 0), (17, 24, 16392, 0)],
    "f32": [(1, 6148, 2052, 1), (13, 4084, 516, 1), (16, 4, 4, 1), (17, 2052, 1028, 1), (32, 68, 260, 1),
            (16, 5124, 1028, 2), (16, 6140, 260, 2), (32, 5124, 1028, 2), (31, 8196, 260, 2),
            (16, 516, 16388, 0), (32, 2052, 4100, 0), (24, 24580, 1028, 0), (17, 20, 16388, 0)],
}
