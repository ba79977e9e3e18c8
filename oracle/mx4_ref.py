"""4-bit weights (OCP microscaling: E2M1 elements, one E8M0 scale per 32
values), by search over the format's values in float64.  Test infrastructure
only (see the package header).

  * s = clamp(floor(log2(amax)) - 2, -127, 127), -127 for an all-zero block;
    floor(log2) exactly, from frexp;
  * an element is the nearest of the eight magnitudes to |v| / 2^s, ties to the
    even code, the largest (6) for anything above it; the sign of zero is kept;
  * a block with an infinity or NaN: scale byte 255, zero codes, 32 NaNs.
"""

from __future__ import annotations

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def quantize_rows(a):
    """[M, K] -> (codes [M, K] uint8 in 0..15, scale bytes [M, K/32] uint8)."""
    a = np.asarray(a, np.float64)
    M, K = a.shape
    b = a.reshape(M, K // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    s = np.where(amax > 0, np.clip(np.frexp(amax)[1] - 3, -127, 127), -127)
    x = np.abs(b) * np.ldexp(1.0, -s)[:, :, None]
    dist = np.abs(np.minimum(x, 6.0)[..., None] - VALUES)
    # nearest value; of two equally near ones the even code
    best = dist.min(axis=-1, keepdims=True)
    near = dist == best
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(axis=-1, keepdims=True), even, near)
    code = pick.argmax(axis=-1).astype(np.uint8)
    code |= (np.signbit(b).astype(np.uint8) << 3)
    code[bad] = 0
    return code.reshape(M, K), np.where(bad, 255, s + 127).astype(np.uint8)


def pack(codes):
    """Codes [M, K] to bytes [M, K/2], the even column in the low half."""
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(q):
    out = np.empty((q.shape[0], q.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def dequantize_rows(codes, scales):
    M, K = codes.shape
    v = np.where(codes & 8, -1.0, 1.0) * VALUES[codes & 7]
    e = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v.reshape(M, K // BLOCK, BLOCK) * e[:, :, None]).reshape(M, K)


def scales_to_chunks(s):
    """[M, K/32] bytes to the stored order [ceil(K/128)][M][4], 0 past a row's end."""
    M, nb = s.shape
    out = np.zeros((M, -(-nb // 4) * 4), np.uint8)
    out[:, :nb] = s
    return np.ascontiguousarray(out.reshape(M, -1, 4).transpose(1, 0, 2)).reshape(-1)
