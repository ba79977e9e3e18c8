"""4-bit weights: mx_quantize_e2m1 / mx_dequantize_e2m1 bit for bit against the
oracle, and mx_linear_e2m1 against float64.

Tolerance of the product: K additions in fp32 are within (K + 16) 2^-24 of the
sum of the terms' magnitudes in any order; the result is rounded once (bf16:
2^-8 relative).
"""

import numpy as np
import pytest
import torch

from oracle import mx4_ref

from helpers import say, to_np

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _abi():
    from token_routing_grouped_amd import _abi as a

    return a


def _quantize(x):
    abi = _abi()
    rows, cols = x.shape
    q = torch.full((rows, cols // 2), 0xEE, dtype=torch.uint8, device=DEV)
    s = torch.full((abi.mx_scale_bytes(rows, cols),), 0xEE, dtype=torch.uint8, device=DEV)
    abi.mx_quantize_e2m1(x, q, s)
    return q, s


def _check_bits(x):
    abi = _abi()
    codes, sc = mx4_ref.quantize_rows(to_np(x).astype(np.float64))
    q, s = _quantize(x)
    assert np.array_equal(to_np(s), mx4_ref.scales_to_chunks(sc))
    assert np.array_equal(to_np(q), mx4_ref.pack(codes))
    out = torch.empty_like(x)
    abi.mx_dequantize_e2m1(q, s, out)
    want = torch.from_numpy(mx4_ref.dequantize_rows(codes, sc)).to(x.dtype)
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    number = ~torch.isnan(want)
    assert torch.equal(torch.signbit(got)[number], torch.signbit(want)[number])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 128), (3, 96), (5, 160), (17, 256), (129, 2048), (1000, 64)])
def test_quantize_bits(rows, cols, dt):
    say(f"e2m1 bits {rows}x{cols} {dt}")
    g = np.random.default_rng(rows + cols)
    x = g.standard_normal((rows, cols)) * np.exp2(g.integers(-20, 20, (rows, 1)))
    _check_bits(torch.from_numpy(x).to(DEV).to(DT[dt]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_every_bf16_pattern(dt):
    """All 65536 bf16 bit patterns (infinities and NaN among them), alone in
    their block, and in blocks sorted by magnitude so that values meet every
    scale near theirs."""
    bits = np.arange(65536, dtype=np.uint16)
    v = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).to(DEV)
    alone = torch.zeros(65536, 32, dtype=torch.bfloat16, device=DEV)
    alone[torch.arange(65536), torch.arange(65536) % 32] = v
    _check_bits(alone.view(-1, 256).to(DT[dt]).contiguous())
    mags = v[:32640].view(-1, 32)  # finite, by magnitude
    _check_bits(torch.cat([mags, -mags], 0).to(DT[dt]).contiguous())


def test_quantize_borders_and_signs_in_f32():
    """Values on and one fp32 step beside every rounding border, in blocks of
    several scales."""
    b = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9999], np.float32)
    vals = np.concatenate([b, np.nextafter(b, np.float32(0)), np.nextafter(b, np.float32(9)), [0.0, -0.0]])
    vals = np.concatenate([vals, -vals])[:58].astype(np.float32)
    rows = []
    for e in (-126, -125, -100, -3, 0, 5, 100, 124):
        blk = np.zeros(64, np.float32)
        blk[1:30], blk[33:62] = vals[:29], vals[29:]
        blk[0] = blk[32] = 4.0  # the block's scale, unless 6 or more is in it
        rows.append(np.ldexp(blk, e).astype(np.float32))
    _check_bits(torch.from_numpy(np.stack(rows)).to(DEV))


def test_dequantize_every_code_and_scale():
    """Every code under every scale byte (255 stands for NaN), in fp32 and bf16."""
    abi = _abi()
    codes = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 1))
    s = np.arange(256, dtype=np.uint8).reshape(256, 1)
    q = torch.from_numpy(mx4_ref.pack(codes)).to(DEV)
    sd = torch.from_numpy(mx4_ref.scales_to_chunks(s)).to(DEV)
    want = mx4_ref.dequantize_rows(codes, s)
    for dt in DT.values():
        out = torch.empty(256, 32, dtype=dt, device=DEV)
        abi.mx_dequantize_e2m1(q, sd, out)
        ref = torch.from_numpy(want).to(torch.float32).to(dt)
        assert torch.equal(torch.isnan(out.cpu()), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(out.cpu()), torch.nan_to_num(ref))


def _linear(x, q, s, n):
    y = torch.full((x.shape[0], n), float("nan"), dtype=torch.bfloat16, device=DEV)
    _abi().mx_linear_e2m1(x, q, s, y)
    return y


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("n,K", [(1, 32), (16, 256), (40, 96), (33, 1120), (130, 2048), (7, 8192)])
def test_linear(T, n, K):
    say(f"e2m1 linear T={T} n={n} K={K}")
    g = np.random.default_rng(T + n + K)
    x = torch.from_numpy(g.standard_normal((T, K))).to(DEV).to(torch.bfloat16)
    w = torch.from_numpy(g.standard_normal((n, K)) * 0.05).to(DEV).to(torch.bfloat16)
    q, s = _quantize(w)
    y = to_np(_linear(x, q, s, n)).astype(np.float64)
    wv = mx4_ref.dequantize_rows(*mx4_ref.quantize_rows(to_np(w).astype(np.float64)))
    xv = to_np(x).astype(np.float64)
    ref = xv @ wv.T
    sums = (K + 16) * 2.0 ** -24 * (np.abs(xv) @ np.abs(wv).T)
    assert (np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + sums * (1 + 2.0 ** -8)).all()


def test_linear_is_exact_on_integers():
    """Small whole values: every partial sum is exact in fp32, so the result is
    the exact sum rounded once, whatever the order: each weight and each token
    element meets exactly its own partner."""
    g = np.random.default_rng(1)
    T, n, K = 19, 50, 736
    codes = g.integers(0, 16, (n, K)).astype(np.uint8)
    sc = g.integers(126, 129, (n, K // 32)).astype(np.uint8)
    x = g.integers(-8, 9, (T, K)).astype(np.float32)
    q = torch.from_numpy(mx4_ref.pack(codes)).to(DEV)
    s = torch.from_numpy(mx4_ref.scales_to_chunks(sc)).to(DEV)
    y = _linear(torch.from_numpy(x).to(DEV).to(torch.bfloat16), q, s, n)
    ref = x.astype(np.float64) @ mx4_ref.dequantize_rows(codes, sc).T
    assert torch.equal(y.cpu(), torch.from_numpy(ref).to(torch.bfloat16))


def test_linear_meets_every_scale_byte():
    """One 32-value row per scale byte: subnormal, ordinary, the largest, and
    255 (NaN).  Products that leave bf16's or fp32's range are compared as
    infinities; below 2^-126 a scaled weight times x may be flushed, so those
    scales are held to the smallest normal instead of bit for bit."""
    codes = np.full((256, 32), 0, np.uint8)
    codes[:, 0], codes[:, 31] = 2, 11  # 1 and -1.5
    s = np.arange(256, dtype=np.uint8).reshape(256, 1)
    x = np.zeros((1, 32), np.float32)
    x[0, 0], x[0, 31] = 4.0, 2.0  # 4 - 3 = 1
    y = to_np(_linear(torch.from_numpy(x).to(DEV).to(torch.bfloat16), torch.from_numpy(mx4_ref.pack(codes)).to(DEV),
                      torch.from_numpy(mx4_ref.scales_to_chunks(s)).to(DEV), 256))[0].astype(np.float64)
    assert np.isnan(y[255])
    want = np.ldexp(1.0, np.arange(255) - 127)
    mid = (np.arange(255) >= 4) & (np.arange(255) <= 251)
    assert np.array_equal(y[:255][mid], want[mid])
    assert (np.abs(y[:4] - want[:4]) <= 2.0 ** -124).all()


def test_linear_leaves_what_is_not_its_own():
    """A NaN token, a NaN weight row: only their own column and row."""
    g = np.random.default_rng(3)
    T, n, K = 18, 40, 320
    x = torch.from_numpy(g.standard_normal((T, K))).to(DEV).to(torch.bfloat16)
    w = torch.from_numpy(g.standard_normal((n, K))).to(DEV).to(torch.bfloat16)
    y0 = _linear(x, *_quantize(w), n)
    x[17, 3], w[5, 100] = float("nan"), float("inf")
    y = _linear(x, *_quantize(w), n)
    keep = torch.ones(T, n, dtype=torch.bool, device=DEV)
    keep[17], keep[:, 5] = False, False
    assert torch.equal(y[keep], y0[keep]) and y[~keep].isnan().all()
    big = torch.full((T + 2, n), 7.0, dtype=torch.bfloat16, device=DEV)
    _abi().mx_linear_e2m1(x[:T], *_quantize(w), big[1:T + 1])
    assert (big[0] == 7).all() and (big[T + 1] == 7).all()
