"""Every launch variant of moe_few_fwd and mx_linear_e2m1 (few_variants.py has
the shapes) against float64, computed on the GPU with plain torch.

Tolerance of the layer, elementwise.  u = 2^-24; a sum of n terms in fp32 in any
order is within (n + 16) u of the sum of the terms' magnitudes.
  a, b:   da = (d + 16) u |W1||x|, db likewise with W3
  silu:   |silu'| <= 1.1: its product with b is within 1.1 da |b| + |silu| db +
          8 u |hid|; stored as two bf16 halves it loses 2^-16 |hid| more (fp32: u)
  gate:   the logits are exact (few_variants.py), so a softmax value is within
          (48 + E / 64) u, relatively: exp, a lane's E / 64 additions, the
          wave's, a division
  y:      sum over a token's experts of gate |W2| dhid, plus (2 k h + 16) u of
          gate |W2||hid| (both halves are terms), plus the rounding of y
Relative L2: half a step of y's type (2^-8 bf16, 2^-24 fp32), the hidden
vector's storage, and 4 u sqrt(n) for the longest sum's n terms with signs that
do not conspire.
"""

import numpy as np
import pytest
import torch

import few_variants as fv
from helpers import say, to_np

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
BF = torch.bfloat16


def _abi():
    from token_routing_grouped_amd import _abi as a

    return a


def _random_e2m1(g, E, rows, K):
    """Random codes [E, rows, K/2] and scales of K^-1/2 values, stored order."""
    q = torch.randint(0, 256, (E, rows, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s0 = 127 + int(np.floor(np.log2(K ** -0.5 / 2.9)))
    s = torch.randint(s0, s0 + 2, (-(-K // 128), E, rows, 4), generator=g, device=DEV, dtype=torch.uint8)
    s[-1, :, :, (K - 1) % 128 // 32 + 1:] = 0
    return q, s.view(-1)


def _e2m1_values(q, s):
    """float64 values of codes [rows, K/2] and scales [chunks, rows, 4], from
    the format's fields: a sign, two exponent bits (bias 1), one mantissa bit."""
    rows, K = q.shape[0], q.shape[1] * 2
    c = torch.stack((q & 15, q >> 4), 2).view(rows, K).to(torch.int64)
    ex, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((ex - 1).double()))
    v = torch.where(c >= 8, -v, v)
    e = s.transpose(0, 1).reshape(rows, -1)[:, :K // 32].double() - 127
    return (v.view(rows, K // 32, 32) * torch.exp2(e).unsqueeze(2)).view(rows, K)


class Layer:
    """Inputs, the object under test and the float64 result with its bound."""

    def __init__(self, wt, T, d, E, k, h):
        from token_routing_grouped_amd.layer import MoEDecodeGPU

        self.wt, self.T, self.d, self.E, self.k, self.h = wt, T, d, E, k, h
        dt = torch.float32 if wt == "f32" else BF
        g = torch.Generator(device=DEV).manual_seed(T + 3 * d + 5 * E + 7 * k + 11 * h)
        self.x64, self.wr64 = fv.router_inputs(T, d, E)
        self.x, wr = (torch.from_numpy(a).to(DEV).to(dt) for a in (self.x64, self.wr64))
        self.w, scales = [], {}
        for name, rows, K in (("w1s", h, d), ("w3s", h, d), ("w2s", d, h)):
            if wt == "e2m1":
                q, scales[name] = _random_e2m1(g, E, rows, K)
                self.w.append((q, scales[name].view(-1, E, rows, 4)))
            else:
                self.w.append((torch.randn(E, rows, K, generator=g, device=DEV, dtype=dt) * K ** -0.5,))
        self.m = MoEDecodeGPU(T, k, wr, *(a[0] for a in self.w), **scales)

    def weight(self, i, e):
        return _e2m1_values(self.w[i][0][e], self.w[i][1][:, e]) if self.wt == "e2m1" else self.w[i][0][e].double()

    def expected(self):
        """y, idx, gates, y's bound and the gates' relative one."""
        T, d, E, k, h = self.T, self.d, self.E, self.k, self.h
        L, idx = fv.choose(self.x64, self.wr64, k)
        p = np.exp(L - L.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        gates = np.take_along_axis(p, idx, 1)
        dgate = (48 + E / 64) * U
        x, gt = torch.from_numpy(self.x64).to(DEV), torch.from_numpy(gates).to(DEV)
        y, bound = torch.zeros_like(x), torch.zeros_like(x)
        store = U if self.wt == "f32" else 2.0 ** -16
        for e in np.unique(idx):
            t, j = (torch.from_numpy(a).to(DEV) for a in np.nonzero(idx == e))
            w1, w3, w2 = (self.weight(i, int(e)) for i in range(3))
            xe, ge = x[t], gt[t, j].unsqueeze(1)
            a, b = xe @ w1.t(), xe @ w3.t()
            da, db = ((d + 16) * U * (xe.abs() @ w.abs().t()) for w in (w1, w3))
            s = a * torch.sigmoid(a)
            hid = s * b
            y[t] += ge * (hid @ w2.t())
            dh = 1.1 * da * b.abs() + s.abs() * db + (8 * U + store + dgate) * hid.abs()
            bound[t] += ge * ((dh + (2 * k * h + 16) * U * hid.abs()) @ w2.abs().t())
        half = U if self.wt == "f32" else 2.0 ** -8
        return y, idx, gates, half * y.abs() + (1 + half) * bound, dgate

    def check(self, ref, n=None):
        y, idx, gates, bound, dgate = ref
        n = self.T if n is None else n
        got = self.m.y[:n].double()
        assert np.array_equal(to_np(self.m.topk_idx)[:n], idx[:n])
        assert (np.abs(to_np(self.m.topk_w)[:n] - gates[:n]) <= dgate * gates[:n]).all()
        err = (got - y[:n]).abs()
        assert (err <= bound[:n]).all(), float((err / bound[:n]).max())  # NaN fails
        rel = float((got - y[:n]).norm() / y[:n].norm())
        half, store = (U, U) if self.wt == "f32" else (2.0 ** -8, 2.0 ** -16)
        assert rel <= half + store + 4 * U * np.sqrt(max(self.d, 2 * self.k * self.h)), rel


@pytest.mark.parametrize("case", fv.FEW + fv.PRO, ids=lambda c: "-".join(map(str, c)))
def test_layer_variant(case):
    """Twice, over a workspace and outputs that hold other bytes each time."""
    say("few variant", case)
    c = Layer(*case)
    first = None
    for fill in (0xFF, 0x3C):
        for b in (c.m.ws, c.m.y, c.m.topk_idx, c.m.topk_w):
            b.view(torch.uint8).fill_(fill)
        c.m.forward(c.x)
        out = [b.clone() for b in (c.m.y, c.m.topk_idx, c.m.topk_w)]
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(out, first))
    c.check(c.expected())


# at most 8 tokens: the logits from their own launch (over 16 experts) or not
@pytest.mark.parametrize("wt,T,E", [("bf16", 7, 40), ("bf16", 7, 300), ("bf16", 3, 600), ("f32", 5, 40),
                                    ("e2m1", 6, 16), ("e2m1", 6, 40), ("e2m1", 8, 300), ("e2m1", 2, 700)])
def test_live_count_where_the_projection_routes(wt, T, E):
    say(f"live count, routed in the projection: {wt} T={T} E={E}")
    assert fv.plan(T, 160, E, 3, 96, wt).pro
    c = Layer(wt, T, 160, E, 3, 96)
    ref = c.expected()
    for n in range(T + 1):
        c.m.y.fill_(3)
        c.m.topk_idx.fill_(-3)
        c.m.topk_w.fill_(-3)
        x = c.x.clone()
        x[n:] = float("nan")  # what lies behind is not used
        c.m.forward(x, n_live=torch.tensor([n], dtype=torch.int32, device=DEV))
        assert (c.m.y[n:] == 3).all() and (c.m.topk_idx[n:] == -3).all() and (c.m.topk_w[n:] == -3).all()
        if n:
            c.check(ref, n)


@pytest.mark.parametrize("wt,T,E", [("bf16", 3, 16), ("e2m1", 3, 40), ("bf16", 40, 16), ("e2m1", 40, 300)])
def test_two_objects_on_two_streams_write_their_own(wt, T, E):
    """Interleaved calls on two streams, outputs wiped before them."""
    a, b = (Layer(wt, T, 288, E, 4, 160) for _ in range(2))
    xb = torch.flip(a.x, (0,)).contiguous()
    want = []
    for m, x in ((a.m, a.x), (b.m, xb)):
        m.forward(x)
        want.append([o.clone() for o in (m.y, m.topk_idx, m.topk_w)])
    for m in (a.m, b.m):
        m.y.fill_(7)
        m.topk_idx.fill_(-7)
        m.topk_w.fill_(-7)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(sa):
            a.m.forward(a.x)
        with torch.cuda.stream(sb):
            b.m.forward(xb)
    torch.cuda.synchronize()
    for m, w in zip((a.m, b.m), want):
        assert all(torch.equal(o, v) for o, v in zip((m.y, m.topk_idx, m.topk_w), w))


# K under one 256-value line, ending inside one, and whole lines
@pytest.mark.parametrize("K", [96, 352, 512])
@pytest.mark.parametrize("T", fv.LINEAR_T)
def test_linear_row_tiles(T, K):
    """All row-tile counts: whole values, whose sums are exact in fp32, so that
    the result is the exact sum rounded once; then ordinary values, within
    (K + 16) u of the magnitudes' sum and the rounding."""
    for n in fv.LINEAR_N:
        say(f"linear T={T} n={n} K={K}: {fv.linear_row_tiles(T, n)} row tiles")
        g = torch.Generator(device=DEV).manual_seed(n + K + T)
        q, s = _random_e2m1(g, 1, n, K)
        w = _e2m1_values(q[0], s.view(-1, n, 4))
        buf = torch.full((T * n + 16,), float("nan"), dtype=BF, device=DEV)
        y = buf[8:T * n + 8].view(T, n)
        # in steps of half the smaller scale a term is at most 2 * 12 * 2, a sum under 2^15
        x = torch.randint(-2, 3, (T, K), generator=g, device=DEV).to(BF)
        _abi().mx_linear_e2m1(x, q.view(n, K // 2), s, y)
        assert torch.equal(y, (x.double() @ w.t()).to(BF))
        assert buf[:8].isnan().all() and buf[-8:].isnan().all()
        x = torch.randn(T, K, generator=g, device=DEV, dtype=BF)
        _abi().mx_linear_e2m1(x, q.view(n, K // 2), s, y)
        ref, size = x.double() @ w.t(), x.double().abs() @ w.abs().t()
        err = (y.double() - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * (K + 16) * U * size).all()


@pytest.mark.parametrize("dt", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(6001, 672), (1367, 3104)])
def test_quantize_four_pieces_a_thread(rows, cols, dt):
    """Matrices large enough for four pieces a thread, chunks a row no multiple
    of four and the last one short: codes, scales and values bit for bit."""
    from oracle import mx4_ref

    say(f"e2m1 bits {rows}x{cols} {dt}")
    nch = -(-cols // 128)
    assert rows * nch >= 32768 and nch % 4 and cols % 128
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn(rows, cols, generator=g, device=DEV) * torch.exp2(
        torch.randint(-20, 20, (rows, 1), generator=g, device=DEV).float())
    x[5, 40], x[rows - 1, cols - 1] = float("inf"), float("nan")
    x = x.to(dt)
    q = torch.full((rows, cols // 2), 0xEE, dtype=torch.uint8, device=DEV)
    s = torch.full((_abi().mx_scale_bytes(rows, cols),), 0xEE, dtype=torch.uint8, device=DEV)
    out = torch.full_like(x, 7)
    _abi().mx_quantize_e2m1(x, q, s)
    _abi().mx_dequantize_e2m1(q, s, out)
    x, s, q = to_np(x), to_np(s), to_np(q)
    for r0 in range(0, rows, 512):  # the oracle holds 8 distances a value
        r1 = min(r0 + 512, rows)
        with np.errstate(invalid="ignore"):
            codes, sc = mx4_ref.quantize_rows(x[r0:r1].astype(np.float64))
        assert np.array_equal(q[r0:r1], mx4_ref.pack(codes))
        mine = s.reshape(nch, rows, 4)[:, r0:r1].reshape(-1)
        assert np.array_equal(mine, mx4_ref.scales_to_chunks(sc))
        want = torch.from_numpy(mx4_ref.dequantize_rows(codes, sc)).to(dt)
        got = out[r0:r1].cpu()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


@pytest.mark.parametrize("wt,T,E", [("bf16", 3, 12), ("e2m1", 3, 40), ("f32", 20, 12), ("e2m1", 20, 40)])
def test_layer_without_the_routing_outputs(wt, T, E):
    """topk_idx and topk_w are optional; y is the same without them."""
    c = Layer(wt, T, 288, E, 3, 160)
    want = c.m.forward(c.x).clone()
    y = torch.full_like(want, 7)
    _abi().moe_few_fwd(c.m._args, c.x, y)
    assert torch.equal(y, want)


@pytest.mark.parametrize("T,E", [(3, 12), (3, 40), (20, 40), (64, 6)])
def test_faulty_4bit_expert_reaches_only_its_tokens(T, E):
    """A scale byte of 255 (NaN) or 254 (infinite sums) in one expert's matrices."""
    c = Layer("e2m1", T, 288, E, 2, 160)
    y0 = c.m.forward(c.x).clone()
    idx = c.m.topk_idx.clone()
    e = int(idx[0, 0])
    hit = (idx == e).any(1)
    assert hit.any() and not hit.all()
    for i in range(3):
        for byte in (255, 254):
            s = c.w[i][1]
            old = s[0, e, 7].clone()
            s[0, e, 7, 1] = byte  # block 1 of the expert's row 7
            y = c.m.forward(c.x).clone()
            s[0, e, 7] = old
            assert torch.equal(y[~hit], y0[~hit])
            if byte == 255:
                assert not torch.isfinite(y[hit]).all(1).any()
    assert torch.equal(c.m.forward(c.x), y0)
