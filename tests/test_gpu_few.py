"""moe_few_fwd (the layer for a few tokens) against the float64 oracle.

Tolerance, elementwise, from the magnitudes that meet in each sum.  u = 2^-24;
a sum of n terms in fp32 in any order is within (n + 16) u of the sum of the
terms' magnitudes.
  g, u:   dg = (d + 16) u |W1||x|, du likewise with W3
  silu(g) u: |silu'| <= 1.1, so its error is 1.1 dg |u| + |silu| du + 8 u |h|
  h:      plus its storage as two bf16 halves, 2^-16 |h| (fp32: u |h|)
  gate:   the logits' error dl = (d + 16) u |wr||x| moves a softmax value by at
          most 2 max dl, relatively, plus 16 u
  y:      sum_j gate |W2| dh + (k h + 16) u sum_j gate |W2||h|, and the
          rounding of y itself (2^-8 for bf16)
The same inputs' relative L2 error is held to 2^-8 (bf16) and 2e-6 (fp32) too.
Inputs keep the k-th and the next logit 1e-4 apart (checked), except where ties
are the subject.
"""

import numpy as np
import pytest
import torch

from oracle import moe_ref, mx4_ref

from helpers import rel_l2, say, to_np

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24


def _layer():
    from token_routing_grouped_amd.layer import MoEDecodeGPU

    return MoEDecodeGPU


def _pack(w):
    """[E, n, K] to codes [E, n, K/2] and scales on the device, and the values
    they stand for in float64."""
    E, n, K = w.shape
    c, s = mx4_ref.quantize_rows(w.reshape(E * n, K))
    v = mx4_ref.dequantize_rows(c, s).reshape(E, n, K)
    return (torch.from_numpy(mx4_ref.pack(c)).to(DEV).view(E, n, K // 2),
            torch.from_numpy(mx4_ref.scales_to_chunks(s)).to(DEV), v)


class Case:
    def __init__(self, T, d, E, k, h, wt, seed=0):
        g = np.random.default_rng(seed + T * 7 + d * 3 + E + k + h)
        self.T, self.d, self.E, self.k, self.h, self.wt = T, d, E, k, h, wt
        dt = self.dt = torch.float32 if wt == "f32" else torch.bfloat16
        put = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV).to(dt)
        self.x = put(g.standard_normal((T, d)))
        self.wr = put(g.standard_normal((E, d)) / np.sqrt(d))
        ws = [g.standard_normal(n) / np.sqrt(n[2]) for n in ((E, h, d), (E, h, d), (E, d, h))]
        self.scales = {}
        if wt == "e2m1":
            self.w, self.v = [], []
            for name, a in zip(("w1s", "w3s", "w2s"), ws):
                q, s, v = _pack(a.astype(np.float32).astype(np.float64))
                self.w.append(q)
                self.v.append(v)
                self.scales[name] = s
        else:
            self.w = [put(a) for a in ws]
            self.v = [to_np(a).astype(np.float64) for a in self.w]

    def layer(self, T=None, **kw):
        return _layer()(T or self.T, self.k, self.wr, *self.w, **self.scales, **kw)

    def ref(self, x=None):
        """y, idx, gates and y's bound, float64."""
        x = to_np(self.x if x is None else x).astype(np.float64)
        wr = to_np(self.wr).astype(np.float64)
        w1, w3, w2 = self.v
        f = moe_ref.layer_forward(x, wr, w1, w3, w2, self.k)
        L = np.sort(x @ wr.T, axis=1)
        self.gap = np.min(L[:, -self.k] - L[:, -self.k - 1]) if self.k < self.E else np.inf
        dl = (self.d + 16) * U * (np.abs(x) @ np.abs(wr).T).max()
        dgate = 2 * dl + 16 * U
        store = U if self.wt == "f32" else 2.0 ** -16
        bound = np.zeros_like(f["y"])
        for t in range(x.shape[0]):
            ax = np.abs(x[t])
            for j in range(self.k):
                e, p = f["idx"][t, j], f["w"][t, j]
                a, b = w1[e] @ x[t], w3[e] @ x[t]
                da, db = ((self.d + 16) * U * (np.abs(m) @ ax) for m in (w1[e], w3[e]))
                s = moe_ref.silu(a)
                hid = np.abs(s * b)
                dh = 1.1 * da * np.abs(b) + np.abs(s) * db + (8 * U + store + dgate) * hid
                n = (self.k * self.h + 16) * U
                bound[t] += p * (np.abs(w2[e]) @ (dh + n * hid))
        half = U if self.wt == "f32" else 2.0 ** -8
        return f["y"], f["idx"], f["w"], half * np.abs(f["y"]) + 1.01 * bound, dgate

    def check(self, y, idx=None, w=None, x=None):
        ry, ridx, rw, bound, dgate = self.ref(x)
        assert self.gap > 1e-4 * 0.1, "the inputs leave a tie: choose another seed"
        if idx is not None:
            assert np.array_equal(to_np(idx), ridx)
            assert (np.abs(to_np(w) - rw) <= dgate * rw).all()
        y = to_np(y).astype(np.float64)
        assert np.isfinite(y).all()
        assert (np.abs(y - ry) <= bound).all(), float((np.abs(y - ry) / bound).max())
        assert rel_l2(y, ry) <= (2e-6 if self.wt == "f32" else 2.0 ** -8)


# T, d, E, k, h: one token to the most, one expert to many, ragged rows and
# lines (bf16 lines are 64 values, fp32 32, 4-bit 256), h under one line
SHAPES = [
    (1, 128, 8, 2, 256), (1, 64, 1, 1, 32), (2, 136, 5, 3, 40), (3, 1000, 16, 4, 264), (1, 2048, 8, 4, 128),
    (7, 72, 2, 2, 8), (16, 256, 4, 4, 96), (17, 264, 3, 2, 136), (16, 128, 384, 8, 64), (33, 520, 6, 3, 72),
    (64, 256, 1, 1, 64), (64, 136, 130, 8, 104), (40, 64, 600, 4, 24), (64, 512, 8, 4, 256), (5, 96, 1024, 32, 16),
    (12, 136, 100, 5, 40), (16, 1000, 16, 4, 72), (9, 264, 300, 7, 24), (13, 2048, 13, 4, 64), (8, 72, 700, 8, 40),
    (64, 72, 2, 2, 136), (21, 8200, 3, 1, 8),
]


@pytest.mark.parametrize("T,d,E,k,h", SHAPES)
@pytest.mark.parametrize("wt", ["bf16", "f32"])
def test_few(T, d, E, k, h, wt):
    say(f"few T={T} d={d} E={E} k={k} h={h} {wt}")
    c = Case(T, d, E, k, h, wt)
    m = c.layer()
    c.check(m.forward(c.x), m.topk_idx, m.topk_w)


@pytest.mark.parametrize("T,d,E,k,h", [(1, 128, 8, 2, 256), (1, 32, 1, 1, 32), (2, 160, 5, 3, 96),
                                       (1, 2048, 8, 4, 1024),
                                       (7, 288, 2, 2, 544), (16, 256, 4, 4, 96), (17, 544, 3, 2, 160),
                                       (16, 128, 384, 8, 64), (33, 1056, 6, 3, 288), (64, 256, 8, 4, 256),
                                       (64, 96, 130, 8, 32), (13, 160, 20, 4, 96), (9, 2080, 16, 3, 64),
                                       (64, 128, 2, 1, 64), (12, 1024, 600, 5, 32)])
def test_few_4bit(T, d, E, k, h):
    say(f"few e2m1 T={T} d={d} E={E} k={k} h={h}")
    c = Case(T, d, E, k, h, "e2m1")
    m = c.layer()
    c.check(m.forward(c.x), m.topk_idx, m.topk_w)


# few tokens on both sides of the rule for routing in the up projection (512
# workgroups of 16 rows), and masks of more experts than one batch of loads
@pytest.mark.parametrize("T,d,E,k,h", [(1, 64, 16, 8, 1024), (1, 64, 16, 8, 1056), (8, 64, 8, 2, 1024),
                                       (8, 64, 8, 2, 1056), (1, 96, 40, 32, 256), (1, 96, 40, 32, 288),
                                       (2, 64, 1024, 32, 160), (8, 64, 513, 8, 160), (64, 64, 1024, 2, 32),
                                       (33, 64, 257, 1, 64)])
@pytest.mark.parametrize("wt", ["bf16", "f32", "e2m1"])
def test_few_routed_in_either_place(T, d, E, k, h, wt):
    say(f"few T={T} d={d} E={E} k={k} h={h} {wt}")
    c = Case(T, d, E, k, h, wt)
    m = c.layer()
    c.check(m.forward(c.x), m.topk_idx, m.topk_w)


# every expert has all the tokens: each number of column tiles, with one and more
# row tiles a wave in either projection
@pytest.mark.parametrize("E,d,h", [(2, 136, 72), (32, 64, 512), (32, 2048, 32)])
@pytest.mark.parametrize("T", [16, 17, 32, 33, 48, 49])
@pytest.mark.parametrize("wt", ["bf16", "f32", "e2m1"])
def test_few_every_expert_has_every_token(wt, T, E, d, h):
    if wt == "e2m1":
        d, h = d // 32 * 32, h // 32 * 32
    say(f"few T={T} d={d} E=k={E} h={h} {wt}")
    c = Case(T, d, E, E, h, wt)
    m = c.layer()
    c.check(m.forward(c.x), m.topk_idx, m.topk_w)


@pytest.mark.parametrize("live", [0, 1, 3, 5])
def test_few_live_count_routed_in_its_own_launch(live):
    """More rows than are live, at 1024 workgroups and few tokens."""
    c = Case(5, 64, 200, 8, 416, "bf16")
    n = torch.tensor([live], dtype=torch.int32, device=DEV)
    m = c.layer()
    full = m.forward(c.x).clone()
    m.y.fill_(7)
    m.topk_idx.fill_(-7)
    m.forward(c.x, n_live=n)
    assert torch.equal(m.y[:live], full[:live]) and (m.y[live:] == 7).all() and (m.topk_idx[live:] == -7).all()


@pytest.mark.parametrize("wt", ["bf16", "e2m1"])
def test_few_smaller_batches_of_one_object(wt):
    """Every batch from 0 to the object's T through the same buffers; rows
    behind the batch keep what they held."""
    c = Case(19, 160, 6, 2, 96, wt)
    m = c.layer()
    whole = m.forward(c.x).clone()
    for t in (0, 1, 2, 4, 5, 8, 9, 15, 16, 17, 18, 19):
        m.y.fill_(7)
        m.topk_idx.fill_(-7)
        y = m.forward(c.x[:t])
        assert y.shape == (t, 160) and (m.y[t:] == 7).all() and (m.topk_idx[t:] == -7).all()
        if t:
            c.check(y, m.topk_idx[:t], m.topk_w[:t], c.x[:t])
            # a token's sums run over its own experts in the same order in every batch
            assert rel_l2(to_np(y), to_np(whole[:t])) < 2.0 ** -8


def test_few_workspace_of_an_object_holds_every_smaller_batch():
    from token_routing_grouped_amd import _abi

    for d, E, k, h in ((256, 8, 4, 128), (64, 384, 8, 32), (128, 2, 1, 64), (64, 1024, 32, 32)):
        sizes = [_abi.moe_few_workspace_size(t, d, E, k, h) for t in range(1, 65)]
        assert sizes == sorted(sizes)


def test_few_ties_go_to_the_lower_expert():
    """Equal rows of wr give bitwise equal logits."""
    c = Case(5, 128, 12, 4, 64, "bf16")
    c.wr[:] = c.wr[0].clone()
    m = c.layer()
    m.forward(c.x)
    assert torch.equal(m.topk_idx, torch.arange(4, dtype=torch.int32, device=DEV).expand(5, 4))
    assert (np.abs(to_np(m.topk_w) - 1 / 12) < 1e-6).all()


def test_few_agrees_with_the_layer():
    """The same tokens through MoELayerGPU: the same experts, gates to fp32
    rounding, y to the layer's own bf16 roundings (its G, U, H and Yp are
    stored in bf16: four half steps of at most 2^-8, and y's)."""
    from token_routing_grouped_amd.layer import MoELayerGPU

    c = Case(24, 256, 16, 4, 128, "bf16")
    m, full = c.layer(), MoELayerGPU(24, 256, 16, 4, 128, torch.bfloat16, DEV)
    y = m.forward(c.x)
    ref = full.forward(c.x, c.wr, *c.w)
    assert torch.equal(m.topk_idx, full.topk_idx)
    assert torch.allclose(m.topk_w, full.topk_w, rtol=1e-5, atol=0)
    assert rel_l2(to_np(y), to_np(ref)) <= 5 * 2.0 ** -8


def test_few_live_count_on_the_device():
    c = Case(20, 136, 9, 3, 40, "bf16")
    m = c.layer()
    want = {t: None for t in (0, 1, 16, 17, 20)}
    for t in want:
        m.y.fill_(3)
        m.forward(c.x[:t])
        want[t] = m.y.clone()
    for n, t in ((0, 0), (1, 1), (16, 16), (17, 17), (20, 20), (-5, 0), (99, 20)):  # the routing launch
        m.y.fill_(3)
        m.topk_idx.fill_(-3)
        m.topk_w.fill_(-3)
        x = c.x.clone()
        x[t:] = float("nan")  # what lies behind is not used
        m.forward(x, n_live=torch.tensor([n], dtype=torch.int32, device=DEV))
        assert torch.equal(m.y[t:], want[t][t:]) and (m.topk_idx[t:] == -3).all() and (m.topk_w[t:] == -3).all()
        if t:
            c.check(m.y[:t], m.topk_idx[:t], m.topk_w[:t], c.x[:t])


@pytest.mark.parametrize("T,E,wt", [(7, 9, "bf16"), (16, 40, "bf16"), (11, 16, "e2m1"), (4, 5, "f32")])
def test_few_live_count_where_the_projection_routes(T, E, wt):
    c = Case(T, 160, E, 3, 96, wt)
    m = c.layer()
    for n in range(0, T + 1):
        m.y.fill_(3)
        m.topk_idx.fill_(-3)
        x = c.x.clone()
        x[n:] = float("nan")
        m.forward(x, n_live=torch.tensor([n], dtype=torch.int32, device=DEV))
        assert (m.y[n:] == 3).all() and (m.topk_idx[n:] == -3).all()
        if n:
            c.check(m.y[:n], m.topk_idx[:n], m.topk_w[:n], c.x[:n])


def test_few_captured_once_for_every_batch():
    """One graph, replayed with other tokens and live counts in between, and
    two graphs that share the object's workspace."""
    c = Case(12, 256, 8, 2, 64, "bf16")
    m, n = c.layer(), torch.tensor([12], dtype=torch.int32, device=DEV)
    x = c.x.clone()
    m.forward(x, n_live=n)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.forward(x, n_live=n)
        graphs.append(g)
    for i, t in enumerate((12, 5, 0, 1, 12, 7)):
        x.copy_(c.x.roll(i, 0))
        n.fill_(t)
        eager_y = c.layer()
        eager_y.y.fill_(5)
        eager_y.forward(x, n_live=n)
        m.y.fill_(5)
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(m.y, eager_y.y)
        if t:
            assert torch.equal(m.topk_idx[:t], eager_y.topk_idx[:t])


@pytest.mark.parametrize("T,E,wt", [(6, 8, "bf16"), (1, 40, "e2m1"), (20, 300, "e2m1")])
def test_few_captured_and_replayed(T, E, wt):
    """Each way through (two launches, three, five): replays with other tokens
    equal eager calls bit for bit, whatever ran in between."""
    c = Case(T, 256, E, 2, 64, wt)
    m, e = c.layer(), c.layer()
    x = c.x.clone()
    m.forward(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.forward(x)
    for i in range(4):
        x.copy_(torch.from_numpy(np.random.default_rng(i).standard_normal((T, 256)).astype(np.float32)).to(DEV))
        e.forward(x)
        m.y.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(m.y, e.y) and torch.equal(m.topk_idx, e.topk_idx) and torch.equal(m.topk_w, e.topk_w)


def test_few_two_streams_at_once():
    """Two objects with the same weights on two streams, interleaved."""
    a = Case(3, 520, 16, 4, 256, "bf16")
    b = Case(3, 520, 16, 4, 256, "bf16")
    xb = torch.flip(a.x, (0,)).contiguous()
    ma, mb = a.layer(), _layer()(3, 4, a.wr, *a.w)
    ya, yb = ma.forward(a.x).clone(), mb.forward(xb).clone()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(sa):
            ma.forward(a.x)
        with torch.cuda.stream(sb):
            mb.forward(xb)
    torch.cuda.synchronize()
    assert torch.equal(ma.y, ya) and torch.equal(mb.y, yb)
    assert b.T == 3


@pytest.mark.parametrize("tokens", [6, 12, 18, 36])
def test_few_faulty_token_and_expert_stay_apart(tokens):
    """A NaN token's row is NaN and no other changes; an expert whose weights
    hold an infinity or NaN reaches only the tokens that chose it."""
    T = tokens
    c = Case(T, 136, 8, 2, 72, "bf16")
    m = c.layer()
    y0, i0 = m.forward(c.x).clone(), m.topk_idx.clone()
    x = c.x.clone()
    x[4, 10] = float("nan")
    y = m.forward(x)
    keep = torch.arange(T, device=DEV) != 4
    assert torch.equal(y[keep], y0[keep]) and torch.equal(m.topk_idx[keep], i0[keep]) and y[4].isnan().all()
    for which in range(3):
        for bad in (float("inf"), float("nan")):
            w = [a.clone() for a in c.w]
            e = int(i0[0, 0])
            w[which][e, 3, 5] = bad
            y = _layer()(T, 2, c.wr, *w).forward(c.x)
            hit = (i0 == e).any(1)
            assert hit.any()
            if hit.all():
                continue
            assert torch.equal(y[~hit], y0[~hit]) and not torch.isfinite(y[hit]).all(1).any()


@pytest.mark.parametrize("wt,d,h", [("bf16", 72, 40), ("f32", 40, 24), ("e2m1", 288, 96)])
@pytest.mark.parametrize("T", [2, 12, 20, 40])
def test_few_infinity_in_a_rows_last_values_stays_one(T, wt, d, h):
    """Rows that end inside a line: an infinite hidden value in the last place
    times a zero weight elsewhere must not turn into NaN.  x's last value is
    infinite and the matrices keep every sum a single infinity: W1 and W3 take
    x's last value with weight 1 into the last hidden value and 0 elsewhere, W2
    takes that into output 0; the other outputs read finite hidden values."""
    c = Case(T, d, 4, 1, h, "bf16" if wt == "e2m1" else wt)
    w1, w2 = torch.zeros(4, h, d), torch.zeros(4, d, h)
    w1[:, :, 0] = 1.0   # every hidden value from x[0]
    w2[:, :, 0] = 1.0   # every output from hidden 0
    x = torch.zeros(T, d)
    x[:, 0] = 1.0
    x[T - 1, d - 1] = 3e38  # finite, and infinite once squared by the SwiGLU
    w1[:, h - 1, d - 1] = 4.0
    w2[:, :, h - 1] = 0.5
    wr = torch.zeros(4, d)
    wr[0, 0] = 1.0
    put = lambda a: a.to(DEV).to(c.dt)
    if wt == "e2m1":
        q1, s1, _ = _pack(w1.numpy().astype(np.float64))
        q2, s2, _ = _pack(w2.numpy().astype(np.float64))
        m = _layer()(T, 1, put(wr), q1, q1, q2, w1s=s1, w3s=s1, w2s=s2)
    else:
        m = _layer()(T, 1, put(wr), put(w1), put(w1), put(w2))
    y = m.forward(put(x))
    assert torch.isfinite(y[:T - 1]).all() and (y[T - 1] == float("inf")).all()


def test_few_faulty_logits():
    """NaN and infinite router rows: a NaN logit never wins while others are
    left, indices stay distinct and in range."""
    c = Case(4, 128, 6, 3, 32, "bf16")
    wr = c.wr.clone()
    wr[2] = float("nan")
    m = _layer()(4, 3, wr, *c.w)
    m.forward(c.x)
    idx = to_np(m.topk_idx)
    assert (idx != 2).all() and all(len(set(r)) == 3 for r in idx)
    wr[:] = float("nan")
    m.forward(c.x)
    idx = to_np(m.topk_idx)
    assert all(sorted(r) == [0, 1, 2] for r in idx)


@pytest.mark.parametrize("wt", ["bf16", "f32", "e2m1"])
def test_few_writes_only_its_own(wt):
    """Guard bands around every buffer that is written."""
    from token_routing_grouped_amd import _abi

    c = Case(21, 160, 7, 3, 96, wt)
    m = c.layer()
    want = m.forward(c.x).clone()
    n = _abi.moe_few_workspace_size(21, 160, 7, 3, 96)
    ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    y = torch.full((23, 160), 9.0, dtype=c.dt, device=DEV)
    idx = torch.full((29, 3), -9, dtype=torch.int32, device=DEV)
    gate = torch.full((29, 3), -9.0, device=DEV)
    a = _abi.few_args(3, c.wr, *c.w, ws[256:256 + n], **c.scales)
    _abi.moe_few_fwd(a, c.x, y[1:22], idx[4:25], gate[4:25])
    assert (ws[:256] == 0xA5).all() and (ws[256 + n:] == 0xA5).all()
    assert (y[0] == 9).all() and (y[22] == 9).all()
    for b in (idx, gate):
        assert (b[:4] == -9).all() and (b[25:] == -9).all()
    assert torch.equal(y[1:22], want)


def test_few_refuses_what_does_not_fit():
    from token_routing_grouped_amd import _abi

    c = Case(4, 128, 6, 3, 32, "bf16")
    m = c.layer()
    for bad, text in ((c.x[:, :64].contiguous(), "columns"), (c.x.float(), "must be"),
                      (torch.cat([c.x, c.x]), "buffers are for")):
        with pytest.raises(_abi.MoeError, match=text):
            m.forward(bad)
    with pytest.raises(_abi.MoeError, match="contiguous"):
        m.forward(torch.cat([c.x, c.x], 1)[:, :128])
    with pytest.raises(_abi.MoeError, match="norm_w"):
        m.forward(c.x, res=c.x)
    with pytest.raises(_abi.MoeError, match="w2 must be"):
        _layer()(4, 3, c.wr, c.w[0], c.w[1], c.w[1])
    with pytest.raises(_abi.MoeError, match="T must be"):
        _layer()(65, 3, c.wr, *c.w)
    p = Case(4, 128, 6, 3, 32, "e2m1")
    with pytest.raises(_abi.MoeError, match="w3s is needed"):
        _layer()(4, 3, p.wr, *p.w, w1s=p.scales["w1s"])
    with pytest.raises(_abi.MoeError, match="packed weights only"):
        _layer()(4, 3, c.wr, *c.w, w1s=p.scales["w1s"])


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The library launches on the current device: tensors of another one are
    refused before the call.  (The current device's number is changed for the
    check alone; nothing is launched.)"""
    from token_routing_grouped_amd import _abi

    c = Case(4, 128, 6, 3, 32, "bf16")
    m = c.layer()
    monkeypatch.setattr(_abi.torch.cuda, "current_device", lambda: 1)
    with pytest.raises(_abi.MoeError, match="current device is cuda:1"):
        m.forward(c.x)


@pytest.mark.parametrize("wt", ["bf16", "e2m1"])
def test_decode_block_together(wt):
    """A run as a server makes it: norm with residual, layer, and the stream
    handed to the next step's norm, three steps, against float64.  Between the
    steps the values are the stored bf16 ones."""
    from oracle import norm_ref

    c = Case(6, 288, 8, 2, 96, wt)
    g = np.random.default_rng(9)
    nw = torch.from_numpy(1 + 0.1 * g.standard_normal(288)).to(DEV).to(torch.bfloat16)
    m = c.layer(norm_w=nw, eps=1e-5)
    x, res = c.x.clone(), None
    for _ in range(3):
        y = m.forward(x, res=res).clone()
        s = m.s.clone()
        ry, rs, _ = norm_ref.forward(to_np(x), to_np(nw), 1e-5, None if res is None else to_np(res))
        assert (np.abs(to_np(s) - rs) <= (2.0 ** -8 + 2 * U) * np.abs(rs)).all()
        xn = to_np(m.xn)
        assert (np.abs(xn - ry) <= (2.0 ** -8 + 128 * U) * np.abs(ry)).all()
        c.check(y, m.topk_idx, m.topk_w, m.xn)
        x, res = y, s


def test_dense_expert_from_the_norms_mx_copy():
    """moe_rmsnorm_fwd's MXFP8 copy straight into the scaled grouped GEMM with
    one expert (a dense or shared FFN): the same result, bit for bit, as
    quantising the fp32-normed rows in a pass of their own."""
    from token_routing_grouped_amd import _abi

    T, d, h, bf, u8 = 70, 256, 128, torch.bfloat16, torch.uint8
    g = np.random.default_rng(2)
    t = lambda *n, sc=1.0, dt=bf: (torch.from_numpy(g.standard_normal(n)) * sc).to(DEV).to(dt)
    x, res, nw = t(T, d, dt=torch.float32), t(T, d, dt=torch.float32), t(d, dt=torch.float32)
    ws = [t(h, d, sc=0.1), t(h, d, sc=0.1), t(d, h, sc=0.1)]
    e = lambda *n, dt=u8: torch.zeros(*n, dtype=dt, device=DEV)
    wq = []
    for w in ws:
        q, s = e(*w.shape), e(_abi.mx_scale_bytes(*w.shape))
        _abi.mx_quantize(w, w.shape[0], q, s, seg_rows=w.shape[0])
        wq += [q, s]
    rc = (T + 127 + 127) // 128 * 128
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    off128 = torch.tensor([0, 128], dtype=torch.int32, device=DEV)

    def ffn(xq, xs):
        yp = e(T, d, dt=bf)
        _abi.moe_grouped_gemm_fwd_mx(E=1, R=T, d=d, h=h, rcap=rc, offsets=off, off128=off128, xq=xq, xs=xs, w1q=wq[0],
                                     w1s=wq[1], w3q=wq[2], w3s=wq[3], w2q=wq[4], w2s=wq[5], g=None, u=None,
                                     hbuf=e(T, h, dt=bf), hq=e(T, h), hs=e(T * h // 32), hqT=e(h * rc),
                                     hsT=e(h * rc // 32), yp=yp, ws=e(16), ws_bytes=16)
        return yp

    y32, q, qs = torch.empty_like(x), e(T, d), e(_abi.mx_scale_bytes(T, d))
    _abi.moe_rmsnorm_fwd(x, nw, 1e-6, y32, res=res, q=q, qs=qs)
    q2, qs2 = e(T, d), e(_abi.mx_scale_bytes(T, d))
    _abi.mx_quantize(y32, T, q2, qs2, seg_rows=T)
    out = ffn(q, qs)
    assert torch.equal(out, ffn(q2, qs2)) and out.float().abs().max() > 0


def test_training_block_gradients():
    """MoEBlockGPU: one step of norm and layer, forward and backward, against
    the composed float64 oracles (the layer's own bounds: rel-L2 1e-2)."""
    from oracle import norm_ref
    from token_routing_grouped_amd.layer import MoEBlockGPU, MoELayerGPU

    T, d, E, k, h = 96, 256, 8, 2, 128
    c = Case(64, d, E, k, h, "bf16")
    g = np.random.default_rng(4)
    t = lambda *n, sc=1.0: (torch.from_numpy(g.standard_normal(n)) * sc).to(DEV).to(torch.bfloat16)
    x, res, dy, ds, nw = t(T, d), t(T, d), t(T, d), t(T, d), (1 + 0.1 * t(d)).to(torch.bfloat16)
    b = MoEBlockGPU(MoELayerGPU(T, d, E, k, h, torch.bfloat16, DEV), eps=1e-5)
    y = b.forward(x, nw, c.wr, *c.w, res=res)
    dx = b.backward(dy, nw, c.wr, *c.w, ds=ds)
    f64 = lambda a: to_np(a).astype(np.float64)
    xn, s, rstd = norm_ref.forward(f64(x), f64(nw), 1e-5, f64(res))
    f = moe_ref.layer_forward(xn, f64(c.wr), *c.v, k, logits=to_np(b.layer.logits))
    lb = moe_ref.layer_backward(f, f64(dy), xn, f64(c.wr), *c.v)
    rdx, rdw = norm_ref.backward(lb["dx"], s, f64(nw), rstd, f64(ds))
    for name, got, ref in (("y", y, f["y"]), ("s", b.s, s), ("dx", dx, rdx), ("dnorm_w", b.dnorm_w, rdw),
                           ("dw1", b.layer.dw1, lb["dw1"]), ("dwr", b.layer.dwr, lb["dwr"])):
        assert rel_l2(to_np(got), ref) <= 1e-2, name
