"""moe_orthogonalize / moe_muon_step against the float64 oracle.

Tolerances.  The library's error is that of what it stores: every iterate, A
and B once rounded to fp16 (bf16 matrices) or to two fp16 planes (fp32 ones),
sums in fp32.  The oracle runs the same iteration with the same roundings (and,
for the planes, whose steps are as fine as fp32's sums, with fp32 products);
its distance from the exact result, from singular values, is E.  The library's
roundings are the same ones but for those where its sums' last bits decide, so
its own distance is allowed 2 E (fp32: 4 E, its sums being other sums of the
same fineness), in the Frobenius norm, and 4 times the oracle's largest for
single entries, plus the output's own rounding.

What that model leaves out is the evaluation in fp32 (evaluation() below), which
for a few rows of fp32 values is as large as E.  Of a step with singular values
s (so |X|_F = |s|, |A|_F = |s^2|), in units of 4 2^-24:
  B = a + b A + c A^2 from rounded a, b and c, two products, two sums: under 4
  roundings of a |I| + |b| |A| + |c| |A^2| (r values s: |I| = sqrt(r)), times X:
  (a sqrt(r) + |b| |s^2| + |c| |s^4|) max s;
  the planes' lo lo products, left out: 2^-22 of the products' terms, at most
  |X|_F^2 in A (whence |b| + 2 |c| max s^2 and X: times max s), |c| |A|_F^2 in
  A^2 (times max s), |B|_F |X|_F in B X.
An error at step k reaches the end through the later steps' maps, whose
Lipschitz constant in the Frobenius norm is at most the largest of |p'| and
p(s) / s over the interval of that step's singular values.
"""

import numpy as np
import pytest
import torch

from oracle import dense_ref as ref

from helpers import say, to_np

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
FAR = {"bf16": 2.0, "f32": 4.0}


def _abi():
    from token_routing_grouped_amd import _abi as a

    return a


def _f64(t):
    return to_np(t).astype(np.float64)


def _model(dt):
    if dt == "bf16":
        return dict(store=ref.store_f16)
    return dict(store=ref.store_2f16, mul=ref.mul_f32)


def _gradients(B, rows, cols, dt, seed=0, std=1e-3):
    g = np.random.default_rng(seed + 7 * rows + cols)
    v = g.standard_normal((B, rows, cols)) * std
    v += np.einsum("bri,bic->brc", g.standard_normal((B, rows, 2)), g.standard_normal((B, 2, cols))) * std
    return torch.from_numpy(v.astype(np.float32)).to(DEV).to(DT[dt])


def _ws(abi, t):
    return abi.workspace(abi.moe_orthogonalize_workspace_size(*t.shape, t.dtype), DEV).fill_(0xFF)


def evaluation(u, steps, eps, planes):
    """Frobenius-norm bound on what fp32 evaluation adds (module docstring)."""
    a, b, c = ref.A, abs(ref.B), abs(ref.C)
    s = np.linalg.svd(u, compute_uv=False)
    s = s / (np.sqrt((s * s).sum()) + eps)
    n = np.linalg.norm
    total = 2.0 ** -24 * n(s) * 4  # the first X from u
    for k in range(steps):
        t = np.linspace(s.min(), s.max(), 257)
        t = t[t > 0]
        if t.size:
            total *= max(np.abs(ref.A + 3 * ref.B * t ** 2 + 5 * ref.C * t ** 4).max(), (ref.quintic(t) / t).max())
        top, m = s.max(), a * len(s) ** 0.5 + b * n(s ** 2) + c * n(s ** 4)
        d = m * top
        if planes:
            d += n(s) ** 2 * (b + 2 * c * top ** 2) * top + c * n(s ** 2) ** 2 * top + m * n(s)
        total += 2.0 ** -22 * d
        s = ref.quintic(s)
    return total


def _check_one(got, u, dt, steps=5, scale=1.0, base=0.0, eps=1e-7, half=None):
    """got [rows, cols] against base + scale * orthogonalised u, all float64."""
    exact, model = ref.orthogonalize(u, steps, eps), ref.iterate(u, steps, eps, **_model(dt))
    e = np.abs(scale) * (model - exact)
    want = base + scale * exact
    err = np.abs(got - want)
    half = HALF[dt] if half is None else half
    out = half * np.linalg.norm(want) + 2.0 ** -23 * (np.linalg.norm(base) + np.abs(scale) * np.linalg.norm(exact))
    ev = np.abs(scale) * evaluation(u, steps, eps, dt == "f32")
    assert np.linalg.norm(err) <= FAR[dt] * np.linalg.norm(e) + ev + out + 1e-30, (np.linalg.norm(err), np.linalg.norm(e))
    one = half * np.abs(want) + 2.0 ** -23 * (np.abs(base) + np.abs(scale * exact)).max()
    assert (err <= 4 * np.abs(e).max() + ev + one + 1e-30).all()


# vectors, squares, wide and tall, ragged sides, several tiles, several K parts
SHAPES = [(1, 1, 8), (2, 1, 64), (2, 8, 8), (3, 9, 24), (2, 64, 64), (2, 40, 136), (2, 136, 40), (1, 100, 600),
          (1, 601, 96), (2, 130, 136), (1, 128, 2048), (1, 300, 264), (1, 7, 1000)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,rows,cols", SHAPES)
def test_orthogonalize(B, rows, cols, dt):
    if dt == "f32" and cols > 8:
        cols += 4  # a row that ends inside 8 values
    say(f"orthogonalize {B} {rows} {cols} {dt}")
    abi = _abi()
    g = _gradients(B, rows, cols, dt)
    out = torch.full_like(g, np.nan)
    ws = _ws(abi, g)
    abi.moe_orthogonalize(g, out, ws)
    for b in range(B):
        _check_one(_f64(out[b]), _f64(g[b]), dt)
    same = g.clone()  # in place, and again
    abi.moe_orthogonalize(same, same, ws.fill_(0xFF))
    assert torch.equal(same, out)


@pytest.mark.parametrize("steps", [1, 2, 8])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_steps(steps, dt):
    abi = _abi()
    g = _gradients(2, 48, 72, dt, 3)
    out = torch.empty_like(g)
    abi.moe_orthogonalize(g, out, _ws(abi, g), steps=steps)
    for b in range(2):
        _check_one(_f64(out[b]), _f64(g[b]), dt, steps)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("std", [1e-30, 1e-15, 1e15, 1e30])
def test_any_scale(std, dt):
    """Squares of these values leave fp32's range; the norm does not."""
    abi = _abi()
    g = _gradients(1, 40, 64, dt, 4, std)
    out = torch.empty_like(g)
    abi.moe_orthogonalize(g, out, _ws(abi, g), eps=0.0)
    _check_one(_f64(out[0]), _f64(g[0]), dt, eps=0.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [0.0, 1e-7])
def test_zero_and_non_finite_matrices(dt, eps):
    """A matrix of zeros (an expert without tokens) gives zeros; one with an
    infinity or NaN gives NaNs; the others are what they are by themselves."""
    abi = _abi()
    g = _gradients(5, 72, 40, dt, 5)
    g[1] = 0
    g[2, 71, 39] = float("inf")
    g[3, 0, 0] = float("nan")
    out = torch.empty_like(g)
    abi.moe_orthogonalize(g, out, _ws(abi, g), eps=eps)
    assert (out[1] == 0).all() and out[2].isnan().all() and out[3].isnan().all()
    for b in (0, 4):
        _check_one(_f64(out[b]), _f64(g[b]), dt, eps=eps)


def test_what_lies_around_is_not_read_or_written():
    abi, pad = _abi(), 512
    for shape in ((2, 42, 72), (2, 72, 40)):
        g = _gradients(*shape, "bf16", 6)
        n = g.numel()
        big = torch.full((n + 2 * pad,), np.nan, dtype=g.dtype, device=DEV)
        big[pad:pad + n] = g.view(-1)
        bo = torch.full_like(big, 7.0)
        ws = _ws(abi, g)
        abi.moe_orthogonalize(big[pad:pad + n].view(shape), bo[pad:pad + n].view(shape), ws)
        want = torch.empty_like(g)
        abi.moe_orthogonalize(g, want, ws)
        assert torch.equal(bo[pad:pad + n].view(shape), want)
        assert (bo[:pad] == 7).all() and (bo[pad + n:] == 7).all()


@pytest.mark.parametrize("dt,master", [("bf16", True), ("bf16", False), ("f32", False), ("f32", True)])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("rows,cols", [(72, 136), (136, 72)])
def test_muon_step(rows, cols, dt, master, nesterov):
    say(f"muon {rows} {cols} {dt} master={master} nesterov={nesterov}")
    abi, B = _abi(), 2
    g = _gradients(B, rows, cols, dt, 8)
    buf = _gradients(B, rows, cols, "f32", 9)
    w32 = torch.randn(B, rows, cols, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).mul_(0.05)
    w = w32.to(DT[dt], copy=True)
    m = w32 if master else None
    new = dict(w_out=torch.full_like(w, np.nan), buf_out=torch.full_like(buf, np.nan),
               master_out=torch.full_like(w32, np.nan) if master else None)
    scale = torch.tensor(0.5, device=DEV)
    kw = dict(step=0.3, decay=0.02, momentum=0.9, nesterov=nesterov, master=m, lr_scale=scale)
    ws = _ws(abi, g)
    abi.moe_muon_step(w, g, buf, ws, **kw, **new)
    for b in range(B):
        wb, gb, bb = (_f64(t[b]) for t in (w32 if master else w, g, buf))
        _, rb = ref.muon(wb, gb, bb, 0, 0, 0.9, nesterov)
        assert (np.abs(_f64(new["buf_out"][b]) - rb) <= 2.0 ** -23 * (np.abs(0.9 * bb) + np.abs(gb))).all()
        u = gb + 0.9 * rb if nesterov else rb
        # u itself is rounded to fp32 (relative 2^-22 of its terms), far below what is stored of it in fp16; in
        # planes it is of their fineness, which the tolerance's factor has room for
        _check_one(_f64(new["w_out"][b]), u, dt, scale=-0.15, base=wb * 0.99)
        if master:
            _check_one(_f64(new["master_out"][b]), u, dt, scale=-0.15, base=wb * 0.99, half=HALF["f32"])
    if master:
        assert torch.equal(new["master_out"].to(w.dtype), new["w_out"])
    # in place
    abi.moe_muon_step(w, g, buf, ws.fill_(0xFF), **kw)
    assert torch.equal(w, new["w_out"]) and torch.equal(buf, new["buf_out"])
    if master:
        assert torch.equal(w32, new["master_out"])


def test_no_matrices():
    abi = _abi()
    g = torch.empty(0, 16, 16, device=DEV)
    abi.moe_orthogonalize(g, g, _ws(abi, g))
    abi.moe_muon_step(g, g, g, _ws(abi, g), step=0.1)


def test_captured_and_replayed():
    """A step in a graph, replayed: the same as eager steps, with the schedule's
    factor changed on the device in between."""
    abi = _abi()
    g = _gradients(3, 72, 264, "bf16", 11)
    w0 = torch.randn(3, 72, 264, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)).mul_(0.05)
    scale = torch.ones((), device=DEV)
    a = [w0.bfloat16(), torch.zeros_like(w0), w0.clone(), _ws(abi, g)]
    b = [t.clone() for t in a]

    def step(t):
        abi.moe_muon_step(t[0], g, t[1], t[3], step=0.1, decay=0.01, master=t[2], lr_scale=scale)

    step(a)
    step(b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step(a)
    torch.cuda.current_stream().wait_stream(s)
    for rep in range(4):
        scale.fill_(1.0 / (rep + 1))
        g.copy_(_gradients(3, 72, 264, "bf16", 40 + rep))
        step(b)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(a[:3], b[:3]):
            assert torch.equal(p, q), rep
