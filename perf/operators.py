"""The token-sized and 4-bit operators around the expert layer, in their plain
form (elementary torch operations in 32 bits) and as calls of the framework's
own kernels, over the sizes they are used at.

  norm     the block's root-mean-square norm with the residual's addition in
           front of the layer, optionally with the MXFP8 copy of its output
  norm_bwd its gradients (input and weight)
  few      a whole mixture-of-experts layer for a few tokens (serving): router,
           top-k, the chosen experts' SwiGLU FFNs and the gated sum, with the
           experts' weights in fp32, bf16 or 4 bits (E2M1, one scale per 32)
  linear   a few tokens through one dense matrix of 4-bit weights
  quant    weights to 4 bits and back to the values they stand for

A case is a dict of plain values.  `own` chooses between the plain form and the
framework's calls; prepare() makes the same inputs for both.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
#: Values of the eight E2M1 magnitudes; a code's bit 3 is its sign.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decode step, in front of the layer
        {"name": "norm_one_token", "op": "norm", "T": 1, "d": 2048, "dt": "bf16", "res": True, "mx": False},
        # a training step's tokens, with the MXFP8 copy for the scaled products
        {"name": "norm_step_mx", "op": "norm", "T": 16384, "d": 2048, "dt": "bf16", "res": True, "mx": True},
        # the same step's backward, the residual's gradient coming in beside it
        {"name": "norm_bwd_step", "op": "norm_bwd", "T": 16384, "d": 2048, "dt": "bf16", "ds": True},
        # an odd number of wide rows in fp32, as a last ragged micro-batch has
        {"name": "norm_bwd_ragged_f32", "op": "norm_bwd", "T": 1021, "d": 6144, "dt": "f32", "ds": False},
        # one sequence decoding through the 8-expert layer
        {"name": "few_one_small", "op": "few", "T": 1, "d": 2048, "E": 8, "k": 4, "h": 1024, "wt": "bf16"},
        # a decode batch through the widest layer: most of its weights are read
        {"name": "few_24_trillion", "op": "few", "T": 24, "d": 6144, "E": 384, "k": 8, "h": 2048, "wt": "bf16"},
        # one sequence through the 128-expert layer, its experts held in 4 bits
        {"name": "few_one_wide_e2m1", "op": "few", "T": 1, "d": 2048, "E": 128, "k": 4, "h": 1024, "wt": "e2m1"},
        # a full odd batch through it: about two tokens an expert
        {"name": "few_61_wide_e2m1", "op": "few", "T": 61, "d": 2048, "E": 128, "k": 4, "h": 1024, "wt": "e2m1"},
        # a dense projection beside the experts, one token
        {"name": "linear_one", "op": "linear", "T": 1, "n": 6144, "K": 2048},
        # a wide dense projection, a small batch (speculative or several users)
        {"name": "linear_13_wide", "op": "linear", "T": 13, "n": 24576, "K": 6144},
        # a small odd matrix, as one expert loaded by itself
        {"name": "quant_small_f32", "op": "quant", "rows": 1023, "cols": 2048, "dt": "f32"},
        # all of one projection of the 8-expert layer
        {"name": "quant_experts", "op": "quant", "rows": 8192, "cols": 2048, "dt": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step - 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "few", "few", "linear", "quant"])
    if op in ("norm", "norm_bwd"):
        dt = rng.choice(["bf16", "bf16", "f32"])
        mx = op == "norm" and rng.random() < 0.5
        d = _log(rng, 128, 8192, 128 if mx else 8)
        T = _log(rng, 1, min(16384, (1 << 24) // d))
        if op == "norm":
            return {"op": op, "T": T, "d": d, "dt": dt, "res": rng.random() < 0.7, "mx": mx}
        return {"op": op, "T": T, "d": d, "dt": dt, "ds": rng.random() < 0.5}
    if op == "few":
        wt = rng.choice(["bf16", "bf16", "e2m1", "e2m1", "f32"])
        step = 32 if wt == "e2m1" else 8
        while True:
            d, h = _log(rng, 128, 6144, step), _log(rng, 64, 2048, step)
            E, T = _log(rng, 2, 384), _log(rng, 1, 64)
            k = rng.randint(1, min(E, 8))
            if E * d * h <= 1 << 28 and T * k * d * h <= 1 << 31:
                return {"op": op, "T": T, "d": d, "E": E, "k": k, "h": h, "wt": wt}
    if op == "linear":
        n, K = _log(rng, 64, 24576), _log(rng, 128, 8192, 32)
        return {"op": op, "T": _log(rng, 1, 64), "n": n, "K": K}
    return {"op": op, "rows": _log(rng, 64, 8192), "cols": _log(rng, 64, 2048, 32), "dt": rng.choice(["bf16", "f32"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _scale_bytes(rows, K):
    return -(-K // 128) * rows * 4


def _scales_to_bytes(e, rows, K):
    """Exponents [rows, K/32] as the library's K-chunk-major bytes
    [ceil(K/128), rows, 4] (a short last chunk's places hold 0)."""
    out = torch.zeros(rows, -(-K // 128) * 4, dtype=torch.uint8, device=e.device)
    out[:, :K // 32] = (e + 127).to(torch.uint8)
    return out.view(rows, -1, 4).transpose(0, 1).contiguous().view(-1)


def _scales_of_bytes(b, rows, K):
    """2^s of the library's scale bytes, [rows, K/32] fp32."""
    e = b.view(-1, rows, 4).transpose(0, 1).reshape(rows, -1)[:, :K // 32].to(torch.int32) - 127
    return torch.ldexp(torch.ones((), device=b.device), e)


def _to_e2m1(w):
    """Plain E2M1 quantisation of [rows, K]: packed codes (two to a byte, the
    even value in the low half) and scale bytes."""
    rows, K = w.shape
    b = w.float().view(rows, K // 32, 32)
    amax = b.abs().amax(2)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 3).clamp(-127, 127), -127)
    a = torch.ldexp(b.abs(), -e.unsqueeze(2)).clamp(max=6.0)
    # round to nearest, ties to the even code: steps of 1/2 below 2, 1 below 4, 2 above
    mag = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    c = (mag.to(torch.uint8) | (torch.signbit(b).to(torch.uint8) << 3)).view(rows, K // 2, 2)
    return c[:, :, 0] | (c[:, :, 1] << 4), _scales_to_bytes(e, rows, K)


def _of_e2m1(q, s, rows, K):
    """fp32 values of packed codes and scale bytes, [rows, K]."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=q.device)
    c = torch.stack((q & 15, q >> 4), 2).view(rows, K)
    return (v[c.int()].view(rows, K // 32, 32) * _scales_of_bytes(s, rows, K).unsqueeze(2)).view(rows, K)


def _normal(g, *shape, std=1.0, dt=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dt).mul_(std)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        dt, T, d = TYPES[c["dt"]], c["T"], c["d"]
        w = (1 + 0.1 * _normal(g, d, dt=torch.float32)).to(dt)
        if op == "norm":
            c.update(x=_normal(g, T, d, dt=dt), w=w, r=_normal(g, T, d, std=2.0, dt=dt) if c["res"] else None)
        else:
            s = _normal(g, T, d, std=2.0, dt=dt)
            c.update(s=s, w=w, rstd=torch.rsqrt(s.float().square().mean(1) + EPS), dy=_normal(g, T, d, dt=dt),
                     dsum=_normal(g, T, d, dt=dt) if c["ds"] else None)
    elif op == "few":
        T, d, E, h, wt = c["T"], c["d"], c["E"], c["h"], c["wt"]
        dt = torch.float32 if wt == "f32" else torch.bfloat16
        c.update(x=_normal(g, T, d, dt=dt), wr=_normal(g, E, d, std=0.02, dt=dt))
        for n, rows, K in (("w1", E * h, d), ("w3", E * h, d), ("w2", E * d, h)):
            w = _normal(g, rows, K, std=0.02, dt=dt)
            if wt == "e2m1":
                q, c[n + "s"] = _to_e2m1(w)
                c[n] = q.view(E, rows // E, K // 2)
            else:
                c[n] = w.view(E, rows // E, K)
    elif op == "linear":
        c["x"] = _normal(g, c["T"], c["K"])
        c["q"], c["s"] = _to_e2m1(_normal(g, c["n"], c["K"], std=0.02))
    else:
        c["w"] = _normal(g, c["rows"], c["cols"], std=0.02, dt=TYPES[c["dt"]])
    return c


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(c):
    return (_OWN if own else _PLAIN)[c["op"]](c)


def _norm(c):
    T, d = c["T"], c["d"]
    v = c["x"].float() if c["r"] is None else c["x"].float() + c["r"].float()
    rstd = torch.rsqrt(v.square().mean(1) + EPS)
    y = v * rstd.unsqueeze(1) * c["w"].float()
    out = {"y": y.to(c["x"].dtype), "rstd": rstd}
    if c["r"] is not None:
        out["s"] = v.to(c["x"].dtype)
    if c["mx"]:
        b = y.view(T, d // 32, 32)
        amax = b.abs().amax(2)
        e = torch.where(amax > 0, (torch.frexp(amax)[1] - 9).clamp(-127, 127), -127)
        q = torch.ldexp(b, -e.unsqueeze(2)).clamp(-448.0, 448.0)
        out["q"] = q.to(torch.float8_e4m3fn).view(T, d)
        out["qs"] = _scales_to_bytes(e, T, d).view(torch.float8_e8m0fnu)
    return out


def _norm_bwd(c):
    xh = c["s"].float() * c["rstd"].unsqueeze(1)
    dy = c["dy"].float()
    g = dy * c["w"].float()
    dx = c["rstd"].unsqueeze(1) * (g - xh * (g * xh).mean(1, keepdim=True))
    if c["dsum"] is not None:
        dx = dx + c["dsum"].float()
    return {"dx": dx.to(c["s"].dtype), "dw": (dy * xh).sum(0).to(c["w"].dtype)}


def _expert_weight(c, n, idx):
    """fp32 weights of the experts idx [R], [R, rows, K]."""
    w = c[n][idx]
    if c["wt"] != "e2m1":
        return w.float()
    E, rows, K = c["E"], w.shape[1], w.shape[2] * 2
    s = c[n + "s"].view(-1, E, rows, 4)[:, idx].reshape(-1, idx.numel() * rows, 4)
    return _of_e2m1(w.reshape(-1, K // 2), s.reshape(-1), idx.numel() * rows, K).view(-1, rows, K)


def _few(c):
    T, d, k = c["T"], c["d"], c["k"]
    x = c["x"].float()
    p = torch.softmax(x @ c["wr"].float().t(), 1)
    order = torch.sort(p, dim=1, descending=True, stable=True)  # ties: the lower expert first
    gate, idx = order.values[:, :k].contiguous(), order.indices[:, :k].contiguous()
    e = idx.view(-1)
    xr = x.repeat_interleave(k, 0).unsqueeze(2)
    a = torch.bmm(_expert_weight(c, "w1", e), xr)
    b = torch.bmm(_expert_weight(c, "w3", e), xr)
    hid = a * torch.sigmoid(a) * b
    yp = torch.bmm(_expert_weight(c, "w2", e), hid).view(T, k, d)
    return {"y": (gate.unsqueeze(2) * yp).sum(1).to(c["x"].dtype), "topk_idx": idx.int(), "topk_w": gate}


def _linear(c):
    return (c["x"].float() @ _of_e2m1(c["q"], c["s"], c["n"], c["K"]).t()).to(c["x"].dtype)


def _quant(c):
    q, s = _to_e2m1(c["w"])
    return {"w": _of_e2m1(q, s, c["rows"], c["cols"]).to(c["w"].dtype), "s": s.view(torch.float8_e8m0fnu)}


_PLAIN = {"norm": _norm, "norm_bwd": _norm_bwd, "few": _few, "linear": _linear, "quant": _quant}


def _own_norm(c):
    from token_routing_grouped_amd import _abi

    x, T, d = c["x"], c["T"], c["d"]
    if "out" not in c:  # a program's own buffers, kept from step to step
        o = c["out"] = {"y": torch.empty_like(x), "rstd": torch.empty(T, device=DEV)}
        if c["r"] is not None:
            o["s"] = torch.empty_like(x)
        if c["mx"]:
            o["q"] = torch.empty(T, d, dtype=torch.uint8, device=DEV)
            o["qs"] = torch.empty(_scale_bytes(T, d), dtype=torch.uint8, device=DEV)
    o = c["out"]
    _abi.moe_rmsnorm_fwd(x, c["w"], EPS, o["y"], res=c["r"], s=o.get("s"), q=o.get("q"), qs=o.get("qs"), rstd=o["rstd"])
    if not c["mx"]:
        return o
    return dict(o, q=o["q"].view(torch.float8_e4m3fn), qs=o["qs"].view(torch.float8_e8m0fnu))


def _own_norm_bwd(c):
    from token_routing_grouped_amd import _abi

    s, T, d = c["s"], c["T"], c["d"]
    if "out" not in c:
        c["ws"] = _abi.workspace(_abi.moe_rmsnorm_bwd_workspace_size(T, d), DEV)
        c["out"] = {"dx": torch.empty_like(s), "dw": torch.empty_like(c["w"])}
    o = c["out"]
    _abi.moe_rmsnorm_bwd(c["dy"], s, c["w"], c["rstd"], o["dx"], o["dw"], c["ws"], ds=c["dsum"])
    return o


def _own_few(c):
    from token_routing_grouped_amd.layer import MoEDecodeGPU

    if "layer" not in c:  # the layer's buffers and workspace, for these weights
        scales = {n + "s": c[n + "s"] for n in ("w1", "w3", "w2")} if c["wt"] == "e2m1" else {}
        c["layer"] = MoEDecodeGPU(c["T"], c["k"], c["wr"], c["w1"], c["w3"], c["w2"], **scales)
    m = c["layer"]
    m.forward(c["x"])
    return {"y": m.y, "topk_idx": m.topk_idx, "topk_w": m.topk_w}


def _own_linear(c):
    from token_routing_grouped_amd import _abi

    if "out" not in c:
        c["out"] = torch.empty(c["T"], c["n"], dtype=c["x"].dtype, device=DEV)
    _abi.mx_linear_e2m1(c["x"], c["q"], c["s"], c["out"])
    return c["out"]


def _own_quant(c):
    from token_routing_grouped_amd import _abi

    w, rows, cols = c["w"], c["rows"], c["cols"]
    if "out" not in c:
        c["codes"] = torch.empty(rows, cols // 2, dtype=torch.uint8, device=DEV)
        c["out"] = {"w": torch.empty_like(w), "s": torch.empty(_scale_bytes(rows, cols), dtype=torch.uint8, device=DEV)}
    o = c["out"]
    _abi.mx_quantize_e2m1(w, c["codes"], o["s"])
    _abi.mx_dequantize_e2m1(c["codes"], o["s"], o["w"])
    return {"w": o["w"], "s": o["s"].view(torch.float8_e8m0fnu)}


_OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "few": _own_few, "linear": _own_linear, "quant": _own_quant}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _weight_bytes(n, wt):
    return n * {"f32": 4, "bf16": 2, "e2m1": 17 / 32}[wt]


def work(case):
    c, op = case, case["op"]
    if op == "norm":
        n, es = c["T"] * c["d"], 4 if c["dt"] == "f32" else 2
        b = n * es * (4 if c["res"] else 2) + (n * 33 / 32 if c["mx"] else 0) + 4 * c["T"] + c["d"] * es
        return {"bytes": b, "flops": n * (8 if c["mx"] else 5)}
    if op == "norm_bwd":
        n, es = c["T"] * c["d"], 4 if c["dt"] == "f32" else 2
        return {"bytes": n * es * (4 if c["ds"] else 3) + 4 * c["T"] + 2 * c["d"] * es, "flops": 10 * n}
    if op == "few":
        T, d, E, k, h = (c[n] for n in "TdEkh")
        es = 4 if c["wt"] == "f32" else 2
        hit = E * (1 - (1 - k / E) ** T)  # experts that T tokens choose, with even routing
        b = hit * _weight_bytes(3 * d * h, c["wt"]) + E * d * es + 2 * T * d * es + 8 * T * k
        return {"bytes": b, "flops": 6 * T * k * d * h + 2 * T * E * d}
    if op == "linear":
        T, n, K = c["T"], c["n"], c["K"]
        return {"bytes": _weight_bytes(n * K, "e2m1") + 2 * T * (n + K), "flops": 2 * T * n * K}
    n = c["rows"] * c["cols"]
    # the values in, the codes and scales out and in again, the values out
    return {"bytes": n * (2 * (4 if c["dt"] == "f32" else 2) + 2 * 17 / 32), "flops": 4 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _e2m1_exact(q, s, rows, K):
    """Values of packed codes in 64 bits, from the format's fields: sign, two
    exponent bits (bias 1), one mantissa bit; exponent 0 is subnormal."""
    c = torch.empty(rows, K, dtype=torch.int64, device=q.device)
    c[:, 0::2], c[:, 1::2] = q.view(rows, -1) & 15, q.view(rows, -1) >> 4
    ex, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((ex - 1).double()))
    col = torch.arange(K, device=q.device) // 32
    at = (col // 4 * rows).unsqueeze(0) * 4 + torch.arange(rows, device=q.device).unsqueeze(1) * 4 + col % 4
    return torch.where(c >= 8, -mag, mag) * torch.exp2(s[at].double() - 127)


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op == "norm":
        v = c["x"].double()
        if c["r"] is not None:
            v = v + c["r"].double()
        ms = (v * v).sum(1, keepdim=True) / c["d"] + EPS
        y = v / ms.sqrt() * c["w"].double()
        out = {"y": y, "rstd": 1 / ms.sqrt().view(-1)}
        if c["r"] is not None:
            out["s"] = v
        if c["mx"]:
            # the value that each 8-bit element stands for, before its rounding;
            # the scales are steps of the data and have no value between
            top = y.abs().view(c["T"], -1, 32).amax(2, keepdim=True)
            scale = torch.exp2(torch.frexp(top)[1].double() - 9)
            out["q"] = (y.view(c["T"], -1, 32) / scale).clamp(-448, 448).view(c["T"], -1)
            out["qs"] = None
        return out
    if op == "norm_bwd":
        s, r, dy, w = c["s"].double(), c["rstd"].double().view(-1, 1), c["dy"].double(), c["w"].double()
        inner = (dy * w * s).sum(1, keepdim=True) / c["d"]
        dx = r * dy * w - r ** 3 * s * inner
        return {"dx": dx if c["dsum"] is None else dx + c["dsum"].double(), "dw": (dy * s * r).sum(0)}
    if op == "few":
        E, h, d, k = c["E"], c["h"], c["d"], c["k"]
        x = c["x"].double()
        z = x @ c["wr"].double().t()
        z = torch.exp(z - z.amax(1, keepdim=True))
        p = z / z.sum(1, keepdim=True)
        top, chosen = torch.topk(p, k, dim=1)
        y = torch.zeros_like(x)
        for e in torch.unique(chosen).tolist():  # one expert after the other
            t, j = torch.nonzero(chosen == e, as_tuple=True)
            mats = []
            for n, rows, K in (("w1", h, d), ("w3", h, d), ("w2", d, h)):
                if c["wt"] == "e2m1":
                    sc = c[n + "s"].view(-1, E, rows, 4)[:, e].contiguous().view(-1)
                    mats.append(_e2m1_exact(c[n][e], sc, rows, K))
                else:
                    mats.append(c[n][e].double())
            a = x[t] @ mats[0].t()
            y[t] += top[t, j].unsqueeze(1) * ((a / (1 + torch.exp(-a)) * (x[t] @ mats[1].t())) @ mats[2].t())
        return {"y": y, "topk_idx": None, "topk_w": top}
    if op == "linear":
        return c["x"].double() @ _e2m1_exact(c["q"], c["s"], c["n"], c["K"]).t()
    # the nearest value of the format, ties to the even code
    b = c["w"].double().view(c["rows"], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    scale = torch.where(top > 0, torch.exp2(torch.frexp(top)[1].double() - 3), 2.0 ** -127)
    a = b.abs() / scale
    mag = 0.5 * ((a > 0.25).double() + (a >= 0.75).double() + (a > 1.25).double() + (a >= 1.75).double())
    mag = mag + (a > 2.5).double() + (a >= 3.5).double() + 2 * (a > 5).double()
    sb = torch.zeros(c["rows"], -(-c["cols"] // 128) * 4, dtype=torch.float64, device=b.device)
    sb[:, :c["cols"] // 32] = scale.view(c["rows"], -1)
    sb[:, c["cols"] // 32:] = 2.0 ** -127
    return {"w": (torch.sign(b) * mag * scale).view(c["rows"], -1), "s": sb.view(c["rows"], -1, 4).transpose(0, 1).reshape(-1)}
