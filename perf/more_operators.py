"""The dense products beside the expert layer and the update of its weights, in
their plain form (elementary torch operations in 32 bits) and as calls of the
framework's own kernels, over the sizes they are used at.

  linear      a matrix product with bias, activation and residual:
              z = x W^T + b, y = act(z) + res
  linear_bwd  its gradients: dz = dy act'(z), dx = dz W, dW = dz^T x, db = sum dz
  ortho       a batch of matrices (the experts' gradients), each orthogonalised
              by Newton-Schulz products: X <- a X + (b A + c A^2) X, A = X X^T
  muon        a weight update with it: momentum, orthogonalised, weights moved

A case is a dict of plain values.  `own` chooses between the plain form and the
framework's calls; prepare() makes the same inputs for both.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "silu")
#: The quintic of the orthogonalisation and its number of steps.
A, B, C = 3.4445, -4.7750, 2.0315
STEPS = 5
EPS = 1e-7
MOMENTUM = 0.95
DECAY, STEP = 3e-5, 0.002


def listed():
    return [
        # one token of a decode step through a projection beside the experts
        {"name": "linear_one", "op": "linear", "T": 1, "n": 6144, "K": 2048, "dt": "bf16", "act": "silu", "bias": True,
         "res": False, "keep": False},
        # an odd decode batch through a wide projection back onto the residual stream
        {"name": "linear_61_wide", "op": "linear", "T": 61, "n": 2048, "K": 6144, "dt": "bf16", "act": "none",
         "bias": True, "res": True, "keep": False},
        # a training step's tokens, what the activation had kept for its gradient
        {"name": "linear_step", "op": "linear", "T": 16384, "n": 6144, "K": 2048, "dt": "bf16", "act": "gelu",
         "bias": True, "res": False, "keep": True},
        # a ragged micro-batch of an fp32 model
        {"name": "linear_ragged_f32", "op": "linear", "T": 1021, "n": 1000, "K": 2048, "dt": "f32", "act": "silu",
         "bias": True, "res": True, "keep": True},
        # a short odd sequence's gradients: few output tiles, and a short sum for the weights
        {"name": "linear_bwd_short", "op": "linear_bwd", "T": 253, "n": 2048, "K": 2048, "dt": "bf16", "act": "silu"},
        # the training step's gradients
        {"name": "linear_bwd_step", "op": "linear_bwd", "T": 16384, "n": 6144, "K": 2048, "dt": "bf16", "act": "gelu"},
        # the ragged micro-batch's
        {"name": "linear_bwd_ragged_f32", "op": "linear_bwd", "T": 1021, "n": 1000, "K": 2048, "dt": "f32",
         "act": "relu"},
        # all experts of the smallest layer, tall matrices
        {"name": "ortho_tiny_f32", "op": "ortho", "B": 8, "rows": 256, "cols": 128, "dt": "f32"},
        # one up projection of the 8-expert layer
        {"name": "ortho_experts", "op": "ortho", "B": 8, "rows": 1024, "cols": 2048, "dt": "bf16"},
        # one wide matrix by itself, in fp32
        {"name": "ortho_one_wide_f32", "op": "ortho", "B": 1, "rows": 2048, "cols": 6144, "dt": "f32"},
        # the update of a small layer's down projection
        {"name": "muon_tiny", "op": "muon", "B": 8, "rows": 128, "cols": 256, "dt": "bf16", "master": False},
        # the update of all 128 experts' down projections, fp32 master weights
        {"name": "muon_wide", "op": "muon", "B": 128, "rows": 2048, "cols": 1024, "dt": "bf16", "master": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step - 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "ortho", "muon"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    while True:
        if op in ("linear", "linear_bwd"):
            T, n, K = _log(rng, 1, 16384), _log(rng, 64, 8192, 8), _log(rng, 64, 8192, 8)
            if T * n * K > 16384 * 6144 * 2048 // (4 if dt == "f32" else 1):
                continue
            c = {"op": op, "T": T, "n": n, "K": K, "dt": dt, "act": rng.choice(ACTS)}
            if op == "linear":
                c.update(bias=rng.random() < 0.7, res=rng.random() < 0.5, keep=rng.random() < 0.5)
            return c
        b, rows, cols = _log(rng, 1, 128), _log(rng, 16, 4096), _log(rng, 16, 6144, 8)
        c = {"op": op, "B": b, "rows": rows, "cols": cols, "dt": dt}
        if op == "muon":
            c["master"] = dt == "bf16" and rng.random() < 0.5
        if b * rows * cols <= 1 << 25 and work(c)["flops"] * (4 if dt == "f32" else 1) <= 4e12:
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, *shape, std=1.0, dt=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dt).mul_(std)


def _gradient(g, b, rows, cols, dt):
    """A weight gradient as a step gives it: a few strong directions over noise."""
    v = _normal(g, b, rows, cols, std=1e-4, dt=torch.float32)
    p, q = _normal(g, b, rows, 8, dt=torch.float32), _normal(g, b, 8, cols, std=3e-5, dt=torch.float32)
    return v.add_(torch.bmm(p, q)).to(dt)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    dt, op = TYPES[c["dt"]], c["op"]
    if op in ("linear", "linear_bwd"):
        T, n, K = c["T"], c["n"], c["K"]
        c.update(x=_normal(g, T, K, dt=dt), w=_normal(g, n, K, std=0.02, dt=dt))
        if op == "linear":
            c["b"] = _normal(g, n, std=0.1, dt=dt) if c["bias"] else None
            c["r"] = _normal(g, T, n, std=2.0, dt=dt) if c["res"] else None
        else:
            c["dy"] = _normal(g, T, n, dt=dt)
            c["z"] = _normal(g, T, n, dt=dt) if c["act"] != "none" else None
        return c
    b, rows, cols = c["B"], c["rows"], c["cols"]
    c["g"] = _gradient(g, b, rows, cols, dt)
    if op == "muon":
        c["buf"] = _gradient(g, b, rows, cols, torch.float32).mul_(10.0)
        w = _normal(g, b, rows, cols, std=0.02, dt=torch.float32)
        c["w"] = w.to(dt)
        c["w32"] = w if c["master"] else None
    return c


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(c):
    return (_OWN if own else _PLAIN)[c["op"]](c)


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _linear(c):
    dt = c["x"].dtype
    z = c["x"].float() @ c["w"].float().t()
    if c["b"] is not None:
        z = z + c["b"].float()
    y = _act(z, c["act"])
    if c["r"] is not None:
        y = y + c["r"].float()
    out = {"y": y.to(dt)}
    if c["keep"]:
        out["z"] = z.to(dt)
    return out


def _linear_bwd(c):
    dt = c["x"].dtype
    dz = c["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(c["z"].float(), c["act"])
    return {"dx": (dz @ c["w"].float()).to(dt), "dw": (dz.t() @ c["x"].float()).to(dt), "dbias": dz.sum(0).to(dt)}


def _newton_schulz(u):
    """Orthogonalised matrices of u [B, rows, cols], fp32 in and out."""
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2).contiguous() if tall else u
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        gram = torch.bmm(x, x.transpose(1, 2))
        x = A * x + torch.bmm(B * gram + C * torch.bmm(gram, gram), x)
    return x.transpose(1, 2) if tall else x


def _ortho(c):
    return _newton_schulz(c["g"].float()).to(c["g"].dtype).contiguous()


def _muon(c):
    buf = MOMENTUM * c["buf"] + c["g"].float()
    o = _newton_schulz(c["g"].float() + MOMENTUM * buf)
    w = (c["w32"] if c["master"] else c["w"].float()) * (1.0 - DECAY) - STEP * o
    out = {"w": w.to(c["w"].dtype), "buf": buf}
    if c["master"]:
        out["master"] = w
    return out


_PLAIN = {"linear": _linear, "linear_bwd": _linear_bwd, "ortho": _ortho, "muon": _muon}


def _own_linear(c):
    from token_routing_grouped_amd import _abi

    x, w = c["x"], c["w"]
    T, n, K = c["T"], c["n"], c["K"]
    if "out" not in c:  # a program's own buffers, kept from step to step
        c["ws"] = _abi.workspace(_abi.moe_linear_workspace_size(T, n, K, x.dtype), DEV)
        o = c["out"] = {"y": torch.empty(T, n, dtype=x.dtype, device=DEV)}
        if c["keep"]:
            o["z"] = torch.empty_like(o["y"])
    o = c["out"]
    _abi.moe_linear_fwd(x, w, o["y"], c["ws"], bias=c["b"], res=c["r"], act=c["act"], z=o.get("z"))
    return o


def _own_linear_bwd(c):
    from token_routing_grouped_amd import _abi

    x, w = c["x"], c["w"]
    T, n, K = c["T"], c["n"], c["K"]
    if "out" not in c:
        c["ws"] = _abi.workspace(_abi.moe_linear_bwd_workspace_size(T, n, K, x.dtype), DEV)
        c["out"] = {"dx": torch.empty_like(x), "dw": torch.empty_like(w), "dbias": torch.empty_like(w[:, 0])}
    o = c["out"]
    _abi.moe_linear_bwd(c["dy"], x, w, c["ws"], act=c["act"], z=c["z"], dx=o["dx"], dw=o["dw"], dbias=o["dbias"])
    return o


def _own_ortho(c):
    from token_routing_grouped_amd import _abi

    g = c["g"]
    if "out" not in c:
        c["ws"] = _abi.workspace(_abi.moe_orthogonalize_workspace_size(*g.shape, g.dtype), DEV)
        c["out"] = torch.empty_like(g)
    _abi.moe_orthogonalize(g, c["out"], c["ws"], steps=STEPS, eps=EPS)
    return c["out"]


def _own_muon(c):
    from token_routing_grouped_amd import _abi

    w = c["w"]
    if "out" not in c:
        c["ws"] = _abi.workspace(_abi.moe_orthogonalize_workspace_size(*w.shape, w.dtype), DEV)
        c["out"] = {"w": torch.empty_like(w), "buf": torch.empty_like(c["buf"])}
        if c["master"]:
            c["out"]["master"] = torch.empty_like(c["w32"])
    o = c["out"]
    _abi.moe_muon_step(w, c["g"], c["buf"], c["ws"], step=STEP, decay=DECAY, momentum=MOMENTUM, nesterov=True,
                       steps=STEPS, eps=EPS, master=c["w32"], w_out=o["w"], buf_out=o["buf"],
                       master_out=o.get("master"))
    return o


_OWN = {"linear": _own_linear, "linear_bwd": _own_linear_bwd, "ortho": _own_ortho, "muon": _own_muon}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c, op = case, case["op"]
    es = 4 if c["dt"] == "f32" else 2
    if op in ("linear", "linear_bwd"):
        T, n, K = c["T"], c["n"], c["K"]
        if op == "linear":
            b = es * (T * K + n * K + T * n * (1 + c["res"] + c["keep"]) + n * c["bias"])
            return {"bytes": b, "flops": 2 * T * n * K}
        b = es * (2 * (T * K + n * K) + T * n * (1 if c["act"] == "none" else 2) + n)
        return {"bytes": b, "flops": 4 * T * n * K}
    v = c["B"] * c["rows"] * c["cols"]
    m, n = min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
    # the two symmetric products count half
    f = c["B"] * STEPS * (m * m * n + m * m * m + 2 * m * m * n)
    if op == "ortho":
        return {"bytes": 2 * es * v, "flops": f}
    return {"bytes": v * (3 * es + 8 + (8 - es if c["master"] else 0)), "flops": f}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_ortho(u):
    """The same polynomial of u's singular values by products of m x m matrices
    alone: with G = X X^T, a step multiplies X by P = a + b G + c G^2 from the
    left and turns G into P G P, so the steps' P multiply to the map of the
    first X."""
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2).contiguous() if tall else u
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + EPS)
    gram = torch.bmm(x, x.transpose(1, 2).contiguous())
    total = None
    for _ in range(STEPS):
        p = B * gram + C * torch.bmm(gram, gram)
        p.diagonal(dim1=1, dim2=2).add_(A)
        total = p if total is None else torch.bmm(p, total)
        gram = torch.bmm(torch.bmm(p, gram), p)
    x = torch.bmm(total, x)
    return x.transpose(1, 2).contiguous() if tall else x


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op in ("linear", "linear_bwd"):
        x, w, act = c["x"].double(), c["w"].double(), c["act"]
        half_erfc = lambda v: 0.5 * torch.special.erfc(-v / math.sqrt(2.0))  # the normal distribution function
        if op == "linear":
            z = torch.mm(x, w.t().contiguous())
            z = z if c["b"] is None else z + c["b"].double().unsqueeze(0)
            y = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, torch.zeros_like(z)),
                 "gelu": lambda: z * half_erfc(z), "silu": lambda: z * torch.special.expit(z)}[act]()
            y = y if c["r"] is None else y + c["r"].double()
            return {"y": y, "z": z} if c["keep"] else {"y": y}
        dz = c["dy"].double()
        if act != "none":
            z = c["z"].double()
            p = torch.special.expit(z)
            dz = dz * {"relu": lambda: torch.where(z > 0, 1.0, 0.0).double(),
                       "gelu": lambda: half_erfc(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi),
                       "silu": lambda: p + z * p * torch.special.expit(-z)}[act]()
        return {"dx": torch.mm(dz, w), "dw": torch.mm(dz.t().contiguous(), x), "dbias": dz.sum(0)}
    if op == "ortho":
        return _exact_ortho(c["g"].double())
    g = c["g"].double()
    buf = c["buf"].double() * MOMENTUM + g
    u = g + buf * MOMENTUM
    base = c["w32"] if c["master"] else c["w"]
    w = base.double() - DECAY * base.double() - STEP * _exact_ortho(u)
    return {"w": w, "buf": buf, "master": w} if c["master"] else {"w": w, "buf": buf}
