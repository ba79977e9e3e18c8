"""Refusals of the dense and weight-update calls, all on the host before
anything is enqueued (no GPU needed)."""

import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "token_routing_grouped_amd", "libtrg_moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")

P = [ctypes.c_void_p(1 << 20 | i << 12) for i in range(12)]
ODD = ctypes.c_void_p((1 << 20) + 8)
INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def _abi():
    from token_routing_grouped_amd import _abi

    return _abi


def _says(status, want, text):
    msg = _abi().lib().moe_last_error_string().decode()
    assert status == want and text in msg, (status, msg)


def test_linear_forward_refusals():
    f = _abi().lib().moe_linear_fwd
    names = ["x", "w", "bias", "res", "T", "n", "K", "act", "dt", "z", "y", "ws", "bytes", "stream"]
    ok = [P[0], P[1], None, None, 4, 64, 64, 0, 1, None, P[2], P[3], BIG, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)

    _says(call(dt=4), UNSUPPORTED, "dt must be")
    _says(call(T=-1), INVALID, "T must be")
    _says(call(n=0), INVALID, "n must be positive")
    _says(call(K=-8), INVALID, "K must be positive")
    _says(call(n=12), ALIGN, "n * element size")
    _says(call(K=62), ALIGN, "K * element size")
    _says(call(K=66, dt=0), ALIGN, "K * element size")
    _says(call(n=(1 << 20) + 8), UNSUPPORTED, "at most")
    _says(call(K=(1 << 20) + 8), UNSUPPORTED, "at most")
    _says(call(T=(1 << 31) - 1, n=1 << 20), UNSUPPORTED, "too large")
    for act in (-1, 4):
        _says(call(act=act), INVALID, "act must be")
    for p in ("x", "w", "y"):
        _says(call(**{p: None}), INVALID, f"{p} is null")
        _says(call(**{p: ODD}), ALIGN, f"{p} is not")
    for p in ("bias", "res", "z"):
        _says(call(**{p: ODD}), ALIGN, f"{p} is not")
    for p in (P[0], P[1]):
        _says(call(y=p), INVALID, "different buffers")
    _says(call(z=P[2]), INVALID, "different buffers")
    assert call(T=0, x=None, w=None, y=None, ws=None, bytes=0) == 0
    size = _abi().lib().moe_linear_workspace_size
    assert size(-1, 64, 64, 1) == 0 and size(4, 60, 64, 1) == 0 and size(4, 64, 64, 3) == 0 and size(0, 64, 64, 1) > 0
    need = size(128, 64, 8192, 1)  # few tiles, a long sum: in parts
    assert need > 16
    _says(call(T=128, K=8192, ws=None), WORKSPACE, "workspace needs")
    _says(call(T=128, K=8192, bytes=need - 17), WORKSPACE, "workspace needs")
    _says(call(T=128, K=8192, ws=ODD), ALIGN, "ws is not")


def test_linear_backward_refusals():
    f = _abi().lib().moe_linear_bwd
    names = ["dy", "x", "w", "z", "T", "n", "K", "act", "dt", "dx", "dw", "db", "ws", "bytes", "stream"]
    ok = [P[0], P[1], P[2], P[3], 4, 64, 64, 3, 1, P[4], P[5], P[6], P[7], BIG, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)

    _says(call(act=9), INVALID, "act must be")
    _says(call(dx=None, dw=None, db=None), INVALID, "nothing to write")
    _says(call(dy=None), INVALID, "dy is null")
    _says(call(w=None), INVALID, "w is null")
    _says(call(x=None), INVALID, "x is null")
    _says(call(z=None), INVALID, "z is null")
    for p in ("dx", "dw"):
        for q in (0, 1, 2, 3):
            _says(call(**{p: P[q]}), INVALID, f"{p} must be a buffer of its own")
    _says(call(dw=P[4]), INVALID, "dw must be a buffer of its own")
    for p, n in (("dx", "dx"), ("dw", "dw"), ("db", "dbias")):
        _says(call(**{p: ODD}), ALIGN, f"{n} is not")
    _says(call(ws=None), WORKSPACE, "workspace needs")
    _says(call(bytes=16), WORKSPACE, "workspace needs")
    _says(call(ws=ODD), ALIGN, "ws is not")


def _muon(**kw):
    abi = _abi()
    a = abi.MuonArgs(B=2, rows=8, cols=16, dt=1, steps=5, nesterov=1, eps=1e-7, momentum=0.9, step=0.1, decay=0.0)
    for i, n in enumerate(("w", "g", "buf", "w_out", "buf_out", "ws")):
        setattr(a, n, P[i].value)
    a.ws_bytes = BIG
    for k, v in kw.items():
        setattr(a, k, v.value if isinstance(v, ctypes.c_void_p) else v)
    return abi.lib().moe_muon_step(ctypes.byref(a), None)


def test_orthogonalize_refusals():
    lib = _abi().lib()
    names = ["g", "B", "rows", "cols", "dt", "steps", "eps", "out", "ws", "bytes", "stream"]
    ok = [P[0], 2, 8, 16, 1, 5, 1e-7, P[1], P[2], BIG, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[names.index(k)] = v
        return lib.moe_orthogonalize(*a)

    for f in (call, _muon):
        _says(f(dt=3), UNSUPPORTED, "dt must be")
        _says(f(B=-1), INVALID, "B must be")
        _says(f(rows=0), INVALID, "rows must be positive")
        _says(f(cols=0), INVALID, "cols must be positive")
        _says(f(cols=12), ALIGN, "cols * element size")
        _says(f(cols=6, dt=0), ALIGN, "cols * element size")
        _says(f(rows=(1 << 20) + 1), UNSUPPORTED, "at most")
        _says(f(cols=(1 << 20) + 8), UNSUPPORTED, "at most")
        for steps in (0, 33):
            _says(f(steps=steps), INVALID, "steps must be")
        for eps in (-1e-9, NAN, INF):
            _says(f(eps=eps), INVALID, "eps must be")
        _says(f(ws=None), WORKSPACE, "workspace needs")
        _says(f(ws=ODD), ALIGN, "ws is not")
        _says(f(g=None), INVALID, "g is null")
        _says(f(g=ODD), ALIGN, "g is not")
    _says(call(out=None), INVALID, "out is null")
    _says(call(bytes=1000), WORKSPACE, "workspace needs")
    assert call(B=0, g=None, out=None, ws=None) == 0
    size = lib.moe_orthogonalize_workspace_size
    assert size(2, 0, 16, 1) == 0 and size(2, 8, 10, 1) == 0
    assert size(1, 2048, 6144, 0) >= size(1, 2048, 6144, 1) > 0
    # many large matrices go through in chunks
    assert size(384, 2048, 6144, 1) < 3 << 30


def test_muon_refusals():
    for n in ("step", "decay", "momentum"):
        for v in (NAN, INF, -INF):
            _says(_muon(**{n: v}), INVALID, f"{n} must be finite")
    _says(_muon(master=P[8]), INVALID, "go together")
    _says(_muon(master_out=P[8]), INVALID, "go together")
    for n in ("w", "buf", "w_out", "buf_out"):
        _says(_muon(**{n: None}), INVALID, f"{n} is null")
        _says(_muon(**{n: ODD}), ALIGN, f"{n} is not")
    _says(_muon(lr_scale=ctypes.c_void_p(4098)), ALIGN, "lr_scale")
    for kw in (dict(w_out=P[1]), dict(w_out=P[2]), dict(buf_out=P[0]), dict(buf_out=P[3]), dict(buf_out=P[1]),
               dict(master=P[8], master_out=P[0]), dict(master=P[8], master_out=P[4]), dict(master=P[8], master_out=P[1])):
        _says(_muon(**kw), INVALID, "may be its own input")
    assert _abi().lib().moe_muon_step(None, None) == INVALID
    assert _muon(B=0, w=None, g=None) == 0


def test_binding_refusals():
    abi = _abi()
    bf = torch.bfloat16
    x, w, y, ws = torch.zeros(4, 64, dtype=bf), torch.zeros(48, 64, dtype=bf), torch.zeros(4, 48, dtype=bf), torch.zeros(16)
    with pytest.raises(abi.MoeError, match="expected the GPU"):
        abi.moe_linear_fwd(x, w, y, ws)
    with pytest.raises(abi.MoeError, match="w must have 64 columns"):
        abi.moe_linear_fwd(x, torch.zeros(48, 32, dtype=bf), y, ws)
    with pytest.raises(abi.MoeError, match="expected the GPU"):
        abi.moe_linear_bwd(y, x, w, ws)
    with pytest.raises(abi.MoeError, match="expected the GPU"):
        abi.moe_orthogonalize(w, w, ws)
    with pytest.raises(abi.MoeError, match="expected the GPU"):
        abi.moe_muon_step(w, w, w.float(), ws, step=0.1)
    with pytest.raises(abi.MoeError, match="must be a matrix"):
        abi.moe_orthogonalize(w[0], w[0], ws)
    with pytest.raises(abi.MoeError, match="act must be one of"):
        abi._act("tanh")
    with pytest.raises(abi.MoeError, match="unsupported dtype"):
        abi.moe_linear_workspace_size(4, 64, 64, torch.float16)
    with pytest.raises(abi.MoeError, match="16 bytes"):
        abi.moe_linear_workspace_size(4, 60, 64, bf)
    with pytest.raises(abi.MoeError, match="rows must be positive"):
        abi.moe_orthogonalize_workspace_size(2, 0, 64, bf)


def test_outputs_that_are_inputs():
    lib = _abi().lib()
    x, w, bias, res, z, y, ws = P[:7]

    def fwd(z, y, bias=bias, res=res):
        return lib.moe_linear_fwd(x, w, bias, res, 4, 64, 64, 2, 1, z, y, ws, BIG, None)

    _says(fwd(z, bias), INVALID, "an output is also an input")
    for p in (x, w, bias, res):
        _says(fwd(p, y), INVALID, "an output is also an input")
    _says(fwd(res, res), INVALID, "different buffers")
    dx, dw = P[7], P[8]
    for p in (x, w, z, y, dx, dw):
        _says(lib.moe_linear_bwd(y, x, w, z, 4, 64, 64, 2, 1, dx, dw, p, ws, BIG, None), INVALID, "dbias must be")
