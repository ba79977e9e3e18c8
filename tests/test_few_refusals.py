"""Refusals of the norm, 4-bit and few-token calls, all on the host before
anything is enqueued (no GPU needed)."""

import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "token_routing_grouped_amd", "libtrg_moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")

C = ctypes.c_void_p(64)
INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4


def _lib():
    from token_routing_grouped_amd import _abi

    return _abi.lib()


def _says(status, want, text):
    lib = _lib()
    msg = lib.moe_last_error_string().decode()
    assert status == want and text in msg, (status, msg)


def test_norm_refusals():
    f = _lib().moe_rmsnorm_fwd
    #      x  res  w  T  d   eps  dt s  y  q  qs rstd stream
    ok = [C, None, C, 4, 64, 1e-6, 1, None, C, None, None, None, None]

    def call(**kw):
        names = ["x", "res", "w", "T", "d", "eps", "dt", "s", "y", "q", "qs", "rstd", "stream"]
        a = list(ok)
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)

    odd = ctypes.c_void_p(72)
    _says(call(dt=4), UNSUPPORTED, "dt must be")
    _says(call(T=-1), INVALID, "T must be")
    _says(call(d=0), INVALID, "d must be positive")
    _says(call(d=12), ALIGN, "multiple of 16 bytes")
    _says(call(d=65544), UNSUPPORTED, "128 KiB")
    _says(call(d=32772, dt=0), UNSUPPORTED, "128 KiB")
    for eps in (-1e-9, float("nan"), float("inf")):
        _says(call(eps=eps), INVALID, "eps")
    _says(call(q=C), INVALID, "go together")
    _says(call(y=None), INVALID, "nothing to write")
    _says(call(d=72, q=C, qs=C), INVALID, "d % 32")
    _says(call(x=None), INVALID, "x is null")
    _says(call(res=odd), ALIGN, "res is not")
    _says(call(s=odd), ALIGN, "s is not")
    _says(call(y=odd), ALIGN, "y is not")
    _says(call(q=C, qs=ctypes.c_void_p(66)), ALIGN, "qs and rstd")
    _says(call(rstd=ctypes.c_void_p(66)), ALIGN, "qs and rstd")
    _says(call(s=C), INVALID, "different buffers")
    assert call(T=0, x=None, w=None) == 0
    g = _lib().moe_rmsnorm_bwd
    #      dy  ds    s  w  rstd T  d  dt dx dw ws bytes stream
    _says(g(C, None, C, C, C, 4, 64, 1, C, C, C, 0, None), WORKSPACE, "workspace needs")
    big = 1 << 30
    _says(g(C, None, C, C, None, 4, 64, 1, C, C, C, big, None), INVALID, "rstd is null")
    _says(g(C, odd, C, C, C, 4, 64, 1, C, C, C, big, None), ALIGN, "ds is not")
    _says(g(C, None, C, C, C, 4, 64, 1, C, None, C, big, None), INVALID, "dw is null")
    _says(g(C, None, C, C, C, 4, 64, 1, C, C, odd, big, None), ALIGN, "ws is not")
    size = _lib().moe_rmsnorm_bwd_workspace_size
    assert size(-1, 64) == 0 and size(4, 0) == 0 and size(0, 64) == 64 * 4 and size(1 << 20, 64) == 512 * 64 * 4


def test_e2m1_refusals():
    lib = _lib()
    _says(lib.mx_quantize_e2m1(C, 2, 4, 64, C, C, None), UNSUPPORTED, "dt must be")
    _says(lib.mx_quantize_e2m1(C, 1, -1, 64, C, C, None), INVALID, "rows")
    _says(lib.mx_quantize_e2m1(C, 1, 4, 48, C, C, None), INVALID, "multiple of 32")
    _says(lib.mx_quantize_e2m1(C, 1, 1 << 26, 32, C, C, None), UNSUPPORTED, "too large")
    _says(lib.mx_dequantize_e2m1(C, C, 0, 1 << 20, 8192, C, None), UNSUPPORTED, "too large")
    _says(lib.mx_quantize_e2m1(C, 1, 4, 64, None, C, None), INVALID, "q is null")
    _says(lib.mx_quantize_e2m1(C, 1, 4, 64, C, None, None), INVALID, "s is null")
    _says(lib.mx_quantize_e2m1(C, 1, 4, 64, ctypes.c_void_p(72), C, None), ALIGN, "q is not")
    _says(lib.mx_quantize_e2m1(C, 1, 4, 64, C, ctypes.c_void_p(66), None), ALIGN, "s is not")
    _says(lib.mx_dequantize_e2m1(C, C, 1, 4, 64, None, None), INVALID, "out is null")
    assert lib.mx_quantize_e2m1(None, 1, 0, 64, None, None, None) == 0
    assert lib.mx_dequantize_e2m1(None, None, 1, 0, 64, None, None) == 0
    _says(lib.mx_linear_e2m1(C, C, C, 65, 4, 64, C, None), INVALID, "T must be")
    _says(lib.mx_linear_e2m1(C, C, C, -1, 4, 64, C, None), INVALID, "T must be")
    _says(lib.mx_linear_e2m1(C, C, C, 4, 0, 64, C, None), INVALID, "n must be")
    _says(lib.mx_linear_e2m1(C, C, C, 4, 4, 40, C, None), INVALID, "multiple of 32")
    _says(lib.mx_linear_e2m1(C, C, C, 4, 4, 65568, C, None), UNSUPPORTED, "K must be")
    _says(lib.mx_linear_e2m1(C, C, C, 4, 65536, 65536, C, None), UNSUPPORTED, "2 GiB")
    _says(lib.mx_linear_e2m1(None, C, C, 4, 4, 64, C, None), INVALID, "x is null")
    assert lib.mx_linear_e2m1(None, C, C, 0, 4, 64, None, None) == 0


def _few(**kw):
    from token_routing_grouped_amd import _abi

    a = dict(T=4, d=64, E=8, k=2, h=64, dt=1, wt=1, x=64, wr=64, w1=64, w3=64, w2=64, y=64, ws=64, ws_bytes=1 << 30)
    a.update(kw)
    return _lib().moe_few_fwd(ctypes.byref(_abi.FewArgs(**a)), None)


def test_few_refusals():
    _says(_lib().moe_few_fwd(None, None), INVALID, "args is null")
    _says(_few(dt=2), UNSUPPORTED, "dt must be")
    for T in (-1, 65):
        _says(_few(T=T), INVALID, "T must be")
    for E in (0, 1025):
        _says(_few(E=E), INVALID, "E must be")
    for k in (0, 33):
        _says(_few(k=k, E=64), INVALID, "k must be")
    _says(_few(k=9), INVALID, "k (9) > E (8)")
    _says(_few(d=0), INVALID, "must be positive")
    _says(_few(h=65544), UNSUPPORTED, "at most")
    _says(_few(d=68), ALIGN, "multiple of 16 bytes")
    _says(_few(h=4), ALIGN, "multiple of 16 bytes")
    _says(_few(wt=0), UNSUPPORTED, "wt must be")
    _says(_few(wt=3), UNSUPPORTED, "wt must be")
    _says(_few(wt=4, dt=0), UNSUPPORTED, "need dt MOE_BF16")
    _says(_few(wt=4, d=72), INVALID, "% 32")
    _says(_few(wt=4, h=72), INVALID, "% 32")
    _says(_few(d=65536, h=16384), UNSUPPORTED, "2 GiB")
    _says(_few(dt=0, wt=0, d=32768, h=16384), UNSUPPORTED, "2 GiB")
    _says(_few(wt=4, E=1024, d=65536, h=32768), UNSUPPORTED, "too large")
    _says(_few(wt=4), INVALID, "w1s is null")
    _says(_few(wt=4, w1s=64, w3s=66, w2s=64), ALIGN, "w3s is not")
    for n in ("x", "wr", "w1", "w3", "w2", "y"):
        _says(_few(**{n: None}), INVALID, f"{n} is null")
        _says(_few(**{n: 72}), ALIGN, f"{n} is not")
    _says(_few(topk_idx=72), ALIGN, "topk_idx is not")
    _says(_few(n_live=66), ALIGN, "n_live is not")
    _says(_few(ws=None), WORKSPACE, "workspace needs")
    _says(_few(ws_bytes=16), WORKSPACE, "workspace needs")
    _says(_few(ws=72), ALIGN, "ws is not")
    assert _few(T=0, x=None, y=None, ws=None, ws_bytes=0) == 0
    size = _lib().moe_few_workspace_size
    assert size(65, 64, 8, 2, 64) == 0 and size(4, 64, 1, 2, 64) == 0 and size(4, 64, 8, 2, 64) > 0


def test_few_arg_struct_matches_the_header(tmp_path):
    from token_routing_grouped_amd import _abi

    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe.h"', "int main(void) {",
             'printf("%zu %d\\n", sizeof(moe_few_args), MOE_E2M1);']
    lines += [f'printf("%zu\\n", offsetof(moe_few_args, {f}));' for f, _ in _abi.FewArgs._fields_]
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out[:2]] == [ctypes.sizeof(_abi.FewArgs), _abi.MOE_E2M1]
    assert [int(v) for v in out[2:]] == [getattr(_abi.FewArgs, f).offset for f, _ in _abi.FewArgs._fields_]


def test_host_tensors_and_wrong_shapes_are_refused():
    from token_routing_grouped_amd import _abi

    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(64, dtype=bf)
    with pytest.raises(_abi.MoeError, match="x: tensor on cpu"):
        _abi.moe_rmsnorm_fwd(x, w, 1e-6, x.clone())
    with pytest.raises(_abi.MoeError, match="must be a matrix"):
        _abi.moe_rmsnorm_fwd(w, w, 1e-6, w)
    with pytest.raises(_abi.MoeError, match="tensor on cpu"):
        _abi.mx_quantize_e2m1(x, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(_abi.MoeError, match="must have 4 rows"):
        _abi.mx_linear_e2m1(x, w, w, torch.zeros(3, 8, dtype=bf))
    with pytest.raises(_abi.MoeError, match="w1 must be"):
        _abi.few_args(2, torch.zeros(8, 64, dtype=bf), x, x, x, w)


def test_norms_refuse_more_rows_than_a_launch_has_threads_for():
    """64 threads a row up to 4 KiB, 256 up to 16 KiB, 1024 above: 2^32 in all."""
    lib = _lib()
    for T, d, dt in ((1 << 26, 8, 1), (1 << 26, 1024, 0), (1 << 24, 2056, 1), (1 << 22, 16384, 1),
                     (2 ** 31 - 1, 64, 1)):
        _says(lib.moe_rmsnorm_fwd(C, None, C, T, d, 1e-6, dt, None, C, None, None, None, None), UNSUPPORTED,
              "too large")
        _says(lib.moe_rmsnorm_bwd(C, None, C, C, C, T, d, dt, C, C, C, 1 << 40, None), UNSUPPORTED, "too large")


def test_decode_layer_of_no_tokens_is_refused():
    from token_routing_grouped_amd import _abi
    from token_routing_grouped_amd.layer import MoEDecodeGPU

    w = torch.zeros(4, 64, 64)
    for T in (0, -3):
        with pytest.raises(_abi.MoeError, match="at least 1"):
            MoEDecodeGPU(T, 2, torch.zeros(4, 64), w, w, w)
    with pytest.raises(_abi.MoeError, match="T must be"):
        MoEDecodeGPU(65, 2, torch.zeros(4, 64), w, w, w)
