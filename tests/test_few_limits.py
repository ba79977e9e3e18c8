"""Size limits of the norm and 4-bit calls at their last accepted and first
refused values, all on the host before anything is enqueued (no GPU needed)."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "token_routing_grouped_amd", "libtrg_moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")

C = ctypes.c_void_p(64)
INVALID, UNSUPPORTED = 1, 2


def _lib():
    from token_routing_grouped_amd import _abi

    return _abi.lib()


def _says(status, want, text):
    msg = _lib().moe_last_error_string().decode()
    assert status == want and text in msg, (status, msg)


@pytest.mark.parametrize("d,dt,last", [
    (8, 1, 2 ** 26 - 4), (2048, 1, 2 ** 26 - 4), (1024, 0, 2 ** 26 - 4),  # four rows a workgroup of 256 threads
    (2056, 1, 2 ** 24 - 1), (4096, 0, 2 ** 24 - 1),                      # a row a workgroup of 256
    (8200, 1, 2 ** 22 - 1), (16384, 0, 2 ** 22 - 1)])                    # and of 1024
def test_norm_rows_end_where_a_launch_has_2_32_threads(d, dt, last):
    """Workgroups are whole, so rows count in the fours that a workgroup takes.
    A size that is accepted is then refused for its missing input."""
    lib = _lib()

    def fwd(T):
        return lib.moe_rmsnorm_fwd(None, None, C, T, d, 1e-6, dt, None, C, None, None, None, None)

    def bwd(T):
        return lib.moe_rmsnorm_bwd(None, None, C, C, C, T, d, dt, C, C, C, 1 << 40, None)

    _says(fwd(last), INVALID, "x is null")
    _says(bwd(last), INVALID, "dy is null")
    for T in (last + 1, last + 2, last + 3, last + 4):
        _says(fwd(T), UNSUPPORTED, "too large")
        _says(bwd(T), UNSUPPORTED, "too large")


def test_e2m1_columns_end_where_rounding_up_to_a_chunk_passes_31_bits():
    """cols + 127 is taken in 32 bits.  (Accepted sizes are then refused for
    their missing buffers, or have no rows.)"""
    lib = _lib()
    last = 2 ** 31 - 128
    for rows in (1, 2, 3):
        _says(lib.mx_quantize_e2m1(C, 1, rows, last, None, C, None), INVALID, "q is null")
        _says(lib.mx_dequantize_e2m1(None, C, 0, rows, last, C, None), INVALID, "q is null")
    for cols in (last + 32, last + 64, last + 96):
        for rows in (0, 1, 2, 3):
            _says(lib.mx_quantize_e2m1(C, 1, rows, cols, None, C, None), UNSUPPORTED, "cols must be at most")
            _says(lib.mx_dequantize_e2m1(None, C, 0, rows, cols, C, None), UNSUPPORTED, "cols must be at most")


def test_norm_takes_every_finite_eps():
    lib = _lib()
    for eps in (0.0, 1e-45, 1e30, 2e30, 3.4028234e38):
        assert lib.moe_rmsnorm_fwd(None, None, None, 0, 64, eps, 1, None, None, None, None, None, None) == 0
    for eps in (-1e-45, float("inf"), float("nan")):
        _says(lib.moe_rmsnorm_fwd(None, None, None, 0, 64, eps, 1, None, None, None, None, None, None), INVALID, "eps")
