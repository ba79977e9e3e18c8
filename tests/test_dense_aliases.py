"""What the header lets two arguments share, no kernel promises the compiler to
be apart (host only: the promise is in the source, what it may break is not)."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "token_routing_grouped_amd", "csrc")


def _kernels(name):
    """(kernel, its parameters) of a source file."""
    text = open(os.path.join(CSRC, name)).read()
    return re.findall(r"__global__[^;{]*?\bvoid\s+(\w+)\s*\(([^{;]*)\)\s*\{", text)


def test_residual_and_result():
    """moe_linear_fwd: y may be res."""
    found = 0
    for kernel, params in _kernels("dense.hip"):
        names = {p.split()[-1].strip("*&"): p for p in params.split(",")}
        if "res" in names and "y" in names:
            found += 1
            assert "__restrict__" not in names["res"] and "__restrict__" not in names["y"], kernel
    assert found == 1


def test_gradient_and_orthogonalised_matrix():
    """moe_orthogonalize: out may be g.  Only the first two passes read g through
    a pointer of its own, and neither has the result."""
    kernels = dict(_kernels("muon.hip"))
    assert set(kernels) == {"sumsq_kernel", "scale_kernel"}
    for params in kernels.values():
        assert not re.search(r"\bout\b|\bUpdate\b", params)
