"""MuonGPU refuses, before anything moves, whatever one of its weights' updates
would refuse after others have moved."""

import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "token_routing_grouped_amd", "libtrg_moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")


def _muon(*weights):
    from token_routing_grouped_amd.layer import MuonGPU

    return MuonGPU(weights)


def _error():
    from token_routing_grouped_amd import _abi

    return _abi.MoeError


def test_weights():
    """(Host tensors: they are looked at before any call.)"""
    a, b = torch.zeros(2, 16, 24), torch.zeros(64, 32)
    flat = torch.zeros(16 * 24 + 1)
    for bad, says in ((b.t(), "weight 1 must be contiguous"), (b[:, :16], "weight 1 must be contiguous"),
                      (flat[1:].view(16, 24), "16-byte aligned"), (torch.zeros(16, 24, device="meta"), "weight 1 is on meta"),
                      (a, "given twice"), (a[:1], "given twice"), (a[1:], "weights 0 and 1 overlap")):
        with pytest.raises(_error(), match=says):
            _muon(a, bad)
    with pytest.raises(_error(), match="weights 0 and 2 overlap"):
        _muon(b[8:24], a, b[:16])
    _muon(b[8:24], a, b[:8], b[24:], torch.zeros(0, 8, 8), torch.zeros(0, 8, 8))  # neighbours, and empty ones


def test_masters_hold_no_graph():
    w = torch.nn.Parameter(torch.ones(16, 32, dtype=torch.bfloat16))
    opt = _muon(w)
    assert not opt.masters[0].requires_grad and not opt.bufs[0].requires_grad


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_nothing_moves_when_the_second_gradient_is_refused(dt):
    dev = torch.device("cuda:0")
    one = lambda *s: torch.ones(*s, device=dev, dtype=dt)
    w = [one(2, 16, 24), one(16, 32)]
    opt = _muon(*w)
    state = [*opt.weights, *opt.bufs, *(m for m in opt.masters if m is not None)]
    before = [t.clone() for t in state]
    shifted = torch.ones(16 * 32 + 1, device=dev, dtype=dt)[1:].view(16, 32)
    own = [opt.weights[1]] + ([opt.bufs[1]] if dt == torch.float32 else [])
    for bad, says in [(shifted, "gradient 1 must be 16-byte aligned")] + [(t, "gradient 1 is a weight") for t in own]:
        with pytest.raises(_error(), match=says):
            opt.step([one(2, 16, 24), bad])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(state, before))
    opt.step([one(2, 16, 24), one(16, 32)])
    # (in bf16 a weight's own step may round to nothing)
    assert not any(torch.equal(p, q) for p, q in zip(state, before) if p.dtype == torch.float32)
