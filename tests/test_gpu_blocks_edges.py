"""Root-mean-square norm, rotary positions and AdamW on the GPU where their
contracts end: numbers at the borders of fp32, skipped updates, outputs on
inputs, rows past 32 bits in the kernels of whole rows."""

import math

import pytest
import torch

import blocks_ref as ref
from test_gpu_adamw import everything, make, same
from test_gpu_rms_norm import EPS, TYPES, _cuda, check_backward, check_codes, check_forward, inputs, normal  # noqa: F401
from transposed_convolution_02_b200 import ct

pytestmark = pytest.mark.gpu


# ---- AdamW -----------------------------------------------------------------------

@pytest.mark.parametrize("bits", [32, 8])
def test_device_steps_and_rates_that_skip(bits):
    """A step below 1 (a counter that the graph counts up only behind the update) and a rate that is no rate leave
    every bit as it was."""
    params, grads = make(130)
    lr, step = torch.tensor([1e-2], device="cuda"), torch.ones(1, dtype=torch.int64, device="cuda")
    opt = ct.AdamW(params, lr=lr, bits=bits)
    opt.step(grads, step=step)
    kept = everything(opt)
    for t in (0, -1, -(1 << 63)):
        step.fill_(t)
        opt.step(grads, step=step)
        assert same(everything(opt), kept), t
    step.fill_(2)
    for bad in (-1e-3, float("nan"), float("inf"), -float("inf")):
        lr.fill_(bad)
        opt.step(grads, step=step)
        assert same(everything(opt), kept), bad
    lr.fill_(1e-2)
    opt.step(grads, step=step)
    assert not same(everything(opt), kept)
    assert all(bool(p.isfinite().all()) for p in params)


# ---- rotary positions ---------------------------------------------------------------

@pytest.mark.parametrize("base", [1e-36, 1e-38, 1e-40, 1e-100, 1e-300])
def test_frequencies_that_fp32_does_not_hold(base):
    """Position 0 turns nothing whatever the frequency; others stay turns."""
    x = normal([2, 3, 2, 132], 3)
    for kind in (None, torch.int32, torch.int64, torch.float32):
        at = None if kind is None else torch.tensor([[0], [0], [2]], dtype=kind, device="cuda")
        for pairs in ("adjacent", "halves"):
            y = ct.rotary_nhwc(x, [128], base=base, pairs=pairs, positions=at)
            still = 1 if kind is None else 2
            assert torch.equal(y[:, :still], x[:, :still])
            assert bool(y.isfinite().all())
            # a turn keeps lengths: c and s are good to 1.5 u each (2.2 u of a pair's length), two products and a
            # sum of each side lose 2 u, twice that of the squares
            assert torch.allclose((y.double() ** 2).sum(-1), (x.double() ** 2).sum(-1), rtol=16 * ref.U, atol=0)
            # the first pair turns by its position, 2
            i, k = (0, 1) if pairs == "adjacent" else (0, 64)
            v, w = x[:, 2, :, i].double(), x[:, 2, :, k].double()
            want = v * math.cos(2.0) - w * math.sin(2.0)
            assert bool(((y[:, 2, :, i].double() - want).abs() <= 5 * ref.U * (v.abs() + w.abs())).all())
