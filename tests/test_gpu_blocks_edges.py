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
