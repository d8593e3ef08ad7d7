"""Root-mean-square norm, rotary positions and AdamW without a GPU: calls that
the binding has to refuse, and settings that may not be kept by what they are."""

import ctypes

import pytest
import torch
from torch.autograd import forward_ad

from test_blocks_host import FLAT, HEADS, OUT, R, X, Card, adamw_status, card, rotary_desc
from transposed_convolution_02_b200 import ct


def test_parameters_that_change_where_they_lie():
    """Everything that the kernel relies on is looked at again: a parameter at its old address with other strides,
    another type or another number of elements, and lists that lost or gained one."""
    def made():
        p, q = card(4, 4), card(6, dtype=torch.float16)
        return p, q, ct.AdamW([p, q]), [card(4, 4), card(6, dtype=torch.float16)]

    p, q, opt, g = made()
    p.data = p.data.t()
    with pytest.raises(ValueError, match="parameter 0"):
        opt.step(g)
    p, q, opt, g = made()
    q.data = q.data.view(torch.bfloat16)
    with pytest.raises(ValueError, match="parameter 1"):
        opt.step(g)
    p, q, opt, g = made()
    p.data = p.data.view(torch.float16)[:, ::2]                    # 16 elements, 2 bytes each, at the same address
    with pytest.raises(ValueError, match="parameter 0"):
        opt.step(g)
    p, q, opt, g = made()
    with pytest.raises(ValueError, match="parameters"):
        opt.params.pop(0)
        opt.step(g[1:])
    p, q, opt, g = made()
    opt.params.append(card(3))
    with pytest.raises(ValueError, match="parameters"):
        opt.step(g + [card(3)])


def test_states_that_change_where_they_lie():
    opt = ct.AdamW([card(40)])
    kept = opt.exp_avg
    for other in (kept.view(torch.int32), kept.view(16, 16).t()):
        opt.exp_avg = other
        with pytest.raises(ValueError, match="exp_avg"):
            opt.step([card(40)])
    opt = ct.AdamW([card(40)], bits=8)
    opt.exp_avg_sq = opt.exp_avg_sq.view(torch.uint8)
    with pytest.raises(ValueError, match="exp_avg_sq"):
        opt.step([card(40)])


def needs(t):
    return t.clone().as_subclass(Card).requires_grad_()


@pytest.mark.parametrize("call", [
    lambda: ct.rms_norm_nhwc(X.as_subclass(Card), out=needs(OUT)),
    lambda: ct.rms_norm_nhwc(X.as_subclass(Card), residual=R, sum_out=needs(OUT)),
    lambda: ct.rms_norm_nhwc_e4m3(X.as_subclass(Card), residual=R, sum_out=needs(OUT)),
    lambda: ct.rotary_nhwc(HEADS.as_subclass(Card), [4, 8], out=needs(HEADS)),
    lambda: ct.rotary_nhwc_backward(HEADS.as_subclass(Card), [4, 8], out=needs(HEADS)),
    lambda: ct.dropout(X.as_subclass(Card), 0.5, out=needs(OUT)),
    lambda: ct.group_norm_nhwc(X.as_subclass(Card), 3, out=needs(OUT))])
def test_outputs_that_require_a_gradient(call):
    """They are refused as inputs are; under no_grad they are taken (and refused further on, for want of a device)."""
    with pytest.raises(ValueError, match="gradient"):
        call()
    with torch.no_grad(), pytest.raises(Exception) as e:
        call()
    assert "gradient" not in str(e.value)


@pytest.mark.parametrize("call", [
    lambda: ct.grad_norm([card(3), needs(FLAT[:3])]),
    lambda: ct.grad_norm([needs(FLAT[:3]) * 2]),
    lambda: ct.AdamW([card(3)]).step([needs(FLAT[:3])]),
    lambda: ct.AdamW([card(3), card(2)]).step([needs(FLAT[:3]) * 2, None])])
def test_gradients_that_would_be_dropped(call):
    """Gradients that carry a graph are refused as inputs are."""
    with pytest.raises(ValueError, match="gradient"):
        call()


def test_tangents_that_would_be_dropped():
    for call in (lambda g: ct.grad_norm([card(3), g]), lambda g: ct.AdamW([card(2), card(3)]).step([None, g]),
                 lambda g: ct.AdamW([card(3)]).step([g])):
        with forward_ad.dual_level(), torch.no_grad():
            g = forward_ad.make_dual(torch.zeros(3), torch.ones(3)).as_subclass(Card)
            with pytest.raises(ValueError, match="tangent"):
                call(g)


def test_numbers_are_kept_by_value():
    """Settings given as tensors that then change: descriptors are those of the present value."""
    eps = torch.tensor(1e-6)
    assert ct._rms_of(X, None, 0, eps).desc.eps == pytest.approx(1e-6)
    eps.fill_(1e-3)
    assert ct._rms_of(X, None, 0, eps).desc.eps == pytest.approx(1e-3)
    assert ct._norm_of(X, 3, None, None, "relu", eps).desc.eps == pytest.approx(1e-3)
    eps.fill_(1e-2)
    assert ct._norm_of(X, 3, None, None, "relu", eps).desc.eps == pytest.approx(1e-2)

    ct._ROTARY.clear()
    for base, sections in ((torch.tensor(100.0), [4, 8]), (100.0, [torch.tensor(4), 8]), (100.0, [4, 8])):
        with pytest.raises(ValueError, match="CUDA"):
            ct.rotary_nhwc(HEADS, sections, base=base)
    assert [r.desc.base for r in ct._ROTARY.values()] == [100.0]
    assert not any(isinstance(v, torch.Tensor) for key in ct._ROTARY for v in key + key[3])


@pytest.mark.parametrize("base, status", [(1e-300, 0), (1e-40, 0), (5e-324, 4), (1e-310, 0), (1e-315, 4)])
def test_frequencies_past_64_bits(base, status):
    """They are refused; all others are taken (nothing is launched for no images).  The last of 256 pairs has
    base^(-255 / 256) / 2 pi: 9.8e307 for 1e-310."""
    d = rotary_desc(base=base, sections=[0, 512, 0], dim=512, N=0)
    assert ct.lib().ct_rotary(ctypes.byref(d), None, None, None, None) == status


@pytest.mark.parametrize("over", [dict(lr=1e39), dict(eps=1e39), dict(rows=((10, 0, 0, 1e39),))])
def test_settings_that_fp32_does_not_hold(over):
    """They would become infinite on the way to the kernel."""
    assert adamw_status(**over) == 4
