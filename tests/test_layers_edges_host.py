"""Group norm and dropout without a GPU: the edges of the accepted sizes and
arguments."""

import ctypes
import os

import numpy
import pytest
import torch

from transposed_convolution_02_b200 import ct

CSRC = os.path.join(os.path.dirname(os.path.abspath(ct.__file__)), "csrc")


def workspace(dtype, n, s, c, groups):
    """(forward, backward) workspace bytes of a group norm."""
    d = ct.ct_group_norm_desc(dtype, 0, 0, 0, n, s, c, groups, 1e-5)
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert ct.lib().ct_group_norm_workspace_bytes(ctypes.byref(d), ctypes.byref(f), ctypes.byref(b)) == 0
    return f.value, b.value


@pytest.mark.parametrize("dtype", [ct.CT_F32, ct.CT_F16])
@pytest.mark.parametrize("n,c,groups", [(3, 8, 2), (700, 4099, 1), (1 << 21, (1 << 24) - 1, 1),
                                        (1 << 30, 1 << 24, 1 << 24)])
def test_no_pixels_need_no_workspace(dtype, n, c, groups):
    assert workspace(dtype, n, 0, c, groups) == (0, 0)


def test_cluster_barriers_have_their_warp_together():
    """The aligned forms of the cluster's barrier are undefined where a warp's
    lanes arrive apart, which no run shows: in the group norm's kernels, which
    meet it after branches by lane, each stands directly behind a warp barrier."""
    with open(os.path.join(CSRC, "group_norm_kernels.cuh")) as f:
        lines = [line.strip() for line in f]
    at = [i for i, line in enumerate(lines) if "barrier.cluster" in line]
    assert len(at) == 2 and all(lines[i - 1] == "__syncwarp();" for i in at)
    assert not any("cluster_sync" in line for line in lines)


@pytest.mark.parametrize("n,s,c,groups", [
    (1024, 1, 65537, 1), (1, 1, 1 << 20, 1), (1, 1, 1 << 24, 1 << 24), (1, 1, (1 << 24) - 1, 1),
    (1, 1, (1 << 24) - 1, (1 << 24) - 1), (1, 1, 100001, 1), (7, 3, 70007, 7), (64, 1, 1 << 20, 32),
    (3, 5, 4099, 1), (2, 64, 8200, 50), (1 << 10, 1, 1 << 24, 1 << 12)])
@pytest.mark.parametrize("dtype", [ct.CT_F32, ct.CT_F16, ct.CT_BF16])
def test_workspace_of_wide_pixels(dtype, n, s, c, groups):
    """The workspace is a small multiple of X, however many channels a pixel
    has: 16 bytes for a group and 8 for a group and a channel, at most twice
    (an image that starts inside a vector reaches into a second copy of the
    channels) and in every block of the GPU (the constant)."""
    x = n * s * c * (4 if dtype == ct.CT_F32 else 2)
    f, b = workspace(dtype, n, s, c, groups)
    assert f <= 16 * x + (1 << 20) and b <= 16 * x + (1 << 20)


FLAT = torch.zeros(400)
PIXELS, OUT = FLAT[:72].view(2, 3, 12), FLAT[100:172].view(2, 3, 12)
WORDS = FLAT[168:176].view(torch.int64)       # the first two lie in OUT, the last two behind it


@pytest.mark.parametrize("call,refusal", [
    (lambda: ct.group_norm_nhwc(PIXELS, 4, FLAT[100:112], out=OUT), "overlaps"),
    (lambda: ct.group_norm_nhwc(PIXELS, 4, FLAT[89:101], out=OUT), "overlaps"),
    (lambda: ct.group_norm_nhwc(PIXELS, 4, FLAT[200:212], FLAT[171:183], out=OUT), "overlaps"),
    (lambda: ct.group_norm_nhwc(PIXELS, 4, p=0.5, rng=WORDS[:2], out=OUT), "overlaps"),
    (lambda: ct.dropout(PIXELS, 0.5, rng=WORDS[:2], out=OUT), "overlaps"),
    (lambda: ct.dropout(PIXELS, 0.5, rng=FLAT[100:104].view(torch.int64), out=OUT), "overlaps"),
    (lambda: ct.dropout_backward(PIXELS, 0.5, rng=WORDS[1:3], out=OUT), "overlaps"),
    # beside it: refused for the device alone
    (lambda: ct.group_norm_nhwc(PIXELS, 4, FLAT[88:100], FLAT[172:184], p=0.5, rng=WORDS[2:], out=OUT), "CUDA"),
    (lambda: ct.dropout(PIXELS, 0.5, rng=WORDS[2:], out=OUT), "CUDA"),
    (lambda: ct.dropout(OUT, 0.5, rng=WORDS[2:], residual=PIXELS, out=OUT), "CUDA")])
def test_output_over_parameters(call, refusal):
    """Blocks still read the parameters and the random words while others
    write the output: it may not lie over them."""
    with pytest.raises(ValueError, match=refusal):
        call()


def test_tangents_are_refused():
    """Forward-mode tangents would be dropped silently, under no_grad too."""
    class OnCuda(torch.Tensor):
        is_cuda = True

    x, w = torch.zeros(3).as_subclass(OnCuda), torch.zeros(3)
    with torch.autograd.forward_ad.dual_level():
        ct._check_cuda(x, w, None)
        dual = torch.autograd.forward_ad.make_dual(w, torch.ones(3))
        for grad in (True, False):
            with torch.set_grad_enabled(grad):
                with pytest.raises(ValueError, match="tangent"):
                    ct._check_cuda(x, None, dual)
                with pytest.raises(ValueError, match="tangent"):
                    ct._check_cuda(dual.as_subclass(OnCuda), w)
    ct._check_cuda(x, w)


@pytest.mark.parametrize("groups", [2.5, 1.25, numpy.float64(2.5)])
def test_group_counts_are_whole_numbers(groups):
    """A fraction that divides the channels (20 by 2.5) is no number of groups."""
    x = torch.zeros(2, 3, 20)
    with pytest.raises(ValueError, match="groups"):
        ct._norm_of(x, groups, None, None, "silu", 1e-5)
    for whole in (4, 4.0, numpy.int64(4)):
        assert ct._norm_of(x, whole, None, None, "silu", 1e-5).stats == (2, 4)
