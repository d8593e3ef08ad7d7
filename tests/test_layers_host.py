"""Group norm and dropout without a GPU: the plain forms against published
values and differences, and the refusals of the C entries and the binding."""

import ctypes

import numpy as np
import pytest
import torch

import layers_ref as ref
from transposed_convolution_02_b200 import ct


def test_philox_known_answers():
    """The known-answer vectors published with the generator."""
    ones, zero = 0xFFFFFFFF, 0
    cases = [([zero] * 4, [zero] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
             ([ones] * 4, [ones] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
             ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
              [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])]
    for counter, key, want in cases:
        assert [int(v) for v in ref.philox([counter], key)[0]] == want


def test_keep_mask_rate_and_independence():
    n = 1 << 18
    for p in (0.0, 0.1, 0.5, 0.97, 1.0):
        m = ref.keep_mask(n, p, 11, 3)
        q = 1 - ref.threshold(p) / 65536
        # six standard deviations of a binomial count
        assert abs(m.sum() - n * q) <= 6 * np.sqrt(n * q * (1 - q))
    a, b, c = (ref.keep_mask(n, 0.5, s, o) for s, o in ((11, 3), (12, 3), (11, 4)))
    for u, v in ((a, b), (a, c)):
        assert abs((u == v).sum() - n / 2) <= 6 * np.sqrt(n) / 2
    assert np.array_equal(ref.keep_mask(100, 0.5, 11, 3, first=37), a[37:137])


@pytest.mark.parametrize("activation", ["identity", "relu", "silu", "gelu"])
def test_formulas_against_differences(activation):
    """The backward formulas against central differences of the forward, in fp64."""
    g = torch.Generator().manual_seed(5)
    n, s, c, groups = 2, 5, 6, 3
    x, dy = (torch.randn(n, s, c, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(c, generator=g, dtype=torch.float64) for _ in range(2))
    f = ref.factor((n, s, c), 0.3, 9, 1)

    def loss(x, w, b):
        return float((ref.forward(x, groups, w, b, 1e-3, activation, f)[0] * dy).sum())

    y, mean, rstd, a = ref.forward(x, groups, w, b, 1e-3, activation, f)
    assert float(a.abs().min()) > 1e-4          # clear of relu's jump
    grads = ref.backward(dy, x, mean, rstd, groups, w, b, activation, f)
    step = 1e-6
    for which, (t, gr) in enumerate(zip((x, w, b), grads)):
        for i in range(0, t.numel(), max(1, t.numel() // 12)):
            args = [x.clone(), w.clone(), b.clone()]
            args[which].view(-1)[i] += step
            hi = loss(*args)
            args[which].view(-1)[i] -= 2 * step
            lo = loss(*args)
            # rounding of the difference: 1e-16 * |loss| / step
            assert abs((hi - lo) / (2 * step) - float(gr.reshape(-1)[i])) < 1e-6


def _desc(**over):
    d = ct.ct_group_norm_desc(1, 0, 2, 0, 2, 9, 12, 4, 1e-5)
    for k, v in over.items():
        setattr(d, k, v)
    return d


def _ws_status(d):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    return ct.lib().ct_group_norm_workspace_bytes(ctypes.byref(d) if d is not None else None,
                                                  ctypes.byref(f), ctypes.byref(b))


@pytest.mark.parametrize("over, status", [
    ({}, 0), (dict(dtype=2), 0), (dict(param_dtype=1), 0), (dict(N=0), 0), (dict(S=0), 0),
    (dict(eps=0.0), 0), (dict(dtype=3), 3), (dict(dtype=-1), 3), (dict(param_dtype=2), 3),
    (dict(dtype=0, param_dtype=1), 3), (dict(activation=4), 4), (dict(activation=-1), 4),
    (dict(groups=5), 1), (dict(groups=0), 1), (dict(groups=-4), 1), (dict(C=0), 1), (dict(C=-4), 1),
    (dict(C=1 << 25, groups=1), 1), (dict(N=-1), 4), (dict(N=(1 << 30) + 1), 4), (dict(S=-1), 4),
    (dict(S=1 << 60), 4), (dict(N=1 << 30, S=1 << 30), 4), (dict(S=1 << 62), 4),
    (dict(eps=-1e-5), 4), (dict(eps=float("nan")), 4), (dict(eps=float("inf")), 4)])
def test_group_norm_desc_refusals(over, status):
    assert _ws_status(_desc(**over)) == status


def test_group_norm_null_and_workspace():
    assert _ws_status(None) == 6
    L = ct.lib()
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    big = _desc(S=1 << 20)         # long images: both directions need a workspace
    assert L.ct_group_norm_workspace_bytes(ctypes.byref(big), ctypes.byref(f), ctypes.byref(b)) == 0
    assert f.value > 0 and b.value > 0
    d = ctypes.byref(big)
    a = 1 << 20          # an aligned address that is never followed: every call is refused before a launch
    args = [d, a, a, a, 0.1, 1, 2, None, a, None, None, a, None]
    def fwd(**over):
        v = list(args)
        for k, x in over.items():
            v[int(k[1:])] = x
        return L.ct_group_norm(*v)
    assert fwd(_0=None) == 6
    assert fwd(_1=None) == 6 and fwd(_8=None) == 6
    assert fwd(_11=None) == 8
    assert fwd(_11=a + 16) == 5 and fwd(_1=a + 1) == 5 and fwd(_8=a + 1) == 5 and fwd(_2=a + 2) == 5
    assert fwd(_7=a + 4) == 5 and fwd(_9=a + 2) == 5
    for p in (-0.1, 1.1, float("nan"), float("inf")):
        assert fwd(_4=p) == 4
    back = [d, a, a, a, a, a, a, 0.1, 1, 2, None, a, a, a, a, None]
    def bwd(**over):
        v = list(back)
        for k, x in over.items():
            v[int(k[1:])] = x
        return L.ct_group_norm_backward(*v)
    for i in (0, 1, 2, 3, 4):
        assert bwd(**{"_%d" % i: None}) == 6
    assert bwd(_14=None) == 8
    assert bwd(_11=a + 1) == 5 and bwd(_12=a + 2) == 5 and bwd(_13=a + 2) == 5 and bwd(_3=a + 2) == 5
    assert bwd(_7=2.0) == 4
    assert bwd(_11=None, _12=None, _13=None) == 0     # nothing wanted
    if not torch.cuda.is_available():
        assert fwd() == 7 and bwd() == 7


def test_dropout_refusals():
    L = ct.lib()
    a = 1 << 20
    def drop(dtype=1, n=8, x=a, res=None, p=0.5, rng=None, y=a):
        return L.ct_dropout(dtype, n, x, res, p, 1, 2, rng, y, None)
    assert drop(dtype=3) == 3 and drop(dtype=-1) == 3
    assert drop(n=-1) == 4 and drop(n=(1 << 60) + 1) == 4
    assert drop(p=-0.1) == 4 and drop(p=1.5) == 4 and drop(p=float("nan")) == 4
    assert drop(x=None) == 6 and drop(y=None) == 6
    assert drop(x=a + 1) == 5 and drop(y=a + 1) == 5 and drop(res=a + 1) == 5 and drop(rng=a + 4) == 5
    assert drop(dtype=0, x=a + 2) == 5
    assert drop(n=0, x=None, y=None) == 0
    if not torch.cuda.is_available():
        assert drop() == 7


def test_new_types_and_activations_stay_out_of_conv_transpose():
    d = ct.make_desc([1, 4, 5], [4, 3, 3], dtype=torch.float16)
    d.dtype = ct.CT_BF16
    with pytest.raises(ct.CtError) as e:
        ct.ct_output_shape(d)
    assert e.value.status == 3
    for name in ("silu", "gelu"):
        with pytest.raises(ct.CtError) as e:
            ct.ct_output_shape(ct.make_desc([1, 4, 5], [4, 3, 3], dtype=torch.float16, activation=name))
        assert e.value.status == 4


X = torch.zeros(2, 3, 3, 12, dtype=torch.float16)
W = torch.zeros(12)


@pytest.mark.parametrize("call", [
    lambda: ct.group_norm_nhwc(X.double(), 4),
    lambda: ct.group_norm_nhwc(X[0, 0, 0], 4),
    lambda: ct.group_norm_nhwc(X, 5),
    lambda: ct.group_norm_nhwc(X, 0),
    lambda: ct.group_norm_nhwc(X, 4, activation="tanh"),
    lambda: ct.group_norm_nhwc(X, 4, W[:11], W),
    lambda: ct.group_norm_nhwc(X, 4, W.double(), W.double()),
    lambda: ct.group_norm_nhwc(X, 4, W.bfloat16(), W.bfloat16()),
    lambda: ct.group_norm_nhwc(X, 4, W.half(), W),
    lambda: ct.group_norm_nhwc(X, 4, W.to("meta"), W),
    lambda: ct.group_norm_nhwc(X, 4, p=1.5),
    lambda: ct.group_norm_nhwc(X, 4, p=float("nan")),
    lambda: ct.group_norm_nhwc(X, 4, p=0.5, seed=-1),
    lambda: ct.group_norm_nhwc(X, 4, p=0.5, offset=1 << 64),
    lambda: ct.group_norm_nhwc(X, 4, p=0.5, rng=torch.zeros(2)),
    lambda: ct.group_norm_nhwc(X, 4, p=0.5, rng=torch.zeros(3, dtype=torch.int64)),
    lambda: ct.group_norm_nhwc(X, 4, p=0.5, rng=torch.zeros(4, dtype=torch.int64)[::2]),
    lambda: ct.group_norm_nhwc(X, 4, out=X.float()),
    lambda: ct.group_norm_nhwc(X, 4, out=X[:1]),
    lambda: ct.group_norm_nhwc(X, 4, out=torch.zeros(2, 3, 12, 3, dtype=torch.float16).transpose(2, 3)),
    lambda: ct.group_norm_nhwc(X, 4, out=X),
    lambda: ct.group_norm_nhwc(X, 4),                         # not on a GPU
    lambda: ct.group_norm_nhwc_backward(X.float(), X, torch.zeros(2, 4), torch.zeros(2, 4), 4),
    lambda: ct.group_norm_nhwc_backward(X, X, torch.zeros(2, 3), torch.zeros(2, 4), 4),
    lambda: ct.group_norm_nhwc_backward(X, X, torch.zeros(2, 4), torch.zeros(2, 4).half(), 4),
    lambda: ct.group_norm_nhwc_backward(X, X, torch.zeros(2, 4), torch.zeros(2, 4), 4),
    lambda: ct.dropout(X.double(), 0.5),
    lambda: ct.dropout(X, -0.5),
    lambda: ct.dropout(X, 0.5, residual=X[:1]),
    lambda: ct.dropout(X, 0.5, residual=X.float()),
    lambda: ct.dropout(X[:, :2], 0.5, out=X[:, 1:]),
    lambda: ct.dropout(X, 0.5, out=X.transpose(1, 2)),
    lambda: ct.dropout(X, 0.5),
    lambda: ct.dropout_backward(X, 2.0),
])
def test_binding_refusals(call):
    with pytest.raises(ValueError):
        call()


def test_checks_of_overlap_and_gradients():
    flat = torch.zeros(100)
    ct.check_out(flat[:40], flat[:40], (flat[40:80],))
    ct.check_out(flat[:40], flat[:40], (flat[:40],), in_place=True)
    with pytest.raises(ValueError):
        ct.check_out(flat[:40], flat[:40], (flat[39:79],))
    with pytest.raises(ValueError):
        ct.check_out(flat[:40], flat[:40], (flat[1:41],), in_place=True)
    with pytest.raises(ValueError, match="CUDA"):
        ct._check_cuda(flat)

    class OnCuda:
        is_cuda, requires_grad = True, False

    leaf = torch.zeros(3, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        ct._check_cuda(OnCuda(), leaf)
    with torch.no_grad():
        ct._check_cuda(OnCuda(), leaf)


def test_descriptor_follows_sizes():
    a = ct._norm_of(torch.zeros(2, 3, 5, 8, dtype=torch.float16), 4, None, None, "silu", 1e-5)
    assert (a.desc.N, a.desc.S, a.desc.C, a.desc.groups) == (2, 15, 8, 4)
    assert (a.desc.dtype, a.desc.param_dtype, a.desc.activation) == (1, 0, 2)
    b = ct._norm_of(torch.zeros(2, 8, dtype=torch.bfloat16), 4, None, torch.zeros(8, dtype=torch.bfloat16),
                    "gelu", 0)
    assert (b.desc.S, b.desc.dtype, b.desc.param_dtype, b.desc.activation) == (1, 2, 2, 3)
    assert a.stats == (2, 4) and a.forward_bytes >= 0 and a.backward_bytes > 0


def test_checks_hold_on_sizes_seen_before():
    """The checks by size are made once; those of the parameters every time."""
    x, w = torch.zeros(2, 3, 24), torch.zeros(24)
    for _ in range(2):
        ct._norm_of(x, 4, w, w, "silu", 1e-5)
        for bad in (w[:23], w.half(), w.to("meta"), w.view(4, 6)):
            with pytest.raises(ValueError):
                ct._norm_of(x, 4, w, bad, "silu", 1e-5)
            with pytest.raises(ValueError):
                ct._norm_of(x, 4, bad, w, "silu", 1e-5)
        with pytest.raises(ValueError):
            ct._norm_of(x, 5, w, w, "silu", 1e-5)
        with pytest.raises(ct.CtError):
            ct._norm_of(x, 4, w, w, "silu", -1.0)
