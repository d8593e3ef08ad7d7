"""Group norm and dropout on the GPU: the edges of the accepted sizes and
arguments, against fp64."""

import pytest
import torch

import layers_ref as ref
from test_gpu_layers import EPS, TYPES, both_ways
from transposed_convolution_02_b200 import ct

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    major, _ = torch.cuda.get_device_capability()
    assert major == 10, "these kernels are built for sm_100a"


def raw_stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("n,c,groups", [(3, 8, 2), (5, 30, 3), (2, 4099, 1)])
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_no_pixels_without_statistics(dtype, n, c, groups):
    """Images of no pixels through the C entries: no statistics are read or
    needed, the parameters' gradients are 0."""
    x = torch.empty(n, 0, c, dtype=TYPES[dtype], device="cuda")
    norm = ct._norm_of(x, groups, None, None, "silu", EPS)
    dw, db = (torch.full((c,), 7.25, device="cuda") for _ in range(2))
    for p in (0.0, 0.5):
        assert ct.lib().ct_group_norm_backward(norm.desc, None, None, None, None, None, None, p, 1, 2, None, None,
                                               dw.data_ptr(), db.data_ptr(), None, raw_stream()) == 0
        torch.cuda.synchronize()
        assert not dw.any() and not db.any()
        dw.fill_(7.25), db.fill_(7.25)
        mean, rstd = (torch.full((n, groups), 7.25, device="cuda") for _ in range(2))
        assert ct.lib().ct_group_norm(norm.desc, None, None, None, p, 1, 2, None, None, mean.data_ptr(),
                                      rstd.data_ptr(), None, raw_stream()) == 0
        assert ct.lib().ct_group_norm(norm.desc, None, None, None, p, 1, 2, None, None, None, None, None,
                                      raw_stream()) == 0
        torch.cuda.synchronize()
        assert not mean.any()
        # a square root, a quotient and eps itself rounded: half a step each, the root of eps' halved
        assert bool(((rstd.double() * EPS ** 0.5 - 1).abs() <= 3 * 2.0 ** -24).all())


def test_any_number_of_images_of_no_pixels():
    """The number of empty images is bounded by no memory: no kernel may walk
    them one by one."""
    x = torch.empty(1 << 30, 0, 1 << 24, dtype=torch.float16, device="cuda")
    assert ct.group_norm_nhwc(x, 1, activation="silu").shape == x.shape
    x = torch.empty(1 << 24, 0, 1 << 22, dtype=torch.float16, device="cuda")
    y, mean, rstd = ct.group_norm_nhwc(x, 2, return_stats=True)
    w = torch.ones(1 << 22, device="cuda")
    dx, dw, db = ct.group_norm_nhwc_backward(x, x, mean, rstd, 2, w, w)
    torch.cuda.synchronize()
    assert dx.shape == x.shape and not dw.any() and not db.any() and not mean.any()


WIDE = [
    ([40, 1, 65537], 1), ([9, 1, 4099], 4099), ([3, 2, 100001], 11), ([5, 3, 70004], 2), ([9, 5, 2570], 10),
    ([2, 9, 4112], 257), ([3, 7, 2052], 1026), ([1, 1, 1 << 20], 1 << 20), ([6, 2, 16388], 17), ([17, 1, 2058], 3),
    ([1, 1, (1 << 24) - 1], 1), ([1, 2, 1 << 22], 1 << 10), ([2, 500, 4101], 3), ([1, 900, 2316], 193),
]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("i", range(len(WIDE)))
def test_wide_pixels(i, dtype):
    """Pixels of more channels than one column tile takes: few and many
    groups, tiles that start and end inside groups, images that start inside a
    vector, fewer pixels than copies of the channels along a row."""
    shape, groups = WIDE[i]
    both_ways(shape, groups, TYPES[dtype], ["silu", "identity", "gelu"][(i + len(dtype)) % 3], [0.0, 0.3][i % 2],
              seed=2000 + 10 * i, affine=i % 4 != 3)


@pytest.mark.parametrize("dtype,shape,groups", [
    ("fp32", [2, 3000, 2116], 23), ("fp32", [1, 5000, 2068], 47), ("fp16", [2, 4000, 4416], 23),
    ("bf16", [3, 2500, 4098], 6), ("fp32", [2, 2001, 2565], 27)])
def test_tiles_that_share_a_group_agree(dtype, shape, groups):
    """A group whose channels lie in two column tiles is joined by the blocks
    of both. Where all of its channels are alike, so are the outputs, to the
    bit: the tiles' statistics and means may differ in no bit, or what mean
    and rstd hold depends on which block is last."""
    n, s, c = shape
    g = torch.Generator(device="cuda").manual_seed(c)
    for _ in range(4):
        x, dy = (torch.randn(n, s, groups, 1, generator=g, device="cuda").expand(n, s, groups, c // groups)
                 .reshape(shape).to(TYPES[dtype]) for _ in range(2))
        x = x * 3 + 1
        y, mean, rstd = ct.group_norm_nhwc(x, groups, activation="silu", return_stats=True)
        dx, _, _ = ct.group_norm_nhwc_backward(dy, x, mean, rstd, groups, activation="silu")
        for t in (y, dx):
            t = t.view(n, s, groups, -1)
            assert torch.equal(t, t[..., :1].expand(t.shape))
        for _ in range(3):
            again = ct.group_norm_nhwc(x, groups, activation="silu", return_stats=True)
            assert all(torch.equal(a, b) for a, b in zip(again, (y, mean, rstd)))


def test_inputs_whose_derivatives_would_be_lost():
    """No call records a derivative: inputs that carry one are refused, the
    statistics of the backward call as well."""
    x, w, b = torch.randn(2, 9, 8, device="cuda"), torch.ones(8, device="cuda"), torch.zeros(8, device="cuda")
    _, mean, rstd = ct.group_norm_nhwc(x, 2, w, b, return_stats=True)
    with torch.autograd.forward_ad.dual_level(), torch.no_grad():
        def dual(t):
            return torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))
        for call in (lambda: ct.group_norm_nhwc(dual(x), 2, w, b), lambda: ct.group_norm_nhwc(x, 2, dual(w), b),
                     lambda: ct.group_norm_nhwc(x, 2, w, dual(b)), lambda: ct.dropout(dual(x), 0.5),
                     lambda: ct.dropout(x, 0.5, residual=dual(x)), lambda: ct.dropout_backward(dual(x), 0.5),
                     lambda: ct.group_norm_nhwc_backward(dual(x), x, mean, rstd, 2, w, b),
                     lambda: ct.group_norm_nhwc_backward(x, x, dual(mean), rstd, 2, w, b),
                     lambda: ct.group_norm_nhwc_backward(x, x, mean, dual(rstd), 2, w, b)):
            with pytest.raises(ValueError, match="tangent"):
                call()
    for call in (lambda m: ct.group_norm_nhwc_backward(x, x, m, rstd, 2, w, b),
                 lambda m: ct.group_norm_nhwc_backward(x, x, mean, m, 2, w, b)):
        leaf = rstd.clone().requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            call(leaf)
        with torch.no_grad():
            call(leaf)


# pixels of an image of s that lie far from the others: the first one, a column
# at the image's border, a band at its top
FAR_PIXELS = {"first": lambda s: slice(0, 1), "column": lambda s: slice(0, s, 256), "band": lambda s: slice(0, s // 290)}


@pytest.mark.parametrize("far", [0.0, 20.0, 100.0, 1e4])
@pytest.mark.parametrize("where", sorted(FAR_PIXELS))
@pytest.mark.parametrize("dtype,shape,groups", [
    ("fp16", [300, 60000, 8], 4), ("bf16", [160, 60000, 8], 2), ("fp32", [300, 30000, 8], 4),
    ("fp32", [1, 2000000, 8], 4), ("fp32", [300, 30000, 7], 1), ("fp16", [2, 300001, 24], 3),
    ("fp32", [8, 16384, 128], 32)])
def test_far_pixels_in_long_images(dtype, shape, groups, where, far):
    """Pixels far from all others, those among them that sums and joins are
    shifted by: the statistics keep the bound that they have without them,
    however many pixels follow."""
    n, s, c = shape
    x = torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(s), device="cuda")
    if far:
        at = FAR_PIXELS[where](s)
        x[:, at] = far
        x[::3, at, c // 2:] = -far
    x = x.to(TYPES[dtype])
    y, mean, rstd = ct.group_norm_nhwc(x, groups, eps=EPS, return_stats=True)
    g = x.view(n, s, groups, -1).double()
    m = g.mean(dim=(1, 3))
    d = g - m[:, None, :, None]
    r = 1 / torch.sqrt((d * d).mean(dim=(1, 3)) + EPS)
    spread = d.abs().mean(dim=(1, 3))
    assert bool(((mean - m).abs() <= ref.U * (ref.CHAIN * 2 * spread + 4 * m.abs())).all())
    assert float((rstd / r - 1).abs().max()) <= ref.U * (ref.CHAIN + 8)
    del d, g
    # y from the fp64 statistics, pixels of the image's start, middle and end
    for at in (0, s // 2, s - 100):
        h = (x[:, at: at + 100].double().view(n, 100, groups, -1) - m[:, None, :, None]) * r[:, None, :, None]
        e = (6 + ref.CHAIN / 2) * h.abs() + ref.CHAIN * 2 + 4 * (m.abs() * r)[:, None, :, None]
        off = (y[:, at: at + 100].double().view(h.shape) - h).abs()
        assert bool((off <= 1.01 * (ref.HALF[TYPES[dtype]] * h.abs() + ref.U * e) + ref.TINY[TYPES[dtype]]).all())


@pytest.mark.parametrize("c,rows,groups", [(8, 128, 4), (7, 36 * 4, 1), (64, 16, 8)])
def test_threads_that_sum_a_thousand_vectors(c, rows, groups, monkeypatch):
    """As many images as fill the GPU, each the work of one block, so long that
    a thread adds 1000 vectors (`rows` pixels of a block at a time): forward and
    backward against fp64. The longest chain of additions is a thread's 1024, a
    column's 256 and 64 for lanes, parts and images."""
    monkeypatch.setattr(ref, "CHAIN", 1024 + 256 + 64)
    n, s = 300, 1000 * rows - 3
    gen = torch.Generator(device="cuda").manual_seed(c)
    x, dy = (torch.randn(n, s, c, generator=gen, device="cuda") for _ in range(2))
    w, b = (torch.randn(c, generator=gen, device="cuda") for _ in range(2))
    y, mean, rstd = ct.group_norm_nhwc(x, groups, w, b, eps=EPS, activation="silu", return_stats=True)
    dx, dw, db = ct.group_norm_nhwc_backward(dy, x, mean, rstd, groups, w, b, activation="silu")
    w64, b64, one = w.double(), b.double(), torch.ones(1, dtype=torch.float64, device="cuda")
    sums = [torch.zeros(c, dtype=torch.float64, device="cuda") for _ in range(4)]
    part = 30                                   # images at a time
    for i in range(0, n, part):
        v, g = x[i: i + part].double(), dy[i: i + part].double()
        want, m, r, a = ref.forward(v, groups, w64, b64, EPS, "silu")
        spread = (v - ref._spread(m, v, groups)).abs().view(part, s, groups, -1).mean(dim=(1, 3))
        assert bool(((mean[i: i + part] - m).abs() <= ref.U * (ref.CHAIN * 2 * spread + 4 * m.abs())).all())
        assert bool(((rstd[i: i + part] / r - 1).abs() <= ref.U * (ref.CHAIN + 8)).all())
        bound = ref.forward_bound(v, m, r, groups, w64, b64, a, want, torch.float32, 1.0)
        assert bool(((y[i: i + part] - want).abs() <= bound).all())
        del want, a, bound
        # the gradients with the statistics as they are
        m, r = mean[i: i + part].double(), rstd[i: i + part].double()
        want = ref.backward(g, v, m, r, groups, w64, b64, "silu")
        bounds = ref.backward_bounds(g, v, m, r, groups, w64, b64, "silu", one, torch.float32, torch.float32, *want)
        assert bool(((dx[i: i + part] - want[0]).abs() <= bounds[0]).all())
        for j in (1, 2):
            sums[j - 1] += want[j]
            sums[j + 1] += bounds[j]            # the roundings of the parts bound that of their sum
    assert bool(((dw - sums[0]).abs() <= sums[2]).all()) and bool(((db - sums[1]).abs() <= sums[3]).all())
