"""Group norm and dropout on the GPU against their plain fp64 forms."""

import math

import pytest
import torch

import layers_ref as ref
from transposed_convolution_02_b200 import ct
from transposed_convolution_02_b200.workloads import draw

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    major, _ = torch.cuda.get_device_capability()
    assert major == 10, "these kernels are built for sm_100a"


def inputs(shape, dtype, seed, pdtype=torch.float32, shift=2.0):
    c = shape[-1]
    x = draw(shape, ("normal", 1.0), seed, torch.float32)
    x = x * (0.5 + draw([c], ("normal", 1.0), seed + 1, torch.float32).abs())
    x = (x + shift * draw([c], ("normal", 1.0), seed + 2, torch.float32)).to(dtype)
    w = (1 + 0.3 * draw([c], ("normal", 1.0), seed + 3, torch.float32)).to(pdtype)
    b = draw([c], ("normal", 0.3), seed + 4, pdtype)
    dy = draw(shape, ("normal", 1.0), seed + 5, dtype)
    return x, w, b, dy


def check(got, want, bound, where):
    got = got.double().cpu()
    assert got.shape == want.shape, where
    err = (got - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its bound" % (
        where, int(bad.sum()), bad.numel(), float((err / bound).nan_to_num(float("inf")).max()))


def both_ways(shape, groups, dtype, activation="identity", p=0.0, seed=100, pdtype=torch.float32, affine=True,
              shift=2.0, data=None, rng=False):
    """Forward and backward, compared as a whole; relu's backward away from its jump only."""
    x, w, b, dy = inputs(shape, dtype, seed, pdtype, shift) if data is None else data
    s, o = (1 << 40) + seed, (3 << 33) + 7
    xd, dyd = x.cuda(), dy.cuda()
    wd, bd = (w.cuda(), b.cuda()) if affine else (None, None)
    how = dict(activation=activation, p=p)
    how.update({"rng": torch.tensor([s, o], device="cuda")} if rng else {"seed": s, "offset": o})
    y, mean, rstd = ct.group_norm_nhwc(xd, groups, wd, bd, eps=EPS, return_stats=True, **how)
    dx, dw, db = ct.group_norm_nhwc_backward(dyd, xd, mean, rstd, groups, wd, bd, **how)
    torch.cuda.synchronize()
    w64 = w.double() if affine else torch.ones(shape[-1], dtype=torch.float64)
    b64 = b.double() if affine else torch.zeros(shape[-1], dtype=torch.float64)
    x64 = x.double()
    f = ref.factor(shape, p, s, o) if p else torch.ones(shape, dtype=torch.float64)
    scale = ref.drop_scale(p)
    where = "%s %s %s p=%g " % (shape, dtype, activation, p)
    yr, mr, rr, a = ref.forward(x64, groups, w64, b64, EPS, activation, f)
    spread = ((x64 - ref._spread(mr, x64, groups)).abs()).reshape(shape[0], -1, groups, shape[-1] // groups)
    check(mean, mr, ref.U * (ref.CHAIN * 2 * spread.mean(dim=(1, 3)) + 4 * mr.abs()) + 1e-38, where + "mean")
    # var's sum has CHAIN u of itself, the mean's error enters squared; sqrt halves it
    check(rstd, rr, ref.U * (ref.CHAIN + 8) * rr, where + "rstd")
    check(y, yr, ref.forward_bound(x64, mr, rr, groups, w64, b64, a, yr, dtype, scale), where + "y")
    if p:
        assert bool((y.cpu()[f == 0] == 0).all()), where + "dropped elements are 0"
    m64, r64 = mean.double().cpu(), rstd.double().cpu()
    want = ref.backward(dy.double(), x64, m64, r64, groups, w64, b64, activation, f)
    bounds = ref.backward_bounds(dy.double(), x64, m64, r64, groups, w64, b64, activation, f, dtype, pdtype, *want)
    check(dx, want[0], bounds[0], where + "dx")
    if affine:
        check(dw, want[1], bounds[1], where + "dweight")
        check(db, want[2], bounds[2], where + "dbias")
    else:
        assert dw is None and db is None
    return y, mean, rstd, dx, dw, db


SHAPES = [
    ([1, 1], 1), ([1, 8], 8), ([2, 1, 1, 32], 32), ([3, 5], 1), ([3, 1, 1000], 1),   # one pixel
    ([1, 2, 3], 3), ([5, 9, 7], 7), ([4, 2, 3, 4, 24], 3), ([3, 7, 5, 30], 5),      # small and odd
    ([2, 13, 17, 65], 13), ([7, 11, 3, 9], 1), ([9, 5, 12], 4), ([33, 3, 20], 5),
    ([2, 40, 515], 5), ([2, 33, 2056], 8), ([1, 5, 4099], 1), ([2, 3, 2050], 41),   # rows wider than a block
    ([1, 4099, 16], 2), ([1, 50000, 8], 4), ([1, 20011, 3], 3),                     # one long image
    ([2, 64, 64, 128], 32), ([16, 8, 8, 512], 32), ([1, 8, 8, 256], 32), ([3, 100, 1024], 16),
    ([16, 35, 2], 2), ([5, 33, 3], 3), ([4, 13, 5], 1), ([3, 77, 1], 1), ([40, 9, 3], 1), ([3, 41, 6], 2),   # below a vector
    ([70, 4, 16], 4), ([2, 57, 91, 30], 5), ([1, 31, 2048], 2048), ([6, 300, 96], 96),
    ([2, 40, 4096], 32), ([1, 3000, 4096], 16), ([2, 700, 4104], 27), ([2, 5, 8192], 8192),  # column tiles of whole groups
    ([700, 33, 64], 8), ([70000, 1, 8], 2), ([5, 20000, 56], 7), ([1, 30001, 70], 14),       # many images, long ones
]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_group_norm(i, dtype):
    shape, groups = SHAPES[i]
    act = ["silu", "gelu", "identity"][(i + len(dtype)) % 3]
    p = [0.0, 0.25, 0.0, 0.6][i % 4]
    t = TYPES[dtype]
    both_ways(shape, groups, t, act, p, seed=1000 + 10 * i, pdtype=[torch.float32, t][i % 2],
              affine=i % 5 != 3, rng=i % 3 == 1)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("activation", ["identity", "relu", "silu", "gelu"])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_activations(dtype, activation, p):
    shape, groups = [3, 6, 10, 24], 4
    x, w, b, dy = inputs(shape, TYPES[dtype], 77)
    if activation == "relu":   # dy is 0 where a is near relu's jump, where the side it falls on is rounding
        a = ref.forward(x.double(), groups, w.double(), b.double(), EPS, "identity")[3]
        dy = torch.where(a.abs() < 1e-3, torch.zeros_like(dy), dy)
    both_ways(shape, groups, TYPES[dtype], activation, p, data=(x, w, b, dy))


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_far_mean(dtype):
    """Means many deviations from 0: the statistics stay those of the values
    given (a sum of squares would lose them all)."""
    both_ways([2, 37, 40], 5, TYPES[dtype], "silu", shift=300.0 if dtype == "fp32" else 30.0, seed=55)
    g = torch.Generator().manual_seed(3)
    x = (1000.0 + torch.randn(2, 500, 32, generator=g)).to(TYPES[dtype])
    _, w, b, dy = inputs([2, 500, 32], TYPES[dtype], 56)
    both_ways([2, 500, 32], 8, TYPES[dtype], "identity", data=(x, w, b, dy))


def test_constant_and_one_far_value():
    """A constant group has variance 0; one value far from all others, first
    in its thread or not, leaves the variance exact to its bound."""
    shape, groups = [2, 300, 16], 4
    _, w, b, dy = inputs(shape, torch.float32, 91)
    for at in (0, 1, 299):
        x = torch.full(shape, 3.0)
        x[:, at, 5] = 1e4
        x[1, :, 8:] = 0.0
        y, mean, rstd, *_ = both_ways(shape, groups, torch.float32, "identity", data=(x, w, b, dy))
        assert abs(float(rstd[1, 3]) - EPS ** -0.5) <= 8 * ref.U * EPS ** -0.5
        assert torch.equal(y[1, :, 12:].cpu(), b[12:].expand(300, 4))


def test_not_finite_stays_in_its_group():
    shape, groups = [2, 50, 24], 3
    x, w, b, dy = inputs(shape, torch.float16, 15)
    clean = ct.group_norm_nhwc(x.cuda(), groups, w.cuda(), b.cuda(), activation="silu")
    x2 = x.clone()
    x2[0, 7, 9], x2[1, 49, 23] = float("inf"), float("nan")
    y, mean, rstd = ct.group_norm_nhwc(x2.cuda(), groups, w.cuda(), b.cuda(), activation="silu",
                                       return_stats=True)
    dx, _, _ = ct.group_norm_nhwc_backward(dy.cuda(), x2.cuda(), mean, rstd, groups, w.cuda(), b.cuda(),
                                           activation="silu")
    for t in (y, dx):
        assert bool(t[0, :, 8:16].isnan().any()) and bool(t[1, :, 16:].isnan().all())
        ok = t.clone()
        ok[0, :, 8:16] = 0
        ok[1, :, 16:] = 0
        assert bool(ok.isfinite().all())
    assert math.isnan(float(rstd[0, 1])) and math.isnan(float(rstd[1, 2])) and int(rstd.isnan().sum()) == 2
    assert torch.equal(y[0, :, :8], clean[0, :, :8]) and torch.equal(y[1, :, :16], clean[1, :, :16])


def test_overflow_rounds_to_infinity():
    x = torch.tensor([[[60000.0], [-60000.0]]], dtype=torch.float16).cuda()
    big = torch.full((1,), 60000.0, dtype=torch.float16).cuda()
    y = ct.group_norm_nhwc(x, 1, big, big)
    assert y.flatten().tolist() == [math.inf, 0.0]
    d = ct.dropout(torch.full((64,), 60000.0, dtype=torch.float16, device="cuda"), 0.5, seed=1)
    assert set(d.tolist()) == {math.inf, 0.0}


def test_empty():
    x = torch.empty(0, 4, 8, dtype=torch.float16, device="cuda")
    w = torch.ones(8, device="cuda")
    y, mean, rstd = ct.group_norm_nhwc(x, 2, w, w, return_stats=True)
    assert y.shape == (0, 4, 8) and mean.shape == (0, 2)
    dx, dw, db = ct.group_norm_nhwc_backward(x, x, mean, rstd, 2, w, w)
    assert dx.shape == x.shape and not dw.any() and not db.any() and dw.shape == (8,)
    x = torch.empty(3, 0, 8, dtype=torch.float16, device="cuda")
    y, mean, rstd = ct.group_norm_nhwc(x, 2, w, w, return_stats=True)
    assert y.shape == (3, 0, 8) and not mean.any()
    dx, dw, db = ct.group_norm_nhwc_backward(x, x, mean, rstd, 2, w, w)
    assert dx.shape == x.shape and not dw.any() and not db.any()
    assert ct.dropout(x, 0.5).shape == x.shape


def guarded(shape, dtype, offset):
    """A tensor `offset` elements into a buffer of a marker value, and the buffer."""
    n = math.prod(shape)
    buf = torch.full((n + 64,), 7.25, dtype=dtype, device="cuda")
    return buf[offset: offset + n].view(shape), buf


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("shape,groups", [([3, 7, 5, 30], 5), ([2, 9, 16], 4), ([5, 3, 3], 1)])
@pytest.mark.parametrize("xo,yo", [(1, 1), (0, 3), (5, 0), (8, 16)])
def test_alignment_and_neighbours(dtype, shape, groups, xo, yo):
    """Tensors at any element offset give the same bits, and nothing around the outputs is written."""
    t = TYPES[dtype]
    x, w, b, dy = inputs(shape, t, 300)
    how = dict(activation="silu", p=0.3, seed=5, offset=6)
    want = ct.group_norm_nhwc(x.cuda(), groups, w.cuda(), b.cuda(), **how)
    xd, _ = guarded(shape, t, xo)
    xd.copy_(x)
    yd, buf = guarded(shape, t, yo)
    wb = torch.zeros(2 * shape[-1] + 2, device="cuda")
    wd, bd = wb[1: 1 + shape[-1]], wb[1 + shape[-1]: 1 + 2 * shape[-1]]
    wd.copy_(w)
    bd.copy_(b)
    got, mean, rstd = ct.group_norm_nhwc(xd, groups, wd, bd, out=yd, return_stats=True, **how)
    assert got is yd and torch.equal(got, want)
    n = math.prod(shape)
    assert bool((buf[:yo] == 7.25).all()) and bool((buf[yo + n:] == 7.25).all())
    dyd, _ = guarded(shape, t, yo)
    dyd.copy_(dy)
    a = ct.group_norm_nhwc_backward(dy.cuda(), x.cuda(), mean, rstd, groups, w.cuda(), b.cuda(), **how)
    c = ct.group_norm_nhwc_backward(dyd, xd, mean, rstd, groups, wd, bd, **how)
    assert all(torch.equal(u, v) for u, v in zip(a, c))
    # dropout, at the same offsets
    want = ct.dropout(x.cuda(), 0.4, seed=8, offset=9, residual=dy.cuda())
    yd, buf = guarded(shape, t, yo)
    got = ct.dropout(xd, 0.4, seed=8, offset=9, residual=dyd, out=yd)
    assert torch.equal(got, want)
    assert bool((buf[:yo] == 7.25).all()) and bool((buf[yo + n:] == 7.25).all())


def test_backward_does_not_write_around_dx():
    """The C entry with every output in a guarded buffer."""
    shape, groups, t = [3, 11, 10], 5, torch.float16
    x, w, b, dy = (v.cuda() for v in inputs(shape, t, 310))
    _, mean, rstd = ct.group_norm_nhwc(x, groups, w, b, return_stats=True)
    want = ct.group_norm_nhwc_backward(dy, x, mean, rstd, groups, w, b)
    norm = ct._norm_of(x, groups, w, b, "identity", 0.0)
    desc, nb = norm.desc, norm.backward_bytes
    ws = torch.full((nb + 256,), 0xFF, dtype=torch.uint8, device="cuda")   # a workspace of NaNs
    for off in (0, 3):
        dx, xbuf = guarded(shape, t, off)
        dw, wbuf = guarded([10], torch.float32, off)
        db, bbuf = guarded([10], torch.float32, off)
        st = ct.lib().ct_group_norm_backward(desc, dy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                             w.data_ptr(), b.data_ptr(), 0.0, 0, 0, None, dx.data_ptr(),
                                             dw.data_ptr(), db.data_ptr(), ws.data_ptr(),
                                             torch.cuda.current_stream().cuda_stream)
        assert st == 0
        for got, buf, ref_ in ((dx, xbuf, want[0]), (dw, wbuf, want[1]), (db, bbuf, want[2])):
            assert torch.equal(got, ref_)
            n = got.numel()
            assert bool((buf[:off] == 7.25).all()) and bool((buf[off + n:] == 7.25).all())
    assert bool((ws[nb:] == 0xFF).all())
    # dx alone, or the parameters' gradients alone
    dx, none_w, none_b = ct.group_norm_nhwc_backward(dy, x, mean, rstd, groups)
    assert none_w is None and none_b is None
    none, dw, db = ct.group_norm_nhwc_backward(dy, x, mean, rstd, groups, w, b, need_x_grad=False)
    assert none is None and torch.equal(dw, want[1]) and torch.equal(db, want[2])
    _, dw, none = ct.group_norm_nhwc_backward(dy, x, mean, rstd, groups, w, None)
    assert none is None and dw.shape == (10,)


def test_strides_and_orders():
    """A permuted channels-first tensor, a channel slice, an expanded dy, every other weight."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(2, 24, 6, 5, generator=g).cuda()
    w, b = torch.randn(48, generator=g).cuda()[::2], torch.randn(24, generator=g).cuda()
    for v in (x.permute(0, 2, 3, 1), torch.randn(2, 6, 5, 50, generator=g).cuda()[..., 7:31]):
        y, mean, rstd = ct.group_norm_nhwc(v, 4, w, b, activation="gelu", return_stats=True)
        y2 = ct.group_norm_nhwc(v.contiguous(), 4, w.contiguous(), b, activation="gelu")
        assert torch.equal(y, y2) and y.is_contiguous()
        dy = torch.ones(1, 1, 1, 24, device="cuda").expand(2, 6, 5, 24)
        a = ct.group_norm_nhwc_backward(dy, v, mean, rstd, 4, w, b, activation="gelu")
        c = ct.group_norm_nhwc_backward(dy.contiguous(), v.contiguous(), mean, rstd, 4, w.contiguous(), b,
                                        activation="gelu")
        assert all(torch.equal(s, t) for s, t in zip(a, c))
        assert torch.equal(ct.dropout(v, 0.5, seed=3), ct.dropout(v.contiguous(), 0.5, seed=3))


def test_same_bits_again_and_while_others_run():
    """No result depends on timing: the same call gives the same bits, alone
    and while the same operators run on a second stream."""
    x, w, b, dy = (v.cuda() for v in inputs([8, 40, 40, 96], torch.bfloat16, 500))
    how = dict(activation="silu", p=0.2, seed=1, offset=2)

    def step():
        y, mean, rstd = ct.group_norm_nhwc(x, 8, w, b, return_stats=True, **how)
        return (y, mean, rstd) + ct.group_norm_nhwc_backward(dy, x, mean, rstd, 8, w, b, **how)

    first = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x2 = x.clone()
    torch.cuda.synchronize()
    for _ in range(5):
        got = step()
        o = ct.group_norm_nhwc(x2, 8, w, b, return_stats=True, stream=side, **how)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(first, got))
        assert all(torch.equal(u, v) for u, v in zip(first[:3], o))


def test_other_stream():
    x, w, b, dy = (v.cuda() for v in inputs([4, 64, 64, 64], torch.float16, 510))
    torch.cuda.synchronize()
    want = ct.group_norm_nhwc(x, 8, w, b, return_stats=True)
    wantb = ct.group_norm_nhwc_backward(dy, x, want[1], want[2], 8, w, b)
    wantd = ct.dropout(x, 0.5, seed=4, residual=dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = ct.group_norm_nhwc(x, 8, w, b, return_stats=True, stream=side)
    gotb = ct.group_norm_nhwc_backward(dy, x, got[1], got[2], 8, w, b, stream=side)
    gotd = ct.dropout(x, 0.5, seed=4, residual=dy, stream=side)
    junk = [torch.full_like(x, float("nan")) for _ in range(8)]   # would land in memory freed too early
    side.synchronize()
    for u, v in zip(want + wantb + (wantd,), got + gotb + (gotd,)):
        assert torch.equal(u, v)
    del junk


def test_graph_replays_draw_new_masks():
    """A captured step: the inputs and the random numbers change between
    replays, two graphs with the same tensors do not disturb each other."""
    shape, groups = [2, 20, 20, 32], 8
    x, w, b, dy = (v.cuda() for v in inputs(shape, torch.float16, 520))
    rng = torch.tensor([77, 0], device="cuda")

    def step():
        y, mean, rstd = ct.group_norm_nhwc(x, groups, w, b, activation="silu", p=0.25, rng=rng, return_stats=True)
        z = ct.dropout(y, 0.5, rng=rng, residual=x)
        dz = ct.dropout_backward(dy, 0.5, rng=rng)
        return (y, z) + ct.group_norm_nhwc_backward(dz, x, mean, rstd, groups, w, b, activation="silu", p=0.25,
                                                    rng=rng)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
            rng[1] += 1
        graphs.append((g, out))
    rng.copy_(torch.tensor([77, 0]))
    seen = []
    for k in range(4):
        if k == 2:
            x.mul_(1.5)
        g, out = graphs[k % 2]
        want_rng = torch.tensor([77, k], device="cuda")
        assert torch.equal(rng, want_rng)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        rng.copy_(want_rng)
        for u, v in zip(got, step()):
            assert torch.equal(u, v)
        assert torch.equal(got[0], ct.group_norm_nhwc(x, groups, w, b, activation="silu", p=0.25, seed=77, offset=k))
        rng.add_(torch.tensor([0, 1], device="cuda"))
        seen.append(got[0] == 0)
    assert not torch.equal(seen[0], seen[1])


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("n", [1, 7, 8, 9, 1023, 4096, 100001])
@pytest.mark.parametrize("p", [0.0, 1e-6, 0.1, 0.5, 0.999, 1.0])
def test_dropout(dtype, n, p):
    t = TYPES[dtype]
    x, r = draw([n], ("normal", 1.0), 600 + n, t), draw([n], ("normal", 1.0), 601 + n, t)
    seed, offset = (1 << 64) - 3, (1 << 63) + n
    f = ref.factor([n], p, seed, offset)
    y = ct.dropout(x.cuda(), p, seed=seed, offset=offset)
    z = ct.dropout(x.cuda(), p, seed=seed, offset=offset, residual=r.cuda())
    d = ct.dropout_backward(r.cuda(), p, seed=seed, offset=offset)
    # one fp32 step for the scale and one for the product, then the type's rounding
    for got, want, size in ((y, x.double() * f, x), (z, x.double() * f + r.double(), x), (d, r.double() * f, r)):
        part = size.double().abs() * f
        check(got, want, 1.01 * (ref.HALF[t] * want.abs() + 3 * ref.U * (part + want.abs())) + ref.TINY[t], "dropout")
    assert torch.equal(y.cpu() == 0, (f == 0) | (x == 0))
    assert torch.equal(d.cpu() == 0, (f == 0) | (r == 0))
    zc = z.cpu()
    assert torch.equal(zc[f == 0], r[f == 0])      # the residual comes through as it is


def test_dropout_of_not_finite_values():
    x = torch.full((4096,), float("inf"), device="cuda")
    x[::2] = float("nan")
    f = ref.factor([4096], 0.5, 5, 6)
    y = ct.dropout(x, 0.5, seed=5, offset=6).cpu()
    assert bool((y[f == 0] == 0).all())
    assert bool(y[f != 0][x.cpu()[f != 0].isnan()].isnan().all())
    assert bool((ct.dropout(x, 1.0) == 0).all())


def test_dropout_in_place_and_rng():
    x = draw([3, 333], ("normal", 1.0), 640, torch.bfloat16).cuda()
    r = draw([3, 333], ("normal", 1.0), 641, torch.bfloat16).cuda()
    want = ct.dropout(x, 0.3, seed=9, offset=10, residual=r)
    rng = torch.tensor([9, 10], device="cuda")
    assert torch.equal(ct.dropout(x, 0.3, rng=rng, residual=r), want)
    a, b = x.clone(), r.clone()
    assert ct.dropout(a, 0.3, seed=9, offset=10, residual=r, out=a) is a and torch.equal(a, want)
    assert ct.dropout(x, 0.3, seed=9, offset=10, residual=b, out=b) is b and torch.equal(b, want)
    assert torch.equal(ct.dropout(x, 0.3, seed=9, offset=10, residual=x), ct.dropout(x, 0.3, rng=rng, residual=x))
    neg = torch.tensor([-1, -2], device="cuda")    # the same 64 bits
    assert torch.equal(ct.dropout(x, 0.3, rng=neg), ct.dropout(x, 0.3, seed=(1 << 64) - 1, offset=(1 << 64) - 2))


def test_dropout_past_32_bits():
    """Indices beyond 2^32: the last elements of 2^32 + 24 take their own counters."""
    n = (1 << 32) + 24
    x = torch.ones(n, dtype=torch.float16, device="cuda")
    ct.dropout(x, 0.5, seed=21, offset=4, out=x)
    for first in (0, (1 << 31) - 100, (1 << 32) - 100, n - 124):
        got = x[first: first + 124].cpu() != 0
        assert torch.equal(got, torch.from_numpy(ref.keep_mask(124, 0.5, 21, 4, first=first)))
    del x
    torch.cuda.empty_cache()


def test_group_norm_past_32_bits():
    """An image that lies wholly beyond 2^32 elements."""
    n, s, c, groups = 3, 1 << 24, 96, 12        # 3 images of 1.6e9 elements
    x = torch.zeros(n, s, c, dtype=torch.float16, device="cuda")
    small = draw([1, 4096, c], ("normal", 1.0), 650, torch.float16).cuda()
    x[2].view(-1, 4096, c).copy_(small.expand(s // 4096, 4096, c))
    y, mean, rstd = ct.group_norm_nhwc(x, groups, activation="silu", return_stats=True)
    want, wm, wr = ct.group_norm_nhwc(small, groups, activation="silu", return_stats=True)
    assert bool((mean[:2] == 0).all())
    # the same values 4096 times over: statistics of the same numbers, each within its own bound
    assert float((mean[2] - wm[0]).abs().max()) <= 4 * ref.U * ref.CHAIN
    assert float((rstd[2] / wr[0] - 1).abs().max()) <= 2 * ref.U * ref.CHAIN
    for at in (0, 1 << 12, s - 4096):
        d = (y[2, at: at + 4096].float() - want[0].float()).abs()
        assert bool((d <= 2 * ref.HALF[torch.float16] * want[0].float().abs() + 1e-4).all())
    assert not bool(y[:2].any())
    del x, y
    torch.cuda.empty_cache()


def test_decoder_block():
    """The operators together, as a decoder runs them: upsample, norm with
    SiLU, dropout added to a skip; then the gradients back to the norm's input."""
    n, cin, c, groups = 2, 64, 48, 8
    x = draw([n, 9, 10, cin], ("normal", 1.0), 700, torch.float16)
    wt = draw([cin, 4, 4, c], ("normal", 0.09), 701, torch.float16)
    op = ct.ConvTranspose(wt.cuda(), list(x.shape), layout="nhwc", strides=[2, 2], pads=[1, 1, 1, 1])
    up = op(x.cuda())
    assert list(up.shape) == [n, 18, 20, c]
    skip = draw(list(up.shape), ("normal", 1.0), 702, torch.float16)
    w, b = 1 + draw([c], ("normal", 0.2), 703, torch.float32), draw([c], ("normal", 0.2), 704, torch.float32)
    dz = draw(list(up.shape), ("normal", 1.0), 705, torch.float16)
    h, mean, rstd = ct.group_norm_nhwc(up, groups, w.cuda(), b.cuda(), activation="silu", return_stats=True)
    z = ct.dropout(h, 0.2, seed=31, offset=1, residual=skip.cuda())
    dh = ct.dropout_backward(dz.cuda(), 0.2, seed=31, offset=1)
    dup, dw, db = ct.group_norm_nhwc_backward(dh, up, mean, rstd, groups, w.cuda(), b.cuda(), activation="silu")
    up64, t = up.cpu().double(), torch.float16
    f = ref.factor(list(up.shape), 0.2, 31, 1)
    y, mr, rr, a = ref.forward(up64, groups, w.double(), b.double(), EPS, "silu")
    bh = ref.forward_bound(up64, mr, rr, groups, w.double(), b.double(), a, y, t, 1.0)
    check(h, y, bh, "norm")
    want = y * f + skip.double()
    check(z, want, f * bh + 1.01 * (ref.HALF[t] * want.abs() + 4 * ref.U * (1 + want.abs())) + ref.TINY[t], "block")
    m64, r64 = mean.cpu().double(), rstd.cpu().double()
    # dh is rounded to its type between the two calls, so the norm's gradients are checked at dh as it is
    g = ref.backward(dh.cpu().double(), up64, m64, r64, groups, w.double(), b.double(), "silu")
    bounds = ref.backward_bounds(dh.cpu().double(), up64, m64, r64, groups, w.double(), b.double(), "silu", 1.0, t,
                                 torch.float32, *g)
    for got, val, bound in zip((dup, dw, db), g, bounds):
        check(got, val, bound, "block gradient")
    # dropout inside the norm's pass: the same mask, one rounding fewer
    fused = ct.group_norm_nhwc(up, groups, w.cuda(), b.cuda(), activation="silu", p=0.2, seed=31, offset=1)
    assert torch.equal(fused.cpu() == 0, (f == 0) | (fused.cpu() == 0)) and bool((fused.cpu()[f == 0] == 0).all())
    check(fused, y * f, ref.forward_bound(up64, mr, rr, groups, w.double(), b.double(), a, y * f, t,
                                          ref.drop_scale(0.2)), "norm with dropout")
