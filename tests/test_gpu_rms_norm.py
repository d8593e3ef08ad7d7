"""Root-mean-square norm on the GPU against its plain fp64 form."""

import pytest
import torch

import blocks_ref as ref
from transposed_convolution_02_b200 import ct

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    major, _ = torch.cuda.get_device_capability()
    assert major == 10, "these kernels are built for sm_100a"


def normal(shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def inputs(shape, dtype, seed, pdtype=torch.float32):
    c = shape[-1]
    spread = 0.3 + normal([c], seed).abs() ** 3
    x, r = ((normal(shape, seed + k) * spread).to(dtype) for k in (1, 2))
    w = (1 + 0.3 * normal([c], seed + 3)).to(pdtype)
    return x, r, w, normal(shape, seed + 4, dtype), normal(shape, seed + 5, dtype)


def as64(t):
    return None if t is None else t.double()


def check_forward(x, r, w, got, where):
    """got: (y[, sum], rstd)"""
    one = torch.ones(x.shape[-1], device="cuda", dtype=torch.float64) if w is None else w.double()
    y, h, rstd = ref.rms_forward(x.double(), as64(r), one, EPS)
    by, bh, br = ref.rms_bounds(y, h, rstd, x.dtype)
    ref.check(got[-1], rstd, br, where + " rstd")
    ref.check(got[0], y, by, where + " y")
    if r is not None:
        ref.check(got[1], h, bh, where + " sum")


def check_codes(x, r, w, block, got, where):
    """got: (q, scale[, sum], rstd); codes against y over the returned scale."""
    one = torch.ones(x.shape[-1], device="cuda", dtype=torch.float64) if w is None else w.double()
    y, h, rstd = ref.rms_forward(x.double(), as64(r), one, EPS)
    scale = ref.block_scales(y, block)
    assert got[0].dtype == torch.float8_e4m3fn and got[1].dtype == torch.float32
    ref.check(got[1], scale, (ref.CHAIN / 2 + 10) * ref.U * scale, where + " scale")
    v = y / ref.spread_scales(got[1].double(), block, x.shape[-1])
    ref.check(got[0].float(), v, ref.e4m3_bound(v), where + " codes")
    ref.check(got[-1], rstd, ref.rms_bounds(y, h, rstd, x.dtype)[2], where + " rstd")
    if r is not None:
        ref.check(got[2], h, ref.rms_bounds(y, h, rstd, x.dtype)[1], where + " sum")


def check_backward(dy, h, rstd, w, dsum, got, where):
    one = torch.ones(h.shape[-1], device="cuda", dtype=torch.float64) if w is None else w.double()
    args = (dy.double(), h.double(), rstd.double(), one, as64(dsum))
    dx, dw = ref.rms_backward(*args)
    bx, bw = ref.rms_backward_bounds(*args, dx, dw, h.dtype, torch.float32 if w is None else w.dtype)
    if got[0] is not None:
        ref.check(got[0], dx, bx, where + " dx")
    if w is None:
        assert got[1] is None
    else:
        ref.check(got[1], dw, bw, where + " dweight")


def all_ways(shape, dtype, seed, residual=True, weight=True, pdtype=torch.float32, block=0, data=None):
    x, r, w, dy, dsum = inputs(shape, dtype, seed, pdtype) if data is None else data
    r, dsum = (r, dsum) if residual else (None, None)
    w = w if weight else None
    where = "%s %s res=%s block=%d" % (shape, dtype, residual, block)
    out = ct.rms_norm_nhwc(x, w, eps=EPS, residual=r, return_rstd=True)
    check_forward(x, r, w, out, where)
    check_codes(x, r, w, block, ct.rms_norm_nhwc_e4m3(x, w, block=block or None, eps=EPS, residual=r, return_rstd=True),
                where)
    h = x if r is None else out[1]
    back = ct.rms_norm_nhwc_backward(dy, h, out[-1], w, dsum=dsum)
    check_backward(dy, h, out[-1], w, dsum, back, where)
    return out, back


CHANNELS = [1, 2, 3, 7, 8, 9, 16, 24, 31, 32, 33, 40, 64, 65, 72, 96, 127, 128, 129, 136, 160, 255, 256, 257, 264, 320,
            500, 511, 512, 513, 520, 1000, 1024, 1025, 1032, 2000, 2048, 2049, 2056, 4095, 4096, 4100, 4104, 5000, 8192,
            8193, 8200, 10000, 16383, 16384, 16385, 16392, 20000, 32768, 32776, 40001]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("c", CHANNELS)
def test_channels(c, dtype):
    """Every way at every number of channels where the choice of threads,
    vectors and walks changes, in a few rows and in more than a round of blocks."""
    t = TYPES[dtype]
    i = CHANNELS.index(c)
    for k, rows in enumerate([[1], [3, 5], [2, 9, 41], [1200 if c > 600 else 5000]]):
        if rows[0] * c > 6e6:
            continue
        all_ways(rows + [c], t, 100 * i + 10 * k, residual=(i + k) % 3 != 0, weight=(i + k) % 4 != 1,
                 pdtype=[torch.float32, t][(i + k) % 2], block=[0, 32, 64, 128][(i + 3 * k) % 4])


WARPS = [320, 384, 448, 640, 768, 896, 1152, 1280, 1536, 1792, 2304, 2560, 3584, 5120, 6144, 7168, 10240, 12288, 14336]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("c", WARPS)
def test_rows_of_any_number_of_warps(c, dtype):
    """Rows of 3, 5, 6, 7 ... warps and of 24 elements a thread: whole ones, and with rows that no slot has."""
    for k, rows in enumerate((1, 6, 7, 1200 if c < 2000 else 450)):
        all_ways([rows, c], TYPES[dtype], c + k, residual=k % 2 == 0, weight=k != 2,
                 pdtype=[torch.float32, TYPES[dtype]][k // 2], block=[0, 128, 32, 0][k])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("c", [32, 33, 34, 36, 100, 255, 1001, 2047, 8191, 12001, 16381, 24001, 32765])
def test_neighbours_in_a_vector(c, residual, dtype):
    """Rows that share vectors with their neighbours: NaN and infinities in those leave a row to the bit what it
    is beside zeros, and what is not written stays; one round of blocks and several."""
    t = TYPES[dtype]
    for rows in (3, 11, 60000 if c <= 100 else 3000 if c <= 1001 else 301):
        x, r, w, _, _ = inputs([rows, c], t, c + rows)
        r = r if residual else None
        for first in (0, 1):
            clean, foul = x.clone(), x.clone()
            clean[1 - first::2] = 0
            foul[1 - first::2] = float("nan")
            foul[1 - first::4] = float("inf")
            own = slice(first, None, 2)
            for call in (ct.rms_norm_nhwc, ct.rms_norm_nhwc_e4m3):
                a, b = (call(v, w, eps=EPS, residual=r, return_rstd=True) for v in (clean, foul))
                for p, q in zip(a, b):
                    p, q = (v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v for v in (p, q))
                    assert torch.equal(p[own], q[own])
        flat = torch.full((rows * c + 16,), 7.0, dtype=t, device="cuda")
        out = flat[8:-8].view(rows, c)
        ct.rms_norm_nhwc(x, w, eps=EPS, residual=r, out=out)
        assert bool((flat[:8] == 7).all()) and bool((flat[-8:] == 7).all())
        want = ct.rms_norm_nhwc(x, w, eps=EPS, residual=r)
        assert torch.equal(out, want[0] if residual else want)
        over, into = x.clone(), None if r is None else r.clone()               # in place
        ct.rms_norm_nhwc(over, w, eps=EPS, residual=into, out=over, sum_out=into)
        assert torch.equal(over, out) and (r is None or torch.equal(into, want[1]))


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("block", [0, 32, 64, 128])
@pytest.mark.parametrize("c", [32, 33, 100, 128, 200, 264, 511, 1024, 2056, 16400, 33000])
def test_blocks(c, block, dtype):
    x, r, w, _, _ = inputs([5, c], TYPES[dtype], 7)
    for res in (None, r):
        got = ct.rms_norm_nhwc_e4m3(x, w, block=block or None, eps=EPS, residual=res, return_rstd=True)
        check_codes(x, res, w, block, got, "C=%d block=%d" % (c, block))


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("c", [64, 511, 4096])
def test_alignment_and_strides(c, dtype):
    """Tensors that start inside a vector, weights too, and views that are not
    contiguous."""
    t, rows = TYPES[dtype], 37
    x, r, w, dy, dsum = inputs([rows, c], t, 31)

    def moved(v, by):
        flat = torch.empty(v.numel() + by, dtype=v.dtype, device="cuda")
        flat[by:] = v.reshape(-1)
        return flat[by:].view(v.shape)

    for k in range(5):
        data = [moved(v, 1 if k == j else 0) for j, v in enumerate((x, r, w, dy, dsum))]
        all_ways([rows, c], t, 0, data=data, block=64)
    wide = torch.cat((x, r, dy, dsum), dim=1)                # slices: rows a stride apart
    data = [wide[:, k * c:(k + 1) * c] for k in range(4)]
    all_ways([rows, c], t, 0, data=(data[0], data[1], w.repeat_interleave(2)[::2], data[2], data[3]))
    y = torch.empty(rows * c + 1, dtype=t, device="cuda")[1:].view(rows, c)
    s = torch.empty(rows * c + 3, dtype=t, device="cuda")[3:].view(rows, c)
    out = ct.rms_norm_nhwc(x, w, eps=EPS, residual=r, out=y, sum_out=s, return_rstd=True)
    assert out[0] is y and out[1] is s
    check_forward(x, r, w, out, "odd outputs")


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("c", [48, 511, 2048, 40000])
def test_in_place(c, dtype):
    """Outputs on the inputs give the bits that outputs beside them give."""
    x, r, w, _, _ = inputs([33, c], TYPES[dtype], 41)
    want = ct.rms_norm_nhwc(x, w, eps=EPS, residual=r)
    for swap in (False, True):
        a, b = x.clone(), r.clone()
        out, s = (b, a) if swap else (a, b)
        ct.rms_norm_nhwc(a, w, eps=EPS, residual=b, out=out, sum_out=s)
        assert torch.equal(out, want[0]) and torch.equal(s, want[1])
    a = x.clone()
    assert torch.equal(ct.rms_norm_nhwc(a, w, eps=EPS, out=a), ct.rms_norm_nhwc(x, w, eps=EPS))
    for block in (None, 32, 128):
        want = ct.rms_norm_nhwc_e4m3(x, w, block=block, eps=EPS, residual=r)
        b = r.clone()
        got = ct.rms_norm_nhwc_e4m3(x, w, block=block, eps=EPS, residual=b, sum_out=b)
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, want))


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_values_at_the_edges(dtype):
    """Rows of zeros, infinities and NaN keep to themselves; scales never are 0."""
    t = TYPES[dtype]
    for c in (40, 64, 511, 4096, 40000):
        x = normal([9, c], 51, t)
        plain = x.clone()
        x[2] = 0
        x[4, c // 2] = float("inf")
        x[6, 3] = float("nan")
        x[7] = 2.0 ** -14            # eps is larger than the squares
        rest = [0, 1, 3, 5, 8]
        y, rstd = ct.rms_norm_nhwc(x, None, eps=EPS, return_rstd=True)
        want = ct.rms_norm_nhwc(plain, None, eps=EPS)
        assert torch.equal(y[rest], want[rest])
        assert not y[2].any() and abs(float(rstd[2]) * EPS ** 0.5 - 1) < 1e-6
        assert float(rstd[4]) == 0 and bool(y[4, c // 2].isnan()) and not y[4, :c // 2].any()
        assert bool(y[6].isnan().all()) and bool(rstd[6].isnan())
        check_forward(x[7:8], None, None, (y[7:8], rstd[7:8]), "small row")
        for block in (None, 32):
            q, scale = ct.rms_norm_nhwc_e4m3(x, None, block=block, eps=EPS)
            v = q.float() * ref.spread_scales(scale, block or 0, c)
            assert not v[2].any() and bool((scale[2] == ref.LEAST_SCALE).all())
            assert bool(v[6].isnan().all()) and bool(v[4, c // 2].isnan())
            assert bool(v[rest].isfinite().all())
        dx, dw = ct.rms_norm_nhwc_backward(plain, x, rstd, torch.ones(c, device="cuda"))
        assert bool(dx[rest].isfinite().all()) and bool(dx[6].isnan().all())


@pytest.mark.parametrize("c", [12, 511, 20000])
def test_no_rows(c):
    x = torch.empty(2, 0, c, device="cuda", dtype=torch.float16)
    w = torch.ones(c, device="cuda")
    y, s, rstd = ct.rms_norm_nhwc(x, w, residual=x, return_rstd=True)
    assert y.shape == s.shape == x.shape and rstd.shape == (2, 0)
    q, scale = ct.rms_norm_nhwc_e4m3(x, w, block=32)
    assert q.shape == x.shape and scale.shape == (2, 0, -(-c // 32))
    dx, dw = ct.rms_norm_nhwc_backward(x, x, rstd, w)
    assert dx.shape == x.shape and not dw.any() and dw.shape == w.shape


def test_what_is_not_wanted():
    x, r, w, dy, _ = inputs([300, 520], torch.float16, 61)
    y, rstd = ct.rms_norm_nhwc(x, w, eps=EPS, return_rstd=True)
    assert torch.equal(ct.rms_norm_nhwc(x, w, eps=EPS), y)
    full = ct.rms_norm_nhwc_backward(dy, x, rstd, w)
    only = ct.rms_norm_nhwc_backward(dy, x, rstd, w, need_x_grad=False)
    assert only[0] is None and torch.equal(only[1], full[1])
    assert ct.rms_norm_nhwc_backward(dy, x, rstd, None)[1] is None


@pytest.mark.parametrize("shape", [[50000, 64], [3000, 511], [2000, 4096], [600, 20000]])
def test_same_bits(shape):
    x, r, w, dy, dsum = inputs(shape, torch.bfloat16, 71)
    first = None
    for _ in range(3):
        out = ct.rms_norm_nhwc(x, w, residual=r, return_rstd=True)
        got = out + ct.rms_norm_nhwc_backward(dy, out[1], out[2], w, dsum=dsum)
        first = got if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_rows_past_32_bits():
    """Offsets above 2^31 elements: the last rows are as they are alone."""
    rows, c = (1 << 31) // 4096 + 9, 4096
    x = torch.empty(rows, c, dtype=torch.float16, device="cuda")
    x[:-8] = 1.0
    x[-8:] = normal([8, c], 81, torch.float16)
    y, s, rstd = ct.rms_norm_nhwc(x, None, eps=EPS, residual=x, return_rstd=True)
    ya, sa, ra = ct.rms_norm_nhwc(x[-8:].clone(), None, eps=EPS, residual=x[-8:].clone(), return_rstd=True)
    assert torch.equal(y[-8:], ya) and torch.equal(s[-8:], sa) and torch.equal(rstd[-8:], ra)
    assert bool((y[:-8].float().sub_(1).abs_() < 1e-3).all())
    del y, s
    dx, _ = ct.rms_norm_nhwc_backward(x, x, rstd, None)
    assert torch.equal(dx[-8:], ct.rms_norm_nhwc_backward(x[-8:].clone(), x[-8:].clone(), ra, None)[0])


def test_streams_and_graphs():
    """On another stream than the current one; two captured graphs that share
    no workspace, replayed on new data at the same time."""
    x, r, w, dy, dsum = inputs([700, 1024], torch.float16, 91)
    want = ct.rms_norm_nhwc(x, w, residual=r, return_rstd=True)
    want += ct.rms_norm_nhwc_backward(dy, want[1], want[2], w, dsum=dsum)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ct.rms_norm_nhwc(x, w, residual=r, return_rstd=True, stream=side)
    got += ct.rms_norm_nhwc_backward(dy, got[1], got[2], w, dsum=dsum, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for k in range(2):
        ins = [v.clone() for v in (x, r, dy)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ct.rms_norm_nhwc(ins[0], w, residual=ins[1], return_rstd=True)
            out += ct.rms_norm_nhwc_backward(ins[2], out[1], out[2], w, dsum=dsum)
        graphs.append((g, ins, out))
    for k, (g, ins, out) in enumerate(graphs):
        for j, v in enumerate(ins):
            v.copy_(normal(v.shape, 200 + 10 * k + j, torch.float16))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for (g, ins, out), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for g, ins, out in graphs:
        want = ct.rms_norm_nhwc(ins[0], w, residual=ins[1], return_rstd=True)
        want += ct.rms_norm_nhwc_backward(ins[2], want[1], want[2], w, dsum=dsum)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_inputs_that_require_gradients():
    x = torch.zeros(3, 8, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        ct.rms_norm_nhwc(x)
    with torch.no_grad():
        ct.rms_norm_nhwc(x)
