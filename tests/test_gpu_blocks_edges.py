"""Root-mean-square norm, rotary positions and AdamW on the GPU where their
contracts end: numbers at the borders of fp32, skipped updates, outputs on
inputs, rows past 32 bits in the kernels of whole rows."""

import math

import pytest
import torch

import blocks_ref as ref
from test_gpu_adamw import everything, make, same
from test_gpu_rms_norm import EPS, TYPES, _cuda, check_backward, check_forward, inputs, normal  # noqa: F401
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


def test_parameters_without_a_gradient_stay_valid():
    """What a backward pass still needs of a parameter that an update left as it was is not refused."""
    p, q = (torch.nn.Parameter(normal([40], k)) for k in (1, 2))
    opt = ct.AdamW([p, q], lr=1e-2)
    loss = (q * q).sum()
    opt.step([normal([40], 3), None])
    loss.backward()
    assert torch.equal(q.grad, 2 * q.detach())
    loss = (p * p).sum()
    opt.step([normal([40], 4), None])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


# ---- outputs that lie on inputs -----------------------------------------------------

def outputs(x, r):
    w = torch.ones(x.shape[-1], device="cuda")
    heads = x.view(x.shape[0], -1, 2, x.shape[-1] // 2)
    return {
        "norm": (x, lambda: ct.rms_norm_nhwc(x, w, out=x)),
        "norm of a sum": (x, lambda: ct.rms_norm_nhwc(x, w, residual=r, out=x)),
        "sum": (r, lambda: ct.rms_norm_nhwc(x, w, residual=r, sum_out=r)),
        "e4m3 sum": (r, lambda: ct.rms_norm_nhwc_e4m3(x, w, residual=r, sum_out=r)),
        "rotary": (x, lambda: ct.rotary_nhwc(heads, [8], out=heads)),
        "rotary slice": (x, lambda: ct.rotary_nhwc(heads[:, :, :1], [8], out=heads[:, :, :1])),
        "rotary back": (x, lambda: ct.rotary_nhwc_backward(heads, [8], out=heads)),
        "dropout": (x, lambda: ct.dropout(x, 0.5, out=x)),
        "group norm": (x, lambda: ct.group_norm_nhwc(r, 2, out=x)),
    }


@pytest.mark.parametrize("name", ["norm", "norm of a sum", "sum", "e4m3 sum", "rotary", "rotary slice", "rotary back",
                                  "dropout", "group norm"])
def test_writes_are_seen_by_autograd(name):
    """A tensor that a backward pass still needs is not overwritten unnoticed."""
    x, r = normal([3, 5, 16], 1), normal([3, 5, 16], 2)
    target, call = outputs(x, r)[name]
    a = torch.ones_like(target, requires_grad=True)
    loss = (a * target).sum()
    call()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


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


@pytest.mark.parametrize("top", [1 << 10, 1 << 17, 1 << 21, (1 << 24) - 1, 1 << 29])
def test_cosines_and_sines(top):
    """Pairs (1, 0) turn into the cosine and the sine.  Of the kernel's forms, u = 2^-24: the angle's remainder
    within an eighth of a turn is rounded to u / 2 once it is an angle; the cosine's polynomial adds the last sum's
    u / 2, a quarter of u from the square and a sixth from the sum before it, and 0.35 u of the angle: 1.3 u, the
    sine's 1.15 u, terms left out 0.03 u.  The position's product with a frequency of 48 bits, and the parts that it
    is made of, lose at most 2^-45 of the angle; beyond 2^24, in 64 bits, 2^-51."""
    n = 4096
    g = torch.Generator(device="cuda").manual_seed(top % 1000)
    at = torch.randint(-top, top, (n, 1), generator=g, device="cuda")
    for pairs, i, k in (("adjacent", slice(0, None, 2), slice(1, None, 2)), ("halves", slice(0, 64), slice(64, None))):
        x = torch.zeros(1, n, 1, 128, device="cuda")
        x[..., i] = 1.0
        angles = ref.rotary_angles(at.double(), [128], 10000.0)
        for call, sign in ((ct.rotary_nhwc, 1), (ct.rotary_nhwc_backward, -1)):
            y = call(x, [128], pairs=pairs, positions=at)[0, :, 0].double()
            bound = 1.5 * ref.U + angles.abs() * (2.0 ** -45 if top <= 1 << 24 else 2.0 ** -51)
            for got, want in ((y[:, i], torch.cos(angles)), (y[:, k], sign * torch.sin(angles))):
                err = (got - want).abs() / bound
                assert float(err.max()) <= 1, "%.3g of the bound" % float(err.max())


# ---- root-mean-square norm ------------------------------------------------------------

FULL = [256, 512, 768, 1024, 2048, 4096, 8192]       # rows of whole warps, each thread with all of its vectors


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("c", FULL + [64, 100, 511, 40000])
def test_values_at_the_edges_with_weights(c, dtype):
    """Rows of zeros, infinities and NaN in the kernels that whole rows with a weight have: they keep to themselves,
    with a residual and without, weights in both types."""
    t, rows = TYPES[dtype], 64
    for pdtype in (torch.float32, t):
        for residual in (False, True):
            x, r, w, _, _ = inputs([rows, c], t, 151, pdtype)
            r = r if residual else None
            foul, clean = x.clone(), x
            foul[2] = 0
            foul[4, c // 2] = float("inf")
            foul[6, 3] = float("nan")
            foul[9, c - 1] = -float("inf")
            foul[17, 0] = float("nan")
            odd = [2, 4, 6, 9, 17]
            rest = [i for i in range(rows) if i not in odd]
            if r is not None:
                r[2] = 0
            for block in (None, 0, 32, 128):       # None: the type's own output
                def call(v):
                    if block is None:
                        return ct.rms_norm_nhwc(v, w, eps=EPS, residual=r, return_rstd=True)
                    return ct.rms_norm_nhwc_e4m3(v, w, block=block or None, eps=EPS, residual=r, return_rstd=True)
                a, b = call(clean), call(foul)
                for p, q in zip(a, b):
                    p, q = (v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v for v in (p, q))
                    assert torch.equal(p[rest], q[rest])
                rstd = b[-1]
                assert bool(rstd[[6, 17]].isnan().all()) and not rstd[[4, 9]].any()
                assert abs(float(rstd[2]) * EPS ** 0.5 - 1) < 1e-6
                y = b[0].float() if block is None else b[0].float() * ref.spread_scales(b[1], block, c)
                assert not y[2].any() and bool(y[[6, 17]].isnan().all())
                assert bool(y[4, c // 2].isnan()) and bool(y[9, c - 1].isnan())
                if block is not None:
                    assert bool((b[1][2] == ref.LEAST_SCALE).all()) and bool(b[1][[6, 17]].isnan().all())
                    at = c // 2 // block if block and block < c else None
                    assert bool((b[1][4] if at is None else b[1][4][at]).isnan().all())
                    if at is not None:             # blocks beside the infinity's are of zeros
                        assert int(b[1][4].isnan().sum()) == 1


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("c", [32, 64, 100, 256, 511, 1024, 4096, 20000])
def test_products_that_overflow(c, dtype):
    """A block whose y is infinite though its x is not has a scale of NaN, as every block with an infinity has."""
    t = TYPES[dtype]
    x = 1 + normal([8, c], 5).abs().to(t)
    for how in (float("inf"), 3e38):
        w = torch.ones(c, device="cuda")
        w[c // 3] = how
        x[3, c // 3] = 8.0 * c ** 0.5             # alone it is most of the row: 3e38 times its share of sqrt(c)
        for block in (0, 32, 128):
            y = (x.double() / ((x.double() ** 2).mean(-1, keepdim=True) + EPS).sqrt() * w.double()).float()
            q, scale = ct.rms_norm_nhwc_e4m3(x, w, block=block or None, eps=EPS)
            width = block or c
            for b in range(-(-c // width)):
                part, s = y[:, b * width:(b + 1) * width], (scale[:, b] if block else scale)
                assert torch.equal(s.isnan(), part.isinf().any(-1)), (how, block, b)
            v = q.float() * ref.spread_scales(scale, block, c)
            assert bool(v[y.isinf()].isnan().all())


@pytest.mark.parametrize("c", [64, 511, 4096, 40000])
def test_where_squares_end(c):
    """Rows whose squares' sum fp32 holds come out right; beyond it rstd is 0."""
    x = normal([4, c], 7)
    x[0] *= 1.7e19 / float(torch.linalg.vector_norm(x[0].double()))
    x[1] *= 2.0e19 / float(torch.linalg.vector_norm(x[1].double()))
    x[2] = 1.7e19 / c ** 0.5
    x[3] = 2.0e19 / c ** 0.5
    y, rstd = ct.rms_norm_nhwc(x, None, eps=EPS, return_rstd=True)
    check_forward(x[::2], None, None, (y[::2], rstd[::2]), "%d channels" % c)
    assert not rstd[1::2].any() and not y[1::2].any()


@pytest.mark.parametrize("c", [1 << 20, 1 << 24])
def test_sums_of_the_longest_rows(c):
    """Terms that are all alike round alike: sums of the longest rows still hold to their bound."""
    for value in (1.1, -1.3, 0.7):
        x = torch.full([2, c], value, device="cuda")
        y, rstd = ct.rms_norm_nhwc(x, None, eps=EPS, return_rstd=True)
        check_forward(x, None, None, (y, rstd), "%d channels" % c)
        dy = torch.full_like(x, 0.3)
        w = torch.full([c], 0.9, device="cuda")
        check_backward(dy, x, rstd, w, None, ct.rms_norm_nhwc_backward(dy, x, rstd, w), "%d channels" % c)


@pytest.mark.parametrize("c", [1024, 4096])
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("residual", [True, False])
def test_whole_rows_past_32_bits(c, wide, residual):
    """Offsets above 2^31 elements in the kernels that whole rows with a weight have: the last rows, and those
    around the 32nd bit, are as they are alone."""
    rows = (1 << 31) // c + 64
    t = torch.float16
    w = (1 + 0.1 * normal([c], 9)).to(torch.float32 if wide else t)
    x = torch.empty(rows, c, dtype=t, device="cuda")
    x[:] = 1.0
    at = [slice(0, 64), slice(rows - 128, rows - 64), slice(rows - 64, rows)]
    for i, s in enumerate(at):
        x[s] = normal([64, c], 10 + i, t)
    r = x if residual else None

    def own(out, s):
        return [v[s].clone() for v in out]

    for call in (lambda a, b: ct.rms_norm_nhwc(a, w, eps=EPS, residual=b, return_rstd=True),
                 lambda a, b: ct.rms_norm_nhwc_e4m3(a, w, eps=EPS, residual=b, return_rstd=True),
                 lambda a, b: ct.rms_norm_nhwc_e4m3(a, w, block=128, eps=EPS, residual=b, return_rstd=True)):
        got = call(x, r)
        parts = [own(got, s) for s in at]
        middle = [v[1000:1064].clone() for v in got], [v[rows // 2:rows // 2 + 64].clone() for v in got]
        del got
        for s, part in zip(at, parts):
            alone = x[s].clone()
            for p, q in zip(part, call(alone, alone if residual else None)):
                p, q = (v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v for v in (p, q))
                assert torch.equal(p, q)
        for p, q in zip(*middle):
            p, q = (v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v for v in (p, q))
            assert torch.equal(p, q)
