"""Root-mean-square norm, rotary positions and AdamW without a GPU: the plain
forms against differences and by hand, and the refusals of the C entries and
the binding."""

import ctypes
import math

import pytest
import torch

import blocks_ref as ref
from transposed_convolution_02_b200 import ct


def differences(loss, leaves, grads, step=1e-6, tol=1e-6):
    """Central differences of loss(*leaves) against grads, at some elements of each."""
    for which, (t, gr) in enumerate(zip(leaves, grads)):
        for i in range(0, t.numel(), max(1, t.numel() // 12)):
            args = [v.clone() for v in leaves]
            args[which].view(-1)[i] += step
            hi = loss(*args)
            args[which].view(-1)[i] -= 2 * step
            # rounding of the difference: 1e-16 * |loss| / step
            assert abs((hi - loss(*args)) / (2 * step) - float(gr.reshape(-1)[i])) < tol


def test_rms_formulas_against_differences():
    g = torch.Generator().manual_seed(5)
    x, r, dy, dsum = (torch.randn(3, 4, 7, generator=g, dtype=torch.float64) for _ in range(4))
    w = torch.randn(7, generator=g, dtype=torch.float64)

    def loss(x, r, w):
        y, h, _ = ref.rms_forward(x, r, w, 1e-3)
        return float((y * dy).sum() + (h * dsum).sum())

    _, h, rstd = ref.rms_forward(x, r, w, 1e-3)
    dx, dw = ref.rms_backward(dy, h, rstd, w, dsum)
    differences(loss, (x, r, w), (dx, dx, dw))


def rms_desc(**over):
    d = ct.ct_rms_norm_desc(1, 0, 0, 0, 6, 12, 1e-6)
    for k, v in over.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("over, status", [
    ({}, 0), (dict(dtype=2), 0), (dict(param_dtype=1), 0), (dict(rows=0), 0), (dict(eps=0.0), 0),
    (dict(block=5), 0), (dict(dtype=3), 3), (dict(dtype=-1), 3), (dict(param_dtype=2), 3),
    (dict(dtype=0, param_dtype=1), 3), (dict(C=0), 1), (dict(C=-4), 1), (dict(C=(1 << 24) + 1), 1),
    (dict(rows=-1), 4), (dict(rows=1 << 60), 4), (dict(rows=1 << 62), 4),
    (dict(eps=-1e-6), 4), (dict(eps=float("nan")), 4), (dict(eps=float("inf")), 4)])
def test_rms_desc_refusals(over, status):
    b = ctypes.c_size_t()
    assert ct.lib().ct_rms_norm_workspace_bytes(ctypes.byref(rms_desc(**over)), ctypes.byref(b)) == status
    assert ct.lib().ct_rms_norm_workspace_bytes(None, ctypes.byref(b)) == 6
    assert ct.lib().ct_rms_norm_workspace_bytes(ctypes.byref(rms_desc()), None) == 6


def refused(fn, args, over, status):
    v = list(args)
    for k, x in over.items():
        v[k] = x
    return fn(*v) == status


# an aligned address that is never followed: every call is refused before a launch
A = 1 << 20


def test_rms_call_refusals():
    L = ct.lib()
    d = ctypes.byref(rms_desc())
    fwd = [d, A, A, A, A, A, A, None]
    for over, status in [({0: None}, 6), ({1: None}, 6), ({4: None}, 6), ({2: None}, 6), ({1: A + 1}, 5),
                         ({2: A + 1}, 5), ({3: A + 2}, 5), ({4: A + 1}, 5), ({5: A + 1}, 5), ({6: A + 2}, 5),
                         ({0: ctypes.byref(rms_desc(dtype=7))}, 3), ({0: ctypes.byref(rms_desc(rows=0)), 1: None}, 0)]:
        assert refused(L.ct_rms_norm, fwd, over, status), (over, status)
    quant = [d, A, A, A, A + 1, A, A, A, None]      # codes are bytes: any address
    for over, status in [({0: None}, 6), ({1: None}, 6), ({4: None}, 6), ({5: None}, 6), ({2: None}, 6),
                         ({5: A + 2}, 5), ({6: A + 1}, 5), ({7: A + 1}, 5)] + \
            [({0: ctypes.byref(rms_desc(block=b))}, 4) for b in (-32, 1, 16, 31, 33, 96, 256)]:
        assert refused(L.ct_rms_norm_e4m3, quant, over, status), (over, status)
    back = [d, A, A, A, A, A, A, A, A, None]
    for over, status in [({0: None}, 6), ({1: None}, 6), ({2: None}, 6), ({3: None}, 6), ({8: None}, 8),
                         ({8: A + 16}, 5), ({1: A + 1}, 5), ({2: A + 1}, 5), ({3: A + 2}, 5), ({4: A + 2}, 5),
                         ({5: A + 1}, 5), ({6: A + 1}, 5), ({7: A + 2}, 5), ({6: None, 7: None}, 0)]:
        assert refused(L.ct_rms_norm_backward, back, over, status), (over, status)
    if not torch.cuda.is_available():
        for fn, args in ((L.ct_rms_norm, fwd), (L.ct_rms_norm_e4m3, quant), (L.ct_rms_norm_backward, back)):
            assert refused(fn, args, {}, 7)


FLAT = torch.zeros(400)
X, R, OUT = FLAT[:72].view(2, 3, 12), FLAT[80:152].view(2, 3, 12), FLAT[160:232].view(2, 3, 12)
RSTD = FLAT[300:306].view(2, 3)


@pytest.mark.parametrize("call, refusal", [
    (lambda: ct.rms_norm_nhwc(X.double()), "float32"),
    (lambda: ct.rms_norm_nhwc(X.int()), "float32"),
    (lambda: ct.rms_norm_nhwc(torch.zeros(())), "shape"),
    (lambda: ct.rms_norm_nhwc(torch.zeros(4, 0)), "shape"),
    (lambda: ct.rms_norm_nhwc(X, FLAT[:11]), "weight"),
    (lambda: ct.rms_norm_nhwc(X, FLAT[:12].half()), "weight"),
    (lambda: ct.rms_norm_nhwc(X, FLAT[:12].view(1, 12)), "weight"),
    (lambda: ct.rms_norm_nhwc(X, residual=R[:1]), "residual"),
    (lambda: ct.rms_norm_nhwc(X, residual=R.half()), "residual"),
    (lambda: ct.rms_norm_nhwc(X, sum_out=OUT), "residual"),
    (lambda: ct.rms_norm_nhwc(X, out=OUT.half()), "out"),
    (lambda: ct.rms_norm_nhwc(X, out=OUT.transpose(0, 1)), "out"),
    (lambda: ct.rms_norm_nhwc(X, out=FLAT[4:76].view(2, 3, 12)), "overlaps"),
    (lambda: ct.rms_norm_nhwc(X, FLAT[165:177], out=OUT), "overlaps"),
    (lambda: ct.rms_norm_nhwc(X, residual=R, sum_out=FLAT[84:156].view(2, 3, 12)), "overlaps"),
    (lambda: ct.rms_norm_nhwc(X, residual=R, out=X, sum_out=X), "overlap"),
    (lambda: ct.rms_norm_nhwc(X, residual=R, out=OUT, sum_out=FLAT[231:303].view(2, 3, 12)), "overlap"),
    (lambda: ct.rms_norm_nhwc(X, residual=R, out=X, sum_out=R), "CUDA"),
    (lambda: ct.rms_norm_nhwc(X, eps=-1.0), "CT_ERR_ATTR"),
    (lambda: ct.rms_norm_nhwc_e4m3(X, block=16), "block"),
    (lambda: ct.rms_norm_nhwc_e4m3(X, block=48.0), "block"),
    (lambda: ct.rms_norm_nhwc_e4m3(X, sum_out=OUT), "residual"),
    (lambda: ct.rms_norm_nhwc_e4m3(X, block=64), "CUDA"),
    (lambda: ct.rms_norm_nhwc_backward(R[:1], X, RSTD), "dy"),
    (lambda: ct.rms_norm_nhwc_backward(R, X, RSTD, dsum=R.half()), "dsum"),
    (lambda: ct.rms_norm_nhwc_backward(R, X, RSTD.double()), "rstd"),
    (lambda: ct.rms_norm_nhwc_backward(R, X, RSTD.view(6)), "rstd"),
    (lambda: ct.rms_norm_nhwc_backward(R, X, RSTD, FLAT[:13]), "weight"),
    (lambda: ct.rms_norm_nhwc_backward(R, X, RSTD, FLAT[:12]), "CUDA")])
def test_rms_binding_refusals(call, refusal):
    with pytest.raises((ValueError, ct.CtError), match=refusal):
        call()


# ---- rotary positions ---------------------------------------------------------

@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_rotary_formula(pairs):
    """Turns keep lengths, add up, and the gradient is the turn back."""
    g = torch.Generator().manual_seed(6)
    x, dy = (torch.randn(2, 3, 4, 5, 9, generator=g, dtype=torch.float64) for _ in range(2))
    angles = ref.rotary_angles(ref.grid_positions([3, 4]), [6, 2], 100.0)
    y = ref.rotary(x, angles, pairs)
    assert torch.allclose((y * y).sum(-1), (x * x).sum(-1)) and torch.equal(y[..., 8], x[..., 8])
    assert torch.allclose(ref.rotary(y, angles, pairs), ref.rotary(x, 2 * angles, pairs))
    differences(lambda v: float((ref.rotary(v, angles, pairs) * dy).sum()), (x,), (ref.rotary(dy, -angles, pairs),))
    i, k = (0, 1) if pairs == "adjacent" else (0, 4)         # a turn by hand: pixel (2, 3), axis 0's first pair
    a, b = float(x[1, 2, 3, 4, i]), float(x[1, 2, 3, 4, k])
    assert abs(float(y[1, 2, 3, 4, i]) - (a * math.cos(2.0) - b * math.sin(2.0))) < 1e-12


def rotary_desc(**over):
    d = ct.ct_rotary_desc(1, 2, 0, 0, 0, 0, 2)
    d.grid[:] = [3, 4, 0]
    d.heads, d.dim, d.base = 5, 16, 10000.0
    d.sections[:] = [4, 8, 0]
    d.x_strides[:] = d.y_strides[:] = [960, 80, 16]
    for k, v in over.items():
        if isinstance(v, list):
            getattr(d, k)[:] = v
        else:
            setattr(d, k, v)
    return d


@pytest.mark.parametrize("over, status", [
    (dict(N=0), 0), (dict(heads=0), 0), (dict(grid=[0, 4, 0]), 0), (dict(dtype=3), 3), (dict(axes=0), 2),
    (dict(axes=4), 2), (dict(pairs=2), 4), (dict(inverse=2), 4), (dict(position_type=4), 4),
    (dict(position_images=2), 4),
    (dict(base=0.0), 4), (dict(base=-1.0), 4), (dict(base=float("nan")), 4), (dict(base=float("inf")), 4),
    (dict(N=-1), 4), (dict(heads=-1), 4), (dict(dim=0), 4), (dict(grid=[3, -1, 0]), 4), (dict(N=1 << 31), 4),
    (dict(N=1 << 30, grid=[1 << 30, 1 << 30, 0]), 4), (dict(sections=[3, 4, 0]), 1), (dict(sections=[-2, 4, 0]), 1),
    (dict(sections=[10, 8, 0]), 1), (dict(dim=600, sections=[500, 14, 0]), 1), (dict(sections=[1 << 40, 8, 0]), 1),
    (dict(x_strides=[1 << 59, 80, 16]), 4), (dict(x_strides=[-(1 << 58), 80, 16]), 4),
    (dict(y_strides=[960, 80, -16]), 4),
    (dict(y_strides=[960, 80, 15]), 4), (dict(y_strides=[960, 79, 16]), 4), (dict(y_strides=[959, 80, 16]), 4),
    (dict(y_strides=[960, 0, 16]), 4), (dict(y_strides=[0, 80, 16]), 4)])
def test_rotary_desc_refusals(over, status):
    assert ct.lib().ct_rotary(ctypes.byref(rotary_desc(**over)), A, None, A, None) == status


def test_rotary_call_refusals():
    L = ct.lib()
    d = ctypes.byref(rotary_desc())
    given = ctypes.byref(rotary_desc(position_type=2))
    for args, status in [((None, A, None, A), 6), ((d, None, None, A), 6), ((d, A, None, None), 6),
                         ((given, A, None, A), 6), ((given, A, A + 4, A), 5), ((d, A + 1, None, A), 5),
                         ((d, A, None, A + 1), 5)]:
        assert L.ct_rotary(*args, None) == status
    if not torch.cuda.is_available():
        for over in ({}, dict(x_strides=[0, 0, 0]), dict(y_strides=[960, 16, 192]), dict(y_strides=[16, 32, 384]),
                     dict(N=1, y_strides=[0, 80, 16]), dict(sections=[0, 0, 0])):
            assert L.ct_rotary(ctypes.byref(rotary_desc(**over)), A, None, A, None) == 7


HEADS = torch.zeros(2, 3, 4, 5, 16)
AT = torch.zeros(3, 4, 2)


@pytest.mark.parametrize("call, refusal", [
    (lambda: ct.rotary_nhwc(HEADS.double(), [4, 8]), "float32"),
    (lambda: ct.rotary_nhwc(HEADS, []), "axes"),
    (lambda: ct.rotary_nhwc(HEADS, [2, 2, 2, 2]), "axes"),
    (lambda: ct.rotary_nhwc(HEADS, [3, 8]), "even"),
    (lambda: ct.rotary_nhwc(HEADS, [2.5, 8]), "even"),
    (lambda: ct.rotary_nhwc(HEADS, [-2, 8]), "even"),
    (lambda: ct.rotary_nhwc(HEADS, [10, 8]), "fit"),
    (lambda: ct.rotary_nhwc(torch.zeros(1, 1, 1, 600), [514]), "fit"),
    (lambda: ct.rotary_nhwc(HEADS, [4]), "positions"),
    (lambda: ct.rotary_nhwc(HEADS[0, 0], [4, 8]), "shape"),
    (lambda: ct.rotary_nhwc(HEADS, [4, 8], pairs="even"), "pairs"),
    (lambda: ct.rotary_nhwc(HEADS, [4, 8], base=0), "base"),
    (lambda: ct.rotary_nhwc(HEADS, [4, 8], base=float("nan")), "base"),
    (lambda: ct.rotary_nhwc(HEADS, [4, 8], positions=AT.double()), "positions"),
    (lambda: ct.rotary_nhwc(HEADS, [4, 8], positions=AT[:2]), "positions"),
    (lambda: ct.rotary_nhwc(HEADS, [4, 8], positions=AT[..., :1]), "positions"),
    (lambda: ct.rotary_nhwc(HEADS, [4, 8], out=HEADS[:1]), "out"),
    (lambda: ct.rotary_nhwc(HEADS, [4, 8], out=torch.zeros(2, 3, 4, 16, 5).transpose(3, 4)), "neighbours"),
    (lambda: ct.rotary_nhwc(HEADS[:1], [4, 8], out=HEADS.view(-1)[16:976].view(1, 3, 4, 5, 16)), "overlaps"),
    (lambda: ct.rotary_nhwc(HEADS, [4, 8], out=HEADS), "CUDA"),
    (lambda: ct.rotary_nhwc_backward(HEADS, [4, 8], positions=AT, out=HEADS), "CUDA")])
def test_rotary_binding_refusals(call, refusal):
    with pytest.raises(ValueError, match=refusal):
        call()


def test_pixel_strides():
    """Pixels one stride apart are found in slices and permuted layouts."""
    def of(t):
        return ct._head_strides(t.shape, t.stride())
    qkv = torch.zeros(2, 3, 4, 15, 16)
    assert of(qkv) == (2880, 240, 16) and of(qkv[..., 5:10, :]) == (2880, 240, 16)
    assert of(qkv[:, :, ::2]) == (2880, 480, 16)           # rows of pixels that go on at the same stride
    assert of(qkv[:, :, :3]) is None and of(qkv[:, ::2]) is None and of(qkv[..., ::2]) is None
    assert of(qkv[:, :1, :3]) == (2880, 240, 16) and of(qkv[:, :, :1]) == (2880, 960, 16)
    assert of(torch.zeros(2, 5, 3, 4, 16).permute(0, 2, 3, 1, 4)) == (960, 16, 192)
    assert of(torch.zeros(2, 1, 5, 16)) == (80, 0, 16)


# ---- AdamW and the gradients' norm ------------------------------------------------

def test_adamw_formula():
    """A constant gradient moves by lr a step whatever its size; decay alone
    shrinks; the codes' grid is e4m3's and the random choice right on average."""
    p = m = v = torch.zeros(3, dtype=torch.float64)
    g = torch.tensor([1e-3, -2.0, 50.0], dtype=torch.float64)
    for t in range(1, 6):
        p, m, v, _ = ref.adamw(p, g, m, v, 0.01, (0.9, 0.999), 1e-30, 0.0, t)
        assert torch.allclose(p, -0.01 * t * g.sign())
    q = ref.adamw(p, 0 * g, 0 * g, 0 * g, 0.01, (0.9, 0.999), 1e-8, 0.5, 1)[0]
    assert torch.allclose(q, p * (1 - 0.005))
    x = torch.linspace(-448, 448, 100001, dtype=torch.float64)
    x = torch.cat((x, x / 448, x / 448 / 100, x / 448 / 5000))
    low, step = ref.code_steps(x)
    for c in (low, low + step):
        assert torch.equal(c.clamp(max=448).float().to(torch.float8_e4m3fn).double(), c.clamp(max=448))
    assert bool((low <= x.abs()).all()) and bool((x.abs() < low + step).all())
    r = torch.arange(65536, dtype=torch.float64)
    for value in (0.3, 1.07, 100.0, 0.001, 0.017):
        mean = ref.random_codes(torch.full_like(r, value), r)[0].mean()
        assert abs(float(mean) - value) <= float(ref.code_steps(torch.tensor(value).double())[1]) / 65536


def shapes(*rows):
    return (ct.ct_param * max(1, len(rows)))(*[ct.ct_param(*r) for r in rows])


def addresses(*values):
    return ct._pointers(list(values) or [0])


def adamw_status(desc=None, rows=((10, 0, 0, 0.1),), params=(A,), grads=(A,), m=A, v=A, ms=None, vs=None, master=None,
                 count=None, **over):
    d = ct.ct_adamw_desc(32, 0, 1e-3, 0.9, 0.999, 1e-8, 1, 3)
    for k, x in over.items():
        setattr(d, k, x)
    p, g = addresses(*params), addresses(*grads)
    return ct.lib().ct_adamw(ctypes.byref(d) if desc is None else None, len(rows) if count is None else count,
                             shapes(*rows), p.buffer_info()[0], g.buffer_info()[0], m, v, ms, vs, master, None)


@pytest.mark.parametrize("over, status", [
    (dict(desc=0), 6), (dict(bits=16), 4), (dict(lr=-1.0), 4), (dict(lr=float("nan")), 4), (dict(lr=float("inf")), 4),
    (dict(beta1=1.0), 4), (dict(beta2=-0.1), 4), (dict(beta2=float("nan")), 4), (dict(eps=0.0), 4),
    (dict(eps=float("inf")), 4), (dict(step=0), 4), (dict(count=-1), 4), (dict(count=(1 << 20) + 1), 4),
    (dict(rows=((10, 3, 3, 0.0),)), 3), (dict(rows=((10, 0, 1, 0.0),)), 3), (dict(rows=((10, 1, 2, 0.0),)), 3),
    (dict(rows=((-1, 0, 0, 0.0),)), 4), (dict(rows=(((1 << 40) + 1, 0, 0, 0.0),)), 4),
    (dict(rows=((1 << 40, 0, 0, 0.0), (1, 0, 0, 0.0)), params=(A, A), grads=(A, A)), 4),
    (dict(rows=((10, 0, 0, -0.1),)), 4), (dict(rows=((10, 0, 0, float("nan")),)), 4), (dict(params=(0,)), 6),
    (dict(params=(A + 2,)), 5), (dict(grads=(A + 2,)), 5), (dict(rows=((10, 1, 1, 0.0),)), 6),
    (dict(rows=((10, 1, 1, 0.0),), master=A, params=(A + 1,)), 5), (dict(m=None), 6), (dict(v=None), 6),
    (dict(m=A + 128), 5), (dict(bits=8), 6), (dict(bits=8, ms=A), 6), (dict(bits=8, ms=A, vs=A + 4), 5),
    (dict(master=A + 4), 5), (dict(lr_device=A + 2), 5), (dict(step_device=A + 4), 5), (dict(grad_scale=A + 2), 5),
    (dict(grads=(0,), params=(0,), m=None), 0), (dict(rows=((0, 0, 0, 0.0),), m=None), 0), (dict(count=0, m=None), 0)])
def test_adamw_refusals(over, status):
    assert adamw_status(**over) == status


def test_grad_norm_refusals():
    L = ct.lib()
    n = ctypes.c_size_t()
    assert L.ct_grad_norm_workspace_bytes(5, None) == 6 and L.ct_grad_norm_workspace_bytes(-1, ctypes.byref(n)) == 4
    assert L.ct_grad_norm_workspace_bytes(600, ctypes.byref(n)) == 0 and n.value >= 8 * 2 * 592
    s, g = shapes((10, 0, 0, 0.0)), addresses(A)

    def status(count=1, shapes_=s, grads=g.buffer_info()[0], most=1.0, norm=A, scale=A, ws=A):
        return L.ct_grad_norm(count, shapes_, grads, most, norm, scale, ws, None)

    assert status(count=-1) == 4 and status(shapes_=None) == 6 and status(grads=None) == 6
    assert status(most=0.0) == 4 and status(most=-1.0) == 4 and status(most=float("nan")) == 4
    assert status(norm=None) == 6 and status(ws=None) == 8 and status(ws=A + 8) == 5 and status(scale=A + 1) == 5
    if not torch.cuda.is_available():
        assert status() == 7 and status(scale=None, most=float("inf")) == 7 and adamw_status() == 7


class Card(torch.Tensor):
    """A CPU tensor that passes for one on a device, for the binding's checks."""
    is_cuda = True


def card(*size, dtype=torch.float32):
    return torch.zeros(*size, dtype=dtype).as_subclass(Card)


@pytest.mark.parametrize("make, refusal", [
    (lambda: ct.AdamW([]), "no parameter"),
    (lambda: ct.AdamW([torch.zeros(3)]), "CUDA"),
    (lambda: ct.AdamW([card(3, dtype=torch.float64)]), "float32"),
    (lambda: ct.AdamW([card(3, 4).t()]), "contiguous"),
    (lambda: ct.AdamW([card(3)], bits=16), "bits"),
    (lambda: ct.AdamW([card(3)], seed=-1), "seed"),
    (lambda: ct.AdamW([card(3)], betas=(0.9, 1.0)), "betas"),
    (lambda: ct.AdamW([card(3)], eps=0.0), "eps"),
    (lambda: ct.AdamW([card(3)], weight_decay=-0.1), "weight_decay"),
    (lambda: ct.AdamW([card(3)], weight_decay=[0.1, 0.2]), "weight_decay"),
    (lambda: ct.AdamW([TWICE, TWICE]), "overlap"),
    (lambda: ct.AdamW([TWICE[:2], TWICE[1:]]), "overlap"),
    (lambda: ct.grad_norm([]), "no gradient"),
    (lambda: ct.grad_norm([None, None]), "no gradient"),
    (lambda: ct.grad_norm([torch.zeros(3)]), "CUDA"),
    (lambda: ct.grad_norm([card(3)], max_norm=0.0), "max_norm"),
    (lambda: ct.grad_norm([card(3)], max_norm=float("nan")), "max_norm"),
    (lambda: ct.grad_norm([card(3, dtype=torch.int32)]), "float32")])
def test_adamw_binding_refusals(make, refusal):
    with pytest.raises(ValueError, match=refusal):
        make()


TWICE = card(3)


def test_adamw_step_refusals():
    p, q = card(2, 3), card(5, dtype=torch.float16)
    opt = ct.AdamW([p, q])
    g = [card(2, 3), card(5, dtype=torch.float16)]
    one = card(1)
    for grads, how, refusal in [
            (g[:1], {}, "2 parameters"), ([g[0].view(3, 2), g[1]], {}, "gradient 0"),
            ([g[0].half(), g[1]], {}, "gradient 0"),
            ([g[0], card(5, dtype=torch.bfloat16)], {}, "gradient 1"), ([g[0], torch.zeros(5)], {}, "CUDA"),
            (g, dict(grad_scale=one.double()), "grad_scale"), (g, dict(grad_scale=card(2)), "grad_scale"),
            (g, dict(step=one), "step")]:
        with pytest.raises(ValueError, match=refusal):
            opt.step(grads, **how)
    for lr in (-1.0, float("nan"), float("inf")):
        opt.lr = lr
        with pytest.raises(ValueError, match="lr"):
            opt.step(g)
    opt.lr = 1e-3
    kept = opt.exp_avg
    for other in (kept[:256], kept.half(), torch.zeros(2, 512)[:, ::2].reshape(-1)[::2], None):
        opt.exp_avg = other
        with pytest.raises(ValueError, match="exp_avg"):
            opt.step(g)
    opt.exp_avg, opt.master = kept, None
    with pytest.raises(ValueError, match="master"):
        opt.step(g)
    opt.master = torch.zeros(256)
    q.data = q.data[:4]
    with pytest.raises(ValueError, match="parameter 1"):
        opt.step(g)
    assert opt.steps == 0
