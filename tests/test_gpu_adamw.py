"""AdamW and the gradients' norm on the GPU against their plain fp64 forms, and
a training step of the operators together."""

import math

import numpy as np
import pytest
import torch

import blocks_ref as ref
import layers_ref
from test_gpu_rms_norm import TYPES, _cuda, normal  # noqa: F401
from transposed_convolution_02_b200 import ct

pytestmark = pytest.mark.gpu

BLOCK = 256
SIZES = [[1], [3], [0], [2, 5], [255], [256], [257], [31, 33], [8, 4, 3, 3], [1024], [4099], [70, 1000], [7]]
KINDS = [torch.float32, torch.bfloat16, torch.float16]


def blocks(n):
    return -(-n // BLOCK)


def spread(opt, flat, i, low=False):
    """Parameter i's part of a buffer (masters: of the 16-bit parameters alone)."""
    at = sum(blocks(p.numel()) for p in opt.params[:i] if not low or p.dtype != torch.float32) * BLOCK
    return flat[at:at + opt.params[i].numel()]


def held(opt):
    """What the next update starts from, in fp64: (p, m, v) for each parameter."""
    m, v = opt.exp_avg.double(), opt.exp_avg_sq.double()
    if opt.bits == 8:
        m = m * opt.exp_avg_scale.double().repeat_interleave(BLOCK)
        v = (v * opt.exp_avg_sq_scale.double().repeat_interleave(BLOCK)) ** 2
    out = []
    for i, p in enumerate(opt.params):
        w = p.detach().double().reshape(-1) if p.dtype == torch.float32 else spread(opt, opt.master, i, True).double()
        out.append((w, spread(opt, m, i).clone(), spread(opt, v, i).clone()))
    return out


def random16(n, seed, step):
    i = np.arange(-(-n // 8), dtype=np.uint64)
    c = np.stack([i & np.uint64(0xFFFFFFFF), i >> np.uint64(32), np.full_like(i, step & 0xFFFFFFFF),
                  np.full_like(i, step >> 32)], axis=1)
    w = layers_ref.philox(c, [seed & 0xFFFFFFFF, seed >> 32])
    return torch.from_numpy(np.stack([w & 0xFFFF, w >> 16], axis=2).reshape(-1)[:n].astype(np.float64)).cuda()


def check_step(opt, old, grads, scale, step, lr, where):
    """The parameters and states that an update left, from what it started with."""
    bits = random16(opt.exp_avg.numel(), opt.seed, step) if opt.bits == 8 else None
    for i, (p, g) in enumerate(zip(opt.params, grads)):
        if g is None or p.numel() == 0:
            continue
        w, m, v = old[i]
        decay = opt._decay[i]
        g64 = g.double().reshape(-1) * scale
        args = (lr, opt.betas, opt.eps, decay, step)
        new = ref.adamw(w, g64, m, v, *args)
        bp, bm, bv = ref.adamw_bounds(w, g64, m, v, new, *args)
        at = "%s parameter %d %s %s" % (where, i, list(p.shape), p.dtype)
        got = p.detach().reshape(-1)
        if p.dtype != torch.float32:
            held_ = spread(opt, opt.master, i, True)
            assert torch.equal(held_.to(p.dtype), got), at + " is its master rounded"
            got = held_
        ref.check(got, new[0], bp, at + " p")
        if opt.bits == 32:
            ref.check(spread(opt, opt.exp_avg, i), new[1], bm, at + " m")
            ref.check(spread(opt, opt.exp_avg_sq, i), new[2], bv, at + " v")
            continue
        first = sum(blocks(q.numel()) for q in opt.params[:i])
        n = p.numel()
        r = bits[first * BLOCK:first * BLOCK + n]
        for what, value, flat, scales in (("m", new[1], opt.exp_avg, opt.exp_avg_scale),
                                          ("root", torch.sqrt(new[2]), opt.exp_avg_sq, opt.exp_avg_sq_scale)):
            sc = scales[first:first + blocks(n)].double()
            full = torch.nn.functional.pad(value, (0, -n % BLOCK)).view(-1, BLOCK).abs().amax(dim=1)
            # m as bm says, against the block's largest; a root to 8 u; the quotient by 448
            most = torch.nn.functional.pad(bm, (0, -n % BLOCK)).view(-1, BLOCK).amax(dim=1)
            ref.check(sc, (full / 448).clamp(min=ref.LEAST_SCALE), 12 * ref.U * full / 448 + most / 448 + 2.0 ** -149,
                      at + " scale of " + what)
            x = value / sc.repeat_interleave(BLOCK)[:n]
            # an m that two terms nearly cancel in is good to what they were
            sure = torch.ones_like(x, dtype=torch.bool) if what == "root" else \
                bm <= 12 * ref.U * value.abs() + ref.U * 2.0 ** -9 * sc.repeat_interleave(BLOCK)[:n]
            want, close = ref.random_codes(x, r)
            if what == "root":
                want = torch.where(value > 0, want.clamp(min=2.0 ** -9), want)
            code = spread(opt, flat, i).double()
            assert bool(((code == want) | close | ~sure).all()), at + " codes of " + what
            assert bool(((code - x).abs() <= 1.001 * ref.code_steps(x)[1] + 1e-6).all()), at + " codes of " + what


def make(seed, sizes=SIZES, kinds=KINDS, moved=0):
    params, grads = [], []
    for i, size in enumerate(sizes):
        t = kinds[i % len(kinds)]
        n = math.prod(size)
        flat = torch.zeros(n + moved, dtype=t, device="cuda")
        params.append(flat[moved:].view(size).copy_(normal(size, seed + 2 * i, scale=0.1)))
        gt = t if (i // len(kinds)) % 2 == 0 else torch.float32
        g = torch.zeros(n + moved, dtype=gt, device="cuda")[moved:].view(size)
        grads.append(g.copy_(normal(size, seed + 2 * i + 1, scale=10.0 ** (-(i % 4)))))
    return params, grads


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("moved", [0, 1, 2, 4])
def test_adamw(moved, bits):
    """Sizes around a block, mixed types, several steps; tensors that start
    inside a vector."""
    params, _ = make(100, moved=moved)
    decay = [0.0 if i % 3 == 1 else 0.05 for i in range(len(params))]
    opt = ct.AdamW(params, lr=3e-3, betas=(0.8, 0.95), eps=1e-8, weight_decay=decay, bits=bits, seed=(1 << 50) + 9)
    assert (opt.master is not None) and opt.exp_avg.numel() % BLOCK == 0
    for step in range(1, 5):
        old, (_, grads) = held(opt), make(1000 * step, moved=moved)
        if step == 3:
            grads[5] = torch.zeros_like(grads[5])
        opt.step(grads)
        assert opt.steps == step
        check_step(opt, old, grads, 1.0, step, 3e-3, "step %d" % step)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("betas", [(0.0, 0.0), (0.9, 0.999), (0.99, 0.9999)])
def test_betas_and_far_steps(betas, bits):
    params, grads = make(7)
    for at in (0, 5, 100000):
        opt = ct.AdamW([p.clone() for p in params], lr=1e-3, betas=betas, bits=bits, eps=1e-6, weight_decay=0.1)
        opt.steps = at
        old = held(opt)
        opt.step(grads)
        check_step(opt, old, grads, 1.0, at + 1, 1e-3, "step %d" % at)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """More than one table of them, parameters without a gradient in between:
    those keep every bit."""
    sizes = [[1 + (37 * i) % 700] for i in range(1100)]
    params, grads = make(50, sizes)
    for i in range(0, 1100, 7):
        grads[i] = None
    opt = ct.AdamW(params, lr=1e-2, bits=bits, seed=5)
    for state in (opt.exp_avg.view(torch.uint8), opt.exp_avg_sq.view(torch.uint8)):
        state.copy_(torch.randint(0, 60, (state.numel(),), device="cuda"))
    if bits == 8:
        opt.exp_avg_scale.fill_(1e-3), opt.exp_avg_sq_scale.fill_(1e-2)
    before = [p.clone() for p in params], opt.exp_avg.view(torch.uint8).clone(), opt.master.clone()
    old = held(opt)
    opt.step(grads)
    check_step(opt, old, grads, 1.0, 1, 1e-2, "many")
    for i in range(0, 1100, 7):
        assert torch.equal(params[i], before[0][i])
        assert torch.equal(spread(opt, opt.exp_avg, i).view(torch.uint8),
                           spread(opt, before[1].view(opt.exp_avg.dtype), i).view(torch.uint8))
        if params[i].dtype != torch.float32:
            assert torch.equal(spread(opt, opt.master, i, True), spread(opt, before[2], i, True))


def everything(opt):
    return [t.clone() for t in list(opt.params) + [opt.exp_avg.view(torch.uint8), opt.exp_avg_sq.view(torch.uint8),
                                                  opt.exp_avg_scale, opt.exp_avg_sq_scale, opt.master] if t is not None]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.numel() else x, y.view(torch.uint8) if y.numel() else y)
               for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [32, 8])
def test_scaled_and_skipped(bits):
    params, grads = make(60)
    opt = ct.AdamW(params, lr=1e-2, bits=bits)
    old = held(opt)
    opt.step(grads, grad_scale=torch.tensor(0.125, device="cuda"))
    check_step(opt, old, grads, 0.125, 1, 1e-2, "scaled")
    kept = everything(opt)
    for bad in (0.0, -1.0, float("nan"), float("inf"), -float("inf")):
        opt.step(grads, grad_scale=torch.tensor([bad], device="cuda"))
        assert same(everything(opt), kept), bad
    assert opt.steps == 6


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_are_not_finite(bits):
    """They stay in their element, with 8-bit states in their block."""
    params, grads = make(70, kinds=[torch.float32])
    opt, plain = (ct.AdamW([p.clone() for p in params], lr=1e-2, bits=bits) for _ in range(2))
    plain.step(grads)
    grads[11] = grads[11].clone()
    grads[11].view(-1)[300] = float("nan")
    grads[11].view(-1)[5000] = float("inf")
    opt.step(grads)
    for i, (p, q) in enumerate(zip(opt.params, plain.params)):
        odd = torch.zeros(p.numel(), dtype=torch.bool, device="cuda")
        if i == 11:
            odd[300] = odd[5000] = True
        assert torch.equal(p.view(-1)[~odd], q.view(-1)[~odd]) and bool(p.view(-1)[odd].isnan().all())
    m = spread(opt, opt.exp_avg if bits == 32 else
               opt.exp_avg.float() * opt.exp_avg_scale.repeat_interleave(BLOCK), 11)
    bad = ~m.isfinite()
    if bits == 32:
        assert int(bad.sum()) == 2 and bool(bad[300]) and bool(bad[5000])
    else:
        assert bool(bad[256:512].all()) and bool(bad[19 * 256:20 * 256].all()) and int(bad.sum()) == 512


def test_random_rounding_is_right_on_average():
    """States that decay by 1e-4 a step, a thousandth of a code's step, beside
    one in each block that stays: they decay at that rate."""
    n = 1 << 20
    p = torch.zeros(n, device="cuda")
    opt = ct.AdamW([p], lr=0.0, betas=(1 - 1e-4, 1 - 2e-4), bits=8, seed=77, weight_decay=0.0)
    values = 0.1 + 0.9 * torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    values.view(-1, BLOCK)[:, 0] = 1.0
    opt.exp_avg.copy_(values * 448), opt.exp_avg_sq.copy_(values * 448)
    opt.exp_avg_scale.fill_(1 / 448), opt.exp_avg_sq_scale.fill_(1 / 448)

    def mean(codes, scale):
        return float((codes.float().view(-1, BLOCK)[:, 1:] * scale[:, None]).double().mean())

    start = mean(opt.exp_avg, opt.exp_avg_scale)
    assert start == mean(opt.exp_avg_sq, opt.exp_avg_sq_scale)
    g = torch.zeros(n, device="cuda")
    g.view(-1, BLOCK)[:, 0] = 1.0
    for _ in range(50):
        opt.step([g])
    # m falls by (1 - 1e-4)^50, the root by the square root of (1 - 2e-4)^50.  An update moves a value by a step d
    # (at most 2^-3) with probability 1e-4 value / d: a variance below 1e-4 * 2^-3, and 50 * 2^20 of them are
    # independent, so six deviations of the mean are 1.5e-4.  Parts of a step below 2^-16 are dropped: at most
    # 50 * 2^-16 * 2^-3 = 1e-4.  Both against a mean of 0.55.
    for c, s in ((opt.exp_avg, opt.exp_avg_scale), (opt.exp_avg_sq, opt.exp_avg_sq_scale)):
        assert abs(mean(c, s) / start - (1 - 1e-4) ** 50) < 5e-4


@pytest.mark.parametrize("bits", [32, 8])
def test_device_step_and_rate_in_graphs(bits):
    """Step, rate and scale read on the device; two captured optimizers replayed
    at the same time; a captured step without a device step is refused."""
    lr, step, scale = (torch.tensor([v], device="cuda") for v in (5e-3, 1.0, 0.5))
    step = step.long()
    work = []
    for k in range(2):
        params, grads = make(80 + k, kinds=[torch.float32, torch.bfloat16])
        work.append((ct.AdamW(params, lr=lr, bits=bits, seed=k), grads))
    opt, grads = work[0]
    for t in (1, 2):
        old = held(opt)
        step.fill_(t)
        opt.step(grads, step=step, grad_scale=scale)
        check_step(opt, old, grads, 0.5, t, 5e-3, "device step %d" % t)
    assert opt.steps == 0
    graphs = []
    for opt, grads in work:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            with pytest.raises(ValueError, match="captured"):
                opt.step(grads)
            opt.step(grads, step=step, grad_scale=scale)
        graphs.append(g)
    for t in (3, 4):
        step.fill_(t), lr.fill_(1e-2 / t), scale.fill_(0.25 * t)
        old = [held(opt) for opt, _ in work]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (opt, grads), o in zip(work, old):
            check_step(opt, o, grads, 0.25 * t, t, float(lr), "replay %d" % t)


def test_gradients_of_other_layouts_and_streams():
    params, grads = make(90, [[30, 40], [7, 9, 11]], [torch.float32])
    turned = [g.transpose(0, 1).contiguous().transpose(0, 1) for g in grads]
    assert not turned[0].is_contiguous()
    a, b = (ct.AdamW([p.clone() for p in params], lr=1e-2) for _ in range(2))
    a.step(grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.step(turned, stream=side)
    side.synchronize()
    assert same(everything(a), everything(b))
    p = torch.nn.Parameter(params[0].clone())      # a leaf under grad mode, and a value that backward still needs
    opt = ct.AdamW([p], lr=1e-2)
    loss = (p * p).sum()
    opt.step([grads[0]])
    assert torch.equal(p, a.params[0])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_parameters_that_move():
    params, grads = make(95, [[40], [50]], [torch.float32])
    opt = ct.AdamW(params, lr=1e-2)
    opt.step(grads)
    want = [p.clone() for p in params]
    moved = params[0].clone()
    opt.params[0].data = moved
    opt.step(grads)
    assert opt.params[0].data_ptr() == moved.data_ptr() and not torch.equal(moved, want[0])
    opt.params[1].data = moved[:0].new_zeros(50)[:49]
    with pytest.raises(ValueError, match="parameter 1"):
        opt.step(grads)
    opt.params[1].data = moved.new_empty(0).set_(moved.untyped_storage(), 0, (40,), (1,))
    with pytest.raises(ValueError, match="parameter 1"):
        opt.step(grads)


def test_past_32_bits():
    """More than 2^31 elements: the last ones move as they do alone."""
    n, tail = (1 << 31) + 300, 700
    p = torch.zeros(n, dtype=torch.float16, device="cuda")
    g = torch.zeros(n, dtype=torch.float16, device="cuda")
    p[-tail:], g[-tail:] = normal([tail], 1, torch.float16), normal([tail], 2, torch.float16)
    small, gs = p[-tail:].clone(), g[-tail:].clone()
    a, b = ct.AdamW([p], lr=1e-2, bits=8), ct.AdamW([small], lr=1e-2, bits=8)
    norm, _ = ct.grad_norm([g])
    a.step([g]), b.step([gs])
    assert torch.equal(p[-tail:], small) and not p[:-tail].any()
    assert abs(float(norm) / float(torch.linalg.vector_norm(gs.double())) - 1) < 8 * ref.U
    assert not a.exp_avg[:1 << 30].view(torch.uint8).any()


@pytest.mark.parametrize("moved", [0, 1, 4])
def test_grad_norm(moved):
    for sizes in (SIZES, [[1]], [[0], [0]], [[5000000], [3]], [[1 + (37 * i) % 700] for i in range(1100)]):
        _, grads = make(110, sizes, moved=moved)
        want = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
        for most in (None, 0.5 * want + 1e-9, 2 * want + 1e-9):
            norm, scale = ct.grad_norm(grads, most)
            # 64 bits, and the result's rounding
            assert abs(float(norm) - want) <= 1.01 * ref.U * want
            clip = 1.0 if most is None or want <= most else most / want
            assert abs(float(scale) - clip) <= 1.01 * ref.U
        assert all(torch.equal(a, b) for a, b in zip(ct.grad_norm(grads, 1.0), ct.grad_norm(grads + [None], 1.0)))
    turned = normal([50, 60], 3).t()
    assert torch.equal(ct.grad_norm([turned])[0], ct.grad_norm([turned.contiguous()])[0])
    for bad in (float("nan"), float("inf"), -float("inf")):
        grads[3].view(-1)[0] = bad
        norm, scale = ct.grad_norm(grads, 1.0)
        assert not math.isfinite(float(norm)) and float(scale) == 0.0
    norm, scale = ct.grad_norm([torch.full((9,), 1e30, device="cuda")], 1.0)       # squares that fp32 does not hold
    assert abs(float(norm) / 3e30 - 1) < 4 * ref.U and abs(float(scale) * 3e30 - 1) < 4 * ref.U
    norm, scale = ct.grad_norm([torch.full((9,), 3e38, device="cuda")], 1.0)       # nor their norm
    assert math.isinf(float(norm)) and float(scale) == 0.0
    norm, scale = ct.grad_norm([torch.full((9,), 1e-30, device="cuda")], 1.0)
    assert abs(float(norm) / 3e-30 - 1) < 4 * ref.U and float(scale) == 1.0
    zero, scale = ct.grad_norm([torch.zeros(5, device="cuda")], 1.0)
    assert float(zero) == 0 and float(scale) == 1


# ---- together ------------------------------------------------------------------------

def train_block(x, res, weight, target, sections, opt, step):
    """Norm of the residual stream, positions, a loss against `target` (its
    gradient is -target), and back; one update with clipping."""
    n, h, w, c = x.shape
    y, s, rstd = ct.rms_norm_nhwc(x, weight, residual=res, return_rstd=True)
    turned = ct.rotary_nhwc(y.view(n, h, w, 4, c // 4), sections, pairs="halves")
    dy = ct.rotary_nhwc_backward(-target, sections, pairs="halves").view(x.shape)
    dx, dweight = ct.rms_norm_nhwc_backward(dy, s, rstd, weight)
    norm, scale = ct.grad_norm([dweight], 0.5)
    opt.step([dweight], grad_scale=scale, step=step)
    return turned, dx, dweight, norm


def test_training_step_together():
    """Forward, backward, clip and update through the framework's calls, eager
    and as one captured graph replayed; gradients against autograd in fp64."""
    sections = [16, 8]
    x, res = normal([2, 5, 6, 128], 1, torch.bfloat16), normal([2, 5, 6, 128], 2, torch.bfloat16)
    target = normal([2, 5, 6, 4, 32], 3, torch.bfloat16)
    w0 = 1 + 0.1 * normal([128], 4)
    x64, w64 = x.double().requires_grad_(), w0.double().requires_grad_()
    y64, _, _ = ref.rms_forward(x64, res.double(), w64, 1e-6)
    angles = ref.rotary_angles(ref.grid_positions([5, 6], "cuda"), sections, 10000.0)
    turned64 = ref.rotary(y64.view(2, 5, 6, 4, 32), angles, "halves").reshape(-1)
    (-(turned64 * target.double().reshape(-1)).sum()).backward()
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    runs = []
    for captured in (False, True):
        w = w0.clone()
        opt = ct.AdamW([w], lr=1e-2)
        step.fill_(1)
        if captured:
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                out = train_block(x, res, w, target, sections, opt, step)
                step.add_(1)
            for k in range(3):
                g.replay()
                if k == 0:
                    first = [t.clone() for t in out]
        else:
            for k in range(3):
                out = train_block(x, res, w, target, sections, opt, step)
                step.add_(1)
                if k == 0:
                    first = [t.clone() for t in out]
        torch.cuda.synchronize()
        runs.append(first + [w, opt.exp_avg, opt.exp_avg_sq])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    turned, dx, dw, norm = runs[0][:4]
    # bf16 at each hand-over (y, the turn, its gradient, the sum that backward reads, dx): five roundings of 2^-8 of
    # values that a turn mixes in pairs; in the 2-norm at most 5 * 2^-8 * 1.5
    for got, want in ((turned.reshape(-1), turned64.detach()), (dx, x64.grad), (dw, w64.grad)):
        off = torch.linalg.vector_norm(got.double() - want) / torch.linalg.vector_norm(want)
        assert float(off) < 7.5 * 2.0 ** -8
    assert abs(float(norm) / float(torch.linalg.vector_norm(dw.double())) - 1) < 8 * ref.U


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_grad_norm_of_wide_ranges(dtype):
    """Sums of 16-bit squares over many orders, whole blocks and rests: to the
    rounding of the result."""
    g = normal([3 * 8192 + 77], 5) * torch.exp2(torch.linspace(-24, 12, 3 * 8192 + 77, device="cuda"))
    for scale in (1.0, 2.0 ** -100, 2.0 ** 90) if dtype == "bf16" else (1.0, 0.01):
        t = (g * scale).to(TYPES[dtype])
        norm, _ = ct.grad_norm([t, t[1:], t[:5]])
        want = float(torch.linalg.vector_norm(torch.cat((t, t[1:], t[:5])).double()))
        assert abs(float(norm) - want) <= 1.01 * ref.U * want
    bad = t.clone()
    bad[5000] = float("nan")
    assert math.isnan(float(ct.grad_norm([bad])[0]))


def test_restart():
    """States copied, or put in their place, go on as the ones they come from; changed settings take effect."""
    params, grads = make(120)
    a = ct.AdamW(params, lr=1e-2, bits=8, seed=3)
    a.step(grads)
    b = ct.AdamW([p.clone() for p in params], lr=1e-2, bits=8, seed=3)
    for name in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        getattr(b, name).copy_(getattr(a, name))
    b.master = a.master.clone()
    b.steps = a.steps
    for opt in (a, b):
        opt.step(grads)
        opt.betas, opt.eps = (0.5, 0.6), 1e-3
        opt.step(grads)
    assert same(everything(a), everything(b))
    c = ct.AdamW([p.clone() for p in params], lr=1e-2, bits=32)
    old = held(c)
    c.betas, c.eps = (0.5, 0.6), 1e-3
    c.step(grads)
    check_step(c, old, grads, 1.0, 1, 1e-2, "changed settings")
