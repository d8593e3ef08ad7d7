"""Plain fp64 forms of the root-mean-square norm, of rotary positions and of
AdamW, for the tests: written from the definitions, sharing nothing with the
library.  They run wherever their inputs lie.

Rounding bounds: u = 2^-24 is half a step of fp32.  The library computes in
fp32 and rounds once; CHAIN bounds the relative error of a sum against the sum
of its terms' magnitudes in units of u (a thread's own terms, lanes, warps,
rows of a block, parts, one after the other).
"""

import torch

U = 2.0 ** -24
CHAIN = 256
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}
LEAST_SCALE = 2.0 ** -126


def check(got, want, bound, where):
    """Elementwise |got - want| <= bound; NaN and infinities have to agree."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, "%s: shape %s, not %s" % (where, list(got.shape), list(want.shape))
    err = (got - want).abs()
    bad = ~(err <= bound) & ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its bound" % (
        where, int(bad.sum()), bad.numel(), float((err / bound)[bad].nan_to_num(float("inf")).max()))


# ---- root-mean-square norm ----------------------------------------------------

def rms_forward(x, residual, weight, eps):
    """fp64 -> y, h, rstd."""
    h = x if residual is None else x + residual
    rstd = 1 / torch.sqrt((h * h).mean(dim=-1) + eps)
    return h * rstd[..., None] * weight, h, rstd


def rms_bounds(y, h, rstd, dtype):
    """(y, sum, rstd): the squares' sum is good to CHAIN u of itself, and half
    of that enters rstd; a square root, a quotient, h, and two products lose
    half a step each."""
    return (1.01 * (HALF[dtype] + (CHAIN / 2 + 8) * U) * y.abs() + TINY[dtype],
            1.01 * (HALF[dtype] + U) * h.abs() + TINY[dtype], (CHAIN / 2 + 6) * U * rstd)


def rms_backward(dy, h, rstd, weight, dsum):
    """fp64 -> dx, dweight."""
    hat = h * rstd[..., None]
    t = dy * weight
    dx = rstd[..., None] * (t - hat * (t * hat).mean(dim=-1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum
    return dx, (dy * hat).sum(dim=tuple(range(dy.dim() - 1)))


def rms_backward_bounds(dy, h, rstd, weight, dsum, dx, dw, dtype, pdtype):
    hat = (h * rstd[..., None]).abs()
    t = (dy * weight).abs()
    e = rstd[..., None] * (6 * t + (CHAIN + 8) * hat * (t * hat).mean(dim=-1, keepdim=True))
    if dsum is not None:
        e = e + 2 * dsum.abs()
    terms = (dy.abs() * hat).sum(dim=tuple(range(dy.dim() - 1)))
    return (1.01 * (HALF[dtype] * dx.abs() + U * e) + TINY[dtype],
            1.01 * (HALF[pdtype] * dw.abs() + (CHAIN + 4) * U * terms) + TINY[pdtype])


def block_scales(y, block):
    """The scales of y's blocks (0: whole rows), without their last axis then."""
    c = y.shape[-1]
    width = block or c
    scale = torch.stack([y[..., k:k + width].abs().amax(dim=-1) for k in range(0, c, width)], dim=-1) / 448
    return scale.clamp(min=LEAST_SCALE) if block else scale[..., 0].clamp(min=LEAST_SCALE)


def spread_scales(scale, block, c):
    """One scale for each of c channels."""
    return scale.repeat_interleave(block, dim=-1)[..., :c] if block else scale[..., None].expand(*scale.shape, c)


def e4m3_bound(v, steps=0.5):
    """How far a code may lie from v: `steps` of the grid there, 2^-3 of the
    power of two below v, 2^-9 at the least; and v's own error."""
    return steps * torch.maximum(v.abs() * 2.0 ** -3, torch.full_like(v, 2.0 ** -9)) + (CHAIN + 16) * U * v.abs()


# ---- rotary positions ---------------------------------------------------------

def rotary_angles(at, sections, base):
    """Positions [.., axes] in fp64 -> angles [.., pairs]."""
    freq = [base ** (-torch.arange(0, d, 2, dtype=torch.float64, device=at.device) / d) for d in sections]
    return torch.cat([at[..., a, None] * f for a, f in enumerate(freq)], dim=-1)


def grid_positions(dims, device="cpu"):
    return torch.stack(torch.meshgrid(*[torch.arange(d, device=device, dtype=torch.float64) for d in dims],
                                      indexing="ij"), dim=-1)


def rotary(x, angles, pairs):
    """x [.., heads, dim] in fp64, angles [.., pairs]."""
    half = angles.shape[-1]
    c, s = torch.cos(angles)[..., None, :], torch.sin(angles)[..., None, :]
    i = torch.arange(half, device=x.device)
    i, k = (i, i + half) if pairs == "halves" else (2 * i, 2 * i + 1)
    y = x.clone()
    y[..., i], y[..., k] = x[..., i] * c - x[..., k] * s, x[..., i] * s + x[..., k] * c
    return y


def rotary_bound(x, y, angles, pairs, dtype):
    """The angle is good to 2^-52 of itself (the frequency, the position's
    product), and its fraction of half a turn to half a step of fp32; sincospi
    to 4 steps; two products and a sum lose half a step of the terms each."""
    half = angles.shape[-1]
    off = (angles.abs() * 2.0 ** -51 + 12 * U)[..., None, :]
    i = torch.arange(half, device=x.device)
    i, k = (i, i + half) if pairs == "halves" else (2 * i, 2 * i + 1)
    e = torch.zeros_like(x)
    both = (x[..., i].abs() + x[..., k].abs()) * off
    e[..., i], e[..., k] = both, both
    return 1.01 * (HALF[dtype] * y.abs() + e) + torch.where(e > 0, TINY[dtype], 0.0)


# ---- AdamW --------------------------------------------------------------------

def adamw(p, g, m, v, lr, betas, eps, decay, step):
    """fp64 -> p, m, v and the update by m / sqrt(v) alone."""
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    update = lr * (m / (1 - betas[0] ** step)) / (torch.sqrt(v / (1 - betas[1] ** step)) + eps)
    return p - lr * decay * p - update, m, v, update


def adamw_bounds(p, g, m, v, new, lr, betas, eps, decay, step):
    """(p, m, v) bounds of the fp32 update from the old p, m, v.  m: the
    gradient's scale, both factors, products and the sum.  v the same with the
    square.  The update: m's error over the same root, and sqrt (2^-23), the
    quotient (4 u), the corrections (expm1 and its argument, or rounded once),
    eps and products: 40 u in all."""
    pn, mn, vn, update = new
    em = 6 * U * (betas[0] * m.abs() + (1 - betas[0]) * g.abs())
    ev = 8 * U * vn
    slope = (lr / (1 - betas[0] ** step)) / (torch.sqrt(vn / (1 - betas[1] ** step)) + eps)
    ep = em * slope + 40 * U * update.abs() + 4 * U * lr * decay * p.abs()
    return 1.01 * (U * pn.abs() + ep) + 2.0 ** -126, em + 2.0 ** -126, ev + 2.0 ** -126


def code_steps(x):
    """The grid below |x| (fp64, at most 448): the code below and the distance to the next."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))) * 2.0 ** -3
    return torch.floor(a / step) * step, step


def random_codes(x, r):
    """Where x lies between two codes and r's 16 bits choose the upper one ->
    the code (fp64), and whether the choice is one that rounding can turn: x is
    good to some 60 u, 2^4 steps of the grid at most, that is 4 of 2^16."""
    low, step = code_steps(x)
    part = (x.abs() - low) / step * 65536 + r
    code = torch.where(part >= 65536, low + step, low).clamp(max=448.0)
    close = ((part - 65536).abs() < 6) | (part < r + 6) | (part > r + 65530)
    return torch.copysign(code, x), close
