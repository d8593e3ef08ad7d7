"""Plain fp64 forms of the group norm and of dropout, for the tests: written
from the definitions, sharing nothing with the library.

Rounding bounds: u = 2^-24 is half a step of fp32.  The library computes in
fp32 and rounds once, so an output may be off by half a step of its type plus
what the fp32 operations in front of it lose; ``forward_bound`` and
``backward_bounds`` add these up from the values themselves.
"""

import math

import numpy as np
import torch

U = 2.0 ** -24
# Length of the longest chain of additions behind one sum, which bounds its
# relative error against the sum of magnitudes: a thread's own values, the
# block's, then the parts of the image and the images.
CHAIN = 256
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}


def philox(counter, key):
    """Philox4x32-10 of Salmon et al. (2011): counter [n, 4], key [2] -> [n, 4]."""
    c = np.array(counter, dtype=np.uint64).reshape(-1, 4)
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[:, 0] * np.uint64(0xD2511F53), c[:, 2] * np.uint64(0xCD9E8D57)
        c = np.stack([(p1 >> np.uint64(32)) ^ c[:, 1] ^ np.uint64(k[0]), p1 & low,
                      (p0 >> np.uint64(32)) ^ c[:, 3] ^ np.uint64(k[1]), p0 & low], axis=1)
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c.astype(np.uint32)


def threshold(p):
    return math.floor(p * 65536 + 0.5)


def drop_scale(p):
    t = threshold(p)
    return 65536 / (65536 - t) if t < 65536 else 0.0


def keep_mask(n, p, seed, offset, first=0):
    """Whether elements first .. first+n-1 are kept (a bool array)."""
    b0, b1 = first // 8, (first + n + 7) // 8
    i = np.arange(b0, max(b1, b0), dtype=np.uint64)
    o = np.full_like(i, 1)
    c = np.stack([i & np.uint64(0xFFFFFFFF), i >> np.uint64(32), o * np.uint64(offset & 0xFFFFFFFF),
                  o * np.uint64(offset >> 32)], axis=1)
    w = philox(c, [seed & 0xFFFFFFFF, seed >> 32])
    v = np.stack([w & 0xFFFF, w >> 16], axis=2).reshape(-1)
    return v[first - 8 * b0: first - 8 * b0 + n] >= threshold(p)


def factor(shape, p, seed, offset):
    """0 where dropped, the scale where kept (fp64)."""
    n = math.prod(shape)
    m = torch.from_numpy(keep_mask(n, p, seed, offset)).view(shape)
    return m.double() * drop_scale(p)


def act(a, name):
    if name == "silu":
        return a * torch.sigmoid(a)
    if name == "gelu":
        return a * 0.5 * torch.special.erfc(-a / math.sqrt(2.0))
    return a.clamp(min=0) if name == "relu" else a


def act_slope(a, name):
    if name == "silu":
        s = torch.sigmoid(a)
        return s + a * s * (1 - s)
    if name == "gelu":
        return (0.5 * torch.special.erfc(-a / math.sqrt(2.0))
                + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi))
    return (a > 0).to(a.dtype) if name == "relu" else torch.ones_like(a)


def stats(x, groups, eps):
    n, c = x.shape[0], x.shape[-1]
    g = x.reshape(n, -1, groups, c // groups)
    mean = g.mean(dim=(1, 3))
    var = ((g - mean[:, None, :, None]) ** 2).mean(dim=(1, 3))
    return mean, 1 / torch.sqrt(var + eps)


def _spread(t, x, groups):
    """[N, G] -> broadcast over X's pixels and channels."""
    n, c = x.shape[0], x.shape[-1]
    return t.repeat_interleave(c // groups, dim=1).view([n] + [1] * (x.dim() - 2) + [c])


def forward(x, groups, weight, bias, eps, activation, f=1.0, mean_rstd=None):
    """x in fp64 -> y, mean, rstd, a."""
    mean, rstd = stats(x, groups, eps) if mean_rstd is None else mean_rstd
    h = (x - _spread(mean, x, groups)) * _spread(rstd, x, groups)
    a = h * weight + bias
    return act(a, activation) * f, mean, rstd, a


def backward(dy, x, mean, rstd, groups, weight, bias, activation, f=1.0):
    n, c = x.shape[0], x.shape[-1]
    rs = _spread(rstd, x, groups)
    h = (x - _spread(mean, x, groups)) * rs
    da = dy * f * act_slope(h * weight + bias, activation)
    axes = tuple(range(x.dim() - 1))
    dw, db = (da * h).sum(dim=axes), da.sum(dim=axes)
    dh = da * weight
    split = [n, -1, groups, c // groups]
    m0 = _spread(dh.reshape(split).mean(dim=(1, 3)), x, groups)
    m1 = _spread((dh * h).reshape(split).mean(dim=(1, 3)), x, groups)
    return rs * (dh - m0 - h * m1), dw, db


def _a_error(x, mean, rstd, groups, weight, bias, own_stats):
    """How far a may be off in fp32.  (x - mean) loses half a step of the
    difference, the products and the sum one each; with the library's own
    statistics the mean is off by CHAIN u of the values' distance from any of
    them plus two steps of itself, and rstd by half of var's CHAIN u, that is
    CHAIN / 2 u of itself."""
    mc, rc = _spread(mean, x, groups), _spread(rstd, x, groups)
    h = ((x - mc) * rc).abs()
    e = 6 * h * weight.abs() + 2 * bias.abs()
    if own_stats:
        e = e + (CHAIN / 2 * h + CHAIN * 2 + 4 * mc.abs() * rc) * weight.abs()
    return U * e


def forward_bound(x, mean, rstd, groups, weight, bias, a, y, dtype, scale, own_stats=True):
    """The slope of each activation is below 1.2; exp and the division of
    silu, and erf, are good to 8 steps of their values."""
    e = 1.2 * _a_error(x, mean, rstd, groups, weight, bias, own_stats) + 8 * U * a.abs()
    return 1.01 * (HALF[dtype] * y.abs() + scale * e) + TINY[dtype]


def backward_bounds(dy, x, mean, rstd, groups, weight, bias, activation, f, dtype, pdtype, dx, dw, db):
    """(dx, dw, db) bounds with the statistics given (no error of their own).
    The slopes' own slope is below 1 (relu: 0 away from the jump, which the
    tests keep clear of), and a slope is good to 16 steps of 1 + |a|."""
    n, c = x.shape[0], x.shape[-1]
    rs = _spread(rstd, x, groups)
    h = (x - _spread(mean, x, groups)) * rs
    a = h * weight + bias
    g = (dy * f).abs()
    eda = g * (_a_error(x, mean, rstd, groups, weight, bias, False) + 16 * U * (1 + a.abs()))
    da = g * act_slope(a, activation).abs()
    axes = tuple(range(x.dim() - 1))
    split = [n, -1, groups, c // groups]

    def mean_of(t):
        return _spread(t.reshape(split).mean(dim=(1, 3)), x, groups)

    wa, ha = weight.abs(), h.abs()
    em0 = mean_of(wa * (eda + CHAIN * U * da))
    em1 = mean_of(wa * ha * (eda + CHAIN * U * da))
    terms = wa * da + mean_of(wa * da) + ha * mean_of(wa * da * ha)
    edx = rs * (wa * eda + em0 + ha * em1 + 8 * U * terms)
    bdx = 1.01 * (HALF[dtype] * dx.abs() + edx) + TINY[dtype]
    bdw = 1.01 * (HALF[pdtype] * dw.abs() + (ha * (eda + CHAIN * U * da)).sum(dim=axes)) + TINY[pdtype]
    bdb = 1.01 * (HALF[pdtype] * db.abs() + (eda + CHAIN * U * da).sum(dim=axes)) + TINY[pdtype]
    return bdx, bdw, bdb
