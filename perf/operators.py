"""The operators around a transposed convolution in a decoder, as cases that can be timed: channels-last group norm
with its activation and dropout (forward, backward, both), and dropout with a residual.

The plain forms here state what each operator computes; the framework's own calls are made where ``own`` is true.
"""

import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = {"fp16": 2, "bf16": 2, "fp32": 4}
EPS = 1e-5


def _gn(name, way, dtype, n, s, c, groups, act, p=0.0):
    return {"name": name, "op": "group_norm", "way": way, "dtype": dtype, "n": n, "s": s, "c": c, "groups": groups,
            "act": act, "p": p}


def _drop(name, way, dtype, n, c, p, rng=False):
    return {"name": name, "op": "dropout", "way": way, "dtype": dtype, "n": n, "c": c, "p": p, "rng": rng}


def listed():
    return [
        # one image at a decoder's lowest resolution, answered alone: latency
        _gn("gn_one_8x8x256_fp16", "forward", "fp16", 1, 8 * 8, 256, 32, "silu"),
        # the output of the 2-D decoder upsample (X[8,256,64,64] -> [8,128,128,128]), channels last
        _gn("gn_decoder_128x128x128_fp16", "forward", "fp16", 8, 128 * 128, 128, 32, "silu"),
        # the output of the 3-D volumetric upsample: few channels, long images
        _gn("gn_volume_64cubed_x32_fp16", "forward", "fp16", 2, 64 * 64 * 64, 32, 8, "relu"),
        # the output of the 1-D fp32 vocoder upsample: the largest forward pass
        _gn("gn_vocoder_16384x256_fp32", "forward", "fp32", 16, 16384, 256, 16, "gelu"),
        # sizes that fit no vector: 57 x 91 pixels of 30 channels
        _gn("gn_odd_57x91x30_bf16", "forward", "bf16", 3, 57 * 91, 30, 5, "gelu"),
        # the backward pass at the grouped 2-D upsample's output (16 images of 112 x 112, 512 channels): the largest
        _gn("gn_back_112x112x512_fp16", "backward", "fp16", 16, 112 * 112, 512, 32, "silu"),
        # the backward pass of a small odd batch, single precision
        _gn("gn_back_13x17x65_fp32", "backward", "fp32", 2, 13 * 17, 65, 13, "gelu"),
        # a training step through a decoder's inner block: forward with dropout, then backward
        _gn("gn_train_32x32x512_bf16", "train", "bf16", 16, 32 * 32, 512, 32, "silu", 0.1),
        # dropout of a decoder block's output, added to the block's input
        _drop("drop_add_decoder_bf16", "residual", "bf16", 8 * 128 * 128, 256, 0.1),
        # dropout of a few odd rows: latency
        _drop("drop_small_31x33_fp16", "forward", "fp16", 31, 33, 0.25),
        # the gradient through dropout in a replayable step: seed and offset lie on the device
        _drop("drop_back_odd_fp32", "backward", "fp32", 57 * 91 * 3, 511, 0.5, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["fp16", "bf16", "fp32"])
    if rng.random() < 0.3:
        way = rng.choice(["forward", "residual", "backward"])
        c = _log(rng, 1, 2000)
        n = max(1, _log(rng, 100, 32e6) // c)
        return _drop("", way, dtype, n, c, round(rng.uniform(0.02, 0.9), 3), rng.random() < 0.5)
    groups = rng.choice([1, 2, 3, 5, 8, 16, 32, 32, 32])
    c = groups * max(1, _log(rng, 8, 1024) // groups)
    n = _log(rng, 1, 32)
    s = max(-(-64 // (c // groups)), _log(rng, 16, 24e6) // (n * c))  # 64 values in a group at least
    way = rng.choice(["forward", "backward", "train"])
    # relu's derivative jumps at 0, where two right answers may fall on either side: forward only
    act = rng.choice(["silu", "silu", "gelu", "identity"] + (["relu"] if way == "forward" else []))
    p = round(rng.uniform(0.02, 0.5), 3) if rng.random() < 0.4 else 0.0
    return _gn("", way, dtype, n, s, c, groups, act, p)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    st = {"case": case, "seed": (seed * 0x9E3779B97F4A7C15) % (1 << 63), "offset": seed % 1000}
    if case["op"] == "dropout":
        st["x"] = normal(case["n"], case["c"]).to(t)
        if case["way"] == "residual":
            st["residual"] = normal(case["n"], case["c"]).to(t)
        st["rng"] = torch.tensor([st["seed"], st["offset"]], dtype=torch.int64, device="cuda") if case["rng"] else None
        return st
    n, s, c = case["n"], case["s"], case["c"]
    # a convolution's outputs: every channel with a scale and a mean of its own
    st["x"] = (normal(n, s, c) * (0.5 + normal(c).abs()) + 2.0 * normal(c)).to(t)
    st["weight"], st["bias"] = 1.0 + 0.2 * normal(c), 0.2 * normal(c)
    if case["way"] != "forward":
        st["dy"] = (0.1 * normal(n, s, c)).to(t)
    if case["way"] == "backward":  # what the forward pass left
        xg = st["x"].double().view(n, s, case["groups"], -1)
        var, mean = torch.var_mean(xg, dim=(1, 3), correction=0)
        st["mean"], st["rstd"] = mean.float(), (1.0 / torch.sqrt(var + EPS)).float()
    return st


# ---- the plain forms ----------------------------------------------------------------------------------------------

LOW = 0xFFFFFFFF


def _kept(n, st, p):
    """Which of n elements stay: element i takes 16-bit value i % 8 of Philox4x32-10 (Salmon et al., 2011) at counter
    (i // 8, offset) under the key seed, and stays where that is at least p * 65536 (rounded)."""
    if st.get("rng") is not None:
        seed, offset = st["rng"][0], st["rng"][1]
    else:
        seed, offset = st["seed"], st["offset"]
    i = torch.arange((n + 7) // 8, device="cuda", dtype=torch.int64)
    zero = torch.zeros_like(i)
    c0, c1, c2, c3 = i & LOW, i >> 32, zero + (offset & LOW), zero + ((offset >> 32) & LOW)
    k0, k1 = seed & LOW, (seed >> 32) & LOW
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & LOW) ^ c1 ^ k0, p1 & LOW, ((p0 >> 32) & LOW) ^ c3 ^ k1, p0 & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    words = torch.stack((c0, c1, c2, c3), dim=1)
    return torch.stack((words & 0xFFFF, words >> 16), dim=2).reshape(-1)[:n] >= _threshold(p)


def _threshold(p):
    return math.floor(p * 65536 + 0.5)


def _drop_plain(v, st, p):
    """v where it stays, scaled so that the expectation is v; zero elsewhere."""
    t = _threshold(p)
    if t == 0:
        return v
    keep = _kept(v.numel(), st, p).view(v.shape)
    return torch.where(keep, v * (65536 / (65536 - t) if t < 65536 else 0.0), torch.zeros_like(v))


def _act(a, act):
    if act == "silu":
        return a / (1 + torch.exp(-a))
    if act == "gelu":
        return 0.5 * a * (1 + torch.erf(a * math.sqrt(0.5)))
    return torch.clamp(a, min=0) if act == "relu" else a


def _act_slope(a, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-a))
        return s * (1 + a * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(a * math.sqrt(0.5))) + a * torch.exp(-0.5 * a * a) * (1 / math.sqrt(2 * math.pi))
    return (a > 0).to(a.dtype) if act == "relu" else torch.ones_like(a)


def _forward_plain(st):
    c = st["case"]
    x = st["x"].float().view(c["n"], c["s"], c["groups"], -1)
    mean = x.mean(dim=(1, 3), keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(dim=(1, 3), keepdim=True) + EPS)
    a = (d * rstd).view(st["x"].shape) * st["weight"] + st["bias"]
    y = _drop_plain(_act(a, c["act"]), st, c["p"])
    return y.to(st["x"].dtype), mean.view(c["n"], -1), rstd.view(c["n"], -1)


def _backward_plain(st, mean, rstd):
    c = st["case"]
    split = (c["n"], c["s"], c["groups"], -1)
    rs = rstd.view(c["n"], 1, -1, 1)
    hat = (st["x"].float().view(split) - mean.view(c["n"], 1, -1, 1)) * rs
    a = hat.view(st["x"].shape) * st["weight"] + st["bias"]
    da = _drop_plain(st["dy"].float(), st, c["p"]) * _act_slope(a, c["act"])
    dweight, dbias = (da * hat.view(a.shape)).sum(dim=(0, 1)), da.sum(dim=(0, 1))
    dh = (da * st["weight"]).view(split)
    m0, m1 = dh.mean(dim=(1, 3), keepdim=True), (dh * hat).mean(dim=(1, 3), keepdim=True)
    return ((dh - m0 - hat * m1) * rs).view(a.shape).to(st["x"].dtype), dweight, dbias


def _run_plain(st):
    c = st["case"]
    if c["op"] == "dropout":
        y = _drop_plain(st["x"].float(), st, c["p"])
        return (y + st["residual"].float() if c["way"] == "residual" else y).to(st["x"].dtype)
    if c["way"] == "backward":
        return _backward_plain(st, st["mean"], st["rstd"])
    y, mean, rstd = _forward_plain(st)
    return (y, mean, rstd) + (_backward_plain(st, mean, rstd) if c["way"] == "train" else ())


# ---- the framework's calls ----------------------------------------------------------------------------------------

def _run_own(st):
    from transposed_convolution_02_b200 import ct

    c = st["case"]
    if c["op"] == "dropout":
        how = {"rng": st["rng"]} if c["rng"] else {"seed": st["seed"], "offset": st["offset"]}
        if c["way"] == "backward":
            return ct.dropout_backward(st["x"], c["p"], **how)
        return ct.dropout(st["x"], c["p"], residual=st.get("residual"), **how)
    how = {"activation": c["act"], "p": c["p"], "seed": st["seed"], "offset": st["offset"]}
    if c["way"] == "backward":
        return ct.group_norm_nhwc_backward(st["dy"], st["x"], st["mean"], st["rstd"], c["groups"], st["weight"],
                                           st["bias"], **how)
    y, mean, rstd = ct.group_norm_nhwc(st["x"], c["groups"], st["weight"], st["bias"], eps=EPS, return_stats=True,
                                       **how)
    if c["way"] == "forward":
        return y, mean, rstd
    return (y, mean, rstd) + tuple(ct.group_norm_nhwc_backward(st["dy"], st["x"], mean, rstd, c["groups"],
                                                               st["weight"], st["bias"], **how))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    """Every input read once, every output written once; the operations of the formulas, and 80 for eight elements'
    random values."""
    size = SIZES[case["dtype"]]
    if case["op"] == "dropout":
        e = case["n"] * case["c"]
        return {"bytes": e * size * (3 if case["way"] == "residual" else 2), "flops": 12 * e}
    e = case["n"] * case["s"] * case["c"]
    tensors, ops = {"forward": (2, 12), "backward": (3, 24), "train": (4, 36)}[case["way"]]
    params = 2 if case["way"] == "forward" else 4
    return {"bytes": e * size * tensors + 4 * (params * case["c"] + 2 * case["n"] * case["groups"]),
            "flops": (ops + (10 * tensors // 2 if case["p"] else 0)) * e}


# ---- the definition in 64 bits ------------------------------------------------------------------------------------

def _mul32(a, m):
    """(high, low) 32 bits of a * m, from 16-bit parts."""
    al, ah, ml, mh = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    mid = ah * ml + ((al * ml) >> 16)
    mid2 = al * mh + (mid & 0xFFFF)
    return ah * mh + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((al * ml) & 0xFFFF)


def _mask_exact(count, seed, offset, p):
    blocks = -(-count // 8)
    at = torch.arange(blocks, device="cuda")
    state = [at % 2 ** 32, torch.div(at, 2 ** 32, rounding_mode="floor"), torch.full_like(at, offset % 2 ** 32),
             torch.full_like(at, offset // 2 ** 32)]
    for r in range(10):
        key = [(seed + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
        h0, l0 = _mul32(state[0], 0xD2511F53)
        h1, l1 = _mul32(state[2], 0xCD9E8D57)
        state = [h1 ^ state[1] ^ key[0], l1, h0 ^ state[3] ^ key[1], l0]
    values = torch.empty(blocks, 8, device="cuda", dtype=torch.int64)
    for k in range(8):
        values[:, k] = (state[k // 2] >> (16 * (k % 2))) % 65536
    cut = int(p * 65536 + 0.5)
    factor = 65536.0 / (65536 - cut) if cut < 65536 else 0.0
    return (values.flatten()[:count] >= cut).double() * factor


def exact(case, seed):
    st = prepare(case, seed)
    x = st["x"].double()
    m = _mask_exact(x.numel(), st["seed"], st["offset"], case["p"]).view(x.shape) if case["p"] else 1.0
    if case["op"] == "dropout":
        return m * x + st["residual"].double() if case["way"] == "residual" else m * x
    n, s, c, k = case["n"], case["s"], case["c"], case["groups"]
    each = c // k
    w, b = st["weight"].double(), st["bias"].double()
    # per channel first, then over the channels of a group
    if case["way"] == "backward":
        mean, rstd = st["mean"].double(), st["rstd"].double()
    else:
        of_channel = x.sum(1) / s
        mean = of_channel.view(n, k, each).sum(2) / each
        off = x - mean.repeat_interleave(each, 1)[:, None]
        rstd = ((off ** 2).sum(1).view(n, k, each).sum(2) / (each * s) + EPS) ** -0.5
        del off
    mc, rc = mean.repeat_interleave(each, 1)[:, None], rstd.repeat_interleave(each, 1)[:, None]
    h = (x - mc) * rc
    del x
    a = h * w + b
    if case["act"] == "silu":
        value, slope = a * torch.sigmoid(a), torch.sigmoid(a) * (1 + a * torch.sigmoid(-a))
    elif case["act"] == "gelu":
        half = torch.special.erfc(-a / 2 ** 0.5) / 2
        value, slope = a * half, half + a * torch.exp(-a ** 2 / 2) / (2 * math.pi) ** 0.5
    elif case["act"] == "relu":
        value, slope = a.relu(), (a > 0).double()
    else:
        value, slope = a, 1.0
    if case["way"] == "forward":
        return value * m, mean, rstd
    u = st["dy"].double() * m * slope
    db, dw = u.sum(1), (u * h).sum(1)
    t0 = ((db * w).view(n, k, each).sum(2) / (each * s)).repeat_interleave(each, 1)[:, None]
    t1 = ((dw * w).view(n, k, each).sum(2) / (each * s)).repeat_interleave(each, 1)[:, None]
    grads = ((u * w - t0 - h * t1) * rc, dw.sum(0), db.sum(0))
    return grads if case["way"] == "backward" else (value * m, mean, rstd) + grads
