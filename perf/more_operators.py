"""The operators around the matrix products of a channels-last decoder's blocks, and its training step, as cases that
can be timed: root-mean-square norm (with a residual, with an e4m3 output, backward), rotary positions of several
axes, and AdamW over many tensors with states in 32 or 8 bits, after the gradients' global norm.

The plain forms here state what each operator computes; the framework's own calls are made where ``own`` is true.
"""

import math
import random

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = {"fp16": 2, "bf16": 2, "fp32": 4}
EPS = 1e-6
E4M3 = torch.float8_e4m3fn
TINY = 2.0 ** -126          # the smallest scale of a block of 8-bit values
LR, BETAS, ADAM_EPS, DECAY, MAX_NORM = 1e-4, (0.9, 0.999), 1e-8, 0.01, 1.0
BLOCK = 256                 # of 8-bit states under one scale; every parameter's states start at a multiple of it

# the parameters of a decoder: transposed convolutions with their biases, the norms behind them
DECODER = [256 * 128 * 16, 128, 128, 128, 64 * 32 * 27, 32, 32, 512 * 256 * 16, 256, 256, 256, 512 * 16 * 9, 512, 512,
           512, 8 * 4 * 9, 4, 30, 65]


def _norm(name, way, dtype, n, s, c, residual=False, block=0):
    return {"name": name, "op": "norm", "way": way, "dtype": dtype, "n": n, "s": s, "c": c, "residual": residual,
            "block": block}


def _rotary(name, way, dtype, n, dims, heads, dim, sections, pairs, explicit=False):
    return {"name": name, "op": "rotary", "way": way, "dtype": dtype, "n": n, "dims": dims, "heads": heads, "dim": dim,
            "sections": sections, "pairs": pairs, "explicit": explicit}


def _adamw(name, dtype, bits, count, total, pick, clip):
    return {"name": name, "op": "adamw", "dtype": dtype, "bits": bits, "count": count, "total": total, "pick": pick,
            "clip": clip}


def listed():
    return [
        # one token on its way through a decoder that answers token by token: latency
        _norm("norm_token_4096_bf16", "forward", "bf16", 1, 1, 4096, True),
        # a batch of feature maps (64 x 64) between two blocks, the residual stream carried on
        _norm("norm_add_64x64x1024_bf16", "forward", "bf16", 8, 64 * 64, 1024, True),
        # a long prompt in front of an 8-bit matrix product: the largest forward pass
        _norm("norm_e4m3_4096_fp16", "e4m3", "fp16", 8, 4096, 4096, True),
        # the backward pass at the grouped 2-D upsample's output (16 images of 112 x 112, 512 channels)
        _norm("norm_back_112x112x512_fp16", "backward", "fp16", 16, 112 * 112, 512, True),
        # a training step's forward and backward on a small odd batch, single precision
        _norm("norm_train_13x17x65_fp32", "train", "fp32", 2, 13 * 17, 65),
        # queries and keys of a video block: 16 frames of 32 x 32
        _rotary("rotary_video_16x32x32_bf16", "forward", "bf16", 2, "16,32,32", 24, 128, "16,56,56", "halves"),
        # the next token of 16 requests, each at a far position of its own: latency
        _rotary("rotary_token_fp16", "forward", "fp16", 16, "1", 32, 128, "16,56,56", "halves", True),
        # the gradient at an image block of odd sizes, part of each head unrotated
        _rotary("rotary_back_57x91_fp32", "backward", "fp32", 3, "57,91", 5, 72, "24,40", "adjacent"),
        # a small decoder's step with clipping: dozens of tensors, most of them tiny
        _adamw("adamw_decoder_fp32", "fp32", 32, 0, 0, 3, True),
        # a large step in mixed precision (bf16 parameters and gradients, fp32 masters) with clipping: the largest
        _adamw("adamw_134M_bf16", "bf16", 32, 150, 1 << 27, 1, True),
        # the same decoder with 8-bit states, fp16 with masters
        _adamw("adamw_8bit_decoder_fp16", "fp16", 8, 0, 0, 3, False),
        # a large step where the states have to fit beside a model
        _adamw("adamw_8bit_67M_fp32", "fp32", 8, 60, 1 << 26, 2, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["fp16", "bf16", "fp32"])
    op = rng.choice(["norm", "norm", "rotary", "adamw"])
    if op == "norm":
        way = rng.choice(["forward", "e4m3", "backward", "train"])
        c = _log(rng, 8, 16384)
        if rng.random() < 0.6:
            c = max(8, c // 64 * 64) if c >= 64 else max(8, c // 8 * 8)
        rows = max(1, _log(rng, 1000, 4e7) // c)
        n = rng.choice([1, 2, 3, 8, 16])
        return _norm("", way, dtype, n, max(1, rows // n), c, rng.random() < 0.5,
                     rng.choice([0, 32, 64, 128]) if way == "e4m3" else 0)
    if op == "rotary":
        axes = rng.choice([1, 2, 3])
        explicit = rng.random() < 0.4
        sections = [2 * rng.randint(1, 64 // axes) for _ in range(axes)]
        dim = sum(sections) + rng.choice([0, 0, 8, 17])
        heads, n = _log(rng, 1, 64), _log(rng, 1, 16)
        s = max(1, _log(rng, 1000, 4e7) // (heads * n * dim))
        if explicit:
            dims = [s]
        else:
            dims = [max(1, int(round(s ** (1 / axes) * rng.uniform(0.6, 1.4)))) for _ in range(axes)]
        return _rotary("", rng.choice(["forward", "backward"]), dtype, n, ",".join(map(str, dims)), heads, dim,
                       ",".join(map(str, sections)), rng.choice(["adjacent", "halves"]), explicit)
    total = _log(rng, 1000, 6e7)
    return _adamw("", dtype, rng.choice([32, 8]), min(_log(rng, 1, 300), total), total, rng.randrange(1 << 20),
                  rng.random() < 0.5)


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _sizes(case):
    """The parameters' element counts: the decoder's `pick` times over, or `total` elements split over `count` tensors
    of very different sizes."""
    if not case["count"]:
        return DECODER * case["pick"]
    r = random.Random(case["pick"])
    share = [math.exp(r.uniform(0, 9)) for _ in range(case["count"])]
    spare = case["total"] - case["count"]
    sizes = [1 + int(spare * v / sum(share)) for v in share]
    sizes[-1] += case["total"] - sum(sizes)
    return sizes


def _starts(sizes):
    """Where each parameter starts in a buffer that holds all of them, at multiples of BLOCK; and the buffer's size."""
    at, starts = 0, []
    for n in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    return starts, at


def _dims(text):
    return [int(v) for v in text.split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    st = {"case": case}
    if case["op"] == "norm":
        n, s, c = case["n"], case["s"], case["c"]
        # a residual stream: some channels far larger than the others
        spread = 0.5 + normal(c).abs() ** 3
        st["x"] = (normal(n, s, c) * spread).to(t)
        st["weight"] = 1.0 + 0.2 * normal(c)
        if case["way"] in ("backward", "train"):
            st["dy"] = (0.1 * normal(n, s, c)).to(t)
            st["dsum"] = (0.1 * normal(n, s, c)).to(t) if case["residual"] else None
        if case["way"] == "backward":      # what the forward pass left
            st["rstd"] = ((st["x"].double() ** 2).mean(dim=-1) + EPS).rsqrt().float()
        else:
            st["residual"] = (normal(n, s, c) * spread).to(t) if case["residual"] else None
        return st
    if case["op"] == "rotary":
        st["x"] = normal(case["n"], *_dims(case["dims"]), case["heads"], case["dim"]).to(t)
        st["positions"] = None
        if case["explicit"]:
            st["positions"] = torch.randint(0, 1 << 17, (case["n"], *_dims(case["dims"]), len(_dims(case["sections"]))),
                                            generator=g, device="cuda")
        return st
    sizes = _sizes(case)
    starts, total = _starts(sizes)

    def views(flat):
        return [flat[a:a + n] for a, n in zip(starts, sizes)]

    def filled(make):
        flat = torch.zeros(total, device="cuda", dtype=torch.float32)
        for v in views(flat):
            v.copy_(make(v.numel()))
        return flat

    # a run some hundred steps old; each tensor's gradients have a size of their own
    scales = [0.002 * math.exp(2 * v) for v in normal(len(sizes)).tolist()]
    of = iter(scales * 3)
    st["step"] = 100 + seed % 1000
    st["seed"] = (seed * 0x9E3779B97F4A7C15) % (1 << 63)
    master = filled(lambda n: 0.1 * normal(n))
    st["p"] = master.to(t)
    st["master"] = None if t == torch.float32 else master
    st["g"] = filled(lambda n: next(of) * normal(n)).to(t)
    m = filled(lambda n: 0.3 * next(of) * normal(n))
    root = filled(lambda n: next(of) * (0.5 + normal(n).abs()))
    if case["bits"] == 32:
        st["m"], st["v"] = m, root * root
    else:
        for name, value in (("m", m), ("v", root)):
            scale = _scales(value)
            st[name], st[name + "_scale"] = (value.view(-1, BLOCK) / scale[:, None]).view(-1).to(E4M3), scale
    st["grads"] = views(st["g"])
    st["params"] = views(st["p"])
    if own:                      # the optimizer that a program keeps, with the states at this step
        from transposed_convolution_02_b200 import ct

        opt = ct.AdamW(st["params"], lr=LR, betas=BETAS, eps=ADAM_EPS, weight_decay=DECAY, bits=case["bits"],
                       seed=st["seed"])
        opt.steps = st["step"]
        opt.exp_avg.copy_(st.pop("m"))
        opt.exp_avg_sq.copy_(st.pop("v"))
        if case["bits"] == 8:
            opt.exp_avg_scale.copy_(st.pop("m_scale"))
            opt.exp_avg_sq_scale.copy_(st.pop("v_scale"))
        if st["master"] is not None:
            opt.master.copy_(st.pop("master"))
        st["opt"] = opt
    return st


# ---- the plain forms ------------------------------------------------------------------------------------------------

def _norm_forward(st):
    c = st["case"]
    h = st["x"].float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
    rstd = 1 / torch.sqrt((h * h).mean(dim=-1, keepdim=True) + EPS)
    return h, h * rstd * st["weight"], rstd.view(c["n"], c["s"])


def _blocks(y, block):
    """[.., C] -> [.., blocks, block], the last one filled up with zeros; one block of all channels for 0."""
    if block == 0:
        return y[..., None, :]
    return torch.nn.functional.pad(y, (0, -y.shape[-1] % block)).unflatten(-1, (-1, block))


def _norm_e4m3(st):
    c = st["case"]
    h, y, rstd = _norm_forward(st)
    parts = _blocks(y, c["block"])
    scale = torch.clamp(parts.abs().amax(dim=-1) / 448, min=TINY)
    q = (parts / scale[..., None]).flatten(-2)[..., :c["c"]].to(E4M3)
    scale = scale if c["block"] else scale[..., 0]
    return (q, scale, h.to(st["x"].dtype), rstd) if st["residual"] is not None else (q, scale, rstd)


def _norm_backward(st, h, rstd):
    h, dy, r = h.float(), st["dy"].float(), rstd[..., None]
    hat, t = h * r, dy * st["weight"]
    dx = r * (t - hat * (t * hat).mean(dim=-1, keepdim=True))
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return dx.to(st["x"].dtype), (dy * hat).sum(dim=(0, 1))


def _norm_plain(st):
    way, t = st["case"]["way"], st["x"].dtype
    if way == "backward":
        return _norm_backward(st, st["x"], st["rstd"])
    if way == "e4m3":
        return _norm_e4m3(st)
    h, y, rstd = _norm_forward(st)
    out = (y.to(t), h.to(t), rstd) if st["residual"] is not None else (y.to(t), rstd)
    return out + _norm_backward(st, h.to(t), rstd) if way == "train" else out


def _angles(st, shape):
    """cos and sin [.., pairs] of positions times frequencies: in 64 bits, where a far position times a frequency
    keeps its fraction of a turn."""
    c = st["case"]
    sections = _dims(c["sections"])
    if st["positions"] is not None:
        at = st["positions"].double()
    else:
        at = torch.stack(torch.meshgrid(*[torch.arange(d, device="cuda", dtype=torch.float64) for d in shape],
                                        indexing="ij"), dim=-1)
    freq = [10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d) for d in sections]
    angle = torch.cat([at[..., a, None] * f for a, f in enumerate(freq)], dim=-1)[..., None, :]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotary_plain(st):
    c = st["case"]
    x = st["x"].float()
    cos, sin = _angles(st, st["x"].shape[1:-2])
    if c["way"] == "backward":
        sin = -sin
    rot = 2 * cos.shape[-1]
    if c["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), dim=-1).to(st["x"].dtype)


LOW = 0xFFFFFFFF


def _random16(n, seed, offset):
    """16 bits for each of n elements: part i % 8 of Philox4x32-10 (Salmon et al., 2011) at counter (i // 8, offset)."""
    i = torch.arange(n // 8, device="cuda", dtype=torch.int64)
    zero = torch.zeros_like(i)
    c0, c1, c2, c3 = i & LOW, i >> 32, zero + (offset & LOW), zero + (offset >> 32)
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & LOW) ^ c1 ^ k0, p1 & LOW, ((p0 >> 32) & LOW) ^ c3 ^ k1, p0 & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    words = torch.stack((c0, c1, c2, c3), dim=1)
    return torch.stack((words & 0xFFFF, words >> 16), dim=2).reshape(-1).int()


def _scales(v):
    return torch.clamp(v.view(-1, BLOCK).abs().amax(dim=1) / 448, min=TINY)


def _codes(v, scale, r):
    """v / scale in e4m3, up to the next value with the probability of the part that lies beyond the last: the 16
    random bits are added below the three bits that stay.  Below 2^-6 values lie 2^-9 apart, as they do above it."""
    x = (v.view(-1, BLOCK) / scale[:, None]).view(-1)
    a = x.abs()
    low = a < 2.0 ** -6
    b = torch.where(low, a + 2.0 ** -6, a)
    b = ((b.view(torch.int32) + (r << 4)) & ~0xFFFFF).view(torch.float32)
    b = torch.clamp(torch.where(low, b - 2.0 ** -6, b), max=448.0)
    return torch.copysign(b, x)


def _adamw_plain(st):
    c = st["case"]
    st["step"] += 1
    g = st["g"].float()
    out = {}
    if c["clip"]:
        norm = torch.sqrt((st["g"].double() ** 2).sum())
        scale = torch.clamp(MAX_NORM / norm, max=1.0).float()
        g = g * scale
        out["norm"], out["scale"] = norm.float(), scale
    if c["bits"] == 32:
        m, v = st["m"], st["v"]
    else:
        m = (st["m"].float().view(-1, BLOCK) * st["m_scale"][:, None]).view(-1)
        v = (st["v"].float().view(-1, BLOCK) * st["v_scale"][:, None]).view(-1) ** 2
    m = BETAS[0] * m + (1 - BETAS[0]) * g
    v = BETAS[1] * v + (1 - BETAS[1]) * (g * g)
    c1, c2 = 1 - BETAS[0] ** st["step"], 1 - BETAS[1] ** st["step"]
    p = st["p"] if st["master"] is None else st["master"]
    p.copy_(p * (1 - LR * DECAY) - LR * (m / c1) / (torch.sqrt(v / c2) + ADAM_EPS))
    if st["master"] is not None:
        st["p"].copy_(p.to(st["p"].dtype))
        out["master"] = p
    if c["bits"] == 32:
        st["m"].copy_(m)
        st["v"].copy_(v)
    else:
        r = _random16(m.numel(), st["seed"], st["step"])
        root = torch.sqrt(v)
        st["m_scale"], st["v_scale"] = _scales(m), _scales(root)
        st["m"] = _codes(m, st["m_scale"], r).to(E4M3)
        code = _codes(root, st["v_scale"], r)
        st["v"] = torch.where(root > 0, torch.clamp(code, min=2.0 ** -9), code).to(E4M3)
        out["m_scale"], out["v_scale"] = st["m_scale"], st["v_scale"]
    return {**out, "p": st["p"], "m": st["m"], "v": st["v"]}


def _run_plain(st):
    op = st["case"]["op"]
    return _norm_plain(st) if op == "norm" else _rotary_plain(st) if op == "rotary" else _adamw_plain(st)


# ---- the framework's calls ------------------------------------------------------------------------------------------

def _run_own(st):
    from transposed_convolution_02_b200 import ct

    c = st["case"]
    if c["op"] == "rotary":
        call = ct.rotary_nhwc if c["way"] == "forward" else ct.rotary_nhwc_backward
        return call(st["x"], _dims(c["sections"]), pairs=c["pairs"], positions=st["positions"])
    if c["op"] == "adamw":
        opt, out, scale = st["opt"], {}, None
        if c["clip"]:
            norm, scale = ct.grad_norm(st["grads"], max_norm=MAX_NORM)
            out["norm"], out["scale"] = norm, scale
        opt.step(st["grads"], grad_scale=scale)
        if opt.master is not None:
            out["master"] = opt.master
        if c["bits"] == 8:
            out["m_scale"], out["v_scale"] = opt.exp_avg_scale, opt.exp_avg_sq_scale
        return {**out, "p": st["p"], "m": opt.exp_avg, "v": opt.exp_avg_sq}
    if c["way"] == "backward":
        return ct.rms_norm_nhwc_backward(st["dy"], st["x"], st["rstd"], st["weight"], dsum=st["dsum"])
    how = {"eps": EPS, "residual": st["residual"], "return_rstd": True}
    if c["way"] == "e4m3":
        return ct.rms_norm_nhwc_e4m3(st["x"], st["weight"], block=c["block"] or None, **how)
    out = ct.rms_norm_nhwc(st["x"], st["weight"], **how)
    if c["way"] == "forward":
        return out
    h = out[1] if st["residual"] is not None else st["x"]
    return out + tuple(ct.rms_norm_nhwc_backward(st["dy"], h, out[-1], st["weight"], dsum=st["dsum"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    """Every input read once, every output written once; the operations of the formulas."""
    size = SIZES[case["dtype"]]
    if case["op"] == "norm":
        rows, c = case["n"] * case["s"], case["c"]
        e, res = rows * c, case["residual"]
        forward = e * size * (4 if res else 2) + 4 * rows
        backward = e * size * (4 if res else 3) + 4 * rows
        if case["way"] == "e4m3":
            forward += e * (1 - size) + 4 * rows * (-(-c // case["block"]) if case["block"] else 1)
        moved = {"backward": backward, "train": forward + backward}.get(case["way"], forward)
        ops = {"forward": 5, "e4m3": 8, "backward": 12, "train": 17}[case["way"]]
        return {"bytes": moved + 8 * c, "flops": ops * e}
    if case["op"] == "rotary":
        pixels = case["n"] * math.prod(_dims(case["dims"]))
        e = pixels * case["heads"] * case["dim"]
        return {"bytes": 2 * e * size + (8 * pixels * len(_dims(case["sections"])) if case["explicit"] else 0),
                "flops": 3 * e}
    e = sum(_sizes(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK           # both states, read and written
    weight = 8 if case["dtype"] == "fp32" else 8 + size            # read and written; masters, and the 16-bit copy
    return {"bytes": e * (state + weight + size * (2 if case["clip"] else 1)),
            "flops": e * (18 if case["bits"] == 32 else 45)}


# ---- the definition in 64 bits --------------------------------------------------------------------------------------

def _norm_exact(case, st):
    x, w = st["x"].double(), st["weight"].double()
    res = case["residual"]
    if case["way"] == "backward":
        h, inv = x, st["rstd"].double()
    else:
        h = x + st["residual"].double() if res else x
        inv = (torch.linalg.vector_norm(h, dim=-1) ** 2 / case["c"] + EPS) ** -0.5
    out = ()
    if case["way"] != "backward":
        y = h * inv.unsqueeze(-1) * w
        if case["way"] == "e4m3":
            width = case["block"] or case["c"]
            count = -(-case["c"] // width)
            scale = torch.stack([y[..., k * width:(k + 1) * width].abs().amax(-1) / 448 for k in range(count)], -1)
            q = y / scale.repeat_interleave(width, -1)[..., :case["c"]].clamp(min=1e-300)
            out = (q, scale if case["block"] else scale.squeeze(-1))
        else:
            out = (y,)
        out += (h, inv) if res else (inv,)
        del y
    if case["way"] in ("backward", "train"):
        dy = st["dy"].double()
        dot = (dy * w * h).sum(-1) / case["c"]
        dx = dy * w * inv.unsqueeze(-1) - h * (dot * inv ** 3).unsqueeze(-1)
        if st["dsum"] is not None:
            dx += st["dsum"].double()
        out += (dx, torch.einsum("nsc,ns->c", dy * h, inv))
    return out


def _rotary_exact(case, st):
    x = st["x"].double()
    y = x.clone()
    sections = _dims(case["sections"])
    half, pair = sum(sections) // 2, 0
    for a, d in enumerate(sections):
        if case["explicit"]:
            at = st["positions"][..., a].double()
        else:
            at = torch.arange(x.shape[1 + a], device="cuda").double()
            at = at.view([-1 if k == a else 1 for k in range(len(sections))]).expand(x.shape[1:-2])
        for j in range(d // 2):
            i, k = (2 * pair, 2 * pair + 1) if case["pairs"] == "adjacent" else (pair, half + pair)
            turn = torch.polar(torch.ones_like(at), at * math.exp(-2 * j / d * math.log(10000.0)))
            if case["way"] == "backward":
                turn = turn.conj()
            z = torch.complex(x[..., i], x[..., k]) * turn.unsqueeze(-1)
            y[..., i], y[..., k] = z.real, z.imag
            pair += 1
    return y


def _adamw_exact(case, st):
    f = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor)}
    g, t, out = f["g"], st["step"] + 1, {}
    if case["clip"]:
        out["norm"] = torch.linalg.vector_norm(g)
        out["scale"] = (MAX_NORM / out["norm"]).clamp(max=1.0)
        g = g * out["scale"]
    m, v = f["m"], f["v"]
    if case["bits"] == 8:
        m = m * f["m_scale"].repeat_interleave(BLOCK)
        v = (v * f["v_scale"].repeat_interleave(BLOCK)) ** 2
    m = m + (1 - BETAS[0]) * (g - m)
    v = v + (1 - BETAS[1]) * (g ** 2 - v)
    p = f.get("master", f["p"])
    p = p - LR * DECAY * p - LR / (1 - BETAS[0] ** t) * m / ((v / (1 - BETAS[1] ** t)).sqrt() + ADAM_EPS)
    if "master" in f:
        out["master"] = p
    if case["bits"] == 8:                  # the states before they are rounded
        for name, value in (("m", m), ("v", v.sqrt())):
            out[name + "_scale"] = value.view(-1, BLOCK).abs().amax(1) / 448
            value /= out[name + "_scale"].clamp(min=1e-300).repeat_interleave(BLOCK)
            m, v = (value, v) if name == "m" else (m, value)
    return {**out, "p": p, "m": m, "v": v}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(case, st)
    return _rotary_exact(case, st) if case["op"] == "rotary" else _adamw_exact(case, st)
