"""Rotary positions on the GPU against their plain fp64 form."""

import pytest
import torch

import blocks_ref as ref
from test_gpu_rms_norm import TYPES, _cuda, normal  # noqa: F401
from transposed_convolution_02_b200 import ct

pytestmark = pytest.mark.gpu


def compare(x, sections, pairs, positions=None, base=10000.0, backward=False, **how):
    call = ct.rotary_nhwc_backward if backward else ct.rotary_nhwc
    x64 = x.double()
    y = call(x, sections, base=base, pairs=pairs, positions=positions, **how)
    at = ref.grid_positions(x.shape[1:-2], "cuda") if positions is None else positions.double()
    angles = ref.rotary_angles(at, sections, base) * (-1 if backward else 1)
    want = ref.rotary(x64, angles, pairs)
    where = "%s %s %s" % (list(x.shape), sections, pairs)
    ref.check(y, want, ref.rotary_bound(x64, want, angles, pairs, x.dtype), where)
    assert torch.equal(y[..., sum(sections):], x64[..., sum(sections):].to(x.dtype)), where + " rest"
    return y


CASES = [   # dims, heads, dim, sections
    ([1], 1, 1, [0]), ([1], 1, 2, [2]), ([7], 3, 8, [8]), ([50], 4, 64, [64]), ([9], 2, 128, [32]), ([3], 5, 17, [16]),
    ([4], 1, 600, [512]), ([5], 9, 72, [36]), ([600], 33, 40, [24]), ([2], 64, 24, [16]), ([1], 13, 32, [32]),
    ([3, 5], 2, 16, [8, 8]), ([6, 7], 7, 72, [24, 40]), ([1, 9], 3, 20, [2, 14]), ([5, 1], 4, 128, [64, 64]),
    ([33, 35], 5, 80, [16, 64]), ([2, 3], 1, 26, [0, 26]), ([8, 8], 6, 48, [30, 2]),
    ([2, 3, 4], 3, 32, [8, 8, 16]), ([3, 1, 5], 24, 128, [16, 56, 56]), ([4, 4, 4], 2, 38, [4, 6, 10]),
    ([7, 3], 5, 36, [12, 20]), ([90], 9, 44, [44]), ([110], 17, 28, [24]), ([30, 40], 12, 72, [20, 50]),
    ([9, 17, 19], 2, 64, [16, 24, 24]), ([1, 1, 1], 8, 96, [32, 32, 32]), ([5, 6, 7], 1, 51, [2, 2, 46]),
]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_rotary(i, pairs, dtype):
    dims, heads, dim, sections = CASES[i]
    for n in (1, 3):
        x = normal([n] + dims + [heads, dim], 100 + i, TYPES[dtype])
        compare(x, sections, pairs, base=[10000.0, 100.0, 5e5][i % 3], backward=(i + n) % 2 == 0)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("kind", [torch.int32, torch.int64, torch.float32])
@pytest.mark.parametrize("images", [False, True])
def test_given_positions(kind, images, dtype):
    """Positions of every type, for each image or for all, far ones and
    fractions among them; negative ones too."""
    for pairs, sections in (("halves", [16, 24, 24]), ("adjacent", [10, 6])):
        x = normal([3, 5, 7, 4, 72], 7, TYPES[dtype])
        g = torch.Generator().manual_seed(3)
        at = torch.randint(-1000, 1 << 20, ([3] if images else []) + [5, 7, len(sections)], generator=g)
        at.view(-1)[:3] = torch.tensor([0, (1 << 31) - 1, -(1 << 31)])
        if kind == torch.float32:
            at = at * 0.37 + 0.001
        compare(x, sections, pairs, positions=at.to(kind).cuda())
        compare(x, sections, pairs, positions=at.to(kind).cuda(), backward=True)
        wide = at.to(kind).cuda().repeat_interleave(2, dim=-1)[..., ::2]       # not contiguous
        compare(x, sections, pairs, positions=wide)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_layouts(pairs, dtype):
    """Slices, permuted heads, repeated pixels, tensors that start inside a
    vector; in place, with what lies around left as it was."""
    t = TYPES[dtype]
    sections = [16, 48]
    qkv = normal([2, 5, 6, 9, 64], 11, t)
    want = compare(qkv[..., 2:7, :], sections, pairs)
    for view in (qkv[:, :, ::2], qkv[:, :, 1:4], qkv[..., ::2, :], qkv[1:, 1:2]):
        compare(view, sections, pairs)
    assert ct.rotary_nhwc(qkv[..., 2:7, :], sections, pairs=pairs).is_contiguous()
    packed = qkv.clone()
    part = packed[..., 2:7, :]
    assert ct.rotary_nhwc(part, sections, pairs=pairs, out=part) is part
    assert torch.equal(part, want)
    assert torch.equal(packed[..., :2, :], qkv[..., :2, :]) and torch.equal(packed[..., 7:, :], qkv[..., 7:, :])
    back = ct.rotary_nhwc_backward(part, sections, pairs=pairs, out=part)
    # values below 6: a rounding of 1.5 times that each way, and rotary_bound's 12 u of both sides of a pair
    assert bool(((back.double() - qkv[..., 2:7, :].double()).abs() <= 18 * ref.HALF[t] + 288 * ref.U).all())
    outside = normal([2, 9, 5, 6, 64], 12, t).permute(0, 2, 3, 1, 4)           # heads outside the pixels
    want = compare(outside, sections, pairs)
    into = torch.full((2, 9, 5, 6, 64), 7.0, dtype=t, device="cuda").permute(0, 2, 3, 1, 4)
    assert torch.equal(ct.rotary_nhwc(outside, sections, pairs=pairs, out=into), want)
    compare(qkv[:, :1, :1].expand(2, 5, 6, 9, 64), sections, pairs)
    for cut, moved in ((0, 1), (1, 0), (2, 3)):
        flat = torch.zeros(qkv.numel() + 4, dtype=t, device="cuda")
        odd = flat[cut:cut + qkv.numel()].view(qkv.shape)
        odd.copy_(qkv)
        out = torch.zeros(qkv.numel() + 4, dtype=t, device="cuda")[moved:moved + qkv.numel()].view(qkv.shape)
        compare(odd, sections, pairs, out=out)
    narrow = normal([2, 5, 6, 9, 63], 13, t)                                    # heads that start inside a vector
    compare(narrow, [16, 46], pairs)
    copied = normal([2, 5, 6, 64, 9], 14, t).transpose(3, 4)                    # copied first
    compare(copied, sections, pairs)
    with pytest.raises(ValueError, match="overlaps"):
        ct.rotary_nhwc(part, sections, out=packed[..., 3:8, :])
    with pytest.raises(ct.CtError, match="CT_ERR_ATTR"):                        # an output that lies on itself
        ct.rotary_nhwc(qkv, sections, out=torch.zeros(64, dtype=t, device="cuda").expand(qkv.shape))


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("heads", [1, 2, 3, 4])
def test_images_that_share_positions(heads, dtype):
    """More images than heads, with one grid, given positions for all or for
    each: to the bit what each image gives alone; slices of images, one image
    for all, images behind pixels."""
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(5)
    for n, pairs, sections in ((5, "halves", [16, 24, 24]), (19, "adjacent", [10, 6]), (33, "halves", [50])):
        dims = {3: [3, 2, 4], 2: [3, 7], 1: [11]}[len(sections)]
        x = normal([n] + dims + [heads, 72], 17 + n, t)
        at = torch.randint(-99, 1 << 18, [n] + dims + [len(sections)], generator=g).cuda()
        turned = x.movedim(0, -3).contiguous().movedim(-3, 0)
        for images, positions in ((x, None), (x, at[0]), (x, at), (x[::2], None), (x[1::2], at[0]),
                                  (x[:1].expand(x.shape), at[1]), (turned, None)):
            y = compare(images, sections, pairs, positions=positions)
            for i in (0, len(images) - 1):
                own = positions[i:i + 1] if positions is at else positions
                assert torch.equal(y[i:i + 1], ct.rotary_nhwc(images[i:i + 1], sections, pairs=pairs, positions=own))
        compare(x, sections, pairs, positions=at[0], backward=True)


@pytest.mark.parametrize("base", [1e-4, 0.5, 1.0, 1e30])
def test_bases(base):
    """Frequencies above a turn a position, none that differ, and vanishing ones; positions around 2^24, where
    floats stop holding them."""
    x = normal([1, 9, 2, 40], 17)
    for kind in (torch.int64, torch.float32):
        at = torch.tensor([[0], [1], [77], [-1000], [(1 << 24) - 1], [1 << 24], [-(1 << 24) - 2], [(1 << 25) + 4],
                           [1 << 30]], device="cuda").to(kind)
        for pairs in ("adjacent", "halves"):
            compare(x, [32], pairs, positions=at, base=base)


def test_special_values():
    """Position 0 turns nothing, infinities and NaN stay in their pairs."""
    x = normal([1, 6, 2, 24], 21)
    at = torch.tensor([[0], [1], [2], [3], [4], [5]], device="cuda")
    x[0, 2, 0, 1] = float("inf")
    x[0, 3, 1, 2] = float("nan")
    x[0, 4, 0, 20] = float("nan")             # not rotated
    y = ct.rotary_nhwc(x, [16], positions=at)
    assert torch.equal(y[0, 0], x[0, 0])
    odd = torch.zeros_like(x, dtype=torch.bool)
    odd[0, 2, 0, :2] = odd[0, 3, 1, 2:4] = odd[0, 4, 0, 20] = True
    assert torch.equal(y.isfinite(), ~odd)


def test_empty():
    for shape in ([0, 3, 2, 8], [2, 0, 2, 8], [2, 3, 0, 8]):
        x = torch.zeros(shape, device="cuda")
        assert ct.rotary_nhwc(x, [8]).shape == x.shape


@pytest.mark.parametrize("heads,dim,per", [(1, 512, 0), (4, 16, 1)])
def test_heads_past_32_bits(heads, dim, per):
    """Offsets above 2^31 elements, and more threads than 2^31 / 4."""
    s = (1 << 31) // (heads * dim) + 77
    x = torch.zeros(1, s, heads, dim, dtype=torch.float16, device="cuda")
    x[:, -50:] = normal([1, 50, heads, dim], 31, torch.float16)
    y = ct.rotary_nhwc(x, [16], pairs="halves", out=x.clone() if per else None)
    at = torch.arange(s - 50, s, device="cuda")[:, None]
    assert torch.equal(y[:, -50:], ct.rotary_nhwc(x[:, -50:], [16], pairs="halves", positions=at))
    assert not y[:, :-50].any()


def test_streams_and_graphs():
    x = normal([2, 9, 11, 6, 64], 41, torch.bfloat16)
    want = ct.rotary_nhwc(x, [16, 48])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ct.rotary_nhwc(x, [16, 48], stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    at = torch.zeros(9, 11, 2, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ct.rotary_nhwc(x, [16, 48], positions=at)
    at.copy_(ref.grid_positions([9, 11], "cuda"))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(ValueError, match="gradient"):
        ct.rotary_nhwc(torch.zeros(1, 1, 1, 2, device="cuda", requires_grad=True), [2])
