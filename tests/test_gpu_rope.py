"""Rotary positions on the GPU against the definition in 64 bits: layouts, part of the head, axes,
scalings, far positions, strides, in place, and the gradient."""
import math

import pytest
import torch

import block_sparse_attention_lf_b200 as L
from tests import block_ref as R

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _bound(ref, size, dtype, reach=0.0):
    """Error of one element: half a step of its rounding, and for each member of the pair what the fp32 factor
    cos or sin may be off: the remaining half turn rounded to fp32 (2^-26 turns, 9.4e-8 rad), sincospif (2 ulp,
    1.2e-7), the amplitude and its product (2 * 2^-24), the product and the sum (2 * 2^-24): below 5e-7. `reach`:
    2^-50 times the largest angle, for the roundings of position times frequency in 64 bits on both sides.
    fp16 rounds below 2^-14 in steps of 2^-24."""
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return R.EPS[dtype] * ref.abs() + (5e-7 + reach) * size + tiny


def _check(plan, f, xs, pos, layout, rot, rotate, backward, outs):
    freq, axis, amp = f
    reach = float((pos.double().abs().amax() * freq.max()) * 2.0 ** -50)
    for x, o, turn in zip(xs, outs, rotate):
        if not turn:
            assert torch.equal(o.cpu(), x.cpu())
            continue
        ref, size = R.rope(x.double().cpu(), pos, freq, axis, amp, layout, rot, backward)
        err = (o.double().cpu() - ref).abs()
        assert (err <= _bound(ref, size, x.dtype, reach)).all(), float((err - _bound(ref, size, x.dtype, reach)).max())


CASES = [
    # B, H, T, D, rot, axis dims, layout, dtype, scaling, factor, original, start
    (1, 1, 1, 128, 128, (128,), "half", "bf16", "none", 1.0, 0, 0),
    (2, 3, 17, 128, 128, (44, 42, 42), "interleaved", "bf16", "none", 1.0, 0, 0),
    (1, 12, 65, 64, 64, (64,), "interleaved", "fp16", "linear", 4.0, 0, 1000),
    (2, 5, 33, 128, 64, (64,), "half", "fp32", "ntk", 2.5, 0, 70000),
    (1, 7, 9, 80, 80, (80,), "half", "bf16", "yarn", 8.0, 2048, 123456),
    (1, 2, 5, 96, 38, (20, 18), "interleaved", "fp16", "none", 1.0, 0, 0),      # odd spans: one pair at a time
    (1, 2, 5, 66, 66, (66,), "half", "bf16", "none", 1.0, 0, 5),
    (3, 2, 4, 7, 6, (6,), "half", "fp32", "none", 1.0, 0, 5),                    # an odd head
    (1, 1, 3, 2, 2, (2,), "interleaved", "bf16", "linear", 2.0, 0, 0),
    (1, 24, 40, 256, 192, (64, 64, 64), "half", "bf16", "none", 1.0, 0, 0),
    (1, 2, 3, 256, 256, (256,), "interleaved", "fp32", "yarn", 32.0, 512, (1 << 31) - 8),   # the farthest positions
    (1, 2, 700, 128, 128, (128,), "half", "bf16", "none", 1.0, 0, -350),         # negative ones
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_rope(case, backward):
    B, H, n, D, rot, dims, layout, dt, scaling, factor, original, start = case
    g = torch.Generator().manual_seed(n + D)
    x = torch.randn(B, n, 3, H, D, generator=g).to(T[dt]).cuda()             # token-major projection
    pos = (start + torch.arange(n)).unsqueeze(-1) if len(dims) == 1 else \
        torch.stack([torch.arange(n) // (3 ** (len(dims) - 1 - a)) for a in range(len(dims))], -1)
    plan = L.RopePlan.make(D, rot, layout, dims, 10000.0, scaling, factor, original)
    f = R.rope_frequencies(dims, 10000.0, scaling, factor, original)
    out = torch.full((3, B, H, n, D), 7.0, dtype=T[dt], device="cuda")
    xs, rotate = x.permute(2, 0, 3, 1, 4).unbind(0), (True, True, False)
    L.lf_rope(plan, xs, out.unbind(0), pos.int().cuda(), rotate, backward)
    _check(plan, f, xs, pos, layout, rot, rotate, backward, out.unbind(0))


def test_rope_heads_differ_positions_per_sample_and_cache_slot():
    """Grouped keys (fewer heads), positions of each sample, and a destination inside a longer cache."""
    g = torch.Generator().manual_seed(9)
    B, n, D = 2, 30, 128
    q, k = (torch.randn(B, n, h, D, generator=g).to(torch.bfloat16).cuda() for h in (6, 2))
    cache = torch.full((B, 2, 100, D), 3.0, dtype=torch.bfloat16, device="cuda")
    before = cache.clone()
    oq = torch.empty(B, 6, n, D, dtype=torch.bfloat16, device="cuda")
    pos = torch.randint(0, 5000, (B, n, 1), generator=g)
    plan = L.RopePlan.make(D, layout="half")
    L.lf_rope(plan, [q.transpose(1, 2), k.transpose(1, 2)], [oq, cache[:, :, 41:71]], pos.int().cuda())
    f = R.rope_frequencies((128,), 10000.0)
    _check(plan, f, [q.transpose(1, 2), k.transpose(1, 2)], pos, "half", 128, (True, True), False,
           [oq, cache[:, :, 41:71]])
    assert torch.equal(cache[:, :, :41], before[:, :, :41]) and torch.equal(cache[:, :, 71:], before[:, :, 71:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_rope_in_place_and_unaligned(layout, shift):
    """In place; the same values whether or not the 16-byte path is open; rows around the tensor untouched."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(2 * 3 * 20 * 64, generator=g).to(torch.float16)
    plan, pos = L.RopePlan.make(64, 32, layout), torch.arange(20).unsqueeze(-1).int().cuda()
    want = torch.empty(2, 3, 20, 64, dtype=torch.float16, device="cuda")
    L.lf_rope(plan, [x.view(2, 3, 20, 64).cuda()], [want], pos)
    buf = torch.full((x.numel() + 16,), 5.0, dtype=torch.float16, device="cuda")
    view = buf[shift:shift + x.numel()].view(2, 3, 20, 64)
    view.copy_(x.view(2, 3, 20, 64))
    L.lf_rope(plan, [view], [view], pos)
    assert torch.equal(view, want)
    assert (buf[:shift] == 5).all() and (buf[shift + x.numel():] == 5).all()


def test_rope_broadcast_input_and_empty():
    x = torch.randn(1, 1, 4, 64, device="cuda").expand(3, 5, 4, 64)
    out, pos = torch.empty(3, 5, 4, 64, device="cuda"), torch.arange(4, device="cuda").unsqueeze(-1).int()
    plan = L.RopePlan.make(64)
    L.lf_rope(plan, [x], [out], pos)
    assert torch.equal(out, out[:1, :1].expand(3, 5, 4, 64))
    with pytest.raises(L.LfError):
        L.lf_rope(plan, [out], [x], pos)           # an output whose heads share memory
    none = torch.empty(2, 3, 0, 64, device="cuda")
    L.lf_rope(plan, [none], [none], torch.empty(0, 1, dtype=torch.int32, device="cuda"))


def test_rope_refusals():
    plan, pos = L.RopePlan.make(64), torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 2, 4, 64, device="cuda")
    with pytest.raises(ValueError):
        L.lf_rope(plan, [x], [x[:, :1]], pos)
    with pytest.raises(ValueError):
        L.lf_rope(plan, [x, x[:, :, :3]], [x, x[:, :, :3]], pos)
    with pytest.raises(ValueError):
        L.lf_rope(plan, [x.transpose(2, 3)], [x], pos)
    with pytest.raises(ValueError):
        L.lf_rope(plan, [x], [x], pos[:3])
    with pytest.raises(TypeError):
        L.lf_rope(plan, [x], [x.half()], pos)
    with pytest.raises(TypeError):
        L.lf_rope(plan, [x.double()], [x.double()], pos)
    with pytest.raises(ValueError):
        L.lf_rope(L.RopePlan.make(128), [x], [x], pos)
    with pytest.raises(ValueError):
        L.lf_rope(plan, [x.cpu()], [x.cpu()], pos)
    with pytest.raises(ValueError):
        L.lf_rope(plan, [], [], pos)


def test_rope_gradient_against_differences():
    """<dx, d> of the kernel's gradient against differences of the kernel's forward (fp32): the map is linear,
    so the difference at step 1 is exact but for rounding (2^-20 of the sums' sizes)."""
    g = torch.Generator().manual_seed(13)
    x, d, dy = (torch.randn(2, 3, 50, 64, generator=g).cuda() for _ in range(3))
    plan = L.RopePlan.make(64, 48, "half", (24, 24), scaling="yarn", factor=3.0, original_length=40)
    pos = torch.randint(0, 1000, (50, 2), generator=g).int().cuda()
    up, down, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    L.lf_rope(plan, [x + d], [up], pos)
    L.lf_rope(plan, [x - d], [down], pos)
    L.lf_rope(plan, [dy], [dx], pos, backward=True)
    a = float(((up - down).double() / 2 * dy.double()).sum())
    b = float((dx.double() * d.double()).sum())
    assert abs(a - b) <= 2.0 ** -20 * float((up.abs().double() * dy.abs().double()).sum())


def test_rope_stream_and_graph():
    g = torch.Generator().manual_seed(15)
    x = torch.randn(1, 4, 100, 128, generator=g).to(torch.bfloat16).cuda()
    plan, pos = L.RopePlan.make(128), torch.arange(100).unsqueeze(-1).int().cuda()
    want, out = torch.empty_like(x), torch.zeros_like(x)
    L.lf_rope(plan, [x], [want], pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.lf_rope(plan, [x], [out], pos)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lf_rope(plan, [x], [out], pos)
    x.copy_(x.flip(2))
    out.zero_()
    graph.replay()
    L.lf_rope(plan, [x], [want], pos)
    assert torch.equal(out, want) and math.isfinite(float(out.float().sum()))


MANY = [
    # B, heads of the tensors, T, D, rot, layout, dtype, odd (elements a head is apart beyond D), what it runs
    (1, (5, 3, 4), 19009, 128, 128, "half", "bf16", 0),          # a thread takes all twelve heads of three tensors
    (1, (5, 3, 4), 4001, 128, 128, "interleaved", "bf16", 0),    # four heads a thread: one meets two tensors
    (2, (7, 1), 6001, 64, 64, "half", "fp16", 0),                # a tensor of one head behind one of seven
    (1, (4,), 12001, 128, 64, "half", "fp32", 0),                # three heads asked for, then one; half of each copied
    (1, (2, 1, 1), 5003, 128, 128, "interleaved", "fp32", 0),
    (1, (3, 2), 9001, 66, 66, "interleaved", "bf16", 1),         # single elements: a pair is two loads
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("case", MANY)
def test_rope_threads_of_several_heads(case, backward):
    """So many tokens that a thread takes several heads: later heads are asked for before earlier ones are stored,
    across the tensors of a call, into other tensors and in place."""
    B, heads, n, D, rot, layout, dt, odd = case
    rows = 1 if odd else (8 if dt == "fp16" or dt == "bf16" else 4)
    spans = (rot // 2 if layout == "half" else rot // (2 if odd else 1)) // rows + (D - rot) // rows
    want = -(-148 * 1024 // (B * n * spans))                     # groups of heads the launch asks for
    assert -(-sum(heads) // min(want, sum(heads))) >= 2          # heads a thread takes
    g = torch.Generator().manual_seed(n + D)
    wide = [torch.randn(B, h, n, D + odd, generator=g).to(T[dt]).cuda() for h in heads]
    xs = [t[..., :D] for t in wide]
    pos = torch.randint(-3000, 90000, (n, 1), generator=g)
    plan, f = L.RopePlan.make(D, rot, layout), R.rope_frequencies((rot,), 10000.0)
    rotate = (True, True, False)[:len(heads)] if len(heads) > 1 else (True,)
    outs = [torch.full((B, h, n, D), 7.0, dtype=T[dt], device="cuda") for h in heads]
    L.lf_rope(plan, xs, outs, pos.int().cuda(), rotate, backward)
    _check(plan, f, xs, pos, layout, rot, rotate, backward, outs)
    L.lf_rope(plan, xs, xs, pos.int().cuda(), rotate, backward)
    assert all(torch.equal(x, o) for x, o in zip(xs, outs))
