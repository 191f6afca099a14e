"""The attention's log-sum-exp and gradient on the GPU against the definition in 64 bits, with bounds derived
element by element from the roundings: ragged frames, frames shorter than a block, head_dim 64 and 128, strided
caches, uneven and empty lists, unlisted blocks, sharp softmaxes, split forward, bad lists."""
import pytest
import torch

import block_sparse_attention_lf_b200 as L
from tests import block_ref as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _lists(g, B, H, Rq, Nkv, cap, counts):
    """Lists of distinct ids in any order; `counts`: full, ragged (0 .. cap) or empty."""
    lists = torch.argsort(torch.rand(B, H, Rq, Nkv, generator=g), -1)[..., :cap].int()
    if counts == "full":
        return lists, torch.full((B, H, Rq), cap, dtype=torch.int32)
    if counts == "empty":
        return lists, torch.zeros(B, H, Rq, dtype=torch.int32)
    n = torch.randint(0, cap + 1, (B, H, Rq), generator=g, dtype=torch.int32)
    n.view(-1)[0], n.view(-1)[-1] = 0, cap
    return lists, n


def _call(shape, q, k, v, do, lists, count, scale=0.0, tail_pieces=1, dk=None, dv=None):
    dev = [t.cuda().contiguous() for t in (q, k, v, do, lists, count)]
    q, k, v, do, lists, count = dev
    cap = lists.shape[-1]
    out, lo, lse = torch.full_like(q, 9.0), torch.full_like(q, 9.0), torch.full(q.shape[:3], 9.0, device="cuda")
    ws = None  # 148 SMs' pieces, and room for out_lo's sums
    if tail_pieces != 1:
        ws = torch.empty(148 * tail_pieces * 64 * (q.shape[-1] + 3) * 4, dtype=torch.uint8, device="cuda")
    L.lf_block_sparse_attn_lse(shape, q, k, v, lists, count, cap, scale, out, lse, ws, tail_pieces, out_lo=lo)
    dq = torch.full_like(q, 9.0)
    dk = torch.full_like(k, 9.0) if dk is None else dk
    dv = torch.full_like(k, 9.0) if dv is None else dv
    bws = torch.full((L.lf_attn_bwd_workspace(shape),), 255, dtype=torch.uint8, device="cuda")
    L.lf_block_sparse_attn_bwd(shape, q, k, v, out, do, lse, lists, count, cap, scale, dq, dk, dv, bws, out_lo=lo)
    # out_lo is the rounding of out (2^-8) and of the weights' sum (2^-8 of the row), rounded
    assert ((lo.float().abs() <= 2.1 * 2.0 ** -8 * out.float().abs() + 1e-30) | ~torch.isfinite(out)).all()
    return out, lse, dq, dk, dv


def _hold(name, got, ref, bound):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), name
    worst = float(((got - ref).abs() - bound).max())
    assert worst <= 0, (name, worst)
    n = float(ref.norm())
    assert float((got - ref).norm()) <= 2.0 ** -7 * n + 1e-12, (name, float((got - ref).norm()) / max(n, 1e-30))


def _check(shape, q, k, v, do, lists, count, scale, got):
    Lkv, s = shape.Lkv, scale if scale > 0 else shape.head_dim ** -0.5
    mask = R.token_mask(shape.batch, shape.heads, shape.frame_tokens, shape.n_cur, shape.n_frames, lists, count)
    d = [t.double() for t in (q, k[:, :, :Lkv], v[:, :, :Lkv], do)]
    (out, lse, dq, dk, dv), (tq, tk, tv), logit = R.attention_grads(*d, mask, s)
    o, l, gq, gk, gv = got
    _hold("dq", gq, dq, tq)
    _hold("dk", gk[:, :, :Lkv], dk, tk)
    _hold("dv", gv[:, :, :Lkv], dv, tv)
    # lse: fp32 sums of the scores (2^-16 of their terms' sizes) and of the row, one logarithm
    some = mask.any(-1)
    lim = 2.0 ** -16 * (1 + (logit * mask).amax(-1)) + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0)
    err = (l.double().cpu() - lse).abs()
    assert (err[some] <= lim[some]).all() and (l.cpu()[~some] == -float("inf")).all()
    # out as in the forward's own parity tests
    assert float((o.double().cpu() - out).abs().max()) <= 3e-2
    assert float((o.double().cpu() - out).norm()) <= 1e-2 * float(out.norm()) + 1e-12
    assert (o.cpu()[~some] == 0).all() and (gq.cpu()[~some] == 0).all()


CASES = [
    # name, B, H, D, F, frames, sink, recent, cur, list length, counts, key scale, pad
    ("one_block", 1, 1, 128, 64, 2, 0, 0, 1, 1, "full", 1.0, 0),
    ("one_token", 1, 2, 64, 1, 3, 1, 0, 1, 2, "full", 1.0, 0),
    ("pair_d128", 1, 2, 128, 128, 3, 0, 1, 1, 4, "full", 1.0, 0),
    ("odd_lists_d64", 2, 3, 64, 100, 5, 1, 1, 2, 5, "full", 1.0, 0),
    ("ragged_d128", 2, 3, 128, 200, 6, 1, 1, 3, 11, "ragged", 1.0, 0),
    ("ragged_d64", 1, 4, 64, 333, 4, 0, 0, 2, 13, "ragged", 1.0, 0),
    ("short_frames", 1, 2, 128, 40, 9, 1, 1, 2, 7, "ragged", 1.0, 0),
    ("strided", 2, 2, 128, 150, 5, 1, 1, 2, 9, "ragged", 1.0, 77),
    ("all_empty", 1, 2, 128, 70, 3, 0, 0, 1, 3, "empty", 1.0, 0),
    ("dense", 1, 2, 128, 260, 3, 0, 0, 3, 15, "full", 1.0, 0),
    ("sharp", 1, 2, 128, 300, 4, 1, 1, 2, 12, "full", 8.0, 0),
    ("many_rows", 1, 1, 128, 1100, 3, 0, 0, 3, 20, "ragged", 1.0, 0),   # 54 query blocks: two words of a list's bits
    ("many_blocks", 1, 1, 64, 65, 600, 1, 1, 1, 30, "full", 1.0, 0),    # 1200 KV blocks: two CTAs of the transposition
]


def _inputs(case):
    name, B, H, D, F, NF, ns, nr, nc, cap, counts, ks, pad = case
    g = torch.Generator().manual_seed(len(name) * 1000 + F)
    bpf = -(-F // 64)
    stride = NF * F + pad if pad else 0
    shape = L.LfShape.make(B, H, D, F, NF, ns, nr, nc, kv_stride=stride)
    r = lambda n, by=1.0: (torch.randn(B, H, n, D, generator=g) * by).to(BF)  # noqa: E731
    q, k, v, do = r(nc * F), r(NF * F + pad, ks), r(NF * F + pad), r(nc * F)
    lists, count = _lists(g, B, H, nc * bpf, NF * bpf, cap, counts)
    return shape, q, k, v, do, lists, count


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_gradients(case):
    shape, q, k, v, do, lists, count = _inputs(case)
    got = _call(shape, q, k, v, do, lists, count)
    _check(shape, q, k, v, do, lists, count, 0.0, got)
    if case[-1]:  # rows past the used length are left as they were
        assert (got[3][:, :, shape.Lkv:] == 9).all() and (got[4][:, :, shape.Lkv:] == 9).all()
    assert L.lf_get_device_error() == (0, 0)
    again = _call(shape, q, k, v, do, lists, count)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_scale_and_forward_equals_plain_call():
    shape, q, k, v, do, lists, count = _inputs(CASES[4])
    got = _call(shape, q, k, v, do, lists, count, scale=0.3)
    _check(shape, q, k, v, do, lists, count, 0.3, got)
    out = torch.empty_like(got[0])
    L.lf_block_sparse_attn(shape, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), count.cuda(), lists.shape[-1], 0.3, out)
    assert torch.equal(out, got[0])


@pytest.mark.parametrize("pieces", [2, 5])
def test_split_forward(pieces):
    """The log-sum-exp of rows whose lists are split and merged."""
    for c in (CASES[4], CASES[5]):
        shape, q, k, v, do, lists, count = _inputs(c)
        got = _call(shape, q, k, v, do, lists, count, tail_pieces=pieces)
        _check(shape, q, k, v, do, lists, count, 0.0, got)


def test_list_longer_than_the_shared_copy():
    """1030 blocks of a list (the forward keeps 1024 in shared memory), and a capacity above the count."""
    g = torch.Generator().manual_seed(77)
    shape = L.LfShape.make(1, 1, 64, 2, 1030, 6, 0, 1)
    q, do = (torch.randn(1, 1, 2, 64, generator=g).to(BF) for _ in range(2))
    k, v = (torch.randn(1, 1, 2060, 64, generator=g).to(BF) for _ in range(2))
    lists = torch.full((1, 1, 1, 1050), -5, dtype=torch.int32)
    lists[..., :1030] = torch.randperm(1030, generator=g)
    count = torch.full((1, 1, 1), 1030, dtype=torch.int32)
    got = _call(shape, q, k, v, do, lists, count)
    _check(shape, q, k, v, do, lists, count, 0.0, got)
    assert L.lf_get_device_error() == (0, 0)


def test_garbage_between_heads_and_behind_frames():
    """NaN and infinities in the rows between a head's used tokens and its stride reach no gradient."""
    case = CASES[7]
    shape, q, k, v, do, lists, count = _inputs(case)
    want = _call(shape, q, k, v, do, lists, count)
    k[:, :, shape.Lkv:], v[:, :, shape.Lkv:] = float("nan"), float("inf")
    got = _call(shape, q, k, v, do, lists, count)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_nonfinite_token_stays_with_its_readers():
    """A NaN key changes only the gradients of rows and blocks that meet it."""
    shape, q, k, v, do, lists, count = _inputs(CASES[4])
    want = _call(shape, q, k, v, do, lists, count)
    bad = 3  # block 3 of head (0, 1)
    bpf, F = shape.bpf, shape.frame_tokens
    tok = (bad // bpf) * F + (bad % bpf) * 64
    k[0, 1, tok] = float("nan")
    got = _call(shape, q, k, v, do, lists, count)
    n = count[0, 1]
    reads = torch.tensor([bad in lists[0, 1, r, :int(n[r])].tolist() for r in range(shape.Rq)])
    assert reads.any() and not reads.all()
    for r in range(shape.Rq):
        f, j = divmod(r, bpf)
        rows = slice(f * F + 64 * j, f * F + min(64 * j + 64, F))
        same = torch.equal(got[2][0, 1, rows], want[2][0, 1, rows])
        assert same == (not reads[r]) and (reads[r] or torch.isfinite(got[2][0, 1, rows]).all())
    for i in range(5):
        assert torch.equal(got[i][1], want[i][1]) and torch.equal(got[i][0, 0], want[i][0, 0])


def test_bad_lists_are_reported():
    """Ids out of range are skipped, counts clamped, repeated blocks reported; no gradient is out of bounds."""
    shape, q, k, v, do, lists, count = _inputs(CASES[4])
    good = _call(shape, q, k, v, do, lists, torch.full_like(count, 4))
    broken = lists.clone()
    broken[..., 4] = shape.Nkv
    broken[..., 5] = -1
    got = _call(shape, q, k, v, do, broken, torch.full_like(count, 6))
    assert L.lf_get_device_error()[0] == 10
    # the same blocks in other pairs of a tile: the same sums
    for a, b in zip(got, good):
        assert float((a.double() - b.double()).norm()) <= 2.0 ** -7 * float(b.double().norm())
    twice = lists.clone()
    twice[0, 0, 1, 1] = twice[0, 0, 1, 0]
    _call(shape, q, k, v, do, twice, torch.full_like(count, 4))
    assert L.lf_get_device_error()[0] == 10
    long = count.clone()
    long[0, 0, 0] = lists.shape[-1] + 1
    _call(shape, q, k, v, do, lists, long)
    assert L.lf_get_device_error()[0] == 10
    assert L.lf_get_device_error() == (0, 0)


def test_shapes_are_checked():
    shape, q, k, v, do, lists, count = [t.cuda() if torch.is_tensor(t) else t for t in _inputs(CASES[2])]
    ws = torch.empty(L.lf_attn_bwd_workspace(shape), dtype=torch.uint8, device="cuda")
    lse = torch.zeros(q.shape[:3], device="cuda")
    run = lambda **kw: L.lf_block_sparse_attn_bwd(**{**dict(  # noqa: E731
        shape=shape, q=q, k=k, v=v, out=q, dout=do, lse=lse, block_list=lists, block_count=count,
        list_cap=lists.shape[-1], softmax_scale=0.0, dq=torch.empty_like(q), dk=torch.empty_like(k),
        dv=torch.empty_like(k), workspace=ws), **kw})
    for bad in (dict(q=q[:, :1]), dict(dk=q), dict(lse=lse[..., :3]), dict(list_cap=3), dict(block_count=count[:, :1]),
                dict(dout=do.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            run(**bad)
    with pytest.raises(TypeError):
        run(out=q.half())
    with pytest.raises(L.LfError):
        run(workspace=ws[:16])


def test_directional_difference():
    """<gradients of the kernel, d> against central differences of the definition in 64 bits: the kernel's gradients
    are within 2^-7 in norm, so the product within that of |g||d| per tensor."""
    shape, q, k, v, do, lists, count = _inputs(CASES[4])
    got = _call(shape, q, k, v, do, lists, count)
    mask = R.token_mask(shape.batch, shape.heads, shape.frame_tokens, shape.n_cur, shape.n_frames, lists, count)
    g = torch.Generator().manual_seed(31)
    x = [t.double() for t in (q, k, v)]
    d = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in x]
    e, s = 1e-6, shape.head_dim ** -0.5
    f = lambda sign: float((R.attention(*[a + sign * e * b for a, b in zip(x, d)], mask, s)[0] * do.double()).sum())  # noqa: E731
    want = sum(float((t.double().cpu() * b).sum()) for t, b in zip(got[2:], d))
    size = sum(float(t.double().norm() * b.norm()) for t, b in zip(got[2:], d))
    assert abs((f(1) - f(-1)) / (2 * e) - want) <= 2.0 ** -7 * size


def test_stream_graph_and_two_workspaces():
    shape, q, k, v, do, lists, count = [t.cuda() if torch.is_tensor(t) else t for t in _inputs(CASES[4])]
    cap = lists.shape[-1]

    def buffers():
        return [torch.zeros_like(q), torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda"), torch.zeros_like(q), torch.zeros_like(k),
                torch.zeros_like(k), torch.empty(L.lf_attn_bwd_workspace(shape), dtype=torch.uint8, device="cuda")]

    def step(b):
        L.lf_block_sparse_attn_lse(shape, q, k, v, lists, count, cap, 0.0, b[0], b[2], out_lo=b[1])
        L.lf_block_sparse_attn_bwd(shape, q, k, v, b[0], do, b[2], lists, count, cap, 0.0, *b[3:], out_lo=b[1])

    want = buffers()
    step(want)
    torch.cuda.synchronize()
    sets, streams = [buffers(), buffers()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(sets, streams):
            with torch.cuda.stream(s):
                step(b)
    torch.cuda.synchronize()
    assert all(torch.equal(a, w) for b in sets for a, w in zip(b[:6], want[:6]))
    b, graph = buffers(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(a, w) for a, w in zip(b[:6], want[:6]))


def test_call_trains_and_loads():
    """A transformer block's attention as a training step runs it: fused projection, rotary positions into the call's
    tensors, pooling, selection, attention, and back to the projection's gradient, against the definition in 64 bits
    on the selected lists."""
    B, H, D, F, NF, nc = 1, 3, 128, 100, 6, 2
    shape = L.LfShape.make(B, H, D, F, NF, 1, 1, nc)
    g = torch.Generator().manual_seed(41)
    qkv = torch.randn(B, nc * F, 3, H, D, generator=g).to(BF).cuda()
    k, v = (torch.randn(B, H, NF * F, D, generator=g).to(BF).cuda() for _ in range(2))
    do = torch.randn(B, H, nc * F, D, generator=g).to(BF).cuda()
    past = k[:, :, :(NF - nc) * F].clone()
    t = torch.arange(nc * F)
    pos = torch.stack([(NF - nc) + t // F, (t % F) // 10, t % 10], -1)
    plan = L.RopePlan.make(D, layout="interleaved", axis_dims=(44, 42, 42))
    q = torch.empty(B, H, nc * F, D, dtype=BF, device="cuda")
    call = L.HSACall(shape, 2, 2, 1, train=True)
    call.load(plan, qkv, pos.int().cuda(), q, k, v)
    out = call(q, k, v)
    dq, dk, dv, dqkv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(qkv)
    call.backward(q, k, v, do, dq, dk, dv)
    call.load_bwd(plan, dq, dk, dv, pos.int().cuda(), dqkv)
    assert torch.equal(k[:, :, :(NF - nc) * F], past)
    lists, count = call.buf.block_list.cpu(), call.buf.block_count.cpu()
    _check(shape, q.cpu(), k.cpu(), v.cpu(), do.cpu(), lists, count, 0.0, (out, call.lse, dq, dk, dv))
    # the rotation's gradient of the kernel's own dq and dk
    f, axis, amp = R.rope_frequencies((44, 42, 42), 10000.0)
    for i, t in enumerate((dq, dk[:, :, (NF - nc) * F:])):
        ref, size = R.rope(t.double().cpu(), pos, f, axis, amp, "interleaved", D, backward=True)
        err = (dqkv[:, :, i].transpose(1, 2).double().cpu() - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + 5e-7 * size).all()
    assert torch.equal(dqkv[:, :, 2].transpose(1, 2), dv[:, :, (NF - nc) * F:])
    with pytest.raises(ValueError):
        L.HSACall(shape, 2, 2, 1).backward(q, k, v, do, dq, dk, dv)


def test_train_call_splits_as_the_plain_one():
    """The last wave's lists are cut into as many pieces with the sums that training adds, so out keeps its bits."""
    shape = L.LfShape.make(1, 1, 128, 320, 8, 1, 1, 2)
    g = torch.Generator().manual_seed(43)
    q = torch.randn(1, 1, 640, 128, generator=g).to(BF).cuda()
    k, v = (torch.randn(1, 1, 8 * 320, 128, generator=g).to(BF).cuda() for _ in range(2))
    plain, train = (L.HSACall(shape, 2, 2, 5, train=t) for t in (False, True))
    tail, pieces = train.split
    assert (tail, pieces) == plain.split and pieces >= 2
    assert train.workspace.numel() == tail * pieces * 64 * (128 + 3) * 4
    assert torch.equal(plain(q, k, v), train(q, k, v))


def test_gradient_before_a_call_is_refused():
    shape = L.LfShape.make(1, 1, 64, 64, 4, 1, 1, 1)
    t = [torch.zeros(1, 1, n, 64, dtype=BF, device="cuda") for n in (64, 256, 256, 64, 64, 256, 256)]
    with pytest.raises(ValueError):
        L.HSACall(shape, 2, 1, 1, train=True).backward(*t)


@pytest.mark.parametrize("pieces", [1, 2, 5])
@pytest.mark.parametrize("case", [CASES[4], CASES[5]], ids=lambda c: c[0])
def test_a_nan_shows_however_lists_are_split(case, pieces):
    """A NaN key makes out and lse of every row that lists it NaN, a NaN query those of its own row, with the lists
    whole or cut into pieces, in the training call and the plain one; the other rows keep their bits."""
    shape, q, k, v, do, lists, count = _inputs(case)
    cap, bpf, F = lists.shape[-1], shape.bpf, shape.frame_tokens
    want = _call(shape, q, k, v, do, lists, count, tail_pieces=pieces)
    b, h, bad = 0, 1, 3
    k[b, h, (bad // bpf) * F + (bad % bpf) * 64] = float("nan")
    own = next(r for r in range(shape.Rq) if int(count[b, h, r]) > 0 and bad not in lists[b, h, r, :int(count[b, h, r])])
    row = own // bpf * F + own % bpf * 64 + 7
    q[b, h, row] = float("nan")
    hit = torch.zeros(q.shape[:3], dtype=torch.bool)
    hit[b, h, row] = True
    for r in range(shape.Rq):
        if bad in lists[b, h, r, :int(count[b, h, r])]:
            f, j = divmod(r, bpf)
            hit[b, h, f * F + 64 * j:f * F + min(64 * j + 64, F)] = True
    assert 1 < int(hit.sum()) < hit.numel()
    out, lse, dq, _, _ = _call(shape, q, k, v, do, lists, count, tail_pieces=pieces)
    plain, ws = torch.empty_like(out), None
    if pieces > 1:
        ws = torch.empty(148 * pieces * 64 * (shape.head_dim + 2) * 4, dtype=torch.uint8, device="cuda")
    L.lf_block_sparse_attn_ws(shape, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), count.cuda(), cap, 0.0, plain, ws, pieces)
    for t in (out, plain, dq):
        assert t.cpu()[hit].isnan().all() and torch.isfinite(t.cpu()[~hit]).all()
    assert lse.cpu()[hit].isnan().all()
    for t, w in ((out, want[0]), (plain, want[0]), (lse, want[1])):
        assert torch.equal(t.cpu()[~hit], w.cpu()[~hit])


def test_planned_workspace_gives_the_planned_pieces():
    """A training call with a workspace of exactly the planned size is cut as the plain call with its own, so out keeps
    its bits; with the plain call's size it would be a piece short."""
    shape = L.LfShape.make(1, 1, 128, 320, 8, 1, 1, 2)
    g = torch.Generator().manual_seed(47)
    q = torch.randn(1, 1, 640, 128, generator=g).to(BF).cuda()
    k, v = (torch.randn(1, 1, 8 * 320, 128, generator=g).to(BF).cuda() for _ in range(2))
    lists, count = (t.cuda() for t in _lists(g, 1, 1, shape.Rq, shape.Nkv, 30, "full"))
    outs = []
    for plan in (L.lf_attn_split_plan, L.lf_attn_lse_split_plan):
        tail, pieces, nbytes = plan(shape, 30)
        assert (tail, pieces) == (10, 3)
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        outs.append(torch.empty_like(q))
        if plan is L.lf_attn_split_plan:
            L.lf_block_sparse_attn_ws(shape, q, k, v, lists, count, 30, 0.0, outs[-1], ws)
        else:
            L.lf_block_sparse_attn_lse(shape, q, k, v, lists, count, 30, 0.0, outs[-1],
                                       torch.empty(1, 1, 640, device="cuda"), ws, out_lo=torch.empty_like(q))
    assert torch.equal(*outs)


LONG_LISTS = [
    # name, B, H, D, F, frames, sink, recent, cur, list length, counts
    # more query blocks list a KV block than two 32-entry windows of its list hold, an odd number of them
    ("key_lists_d128", 1, 2, 128, 33, 73, 1, 1, 71, 73, "full", 1.0, 0),
    ("key_lists_d64", 1, 2, 64, 33, 73, 1, 1, 71, 73, "full", 1.0, 0),
    ("uneven_key_lists", 2, 1, 128, 70, 52, 1, 1, 50, 104, "ragged", 1.0, 0),   # two blocks a frame, one of six tokens
    # more query blocks than the transposition takes at once (256)
    ("many_query_blocks", 1, 2, 128, 3, 320, 6, 4, 300, 90, "ragged", 1.0, 0),
    ("three_sweeps_d64", 1, 1, 64, 2, 606, 4, 2, 600, 120, "ragged", 1.0, 0),
]


@pytest.mark.parametrize("case", LONG_LISTS, ids=[c[0] for c in LONG_LISTS])
def test_long_key_lists(case):
    """Key items of many tiles, whose list ids and row statistics are fetched anew every 32 entries, and transpositions
    of more than one sweep."""
    shape, q, k, v, do, lists, count = _inputs(case)
    listed = torch.zeros(shape.batch * shape.heads, shape.Nkv, dtype=torch.int64)
    flat, n = lists.reshape(-1, shape.Rq, lists.shape[-1]).long(), count.reshape(-1, shape.Rq, 1)
    for u in range(flat.shape[0]):
        listed[u] = torch.bincount(flat[u][torch.arange(flat.shape[-1]) < n[u]], minlength=shape.Nkv)
    if case[10] == "full":
        assert (listed == shape.Rq).all() and shape.Rq == 71
    elif shape.Rq > 256:
        assert shape.Rq > 256 and int(listed.max()) > 64
    else:
        assert int((listed > 32).sum()) > 50 and len(listed.unique()) > 10
    got = _call(shape, q, k, v, do, lists, count)
    _check(shape, q, k, v, do, lists, count, 0.0, got)
    assert L.lf_get_device_error() == (0, 0)
    again = _call(shape, q, k, v, do, lists, count)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
