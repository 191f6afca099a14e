"""Refusals, sizes and host logic of the operators around the HSA call (no GPU is touched), and
the 64-bit definitions against differences."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_lf_b200 as L
from tests import block_ref as R

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced (validation fails first)
P = ctypes.c_void_p
p, mis = P(FAKE), P(FAKE + 8)


# ---------------------------------------------------------------- rotary plan
@pytest.mark.parametrize("dims,rot,D", [((128,), 128, 128), ((44, 42, 42), 128, 128), ((32, 32), 64, 96), ((2,), 2, 2)])
@pytest.mark.parametrize("scaling,factor,original", [("none", 1.0, 0), ("linear", 4.0, 0), ("ntk", 2.5, 0),
                                                    ("yarn", 16.0, 8192), ("yarn", 1.0, 100)])
def test_rope_plan_frequencies(dims, rot, D, scaling, factor, original):
    if scaling == "ntk" and dims[0] == 2:
        with pytest.raises(L.LfError):
            L.RopePlan.make(D, rot, axis_dims=dims, scaling=scaling, factor=factor)
        return
    plan = L.RopePlan.make(D, rot, "half", dims, 10000.0, scaling, factor, original)
    f, _, amp = R.rope_frequencies(dims, 10000.0, scaling, factor, original)
    assert list(plan.axis_dims)[:len(dims)] == list(dims) and plan.n_axes == len(dims)
    got = torch.tensor(list(plan.turns)[:rot // 2], dtype=torch.float64) * 2 * math.pi
    # a few fp64 roundings in pow, the scaling and the division by 2 pi
    torch.testing.assert_close(got, f, rtol=64 * 2.0 ** -53, atol=0)
    assert plan.amplitude == pytest.approx(amp, rel=2.0 ** -24)
    assert all(t == 0.0 for t in list(plan.turns)[rot // 2:])


@pytest.mark.parametrize("kw", [
    dict(head_dim=257), dict(head_dim=1), dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=130), dict(axis_dims=[64, 62]),
    dict(axis_dims=[63, 65]), dict(axis_dims=[32, 32, 32, 32]), dict(base=1.0), dict(base=math.inf),
    dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=math.nan), dict(scaling="yarn", factor=2.0),
    dict(scaling="yarn", factor=2.0, original_length=100, beta_fast=1.0, beta_slow=1.0),
    dict(scaling="yarn", factor=2.0, original_length=100, beta_slow=0.0)])
def test_rope_plan_refusals(kw):
    with pytest.raises(L.LfError):
        L.RopePlan.make(**{**dict(head_dim=128), **kw})
    with pytest.raises(ValueError):
        L.RopePlan.make(128, layout="other")
    with pytest.raises(ValueError):
        L.RopePlan.make(128, scaling="other")


def _io(n=1, **kw):
    io = (L._RopeIo * n)()
    for i in range(n):
        io[i].x, io[i].out, io[i].heads, io[i].rotate = FAKE, FAKE, 2, 1
        io[i].x_stride[:] = io[i].out_stride[:] = (2560, 1280, 128)
        for name, value in kw.items():
            if name in ("x_stride", "out_stride"):
                getattr(io[i], name)[:] = value
            else:
                setattr(io[i], name, value)
    return io


def test_rope_refusals():
    plan = L.RopePlan.make(128)
    f = lambda pl=plan, batch=2, tokens=10, dtype=1, pos=p, pb=0, io=_io(), n=1: L.lib.lf_rope(  # noqa: E731
        None if pl is None else ctypes.byref(pl), batch, tokens, dtype, pos, pb, io, n, 0, None)
    assert f(pl=None) == 1 and f(io=None) == 1 and f(pos=None) == 1
    assert f(io=_io(x=None)) == 1 and f(io=_io(out=None)) == 1
    assert f(n=0) == 3 and f(io=_io(4), n=4) == 3 and f(batch=-1) == 3 and f(tokens=-1) == 3
    assert f(io=_io(heads=0)) == 3 and f(io=_io(heads=20000)) == 3 and f(tokens=1 << 24) == 3
    assert f(dtype=3) == 9 and f(dtype=-1) == 9 and f(pb=-1) == 9
    assert f(io=_io(x_stride=(-1, 1, 1))) == 9 and f(io=_io(out_stride=(0, 1280, 128))) == 9
    assert f(io=_io(x=FAKE + 1)) == 2 and f(dtype=0, io=_io(out=FAKE + 2)) == 2 and f(pos=P(FAKE + 2)) == 2
    for name, value in (("rot_dim", 3), ("rot_dim", 130), ("n_axes", 0), ("n_axes", 4), ("layout", 2), ("head_dim", 300)):
        bad = L.RopePlan.from_buffer_copy(plan)
        setattr(bad, name, value)
        assert f(pl=bad) == 9
    bad = L.RopePlan.from_buffer_copy(plan)
    bad.turns[5] = math.nan
    assert f(pl=bad) == 9
    bad = L.RopePlan.from_buffer_copy(plan)
    bad.axis_dims[0] = 126
    assert f(pl=bad) == 9
    assert f(batch=0) == 0 and f(tokens=0) == 0  # nothing to do, nothing launched


# ---------------------------------------------------------------- norms
def _vec(**kw):
    v = L._NormVectors()
    for n, a in kw.items():
        setattr(v, n, a)
    return v


def test_norm_refusals():
    def f(x=p, y=p, r=p, h=p, v=None, **kw):
        s = L.NormGateShape.make(**{**dict(rows=4, dim=64, post="rms"), **kw})
        return L.lib.lf_norm_gate(ctypes.byref(s), None if v is None else ctypes.byref(v), x, y, r, h, None)

    def raw(**kw):
        s = L.NormGateShape.make(4, 64)
        for n, a in kw.items():
            setattr(s, n, a)
        return L.lib.lf_norm_gate(ctypes.byref(s), None, p, p, p, p, None)

    assert L.lib.lf_norm_gate(None, None, p, p, p, p, None) == 1
    assert f(x=None) == 1 and f(r=None, h=None) == 1
    assert f(rows=-1) == 3 and f(dim=0) == 3 and f(dim=16385) == 3 and f(rows_per_group=0) == 3 and f(rows=1 << 31) == 3
    assert raw(x_dtype=3) == 9 and raw(y_dtype=-1) == 9 and raw(x_dtype=1, y_dtype=2) == 9 and raw(x_dtype=1, y_dtype=0) == 9
    assert raw(pre_norm=3) == 9 and raw(post_norm=-1) == 9
    assert f(eps=-1.0) == 9 and f(eps=math.nan) == 9 and f(residual_scale=math.inf) == 9
    assert f(pre="none") == 9                      # h without a norm
    assert f(y=None) == 9                          # a post norm without y
    assert f(post="none", v=_vec(post_w=FAKE)) == 9
    assert f(pre="none", h=None, v=_vec(scale=FAKE)) == 9
    assert f(y=None, post="none", v=_vec(gate=FAKE)) == 9
    assert f(v=_vec(scale=FAKE + 4)) == 2
    for n in "xyrh":
        assert f(**{n: mis}) == 2
    assert f(rows=0) == 0


def test_norm_bwd_refusals():
    s = L.NormGateShape.make(4, 64, post="rms")
    need = L.lf_norm_gate_bwd_workspace(s)
    assert need == (4 + 4 + 1) * 4 * 64 * 4

    def f(x=p, y=p, dr=p, dh=p, dx=p, dy=p, v=None, g=None, ws=p, n=need, s=s):
        ref = lambda t: None if t is None else ctypes.byref(t)  # noqa: E731
        return L.lib.lf_norm_gate_bwd(ctypes.byref(s), ref(v), x, y, dr, dh, dx, dy, ref(g), ws, n, None)

    assert f(x=None) == 1 and f(ws=None) == 1
    assert f(n=need - 1) == 12 and f(n=-1) == 9
    assert f(y=None) == 9 and f(g=_vec(gate=FAKE + 8)) == 2
    none = L.NormGateShape.make(4, 64)
    assert f(s=none, y=None) == 9                  # dy without y
    assert f(s=none, g=_vec(post_b=FAKE)) == 9
    for n in ("x", "y", "dr", "dh", "dx", "dy", "ws"):
        assert f(**{n: mis}) == 2
    assert L.lib.lf_norm_gate_bwd_workspace(None) == -1
    with pytest.raises(L.LfError):
        L.lf_norm_gate_bwd_workspace(L.NormGateShape.make(4, 0))
    big = L.NormGateShape.make(10 ** 6, 100, rows_per_group=1 << 62)
    assert L.lf_norm_gate_bwd_workspace(big) == (148 + 148 + 1) * 4 * 104 * 4


# ---------------------------------------------------------------- attention gradient
def test_attn_grad_refusals():
    sh = L.LfShape.make(1, 2, 128, 1560, 21, 1, 1, 3)
    need = L.lf_attn_bwd_workspace(sh)
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    assert need == 256 + up(2 * 4680 * 4) + up(2 * 525 * 4) + up(2 * 525 * 75 * 4)

    def f(s=sh, ws=p, n=need, cap=108, scale=0.0, **kw):
        a = dict(q=p, k=p, v=p, out=p, lo=p, dout=p, lse=p, lists=p, count=p, dq=p, dk=p, dv=p)
        a.update(kw)
        return L.lib.lf_block_sparse_attn_bwd(None if s is None else ctypes.byref(s), a["q"], a["k"], a["v"], a["out"],
                                              a["lo"], a["dout"], a["lse"], a["lists"], a["count"], cap, scale, a["dq"], a["dk"],
                                              a["dv"], ws, n, None)

    assert f(s=None) == 1 and f(ws=None) == 1 and f(ws=mis) == 2 and f(n=need - 1) == 12
    assert f(cap=-1) == 5 and f(scale=math.nan) == 9 and f(scale=math.inf) == 9
    assert f(s=L.LfShape.make(1, 2, 96, 1560, 21, 1, 1, 3)) == 3
    for n in ("q", "k", "v", "out", "dout", "lse", "lists", "count", "dq", "dk", "dv"):
        assert f(**{n: None}) == 1 and f(**{n: mis}) == 2
    assert f(lo=mis) == 2
    S = ctypes.byref(sh)
    g = L.lib.lf_block_sparse_attn_lse
    assert g(S, p, p, p, p, p, 108, 0.0, p, p, None, 0, p, 1 << 20, None) == 1
    assert g(S, p, p, p, p, p, 108, 0.0, p, p, mis, 0, p, 1 << 20, None) == 2
    assert g(S, p, p, p, p, p, 108, 0.0, p, mis, p, 0, p, 1 << 20, None) == 2
    assert g(S, p, p, p, p, p, -1, 0.0, p, None, p, 0, p, 1 << 20, None) == 5
    assert g(S, p, None, p, p, p, 108, 0.0, p, None, p, 0, p, 1 << 20, None) == 1
    assert L.lib.lf_attn_bwd_workspace(None) == -1
    with pytest.raises(L.LfError):
        L.lf_attn_bwd_workspace(L.LfShape.make(1, 2, 96, 1560, 21, 1, 1, 3))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,nc,kb,sm", [(1, 12, 3, 12, 148), (1, 2, 3, 12, 148), (1, 1, 1, 12, 148), (1, 12, 3, 1, 148),
                                          (1, 4, 37, 12, 148), (1, 12, 3, 12, 132), (1, 24, 3, 12, 148)])
def test_training_split_plan(B, H, nc, kb, sm, D):
    """The plain call's plan, with the slots that out_lo's sums need."""
    sh = L.LfShape.make(B, H, D, 1560, 18 + nc, 1, 1, nc)
    cap = L.lf_list_capacity(sh, 2, 4, kb)
    t, k, nbytes = L.lf_attn_lse_split_plan(sh, cap, sm)
    assert (t, k) == L.lf_attn_split_plan(sh, cap, sm)[:2]
    assert nbytes == t * k * 64 * (D + 3) * 4


def test_training_split_plan_refusals():
    sh, f = L.LfShape.make(1, 2, 128, 1560, 21, 1, 1, 3), L.lib.lf_attn_lse_split_plan
    t, k, b = (ctypes.byref(c()) for c in (ctypes.c_int32, ctypes.c_int32, ctypes.c_int64))
    assert f(None, 108, 148, t, k, b) == 1 and f(ctypes.byref(sh), -1, 148, t, k, b) == 5
    for args in ((None, k, b), (t, None, b), (t, k, None)):
        assert f(ctypes.byref(sh), 108, 148, *args) == 1
    with pytest.raises(L.LfError):
        L.lf_attn_lse_split_plan(L.LfShape.make(1, 2, 96, 1560, 21, 1, 1, 3), 108, 148)


def test_bindings_reject_cpu_tensors():
    x = torch.zeros(1, 2, 4, 128)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        L.lf_rope(L.RopePlan.make(128), [x], [x], torch.zeros(4, 1, dtype=torch.int32))


class _Steps:
    """An HSACall on the CPU whose library calls are counted, or refused, in place of running."""

    def __init__(self, monkeypatch):
        self.refuse, self.gradients = False, 0
        monkeypatch.setattr(L, "lf_pool", lambda *a, **k: None)
        monkeypatch.setattr(L, "lf_select_mask", self._step)
        monkeypatch.setattr(L, "lf_block_sparse_attn_lse", self._step)
        monkeypatch.setattr(L, "lf_block_sparse_attn_bwd", self._gradient)
        self.call = L.HSACall(L.LfShape.make(1, 1, 64, 64, 4, 1, 1, 1), 2, 1, 1, device="cpu", tail_pieces=1, train=True)

    def _step(self, *a, **k):
        if self.refuse:
            raise ValueError("refused")

    def _gradient(self, *a, **k):
        self.gradients += 1

    def backward(self):
        self.call.backward(*[None] * 7)


def test_gradient_after_a_refused_call_is_refused(monkeypatch):
    """An attention that did not run leaves nothing to take a gradient of, neither the first one nor a later one."""
    s = _Steps(monkeypatch)
    s.refuse = True
    with pytest.raises(ValueError, match="refused"):
        s.call.attend(None, None, None)
    with pytest.raises(ValueError, match="HSACall.backward"):
        s.backward()
    s.refuse = False
    s.call(None, None, None)
    s.backward()
    s.backward()  # the same call's gradient of another dout
    assert s.gradients == 2
    s.refuse = True
    with pytest.raises(ValueError, match="refused"):
        s.call.attend(None, None, None)
    with pytest.raises(ValueError, match="HSACall.backward"):
        s.backward()
    assert s.gradients == 2


def test_gradient_after_another_selection_is_refused(monkeypatch):
    """select() replaces the lists that the attention's log-sum-exp belongs to; attend() brings the two together again."""
    s = _Steps(monkeypatch)
    s.call(None, None, None)
    s.call.pool(None, None)  # the pooled vectors are not the gradient's
    s.backward()
    s.call.select()
    with pytest.raises(ValueError, match="HSACall.backward"):
        s.backward()
    s.call.attend(None, None, None)
    s.backward()
    s.refuse = True
    with pytest.raises(ValueError, match="refused"):
        s.call.select()      # it may have written some of the lists
    with pytest.raises(ValueError, match="HSACall.backward"):
        s.backward()
    assert s.gradients == 2


# ---------------------------------------------------------------- definitions against differences
def _difference(f, inputs, grads, seed):
    """<grad, d> against (f(x + e d) - f(x - e d)) / 2 e for a random direction of every input."""
    g = torch.Generator().manual_seed(seed)
    d = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in inputs]
    e = 1e-6
    up, down = f([t + e * u for t, u in zip(inputs, d)]), f([t - e * u for t, u in zip(inputs, d)])
    want = sum(float((a * u).sum()) for a, u in zip(grads, d))
    # central differences: e^2 of the third derivative (~1e-12) and 2^-53 |f| / e of the cancellation
    assert (up - down) / (2 * e) == pytest.approx(want, rel=1e-7, abs=1e-7 * (1 + abs(up)))


def test_attention_formula_against_differences():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, do = r(1, 2, 70, 16), r(1, 2, 140, 16), r(1, 2, 140, 16), r(1, 2, 70, 16)
    lists = torch.tensor([[[[0, 3], [2, 1]], [[1, 0], [3, 0]]]])
    mask = R.token_mask(1, 2, 70, 1, 2, lists, torch.tensor([[[2, 1], [0, 2]]]))
    (out, lse, dq, dk, dv), _, _ = R.attention_grads(q, k, v, do, mask, 0.3)
    _difference(lambda t: float((R.attention(*t, mask, 0.3)[0] * do).sum()), [q, k, v], [dq, dk, dv], 5)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_formula_against_differences(layout):
    g = torch.Generator().manual_seed(4)
    x, dy = (torch.randn(1, 2, 5, 12, generator=g, dtype=torch.float64) for _ in range(2))
    pos = torch.arange(5).unsqueeze(-1) * 7
    f, axis, amp = R.rope_frequencies((8,), 100.0, "yarn", 4.0, 16)
    dx, _ = R.rope(dy, pos, f, axis, amp, layout, 8, backward=True)
    _difference(lambda t: float((R.rope(t[0], pos, f, axis, amp, layout, 8)[0] * dy).sum()), [x], [dx], 6)
