"""The gated residual norms on the GPU against the definition in 64 bits: kinds, types, odd sizes, ragged
groups, absent parts, in place, outliers, and every gradient."""
import pytest
import torch

import block_sparse_attention_lf_b200 as L
from tests import block_ref as R

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NAMES = ("gate", "scale", "shift", "pre_w", "pre_b", "post_w", "post_b")
# A row sum adds at most 2 * 32 (a thread's elements) + 5 (its warp) + 16 (the team) terms one after another: each
# statistic is within 85 * 2^-24 = 5.1e-6 of its terms' sum, and up to three follow one another (post, pre, gradient).
SUM = 85 * 2.0 ** -24

CASES = [
    # rows, dim, per group, x, y, pre, post, vectors
    (1, 1536, 1, "bf16", "bf16", "layer", "none", "gate scale shift"),
    (37, 1536, 10, "fp32", "bf16", "rms", "rms", "gate scale shift pre_w post_w"),
    (300, 128, 7, "bf16", "bf16", "layer", "layer", " ".join(NAMES)),
    (65, 64, 65, "fp16", "fp16", "rms", "none", "gate scale"),
    (9, 2049, 4, "fp32", "fp32", "layer", "rms", " ".join(NAMES)),        # odd: no wide loads
    (50, 777, 50, "bf16", "bf16", "rms", "layer", "gate pre_w post_b"),
    (5, 1, 2, "fp32", "fp32", "rms", "rms", "gate scale shift"),          # one element a row
    (3, 3, 1, "fp16", "fp16", "layer", "none", "shift"),
    (12, 8192, 5, "fp32", "fp16", "layer", "rms", " ".join(NAMES)),       # two groups of eight a thread
    (4, 16384, 4, "bf16", "bf16", "rms", "layer", " ".join(NAMES)),       # four
    (6, 12289, 4, "fp32", "bf16", "layer", "layer", "gate post_w"),
    (2000, 256, 1, "bf16", "bf16", "layer", "none", "gate scale shift"),  # a group a row
    (1111, 320, 600, "fp32", "fp32", "rms", "rms", " ".join(NAMES)),      # groups cross the CTAs' rows
    # more rows than four an SM: a CTA's teams share a group's vectors, or keep their own for short groups
    (700, 1536, 130, "bf16", "bf16", "layer", "layer", " ".join(NAMES)),
    (1300, 512, 64, "bf16", "bf16", "rms", "rms", " ".join(NAMES)),       # a CTA meets two groups
    (650, 2048, 100, "fp32", "fp32", "rms", "layer", " ".join(NAMES)),    # no room for a ring
    (601, 1000, 64, "fp32", "bf16", "layer", "rms", "gate shift pre_w"),  # threads past the row's end
    (777, 1333, 300, "fp16", "fp16", "layer", "layer", " ".join(NAMES)),  # odd
    (900, 1992, 3, "fp32", "bf16", "rms", "rms", "gate scale shift"),
    (640, 1024, 63, "bf16", "bf16", "layer", "none", "scale shift"),
]


def _inputs(case, seed=0):
    rows, dim, per, xt, yt, pre, post, names = case
    g = torch.Generator().manual_seed(rows * 7 + dim + seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    groups = -(-rows // per)
    x, y = (r(rows, dim) * 2 + 0.3).to(T[xt]), (r(rows, dim) - 0.2).to(T[yt])
    dr, dh = r(rows, dim).to(T[xt]), r(rows, dim).to(T[yt])
    v = {}
    for n in NAMES:
        if n in names.split():
            v[n] = r(groups, dim) * 0.5 if n in NAMES[:3] else r(dim) * 0.2 + (1.0 if n.endswith("w") else 0.0)
    shape = L.NormGateShape.make(rows, dim, per, T[xt], T[yt], pre, post, 1e-6, 0.75)
    return shape, x, y, dr, dh, v


def _ref(case, x, y, dr, dh, v, alpha=0.75):
    _, _, per, _, _, pre, post, _ = case
    leaf = {n: t.double().requires_grad_() for n, t in v.items()}
    xx = x.double().requires_grad_()
    yy = None if y is None else y.double().requires_grad_()
    r, h = R.norm_gate(xx, yy, per, alpha, pre, post, 1e-6, leaf)
    loss = 0.0
    if dr is not None:
        loss = loss + (r * dr.double()).sum()
    if dh is not None and h is not None:
        loss = loss + (h * dh.double()).sum()
    wrt = [xx] + ([yy] if yy is not None else []) + list(leaf.values())
    got = torch.autograd.grad(loss, wrt, allow_unused=True) if torch.is_tensor(loss) else [None] * len(wrt)
    got = [torch.zeros_like(w) if t is None else t for t, w in zip(got, wrt)]
    grads = dict(zip(["x"] + (["y"] if yy is not None else []) + list(leaf), got))
    return r.detach(), None if h is None else h.detach(), grads


def _close(got, ref, dtype, steps, what, axis=-1):
    """Within half a rounding step of each element, and of `steps` chained row sums of the row's size (2-norm / sqrt n,
    times 8 for the largest of a row's elements that one sum's error can meet)."""
    got, ref = got.double().cpu(), ref.double()
    assert torch.isfinite(got).all()
    rms = ref.square().mean(axis, keepdim=True).sqrt()
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    bound = R.EPS[dtype] * ref.abs() + steps * SUM * 8 * torch.maximum(rms, ref.abs()) + tiny
    worst = ((got - ref).abs() - bound).max()
    assert worst <= 0, (what, float(worst))
    off = float((got - ref).norm() / ref.norm().clamp_min(1e-30))
    assert off <= R.EPS[dtype] + steps * SUM, (what, off)


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    shape, x, y, _, _, v = _inputs(case)
    xd, yd, vd = x.cuda(), y.cuda(), {n: t.cuda() for n, t in v.items()}
    r, h = torch.empty_like(xd), torch.empty_like(yd)
    L.lf_norm_gate(shape, xd, yd, r, h, **vd)
    rr, hh, _ = _ref(case, x, y, None, None, v)
    if case[1] > 3:
        _close(r, rr, r.dtype, 1, "r")
        _close(h, hh, h.dtype, 2, "h")
    else:
        _tiny_rows(r, rr)
        _tiny_rows(h, hh)
    # in place
    L.lf_norm_gate(shape, xd, yd, xd, yd, **vd)
    assert torch.equal(xd, r) and torch.equal(yd, h)


def _tiny_rows(got, ref):
    """Rows of one to three elements: a layer or RMS norm of few elements is +-1, or amplifies x's rounding where they
    nearly agree, so only the size of the deviation is held (half a step and 2^-12 of the largest value)."""
    got, ref = got.double().cpu(), ref.double()
    bound = R.EPS[torch.float16] * 2 * ref.abs() + 2.0 ** -12 * ref.abs().max()
    assert ((got - ref).abs() <= bound).all()


@pytest.mark.parametrize("case", CASES)
def test_gradients(case):
    shape, x, y, dr, dh, v = _inputs(case, 1)
    xd, yd, drd, dhd = x.cuda(), y.cuda(), dr.cuda(), dh.cuda()
    vd = {n: t.cuda() for n, t in v.items()}
    dx, dy = torch.empty_like(xd), torch.empty_like(yd)
    grads = {n: torch.full_like(t, 9.0) for n, t in vd.items()}
    ws = torch.full((L.lf_norm_gate_bwd_workspace(shape),), 255, dtype=torch.uint8, device="cuda")  # NaN patterns
    L.lf_norm_gate_bwd(shape, xd, yd, drd, dhd, dx, dy, grads, ws, **vd)
    _, _, ref = _ref(case, x, y, dr, dh, v)
    if case[1] > 3:
        _close(dx, ref["x"], dx.dtype, 3, "dx")
        _close(dy, ref["y"], dy.dtype, 3, "dy")
    for n, t in grads.items():
        # column sums: at most 296 CTAs' partial sums and a CTA's rows, one after another, over terms that are
        # themselves within three chained row sums
        terms = case[0] ** 0.5
        bound = (3 * SUM * 8 + 400 * 2.0 ** -24) * (ref[n].abs() + 8 * terms) * 4
        if case[1] <= 3:
            bound = bound + 2.0 ** -8
        err = (t.double().cpu() - ref[n]).abs()
        assert (err <= bound).all(), (n, float((err - bound).max()))
    # the same bits again, whatever the workspace held; and in place
    again = {n: torch.empty_like(t) for n, t in grads.items()}
    ws.zero_()
    L.lf_norm_gate_bwd(shape, xd, yd, drd, dhd, drd, dhd, again, ws, **vd)
    assert torch.equal(drd, dx) and torch.equal(dhd, dy)
    assert all(torch.equal(again[n], t) for n, t in grads.items())


@pytest.mark.parametrize("part", ["no_y", "no_pre", "no_dr", "no_dh", "only_dx", "no_vectors"])
def test_absent_parts(part):
    case = (70, 512, 32, "fp32", "bf16", "none" if part == "no_pre" else "layer", "none" if part == "no_y" else "rms",
            "" if part == "no_vectors" else {"no_y": "scale shift pre_w", "no_pre": "gate post_w post_b"}.get(
                part, "gate scale shift pre_w post_b"))
    shape, x, y, dr, dh, v = _inputs(case, 2)
    if part == "no_y":
        y = None
    if part == "no_pre" or part == "no_dh":
        dh = None
    if part == "no_dr":
        dr = None
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    xd, yd, vd = c(x), c(y), {n: t.cuda() for n, t in v.items()}
    r, h = torch.empty_like(xd), None if part == "no_pre" else torch.empty(70, 512, dtype=torch.bfloat16, device="cuda")
    L.lf_norm_gate(shape, xd, yd, None if part == "no_vectors" else r, h, **vd)
    rr, hh, ref = _ref(case, x, y, dr, dh, v)
    if part != "no_vectors":
        _close(r, rr, r.dtype, 1, "r")
    if h is not None:
        _close(h, hh, h.dtype, 2, "h")
    dx = torch.empty_like(xd)
    dy = None if y is None or part == "only_dx" else torch.empty_like(yd)
    grads = {} if part == "only_dx" else {n: torch.empty_like(t) for n, t in vd.items()}
    ws = torch.empty(L.lf_norm_gate_bwd_workspace(shape), dtype=torch.uint8, device="cuda")
    L.lf_norm_gate_bwd(shape, xd, yd, c(dr), c(dh), dx, dy, grads, ws, **vd)
    _close(dx, ref["x"], dx.dtype, 3, "dx")
    if dy is not None:
        _close(dy, ref["y"], dy.dtype, 3, "dy")
    for n, t in grads.items():
        bound = (3 * SUM * 8 + 400 * 2.0 ** -24) * (ref[n].abs() + 8 * 70 ** 0.5) * 4
        assert ((t.double().cpu() - ref[n]).abs() <= bound).all(), n


def test_gradient_of_a_gate_that_is_not_there():
    """A gate of ones may be left out and its gradient still taken."""
    case = (40, 128, 40, "fp32", "fp32", "rms", "layer", "")
    shape, x, y, dr, dh, _ = _inputs(case, 3)
    ws = torch.empty(L.lf_norm_gate_bwd_workspace(shape), dtype=torch.uint8, device="cuda")
    args = [t.cuda() for t in (x, y, dr, dh)]
    g = {"gate": torch.empty(1, 128, device="cuda"), "pre_b": torch.empty(128, device="cuda")}
    L.lf_norm_gate_bwd(shape, *args, None, None, g, ws)
    h = {"gate": torch.empty(1, 128, device="cuda"), "pre_b": torch.empty(128, device="cuda")}
    L.lf_norm_gate_bwd(shape, *args, None, None, h, ws, gate=torch.ones(1, 128, device="cuda"),
                       pre_b=torch.zeros(128, device="cuda"))
    assert torch.equal(g["gate"], h["gate"]) and torch.equal(g["pre_b"], h["pre_b"])


def test_mean_far_from_deviation():
    """Rows of mean 1000 and deviation 1: a difference of squares in fp32 would keep no digit of the variance. The mean
    itself is within 85 * 2^-24 * 1000 = 5e-3 worst, so values are held to 1e-2 of a deviation."""
    g = torch.Generator().manual_seed(21)
    x = torch.randn(16, 1536, generator=g) + 1000
    shape = L.NormGateShape.make(16, 1536, None, torch.float32, torch.float32, "layer", "none")
    h = torch.empty(16, 1536, device="cuda")
    L.lf_norm_gate(shape, x.cuda(), None, None, h)
    ref = R.norm(x.double(), "layer", 1e-6)
    assert float((h.double().cpu() - ref).abs().max()) < 1e-2
    x = torch.zeros(4, 1536)
    x[:, 0] = 3e4
    L.lf_norm_gate(L.NormGateShape.make(4, 1536, None, torch.float32, torch.float32, "layer"), x.cuda(), None, None, h[:4])
    ref = R.norm(x.double(), "layer", 1e-6)
    assert float((h[:4].double().cpu() - ref).abs().max() / ref.abs().max()) < 4 * SUM


def test_nonfinite_rows_stay_theirs():
    """A row with a NaN or an infinity changes no other row."""
    case = (33, 256, 33, "bf16", "bf16", "layer", "rms", "gate scale shift")
    shape, x, y, _, _, v = _inputs(case, 4)
    vd = {n: t.cuda() for n, t in v.items()}
    r, h, r2, h2 = (torch.empty(33, 256, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    L.lf_norm_gate(shape, x.cuda(), y.cuda(), r, h, **vd)
    x[5, 7], y[9, 0] = float("nan"), float("inf")
    L.lf_norm_gate(shape, x.cuda(), y.cuda(), r2, h2, **vd)
    keep = torch.ones(33, dtype=torch.bool)
    keep[[5, 9]] = False
    assert torch.equal(r[keep], r2[keep]) and torch.equal(h[keep], h2[keep])
    assert h2[5].isnan().all() and h2[9].isnan().any()


def test_no_rows():
    shape = L.NormGateShape.make(0, 64, post="rms")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    L.lf_norm_gate(shape, e, e, e, e)
    g = {"pre_w": torch.ones(64, device="cuda"), "gate": torch.empty(0, 64, device="cuda")}
    L.lf_norm_gate_bwd(shape, e, e, e, e, e, e, g, torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert (g["pre_w"] == 0).all()


def test_shapes_are_checked():
    shape = L.NormGateShape.make(4, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        L.lf_norm_gate(shape, x[:3], x, x, x)
    with pytest.raises(TypeError):
        L.lf_norm_gate(shape, x.float(), x, x, x)
    with pytest.raises(ValueError):
        L.lf_norm_gate(shape, x, x, x, x, gate=torch.zeros(2, 64, device="cuda"))
    with pytest.raises(ValueError):
        L.lf_norm_gate(shape, torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")[:, ::2], x, x, x)
    with pytest.raises(ValueError):
        L.lf_norm_gate_bwd(shape, x, x, x, x, x, x, {"bias": x}, x.view(torch.uint8))


def test_gradient_against_differences():
    """<gradients, d> against differences of the kernel's forward in fp32. Step 2^-7: the differences' own error is
    e^2 / 6 of the third derivative (about 1e-5 of the sum) and 2^-20 sqrt(n) |h| / e of rounding (about 1e-4)."""
    case = (24, 96, 9, "fp32", "fp32", "layer", "rms", " ".join(NAMES))
    shape, x, y, dr, dh, v = _inputs(case, 5)
    g = torch.Generator().manual_seed(23)
    ts = {"x": x.cuda(), "y": y.cuda(), **{n: t.cuda() for n, t in v.items()}}
    ds = {n: torch.randn(t.shape, generator=g).cuda() for n, t in ts.items()}
    e = 2.0 ** -7

    def loss(sign):
        a = {n: t + sign * e * ds[n] for n, t in ts.items()}
        r, h = torch.empty_like(ts["x"]), torch.empty_like(ts["x"])
        L.lf_norm_gate(shape, a.pop("x"), a.pop("y"), r, h, **a)
        return float((r.double() * dr.cuda().double()).sum() + (h.double() * dh.cuda().double()).sum())

    got = {n: torch.empty_like(t) for n, t in ts.items()}
    ws = torch.empty(L.lf_norm_gate_bwd_workspace(shape), dtype=torch.uint8, device="cuda")
    L.lf_norm_gate_bwd(shape, ts["x"], ts["y"], dr.cuda(), dh.cuda(), got["x"], got["y"],
                       {n: got[n] for n in v}, ws, **{n: ts[n] for n in v})
    want = sum(float((got[n].double() * ds[n].double()).sum()) for n in ts)
    size = sum(float((got[n].double() * ds[n].double()).square().sum()) for n in ts) ** 0.5
    assert abs((loss(1) - loss(-1)) / (2 * e) - want) <= 2e-3 * size


def test_graph_and_stream():
    case = (100, 256, 50, "bf16", "bf16", "layer", "rms", " ".join(NAMES))
    shape, x, y, dr, dh, v = _inputs(case, 6)
    a = [t.cuda() for t in (x, y, dr, dh)]
    vd = {n: t.cuda() for n, t in v.items()}
    ws = torch.empty(L.lf_norm_gate_bwd_workspace(shape), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(a[0]) for _ in range(4)]
    grads = {n: torch.empty_like(t) for n, t in vd.items()}

    def step():
        L.lf_norm_gate(shape, a[0], a[1], out[0], out[1], **vd)
        L.lf_norm_gate_bwd(shape, *a, out[2], out[3], grads, ws, **vd)

    step()
    want = [t.clone() for t in out + list(grads.values())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in out + list(grads.values()):
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(t, w) for t, w in zip(out + list(grads.values()), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in out + list(grads.values()):
        t.zero_()
    graph.replay()
    assert all(torch.equal(t, w) for t, w in zip(out + list(grads.values()), want))


# ---------------------------------------------------------------- many rows a team
def _terms(shape, x, y, dr, dh, v):
    """In 64 bits: (r, h, dx, dy, what each row adds to each vector's gradient), and for dx and dy the size of the
    terms that their last subtraction takes apart. Written from the formulas of the gradient, not by autograd."""
    f = lambda t: None if t is None else t.double()  # noqa: E731
    per, alpha, eps = shape.rows_per_group, float(shape.residual_scale), float(shape.eps)
    at = torch.arange(shape.rows, device=x.device) // per
    one, zero = torch.ones((), dtype=torch.float64, device=x.device), torch.zeros((), dtype=torch.float64, device=x.device)
    vec = {n: f(v[n]) if n in v else (zero if n in ("shift", "scale") or n.endswith("b") else one) for n in NAMES}
    gate, scale, shift = (vec[n][at] if n in v else vec[n] for n in NAMES[:3])
    w1, b1, w2, b2 = (vec[n] for n in NAMES[3:])
    x, y, dr, dh = f(x), f(y), f(dr), f(dh)

    def hat(t, kind):
        if kind == 0:
            return t, 1.0
        t = t - t.mean(-1, keepdim=True) if kind == 2 else t
        rs = torch.rsqrt(t.square().mean(-1, keepdim=True) + eps)
        return t * rs, rs

    def back(d, n, rs, kind):
        if kind == 0:
            return d, d.abs()
        size = rs * (d.abs() + n.abs() * (d * n).abs().mean(-1, keepdim=True))
        out = d - n * (d * n).mean(-1, keepdim=True)
        if kind == 2:
            out, size = out - d.mean(-1, keepdim=True), size + rs * d.abs().mean(-1, keepdim=True)
        return rs * out, size

    m, rs2 = hat(y, shape.post_norm)
    u = m * w2 + b2
    r = alpha * x + gate * u
    n, rs1 = hat(r, shape.pre_norm)
    a = n * w1 + b1
    d, s1 = back(dh * (1 + scale) * w1, n, rs1, shape.pre_norm)
    d, s1 = d + dr, s1 + dr.abs()
    dy, s2 = back(d * gate * w2, m, rs2, shape.post_norm)
    s2 = s2 + (rs2 * (gate * w2).abs() * s1 if shape.post_norm else (gate * w2).abs() * s1)
    terms = {"gate": d * u, "scale": dh * a, "shift": dh, "pre_w": dh * (1 + scale) * n, "pre_b": dh * (1 + scale),
             "post_w": d * gate * m, "post_b": d * gate}
    return r, a * (1 + scale) + shift, (alpha * d, abs(alpha) * s1), (dy, s2), {k: t.expand_as(x) for k, t in terms.items()}


def _sums(t, name, shape):
    """Sums over a group's rows, or over all."""
    if name not in NAMES[:3]:
        return t.sum(0)
    pad = torch.zeros(shape.groups * shape.rows_per_group - shape.rows, shape.dim, dtype=t.dtype, device=t.device)
    return torch.cat([t, pad]).view(shape.groups, shape.rows_per_group, shape.dim).sum(1)


MANY = [
    # the group kernel, threads with every column of a row: eight rows a team over a ring of four
    (9001, 1536, 1560, "bf16", "bf16", "layer", "layer", " ".join(NAMES)),
    (7000, 1536, 3000, "fp32", "bf16", "rms", "rms", "gate scale shift pre_w post_w"),
    (12000, 512, 700, "bf16", "bf16", "layer", "none", "gate scale shift"),
    (6000, 768, 97, "fp16", "fp16", "rms", "layer", " ".join(NAMES)),      # threads past the row's end
    (3000, 2048, 400, "fp32", "fp32", "layer", "rms", " ".join(NAMES)),    # no ring forward
    (6001, 1333, 500, "bf16", "bf16", "rms", "none", "gate scale"),        # odd: loaded directly
    # the register kernel: every team its own groups
    (20000, 1024, 16, "bf16", "bf16", "layer", "rms", "gate scale shift"),
    (9000, 512, 1, "bf16", "bf16", "layer", "none", "gate scale shift"),
    (12003, 256, 50, "fp32", "fp16", "rms", "rms", " ".join(NAMES)),
    # rows of a CTA each
    (1500, 4096, 200, "bf16", "bf16", "layer", "layer", " ".join(NAMES)),
    (1300, 5120, 1300, "fp32", "bf16", "rms", "rms", "gate scale shift pre_w post_w"),
    (1200, 8192, 64, "fp16", "fp16", "layer", "none", "gate scale shift"),
    (900, 12288, 300, "bf16", "bf16", "rms", "layer", " ".join(NAMES)),
    (800, 16384, 100, "fp32", "fp32", "layer", "rms", " ".join(NAMES)),
    (1000, 2600, 7, "bf16", "bf16", "layer", "layer", "gate scale shift post_b"),
    (700, 4099, 150, "fp32", "bf16", "rms", "none", "gate scale"),
]


@pytest.mark.parametrize("case", MANY)
def test_many_rows_a_team(case):
    """Rings whose stages are used again and again, several groups a CTA, and gradients of vectors held row by row."""
    shape, *ts, v = _inputs(case, 7)
    x, y, dr, dh = (t.cuda() for t in ts)
    vd = {n: t.cuda() for n, t in v.items()}
    r, h, dx, dy = torch.empty_like(x), torch.empty_like(y), torch.empty_like(x), torch.empty_like(y)
    grads = {n: torch.full_like(t, 9.0) for n, t in vd.items()}
    ws = torch.full((L.lf_norm_gate_bwd_workspace(shape),), 255, dtype=torch.uint8, device="cuda")
    L.lf_norm_gate(shape, x, y, r, h, **vd)
    L.lf_norm_gate_bwd(shape, x, y, dr, dh, dx, dy, grads, ws, **vd)
    rr, hh, (dxr, _), (dyr, _), terms = _terms(shape, x, y, dr, dh, vd)
    for got, ref, steps, what in ((r, rr, 1, "r"), (h, hh, 2, "h"), (dx, dxr, 3, "dx"), (dy, dyr, 3, "dy")):
        _close(got, ref.cpu(), got.dtype, steps, what)
    _hold_vectors(shape, grads, terms)
    # in place, and the same bits
    again = {n: torch.empty_like(t) for n, t in grads.items()}
    L.lf_norm_gate_bwd(shape, x, y, dr, dh, dr, dh, again, ws, **vd)
    assert torch.equal(dr, dx) and torch.equal(dh, dy) and all(torch.equal(again[n], t) for n, t in grads.items())
    L.lf_norm_gate(shape, x, y, x, y, **vd)
    assert torch.equal(x, r) and torch.equal(y, h)


def _hold_vectors(shape, grads, terms):
    """A row's term is within three chained row sums (as dx is, _close); a column adds at most its rows, or the rows
    of a CTA and then 148 CTAs' partial sums by 32 threads, one after another, 2^-24 of the terms' sizes each; and two
    products. In norm: the terms' errors add up as the terms do."""
    for n, got in grads.items():
        t, got = terms[n], got.double()
        ref, size = _sums(t, n, shape), _sums(t.abs(), n, shape)
        rms = _sums(t.square().mean(-1, keepdim=True).sqrt().expand_as(t), n, shape)
        chain = min(shape.rows_per_group if n in NAMES[:3] else shape.rows, -(-shape.rows // 148) + 148) + 4
        bound = 3 * SUM * 8 * torch.maximum(rms, size) + chain * 2.0 ** -24 * size
        worst = float(((got - ref).abs() - bound).max())
        assert torch.isfinite(got).all() and worst <= 0, (n, worst)
        off = float((got - ref).norm() / ref.norm().clamp_min(1e-30))
        assert off <= 3 * SUM + chain * 2.0 ** -24, (n, off)


TIGHT = [c for c in CASES if c[1] > 3] + [
    (2001, 256, 1, "bf16", "bf16", "rms", "layer", " ".join(NAMES)),
]


@pytest.mark.parametrize("case", TIGHT)
def test_vector_gradients_row_by_row(case):
    """The gradients of gate, scale, shift, weights and biases within what their own group's rows allow."""
    shape, *ts, v = _inputs(case, 8)
    x, y, dr, dh = (t.cuda() for t in ts)
    vd = {n: t.cuda() for n, t in v.items()}
    grads = {n: torch.full_like(t, 9.0) for n, t in vd.items()}
    ws = torch.empty(L.lf_norm_gate_bwd_workspace(shape), dtype=torch.uint8, device="cuda")
    L.lf_norm_gate_bwd(shape, x, y, dr, dh, None, None, grads, ws, **vd)
    _hold_vectors(shape, grads, _terms(shape, x, y, dr, dh, vd)[4])


@pytest.mark.parametrize("dim", [1, 2, 3])
@pytest.mark.parametrize("pre,post", [("rms", "rms"), ("layer", "rms"), ("rms", "layer"), ("layer", "none")])
@pytest.mark.parametrize("types", [("fp32", "fp32"), ("bf16", "bf16"), ("fp32", "fp16")])
def test_rows_of_few_elements(dim, pre, post, types):
    """Rows of one to three elements, with eps = 1 so that no norm divides by almost nothing: half a step, and three
    chained statistics of the terms that the gradient's subtractions take apart. A statistic is off by 2^-24 for each
    of its sum's dim terms (zeros add no error), four for 2 ulp of 1 / deviation, three for eps, the mean and the
    product; 1 / deviation is at most 1, and a row's values, of size `big`, move it by as much at most."""
    case = (45, dim, 9, *types, pre, post, "gate scale shift pre_w" + (" post_w post_b" if post != "none" else ""))
    _, *ts, v = _inputs(case, 9)
    shape = L.NormGateShape.make(45, dim, 9, T[types[0]], T[types[1]], pre, post, 1.0, 0.75)
    x, y, dr, dh = (t.cuda() for t in ts)
    vd = {n: t.cuda() for n, t in v.items()}
    r, h, dx, dy = torch.empty_like(x), torch.empty_like(y), torch.empty_like(x), torch.empty_like(y)
    grads = {n: torch.full_like(t, 9.0) for n, t in vd.items()}
    ws = torch.empty(L.lf_norm_gate_bwd_workspace(shape), dtype=torch.uint8, device="cuda")
    L.lf_norm_gate(shape, x, y, r, h, **vd)
    L.lf_norm_gate_bwd(shape, x, y, dr, dh, dx, dy, grads, ws, **vd)
    rr, hh, *sized, terms = _terms(shape, x, y, dr, dh, vd)
    big, few = max(float(t.abs().max()) for t in (x, y)), 3 * (dim + 7) * 2.0 ** -24
    for got, (ref, size) in zip((r, h, dx, dy), ((rr, big * (1 + rr.abs())), (hh, big * (1 + hh.abs())), *sized)):
        tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
        bound = R.EPS[got.dtype] * ref.abs() + few * (1 + big) * size + tiny
        err = (got.double() - ref).abs()
        assert (err <= bound).all(), float((err - bound).max())
    for n, t in grads.items():
        size = _sums(terms[n].abs(), n, shape) + _sums(torch.ones_like(terms[n]), n, shape)
        assert ((t.double() - _sums(terms[n], n, shape)).abs() <= few * (1 + big) * size).all(), n
