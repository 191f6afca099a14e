"""Work measured for the training and block-level operators around an HSA call.

Three kinds of case: ``attn`` (block-sparse attention with its log-sum-exp, then
its gradient), ``rope`` (rotary positions from token-major projections to the
call's head-major layout, and the gradient) and ``norm`` (residual update with
gate and norms on both sides of a block, and its gradient). ``run`` computes a
case with elementary torch operations, or through the library where ``own`` is
true. Sizes are those of the 480p workloads (30 x 52 = 1560 tokens a frame,
three-frame chunks, 12 heads of 128, model width 1536) and of the tiny one.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZEOF = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases
def _attn(name, B, H, D, F, frames, sink, recent, cur, kf, kb, ragged=False):
    c = dict(kind="attn", B=B, H=H, D=D, F=F, frames=frames, sink=sink, recent=recent, cur=cur, kf=kf, kb=kb,
             ragged=ragged)
    return dict(c, name=name) if name else c


def _rope(name, B, H, L, D, rot, layout, axes, dtype, scaling="none", factor=1.0, original=0, start=0,
          fused=True, backward=False, base=10000.0):
    c = dict(kind="rope", B=B, H=H, L=L, D=D, rot=rot, layout=layout, axes=axes, dtype=dtype, scaling=scaling,
             factor=factor, original=original, start=start, fused=fused, backward=backward, base=base)
    return dict(c, name=name) if name else c


def _norm(name, rows, dim, per_group, x_dtype, y_dtype, pre, post, affine, backward, alpha=1.0):
    c = dict(kind="norm", rows=rows, dim=dim, per_group=per_group, x_dtype=x_dtype, y_dtype=y_dtype, pre=pre,
             post=post, affine=affine, backward=backward, alpha=alpha)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a fine-tuning step's attention in the smallest model: launches count
        _attn("attn_tiny", 1, 2, 64, 256, 9, 1, 1, 2, 2, 2),
        # one layer of the 480p model at 80 % sparsity, forward and gradient
        _attn("attn_layer480p", 1, 12, 128, 1560, 21, 1, 1, 3, 4, 12),
        # a frame that no block size divides, uneven lists, some of them empty
        _attn("attn_ragged", 2, 5, 128, 777, 13, 1, 1, 2, 3, 7, ragged=True),
        # the same layer deep into a long video, 90 % sparsity
        _attn("attn_longvideo480p", 1, 12, 128, 1560, 65, 1, 1, 3, 4, 18),
        # one new token of a sequence far past the trained length
        _rope("rope_one_token", 1, 12, 1, 128, 128, "half", 1, "bf16", scaling="yarn", factor=16.0, original=8192,
              start=100003),
        # a chunk's fused projection: q and k rotated in time, height and width, v moved, all to head-major
        _rope("rope_chunk480p", 1, 12, 4680, 128, 128, "interleaved", 3, "bf16"),
        # its gradient in fp32, half of each head rotated, the time axis stretched
        _rope("rope_grad_partial", 2, 12, 4680, 128, 64, "half", 1, "fp32", scaling="linear", factor=4.0, start=12345,
              backward=True),
        # all 21 frames of a rollout's keys re-rotated at once
        _rope("rope_rollout480p", 1, 12, 32760, 128, 128, "half", 3, "bf16", scaling="ntk", factor=2.0, fused=False),
        # the residual update of one token when serving
        _norm("norm_one_token", 1, 1536, 1, "bf16", "bf16", "rms", "rms", True, False),
        # a chunk between two blocks, modulation per frame
        _norm("norm_chunk480p", 4680, 1536, 1560, "bf16", "bf16", "layer", "none", False, False),
        # a training step of the same with an fp32 residual stream, norms on both sides
        _norm("norm_step_chunk480p", 4680, 1536, 1560, "fp32", "bf16", "rms", "rms", True, True),
        # a training step over a whole rollout
        _norm("norm_step_rollout480p", 32760, 1536, 1560, "bf16", "bf16", "layer", "layer", True, True, alpha=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["attn", "rope", "norm"])
    if kind == "attn":
        while True:
            F = _log(rng, 1, 1560)
            bpf = -(-F // 64)
            cur, sink, recent = rng.randint(1, 3), rng.randint(0, 2), rng.randint(0, 2)
            frames = cur + sink + recent + _log(rng, 1, 61) - 1
            c = _attn(None, rng.randint(1, 2), rng.randint(1, 12), rng.choice([64, 128, 128]), F, frames, sink, recent,
                      cur, rng.randint(1, 6), rng.randint(1, bpf), ragged=rng.random() < 0.5)
            cap = (sink + recent + cur + min(c["kf"], frames - sink - recent - cur)) * c["kb"]
            if c["B"] * c["H"] * cur * bpf * cap <= 900 * 162 and c["B"] * c["H"] * frames * F <= 12 * 65 * 1560:
                return c
    if kind == "rope":
        D = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256])
        rot = D if rng.random() < 0.6 else 2 * rng.randint(3, D // 2)
        axes = 1 if rot < 12 else rng.choice([1, 1, 2, 3])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        while True:
            B, H, L = rng.randint(1, 2), rng.randint(1, 24), _log(rng, 1, 32760)
            if B * H * L * D * SIZEOF[dtype] <= 2 * 12 * 4680 * 128 * 4:
                break
        factor = 1.0 if scaling == "none" else rng.uniform(1.5, 32.0)
        return _rope(None, B, H, L, D, rot, rng.choice(["interleaved", "half"]), axes, dtype, scaling=scaling,
                     factor=factor, original=_log(rng, 64, 16384) if scaling == "yarn" else 0,
                     start=0 if axes > 1 else _log(rng, 1, 1 << 20) - 1, fused=rng.random() < 0.5,
                     backward=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]))
    while True:
        rows, dim = _log(rng, 1, 32760), _log(rng, 64, 8192)
        if rng.random() < 0.7:
            dim = -(-dim // 8) * 8
        if rows * dim <= 32760 * 1536:
            break
    x_dtype, y_dtype = rng.choice([("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16"),
                                   ("fp32", "fp16")])
    if x_dtype == "fp32":
        rows = max(1, rows // 2)
    return _norm(None, rows, dim, _log(rng, max(1, rows // 64), rows), x_dtype, y_dtype,
                 rng.choice(["rms", "layer"]), rng.choice(["none", "rms", "layer"]), rng.random() < 0.5,
                 rng.random() < 0.5, alpha=rng.choice([1.0, 0.5]))


def work(case):
    c = case
    if c["kind"] == "attn":
        bpf = -(-c["F"] // 64)
        mean = c["F"] / bpf                      # tokens a block holds on average
        rows = c["B"] * c["H"] * c["cur"] * bpf
        cap = _cap(c) * (0.5 if c["ragged"] else 1.0)
        pairs = rows * cap * mean * mean
        q = c["B"] * c["H"] * c["cur"] * c["F"] * c["D"] * 2
        kv = c["B"] * c["H"] * c["frames"] * c["F"] * c["D"] * 2
        # read q, k, v, dout; write out, dq, dk, dv and the row's log-sum-exp
        return {"bytes": 4 * q + 4 * kv + c["B"] * c["H"] * c["cur"] * c["F"] * 4, "flops": 7 * 2 * pairs * c["D"]}
    if c["kind"] == "rope":
        n = c["B"] * c["H"] * c["L"] * c["D"] * (3 if c["fused"] else 1)
        return {"bytes": 2 * n * SIZEOF[c["dtype"]] + 4 * c["L"] * c["axes"], "flops": 4 * n}
    n = c["rows"] * c["dim"]
    x, y = SIZEOF[c["x_dtype"]], SIZEOF[c["y_dtype"]]
    groups = -(-c["rows"] // c["per_group"])
    if not c["backward"]:
        return {"bytes": n * (2 * x + 2 * y) + 3 * groups * c["dim"] * 4, "flops": 16 * n}
    # x, y, dr, dh read; r, h, dx, dy written; vectors and their gradients
    return {"bytes": n * (4 * x + 4 * y) + 6 * groups * c["dim"] * 4, "flops": 48 * n}


# ---------------------------------------------------------------- inputs
def _cap(c):
    forced = c["sink"] + c["recent"] + c["cur"]
    return (forced + min(c["kf"], c["frames"] - forced)) * c["kb"]


def _axis_dims(c):
    """Rotated dimensions of each axis: even parts, the first one takes what is left."""
    each = (c["rot"] // c["axes"]) // 2 * 2
    return [c["rot"] - (c["axes"] - 1) * each] + [each] * (c["axes"] - 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, by=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * by).to(dtype)

    if case["kind"] == "attn":
        return _prepare_attn(case, g, normal)
    if case["kind"] == "rope":
        return _prepare_rope(case, g, normal)
    return _prepare_norm(case, g, normal)


def _prepare_attn(c, g, normal):
    B, H, D, F, NF = c["B"], c["H"], c["D"], c["F"], c["frames"]
    bpf = -(-F // 64)
    Rq = c["cur"] * bpf
    bf = torch.bfloat16
    forced = c["sink"] + c["recent"] + c["cur"]
    n_mem = NF - forced
    kf = min(c["kf"], n_mem)
    # queries and keys share a direction per frame, so that the softmax is neither flat nor one-hot
    k = (normal(B, H, NF, F, D) + normal(B, H, NF, 1, D, by=0.5)).reshape(B, H, NF * F, D).to(bf)
    q = (normal(B, H, c["cur"] * F, D) + normal(B, H, 1, D, by=0.5)).to(bf)
    v = normal(B, H, NF * F, D, dtype=bf)
    dout = normal(B, H, c["cur"] * F, D, dtype=bf)
    # lists as the two-level selection writes them: kf memory frames besides the forced ones, kb blocks of each
    pick = torch.rand(B, H, Rq, n_mem, generator=g, device="cuda").topk(kf, dim=-1).indices + c["sink"]
    keep = torch.cat([torch.arange(c["sink"], device="cuda"), torch.arange(NF - c["recent"] - c["cur"], NF,
                                                                          device="cuda")])
    sel = torch.cat([pick, keep.expand(B, H, Rq, -1)], dim=-1).sort(dim=-1).values
    blk = torch.rand(B, H, Rq, sel.shape[-1], bpf, generator=g, device="cuda").topk(c["kb"], dim=-1).indices
    blk = blk.sort(dim=-1).values
    lists = (sel.unsqueeze(-1) * bpf + blk).reshape(B, H, Rq, -1).to(torch.int32).contiguous()
    cap = lists.shape[-1]
    count = torch.full((B, H, Rq), cap, dtype=torch.int32, device="cuda")
    if c["ragged"]:
        # uneven lists (0 ... cap, half of cap on average), about one in sixteen of them empty
        u = torch.rand(B, H, Rq, generator=g, device="cuda")
        count = (u * (cap + 1)).floor().clamp(0, cap).to(torch.int32)
        count = torch.where(u < 1 / 16, torch.zeros_like(count), count)
    return dict(case=c, q=q, k=k, v=v, dout=dout, lists=lists, count=count, cap=cap,
                out=torch.empty_like(q), lse=torch.empty(B, H, c["cur"] * F, device="cuda"),
                dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))


def _prepare_rope(c, g, normal):
    B, H, L, D, dt = c["B"], c["H"], c["L"], c["D"], DTYPES[c["dtype"]]
    n = 3 if c["fused"] else 1
    if c["axes"] == 1:
        pos = (c["start"] + torch.arange(L, device="cuda")).unsqueeze(-1)
    else:  # token t of a 30 x 52 grid: frame, row, column (two axes: frame, place)
        t = torch.arange(L, device="cuda")
        pos = torch.stack([t // 1560, (t // 52) % 30, t % 52], -1) if c["axes"] == 3 else \
            torch.stack([t // 1560, t % 1560], -1)
    tok = normal(B, L, n, H, D, dtype=dt)       # a projection's output, token-major
    head = normal(n, B, H, L, D, dtype=dt)      # the call's layout, head-major
    src, dst = (head, tok) if c["backward"] else (tok, head)
    return dict(case=c, src=src, dst=torch.empty_like(dst), pos=pos.to(torch.int32).contiguous())


def _prepare_norm(c, g, normal):
    rows, dim = c["rows"], c["dim"]
    xd, yd = DTYPES[c["x_dtype"]], DTYPES[c["y_dtype"]]
    groups = -(-rows // c["per_group"])
    s = dict(case=c, x=normal(rows, dim, dtype=xd, by=2.0) + 0.25, y=normal(rows, dim, dtype=yd),
             gate=normal(groups, dim, by=0.5), scale=normal(groups, dim, by=0.3), shift=normal(groups, dim, by=0.3),
             pre_w=None, pre_b=None, post_w=None, post_b=None)
    if c["affine"]:
        s["pre_w"] = 1 + normal(dim, by=0.1)
        s["pre_b"] = normal(dim, by=0.1) if c["pre"] == "layer" else None
        if c["post"] != "none":
            s["post_w"] = 1 + normal(dim, by=0.1)
            s["post_b"] = normal(dim, by=0.1) if c["post"] == "layer" else None
    s["r"], s["h"] = torch.empty_like(s["x"]), torch.empty_like(s["y"])
    if c["backward"]:
        s["dr"], s["dh"] = normal(rows, dim, dtype=xd), normal(rows, dim, dtype=yd)
        s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["y"])
        s["grads"] = {n: torch.empty_like(s[n]) for n in PARAMS if s[n] is not None}
    return s


PARAMS = ("gate", "scale", "shift", "pre_w", "pre_b", "post_w", "post_b")


# ---------------------------------------------------------------- one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"attn": _own_attn, "rope": _own_rope, "norm": _own_norm}[kind](state)
    return {"attn": _plain_attn, "rope": _plain_rope, "norm": _plain_norm}[kind](state)


def _own_attn(s):
    import block_sparse_attention_lf_b200 as lf
    c = s["case"]
    if "shape" not in s:
        s["shape"] = lf.LfShape.make(c["B"], c["H"], c["D"], c["F"], c["frames"], c["sink"], c["recent"], c["cur"])
        tail, pieces, _ = lf.lf_attn_split_plan(s["shape"], s["cap"])
        fwd = tail * pieces * 64 * (c["D"] + 3) * 4  # a piece's slot in a training call
        s["ws"] = torch.empty(fwd, dtype=torch.uint8, device="cuda") if fwd else None
        s["out_lo"] = torch.empty_like(s["out"])
        s["ws_bwd"] = torch.empty(lf.lf_attn_bwd_workspace(s["shape"]), dtype=torch.uint8, device="cuda")
    sh = s["shape"]
    lf.lf_block_sparse_attn_lse(sh, s["q"], s["k"], s["v"], s["lists"], s["count"], s["cap"], 0.0, s["out"], s["lse"],
                                workspace=s["ws"], out_lo=s["out_lo"])
    lf.lf_block_sparse_attn_bwd(sh, s["q"], s["k"], s["v"], s["out"], s["dout"], s["lse"], s["lists"], s["count"],
                                s["cap"], 0.0, s["dq"], s["dk"], s["dv"], s["ws_bwd"], out_lo=s["out_lo"])
    return {n: s[n] for n in ("out", "lse", "dq", "dk", "dv")}


def _own_rope(s):
    import block_sparse_attention_lf_b200 as lf
    c = s["case"]
    if "plan" not in s:
        s["plan"] = lf.RopePlan.make(c["D"], rot_dim=c["rot"], layout=c["layout"], axis_dims=_axis_dims(c),
                                     base=c["base"], scaling=c["scaling"], factor=c["factor"],
                                     original_length=c["original"])
    tok, head = (s["dst"], s["src"]) if c["backward"] else (s["src"], s["dst"])
    tok = tok.permute(2, 0, 3, 1, 4)             # [n, B, H, L, D] view of the token-major tensor
    src, dst = (head, tok) if c["backward"] else (tok, head)
    lf.lf_rope(s["plan"], src.unbind(0), dst.unbind(0), s["pos"], rotate=(True, True, False)[:src.shape[0]],
               backward=c["backward"])
    return s["dst"]


def _own_norm(s):
    import block_sparse_attention_lf_b200 as lf
    c = s["case"]
    if "shape" not in s:
        s["shape"] = lf.NormGateShape.make(c["rows"], c["dim"], rows_per_group=c["per_group"], x_dtype=s["x"].dtype,
                                           y_dtype=s["y"].dtype, pre=c["pre"], post=c["post"], eps=1e-6,
                                           residual_scale=c["alpha"])
        if c["backward"]:
            s["ws"] = torch.empty(lf.lf_norm_gate_bwd_workspace(s["shape"]), dtype=torch.uint8, device="cuda")
    p = {n: s[n] for n in PARAMS}
    lf.lf_norm_gate(s["shape"], s["x"], s["y"], s["r"], s["h"], **p)
    if not c["backward"]:
        return {"r": s["r"], "h": s["h"]}
    lf.lf_norm_gate_bwd(s["shape"], s["x"], s["y"], s["dr"], s["dh"], s["dx"], s["dy"], s["grads"], s["ws"], **p)
    return {"r": s["r"], "h": s["h"], "dx": s["dx"], "dy": s["dy"], **{"d" + n: t for n, t in s["grads"].items()}}


def _plain_attn(s):
    c = s["case"]
    BH, D, F, NF = c["B"] * c["H"], c["D"], c["F"], c["frames"]
    bpf = -(-F // 64)
    Rq, cap = c["cur"] * bpf, s["cap"]
    dev = s["q"].device
    scale = D ** -0.5
    # query rows [BH, Rq, 64] and listed key rows [BH, Rq, cap * 64] as token indices, with what is valid of them
    o64 = torch.arange(64, device=dev)
    r = torch.arange(Rq, device=dev)
    qt = (r % bpf).unsqueeze(-1) * 64 + o64
    q_ok = qt < F
    qi = torch.where(q_ok, (r // bpf).unsqueeze(-1) * F + qt, torch.zeros_like(qt))
    g = s["lists"].reshape(BH, Rq, cap).long()
    listed_ = torch.arange(cap, device=dev) < s["count"].reshape(BH, Rq, 1)
    g = torch.where(listed_, g, torch.zeros_like(g))
    kt = (g % bpf).unsqueeze(-1) * 64 + o64
    k_ok = ((kt < F) & listed_.unsqueeze(-1)).reshape(BH, Rq, 1, cap * 64)
    ki = torch.where(kt < F, (g // bpf).unsqueeze(-1) * F + kt, torch.zeros_like(kt)).reshape(BH, Rq * cap * 64)
    heads = torch.arange(BH, device=dev).unsqueeze(-1)
    flat = ki + heads * (NF * F)                                  # rows of the flattened keys
    qflat = (qi.reshape(1, -1) + heads * (c["cur"] * F))
    q = s["q"].reshape(-1, D)[qflat].float().reshape(BH * Rq, 64, D) * q_ok.repeat(BH, 1).unsqueeze(-1)
    do = s["dout"].reshape(-1, D)[qflat].float().reshape(BH * Rq, 64, D) * q_ok.repeat(BH, 1).unsqueeze(-1)
    k = s["k"].reshape(-1, D)[flat].float().reshape(BH * Rq, cap * 64, D)
    v = s["v"].reshape(-1, D)[flat].float().reshape(BH * Rq, cap * 64, D)
    ok = k_ok.reshape(BH * Rq, 1, cap * 64)
    sc = (torch.bmm(q, k.transpose(1, 2)) * scale).masked_fill_(~ok, -math.inf)
    m = sc.amax(dim=-1, keepdim=True)
    p = torch.exp(sc.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)))
    l = p.sum(dim=-1, keepdim=True)
    lse = (m + torch.log(l)).squeeze(-1)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    o = torch.bmm(p, v)
    dp = torch.bmm(do, v.transpose(1, 2))
    ds = dp.sub_((do * o).sum(dim=-1, keepdim=True)).mul_(p)
    dq = torch.bmm(ds, k) * scale
    del sc, k, v
    dv = torch.zeros(BH * NF * F, D, device=dev).index_add_(0, flat.reshape(-1),
                                                            torch.bmm(p.transpose(1, 2), do).reshape(-1, D))
    del p, dp
    dk = torch.zeros(BH * NF * F, D, device=dev).index_add_(0, flat.reshape(-1),
                                                            torch.bmm(ds.transpose(1, 2), q).reshape(-1, D))
    bf = torch.bfloat16
    take = q_ok.reshape(-1)
    B, H, Lq = c["B"], c["H"], c["cur"] * F
    rows = lambda t: t.reshape(BH, Rq * 64, D)[:, take].reshape(B, H, Lq, D).to(bf)  # noqa: E731
    return {"out": rows(o), "lse": lse.reshape(BH, Rq * 64)[:, take].reshape(B, H, Lq), "dq": rows(dq),
            "dk": (dk * scale).to(bf).reshape(B, H, NF * F, D), "dv": dv.to(bf).reshape(B, H, NF * F, D)}


def _frequencies(c, dev):
    """Angle per position of each pair, the axis of each pair and the factor on the result (64 bits)."""
    f64 = torch.float64
    dims = _axis_dims(c)
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=dev), torch.tensor([d // 2 for d in dims],
                                                                                     device=dev))
    d = torch.tensor(dims, dtype=f64, device=dev)[axis]
    at = torch.arange(c["rot"] // 2, device=dev) - torch.tensor([0] + [sum(dims[:1]) // 2, sum(dims[:2]) // 2],
                                                                device=dev)[axis]
    f = c["base"] ** (-2.0 * at.to(f64) / d)
    d0, first = float(dims[0]), axis == 0
    if c["scaling"] == "linear":
        f = torch.where(first, f / c["factor"], f)
    if c["scaling"] == "ntk":
        base = c["base"] * c["factor"] ** (d0 / (d0 - 2.0))
        f = torch.where(first, base ** (-2.0 * at.to(f64) / d0), f)
    if c["scaling"] == "yarn":
        place = lambda turns: d0 * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(c["base"]))  # noqa: E731
        low = min(max(math.floor(place(32.0)), 0), dims[0] - 1)
        high = min(max(math.ceil(place(1.0)), 0), dims[0] - 1)
        ramp = ((at.to(f64) - low) / max(high - low, 0.001)).clamp(0, 1)
        f = torch.where(first, f / c["factor"] * ramp + f * (1 - ramp), f)
    m = 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" and c["factor"] > 1 else 1.0
    return f, axis, m


def _plain_rope(s):
    c = s["case"]
    f, axis, m = _frequencies(c, s["pos"].device)
    angle = s["pos"].to(torch.float64)[:, axis] * f               # [L, rot / 2]
    cos = (torch.cos(angle) * m).float()
    sin = (torch.sin(angle) * (-m if c["backward"] else m)).float()
    x = s["src"].float() if c["backward"] else s["src"].permute(2, 0, 3, 1, 4).float()   # [n, B, H, L, D]
    n, rot = x.shape[0], c["rot"]
    turn, rest, move = x[:2, ..., :rot], x[:2, ..., rot:], x[2:]
    if c["layout"] == "half":
        a, b = turn[..., :rot // 2], turn[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    else:
        a, b = turn[..., 0::2], turn[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    y = torch.cat([torch.cat([y, rest], dim=-1), move], dim=0).to(DTYPES[c["dtype"]])
    return y.permute(1, 3, 0, 2, 4).contiguous() if c["backward"] else y.contiguous()


def _hat(t, kind):
    """Normalised rows and 1 / deviation (None: no norm)."""
    if kind == "none":
        return t, None
    z = t - t.mean(dim=-1, keepdim=True) if kind == "layer" else t
    rstd = torch.rsqrt((z * z).mean(dim=-1, keepdim=True) + 1e-6)
    return z * rstd, rstd


def _hat_grad(dn, n, rstd, kind):
    if kind == "none":
        return dn
    d = dn - n * (dn * n).mean(dim=-1, keepdim=True)
    return (d - dn.mean(dim=-1, keepdim=True) if kind == "layer" else d) * rstd


def _plain_norm(s):
    c = s["case"]
    rows, dim, per = c["rows"], c["dim"], c["per_group"]
    groups = -(-rows // per)
    group = torch.arange(rows, device=s["x"].device) // per
    one = lambda t, other: other if t is None else t  # noqa: E731
    w1, b1, w2, b2 = one(s["pre_w"], 1.0), one(s["pre_b"], 0.0), one(s["post_w"], 1.0), one(s["post_b"], 0.0)
    gate, scale, shift = s["gate"][group], s["scale"][group], s["shift"][group]
    m, m_rstd = _hat(s["y"].float(), c["post"])
    u = m * w2 + b2
    r = c["alpha"] * s["x"].float() + gate * u
    n, n_rstd = _hat(r, c["pre"])
    a = n * w1 + b1
    h = a * (1 + scale) + shift
    res = {"r": r.to(s["x"].dtype), "h": h.to(s["y"].dtype)}
    if not c["backward"]:
        return res
    dh = s["dh"].float()

    def by_group(t):
        pad = torch.zeros(groups * per - rows, dim, device=t.device)
        return torch.cat([t, pad]).reshape(groups, per, dim).sum(dim=1)

    da = dh * (1 + scale)
    dr = s["dr"].float() + _hat_grad(da * w1, n, n_rstd, c["pre"])
    du = dr * gate
    res["dx"], res["dy"] = (c["alpha"] * dr).to(s["x"].dtype), _hat_grad(du * w2, m, m_rstd, c["post"]).to(s["y"].dtype)
    res["dgate"], res["dscale"], res["dshift"] = by_group(dr * u), by_group(dh * a), by_group(dh)
    if s["pre_w"] is not None:
        res["dpre_w"] = (da * n).sum(dim=0)
    if s["pre_b"] is not None:
        res["dpre_b"] = da.sum(dim=0)
    if s["post_w"] is not None:
        res["dpost_w"] = (du * m).sum(dim=0)
    if s["post_b"] is not None:
        res["dpost_b"] = du.sum(dim=0)
    return res


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "rope": _exact_rope, "norm": _exact_norm}[case["kind"]](s)


def _exact_attn(s):
    c = s["case"]
    F, D, cur = c["F"], c["D"], c["cur"]
    bpf = -(-F // 64)
    B, H = c["B"], c["H"]
    lists, count = s["lists"].tolist(), s["count"].tolist()
    q, k, v, do = (s[n].double() for n in ("q", "k", "v", "dout"))
    out, dq, dk, dv = (torch.zeros_like(t) for t in (q, q, k, v))
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)
    span = torch.arange(64, device=q.device)
    for b in range(B):
        for h in range(H):
            for r in range(cur * bpf):
                n = count[b][h][r]
                if n == 0:
                    continue
                f, j = divmod(r, bpf)
                rows = slice(f * F + 64 * j, f * F + min(64 * j + 64, F))
                ids = s["lists"][b, h, r, :n].long()
                place = (ids % bpf).unsqueeze(-1) * 64 + span
                cols = ((ids // bpf).unsqueeze(-1) * F + place)[place < F]
                kk, vv, qq, oo = k[b, h, cols], v[b, h, cols], q[b, h, rows], do[b, h, rows]
                z = qq @ kk.T / math.sqrt(D)
                ls = torch.logsumexp(z, dim=-1)
                w = torch.exp(z - ls[:, None])
                y = w @ vv
                e = oo @ vv.T
                e = w * (e - (w * e).sum(dim=-1, keepdim=True))
                out[b, h, rows], lse[b, h, rows], dq[b, h, rows] = y, ls, e @ kk / math.sqrt(D)
                dk[b, h, cols] += e.T @ qq / math.sqrt(D)
                dv[b, h, cols] += w.T @ oo
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _exact_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    dims = _axis_dims(c)
    freq, axis = [], []
    for a, d in enumerate(dims):
        for j in range(d // 2):
            w = math.exp(-2.0 * j / d * math.log(c["base"]))
            if a == 0 and c["scaling"] == "linear":
                w /= c["factor"]
            elif a == 0 and c["scaling"] == "ntk":
                w = math.exp(-2.0 * j / d * (math.log(c["base"]) + d / (d - 2.0) * math.log(c["factor"])))
            elif a == 0 and c["scaling"] == "yarn":
                edge = [d * math.log(c["original"] / (2 * math.pi * t)) / (2 * math.log(c["base"])) for t in (32.0, 1.0)]
                lo, hi = max(0, min(d - 1, math.floor(edge[0]))), max(0, min(d - 1, math.ceil(edge[1])))
                mix = max(0.0, min(1.0, (j - lo) / max(hi - lo, 0.001)))
                w = w * (1 - mix) + w / c["factor"] * mix
            freq.append(w)
            axis.append(a)
    amp = 1.0 + 0.1 * math.log(c["factor"]) if c["scaling"] == "yarn" and c["factor"] > 1 else 1.0
    dev = s["src"].device
    theta = s["pos"].double()[:, axis] * torch.tensor(freq, dtype=torch.float64, device=dev)
    if c["backward"]:
        theta = -theta
    turn = torch.polar(torch.full_like(theta, amp), theta)        # a rotation is a complex product
    x = s["src"] if c["backward"] else s["src"].permute(2, 0, 3, 1, 4)
    y = []
    for i in range(x.shape[0]):
        t = x[i].double()
        if i < 2:
            first, second = (slice(0, half), slice(half, rot)) if c["layout"] == "half" else (slice(0, rot, 2),
                                                                                             slice(1, rot, 2))
            z = torch.complex(t[..., first], t[..., second]) * turn
            t = t.clone()
            t[..., first], t[..., second] = z.real, z.imag
        y.append(t)
    y = torch.stack(y)
    return y.permute(1, 3, 0, 2, 4).contiguous() if c["backward"] else y


def _exact_norm(s):
    c = s["case"]
    names = [n for n in PARAMS if s[n] is not None]
    leaf = {n: s[n].double().requires_grad_(c["backward"]) for n in names + ["x", "y"]}
    per, rows = c["per_group"], c["rows"]

    def norm(t, kind):
        if kind == "none":
            return t
        var, mean = torch.var_mean(t, dim=1, correction=0, keepdim=True)
        return (t - mean) / torch.sqrt(var + 1e-6) if kind == "layer" else \
            t / torch.sqrt(t.square().mean(dim=1, keepdim=True) + 1e-6)

    def affine(t, w, b):
        t = t * leaf[w] if w in leaf else t
        return t + leaf[b] if b in leaf else t

    spread = {n: leaf[n].repeat_interleave(per, dim=0)[:rows] for n in ("gate", "scale", "shift")}
    r = c["alpha"] * leaf["x"] + spread["gate"] * affine(norm(leaf["y"], c["post"]), "post_w", "post_b")
    h = affine(norm(r, c["pre"]), "pre_w", "pre_b") * (1 + spread["scale"]) + spread["shift"]
    res = {"r": r.detach(), "h": h.detach()}
    if c["backward"]:
        order = ["x", "y"] + names
        got = torch.autograd.grad([r, h], [leaf[n] for n in order], [s["dr"].double(), s["dh"].double()])
        res.update({"d" + n: t for n, t in zip(order, got)})
    return res
