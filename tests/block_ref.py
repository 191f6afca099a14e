"""Definitions in 64 bits (plain torch, CPU) of the operators around the HSA call, and the
inputs their tests use. Nothing here calls the library."""
import math

import torch

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative


# ---------------------------------------------------------------- rotary positions
def rope_frequencies(dims, base, scaling="none", factor=1.0, original=0.0, fast=32.0, slow=1.0):
    """(angle per position of each pair, axis of each pair, amplitude)."""
    f, axis = [], []
    for a, d in enumerate(dims):
        for j in range(d // 2):
            w = base ** (-2.0 * j / d)
            if a == 0 and scaling == "linear":
                w = w / factor
            if a == 0 and scaling == "ntk":
                w = (base * factor ** (d / (d - 2.0))) ** (-2.0 * j / d)
            if a == 0 and scaling == "yarn":
                lo, hi = (d * math.log(original / (2 * math.pi * b)) / (2 * math.log(base)) for b in (fast, slow))
                lo, hi = min(max(math.floor(lo), 0), d - 1), min(max(math.ceil(hi), 0), d - 1)
                r = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
                w = w * (1 - r) + w / factor * r
            f.append(w)
            axis.append(a)
    amp = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    return torch.tensor(f, dtype=torch.float64), torch.tensor(axis), amp


def rope(x, pos, f, axis, amp, layout, rot, backward=False):
    """x [B, H, T, D] float64, pos [T, n] or [B, T, n]: rotated, and the size sum |a| + |b| of what each element adds."""
    pos = pos if pos.dim() == 3 else pos.unsqueeze(0)
    th = pos.double()[..., axis] * f                               # [B or 1, T, rot / 2]
    c, s = amp * torch.cos(th).unsqueeze(1), amp * torch.sin(th).unsqueeze(1)
    if backward:
        s = -s
    ia = torch.arange(rot // 2) * (1 if layout == "half" else 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    a, b = x[..., ia], x[..., ib]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = amp * (a.abs() + b.abs())
    return y, size


# ---------------------------------------------------------------- gated residual norms
def norm(t, kind, eps):
    if kind == "none":
        return t
    if kind == "layer":
        t = t - t.mean(-1, keepdim=True)
    return t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)


def norm_gate(x, y, per, alpha, pre, post, eps, v):
    """(r, h) of float64 inputs; v: vectors by name, absent ones missing."""
    rows = x.shape[0]
    spread = lambda n: v[n].repeat_interleave(per, 0)[:rows]  # noqa: E731
    r = alpha * x
    if y is not None:
        u = norm(y, post, eps)
        u = u * v["post_w"] if "post_w" in v else u
        u = u + v["post_b"] if "post_b" in v else u
        r = r + (spread("gate") * u if "gate" in v else u)
    if pre == "none":
        return r, None
    h = norm(r, pre, eps)
    h = h * v["pre_w"] if "pre_w" in v else h
    h = h + v["pre_b"] if "pre_b" in v else h
    h = h * (1 + spread("scale")) if "scale" in v else h
    return r, h + spread("shift") if "shift" in v else h


# ---------------------------------------------------------------- block-sparse attention
def token_mask(B, H, F, n_cur, n_frames, lists, count):
    """[B, H, Lq, Lkv] truth values: query t attends to token s."""
    bpf = -(-F // 64)
    m = torch.zeros(B, H, n_cur * F, n_frames * F, dtype=torch.bool)
    for b in range(B):
        for h in range(H):
            for r in range(n_cur * bpf):
                f, j = divmod(r, bpf)
                rows = slice(f * F + 64 * j, f * F + min(64 * j + 64, F))
                for g in lists[b, h, r, :int(count[b, h, r])].tolist():
                    t, jj = divmod(g, bpf)
                    m[b, h, rows, t * F + 64 * jj:t * F + min(64 * jj + 64, F)] = True
    return m


def attention(q, k, v, mask, scale):
    """(out, lse) in 64 bits; rows without a token give 0 and -inf."""
    s = (q @ k.transpose(-1, -2)) * scale
    s = s.masked_fill(~mask, -math.inf)
    some = mask.any(-1, keepdim=True)
    lse = torch.logsumexp(s.masked_fill(~some, 0.0), -1, keepdim=True)
    p = torch.where(mask, torch.exp(s - lse), torch.zeros_like(s))
    return p @ v, torch.where(some, lse, torch.full_like(lse, -math.inf)).squeeze(-1), p


def attention_grads(q, k, v, do, mask, scale):
    """Gradients by the formula, and for each the bound of its error when P and dS are rounded to bf16
    (half a step, 2^-8 relative), delta is the mean of dout v^T under weights rounded to bf16 that sum to one
    (so off by 2^-8 of the mean |dout v^T - delta|, and 2^-16 of |dout||out| for how it is stored), products are exact in fp32 sums (2^-16 of the
    terms' sizes: sums of up to 2^7 terms a step and 2^8 relative steps of 2^-24 each), and the result is rounded
    to bf16."""
    out, lse, p = attention(q, k, v, mask, scale)
    e, f = 2.0 ** -8, 2.0 ** -16
    dp = do @ v.transpose(-1, -2)
    delta = (do * out).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    dq, dk, dv = scale * ds @ k, scale * ds.transpose(-1, -2) @ q, p.transpose(-1, -2) @ do
    # error of one element of dS: its own rounding, delta's (out rounded), the fp32 sums behind dP and S
    size = do.abs() @ v.abs().transpose(-1, -2)
    logit = scale * (q.abs() @ k.abs().transpose(-1, -2))
    err_p = p * (f * (1 + logit))
    err_ds = ds.abs() * e + p * (2 * e * (p * (dp - delta).abs()).sum(-1, keepdim=True) + f * size
                                 + f * (do.abs() * out.abs()).sum(-1, keepdim=True)) + err_p * (dp - delta).abs()
    err_dv = (p * e + err_p).transpose(-1, -2) @ do.abs()
    t_dq = e * dq.abs() + (1 + e) * scale * err_ds @ k.abs()
    t_dk = e * dk.abs() + (1 + e) * scale * err_ds.transpose(-1, -2) @ q.abs()
    t_dv = e * dv.abs() + (1 + e) * err_dv
    return (out, lse, dq, dk, dv), (t_dq, t_dk, t_dv), logit
