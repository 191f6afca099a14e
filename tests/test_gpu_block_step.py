"""The operators together as a fine-tuning step of one transformer block runs them: gated norm into the block, fused
projection, rotary positions into the call's tensors, pooling and selection, attention, output projection, gated norm
out of the block, and the whole way back; against 64-bit automatic differentiation of the definitions on the blocks
that were selected."""
import pytest
import torch

import block_sparse_attention_lf_b200 as L
from tests import block_ref as R

pytestmark = pytest.mark.gpu


def test_block_step():
    B, H, D, F, NF, nc = 1, 2, 64, 96, 5, 2
    T, C = nc * F, H * D
    bf = torch.bfloat16
    g = torch.Generator().manual_seed(51)
    r = lambda *s, by=1.0: torch.randn(*s, generator=g) * by  # noqa: E731
    x0, y0 = r(B * T, C), r(B * T, C).to(bf)                      # fp32 stream, the block before's output
    w_qkv, w_o = r(C, 3 * C, by=C ** -0.5).to(bf), r(C, C, by=C ** -0.5).to(bf)
    past_k, past_v = r(B, H, (NF - nc) * F, D).to(bf), r(B, H, (NF - nc) * F, D).to(bf)
    mod = {n: r(nc, C, by=0.3) for n in ("gate", "scale", "shift")}
    mod2 = {n: r(nc, C, by=0.3) for n in ("gate", "scale", "shift")}
    post_w = 1 + r(C, by=0.1)
    dr, dh = r(B * T, C), r(B * T, C).to(bf)
    t = torch.arange(T)
    pos = torch.stack([(NF - nc) + t // F, (t % F) // 12, t % 12], -1)
    dims = (24, 20, 20)

    # forward and gradient on the GPU
    c = lambda v: v.cuda()  # noqa: E731
    n1 = L.NormGateShape.make(B * T, C, F, torch.float32, bf, "layer", "none")
    n2 = L.NormGateShape.make(B * T, C, F, torch.float32, bf, "layer", "rms")
    x, y = c(x0), c(y0)
    m1, m2 = {n: c(v) for n, v in mod.items()}, {n: c(v) for n, v in mod2.items()}
    res, h = torch.empty_like(x), torch.empty_like(y)
    L.lf_norm_gate(n1, x, y, res, h, **m1)
    qkv = (h @ c(w_qkv)).view(B, T, 3, H, D)
    shape = L.LfShape.make(B, H, D, F, NF, 1, 1, nc)
    call = L.HSACall(shape, 2, 1, 1, train=True)
    plan = L.RopePlan.make(D, layout="half", axis_dims=dims)
    q = torch.empty(B, H, T, D, dtype=bf, device="cuda")
    k, v = (torch.cat([c(p), torch.empty(B, H, T, D, dtype=bf, device="cuda")], 2) for p in (past_k, past_v))
    p32 = c(pos.int())
    call.load(plan, qkv, p32, q, k, v)
    o = call(q, k, v)
    o_tok = o.transpose(1, 2).reshape(B * T, C).contiguous()
    y2 = o_tok @ c(w_o)
    res2, h2 = torch.empty_like(x), torch.empty_like(y)
    L.lf_norm_gate(n2, res, y2, res2, h2, post_w=c(post_w), **m2)

    ws1, ws2 = (torch.empty(L.lf_norm_gate_bwd_workspace(s), dtype=torch.uint8, device="cuda") for s in (n1, n2))
    dres, dy2 = torch.empty_like(x), torch.empty_like(y2)
    g2 = {n: torch.empty_like(w) for n, w in m2.items()}
    g2["post_w"] = torch.empty(C, device="cuda")
    L.lf_norm_gate_bwd(n2, res, y2, c(dr), c(dh), dres, dy2, g2, ws2, post_w=c(post_w), **m2)
    do = (dy2 @ c(w_o).T).view(B, T, H, D).transpose(1, 2).contiguous()
    dq, dk, dv, dqkv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(qkv)
    call.backward(q, k, v, do, dq, dk, dv)
    call.load_bwd(plan, dq, dk, dv, p32, dqkv)
    dh1 = dqkv.view(B * T, 3 * C) @ c(w_qkv).T
    dx, dy = torch.empty_like(x), torch.empty_like(y)
    g1 = {n: torch.empty_like(w) for n, w in m1.items()}
    L.lf_norm_gate_bwd(n1, x, y, dres, dh1, dx, dy, g1, ws1, **m1)

    # the same in 64 bits
    leaf = lambda v: v.double().requires_grad_()  # noqa: E731
    X, Y, A1, A2, PW = leaf(x0), leaf(y0), {n: leaf(w) for n, w in mod.items()}, {n: leaf(w) for n, w in mod2.items()}, leaf(post_w)
    R1, H1 = R.norm_gate(X, Y, F, 1.0, "layer", "none", 1e-6, A1)
    Q, K, V = (H1 @ w_qkv.double()).view(B, T, 3, H, D).permute(2, 0, 3, 1, 4).unbind(0)
    f, axis, amp = R.rope_frequencies(dims, 10000.0)
    th = pos.double()[:, axis] * f
    turn = lambda u: torch.cat([u[..., :D // 2] * th.cos() - u[..., D // 2:] * th.sin(),  # noqa: E731
                                u[..., :D // 2] * th.sin() + u[..., D // 2:] * th.cos()], -1)
    K, V = torch.cat([past_k.double(), turn(K)], 2), torch.cat([past_v.double(), V], 2)
    mask = R.token_mask(B, H, F, nc, NF, call.buf.block_list.cpu(), call.buf.block_count.cpu())
    O, lse, _ = R.attention(turn(Q), K, V, mask, D ** -0.5)
    Y2 = O.transpose(1, 2).reshape(B * T, C) @ w_o.double()
    R2, H2 = R.norm_gate(R1, Y2, F, 1.0, "layer", "rms", 1e-6, {**A2, "post_w": PW})
    names = ["x", "y"] + list(A1) + ["2" + n for n in A2] + ["post_w"]
    got = torch.autograd.grad((R2 * dr.double()).sum() + (H2 * dh.double()).sum(),
                              [X, Y, *A1.values(), *A2.values(), PW])
    here = [dx, dy, *g1.values(), *[g2[n] for n in A2], g2["post_w"]]
    # Every one of the chain's tensors between the operators (h, the projection, q, k, o, y2 and the seven gradients
    # between them) is rounded to bf16, at most 2^-8 of each element, and P and dS once each; independent roundings
    # add in squares: sqrt(15) * 2^-8 of the norm, and twice that for what the norms' and the softmax's derivatives
    # (below 2 here) make of them.
    lim = 2 * 15 ** 0.5 * 2.0 ** -8
    off = {n: float((a.double().cpu() - b).norm() / b.norm()) for n, a, b in zip(names, here, got)}
    assert all(e <= lim for e in off.values()), off
    assert float((h2.double().cpu() - H2.detach()).norm() / H2.detach().norm()) <= lim
    assert float((res2.double().cpu() - R2.detach()).norm() / R2.detach().norm()) <= lim
    assert float((call.lse.double().cpu() - lse.detach()).abs().max()) <= 0.1
    assert L.lf_get_device_error() == (0, 0)
