"""Training a router whose experts are no multiple of 8: its products over the next multiple, the rest closed by the bias."""

import pytest
import torch

import sparse_moe_ffn_route_amd as moe

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
D = 256


def padded_step(x, wr, bias, d_w, d_loss, E, k, renorm, dtype):
    """Routing, grouping, losses and both products' gradients over P >= E experts."""
    T, P = x.shape[0], wr.shape[0]
    d = moe.make_dims(T, D, P, k, 64, 0, 0, E, renorm, dtype, dtype, dtype)
    new = lambda *s, t: torch.full(s, 77, dtype=t, device="cuda")  # noqa: E731
    i32, f32 = torch.int32, torch.float32
    ws, logits, packed = moe.workspace(d), new(T, P, t=f32), new(T, 2, k, t=i32)
    moe.moe_route(d, x, wr, logits, bias, packed, ws)
    counts, offsets, perm, inv = new(E, t=i32), new(E + 1, t=i32), new(T * k, t=i32), new(T, k, t=i32)
    moe.moe_permute(d, packed, counts, offsets, perm, inv, ws=ws)
    loss, load = new(2, t=f32), new(P + 1, t=i32)
    moe.moe_route_loss(d, logits, bias, packed, loss, load, ws=moe.route_loss_workspace(d))
    d_logits, dx, dwr = new(T, P, t=x.dtype), new(T, D, t=x.dtype), new(P, D, t=x.dtype)
    moe.moe_route_backward(d, logits, bias, packed, d_w, load, d_loss, d_logits)
    g = moe.make_groups(1, T, P, D, dtype)
    all_t, gws = torch.tensor([0, T], dtype=i32, device="cuda"), moe.grouped_gemm_workspace(g)
    moe.moe_grouped_gemm_backward_rows(g, d_logits, all_t, wr, dx, ws=gws)
    moe.moe_grouped_gemm_backward_weights(g, d_logits, x, all_t, dwr, ws=gws)
    return packed, inv, offsets, loss, load, d_logits, dx, dwr


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 3, 1), (70, 5, 5), (200, 60, 4), (300, 257, 10)])
def test_gradients_are_those_of_the_experts_that_are_there(T, E, k, renorm, dtype):
    """2-norms, against float64 autograd over E experts.  Two roundings to the type lie between inputs and a gradient
    (d_logits, the result), 2^-24 or 2^-8 each; logits, losses and products are fp32 sums of up to 300 terms, 300 * 2^-24
    each at most, on five of them."""
    P = -(-E // 8) * 8
    g = torch.Generator().manual_seed(T + E)
    x, wr = torch.randn(T, D, generator=g).to(DT[dtype]), (torch.randn(E, D, generator=g) * D ** -0.5).to(DT[dtype])
    bias, d_w = torch.randn(E, generator=g) * 0.3, torch.randn(T, k, generator=g) / T
    c = torch.tensor([0.5, 0.01])
    wr_p = torch.zeros(P, D, dtype=DT[dtype])
    wr_p[:E] = wr
    bias_p = torch.full((P,), -float("inf"))
    bias_p[:E] = bias
    packed, inv, offsets, loss, load, d_logits, dx, dwr = (t.cpu() for t in padded_step(
        x.cuda(), wr_p.cuda(), bias_p.cuda(), d_w.cuda(), (c * torch.tensor([E / P, 1.0])).cuda(), E, k, renorm, dtype))
    ids = packed[:, 0].long()
    assert (ids < E).all() and (inv >= 0).all() and offsets[E] == T * k and not load[E:P].any() and load[P] == T
    assert not d_logits[:, E:].any() and not dwr[E:].any()

    x64, wr64 = x.double().requires_grad_(), wr.double().requires_grad_()
    key = x64 @ wr64.T + bias.double()
    prob = torch.softmax(key, 1)
    w = torch.softmax(torch.gather(key, 1, ids), 1) if renorm else torch.gather(prob, 1, ids)
    counted = torch.bincount(ids.reshape(-1), minlength=E).double()
    balance = E / (k * T) * (counted * prob.sum(0)).sum() / T
    z = (torch.logsumexp(key, 1) ** 2).mean()
    total = (w * d_w.double()).sum() + c[0].double() * balance + c[1].double() * z
    ref_dx, ref_dwr = torch.autograd.grad(total, (x64, wr64))
    bar = 2 * (2.0 ** -24 if dtype == "f32" else 2.0 ** -8) + 5 * 300 * 2.0 ** -24
    assert (dx.double() - ref_dx).norm() <= bar * ref_dx.norm()
    assert (dwr[:E].double() - ref_dwr).norm() <= bar * ref_dwr.norm()
    ref_loss = torch.stack([balance * P / E, z]).detach()
    assert ((loss.double() - ref_loss).abs() <= 5 * 300 * 2.0 ** -24 * ref_loss).all()


def test_products_of_other_widths_are_refused():
    for E in (3, 60, 257):
        assert moe.library().moe_grouped_gemm_workspace_bytes(moe.make_groups(1, 16, E, D)) == 0
