"""Gradients of the combine and the permutation, and a whole backward pass of the layer, against float64.

Whole numbers and powers of two make the combine's products and sums exact: equality.
"""

import ctypes

import pytest
import torch

import sparse_moe_ffn_route_amd as moe
from test_dropout import mask_of

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def routing(T, E, k, begin, local, seed):
    """ids, weights (powers of two), inv_pos of a local slice with the rows in a random order, rows in use."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).topk(k, 1)[1]
    w = 2.0 ** -torch.randint(0, 6, (T, k), generator=g).float()
    here = (ids >= begin) & (ids < begin + local)
    inv = torch.full((T, k), -1, dtype=torch.int32)
    used = int(here.sum())
    inv[here] = torch.randperm(used, generator=g).int()
    return ids, w, inv, used


def whole(shape, seed):
    return torch.randint(-4, 5, shape, generator=torch.Generator().manual_seed(seed)).float()


COMBINE = [(1, 64, 4, 1, 4), (1, 4096, 512, 10, 512), (7, 64, 16, 8, 16), (33, 2112, 40, 9, 13), (50, 320, 64, 32, 20),
           (3, 128, 8, 2, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("act,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,D,E,k,local", COMBINE)
def test_combine_backward(T, D, E, k, local, act, out):
    begin = (E - local) // 2
    ids, w, inv, used = routing(T, E, k, begin, local, T + D)
    d = moe.make_dims(T, D, E, k, 64, 0, begin, local, True, act, act, out)
    dy, rows = whole((T, D), 1).to(DT[out]), whole((T * k, D), 2).to(DT[out])
    rows[used:] = float("nan")
    packed = torch.stack([ids.int(), w.view(torch.int32)], 1).contiguous().cuda()
    d_rows = torch.full((T * k, D), 777.0, dtype=DT[act], device="cuda")
    d_w = torch.full((T, k), 777.0, device="cuda")
    moe.moe_unpermute_combine_backward(d, dy.cuda(), packed, inv.cuda(), rows.cuda(), d_rows, d_w)
    want_rows = torch.full((T * k, D), 777.0, dtype=torch.float64)
    want_w = torch.zeros(T, k, dtype=torch.float64)
    for t, j in (inv >= 0).nonzero().tolist():
        want_rows[inv[t, j]] = w[t, j].double() * dy[t].double()
        want_w[t, j] = dy[t].double() @ rows[inv[t, j]].double()
    assert torch.equal(d_rows.cpu(), want_rows.to(DT[act])) and torch.equal(d_w.cpu().double(), want_w)
    again = torch.full_like(d_rows, 777.0)
    moe.moe_unpermute_combine_backward(d, dy.cuda(), packed, inv.cuda(), None, again, None)
    assert torch.equal(again, d_rows)


@pytest.mark.gpu
@pytest.mark.parametrize("act", list(DT))
@pytest.mark.parametrize("T,D,E,k,local", COMBINE)
def test_permute_backward(T, D, E, k, local, act):
    begin = (E - local) // 2
    _, _, inv, used = routing(T, E, k, begin, local, T + D)
    d = moe.make_dims(T, D, E, k, 64, 0, begin, local, True, act, act, act)
    rows, add = whole((T * k, D), 3).to(DT[act]), whole((T, D), 4).to(DT[act])
    rows[used:] = float("nan")
    want = torch.zeros(T, D, dtype=torch.float64)
    for t, j in (inv >= 0).nonzero().tolist():
        want[t] += rows[inv[t, j]].double()
    dx = torch.full((T, D), 777.0, dtype=DT[act], device="cuda")
    moe.moe_permute_backward(d, rows.cuda(), inv.cuda(), dx)
    assert torch.equal(dx.cpu(), want.to(DT[act]))
    dx.copy_(add)
    moe.moe_permute_backward(d, rows.cuda(), inv.cuda(), dx, add=dx)
    assert torch.equal(dx.cpu(), (want + add.double()).to(DT[act]))


@pytest.mark.gpu
@pytest.mark.parametrize("act", list(DT))
@pytest.mark.parametrize("T,D,k", [(1, 64, 1), (700, 576, 10), (4096, 1024, 32)])
def test_adding_in_place_gives_the_same_bits(T, D, k, act):
    """d_x = add's own memory, call after call, against d_x apart from it."""
    g = torch.Generator(device="cuda").manual_seed(T)
    d = moe.make_dims(T, D, 32, k, 64, act=act, w=act, out=act)
    rows = torch.randn(T * k, D, generator=g, device="cuda").to(DT[act])
    inv = torch.randperm(T * k, generator=g, device="cuda").int().reshape(T, k)
    inv[::3, k // 2] = -1
    here, apart = torch.randn(T, D, generator=g, device="cuda").to(DT[act]), torch.empty(T, D, dtype=DT[act], device="cuda")
    for _ in range(3):
        moe.moe_permute_backward(d, rows, inv, apart, add=here)
        moe.moe_permute_backward(d, rows, inv, here, add=here)
        assert torch.equal(here, apart)


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [((1 << 26) + 3, 64), ((1 << 25) + 3, 576)])
def test_more_tokens_than_a_grid_dimension_holds(T, D):
    """2^26 waves and more, which are 2^32 threads: the permutation's gradient and the combine itself, every row."""
    d = moe.make_dims(T, D, 2, 1, 64)
    rows = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").random_(-8, 9)
    inv = torch.arange(T, device="cuda", dtype=torch.int32).flip(0).contiguous()
    inv[::7] = -1
    packed = torch.zeros(T, 2, 1, dtype=torch.int32, device="cuda")
    packed[:, 1] = torch.tensor(2.0).view(torch.int32).item()
    out = torch.empty_like(rows)
    for weight, call in ((1, lambda: moe.moe_permute_backward(d, rows, inv, out)),
                         (2, lambda: moe.moe_unpermute_combine(d, rows, packed, inv, None, out))):
        out.fill_(777.0)
        call()
        for t in range(0, T, 1 << 21):
            at = inv[t:t + (1 << 21), None].long()
            want = torch.where(at >= 0, rows[at[:, 0].clamp_min(0)] * weight, 0)
            assert torch.equal(out[t:t + (1 << 21)], want), (weight, t)
    del rows, inv, packed, out, want
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_combine_backward_random_values():
    """Random weights and rows: a product and its rounding per row value; dots of D exact products and as many sums."""
    T, D, E, k = 40, 1024, 32, 6
    ids, _, inv, used = routing(T, E, k, 0, E, 5)
    g = torch.Generator().manual_seed(1)
    w, dy, rows = torch.rand(T, k, generator=g), torch.randn(T, D, generator=g).bfloat16(), torch.randn(T * k, D, generator=g).bfloat16()
    d = moe.make_dims(T, D, E, k, 64)
    d_rows, d_w = torch.zeros(T * k, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, k, device="cuda")
    packed = torch.stack([ids.int(), w.view(torch.int32)], 1).contiguous().cuda()
    moe.moe_unpermute_combine_backward(d, dy.cuda(), packed, inv.cuda(), rows.cuda(), d_rows, d_w)
    r = rows.double()[inv.long()]
    dots = (dy.double()[:, None] * r).sum(2)
    mag = (dy.double()[:, None] * r).abs().sum(2)
    assert ((d_w.cpu().double() - dots).abs() <= D * 2.0 ** -24 * mag).all()
    want = w.double()[..., None] * dy.double()[:, None]
    got = d_rows.cpu().double()[inv.long()]
    assert ((got - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs()).all()


# ---------------------------------------------------------------------------
# The whole layer, forward and backward
# ---------------------------------------------------------------------------

def train_step(x, wr, wg, wu, wd, dy, d_loss, k, p, rng, dtype):
    """A training step's calls; rows in moe_permute's order.  Returns the gradients, y and the routing."""
    T, D = x.shape
    E, I = wg.shape[0], wg.shape[1]
    d = moe.make_dims(T, D, E, k, I, act=dtype, w=dtype, out=dtype)
    dev, dt, R = x.device, x.dtype, T * k
    new = lambda *s, t=dt: torch.empty(s, dtype=t, device=dev)  # noqa: E731
    i32 = torch.int32
    ws, logits, packed = moe.workspace(d), new(T, E, t=torch.float32), new(T, 2, k, t=i32)
    moe.moe_route(d, x, wr, logits, None, packed, ws)
    loss, load, lws = new(2, t=torch.float32), new(E + 1, t=i32), moe.route_loss_workspace(d)
    moe.moe_route_loss(d, logits, None, packed, loss, load, ws=lws)
    counts, offsets, perm, inv = new(E, t=i32), new(E + 1, t=i32), new(R, t=i32), new(T, k, t=i32)
    moe.moe_permute(d, packed, counts, offsets, perm, inv, ws=ws)
    up, down = moe.make_groups(E, R, I, D, dtype), moe.make_groups(E, R, D, I, dtype)
    router = moe.make_groups(1, T, E, D, dtype)
    gws = [moe.grouped_gemm_workspace(g) for g in (up, down, router)]
    gate, upv, h, rows, y = new(R, I), new(R, I), new(R, I), new(R, D), new(T, D)
    moe.moe_grouped_gemm(up, x, offsets, wg, gate, index=perm, ws=gws[0])
    moe.moe_grouped_gemm(up, x, offsets, wu, upv, index=perm, ws=gws[0])
    used = offsets[E:]
    moe.moe_swiglu(gate, upv, h, n_rows=used, p=p, rng=rng)
    moe.moe_grouped_gemm(down, h, offsets, wd, rows, ws=gws[1])
    moe.moe_unpermute_combine(d, rows, packed, inv, None, y)

    d_rows, d_w, d_h, d_gate, d_up = new(R, D), new(T, k, t=torch.float32), new(R, I), new(R, I), new(R, I)
    moe.moe_unpermute_combine_backward(d, dy, packed, inv, rows, d_rows, d_w)
    moe.moe_grouped_gemm_backward_rows(down, d_rows, offsets, wd, d_h, ws=gws[1])
    moe.moe_swiglu_backward(d_h, gate, upv, d_gate, d_up, h=h, n_rows=used, p=p, rng=rng)
    dwd, dwg, dwu, dwr = (torch.empty_like(t) for t in (wd, wg, wu, wr))
    moe.moe_grouped_gemm_backward_weights(down, d_rows, h, offsets, dwd, ws=gws[1])
    moe.moe_grouped_gemm_backward_weights(up, d_gate, x, offsets, dwg, index=perm, ws=gws[0])
    moe.moe_grouped_gemm_backward_weights(up, d_up, x, offsets, dwu, index=perm, ws=gws[0])
    d_x_rows, dx, d_logits = new(R, D), new(T, D), new(T, E)
    moe.moe_grouped_gemm_backward_rows(up, d_gate, offsets, wg, d_x_rows, ws=gws[0])
    moe.moe_grouped_gemm_backward_rows(up, d_up, offsets, wu, d_x_rows, add=d_x_rows, ws=gws[0])
    moe.moe_route_backward(d, logits, None, packed, d_w, load, d_loss, d_logits)
    all_t = torch.zeros(2, dtype=i32, device=dev)
    all_t[1:].fill_(T)
    moe.moe_grouped_gemm_backward_rows(router, d_logits, all_t, wr, dx, ws=gws[2])
    moe.moe_permute_backward(d, d_x_rows, inv, dx, add=dx)
    moe.moe_grouped_gemm_backward_weights(router, d_logits, x, all_t, dwr, ws=gws[2])
    return dict(dx=dx, dwr=dwr, dwg=dwg, dwu=dwu, dwd=dwd), y, loss, packed, inv, offsets


def reference_step(x, wr, wg, wu, wd, dy, d_loss, k, ids, inv, keep):
    """Float64 autograd of the same step, the chosen experts given; keep: factors of h's elements [T * k][I]."""
    leaves = [t.double().requires_grad_() for t in (x, wr, wg, wu, wd)]
    x, wr, wg, wu, wd = leaves
    T, E = x.shape[0], wr.shape[0]
    logits = x @ wr.T
    prob = torch.softmax(logits, 1)
    w = torch.softmax(torch.gather(logits, 1, ids), 1)
    y = torch.zeros(T, x.shape[1], dtype=torch.float64)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            g, u = x[t] @ wg[e].T, x[t] @ wu[e].T
            h = torch.nn.functional.silu(g) * u * keep[inv[t, j].long()]
            y = y.index_add(0, t, w[t, j, None] * (h @ wd[e].T))
    load = torch.bincount(ids.reshape(-1), minlength=E).double()
    loss = torch.stack([E / (k * T) * (load * prob.sum(0)).sum() / T, (torch.logsumexp(logits, 1) ** 2).mean()])
    total = (y * dy.double()).sum() + (d_loss.double() * loss).sum()
    grads = torch.autograd.grad(total, leaves)
    return dict(zip(("dx", "dwr", "dwg", "dwu", "dwd"), grads)), y.detach(), loss.detach()


def step_inputs(T, D, E, I, dtype):
    g = torch.Generator().manual_seed(T)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DT[dtype])  # noqa: E731
    return (r(T, D), r(E, D, std=D ** -0.5), r(E, I, D, std=D ** -0.5), r(E, I, D, std=D ** -0.5),
            r(E, D, I, std=I ** -0.5), r(T, D, std=0.1), torch.tensor([0.5, 0.01]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,p", [(1, 0.0), (5, 0.5), (200, 0.1)])
def test_a_training_step(T, p, dtype):
    """2-norms.  Every intermediate tensor is rounded once to its type, half a step (2^-24 or 2^-8) of each value; up to
    8 of them lie between a gradient and its inputs (gate, up, h, rows or d_rows, d_h, d_gate, d_x_rows, the result), and
    random weights pass a relative error of a tensor on as one of the product.  fp32 sums of up to 256 terms add
    256 * 2^-24 each at most, on five products."""
    D, E, I, k = 256, 8, 128, 2
    inputs = step_inputs(T, D, E, I, dtype)
    rng = torch.tensor([11, 22], dtype=torch.int64, device="cuda")
    grads, y, loss, packed, inv, offsets = train_step(*(t.cuda() for t in inputs), k, p, rng, dtype)
    ids = packed[:, 0].long().cpu()
    keep = mask_of(T * k * I, p, (11, 22)).reshape(T * k, I)
    ref, ref_y, ref_loss = reference_step(*inputs, k, ids, inv.cpu(), keep)
    bar = 8 * (2.0 ** -24 if dtype == "f32" else 2.0 ** -8) + 5 * 256 * 2.0 ** -24
    for name, got in (*grads.items(), ("y", y)):
        want = ref_y if name == "y" else ref[name]
        assert (got.cpu().double() - want).norm() <= bar * want.norm(), name
    assert ((loss.cpu().double() - ref_loss).abs() <= 1e-5 * ref_loss).all()


@pytest.mark.gpu
def test_a_training_step_captured():
    """The whole step in one graph: replays on new tokens equal eager steps on the same workspaces' sizes, bit for bit."""
    T, D, E, I, k, p = 64, 128, 8, 64, 2, 0.25
    inputs = [t.cuda() for t in step_inputs(T, D, E, I, "bf16")]
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    want = train_step(*inputs, k, p, rng, "bf16")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = train_step(*inputs, k, p, rng, "bf16")
    for i in range(3):
        inputs[0].copy_(torch.randn(T, D, generator=torch.Generator().manual_seed(i)))
        rng[1] += 1
        graph.replay()
        want = train_step(*inputs, k, p, rng, "bf16")
        torch.cuda.synchronize()
        for name in want[0]:
            assert torch.equal(got[0][name], want[0][name]), name
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------

FAKE, OFF = ctypes.c_void_p(256), ctypes.c_void_p(264)


def test_refusals():
    lib = moe.library()

    def combine(T=8, dy=FAKE, packed=FAKE, inv=FAKE, rows=FAKE, d_rows=FAKE, d_w=FAKE):
        return lib.moe_unpermute_combine_backward(ctypes.byref(moe.make_dims(T, 64, 8, 2, 64)), dy, packed, inv, rows, d_rows,
                                                  d_w, None)

    assert combine(T=0) == moe.OK and combine(T=-1) == moe.ERR_BAD_DIMS
    for bad in (dict(dy=None), dict(packed=None), dict(inv=None), dict(d_rows=None), dict(rows=None), dict(d_w=None)):
        assert combine(**bad) == moe.ERR_NULL_ARG, bad
    for bad in (dict(dy=OFF), dict(rows=OFF), dict(d_rows=OFF)):
        assert combine(**bad) == moe.ERR_UNSUPPORTED, bad

    def permute(T=8, rows=FAKE, inv=FAKE, add=None, dx=FAKE):
        return lib.moe_permute_backward(ctypes.byref(moe.make_dims(T, 64, 8, 2, 64)), rows, inv, add, dx, None)

    assert permute(T=0) == moe.OK and permute(T=-1) == moe.ERR_BAD_DIMS
    for bad in (dict(rows=None), dict(inv=None), dict(dx=None)):
        assert permute(**bad) == moe.ERR_NULL_ARG, bad
    for bad in (dict(rows=OFF), dict(add=OFF), dict(dx=OFF)):
        assert permute(**bad) == moe.ERR_UNSUPPORTED, bad


def test_binding_refusals(monkeypatch):
    monkeypatch.setattr(moe, "_device", lambda: -1)   # where these tensors are: types and sizes are what is refused
    d = moe.make_dims(4, 64, 8, 2, 64)
    dy, rows = torch.zeros(4, 64).bfloat16(), torch.zeros(8, 64).bfloat16()
    pk, inv, dw = torch.zeros(4, 2, 2, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for args, what in (((dy[:3], pk, inv, rows, rows, dw), "dy"), ((dy, pk, inv.long(), rows, rows, dw), "inv_pos"),
                       ((dy, pk, inv, rows.float(), rows, dw), "out_rows"), ((dy, pk, inv, rows, rows[:7], dw), "d_rows"),
                       ((dy, pk, inv, rows, rows, dw.bfloat16()), "d_weights")):
        with pytest.raises(ValueError, match=what):
            moe.moe_unpermute_combine_backward(d, *args)
    with pytest.raises(ValueError, match="d_x_perm"):
        moe.moe_permute_backward(d, rows.float(), inv, dy)
    with pytest.raises(ValueError, match="add"):
        moe.moe_permute_backward(d, rows, inv, dy, add=dy[:1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_no_rows(dtype):
    """No tokens at all: every call succeeds, gradients of weights are zeros."""
    dt = DT[dtype]
    g = moe.make_groups(3, 0, 64, 32, dtype)
    e = lambda *s, t=dt: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    off, w, d_w = torch.zeros(4, dtype=torch.int32, device="cuda"), e(3, 64, 32), torch.ones(3, 64, 32, dtype=dt, device="cuda")
    ws = moe.grouped_gemm_workspace(g)
    moe.moe_grouped_gemm(g, e(0, 32), off, w, e(0, 64), ws=ws)
    moe.moe_grouped_gemm_backward_rows(g, e(0, 64), off, w, e(0, 32), ws=ws)
    moe.moe_grouped_gemm_backward_weights(g, e(0, 64), e(0, 32), off, d_w, ws=ws)
    assert not d_w.any()
    moe.moe_swiglu(e(0, 8), e(0, 8), e(0, 8))
    moe.moe_dropout(e(0), e(0), 0.5, torch.zeros(2, dtype=torch.int64, device="cuda"))
    d = moe.make_dims(0, 64, 8, 2, 64, act=dtype, w=dtype, out=dtype)
    i32 = lambda *s: e(*s, t=torch.int32)  # noqa: E731
    moe.moe_unpermute_combine_backward(d, e(0, 64), i32(0, 2, 2), i32(0, 2), e(0, 64), e(0, 64), e(0, 2, t=torch.float32))
    moe.moe_permute_backward(d, e(0, 64), i32(0, 2), e(0, 64))
