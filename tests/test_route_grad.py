"""Router losses and the gradient of the logits (moe_route_loss, moe_route_backward), against float64 and differences.

Bars.  A probability is exp(key - max) / sum: the difference is off by half a step of itself (|key - max| <= 32 here), the
exponential by 2 steps, a sum of up to 1024 positive values in 16 serial and 6 pairwise steps by 22, the division
by 2: P = 64 * 2^-24 relative in all.  Each further product or sum adds 2^-24 of the magnitudes that it takes, at
most 16 of them on any way through either call; bf16 results add their rounding, 2^-8 of the value.
"""

import ctypes

import pytest
import torch

import sparse_moe_ffn_route_amd as moe

U = 2.0 ** -24
P = 64 * U
HALF = {"f32": U, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    def __init__(self, T, E, k, renorm, mask, bias, seed=0):
        g = torch.Generator().manual_seed(seed + 100 * T + E)
        self.T, self.E, self.k, self.renorm = T, E, k, renorm
        self.logits = torch.randn(T, E, generator=g) * 1.5
        self.bias = None
        if bias:
            self.bias = torch.randn(E, generator=g) * 0.5
            self.bias[torch.randperm(E, generator=g)[:(E - k) // 3]] = -float("inf")
        self.key = self.logits if self.bias is None else self.logits + self.bias
        top, ids = self.key.double().sort(dim=1, descending=True, stable=True)
        w = torch.softmax(top, 1)[:, :k]
        self.w = (w / w.sum(1, keepdim=True) if renorm else w).float()
        self.ids = ids[:, :k]
        self.mask = (torch.rand(T, generator=g) < 0.7).to(torch.uint8) if mask else None
        self.d_w = torch.randn(T, k, generator=g)
        self.d_loss = torch.tensor([0.5, 0.25])
        self.dims = moe.make_dims(T, 64, E, k, 64, renormalize=renorm)

    def on_gpu(self):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        packed = torch.stack([self.ids.int(), self.w.view(torch.int32)], 1).contiguous()
        return c(self.logits), c(self.bias), packed.cuda(), c(self.mask)

    def run(self, out="f32", d_w=True, d_loss=True):
        logits, bias, packed, mask = self.on_gpu()
        loss, load = torch.full((2,), 9.0, device="cuda"), torch.full((self.E + 1,), 9, dtype=torch.int32, device="cuda")
        moe.moe_route_loss(self.dims, logits, bias, packed, loss, load, mask=mask, ws=moe.route_loss_workspace(self.dims))
        d = torch.full((self.T, self.E), 777.0, dtype=DT[out], device="cuda")
        moe.moe_route_backward(self.dims, logits, bias, packed, self.d_w.cuda() if d_w else None,
                               load if d_loss else None, self.d_loss.cuda() if d_loss else None, d, mask=mask)
        return loss.cpu(), load.cpu(), d.cpu()

    def reference(self, d_w=True, d_loss=True):
        """Losses, load and the gradient by float64 autograd, and the magnitudes that its fp32 errors are relative to."""
        on = torch.ones(self.T, dtype=torch.bool) if self.mask is None else self.mask != 0
        load = torch.bincount(self.ids[on].reshape(-1), minlength=self.E)
        n = int(on.sum())
        key = self.key.double().requires_grad_()
        p, lse = torch.softmax(key, 1), torch.logsumexp(key, 1)
        many = max(n, 1)
        bal = self.E / (self.k * many) * (load * p[on].sum(0)).sum() / many
        z = (lse[on] ** 2).sum() / many
        # renormalised: the softmax of the kept keys alone, whose gradient elsewhere is zero in float64, too
        w = torch.softmax(torch.gather(key, 1, self.ids), 1) if self.renorm else torch.gather(p, 1, self.ids)
        total = 0
        if d_w:
            total = total + (w * self.d_w.double()).sum()
        if d_loss:
            total = total + self.d_loss[0].double() * bal + self.d_loss[1].double() * z
        grad, = torch.autograd.grad(total, key)
        p, lse, w = p.detach(), lse.detach(), w.detach()
        err = torch.zeros_like(p)
        if d_w:
            dw = self.d_w.double().abs()
            mean = (w * dw).sum(1, keepdim=True)
            if self.renorm:
                err.scatter_add_(1, self.ids, w * (dw + mean) * 16 * U)
            else:
                err += p * (torch.zeros_like(p).scatter_add_(1, self.ids, dw) + mean) * (P + 16 * U)
        if d_loss:
            q = (p * load).sum(1, keepdim=True)
            top = torch.where(self.key.isfinite(), self.key.double(), 0.0).abs().amax(1, keepdim=True)
            aux = self.d_loss[0] * self.E / self.k / many / many * p * (load + q) * (2 * P + 16 * U)
            aux = aux + self.d_loss[1] * 2 / many * p * (lse.abs()[:, None] * (P + 16 * U) + (top + 8) * P)
            err += aux * on[:, None]
        return torch.stack([bal, z]).detach(), torch.cat([load, torch.tensor([n])]), grad, err


CASES = [(1, 2, 1), (5, 16, 2), (64, 16, 16), (33, 63, 5), (40, 100, 10), (130, 256, 8), (70, 257, 1), (300, 512, 10),
         (9, 1000, 32), (1100, 1024, 10)]


@pytest.mark.gpu
@pytest.mark.parametrize("mask,bias", [(False, False), (True, True)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", CASES)
def test_losses_and_gradient(T, E, k, renorm, mask, bias):
    c = Case(T, E, k, renorm, mask, bias)
    fin = c.key.masked_fill(c.key.isinf(), 0)
    assert (fin.amax(1) - fin.amin(1)).max() <= 32
    for parts in ((True, True), (True, False), (False, True)):
        ref_loss, ref_load, ref, err = c.reference(*parts)
        for out in DT:
            loss, load, d = c.run(out, *parts)
            assert torch.equal(load.long(), ref_load)
            # positive terms: serial over a wave's tokens, 8 waves, 128 workgroups, then 1024 experts by 16 waves
            steps = T / 8 + 8 + 128 + 32
            top = c.key[c.key.isfinite()].abs().max()
            assert abs(loss[0] - ref_loss[0]) <= (steps * U + P + 8 * U) * ref_loss[0]
            z_mag = ref_loss[1] + (2 * (top + 8) * ref_loss[1].sqrt())
            assert abs(loss[1] - ref_loss[1]) <= (steps * U + P + 8 * U) * z_mag
            assert ((d.double() - ref).abs() <= err + HALF[out] * ref.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mask,bias", [(False, False), (True, True)])
@pytest.mark.parametrize("T,E,k", CASES + [(5000, 64, 4), (9000, 512, 10)])
def test_losses_are_sums_of_few_steps(T, E, k, mask, bias):
    """The losses to the steps that their sums have.  Tokens go round 128 workgroups of 16 waves: a wave adds up its own
    ceil(T / 2048), a workgroup its 16 waves, the join b / f workgroups and f such sums, with f = 1024 over the experts'
    next power of two (64 at least), then over a wave in 6 and 16 of those; and up to 8 products and quotients.  The
    log of a sum that is off by P is off by P, and rounded with the largest key, U of each."""
    c = Case(T, E, k, True, mask, bias)
    (bal, z), _, _, _ = c.reference(False, True)
    loss, _, _ = c.run("f32", False, True)
    blocks, f = min(128, -(-T // 16)), 1024 // max(64, 1 << (E - 1).bit_length())
    steps = -(-T // 2048) + 16 + -(-blocks // f) + f + 6 + 16 + 8
    top = float(c.key[c.key.isfinite()].abs().max())
    assert abs(loss[0] - bal) <= (steps * U + P) * bal
    assert abs(loss[1] - z) <= steps * U * z + 2 * z.sqrt() * (P + 2 * U * (top + 8))


@pytest.mark.gpu
def test_calls_repeat_bit_for_bit():
    c = Case(3000, 512, 10, True, True, True)
    a, b = c.run(), c.run()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_masked_tokens_hold_anything():
    """Tokens outside the mask: NaN logits, ids of no expert; and a mask that leaves no token."""
    c = Case(50, 96, 4, True, True, False)
    c.mask[7] = 1
    ref = c.reference(False, True)
    off = c.mask == 0
    c.logits[off] = float("nan")
    c.ids[off] = 4096
    loss, load, d = c.run("f32", False, True)
    assert torch.equal(load.long(), ref[1]) and loss.isfinite().all()
    assert (d[off] == 0).all() and ((d.double() - ref[2]).abs() <= ref[3] + U * ref[2].abs())[~off].all()
    c.mask.zero_()
    loss, load, d = c.run("f32", False, True)
    assert not loss.any() and not load.any() and not d.any()


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [True, False])
def test_tokens_without_a_finite_key(renorm):
    """All keys -inf: nothing in the losses, nothing in the gradient from them."""
    c = Case(6, 40, 2, renorm, False, False)
    c.logits[2] = -float("inf")
    loss, load, d = c.run("f32", False, True)
    assert loss.isfinite().all() and d.isfinite().all() and not d[2].any()
    others = [0, 1, 3, 4, 5]
    z = torch.logsumexp(c.logits[others].double(), 1).square().sum() / 6
    assert abs(loss[1] - z) <= 256 * U * z


@pytest.mark.gpu
@pytest.mark.parametrize("weight", [float("nan"), 0.0])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [40, 63, 512, 1000])
def test_no_gradient_from_the_weights_of_a_token_without_a_finite_key(E, renorm, weight):
    """All keys -inf: no gradient from weights that are their softmax's NaN, or 0."""
    for parts in ((True, False), (True, True)):
        c = Case(6, E, 2, renorm, False, False)
        c.bias = torch.linspace(-1, 1, E)
        c.key = c.logits + c.bias
        top, ids = c.key.double().sort(dim=1, descending=True, stable=True)
        c.ids, w = ids[:, :2], torch.softmax(top, 1)[:, :2]
        c.w = (w / w.sum(1, keepdim=True) if renorm else w).float()
        on = torch.tensor([1, 1, 0, 1, 1, 1], dtype=torch.uint8)
        c.mask = on
        _, _, ref, err = c.reference(*parts)   # of the other tokens, with token 2 outside the losses
        c.logits[2] = -float("inf")
        c.w[2] = weight
        for c.mask in (on, None):
            loss, load, d = c.run("f32", *parts)
            assert loss.isfinite().all() and not d[2].any()
            if c.mask is not None or not parts[1]:
                assert ((d.double() - ref).abs() <= err + U * ref.abs())[on != 0].all()


@pytest.mark.gpu
@pytest.mark.parametrize("E", [40, 512, 1000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_counted_token_that_is_not_finite(E, bad):
    """NaN, or an infinity's NaN, reaches the losses and that token's gradient, and no other token's."""
    for whole_row in (False, True):
        c = Case(6, E, 2, False, False, False)
        ref = c.reference()
        c.logits[2, slice(None) if whole_row else E - 1] = bad
        loss, load, d = c.run()
        assert loss.isnan().all() and d[2].isnan().all() and torch.equal(load.long(), ref[1])
        c.mask = torch.tensor([1, 1, 0, 1, 1, 1], dtype=torch.uint8)
        loss, load, d = c.run("f32", False, True)
        ref = c.reference(False, True)
        others = [0, 1, 3, 4, 5]
        assert loss.isfinite().all() and not d[2].any()
        assert ((d.double() - ref[2]).abs() <= ref[3] + U * ref[2].abs())[others].all()


@pytest.mark.gpu
@pytest.mark.parametrize("low", [-1e4, -1e30, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("renorm", [True, False])
def test_keys_of_the_lowest_value(renorm, low):
    """Experts masked by a large negative number instead of -inf have probability 0, a token of nothing else equal ones.

    Its lse is low + log E, whose log E fp32 drops at the larger two: the z loss of that token is left out of the comparison.
    """
    c = Case(8, 96, 4, renorm, False, False)
    free = torch.ones(8, 96, dtype=torch.bool).scatter_(1, c.ids, False)
    c.logits[free] = low
    c.logits[5] = low
    c.key = c.logits
    top = torch.gather(c.logits.double(), 1, c.ids)
    c.w = torch.softmax(top, 1).float()
    if not renorm:
        c.w[5] = 1 / 96
    c.d_loss = torch.tensor([0.5, 0.0])
    _, ref_load, ref, err = c.reference()
    loss, load, d = c.run()
    on = torch.tensor([0, 1, 2, 3, 4, 6, 7])
    assert torch.equal(load.long(), ref_load) and d.isfinite().all()
    assert ((d.double() - ref).abs() <= err + U * ref.abs()).all()
    assert not d[on][free[on]].any()


@pytest.mark.gpu
def test_workspace_is_as_large_as_said():
    """Bytes behind the workspace stay, and what it held before does not matter."""
    for T, E in ((1, 8), (17, 63), (3000, 512)):
        c = Case(T, E, 2, True, False, False)
        logits, bias, packed, mask = c.on_gpu()
        need = moe.route_loss_workspace(c.dims).nbytes
        results = []
        for fill in (0, 255):
            ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
            ws[need:] = 171
            loss, load = torch.empty(2, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
            moe.moe_route_loss(c.dims, logits, bias, packed, loss, load, mask=mask, ws=ws[:need])
            assert (ws[need:] == 171).all()
            results.append((loss, load))
        assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


@pytest.mark.gpu
def test_an_expert_named_twice():
    """Gradients of slots with one id add up at that expert."""
    c = Case(4, 32, 4, True, False, False)
    c.ids[1] = torch.tensor([5, 5, 9, 5])
    loss, load, d = c.run("f32", True, False)
    w, dw = c.w[1].double(), c.d_w[1].double()
    x = w * (dw - (w * dw).sum())
    want = torch.zeros(32, dtype=torch.float64).index_add_(0, c.ids[1], x)
    assert ((d[1].double() - want).abs() <= 32 * U * (w * (dw.abs() + (w * dw.abs()).sum())).sum()).all()
    assert load[5] == int((c.ids == 5).sum())


@pytest.mark.gpu
def test_no_tokens():
    c = Case(0, 16, 2, True, False, False)
    loss, load, _ = c.run()
    assert not loss.any() and not load.any()


@pytest.mark.gpu
def test_gradient_against_differences():
    """Differences of the losses that moe_route_loss returns, step e = 2^-3 of one logit of every token at a time.

    A loss's third derivative by a logit is below 4 / n times its scale (E / k max load / n for the balance; 8 |lse| + 8 for
    z), so differences are off by e^2 / 6 of it; the losses' fp32 sums by 2^-17 of their value over 2 e.
    """
    T, E, k, e = 6, 12, 2, 2.0 ** -3
    c = Case(T, E, k, True, True, True, seed=3)
    c.mask[:] = torch.tensor([1, 1, 0, 1, 1, 1], dtype=torch.uint8)
    c.bias = None
    for which in (0, 1):
        c.d_loss = torch.eye(2)[which].contiguous()
        base, load, d = c.run("f32", False, True)
        scale = E / k * float(load[:E].max()) / 5 if which == 0 else 8 * float(torch.logsumexp(c.logits, 1).abs().max()) + 8
        for t in range(T):
            for x in range(E):
                got = []
                for step in (e, -e):
                    saved = c.logits[t, x].item()
                    c.logits[t, x] = saved + step
                    got.append(c.run("f32", False, True)[0][which].double())
                    c.logits[t, x] = saved
                bound = e * e / 6 * 4 / 5 * scale + 2.0 ** -17 * float(base[which]) / e
                assert abs((got[0] - got[1]) / (2 * e) - d[t, x]) <= bound


@pytest.mark.gpu
def test_capture():
    """The pair captured: replays on new logits between eager calls on the same workspace, bit for bit."""
    c = Case(200, 64, 4, True, True, False)
    logits, bias, packed, mask = c.on_gpu()
    ws = moe.route_loss_workspace(c.dims)
    loss, load = torch.empty(2, device="cuda"), torch.empty(65, dtype=torch.int32, device="cuda")
    d, d_w, d_loss = torch.empty(200, 64, device="cuda"), c.d_w.cuda(), c.d_loss.cuda()

    def both():
        moe.moe_route_loss(c.dims, logits, bias, packed, loss, load, mask=mask, ws=ws)
        moe.moe_route_backward(c.dims, logits, bias, packed, d_w, load, d_loss, d, mask=mask)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in range(4):
        logits.copy_(torch.randn(200, 64, generator=torch.Generator().manual_seed(i)))
        mask.copy_((torch.rand(200, generator=torch.Generator().manual_seed(i)) < 0.5).to(torch.uint8))
        graph.replay()
        replayed = [t.clone() for t in (loss, load, d)]
        both()
        assert all(torch.equal(x, y) for x, y in zip(replayed, (loss, load, d)))


FAKE = ctypes.c_void_p(256)


def test_refusals():
    lib = moe.library()
    d = moe.make_dims(8, 64, 16, 2, 64)
    need = lib.moe_route_loss_workspace_bytes(ctypes.byref(d))
    assert need > 0 and lib.moe_route_loss_workspace_bytes(ctypes.byref(moe.make_dims(8, 64, 16, 17, 64))) == 0

    def loss(d=d, logits=FAKE, packed=FAKE, out=FAKE, load=FAKE, ws=FAKE, nb=need):
        return lib.moe_route_loss(ctypes.byref(d), logits, None, packed, None, out, load, ws, nb, None)

    for bad in (dict(logits=None), dict(packed=None), dict(out=None), dict(load=None), dict(ws=None)):
        assert loss(**bad) == moe.ERR_NULL_ARG, bad
    assert loss(nb=need - 1) == moe.ERR_WORKSPACE
    assert loss(ws=ctypes.c_void_p(264)) == moe.ERR_UNSUPPORTED
    assert loss(d=moe.make_dims(8, 64, 2048, 2, 64)) == moe.ERR_UNSUPPORTED
    assert loss(d=moe.make_dims(-1, 64, 16, 2, 64)) == moe.ERR_BAD_DIMS

    def grad(logits=FAKE, packed=FAKE, d_w=FAKE, load=FAKE, d_loss=FAKE, dt=moe.F32, out=FAKE):
        return lib.moe_route_backward(ctypes.byref(d), logits, None, packed, None, d_w, load, d_loss, dt, out, None)

    for bad in (dict(logits=None), dict(packed=None), dict(out=None), dict(load=None), dict(d_w=None, d_loss=None)):
        assert grad(**bad) == moe.ERR_NULL_ARG, bad
    assert grad(dt=moe.E4M3) == moe.ERR_UNSUPPORTED


def test_binding_refusals(monkeypatch):
    monkeypatch.setattr(moe, "_device", lambda: -1)   # where these tensors are: types and sizes are what is refused
    d = moe.make_dims(8, 64, 16, 2, 64)
    lg, pk = torch.zeros(8, 16), torch.zeros(8, 2, 2, dtype=torch.int32)
    loss, load = torch.zeros(2), torch.zeros(17, dtype=torch.int32)
    for args, what in (((lg.double(), None, pk, loss, load), "logits"), ((lg, None, pk[:4], loss, load), "packed"),
                       ((lg, None, pk, loss[:1], load), "loss"), ((lg, None, pk, loss, load[:16]), "load"),
                       ((lg, lg[0, :8], pk, loss, load), "bias")):
        with pytest.raises(ValueError, match=what):
            moe.moe_route_loss(d, *args)
    with pytest.raises(ValueError, match="mask"):
        moe.moe_route_loss(d, lg, None, pk, loss, load, mask=lg)
    with pytest.raises(ValueError, match="d_logits"):
        moe.moe_route_backward(d, lg, None, pk, None, load, loss, lg[:4])
    with pytest.raises(ValueError, match="d_weights"):
        moe.moe_route_backward(d, lg, None, pk, lg[0, :8], load, loss, lg)
