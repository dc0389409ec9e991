"""Counter-based dropout (moe_dropout) and the activation that holds it (moe_swiglu, moe_swiglu_backward).

The generator is checked against an implementation in Python's whole numbers and against Philox-4x32-10's published
known answers; the activation against float64.  Bars: half a step of the result's type (2^-8 bf16, 2^-24 fp32) of its
value, plus the fp32 arithmetic.  That is, in units of 2^-24 of the magnitudes that are added: each product and sum 1;
the sigmoid 1 for the division or 2 for the hardware reciprocal and its sum, and for the exponential e^-g either 2 or,
through the hardware's base-2 one, 2 + |g| (the product with log2 e is off by half a step of |g| log2 e, an absolute
error that the power makes relative).  With |g| <= 16 that is at most 24 for the sigmoid and 32 for any result.
"""

import ctypes

import numpy as np
import pytest
import torch

import sparse_moe_ffn_route_amd as moe

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
ARITH = 32 * 2.0 ** -24
M = 0xFFFFFFFF


def philox(c, k):
    """Philox-4x32-10 in Python's whole numbers."""
    c, k = list(c), list(k)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & M, (a >> 32) ^ c[3] ^ k[1], a & M]
        k = [(k[0] + 0x9E3779B9) & M, (k[1] + 0xBB67AE85) & M]
    return c


def mask_of(n, p, rng, first=0):
    """Factors (0 or 1 / (1 - p)) of elements first .. first + n - 1."""
    seed, offset = (v & (2 ** 64 - 1) for v in rng)
    low = round(p * 65536)
    out, block, words = np.zeros(n), -1, None
    for i in range(n):
        e = first + i
        if e // 8 != block:
            block = e // 8
            words = philox([block & M, block >> 32, offset & M, offset >> 32], [seed & M, seed >> 32])
        bits = words[e % 8 // 2] >> (16 * (e % 2)) & 0xFFFF
        out[i] = 65536 / (65536 - low) if bits >= low else 0.0
    return torch.from_numpy(out)


def test_known_answers():
    """The generator's published test vectors."""
    assert philox([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert philox([M] * 4, [M] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert philox([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0]) == \
        [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


RNGS = [(0, 0), (12345, 7), (-1, -2), (0x123456789ABCDEF0, 1 << 40)]


def rand(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(DT[dtype])


def rng_of(rng):
    return torch.tensor(rng, dtype=torch.int64, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("rng", RNGS)
@pytest.mark.parametrize("n,p", [(1, 0.5), (7, 0.5), (8, 0.1), (1000, 0.1), (4096, 0.5), (20011, 0.9)])
def test_dropout_mask_and_sum(n, p, rng):
    keep = mask_of(n, p, rng)
    for dtype in DT:
        x, r = rand((n,), dtype, 1), rand((n,), dtype, 2)
        out = torch.empty_like(x, device="cuda")
        moe.moe_dropout(torch.ones_like(x).cuda(), out, p, rng_of(rng))
        assert torch.equal(out.cpu(), keep.to(torch.float32).to(DT[dtype]))
        for residual in (None, r):
            moe.moe_dropout(x.cuda(), out, p, rng_of(rng), residual=None if residual is None else r.cuda())
            ref = keep * x.double() + (0 if residual is None else r.double())
            mag = (keep * x.double()).abs() + (0 if residual is None else r.double().abs())
            # the factor, its product and the sum
            assert ((out.cpu().double() - ref).abs() <= 3 * 2.0 ** -24 * mag + HALF[dtype] * ref.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_dropout_ends_of_p(dtype):
    x, r = rand((3, 77), dtype, 1), rand((3, 77), dtype, 2)
    x[1] = float("nan")
    x[2, :5] = float("inf")
    out = torch.empty_like(x, device="cuda")
    moe.moe_dropout(x.cuda(), out, 1.0, rng_of((1, 2)), residual=r.cuda())
    assert torch.equal(out.cpu(), r)                       # all dropped, whatever they hold
    moe.moe_dropout(x.cuda(), out, 0.0)
    assert torch.equal(out.cpu().nan_to_num(9.0), x.nan_to_num(9.0))
    moe.moe_dropout(x.cuda(), out, 2.0 ** -18)             # rounds to nothing dropped
    assert torch.equal(out.cpu().nan_to_num(9.0), x.nan_to_num(9.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_dropout_in_place_and_off_16_bytes(dtype):
    n, p, rng = 1003, 0.3, (5, 6)
    x, r = rand((n,), dtype, 1), rand((n,), dtype, 2)
    want = torch.empty_like(x, device="cuda")
    moe.moe_dropout(x.cuda(), want, p, rng_of(rng), residual=r.cuda())
    for over in ("x", "residual"):
        xs, rs = x.cuda(), r.cuda()
        moe.moe_dropout(xs, xs if over == "x" else rs, p, rng_of(rng), residual=rs)
        assert torch.equal(xs if over == "x" else rs, want)
    wide = torch.full((n + 9,), 555.0, dtype=DT[dtype], device="cuda")
    xs = torch.cat([x[:3], x]).cuda()[3:]
    moe.moe_dropout(xs, wide[1:n + 1], p, rng_of(rng), residual=r.cuda())
    assert torch.equal(wide[1:n + 1], want) and wide[0] == 555 and (wide[n + 1:] == 555).all()


@pytest.mark.gpu
def test_dropped_share_and_independence():
    """Of 2^20 elements the dropped ones' number is within 5 standard deviations; other offsets and seeds agree by chance."""
    n, p = 1 << 20, 0.25
    ones, out = torch.ones(n, device="cuda"), torch.empty(n, device="cuda")
    masks = []
    for rng in ((1, 1), (1, 2), (2, 1)):
        moe.moe_dropout(ones, out, p, rng_of(rng))
        masks.append(out == 0)
        assert abs(int(masks[-1].sum()) - n * p) <= 5 * (n * p * (1 - p)) ** 0.5
    for a, b in ((0, 1), (0, 2), (1, 2)):
        q = p * p
        assert abs(int((masks[a] & masks[b]).sum()) - n * q) <= 5 * (n * q * (1 - q)) ** 0.5


@pytest.mark.gpu
def test_dropout_past_32_bits():
    """Elements past 2^32: their block number needs the counter's second word only past 2^35, their place 64 bits."""
    n, p, rng = (1 << 32) + 24, 0.5, (9, 3)
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    moe.moe_dropout(x, x, p, rng_of(rng))
    for first in (0, (1 << 31) - 4, (1 << 32) - 4):
        got = x[first:first + 24].cpu().double()
        assert torch.equal(got, mask_of(24, p, rng, first))


def swiglu_reference(g, u, d, keep):
    g, u, d = g.double(), u.double(), d.double() * keep
    s = torch.sigmoid(g)
    h, dg, du = keep * g * s * u, d * u * s * (1 + g * (1 - s)), d * g * s
    # magnitudes of what the fp32 steps add up: 1 + g (1 - s)
    return (h, dg, du), (h.abs(), d.abs() * u.abs() * s * (1 + g.abs() * (1 - s) + g.abs()), du.abs())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,I,p", [(1, 8, 0.1), (1, 1, 0.5), (3, 7, 0.5), (5, 33, 0.0), (40, 64, 0.1), (17, 136, 0.9)])
def test_swiglu(rows, I, p, dtype):
    rng = (77, rows)
    g, u, d = rand((rows, I), dtype, 1, 3.0).clamp(-16, 16), rand((rows, I), dtype, 2), rand((rows, I), dtype, 3)
    keep = mask_of(rows * I, p, rng).reshape(rows, I)
    refs, mags = swiglu_reference(g, u, d, keep)
    gs, us, ds = g.cuda(), u.cuda(), d.cuda()
    h, h2, dg, du = (torch.empty_like(gs) for _ in range(4))
    moe.moe_swiglu(gs, us, h, p=p, rng=rng_of(rng))
    moe.moe_swiglu_backward(ds, gs, us, dg, du, h=h2, p=p, rng=rng_of(rng))
    assert torch.equal(h, h2)
    for got, ref, mag in zip((h, dg, du), refs, mags):
        assert ((got.cpu().double() - ref).abs() <= ARITH * mag + HALF[dtype] * ref.abs()).all()
        assert (got.cpu()[keep == 0] == 0).all()
    # halves of one tensor, n_rows, without h
    both = torch.cat([gs, us], 1)
    d_both = torch.full_like(both, 555.0)
    used = torch.tensor([rows - 1], dtype=torch.int32, device="cuda")
    h2.fill_(555.0)
    moe.moe_swiglu(both[:, :I], both[:, I:], h2, n_rows=used, p=p, rng=rng_of(rng))
    moe.moe_swiglu_backward(ds, both[:, :I], both[:, I:], d_both[:, :I], d_both[:, I:], n_rows=used, p=p, rng=rng_of(rng))
    assert torch.equal(h2[:-1], h[:-1]) and torch.equal(d_both[:-1], torch.cat([dg, du], 1)[:-1])
    assert (h2[-1] == 555).all() and (d_both[-1] == 555).all()
    # in place
    moe.moe_swiglu_backward(ds, gs, us, gs, us, h=ds, p=p, rng=rng_of(rng))
    assert torch.equal(gs, dg) and torch.equal(us, du) and torch.equal(ds, h)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_swiglu_extremes(dtype):
    """Gates past the exponential's range; dropped elements that hold infinities and NaN."""
    g = torch.tensor([[-1e4, -200.0, -89.0, 89.0, 200.0, 1e4, 0.0, -0.0]]).to(DT[dtype])
    u, d = torch.full_like(g, 2.0), torch.full_like(g, 0.5)
    h, dg, du = (torch.empty_like(g, device="cuda") for _ in range(3))
    moe.moe_swiglu_backward(d.cuda(), g.cuda(), u.cuda(), dg, du, h=h)
    assert torch.equal(dg.cpu()[0, [0, 1, 4, 5]], torch.tensor([0.0, 0.0, 1.0, 1.0]).to(DT[dtype]))
    assert torch.equal(h.cpu()[0, [0, 1, 4, 5]].float(), torch.stack([g[0, 0] * 0, g[0, 0] * 0, g[0, 4] * 2, g[0, 5] * 2]).float())
    assert dg.isfinite().all() and du.isfinite().all() and (dg[0, 6:] == 0.5).all()
    n, p, rng = 512, 0.5, (3, 3)
    keep = mask_of(n, p, rng).reshape(1, n)
    g, u, d = rand((1, n), dtype, 1), rand((1, n), dtype, 2), rand((1, n), dtype, 3)
    for t, v in ((g, float("nan")), (u, float("inf")), (d, float("-inf"))):
        t[keep == 0] = v
    h, dg, du = (torch.empty_like(g, device="cuda") for _ in range(3))
    moe.moe_swiglu_backward(d.cuda(), g.cuda(), u.cuda(), dg, du, h=h, p=p, rng=rng_of(rng))
    for t in (h, dg, du):
        assert t.isfinite().all() and (t.cpu()[keep == 0] == 0).all()


@pytest.mark.gpu
def test_swiglu_gradient_against_differences():
    """fp32, against differences of the forward call in float64 sums: step 2^-7, whose error is a third derivative's."""
    rows, I, p, rng = 3, 16, 0.25, (4, 4)
    g, u, d = rand((rows, I), "f32", 1).cuda(), rand((rows, I), "f32", 2).cuda(), rand((rows, I), "f32", 3).cuda()
    dg, du = torch.empty_like(g), torch.empty_like(g)
    moe.moe_swiglu_backward(d, g, u, dg, du, p=p, rng=rng_of(rng))

    def loss(g, u):
        h = torch.empty_like(g)
        moe.moe_swiglu(g, u, h, p=p, rng=rng_of(rng))
        return h.double() * d.double()

    e = 2.0 ** -7
    scale = (d * u).abs().double() / (1 - p)
    by_g = (loss(g + e, u) - loss(g - e, u)) / (2 * e)
    # |silu'''| < 0.6: e^2 / 6 of it; fp32 values of the loss, up to 8 times scale, off by 32 * 2^-24 over the step
    assert ((by_g - dg.double()).abs() <= scale * (0.1 * e * e + 8 * ARITH / e) + 1e-6).all()
    by_u = (loss(g, u + e) - loss(g, u - e)) / (2 * e)
    assert ((by_u - du.double()).abs() <= (d * g).abs().double() / (1 - p) * 8 * ARITH / e + 1e-5).all()


@pytest.mark.gpu
def test_replays_read_new_numbers():
    """A captured forward and backward pair: each replay takes the seed and offset that rng then holds."""
    rows, I, p = 9, 40, 0.5
    g, u, d = (rand((rows, I), "bf16", i).cuda() for i in (1, 2, 3))
    rng = rng_of((1, 0))
    h, dg, du = (torch.empty_like(g) for _ in range(3))
    side = torch.cuda.Stream()
    moe.moe_swiglu(g, u, h, p=p, rng=rng, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_swiglu(g, u, h, p=p, rng=rng)
        moe.moe_swiglu_backward(d, g, u, dg, du, p=p, rng=rng)
        rng[1] += 1
    for step in range(4):
        torch.cuda.synchronize()
        now = rng.tolist()
        assert now == [1, step]
        graph.replay()
        keep = mask_of(rows * I, p, now).reshape(rows, I) > 0
        live = (g.cpu() != 0) & (u.cpu() != 0) & (d.cpu() != 0)
        assert torch.equal((h.cpu() != 0)[live], keep[live]) and torch.equal((du.cpu() != 0)[live], keep[live])
        e = torch.empty_like(h)
        moe.moe_swiglu(g, u, e, p=p, rng=rng_of(now))
        assert torch.equal(e, h)


FAKE = ctypes.c_void_p(256)


def test_refusals():
    lib = moe.library()

    def swiglu(rows=2, I=8, ld=8, dt=moe.BF16, p=0.5, g=FAKE, u=FAKE, rng=FAKE, h=FAKE):
        f = lib.moe_swiglu(rows, I, ld, dt, None, g, u, p, rng, h, None)
        b = lib.moe_swiglu_backward(rows, I, ld, dt, None, FAKE, g, u, p, rng, h, FAKE, None, None)
        assert f == b
        return f

    assert swiglu(rows=0) == moe.OK
    for bad in (dict(rows=-1), dict(I=0), dict(ld=7), dict(p=-0.1), dict(p=1.5), dict(p=float("nan"))):
        assert swiglu(**bad) == moe.ERR_BAD_DIMS, bad
    for bad in (dict(dt=moe.E4M3), dict(rows=1 << 40)):
        assert swiglu(**bad) == moe.ERR_UNSUPPORTED, bad
    for bad in (dict(g=None), dict(u=None), dict(h=None), dict(rng=None)):
        assert swiglu(**bad) == moe.ERR_NULL_ARG, bad
    assert lib.moe_swiglu_backward(2, 8, 8, moe.F32, None, None, FAKE, FAKE, 0.0, None, FAKE, FAKE, None, None) == moe.ERR_NULL_ARG
    assert lib.moe_dropout(0, moe.F32, None, None, 0.5, FAKE, None, None) == moe.OK
    assert lib.moe_dropout(-1, moe.F32, FAKE, None, 0.5, FAKE, FAKE, None) == moe.ERR_BAD_DIMS
    assert lib.moe_dropout(8, moe.MXFP4, FAKE, None, 0.5, FAKE, FAKE, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_dropout(8, moe.F32, FAKE, None, 0.5, None, FAKE, None) == moe.ERR_NULL_ARG
    assert lib.moe_dropout(8, moe.F32, FAKE, None, 2.0, FAKE, FAKE, None) == moe.ERR_BAD_DIMS
    assert lib.moe_dropout(8, moe.F32, None, None, 0.5, FAKE, FAKE, None) == moe.ERR_NULL_ARG


def test_binding_refusals(monkeypatch):
    monkeypatch.setattr(moe, "_device", lambda: -1)   # where these tensors are: types and sizes are what is refused
    g = torch.zeros(4, 16)
    h = torch.zeros(4, 16)
    for args in ((g, g[:3], h), (g, g.bfloat16(), h), (g, torch.zeros(4, 32)[:, :16], h), (g.t(), g.t(), h)):
        with pytest.raises(ValueError):
            moe.moe_swiglu(*args)
    with pytest.raises(ValueError, match="h"):
        moe.moe_swiglu(g, g, h[:2])
    with pytest.raises(ValueError, match="rng"):
        moe.moe_dropout(g, h, 0.5, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="residual"):
        moe.moe_dropout(g, h, 0.5, residual=g.bfloat16())
    monkeypatch.undo()
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_dropout(g, h, 0.0)
