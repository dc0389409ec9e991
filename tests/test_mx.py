"""Microscaled FP4 weights: the packed images, the grouped experts on them, and the whole layer.

Bars.  Images and unpacked values: bit-exact.  Grouped experts: |out - ref| <= half a step of the output type
times |ref| (2^-8 bf16, 2^-24 fp32), plus 1e-4 of the row's largest value for the fp32 sums (the bar of the fp32
layer), plus the slack of values of h that lie on a rounding border (mx_reference.grouped_ffn).
"""

import ctypes

import numpy as np
import pytest
import torch

import mx_reference as mx
import oracle
import sparse_moe_ffn_route_amd as moe
from harness import to_np


# ---------------------------------------------------------------------------
# Host
# ---------------------------------------------------------------------------

def test_weight_bytes():
    # one 16-row fragment: whole groups of 512 are 4 KB of codes and 256 bytes of scales
    assert moe.moe_mx_weight_bytes(1, 16, 512) == 4096 + 256
    assert moe.moe_mx_weight_bytes(3, 32, 1024) == 3 * 2 * 2 * 4352
    assert moe.moe_mx_weight_bytes(1, 16, 64) == 1024 + 256
    assert moe.moe_mx_weight_bytes(1, 16, 704) == 6 * 1024 + 2 * 256
    assert moe.moe_mx_weight_bytes(0, 16, 64) == 0
    for bad in ((1, 24, 64), (1, 16, 96), (-1, 16, 64), (1, -16, 64), (1, 65536, 65536)):
        assert moe.moe_mx_weight_bytes(*bad) == 0


def test_pack_and_unpack_argument_checks():
    lib = moe.library()
    fake = ctypes.c_void_p(256)
    for f in (lib.moe_mx_pack_weights, lib.moe_mx_unpack_weights):
        assert f(moe.E4M3, 1, 16, 64, fake, fake, None) == moe.ERR_UNSUPPORTED
        assert f(moe.MXFP4, 1, 16, 64, fake, fake, None) == moe.ERR_UNSUPPORTED
        assert f(moe.BF16, 1, 8, 64, fake, fake, None) == moe.ERR_UNSUPPORTED
        assert f(moe.BF16, 1, 16, 32, fake, fake, None) == moe.ERR_UNSUPPORTED
        assert f(moe.BF16, -1, 16, 64, fake, fake, None) == moe.ERR_BAD_DIMS
        assert f(moe.BF16, 1 << 62, 16, 64, fake, fake, None) == moe.ERR_UNSUPPORTED
        assert f(moe.BF16, 1, 16, 64, None, fake, None) == moe.ERR_NULL_ARG
        assert f(moe.BF16, 1, 16, 64, fake, None, None) == moe.ERR_NULL_ARG
        assert f(moe.BF16, 0, 16, 64, None, None, None) == moe.OK
        assert f(moe.BF16, 1, 16, 64, ctypes.c_void_p(264), fake, None) == moe.ERR_UNSUPPORTED  # off 16 bytes
        assert f(moe.BF16, 1, 16, 64, fake, ctypes.c_void_p(264), None) == moe.ERR_UNSUPPORTED
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        moe.moe_mx_pack_weights(torch.zeros(16, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="images"):
        moe.moe_mx_pack_weights(torch.zeros(16, 64), dst=torch.zeros(10, dtype=torch.uint8))
    with pytest.raises(ValueError, match="images"):
        moe.moe_mx_unpack_weights(torch.zeros(1281, dtype=torch.uint8), 16, 64)


def test_dims_take_mxfp4_with_packed_bf16_only():
    ok = dict(T=8, D=64, E=8, top_k=2, I=64, act="bf16", w="mxfp4", out="bf16", layout="packed")
    assert moe.moe_workspace_bytes(moe.make_dims(**ok)) > 0
    assert moe.moe_workspace_bytes(moe.make_dims(**{**ok, "out": "f32"})) > 0
    for bad in (dict(layout="rows"), dict(act="f32"), dict(act="f32", out="f32"), dict(D=96)):
        assert moe.moe_workspace_bytes(moe.make_dims(**{**ok, **bad})) == 0
    lib = moe.library()
    d, fake = moe.make_dims(**ok), ctypes.c_void_p(256)
    w = moe.moe_weights(fake, fake, fake, fake, None, None, None, None, None, None)
    off = ctypes.c_void_p(264)
    for i in range(5):                          # rows, images, output off a 16-byte boundary
        p = [off if i == j else fake for j in range(5)]
        assert lib.moe_grouped_ffn(ctypes.byref(d), p[0], None, None, fake, p[1], p[2], p[3], None, None, None, p[4],
                                   fake, 1 << 30, None) == moe.ERR_UNSUPPORTED
    assert lib.moe_audit_workspace_bytes(ctypes.byref(d), 4) == 0
    assert lib.moe_audit(ctypes.byref(d), ctypes.byref(w), fake, fake, fake, fake, 4, None, fake, fake, 1 << 30,
                         None) == moe.ERR_UNSUPPORTED


def test_reference_rounding():
    """The reference itself, on values whose answers are known."""
    v = np.zeros(64)
    v[:12] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.76, 7.9, 0.1]
    v[32:34] = [1.0, 0.0625]
    q = mx.quantise(v)
    np.testing.assert_array_equal(q[:12], [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.0, -1.0, 6.0, 0.0])
    np.testing.assert_array_equal(q[32:34], [1.0, 0.0])   # scale 1/4: 1/16 lies on the tie between 0 and 1/8


# ---------------------------------------------------------------------------
# Images
# ---------------------------------------------------------------------------

def _source(rng, shape, dtype):
    v = rng.standard_normal(shape).astype(np.float32)
    v.reshape(-1, 32)[1::7] *= 2.0 ** rng.integers(-40, 40, (len(v.reshape(-1, 32)[1::7]), 1))
    v.reshape(-1, 32)[2::11] = 0.0                                   # zero blocks
    v.reshape(-1, 32)[3::13] = rng.choice([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -5.0],
                                          (len(v.reshape(-1, 32)[3::13]), 32))   # ties
    v.reshape(-1, 32)[4::17] *= 2.0 ** -130                          # subnormal magnitudes
    return torch.from_numpy(v).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,rows,cols", [(1, 16, 64), (2, 48, 512), (3, 32, 704), (1, 16, 1088), (5, 64, 128)])
def test_pack_weights_image_and_values(n, rows, cols, dtype):
    src = _source(np.random.default_rng(cols + n), (n, rows, cols), dtype)
    codes, exps = mx.encode(src.to(torch.float64).numpy())
    guard = torch.full((n * moe.moe_mx_weight_bytes(1, rows, cols) + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    moe.moe_mx_pack_weights(src.cuda(), guard)
    np.testing.assert_array_equal(guard[:-64].cpu().numpy().reshape(n, -1), mx.image(codes, exps))
    assert (guard[-64:] == 0xA5).all()
    for out in (torch.bfloat16, torch.float32):
        got = moe.moe_mx_unpack_weights(guard[:-64], rows, cols, out)
        # bf16's smallest subnormal is 2^-133: a value below half of it is out of bf16's reach
        want = mx.decode(codes, exps)
        if out == torch.bfloat16:
            want = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16).to(torch.float64).numpy()
        np.testing.assert_array_equal(to_np(got), want)


def _around_every_border(dtype):
    """Per exponent field: a largest value, and what lies around every rounding border below it, as [16][cols]."""
    if dtype == torch.bfloat16:
        man = torch.arange(128)
        field = torch.arange(1, 255)[:, None, None]
        v = ((field - torch.arange(5)[:, None]).clamp(min=0) << 7 | man).reshape(254, -1)  # five binades' values
        top = (torch.arange(1, 255) << 7 | 127)
        bits = torch.cat([v, v | 0x8000], 1)
    else:
        tie = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]).view(torch.int32)
        tie = torch.cat([tie - 1, tie, tie + 1]).long()
        field = torch.arange(1, 255)
        v = torch.where(field[:, None] > 6, tie + ((field[:, None] - 129) << 23), torch.randint(1 << 22, (254, 24)))
        top = field << 23 | 0x7FFFFF
        bits = torch.cat([v, v | 0x80000000], 1)
    n = -(-bits.shape[1] // 31)
    out = torch.zeros(254, n, 32, dtype=torch.int64)
    out[:, :, 31] = top[:, None]
    flat = torch.zeros(254, n * 31, dtype=torch.int64)
    flat[:, :bits.shape[1]] = bits
    out[:, :, :31] = flat.reshape(254, n, 31)
    flat = out.reshape(-1)
    cols = -(-flat.numel() // 16 // 64) * 64
    flat = torch.cat([flat, torch.zeros(16 * cols - flat.numel(), dtype=torch.int64)]).reshape(16, cols)
    if dtype == torch.bfloat16:
        return torch.where(flat > 32767, flat - 65536, flat).to(torch.int16).view(torch.bfloat16)
    return torch.where(flat > 2 ** 31 - 1, flat - 2 ** 32, flat).to(torch.int32).view(torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pack_weights_around_every_border(dtype):
    v = _around_every_border(dtype)
    codes, exps = mx.encode(v.double().numpy()[None])
    img = moe.moe_mx_pack_weights(v.cuda()[None])
    np.testing.assert_array_equal(img.cpu().numpy().reshape(1, -1), mx.image(codes, exps))
    back = moe.moe_mx_unpack_weights(img, *v.shape, dtype=torch.float32).cpu().numpy()
    np.testing.assert_array_equal(back, mx.decode(codes, exps).astype(np.float32))


@pytest.mark.gpu
def test_pack_weights_non_finite_blocks():
    """A NaN or an infinity makes its block NaN and no other."""
    src = torch.randn(1, 16, 128)
    src[0, 3, 40], src[0, 5, 0], src[0, 7, 127] = float("nan"), float("inf"), float("-inf")
    got = to_np(moe.moe_mx_unpack_weights(moe.moe_mx_pack_weights(src.cuda()), 16, 128))[0]
    want = mx.quantise(src[0].numpy())
    np.testing.assert_array_equal(got, want)
    assert np.isnan(got[3, 32:64]).all() and np.isnan(got[5, :32]).all() and np.isnan(got[7, 96:]).all()
    assert np.isnan(got).sum() == 96


# ---------------------------------------------------------------------------
# Grouped experts
# ---------------------------------------------------------------------------

def _weights(rng, n, D, I):
    """(bf16 source tensors, images, decoded values) of gate, up, down."""
    src = [torch.from_numpy((rng.standard_normal(s) / np.sqrt(s[-1])).astype(np.float32)).to(torch.bfloat16)
           for s in ((n, I, D), (n, I, D), (n, D, I))]
    img = [moe.moe_mx_pack_weights(s.cuda()) for s in src]
    val = [mx.quantise(to_np(s)) for s in src]
    return src, img, val


def _check_rows(got, ref, slack, half_step):
    lim = half_step * np.abs(ref) + 1e-4 * np.abs(ref).max(1, keepdims=True) + slack * (1 + half_step)
    assert (np.abs(got - ref) <= lim).all(), float((np.abs(got - ref) - lim).max())


FFN = [
    # (rows of each group, D, I, out): tiles of 32 or 128 rows, by the average and the number of tiles
    ([1], 64, 64, "bf16"),
    ([5, 0, 16, 17, 1, 0, 3], 256, 128, "f32"),
    ([20, 31, 33, 0, 16], 704, 320, "bf16"),
    ([130, 1, 128, 0, 300, 64, 97], 576, 192, "bf16"),
    ([260, 40], 1088, 576, "f32"),
    ([0, 0, 40, 0], 128, 64, "bf16"),
    ([70], 4224, 64, "bf16"),
    ([200, 50], 128, 1088, "bf16"),             # h wider than the LDS, in tall tiles and in short ones
    ([8, 30], 64, 4224, "f32"),
    ([0, 2, 0, 1] * 256, 64, 64, "bf16"),       # the most groups
    ([40] * 70 + [0] * 5, 64, 64, "f32"),
    # enough work for the taller tiles: one to four units, one tile of a group or several; rows resident
    # or through the ring, in either launch
    ([130, 1, 128, 0, 300, 64, 97, 33, 96, 160, 129, 5] * 2, 576, 576, "bf16"),
    ([130, 1, 128, 0, 300, 64, 97, 33, 96, 160, 129, 5] * 2, 1088, 576, "f32"),
    ([70, 128, 31, 200, 0, 160, 257, 65, 96, 40, 100, 150], 128, 1088, "bf16"),
    ([70, 128, 31, 200, 0, 160, 257, 65, 96, 40, 100, 150], 704, 1088, "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("counts,D,I,out", FFN)
def test_grouped_ffn(counts, D, I, out, gathered):
    rng = np.random.default_rng(D + I + len(counts))
    n, N = len(counts), int(sum(counts))
    _, img, val = _weights(rng, n, D, I)
    T = N if not gathered else max(1, N // 2)
    k = 1 if not gathered else -(-N // T)      # T * k bounds the grouped rows
    k = min(k, n)
    T = max(T, -(-N // k))
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16)
    perm = rng.integers(0, T, N).astype(np.int32) if gathered else np.arange(N, dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    d = moe.make_dims(T, D, n, k, I, act="bf16", w="mxfp4", out=out, layout="packed")
    dt = torch.float32 if out == "f32" else torch.bfloat16
    rows = torch.full((T * k, D), 7.0, dtype=dt, device="cuda")
    ws = moe.workspace(d)
    ws.fill_(0xFF)                              # scale bytes left unwritten would be NaN
    moe.moe_grouped_ffn(d, x.cuda(), None, torch.from_numpy(perm).cuda() if gathered else None,
                        torch.from_numpy(offsets).cuda(), *img, None, None, None, rows, ws)
    got = to_np(rows)
    assert (got[N:] == 7.0).all()               # rows behind the last group
    ref, slack = mx.grouped_ffn(to_np(x), perm, offsets, *val)
    _check_rows(got[:N], ref, slack, 2.0 ** -24 if out == "f32" else 2.0 ** -8)


@pytest.mark.gpu
def test_grouped_ffn_keeps_nan_to_its_row_and_expert():
    """A NaN in a token reaches that token's rows only; a NaN weight block reaches that expert's rows only."""
    rng = np.random.default_rng(5)
    counts, D, I = [20, 18, 25], 256, 128
    src, img, _ = _weights(rng, 3, D, I)
    bad = src[0].clone()
    bad[1, 3, 7] = float("nan")
    img_bad = moe.moe_mx_pack_weights(bad.cuda())
    T = sum(counts)
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16)
    x_bad = x.clone()
    x_bad[4, 100] = float("inf")
    offsets = torch.tensor([0, 20, 38, 63], dtype=torch.int32, device="cuda")
    d = moe.make_dims(T, D, 3, 1, I, act="bf16", w="mxfp4", out="bf16", layout="packed")
    ws = moe.workspace(d)
    outs = []
    for xx, wg in ((x, img[0]), (x_bad, img[0]), (x, img_bad)):
        o = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_ffn(d, xx.cuda(), None, None, offsets, wg, img[1], img[2], None, None, None, o, ws)
        outs.append(to_np(o))
    clean, by_x, by_w = outs
    assert np.isnan(by_x[4]).all()
    np.testing.assert_array_equal(np.delete(by_x, 4, 0), np.delete(clean, 4, 0))
    assert np.isnan(by_w[20:38]).all()
    np.testing.assert_array_equal(by_w[:20], clean[:20])
    np.testing.assert_array_equal(by_w[38:], clean[38:])


# ---------------------------------------------------------------------------
# The layer
# ---------------------------------------------------------------------------

LAYERS = [
    # (T, D, E, k, I, I_shared, begin, n_local, given)
    (40, 256, 16, 3, 128, 64, 0, 16, False),
    (300, 448, 24, 4, 192, 128, 0, 24, False),
    (700, 320, 8, 2, 64, 0, 2, 5, True),
    (400, 256, 32, 4, 640, 64, 0, 32, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,E,k,I,Is,begin,nl,given", LAYERS)
def test_layer_forward(T, D, E, k, I, Is, begin, nl, given):
    rng = np.random.default_rng(T)
    bf = lambda a: torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    x, wr = bf(rng.standard_normal((T, D))), bf(rng.standard_normal((E, D)) / np.sqrt(D))
    _, img, val = _weights(rng, nl, D, I)
    sh = [bf(rng.standard_normal(s) / np.sqrt(s[-1])) for s in ((Is, D), (Is, D), (D, Is))] if Is else [None] * 3
    d = moe.make_dims(T, D, E, k, I, Is, begin, nl, True, "bf16", "mxfp4", "f32", "packed")
    w = [None if s is None else moe.moe_pack_weights(s.cuda()) for s in sh]
    wts = moe.make_weights(wr.cuda(), *img, None, None, None, *w)
    packed_in = None
    if given:
        ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
        packed_in = torch.from_numpy(oracle.pack_routing(ids, rng.random((T, k)).astype(np.float32))).cuda()
    y = torch.empty(T, D, dtype=torch.float32, device="cuda")
    blob = torch.empty(T, 2, k, dtype=torch.int32, device="cuda")
    moe.moe_layer_forward(d, wts, x.cuda(), packed_in, None, y, None, blob, moe.workspace(d))
    ids, wt = oracle.unpack_routing(blob.cpu().numpy())
    x64 = to_np(x)
    ref, lim = np.zeros((T, D)), np.zeros((T, D))
    for e in range(nl):
        t, j = np.nonzero(ids == begin + e)
        rows, slack = mx.grouped_ffn(x64, t, [0, len(t)], *(v[e:e + 1] for v in val))
        np.add.at(ref, t, wt[t, j][:, None] * rows)
        np.add.at(lim, t, wt[t, j][:, None] * slack)
    if Is:
        g, u, dn = (to_np(s) for s in sh)
        h = mx.silu(x64 @ g.T) * (x64 @ u.T)
        ref += h @ dn.T
        lim += 2.0 ** -8 * (np.abs(h) @ np.abs(dn).T)       # the shared h is stored in bf16
    lim += 1e-4 * np.abs(ref).max(1, keepdims=True)
    assert (np.abs(to_np(y) - ref) <= lim).all(), float((np.abs(to_np(y) - ref) - lim).max())


@pytest.mark.gpu
def test_layer_captured_and_without_a_workspace():
    """The layer captured and replayed, with eager calls between, and on the library's own scratch: the same bits."""
    rng = np.random.default_rng(3)
    D, E, k, I, Is = 256, 16, 3, 128, 64
    bf = lambda *s: torch.from_numpy((rng.standard_normal(s) / np.sqrt(s[-1])).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    _, img, _ = _weights(rng, E, D, I)
    keep = [bf(E, D).cuda(), *img, *[moe.moe_pack_weights(bf(*s).cuda()) for s in ((Is, D), (Is, D), (D, Is))]]
    wts = moe.make_weights(*keep[:4], None, None, None, *keep[4:])
    for T in (1, 30, 300):
        d = moe.make_dims(T, D, E, k, I, Is, 0, E, True, "bf16", "mxfp4", "bf16", "packed")
        xs = [bf(T, D).cuda() for _ in range(3)]
        ws = moe.workspace(d)
        x, y, y2 = (torch.empty_like(xs[0]) for _ in range(3))
        want = []
        for v in xs:
            moe.moe_layer_forward(d, wts, v, None, None, y, ws=ws)
            want.append(y.clone())
            moe.moe_layer_forward_noalloc(d, wts, v, None, None, y2)
            assert torch.equal(y2, y)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        moe.moe_layer_forward(d, wts, xs[1], None, None, y2, ws=ws, stream=side)
        side.synchronize()
        assert torch.equal(y2, want[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_layer_forward(d, wts, x, None, None, y, ws=ws)
        for i in (0, 2, 1, 0):
            x.copy_(xs[i])
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[i])
            moe.moe_layer_forward(d, wts, xs[(i + 1) % 3], None, None, y2, ws=ws)
            assert torch.equal(y2, want[(i + 1) % 3])


@pytest.mark.gpu
def test_rows_behind_four_gigabytes():
    """Grouped rows whose fp32 results pass 4 GiB: the last rows equal those of a small call on the same tokens."""
    D, I, T = 8192, 64, 140000
    g = torch.Generator(device="cuda").manual_seed(2)
    mats = [torch.randn(s, generator=g, device="cuda") / s[-1] ** 0.5 for s in ((1, I, D), (1, I, D), (1, D, I))]
    img = [moe.moe_mx_pack_weights(m) for m in mats]
    x = torch.randn(T, D, generator=g, device="cuda", dtype=torch.bfloat16)
    res = []
    for n in (T, 200):
        d = moe.make_dims(n, D, 1, 1, I, act="bf16", w="mxfp4", out="f32", layout="packed")
        out = torch.empty(n, D, device="cuda")
        offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        moe.moe_grouped_ffn(d, x[T - n:], None, None, offsets, *img, None, None, None, out, moe.workspace(d))
        res.append(out[-200:].clone())
        del out
    assert torch.equal(res[0], res[1]) and res[0].abs().max() > 0.1
