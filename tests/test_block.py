"""Leaving and entering blocks (moe_block_norm) and a whole block (moe_block_forward), against float64.

Bar of the norm: half a step of the output type per value (2^-8 bf16, 2^-24 fp32) of its magnitude, plus fp32
arithmetic: 16 roundings of 2^-24 of the magnitudes that are added, and the mean square's own error (a sum of D
squares in D / 256 serial steps and a tree, below 2^-24 * (D / 256 + 16) relative, halved by the root).
"""

import ctypes

import numpy as np
import pytest
import torch

import mx_reference as mx
import oracle
import sparse_moe_ffn_route_amd as moe
from harness import to_np
from test_few import Layer

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def test_block_norm_argument_checks():
    lib = moe.library()
    fake = ctypes.c_void_p(256)

    def call(T=2, D=64, act=moe.BF16, yd=moe.BF16, y=fake, r=fake, r_out=fake, x=fake, **kw):
        n = dict(w_post=None, gate=None, w_next=fake, gate_kind=0, res_scale=1.0, eps=1e-6)
        n.update(kw)
        n = moe.moe_norm(**n)
        return lib.moe_block_norm(T, D, act, yd, ctypes.byref(n), y, r, r_out, x, None)

    assert call(T=0) == moe.OK
    assert call(T=-1) == moe.ERR_BAD_DIMS
    assert call(D=0) == moe.ERR_BAD_DIMS
    assert call(D=16385) == moe.ERR_UNSUPPORTED
    assert call(act=moe.E4M3) == moe.ERR_UNSUPPORTED
    assert call(act=moe.F32, yd=moe.BF16) == moe.ERR_UNSUPPORTED
    assert call(gate_kind=4, gate=fake) == moe.ERR_BAD_DIMS
    assert call(eps=-1.0) == moe.ERR_BAD_DIMS
    assert call(eps=float("nan")) == moe.ERR_BAD_DIMS
    assert call(gate_kind=1) == moe.ERR_NULL_ARG                      # a kind without a gate, a gate without a kind
    assert call(gate=fake) == moe.ERR_NULL_ARG
    assert call(r=None) == moe.ERR_NULL_ARG
    assert call(r_out=None) == moe.ERR_NULL_ARG                       # leaving without a place for the stream
    assert call(y=None) == moe.ERR_NULL_ARG                           # entering writes no r_out
    assert call(x=None) == moe.ERR_NULL_ARG
    assert call(w_next=None) == moe.ERR_NULL_ARG
    assert call(y=None, r_out=None, w_next=None, x=None) == moe.ERR_NULL_ARG   # nothing to do
    assert lib.moe_block_norm(2, 64, moe.BF16, moe.BF16, None, fake, fake, fake, fake, None) == moe.ERR_NULL_ARG


def test_block_norm_binding_checks():
    r = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="w_next"):
        moe.moe_block_norm(None, r, w_next=w.float(), x_next=r)
    with pytest.raises(ValueError, match="gate_kind"):
        moe.moe_block_norm(r, r, r, gate=w)
    with pytest.raises(ValueError, match="token gate"):
        moe.moe_block_norm(r, r, r, gate=w, gate_kind="token")
    with pytest.raises(ValueError, match="w_post"):
        moe.moe_block_norm(r, r, r, w_post=w[:32])
    with pytest.raises(ValueError, match="r_out"):
        moe.moe_block_norm(r, r, r[:2])
    with pytest.raises(ValueError, match="y"):
        moe.moe_block_norm(r[:2], r, r)


def test_block_forward_argument_checks():
    lib = moe.library()
    fake = ctypes.c_void_p(256)
    d = moe.make_dims(8, 64, 8, 2, 64)
    w = moe.moe_weights(fake, fake, fake, fake, None, None, None, None, None, None)
    n = moe.moe_norm(None, None, None, 0, 1.0, 1e-6)
    need = lib.moe_block_workspace_bytes(ctypes.byref(d))
    assert need >= moe.moe_workspace_bytes(d) + 2 * 8 * 64 * 2

    def call(d=d, w=w, w_in=fake, x_in=None, n=n, r=fake, r_out=fake, x_next=None, ws=fake, nb=need):
        return lib.moe_block_forward(ctypes.byref(d), ctypes.byref(w), w_in, x_in, None, ctypes.byref(n) if n else None,
                                     r, r_out, x_next, ws, nb, None)

    assert call(d=moe.make_dims(0, 64, 8, 2, 64)) == moe.OK
    assert call(x_in=fake) == moe.ERR_NULL_ARG                        # both
    assert call(w_in=None) == moe.ERR_NULL_ARG                        # neither
    assert call(n=None) == moe.ERR_NULL_ARG
    assert call(r=None) == moe.ERR_NULL_ARG
    assert call(r_out=None) == moe.ERR_NULL_ARG
    assert call(x_next=fake) == moe.ERR_NULL_ARG                      # no w_next
    assert call(nb=need - 1) == moe.ERR_WORKSPACE
    assert call(w=moe.moe_weights(None, fake, fake, fake, None, None, None, None, None, None)) == moe.ERR_NULL_ARG
    assert call(d=moe.make_dims(8, 96, 8, 2, 64)) == moe.ERR_UNSUPPORTED
    wide = moe.make_dims(8, 32768, 8, 2, 64)
    assert call(d=wide, nb=lib.moe_block_workspace_bytes(ctypes.byref(wide))) == moe.ERR_UNSUPPORTED
    assert lib.moe_block_workspace_bytes(ctypes.byref(moe.make_dims(8, 96, 8, 2, 64))) == 0


# ---------------------------------------------------------------------------
# The norm
# ---------------------------------------------------------------------------

def _rms(v, w, eps):
    return v / np.sqrt((v * v).mean(1, keepdims=True) + eps) * w


def _reference(y, r, w_post, gate, kind, scale, eps, w_next):
    """(r_out, its fp32 error, x_next, its fp32 error)."""
    u = 2.0 ** -24
    out, err = r, 0.0 * r
    if y is not None:
        z = y if w_post is None else _rms(y, w_post, eps)
        g = {"none": 1.0, "token": None if gate is None else gate.reshape(-1, 1), "channel": gate, "full": gate}[kind]
        z = z * g
        out = scale * r + z
        err = u * (16 + r.shape[1] / 256 + 16) * (np.abs(scale * r) + np.abs(z))
    x = err_x = None
    if w_next is not None:
        x = _rms(out, w_next, eps)
        inv = 1 / np.sqrt((out * out).mean(1, keepdims=True) + eps)
        # the mean square moves by twice the relative error of out in the mean
        shift = np.sqrt((err * err).mean(1, keepdims=True)) * inv
        err_x = err * inv * np.abs(w_next) + np.abs(x) * (shift + u * (32 + r.shape[1] / 256))
    return out, err, x, err_x


NORMS = [
    # (T, D, gate, post, next, leave)
    (1, 1, "none", False, True, True),
    (1, 4096, "channel", True, True, True),
    (3, 8, "token", True, True, True),
    (5, 705, "full", True, True, True),          # odd width: single values
    (2, 2048, "full", False, True, True),
    (7, 2056, "token", True, False, True),       # just past one sweep of 256 threads
    (4, 16384, "channel", True, True, True),
    (2, 16383, "full", True, True, True),
    (33, 320, "none", False, True, False),       # only entering
    (300, 64, "none", True, False, True),
    (2, 8200, "none", True, True, True),
    (3, 3001, "channel", True, True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("act,yd", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,D,gate,post,nxt,leave", NORMS)
def test_block_norm(T, D, gate, post, nxt, leave, act, yd):
    rng = np.random.default_rng(D + T)
    put = lambda a, dt: torch.from_numpy(np.asarray(a, np.float32)).to(dt).cuda()  # noqa: E731
    r = put(rng.standard_normal((T, D)) * 3, DT[act])
    y = put(rng.standard_normal((T, D)) * 0.5, DT[yd]) if leave else None
    wp = put(1 + 0.2 * rng.standard_normal(D), DT[act]) if post and leave else None
    wn = put(1 + 0.2 * rng.standard_normal(D), DT[act]) if nxt else None
    shape = {"none": None, "token": (T,), "channel": (D,), "full": (T, D)}[gate]
    g = None if shape is None else put(rng.standard_normal(shape), torch.float32 if gate == "token" else DT[act])
    r_out = torch.full((T + 1, D), 5.0, dtype=DT[act], device="cuda") if leave else None
    x = torch.full((T + 1, D), 5.0, dtype=DT[act], device="cuda") if nxt else None
    moe.moe_block_norm(y, r, r_out, wp, g, gate, 0.875, 1e-5, wn, x)
    n64 = lambda t: None if t is None else to_np(t)  # noqa: E731
    out, err, xx, err_x = _reference(n64(y), n64(r), n64(wp), n64(g), gate, 0.875, 1e-5, n64(wn))
    if leave:
        assert (np.abs(to_np(r_out)[:T] - out) <= HALF[act] * np.abs(out) + 2 * err).all()
        assert (r_out[T] == 5.0).all()
    if nxt:
        assert (np.abs(to_np(x)[:T] - xx) <= HALF[act] * np.abs(xx) + 2 * err_x).all()
        assert (x[T] == 5.0).all()
    if leave:                                     # in place, the same bits
        r2 = r.clone()
        moe.moe_block_norm(y, r2, r2, wp, g, gate, 0.875, 1e-5, wn, x)
        assert torch.equal(r2, r_out[:T])


@pytest.mark.gpu
def test_block_norm_unaligned_rows_and_non_finite_values():
    """Tensors off a 16-byte boundary give the same values; a zero row with eps stays zero; NaN stays in its row."""
    rng = np.random.default_rng(1)
    T, D = 6, 264
    base = torch.from_numpy(rng.standard_normal(T * D * 2 + 8).astype(np.float32)).to(torch.bfloat16).cuda()
    off_r, off_y = base[1:1 + T * D].view(T, D), base[T * D + 3:2 * T * D + 3].view(T, D)
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    res = []
    for r, y in ((off_r, off_y), (off_r.clone(), off_y.clone())):
        r_out, x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_norm(y, r, r_out, w_post=w, w_next=w, x_next=x)
        res.append((to_np(r_out), to_np(x)))
    for a, b in zip(*res):                        # another order of the sum of squares: at most one bf16 step apart
        np.testing.assert_allclose(a, b, rtol=2.0 ** -7, atol=1e-6)
    r, y = off_r.clone(), off_y.clone()
    y[2], r[2] = 0.0, 0.0
    y[4, 7] = float("nan")
    r_out, x = torch.empty_like(r), torch.empty_like(r)
    moe.moe_block_norm(y, r, r_out, w_post=w, w_next=w, x_next=x)
    assert (to_np(r_out)[2] == 0).all() and (to_np(x)[2] == 0).all()
    assert np.isnan(to_np(r_out)[4]).all() and np.isnan(to_np(x)[4]).all()
    for t in (0, 1, 3, 5):
        np.testing.assert_array_equal(to_np(x)[t], res[1][1][t])


# ---------------------------------------------------------------------------
# Blocks
# ---------------------------------------------------------------------------

def _block_reference(layer, r, w_in, x_in, w_post, gate, kind, scale, eps, w_next, k, act, quantised):
    x = x_in if x_in is not None else _rms(r, w_in, eps)
    x = to_np(torch.from_numpy(x).to(DT[act]))
    ids, wt = oracle.route((x @ to_np(layer.router).T).astype(np.float32), k)
    y = layer.reference(mx.quantise(x) if quantised else x, ids, wt, 0)
    return _reference(y, r, w_post, gate, kind, scale, eps, w_next)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 16, 17, 90])
@pytest.mark.parametrize("w", ["f32", "bf16"])
def test_two_blocks_in_a_row(T, w):
    """Two blocks chained through x_next, as a model runs them, against float64.

    Bar, relative to the largest value: per block the layer's y within 1e-2 (bf16) or 1e-4 (fp32) of its largest
    value, which the post-norm and a gate of at most 0.5 carry into r; norms divide by an rms near one.  The second
    block's x differs from the reference's by the first's error, and so does its y: twice the bar.
    """
    rng = np.random.default_rng(T)
    D, E, k, I, Is = 256, 16, 3, 128, 64
    tol = 1e-4 if w == "f32" else 1e-2
    layers = [Layer(rng, D, E, E, I, Is, w) for _ in range(2)]
    dt = layers[0].f
    put = lambda a: torch.from_numpy(np.asarray(a, np.float32)).to(dt)  # noqa: E731
    r = put(rng.standard_normal((T, D)))
    ws = [put(1 + 0.1 * rng.standard_normal(D)) for _ in range(5)]
    gate = put(rng.uniform(-0.5, 0.5, D))
    d = moe.make_dims(T, D, E, k, I, Is, 0, E, True, w, w, w, "packed")
    scratch = moe.block_workspace(d)
    cu = [v.cuda() for v in ws]
    r1, x1, r2 = (torch.empty(T, D, dtype=dt, device="cuda") for _ in range(3))
    moe.moe_block_forward(d, layers[0].on_gpu(True), r.cuda(), r1, w_in=cu[0], w_post=cu[1], gate=gate.cuda(),
                          gate_kind="channel", res_scale=0.75, w_next=cu[2], x_next=x1, ws=scratch)
    moe.moe_block_forward(d, layers[1].on_gpu(True), r1, r2, x_in=x1, w_post=cu[3], gate=gate.cuda(),
                          gate_kind="channel", res_scale=0.75, ws=scratch)
    n = [to_np(v) for v in ws]
    out, _, xx, _ = _block_reference(layers[0], to_np(r), n[0], None, n[1], to_np(gate), "channel", 0.75, 1e-6, n[2],
                                     k, w, False)
    big = lambda a, b: np.abs(a - b).max() / np.abs(b).max()  # noqa: E731
    assert big(to_np(r1), out) <= tol and big(to_np(x1), xx) <= 2 * tol
    # the second block on what the first one really gave
    out2, _, _, _ = _block_reference(layers[1], to_np(r1), None, to_np(x1), n[3], to_np(gate), "channel", 0.75, 1e-6,
                                     None, k, w, False)
    assert big(to_np(r2), out2) <= tol


@pytest.mark.gpu
def test_block_forward_is_its_three_calls():
    """With 4-bit experts, on both sides of the few-token limit: the block equals its calls made one by one."""
    rng = np.random.default_rng(3)
    D, E, k, I, Is = 320, 12, 3, 192, 64
    layer = Layer(rng, D, E, E, I, Is, "mxfp4")
    wts = layer.on_gpu(True)
    wi = torch.randn(D).to(torch.bfloat16).cuda()
    for T in (2, 16, 17, 200):
        r = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16).cuda()
        d = moe.make_dims(T, D, E, k, I, Is, 0, E, True, "bf16", "mxfp4", "bf16", "packed")
        r1, x1 = torch.empty_like(r), torch.empty_like(r)
        moe.moe_block_forward(d, wts, r, r1, w_in=wi, w_post=wi, res_scale=0.5, w_next=wi, x_next=x1,
                              ws=moe.block_workspace(d))
        x, y, r2, x2 = (torch.empty_like(r) for _ in range(4))
        moe.moe_block_norm(None, r, w_next=wi, x_next=x)
        call = moe.moe_layer_forward_few if T <= moe.FEW_MAX_T else moe.moe_layer_forward
        call(d, wts, x, None, None, y, ws=moe.workspace(d))
        moe.moe_block_norm(y, r, r2, w_post=wi, res_scale=0.5, w_next=wi, x_next=x2)
        assert torch.equal(r1, r2) and torch.equal(x1, x2)


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,E,k,w,off", [(1, 64, 4, 1, "bf16", 0), (16, 4160, 70, 3, "bf16", 0), (7, 8192, 5, 2, "f32", 0),
                                           (16, 2048, 600, 4, "f32", 0), (3, 320, 12, 3, "bf16", 1), (3, 320, 12, 3, "f32", 1)])
def test_entering_inside_the_layer(T, D, E, k, w, off):
    """Few tokens enter in the layer's first launch (or, off a 16-byte boundary, before it): the same bits as the
    three calls, in place as well."""
    rng = np.random.default_rng(D)
    layer = Layer(rng, D, E, E, 64, 0, w)
    wts = layer.on_gpu(True)
    flat = torch.from_numpy(rng.standard_normal(T * D + 8).astype(np.float32)).to(layer.f).cuda()
    r = flat[off:off + T * D].view(T, D)
    wi = torch.from_numpy((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)).to(layer.f).cuda()
    d = moe.make_dims(T, D, E, k, 64, 0, 0, E, True, w, w, w, "packed")
    r1, x1 = torch.empty(T, D, dtype=layer.f, device="cuda"), torch.empty(T, D, dtype=layer.f, device="cuda")
    moe.moe_block_forward(d, wts, r, r1, w_in=wi, w_post=wi, eps=1e-3, w_next=wi, x_next=x1, ws=moe.block_workspace(d))
    x, y, r2, x2 = (torch.empty_like(r1) for _ in range(4))
    moe.moe_block_norm(None, r, w_next=wi, x_next=x, eps=1e-3)
    moe.moe_layer_forward_few(d, wts, x, None, None, y, ws=moe.workspace(d))
    moe.moe_block_norm(y, r, r2, w_post=wi, w_next=wi, x_next=x2, eps=1e-3)
    assert torch.equal(r1, r2) and torch.equal(x1, x2)
    moe.moe_block_forward(d, wts, r, r, w_in=wi, w_post=wi, eps=1e-3, ws=moe.block_workspace(d))
    assert torch.equal(r, r2)


@pytest.mark.gpu
def test_block_captured_and_replayed():
    rng = np.random.default_rng(7)
    D, E, k, I = 128, 8, 2, 64
    layer = Layer(rng, D, E, E, I, 64, "bf16")
    wts = layer.on_gpu(True)
    wi = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    for T in (3, 40):
        rs = [torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(3)]
        d = moe.make_dims(T, D, E, k, I, 64, 0, E, True, "bf16", "bf16", "bf16", "packed")
        ws = moe.block_workspace(d)
        r, out, x = (torch.empty_like(rs[0]) for _ in range(3))
        want = []
        for v in rs:
            moe.moe_block_forward(d, wts, v, out, w_in=wi, w_next=wi, x_next=x, ws=ws)
            want.append((out.clone(), x.clone()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_block_forward(d, wts, r, out, w_in=wi, w_next=wi, x_next=x, ws=ws)
        for i in (0, 1, 2, 0):
            r.copy_(rs[i])
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[i][0]) and torch.equal(x, want[i][1])
            o2, x2 = torch.empty_like(out), torch.empty_like(x)
            moe.moe_block_forward(d, wts, rs[(i + 1) % 3], o2, w_in=wi, w_next=wi, x_next=x2, ws=ws)
            assert torch.equal(o2, want[(i + 1) % 3][0])
