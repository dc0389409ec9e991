"""The MoE layer for up to 16 tokens, for every weight type and layout, against the fp64 oracle.

Bar: max |y - ref| <= (half a step of the output type + 1e-4) * max |ref|: one rounding of y (2^-8 bf16) and the
fp32 sums at the fp32 layer's bar; weights are exact in the products and h keeps 16 bits or more (2^-17 of a
term), which the 1e-4 covers.  Routing ids are exact on the kernel's own logits.
"""

import ctypes

import numpy as np
import pytest
import torch

import mx_reference as mx
import oracle
import sparse_moe_ffn_route_amd as moe
from harness import logit_bound, rel_err, to_np


def _dims(**kw):
    base = dict(T=8, D=64, E=8, top_k=2, I=64, act="bf16", w="bf16", out="bf16", layout="packed")
    base.update(kw)
    return moe.make_dims(**base)


def test_argument_checks():
    lib = moe.library()
    fake = ctypes.c_void_p(256)
    w = moe.moe_weights(fake, fake, fake, fake, None, None, None, None, None, None)

    def call(d, x=fake, packed=None, y=fake, ws=fake, n=1 << 30, w=w):
        return lib.moe_layer_forward_few(ctypes.byref(d), ctypes.byref(w) if w else None, x, packed, None, y, None,
                                         None, ws, n, None)

    assert call(_dims(T=moe.FEW_MAX_T + 1)) == moe.ERR_UNSUPPORTED
    assert call(_dims(T=-1)) == moe.ERR_BAD_DIMS
    assert call(_dims(), x=None) == moe.ERR_NULL_ARG
    assert call(_dims(), y=None) == moe.ERR_NULL_ARG
    assert call(_dims(), ws=None) == moe.ERR_NULL_ARG
    assert call(_dims(), w=None) == moe.ERR_NULL_ARG
    assert call(_dims(w="e4m3")) == moe.ERR_NULL_ARG                       # scales missing
    assert call(_dims(I_shared=64)) == moe.ERR_NULL_ARG                    # shared weights missing
    no_router = moe.moe_weights(None, fake, fake, fake, None, None, None, None, None, None)
    assert call(_dims(), w=no_router) == moe.ERR_NULL_ARG
    assert call(_dims(), n=moe.moe_workspace_bytes(_dims()) - 1) == moe.ERR_WORKSPACE
    assert call(_dims(T=0)) == moe.OK
    off = ctypes.c_void_p(258)
    assert call(_dims(), x=off) == moe.ERR_UNSUPPORTED                     # off a 16-byte boundary
    assert call(_dims(), ws=off) == moe.ERR_UNSUPPORTED
    for i in range(4):
        ptr = [off if i == j else fake for j in range(4)]
        assert call(_dims(), w=moe.moe_weights(*ptr, *[None] * 6)) == moe.ERR_UNSUPPORTED
    with pytest.raises(ValueError, match="x:"):
        moe.moe_layer_forward_few(_dims(), w, torch.zeros(4, 64, dtype=torch.bfloat16), None, None,
                                  torch.zeros(8, 64, dtype=torch.bfloat16))


class Layer:
    """Random weights of one layer: what the library takes (rows or packed) and their fp64 values."""

    def __init__(self, rng, D, E, n, I, Is, w):
        f = torch.float32 if w == "f32" else torch.bfloat16
        draw = lambda *s: torch.from_numpy((rng.standard_normal(s) / np.sqrt(s[-1])).astype(np.float32))  # noqa: E731
        self.w, self.f = w, f
        self.router = draw(E, D).to(f)
        self.routed = [draw(n, I, D), draw(n, I, D), draw(n, D, I)]
        self.shared = [draw(Is, D).to(f), draw(Is, D).to(f), draw(D, Is).to(f)] if Is else None
        self.scales = [None] * 3
        if w == "e4m3":
            amax = [m.abs().amax(-1) for m in self.routed]
            self.scales = [a / 448 for a in amax]
            self.routed = [(m * (448 / a)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
                           for m, a in zip(self.routed, amax)]
            self.values = [to_np(m) * to_np(s)[..., None] for m, s in zip(self.routed, self.scales)]
        elif w == "mxfp4":
            self.values = [mx.quantise(to_np(m)) for m in self.routed]
        else:
            self.routed = [m.to(f) for m in self.routed]
            self.values = [to_np(m) for m in self.routed]

    def on_gpu(self, packed):
        lay = (lambda t: moe.moe_pack_weights(t.cuda())) if packed else (lambda t: t.cuda())
        routed = [moe.moe_mx_pack_weights(m.cuda()) if self.w == "mxfp4" else lay(m) for m in self.routed]
        sh = [lay(m) for m in self.shared] if self.shared else [None] * 3
        self.alive = [self.router.cuda(), *routed, *[None if s is None else s.cuda() for s in self.scales], *sh]
        return moe.make_weights(*self.alive)

    def reference(self, x, ids, wt, begin):
        y = np.zeros_like(x)
        for e in range(len(self.values[0])):
            t, j = np.nonzero(ids == begin + e)
            g, u, d = (v[e] for v in self.values)
            np.add.at(y, t, wt[t, j][:, None] * ((mx.silu(x[t] @ g.T) * (x[t] @ u.T)) @ d.T))
        if self.shared:
            g, u, d = (to_np(m) for m in self.shared)
            y += (mx.silu(x @ g.T) * (x @ u.T)) @ d.T
        return y


CASES = [
    # (T, D, E, k, I, I_shared, begin, n_local, given, renorm)
    (1, 64, 4, 1, 64, 0, 0, 4, False, True),
    (1, 1024, 64, 8, 256, 128, 0, 64, False, True),
    (3, 704, 20, 5, 320, 192, 0, 20, False, False),
    (7, 320, 600, 10, 64, 64, 0, 600, False, True),
    (16, 256, 40, 32, 128, 0, 0, 40, False, True),
    (16, 448, 24, 4, 192, 64, 8, 6, False, True),
    (13, 576, 64, 6, 128, 0, 16, 16, True, True),
    (5, 128, 32, 2, 64, 0, 30, 1, True, True),
    (2, 4160, 8, 2, 64, 64, 0, 8, False, True),
    (16, 8192, 4, 2, 64, 64, 0, 4, False, True),       # x past the LDS
    (16, 4096, 6, 3, 128, 192, 0, 6, True, True),      # x in the LDS as 4-bit terms or not at all
    (11, 2048, 6, 3, 1088, 0, 0, 6, False, True),
]


def _run(layer, x, packed, T, D, E, k, I, Is, begin, nl, renorm, out, blob_in=None, bias=None, ws=None, stream=None):
    act = "f32" if layer.w == "f32" else "bf16"
    d = moe.make_dims(T, D, E, k, I, Is, begin, nl, renorm, act, layer.w, out, "packed" if packed else "rows")
    y = torch.full((T, D), float("nan"), dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    logits = None if blob_in is not None else torch.empty(T, E, dtype=torch.float32, device="cuda")
    blob = torch.empty(T, 2, k, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = moe.workspace(d)
        ws.fill_(0xFF)
    w = layer.on_gpu(packed)
    moe.moe_layer_forward_few(d, w, x, blob_in, bias, y, logits, blob, ws, stream=stream)
    torch.cuda.synchronize()
    return y, logits, blob, ws


@pytest.mark.gpu
@pytest.mark.parametrize("w,packed,out", [("f32", False, "f32"), ("f32", True, "f32"), ("bf16", False, "bf16"),
                                          ("bf16", True, "f32"), ("e4m3", False, "f32"), ("e4m3", True, "bf16"),
                                          ("mxfp4", True, "f32"), ("mxfp4", True, "bf16")])
@pytest.mark.parametrize("case", CASES)
def test_few_matches_the_oracle(case, w, packed, out):
    T, D, E, k, I, Is, begin, nl, given, renorm = case
    rng = np.random.default_rng(T * 31 + D)
    layer = Layer(rng, D, E, nl, I, Is, w)
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(layer.f)
    blob_in = None
    if given:
        ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
        blob_in = torch.from_numpy(oracle.pack_routing(ids, rng.random((T, k)).astype(np.float32))).cuda()
    y, logits, blob, ws = _run(layer, x.cuda(), packed, T, D, E, k, I, Is, begin, nl, renorm, out, blob_in)
    ids, wt = oracle.unpack_routing(blob.cpu().numpy())
    if given:
        np.testing.assert_array_equal(blob.cpu().numpy(), blob_in.cpu().numpy())
    else:
        l_ref = oracle.router_logits(to_np(x), to_np(layer.router)).astype(np.float64)
        assert (np.abs(to_np(logits) - l_ref) <= logit_bound(to_np(x), to_np(layer.router), l_ref)).all()
        ids_ref, w_ref = oracle.route(logits.cpu().numpy(), k, renormalize=renorm)
        np.testing.assert_array_equal(ids, ids_ref)
        np.testing.assert_allclose(wt, w_ref, rtol=0, atol=1e-6)
    assert int(moe.workspace_error_count(ws).cpu()[0]) == 0
    ref = layer.reference(to_np(x), ids, wt.astype(np.float64), begin)
    assert rel_err(to_np(y), ref) <= (2.0 ** -8 if out == "bf16" else 2.0 ** -24) + 1e-4


@pytest.mark.gpu
def test_bias_excludes_experts():
    rng = np.random.default_rng(2)
    layer = Layer(rng, 256, 48, 48, 64, 0, "bf16")
    x = torch.from_numpy(rng.standard_normal((9, 256)).astype(np.float32)).to(torch.bfloat16)
    bias = rng.standard_normal(48).astype(np.float32)
    bias[::3] = -np.inf
    y, logits, blob, _ = _run(layer, x.cuda(), True, 9, 256, 48, 6, 64, 0, 0, 48, True, "f32",
                              bias=torch.from_numpy(bias).cuda())
    ids, wt = oracle.unpack_routing(blob.cpu().numpy())
    ids_ref, _ = oracle.route(logits.cpu().numpy(), 6, bias=bias)
    np.testing.assert_array_equal(ids, ids_ref)
    assert (ids % 3 != 0).all()
    assert rel_err(to_np(y), layer.reference(to_np(x), ids, wt.astype(np.float64), 0)) <= 1e-4 + 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["bf16", "mxfp4"])
def test_given_routing_with_bad_and_repeated_ids(w):
    """Ids outside [0, E) are skipped and counted, a repeated expert is summed, a token with nothing local is 0."""
    rng = np.random.default_rng(4)
    T, D, E, k, I, begin, nl = 6, 192, 12, 4, 128, 3, 5
    layer = Layer(rng, D, E, nl, I, 0, w)
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16)
    ids = np.array([[3, 3, 7, -1], [12, 2 ** 30, -2 ** 31, 4], [0, 1, 2, 8], [5, 6, 5, 5], [7, 6, 5, 4], [9, 10, 11, 3]],
                   dtype=np.int32)
    wt = rng.random((T, k)).astype(np.float32)
    blob = torch.from_numpy(oracle.pack_routing(ids, wt)).cuda()
    y, _, _, ws = _run(layer, x.cuda(), True, T, D, E, k, I, 0, begin, nl, True, "f32", blob)
    assert int(moe.workspace_error_count(ws).cpu()[0]) == 4
    got = to_np(y)
    assert (got[2] == 0).all()
    ref = layer.reference(to_np(x), ids.astype(np.int64), wt.astype(np.float64), begin)
    assert rel_err(got, ref) <= 1e-4 + 2.0 ** -24


@pytest.mark.gpu
def test_non_finite_values_stay_with_their_token_and_expert():
    rng = np.random.default_rng(8)
    T, D, E, k, I = 8, 128, 6, 2, 64
    ids = np.array([[t % E, (t + 1) % E] for t in range(T)], dtype=np.int32)
    blob = torch.from_numpy(oracle.pack_routing(ids, np.full((T, k), 0.5, np.float32))).cuda()
    layer = Layer(rng, D, E, E, I, 64, "bf16")
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16)
    args = (True, T, D, E, k, I, 64, 0, E, True, "bf16", blob)
    clean = to_np(_run(layer, x.cuda(), *args)[0])
    x_bad = x.clone()
    x_bad[3, 5] = float("inf")
    got = to_np(_run(layer, x_bad.cuda(), *args)[0])
    assert not np.isfinite(got[3]).any()
    np.testing.assert_array_equal(np.delete(got, 3, 0), np.delete(clean, 3, 0))
    for m in (0, 2):                                                       # the gate, then the down projection
        layer.routed[m][2, 1, 1] = float("nan")
        got = to_np(_run(layer, x.cuda(), *args)[0])
        hit = (ids == 2).any(1)
        assert np.isnan(got[hit]).any(1).all()
        np.testing.assert_array_equal(got[~hit], clean[~hit])
        layer.routed[m][2, 1, 1] = 0.01


@pytest.mark.gpu
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("w", ["e4m3", "mxfp4"])
def test_non_finite_tokens_on_narrow_weights(w, given):
    """A token with an infinity or a NaN is NaN and changes no other token's row, however many share its experts."""
    rng = np.random.default_rng(18)
    T, D, E, k, I = 16, 704, 4, 2, 192
    layer = Layer(rng, D, E, E, I, 64, w)
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16)
    blob = _run(layer, x.cuda(), True, T, D, E, k, I, 64, 0, E, True, "f32")[2]
    args = (True, T, D, E, k, I, 64, 0, E, True, "f32", blob if given else None)
    clean = to_np(_run(layer, x.cuda(), *args)[0])
    for t, c, v in ((0, 0, "inf"), (9, 703, "nan"), (15, 350, "-inf")):
        bad = x.clone()
        bad[t, c] = float(v)
        got = to_np(_run(layer, bad.cuda(), *args)[0])
        assert not np.isfinite(got[t]).any()
        rest = np.delete(np.arange(T), t)
        # with its own routing the NaN token names other experts, and the order of a sum may change
        if given:
            np.testing.assert_array_equal(got[rest], clean[rest])
        else:
            assert rel_err(got[rest], clean[rest]) <= 2 * (1e-4 + 2.0 ** -24)


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["f32", "bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("Is", [0, 128])
def test_no_token_chose_a_local_expert(w, Is):
    rng = np.random.default_rng(1)
    T, D, E, k, I = 4, 192, 12, 2, 64
    layer = Layer(rng, D, E, 3, I, Is, w)
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(layer.f)
    ids = np.tile(np.array([[0, 11]], np.int32), (T, 1))
    blob = torch.from_numpy(oracle.pack_routing(ids, np.ones((T, k), np.float32))).cuda()
    y, _, _, ws = _run(layer, x.cuda(), True, T, D, E, k, I, Is, 4, 3, True, "f32", blob)
    assert int(moe.workspace_error_count(ws).cpu()[0]) == 0
    if Is:
        ref = layer.reference(to_np(x), ids, np.ones((T, k)), 4)
        assert rel_err(to_np(y), ref) <= 1e-4 + 2.0 ** -24
    else:
        assert (to_np(y) == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["bf16", "mxfp4", "f32"])
def test_streams_graphs_and_repeats(w):
    """The call on another stream, captured and replayed between eager calls on other inputs and the same
    workspace, gives the eager result bit for bit."""
    rng = np.random.default_rng(6)
    T, D, E, k, I, Is = 4, 256, 32, 4, 128, 64
    layer = Layer(rng, D, E, E, I, Is, w)
    xs = [torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(layer.f).cuda() for _ in range(3)]
    act = "f32" if w == "f32" else "bf16"
    d = moe.make_dims(T, D, E, k, I, Is, 0, E, True, act, w, act, "packed")
    wts, ws = layer.on_gpu(True), moe.workspace(d)
    x, y = torch.empty_like(xs[0]), torch.empty_like(xs[0])
    want = []
    for v in xs:
        moe.moe_layer_forward_few(d, wts, v, None, None, y, ws=ws)
        want.append(y.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = torch.empty_like(y)
    moe.moe_layer_forward_few(d, wts, xs[1], None, None, y2, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(y2, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_layer_forward_few(d, wts, x, None, None, y, ws=ws)
    for i in (0, 2, 1, 0):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        moe.moe_layer_forward_few(d, wts, xs[(i + 1) % 3], None, None, y2, ws=ws)
        assert torch.equal(y2, want[(i + 1) % 3])


@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(8, 2), (100, 7), (130, 32), (600, 5), (1024, 32)])
def test_equal_and_nan_logits(E, k):
    """Equal logits keep the lowest ids; tokens with a NaN, with equal and with ordinary logits in one call route as
    the full layer routes them, and the ordinary ones' results stay within the bar (the experts of a call are summed
    in the order in which its tokens name them, so another token's choice may change a sum's order)."""
    rng = np.random.default_rng(E)
    T, D, I = 6, 128, 64
    layer = Layer(rng, D, E, E, I, 0, "bf16")
    layer.router[::2] = layer.router[0]                                    # half of the experts in a tie
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16)
    x[1] = 0                                                               # all of them
    clean, logits, blob, _ = _run(layer, x.cuda(), True, T, D, E, k, I, 0, 0, E, True, "f32")
    ids, wt = oracle.unpack_routing(blob.cpu().numpy())
    np.testing.assert_array_equal(ids, oracle.route(logits.cpu().numpy(), k)[0])
    np.testing.assert_array_equal(ids[1], np.arange(k))
    assert rel_err(to_np(clean), layer.reference(to_np(x), ids, wt.astype(np.float64), 0)) <= 1e-4 + 2.0 ** -24
    x[3, 5] = float("nan")
    got, _, blob, ws = _run(layer, x.cuda(), True, T, D, E, k, I, 0, 0, E, True, "f32")
    rest = [0, 1, 2, 4, 5]
    assert rel_err(to_np(got)[rest], to_np(clean)[rest]) <= 2 * (1e-4 + 2.0 ** -24)
    d = moe.make_dims(T, D, E, k, I, 0, 0, E, True, "bf16", "bf16", "f32", "packed")
    full = torch.empty_like(blob)
    y2 = torch.empty(T, D, device="cuda")
    moe.moe_layer_forward(d, layer.on_gpu(True), x.cuda(), None, None, y2, None, full, moe.workspace(d))
    np.testing.assert_array_equal(blob[:, 0].cpu().numpy(), full[:, 0].cpu().numpy())
    assert np.isnan(to_np(got)[3]).all() == np.isnan(to_np(y2)[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["bf16", "e4m3", "mxfp4"])
def test_two_calls_at_once(w):
    """Two layers on two streams, each with its workspace: both give what they give alone."""
    rng = np.random.default_rng(9)
    shapes = [(7, 256, 32, 4, 128, 64), (16, 512, 24, 3, 192, 0)]
    jobs = []
    for T, D, E, k, I, Is in shapes:
        layer = Layer(rng, D, E, E, I, Is, w)
        x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(layer.f).cuda()
        d = moe.make_dims(T, D, E, k, I, Is, 0, E, True, "bf16", w, "bf16", "packed")
        wts, ws = layer.on_gpu(True), moe.workspace(d)
        y = torch.empty_like(x)
        moe.moe_layer_forward_few(d, wts, x, None, None, y, ws=ws)
        torch.cuda.synchronize()
        jobs.append((layer, d, wts, x, ws, y, torch.cuda.Stream()))
    outs = [[torch.empty_like(j[3]) for _ in range(8)] for j in jobs]
    torch.cuda.synchronize()
    for i in range(8):
        for o, (_, d, wts, x, ws, _, s) in zip(outs, jobs):
            moe.moe_layer_forward_few(d, wts, x, None, None, o[i], ws=ws, stream=s)
    torch.cuda.synchronize()
    for o, j in zip(outs, jobs):
        assert all(torch.equal(v, j[5]) for v in o)


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["bf16", "mxfp4"])
def test_experts_behind_four_gigabytes(w):
    """A call that takes the last of so many experts that their matrices pass 4 GiB, against the same one alone."""
    T, D, I, k = 3, 4096, 2048, 1
    one = moe.moe_mx_weight_bytes(1, I, D) if w == "mxfp4" else I * D * 2
    n = (1 << 32) // one + 2
    g = torch.Generator(device="cuda").manual_seed(1)
    mats = [torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16) / s[-1] ** 0.5
            for s in ((1, I, D), (1, I, D), (1, D, I))]
    pack = moe.moe_mx_pack_weights if w == "mxfp4" else moe.moe_pack_weights
    small = [pack(m).view(torch.uint8).reshape(-1) for m in mats]
    big = [torch.zeros(n * one, dtype=torch.uint8, device="cuda") for _ in small]
    for b, s in zip(big, small):
        b[-one:] = s
    x = torch.randn(T, D, generator=g, device="cuda").to(torch.bfloat16)
    wt = torch.tensor([[0.5], [1.0], [0.25]])
    ys = []
    for count, m in ((n, big), (1, small)):
        ids = np.full((T, 1), count - 1, np.int32)
        blob = torch.from_numpy(oracle.pack_routing(ids, wt.numpy())).cuda()
        d = moe.make_dims(T, D, count, k, I, 0, 0, count, True, "bf16", w, "f32", "packed")
        wts = moe.make_weights(None, *m)
        for call in (moe.moe_layer_forward_few, moe.moe_layer_forward):
            y = torch.empty(T, D, device="cuda")
            call(d, wts, x, blob, None, y, ws=moe.workspace(d))
            ys.append(y)
    assert torch.equal(ys[0], ys[2]) and torch.equal(ys[1], ys[3])
    assert ys[0].abs().max() > 0.1


@pytest.mark.gpu
def test_agrees_with_the_full_layer():
    """Same routing, same experts: moe_layer_forward's y within its own bf16 roundings of h and expert rows."""
    rng = np.random.default_rng(12)
    T, D, E, k, I, Is = 11, 512, 32, 4, 192, 128
    layer = Layer(rng, D, E, E, I, Is, "bf16")
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    y, _, blob, _ = _run(layer, x, True, T, D, E, k, I, Is, 0, E, True, "bf16")
    d = moe.make_dims(T, D, E, k, I, Is, 0, E, True, "bf16", "bf16", "bf16", "packed")
    y2, blob2 = torch.empty_like(y), torch.empty_like(blob)
    moe.moe_layer_forward(d, layer.on_gpu(True), x, None, None, y2, None, blob2, moe.workspace(d))
    np.testing.assert_array_equal(blob[:, 0].cpu().numpy(), blob2[:, 0].cpu().numpy())
    assert rel_err(to_np(y), to_np(y2)) <= 1e-2
