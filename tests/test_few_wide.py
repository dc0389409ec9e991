"""The few-token layer where its parts do not fit the LDS, and how many bits of h it keeps.

Widths: x of 16 tokens as 4-bit terms takes 2 * 16 * (D + 16 + D / 32) bytes, 270848 at D 8192, where a
workgroup has 152792 beside its routing: the terms go through memory, made by a launch of their own where the logits' launch did not
make them (routing given, or the norm entered there).
"""

import numpy as np
import pytest
import torch

import mx_reference as mx
import oracle
import sparse_moe_ffn_route_amd as moe
from harness import rel_err, to_np
from test_few import Layer, _run


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["mxfp4", "bf16", "e4m3"])
@pytest.mark.parametrize("T,D,Is", [(16, 8192, 0), (16, 8192, 128), (10, 8256, 64)])
def test_given_routing_past_the_lds(T, D, Is, w):
    """Bar as in test_few.py."""
    rng = np.random.default_rng(D + Is)
    E, k, I = 5, 3, 64
    layer = Layer(rng, D, E, E, I, Is, w)
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    wt = rng.random((T, k)).astype(np.float32)
    blob = torch.from_numpy(oracle.pack_routing(ids, wt)).cuda()
    y, _, _, ws = _run(layer, x.cuda(), True, T, D, E, k, I, Is, 0, E, True, "f32", blob)
    assert int(moe.workspace_error_count(ws).cpu()[0]) == 0
    assert rel_err(to_np(y), layer.reference(to_np(x), ids, wt.astype(np.float64), 0)) <= 1e-4 + 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,E,Is", [(16, 8192, 20, 0), (16, 8192, 6, 64), (9, 16384, 4, 128)])
def test_a_wide_block_of_narrow_weights_is_its_three_calls(T, D, E, Is):
    rng = np.random.default_rng(T + E)
    layer = Layer(rng, D, E, E, 64, Is, "mxfp4")
    wts = layer.on_gpu(True)
    r = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    wi = torch.from_numpy((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)).to(torch.bfloat16).cuda()
    d = moe.make_dims(T, D, E, 3, 64, Is, 0, E, True, "bf16", "mxfp4", "bf16", "packed")
    r1, x1 = torch.empty_like(r), torch.empty_like(r)
    moe.moe_block_forward(d, wts, r, r1, w_in=wi, w_post=wi, w_next=wi, x_next=x1, ws=moe.block_workspace(d))
    x, y, r2, x2 = (torch.empty_like(r) for _ in range(4))
    moe.moe_block_norm(None, r, w_next=wi, x_next=x)
    blob = torch.empty(T, 2, 3, dtype=torch.int32, device="cuda")
    moe.moe_layer_forward_few(d, wts, x, None, None, y, None, blob, moe.workspace(d))
    moe.moe_block_norm(y, r, r2, w_post=wi, w_next=wi, x_next=x2)
    assert torch.equal(r1, r2) and torch.equal(x1, x2)
    given = torch.empty_like(y)                                # and the layer call with that routing given
    moe.moe_layer_forward_few(d, wts, x, blob, None, given, ws=moe.workspace(d))
    assert torch.equal(given, y)
    ids, wt = oracle.unpack_routing(blob.cpu().numpy())
    assert rel_err(to_np(y), layer.reference(to_np(x), ids, wt.astype(np.float64), 0)) <= 1e-4 + 2.0 ** -8


# ---------------------------------------------------------------------------
# How many bits of h are kept
# ---------------------------------------------------------------------------

T, D, I, CH = 16, 64, 64, 37


def _terms(h, n):
    """h as the sum of n e4m3 terms, each 2^5 finer than the one before, the first at 2^(floor(log2 |h|) - 7)."""
    unit = np.exp2(np.floor(np.log2(np.abs(h))) - 7)
    rest, total = h / unit, np.zeros_like(h)
    for i in range(n):
        t = torch.from_numpy(rest).to(torch.float8_e4m3fn).double().numpy()
        total += t * 2.0 ** (-5 * i)
        rest = (rest - t) * 32
    return total * unit


def _one_channel():
    """Two experts with one channel that is not zero; x whose gate there is 16: (layer, x, ids, weights)."""
    rng = np.random.default_rng(40)
    gate, up, down = np.zeros((2, I, D)), np.zeros((2, I, D)), np.zeros((2, D, I))
    gate[:, CH, 0], up[:, CH, 1] = 4.0, 1.0
    down[:, :, CH] = rng.choice([-6.0, -3.0, -1.0, 0.5, 1.5, 2.0, 4.0], (2, D))
    x = rng.standard_normal((T, D))
    x[:, 0], x[:, 1] = 4.0, rng.choice([-1, 1], T) * rng.uniform(1, 2, T)
    ids = (np.arange(T) % 2).astype(np.int32)[:, None]
    return (gate, up, down), torch.from_numpy(x).to(torch.bfloat16), ids, rng.uniform(0.1, 1, (T, 1)).astype(np.float32)


def _h(x, wt):
    return wt[:, 0].astype(np.float64) * mx.silu(16.0) * to_np(x)[:, 1]


# h to 2^-17 of itself; twenty roundings of 2^-24 at most in g, u, silu, the products with the weight and the
# scales and the sums (each of one product that is not zero), 2^-19 in all
BITS = 2.0 ** -17 + 2.0 ** -19


def test_a_lost_term_of_h_is_seen():
    _, x, _, wt = _one_channel()
    h = _h(x, wt)
    assert np.abs(_terms(h, 4) / h - 1).max() <= 2.0 ** -17
    assert np.abs(_terms(h, 3) / h - 1).max() > 2 * BITS
    assert np.abs(torch.from_numpy(h).to(torch.bfloat16).double().numpy() / h - 1).max() > 2 * BITS


@pytest.mark.gpu
@pytest.mark.parametrize("w,packed", [("mxfp4", True), ("bf16", True), ("bf16", False), ("e4m3", True), ("e4m3", False),
                                      ("f32", True)])
def test_h_keeps_sixteen_bits(w, packed):
    mats, x, ids, wt = _one_channel()
    layer = Layer(np.random.default_rng(0), D, 2, 2, I, 0, w)
    kind = {"mxfp4": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "f32": torch.float32}[w]
    layer.routed = [torch.from_numpy(m).to(kind) for m in mats]           # exact in every type
    layer.scales = [torch.ones(m.shape[:2]) if w == "e4m3" else None for m in mats]
    for m, t in zip(mats, layer.routed):
        np.testing.assert_array_equal(mx.quantise(m) if w == "mxfp4" else to_np(t), m)
    blob = torch.from_numpy(oracle.pack_routing(ids, wt)).cuda()
    y, _, _, _ = _run(layer, x.to(layer.f).cuda(), packed, T, D, 2, 1, I, 0, 0, 2, True, "f32", blob)
    ref = _h(x, wt)[:, None] * mats[2][ids[:, 0], :, CH]
    assert (np.abs(to_np(y) - ref) <= BITS * np.abs(ref)).all(), float(np.abs(to_np(y) / ref - 1).max())
