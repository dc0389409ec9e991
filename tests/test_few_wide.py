"""The few-token layer where its parts do not fit the LDS.

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
