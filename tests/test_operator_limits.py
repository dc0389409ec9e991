"""Limits of the calls beside the full layer: workspaces, refusals before any launch, the largest calls."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_ffn_route_amd as moe
from harness import to_np
from test_few import Layer

WORKSPACES = [
    dict(D=4096, E=512, top_k=10, I=1024, I_shared=1024),
    dict(D=4096, E=512, top_k=10, I=1024, I_shared=1024, w="e4m3"),
    dict(D=4096, E=128, top_k=8, I=1024, I_shared=1024, w="mxfp4", layout="packed"),
    dict(D=1024, E=64, top_k=2, I=4096),                       # h of the few-token layer wider than the rows
    dict(D=256, E=512, top_k=1, I=64),
    dict(D=64, E=8, top_k=8, I=64, I_shared=4096, act="f32", w="f32", out="f32"),
]


@pytest.mark.parametrize("kw", WORKSPACES)
def test_a_workspace_serves_fewer_tokens(kw):
    """One sized for a few more tokens than the few-token layer takes holds every call of its size or less."""
    lib = moe.library()
    dims = {T: moe.make_dims(T, **kw) for T in range(1, 33)}
    for size in (moe.moe_workspace_bytes, lambda d: lib.moe_block_workspace_bytes(ctypes.byref(d))):
        n = [size(dims[T]) for T in range(1, 33)]
        assert n[0] > 0 and n == sorted(n)


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["bf16", "mxfp4"])
def test_calls_on_the_workspace_of_more_tokens(w):
    """Both layer calls on the workspace of one token more than the few-token layer takes, and the block on its own:
    as on one of their size; nothing behind the workspace is written."""
    rng = np.random.default_rng(17)
    D, E, k, I, Is = 64, 16, 8, 256, 192
    layer = Layer(rng, D, E, E, I, Is, w)
    wts = layer.on_gpu(True)
    dims = lambda T: moe.make_dims(T, D, E, k, I, Is, 0, E, True, "bf16", w, "bf16", "packed")  # noqa: E731
    n, nb = moe.moe_workspace_bytes(dims(17)), moe.block_workspace(dims(17)).numel()
    ones = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    for T in (1, 8, 15, 16):
        d, x = dims(T), torch.randn(T, D, device="cuda").to(torch.bfloat16)
        for call, size in ((moe.moe_layer_forward, n), (moe.moe_layer_forward_few, n), (moe.moe_block_forward, nb)):
            got = []
            for bytes_ in (None, size):
                guard = torch.full((bytes_ + 256,), 0xA5, dtype=torch.uint8, device="cuda") if bytes_ else None
                ws = guard[:bytes_] if bytes_ else moe.block_workspace(d)
                y = torch.empty_like(x)
                if call is moe.moe_block_forward:
                    call(d, wts, x, y, w_in=ones, ws=ws)
                else:
                    call(d, wts, x, None, None, y, ws=ws)
                got.append(y)
                assert guard is None or (guard[bytes_:] == 0xA5).all()
            assert torch.equal(*got)
