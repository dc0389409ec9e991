"""Routing and grouping of more tokens than one grid dimension holds threads for (a launch of more runs in part, without an error)."""

import pytest
import torch

import sparse_moe_ffn_route_amd as moe

pytestmark = pytest.mark.gpu
STEP = 1 << 22


def gpu(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def grouped(T, k, E, dtype, D=64):
    """moe_permute of whole-number tokens with a cheap routing: counts, offsets, perm_token, inv_pos and the rows."""
    d = moe.make_dims(T, D, E, k, 64, w=dtype)
    ids = torch.arange(T, device="cuda").mul_(7).remainder_(E)
    packed = gpu(T, 2, k).zero_()
    for j in range(k):
        packed[:, 0, j] = (ids + j) % E
    del ids
    x = gpu(T, D, dtype=torch.bfloat16).random_(-8, 9)
    counts, offsets, perm, inv = gpu(E), gpu(E + 1), gpu(T * k), gpu(T, k)
    x_perm = gpu(T * k, D, dtype=torch.bfloat16 if dtype == "bf16" else torch.uint8).fill_(77)
    scale = None if dtype == "bf16" else gpu(T * k, dtype=torch.float32).fill_(77)
    moe.moe_permute(d, packed, counts, offsets, perm, inv, x, x_perm, scale, ws=moe.workspace(d))
    for j in range(k):
        for t in range(0, T, STEP):
            at = inv[t:t + STEP, j].long()
            assert torch.equal(perm[at].long(), torch.arange(t, min(T, t + STEP), device="cuda"))
            of = torch.bucketize(at, offsets[1:].long(), right=True)
            assert torch.equal(of.int(), packed[t:t + STEP, 0, j])
    return x, perm, x_perm, scale


@pytest.mark.parametrize("T,k", [((1 << 24) + 5, 1), ((1 << 23) + 7, 2), ((1 << 22) - 1, 5)])
def test_every_row_is_gathered(T, k):
    x, perm, x_perm, _ = grouped(T, k, 5, "bf16")
    for r in range(0, T * k, STEP):
        assert torch.equal(x_perm[r:r + STEP], x[perm[r:r + STEP].long()]), r
    del x, perm, x_perm
    torch.cuda.empty_cache()


def test_every_token_is_quantised():
    """2^26 tokens and more to e4m3: scale = amax / 448 exactly; values within half a step, 2^-4 of the value (and a
    thousandth of that for the fp32 roundings of the division and of this test) or, of the smallest, 2^-10 (twice that)."""
    T = (1 << 26) + 5
    x, perm, x_perm, scale = grouped(T, 1, 3, "e4m3")
    for r in range(0, T, STEP):
        v = x[perm[r:r + STEP].long()].float()
        amax = v.abs().amax(1)
        s = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, 448))
        assert torch.equal(scale[r:r + STEP], s), r
        got = x_perm[r:r + STEP].view(torch.float8_e4m3fn).float() * s[:, None]
        assert ((got - v).abs() <= v.abs() * 2.0 ** -4 * 1.001 + s[:, None] * 2.0 ** -9).all(), r
    del x, perm, x_perm, scale
    torch.cuda.empty_cache()


def test_every_token_is_routed():
    T, E, k = (1 << 26) + 5, 4, 2
    d = moe.make_dims(T, 64, E, k, 64)
    logits, packed = gpu(T, E, dtype=torch.float32).normal_(), gpu(T, 2, k).fill_(-7)
    moe.moe_route(d, None, None, logits, None, packed)
    for t in range(0, T, STEP):
        top, ids = logits[t:t + STEP].sort(dim=1, descending=True, stable=True)
        assert torch.equal(packed[t:t + STEP, 0], ids[:, :k].int()), t
        w = packed[t:t + STEP, 1].contiguous().view(torch.float32)
        assert (w - torch.softmax(top[:, :k], 1)).abs().max() <= 16 * 2.0 ** -24, t
    del logits, packed, top, ids, w
    torch.cuda.empty_cache()
