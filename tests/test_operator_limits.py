"""Limits of the calls beside the full layer: workspaces, refusals before any launch, the largest calls."""

import ctypes

import numpy as np
import pytest
import torch

import sparse_moe_ffn_route_amd as moe
import test_mx
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


# ---------------------------------------------------------------------------
# Nothing is launched by a refused call
# ---------------------------------------------------------------------------

FAKE, OFF = ctypes.c_void_p(256), ctypes.c_void_p(264)


def _layer_weights(off):
    """Router, gate, up and down at 16-byte boundaries but for the one at index `off`."""
    return moe.moe_weights(*[OFF if i == off else FAKE for i in range(4)], *[None] * 6)


def test_the_layer_checks_alignment_before_any_launch():
    lib = moe.library()
    for T in (8, 40):
        d = moe.make_dims(T, 64, 8, 2, 64, act="bf16", w="mxfp4", out="bf16", layout="packed")

        def call(x=FAKE, off=None, ws=FAKE):
            return lib.moe_layer_forward(ctypes.byref(d), ctypes.byref(_layer_weights(off)), x, None, None, FAKE, None,
                                         None, ws, 1 << 30, None, None)

        assert call(x=OFF) == call(ws=OFF) == moe.ERR_UNSUPPORTED
        for i in (1, 2, 3):
            assert call(off=i) == moe.ERR_UNSUPPORTED


def test_the_block_checks_alignment_before_any_launch():
    lib = moe.library()
    n = moe.moe_norm(None, None, None, 0, 1.0, 1e-6)

    def call(T, w, off=None, r=FAKE, x_in=None, ws=FAKE):
        d = moe.make_dims(T, 64, 8, 2, 64, act="bf16", w=w, out="bf16", layout="packed")
        return lib.moe_block_forward(ctypes.byref(d), ctypes.byref(_layer_weights(off)), None if x_in else FAKE, x_in,
                                     None, ctypes.byref(n), r, FAKE, None, ws, 1 << 30, None)

    for T, w in ((8, "bf16"), (8, "mxfp4"), (40, "mxfp4")):
        assert call(T, w, ws=OFF) == moe.ERR_UNSUPPORTED
        assert call(T, w, x_in=OFF) == moe.ERR_UNSUPPORTED
        for i in range(0 if T == 8 else 1, 4):
            assert call(T, w, off=i) == moe.ERR_UNSUPPORTED
            assert call(T, w, off=i, r=OFF) == moe.ERR_UNSUPPORTED       # r off a boundary: entered before the layer


@pytest.mark.gpu
def test_a_refused_layer_call_writes_nothing():
    """4-bit images off a 16-byte boundary: logits, blob, output and workspace stay as they were."""
    rng = np.random.default_rng(3)
    T, D, E, k, I = 40, 128, 8, 2, 64
    layer = Layer(rng, D, E, E, I, 0, "mxfp4")
    layer.on_gpu(True)
    router, gate, up, down = layer.alive[:4]
    moved = torch.empty(up.numel() + 8, dtype=torch.uint8, device="cuda")[8:].copy_(up.reshape(-1))
    d = moe.make_dims(T, D, E, k, I, 0, 0, E, True, "bf16", "mxfp4", "bf16", "packed")
    x = torch.randn(T, D, device="cuda").to(torch.bfloat16)
    outs = [torch.full((T, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, E), 7.0, device="cuda"),
            torch.full((T, 2, k), 7, dtype=torch.int32, device="cuda"),
            torch.full((moe.block_workspace(d).numel(),), 7, dtype=torch.uint8, device="cuda")]
    y, logits, blob, ws = outs
    w = moe.make_weights(router, gate, moved, down)
    with pytest.raises(moe.MoeError, match="unsupported"):
        moe.moe_layer_forward(d, w, x, None, None, y, logits, blob, ws)
    with pytest.raises(moe.MoeError, match="unsupported"):
        moe.moe_block_forward(d, w, x, y, w_in=x[0], ws=ws)
    assert all((t == 7).all() for t in outs)
    moe.moe_layer_forward(d, moe.make_weights(router, gate, up, down), x, None, None, y, logits, blob, ws)
    assert torch.isfinite(y.float()).all() and (y != 7).any()


# ---------------------------------------------------------------------------
# An expert slice
# ---------------------------------------------------------------------------

def test_the_block_refuses_an_expert_slice():
    """The layer of a slice gives partial sums, to be added over the devices before any norm."""
    lib = moe.library()
    n = moe.moe_norm(None, None, None, 0, 1.0, 1e-6)
    w = _layer_weights(None)
    for T in (4, 40):
        for begin, local in ((0, 4), (4, 4), (1, 7)):
            d = moe.make_dims(T, 64, 8, 2, 64, 0, begin, local, layout="packed")
            assert lib.moe_block_forward(ctypes.byref(d), ctypes.byref(w), FAKE, None, None, ctypes.byref(n), FAKE, FAKE,
                                         None, FAKE, 1 << 30, None) == moe.ERR_UNSUPPORTED
            assert lib.moe_block_workspace_bytes(ctypes.byref(d)) == 0
            assert moe.moe_workspace_bytes(d) > 0


# ---------------------------------------------------------------------------
# The largest calls
# ---------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [((1 << 24) + 5, 8), ((1 << 20) + 1, 3)])
def test_block_norm_of_many_rows(T, D):
    """2^24 rows are 2^32 threads; the second case ends one row behind a grid row.  Bar as in test_block.py: fp32
    outputs, one rounding each of y + r and of products with one fp32 root (a sum of at most 8 squares)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    y, r = (torch.randn(T, D, generator=g, device="cuda") for _ in range(2))
    gate = torch.randn(T, generator=g, device="cuda")
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    r_out, x = (torch.full((T + 1, D), 5.0, device="cuda") for _ in range(2))
    moe.moe_block_norm(y, r, r_out, w_post=w, gate=gate, gate_kind="token", w_next=w, x_next=x, eps=1e-3)
    assert (r_out[T] == 5.0).all() and (x[T] == 5.0).all()
    for a in range(0, T, 1 << 22):
        b = min(a + (1 << 22), T)
        rms = lambda v: v / (v.square().mean(1, keepdim=True) + 1e-3).sqrt()  # noqa: E731
        z = rms(y[a:b].double()) * w * gate[a:b, None]
        out = r[a:b] + z
        nxt = rms(out) * w
        # the roundings of the mean, root, quotient, three products and the sum, and of x's after them
        lim = 2.0 ** -24 * 24 * (r[a:b].abs() + z.abs())
        inv = (out.square().mean(1, keepdim=True) + 1e-3).rsqrt()
        lim_x = lim * inv * w + nxt.abs() * (lim.square().mean(1, keepdim=True).sqrt() * inv + 24 * 2.0 ** -24)
        assert ((r_out[a:b] - out).abs() <= lim).all() and ((x[a:b] - nxt).abs() <= lim_x).all()


def test_pack_and_unpack_refuse_what_a_grid_cannot_hold():
    """One wave per 16 rows and 512 values: 2^26 of them are 2^32 threads."""
    lib = moe.library()
    most = (1 << 26) - 4
    assert moe.moe_mx_weight_bytes(most, 16, 64) == most * 1280
    assert moe.moe_mx_weight_bytes(most // 6, 32, 1088) == most // 6 * 2 * (9 * 1024 + 3 * 256)
    for n, rows, cols in ((most + 1, 16, 64), (1 << 32, 16, 512), (most // 6 + 1, 32, 1088)):
        assert moe.moe_mx_weight_bytes(n, rows, cols) == 0
        for f in (lib.moe_mx_pack_weights, lib.moe_mx_unpack_weights):
            assert f(moe.BF16, n, rows, cols, FAKE, FAKE, None) == moe.ERR_UNSUPPORTED


# ---------------------------------------------------------------------------
# Tile heights of the 4-bit grouped GEMMs
# ---------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("n,D,I,rows,height", [
    (64, 4096, 1024, 10, 32), (64, 4096, 1024, 25, 128), (64, 4096, 1024, 160, 128),
    (24, 704, 320, 42, 32), (16, 256, 128, 625, 32), (32, 1024, 512, 110, 32),   # weights below 32 MB
    (24, 704, 320, 230, 128),
    (8, 4096, 1024, 100, 32), (8, 4096, 1024, 128, 32), (8, 4096, 1024, 150, 128),   # above
])
def test_tile_height_is_the_faster_one(n, D, I, rows, height):
    """The grouping writes the M-tile prefix of the height that the GEMMs will take: found in the workspace."""
    T = n * rows
    ids = torch.arange(T, dtype=torch.int32) % n
    ids[: 7 * n] = 0                                           # uneven: the prefixes of the two heights differ
    blob = torch.stack([ids, torch.ones(T).view(torch.int32)], 1).reshape(T, 2, 1).contiguous().cuda()
    d = moe.make_dims(T, D, n, 1, I, act="bf16", w="mxfp4", out="bf16", layout="packed")
    ws = torch.full((moe.moe_workspace_bytes(d),), 0xFF, dtype=torch.uint8, device="cuda")
    counts, offsets = (torch.empty(n + i, dtype=torch.int32, device="cuda") for i in range(2))
    perm, inv = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
    moe.moe_permute(d, blob, counts, offsets, perm, inv, ws=ws)
    words = ws.cpu().numpy().view(np.int32)
    c = counts.cpu().numpy()
    found = []
    for h in (32, 128):
        want = np.concatenate([[0], np.cumsum(-(-c // h))])
        places = range(0, len(words) - n, 64)                  # parts of a workspace begin at 256 bytes
        found.append(any((words[p:p + n + 1] == want).all() for p in places if words[p + n] == want[n]))
    assert found == [height == 32, height == 128]


TALL = [130, 1, 128, 0, 300, 64, 97, 33, 96, 160, 129, 5]          # one to four units, one tile of a group or several
WIDE = [70, 128, 31, 200, 0, 160, 257, 65, 96, 40, 100, 150]


@pytest.mark.gpu
@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("counts,D,I,out", [(TALL * 3, 576, 576, "bf16"), (TALL * 3, 1088, 576, "f32"),
                                            (WIDE * 2, 128, 1088, "bf16"), (WIDE * 2, 704, 1088, "f32")])
def test_grouped_ffn_in_tall_tiles(counts, D, I, out, gathered):
    """More than two short tiles' workgroups per CU: rows resident or through the ring, in either launch."""
    assert len(counts) * (sum(counts) / len(counts) / 32 + 0.5) * -(-I // 128) > 512
    test_mx.test_grouped_ffn(counts, D, I, out, gathered)


@pytest.mark.gpu
def test_layer_forward_in_tall_tiles():
    assert 32 * (900 * 4 / 32 / 32 + 0.5) * 5 > 512
    test_mx.test_layer_forward(900, 256, 32, 4, 640, 64, 0, 32, False)


# ---------------------------------------------------------------------------
# Tensors of another device
# ---------------------------------------------------------------------------

class _On0(torch.Tensor):
    """A host tensor that says it lives on device 0: host checks only."""

    def get_device(self):
        return 0

    is_cuda = True


class _On1(_On0):
    def get_device(self):
        return 1


class _Calls:
    """In place of the library: counts what reaches it."""

    def __init__(self):
        self.n = 0

    def moe_mx_weight_bytes(self, n, rows, cols):
        return n * (rows // 16) * 1280

    def __getattr__(self, name):
        def call(*args):
            self.n += 1
            return moe.OK
        return call


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _device_cases():
    d = moe.make_dims(4, 64, 8, 2, 64)
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    w = moe.moe_weights()
    few = dict(x=_bf(4, 64), packed_in=torch.zeros(4, 2, 2, dtype=i32), logit_bias=torch.zeros(8), y=_bf(4, 64),
               logits_out=torch.zeros(4, 8), packed_out=torch.zeros(4, 2, 2, dtype=i32), ws=torch.zeros(64, dtype=u8))
    norm = dict(y=_bf(4, 64), r=_bf(4, 64), r_out=_bf(4, 64), w_post=_bf(64), gate=torch.zeros(4, dtype=f32),
                w_next=_bf(64), x_next=_bf(4, 64))
    block = dict(r=_bf(4, 64), r_out=_bf(4, 64), w_in=_bf(64), x_in=_bf(4, 64), logit_bias=torch.zeros(8), w_post=_bf(64),
                 gate=torch.zeros(4, dtype=f32), w_next=_bf(64), x_next=_bf(4, 64), ws=torch.zeros(64, dtype=u8))
    return [
        (lambda **t: moe.moe_layer_forward_few(d, w, **t), few),
        (lambda **t: moe.moe_block_norm(**t, gate_kind="token"), norm),
        (lambda **t: moe.moe_block_forward(d, w, **t, gate_kind="token"), block),
        (moe.moe_mx_pack_weights, dict(src=_bf(16, 64), dst=torch.zeros(1280, dtype=u8))),
        (lambda **t: moe.moe_mx_unpack_weights(rows=16, cols=64, **t), dict(images=torch.zeros(1280, dtype=u8), dst=_bf(16, 64))),
    ]


@pytest.mark.parametrize("case", range(5))
def test_every_tensor_is_on_the_current_device(case, monkeypatch):
    calls = _Calls()
    monkeypatch.setattr(moe, "library", lambda: calls)
    monkeypatch.setattr(moe, "_stream", lambda stream: 0)
    monkeypatch.setattr(moe, "_device", lambda: 0)
    call, tensors = _device_cases()[case]
    near = {k: v.as_subclass(_On0) for k, v in tensors.items()}
    call(**near)
    assert calls.n == 1
    for name, t in tensors.items():
        with pytest.raises(ValueError, match=f"{name} .*cuda:1"):
            call(**{**near, name: t.as_subclass(_On1)})
    assert calls.n == 1
    with pytest.raises(ValueError, match="GPU memory"):
        call(**{**near, next(iter(tensors)): next(iter(tensors.values()))})
