"""Products grouped by expert and both gradients (moe_grouped_gemm*), against float64.

Small whole numbers as inputs make every product and partial sum exact in fp32, so those results have to be equal to
float64's, rounded once.  Random inputs: a sum of R exact products in fp32, in any order, is off by at most
R * 2^-24 of the sum of their magnitudes; adding a tensor and the result's own rounding (2^-8 of the value in bf16,
2^-24 in fp32) come on top.
"""

import ctypes

import pytest
import torch

import sparse_moe_ffn_route_amd as moe

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DIRS = ("fwd", "rows", "weights")

# rows of each group: none, one, either side of the tiles' edges, many; a last group of one row or none
RAGGED = {
    "one_row": [1],
    "none": [0, 0, 0],
    "few": [0, 1, 15, 16, 0, 17, 31, 32, 33, 2, 0],
    "middle": [0, 127, 1, 128, 129, 65, 0, 200],
    "many": [0, 513, 255, 256, 1, 257, 300, 0, 1],
}
WIDTHS = [(8, 8), (64, 128), (136, 72), (264, 328)]


def ints(shape, dtype, seed, top=3):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g).to(DT[dtype])


def offsets_of(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)


def reference(dir, counts, a, d_out, w, index, add, rows):
    """Float64 result; rows behind the last group: NaN (not to be compared)."""
    at = offsets_of(counts).tolist()
    a = a.double() if index is None or a is None else a.double()[index.long()]
    if dir == "weights":
        out = torch.stack([d_out[b:t].double().T @ a[b:t] for b, t in zip(at, at[1:])])
        return out if add is None else out + add.double()
    src = a if dir == "fwd" else d_out.double()
    width = w.shape[1] if dir == "fwd" else w.shape[2]
    out = torch.full((rows, width), float("nan"), dtype=torch.float64)
    for e, (b, t) in enumerate(zip(at, at[1:])):
        m = w[e].double()
        out[b:t] = src[b:t] @ (m.T if dir == "fwd" else m)
    return out if add is None else out + add.double()


def call(dir, g, a, d_out, w, offsets, out, index=None, add=None, ws=None, stream=None):
    ws = moe.grouped_gemm_workspace(g) if ws is None else ws
    if dir == "fwd":
        moe.moe_grouped_gemm(g, a, offsets, w, out, index=index, add=add, ws=ws, stream=stream)
    elif dir == "rows":
        moe.moe_grouped_gemm_backward_rows(g, d_out, offsets, w, out, add=add, ws=ws, stream=stream)
    else:
        moe.moe_grouped_gemm_backward_weights(g, d_out, a, offsets, out, index=index, add=add, ws=ws, stream=stream)


def case(dir, counts, N, K, dtype, out, gather, add, spare=5, seed=0, make=ints):
    """Inputs on the CPU: `spare` rows behind the last group."""
    n, rows = len(counts), sum(counts) + spare
    src = max(1, rows // 2) if gather else rows
    index = torch.randint(0, src, (rows,), generator=torch.Generator().manual_seed(seed + 9)).int() if gather else None
    shape = {"fwd": (rows, N), "rows": (rows, K), "weights": (n, N, K)}[dir]
    return dict(a=make((src, K), dtype, seed + 1), d_out=make((rows, N), dtype, seed + 2), w=make((n, N, K), dtype, seed + 3),
                index=index, add=make(shape, out, seed + 4) if add else None), shape, rows


def run(dir, counts, N, K, dtype, out, gather=False, add=False, spare=5, seed=0, make=ints):
    c, shape, rows = case(dir, counts, N, K, dtype, out, gather, add, spare, seed, make)
    gpu = {k: None if v is None else v.cuda() for k, v in c.items()}
    result = torch.full(shape, 777.0, dtype=DT[out], device="cuda")
    g = moe.make_groups(len(counts), rows, N, K, dtype, out)
    call(dir, g, gpu["a"], gpu["d_out"], gpu["w"], offsets_of(counts).cuda(), result, gpu["index"], gpu["add"])
    return result.cpu(), reference(dir, counts, c["a"], c["d_out"], c["w"], c["index"], c["add"], rows), c


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("N,K", WIDTHS)
@pytest.mark.parametrize("counts", list(RAGGED))
@pytest.mark.parametrize("dir", DIRS)
def test_whole_numbers_are_exact(dir, counts, N, K, dtype, out):
    counts = RAGGED[counts]
    for gather, add in ((False, False), (dir != "rows", True)):
        got, ref, _ = run(dir, counts, N, K, dtype, out, gather, add)
        used = sum(counts)
        if dir != "weights":
            assert (got[used:] == 777.0).all()              # rows behind the last group
            got, ref = got[:used], ref[:used]
        assert torch.equal(got, ref.to(DT[out])), (gather, add)


# Sizes that take the other tile shapes, and reductions in parts, in one direction or another: ends of tiles in every
# dimension, a group that ends a few rows into a tile, empty ones.
LARGE = [([4100], 4104, 1032), ([2100, 0, 2200], 2056, 4104), ([700, 0, 130, 1100, 3, 40], 1032, 2056), ([9000], 520, 1032),
         ([5003], 264, 264), ([3, 1, 5, 0, 2], 1544, 2056), ([3] * 60 + [0, 17, 1], 1032, 1032)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("counts,N,K", LARGE)
@pytest.mark.parametrize("dir", DIRS)
def test_whole_numbers_are_exact_at_large_sizes(dir, counts, N, K, dtype, out):
    add = gather = dir != "rows"
    got, ref, _ = run(dir, counts, N, K, dtype, out, gather, add or out == "f32")
    used = sum(counts)
    if dir != "weights":
        assert (got[used:] == 777.0).all()
        got, ref = got[:used], ref[:used]
    assert torch.equal(got, ref.to(DT[out]))


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("dir", DIRS)
def test_whole_numbers_are_exact_at_the_largest_tiles(dir, out):
    """All three directions in their largest tiles; the float64 products on the GPU."""
    counts, N, K = [2000, 0, 300, 5700], 4104, 4104
    c, shape, rows = case(dir, counts, N, K, "bf16", out, False, False)
    gpu = {k: None if v is None else v.cuda() for k, v in c.items()}
    got = torch.full(shape, 777.0, dtype=DT[out], device="cuda")
    call(dir, moe.make_groups(4, rows, N, K, "bf16", out), gpu["a"], gpu["d_out"], gpu["w"], offsets_of(counts).cuda(), got)
    at = offsets_of(counts).tolist()
    for e, (b, t) in enumerate(zip(at, at[1:])):
        a, d, w = gpu["a"][b:t].double(), gpu["d_out"][b:t].double(), gpu["w"][e].double()
        ref = d.T @ a if dir == "weights" else a @ w.T if dir == "fwd" else d @ w
        assert torch.equal(got[e] if dir == "weights" else got[b:t], ref.to(DT[out]))


@pytest.mark.gpu
@pytest.mark.parametrize("dir", DIRS)
def test_tensors_past_32_bits(dir):
    """Rows whose first byte, and first element, lie past 2^32: 1.1 million of 4096 values, a few of them not zero."""
    rows, wide, narrow = (1 << 20) + 70_000, 4096, 8
    N, K = (wide, narrow) if dir == "weights" else (narrow, wide) if dir == "fwd" else (narrow, wide)
    counts = [rows - 40, 0, 33]
    at = offsets_of(counts).tolist()
    some = torch.tensor([0, 1, 524_287, 524_288, 1_048_575, 1_048_576, rows - 41, rows - 40, rows - 20, rows - 8])
    c = dict(a=ints((len(some), K), "bf16", 1), d_out=ints((len(some), N), "bf16", 2), w=ints((3, N, K), "bf16", 3))
    spread = lambda v: torch.zeros(rows, v.shape[1], dtype=v.dtype, device="cuda").index_copy_(0, some.cuda(), v.cuda())  # noqa: E731
    a = spread(c["a"]) if dir != "rows" else None
    d_out = spread(c["d_out"]) if dir != "fwd" else None
    shape = {"fwd": (rows, N), "rows": (rows, K), "weights": (3, N, K)}[dir]
    out = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
    g = moe.make_groups(3, rows, N, K, "bf16", "bf16")
    call(dir, g, a, d_out, c["w"].cuda(), offsets_of(counts).cuda(), out)
    of = torch.bucketize(some, torch.tensor(at[1:]), right=True)
    if dir == "weights":
        ref = torch.stack([c["d_out"][of == e].double().T @ c["a"][of == e].double() for e in range(3)])
        assert torch.equal(out.cpu(), ref.bfloat16())
        return
    m = c["w"].double()[of]
    ref = torch.einsum("rk,rnk->rn", c["a"].double(), m) if dir == "fwd" else torch.einsum("rn,rnk->rk", c["d_out"].double(), m)
    assert torch.equal(out[some.cuda()].cpu(), ref.bfloat16())
    assert (out[rows - 7:] == 7).all()
    out[rows - 7:] = 0
    out[some.cuda()] = 0
    assert not out.any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dir", DIRS)
def test_workspace_is_as_large_as_said(dir, dtype):
    """Reductions in parts: bytes behind the workspace stay, and what it held before does not matter."""
    for counts, N, K in (([16], 1032, 4104), ([5000], 72, 136), ([700, 0, 41], 264, 2056)):
        c, shape, rows = case(dir, counts, N, K, dtype, "f32", False, False)
        gpu = {k: None if v is None else v.cuda() for k, v in c.items()}
        g = moe.make_groups(len(counts), rows, N, K, dtype, "f32")
        need = moe.grouped_gemm_workspace(g).nbytes
        ref = reference(dir, counts, c["a"], c["d_out"], c["w"], None, None, rows)
        for fill in (0, 255):
            ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
            ws[need:] = 171
            got = torch.full(shape, 777.0, device="cuda")
            call(dir, g, gpu["a"], gpu["d_out"], gpu["w"], offsets_of(counts).cuda(), got, ws=ws[:need])
            assert (ws[need:] == 171).all()
            keep = slice(None) if dir == "weights" else slice(0, sum(counts))
            assert torch.equal(got.cpu()[keep].double(), ref[keep])
            assert dir == "weights" or (got[sum(counts):] == 777).all()


@pytest.mark.gpu
def test_a_slice_of_the_groups():
    """Offsets that start behind the first row: rows of the groups before and after stay, a reduction in parts, too."""
    counts, N, K = [70, 5003, 40], 264, 264
    c, _, rows = case("fwd", counts, N, K, "bf16", "f32", False, False)
    for dir in ("fwd", "rows"):
        out = torch.full((rows, N), 777.0, device="cuda")
        off = offsets_of(counts)
        call(dir, moe.make_groups(1, rows, N, K, "bf16", "f32"), c["a"].cuda(), c["d_out"].cuda(), c["w"][1:2].cuda(),
             off[1:3].clone().cuda(), out)
        out = out.cpu()
        assert (out[:70] == 777).all() and (out[5073:] == 777).all()
        ref = c["a"].double() @ c["w"][1].double().T if dir == "fwd" else c["d_out"].double() @ c["w"][1].double()
        assert torch.equal(out[70:5073].double(), ref[70:5073])


@pytest.mark.gpu
@pytest.mark.parametrize("dir", DIRS)
@pytest.mark.parametrize("dtype,out,N,K,counts", [
    ("bf16", "f32", 1024, 712, [40, 0, 700, 3]), ("bf16", "bf16", 512, 1536, [300]), ("f32", "f32", 200, 1288, [31, 170]),
    ("bf16", "bf16", 1536, 2048, [3, 1, 5, 0, 2])])
def test_random_values(dir, dtype, out, N, K, counts):
    def make(shape, dtype, seed):
        return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])

    got, ref, c = run(dir, counts, N, K, dtype, out, False, True, spare=0, make=make)
    mag = reference(dir, counts, c["a"].abs(), c["d_out"].abs(), c["w"].abs(), None, c["add"].abs(), sum(counts))
    R = {"fwd": K, "rows": N, "weights": max(counts)}[dir]
    bound = (R + 2) * 2.0 ** -24 * mag + HALF[out] * ref.abs()
    assert ((got.double() - ref).abs() <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dir", DIRS)
@pytest.mark.parametrize("counts", ["few", "many"])
def test_nothing_leaks_between_groups(dir, counts):
    """Infinities and NaN in one group, its weights and the rows behind the last group stay there."""
    counts = RAGGED[counts]
    N, K = 136, 72
    c, shape, rows = case(dir, counts, N, K, "bf16", "f32", False, False)
    at = offsets_of(counts).tolist()
    bad = 3
    for t, value in ((c["a"], float("nan")), (c["d_out"], float("inf"))):
        t[at[bad]:at[bad + 1]] = value
        t[at[-1]:] = value
    c["w"][bad] = float("nan")
    gpu = {k: None if v is None else v.cuda() for k, v in c.items()}
    out = torch.full(shape, 777.0, device="cuda")
    call(dir, moe.make_groups(len(counts), rows, N, K, "bf16", "f32"), gpu["a"], gpu["d_out"], gpu["w"],
         offsets_of(counts).cuda(), out)
    out = out.cpu()
    ref = reference(dir, counts, c["a"], c["d_out"], c["w"], None, None, rows)
    for e in range(len(counts)):
        r = e if dir == "weights" else slice(at[e], at[e + 1])
        assert e == bad or torch.equal(out[r].double(), ref[r])
    assert not out[bad if dir == "weights" else slice(at[bad], at[bad + 1])].isfinite().any()


@pytest.mark.gpu
@pytest.mark.parametrize("dir", ["fwd", "weights"])
def test_indexes_outside_a_are_rows_of_zeros(dir):
    counts, N, K = [5, 70, 3], 64, 128
    c, shape, rows = case(dir, counts, N, K, "bf16", "f32", True, False)
    c["index"][::3] = torch.tensor([-1, c["a"].shape[0], 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).repeat(rows)[:len(c["index"][::3])]
    gpu = {k: None if v is None else v.cuda() for k, v in c.items()}
    out = torch.zeros(shape, device="cuda")
    call(dir, moe.make_groups(3, rows, N, K, "bf16", "f32"), gpu["a"], gpu["d_out"], gpu["w"], offsets_of(counts).cuda(),
         out, gpu["index"])
    inside = (c["index"] >= 0) & (c["index"] < c["a"].shape[0])
    a = torch.where(inside[:, None], c["a"][c["index"].clamp(0, c["a"].shape[0] - 1).long()].float(), 0.0)
    ref = reference(dir, counts, a, c["d_out"], c["w"], None, None, rows)
    used = sum(counts)
    assert torch.equal((out if dir == "weights" else out[:used]).cpu().double(), ref if dir == "weights" else ref[:used])


@pytest.mark.gpu
@pytest.mark.parametrize("dir", DIRS)
def test_offsets_outside_the_rows_stay_inside(dir):
    """Offsets past `rows`, below zero and falling are taken as the nearest allowed."""
    rows, N, K = 40, 64, 64
    wild = torch.tensor([-5, 7, 3, 1000, 2 ** 31 - 1], dtype=torch.int32)
    bounds = [(0, 7), (7, 7), (3, 40), (40, 40)]
    a, d_out, w = ints((rows, K), "bf16", 1), ints((rows, N), "bf16", 2), ints((4, N, K), "bf16", 3)
    shape = {"fwd": (rows, N), "rows": (rows, K), "weights": (4, N, K)}[dir]
    out = torch.zeros(shape, device="cuda")
    call(dir, moe.make_groups(4, rows, N, K, "bf16", "f32"), a.cuda(), d_out.cuda(), w.cuda(), wild.cuda(), out)
    out = out.cpu().double()
    a, d_out, w = a.double(), d_out.double(), w.double()
    if dir == "weights":
        for e, (b, t) in enumerate(bounds):
            assert torch.equal(out[e], d_out[b:t].T @ a[b:t])
    else:  # rows 3 to 6 belong to two groups here; either may have written them
        f = (lambda e, r: a[r] @ w[e].T) if dir == "fwd" else (lambda e, r: d_out[r] @ w[e])
        assert torch.equal(out[:3], f(0, slice(0, 3))) and torch.equal(out[7:], f(2, slice(7, 40)))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 63, 64, 65, 200, 1000, 1024])
def test_many_groups(n):
    """The search for a tile's group, over groups with and without rows."""
    g = torch.Generator().manual_seed(n)
    counts = (torch.randint(0, 4, (n,), generator=g) * torch.randint(0, 15, (n,), generator=g)).tolist()
    for dir in DIRS:
        got, ref, _ = run(dir, counts, 16, 24, "bf16", "f32")
        used = sum(counts)
        assert torch.equal(got.double() if dir == "weights" else got[:used].double(), ref if dir == "weights" else ref[:used])


@pytest.mark.gpu
@pytest.mark.parametrize("dir", DIRS)
def test_adding_in_place(dir):
    """A running sum: the result is added to its own memory, call after call."""
    counts, N, K = [3, 0, 130, 40], 72, 136
    c, shape, rows = case(dir, counts, N, K, "bf16", "f32", False, False)
    gpu = {k: None if v is None else v.cuda() for k, v in c.items()}
    out = torch.zeros(shape, device="cuda")
    g, off = moe.make_groups(4, rows, N, K, "bf16", "f32"), offsets_of(counts).cuda()
    for _ in range(3):
        call(dir, g, gpu["a"], gpu["d_out"], gpu["w"], off, out, add=out)
    ref = 3 * reference(dir, counts, c["a"], c["d_out"], c["w"], None, None, rows)
    used = slice(None) if dir == "weights" else slice(0, sum(counts))
    assert torch.equal(out.cpu().double()[used], ref[used])


@pytest.mark.gpu
@pytest.mark.parametrize("dir", DIRS)
def test_streams_and_graph(dir):
    """On another stream, and captured: replays on new rows and offsets between eager calls on the same workspace."""
    counts, N, K = [40, 0, 7, 90], 128, 264
    c, shape, rows = case(dir, counts, N, K, "bf16", "bf16", False, False)
    gpu = {k: None if v is None else v.cuda() for k, v in c.items()}
    g, off = moe.make_groups(4, rows, N, K, "bf16", "bf16"), offsets_of(counts).cuda()
    ws = moe.grouped_gemm_workspace(g)
    out = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(dir, g, gpu["a"], gpu["d_out"], gpu["w"], off, out, ws=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(dir, g, gpu["a"], gpu["d_out"], gpu["w"], off, out, ws=ws)
    for i, counts in enumerate(([40, 0, 7, 90], [0, 137, 0, 0], [1, 1, 1, 1])):
        off.copy_(offsets_of(counts))
        for t in ("a", "d_out"):
            gpu[t].copy_(ints(gpu[t].shape, "bf16", 50 + i))
        out.zero_()
        graph.replay()
        replayed = out.clone()
        out.zero_()
        call(dir, g, gpu["a"], gpu["d_out"], gpu["w"], off, out, ws=ws)
        assert torch.equal(replayed, out)
        ref = reference(dir, counts, gpu["a"].cpu(), gpu["d_out"].cpu(), c["w"], None, None, rows).to(torch.bfloat16)
        used = slice(None) if dir == "weights" else slice(0, sum(counts))
        assert torch.equal(out.cpu()[used], ref[used])


# ---------------------------------------------------------------------------
# Refusals, before any launch
# ---------------------------------------------------------------------------

FAKE, OFF = ctypes.c_void_p(256), ctypes.c_void_p(264)


def test_refusals():
    lib = moe.library()

    def all_three(n=2, rows=64, N=64, K=64, i=moe.BF16, o=moe.BF16, p=FAKE, q=FAKE, offsets=FAKE, out=FAKE, index=None,
                  a_rows=64, add=None, ws=FAKE, nb=1 << 40):
        g = ctypes.byref(moe.moe_groups(n, rows, N, K, i, o))
        got = [lib.moe_grouped_gemm(g, p, a_rows, index, offsets, q, add, out, ws, nb, None),
               lib.moe_grouped_gemm_backward_weights(g, p, q, a_rows, index, offsets, add, out, ws, nb, None)]
        if index is None:
            got.append(lib.moe_grouped_gemm_backward_rows(g, p, offsets, q, add, out, ws, nb, None))
        assert len(set(got)) == 1
        return got[0]

    for bad in (dict(n=0), dict(rows=-1), dict(N=0), dict(K=-8)):
        assert all_three(**bad) == moe.ERR_BAD_DIMS
    for bad in (dict(n=1025), dict(N=60), dict(K=4), dict(K=(1 << 20) + 8), dict(i=moe.E4M3), dict(i=moe.F32),
                dict(o=moe.E4M3), dict(p=OFF), dict(q=OFF), dict(out=OFF), dict(add=OFF), dict(ws=OFF),
                dict(index=FAKE, a_rows=1 << 24)):
        assert all_three(**bad) == moe.ERR_UNSUPPORTED, bad
    for bad in (dict(p=None), dict(q=None), dict(offsets=None), dict(out=None)):
        assert all_three(**bad) == moe.ERR_NULL_ARG
    assert all_three(index=FAKE, a_rows=-1) == moe.ERR_BAD_DIMS
    assert lib.moe_grouped_gemm(None, FAKE, 0, None, FAKE, FAKE, None, FAKE, FAKE, 0, None) == moe.ERR_NULL_ARG
    assert lib.moe_grouped_gemm_workspace_bytes(ctypes.byref(moe.moe_groups(1, 1, 60, 64, 1, 1))) == 0
    assert lib.moe_grouped_gemm_workspace_bytes(ctypes.byref(moe.make_groups(1, 1, 64, 64))) >= 256


def test_binding_refusals(monkeypatch):
    monkeypatch.setattr(moe, "_device", lambda: -1)   # where these tensors are: types and sizes are what is refused
    g = moe.make_groups(2, 8, 64, 32)
    a, w, out = torch.zeros(8, 32).bfloat16(), torch.zeros(2, 64, 32).bfloat16(), torch.zeros(8, 64).bfloat16()
    off = torch.zeros(3, dtype=torch.int32)
    for args, what in (((a.float(), off, w, out), "a"), ((a[:7], off, w, out), "a"), ((a, off[:2], w, out), "offsets"),
                       ((a, off.long(), w, out), "offsets"), ((a, off, w[:1], out), "w"), ((a, off, w, out.float()), "out"),
                       ((a, off, w, out[:7]), "out")):
        with pytest.raises(ValueError, match=what):
            moe.moe_grouped_gemm(g, *args)
    with pytest.raises(ValueError, match="index"):
        moe.moe_grouped_gemm(g, a, off, w, out, index=off)
    with pytest.raises(ValueError, match="add"):
        moe.moe_grouped_gemm(g, a, off, w, out, add=out[:1])
    with pytest.raises(ValueError, match="d_a"):
        moe.moe_grouped_gemm_backward_rows(g, out, off, w, a.float())
    with pytest.raises(ValueError, match="d_w"):
        moe.moe_grouped_gemm_backward_weights(g, out, a, off, w[0])
    with pytest.raises(ValueError, match=r"\[a_rows\]\[K\]"):
        moe.moe_grouped_gemm(g, a[:, :16].contiguous(), off, w, out, index=torch.zeros(8, dtype=torch.int32))
    monkeypatch.undo()
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_grouped_gemm(g, a, off, w, out)
