"""Every tile shape of the grouped products, whole and in parts, in every direction.

Which of them a call takes is decided from its sizes (csrc/group_plan.hpp).  The cases below say which one they are
for, and a test without a GPU compiles that decision and holds them to it, so that no change of it empties a test here
unseen.  Small whole numbers make every sum exact: results have to be equal to float64's, rounded once.
"""

import os
import shutil
import subprocess

import pytest
import torch

import sparse_moe_ffn_route_amd as moe
from sparse_moe_ffn_route_amd import build
from test_grouped_gemm import DIRS, DT, call

SHAPES = ("small", "narrow", "middle", "wide", "big", "few")

# rows of each group (and SPARE behind the last), N, K, operand type, tile shape, parts of the reduction; the same plan
# for both result types.  Groups without rows, of one, and ends inside a tile in every dimension.
SPARE = 5
CASES = [
    ("fwd", [5, 1, 0], 8, 1656, "bf16", "few", 4),
    ("fwd", [0, 3], 8, 24, "bf16", "few", 1),
    ("fwd", [3, 1, 5, 0, 2], 1544, 2056, "bf16", "few", 2),
    ("fwd", [25], 8, 2128, "bf16", "small", 8),
    ("fwd", [25], 72, 24, "bf16", "small", 1),
    ("fwd", [60], 4272, 2904, "bf16", "narrow", 4),
    ("fwd", [545], 840, 3744, "bf16", "narrow", 4),
    ("fwd", [300, 0, 170, 200, 1, 313], 1744, 8, "bf16", "narrow", 1),
    ("fwd", [100, 0, 130, 161, 3, 43], 1232, 3464, "bf16", "middle", 4),
    ("fwd", [700, 1100, 0, 22], 496, 4296, "bf16", "middle", 4),
    ("fwd", [2748], 1416, 8, "bf16", "middle", 1),
    ("fwd", [1500, 0, 3045], 1168, 8, "bf16", "wide", 1),
    ("fwd", [400, 0, 1000, 6, 60, 6], 3560, 8, "bf16", "wide", 1),
    ("fwd", [1700, 0, 1, 1294], 4104, 4104, "bf16", "big", 1),
    ("rows", [3], 1224, 8, "bf16", "few", 4),
    ("rows", [0, 3, 0], 8, 8, "bf16", "few", 1),
    ("rows", [7, 0, 3, 12], 1680, 8, "bf16", "few", 4),
    ("rows", [1, 0, 9, 3, 5, 4], 3384, 1264, "bf16", "narrow", 4),
    ("rows", [25], 1048, 8, "bf16", "small", 4),
    ("rows", [0, 60], 16, 16, "bf16", "small", 1),
    ("rows", [5096], 8, 344, "bf16", "narrow", 1),
    ("rows", [484], 4232, 1944, "bf16", "middle", 4),
    ("rows", [2146], 8, 1824, "bf16", "middle", 1),
    ("rows", [4, 0, 1, 2, 0, 2], 3720, 3384, "bf16", "wide", 2),
    ("rows", [20, 1, 0, 20, 0, 3], 3432, 3304, "bf16", "wide", 2),
    ("rows", [1000, 358], 8, 4080, "bf16", "wide", 1),
    ("rows", [2600, 0, 17, 2383], 3688, 2704, "bf16", "big", 1),
    ("weights", [400, 374], 8, 8, "bf16", "small", 2),
    ("weights", [3], 8, 8, "bf16", "small", 1),
    ("weights", [0, 2305], 8, 2216, "bf16", "narrow", 8),
    ("weights", [5, 0, 0, 50, 1, 10], 72, 2936, "bf16", "narrow", 1),
    ("weights", [3000, 0, 1342], 3760, 80, "bf16", "middle", 4),
    ("weights", [5, 0, 1, 0, 0, 3], 200, 2864, "bf16", "middle", 1),
    ("weights", [5000, 0, 209], 328, 944, "bf16", "middle", 4),
    ("weights", [50, 0, 1, 0, 0, 8], 400, 2344, "bf16", "wide", 1),
    ("weights", [5610], 1616, 2952, "bf16", "wide", 2),
    ("weights", [9000, 0, 1, 8503], 1944, 2008, "bf16", "big", 1),
    ("weights", [38000, 694], 4080, 400, "bf16", "big", 4),
    ("fwd", [0, 3], 8, 672, "f32", "small", 4),
    ("fwd", [3], 8, 8, "f32", "small", 1),
    ("fwd", [300, 0, 1, 408], 600, 2512, "f32", "narrow", 4),
    ("fwd", [4285], 504, 8, "f32", "narrow", 1),
    ("rows", [0, 6], 456, 8, "f32", "small", 2),
    ("rows", [4], 8, 8, "f32", "small", 1),
    ("rows", [5, 0, 2, 1], 4048, 2168, "f32", "narrow", 4),
    ("rows", [200, 0, 1, 409, 0, 2], 8, 3040, "f32", "narrow", 1),
    ("weights", [234], 8, 8, "f32", "small", 2),
    ("weights", [4], 8, 8, "f32", "small", 1),
    ("weights", [4000, 488], 8, 4064, "f32", "narrow", 8),
    ("weights", [30, 0, 1, 0, 3, 0], 264, 1096, "f32", "narrow", 1),
]

# One group from the middle of the rows, whose reduction is split: rows before it, of it and after it, N, K, types
SLICES = [
    ("fwd", [20, 16, 15], 1032, 4104, "bf16", "bf16", "small", 16),
    ("fwd", [20, 16, 15], 1032, 4104, "bf16", "f32", "small", 16),
    ("fwd", [30, 300, 11], 264, 4104, "f32", "f32", "small", 8),
    ("rows", [20, 35, 15], 4104, 264, "bf16", "bf16", "few", 16),
    ("rows", [20, 35, 15], 4104, 264, "bf16", "f32", "few", 16),
    ("rows", [70, 500, 25], 4104, 264, "bf16", "bf16", "small", 8),
    ("rows", [70, 500, 25], 4104, 264, "bf16", "f32", "small", 8),
    ("rows", [70, 500, 25], 4104, 264, "f32", "f32", "small", 8),
]

ASK = """
#include <cstdio>
#include "group_plan.hpp"
int main() {
  int dir, n, rows, N, K, f32, out_f32;
  while (std::scanf("%d %d %d %d %d %d %d", &dir, &n, &rows, &N, &K, &f32, &out_f32) == 7) {
    const moe::groups::Plan p = moe::groups::plan(dir, moe::group_sizes(dir, n, rows, N, K), f32, out_f32);
    std::printf("%d %d %d %lld\\n", p.shape, p.parts, p.high, static_cast<long long>(p.blocks));
  }
}
"""


def results_of(dtype):
    return ["f32"] if dtype == "f32" else ["bf16", "f32"]


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """Shape and parts (and a tile's rows and the workgroups) of calls, by the library's own choice, compiled for the host."""
    at = tmp_path_factory.mktemp("plan")
    (at / "ask.cpp").write_text(ASK)
    cc = shutil.which("g++") or os.path.join(os.path.dirname(build._hipcc()), "amdclang++")
    subprocess.run([cc, "-O1", "-std=c++17", "-I", build.CSRC, str(at / "ask.cpp"), "-o", str(at / "ask")], check=True)

    def ask(calls, counts=False):
        lines = "\n".join(f"{DIRS.index(d)} {n} {rows} {N} {K} {int(t == 'f32')} {int(o == 'f32')}"
                          for d, n, rows, N, K, t, o in calls)
        got = subprocess.run([str(at / "ask")], input=lines, text=True, check=True, capture_output=True).stdout.split()
        return [(SHAPES[int(s)], int(p)) + ((int(h), int(b)) if counts else ())
                for s, p, h, b in zip(*(got[i::4] for i in range(4)))]

    return ask


def test_cases_take_the_shapes_they_are_for(plans):
    """Every kernel that the library holds is in a case, and so is a reduction in parts of every direction and type."""
    calls, want = [], []
    for dir, counts, N, K, dtype, shape, parts in CASES:
        for out in results_of(dtype):
            calls.append((dir, len(counts), sum(counts) + SPARE, N, K, dtype, out))
            want.append((shape, parts))
    assert plans(calls) == want
    taken = {(c[0], c[5], c[6], shape) for c, (shape, _) in zip(calls, want)}
    held = {(dir, t, o, s) for dir in DIRS for t, o in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"))
            for s in (SHAPES[:2] if t == "f32" else SHAPES if dir != "weights" else SHAPES[:5])}
    assert taken == held
    assert {(c[0], c[5], c[6]) for c, (_, parts) in zip(calls, want) if parts > 1} == {x[:3] for x in held}


def test_slices_are_split(plans):
    assert plans([(dir, 1, sum(counts) + SPARE, N, K, t, o) for dir, counts, N, K, t, o, _, _ in SLICES]) == \
        [s[6:] for s in SLICES]


def test_counts_of_the_largest_calls_fit(plans):
    """Workgroups in 31 bits and tile rows in 25, up to the sizes that are refused."""
    sizes = [(n, rows, N, K) for n in (1, 3, 1000, 1024) for rows in (0, 1, 1024, 1 << 20, (1 << 30) - 1, 1 << 30)
             for N in (8, 1024, 8192, 1 << 20) for K in (8, 1024, 8192, 1 << 20)]
    types = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]
    fit = [s for s in sizes if max(s[1] * s[2], s[1] * s[3], s[0] * s[2] * s[3]) <= 1 << 40]
    calls = [(dir, *s, t, o) for s in fit for dir in DIRS for t, o in types]
    for (dir, n, rows, *_), (_, _, high, blocks) in zip(calls, plans(calls, True)):
        assert blocks < 1 << 31 and (dir == "weights" or rows // high + n < 1 << 25)
    for n, rows, N, K in sizes:
        for t, o in types:
            need = moe.library().moe_grouped_gemm_workspace_bytes(moe.make_groups(n, rows, N, K, t, o))
            assert (need > 0) == ((n, rows, N, K) in fit)


def test_refusal_of_more_than_2_to_the_40_elements():
    lib, fake = moe.library(), 256
    for n, rows, N, K in ((1024, 8, 1 << 20, 1032), (1, 1 << 30, 1032, 8), (1, 1 << 30, 8, 1032)):
        g = moe.make_groups(n, rows, N, K)
        got = {lib.moe_grouped_gemm(g, fake, 0, None, fake, fake, None, fake, fake, 1 << 40, None),
               lib.moe_grouped_gemm_backward_rows(g, fake, fake, fake, None, fake, fake, 1 << 40, None),
               lib.moe_grouped_gemm_backward_weights(g, fake, fake, 0, None, fake, None, fake, fake, 1 << 40, None)}
        assert got == {moe.ERR_UNSUPPORTED}


def whole(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda").to(DT[dtype])


class Call:
    """Inputs on the GPU; what lies behind the last group is NaN."""

    def __init__(self, dir, counts, N, K, dtype, out, gather, add, seed=0):
        n, used, rows = len(counts), sum(counts), sum(counts) + SPARE
        self.dir, self.used = dir, used
        self.groups = moe.make_groups(n, rows, N, K, dtype, out)
        self.at = [0] + torch.tensor(counts).cumsum(0).tolist()
        self.offsets = torch.tensor(self.at, dtype=torch.int32, device="cuda")
        self.d_out = whole((rows, N), dtype, seed + 1)
        self.d_out[used:] = float("nan")
        self.w = whole((n, N, K), dtype, seed + 2)
        self.index = None
        if gather:  # some rows twice, some outside, and the rows behind the last group from the NaN
            src = max(1, used // 2)
            self.a = whole((src + 1, K), dtype, seed + 3)
            self.index = torch.randint(0, src, (rows,), device="cuda",
                                       generator=torch.Generator(device="cuda").manual_seed(seed + 4)).int()
            self.index[3:used:11] = -1
            self.index[used:] = src
            self.a[src] = float("nan")
            rows_of = torch.where(self.index[:, None] >= 0, self.a[self.index.clamp_min(0).long()], 0)
        else:
            self.a = whole((rows, K), dtype, seed + 3)
            self.a[used:] = float("nan")
            rows_of = self.a
        self.shape = {"fwd": (rows, N), "rows": (rows, K), "weights": (n, N, K)}[dir]
        self.add = whole(self.shape, out, seed + 5) if add else None
        self.rows_of, self.out = rows_of.double(), DT[out]

    def check(self, offsets=None, groups=None, at=None, w=None):
        """The call on a workspace of NaN that ends where it says; rows of no group keep what they held."""
        groups, at, w = groups or self.groups, at or self.at, self.w if w is None else w
        need = moe.grouped_gemm_workspace(groups).nbytes
        ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
        ws[need:] = 171
        got = torch.full(self.shape, 777.0, dtype=self.out, device="cuda")
        call(self.dir, groups, self.a, self.d_out, w, self.offsets if offsets is None else offsets, got, self.index,
             self.add, ws[:need])
        assert (ws[need:] == 171).all()
        d_out = self.d_out.double()
        for e, (b, t) in enumerate(zip(at, at[1:])):
            here = e if self.dir == "weights" else slice(b, t)
            m = w[e].double()
            want = {"fwd": lambda: self.rows_of[b:t] @ m.T, "rows": lambda: d_out[b:t] @ m,
                    "weights": lambda: d_out[b:t].T @ self.rows_of[b:t]}[self.dir]()
            if self.add is not None:
                want += self.add[here].double()
            assert torch.equal(got[here], want.to(self.out)), e
        if self.dir != "weights":
            assert (got[:at[0]] == 777).all() and (got[at[-1]:] == 777).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dir,counts,N,K,dtype,shape,parts", CASES)
def test_whole_numbers_are_exact_in_every_shape(dir, counts, N, K, dtype, shape, parts):
    for out in results_of(dtype):
        for gather in (False, True)[:1 if dir == "rows" else 2]:
            for add in (False, True):
                Call(dir, counts, N, K, dtype, out, gather, add, seed=N).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dir,counts,N,K,dtype,out,shape,parts", SLICES)
def test_a_slice_of_the_groups_in_parts(dir, counts, N, K, dtype, out, shape, parts):
    """Offsets that start behind the first row and a reduction in parts: the rows in front and behind stay."""
    for add in (False, True):
        c = Call(dir, counts, N, K, dtype, out, False, add, seed=K)
        rows = sum(counts) + SPARE
        c.check(c.offsets[1:3].clone(), moe.make_groups(1, rows, N, K, dtype, out), c.at[1:3], c.w[1:2])


@pytest.mark.gpu
@pytest.mark.parametrize("dir,rows,n,dtype,gather", [
    ("fwd", 1 << 29, 3, "f32", False), ("rows", 1 << 29, 100, "f32", False), ("fwd", 1 << 30, 100, "bf16", False),
    ("rows", 1 << 30, 3, "bf16", False), ("fwd", (1 << 29) + 77, 1024, "bf16", True)])
def test_more_tile_rows_than_a_grid_dimension_holds(dir, rows, n, dtype, gather):
    """2^23 tiles and more, whose threads are 2^31 and more: every row of 8 values, in several launches."""
    N = K = 8
    counts = torch.randint(0, 2 * (rows // n), (n,), generator=torch.Generator().manual_seed(n))
    counts[n // 2] = 0
    while counts.sum() > rows - 50:
        counts //= 2
    counts[-1] += rows - 50 - counts.sum()
    offsets = torch.zeros(n + 1, dtype=torch.int64)
    offsets[1:] = counts.cumsum(0)
    src = 1000 if gather else rows
    a, w = torch.empty(src, 8, dtype=DT[dtype], device="cuda").random_(-3, 4), whole((n, N, K), dtype, 1)
    index = torch.empty(rows, dtype=torch.int32, device="cuda").random_(0, src) if gather else None
    out = torch.full((rows, 8), 777.0, dtype=DT[dtype], device="cuda")
    call(dir, moe.make_groups(n, rows, N, K, dtype), a, a, w, offsets.int().cuda(), out, index)
    at, m = offsets.tolist(), w.float()
    for e, (b, t) in enumerate(zip(at, at[1:])):
        for r in range(b, t, 1 << 24):
            r = slice(r, min(t, r + (1 << 24)))
            x = (a[index[r].long()] if gather else a[r]).float()
            assert torch.equal(out[r], (x @ (m[e].T if dir == "fwd" else m[e])).to(DT[dtype])), (e, r)
    assert (out[at[-1]:] == 777).all()
    del a, index, out, x
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_more_tiles_of_weights_than_a_grid_dimension_holds(out):
    """2^23 tiles of the weights' gradient, 8 x 2^20 in each of 1024 groups."""
    n, rows, N, K = 1024, 100, 8, 1 << 20
    d_out, a = whole((rows, N), "bf16", 1), whole((rows, K), "bf16", 2)
    at = [0] * 300 + [40] * 500 + [99] * 225
    got = torch.full((n, N, K), 777.0, dtype=DT[out], device="cuda")
    call("weights", moe.make_groups(n, rows, N, K, "bf16", out), a, d_out, None,
         torch.tensor(at, dtype=torch.int32, device="cuda"), got)
    for e in (299, 799):
        b, t = at[e:e + 2]
        assert torch.equal(got[e], (d_out[b:t].float().T @ a[b:t].float()).to(DT[out]))
        got[e] = 0
    assert not any(got[e:e + 64].any() for e in range(0, n, 64))
    del got
    torch.cuda.empty_cache()
