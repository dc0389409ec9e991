// Ragged grouped GEMM on microscaled 4-bit operands (formats in mx.hpp), gfx950 MFMA.
//
//   SwiGLU launch: h = silu(a W_gate^T) * (a W_up^T), quantised again to 4-bit rows;
//   plain launch:  out = a W^T.
// Both sum code products in fp32 through the 32x32x64 scaled MFMA, which multiplies each
// 32-value block of a row by the two blocks' powers of two, so nothing is decoded first.
// (Measured on register operands: 32x32x64 7.0 PFLOP/s with one wave per SIMD and 7.9 with
// more, 16x16x128 only 2.5 and 4.3.)
//
// A wave holds two pairs of 16-channel fragments (SwiGLU: one of W_gate and the same one of
// W_up, whose 32 channels are one block of h) against up to MU units of 32 token rows.
// Weight runs go from memory into registers as the A operand, four steps (one 512-value
// group) ahead, each reloaded as soon as it has been used; token records are in LDS as the
// B operand, shared by the workgroup's waves, where they arrive straight from memory.
//   resident: the tile's rows stay in LDS over their whole width, and the workgroup runs over a
//             range of channels without a barrier, the next block's weights requested before the
//             last one's results are stored (in the down launch's tall tiles, 22 to 24 spilled registers
//             are reloaded before the stores, which waits for those requests);
//   ring:     rows too wide for that pass through a ring of LDS buffers, one group each; a
//             workgroup does one block of channels.
// Two workgroups of 4 waves per CU cover each other's beginnings and ends.
//
// Measured, 64 experts of D 4096 and I 1024 (428 MB of weights).  10 rows each: gate/up 44 us, down 25 us,
// 6.5 and 6.0 TB/s, bound by the weights' bytes; 50 rows 47 and 31.  160 rows each (258 GFLOP): gate/up 80 us, of which its
// MFMAs alone take 45 and everything but them 76; the weights come from memory once and
// through L2 twice (two M-tiles), and waves wait for the slowest at each group's barrier;
// down 48 us, 4.9 TB/s of which a third is the rows written.  Deeper rings (8 waves, 4 buffers), another order
// of the steps per wave, other parts of the channels, both tiles in one workgroup of 8 waves (83 and 58 us) and
// 64-row resident tiles (105 and 56) were no faster; one 256-row tile with one wave per SIMD took 75 us for
// gate/up here and 123 against 101 at 240 rows each.
// A group's rows are split evenly over the M-tiles it needs, so that no tile streams the
// weights for a few rows only.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"
#include "mx.hpp"

namespace moe {

namespace {

typedef uint32_t u32;
constexpr int kPairs = 2;                    // pairs of weight fragments (32 channels) per wave
constexpr int kUnitRows = 32;                // token rows per unit
constexpr int kWaves = 4;                    // per workgroup, two workgroups per CU
constexpr int kResidentBytes = 70 * 1024;    // LDS rows of a resident tile: two workgroups per CU
constexpr int kRing = 2;                     // LDS buffers of the ring
constexpr int kGroupLoads = 5 * 2 * kPairs;  // a wave's weight loads per group: four steps and the scales
enum : int { OUT_MX = 16 };                  // output: 4-bit rows (SwiGLU launches)

constexpr int mx_bn(bool swiglu) { return kWaves * (swiglu ? kPairs / 2 : kPairs) * 32; }

typedef float f32x16 __attribute__((ext_vector_type(16)));

// c += A B for half a step (64 values); byte S of the scale dwords belongs to it.  Lane l holds row
// (A) or column (B) l % 32, values (l / 32) * 32 .. + 31, and that block's scale.
template <int S>
__device__ __forceinline__ f32x16 mx_mfma(const u32x4& a, const u32x4& b, f32x16 c, u32 sa, u32 sb) {
  const u32x4 z = {0u, 0u, 0u, 0u};  // fp4 operands use the first four registers
  const i32x8 av = __builtin_bit_cast(i32x8, __builtin_shufflevector(a, z, 0, 1, 2, 3, 4, 5, 6, 7));
  const i32x8 bv = __builtin_bit_cast(i32x8, __builtin_shufflevector(b, z, 0, 1, 2, 3, 4, 5, 6, 7));
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, S, static_cast<int>(sa), S,
                                                         static_cast<int>(sb));
}

// One matrix: offsets from 2^31 on read zeros and touch no memory (a matrix is smaller).
constexpr u32 kOutOfRange = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t matrix_rsrc(const void* base) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const u32 lo = static_cast<u32>(__builtin_amdgcn_readfirstlane(static_cast<u32>(a)));
  const u32 hi = static_cast<u32>(__builtin_amdgcn_readfirstlane(static_cast<u32>(a >> 32)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0,
                                           0x7FFFFFFF, 0x00020000);
}

// The tile of one workgroup: group, rows, and which part of the channels.
struct Tile {
  int g, part, row0, nrows;
  bool alone;  // the only M-tile of its group: nothing else reads its weights
};

// Tile L of the order (group, part of the channels, M-tile).
__device__ __forceinline__ Tile locate(const MxGemm& p, int L, int parts) {
  // the group: how many of prefix[1 ..] are at most q, 64 at a time (a search would be a chain of loads)
  const int q = L / parts, lane = threadIdx.x % kWave;
  int lo = 0;
  for (int g0 = 0; g0 < p.n_groups; g0 += kWave) {
    const int n = __popcll(__ballot(g0 + lane < p.n_groups && p.tile_prefix[g0 + lane + 1] <= q));
    lo += n;
    if (n < kWave) break;
  }
  Tile t;
  t.g = __builtin_amdgcn_readfirstlane(lo);
  const int pg = ld_scalar(p.tile_prefix + t.g);
  const int mt = ld_scalar(p.tile_prefix + t.g + 1) - pg;
  const int local = L - pg * parts;
  t.part = __builtin_amdgcn_readfirstlane(local / mt);
  const int beg = ld_scalar(p.offsets + t.g), count = ld_scalar(p.offsets + t.g + 1) - beg;
  // whole units, the same number in every tile but the last
  const int per = ((count + mt - 1) / mt + kUnitRows - 1) / kUnitRows * kUnitRows;
  const int r = __builtin_amdgcn_readfirstlane(local % mt) * per;
  t.row0 = beg + r;
  t.nrows = min(per, count - r);
  t.alone = mt == 1;
  return t;
}

// Weights that only one tile reads bypass the caches' replacement (NT): 64 experts of 50 rows took 47 us for
// gate/up and 31 for down, 59 and 34 without; with two tiles per expert, which share them in L2, it
// is 97 against 81 (160 rows each), and short tiles of 16 experts of 1024 x 512 at 125 rows 9.4 against 7.9.
//
// A wave's weights: pairs of fragments, of both matrices or of one, from channel ncol on.  Half j of a
// step is its blocks 2 j and 2 j + 1: lanes l % 32 < 16 the pair's first fragment, the others its
// second, two pieces of 512 contiguous bytes per load.
template <bool SWIGLU, bool NT>
struct Weights {
  static constexpr int NMAT = SWIGLU ? 2 : 1;
  __amdgpu_buffer_rsrc_t res[NMAT];
  int S, G, N;
  u32 frag_bytes, lane_at, lane_sc;
  u32 at[kPairs];  // byte offset of each pair
  bool on;         // any channel left
  __device__ __forceinline__ Weights(const MxGemm& p, int g, int lane) : S(mx_steps(p.K)), G(mx_groups(p.K)), N(p.N) {
    frag_bytes = static_cast<u32>(mx_fragment_bytes(p.K));
    const u32 second = ((lane >> 4) & 1) * frag_bytes, place = (lane >> 5) * 16 + (lane & 15);
    lane_at = second + place * 16;
    lane_sc = second + place * 4;
    res[0] = matrix_rsrc(static_cast<const uint8_t*>(p.w0) + static_cast<size_t>(g) * p.w_stride);
    if (SWIGLU) res[NMAT - 1] = matrix_rsrc(static_cast<const uint8_t*>(p.w1) + static_cast<size_t>(g) * p.w_stride);
  }
  __device__ __forceinline__ void seek(int ncol, bool there) {
    on = there;
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      const int frag = ncol / 16 + (SWIGLU ? 0 : 2 * q);
      at[q] = static_cast<u32>(min(frag, N / 16 - 2)) * frag_bytes;
    }
  }
  __device__ __forceinline__ void load(u32x4 (&w)[kPairs][2], int grp, int s) const {
    const u32 v = on && grp * 4 + s < S ? lane_at : kOutOfRange;
#pragma unroll
    for (int q = 0; q < kPairs; ++q)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[q][j] = buffer_load16<NT>(res[SWIGLU ? q : 0], v, at[q] + grp * kMxGroupBytes + s * kMxRun + j * 512);
  }
  __device__ __forceinline__ void load_scales(u32 (&sc)[kPairs][2], int grp) const {
    const u32 v = on && grp < G ? lane_sc : kOutOfRange;
    const u32 o = grp * kMxGroupBytes + min(4, S - 4 * grp) * kMxRun;
#pragma unroll
    for (int q = 0; q < kPairs; ++q)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        sc[q][j] = __builtin_amdgcn_raw_buffer_load_b32(res[SWIGLU ? q : 0], v, at[q] + o + j * 128, 0);
  }
};

// One group of the products: acc += w (records at rec, the lane's row), each step's registers refilled
// by next(s) after their use.  MU is the number of units that the tile has, a constant.
template <int MU, typename Next>
__device__ __forceinline__ void group_products(f32x16 (&acc)[kPairs][MU], u32x4 (&w)[4][kPairs][2],
                                               const u32 (&sc)[kPairs][2], const uint8_t* rec, int steps, int half,
                                               Next next) {
  u32 bs[MU][2];
#pragma unroll
  for (int m = 0; m < MU; ++m)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      bs[m][j] = *reinterpret_cast<const u32*>(rec + m * kUnitRows * kMxRecord + 256 + j * 8 + half * 4);
  // Pieces (step, unit, half) are read kAhead before their products, over the ends of the steps too;
  // the scheduling barriers keep it at that, all of them would not fit the registers.
  constexpr int kAhead = 2, kRead = kAhead + 1, kPer = 2 * MU;
  u32x4 b[kRead];
  auto read = [&](int i) {
    const int s = i / kPer, q = i % kPer;
    b[i % kRead] =
        *reinterpret_cast<const u32x4*>(rec + (q >> 1) * kUnitRows * kMxRecord + s * 64 + (q & 1) * 32 + half * 16);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) read(i);
  auto step = [&](auto sc_c) {
    constexpr int s = decltype(sc_c)::value;
    if (s < steps) {
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int i = s * kPer + q, m = q >> 1, j = q & 1;
        if (i + kAhead < 4 * kPer) read(i + kAhead);
#pragma unroll
        for (int f = 0; f < kPairs; ++f)
          acc[f][m] = mx_mfma<s>(w[s][f][j], b[i % kRead], acc[f][m], sc[f][j], bs[m][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    next(s);
  };
  step(std::integral_constant<int, 0>{});
  step(std::integral_constant<int, 1>{});
  step(std::integral_constant<int, 2>{});
  step(std::integral_constant<int, 3>{});
}

// f(integral_constant n) for the n = 1 .. MU in use.
template <int MU, typename F>
__device__ __forceinline__ void with_units(int n, F f) {
  if constexpr (MU == 1) {
    f(std::integral_constant<int, 1>{});
  } else {
    if (n == MU) f(std::integral_constant<int, MU>{});
    else with_units<MU - 1>(n, f);
  }
}

// Exchange a of lanes 32 .. 63 with b of lanes 0 .. 31: then lanes below 32 hold (a, the other half's a),
// the lanes above (the other half's b, b).
__device__ __forceinline__ void swap_halves(u32& a, u32& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// Plain results pass through LDS, 16 rows of 128 bytes at a time in a place of each wave's own, and go
// out as whole lines (stored from where the MFMA leaves them, 16 bytes here and there, they took
// twice the time).
constexpr int kStageRow = 128 + 16;
constexpr int kStage = 16 * kStageRow;

// Rows r0 .. r0 + 15 (of nrows) of the stage -> row r of the output at out + r * stride.
__device__ __forceinline__ void flush_stage(const uint8_t* stage, uint8_t* out, size_t stride, int r0, int nrows, int lane) {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = i * 8 + lane / 8;
    const u32x4 v = *reinterpret_cast<const u32x4*>(stage + r * kStageRow + (lane & 7) * 16);
    if (r0 + r < nrows) *reinterpret_cast<u32x4*>(out + static_cast<size_t>(r0 + r) * stride + (lane & 7) * 16) = v;
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// A wave's results for its channels ncol0 .. -> memory.  Lane l holds column (token) l % 32 and, in
// element 4 i + k, channel 8 i + 4 (l / 32) + k of the pair's 32.
template <int MU, bool SWIGLU, int OUT>
__device__ __forceinline__ void store_tile(const MxGemm& p, const f32x16 (&acc)[kPairs][MU], int row0, int nrows,
                                           int ncol0, int lane, uint8_t* stage) {
  if (ncol0 >= p.N) return;
  const int half = lane >> 5;
#pragma unroll
  for (int m = 0; m < MU; ++m) {
    const int r = m * kUnitRows + (lane & 31);
    const bool live = r < nrows;
    const int64_t grow = row0 + r;
    if constexpr (SWIGLU) {
      // the pair's 32 channels are one block, in two lanes
      float v[2][8];
      u32 mx = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float h = silu(acc[0][m][i]) * acc[1][m][i];
        v[i / 8][i % 8] = h;
        mx = max(mx, mx_abs_bits(h));
      }
      mx = max(mx, static_cast<u32>(__shfl_xor(static_cast<int>(mx), 32, kWave)));
      const u32 byte = mx_scale_byte(mx);
      u32 a = 0, b = 0;  // codes of channels 8 i + 4 half + 0 .. 3, i = 0, 1 and i = 2, 3
      if (byte != 255u) {
        const float inv = mx_inverse_scale(byte);
        a = mx_codes8(v[0], inv);
        b = mx_codes8(v[1], inv);
      }
      swap_halves(a, b);
      if (live) {
        const int blk = ncol0 / 32, bi = blk & 15;
        uint8_t* rec = static_cast<uint8_t*>(p.out) + grow * mx_row_bytes(p.N) + static_cast<int64_t>(blk / 16) * kMxRecord;
        *reinterpret_cast<uint2*>(rec + bi * 16 + half * 8) =
            make_uint2((a & 0xFFFFu) | (b << 16), (a >> 16) | (b & 0xFFFF0000u));
        if (half == 0) rec[256 + (bi & 3) * 4 + (bi >> 2)] = static_cast<uint8_t>(byte);
        if (ncol0 + 32 == p.N && p.N % kMxStep != 0) {
          // two more blocks fill the last step with zeros
#pragma unroll
          for (int e = 1; e <= 2; ++e) {
            const int z = bi + e;
            *reinterpret_cast<uint2*>(rec + z * 16 + half * 8) = make_uint2(0u, 0u);
            if (half == 0) rec[256 + (z & 3) * 4 + (z >> 2)] = 127;
          }
        }
      }
    } else {
      // the wave's 64 channels are all there (N is a multiple of 64)
      constexpr int es = OUT == EL_F32 ? 4 : 2;
      uint8_t* out = static_cast<uint8_t*>(p.out) + (static_cast<size_t>(row0) * p.N + ncol0) * es;
      const size_t stride = static_cast<size_t>(p.N) * es;
      uint8_t* at = stage + (lane & 15) * kStageRow;
#pragma unroll
      for (int part = 0; part < 2; ++part) {  // rows 0 .. 15 and 16 .. 31 of the unit
        const bool mine = ((lane >> 4) & 1) == part;
        if constexpr (OUT == EL_F32) {
#pragma unroll
          for (int f = 0; f < kPairs; ++f) {
            if (mine)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(at + (2 * i + half) * 16) =
                    make_float4(acc[f][m][4 * i], acc[f][m][4 * i + 1], acc[f][m][4 * i + 2], acc[f][m][4 * i + 3]);
            flush_stage(stage, out + f * 128, stride, m * kUnitRows + part * 16, nrows, lane);
          }
        } else {
#pragma unroll
          for (int f = 0; f < kPairs; ++f)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              // lanes below 32 get channels 8 i .. + 7, the lanes above the eight after them
              const f32x16& o = acc[f][m];
              u32 a0 = bf16x2_bits(o[4 * i], o[4 * i + 1]), a1 = bf16x2_bits(o[4 * i + 2], o[4 * i + 3]);
              u32 b0 = bf16x2_bits(o[4 * i + 4], o[4 * i + 5]), b1 = bf16x2_bits(o[4 * i + 6], o[4 * i + 7]);
              swap_halves(a0, b0);
              swap_halves(a1, b1);
              if (mine) *reinterpret_cast<uint4*>(at + (f * 4 + i + half) * 16) = make_uint4(a0, a1, b0, b1);
            }
          flush_stage(stage, out, stride, m * kUnitRows + part * 16, nrows, lane);
        }
      }
    }
  }
}

constexpr int kPieces = kMxRecord / 16;  // 16-byte pieces of a record

// Token records of one group of the tile's rows into LDS, straight from memory: piece i of the tile (row
// i / 17) at 16 * i.  Every thread's pieces are the same in every group, so their rows' offsets are
// looked up once.  Rows of the last unit past the tile's are left as they are: they are columns
// that are never stored.
template <int MU>
struct RowLoader {
  static constexpr int NP = (MU * kUnitRows * kPieces + kWaves * kWave - 1) / (kWaves * kWave);
  __amdgpu_buffer_rsrc_t res;
  u32 off[NP];
  int pieces;
  __device__ __forceinline__ RowLoader(const MxGemm& p, const Tile& t, u32 row_bytes) {
    pieces = t.nrows * kPieces;
    res = buffer_rsrc(p.a);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = threadIdx.x + i * kWaves * kWave;
      const int gr = t.row0 + min(c / kPieces, t.nrows - 1);
      off[i] = static_cast<u32>(p.perm ? p.perm[gr] : gr) * row_bytes + (c % kPieces) * 16;
    }
  }
  __device__ __forceinline__ void load(uint8_t* dst, int grp) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (static_cast<int>(threadIdx.x) + i * kWaves * kWave < pieces)
        buffer_load16_to_lds(res, dst + (wave + i * kWaves) * 1024, off[i], grp * kMxRecord);
  }
};

template <int MF, bool SWIGLU, int OUT, bool NT>
__device__ __forceinline__ void resident_tile(const MxGemm& p, const Tile& t, uint8_t* lds) {
  constexpr int BN = mx_bn(SWIGLU), kBuf = MF * kUnitRows * kMxRecord;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int blocks = (p.N + BN - 1) / BN;  // of channels; this workgroup takes [b0, b1)
  const int b0 = blocks * t.part / p.parts, b1 = blocks * (t.part + 1) / p.parts;
  if (b0 == b1) return;
  Weights<SWIGLU, NT> wt(p, t.g, lane);
  const int S = wt.S, G = wt.G, wcol = wave * (BN / kWaves);
  {
    const RowLoader<MF> rows(p, t, static_cast<u32>(mx_row_bytes(p.K)));
    for (int g = 0; g < G; ++g) rows.load(lds + g * kBuf, g);
  }
  __builtin_amdgcn_sched_barrier(0);  // the waits below count on the rows' loads being the older ones
  const uint8_t* rec = lds + (lane & 31) * kMxRecord;
  with_units<MF>((t.nrows + kUnitRows - 1) / kUnitRows, [&](auto n_c) {
    constexpr int MU = decltype(n_c)::value;
    u32x4 w[4][kPairs][2];
    u32 sc[kPairs][2], nsc[kPairs][2];
    wt.seek(b0 * BN + wcol, true);
    wt.load_scales(sc, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) wt.load(w[s], 0, s);
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<kGroupLoads>();
    bare_barrier();
    for (int b = b0; b < b1; ++b) {
      f32x16 acc[kPairs][MU] = {};
      for (int g = 0; g < G; ++g) {
        const bool last = g + 1 == G;
        const int gn = last ? 0 : g + 1;
        if (last) wt.seek((b + 1) * BN + wcol, b + 1 < b1);
        wt.load_scales(nsc, gn);
        group_products<MU>(acc, w, sc, rec + g * kBuf, S - 4 * g, lane >> 5, [&](int s) {
          __builtin_amdgcn_sched_barrier(0);
          wt.load(w[s], gn, s);
          __builtin_amdgcn_sched_barrier(0);
        });
#pragma unroll
        for (int q = 0; q < kPairs; ++q)
#pragma unroll
          for (int j = 0; j < 2; ++j) sc[q][j] = nsc[q][j];
      }
      store_tile<MU, SWIGLU, OUT>(p, acc, t.row0, t.nrows, b * BN + wcol, lane, lds + G * kBuf + wave * kStage);
    }
  });
}

template <int MF, bool SWIGLU, int OUT>
__global__ __launch_bounds__(kWaves * 64, 2) void mx_resident_kernel(MxGemm p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int total = ld_scalar(p.tile_prefix + p.n_groups) * p.parts;
  if (static_cast<int>(blockIdx.x) >= total) return;
  const Tile t = locate(p, xcd_remap(blockIdx.x, total), p.parts);
  if (t.alone) resident_tile<MF, SWIGLU, OUT, true>(p, t, lds);
  else resident_tile<MF, SWIGLU, OUT, false>(p, t, lds);
}

template <int MF, bool SWIGLU, int OUT, bool NT>
__device__ __forceinline__ void ring_tile(const MxGemm& p, const Tile& t, uint8_t* lds) {
  constexpr int BN = mx_bn(SWIGLU), kBuf = MF * kUnitRows * kMxRecord;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  Weights<SWIGLU, NT> wt(p, t.g, lane);
  const int S = wt.S, G = wt.G, ncol0 = t.part * BN + wave * (BN / kWaves);
  const RowLoader<MF> rows(p, t, static_cast<u32>(mx_row_bytes(p.K)));
  constexpr int kLead = kRing - 1;  // groups of rows requested ahead
#pragma unroll
  for (int g = 0; g < kLead; ++g)
    if (g < G) rows.load(lds + g * kBuf, g);
  __builtin_amdgcn_sched_barrier(0);
  const uint8_t* rec = lds + (lane & 31) * kMxRecord;
  with_units<MF>((t.nrows + kUnitRows - 1) / kUnitRows, [&](auto n_c) {
    constexpr int MU = decltype(n_c)::value;
    u32x4 w[4][kPairs][2];
    u32 sc[kPairs][2], nsc[kPairs][2];
    wt.seek(ncol0, true);
    wt.load_scales(sc, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) wt.load(w[s], 0, s);
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<kGroupLoads>();  // the first kLead groups' rows
    bare_barrier();
    f32x16 acc[kPairs][MU] = {};
    for (int g = 0; g < G; ++g) {
      // buffer (g + kLead) % kRing was last read in group g - 1, which ended with a barrier
      if (g + kLead < G) rows.load(lds + (g + kLead) % kRing * kBuf, g + kLead);
      __builtin_amdgcn_sched_barrier(0);
      wt.load_scales(nsc, g + 1);
      group_products<MU>(acc, w, sc, rec + g % kRing * kBuf, S - 4 * g, lane >> 5, [&](int s) {
        __builtin_amdgcn_sched_barrier(0);
        wt.load(w[s], g + 1, s);
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int q = 0; q < kPairs; ++q)
#pragma unroll
        for (int j = 0; j < 2; ++j) sc[q][j] = nsc[q][j];
      // group g + 1's rows were requested before this group's weight loads, which may stay in flight
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<kLead * kGroupLoads>();
      bare_barrier();
    }
    store_tile<MU, SWIGLU, OUT>(p, acc, t.row0, t.nrows, ncol0, lane, lds + kRing * kBuf + wave * kStage);
  });
}

template <int MF, bool SWIGLU, int OUT>
__global__ __launch_bounds__(kWaves * 64, 2) void mx_ring_kernel(MxGemm p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRing * MF * kUnitRows * kMxRecord + (SWIGLU ? 0 : kWaves * kStage)];
  const int total = ld_scalar(p.tile_prefix + p.n_groups) * p.parts;
  if (static_cast<int>(blockIdx.x) >= total) return;
  const Tile t = locate(p, xcd_remap(blockIdx.x, total), p.parts);
  if (t.alone) ring_tile<MF, SWIGLU, OUT, true>(p, t, lds);
  else ring_tile<MF, SWIGLU, OUT, false>(p, t, lds);
}

// Into how many parts a resident tile's blocks of channels go, one workgroup each.  Tiles of one unit
// are bound by their weights and take as many workgroups as there are blocks (64 such tiles of 16
// blocks: 24.7 us, against 27.9 with half as many).  Taller ones cost about 0.7 of a block's time to
// begin with, and run in rounds of two workgroups per CU: 128 tiles of 16 blocks took 49 us in 4
// parts (one round), 52 in 8 and 58 in 16; 192 tiles 106 us in 3 parts (two rounds, the second
// almost empty), 91 in 5.
int resident_parts(int tiles, int blocks) {
  int best = 1;
  double least = 0.0;
  for (int parts = 1; parts <= blocks; ++parts) {
    const int rounds = (tiles * parts + 511) / 512;
    const double cost = rounds * (static_cast<double>((blocks + parts - 1) / parts) + 0.7);
    if (parts == 1 || cost < least) {
      best = parts;
      least = cost;
    }
  }
  return best;
}

template <int MF, bool SWIGLU, int OUT>
hipError_t launch_mf(MxGemm p, int m_tiles, hipStream_t stream) {
  const int lds = mx_groups(p.K) * MF * kUnitRows * kMxRecord;
  const int blocks = (p.N + mx_bn(SWIGLU) - 1) / mx_bn(SWIGLU);
  if (lds <= kResidentBytes) {
    p.parts = MF == 1 ? blocks : resident_parts(p.busy_tiles, blocks);
    hipLaunchKernelGGL((mx_resident_kernel<MF, SWIGLU, OUT>), dim3(m_tiles * p.parts), dim3(kWaves * 64),
                       lds + (SWIGLU ? 0 : kWaves * kStage), stream, p);
  } else {
    p.parts = blocks;
    hipLaunchKernelGGL((mx_ring_kernel<MF, SWIGLU, OUT>), dim3(m_tiles * p.parts), dim3(kWaves * 64), 0, stream, p);
  }
  return hipGetLastError();
}

template <bool SWIGLU, int OUT>
hipError_t launch_bm(int bm, const MxGemm& p, int m_tiles, hipStream_t stream) {
  switch (bm) {
    case 32: return launch_mf<1, SWIGLU, OUT>(p, m_tiles, stream);
    case 128: return launch_mf<4, SWIGLU, OUT>(p, m_tiles, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_mx_gemm(bool swiglu, int out_el, int bm, const MxGemm& p, int m_tiles, hipStream_t stream) {
  if (m_tiles == 0) return hipSuccess;
  if (swiglu) return launch_bm<true, OUT_MX>(bm, p, m_tiles, stream);
  return out_el == EL_F32 ? launch_bm<false, EL_F32>(bm, p, m_tiles, stream)
                          : launch_bm<false, EL_BF16>(bm, p, m_tiles, stream);
}

}  // namespace moe
