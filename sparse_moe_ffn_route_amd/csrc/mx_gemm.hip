// Ragged grouped GEMM on microscaled 4-bit operands (formats in mx.hpp), gfx950 MFMA.
//
//   SwiGLU launch: h = silu(a W_gate^T) * (a W_up^T), quantised again to 4-bit rows;
//   plain launch:  out = a W^T.
// Both sum code products in fp32 through the 16x16x128 scaled MFMA, which multiplies each
// 32-value block of a row by the two blocks' powers of two, so nothing is decoded first.
//
// A wave holds four fragments of 16 channels (SwiGLU: two of W_gate and the same two of W_up,
// whose 32 channels are one block of h) against up to MF fragments of 16 token rows.
// Weight runs go from memory into registers as the A operand, four steps (one 512-value
// group) ahead, each reloaded as soon as it has been used; token records are in LDS as the
// B operand, shared by the workgroup's waves, where they arrive straight from memory.
//   resident: the tile's rows stay in LDS over their whole width, and the workgroup (4 waves,
//             two per CU) runs over a range of channels without a barrier, its weight stream
//             unbroken from one block of channels to the next;
//   ring:     rows too wide for that pass through a ring of LDS buffers, one group each
//             (8 waves, one workgroup per CU); a workgroup does one block of channels.
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
constexpr int kFR = 4;                       // weight fragments per wave
constexpr int kResidentWaves = 4, kRingWaves = 8;
constexpr int kResidentBytes = 70 * 1024;    // LDS rows of a resident tile: two workgroups per CU
constexpr int kRing = 4;                     // LDS buffers of the ring
constexpr int kGroupLoads = 5 * kFR;         // a wave's weight loads per group: four steps and the scales
enum : int { OUT_MX = 16 };                  // output: 4-bit rows (SwiGLU launches)

constexpr int mx_bn(bool swiglu, int waves) { return waves * (swiglu ? kFR / 2 : kFR) * 16; }

// c += A B for one step; byte S of the scale dwords belongs to it.
template <int S>
__device__ __forceinline__ f32x4 mx_mfma(const u32x4& a, const u32x4& b, f32x4 c, u32 sa, u32 sb) {
  const u32x4 z = {0u, 0u, 0u, 0u};  // fp4 operands use the first four registers
  const i32x8 av = __builtin_bit_cast(i32x8, __builtin_shufflevector(a, z, 0, 1, 2, 3, 4, 5, 6, 7));
  const i32x8 bv = __builtin_bit_cast(i32x8, __builtin_shufflevector(b, z, 0, 1, 2, 3, 4, 5, 6, 7));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, S, static_cast<int>(sa), S,
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
};

// Tile L of the order (group, part of the channels, M-tile).
template <int BM>
__device__ __forceinline__ Tile locate(const MxGemm& p, int L, int parts) {
  int lo = 0, hi = p.n_groups - 1;
  const int q = L / parts;
  while (lo < hi) {  // largest g with prefix[g] <= q
    const int mid = (lo + hi + 1) >> 1;
    if (ld_scalar(p.tile_prefix + mid) <= q) lo = mid; else hi = mid - 1;
  }
  Tile t;
  t.g = __builtin_amdgcn_readfirstlane(lo);
  const int pg = ld_scalar(p.tile_prefix + t.g);
  const int mt = ld_scalar(p.tile_prefix + t.g + 1) - pg;
  const int local = L - pg * parts;
  t.part = __builtin_amdgcn_readfirstlane(local / mt);
  const int beg = ld_scalar(p.offsets + t.g), count = ld_scalar(p.offsets + t.g + 1) - beg;
  // whole fragments, the same number in every tile but the last
  const int per = ((count + mt - 1) / mt + 15) / 16 * 16;
  const int r = __builtin_amdgcn_readfirstlane(local % mt) * per;
  t.row0 = beg + r;
  t.nrows = min(per, count - r);
  return t;
}

// A wave's weights: fragments of both matrices from channel ncol on.
template <bool SWIGLU, bool NT>
struct Weights {
  static constexpr int NMAT = SWIGLU ? 2 : 1, NF = kFR / NMAT;
  __amdgpu_buffer_rsrc_t res[NMAT];
  int S, G, N;
  u32 frag_bytes;
  u32 at[NF];   // byte offset of each fragment
  bool on;      // any channel left
  __device__ __forceinline__ Weights(const MxGemm& p, int g) : S(mx_steps(p.K)), G(mx_groups(p.K)), N(p.N) {
    frag_bytes = static_cast<u32>(mx_fragment_bytes(p.K));
    res[0] = matrix_rsrc(static_cast<const uint8_t*>(p.w0) + static_cast<size_t>(g) * p.w_stride);
    if (SWIGLU) res[NMAT - 1] = matrix_rsrc(static_cast<const uint8_t*>(p.w1) + static_cast<size_t>(g) * p.w_stride);
  }
  __device__ __forceinline__ void seek(int ncol, bool there) {
    on = there;
#pragma unroll
    for (int f = 0; f < NF; ++f) at[f] = static_cast<u32>(min(ncol / 16 + f, N / 16 - 1)) * frag_bytes;
  }
  __device__ __forceinline__ void load(u32x4 (&w)[kFR], int grp, int s, int lane) const {
    const u32 v = on && grp * 4 + s < S ? lane * 16 : kOutOfRange;
#pragma unroll
    for (int a = 0; a < NMAT; ++a)
#pragma unroll
      for (int f = 0; f < NF; ++f) w[a * NF + f] = buffer_load16<NT>(res[a], v, at[f] + grp * kMxGroupBytes + s * kMxRun);
  }
  __device__ __forceinline__ void load_scales(u32 (&sc)[kFR], int grp, int lane) const {
    const u32 v = on && grp < G ? lane * 4 : kOutOfRange;
    const u32 o = grp * kMxGroupBytes + min(4, S - 4 * grp) * kMxRun;
#pragma unroll
    for (int a = 0; a < NMAT; ++a)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        sc[a * NF + f] = __builtin_amdgcn_raw_buffer_load_b32(res[a], v, at[f] + o, 0);
  }
};

// One group of the products: acc += w (records at rec), each step's registers refilled by next(s) after
// their use.  mf: fragments of rows in use.
template <int MF, typename Next>
__device__ __forceinline__ void group_products(f32x4 (&acc)[kFR][MF], u32x4 (&w)[4][kFR], const u32 (&sc)[kFR],
                                               const uint8_t* rec, int steps, int mf, int lgrp, Next next) {
  u32 bs[MF];
#pragma unroll
  for (int m = 0; m < MF; ++m) bs[m] = *reinterpret_cast<const u32*>(rec + m * 16 * kMxRecord + 256 + lgrp * 4);
  auto step = [&](auto sc_c) {
    constexpr int s = decltype(sc_c)::value;
    if (s < steps) {
      u32x4 b = *reinterpret_cast<const u32x4*>(rec + s * 64 + lgrp * 16);
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        // the next fragment is read before this one's products
        u32x4 bn = b;
        if (m + 1 < MF) bn = *reinterpret_cast<const u32x4*>(rec + (m + 1) * 16 * kMxRecord + s * 64 + lgrp * 16);
        if (m == 0 || m < mf) {
#pragma unroll
          for (int f = 0; f < kFR; ++f) acc[f][m] = mx_mfma<s>(w[s][f], b, acc[f][m], sc[f], bs[m]);
        }
        b = bn;
      }
    }
    next(s);
  };
  step(std::integral_constant<int, 0>{});
  step(std::integral_constant<int, 1>{});
  step(std::integral_constant<int, 2>{});
  step(std::integral_constant<int, 3>{});
}

// A wave's results for its channels ncol0 .. -> memory.
template <int MF, bool SWIGLU, int OUT>
__device__ __forceinline__ void store_tile(const MxGemm& p, const f32x4 (&acc)[kFR][MF], int row0, int nrows, int ncol0,
                                           int lane) {
  constexpr int NF = kFR / (SWIGLU ? 2 : 1);
  if (ncol0 >= p.N) return;
  const int lrow = lane & 15, lgrp = lane >> 4;
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    const int r = m * 16 + lrow;
    if (m * 16 >= nrows) break;
    const bool live = r < nrows;
    const int64_t grow = row0 + r;
    if constexpr (SWIGLU) {
      // the wave's 32 channels are one block: lane group lgrp holds channels 4 lgrp .. + 3 of
      // both fragments, the four groups of a token reduce the block's largest magnitude
      float v[8];
      u32 mx = 0;
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[f * 4 + i] = silu(acc[f][m][i]) * acc[NF + f][m][i];
          mx = max(mx, mx_abs_bits(v[f * 4 + i]));
        }
      mx = max(mx, static_cast<u32>(__shfl_xor(static_cast<int>(mx), 16, kWave)));
      mx = max(mx, static_cast<u32>(__shfl_xor(static_cast<int>(mx), 32, kWave)));
      const u32 byte = mx_scale_byte(mx);
      const u32 codes = byte == 255u ? 0u : mx_codes8(v, mx_inverse_scale(byte));
      if (live) {
        const int b = ncol0 / 32, bi = b & 15;
        uint8_t* rec = static_cast<uint8_t*>(p.out) + grow * mx_row_bytes(p.N) + static_cast<int64_t>(b / 16) * kMxRecord;
        *reinterpret_cast<uint16_t*>(rec + bi * 16 + lgrp * 2) = static_cast<uint16_t>(codes);
        *reinterpret_cast<uint16_t*>(rec + bi * 16 + 8 + lgrp * 2) = static_cast<uint16_t>(codes >> 16);
        if (lgrp == 0) rec[256 + (bi & 3) * 4 + (bi >> 2)] = static_cast<uint8_t>(byte);
        if (ncol0 + 32 == p.N && p.N % kMxStep != 0) {
          // two more blocks fill the last step with zeros
#pragma unroll
          for (int e = 1; e <= 2; ++e) {
            const int z = bi + e;
            *reinterpret_cast<u32*>(rec + z * 16 + lgrp * 4) = 0u;
            if (lgrp == 0) rec[256 + (z & 3) * 4 + (z >> 2)] = 127;
          }
        }
      }
    } else if (live) {
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        if (ncol0 + f * 16 >= p.N) continue;
        const size_t idx = static_cast<size_t>(grow) * p.N + ncol0 + f * 16 + lgrp * 4;
        const f32x4 o = acc[f][m];
        if constexpr (OUT == EL_F32)
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + idx) = make_float4(o[0], o[1], o[2], o[3]);
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + idx) =
              make_uint2(bf16x2_bits(o[0], o[1]), bf16x2_bits(o[2], o[3]));
      }
    }
  }
}

constexpr int kPieces = kMxRecord / 16;  // 16-byte pieces of a record

// Token records of one group of the tile's fragments into LDS, straight from memory: piece i of the
// tile (row i / 17) at 16 * i.  Every thread's pieces are the same in every group, so their rows'
// offsets are looked up once; rows past the tile's last re-read it.
template <int MF, int NW>
struct RowLoader {
  static constexpr int NP = (MF * 16 * kPieces + NW * kWave - 1) / (NW * kWave);
  __amdgpu_buffer_rsrc_t res;
  u32 off[NP];
  int pieces;
  __device__ __forceinline__ RowLoader(const MxGemm& p, const Tile& t, u32 row_bytes) {
    pieces = (t.nrows + 15) / 16 * 16 * kPieces;
    res = buffer_rsrc(p.a);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = threadIdx.x + i * NW * kWave;
      const int gr = t.row0 + min(c / kPieces, t.nrows - 1);
      off[i] = static_cast<u32>(p.perm ? p.perm[gr] : gr) * row_bytes + (c % kPieces) * 16;
    }
  }
  __device__ __forceinline__ void load(uint8_t* dst, int grp) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (static_cast<int>(threadIdx.x) + i * NW * kWave < pieces)
        buffer_load16_to_lds(res, dst + (wave + i * NW) * 1024, off[i], grp * kMxRecord);
  }
};

template <int MF, bool SWIGLU, int OUT>
__global__ __launch_bounds__(kResidentWaves * 64, 2) void mx_resident_kernel(MxGemm p) {
  constexpr int BM = 16 * MF, NW = kResidentWaves, BN = mx_bn(SWIGLU, NW);
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int total = ld_scalar(p.tile_prefix + p.n_groups) * p.parts;
  if (static_cast<int>(blockIdx.x) >= total) return;
  const Tile t = locate<BM>(p, xcd_remap(blockIdx.x, total), p.parts);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int mf = (t.nrows + 15) / 16;
  const int blocks = (p.N + BN - 1) / BN;  // of channels; this workgroup takes [b0, b1)
  const int b0 = blocks * t.part / p.parts, b1 = blocks * (t.part + 1) / p.parts;
  if (b0 == b1) return;
  Weights<SWIGLU, MF <= 2> wt(p, t.g);
  const int S = wt.S, G = wt.G, wcol = wave * (BN / NW);
  {
    const RowLoader<MF, NW> rows(p, t, static_cast<u32>(mx_row_bytes(p.K)));
    for (int g = 0; g < G; ++g) rows.load(lds + g * (BM * kMxRecord), g);
  }
  __builtin_amdgcn_sched_barrier(0);  // the waits below count on the rows' loads being the older ones
  u32x4 w[4][kFR];
  u32 sc[kFR], nsc[kFR];
  wt.seek(b0 * BN + wcol, true);
  wt.load_scales(sc, 0, lane);
#pragma unroll
  for (int s = 0; s < 4; ++s) wt.load(w[s], 0, s, lane);
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<kGroupLoads>();
  bare_barrier();
  for (int b = b0; b < b1; ++b) {
    f32x4 acc[kFR][MF];
#pragma unroll
    for (int f = 0; f < kFR; ++f)
#pragma unroll
      for (int m = 0; m < MF; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int g = 0; g < G; ++g) {
      const bool last = g + 1 == G;
      const int gn = last ? 0 : g + 1;
      if (last) wt.seek((b + 1) * BN + wcol, b + 1 < b1);
      wt.load_scales(nsc, gn, lane);
      group_products<MF>(acc, w, sc, lds + g * (BM * kMxRecord) + lrow * kMxRecord, S - 4 * g, mf, lgrp, [&](int s) {
        __builtin_amdgcn_sched_barrier(0);
        wt.load(w[s], gn, s, lane);
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int f = 0; f < kFR; ++f) sc[f] = nsc[f];
    }
    store_tile<MF, SWIGLU, OUT>(p, acc, t.row0, t.nrows, b * BN + wcol, lane);
  }
}

template <int MF, bool SWIGLU, int OUT>
__global__ __launch_bounds__(kRingWaves * 64, 2) void mx_ring_kernel(MxGemm p) {
  constexpr int BM = 16 * MF, NW = kRingWaves, BN = mx_bn(SWIGLU, NW), kBuf = BM * kMxRecord;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRing * kBuf];
  const int total = ld_scalar(p.tile_prefix + p.n_groups) * p.parts;
  if (static_cast<int>(blockIdx.x) >= total) return;
  const Tile t = locate<BM>(p, xcd_remap(blockIdx.x, total), p.parts);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int mf = (t.nrows + 15) / 16;
  Weights<SWIGLU, false> wt(p, t.g);
  const int S = wt.S, G = wt.G, ncol0 = t.part * BN + wave * (BN / NW);
  const RowLoader<MF, NW> rows(p, t, static_cast<u32>(mx_row_bytes(p.K)));
  constexpr int kLead = kRing - 1;  // groups of rows requested ahead
#pragma unroll
  for (int g = 0; g < kLead; ++g)
    if (g < G) rows.load(lds + g * kBuf, g);
  __builtin_amdgcn_sched_barrier(0);
  u32x4 w[4][kFR];
  u32 sc[kFR], nsc[kFR];
  wt.seek(ncol0, true);
  wt.load_scales(sc, 0, lane);
#pragma unroll
  for (int s = 0; s < 4; ++s) wt.load(w[s], 0, s, lane);
  f32x4 acc[kFR][MF];
#pragma unroll
  for (int f = 0; f < kFR; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<kGroupLoads>();  // the first kLead groups' rows
  bare_barrier();
  for (int g = 0; g < G; ++g) {
    // buffer (g + kLead) % kRing was last read in group g - 1, which ended with a barrier
    if (g + kLead < G) rows.load(lds + (g + kLead) % kRing * kBuf, g + kLead);
    __builtin_amdgcn_sched_barrier(0);
    wt.load_scales(nsc, g + 1, lane);
    group_products<MF>(acc, w, sc, lds + g % kRing * kBuf + lrow * kMxRecord, S - 4 * g, mf, lgrp, [&](int s) {
      __builtin_amdgcn_sched_barrier(0);
      wt.load(w[s], g + 1, s, lane);
      __builtin_amdgcn_sched_barrier(0);
    });
#pragma unroll
    for (int f = 0; f < kFR; ++f) sc[f] = nsc[f];
    // Group g + 1's rows were requested in group g - 2, before its weights (or before the loop, and
    // waited for there): three groups' weight loads may stay in flight.
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<3 * kGroupLoads>();
    bare_barrier();
  }
  store_tile<MF, SWIGLU, OUT>(p, acc, t.row0, t.nrows, ncol0, lane);
}

template <int MF, bool SWIGLU, int OUT>
hipError_t launch_mf(MxGemm p, int m_tiles, hipStream_t stream) {
  const int lds = mx_groups(p.K) * 16 * MF * kMxRecord;
  if (lds <= kResidentBytes) {
    // parts of the channels: enough workgroups for two per CU
    const int blocks = (p.N + mx_bn(SWIGLU, kResidentWaves) - 1) / mx_bn(SWIGLU, kResidentWaves);
    p.parts = std::min(blocks, std::max(1, (2 * 256 + p.busy_tiles - 1) / p.busy_tiles));
    hipLaunchKernelGGL((mx_resident_kernel<MF, SWIGLU, OUT>), dim3(m_tiles * p.parts), dim3(kResidentWaves * 64), lds,
                       stream, p);
  } else {
    p.parts = (p.N + mx_bn(SWIGLU, kRingWaves) - 1) / mx_bn(SWIGLU, kRingWaves);
    hipLaunchKernelGGL((mx_ring_kernel<MF, SWIGLU, OUT>), dim3(m_tiles * p.parts), dim3(kRingWaves * 64), 0, stream, p);
  }
  return hipGetLastError();
}

template <bool SWIGLU, int OUT>
hipError_t launch_bm(int bm, const MxGemm& p, int m_tiles, hipStream_t stream) {
  switch (bm) {
    case 16: return launch_mf<1, SWIGLU, OUT>(p, m_tiles, stream);
    case 32: return launch_mf<2, SWIGLU, OUT>(p, m_tiles, stream);
    case 128: return launch_mf<8, SWIGLU, OUT>(p, m_tiles, stream);
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
