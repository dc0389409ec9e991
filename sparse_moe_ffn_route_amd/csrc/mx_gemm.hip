// Ragged grouped GEMM on microscaled 4-bit operands (formats in mx.hpp), gfx950 MFMA.
//
//   SwiGLU launch: h = silu(a W_gate^T) * (a W_up^T), quantised again to 4-bit rows;
//   plain launch:  out = a W^T.
// Both sum code products in fp32 through the 16x16x128 scaled MFMA, which multiplies each
// 32-value block of a row by the two blocks' powers of two, so nothing is decoded first.
//
// Work unit (one workgroup of 8 waves): one (group, N-tile, M-tile); M-tile 16 * MF rows
// gathered through perm, N-tile 8 waves x 4 fragments of 16 channels (SwiGLU: 2 of W_gate
// and the same 2 of W_up, whose 32 channels are one block of h).  Weight runs go from
// memory into registers as the A operand, four steps (one 512-value group) ahead; token
// records are staged in LDS, KC groups at a time, as the B operand shared by the waves.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"
#include "mx.hpp"

namespace moe {

namespace {

typedef uint32_t u32;
constexpr int kNW = 8;             // waves per workgroup
constexpr int kFR = 4;             // weight fragments per wave
enum : int { OUT_MX = 16 };        // output: 4-bit rows (SwiGLU launches)

// Groups of 512 values staged in LDS at a time: 139 KB for the tallest tile.
constexpr int mx_kc(int mf) { return mf == 1 ? 8 : mf == 2 ? 8 : 4; }

// c += A B for one step; byte S of the scale dwords belongs to it.
template <int S>
__device__ __forceinline__ f32x4 mx_mfma(const u32x4& a, const u32x4& b, f32x4 c, u32 sa, u32 sb) {
  const u32x4 z = {0u, 0u, 0u, 0u};  // fp4 operands use the first four registers
  const i32x8 av = __builtin_bit_cast(i32x8, __builtin_shufflevector(a, z, 0, 1, 2, 3, 4, 5, 6, 7));
  const i32x8 bv = __builtin_bit_cast(i32x8, __builtin_shufflevector(b, z, 0, 1, 2, 3, 4, 5, 6, 7));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, S, static_cast<int>(sa), S,
                                                          static_cast<int>(sb));
}

template <bool NT>
__device__ __forceinline__ u32 buffer_load4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, NT ? 2 : 0);
}

template <int MF, bool SWIGLU, int OUT>
__global__ __launch_bounds__(kNW * 64, MF >= 8 ? 2 : 4) void mx_gemm_kernel(MxGemm p) {
  constexpr int NMAT = SWIGLU ? 2 : 1;
  constexpr int NF = kFR / NMAT;
  constexpr int BM = 16 * MF;
  constexpr int BN = kNW * NF * 16;
  constexpr int KC = mx_kc(MF);
  constexpr bool NT = MF <= 2;  // one M-tile reads the weights: stream them past the caches
  __shared__ __attribute__((aligned(16))) uint8_t lds[KC * BM * kMxRecord];
  __shared__ u32 src_row[BM];

  const int n_tiles = (p.N + BN - 1) / BN;
  const int total = ld_scalar(p.tile_prefix + p.n_groups) * n_tiles;
  if (static_cast<int>(blockIdx.x) >= total) return;
  const int L = xcd_remap(blockIdx.x, total);
  int lo = 0, hi = p.n_groups - 1;
  const int q = L / n_tiles;
  while (lo < hi) {  // largest g with prefix[g] <= q
    const int mid = (lo + hi + 1) >> 1;
    if (ld_scalar(p.tile_prefix + mid) <= q) lo = mid; else hi = mid - 1;
  }
  const int g = __builtin_amdgcn_readfirstlane(lo);
  const int pg = ld_scalar(p.tile_prefix + g);
  const int mt = ld_scalar(p.tile_prefix + g + 1) - pg;
  const int local = L - pg * n_tiles;
  const int n_tile = __builtin_amdgcn_readfirstlane(local / mt);
  const int rbeg = __builtin_amdgcn_readfirstlane((local % mt) * BM);
  const int row0 = ld_scalar(p.offsets + g) + rbeg;
  const int nrows = min(BM, ld_scalar(p.offsets + g + 1) - row0);
  const int mf_active = (nrows + 15) / 16;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int S = mx_steps(p.K), G = mx_groups(p.K);
  const u32 frag_bytes = static_cast<u32>(mx_fragment_bytes(p.K));
  const int64_t row_bytes = mx_row_bytes(p.K);
  const int ncol0 = n_tile * BN + wave * NF * 16;

  // rows past the tile's last one re-read it (they are never stored)
  for (int r = threadIdx.x; r < BM; r += kNW * kWave) {
    const int gr = row0 + min(r, nrows - 1);
    src_row[r] = static_cast<u32>(p.perm ? p.perm[gr] : gr);
  }

  __amdgpu_buffer_rsrc_t wres[NMAT];
  wres[0] = buffer_rsrc(static_cast<const uint8_t*>(p.w0) + static_cast<size_t>(g) * p.w_stride);
  if (SWIGLU) wres[NMAT - 1] = buffer_rsrc(static_cast<const uint8_t*>(p.w1) + static_cast<size_t>(g) * p.w_stride);
  const __amdgpu_buffer_rsrc_t none = buffer_rsrc_empty();
  u32 fofs[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) fofs[f] = static_cast<u32>(min(ncol0 / 16 + f, p.N / 16 - 1)) * frag_bytes;

  auto load_step = [&](u32x4 (&w)[kFR], int st) {
    const bool real = st < S;
    const u32 o = real ? static_cast<u32>(st / 4) * kMxGroupBytes + (st % 4) * kMxRun : 0u;
#pragma unroll
    for (int a = 0; a < NMAT; ++a)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        w[a * NF + f] = buffer_load16<NT>(real ? wres[a] : none, lane * 16, fofs[f] + o);
  };
  auto load_scales = [&](u32 (&s)[kFR], int grp) {
    const bool real = grp < G;
    const u32 o = real ? static_cast<u32>(grp) * kMxGroupBytes + static_cast<u32>(min(4, S - 4 * grp)) * kMxRun : 0u;
#pragma unroll
    for (int a = 0; a < NMAT; ++a)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        s[a * NF + f] = buffer_load4<NT>(real ? wres[a] : none, lane * 4, fofs[f] + o);
  };

  auto run = [&](auto mfr_c) {
    constexpr int MFR = decltype(mfr_c)::value;
    f32x4 acc[kFR][MFR];
#pragma unroll
    for (int f = 0; f < kFR; ++f)
#pragma unroll
      for (int m = 0; m < MFR; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 w[4][kFR];
    u32 sc[kFR], nsc[kFR];
    load_scales(sc, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) load_step(w[s], s);

    for (int g0 = 0; g0 < G; g0 += KC) {
      const int gn = min(KC, G - g0);
      __syncthreads();  // src_row is written; the previous groups have been read
      constexpr int kPieces = MFR * 16 * (kMxRecord / 16);
      for (int kc = 0; kc < gn; ++kc) {
        for (int c = threadIdx.x; c < kPieces; c += kNW * kWave) {
          const int r = c / (kMxRecord / 16), col = c % (kMxRecord / 16);
          const uint8_t* src = static_cast<const uint8_t*>(p.a) + src_row[r] * row_bytes +
                               static_cast<int64_t>(g0 + kc) * kMxRecord + col * 16;
          *reinterpret_cast<u32x4*>(lds + kc * (BM * kMxRecord) + c * 16) = *reinterpret_cast<const u32x4*>(src);
        }
      }
      __syncthreads();
      for (int kc = 0; kc < gn; ++kc) {
        const int grp = g0 + kc;
        load_scales(nsc, grp + 1);
        const uint8_t* rec = lds + kc * (BM * kMxRecord) + lrow * kMxRecord;
        auto step = [&](auto sc_c) {
          constexpr int s = decltype(sc_c)::value;
          if (grp * 4 + s < S) {
#pragma unroll
            for (int m = 0; m < MFR; ++m) {
              const uint8_t* r = rec + m * 16 * kMxRecord;
              const u32x4 b = *reinterpret_cast<const u32x4*>(r + s * 64 + lgrp * 16);
              const u32 bs = *reinterpret_cast<const u32*>(r + 256 + lgrp * 4);
#pragma unroll
              for (int f = 0; f < kFR; ++f) acc[f][m] = mx_mfma<s>(w[s][f], b, acc[f][m], sc[f], bs);
            }
          }
          load_step(w[s], (grp + 1) * 4 + s);
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
#pragma unroll
        for (int f = 0; f < kFR; ++f) sc[f] = nsc[f];
      }
    }

    // ---- epilogue -----------------------------------------------------------
    if (ncol0 >= p.N) return;
#pragma unroll
    for (int m = 0; m < MFR; ++m) {
      const int r = m * 16 + lrow;
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
          uint8_t* rec = static_cast<uint8_t*>(p.out) + grow * mx_row_bytes(p.N) +
                         static_cast<int64_t>(b / 16) * kMxRecord;
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
          const int n = ncol0 + f * 16 + lgrp * 4;
          if (ncol0 + f * 16 >= p.N) continue;
          const size_t idx = static_cast<size_t>(grow) * p.N + n;
          const f32x4 o = acc[f][m];
          if constexpr (OUT == EL_F32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + idx) = make_float4(o[0], o[1], o[2], o[3]);
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + idx) =
                make_uint2(bf16x2_bits(o[0], o[1]), bf16x2_bits(o[2], o[3]));
        }
      }
    }
  };
  if constexpr (MF < 8) {
    if (MF == 2 && mf_active == 1) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, MF>{});
  } else {
    // fragments in use, rounded up to two
    switch ((mf_active + 1) / 2) {
      case 1: run(std::integral_constant<int, 2>{}); break;
      case 2: run(std::integral_constant<int, 4>{}); break;
      case 3: run(std::integral_constant<int, 6>{}); break;
      default: run(std::integral_constant<int, 8>{}); break;
    }
  }
}

template <bool SWIGLU, int OUT>
hipError_t launch_bm(int bm, const MxGemm& p, int max_tiles, hipStream_t stream) {
  const dim3 grid(max_tiles), block(kNW * 64);
  if (bm == 16)
    hipLaunchKernelGGL((mx_gemm_kernel<1, SWIGLU, OUT>), grid, block, 0, stream, p);
  else if (bm == 32)
    hipLaunchKernelGGL((mx_gemm_kernel<2, SWIGLU, OUT>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((mx_gemm_kernel<8, SWIGLU, OUT>), grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

int mx_gemm_bn(bool swiglu) { return kNW * (swiglu ? kFR / 2 : kFR) * 16; }

hipError_t launch_mx_gemm(bool swiglu, int out_el, int bm, const MxGemm& p, int max_tiles, hipStream_t stream) {
  if (max_tiles == 0) return hipSuccess;
  if (bm != 16 && bm != 32 && bm != 128) return hipErrorInvalidValue;
  if (swiglu) return launch_bm<true, OUT_MX>(bm, p, max_tiles, stream);
  return out_el == EL_F32 ? launch_bm<false, EL_F32>(bm, p, max_tiles, stream)
                          : launch_bm<false, EL_BF16>(bm, p, max_tiles, stream);
}

}  // namespace moe
