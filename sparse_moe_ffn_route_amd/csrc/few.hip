// The whole MoE layer for 1 to 16 tokens.
//
//   logits kernel    logits = x W_r^T, one workgroup per 16 experts
//   gate/up kernel   every workgroup selects the top-k of all tokens from the logits (a few
//                    KB, in L2), then takes units of (chosen expert or the shared one, 16
//                    channels): h = w * silu(W_gate x) * (W_up x)
//   down kernel      y = sum over experts and channels of W_down h, one workgroup per 16
//                    output channels, which therefore owns their whole sum
// With given routing the first launch is not needed.
//
// All tokens of the call are the 16 columns of one MFMA tile, so each weight byte of a chosen
// expert is read once whichever tokens chose it, and there is no grouping step.  Columns
// of tokens that did not choose the expert are computed and dropped by a select (not by a
// zero weight: an expert's NaN must not reach another expert's token).  Weights of any type
// are turned into bf16 in registers (exact for e4m3 and 4-bit codes) and x is never
// quantised; h, scaled by the routing weight, is carried as a pair of bf16 (value and
// remainder, 16 significant bits), which costs a second MFMA and keeps the rounding of h
// out of y.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"
#include "mx.hpp"
#include "topk.hpp"

namespace moe {

namespace {

typedef uint32_t u32;
constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxPairs = kFewMaxT * 32;

// Weight type W (EL_F32, EL_BF16, EL_E4M3 or EL_MX): a "step" is what 16 bytes per lane cover
// of 16 rows, EPS values of the reduction dimension, of which lane group g holds the
// EPS / 4 from g * EPS / 4 on.  NX: 16-byte pieces of the other operand per lane and step.
constexpr int EL_MX = 3;
template <int W> struct Wt;
template <> struct Wt<EL_F32> { static constexpr int EPS = 16, NX = 1, U = 8; };
template <> struct Wt<EL_BF16> { static constexpr int EPS = 32, NX = 1, U = 8; };
template <> struct Wt<EL_E4M3> { static constexpr int EPS = 64, NX = 2, U = 4; };
template <> struct Wt<EL_MX> { static constexpr int EPS = 128, NX = 4, U = 2; };

// Where the 16 rows of fragment `frag` of a [rows][K] matrix lie, and their steps.
template <int W, bool PACKED> struct Rows {
  const uint8_t* p;  // this lane's first bytes
  int S;
  __device__ __forceinline__ Rows(const void* m, int frag, int K, int lane) {
    S = (K + Wt<W>::EPS - 1) / Wt<W>::EPS;
    const uint8_t* b = static_cast<const uint8_t*>(m);
    if constexpr (W == EL_MX) {
      p = b + frag * mx_fragment_bytes(K);
    } else if constexpr (PACKED) {
      p = b + static_cast<int64_t>(frag) * S * 1024 + lane * 16;
    } else {
      p = b + (static_cast<int64_t>(frag) * 16 + (lane & 15)) * (S * 64) + (lane >> 4) * 16;
    }
  }
  __device__ __forceinline__ u32x4 load(int s, int lane) const {
    const uint8_t* q;
    if constexpr (W == EL_MX) q = p + (s >> 2) * kMxGroupBytes + (s & 3) * kMxRun + lane * 16;
    else q = p + static_cast<int64_t>(s) * (PACKED ? 1024 : 64);
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(q));
  }
  // the block's power of two
  __device__ __forceinline__ float scale(int s, int lane) const {
    if constexpr (W == EL_MX) {
      const int g = s >> 2;
      const u32 d = *reinterpret_cast<const u32*>(p + g * kMxGroupBytes + min(4, S - 4 * g) * kMxRun + lane * 4);
      const u32 b = (d >> (8 * (s & 3))) & 255u;
      return b == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(b << 23);
    } else {
      return 1.0f;
    }
  }
};

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Piece i of a weight step as eight bf16 (f32: the 16 bytes as they are).
template <int W>
__device__ __forceinline__ u32x4 weight_piece(const u32x4& w, int i, float scale) {
  if constexpr (W == EL_E4M3) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const u32 d = w[2 * i + j];
      r[2 * j] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, false));
      r[2 * j + 1] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, true));
    }
    return r;
  } else if constexpr (W == EL_MX) {
    u32x4 r;
    const u32 d = w[i];
    r[0] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0));
    r[1] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1));
    r[2] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2));
    r[3] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3));
    return r;
  } else {
    return w;
  }
}

template <int W>
__device__ __forceinline__ f32x4 mul(const u32x4& a, const u32x4& b, f32x4 c) {
  return mfma_chunk<W == EL_F32 ? EL_F32 : EL_BF16>(a, b, c);
}

// ---------------------------------------------------------------------------
// logits
// ---------------------------------------------------------------------------

template <int EL>
__global__ __launch_bounds__(kThreads) void few_logits_kernel(const void* __restrict__ x, const void* __restrict__ wr,
                                                              int T, int D, int E, float* __restrict__ logits) {
  __shared__ f32x4 red[kWaves][kWave];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int e0 = blockIdx.x * 16;
  constexpr int es = EL == EL_F32 ? 4 : 2;
  const int S = D * es / 64;
  const int s0 = S * wave / kWaves, s1 = S * (wave + 1) / kWaves;
  const int e = min(e0 + lrow, E - 1);
  const uint8_t* wp = static_cast<const uint8_t*>(wr) + static_cast<int64_t>(e) * D * es + lgrp * 16;
  const uint8_t* xp = static_cast<const uint8_t*>(x) + static_cast<int64_t>(min(lrow, T - 1)) * D * es + lgrp * 16;
  const u32x4 z = {0u, 0u, 0u, 0u};
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;
  for (int s = s0; s < s1; s += U) {
    u32x4 a[U], b[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int q = min(s + i, s1 - 1);
      a[i] = *reinterpret_cast<const u32x4*>(wp + static_cast<int64_t>(q) * 64);
      b[i] = *reinterpret_cast<const u32x4*>(xp + static_cast<int64_t>(q) * 64);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (s + i < s1) acc = mfma_chunk<EL>(a[i], lrow < T ? b[i] : z, acc);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 256) {
    const int l = threadIdx.x & 63, r = threadIdx.x >> 6;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += red[w][l][r];
    const int t = l & 15, ee = e0 + (l >> 4) * 4 + r;
    if (t < T && ee < E) logits[static_cast<int64_t>(t) * E + ee] = v;
  }
}

// ---------------------------------------------------------------------------
// The call's (token, slot) pairs and the experts they name
// ---------------------------------------------------------------------------

struct Pairs {
  int32_t blob[2 * kMaxPairs];  // [T][2][k], as the packed routing blob
  u32 mask[1024];               // tokens of each local expert
  uint16_t list[kMaxPairs];     // local experts with a token, ascending
  int count;
};

// All threads, after blob is written.
__device__ void find_experts(Pairs& q, const FewLayer& p) {
  __syncthreads();
  for (int e = threadIdx.x; e < p.n_local; e += kThreads) q.mask[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * p.k; i += kThreads) {
    const int t = i / p.k, id = q.blob[t * 2 * p.k + i % p.k], e = id - p.e_begin;
    if (id >= 0 && id < p.E && e >= 0 && e < p.n_local) atomicOr(&q.mask[e], 1u << t);
  }
  __syncthreads();
  if (threadIdx.x < kWave) {
    int n = 0;
    for (int e0 = 0; e0 < p.n_local; e0 += kWave) {
      const int e = e0 + threadIdx.x;
      const bool on = e < p.n_local && q.mask[e] != 0;
      const uint64_t b = __ballot(on);
      if (on) q.list[n + __popcll(b & ((1ull << threadIdx.x) - 1))] = static_cast<uint16_t>(e);
      n += __popcll(b);
    }
    if (threadIdx.x == 0) q.count = n;
  }
  __syncthreads();
}

// First slot of token t that names local expert e, or -1; weight: the sum over all that do.
__device__ __forceinline__ int slot_of(const Pairs& q, const FewLayer& p, int t, int e, float& weight) {
  int slot = -1;
  weight = 0.f;
  for (int j = 0; j < p.k; ++j)
    if (q.blob[t * 2 * p.k + j] == e + p.e_begin) {
      if (slot < 0) slot = j;
      weight += __int_as_float(q.blob[t * 2 * p.k + p.k + j]);
    }
  return slot;
}

template <int PL>
__device__ void select_all(Pairs& q, const FewLayer& p) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  for (int t = wave; t < p.T; t += kWaves) {
    float key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + i * kWave;
      key[i] = -INFINITY;
      if (e < p.E) {
        key[i] = p.logits[static_cast<int64_t>(t) * p.E + e];
        if (p.bias) key[i] = key[i] + p.bias[e];
      }
    }
    select_topk(key, p.E, p.k, p.renormalize, q.blob + t * 2 * p.k);
  }
}

// ---------------------------------------------------------------------------
// gate/up
// ---------------------------------------------------------------------------

// Products of the two matrices' 16 rows with all tokens over this wave's steps.
template <int W, bool PACKED>
__device__ __forceinline__ void gate_up_range(const void* m0, const void* m1, int frag, const FewLayer& p, int wave,
                                              int lane, f32x4& c0, f32x4& c1) {
  constexpr int EPS = Wt<W>::EPS, NX = Wt<W>::NX, U = Wt<W>::U;
  constexpr int as = W == EL_F32 ? 4 : 2;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const Rows<W, PACKED> r0(m0, frag, p.D, lane), r1(m1, frag, p.D, lane);
  const int s0 = r0.S * wave / kWaves, s1 = r0.S * (wave + 1) / kWaves;
  const uint8_t* xp = static_cast<const uint8_t*>(p.x) + static_cast<int64_t>(min(lrow, p.T - 1)) * p.D * as;
  const bool live = lrow < p.T;
  const u32x4 z = {0u, 0u, 0u, 0u};
  for (int s = s0; s < s1; s += U) {
    u32x4 a[U], b[U], xv[U][NX];
    float fa[U], fb[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int q = min(s + i, s1 - 1);
      a[i] = r0.load(q, lane);
      b[i] = r1.load(q, lane);
      fa[i] = r0.scale(q, lane);
      fb[i] = r1.scale(q, lane);
      const int k0 = q * EPS + lgrp * (EPS / 4);
      const bool in = live && k0 < p.D;
#pragma unroll
      for (int n = 0; n < NX; ++n) xv[i][n] = in ? reinterpret_cast<const u32x4*>(xp + static_cast<int64_t>(k0) * as)[n] : z;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (s + i >= s1) break;
#pragma unroll
      for (int n = 0; n < NX; ++n) {
        c0 = mul<W>(weight_piece<W>(a[i], n, fa[i]), xv[i][n], c0);
        c1 = mul<W>(weight_piece<W>(b[i], n, fb[i]), xv[i][n], c1);
      }
    }
  }
}

// h as two planes of bf16 (value, remainder) of `plane` elements each; fp32 layers one of fp32.
template <bool F32>
__device__ __forceinline__ void store_h(void* h, int64_t plane, int64_t idx, float v) {
  if constexpr (F32) {
    static_cast<float*>(h)[idx] = v;
  } else {
    uint16_t* o = static_cast<uint16_t*>(h);
    const u32 hi = bf16x2_bits(v, 0.f) & 0xFFFFu;
    o[idx] = static_cast<uint16_t>(hi);
    // an infinite value has no remainder
    const float rest = v - bf16_bits_to_f32(hi);
    o[plane + idx] = static_cast<uint16_t>(fabsf(v) <= 3.0e38f ? bf16x2_bits(rest, 0.f) & 0xFFFFu : 0u);
  }
}

template <int W, bool PACKED>
__global__ __launch_bounds__(kThreads) void few_gate_up_kernel(FewLayer p) {
  constexpr bool F32 = W == EL_F32;
  constexpr int SH = F32 ? EL_F32 : EL_BF16;
  __shared__ Pairs q;
  __shared__ f32x4 red[2][2][kWaves][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  if (p.packed_in) {
    for (int i = threadIdx.x; i < p.T * 2 * p.k; i += kThreads) q.blob[i] = p.packed_in[i];
  } else if (p.E <= 8 * kWave) {
    select_all<8>(q, p);
  } else {
    select_all<kMaxKeysPerLane>(q, p);
  }
  find_experts(q, p);
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < p.T * 2 * p.k; i += kThreads) {
      p.packed[i] = q.blob[i];
      if (p.packed_out) p.packed_out[i] = q.blob[i];
    }
    if (wave == 0) {
      int bad = 0;
      for (int i = lane; i < p.T * p.k; i += kWave) {
        const int id = q.blob[i / p.k * 2 * p.k + i % p.k];
        bad += id < 0 || id >= p.E;
      }
      bad = wave_sum_int(bad);
      if (lane == 0) *p.err = bad;
    }
  }

  const int per = p.I / 16;
  const int routed = q.count * per;
  const int units = routed + p.I_shared / 16;
  int parity = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const bool sh = u >= routed;
    const int frag = sh ? u - routed : u % per;
    const int e = sh ? 0 : q.list[u / per];
    f32x4 c0 = {0.f, 0.f, 0.f, 0.f}, c1 = {0.f, 0.f, 0.f, 0.f};
    if (sh)
      gate_up_range<SH, PACKED>(p.sh_gate, p.sh_up, frag, p, wave, lane, c0, c1);
    else
      gate_up_range<W, PACKED>(static_cast<const uint8_t*>(p.w_gate) + e * p.gu_stride,
                               static_cast<const uint8_t*>(p.w_up) + e * p.gu_stride, frag, p, wave, lane, c0, c1);
    red[parity][0][wave][lane] = c0;
    red[parity][1][wave][lane] = c1;
    __syncthreads();
    if (threadIdx.x < 256) {
      // thread -> (channel, token) of the 16 x 16 tile; partial products added in wave order
      const int l = threadIdx.x & 63, r = threadIdx.x >> 6;
      const int t = l & 15, n = frag * 16 + (l >> 4) * 4 + r;
      if (t < p.T) {
        float g = 0.f, v = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          g += red[parity][0][w][l][r];
          v += red[parity][1][w][l][r];
        }
        if (sh) {
          store_h<F32>(p.h_sh, static_cast<int64_t>(p.T) * p.I_shared, static_cast<int64_t>(t) * p.I_shared + n,
                       silu(g) * v);
        } else {
          float wt;
          const int j = slot_of(q, p, t, e, wt);
          if (j >= 0) {
            if constexpr (W == EL_E4M3) {
              g *= p.s_gate[static_cast<int64_t>(e) * p.I + n];
              v *= p.s_up[static_cast<int64_t>(e) * p.I + n];
            }
            store_h<F32>(p.h, static_cast<int64_t>(p.T) * p.k * p.I, (static_cast<int64_t>(t) * p.k + j) * p.I + n,
                         wt * (silu(g) * v));
          }
        }
      }
    }
    parity ^= 1;
  }
}

// ---------------------------------------------------------------------------
// down
// ---------------------------------------------------------------------------

// c += 16 rows of W_down times h over steps [s0, s1); hp: this lane's token's row of h (value
// plane, remainder `plane` elements on), NULL for a lane without one.
template <int W, bool PACKED>
__device__ __forceinline__ f32x4 down_range(const void* m, int frag, int K, const uint8_t* hp, int64_t plane, int s0,
                                            int s1, int lane) {
  constexpr int EPS = Wt<W>::EPS, NX = Wt<W>::NX, U = Wt<W>::U;
  constexpr bool F32 = W == EL_F32;
  constexpr int as = F32 ? 4 : 2;
  const int lgrp = lane >> 4;
  const Rows<W, PACKED> r(m, frag, K, lane);
  const u32x4 z = {0u, 0u, 0u, 0u};
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
  for (int s = s0; s < s1; s += U) {
    u32x4 a[U], hv[U][NX], lv[U][NX];
    float fa[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int q = min(s + i, s1 - 1);
      a[i] = r.load(q, lane);
      fa[i] = r.scale(q, lane);
      const int k0 = q * EPS + lgrp * (EPS / 4);
      const bool in = hp != nullptr && k0 < K;
#pragma unroll
      for (int n = 0; n < NX; ++n) {
        hv[i][n] = in ? reinterpret_cast<const u32x4*>(hp + static_cast<int64_t>(k0) * as)[n] : z;
        if constexpr (!F32)
          lv[i][n] = in ? reinterpret_cast<const u32x4*>(hp + (plane + k0) * as)[n] : z;
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (s + i >= s1) break;
#pragma unroll
      for (int n = 0; n < NX; ++n) {
        const u32x4 w = weight_piece<W>(a[i], n, fa[i]);
        c = mul<W>(w, hv[i][n], c);
        if constexpr (!F32) c = mul<W>(w, lv[i][n], c);
      }
    }
  }
  return c;
}

template <int W, bool PACKED, int OUT>
__global__ __launch_bounds__(kThreads) void few_down_kernel(FewLayer p) {
  constexpr bool F32 = W == EL_F32;
  constexpr int SH = F32 ? EL_F32 : EL_BF16;
  constexpr int as = F32 ? 4 : 2;
  __shared__ Pairs q;
  __shared__ f32x4 red[kWaves][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int t = lane & 15, frag = blockIdx.x;
  for (int i = threadIdx.x; i < p.T * 2 * p.k; i += kThreads) q.blob[i] = p.packed[i];
  find_experts(q, p);

  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const int S = (p.I + Wt<W>::EPS - 1) / Wt<W>::EPS;
  const int total = q.count * S;
  int at = static_cast<int>(static_cast<int64_t>(total) * wave / kWaves);
  const int end = static_cast<int>(static_cast<int64_t>(total) * (wave + 1) / kWaves);
  while (at < end) {
    const int a = at / S, s0 = at - a * S, s1 = min(S, s0 + end - at);
    const int e = q.list[a];
    float wt;
    const int j = t < p.T ? slot_of(q, p, t, e, wt) : -1;
    const uint8_t* hp = j < 0 ? nullptr : static_cast<const uint8_t*>(p.h) + (static_cast<int64_t>(t) * p.k + j) * p.I * as;
    f32x4 c = down_range<W, PACKED>(static_cast<const uint8_t*>(p.w_down) + e * p.dn_stride, frag, p.I, hp,
                                    static_cast<int64_t>(p.T) * p.k * p.I, s0, s1, lane);
    if constexpr (W == EL_E4M3) {
      const float* sd = p.s_down + static_cast<int64_t>(e) * p.D + frag * 16 + (lane >> 4) * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] *= sd[i];
    }
    if (j >= 0) acc += c;
    at += s1 - s0;
  }
  if (p.I_shared) {
    const int Ss = p.I_shared / Wt<SH>::EPS;
    const uint8_t* hp = t < p.T ? static_cast<const uint8_t*>(p.h_sh) + static_cast<int64_t>(t) * p.I_shared * as : nullptr;
    acc += down_range<SH, PACKED>(p.sh_down, frag, p.I_shared, hp, static_cast<int64_t>(p.T) * p.I_shared,
                                  Ss * wave / kWaves, Ss * (wave + 1) / kWaves, lane);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 256) {
    const int r = threadIdx.x & 3, l = (threadIdx.x >> 2) & 63;  // consecutive threads: consecutive channels
    const int tt = l & 15, d = frag * 16 + (l >> 4) * 4 + r;
    if (tt < p.T) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += red[w][l][r];
      const int64_t idx = static_cast<int64_t>(tt) * p.D + d;
      if constexpr (OUT == EL_F32) static_cast<float*>(p.y)[idx] = v;
      else static_cast<uint16_t*>(p.y)[idx] = static_cast<uint16_t>(bf16x2_bits(v, 0.f));
    }
  }
}

// Workgroups of the gate/up launch: two per CU of 256; more units than that are taken in turn.
constexpr int kGateUpBlocks = 512;

template <int W, bool PACKED>
hipError_t launch_w(const FewLayer& p, hipStream_t stream) {
  if (!p.packed_in) {
    constexpr int act = W == EL_F32 ? EL_F32 : EL_BF16;
    hipLaunchKernelGGL((few_logits_kernel<act>), dim3((p.E + 15) / 16), dim3(kThreads), 0, stream, p.x, p.w_router,
                       p.T, p.D, p.E, p.logits);
  }
  const int experts = p.T * p.k < p.n_local ? p.T * p.k : p.n_local;
  const int64_t units = static_cast<int64_t>(experts) * (p.I / 16) + p.I_shared / 16;
  const int grid = static_cast<int>(units < kGateUpBlocks ? (units > 0 ? units : 1) : kGateUpBlocks);
  hipLaunchKernelGGL((few_gate_up_kernel<W, PACKED>), dim3(grid), dim3(kThreads), 0, stream, p);
  if (p.out_el == EL_F32)
    hipLaunchKernelGGL((few_down_kernel<W, PACKED, EL_F32>), dim3(p.D / 16), dim3(kThreads), 0, stream, p);
  else if constexpr (W != EL_F32)
    hipLaunchKernelGGL((few_down_kernel<W, PACKED, EL_BF16>), dim3(p.D / 16), dim3(kThreads), 0, stream, p);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few_layer(int w_el, bool packed, const FewLayer& p, hipStream_t stream) {
  switch (w_el) {
    case EL_F32: return packed ? launch_w<EL_F32, true>(p, stream) : launch_w<EL_F32, false>(p, stream);
    case EL_BF16: return packed ? launch_w<EL_BF16, true>(p, stream) : launch_w<EL_BF16, false>(p, stream);
    case EL_E4M3: return packed ? launch_w<EL_E4M3, true>(p, stream) : launch_w<EL_E4M3, false>(p, stream);
    case EL_MX: return launch_w<EL_MX, true>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace moe
