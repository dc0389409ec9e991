// Device code shared by the kernels of the few-token layer (few.hip, few_mx.hip).
#pragma once

#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"
#include "topk.hpp"

namespace moe {

namespace few {

typedef uint32_t u32;
constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxPairs = kFewMaxT * 32;
constexpr int kCus = 256;
constexpr int kLdsBytes = 160 * 1024;

// Weight type W (EL_F32, EL_BF16 or EL_E4M3): a "step" is what 16 bytes per lane cover
// of 16 rows, EPS values of the reduction dimension, of which lane group g holds the
// EPS / 4 from g * EPS / 4 on.  NX: 16-byte pieces of the other operand per lane and step.
// Gate/up blocks are GB steps of both matrices, GN of them in the ring; down blocks DB steps of
// one matrix with their pieces of h, DN in the ring (DN2 with separate remainders): 2 waves
// per SIMD have 256 registers each.
template <int W> struct Wt;
template <> struct Wt<EL_F32> {
  static constexpr int EPS = 16, NX = 1, GB = 8, GN = 3, DB = 8, DN = 3, DN2 = 3;
};
template <> struct Wt<EL_BF16> {
  static constexpr int EPS = 32, NX = 1, GB = 8, GN = 3, DB = 8, DN = 3, DN2 = 2;
};
template <> struct Wt<EL_E4M3> {
  static constexpr int EPS = 64, NX = 2, GB = 8, GN = 3, DB = 4, DN = 4, DN2 = 2;
};
template <int W> constexpr int act_bytes() { return W == EL_F32 ? 4 : 2; }
template <int W> __host__ __device__ constexpr int steps_of(int k) { return (k + Wt<W>::EPS - 1) / Wt<W>::EPS; }

// Byte offsets within one [rows][K] matrix: lane part, and wave-uniform part of step s of the 16
// rows of fragment `frag`.
template <int W, bool PACKED>
__device__ __forceinline__ u32 lane_offset(int K, int lane) {
  if constexpr (PACKED) return lane * 16;
  else return (lane & 15) * (steps_of<W>(K) * 64) + (lane >> 4) * 16;
}
template <int W, bool PACKED>
__device__ __forceinline__ u32 step_offset(int K, int frag, int s) {
  if constexpr (PACKED)
    return (static_cast<u32>(frag) * steps_of<W>(K) + s) * 1024;
  else
    return static_cast<u32>(frag) * 16 * (steps_of<W>(K) * 64) + s * 64;
}
// Piece i of a weight step as eight bf16 (f32: the 16 bytes as they are).
template <int W>
__device__ __forceinline__ u32x4 weight_piece(const u32x4& w, int i) {
  if constexpr (W == EL_E4M3) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const u32 d = w[2 * i + j];
      r[2 * j] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, false));
      r[2 * j + 1] = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, true));
    }
    return r;
  } else {
    return w;
  }
}

template <int W>
__device__ __forceinline__ f32x4 mul(const u32x4& a, const u32x4& b, f32x4 c) {
  return mfma_chunk<W == EL_F32 ? EL_F32 : EL_BF16>(a, b, c);
}

// A resource of `bytes` bytes: loads at or past its end return zeros and touch no memory.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc_sized(const void* base, u32 bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const u32 lo = static_cast<u32>(__builtin_amdgcn_readfirstlane(static_cast<u32>(a)));
  const u32 hi = static_cast<u32>(__builtin_amdgcn_readfirstlane(static_cast<u32>(a >> 32)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0,
                                           static_cast<int>(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000);
}
constexpr u32 kOutOfRange = 0x80000000u;  // h and every weight matrix is smaller (checked by the host)
// One weight matrix: a step that is not there is a lane offset of kOutOfRange, a select; choosing
// between two resources made branches, with a wait for every load in flight in each.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t weight_rsrc(const void* base) { return buffer_rsrc_sized(base, 0x7FFFFFFFu); }

// This wave's LDS accesses are done, then every wave's: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  bare_barrier();
}

// ---------------------------------------------------------------------------
// The call's (token, slot) pairs and the experts they name
// ---------------------------------------------------------------------------

struct Pairs {
  int32_t blob[2 * kMaxPairs];  // [T][2][k], as the packed routing blob
  int32_t first[1024];          // first pair that names each local expert; before that, selection scratch
  uint16_t list[kMaxPairs];     // local experts with a token, in the order of their first pairs
  int wave_count[kWaves];
  int count;
};

// Top-k of one token by one wave: the same keys, order and weights as select_topk (topk.hpp), in
// about a fifth of its time for 512 keys.  The k-th largest of the lanes' own best keys bounds the
// k-th largest of all from below; the keys that reach it (a few more than k) are ranked against
// each other.  More than 64 of them (many equal keys) take select_topk.
template <int PL>
__device__ __forceinline__ void select_few(const float (&key)[PL], int E, int k, int renormalize,
                                           float2* __restrict__ cand, int32_t* __restrict__ out) {
  const int lane = threadIdx.x % kWave;
  float bk = -INFINITY;
  int bi = 0x7FFFFFFF;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + i * kWave;
    nan |= key[i] != key[i];
    if (e < E && key_before(key[i], e, bk, bi)) {
      bk = key[i];
      bi = e;
    }
  }
  int rank = 0;
#pragma unroll
  for (int j = 0; j < kWave; ++j) {
    const float ok = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bk), j));
    const int oi = __builtin_amdgcn_readlane(bi, j);
    rank += key_before(ok, oi, bk, bi) ? 1 : 0;
  }
  // lanes without a key come last; k <= E lanes or more have one, or every key is a candidate
  const uint64_t at = __ballot(rank == k - 1 && bi < E);
  float lk = -INFINITY;
  int li = 0x7FFFFFFF;
  if (at) {
    const int l = __ffsll(static_cast<unsigned long long>(at)) - 1;
    lk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bk), l));
    li = __builtin_amdgcn_readlane(bi, l);
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + i * kWave;
    const bool on = e < E && !key_before(lk, li, key[i], e);
    const uint64_t b = __ballot(on);
    const int pos = n + __popcll(b & ((1ull << lane) - 1));
    if (on && pos < kWave) cand[pos] = make_float2(key[i], __int_as_float(e));
    n += __popcll(b);
  }
  if (n > kWave || n < k || __any(nan)) {
    select_topk(key, E, k, renormalize, out);
    return;
  }
  // one candidate per lane, through LDS within the wave
  __builtin_amdgcn_wave_barrier();
  float ck = -INFINITY;
  int ci = 0x7FFFFFFF;
  if (lane < n) {
    const float2 c = cand[lane];
    ck = c.x;
    ci = __float_as_int(c.y);
  }
  int r = 0;
  for (int j = 0; j < n; ++j) {
    const float ok = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ck), j));
    const int oi = __builtin_amdgcn_readlane(ci, j);
    r += key_before(ok, oi, ck, ci) ? 1 : 0;
  }
  const bool kept = lane < n && r < k;
  const uint64_t top = __ballot(kept && r == 0);
  const int l0 = top ? __ffsll(static_cast<unsigned long long>(top)) - 1 : 0;
  const float kmax = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ck), l0));
  const float num = kept ? expf(ck - kmax) : 0.0f;
  float den = num;
  if (!renormalize) {
    den = 0.0f;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + i * kWave < E) den += expf(key[i] - kmax);
  }
  den = wave_sum(den);
  if (kept) {
    out[r] = ci;
    out[k + r] = __float_as_int(num / den);
  }
}

template <int PL>
__device__ __forceinline__ void select_all(Pairs& q, const FewLayer& p) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  float2* cand = reinterpret_cast<float2*>(q.first) + wave * kWave;
  for (int t = wave; t < p.T; t += kWaves) {
    float key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + i * kWave;
      key[i] = e < p.E ? p.logits[static_cast<int64_t>(t) * p.E + e] : -INFINITY;
    }
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const int e = lane + i * kWave;
        if (e < p.E) key[i] = key[i] + p.bias[e];
      }
    }
    select_few(key, p.E, p.k, p.renormalize, cand, q.blob + t * 2 * p.k);
  }
}

// The call's routing into q, by all threads: given, or selected from the logits; then the
// distinct local experts.
__device__ __forceinline__ void route_call(Pairs& q, const FewLayer& p) {
  static_assert(sizeof(q.first) >= kWaves * kWave * sizeof(float2), "selection scratch");
  if (p.packed_in) {
    for (int i = threadIdx.x; i < p.T * 2 * p.k; i += kThreads) q.blob[i] = p.packed_in[i];
  } else if (p.E <= 2 * kWave) {
    select_all<2>(q, p);
  } else if (p.E <= 8 * kWave) {
    select_all<8>(q, p);
  } else {
    select_all<kMaxKeysPerLane>(q, p);
  }
  wait_vmcnt<0>();  // x is in LDS, too
  __syncthreads();
  // thread i holds pair i (at most 512)
  const int i = threadIdx.x, wave = i / kWave, lane = i % kWave;
  static_assert(kThreads >= kMaxPairs, "one pair per thread");
  int e = -1;
  if (i < p.T * p.k) {
    const int id = q.blob[i / p.k * 2 * p.k + i % p.k];
    if (id >= 0 && id < p.E && id >= p.e_begin && id - p.e_begin < p.n_local) e = id - p.e_begin;
  }
  if (e >= 0) q.first[e] = 0x7FFFFFFF;
  __syncthreads();
  if (e >= 0) atomicMin(&q.first[e], i);
  __syncthreads();
  const bool on = e >= 0 && q.first[e] == i;
  const uint64_t b = __ballot(on);
  if (lane == 0) q.wave_count[wave] = __popcll(b);
  __syncthreads();
  int n = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int c = q.wave_count[w];
    if (w < wave) n += c;
    all += c;
  }
  if (on) q.list[n + __popcll(b & ((1ull << lane) - 1))] = static_cast<uint16_t>(e);
  if (i == 0) q.count = all;
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

// What the down kernel needs of the routing, written by one workgroup of the gate/up kernel.
__device__ void write_tables(Pairs& q, const FewLayer& p) {
  for (int i = threadIdx.x; i < q.count * 16; i += kThreads) {
    const int a = i / 16, t = i % 16;
    float wt;
    const int j = t < p.T ? slot_of(q, p, t, q.list[a], wt) : -1;
    p.rows[i] = static_cast<int16_t>(j < 0 ? -1 : t * p.k + j);
    if (t == 0) p.list[a] = q.list[a];
  }
  for (int i = threadIdx.x; i < p.T * 2 * p.k; i += kThreads)
    if (p.packed_out) p.packed_out[i] = q.blob[i];
  if (threadIdx.x < kWave) {
    int bad = 0;
    for (int i = threadIdx.x; i < p.T * p.k; i += kWave) {
      const int id = q.blob[i / p.k * 2 * p.k + i % p.k];
      bad += id < 0 || id >= p.E;
    }
    bad = wave_sum_int(bad);
    if (threadIdx.x == 0) {
      *p.err = bad;
      *p.count = q.count;
    }
  }
}

// ---------------------------------------------------------------------------
// gate/up
// ---------------------------------------------------------------------------

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

// Bytes of one token's x in LDS: whole steps (zeros past D) and 16 bytes that put rows into
// different banks.
template <int W> __host__ __device__ constexpr int x_row_bytes(int D) {
  return steps_of<W>(D) * Wt<W>::EPS * act_bytes<W>() + 16;
}

// Units [u0, u1) of 16 channels, one after another by the whole workgroup: wave w multiplies its
// eighth of the reduction dimension, the parts are added in wave order in LDS.
// SHARED: the shared expert's channels; else units of list entry u / (I / 16).
template <int W, bool PACKED, bool XLDS, bool SHARED>
__device__ __forceinline__ void gate_up_units(const FewLayer& p, const Pairs& q, const uint8_t* xs, float* red, int u0,
                                              int u1) {
  constexpr int EPS = Wt<W>::EPS, NX = Wt<W>::NX, B = Wt<W>::GB, NBUF = Wt<W>::GN, as = act_bytes<W>();
  constexpr bool F32 = W == EL_F32;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int S = steps_of<W>(p.D), per = (SHARED ? p.I_shared : p.I) / 16;
  const int s0 = S * wave / kWaves, s1 = S * (wave + 1) / kWaves;
  const int nb = ((S + kWaves - 1) / kWaves + B - 1) / B;  // blocks per unit, the same for every wave
  const int total = (u1 - u0) * nb;
  const u32 voff = lane_offset<W, PACKED>(p.D, lane);
  // columns past the last token repeat it and are never read
  const int t = min(lrow, p.T - 1);
  const uint8_t* xl = xs + t * x_row_bytes<W>(p.D) + lgrp * (EPS / 4) * as;
  const uint8_t* xg = static_cast<const uint8_t*>(p.x) + static_cast<int64_t>(t) * p.D * as;

  struct Block {
    u32x4 w[2][B];
  };
  auto load = [&](Block& b, int i) {
    const int u = u0 + i / nb, j = i % nb;
    const int frag = __builtin_amdgcn_readfirstlane(u % per);
    const bool unit = i < total;
    int64_t eo = 0;
    if (!SHARED && unit) eo = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(q.list[u / per])) * p.gu_stride;
    const __amdgpu_buffer_rsrc_t r0 = weight_rsrc(static_cast<const uint8_t*>(SHARED ? p.sh_gate : p.w_gate) + eo);
    const __amdgpu_buffer_rsrc_t r1 = weight_rsrc(static_cast<const uint8_t*>(SHARED ? p.sh_up : p.w_up) + eo);
#pragma unroll
    for (int n = 0; n < B; ++n) {
      const int s = s0 + j * B + n;
      const bool real = unit && s < s1;
      const u32 v = real ? voff : kOutOfRange, o = step_offset<W, PACKED>(p.D, frag, s);
      b.w[0][n] = buffer_load16<PACKED>(r0, v, o);
      b.w[1][n] = buffer_load16<PACKED>(r1, v, o);
    }
  };

  f32x4 c0 = {0.f, 0.f, 0.f, 0.f}, c1 = {0.f, 0.f, 0.f, 0.f};
  const u32x4 z = {0u, 0u, 0u, 0u};
  float* buf = red;
  int known = -1, slot = -1;  // list entry whose slot and weight this thread's token has looked up
  float wt = 0.f;
  auto finish = [&](int u) {
    if (lrow < p.T) {
      float* o = buf + (wave * p.T + lrow) * 16 + lgrp * 4;
      *reinterpret_cast<f32x4*>(o) = c0;
      *reinterpret_cast<f32x4*>(o + kWaves * p.T * 16) = c1;
    }
    c0 = c1 = f32x4{0.f, 0.f, 0.f, 0.f};
    lds_barrier();
    if (static_cast<int>(threadIdx.x) < p.T * 16) {
      const int tt = threadIdx.x / 16, ch = threadIdx.x % 16, n = (u % per) * 16 + ch;
      float g = 0.f, v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        g += buf[(w * p.T + tt) * 16 + ch];
        v += buf[((kWaves + w) * p.T + tt) * 16 + ch];
      }
      if constexpr (SHARED) {
        store_h<F32>(p.h_sh, static_cast<int64_t>(p.T) * p.I_shared, static_cast<int64_t>(tt) * p.I_shared + n, silu(g) * v);
      } else {
        const int a = u / per, e = q.list[a];
        if (a != known) {
          slot = slot_of(q, p, tt, e, wt);
          known = a;
        }
        if (slot >= 0) {
          if constexpr (W == EL_E4M3) {
            g *= p.s_gate[static_cast<int64_t>(e) * p.I + n];
            v *= p.s_up[static_cast<int64_t>(e) * p.I + n];
          }
          store_h<F32>(p.h, static_cast<int64_t>(p.T) * p.k * p.I, (static_cast<int64_t>(tt) * p.k + slot) * p.I + n,
                       wt * (silu(g) * v));
        }
      }
    }
    // two buffers: the next unit's parts go into the other one; one buffer: wait until it is read
    if (p.red_bufs == 2) buf = buf == red ? red + 2 * kWaves * p.T * 16 : red;
    else lds_barrier();
  };
  auto use = [&](const Block& b, int i) {
    const int j = i % nb;
#pragma unroll
    for (int n = 0; n < B; ++n) {
      const int s = s0 + j * B + n;
      if (s < s1) {
#pragma unroll
        for (int m = 0; m < NX; ++m) {
          u32x4 xv;
          if constexpr (XLDS) {
            xv = *reinterpret_cast<const u32x4*>(xl + s * EPS * as + m * 16);
          } else {
            const int k0 = s * EPS + lgrp * (EPS / 4);
            xv = k0 < p.D ? reinterpret_cast<const u32x4*>(xg + static_cast<int64_t>(k0) * as)[m] : z;
          }
          c0 = mul<W>(weight_piece<W>(b.w[0][n], m), xv, c0);
          c1 = mul<W>(weight_piece<W>(b.w[1][n], m), xv, c1);
        }
      }
    }
    if (j == nb - 1) finish(u0 + i / nb);
  };

  Block ring[NBUF];
#pragma unroll
  for (int j = 0; j < NBUF - 1; ++j) load(ring[j], j);
  for (int i = 0; i < total; i += NBUF) {
#pragma unroll
    for (int j = 0; j < NBUF; ++j) {
      if (j > 0 && i + j >= total) break;
      load(ring[(j + NBUF - 1) % NBUF], i + j + NBUF - 1);
      __builtin_amdgcn_sched_barrier(0);
      use(ring[j], i + j);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// x into LDS rows of whole steps, zeros past D: the loads go straight into LDS and are complete
// after wait_vmcnt<0> and a barrier.
template <int W>
__device__ __forceinline__ void stage_x(const FewLayer& p, uint8_t* xs) {
  const int row = x_row_bytes<W>(p.D), pieces = (row - 16) / 16, real = p.D * act_bytes<W>() / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const __amdgpu_buffer_rsrc_t r = buffer_rsrc(p.x);
  for (int t = 0; t < p.T; ++t) {
    for (int c = wave * kWave; c < real; c += kThreads)
      if (c + lane < real) buffer_load16_to_lds(r, xs + t * row + c * 16, lane * 16, (t * real + c) * 16);
    for (int c = real + threadIdx.x; c < pieces; c += kThreads)
      *reinterpret_cast<u32x4*>(xs + t * row + c * 16) = u32x4{0u, 0u, 0u, 0u};
  }
}

// ---------------------------------------------------------------------------
// down
// ---------------------------------------------------------------------------

// Sum over blocks of 16 rows of W_down times h.  Blocks are DB steps of one matrix; this wave
// takes every `stride`-th from `first` on.  TWO: remainders of h are a second product, else
// columns 8 to 15.  SHARED: one matrix, h_sh; else one per list entry.
template <int W, bool PACKED, bool TWO, bool SHARED>
__device__ __forceinline__ f32x4 down_blocks(const FewLayer& p, const int16_t* rows, int count, int frag, int first,
                                             int stride) {
  constexpr int EPS = Wt<W>::EPS, NX = Wt<W>::NX, B = Wt<W>::DB, NBUF = TWO ? Wt<W>::DN2 : Wt<W>::DN;
  constexpr int as = act_bytes<W>();
  constexpr bool F32 = W == EL_F32;
  constexpr int NP = TWO && !F32 ? 2 : 1;  // pieces of h per weight piece
  const int lane = threadIdx.x % kWave, lrow = lane & 15, lgrp = lane >> 4;
  const int K = SHARED ? p.I_shared : p.I;
  const int S = steps_of<W>(K), nb = (S + B - 1) / B;
  const int blocks = count * nb;
  const u32 voff = lane_offset<W, PACKED>(K, lane);
  const int pair_rows = SHARED ? p.T : p.T * p.k;
  const u32 plane = static_cast<u32>(pair_rows) * K * as;  // bytes of the value plane
  const __amdgpu_buffer_rsrc_t rh = buffer_rsrc_sized(SHARED ? p.h_sh : p.h, F32 ? plane : 2 * plane);
  const int t = F32 || TWO ? lrow : lrow & 7;
  const u32 base = (!F32 && !TWO && lrow >= 8 ? plane : 0u) + lgrp * (EPS / 4) * as;

  struct Block {
    u32x4 w[B], h[B][NX][NP];
    float sd[W == EL_E4M3 ? 4 : 1];
    bool on;
  };
  auto load = [&](Block& b, int i) {
    const int id = first + i * stride;
    const bool there = id < blocks;
    const int a = there ? id / nb : 0, j = there ? id % nb : 0;
    int64_t eo = 0;
    int e = 0, row = t < p.T ? t : -1;
    if constexpr (!SHARED) {
      e = ld_scalar(p.list + a);
      eo = static_cast<int64_t>(e) * p.dn_stride;
      row = rows[a * 16 + t];
    }
    if (!there) row = -1;
    b.on = row >= 0;
    const __amdgpu_buffer_rsrc_t r = weight_rsrc(static_cast<const uint8_t*>(SHARED ? p.sh_down : p.w_down) + eo);
    const u32 ho = base + static_cast<u32>(max(row, 0)) * K * as;
    if constexpr (W == EL_E4M3) {
      const __amdgpu_buffer_rsrc_t rs = weight_rsrc(p.s_down + static_cast<int64_t>(e) * p.D);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        b.sd[n] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, there ? lgrp * 16 : kOutOfRange, (frag * 16 + n) * 4, 0));
    }
#pragma unroll
    for (int n = 0; n < B; ++n) {
      const int s = j * B + n;
      const bool real = there && s < S;
      b.w[n] = buffer_load16<PACKED>(r, real ? voff : kOutOfRange, step_offset<W, PACKED>(K, frag, s));
      // lanes without a row, or past the width, read nothing
      const u32 o = row >= 0 && s * EPS + lgrp * (EPS / 4) < K ? ho : kOutOfRange;
#pragma unroll
      for (int m = 0; m < NX; ++m) {
        b.h[n][m][0] = buffer_load16<false>(rh, o + m * 16, s * EPS * as);
        if constexpr (NP == 2) b.h[n][m][1] = buffer_load16<false>(rh, o + m * 16 + plane, s * EPS * as);
      }
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Block& b, int i) {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
    const int j = (first + i * stride) % nb;
#pragma unroll
    for (int n = 0; n < B; ++n) {
      if (j * B + n < S) {
#pragma unroll
        for (int m = 0; m < NX; ++m) {
          const u32x4 w = weight_piece<W>(b.w[n], m);
          c = mul<W>(w, b.h[n][m][0], c);
          if constexpr (NP == 2) c = mul<W>(w, b.h[n][m][1], c);
        }
      }
    }
    if constexpr (W == EL_E4M3) {
#pragma unroll
      for (int n = 0; n < 4; ++n) c[n] *= b.sd[n];
    }
    if (b.on) acc += c;
  };
  Block ring[NBUF];
  const int mine = first < blocks ? (blocks - first + stride - 1) / stride : 0;
#pragma unroll
  for (int j = 0; j < NBUF - 1; ++j) load(ring[j], j);
  for (int i = 0; i < mine; i += NBUF) {
#pragma unroll
    for (int j = 0; j < NBUF; ++j) {
      if (j > 0 && i + j >= mine) break;
      load(ring[(j + NBUF - 1) % NBUF], i + j + NBUF - 1);
      __builtin_amdgcn_sched_barrier(0);
      use(ring[j], i + j);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  return acc;
}

// Parts (of `parts`) of a launch for work of `part` out of `all`: at least one, not all.
inline int share_of(double part, double all, int parts) {
  const int n = static_cast<int>(parts * part / all + 0.5);
  return n < 1 ? 1 : n > parts - 1 ? parts - 1 : n;
}

// Workgroups (one per CU) and waves for the shared expert, by its share of the bytes, with as many
// distinct experts as T independent draws of k of E give.
inline void deal(FewLayer& p, double w_bytes, double act_bytes) {
  double miss = 1.0;
  for (int t = 0; t < p.T; ++t) miss *= 1.0 - static_cast<double>(p.k) / p.E;
  const double routed = p.n_local * (1.0 - miss) * p.I * w_bytes;
  const double shared = static_cast<double>(p.I_shared) * act_bytes;
  p.shared_blocks = p.I_shared ? share_of(shared, shared + routed, kCus) : 0;
  if (p.shared_blocks > p.I_shared / 16) p.shared_blocks = p.I_shared / 16;
  p.shared_waves = p.I_shared ? share_of(shared, shared + routed, kWaves) : 0;
}

}  // namespace few

void launch_few_logits(int act_el, const FewLayer& p, hipStream_t stream);
hipError_t launch_few_mx(FewLayer p, hipStream_t stream);

}  // namespace moe
