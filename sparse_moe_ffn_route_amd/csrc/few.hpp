// Device code shared by the kernels of the few-token layer (few.hip, few_mx.hip).
#pragma once

#include <type_traits>

#include <algorithm>

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
// Gate/up requests R steps of both matrices ahead; down blocks are DB steps of one matrix with
// their pieces of h, DN of them in the ring: 2 waves per SIMD have 256 registers each.
template <int W> struct Wt;
template <> struct Wt<EL_F32> {
  static constexpr int EPS = 16, NX = 1, R = 8, DB = 8, DN = 3;
};
template <> struct Wt<EL_BF16> {
  static constexpr int EPS = 32, NX = 1, R = 8, DB = 8, DN = 3;
};
template <> struct Wt<EL_E4M3> {
  static constexpr int EPS = 64, NX = 2, R = 8, DB = 4, DN = 4;
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
// Logits
// ---------------------------------------------------------------------------

// 16 waves split the width: at D = 4096 each has all its loads (8 steps of 16 experts) in flight at
// once, so the launch is a few memory latencies long.  (The shared expert's gate/up beside the logits, on CUs
// that are idle here, made this launch 1.5 us longer: one bf16 token 59.0 -> 59.9 us in all, four on 4-bit experts
// 58.2 -> 56.4.)
constexpr int kLogitWaves = 16;
constexpr int kNormWaves = 4;  // parts of a row's sum of squares: the waves of block_norm.hip

// 16 bytes as floats.
template <int EL>
__device__ __forceinline__ void unpack(const u32x4& a, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (EL == EL_F32) {
      v[i] = __uint_as_float(a[i]);
    } else {
      v[2 * i] = bf16_bits_to_f32(a[i] & 0xFFFFu);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}


// NORM: x = rms(r) * w_in, made here (the same arithmetic in the same order as block_norm.hip) and
// written by the first workgroup for the launches after this one.  By a workgroup of kLogitWaves waves.
template <int EL, bool NORM>
__device__ __forceinline__ void logits_block(const FewLayer& p, int block) {
  __shared__ f32x4 red[kLogitWaves][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int e0 = block * 16;
  constexpr int es = EL == EL_F32 ? 4 : 2;
  const int S = p.D * es / 64;
  const int s0 = S * wave / kLogitWaves, s1 = S * (wave + 1) / kLogitWaves;
  const int e = min(e0 + lrow, p.E - 1), t = min(lrow, p.T - 1);
  const uint8_t* wp = static_cast<const uint8_t*>(p.w_router) + static_cast<int64_t>(e) * p.D * es + lgrp * 16;
  const int64_t xo = static_cast<int64_t>(t) * p.D * es + lgrp * 16;
  const uint8_t* xp = static_cast<const uint8_t*>(NORM ? p.norm_r : p.x) + xo;
  const uint8_t* np = static_cast<const uint8_t*>(p.norm_w) + lgrp * 16;
  const u32x4 z = {0u, 0u, 0u, 0u};
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;
  u32x4 a[U], b[U], n[NORM ? U : 1];
  auto load_a = [&](int s) {
#pragma unroll
    for (int i = 0; i < U; ++i) a[i] = *reinterpret_cast<const u32x4*>(wp + static_cast<int64_t>(min(s + i, s1 - 1)) * 64);
  };
  if (s0 < s1) load_a(s0);
  float inv = 1.0f;
  if constexpr (NORM) {
    __shared__ float sums[kFewMaxT][kNormWaves];
    for (int j = wave; j < p.T * kNormWaves; j += kLogitWaves) {
      const int row = j / kNormWaves, part = j % kNormWaves;
      const uint8_t* rp = static_cast<const uint8_t*>(p.norm_r) + static_cast<int64_t>(row) * p.D * es;
      float ss = 0.f;
      for (int d = (part * kWave + lane) * 8; d < p.D; d += kNormWaves * kWave * 8) {
        const u32x4* q = reinterpret_cast<const u32x4*>(rp + static_cast<int64_t>(d) * es);
        float v[8];
        unpack<EL>(q[0], v);
        if constexpr (EL == EL_F32) unpack<EL>(q[1], v + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
      }
      ss = wave_sum(ss);
      if (lane == 0) sums[row][part] = ss;
    }
    __syncthreads();
    float ss = sums[t][0];
#pragma unroll
    for (int i = 1; i < kNormWaves; ++i) ss += sums[t][i];
    inv = 1.0f / sqrtf(ss / p.D + p.norm_eps);
  }
  for (int s = s0; s < s1; s += U) {
    if (s != s0) load_a(s);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int q = min(s + i, s1 - 1);
      b[i] = *reinterpret_cast<const u32x4*>(xp + static_cast<int64_t>(q) * 64);
      if constexpr (NORM) n[i] = *reinterpret_cast<const u32x4*>(np + static_cast<int64_t>(q) * 64);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (s + i >= s1) continue;
      if constexpr (NORM) {
        constexpr int V = 16 / es;
        float v[V], w[V];
        unpack<EL>(b[i], v);
        unpack<EL>(n[i], w);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = v[j] * inv * w[j];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[i][j] = EL == EL_F32 ? __float_as_uint(v[j]) : bf16x2_bits(v[2 * j % V], v[(2 * j + 1) % V]);
        if (block == 0 && lrow < p.T)
          *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(p.norm_x) + xo + static_cast<int64_t>(s + i) * 64) = b[i];
      }
      acc = mfma_chunk<EL>(a[i], lrow < p.T ? b[i] : z, acc);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 256) {
    const int l = threadIdx.x & 63, r = threadIdx.x >> 6;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kLogitWaves; ++w) v += red[w][l][r];
    const int tt = l & 15, ee = e0 + (l >> 4) * 4 + r;
    if (tt < p.T && ee < p.E) p.logits[static_cast<int64_t>(tt) * p.E + ee] = v;
  }
}

// ---------------------------------------------------------------------------
// The call's routing: (token, slot) pairs, and the experts they name
// ---------------------------------------------------------------------------

// An entry is a chosen local expert with up to a kernel's limit of its tokens ("members", by token):
// x: expert | rank0 << 16, y: token mask of the expert | row << 16.  Its members are the ranks
// rank0, rank0 + 1, ... of the mask's tokens, their rows of h the rows from `row` on.
__device__ __forceinline__ int entry_expert(int2 e) { return e.x & 0xFFFF; }
__device__ __forceinline__ int entry_rank0(int2 e) { return static_cast<int>(static_cast<u32>(e.x) >> 16); }
__device__ __forceinline__ u32 entry_mask(int2 e) { return static_cast<u32>(e.y) & 0xFFFFu; }
__device__ __forceinline__ int entry_row(int2 e) { return static_cast<int>(static_cast<u32>(e.y) >> 16); }
__device__ __forceinline__ int entry_members(int2 e, int limit) {
  return min(limit, __popc(entry_mask(e)) - entry_rank0(e));
}

struct Route {
  int32_t blob[2 * kMaxPairs];      // [T][2][k], as the packed routing blob
  float weight[kMaxPairs];          // by row of h: routing weight
  uint8_t token[kMaxPairs];         // and token
  int2 entry[kMaxPairs];
  u32 sums[kWaves];
  int entries;
};
// Scratch of route_call, at the start of the dynamic LDS (the reductions' place later): two words per
// local expert.
constexpr size_t kRouteScratch = 2 * 1024 * sizeof(u32);

// A key's place among keys, in its 16 highest bits: larger for larger keys, equal for both zeros.
__device__ __forceinline__ u32 key_place(float k) {
  const u32 b = __float_as_uint(k + 0.0f);
  return (b & 0x80000000u ? ~b : b | 0x80000000u) >> 16;
}

// Top-k of one token by one wave: the same keys, order and weights as select_topk (topk.hpp), in
// about a fifth of its time for 512 keys.  The k-th largest of the lanes' own best keys bounds the
// k-th largest of all from below, and so does what its 16 highest bits say, which 16 counts over the
// lanes find; the keys that reach it (a few more than k) are ranked against each other.  More than 64
// of them (many equal keys) take select_topk.
template <int PL>
__device__ __forceinline__ void select_few(const float (&key)[PL], int E, int k, int renormalize,
                                           float2* __restrict__ cand, int32_t* __restrict__ out) {
  const int lane = threadIdx.x % kWave;
  u32 best = 0;  // below every key's place
  bool nan = false;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    nan |= key[i] != key[i];
    if (lane + i * kWave < E) best = max(best, key_place(key[i]));
  }
  u32 least = 0;  // min(E, 64) >= k lanes have a key, so at least k reach it
#pragma unroll
  for (int bit = 15; bit >= 0; --bit) {
    const u32 at = least | 1u << bit;
    if (__popcll(__ballot(best >= at)) >= k) least = at;
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + i * kWave;
    const bool on = e < E && key_place(key[i]) >= least;
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

// Every wave's tokens; `beside` runs between the loads of their logits and the selection.
template <int PL, typename F>
__device__ __forceinline__ void select_all(Route& q, const FewLayer& p, const F& beside) {
  constexpr int N = kFewMaxT / kWaves;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  float key[N][PL], bias[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = min(lane + i * kWave, p.E - 1);
#pragma unroll
    for (int n = 0; n < N; ++n)
      key[n][i] = p.logits[static_cast<int64_t>(min(wave + n * kWaves, p.T - 1)) * p.E + e];
    bias[i] = p.bias ? p.bias[e] : 0.0f;
  }
  beside();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int t = wave + n * kWaves;
    if (t >= p.T) break;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      key[n][i] = lane + i * kWave < p.E ? key[n][i] : -INFINITY;
      if (p.bias) key[n][i] = key[n][i] + bias[i];
    }
    select_few(key[n], p.E, p.k, p.renormalize, reinterpret_cast<float2*>(q.entry) + wave * kWave, q.blob + t * 2 * p.k);
  }
}

// The call's routing by all threads: given, or selected from the logits; then the experts it names,
// in the order of the first pairs that do, as entries of up to LIMIT members.  The workgroup
// with `write` set also writes the down kernel's entries (of up to DOWN_LIMIT), the blob and the
// error word.  `beside`, work that needs no routing, runs while the logits are on their way.
template <int LIMIT, int DOWN_LIMIT, typename F>
__device__ __forceinline__ void route_call(Route& q, uint8_t* scratch, const FewLayer& p, bool write, const F& beside) {
  static_assert(sizeof(q.entry) >= kWaves * kWave * sizeof(float2), "selection candidates");
  static_assert(kThreads >= kMaxPairs, "one pair per thread");
  int32_t* first = reinterpret_cast<int32_t*>(scratch);  // first pair that names each expert, then its first row
  u32* mask = reinterpret_cast<u32*>(scratch) + 1024;    // its tokens
  for (int e = threadIdx.x; e < p.n_local; e += kThreads) {
    first[e] = 0x7FFFFFFF;
    mask[e] = 0u;
  }
  if (p.packed_in) {
    constexpr int N = 2 * kMaxPairs / kThreads;
    int32_t v[N];
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = p.packed_in[min(static_cast<int>(threadIdx.x) + n * kThreads, p.T * 2 * p.k - 1)];
    beside();
#pragma unroll
    for (int n = 0; n < N; ++n) q.blob[threadIdx.x + n * kThreads] = v[n];
  } else if (p.E <= 2 * kWave) {
    select_all<2>(q, p, beside);
  } else if (p.E <= 8 * kWave) {
    select_all<8>(q, p, beside);
  } else {
    select_all<kMaxKeysPerLane>(q, p, beside);
  }
  wait_vmcnt<0>();  // loads of x straight into LDS are complete, too
  __syncthreads();
  const int i = threadIdx.x, wave = i / kWave, lane = i % kWave;
  const int t = i / p.k, j = i - t * p.k, pairs = p.T * p.k;
  int e = -1;
  float w = 0.f;
  bool bad = false;
  if (i < pairs) {
    const int32_t* ids = q.blob + t * 2 * p.k;
    const int id = ids[j];
    bad = id < 0 || id >= p.E;
    if (!bad && id >= p.e_begin && id - p.e_begin < p.n_local) e = id - p.e_begin;
    w = __int_as_float(ids[p.k + j]);
    if (p.packed_in && e >= 0) {
      // a given token may name an expert again: its first slot takes all the weights
      for (int n = 0; n < p.k; ++n) {
        if (n == j || ids[n] != id) continue;
        if (n < j) e = -1;
        else w += __int_as_float(ids[p.k + n]);
      }
    }
  }
  if (e >= 0) {
    atomicMin(&first[e], i);
    atomicOr(&mask[e], 1u << t);
  }
  __syncthreads();
  const u32 m = e >= 0 ? mask[e] : 0u;
  const bool lead = e >= 0 && first[e] == i;
  const int members = __popc(m);
  // exclusive sums over the leading pairs before this one: rows, entries, the down kernel's entries
  u32 mine = lead ? members | ((members + LIMIT - 1) / LIMIT) << 10 | ((members + DOWN_LIMIT - 1) / DOWN_LIMIT) << 20 : 0u;
  u32 sum = mine;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const u32 v = static_cast<u32>(__shfl_up(static_cast<int>(sum), o, kWave));
    if (lane >= o) sum += v;
  }
  if (lane == kWave - 1) q.sums[wave] = sum;
  __syncthreads();
  u32 all = 0;
#pragma unroll
  for (int n = 0; n < kWaves; ++n) {
    const u32 v = q.sums[n];
    if (n < wave) sum += v;
    all += v;
  }
  sum -= mine;
  if (lead) {
    const int row = sum & 1023, at = (sum >> 10) & 1023, at_down = sum >> 20;
    first[e] = row;
    for (int n = 0; n * LIMIT < members; ++n)
      q.entry[at + n] = make_int2(e | (n * LIMIT) << 16, static_cast<int>(m | static_cast<u32>(row + n * LIMIT) << 16));
    if (write)
      for (int n = 0; n * DOWN_LIMIT < members; ++n)
        p.entry[at_down + n] =
            make_int2(e | (n * DOWN_LIMIT) << 16, static_cast<int>(m | static_cast<u32>(row + n * DOWN_LIMIT) << 16));
  }
  if (i == 0) q.entries = (all >> 10) & 1023;
  __syncthreads();
  if (e >= 0) {
    const int r = first[e] + __popc(m & ((1u << t) - 1));
    q.weight[r] = w;
    q.token[r] = static_cast<uint8_t>(t);
  }
  if (write) {
    if (p.packed_out)
      for (int n = i; n < 2 * pairs; n += kThreads) p.packed_out[n] = q.blob[n];
    const uint64_t b = __ballot(bad);
    if (lane == 0) q.sums[wave] = __popcll(b);
    __syncthreads();
    if (i == 0) {
      int n = 0;
      for (int v = 0; v < kWaves; ++v) n += q.sums[v];
      *p.err = n;
      *p.entries = all >> 20;
    }
  }
  __syncthreads();
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
// eighth of the reduction dimension, the parts are added in wave order in LDS.  Each wave requests
// R steps ahead, the last R of a unit being followed by the next unit's first; as compiled, the first
// step of each R waits for all of them (few.hip).
// SHARED: the shared expert, every token a column; else units of entry u / (I / 16), its members
// the columns.
template <int W, bool PACKED, bool XLDS, bool SHARED>
__device__ __forceinline__ void gate_up_units(const FewLayer& p, const Route& q, const uint8_t* xs, float* red, int u0,
                                              int u1) {
  constexpr int EPS = Wt<W>::EPS, NX = Wt<W>::NX, R = Wt<W>::R, as = act_bytes<W>();
  constexpr bool F32 = W == EL_F32;
  if (u0 >= u1) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int S = steps_of<W>(p.D), per = (SHARED ? p.I_shared : p.I) / 16;
  const int s0 = S * wave / kWaves, s1 = S * (wave + 1) / kWaves;
  const int turns = ((S + kWaves - 1) / kWaves + R - 1) / R;  // of R steps per unit, the same for every wave
  const u32 voff = lane_offset<W, PACKED>(p.D, lane);
  const u32x4 z = {0u, 0u, 0u, 0u};
  struct Source {
    __amdgpu_buffer_rsrc_t r0, r1;
    u32 at;
    bool on;
  };
  auto source = [&](int u) {
    Source o;
    o.on = u < u1;
    int64_t eo = 0;
    if (!SHARED && o.on) eo = __builtin_amdgcn_readfirstlane(entry_expert(q.entry[u / per])) * p.gu_stride;
    o.r0 = weight_rsrc(static_cast<const uint8_t*>(SHARED ? p.sh_gate : p.w_gate) + eo);
    o.r1 = weight_rsrc(static_cast<const uint8_t*>(SHARED ? p.sh_up : p.w_up) + eo);
    o.at = step_offset<W, PACKED>(p.D, __builtin_amdgcn_readfirstlane(u % per), 0);
    return o;
  };
  u32x4 w0[R], w1[R];
  auto load = [&](int slot, const Source& o, int s) {
    const u32 v = o.on && s < s1 ? voff : kOutOfRange;
    const u32 at = o.at + s * (PACKED ? 1024 : 64);
    w0[slot] = buffer_load16<PACKED>(o.r0, v, at);
    w1[slot] = buffer_load16<PACKED>(o.r1, v, at);
  };
  Source cur = source(u0);
#pragma unroll
  for (int n = 0; n < R; ++n) load(n, cur, s0 + n);
  float* buf = red;
  const int cols = SHARED ? p.T : min(p.T, 16);
  for (int u = u0; u < u1; ++u) {
    // columns past the last member repeat it and are never read
    const int2 en = SHARED ? make_int2(0, 0) : q.entry[u / per];
    const int members = SHARED ? p.T : __popc(entry_mask(en)), row = entry_row(en);
    const int t = SHARED ? min(lrow, p.T - 1) : q.token[row + min(lrow, members - 1)];
    const uint8_t* xl = xs + t * x_row_bytes<W>(p.D) + lgrp * (EPS / 4) * as;
    const uint8_t* xg = static_cast<const uint8_t*>(p.x) + static_cast<int64_t>(t) * p.D * as;
    f32x4 c0 = {0.f, 0.f, 0.f, 0.f}, c1 = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < turns; ++k) {
      const bool last = k + 1 == turns;
      if (last) cur = source(u + 1);
      const int sl = last ? s0 : s0 + (k + 1) * R;
#pragma unroll
      for (int n = 0; n < R; ++n) {
        const int s = s0 + k * R + n;
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
            c0 = mul<W>(weight_piece<W>(w0[n], m), xv, c0);
            c1 = mul<W>(weight_piece<W>(w1[n], m), xv, c1);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        load(n, cur, sl + n);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (lrow < members) {
      float* o = buf + (wave * cols + lrow) * 16 + lgrp * 4;
      *reinterpret_cast<f32x4*>(o) = c0;
      *reinterpret_cast<f32x4*>(o + kWaves * cols * 16) = c1;
    }
    lds_barrier();
    const int c = threadIdx.x / 16, ch = threadIdx.x % 16, n = (u % per) * 16 + ch;
    if (c < members) {
      float g = 0.f, v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        g += buf[(w * cols + c) * 16 + ch];
        v += buf[((kWaves + w) * cols + c) * 16 + ch];
      }
      if constexpr (SHARED) {
        store_h<F32>(p.h_sh, static_cast<int64_t>(p.T) * p.I_shared, static_cast<int64_t>(c) * p.I_shared + n, silu(g) * v);
      } else {
        if constexpr (W == EL_E4M3) {
          const int64_t sc = static_cast<int64_t>(entry_expert(en)) * p.I + n;
          g *= p.s_gate[sc];
          v *= p.s_up[sc];
        }
        store_h<F32>(p.h, static_cast<int64_t>(p.T) * p.k * p.I, static_cast<int64_t>(row + c) * p.I + n,
                     q.weight[row + c] * (silu(g) * v));
      }
    }
    // two buffers: the next unit's parts go into the other one; one buffer: wait until it is read
    if (p.red_bufs == 2) buf = buf == red ? red + 2 * kWaves * cols * 16 : red;
    else lds_barrier();
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

constexpr int kDownMembers = 8;  // per entry: columns 8 to 15 are the remainders

// v in the lane of each of the entry's tokens, from the lane of the member that it is.
__device__ __forceinline__ f32x4 to_tokens(f32x4 v, int2 en, int limit) {
  const int lane = threadIdx.x % kWave, t = lane & 15;
  const u32 m = entry_mask(en);
  const int r = __popc(m & ((1u << t) - 1)) - entry_rank0(en);
  const bool on = ((m >> t) & 1u) && r >= 0 && r < limit;
  f32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float got = __int_as_float(__builtin_amdgcn_ds_bpermute(((lane & 48) + (r & 15)) * 4, __float_as_int(v[i])));
    o[i] = on ? got : 0.0f;
  }
  return o;
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
constexpr int kRor4 = 0x124, kRor8 = 0x128;  // rotate by 4 or 8 lanes within 16

// A wave's blocks first, first + stride, ... of `blocks`, as (hi, lo) = (id / radix, id % radix) without a
// division each; past the last one it stays on it.
struct Cursor {
  int hi, lo, left, dhi, dlo, radix;
  __device__ __forceinline__ Cursor(int first, int stride, int blocks, int r) : radix(r) {
    left = first < blocks ? (blocks - first + stride - 1) / stride : 0;
    hi = first / r;
    lo = first - hi * r;
    dhi = stride / r;
    dlo = stride - dhi * r;
  }
  __device__ __forceinline__ void next() {
    if (--left <= 0) return;
    hi += dhi;
    lo += dlo;
    if (lo >= radix) {
      lo -= radix;
      ++hi;
    }
  }
};

// Sum over blocks of 16 rows of W_down times h, in the lanes of the tokens.  Blocks are DB steps of
// one entry; this wave takes every `stride`-th from `first` on.  SHARED: entries are the call's
// tokens in eights.
template <int W, bool PACKED, bool SHARED>
__device__ __forceinline__ f32x4 down_blocks(const FewLayer& p, int entries, int frag, int first, int stride) {
  constexpr int EPS = Wt<W>::EPS, NX = Wt<W>::NX, B = Wt<W>::DB, NBUF = Wt<W>::DN, as = act_bytes<W>();
  constexpr bool F32 = W == EL_F32;
  const int lane = threadIdx.x % kWave, lrow = lane & 15, lgrp = lane >> 4;
  const int K = SHARED ? p.I_shared : p.I;
  const int S = steps_of<W>(K), nb = (S + B - 1) / B;
  const int blocks = entries * nb;
  if (blocks == 0) return f32x4{0.f, 0.f, 0.f, 0.f};
  const u32 voff = lane_offset<W, PACKED>(K, lane);
  const u32 plane = static_cast<u32>(SHARED ? p.T : p.T * p.k) * K * as;  // bytes of the value plane
  const __amdgpu_buffer_rsrc_t rh = buffer_rsrc_sized(SHARED ? p.h_sh : p.h, F32 ? plane : 2 * plane);
  const int c = lrow & (kDownMembers - 1);
  const u32 base = (!F32 && lrow >= kDownMembers ? plane : 0u) + lgrp * (EPS / 4) * as;

  // the shared expert's entries change first: the second read of a block hits L2
  auto entry = [&](const Cursor& at) {
    if constexpr (SHARED)
      return make_int2(at.lo * kDownMembers << 16, static_cast<int>(((1u << p.T) - 1) | at.lo * kDownMembers << 16));
    else
      return make_int2(ld_scalar(&p.entry[at.hi].x), ld_scalar(&p.entry[at.hi].y));
  };
  auto block_of = [&](const Cursor& at) { return SHARED ? at.hi : at.lo; };
  struct Block {
    u32x4 w[B], h[B][NX];
    float sd[W == EL_E4M3 ? 4 : 1];
  };
  auto load = [&](Block& b, Cursor& at) {
    const bool there = at.left > 0;
    const int2 en = entry(at);
    const int e = entry_expert(en), j = block_of(at);
    at.next();
    const __amdgpu_buffer_rsrc_t r = weight_rsrc(static_cast<const uint8_t*>(SHARED ? p.sh_down : p.w_down) +
                                                 static_cast<int64_t>(e) * p.dn_stride);
    const bool on = there && c < entry_members(en, kDownMembers);
    const u32 ho = base + static_cast<u32>(entry_row(en) + c) * K * as;
    if constexpr (W == EL_E4M3) {
      const __amdgpu_buffer_rsrc_t rs = weight_rsrc(p.s_down + static_cast<int64_t>(e) * p.D);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        b.sd[n] = __uint_as_float(
            __builtin_amdgcn_raw_buffer_load_b32(rs, there ? lgrp * 16 : kOutOfRange, (frag * 16 + n) * 4, 0));
    }
#pragma unroll
    for (int n = 0; n < B; ++n) {
      const int s = j * B + n;
      const bool real = there && s < S;
      b.w[n] = buffer_load16<PACKED>(r, real ? voff : kOutOfRange, step_offset<W, PACKED>(K, frag, s));
      // lanes without a member, or past the width, read nothing
      const u32 o = on && s * EPS + lgrp * (EPS / 4) < K ? ho : kOutOfRange;
#pragma unroll
      for (int m = 0; m < NX; ++m) b.h[n][m] = buffer_load16<false>(rh, o + m * 16, s * EPS * as);
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Block& b, Cursor& at) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    const int j = block_of(at);
    const int2 en = entry(at);
    at.next();
#pragma unroll
    for (int n = 0; n < B; ++n)
      if (j * B + n < S)
#pragma unroll
        for (int m = 0; m < NX; ++m) v = mul<W>(weight_piece<W>(b.w[n], m), b.h[n][m], v);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      if constexpr (W == EL_E4M3) v[n] *= b.sd[n];
      if constexpr (!F32) v[n] = dpp_add<kRor8>(v[n]);
    }
    acc += to_tokens(v, en, kDownMembers);
  };
  Cursor ahead(first, stride, blocks, SHARED ? entries : nb), here = ahead;
  if (here.left == 0) return acc;
  Block ring[NBUF];
#pragma unroll
  for (int j = 0; j < NBUF - 1; ++j) load(ring[j], ahead);
  for (;;) {
#pragma unroll
    for (int j = 0; j < NBUF; ++j) {
      load(ring[(j + NBUF - 1) % NBUF], ahead);
      __builtin_amdgcn_sched_barrier(0);
      use(ring[j], here);
      __builtin_amdgcn_sched_barrier(0);
      if (here.left == 0) return acc;
    }
  }
}

// The waves' sums for 16 channels -> y; red: one f32x4 per thread, written before by this function.
template <int OUT>
__device__ __forceinline__ void finish_down(const FewLayer& p, int frag, f32x4 acc, f32x4 (&red)[kWaves][kWave]) {
  red[threadIdx.x / kWave][threadIdx.x % kWave] = acc;
  __syncthreads();
  const int t = threadIdx.x / 16, ch = threadIdx.x % 16, l = (ch / 4) * 16 + t;
  if (t >= p.T) return;
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) v += red[w][l][ch % 4];
  const int64_t idx = static_cast<int64_t>(t) * p.D + frag * 16 + ch;
  if constexpr (OUT == EL_F32) static_cast<float*>(p.y)[idx] = v;
  else static_cast<uint16_t*>(p.y)[idx] = static_cast<uint16_t>(bf16x2_bits(v, 0.f));
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
