// The few-token layer (few.hip) on microscaled 4-bit weights.
//
// The codes and block scales go into the scaled MFMA as they are; the other operand is the
// activation as a sum of e4m3 terms with a power of two per 32 values,
//   v = t0 2^e + t1 2^(e-5) + t2 2^(e-10) + t3 2^(e-15),  e = floor(log2(max |v|)) - 7,
// each term the rounding of what the terms before it left.  A term carries four significant
// bits and leaves a remainder of at most 2^-4 of itself, so two terms hold a bf16 x exactly
// (to 2^-22 of the block's largest value) and four hold h to 2^-17.  Columns the tokens do
// not need carry the further terms, so up to 8 tokens one product per step does for x, and
// up to 4 tokens for h.  Decoding the weights to bf16 instead takes sixteen conversions and four
// MFMAs per KB and bound both kernels by instruction issue (4.0 TB/s at 4 tokens).
//
// Lane g of a column holds, of a step's 128 values, 16 g .. + 15 and 64 + 16 g .. + 15 in its
// e4m3 operand, and the scale of values 32 g .. + 31.
#include "few.hpp"
#include "mx.hpp"

namespace moe {

namespace {

using namespace few;

constexpr int kTerms = 4;      // terms of h
constexpr int kTermStep = 5;   // exponent between terms
constexpr int kUnit = 32;      // channels per gate/up unit: one block of h

// Two e4m3 values of the low 16 bits.
__device__ __forceinline__ float e4m3_lo(u32 v) { return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(v), 0); }
__device__ __forceinline__ float e4m3_hi(u32 v) { return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(v), 1); }

// Scale byte of term 0 from the block's largest magnitude (255: the block holds a NaN or an
// infinity); the floor keeps every term's byte positive.
__device__ __forceinline__ int term_scale(u32 amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255;
  const int b = static_cast<int>(amax_bits >> 23) - 7;
  return b < 17 ? 17 : b;
}

__device__ __forceinline__ f32x4 mx_mul(const u32x4& a, const u32x4& b0, const u32x4& b1, f32x4 c, u32 sa, u32 sb) {
  const u32x4 z = {0u, 0u, 0u, 0u};
  const i32x8 av = __builtin_bit_cast(i32x8, __builtin_shufflevector(a, z, 0, 1, 2, 3, 4, 5, 6, 7));
  const i32x8 bv = __builtin_bit_cast(i32x8, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7));
  // A: fp4 (format 4); B: e4m3 (format 0); byte 0 of the scale registers
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 0, 0, static_cast<int>(sa), 0,
                                                          static_cast<int>(sb));
}

// Byte offsets in a matrix's image: run of step s of fragment `frag` (lane part lane * 16), and the
// scale byte of step s (lane part lane * 4).
__device__ __forceinline__ u32 run_offset(u32 frag_at, int s) { return frag_at + (s >> 2) * kMxGroupBytes + (s & 3) * kMxRun; }
__device__ __forceinline__ u32 byte_offset(u32 frag_at, int s, int S) {
  const int g = s >> 2;
  return frag_at + g * kMxGroupBytes + min(4, S - 4 * g) * kMxRun + (s & 3);
}

// ---------------------------------------------------------------------------
// x as two terms
// ---------------------------------------------------------------------------

// Rows [token][term], each of whole steps' bytes and 16 more (other banks for other rows), then
// one scale byte per row and block.
__host__ __device__ constexpr int xt_row(int D) { return mx_steps(D) * kMxStep + 16; }
__host__ __device__ constexpr int xt_blocks(int D) { return mx_steps(D) * 4; }
__host__ __device__ constexpr int xt_bytes(int T, int D) { return 2 * T * (xt_row(D) + xt_blocks(D)); }

// By all threads of a workgroup: four lanes a block, eight values each.  first / stride: tokens.
__device__ __forceinline__ void make_terms(const FewLayer& p, uint8_t* xt, int first, int stride) {
  const int row = xt_row(p.D), blocks = xt_blocks(p.D);
  uint8_t* scales = xt + 2 * p.T * row;
  for (int t = first; t < p.T; t += stride)
    for (int c = threadIdx.x; c < blocks * 4; c += kThreads) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (c * 8 < p.D) {
        const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) +
                                                        static_cast<int64_t>(t) * p.D + c * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = bf16_bits_to_f32(a[i] & 0xFFFFu);
          v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
        }
      }
      u32 m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, mx_abs_bits(v[i]));
      m = max(m, static_cast<u32>(__shfl_xor(static_cast<int>(m), 1, kWave)));
      m = max(m, static_cast<u32>(__shfl_xor(static_cast<int>(m), 2, kWave)));
      const int b = term_scale(m);
      u32 t0[2] = {0u, 0u}, t1[2] = {0u, 0u};
      if (b != 255) {
        const float inv = ldexpf(1.0f, 127 - b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a0 = v[2 * i] * inv, a1 = v[2 * i + 1] * inv;
          const u32 hi = f32x2_to_e4m3x2(a0, a1);
          const u32 lo = f32x2_to_e4m3x2((a0 - e4m3_lo(hi)) * 32.0f, (a1 - e4m3_hi(hi)) * 32.0f);
          t0[i / 2] |= hi << (16 * (i & 1));
          t1[i / 2] |= lo << (16 * (i & 1));
        }
      }
      *reinterpret_cast<uint2*>(xt + (2 * t) * row + c * 8) = make_uint2(t0[0], t0[1]);
      *reinterpret_cast<uint2*>(xt + (2 * t + 1) * row + c * 8) = make_uint2(t1[0], t1[1]);
      if ((c & 3) == 0) {
        scales[(2 * t) * blocks + c / 4] = static_cast<uint8_t>(b);
        scales[(2 * t + 1) * blocks + c / 4] = static_cast<uint8_t>(b == 255 ? 255 : b - kTermStep);
      }
    }
}

// For tokens too wide for LDS: the same into the workspace, one workgroup per token.
__global__ __launch_bounds__(kThreads) void few_terms_kernel(FewLayer p) {
  make_terms(p, static_cast<uint8_t*>(p.x_terms), blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------------------
// gate/up
// ---------------------------------------------------------------------------

// Rows of h: [T * k][term] of whole steps' bytes, then a scale byte per row, term and block.
__host__ __device__ constexpr int ht_row(int I) { return mx_steps(I) * kMxStep; }
__host__ __device__ constexpr int ht_blocks(int I) { return mx_steps(I) * 4; }

// Units [u0, u1) of 32 channels of the routed experts; TWO: a product per term, else term 1 in
// columns 8 to 15.
template <bool TWO>
__device__ __forceinline__ void mx_gate_up_units(const FewLayer& p, const Pairs& q, const uint8_t* xt, float* red,
                                                 int u0, int u1) {
  constexpr int B = 2, NBUF = 4, NP = TWO ? 2 : 1;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int S = mx_steps(p.D), per = p.I / kUnit;
  const int s0 = S * wave / kWaves, s1 = S * (wave + 1) / kWaves;
  const int nb = ((S + kWaves - 1) / kWaves + B - 1) / B;
  const int total = (u1 - u0) * nb;
  const u32 frag_bytes = static_cast<u32>(mx_fragment_bytes(p.D));
  const int row = xt_row(p.D), blocks = xt_blocks(p.D);
  const int t = min(TWO ? lrow : lrow & 7, p.T - 1), term = TWO ? 0 : lrow >> 3;
  const uint8_t* xr = xt + (2 * t + term) * row + lgrp * 16;
  const uint8_t* xsc = xt + 2 * p.T * row + (2 * t + term) * blocks + lgrp;

  struct Block {
    u32x4 w[2][2][B];  // matrix, fragment
    u32 sc[2][2][B];
  };
  auto load = [&](Block& b, int i) {
    const int u = u0 + i / nb, j = i % nb;
    const bool unit = i < total;
    int64_t eo = 0;
    if (unit) eo = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(q.list[u / per])) * p.gu_stride;
    const __amdgpu_buffer_rsrc_t r0 = weight_rsrc(static_cast<const uint8_t*>(p.w_gate) + eo);
    const __amdgpu_buffer_rsrc_t r1 = weight_rsrc(static_cast<const uint8_t*>(p.w_up) + eo);
    const u32 f0 = static_cast<u32>(__builtin_amdgcn_readfirstlane(u % per)) * 2 * frag_bytes;
#pragma unroll
    for (int n = 0; n < B; ++n) {
      const int s = s0 + j * B + n;
      const bool real = unit && s < s1;
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const u32 at = f0 + f * frag_bytes;
        const u32 o = run_offset(at, s), so = byte_offset(at, s, S);
        const u32 v = real ? lane * 16 : kOutOfRange, vs = real ? lane * 4 : kOutOfRange;
        b.w[0][f][n] = buffer_load16<true>(r0, v, o);
        b.w[1][f][n] = buffer_load16<true>(r1, v, o);
        b.sc[0][f][n] = __builtin_amdgcn_raw_buffer_load_b8(r0, vs, so, 0);
        b.sc[1][f][n] = __builtin_amdgcn_raw_buffer_load_b8(r1, vs, so, 0);
      }
    }
  };

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 c[2][2] = {{zero, zero}, {zero, zero}};
  float* buf = red;
  int known = -1, slot = -1;
  float wt = 0.f;
  const int tt = threadIdx.x / kUnit, ch = threadIdx.x % kUnit;
  const bool mine = static_cast<int>(threadIdx.x) < p.T * kUnit;
  // this wave's 32 channels of matrix m for every token -> LDS
  auto put = [&](int m, float* o) {
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      f32x4 v = c[m][f];
      if constexpr (!TWO) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v[i]), 0x128, 0xF, 0xF, false));  // row_ror:8
      }
      if (lrow < p.T) *reinterpret_cast<f32x4*>(o + (wave * p.T + lrow) * kUnit + f * 16 + lgrp * 4) = v;
      c[m][f] = zero;
    }
  };
  auto sum = [&](const float* o) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += o[(w * p.T + tt) * kUnit + ch];
    return v;
  };
  auto finish = [&](int u) {
    const int part = kWaves * p.T * kUnit;
    float g = 0.f, v = 0.f;
    if (p.red_bufs == 2) {  // both matrices in each of two buffers: one barrier per unit
      put(0, buf);
      put(1, buf + part);
      lds_barrier();
      if (mine) {
        g = sum(buf);
        v = sum(buf + part);
      }
      buf = buf == red ? red + 2 * part : red;
    } else {                // one matrix at a time
      put(0, red);
      lds_barrier();
      if (mine) g = sum(red);
      lds_barrier();
      put(1, red);
      lds_barrier();
      if (mine) v = sum(red);
      lds_barrier();
    }
    if (!mine) return;
    const int a = u / per;
    if (a != known) {
      slot = slot_of(q, p, tt, q.list[a], wt);
      known = a;
    }
    if (slot < 0) return;  // the same for a token's 32 threads
    const float h = wt * (silu(g) * v);
    u32 m = mx_abs_bits(h);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, static_cast<u32>(__shfl_xor(static_cast<int>(m), o, kWave)));
    const int b = term_scale(m);
    const int hrow = ht_row(p.I), hblocks = ht_blocks(p.I);
    const int64_t r = (static_cast<int64_t>(tt) * p.k + slot) * kTerms;
    uint8_t* out = static_cast<uint8_t*>(p.h);
    uint8_t* out_sc = out + static_cast<int64_t>(p.T) * p.k * kTerms * hrow;
    float rest = b == 255 ? 0.0f : h * ldexpf(1.0f, 127 - b);
#pragma unroll
    for (int i = 0; i < kTerms; ++i) {
      const u32 code = f32x2_to_e4m3x2(rest, 0.0f);
      out[(r + i) * hrow + (u % per) * kUnit + ch] = static_cast<uint8_t>(code);
      rest = (rest - e4m3_lo(code)) * 32.0f;
      if (ch == 0) out_sc[(r + i) * hblocks + u % per] = static_cast<uint8_t>(b == 255 ? 255 : b - i * kTermStep);
    }
  };
  auto use = [&](const Block& b, int i) {
    const int j = i % nb;
#pragma unroll
    for (int n = 0; n < B; ++n) {
      const int s = s0 + j * B + n;
      if (s < s1) {
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          const uint8_t* xp = xr + e * row + s * kMxStep;
          const u32x4 b0 = *reinterpret_cast<const u32x4*>(xp), b1 = *reinterpret_cast<const u32x4*>(xp + 64);
          const u32 sb = xsc[e * blocks + s * 4];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int f = 0; f < 2; ++f) c[m][f] = mx_mul(b.w[m][f][n], b0, b1, c[m][f], b.sc[m][f][n], sb);
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

template <bool TWO, bool XLDS>
__global__ __launch_bounds__(kThreads, 2) void few_mx_gate_up_kernel(FewLayer p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ Pairs q;
  float* red = reinterpret_cast<float*>(lds);
  if (static_cast<int>(blockIdx.x) < p.shared_blocks) {
    // the shared expert is bf16: it takes x as it is
    constexpr int W = EL_BF16;
    uint8_t* xs = lds + p.shared_red_bufs * 2 * kWaves * p.T * 16 * sizeof(float);
    if constexpr (XLDS) {
      stage_x<W>(p, xs);
      wait_vmcnt<0>();
      __syncthreads();
    }
    const int units = p.I_shared / 16, b = blockIdx.x;
    FewLayer ps = p;
    ps.red_bufs = p.shared_red_bufs;
    gate_up_units<W, true, XLDS, true>(ps, q, xs, red, units * b / p.shared_blocks, units * (b + 1) / p.shared_blocks);
    return;
  }
  uint8_t* xt = XLDS ? lds + (p.red_bufs == 2 ? 4 : 1) * kWaves * p.T * kUnit * sizeof(float)
                     : static_cast<uint8_t*>(p.x_terms);
  if constexpr (XLDS) make_terms(p, xt, 0, 1);
  route_call(q, p);
  const int b = blockIdx.x - p.shared_blocks, blocks = gridDim.x - p.shared_blocks;
  if (b == blocks - 1) write_tables(q, p);
  const int units = __builtin_amdgcn_readfirstlane(q.count) * (p.I / kUnit);
  mx_gate_up_units<TWO>(p, q, xt, red, static_cast<int>(static_cast<int64_t>(units) * b / blocks),
                        static_cast<int>(static_cast<int64_t>(units) * (b + 1) / blocks));
}

// ---------------------------------------------------------------------------
// down
// ---------------------------------------------------------------------------

// NB products per step: 1 (all four terms in columns, up to 4 tokens), 2 (two in columns, up to 8) or
// 4.  Blocks of DB steps, DN in the ring.
template <int NB> struct MxDown;
template <> struct MxDown<1> { static constexpr int DB = 2, DN = 6; };
template <> struct MxDown<2> { static constexpr int DB = 2, DN = 4; };
template <> struct MxDown<4> { static constexpr int DB = 1, DN = 5; };

template <int NB>
__device__ __forceinline__ f32x4 mx_down_blocks(const FewLayer& p, const int16_t* rows, int count, int frag, int first,
                                                int stride) {
  constexpr int B = MxDown<NB>::DB, NBUF = MxDown<NB>::DN;
  const int lane = threadIdx.x % kWave, lrow = lane & 15, lgrp = lane >> 4;
  const int S = mx_steps(p.I), nb = (S + B - 1) / B;
  const int blocks = count * nb;
  const u32 frag_at = static_cast<u32>(frag) * static_cast<u32>(mx_fragment_bytes(p.I));
  const int hrow = ht_row(p.I), hblocks = ht_blocks(p.I);
  const u32 codes = static_cast<u32>(p.T) * p.k * kTerms * hrow;  // bytes of the terms, then their scales
  const __amdgpu_buffer_rsrc_t rh = buffer_rsrc_sized(p.h, codes + static_cast<u32>(p.T) * p.k * kTerms * hblocks);
  constexpr int kCols = 4 * NB;  // tokens in columns
  const int t = lrow & (kCols - 1), term = lrow / kCols;
  struct Block {
    u32x4 w[B], h[B][NB][2];
    u32 sc[B], hs[B][NB];
    bool on;
  };
  auto load = [&](Block& b, int i) {
    const int id = first + i * stride;
    const bool there = id < blocks;
    const int a = there ? id / nb : 0, j = there ? id % nb : 0;
    const int row = there ? rows[a * 16 + t] : -1;
    b.on = row >= 0;
    const __amdgpu_buffer_rsrc_t r =
        weight_rsrc(static_cast<const uint8_t*>(p.w_down) + static_cast<int64_t>(ld_scalar(p.list + a)) * p.dn_stride);
#pragma unroll
    for (int n = 0; n < B; ++n) {
      const int s = j * B + n;
      const bool real = there && s < S;
      b.w[n] = buffer_load16<true>(r, real ? lane * 16 : kOutOfRange, run_offset(frag_at, s));
      b.sc[n] = __builtin_amdgcn_raw_buffer_load_b8(r, real ? lane * 4 : kOutOfRange, byte_offset(frag_at, s, S), 0);
#pragma unroll
      for (int e = 0; e < NB; ++e) {
        // terms e * 4 / NB + (column's own); values past the width are padded by zero weights, whose
        // operand must not be a stray NaN: their blocks read nothing
        const u32 rt = static_cast<u32>(max(row, 0)) * kTerms + e * (4 / NB) + term;
        const int k0 = s * kMxStep + lgrp * 16;
        const u32 at = row >= 0 && s < S ? rt * hrow + k0 : kOutOfRange;
        const u32 at_sc = row >= 0 && s < S ? codes + rt * hblocks + s * 4 + lgrp : kOutOfRange;
        b.h[n][e][0] = buffer_load16<false>(rh, at, 0);
        b.h[n][e][1] = buffer_load16<false>(rh, k0 + 64 < p.I ? at + 64 : kOutOfRange, 0);
        b.hs[n][e] = __builtin_amdgcn_raw_buffer_load_b8(rh, s * kMxStep + lgrp * 32 < p.I ? at_sc : kOutOfRange, 0, 0);
      }
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Block& b, int i) {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
    const int j = (first + i * stride) % nb;
#pragma unroll
    for (int n = 0; n < B; ++n)
      if (j * B + n < S)
#pragma unroll
        for (int e = 0; e < NB; ++e) c = mx_mul(b.w[n], b.h[n][e][0], b.h[n][e][1], c, b.sc[n], b.hs[n][e]);
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

template <int NB, int OUT>
__global__ __launch_bounds__(kThreads, 2) void few_mx_down_kernel(FewLayer p) {
  __shared__ int16_t rows[kMaxPairs * 16];
  __shared__ f32x4 red[kWaves][kWave], red_sh[kWaves][kWave];
  constexpr bool TWO = NB == 4;  // as the shared expert's bf16 h counts it: more than 8 tokens
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int frag = blockIdx.x, routed = kWaves - p.shared_waves;
  const int count = ld_scalar(p.count);
  for (int i = threadIdx.x; i < count * 16; i += kThreads) rows[i] = p.rows[i];
  __syncthreads();
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 c = zero, cs = zero;
  if (wave < routed) c = mx_down_blocks<NB>(p, rows, count, frag, wave, routed);
  else cs = down_blocks<EL_BF16, true, TWO, true>(p, rows, 1, frag, wave - routed, p.shared_waves);
  red[wave][lane] = c;
  red_sh[wave][lane] = cs;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < p.T * 16) {
    const int tt = threadIdx.x / 16, ch = threadIdx.x % 16;
    const int l = (ch / 4) * 16 + tt;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
#pragma unroll
      for (int o = 0; o < 16; o += 4 * NB) v += red[w][l + o][ch % 4];
      v += red_sh[w][l][ch % 4];
      if constexpr (!TWO) v += red_sh[w][l + 8][ch % 4];
    }
    const int64_t idx = static_cast<int64_t>(tt) * p.D + frag * 16 + ch;
    if constexpr (OUT == EL_F32) static_cast<float*>(p.y)[idx] = v;
    else static_cast<uint16_t*>(p.y)[idx] = static_cast<uint16_t>(bf16x2_bits(v, 0.f));
  }
}

template <bool XLDS>
void launch_gate_up(const FewLayer& p, int grid, size_t lds, hipStream_t stream) {
  if (p.T > 8) hipLaunchKernelGGL((few_mx_gate_up_kernel<true, XLDS>), dim3(grid), dim3(kThreads), lds, stream, p);
  else hipLaunchKernelGGL((few_mx_gate_up_kernel<false, XLDS>), dim3(grid), dim3(kThreads), lds, stream, p);
}

template <int OUT>
void launch_down(const FewLayer& p, hipStream_t stream) {
  const dim3 grid(p.D / 16), block(kThreads);
  if (p.T <= 4) hipLaunchKernelGGL((few_mx_down_kernel<1, OUT>), grid, block, 0, stream, p);
  else if (p.T <= 8) hipLaunchKernelGGL((few_mx_down_kernel<2, OUT>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((few_mx_down_kernel<4, OUT>), grid, block, 0, stream, p);
}

}  // namespace

size_t few_mx_x_bytes(int T, int D) { return static_cast<size_t>(xt_bytes(T, D)); }
size_t few_mx_h_bytes(int T, int k, int I) {
  return static_cast<size_t>(T) * k * kTerms * (ht_row(I) + ht_blocks(I));
}

hipError_t launch_few_mx(FewLayer p, hipStream_t stream) {
  if (!p.packed_in) launch_few_logits(EL_BF16, p, stream);
  deal(p, 17.0 / 32, 2.0);
  const int64_t most = static_cast<int64_t>(p.T * p.k < p.n_local ? p.T * p.k : p.n_local) * (p.I / kUnit);
  const int blocks = most < kCus - p.shared_blocks ? static_cast<int>(most) : kCus - p.shared_blocks;
  const int grid = p.shared_blocks + blocks;
  // LDS of the routed workgroups (terms of x) and of the shared ones (x), whichever is larger
  const size_t room = kLdsBytes - sizeof(Pairs) - 256;
  const size_t part = static_cast<size_t>(kWaves) * p.T * kUnit * sizeof(float);
  const size_t xt = few_mx_x_bytes(p.T, p.D);
  p.red_bufs = 4 * part + xt <= room ? 2 : 1;
  const size_t routed = (p.red_bufs == 2 ? 4 : 1) * part;
  const size_t red_sh = static_cast<size_t>(2) * kWaves * p.T * 16 * sizeof(float);
  const size_t xs = p.shared_blocks ? static_cast<size_t>(p.T) * x_row_bytes<EL_BF16>(p.D) : 0;
  p.shared_red_bufs = 2 * red_sh + xs <= room ? 2 : 1;
  const size_t shared = p.shared_blocks ? p.shared_red_bufs * red_sh : 0;
  if (routed + xt <= room && shared + xs <= room) {
    launch_gate_up<true>(p, grid, routed + xt > shared + xs ? routed + xt : shared + xs, stream);
  } else {
    hipLaunchKernelGGL(few_terms_kernel, dim3(p.T), dim3(kThreads), 0, stream, p);
    launch_gate_up<false>(p, grid, routed > shared ? routed : shared, stream);
  }
  if (p.out_el == EL_F32) launch_down<EL_F32>(p, stream);
  else launch_down<EL_BF16>(p, stream);
  return hipGetLastError();
}

}  // namespace moe
