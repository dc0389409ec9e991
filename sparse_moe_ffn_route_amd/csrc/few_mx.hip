// The few-token layer (few.hip) on microscaled 4-bit weights.
//
// The codes and block scales go into the scaled MFMA as they are; the other operand is the
// activation as a sum of e4m3 terms with a power of two per 32 values,
//   v = t0 2^e + t1 2^(e-5) + t2 2^(e-10) + t3 2^(e-15),  e = floor(log2(max |v|)) - 7,
// each term the rounding of what the terms before it left.  A term carries four significant
// bits and leaves a remainder of at most 2^-4 of itself, so two terms hold a bf16 x exactly
// (to 2^-22 of the block's largest value) and four hold h to 2^-17.  Columns that
// tokens do not need carry the further terms: one product per step does for x of up to 8
// tokens that chose the expert, and for h of up to 4 (more make a second entry of the expert).  Decoding the weights to bf16 instead takes sixteen conversions and four
// MFMAs per KB and bound both kernels by instruction issue (4.0 TB/s at 4 tokens).
//
// Measured, 4 tokens, 8 of 128 experts of D 4096 and I 1024 and a shared bf16 one (221 MB, 33 us at the
// 6.8 TB/s streaming read): 55 to 57 us; traced, logits 7.6, gate/up 30.9 (145 MB; the experts are known 4 to 5 us
// after its start, 5.5 TB/s from there on), down 17.3 (74 MB; 5.2 TB/s after the first 3).  Gate/up works in batches
// as the other weights' does (few.hip), and waits a second time in each, where the byte-sized scales of the
// next one are widened.  Terms past the LDS are read from memory at each product: 8 of 128 experts at D 7168, 8
// tokens (606 MB) 132 us, 10 (714 MB) 161, 16 (966 MB) 208.
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

// BYTE: of both scale registers.
template <int BYTE = 0>
__device__ __forceinline__ f32x4 mx_mul(const u32x4& a, const u32x4& b0, const u32x4& b1, f32x4 c, u32 sa, u32 sb) {
  const u32x4 z = {0u, 0u, 0u, 0u};
  const i32x8 av = __builtin_bit_cast(i32x8, __builtin_shufflevector(a, z, 0, 1, 2, 3, 4, 5, 6, 7));
  const i32x8 bv = __builtin_bit_cast(i32x8, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7));
  // A: fp4 (format 4); B: e4m3 (format 0)
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 0, BYTE, static_cast<int>(sa), BYTE,
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
__host__ __device__ constexpr int xt_bytes(int T, int D) { return (2 * T * (xt_row(D) + xt_blocks(D)) + 15) & ~15; }

// By all THREADS of a workgroup: four lanes a block, eight values each, of four tokens at a time, whose
// loads are in flight together.  first / stride: tokens.
template <int THREADS>
__device__ __forceinline__ void make_terms(const FewLayer& p, uint8_t* xt, int first, int stride) {
  constexpr int N = 4;
  const int row = xt_row(p.D), blocks = xt_blocks(p.D);
  uint8_t* scales = xt + 2 * p.T * row;
  for (int t0 = first; t0 < p.T; t0 += N * stride)
    for (int c = threadIdx.x; c < blocks * 4; c += THREADS) {
      u32x4 x[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int t = min(t0 + n * stride, p.T - 1), k = min(c * 8, p.D - 8);
        x[n] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) + static_cast<int64_t>(t) * p.D + k);
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int t = t0 + n * stride;
        if (t >= p.T) break;
        float v[8];
        u32 m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u32 w = c * 8 < p.D ? x[n][i] : 0u;  // zeros behind the last value
          v[2 * i] = bf16_bits_to_f32(w & 0xFFFFu);
          v[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
          m = max(m, max(mx_abs_bits(v[2 * i]), mx_abs_bits(v[2 * i + 1])));
        }
        m = max(m, static_cast<u32>(__shfl_xor(static_cast<int>(m), 1, kWave)));
        m = max(m, static_cast<u32>(__shfl_xor(static_cast<int>(m), 2, kWave)));
        const int b = term_scale(m);
        u32 t0s[2] = {0u, 0u}, t1s[2] = {0u, 0u};
        if (b != 255) {
          const float inv = ldexpf(1.0f, 127 - b);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a0 = v[2 * i] * inv, a1 = v[2 * i + 1] * inv;
            const u32 hi = f32x2_to_e4m3x2(a0, a1);
            const u32 lo = f32x2_to_e4m3x2((a0 - e4m3_lo(hi)) * 32.0f, (a1 - e4m3_hi(hi)) * 32.0f);
            t0s[i / 2] |= hi << (16 * (i & 1));
            t1s[i / 2] |= lo << (16 * (i & 1));
          }
        }
        *reinterpret_cast<uint2*>(xt + (2 * t) * row + c * 8) = make_uint2(t0s[0], t0s[1]);
        *reinterpret_cast<uint2*>(xt + (2 * t + 1) * row + c * 8) = make_uint2(t1s[0], t1s[1]);
        if ((c & 3) == 0) {
          scales[(2 * t) * blocks + c / 4] = static_cast<uint8_t>(b);
          scales[(2 * t + 1) * blocks + c / 4] = static_cast<uint8_t>(b == 255 ? 255 : b - kTermStep);
        }
      }
    }
}

// Logits, and beside them on CUs that are idle here the terms of each token, for gate/up to copy: made in
// each of its workgroups they took 2.7 us of 4 tokens and 4.4 of 8 before any weight was asked for.
__global__ __launch_bounds__(kLogitWaves * kWave) void few_mx_first_kernel(FewLayer p) {
  const int block = static_cast<int>(blockIdx.x) - p.T;
  if (block >= 0) logits_block<EL_BF16, false>(p, block);
  else make_terms<kLogitWaves * kWave>(p, static_cast<uint8_t*>(p.x_terms), blockIdx.x, p.T);
}

// Without that launch, tokens too wide for LDS.
__global__ __launch_bounds__(kThreads) void few_terms_kernel(FewLayer p) {
  make_terms<kThreads>(p, static_cast<uint8_t*>(p.x_terms), blockIdx.x, gridDim.x);
}

// Made terms into LDS, complete after wait_vmcnt<0> and a barrier.
__device__ __forceinline__ void stage_terms(const FewLayer& p, uint8_t* xt) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const __amdgpu_buffer_rsrc_t r = buffer_rsrc(p.x_terms);
  const int bytes = xt_bytes(p.T, p.D);
  for (int c = wave * 1024; c < bytes; c += kWaves * 1024)
    if (c + lane * 16 < bytes) buffer_load16_to_lds(r, xt + c, lane * 16, c);
}

// ---------------------------------------------------------------------------
// gate/up
// ---------------------------------------------------------------------------

// Rows of h: [T * k][term] of whole steps' bytes, then a scale byte per row, term and block, 16 per group
// of 512 values: for each lane group the dword of its four steps.
__host__ __device__ constexpr int ht_row(int I) { return mx_steps(I) * kMxStep; }
__host__ __device__ constexpr int ht_blocks(int I) { return mx_groups(I) * 16; }
__host__ __device__ constexpr int ht_scale(int blk) { return (blk & ~15) + (blk & 3) * 4 + ((blk >> 2) & 3); }

constexpr int kGateMembers = 8;  // per entry: columns 8 to 15 are the second terms
constexpr int kHMembers = 4;     // per entry of the down kernel: four terms

// Units [u0, u1) of 32 channels of the routed experts, as gate_up_units (few.hpp).
template <bool XLDS>
__device__ __forceinline__ void mx_gate_up_units(const FewLayer& p, const Route& q, const uint8_t* xt, float* red,
                                                 int u0, int u1) {
  constexpr int R = 4;
  if (u0 >= u1) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int S = mx_steps(p.D), per = p.I / kUnit;
  const int s0 = S * wave / kWaves, s1 = S * (wave + 1) / kWaves;
  const int turns = ((S + kWaves - 1) / kWaves + R - 1) / R;
  const u32 frag_bytes = static_cast<u32>(mx_fragment_bytes(p.D));
  const int row_bytes = xt_row(p.D), blocks = xt_blocks(p.D);
  const int hrow = ht_row(p.I), hblocks = ht_blocks(p.I);
  struct Source {
    __amdgpu_buffer_rsrc_t r0, r1;
    u32 at;
    bool on;
  };
  auto source = [&](int u) {
    Source o;
    o.on = u < u1;
    int64_t eo = 0;
    if (o.on) eo = __builtin_amdgcn_readfirstlane(entry_expert(q.entry[u / per])) * p.gu_stride;
    o.r0 = weight_rsrc(static_cast<const uint8_t*>(p.w_gate) + eo);
    o.r1 = weight_rsrc(static_cast<const uint8_t*>(p.w_up) + eo);
    o.at = static_cast<u32>(__builtin_amdgcn_readfirstlane(u % per)) * 2 * frag_bytes;
    return o;
  };
  u32x4 w[R][2][2];  // step, matrix, fragment
  u32 sc[R][2][2];
  auto load = [&](int n, const Source& o, int s) {
    const bool real = o.on && s < s1;
    const u32 v = real ? lane * 16 : kOutOfRange, vs = real ? lane * 4 : kOutOfRange;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const u32 at = run_offset(o.at + f * frag_bytes, s), so = byte_offset(o.at + f * frag_bytes, s, S);
      w[n][0][f] = buffer_load16<true>(o.r0, v, at);
      w[n][1][f] = buffer_load16<true>(o.r1, v, at);
      sc[n][0][f] = __builtin_amdgcn_raw_buffer_load_b8(o.r0, vs, so, 0);
      sc[n][1][f] = __builtin_amdgcn_raw_buffer_load_b8(o.r1, vs, so, 0);
    }
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  const int cols = min(p.T, kGateMembers), part = kWaves * cols * kUnit;
  Source cur = source(u0);
#pragma unroll
  for (int n = 0; n < R; ++n) load(n, cur, s0 + n);
  float* buf = red;
  for (int u = u0; u < u1; ++u) {
    const int2 en = q.entry[u / per];
    const int members = entry_members(en, kGateMembers), row = entry_row(en);
    const int t = q.token[row + min(lrow & (kGateMembers - 1), members - 1)], term = lrow / kGateMembers;
    const uint8_t* xr = xt + (2 * t + term) * row_bytes + lgrp * 16;
    const uint8_t* xsc = xt + 2 * p.T * row_bytes + (2 * t + term) * blocks + lgrp;
    f32x4 c[2][2] = {{zero, zero}, {zero, zero}};
    for (int k = 0; k < turns; ++k) {
      const bool last = k + 1 == turns;
      if (last) cur = source(u + 1);
      const int sl = last ? s0 : s0 + (k + 1) * R;
#pragma unroll
      for (int n = 0; n < R; ++n) {
        const int s = s0 + k * R + n;
        if (s < s1) {
          const u32x4 b0 = *reinterpret_cast<const u32x4*>(xr + s * kMxStep);
          const u32x4 b1 = *reinterpret_cast<const u32x4*>(xr + s * kMxStep + 64);
          const u32 sb = xsc[s * 4];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int f = 0; f < 2; ++f) c[m][f] = mx_mul(w[n][m][f], b0, b1, c[m][f], sc[n][m][f], sb);
        }
        __builtin_amdgcn_sched_barrier(0);
        load(n, cur, sl + n);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[m][f][i] = dpp_add<kRor8>(c[m][f][i]);
        if (lrow < members)
          *reinterpret_cast<f32x4*>(buf + m * part + (wave * cols + lrow) * kUnit + f * 16 + lgrp * 4) = c[m][f];
      }
    lds_barrier();
    const int cc = threadIdx.x / kUnit, ch = threadIdx.x % kUnit;
    if (cc < members) {
      float g = 0.f, v = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        g += buf[(i * cols + cc) * kUnit + ch];
        v += buf[part + (i * cols + cc) * kUnit + ch];
      }
      const float h = q.weight[row + cc] * (silu(g) * v);
      u32 m = mx_abs_bits(h);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max(m, static_cast<u32>(__shfl_xor(static_cast<int>(m), o, kWave)));
      const int b = term_scale(m);
      uint8_t* out = static_cast<uint8_t*>(p.h);
      uint8_t* out_sc = out + static_cast<int64_t>(p.T) * p.k * kTerms * hrow;
      float rest = b == 255 ? 0.0f : h * ldexpf(1.0f, 127 - b);
#pragma unroll
      for (int i = 0; i < kTerms; ++i) {
        const int64_t r = static_cast<int64_t>(row + cc) * kTerms + i;
        const u32 code = f32x2_to_e4m3x2(rest, 0.0f);
        out[r * hrow + (u % per) * kUnit + ch] = static_cast<uint8_t>(code);
        rest = (rest - e4m3_lo(code)) * 32.0f;
        if (ch == 0) out_sc[r * hblocks + ht_scale(u % per)] = static_cast<uint8_t>(b == 255 ? 255 : b - i * kTermStep);
        // the two blocks that fill the last step have no codes, and a scale that is no NaN
        else if (ch <= 2 && u % per == per - 1 && (p.I & 64)) out_sc[r * hblocks + ht_scale(per - 1 + ch)] = 127;
      }
    }
    if (p.red_bufs == 2) buf = buf == red ? red + 2 * part : red;
    else lds_barrier();
  }
}

template <bool XLDS>
__global__ __launch_bounds__(kThreads, 2) void few_mx_gate_up_kernel(FewLayer p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ Route q;
  float* red = reinterpret_cast<float*>(lds);
  uint8_t* xs = lds + p.red_bytes;
  if (static_cast<int>(blockIdx.x) < p.shared_blocks) {
    // the shared expert is bf16: it takes x as it is
    if constexpr (XLDS) {
      stage_x<EL_BF16>(p, xs);
      wait_vmcnt<0>();
      __syncthreads();
    }
    const int units = p.I_shared / 16, b = blockIdx.x;
    p.red_bufs = p.shared_red_bufs;
    gate_up_units<EL_BF16, true, XLDS, true>(p, q, xs, red, units * b / p.shared_blocks, units * (b + 1) / p.shared_blocks);
    return;
  }
  const int b = blockIdx.x - p.shared_blocks, blocks = gridDim.x - p.shared_blocks;
  route_call<kGateMembers, kHMembers>(q, lds, p, b == blocks - 1, [&] {
    if constexpr (XLDS) {
      if (p.terms_made) stage_terms(p, xs);
      else make_terms<kThreads>(p, xs, 0, 1);
    }
  });
  const int units = __builtin_amdgcn_readfirstlane(q.entries) * (p.I / kUnit);
  mx_gate_up_units<XLDS>(p, q, XLDS ? xs : static_cast<uint8_t*>(p.x_terms), red,
                         static_cast<int>(static_cast<int64_t>(units) * b / blocks),
                         static_cast<int>(static_cast<int64_t>(units) * (b + 1) / blocks));
}

// ---------------------------------------------------------------------------
// down
// ---------------------------------------------------------------------------

// As down_blocks (few.hpp), a block being a group of four steps: entries of up to four members, whose four terms are the columns 4 i + member.
__device__ __forceinline__ f32x4 mx_down_blocks(const FewLayer& p, int entries, int frag, int first, int stride) {
  constexpr int B = kMxGroup / kMxStep, NBUF = 3;
  const int lane = threadIdx.x % kWave, lrow = lane & 15, lgrp = lane >> 4;
  const int S = mx_steps(p.I), nb = (S + B - 1) / B;
  const int blocks = entries * nb;
  const u32 frag_at = static_cast<u32>(frag) * static_cast<u32>(mx_fragment_bytes(p.I));
  const int hrow = ht_row(p.I), hblocks = ht_blocks(p.I);
  const u32 codes = static_cast<u32>(p.T) * p.k * kTerms * hrow;  // bytes of the terms, then their scales
  const __amdgpu_buffer_rsrc_t rh = buffer_rsrc_sized(p.h, codes + static_cast<u32>(p.T) * p.k * kTerms * hblocks);
  const int c = lrow & (kHMembers - 1), term = lrow / kHMembers;
  if (blocks == 0) return f32x4{0.f, 0.f, 0.f, 0.f};
  auto entry = [&](const Cursor& at) { return make_int2(ld_scalar(&p.entry[at.hi].x), ld_scalar(&p.entry[at.hi].y)); };
  struct Block {
    u32x4 w[B], h[B][2];
    u32 sc, hs;  // byte n: step n
  };
  auto load = [&](Block& b, Cursor& at) {
    const bool there = at.left > 0;
    const int2 en = entry(at);
    const int j = at.lo;
    at.next();
    const __amdgpu_buffer_rsrc_t r =
        weight_rsrc(static_cast<const uint8_t*>(p.w_down) + static_cast<int64_t>(entry_expert(en)) * p.dn_stride);
    const bool on = there && c < entry_members(en, kHMembers);
    const u32 rt = static_cast<u32>(entry_row(en) + c) * kTerms + term;
    b.sc = __builtin_amdgcn_raw_buffer_load_b32(r, there ? lane * 4 : kOutOfRange,
                                                frag_at + j * kMxGroupBytes + min(B, S - B * j) * kMxRun, 0);
    b.hs = __builtin_amdgcn_raw_buffer_load_b32(rh, on ? codes + rt * hblocks + j * 16 + lgrp * 4 : kOutOfRange, 0, 0);
#pragma unroll
    for (int n = 0; n < B; ++n) {
      const int s = j * B + n, k0 = s * kMxStep;
      const bool real = there && s < S;
      b.w[n] = buffer_load16<true>(r, real ? lane * 16 : kOutOfRange, run_offset(frag_at, s));
      // lanes without a member, or past the width, read nothing: zeros
      const u32 at = rt * hrow + k0 + lgrp * 16;
      b.h[n][0] = buffer_load16<false>(rh, on && k0 < p.I ? at : kOutOfRange, 0);
      b.h[n][1] = buffer_load16<false>(rh, on && k0 + 64 < p.I ? at + 64 : kOutOfRange, 0);
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Block& b, Cursor& at) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    const int2 en = entry(at);
    const int j = at.lo;
    at.next();
    v = mx_mul<0>(b.w[0], b.h[0][0], b.h[0][1], v, b.sc, b.hs);
    if (j * B + 1 < S) v = mx_mul<1>(b.w[1], b.h[1][0], b.h[1][1], v, b.sc, b.hs);
    if (j * B + 2 < S) v = mx_mul<2>(b.w[2], b.h[2][0], b.h[2][1], v, b.sc, b.hs);
    if (j * B + 3 < S) v = mx_mul<3>(b.w[3], b.h[3][0], b.h[3][1], v, b.sc, b.hs);
#pragma unroll
    for (int n = 0; n < 4; ++n) v[n] = dpp_add<kRor4>(dpp_add<kRor8>(v[n]));
    acc += to_tokens(v, en, kHMembers);
  };
  Cursor ahead(first, stride, blocks, nb), here = ahead;
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

template <int OUT>
__global__ __launch_bounds__(kThreads, 2) void few_mx_down_kernel(FewLayer p) {
  __shared__ f32x4 red[kWaves][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int frag = blockIdx.x, routed = kWaves - p.shared_waves;
  const f32x4 acc = wave < routed ? mx_down_blocks(p, ld_scalar(p.entries), frag, wave, routed)
                                  : down_blocks<EL_BF16, true, true>(p, (p.T + kDownMembers - 1) / kDownMembers, frag,
                                                                     wave - routed, p.shared_waves);
  finish_down<OUT>(p, frag, acc, red);
}

}  // namespace

size_t few_mx_x_bytes(int T, int D) { return static_cast<size_t>(xt_bytes(T, D)); }
size_t few_mx_h_bytes(int T, int k, int I) {
  return static_cast<size_t>(T) * k * kTerms * (ht_row(I) + ht_blocks(I));  // a multiple of 16 bytes
}

hipError_t launch_few_mx(FewLayer p, hipStream_t stream) {
  p.terms_made = !p.packed_in && !p.norm_r;
  if (p.terms_made)
    hipLaunchKernelGGL(few_mx_first_kernel, dim3(p.T + (p.E + 15) / 16), dim3(kLogitWaves * kWave), 0, stream, p);
  else if (!p.packed_in)
    launch_few_logits(EL_BF16, p, stream);
  deal(p, 17.0 / 32, 2.0);
  const int64_t most = static_cast<int64_t>(p.T * p.k < p.n_local ? p.T * p.k : p.n_local) * (p.I / kUnit);
  const int blocks = most < kCus - p.shared_blocks ? static_cast<int>(most) : kCus - p.shared_blocks;
  const int grid = p.shared_blocks + blocks;
  // LDS of the routed workgroups (reductions, terms of x) and of the shared ones (reductions, x)
  const size_t room = kLdsBytes - sizeof(Route) - 256;
  const size_t red = static_cast<size_t>(2) * kWaves * std::min(p.T, kGateMembers) * kUnit * sizeof(float);
  const size_t red_sh = p.shared_blocks ? static_cast<size_t>(2) * kWaves * p.T * 16 * sizeof(float) : 0;
  const size_t xs = p.shared_blocks ? static_cast<size_t>(p.T) * x_row_bytes<EL_BF16>(p.D) : 0;
  const size_t x = std::max(few_mx_x_bytes(p.T, p.D), xs);
  p.red_bufs = 2 * red + x <= room ? 2 : 1;
  p.shared_red_bufs = 2 * red_sh + x <= room ? 2 : 1;
  p.red_bytes = static_cast<int>(std::max({p.red_bufs * red, p.shared_red_bufs * red_sh, kRouteScratch}));
  if (p.red_bytes + x <= room) {
    hipLaunchKernelGGL((few_mx_gate_up_kernel<true>), dim3(grid), dim3(kThreads), p.red_bytes + x, stream, p);
  } else {
    if (!p.terms_made) hipLaunchKernelGGL(few_terms_kernel, dim3(p.T), dim3(kThreads), 0, stream, p);
    hipLaunchKernelGGL((few_mx_gate_up_kernel<false>), dim3(grid), dim3(kThreads), p.red_bytes, stream, p);
  }
  if (p.out_el == EL_F32) hipLaunchKernelGGL((few_mx_down_kernel<EL_F32>), dim3(p.D / 16), dim3(kThreads), 0, stream, p);
  else hipLaunchKernelGGL((few_mx_down_kernel<EL_BF16>), dim3(p.D / 16), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace moe
