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
// The tokens that chose an expert are columns of one 16-column MFMA tile, so each weight byte is
// read once whichever tokens chose it; the grouping is a few hundred pairs that every
// workgroup sorts out for itself.  Weights
// are turned into bf16 in registers (exact for e4m3 codes) and x is
// never quantised; h, scaled by the routing weight, is carried as a pair of bf16 (value and
// remainder, 16 significant bits), which keeps the rounding of h out of y: the remainders are
// columns 8 to 15 of the same MFMA.  4-bit weights have kernels of their
// own (few_mx.hip).
//
// The weights' bytes bound all of it, so both large kernels are built as streams: each wave
// works through its blocks of weight runs with a ring of register buffers, the next blocks'
// loads in flight over the ends of units, their reductions and barriers.
//
// Measured, one token of D 4096 and I 1024, 10 of 512 bf16 experts and a shared one (281 MB, 41 us at
// the chip's 6.8 TB/s streaming read): 59 us; logits 7, gate/up 34, down 17.5.  Inside gate/up
// the weights stream at 6.5 TB/s from 6 us after the start on: launch and x 1.5, the logits'
// latency and the selection 4.5.  13 tokens at 16 or so of 64 local e4m3 experts (182 MB, 27 us): 39 to
// 45 us, by where the allocator puts the matrices.
#include "few.hpp"
#include "mx.hpp"

namespace moe {

namespace {

using namespace few;

// ---------------------------------------------------------------------------
// logits
// ---------------------------------------------------------------------------

// 16 waves split the width: at D = 4096 each has all its loads (8 steps of 16 experts) in flight at
// once, so the launch is a few memory latencies long.  (The shared expert's gate/up beside the logits, on CUs
// that are idle here, made this launch 1.5 us longer and the next hardly shorter.)
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
// written by the first workgroup for the launches after this one.
template <int EL, bool NORM>
__global__ __launch_bounds__(kLogitWaves * kWave) void few_logits_kernel(FewLayer p) {
  __shared__ f32x4 red[kLogitWaves][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int e0 = blockIdx.x * 16;
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
        if (blockIdx.x == 0 && lrow < p.T)
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

// Workgroups [0, shared_blocks) take the shared expert's units and need no routing; the others
// the routed ones.
template <int W, bool PACKED, bool XLDS>
__global__ __launch_bounds__(kThreads, 2) void few_gate_up_kernel(FewLayer p) {
  constexpr int SH = W == EL_F32 ? EL_F32 : EL_BF16;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ Route q;
  float* red = reinterpret_cast<float*>(lds);
  uint8_t* xs = lds + p.red_bytes;
  if (static_cast<int>(blockIdx.x) < p.shared_blocks) {
    if constexpr (XLDS) {
      stage_x<SH>(p, xs);
      wait_vmcnt<0>();
      __syncthreads();
    }
    const int units = p.I_shared / 16, b = blockIdx.x;
    gate_up_units<SH, PACKED, XLDS, true>(p, q, xs, red, units * b / p.shared_blocks, units * (b + 1) / p.shared_blocks);
    return;
  }
  const int b = blockIdx.x - p.shared_blocks, blocks = gridDim.x - p.shared_blocks;
  route_call<16, kDownMembers>(q, lds, p, b == blocks - 1, [&] {
    if constexpr (XLDS) stage_x<W>(p, xs);
  });
  const int units = __builtin_amdgcn_readfirstlane(q.entries) * (p.I / 16);
  gate_up_units<W, PACKED, XLDS, false>(p, q, xs, red, static_cast<int>(static_cast<int64_t>(units) * b / blocks),
                                        static_cast<int>(static_cast<int64_t>(units) * (b + 1) / blocks));
}

// The last shared_waves waves take the shared expert, the others the routed ones.
template <int W, bool PACKED, int OUT>
__global__ __launch_bounds__(kThreads, 2) void few_down_kernel(FewLayer p) {
  constexpr int SH = W == EL_F32 ? EL_F32 : EL_BF16;
  __shared__ f32x4 red[kWaves][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int frag = blockIdx.x, routed = kWaves - p.shared_waves;
  const f32x4 acc = wave < routed
                        ? down_blocks<W, PACKED, false>(p, ld_scalar(p.entries), frag, wave, routed)
                        : down_blocks<SH, PACKED, true>(p, (p.T + kDownMembers - 1) / kDownMembers, frag, wave - routed,
                                                        p.shared_waves);
  finish_down<OUT>(p, frag, acc, red);
}

template <int W, bool PACKED, bool XLDS>
void launch_gate_up(const FewLayer& p, int grid, size_t lds, hipStream_t stream) {
  hipLaunchKernelGGL((few_gate_up_kernel<W, PACKED, XLDS>), dim3(grid), dim3(kThreads), lds, stream, p);
}

template <int W, bool PACKED>
hipError_t launch_w(FewLayer p, hipStream_t stream) {
  constexpr int act = W == EL_F32 ? EL_F32 : EL_BF16;
  if (W == EL_F32 && p.out_el != EL_F32) return hipErrorInvalidValue;
  if (!p.packed_in) launch_few_logits(act, p, stream);
  deal(p, W == EL_E4M3 ? 1.0 : W == EL_BF16 ? 2.0 : 4.0, act_bytes<W>());
  const int64_t most = static_cast<int64_t>(p.T * p.k < p.n_local ? p.T * p.k : p.n_local) * (p.I / 16);
  const int blocks = most < kCus - p.shared_blocks ? static_cast<int>(most) : kCus - p.shared_blocks;
  // x stays in LDS where it fits beside the reduction buffers (two, or one) and the routing
  const size_t red = static_cast<size_t>(2) * kWaves * p.T * 16 * sizeof(float);
  const size_t x = static_cast<size_t>(p.T) * (x_row_bytes<W>(p.D) > x_row_bytes<act>(p.D) ? x_row_bytes<W>(p.D)
                                                                                          : x_row_bytes<act>(p.D));
  const size_t room = kLdsBytes - sizeof(Route) - 256;
  p.red_bufs = std::max(2 * red, kRouteScratch) + x <= room ? 2 : 1;
  p.red_bytes = static_cast<int>(std::max(p.red_bufs * red, kRouteScratch));
  const int grid = p.shared_blocks + blocks;
  if (p.red_bytes + x <= room) launch_gate_up<W, PACKED, true>(p, grid, p.red_bytes + x, stream);
  else launch_gate_up<W, PACKED, false>(p, grid, p.red_bytes, stream);
  if (p.out_el == EL_F32)
    hipLaunchKernelGGL((few_down_kernel<W, PACKED, EL_F32>), dim3(p.D / 16), dim3(kThreads), 0, stream, p);
  else if constexpr (W != EL_F32)
    hipLaunchKernelGGL((few_down_kernel<W, PACKED, EL_BF16>), dim3(p.D / 16), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

void launch_few_logits(int act_el, const FewLayer& p, hipStream_t stream) {
  const dim3 grid((p.E + 15) / 16), block(kLogitWaves * kWave);
#define MOE_LOGITS(EL_, NORM_) hipLaunchKernelGGL((few_logits_kernel<EL_, NORM_>), grid, block, 0, stream, p)
  if (act_el == EL_F32) {
    if (p.norm_r) MOE_LOGITS(EL_F32, true);
    else MOE_LOGITS(EL_F32, false);
  } else {
    if (p.norm_r) MOE_LOGITS(EL_BF16, true);
    else MOE_LOGITS(EL_BF16, false);
  }
#undef MOE_LOGITS
}

hipError_t launch_few_layer(int w_el, bool packed, const FewLayer& p, hipStream_t stream) {
  switch (w_el) {
    case EL_F32: return packed ? launch_w<EL_F32, true>(p, stream) : launch_w<EL_F32, false>(p, stream);
    case EL_BF16: return packed ? launch_w<EL_BF16, true>(p, stream) : launch_w<EL_BF16, false>(p, stream);
    case EL_E4M3: return packed ? launch_w<EL_E4M3, true>(p, stream) : launch_w<EL_E4M3, false>(p, stream);
    case EL_MXFP4: return launch_few_mx(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace moe
