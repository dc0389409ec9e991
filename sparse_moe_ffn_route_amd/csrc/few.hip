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
// works through its blocks of weight runs with register buffers, the next blocks' loads requested
// before the ends of units, their reductions and barriers.  In the down kernel they are a ring; in
// gate/up, as compiled, a batch: the compiler requests a workgroup's first R steps in another order than
// the later ones, and so waits at the first of every R steps for all loads in flight.
//
// Measured, one token of D 4096 and I 1024, 10 of 512 bf16 experts and a shared one (281 MB, 41 us at
// the chip's 6.8 TB/s streaming read): 59 us; logits 7, gate/up 34, down 17.5.  Inside gate/up
// the weights stream at 6.5 TB/s from 6 us after the start on: launch and x 1.5, the logits'
// latency and the selection 4.5.  13 tokens at 16 or so of 64 local e4m3 experts (182 MB, 27 us): 38 to
// 45 us, by where the allocator puts the matrices.  Row-major weights: 68 us for that token, and 91 against 81
// for 4 tokens of 8 of 128 e4m3 experts.
//
// x of more tokens than the LDS holds beside the reductions is read from memory at each product, behind every
// weight load in flight: 8 fp32 tokens of 4 of 64 experts (1.30 GB) 231 us, 9 of them (1.42 GB) 314; bf16 at D 7168,
// 9 tokens (1.24 GB) 229, 10 (1.34 GB) 273.
#include "few.hpp"
#include "mx.hpp"

namespace moe {

namespace {

using namespace few;

// ---------------------------------------------------------------------------
// logits
// ---------------------------------------------------------------------------

template <int EL, bool NORM>
__global__ __launch_bounds__(kLogitWaves * kWave) void few_logits_kernel(FewLayer p) {
  logits_block<EL, NORM>(p, blockIdx.x);
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
