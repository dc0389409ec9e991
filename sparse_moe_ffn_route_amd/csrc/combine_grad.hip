// Gradient of the weighted unpermute-combine y[t] = sum_j w[t][j] * rows[inv_pos[t][j]]:
//   d_rows[inv_pos[t][j]] = w[t][j] * dy[t]        d_w[t][j] = <dy[t], rows[inv_pos[t][j]]>
// slots with inv_pos < 0: no row, d_w = 0.
//
// A wave per slot: it reads its row once and writes the gradient's once, which is all the traffic there has to be but
// for dy[t], which the token's waves, next to each other on one XCD, read from its L2.  The dot product is fp32: each
// lane's own columns in order, then the lanes pairwise.
//
// Bound by memory: 8192 tokens of 10 slots, D = 4096, bf16, move 1.41 GB, rows and gradients once each and past the
// caches' replacement, in 268 us (5.3 TB/s; a copy reaches 5.1).  Four waves a workgroup 268 us, two 272, eight 281;
// a workgroup per token, dy read once into registers, 313 to 350: too little of it under way.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kGridX = 1 << 20;  // a grid dimension holds less than 2^32 threads
constexpr int kAhead = 4;  // pieces of 512 columns under way

// ONCE: past the caches' replacement.
template <int EL, bool ONCE>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&v)[8]) {
  if constexpr (EL == EL_F32) {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + at);
    const f32x4 a = ONCE ? __builtin_nontemporal_load(p) : p[0], b = ONCE ? __builtin_nontemporal_load(p + 1) : p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  } else {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + at);
    const u32x4 w = ONCE ? __builtin_nontemporal_load(p) : p[0];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

template <int EL>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&v)[8]) {
  if constexpr (EL == EL_F32) {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(base) + at);
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, p);
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, p + 1);
  } else {
    const u32x4 w{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7])};
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + at));
  }
}

template <int YEL, int REL>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(CombineGrad p) {
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t total = static_cast<int64_t>(p.T) * p.k;
  const int64_t block = static_cast<int64_t>(blockIdx.y) * gridDim.x + xcd_remap(blockIdx.x, gridDim.x);
  const int64_t q = block * (kThreads / kWave) + wave;
  if (q >= total) return;
  const int64_t t = q / p.k;
  const int row = ld_scalar(p.inv_pos + q);
  const float w = __int_as_float(ld_scalar(p.packed + t * 2 * p.k + p.k + (q - t * p.k)));
  float dot = 0.0f;
  if (row >= 0 && row < total) {
    for (int c0 = lane * 8; c0 < p.D; c0 += kAhead * 512) {
      float dy[kAhead][8], v[kAhead][8];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int c = c0 + x * 512;
        if (c >= p.D) continue;
        load8<YEL, false>(p.dy, t * p.D + c, dy[x]);
        if (p.rows) load8<YEL, true>(p.rows, static_cast<int64_t>(row) * p.D + c, v[x]);
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int c = c0 + x * 512;
        if (c >= p.D) continue;
        if (p.rows) {
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = fmaf(dy[x][i], v[x][i], dot);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) dy[x][i] *= w;
        store8<REL>(p.d_rows, static_cast<int64_t>(row) * p.D + c, dy[x]);
      }
    }
  }
  if (!p.rows) return;
  dot = wave_sum(dot);
  if (lane == 0) p.d_w[q] = dot;
}

}  // namespace

hipError_t launch_combine_grad(int y_el, int row_el, const CombineGrad& p, hipStream_t s) {
  const int64_t slots = static_cast<int64_t>(p.T) * p.k;
  const int64_t blocks = (slots + kThreads / kWave - 1) / (kThreads / kWave), x = std::min<int64_t>(blocks, kGridX);
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>((blocks + x - 1) / x));
  auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, p); };
  if (y_el == EL_BF16) launch(combine_grad_kernel<EL_BF16, EL_BF16>);
  else if (row_el == EL_BF16) launch(combine_grad_kernel<EL_F32, EL_BF16>);
  else launch(combine_grad_kernel<EL_F32, EL_F32>);
  return hipGetLastError();
}

}  // namespace moe
