// Gradient of the weighted unpermute-combine y[t] = sum_j w[t][j] * rows[inv_pos[t][j]]:
//   d_rows[inv_pos[t][j]] = w[t][j] * dy[t]        d_w[t][j] = <dy[t], rows[inv_pos[t][j]]>
// slots with inv_pos < 0: no row, d_w = 0.
//
// One workgroup per token: dy[t] is read once for up to 8 slots (again, from the caches, for the next 8), every row
// of the token is read once and its gradient's row written once, which is all the traffic there has to be.  Sums are
// fp32: each thread's own columns, then the threads of a wave, then the waves, in an order of its own.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256, kBatch = 8;

template <int EL>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&v)[8]) {
  if constexpr (EL == EL_F32) {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + at);
    const f32x4 a = __builtin_nontemporal_load(p), b = __builtin_nontemporal_load(p + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  } else {
    const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + at));
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
    p[0] = f32x4{v[0], v[1], v[2], v[3]};
    p[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + at) =
        u32x4{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7])};
  }
}

template <int YEL, int REL>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(CombineGrad p) {
  __shared__ float part[kThreads / kWave][kBatch];
  const int wave = threadIdx.x / kWave;
  const int64_t t = blockIdx.x;
  const int32_t* inv = p.inv_pos + t * p.k;
  const int32_t* wbits = p.packed + t * 2 * p.k + p.k;
  const int64_t total = static_cast<int64_t>(p.T) * p.k;
  for (int j0 = 0; j0 < p.k; j0 += kBatch) {
    int64_t row[kBatch];
    float w[kBatch], dot[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = min(j0 + u, p.k - 1);
      const int r = inv[j];
      row[u] = j0 + u < p.k && r >= 0 && r < total ? r : -1;
      w[u] = __int_as_float(wbits[j]);
      dot[u] = 0.0f;
    }
    for (int c = threadIdx.x * 8; c < p.D; c += kThreads * 8) {
      float dy[8];
      load8<YEL>(p.dy, t * p.D + c, dy);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (row[u] < 0) continue;  // the same for the whole workgroup
        if (p.rows) {
          float v[8];
          load8<YEL>(p.rows, row[u] * p.D + c, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[u] = fmaf(dy[i], v[i], dot[u]);
        }
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = w[u] * dy[i];
        store8<REL>(p.d_rows, row[u] * p.D + c, d);
      }
    }
    if (!p.rows) continue;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float v = wave_sum(dot[u]);
      if (lane_id() == 0) part[wave][u] = v;
    }
    __syncthreads();
    if (threadIdx.x < kBatch && j0 + static_cast<int>(threadIdx.x) < p.k) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kThreads / kWave; ++i) v += part[i][threadIdx.x];
      p.d_w[t * p.k + j0 + threadIdx.x] = v;
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_combine_grad(int y_el, int row_el, const CombineGrad& p, hipStream_t s) {
  auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(p.T), dim3(kThreads), 0, s, p); };
  if (y_el == EL_BF16) launch(combine_grad_kernel<EL_BF16, EL_BF16>);
  else if (row_el == EL_BF16) launch(combine_grad_kernel<EL_F32, EL_BF16>);
  else launch(combine_grad_kernel<EL_F32, EL_F32>);
  return hipGetLastError();
}

}  // namespace moe
