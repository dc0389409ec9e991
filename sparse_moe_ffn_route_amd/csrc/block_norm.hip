// Leaving one block and entering the next, one pass over the residual stream:
//   z  = rms(y) * w_post   (or y)          rms(v) = v / sqrt(mean(v^2) + eps)
//   r' = res_scale * r + gate * z
//   x  = rms(r') * w_next
// Statistics and every product are fp32; r' and x are each rounded once, x from the
// unrounded r'.
//
// One workgroup per row: the row's y, r and gate are read once into registers (kept there
// through both reductions), so the traffic is the floor: 2 to 3 reads and 1 to 2 writes per
// value.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// V consecutive values as float (V = 8: 16-byte accesses; V = 1: any alignment).
template <int EL, int V>
__device__ __forceinline__ void load_v(const void* base, int64_t idx, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = EL == EL_F32 ? static_cast<const float*>(base)[idx]
                        : bf16_bits_to_f32(static_cast<const uint16_t*>(base)[idx]);
  } else if constexpr (EL == EL_F32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + idx);
    const u32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + idx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_bits_to_f32(a[i] & 0xFFFFu);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

template <int EL, int V>
__device__ __forceinline__ void store_v(void* base, int64_t idx, const float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (EL == EL_F32) static_cast<float*>(base)[idx] = v[0];
    else static_cast<uint16_t*>(base)[idx] = static_cast<uint16_t>(bf16x2_bits(v[0], 0.0f));
  } else if constexpr (EL == EL_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + idx);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + idx) =
        make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
  }
}

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int i = 1; i < kThreads / kWave; ++i) s += red[i];
  return s;
}

// NC: chunks of V values per thread (D <= NC * V * kThreads).
template <int EL, int YEL, int V, int NC>
__global__ __launch_bounds__(kThreads) void block_norm_kernel(BlockNorm p) {
  __shared__ float red[2][kThreads / kWave];
  const int64_t row = blockIdx.x;
  const int64_t base = row * p.D;
  float r[NC][V];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int d = (c * kThreads + threadIdx.x) * V;
    if (d < p.D) load_v<EL, V>(p.r, base + d, r[c]);
  }
  if (p.y) {
    float y[NC][V];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = (c * kThreads + threadIdx.x) * V;
      if (d < p.D) {
        load_v<YEL, V>(p.y, base + d, y[c]);
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(y[c][i], y[c][i], ss);
      }
    }
    float rs = 1.0f;
    if (p.w_post) rs = 1.0f / sqrtf(block_sum(ss, red[0]) / p.D + p.eps);
    const float gt = p.gate_kind == kGateToken ? static_cast<const float*>(p.gate)[row] : 1.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = (c * kThreads + threadIdx.x) * V;
      if (d >= p.D) continue;
      if (p.w_post) {
        float w[V];
        load_v<EL, V>(p.w_post, d, w);
#pragma unroll
        for (int i = 0; i < V; ++i) y[c][i] = y[c][i] * rs * w[i];
      }
      if (p.gate_kind >= kGateChannel) {
        float g[V];
        load_v<EL, V>(p.gate, p.gate_kind == kGateChannel ? d : base + d, g);
#pragma unroll
        for (int i = 0; i < V; ++i) y[c][i] *= g[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) y[c][i] *= gt;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) r[c][i] = fmaf(p.res_scale, r[c][i], y[c][i]);
      store_v<EL, V>(p.r_out, base + d, r[c]);
    }
  }
  if (p.w_next) {
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = (c * kThreads + threadIdx.x) * V;
      if (d < p.D)
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(r[c][i], r[c][i], ss);
    }
    const float rs = 1.0f / sqrtf(block_sum(ss, red[1]) / p.D + p.eps);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = (c * kThreads + threadIdx.x) * V;
      if (d >= p.D) continue;
      float w[V], o[V];
      load_v<EL, V>(p.w_next, d, w);
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = r[c][i] * rs * w[i];
      store_v<EL, V>(p.x_next, base + d, o);
    }
  }
}

template <int EL, int YEL, int V>
hipError_t launch_v(const BlockNorm& p, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(p.T)), block(kThreads);
  const int nc = (p.D + kThreads * V - 1) / (kThreads * V);
#define MOE_NORM(N_) hipLaunchKernelGGL((block_norm_kernel<EL, YEL, V, N_>), grid, block, 0, stream, p)
  if (nc <= 1) MOE_NORM(1);
  else if (nc <= 2) MOE_NORM(2);
  else if (nc <= 4) MOE_NORM(4);
  else if (nc <= 8) MOE_NORM(8);
  else if constexpr (V == 1) {
    if (nc <= 16) MOE_NORM(16);
    else if (nc <= 32) MOE_NORM(32);
    else MOE_NORM(64);
  }
#undef MOE_NORM
  return hipGetLastError();
}

template <int EL, int YEL>
hipError_t launch_el(const BlockNorm& p, bool wide, hipStream_t stream) {
  return wide ? launch_v<EL, YEL, 8>(p, stream) : launch_v<EL, YEL, 1>(p, stream);
}

bool aligned16(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; }

}  // namespace

hipError_t launch_block_norm(int el, int y_el, const BlockNorm& p, hipStream_t stream) {
  // rows of a multiple of 8 values at 16-byte addresses take 16-byte accesses, any other single values
  const bool wide = p.D % 8 == 0 && aligned16(p.y) && aligned16(p.r) && aligned16(p.w_post) &&
                    (p.gate_kind < kGateChannel || aligned16(p.gate)) && aligned16(p.r_out) && aligned16(p.w_next) &&
                    aligned16(p.x_next);
  if (el == EL_F32) return launch_el<EL_F32, EL_F32>(p, wide, stream);
  return y_el == EL_F32 ? launch_el<EL_BF16, EL_F32>(p, wide, stream) : launch_el<EL_BF16, EL_BF16>(p, wide, stream);
}

}  // namespace moe
