// Leaving one block and entering the next, one pass over the residual stream:
//   z  = rms(y) * w_post   (or y)          rms(v) = v / sqrt(mean(v^2) + eps)
//   r' = res_scale * r + gate * z
//   x  = rms(r') * w_next
// Statistics and every product are fp32; r' and x are each rounded once, x from the
// unrounded r'.
//
// One workgroup per row: the row's y, r and gate are read once into registers (kept there
// through both reductions), so the traffic is the floor: 2 to 3 reads and 1 to 2 writes per
// value.  Measured, bf16 rows of 4096 with a gate for every value: 8192 rows (336 MB) in 58 us, 5.8 TB/s (a device
// copy reaches 4.9; 60 us with loads through the caches' ordinary replacement; alternating between two such
// inputs 52 against 60, and 57 with the stores past it, too); one row in 3 us, a few memory latencies.
// Rows of a width that is no multiple of 8, or off a 16-byte boundary, one value per access: 8192 rows of 4095 134 us.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// V consecutive values as stored (V = 8: 16-byte accesses; V = 1: any alignment).
template <int EL, int V>
struct Chunk {
  static constexpr int kWords = V == 1 ? 1 : EL == EL_F32 ? 8 : 4;
  uint32_t w[kWords];

  // NT: past the caches' replacement, for what is read once.
  template <bool NT = false>
  __device__ __forceinline__ void load(const void* base, int64_t idx) {
    if constexpr (V == 1) {
      w[0] = EL == EL_F32 ? static_cast<const uint32_t*>(base)[idx] : static_cast<const uint16_t*>(base)[idx];
    } else {
      const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(base) + idx * (EL == EL_F32 ? 4 : 2));
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const u32x4 a = NT ? __builtin_nontemporal_load(p + i) : p[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = a[j];
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (EL == EL_F32) return __uint_as_float(w[i]);
    else return i % 2 == 0 ? bf16_bits_to_f32(w[i / 2] & 0xFFFFu) : __uint_as_float(w[i / 2] & 0xFFFF0000u);
  }
};

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
constexpr int kGridX = 1 << 20;  // rows per grid row: a grid dimension holds less than 2^32 threads

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
  // Short rows: weights and gate are requested with the row, so that a call of few rows waits for
  // memory once rather than after each sum; longer rows keep the registers.
  constexpr bool kEarly = NC * V <= 16;
  const int64_t row = static_cast<int64_t>(blockIdx.y) * kGridX + blockIdx.x;
  if (row >= p.T) return;
  const int64_t base = row * p.D;
  const bool gated = p.gate_kind >= kGateChannel;
  Chunk<YEL, V> yc[NC];
  Chunk<EL, V> rc[NC], wp[kEarly ? NC : 1], g[kEarly ? NC : 1], wn[kEarly ? NC : 1];
  auto load_post = [&](int c, int d) {
    if (p.w_post) wp[kEarly ? c : 0].load(p.w_post, d);
    if (gated) g[kEarly ? c : 0].template load<true>(p.gate, p.gate_kind == kGateChannel ? d : base + d);
  };
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int d = (c * kThreads + threadIdx.x) * V;
    if (d >= p.D) continue;
    rc[c].template load<true>(p.r, base + d);
    if (p.y) {
      yc[c].template load<true>(p.y, base + d);
      if constexpr (kEarly) load_post(c, d);
    }
    if (kEarly && p.w_next) wn[kEarly ? c : 0].load(p.w_next, d);
  }
  float r[NC][V];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) r[c][i] = rc[c][i];
  if (p.y) {
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = (c * kThreads + threadIdx.x) * V;
      if (d < p.D)
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(yc[c][i], yc[c][i], ss);
    }
    float rs = 1.0f;
    if (p.w_post) rs = 1.0f / sqrtf(block_sum(ss, red[0]) / p.D + p.eps);
    const float gt = p.gate_kind == kGateToken ? static_cast<const float*>(p.gate)[row] : 1.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = (c * kThreads + threadIdx.x) * V, w = kEarly ? c : 0;
      if (d >= p.D) continue;
      if constexpr (!kEarly) load_post(c, d);
      float z[V];
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = p.w_post ? yc[c][i] * rs * wp[w][i] : yc[c][i];
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] *= gated ? g[w][i] : gt;
#pragma unroll
      for (int i = 0; i < V; ++i) r[c][i] = fmaf(p.res_scale, r[c][i], z[i]);
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
      const int d = (c * kThreads + threadIdx.x) * V, w = kEarly ? c : 0;
      if (d >= p.D) continue;
      if constexpr (!kEarly) wn[0].load(p.w_next, d);
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = r[c][i] * rs * wn[w][i];
      store_v<EL, V>(p.x_next, base + d, o);
    }
  }
}

template <int EL, int YEL, int V>
hipError_t launch_v(const BlockNorm& p, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(std::min(p.T, kGridX)), (static_cast<uint32_t>(p.T) + kGridX - 1) / kGridX);
  const dim3 block(kThreads);
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
