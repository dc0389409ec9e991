// Load-balance and z losses of the router, and the gradient of its logits.
//
// With key[t][e] = logits[t][e] + bias[e], p = softmax of a token's keys over all E, lse their log of the sum of
// exponentials, n the tokens whose mask is set, load_e the slots of those tokens that chose e:
//   balance = E sum_e load_e / (k n) * (1/n) sum_t p[t][e]          z = (1/n) sum_t lse[t]^2
// Gradient of a logit, with c = d_loss:
//   kept weights renormalised:  w_j (dw_j - sum_i w_i dw_i) at the expert of slot j
//   softmax entries as they are: p_e (dw of e's slot - sum_i w_i dw_i)
//   + c[0] E / (k n^2) p_e (load_e - sum p load) + c[1] (2 / n) lse p_e      (tokens whose mask is set)
//
// A wave takes one token at a time, its E <= 1024 keys in registers (up to 16 a lane), so each pass reads the logits
// once.  The losses need sums over tokens: waves add up the p of their own tokens in registers, workgroups in
// LDS, and one last workgroup adds the workgroups' sums in their order: no floating-point atomics.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kLossWaves = 8;      // of a workgroup of the loss pass
constexpr int kMaxLossBlocks = 128;
constexpr int kGradWaves = 4;

int loss_blocks(int T) { return std::max(1, std::min(kMaxLossBlocks, (T + kLossWaves - 1) / kLossWaves)); }

// Expert of value c of chunk i of a lane: 4 consecutive ones per lane and chunk.
__device__ __forceinline__ int expert_of(int i, int c) { return (i * 64 + lane_id()) * 4 + c; }

// A token's keys; -inf past E.  VEC: rows start at 16-byte boundaries.
template <int NC, bool VEC>
__device__ __forceinline__ void load_keys(const RouteGrad& p, int64_t t, float (&key)[NC][4]) {
  const float* row = p.logits + t * p.E;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int e = expert_of(i, 0);
    if (VEC) {
      const f32x4 v = e < p.E ? *reinterpret_cast<const f32x4*>(row + e) : f32x4{};
#pragma unroll
      for (int c = 0; c < 4; ++c) key[i][c] = v[c];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) key[i][c] = e + c < p.E ? row[e + c] : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int e = expert_of(i, c);
      if (p.bias && e < p.E) key[i][c] += p.bias[e];
      if (e >= p.E) key[i][c] = -INFINITY;
    }
}

// Softmax in place; the log of the sum of exponentials.  A token without a finite key: zeros, 0.
template <int NC>
__device__ __forceinline__ float softmax(float (&key)[NC][4]) {
  float m = -INFINITY, s = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) m = fmaxf(m, key[i][c]);
  m = wave_max(m);
  const bool none = m == -INFINITY;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      key[i][c] = none ? 0.0f : expf(key[i][c] - m);
      s += key[i][c];
    }
  s = wave_sum(s);
  const float inv = none ? 0.0f : 1.0f / s;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) key[i][c] *= inv;
  return none ? 0.0f : m + logf(s);
}

// Workgroups' sums: [blocks][E] of p, [blocks][E + 1] of the load and the tokens, [blocks] of lse^2.
struct LossParts {
  float* p;
  int32_t* load;
  float* z;
};
__host__ __device__ LossParts loss_parts(void* ws, int blocks, int E) {
  LossParts r;
  r.p = static_cast<float*>(ws);
  r.load = reinterpret_cast<int32_t*>(r.p + static_cast<int64_t>(blocks) * E);
  r.z = reinterpret_cast<float*>(r.load + static_cast<int64_t>(blocks) * (E + 1));
  return r;
}

template <int NC, bool VEC>
__global__ __launch_bounds__(kLossWaves* kWave) void loss_kernel(RouteGrad p, LossParts out) {
  __shared__ float sum[NC * 256];
  __shared__ int32_t load[NC * 256];
  __shared__ float z_of[kLossWaves];
  __shared__ int32_t n_of[kLossWaves];
  const int wave = threadIdx.x / kWave, lane = lane_id();
  for (int e = threadIdx.x; e < NC * 256; e += kLossWaves * kWave) {
    sum[e] = 0.0f;
    load[e] = 0;
  }
  __syncthreads();
  float acc[NC][4] = {}, z = 0.0f;
  int n = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kLossWaves + wave; t < p.T; t += gridDim.x * kLossWaves) {
    if (p.mask && !p.mask[t]) continue;  // the same for the whole wave
    float key[NC][4];
    load_keys<NC, VEC>(p, t, key);
    if (lane < p.k) {
      const int id = p.packed[t * 2 * p.k + lane];
      if (id >= 0 && id < p.E) atomicAdd(&load[id], 1);  // whole numbers: any order
    }
    const float lse = softmax<NC>(key);
    z = fmaf(lse, lse, z);
    ++n;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] += key[i][c];
  }
  for (int w = 0; w < kLossWaves; ++w) {  // waves in order
    __syncthreads();
    if (w == wave) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[expert_of(i, c)] += acc[i][c];
    }
  }
  if (lane == 0) {
    z_of[wave] = z;
    n_of[wave] = n;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kLossWaves * kWave) {
    out.p[static_cast<int64_t>(blockIdx.x) * p.E + e] = sum[e];
    out.load[static_cast<int64_t>(blockIdx.x) * (p.E + 1) + e] = load[e];
  }
  if (threadIdx.x == 0) {
    float zs = 0.0f;
    int ns = 0;
#pragma unroll
    for (int w = 0; w < kLossWaves; ++w) {
      zs += z_of[w];
      ns += n_of[w];
    }
    out.z[blockIdx.x] = zs;
    out.load[static_cast<int64_t>(blockIdx.x) * (p.E + 1) + p.E] = ns;
  }
}

__global__ __launch_bounds__(1024) void loss_finish_kernel(RouteGrad p, LossParts in, int blocks) {
  __shared__ float red[16], zred[16];
  __shared__ int32_t tokens;
  const int e = threadIdx.x;
  float s = 0.0f;
  int load = 0;
  if (e < p.E)
    for (int b = 0; b < blocks; ++b) {
      s += in.p[static_cast<int64_t>(b) * p.E + e];
      load += in.load[static_cast<int64_t>(b) * (p.E + 1) + e];
    }
  if (e == 1023) {  // E <= 1024: a thread with little else to do where E is smaller
    int n = 0;
    for (int b = 0; b < blocks; ++b) n += in.load[static_cast<int64_t>(b) * (p.E + 1) + p.E];
    tokens = n;
  }
  float z = e < blocks ? in.z[e] : 0.0f;
  const float bal = wave_sum(e < p.E ? s * static_cast<float>(load) : 0.0f);
  z = wave_sum(z);
  if (lane_id() == 0) {
    red[e / kWave] = bal;
    zred[e / kWave] = z;
  }
  __syncthreads();
  if (e < p.E) p.load[e] = load;
  if (e == 0) {
    float b = 0.0f, zs = 0.0f;
    for (int i = 0; i < 16; ++i) {
      b += red[i];
      zs += zred[i];
    }
    const float n = static_cast<float>(max(tokens, 1));
    p.loss[0] = b / n / n * (static_cast<float>(p.E) / static_cast<float>(p.k));
    p.loss[1] = zs / n;
    p.load[p.E] = tokens;
  }
}

template <int OEL, int NC, bool VEC>
__global__ __launch_bounds__(kGradWaves* kWave) void route_grad_kernel(RouteGrad p) {
  const int lane = lane_id();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGradWaves + threadIdx.x / kWave;
  if (t >= p.T) return;
  float v[NC][4], d[NC][4] = {};
  const bool aux = p.d_loss && (!p.mask || p.mask[t]);
  float lse = 0.0f;
  if (aux || !p.renormalize) {
    load_keys<NC, VEC>(p, t, v);
    lse = softmax<NC>(v);
  }
  if (p.d_w) {
    int id = -1;
    float w = 0.0f, dw = 0.0f;
    if (lane < p.k) {
      id = p.packed[t * 2 * p.k + lane];
      w = __int_as_float(p.packed[t * 2 * p.k + p.k + lane]);
      dw = p.d_w[t * p.k + lane];
    }
    const float mean = wave_sum(w * dw);
    // of a slot: what is added at its expert
    const float mine = p.renormalize ? w * (dw - mean) : dw;
    for (int j = 0; j < p.k; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float x = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), j));
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) d[i][c] += expert_of(i, c) == e ? x : 0.0f;
    }
    if (!p.renormalize) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) d[i][c] = v[i][c] * (d[i][c] - mean);
    }
  }
  if (aux) {
    const float n = static_cast<float>(max(p.load[p.E], 1));
    const float cb = p.d_loss[0] * static_cast<float>(p.E) / static_cast<float>(p.k) / n / n;
    const float cz = 2.0f * p.d_loss[1] / n * lse;
    float q = 0.0f, load[NC][4];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int e = expert_of(i, c);
        load[i][c] = e < p.E ? static_cast<float>(p.load[e]) : 0.0f;
        q = fmaf(v[i][c], load[i][c], q);
      }
    q = wave_sum(q);
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) d[i][c] = fmaf(v[i][c], fmaf(cb, load[i][c] - q, cz), d[i][c]);
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int e = expert_of(i, 0);
    if (e >= p.E) continue;
    const int64_t at = t * p.E + e;
    if constexpr (OEL == EL_F32) {
      float* o = static_cast<float*>(p.d_logits) + at;
      if (VEC) {
        *reinterpret_cast<f32x4*>(o) = f32x4{d[i][0], d[i][1], d[i][2], d[i][3]};
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (e + c < p.E) o[c] = d[i][c];
      }
    } else {
      uint16_t* o = static_cast<uint16_t*>(p.d_logits) + at;
      if (VEC) {
        *reinterpret_cast<uint2*>(o) = make_uint2(bf16x2_bits(d[i][0], d[i][1]), bf16x2_bits(d[i][2], d[i][3]));
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (e + c < p.E) o[c] = static_cast<uint16_t>(bf16x2_bits(d[i][c], 0.0f));
      }
    }
  }
}

// f(chunks of 256 experts, whether rows are read 16 bytes at a time)
template <typename F>
void by_width(const RouteGrad& p, F f) {
  const bool vec = p.E % 4 == 0 && ((reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.d_logits)) & 15) == 0;
  auto wide = [&](auto nc) {
    if (vec) f(nc, std::true_type{});
    else f(nc, std::false_type{});
  };
  if (p.E <= 256) wide(std::integral_constant<int, 1>{});
  else if (p.E <= 512) wide(std::integral_constant<int, 2>{});
  else wide(std::integral_constant<int, 4>{});
}

}  // namespace

size_t route_loss_workspace(int T, int E) {
  const int b = loss_blocks(T);
  return (static_cast<size_t>(b) * (2 * E + 2) * 4 + 255) & ~static_cast<size_t>(255);
}

hipError_t launch_route_loss(const RouteGrad& p, void* ws, hipStream_t s) {
  const int blocks = loss_blocks(p.T);
  const LossParts parts = loss_parts(ws, blocks, p.E);
  by_width(p, [&](auto nc, auto vec) {
    hipLaunchKernelGGL((loss_kernel<decltype(nc)::value, decltype(vec)::value>), dim3(blocks), dim3(kLossWaves * kWave), 0,
                       s, p, parts);
  });
  hipLaunchKernelGGL(loss_finish_kernel, dim3(1), dim3(1024), 0, s, p, parts, blocks);
  return hipGetLastError();
}

hipError_t launch_route_grad(int out_el, const RouteGrad& p, hipStream_t s) {
  by_width(p, [&](auto nc, auto vec) {
    const dim3 grid((p.T + kGradWaves - 1) / kGradWaves);
    if (out_el == EL_F32)
      hipLaunchKernelGGL((route_grad_kernel<EL_F32, decltype(nc)::value, decltype(vec)::value>), grid,
                         dim3(kGradWaves * kWave), 0, s, p);
    else
      hipLaunchKernelGGL((route_grad_kernel<EL_BF16, decltype(nc)::value, decltype(vec)::value>), grid,
                         dim3(kGradWaves * kWave), 0, s, p);
  });
  return hipGetLastError();
}

}  // namespace moe
