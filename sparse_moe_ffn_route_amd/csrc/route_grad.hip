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
//
// 8192 tokens of 512 experts read 17 MB twice and write 8: 9 us at memory's rate, but each token also costs three
// passes over its registers and three sums over the wave, and there are three launches of 3 us at least: 32 us in
// all, 10.8 the sums over tokens, 6.6 their joining, 11.6 the gradient.  Fewer workgroups of the first pass leave the
// CUs idle, more make the joining longer; 128 of 16 waves was the least of both.  64 tokens of 16 experts: 10 us.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kLossWaves = 16;     // of a workgroup of the loss pass
constexpr int kMaxLossBlocks = 128;
constexpr int kGradWaves = 4;
constexpr int kFinish = 1024;      // threads that add up the workgroups' sums

int loss_blocks(int T) { return std::max(1, std::min(kMaxLossBlocks, (T + kLossWaves - 1) / kLossWaves)); }

// Sum and largest value over the wave, in every lane: shifts within rows of 16 lanes, then each row's last lane to the
// next rows, through the lanes' data paths (six steps through LDS take as long as all else that a token needs).
template <int CTRL, int ROWS>
__device__ __forceinline__ float from_lane(float none, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(v), CTRL, ROWS, 0xf, false));
}
template <typename F>
__device__ __forceinline__ float over_wave(float v, float none, F f) {
  v = f(v, from_lane<0x111, 0xf>(none, v));
  v = f(v, from_lane<0x112, 0xf>(none, v));
  v = f(v, from_lane<0x114, 0xf>(none, v));
  v = f(v, from_lane<0x118, 0xf>(none, v));
  v = f(v, from_lane<0x142, 0xa>(none, v));
  v = f(v, from_lane<0x143, 0xc>(none, v));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float sum_of(float v) {
  return over_wave(v, 0.0f, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float max_of(float v) {
  return over_wave(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}

// e^x for x <= 0 (0 for -inf, NaN for NaN).  x log2(e) is taken to twice fp32's digits, its head through the hardware's
// power of two, the rest as the first term of its series: 2 ulp, in a third of the library function's
// instructions (8192 tokens of 512, both passes: 32.5 us, with expf 34.0).  Where the head is so far down that the
// power is zero the rest can be anything, infinite or NaN, and is bounded.
__device__ __forceinline__ float exp_of(float x) {
  constexpr float kLog2e = 0x1.715476p0f, kLog2eRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float head = x * kLog2e;
  const float rest = __builtin_amdgcn_fmed3f(fmaf(x, kLog2eRest, fmaf(x, kLog2e, -head)), -1.0f, 1.0f);
  const float y = __builtin_amdgcn_exp2f(head);
  return fmaf(y, rest * kLn2, y);
}

// Expert of value c of chunk i of a lane: 4 consecutive ones per lane and chunk.
__device__ __forceinline__ int expert_of(int i, int c) { return (i * 64 + lane_id()) * 4 + c; }

// 4 NC values of a row of E that lane has, 0 past E.  VEC: rows start at 16-byte boundaries.
template <int NC, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, f32x4 (&v)[NC]) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int e = expert_of(i, 0);
    v[i] = f32x4{};
    if (VEC) {
      if (e < E) v[i] = *reinterpret_cast<const f32x4*>(row + e);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (e + c < E) v[i][c] = row[e + c];
    }
  }
}

// Keys of a token's logits; -inf past E.
template <int NC>
__device__ __forceinline__ void to_keys(const f32x4 (&logit)[NC], const f32x4 (&bias)[NC], int E, float (&key)[NC][4]) {
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) key[i][c] = expert_of(i, c) < E ? logit[i][c] + bias[i][c] : -INFINITY;
}

// Softmax in place; the log of the sum of exponentials.  A token whose keys are all -inf: zeros, 0; a NaN or +inf among
// them: NaN.
template <int NC>
__device__ __forceinline__ float softmax(float (&key)[NC][4]) {
  float m = -INFINITY, s = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) m = fmaxf(m, key[i][c]);
  m = max_of(m);
  m = m == -INFINITY ? 0.0f : m;  // all -inf, or NaN, which a maximum passes over
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      key[i][c] = exp_of(key[i][c] - m);
      s += key[i][c];
    }
  s = sum_of(s);
  const bool none = s == 0.0f;
  const float inv = none ? 0.0f : 1.0f / s;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) key[i][c] *= inv;
  return none ? 0.0f : m + logf(s);
}

// Workgroups' sums: [blocks][E] of p and the load, then [blocks] of lse^2 and the tokens.
struct Part {
  float sum;
  int32_t count;
};

template <int NC, bool VEC>
__global__ __launch_bounds__(kLossWaves* kWave) void loss_kernel(RouteGrad p, Part* out) {
  __shared__ float sum[NC * 256];
  __shared__ int32_t load[NC * 256];
  __shared__ float z_of[kLossWaves];
  __shared__ int32_t n_of[kLossWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  for (int e = threadIdx.x; e < NC * 256; e += kLossWaves * kWave) {
    sum[e] = 0.0f;
    load[e] = 0;
  }
  __syncthreads();
  f32x4 bias[NC] = {}, next[NC];
  if (p.bias) load_row<NC, VEC>(p.bias, p.E, bias);
  float acc[NC][4] = {}, z = 0.0f;
  int n = 0, next_id = -1, next_on = 0;
  const int by = gridDim.x * kLossWaves;
  int t = blockIdx.x * kLossWaves + wave;
  // a token's values are asked for while the one before is worked on
  auto ask = [&](int64_t t) {
    if (t >= p.T) return;
    next_on = p.mask ? p.mask[t] : 1;
    next_id = lane < p.k ? p.packed[t * 2 * p.k + lane] : -1;
    load_row<NC, VEC>(p.logits + t * p.E, p.E, next);
  };
  ask(t);
  for (; t < p.T; t += by) {
    float key[NC][4];
    to_keys<NC>(next, bias, p.E, key);
    const int id = next_id, on = __builtin_amdgcn_readfirstlane(next_on);
    ask(static_cast<int64_t>(t) + by);
    if (!on) continue;
    if (id >= 0 && id < p.E) atomicAdd(&load[id], 1);  // whole numbers: any order
    const float lse = softmax<NC>(key);
    z = fmaf(lse, lse, z);
    ++n;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] += key[i][c];
  }
  for (int w = 0; w < min(kLossWaves, p.T); ++w) {  // waves in order
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
  for (int e = threadIdx.x; e < p.E; e += kLossWaves * kWave)
    out[static_cast<int64_t>(blockIdx.x) * p.E + e] = Part{sum[e], load[e]};
  if (threadIdx.x == 0) {
    Part all{0.0f, 0};
#pragma unroll
    for (int w = 0; w < kLossWaves; ++w) {
      all.sum += z_of[w];
      all.count += n_of[w];
    }
    out[static_cast<int64_t>(gridDim.x) * p.E + blockIdx.x] = all;
  }
}

// One workgroup.  `lanes` threads (a power of two, at least E) take an expert each, kFinish / lanes of them
// the same one: each adds up every so many workgroups' sums, kUnder under way at a time.
__global__ __launch_bounds__(kFinish) void loss_finish_kernel(RouteGrad p, const Part* in, int blocks, int lanes) {
  constexpr int kUnder = 16;
  __shared__ float psum[kFinish], red[kFinish / kWave], zred[kFinish / kWave];
  __shared__ int32_t lsum[kFinish], nred[kFinish / kWave];
  const int tid = threadIdx.x, e = tid & (lanes - 1), first = tid / lanes, by = kFinish / lanes;
  // kMaxLossBlocks <= kFinish: a thread per workgroup
  const Part own = tid < blocks ? in[static_cast<int64_t>(blocks) * p.E + tid] : Part{0.0f, 0};
  float s = 0.0f;
  int load = 0;
  if (e < p.E) {
    for (int b0 = first; b0 < blocks; b0 += by * kUnder) {
      Part v[kUnder];
#pragma unroll
      for (int x = 0; x < kUnder; ++x)
        v[x] = b0 + x * by < blocks ? in[static_cast<int64_t>(b0 + x * by) * p.E + e] : Part{0.0f, 0};
#pragma unroll
      for (int x = 0; x < kUnder; ++x) {
        s += v[x].sum;
        load += v[x].count;
      }
    }
  }
  psum[tid] = s;
  lsum[tid] = load;
  const float z = sum_of(own.sum);
  const int n = wave_sum_int(own.count);
  __syncthreads();
  if (tid < lanes)
    for (int g = 1; g < by; ++g) {
      s += psum[g * lanes + tid];
      load += lsum[g * lanes + tid];
    }
  const bool mine = tid < lanes && e < p.E;
  const float bal = sum_of(mine ? s * static_cast<float>(load) : 0.0f);
  if (lane_id() == 0) {
    red[tid / kWave] = bal;
    zred[tid / kWave] = z;
    nred[tid / kWave] = n;
  }
  __syncthreads();
  if (mine) p.load[e] = load;
  if (tid == 0) {
    float b = 0.0f, zs = 0.0f;
    int tokens = 0;
    for (int i = 0; i < kFinish / kWave; ++i) {
      b += red[i];
      zs += zred[i];
      tokens += nred[i];
    }
    const float many = static_cast<float>(max(tokens, 1));
    p.loss[0] = b / many / many * (static_cast<float>(p.E) / static_cast<float>(p.k));
    p.loss[1] = zs / many;
    p.load[p.E] = tokens;
  }
}

template <int OEL, int NC, bool VEC>
__global__ __launch_bounds__(kGradWaves* kWave) void route_grad_kernel(RouteGrad p) {
  const int lane = lane_id();
  const int64_t t = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kGradWaves +
                    __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (t >= p.T) return;
  const bool losses = p.d_loss != nullptr, soft = losses || !p.renormalize;
  // everything is asked for before anything is used
  f32x4 logit[NC] = {}, bias[NC] = {};
  int32_t load[NC][4] = {};
  int id = -1, on = 1;
  float w = 0.0f, dw = 0.0f;
  if (soft) load_row<NC, VEC>(p.logits + t * p.E, p.E, logit);
  if (soft && p.bias) load_row<NC, VEC>(p.bias, p.E, bias);
  if (p.d_w && lane < p.k) {
    id = p.packed[t * 2 * p.k + lane];
    w = __int_as_float(p.packed[t * 2 * p.k + p.k + lane]);
    dw = p.d_w[t * p.k + lane];
  }
  float many = 1.0f, d_bal = 0.0f, d_z = 0.0f;
  if (losses) {
    if (p.mask) on = p.mask[t];
    f32x4 l[NC];
    load_row<NC, VEC>(reinterpret_cast<const float*>(p.load), p.E, l);
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) load[i][c] = __float_as_int(l[i][c]);
    many = static_cast<float>(max(ld_scalar(p.load + p.E), 1));
    d_bal = ld_scalar(p.d_loss);
    d_z = ld_scalar(p.d_loss + 1);
  }
  const bool aux = losses && __builtin_amdgcn_readfirstlane(on) != 0;
  float v[NC][4], d[NC][4] = {};
  float lse = 0.0f;
  if (aux || !p.renormalize) {
    to_keys<NC>(logit, bias, p.E, v);
    lse = softmax<NC>(v);
  }
  if (p.d_w) {
    if (__ballot(w != w)) {
      // Keys that are all -inf have NaN for weights and take no gradient from them; any other NaN goes on.
      bool some = false;
      for (int e = lane; e < p.E; e += kWave)
        some |= !(p.logits[t * p.E + e] + (p.bias ? p.bias[e] : 0.0f) == -INFINITY);
      if (!__ballot(some)) w = dw = 0.0f;
    }
    const float mean = sum_of(w * dw);
    // of a slot: what is added at its expert
    const float mine = p.renormalize ? w * (dw - mean) : dw;
    for (int j = 0; j < p.k; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float x = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), j));
      const float here = lane == ((e >> 2) & 63) ? x : 0.0f;
      const int at = (e >> 8) * 4 + (e & 3);  // the same for the whole wave: one of the lane's registers
#pragma unroll
      for (int i = 0; i < NC * 4; ++i)
        if (at == i) d[i / 4][i % 4] += here;
    }
    if (!p.renormalize) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) d[i][c] = v[i][c] * (d[i][c] - mean);
    }
  }
  if (aux) {
    const float cb = d_bal * static_cast<float>(p.E) / static_cast<float>(p.k) / many / many;
    const float cz = 2.0f * d_z / many * lse;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) q = fmaf(v[i][c], static_cast<float>(load[i][c]), q);
    q = sum_of(q);
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) d[i][c] = fmaf(v[i][c], fmaf(cb, static_cast<float>(load[i][c]) - q, cz), d[i][c]);
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
  const auto at = [](const void* a) { return reinterpret_cast<uintptr_t>(a); };
  const bool vec = p.E % 4 == 0 && ((at(p.logits) | at(p.bias) | at(p.d_logits) | at(p.load)) & 15) == 0;
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
  return (static_cast<size_t>(b) * (E + 1) * sizeof(Part) + 255) & ~static_cast<size_t>(255);
}

hipError_t launch_route_loss(const RouteGrad& p, void* ws, hipStream_t s) {
  const int blocks = loss_blocks(p.T);
  Part* parts = static_cast<Part*>(ws);
  by_width(p, [&](auto nc, auto vec) {
    hipLaunchKernelGGL((loss_kernel<decltype(nc)::value, decltype(vec)::value>), dim3(blocks), dim3(kLossWaves * kWave), 0,
                       s, p, parts);
  });
  int lanes = kWave;
  while (lanes < p.E) lanes *= 2;
  hipLaunchKernelGGL(loss_finish_kernel, dim3(1), dim3(kFinish), 0, s, p, parts, blocks, lanes);
  return hipGetLastError();
}

hipError_t launch_route_grad(int out_el, const RouteGrad& p, hipStream_t s) {
  by_width(p, [&](auto nc, auto vec) {
    const int blocks = (p.T + kGradWaves - 1) / kGradWaves, x = std::min(blocks, 1 << 20);
    const dim3 grid(x, (blocks + x - 1) / x);  // a grid dimension holds less than 2^32 threads
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
