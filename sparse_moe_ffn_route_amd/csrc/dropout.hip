// Dropout whose mask is made from a counter and never stored: inside the experts' SwiGLU, in that activation's
// gradient, and on the branch that joins a residual stream.
//
// Generator: Philox-4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011).
// Key: the seed's two words.  Counter: the number of a block of 8 consecutive elements (64 bits) and the call's
// offset (64 bits), so that the mask of an element depends on the seed, the offset and the element's place only, and
// whoever asks again, the backward pass, a replayed graph, another launch shape, gets the same.  Element i of
// the block owns 16 of the 128 bits; it is dropped where they are below low = round(65536 p).  16 bits an
// element halve the generator's work against 32 and move p by up to 2^-17; the factor of the kept elements is
// 65536 / (65536 - low), by the p that is really applied.
//
// A dropped element's result is chosen, not multiplied, to be zero: what its inputs hold, infinities and NaN too,
// does not reach it.
//
// Bound by memory: a thread has one block of 8 elements, 16 bytes of each tensor, and all accesses go past the
// caches' replacement.  The activation's gradient reads three bf16 tensors and writes three, 403 MB for 32768 rows of
// 1024, in 66 us (6.1 TB/s); the activation 201 MB, and the residual sum as much for 8192 rows of 4096, in 33 us
// each.  The generator's ten rounds, 20 wide products a block, hide behind the memory: with p = 0, which skips them,
// the three calls take as long.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 1 << 16;

// The 8 x 16 bits of block b.
__device__ __forceinline__ u32x4 philox(uint64_t b, uint64_t seed, uint64_t offset) {
  uint32_t c0 = static_cast<uint32_t>(b), c1 = static_cast<uint32_t>(b >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u, p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(p1);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

__device__ __forceinline__ bool kept(const u32x4& bits, int i, uint32_t low) {
  return ((bits[i / 2] >> (i % 2 * 16)) & 0xFFFFu) >= low;
}

// 8 values as stored: 16 bytes at a time, or one by one.
template <int EL>
struct Eight {
  float v[8];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
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
  __device__ __forceinline__ void store(void* base, int64_t at) const {
    if constexpr (EL == EL_F32) {
      f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(base) + at);
      __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, p);
      __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, p + 1);
    } else {
      const u32x4 w{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7])};
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + at));
    }
  }
  static __device__ __forceinline__ float one(const void* base, int64_t at) {
    if constexpr (EL == EL_F32) return static_cast<const float*>(base)[at];
    else return bf16_bits_to_f32(static_cast<const uint16_t*>(base)[at]);
  }
  static __device__ __forceinline__ void put(void* base, int64_t at, float v) {
    if constexpr (EL == EL_F32) static_cast<float*>(base)[at] = v;
    else static_cast<uint16_t*>(base)[at] = static_cast<uint16_t>(bf16x2_bits(v, 0.0f));
  }
};

// 1 / (1 + e^-z).  bf16 results: hardware exponential and reciprocal, each within an ulp or two of fp32, far
// below the rounding to 8 bits; fp32 results: the library's exponential and an IEEE division.
template <int EL>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (EL == EL_F32) return 1.0f / (1.0f + expf(-z));
  else return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// VEC: I and ld are multiples of 8 and every address of 16 bytes, so a block of 8 elements is 16-byte accesses.
template <int EL, bool GRAD, bool VEC>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(SwigluDrop p) {
  int64_t rows = p.rows;
  if (p.n_rows) rows = min(rows, static_cast<int64_t>(max(*p.n_rows, 0)));
  const int64_t n = rows * p.I, blocks = (n + 7) / 8;
  uint64_t seed = 0, offset = 0;
  if (p.low) { seed = p.rng[0]; offset = p.rng[1]; }
  for (int64_t b = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; b < blocks;
       b += gridDim.x * static_cast<int64_t>(kThreads)) {
    const int64_t e = b * 8, r = e / p.I, c = e - r * p.I, at = r * p.ld + c;
    u32x4 bits{};
    auto element = [&](int i, float g, float u, float d, float& h, float& dg, float& du) {
      const bool keep = !p.low || kept(bits, i, p.low);
      const float s = sigmoid<EL>(g), a = g * s;
      h = keep ? a * u * p.factor : 0.0f;
      if constexpr (GRAD) {
        d *= p.factor;
        dg = keep ? d * u * (s * fmaf(g, 1.0f - s, 1.0f)) : 0.0f;
        du = keep ? d * a : 0.0f;
      }
    };
    if constexpr (VEC) {
      Eight<EL> g, u, d{}, h, dg, du;
      g.load(p.gate, at);
      u.load(p.up, at);
      if constexpr (GRAD) d.load(p.d_h, e);
      if (p.low) bits = philox(b, seed, offset);
#pragma unroll
      for (int i = 0; i < 8; ++i) element(i, g.v[i], u.v[i], d.v[i], h.v[i], dg.v[i], du.v[i]);
      if (!GRAD || p.h) h.store(p.h, e);
      if constexpr (GRAD) {
        dg.store(p.d_gate, at);
        du.store(p.d_up, at);
      }
    } else {
      if (p.low) bits = philox(b, seed, offset);
      int64_t row = r, col = c;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (e + i >= n) break;
        const int64_t q = row * p.ld + col;
        float h, dg = 0.f, du = 0.f;
        element(i, Eight<EL>::one(p.gate, q), Eight<EL>::one(p.up, q), GRAD ? Eight<EL>::one(p.d_h, e + i) : 0.0f, h,
                dg, du);
        if (!GRAD || p.h) Eight<EL>::put(p.h, e + i, h);
        if constexpr (GRAD) {
          Eight<EL>::put(p.d_gate, q, dg);
          Eight<EL>::put(p.d_up, q, du);
        }
        if (++col == p.I) { col = 0; ++row; }
      }
    }
  }
}

template <int EL, bool VEC>
__global__ __launch_bounds__(kThreads) void dropout_kernel(Dropout p) {
  const int64_t blocks = (p.n + 7) / 8;
  uint64_t seed = 0, offset = 0;
  if (p.low) { seed = p.rng[0]; offset = p.rng[1]; }
  for (int64_t b = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; b < blocks;
       b += gridDim.x * static_cast<int64_t>(kThreads)) {
    const int64_t e = b * 8;
    u32x4 bits{};
    if (VEC && e + 8 <= p.n) {
      Eight<EL> x, r{};
      x.load(p.x, e);
      if (p.residual) r.load(p.residual, e);
      if (p.low) bits = philox(b, seed, offset);
#pragma unroll
      for (int i = 0; i < 8; ++i) x.v[i] = r.v[i] + (!p.low || kept(bits, i, p.low) ? x.v[i] * p.factor : 0.0f);
      x.store(p.out, e);
    } else {
      if (p.low) bits = philox(b, seed, offset);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (e + i >= p.n) break;
        const float r = p.residual ? Eight<EL>::one(p.residual, e + i) : 0.0f, x = Eight<EL>::one(p.x, e + i);
        Eight<EL>::put(p.out, e + i, r + (!p.low || kept(bits, i, p.low) ? x * p.factor : 0.0f));
      }
    }
  }
}

template <typename... A>
bool at16(const A*... a) { return ((reinterpret_cast<uintptr_t>(a) | ...) & 15) == 0; }

dim3 grid_of(int64_t blocks) {
  return dim3(static_cast<unsigned>(std::min<int64_t>((blocks + kThreads - 1) / kThreads, kMaxBlocks)));
}

}  // namespace

hipError_t launch_swiglu(int el, bool grad, const SwigluDrop& p, hipStream_t s) {
  const bool vec = p.I % 8 == 0 && p.ld % 8 == 0 && at16(p.gate, p.up, p.d_h, p.h, p.d_gate, p.d_up);
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid_of((p.rows * p.I + 7) / 8), dim3(kThreads), 0, s, p);
  };
  auto typed = [&](auto e) {
    constexpr int EL = decltype(e)::value;
    if (grad) vec ? launch(swiglu_kernel<EL, true, true>) : launch(swiglu_kernel<EL, true, false>);
    else vec ? launch(swiglu_kernel<EL, false, true>) : launch(swiglu_kernel<EL, false, false>);
  };
  if (el == EL_F32) typed(std::integral_constant<int, EL_F32>{});
  else typed(std::integral_constant<int, EL_BF16>{});
  return hipGetLastError();
}

hipError_t launch_dropout(int el, const Dropout& p, hipStream_t s) {
  const bool vec = at16(p.x, p.residual, p.out);
  auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid_of((p.n + 7) / 8), dim3(kThreads), 0, s, p); };
  if (el == EL_F32) vec ? launch(dropout_kernel<EL_F32, true>) : launch(dropout_kernel<EL_F32, false>);
  else vec ? launch(dropout_kernel<EL_BF16, true>) : launch(dropout_kernel<EL_BF16, false>);
  return hipGetLastError();
}

}  // namespace moe
