// Microscaled 4-bit storage: weights to the packed image and back, activation rows to
// records (formats in mx.hpp).
//
// All three are streams: pack reads 2 (bf16) or 4 (fp32) bytes and writes 17/32 byte per
// value, unpack the reverse.  Measured, 64 matrices of 1024 x 4096 (537 MB of bf16, 143 MB of images): pack
// 120 us, unpack 122, 5.6 TB/s (a device copy reaches 4.9).  What is read or written once goes past the caches'
// replacement: pack took 158 without that, and unpack 107 after such a pack, whose images it
// then found in the cache before HBM, 128 otherwise.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"
#include "mx.hpp"

namespace moe {

namespace {

typedef uint32_t u32;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16v2 __attribute__((ext_vector_type(2)));

// 8 consecutive values: fp32, or bf16 as they are.
template <int EL>
struct Octet {
  u32 w[EL == EL_F32 ? 8 : 4];

  // NT: past the caches' replacement, for what is read once.
  template <bool NT = false>
  __device__ __forceinline__ void load(const void* base, size_t idx) {
    constexpr int bytes = EL == EL_F32 ? 4 : 2;
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(base) + idx * bytes);
#pragma unroll
    for (int i = 0; i < bytes / 2; ++i) {
      const u32x4 a = NT ? __builtin_nontemporal_load(p + i) : p[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = a[j];
    }
  }

  // Bits of the largest magnitude, as fp32.
  __device__ __forceinline__ u32 abs_max() const {
    if constexpr (EL == EL_F32) {
      u32 m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
      return m;
    } else {
      u16x2 m = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu));
      return static_cast<u32>(m.x > m.y ? m.x : m.y) << 16;
    }
  }

  // Codes of the values divided by scale, a power of two.
  __device__ __forceinline__ u32 codes(float scale) const {
    u32 r = 0;
    if constexpr (EL == EL_F32) {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[0]), __uint_as_float(w[1]), scale, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[2]), __uint_as_float(w[3]), scale, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[4]), __uint_as_float(w[5]), scale, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[6]), __uint_as_float(w[7]), scale, 3);
    } else {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16v2, w[0]), scale, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16v2, w[1]), scale, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16v2, w[2]), scale, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16v2, w[3]), scale, 3);
    }
    return r;
  }
};

// The value of the lane whose index differs by X (1 or 2) from this one's, within its four.
template <int X>
__device__ __forceinline__ u32 quad_xor(u32 v) {
  constexpr int ctrl = X == 1 ? 0xB1 : 0x4E;  // quad_perm 1,0,3,2 and 2,3,0,1
  return static_cast<u32>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), ctrl, 0xF, 0xF, false));
}

// w[i] of lane q becomes w[q] of lane i, within four lanes.
__device__ __forceinline__ void quad_transpose(u32 (&w)[4], int q) {
  const bool odd = (q & 1) != 0, high = (q & 2) != 0;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const u32 got = quad_xor<1>(odd ? w[i] : w[i + 1]);
    if (odd) w[i] = got; else w[i + 1] = got;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const u32 got = quad_xor<2>(high ? w[i] : w[i + 2]);
    if (high) w[i] = got; else w[i + 2] = got;
  }
}

// One wave per (matrix, 16 rows, group).  (Reading 1 KB of one row at a time instead took 172 us against 158.)
// Lane l reads 8 values of row 4 i + l / 16 from (l % 16) * 8 on
// (whole lines), a block's four lanes share its magnitude, and a 4x4 transpose between them makes each
// the holder of one block, so the codes go out as whole 1 KB runs and the scales as one 256-byte store.
template <int EL>
__global__ __launch_bounds__(256) void mx_pack_kernel(const void* __restrict__ src, uint8_t* __restrict__ dst,
                                                      int64_t units, int cols) {
  const int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / kWave;
  if (u >= units) return;
  const int lane = threadIdx.x % kWave;
  const int groups = mx_groups(cols);
  const int g = static_cast<int>(u % groups);
  const int64_t fr = u / groups;  // fragment over all matrices
  const int steps = min(4, mx_steps(cols) - g * 4);
  uint8_t* out = dst + fr * mx_fragment_bytes(cols) + static_cast<int64_t>(g) * kMxGroupBytes;
  const int q = lane & 3, blk = (lane & 15) >> 2, r = lane >> 4;
  const int slot = blk * 16 + q * 4 + r;  // the block that this lane stores
  u32 scales = 0x7F7F7F7Fu;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (s >= steps) continue;
    const int k0 = g * kMxGroup + s * kMxStep + (lane & 15) * 8;
    const int k = min(k0, cols - 8);  // behind the last value: read again, stored as zero
    Octet<EL> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i].template load<true>(src, (static_cast<size_t>(fr) * 16 + i * 4 + r) * cols + k);
    u32 codes[4];
    u32 byte = 127u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32 m = v[i].abs_max();
      m = max(m, quad_xor<1>(m));
      m = max(m, quad_xor<2>(m));
      const u32 b = mx_scale_byte(m);
      const u32 c = v[i].codes(__uint_as_float(b << 23));
      codes[i] = b == 255u || k0 >= cols ? 0u : c;
      byte = i == q ? b : byte;
    }
    if (k0 < cols) scales = (scales & ~(0xFFu << (8 * s))) | (byte << (8 * s));
    quad_transpose(codes, q);
    __builtin_nontemporal_store((u32x4{codes[0], codes[1], codes[2], codes[3]}),
                                reinterpret_cast<u32x4*>(out + s * kMxRun + slot * 16));
  }
  __builtin_nontemporal_store(scales, reinterpret_cast<u32*>(out + steps * kMxRun + slot * 4));
}

// One wave per (matrix, 16 rows, group).  Lane l decodes one dword of codes at a time, 8 values of row
// r0 + l / 16 from (l % 16) * 8 on, so that four rows' 128 values go out as whole lines (a lane that
// decoded a block of its own stored 16 bytes every 64 and took twice the time).
template <int EL>
__global__ __launch_bounds__(256) void mx_unpack_kernel(const uint8_t* __restrict__ src, void* __restrict__ dst,
                                                        int64_t units, int cols) {
  const int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / kWave;
  if (u >= units) return;
  const int lane = threadIdx.x % kWave;
  const int groups = mx_groups(cols);
  const int g = static_cast<int>(u % groups);
  const int64_t fr = u / groups;
  const int steps = min(4, mx_steps(cols) - g * 4);
  const uint8_t* in = src + fr * mx_fragment_bytes(cols) + static_cast<int64_t>(g) * kMxGroupBytes;
  const int blk = (lane & 15) >> 2, r = lane >> 4;
  u32 scales[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    scales[i] = *reinterpret_cast<const u32*>(in + steps * kMxRun + (blk * 16 + i * 4 + r) * 4);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k0 = g * kMxGroup + s * kMxStep + (lane & 15) * 8;
    if (s >= steps || k0 >= cols) continue;
    u32 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = *reinterpret_cast<const u32*>(in + s * kMxRun + blk * 256 + (i * 4 + r) * 16 + (lane & 3) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32 b = (scales[i] >> (8 * s)) & 255u;
      const float scale = __uint_as_float(b == 255u ? 0x7FC00000u : b << 23);  // byte 255 stands for NaN
      const size_t idx = (static_cast<size_t>(fr) * 16 + i * 4 + r) * cols + k0;
      f32x2 v[4];
      v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 0) * scale;
      v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 1) * scale;
      v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 2) * scale;
      v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 3) * scale;
      if constexpr (EL == EL_F32) {
        f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(dst) + idx);
        __builtin_nontemporal_store((f32x4{v[0].x, v[0].y, v[1].x, v[1].y}), p);
        __builtin_nontemporal_store((f32x4{v[2].x, v[2].y, v[3].x, v[3].y}), p + 1);
      } else {
        __builtin_nontemporal_store((u32x4{bf16x2_bits(v[0].x, v[0].y), bf16x2_bits(v[1].x, v[1].y),
                                           bf16x2_bits(v[2].x, v[2].y), bf16x2_bits(v[3].x, v[3].y)}),
                                    reinterpret_cast<u32x4*>(static_cast<uint16_t*>(dst) + idx));
      }
    }
  }
}

// M-tile prefix of at most 1024 groups by one workgroup of 256 threads: four groups per thread.
__device__ void tile_prefix(const int32_t* offsets, int n_groups, int bm, int32_t* prefix) {
  __shared__ int sums[4];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, g0 = threadIdx.x * 4;
  int c[4], mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = g0 + i < n_groups ? (offsets[g0 + i + 1] - offsets[g0 + i] + bm - 1) / bm : 0;
    mine += c[i];
  }
  int sum = mine;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int v = __shfl_up(sum, o, kWave);
    if (lane >= o) sum += v;
  }
  if (lane == kWave - 1) sums[wave] = sum;
  __syncthreads();
  for (int w = 0; w < wave; ++w) sum += sums[w];
  sum -= mine;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (g0 + i <= n_groups) prefix[g0 + i] = sum;
    sum += c[i];
  }
  if (threadIdx.x == 255 && n_groups == 1024) prefix[1024] = sum;
}

// bf16 rows -> records.  Four lanes share a block (8 values each): loads of 16 bytes and
// stores of 4 bytes per lane are contiguous over the wave, one wave per record.
__global__ __launch_bounds__(256) void mx_rows_kernel(const uint16_t* __restrict__ src, int rows,
                                                      const int32_t* __restrict__ n_rows_dev, int cols,
                                                      uint8_t* __restrict__ dst, const int32_t* __restrict__ offsets,
                                                      int n_groups, int bm, int32_t* __restrict__ prefix) {
  if (prefix && blockIdx.x == gridDim.x - 1) {
    tile_prefix(offsets, n_groups, bm, prefix);
    return;
  }
  const int groups = mx_groups(cols);
  const int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / kWave;
  const int64_t row = u / groups;
  const int g = static_cast<int>(u - row * groups);
  const int n = n_rows_dev ? min(rows, ld_scalar(n_rows_dev)) : rows;
  if (row >= n) return;
  const int lane = threadIdx.x % kWave;
  const int k0 = g * kMxGroup + lane * 8;
  Octet<EL_BF16> v = {};
  if (k0 < cols) v.load(src, static_cast<size_t>(row) * cols + k0);
  u32 m = v.abs_max();
  m = max(m, quad_xor<1>(m));
  m = max(m, quad_xor<2>(m));
  const u32 b = mx_scale_byte(m);
  const u32 codes = b == 255u ? 0u : v.codes(__uint_as_float(b << 23));
  uint8_t* out = dst + row * mx_row_bytes(cols) + static_cast<int64_t>(g) * kMxRecord;
  *reinterpret_cast<u32*>(out + lane * 4) = codes;
  const int blk = lane >> 2;  // block of the group: step blk / 4, lane group blk % 4
  if ((lane & 3) == 0) out[256 + (blk & 3) * 4 + (blk >> 2)] = static_cast<uint8_t>(b);
}

}  // namespace

hipError_t launch_mx_pack(int src_el, const void* src, int64_t n_mats, int rows, int cols, void* dst,
                          hipStream_t stream) {
  const int64_t units = n_mats * (rows / 16) * mx_groups(cols);
  if (units == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>((units + 3) / 4));
  if (src_el == EL_F32)
    hipLaunchKernelGGL((mx_pack_kernel<EL_F32>), grid, dim3(256), 0, stream, src, static_cast<uint8_t*>(dst), units,
                       cols);
  else
    hipLaunchKernelGGL((mx_pack_kernel<EL_BF16>), grid, dim3(256), 0, stream, src, static_cast<uint8_t*>(dst), units,
                       cols);
  return hipGetLastError();
}

hipError_t launch_mx_unpack(int dst_el, const void* src, int64_t n_mats, int rows, int cols, void* dst,
                            hipStream_t stream) {
  const int64_t units = n_mats * (rows / 16) * mx_groups(cols);
  if (units == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>((units + 3) / 4));
  if (dst_el == EL_F32)
    hipLaunchKernelGGL((mx_unpack_kernel<EL_F32>), grid, dim3(256), 0, stream, static_cast<const uint8_t*>(src), dst,
                       units, cols);
  else
    hipLaunchKernelGGL((mx_unpack_kernel<EL_BF16>), grid, dim3(256), 0, stream, static_cast<const uint8_t*>(src), dst,
                       units, cols);
  return hipGetLastError();
}

hipError_t launch_mx_rows(const void* src, int rows, const int32_t* n_rows_dev, int cols, void* dst,
                          const int32_t* offsets, int n_groups, int bm, int32_t* prefix, hipStream_t stream) {
  const int64_t units = static_cast<int64_t>(rows) * mx_groups(cols);
  if (units == 0) return hipSuccess;
  hipLaunchKernelGGL(mx_rows_kernel, dim3(static_cast<uint32_t>((units + 3) / 4) + (prefix ? 1 : 0)), dim3(256), 0,
                     stream, static_cast<const uint16_t*>(src), rows, n_rows_dev, cols, static_cast<uint8_t*>(dst),
                     offsets, n_groups, bm, prefix);
  return hipGetLastError();
}

}  // namespace moe
