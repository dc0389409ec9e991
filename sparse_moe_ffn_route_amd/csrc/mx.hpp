// Microscaled 4-bit floating point (OCP MX, E2M1 elements with E8M0 block scales): storage
// and device helpers shared by the kernels that write and read it.
//
// A block is 32 consecutive values of one row; with amax its largest magnitude,
//   e = floor(log2(amax)) - 2 (clamped to [-126, 127]; 0 for a zero block),
//   code = v * 2^-e rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even
//   code, magnitudes above 6 to 6), sign in bit 3; scale byte = e + 127.
// A block that holds a NaN or an infinity gets scale byte 255, which stands for NaN.
//
// Weights ("image", fragment-major like the other packed weights): for each 16 rows and each
// group of 512 values of the reduction dimension, up to four runs of 1 KB (one per "step" of
// 128 values: lane l holds the 16 bytes of row l % 16, values (l / 16) * 32 .. + 31, low
// nibble first), then 256 bytes of scales: lane l's dword holds its block's byte of each of
// the group's steps.  A 16x16x128 MFMA takes a run and one byte of that dword as they are,
// and the scales stream with the codes they belong to.  The last step is padded with zero
// codes where the width is 64 past a multiple of 128.
//
// Rows (activations): each row is ceil(K / 512) records of 272 bytes: 256 bytes of codes
// (block b at 16 * b), then the dwords of scales of the four lane groups.  272 = 17 * 16, so
// the records of 16 rows staged back to back in LDS start in different banks and every
// fragment read is free of conflicts without a swizzle.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int EL_MXFP4 = 3;            // as MOE_MXFP4
constexpr int kMxBlock = 32;
constexpr int kMxStep = 128;           // values per MFMA
constexpr int kMxGroup = 512;          // values per group of four steps
constexpr int kMxRun = 1024;           // bytes of one step of 16 weight rows
constexpr int kMxScales = 256;         // bytes of one group's scales of 16 weight rows
constexpr int kMxGroupBytes = 4 * kMxRun + kMxScales;
constexpr int kMxRecord = 272;         // bytes of one group of an activation row

__host__ __device__ constexpr int mx_steps(int k) { return (k + kMxStep - 1) / kMxStep; }
__host__ __device__ constexpr int mx_groups(int k) { return (k + kMxGroup - 1) / kMxGroup; }
// Bytes of 16 weight rows of width k, and of one activation row.
__host__ __device__ constexpr int64_t mx_fragment_bytes(int k) {
  return static_cast<int64_t>(mx_steps(k)) * kMxRun + static_cast<int64_t>(mx_groups(k)) * kMxScales;
}
__host__ __device__ constexpr int64_t mx_row_bytes(int k) { return static_cast<int64_t>(mx_groups(k)) * kMxRecord; }

// Scale byte of a block from the largest magnitude's bits (sign cleared: a NaN compares
// above infinity, infinity above every finite value).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  if (amax_bits == 0u) return 127u;
  const int biased = static_cast<int>(amax_bits >> 23) - 2;  // floor(log2) + 127 - 2; a subnormal has field 0
  return static_cast<uint32_t>(biased < 1 ? 1 : biased);
}

// 2^-e of a scale byte (1 .. 254 -> 2^126 .. 2^-127, the last a subnormal made by ldexp).
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) { return ldexpf(1.0f, 127 - static_cast<int>(byte)); }

__device__ __forceinline__ float mx_clamp(float v) { return fminf(fmaxf(v, -6.0f), 6.0f); }

// Eight values times inv -> eight codes (value i in nibble i).
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], float inv) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, mx_clamp(v[0] * inv), mx_clamp(v[1] * inv), 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, mx_clamp(v[2] * inv), mx_clamp(v[3] * inv), 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, mx_clamp(v[4] * inv), mx_clamp(v[5] * inv), 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, mx_clamp(v[6] * inv), mx_clamp(v[7] * inv), 1.0f, 3);
  return r;
}

__device__ __forceinline__ uint32_t mx_abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace moe
