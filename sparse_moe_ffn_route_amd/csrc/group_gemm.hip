// Products grouped by expert with ragged sizes, and both gradients, gfx950 MFMA.
//
//   kForward   out[r] = W_e a_r          out[r][n]  = sum_k a[r][k]    w[e][n][k]
//   kRows      d_a[r] = W_e^T d_out_r    out[r][k]  = sum_n d_out[r][n] w[e][n][k]
//   kWeights   dW_e = sum_r d_out_r a_r^T  out[e][n][k] = sum_{r in e} d_out[r][n] a[r][k]
//
// All three are one loop: an output tile of BM x BN is the sum over the reduction index of an operand P
// (indexed by the tile's rows) times an operand Q (by its columns).  They differ in which index of P and Q
// is contiguous in memory: the reduction's (P and Q of kForward, P of kRows), or the tile's ("across": Q of
// kRows, both of kWeights).  Either way the tile goes from memory straight into LDS as it lies, 16 bytes per
// lane, and only the read from LDS differs: 16 bytes of 8 consecutive reduction indexes, or two transposing
// reads that each hand 16 lanes the four reduction indexes of their own column.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// LDS address of tile columns that a lane reads, typed for the transposing read.
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kOut = 0x80000000u;  // a lane offset past every range: reads zeros, touches no memory

__device__ __forceinline__ __amdgpu_buffer_rsrc_t range_rsrc(const uint8_t* base, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a)));
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32)));
  const int n = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0, n,
                                           0x00020000);
}

// Waits until this wave's reads of LDS have returned and at most N of its loads are under way.
template <int N>
__device__ __forceinline__ void wait_step() {
  static_assert(N >= 0 && N <= 63, "vmcnt is 6 bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// One operand's tile of W tile-index values by a step of RB reduction bytes (along) or RB / ES reduction
// rows (across), in LDS, and how a workgroup of NT threads fills it.  16-byte chunks are stored in an order that
// spreads the rows read together over the banks:
//   along: W rows of RB bytes, chunk c of row r at c ^ swizzle(r), so that the 8 lanes of a read's cycle, 8
//     consecutive rows at one chunk, take 8 different 16-byte slots of the 64 banks' 256 bytes;
//   across: RB / ES rows of W values.  A transposing read's half wave touches 32 bytes of each of the rows 0..3 and
//     8..11 (of 16-bit values; a 32-bit read 64 bytes of the rows 0, 4, 8, 12): the run of 16 values is moved by an
//     exclusive or that tells those rows apart.
template <int EL, bool ACROSS, int W, int RB, int NT>
struct Operand {
  static constexpr int ES = EL == EL_F32 ? 4 : 2;
  static constexpr int kBytes = W * RB;
  static constexpr int kLoads = kBytes / 16 / NT;       // 16-byte loads of a thread and step
  static constexpr int kRow = ACROSS ? W * ES : RB;     // bytes of a row as stored
  static constexpr int kChunks = kRow / 16;
  static constexpr int kStep = RB / ES;                 // reduction indexes of a step
  static_assert(kBytes % (16 * NT) == 0, "a tile splits evenly over the threads");

  static __device__ __forceinline__ int turn(int row) {  // in units of 16 values (across) or 16 bytes
    if constexpr (!ACROSS) {
      return RB == 128 ? row & 7 : (row >> 1) & 3;
    } else if constexpr (EL == EL_F32) {
      return (row >> 2) & 3;
    } else {
      return W >= 128 ? (row & 3) | ((row >> 3) & 1) << 2 : ((row >> 1) & 1) | ((row >> 3) & 1) << 1;
    }
  }

  uint32_t voff[kLoads];
  int kc;  // along: first reduction index of this thread's chunk

  // Which of the tile's rows (as stored) load j of this thread is of, and where in the row in bytes.
  static __device__ __forceinline__ void where(int j, int& row, int& byte) {
    const int p = j * NT + threadIdx.x;
    row = p / kChunks;
    const int c = p % kChunks;
    if constexpr (ACROSS) byte = (((c * 16 / (16 * ES)) ^ turn(row)) * 16 * ES) | (c * 16 % (16 * ES));
    else byte = (c ^ turn(row)) * 16;
  }

  // Fragment of tile columns (or rows) 16 * f .. + 15 and reduction chunk ks: lane (g, i) holds 16 bytes of
  // index 16 * f + i, the reduction values g * (16 / ES) .. of the chunk.
  static __device__ __forceinline__ u32x4 frag(const uint8_t* lds, int f, int ks) {
    const int lane = lane_id(), i = lane & 15, g = lane >> 4;
    if constexpr (!ACROSS) {
      return *reinterpret_cast<const u32x4*>(lds + (f * 16 + i) * RB + (((ks * 4 + g) ^ turn(i)) * 16));
    } else if constexpr (EL == EL_F32) {
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = ks * 16 + g * 4 + j;
        v[j] = *reinterpret_cast<const uint32_t*>(lds + r * kRow + ((f ^ turn(r)) * 64) + i * 4);
      }
      return v;
    } else {
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const int r = ks * 32 + g * 8 + i / 4;
      const uint8_t* at = lds + r * kRow + ((f ^ turn(r)) * 32) + (i & 3) * 8;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)at);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at + 4 * kRow));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// A workgroup's tile.
struct Place {
  int g, begin, end;  // group and its rows
  int row0, col0;     // of the tile: kForward, kRows from the group's first row; kWeights within the matrix
  int part;           // of the reduction
};

// Rows of group g, kept inside [0, rows] and in order whatever the offsets hold.
__device__ __forceinline__ int2 group_rows(const GroupGemm& p, int g) {
  const int b = min(max(p.offsets[g], 0), p.rows);
  return make_int2(b, min(max(p.offsets[g + 1], b), p.rows));
}

// Ragged tile rows: each wave counts the groups' tiles itself (lane l those of groups l * per ..), so that
// no launch has to come before this one.  False past the last tile.
template <int BM>
__device__ __forceinline__ bool find_rows(const GroupGemm& p, int n_tiles, int block, Place& at) {
  constexpr int kPer = 16;  // 1024 groups over 64 lanes
  const int lane = lane_id(), per = (p.n_groups + 63) / 64;
  int cnt[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    cnt[i] = 0;
    if (i < per) {  // wave-uniform
      const int g = lane * per + i;
      const int2 r = group_rows(p, min(g, p.n_groups - 1));
      cnt[i] = g < p.n_groups ? (r.y - r.x + BM - 1) / BM : 0;
      mine += cnt[i];
    }
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(upto, o, kWave);
    if (lane >= o) upto += v;
  }
  const int m_tiles = __builtin_amdgcn_readlane(upto, 63);
  const int total = m_tiles * n_tiles * p.parts;
  if (block >= total) return false;
  int L = xcd_remap(block, total);
  at.part = L % p.parts;
  L /= p.parts;
  const int q = L / n_tiles;  // a group's tiles: columns, then rows, so that q is inside its tile rows
  const int who = __popcll(__ballot(upto <= q));
  int before = who ? __builtin_amdgcn_readlane(upto, who ? who - 1 : 0) : 0;
  int g = 0, m = 0, seen = 0;
  // the lane that holds the group looks through its own
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (q - before >= seen && q - before < seen + cnt[i]) { g = lane * per + i; m = cnt[i]; before += seen; seen = 1 << 30; }
    seen += cnt[i];
  }
  at.g = __builtin_amdgcn_readlane(g, who);
  const int mt = __builtin_amdgcn_readlane(m, who);
  const int first = __builtin_amdgcn_readlane(before, who);
  const int local = L - first * n_tiles;
  const int2 r = group_rows(p, at.g);
  at.begin = __builtin_amdgcn_readfirstlane(r.x);
  at.end = __builtin_amdgcn_readfirstlane(r.y);
  at.row0 = local % mt * BM;
  at.col0 = local / mt;
  return true;
}

template <int EL, int OEL, int DIR, int BM, int BN, int RB, int WM, int WN, int ST, int MINB>
__global__ __launch_bounds__(WM * WN * 64, MINB) void group_gemm_kernel(GroupGemm p) {
  constexpr int NT = WM * WN * 64;
  constexpr int ES = EL == EL_F32 ? 4 : 2;
  constexpr int MF = BM / WM / 16, NF = BN / WN / 16;
  using P = Operand<EL, DIR == kWeights, BM, RB, NT>;
  using Q = Operand<EL, DIR != kForward, BN, RB, NT>;
  constexpr int kStage = P::kBytes + Q::kBytes;
  constexpr int kLoads = P::kLoads + Q::kLoads;
  constexpr int STEP = P::kStep, KS = RB / 64;
  __shared__ __attribute__((aligned(256))) uint8_t lds[ST * kStage];

  const int n_tiles = (p.cols + BN - 1) / BN;
  Place at;
  if constexpr (DIR == kWeights) {
    const int m_tiles = (p.out_rows + BM - 1) / BM;
    int L = xcd_remap(blockIdx.x, gridDim.x);
    at.part = L % p.parts;
    L /= p.parts;
    at.row0 = L % m_tiles * BM;
    at.col0 = L / m_tiles % n_tiles;
    at.g = L / m_tiles / n_tiles;
    const int2 r = group_rows(p, at.g);
    at.begin = __builtin_amdgcn_readfirstlane(r.x);
    at.end = __builtin_amdgcn_readfirstlane(r.y);
  } else {
    if (!find_rows<BM>(p, n_tiles, blockIdx.x, at)) return;
  }
  at.col0 *= BN;
  const int tile_rows = min(BM, (DIR == kWeights ? p.out_rows : at.end - at.begin) - at.row0);
  const int tile_cols = min(BN, p.cols - at.col0);

  // this part of the reduction: r0 .. r1
  const int red = DIR == kWeights ? at.end - at.begin : p.red;
  const int per_part = ((red + STEP - 1) / STEP + p.parts - 1) / p.parts * STEP;
  const int r0 = min(red, at.part * per_part), r1 = min(red, r0 + per_part);
  const int steps = (r1 - r0 + STEP - 1) / STEP;

  // ---- where each thread loads from ------------------------------------------
  const uint8_t* pp = static_cast<const uint8_t*>(p.p);
  const uint8_t* pq = static_cast<const uint8_t*>(p.q);
  const int64_t ldp = static_cast<int64_t>(p.ldp) * ES, ldq = static_cast<int64_t>(p.ldq) * ES;
  P op;
  Q oq;
  int64_t p_bytes = 0, q_bytes = 0;
  if constexpr (DIR != kWeights) {
    // rows of the group, as they lie or through the index
    const bool gather = p.index != nullptr;
    const int first = at.begin + at.row0;
    if (!gather) pp += first * ldp;
    p_bytes = gather ? p.src_rows * ldp : tile_rows * ldp;
    pq += static_cast<int64_t>(at.g) * p.w_stride * ES;
    if constexpr (DIR == kForward) {
      pq += at.col0 * ldq;
      q_bytes = tile_cols * ldq;
    }
#pragma unroll
    for (int j = 0; j < P::kLoads; ++j) {
      int row, byte;
      P::where(j, row, byte);
      op.kc = byte / ES;
      uint32_t src = row;
      if (gather) {
        const int at_row = p.index[first + min(row, tile_rows - 1)];
        src = row < tile_rows && static_cast<uint32_t>(at_row) < static_cast<uint32_t>(p.src_rows) ? at_row : -1;
      }
      op.voff[j] = src < 0x7fffffffu && (gather || row < tile_rows) ? static_cast<uint32_t>(src * ldp) + byte : kOut;
    }
  } else {
#pragma unroll
    for (int j = 0; j < P::kLoads; ++j) {
      int row, byte;
      P::where(j, row, byte);
      op.voff[j] = byte < tile_rows * ES ? static_cast<uint32_t>(row * ldp) + at.row0 * ES + byte : kOut;
    }
  }
#pragma unroll
  for (int j = 0; j < Q::kLoads; ++j) {
    int row, byte;
    Q::where(j, row, byte);
    if constexpr (DIR == kForward) {
      oq.kc = byte / ES;
      oq.voff[j] = row < tile_cols ? static_cast<uint32_t>(row * ldq) + byte : kOut;
    } else {
      oq.voff[j] = byte < tile_cols * ES ? static_cast<uint32_t>(row * ldq) + at.col0 * ES + byte : kOut;
    }
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);

  // Loads of step s into its LDS buffer.  Steps past the last read nothing and write zeros, so that every step is as
  // many loads.
  auto load = [&](int s) {
    uint8_t* buf = lds + s % ST * kStage + wave * 1024;
    const int r = r0 + s * STEP;          // first reduction index of the step
    const int left = max(0, r1 - r);      // reduction indexes left
    if constexpr (DIR != kWeights) {
      const __amdgpu_buffer_rsrc_t rp = range_rsrc(pp, p_bytes);
      const bool in = op.kc < left;
#pragma unroll
      for (int j = 0; j < P::kLoads; ++j)
        buffer_load16_to_lds(rp, buf + j * NT * 16, in ? op.voff[j] : kOut, left ? r * ES : 0);
    } else {
      const __amdgpu_buffer_rsrc_t rp = range_rsrc(pp + (at.begin + r) * ldp, min(left, STEP) * ldp);
#pragma unroll
      for (int j = 0; j < P::kLoads; ++j) buffer_load16_to_lds(rp, buf + j * NT * 16, op.voff[j], 0);
    }
    uint8_t* qbuf = buf + P::kBytes;
    if constexpr (DIR == kForward) {
      const __amdgpu_buffer_rsrc_t rq = range_rsrc(pq, q_bytes);
      const bool in = oq.kc < left;
#pragma unroll
      for (int j = 0; j < Q::kLoads; ++j)
        buffer_load16_to_lds(rq, qbuf + j * NT * 16, in ? oq.voff[j] : kOut, left ? r * ES : 0);
    } else if constexpr (DIR == kRows) {
      const __amdgpu_buffer_rsrc_t rq = range_rsrc(pq + r * ldq, min(left, STEP) * ldq);
#pragma unroll
      for (int j = 0; j < Q::kLoads; ++j) buffer_load16_to_lds(rq, qbuf + j * NT * 16, oq.voff[j], 0);
    } else if (!p.index) {
      const __amdgpu_buffer_rsrc_t rq = range_rsrc(pq + (at.begin + r) * ldq, min(left, STEP) * ldq);
#pragma unroll
      for (int j = 0; j < Q::kLoads; ++j) buffer_load16_to_lds(rq, qbuf + j * NT * 16, oq.voff[j], 0);
    } else {
      // A wave's load is of kPer whole rows (64 lanes, kChunks lanes a row): their indexes are wave-uniform.
      constexpr int kPer = 64 / Q::kChunks > 0 ? 64 / Q::kChunks : 1;
      const __amdgpu_buffer_rsrc_t rq = range_rsrc(pq, p.src_rows * ldq);
#pragma unroll
      for (int j = 0; j < Q::kLoads; ++j) {
        const int row = (j * NT + wave * 64) / Q::kChunks;
        const int mine = lane_id() / Q::kChunks;
        uint32_t src = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int v = left ? ld_scalar(p.index + at.begin + r + min(row + i, left - 1)) : -1;
          const uint32_t u = row + i < left && static_cast<uint32_t>(v) < static_cast<uint32_t>(p.src_rows) ? v : kOut;
          src = mine == i ? u : src;
        }
        // voff holds the row's place within the step, too
        const uint32_t col = oq.voff[j] - static_cast<uint32_t>((row + mine) * ldq);
        buffer_load16_to_lds(rq, qbuf + j * NT * 16,
                             src == kOut || oq.voff[j] == kOut ? kOut : static_cast<uint32_t>(src * ldq) + col, 0);
      }
    }
  };

  // ---- the loop ----------------------------------------------------------------
  const int wm = wave % WM, wn = wave / WM;
  f32x4 acc[MF][NF];
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int n = 0; n < NF; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) load(s);
  for (int s = 0; s < steps; ++s) {
    wait_step<(ST - 2) * kLoads>();
    bare_barrier();  // the step is in LDS, and every wave is done with the buffer that is filled next
    load(s + ST - 1);
    const uint8_t* buf = lds + s % ST * kStage;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      u32x4 fp[MF], fq[NF];
#pragma unroll
      for (int n = 0; n < NF; ++n) fq[n] = Q::frag(buf + P::kBytes, wn * NF + n, ks);
#pragma unroll
      for (int m = 0; m < MF; ++m) fp[m] = P::frag(buf, wm * MF + m, ks);
#pragma unroll
      for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int n = 0; n < NF; ++n) acc[m][n] = mfma_chunk<EL>(fq[n], fp[m], acc[m][n]);
    }
  }
  wait_vmcnt<0>();  // no load writes LDS after the workgroup has ended

  // ---- out: lane (g, i) holds columns g * 4 .. + 3 of row i of each fragment ------
  const int lane = lane_id(), i = lane & 15, g = lane >> 4;
  const int64_t base = DIR == kWeights ? static_cast<int64_t>(at.g) * p.out_rows : at.begin;
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    const int r = (wm * MF + m) * 16 + i;
    if (r >= tile_rows) continue;
    const int64_t row = (base + at.row0 + r) * p.cols + at.col0;
#pragma unroll
    for (int n = 0; n < NF; ++n) {
      const int c = (wn * NF + n) * 16 + g * 4;
      if (c >= tile_cols) continue;
      const f32x4 v = acc[m][n];
      if (p.parts > 1) {
        *reinterpret_cast<f32x4*>(p.partial + at.part * p.part_stride + row + c) = v;
      } else if constexpr (OEL == EL_F32) {
        f32x4 o = v;
        if (p.add) o += *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.add) + row + c);
        *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + row + c) = o;
      } else {
        f32x4 o = v;
        if (p.add) {
          const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.add) + row + c);
          o += f32x4{bf16_bits_to_f32(b.x & 0xFFFFu), __uint_as_float(b.x & 0xFFFF0000u), bf16_bits_to_f32(b.y & 0xFFFFu),
                     __uint_as_float(b.y & 0xFFFF0000u)};
        }
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row + c) =
            make_uint2(bf16x2_bits(o[0], o[1]), bf16x2_bits(o[2], o[3]));
      }
    }
  }
}

// Sum of the parts in order, the added tensor, one rounding.  n4: groups of four values; with n_rows (device) only
// the first *n_rows rows of row4 groups each.
template <int OEL>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ partial, int parts, int64_t part_stride,
                                                   const int32_t* __restrict__ n_rows, int64_t row4, int64_t n4,
                                                   const void* add, void* out) {
  if (n_rows) n4 = min(n4, static_cast<int64_t>(max(*n_rows, 0)) * row4);
  for (int64_t q = blockIdx.x * 256ll + threadIdx.x; q < n4; q += gridDim.x * 256ll) {
    f32x4 v = *reinterpret_cast<const f32x4*>(partial + q * 4);
    for (int s = 1; s < parts; ++s) v += *reinterpret_cast<const f32x4*>(partial + s * part_stride + q * 4);
    if constexpr (OEL == EL_F32) {
      if (add) v += static_cast<const f32x4*>(add)[q];
      static_cast<f32x4*>(out)[q] = v;
    } else {
      if (add) {
        const uint2 b = static_cast<const uint2*>(add)[q];
        v += f32x4{bf16_bits_to_f32(b.x & 0xFFFFu), __uint_as_float(b.x & 0xFFFF0000u), bf16_bits_to_f32(b.y & 0xFFFFu),
                   __uint_as_float(b.y & 0xFFFF0000u)};
      }
      static_cast<uint2*>(out)[q] = make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
    }
  }
}

enum Shape { kFew, kMiddle, kBig };
constexpr int kShapeM[] = {32, 128, 256};
constexpr int kShapeN[] = {128, 128, 256};

template <int EL, int OEL, int DIR>
void launch_shape(Shape shape, const GroupGemm& p, int blocks, hipStream_t s) {
  switch (shape) {
    case kFew:
      if constexpr (DIR != kWeights)
        hipLaunchKernelGGL((group_gemm_kernel<EL, OEL, DIR, 32, 128, 128, 1, 4, 3, 2>), dim3(blocks), dim3(256), 0, s, p);
      break;
    case kMiddle:
      hipLaunchKernelGGL((group_gemm_kernel<EL, OEL, DIR, 128, 128, 128, 2, 2, 2, 2>), dim3(blocks), dim3(256), 0, s, p);
      break;
    case kBig:
      hipLaunchKernelGGL((group_gemm_kernel<EL, OEL, DIR, 256, 256, 128, 2, 4, 2, 1>), dim3(blocks), dim3(512), 0, s, p);
      break;
  }
}

template <int DIR>
void launch_types(int el, int oel, Shape shape, const GroupGemm& p, int blocks, hipStream_t s) {
  if (el == EL_F32) launch_shape<EL_F32, EL_F32, DIR>(shape, p, blocks, s);
  else if (oel == EL_F32) launch_shape<EL_BF16, EL_F32, DIR>(shape, p, blocks, s);
  else launch_shape<EL_BF16, EL_BF16, DIR>(shape, p, blocks, s);
}

struct Plan {
  Shape shape;
  int parts;
  int64_t blocks;
};

// Shape, parts of the reduction and most workgroups of a call.
Plan plan(int dir, const GroupGemm& p, int el) {
  const double avg = static_cast<double>(p.rows) / p.n_groups;
  Plan r{};
  if (dir == kWeights) {
    r.shape = p.out_rows > 128 && p.cols > 128 ? kBig : kMiddle;
  } else {
    r.shape = avg <= 32.0 ? kFew : avg <= 128.0 || p.cols <= 128 ? kMiddle : kBig;
  }
  const int bm = kShapeM[r.shape], bn = kShapeN[r.shape];
  const int64_t nt = (p.cols + bn - 1) / bn;
  const int64_t mt = dir == kWeights ? static_cast<int64_t>(p.n_groups) * ((p.out_rows + bm - 1) / bm)
                                     : (static_cast<int64_t>(p.rows) + static_cast<int64_t>(p.n_groups) * (bm - 1)) / bm;
  r.parts = 1;
  r.blocks = mt * nt * r.parts;
  return r;
}

}  // namespace

size_t group_gemm_workspace(int dir, int el, const GroupGemm& p) {
  const Plan r = plan(dir, p, el);
  const int64_t rows = dir == kWeights ? static_cast<int64_t>(p.n_groups) * p.out_rows : p.rows;
  return r.parts > 1 ? static_cast<size_t>(rows) * p.cols * r.parts * 4 : 0;
}

bool group_gemm_fits(int dir, int el, const GroupGemm& p) {
  return plan(dir, p, el).blocks < (1ll << 32) / 512;  // of threads, which a grid dimension counts
}

hipError_t launch_group_gemm(int dir, int el, int oel, GroupGemm p, void* ws, hipStream_t s) {
  const Plan r = plan(dir, p, el);
  if (r.blocks == 0) return hipSuccess;
  const int64_t rows = dir == kWeights ? static_cast<int64_t>(p.n_groups) * p.out_rows : p.rows;
  p.parts = r.parts;
  p.partial = static_cast<float*>(ws);
  p.part_stride = rows * p.cols;
  const int blocks = static_cast<int>(r.blocks);
  if (dir == kForward) launch_types<kForward>(el, oel, r.shape, p, blocks, s);
  else if (dir == kRows) launch_types<kRows>(el, oel, r.shape, p, blocks, s);
  else launch_types<kWeights>(el, oel, r.shape, p, blocks, s);
  if (r.parts > 1) {
    const int64_t n4 = rows * p.cols / 4;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((n4 + 255) / 256, 4096)));
    const int32_t* n_rows = dir == kWeights ? nullptr : p.offsets + p.n_groups;
    if (oel == EL_F32)
      hipLaunchKernelGGL(join_kernel<EL_F32>, grid, dim3(256), 0, s, p.partial, r.parts, p.part_stride, n_rows, p.cols / 4,
                         n4, p.add, p.out);
    else
      hipLaunchKernelGGL(join_kernel<EL_BF16>, grid, dim3(256), 0, s, p.partial, r.parts, p.part_stride, n_rows,
                         p.cols / 4, n4, p.add, p.out);
  }
  return hipGetLastError();
}

}  // namespace moe
