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
// reads that each hand 16 lanes the four reduction indexes of their own column.  The exclusive-or orders below leave the
// larger tiles no bank conflicts (counted) in either.
//
// What bounds them.  10 rows of each of 64 groups, 1024 x 4096: the matrices' 537 MB, read in 86 us (6.3 TB/s; a read
// of memory alone reaches 6.6).  512 rows a group: 275 GFLOP and 0.9 to 2.5 GB, in 320 us (kForward), 355 (kRows,
// with a tensor added), 508 (kWeights, fp32 sums added to sums: 2.5 GB at 4.9 TB/s).  One 4096^3 product: products
// alone 77 us, loads alone 51 to 71, LDS reads 30; they hide behind each other only in part: 102, 105, 112 us (1.35,
// 1.31, 1.23 PFLOP/s).
//   - Two halves of a workgroup's waves in turn (TURNS), one reads LDS and asks for loads while the other multiplies:
//     102 us against 118 to 128 with all waves in step.
//   - A ring of five steps of 64 bytes against two of 128 (one group of 32768 rows, 1024 x 4096, matrices from
//     memory): 235 against 258 us.  kWeights keeps two of 128: its rows are whole lines either way.
//   - Smaller tiles at two or three workgroups a CU fill each other's gaps instead and cover each other's stores,
//     with more to load a product; waves that multiply go first (512 rows a group: kRows in kWide 375 -> 365 us,
//     kForward in kWide 355 -> 344, in kFew 830 -> 773).  kWeights loses by that (506 -> 520) and has it only where a
//     workgroup's halves take turns (kBig).
//   - A reduction that is long for the tiles there are is split into parts (16 x 4096 x 4096 kForward 22 -> 12.5 us,
//     8192 rows into 512 x 512 49 -> 18), summed in order by a second launch: no atomics, the same bits every time.
//   - A matrix that one tile row reads bypasses the caches' replacement (10 rows a group: 104 -> 86 us), as do
//     kWeights' results (631 -> 606 us in kBig, with what they add to).
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

using namespace groups;  // group_plan.hpp

namespace {

// What a lane has of a transposing read: four values of 16 bits.
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kOut = 0x80000000u;  // a lane offset past every range: reads zeros, touches no memory

// Buffer resource of `bytes` bytes from base on, both the same for the whole wave.
__device__ __forceinline__ u32x4 range_rsrc(const uint8_t* base, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a))),
               static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32))) & 0xFFFFu,
               static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(bytes))), 0x00020000u};
}

// Waits until this wave's reads of LDS have returned and at most N of its loads are under way.
template <int N>
__device__ __forceinline__ void wait_step() {
  static_assert(N >= 0 && N <= 63, "vmcnt is 6 bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// buffer_load16_to_lds with the LDS address as a number, as an instruction that the compiler does not count: told of it,
// the compiler waits for all such loads before every transposing read, which it cannot tell apart from them, and
// with that for the step that was only just asked for.  The kernel waits for its steps itself.  The first wait is
// for the scalars' writers, the second for m0's; no other instruction of the kernels here takes m0.
template <bool NT = false>
__device__ __forceinline__ void load16_to_lds(const u32x4& r, uint32_t lds_at, uint32_t voff, uint32_t soff) {
  auto scalar = [](uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(v)); };
  const uint32_t lds = scalar(lds_at), s = scalar(soff);
  const u32x4 rs{scalar(r[0]), scalar(r[1]), scalar(r[2]), scalar(r[3])};
  if constexpr (NT)
    asm volatile("s_nop 4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                 :: "s"(lds), "v"(voff), "s"(rs), "s"(s) : "memory");
  else
    asm volatile("s_nop 4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(lds), "v"(voff), "s"(rs), "s"(s) : "memory");
}

// One operand's tile of W tile-index values by a step of RB reduction bytes (along) or RB / ES reduction
// rows (across), in LDS, and how a workgroup of NT threads fills it.  16-byte chunks are stored in an order that
// spreads the rows read together over the banks:
//   along: W rows of RB bytes, chunk c of row r at c ^ turn(r), so that the lanes of a read's cycle, consecutive rows at
//     one chunk, take different 16-byte slots of the 64 banks' 256 bytes (of 256-byte rows two lanes share a slot: kFew
//     waits for memory, and is no faster with all sixteen apart);
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
      return RB >= 128 ? row & 7 : (row >> 1) & 3;
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

  // Where in the stored tile this lane's part of a fragment lies.  Fragment f is tile indexes 16 * f .. + 15, reduction
  // chunk ks 64 bytes of each: lane (g, i) holds 16 bytes of index 16 * f + i, the reduction values
  // g * (16 / ES) .. of the chunk.  The part of the place that the swizzle mixes with f (across) or ks (along) is in
  // `at`; the rest is a constant that the read's instruction adds.  A wave has the fragments first, first + BY, ...
  template <int BY, int N>
  static __device__ __forceinline__ void places(int first, uint32_t (&at)[N]) {
    const int lane = lane_id(), i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int x = 0; x < N; ++x) {
      if constexpr (!ACROSS) at[x] = (first * 16 + i) * RB + (((x * 4 + g) ^ turn(i)) * 16);
      else if constexpr (EL == EL_F32) at[x] = g * 4 * kRow + (((first + x * BY) ^ turn(g * 4)) * 64) + i * 4;
      else at[x] = (g * 8 + i / 4) * kRow + (((first + x * BY) ^ turn(g * 8 + i / 4)) * 32) + (i & 3) * 8;
    }
  }
  template <int BY, int N>
  static __device__ __forceinline__ u32x4 frag(const uint8_t* lds, const uint32_t (&at)[N], int f, int ks) {
    if constexpr (!ACROSS) {
      return *reinterpret_cast<const u32x4*>(lds + at[ks] + f * BY * 16 * RB);
    } else if constexpr (EL == EL_F32) {
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(lds + at[f] + (ks * 16 + j) * kRow);
      return v;
    } else {
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const uint8_t* p = lds + at[f] + ks * 32 * kRow;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * kRow));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// A workgroup's tile.
struct Place {
  int g, begin, end;  // group and its rows
  int row0, col0;     // of the tile: kForward, kRows from the group's first row; kWeights within the matrix
  int part;           // of the reduction
  int high;           // most rows of the tile
  bool once;          // no other tile reads this one's matrix columns: they bypass the caches' replacement
};

// Rows of group g, kept inside [0, rows] and in order whatever the offsets hold.
__device__ __forceinline__ int2 group_rows(const GroupGemm& p, int g) {
  const int b = min(max(p.offsets[g], 0), p.rows);
  return make_int2(b, min(max(p.offsets[g + 1], b), p.rows));
}

// Tile row and column of tile i of a group: columns of 8 tile rows at a time, so that the tiles that an XCD has at
// work together share both operands in its L2.
__device__ __forceinline__ void tile_at(int i, int m_tiles, int n_tiles, int& row, int& col) {
  const int block = i / (8 * n_tiles), high = min(8, m_tiles - block * 8), in = i - block * 8 * n_tiles;
  row = block * 8 + in % high;
  col = in / high;
}

// Ragged tile rows: each wave counts the groups' tiles itself (lane l those of groups l * per ..), so that
// no launch has to come before this one.  False past the last tile.
__device__ __forceinline__ bool find_rows(const GroupGemm& p, int n_tiles, int block, Place& at) {
  const int lane = lane_id(), per = (p.n_groups + 63) / 64;
  auto tiles_of = [&](int2 r) { return (r.y - r.x + p.high - 1) / p.high; };
  int2 r = make_int2(0, 0);  // of the lane's first group
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int g = lane * per + i;
    const int2 v = group_rows(p, min(g, p.n_groups - 1));
    if (i == 0) r = v;
    if (g < p.n_groups) mine += tiles_of(v);
    mine = min(mine, kMaxTileRows);  // more than any call has: offsets that overlap must not overflow
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(upto, o, kWave);
    if (lane >= o) upto += v;
  }
  const int64_t all = static_cast<int64_t>(__builtin_amdgcn_readlane(upto, 63)) * n_tiles * p.parts;
  const int total = static_cast<int>(min<int64_t>(all, 0x7fffffff));
  if (block >= total) return false;
  int L = xcd_remap(block, total);
  at.part = L % p.parts;
  L /= p.parts;
  const int q = L / n_tiles;  // a group's tiles follow each other, so that q is inside its tile rows
  const int who = __popcll(__ballot(upto <= q));
  int before = __builtin_amdgcn_readlane(upto - mine, who), mt = __builtin_amdgcn_readlane(mine, who);
  at.g = who * per;
  at.begin = __builtin_amdgcn_readlane(r.x, who);
  at.end = __builtin_amdgcn_readlane(r.y, who);
  if (per > 1) {  // the lane's groups in turn, by the whole wave
    mt = tiles_of(make_int2(at.begin, at.end));
    while (q >= before + mt && at.g + 1 < p.n_groups) {
      before += mt;
      const int2 v = group_rows(p, ++at.g);
      at.begin = __builtin_amdgcn_readfirstlane(v.x);
      at.end = __builtin_amdgcn_readfirstlane(v.y);
      mt = tiles_of(make_int2(at.begin, at.end));
    }
  }
  at.once = mt == 1;
  tile_at(L - before * n_tiles, mt, n_tiles, at.row0, at.col0);
  // a group's tiles share its rows evenly, in steps of a fragment
  at.high = ((at.end - at.begin + mt - 1) / mt + 15) / 16 * 16;
  at.row0 *= at.high;
  return true;
}

template <int EL, int OEL, int DIR, int BM, int BN, int RB, int WM, int WN, int ST, int MINB, bool TURNS>
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
    int L = xcd_remap(p.first + blockIdx.x, p.blocks);
    at.part = L % p.parts;
    L /= p.parts;
    at.g = L / (m_tiles * n_tiles);
    tile_at(L - at.g * m_tiles * n_tiles, m_tiles, n_tiles, at.row0, at.col0);
    at.row0 *= BM;
    at.high = BM;
    const int2 r = group_rows(p, at.g);
    at.begin = __builtin_amdgcn_readfirstlane(r.x);
    at.end = __builtin_amdgcn_readfirstlane(r.y);
  } else {
    if (!find_rows(p, n_tiles, p.first + blockIdx.x, at)) return;
  }
  at.col0 *= BN;
  const int tile_rows = min(at.high, (DIR == kWeights ? p.out_rows : at.end - at.begin) - at.row0);
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
  const u32x4 whole_p = range_rsrc(pp, p_bytes), whole_q = range_rsrc(pq, DIR == kWeights ? p.src_rows * ldq : q_bytes);

  // Loads of step s into an LDS buffer.  Steps past the last read nothing and write zeros, so that every
  // step is as many loads.
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
  struct Step {
    u32x4 rp, rq;
    uint32_t buf, soff;
    int r, left;  // first reduction index of the step, indexes from there on
  };
  auto step_at = [&](int s, uint32_t buf) {
    Step t;
    t.buf = buf + lds0 + wave * 1024;
    t.r = r0 + s * STEP;
    t.left = r1 > t.r ? r1 - t.r : 0;
    t.soff = t.left ? t.r * ES : 0;
    auto bytes = [&](int64_t ld) { return t.left >= STEP ? STEP * ld : t.left * ld; };
    t.rp = DIR == kWeights ? range_rsrc(pp + (at.begin + t.r) * ldp, bytes(ldp)) : whole_p;
    t.rq = DIR == kForward || (DIR == kWeights && p.index) ? whole_q
           : range_rsrc(pq + (DIR == kWeights ? at.begin + t.r : t.r) * ldq, bytes(ldq));
    return t;
  };
  // kWeights with an index: a wave's load of Q is of kPer whole rows (64 lanes, kChunks lanes a row), whose sources are
  // the same for the whole wave; they are asked for a step ahead.
  constexpr int kPer = 64 / Q::kChunks > 0 ? 64 / Q::kChunks : 1;
  uint32_t row_at[Q::kLoads * kPer];
  auto rows_ahead = [&](int s) {
    const int r = r0 + s * STEP, left = r1 > r ? r1 - r : 0;
#pragma unroll
    for (int x = 0; x < Q::kLoads * kPer; ++x) {
      const int row = (x / kPer * NT + wave * 64) / Q::kChunks + x % kPer;
      const int v = left ? ld_scalar(p.index + at.begin + r + min(row, left - 1)) : -1;
      row_at[x] = row < left && static_cast<uint32_t>(v) < static_cast<uint32_t>(p.src_rows) ? v : kOut;
    }
  };
  if (DIR == kWeights && p.index) rows_ahead(0);
  auto load_one = [&](const Step& t, int j) {
    if (j < P::kLoads) {
      const uint32_t to = t.buf + j * NT * 16;
      if constexpr (DIR != kWeights) load16_to_lds(t.rp, to, op.kc < t.left ? op.voff[j] : kOut, t.soff);
      else load16_to_lds(t.rp, to, op.voff[j], 0);
      return;
    }
    j -= P::kLoads;
    const uint32_t to = t.buf + P::kBytes + j * NT * 16;
    if constexpr (DIR == kForward) {
      if (RB >= 128 && at.once) load16_to_lds<true>(t.rq, to, oq.kc < t.left ? oq.voff[j] : kOut, t.soff);
      else load16_to_lds(t.rq, to, oq.kc < t.left ? oq.voff[j] : kOut, t.soff);
    } else {
      uint32_t voff = oq.voff[j];
      if (DIR == kWeights && p.index) {
        const int mine = lane_id() / Q::kChunks;
        uint32_t src = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) src = mine == i ? row_at[j * kPer + i] : src;
        // voff holds the row's place within the step, too
        const uint32_t col = voff - static_cast<uint32_t>(((j * NT + wave * 64) / Q::kChunks + mine) * ldq);
        voff = src == kOut || voff == kOut ? kOut : static_cast<uint32_t>(src * ldq) + col;
      }
      if (DIR == kRows && at.once) load16_to_lds<true>(t.rq, to, voff, 0);
      else load16_to_lds(t.rq, to, voff, 0);
    }
  };
  auto load = [&](int s, uint32_t buf) {
    const Step t = step_at(s, buf);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load_one(t, j);
    if (DIR == kWeights && p.index) rows_ahead(s + 1);
  };

  // ---- the loop ----------------------------------------------------------------
  const int wm = wave % WM, wn = wave / WM;
  constexpr int PP = DIR == kWeights ? MF : KS, QP = DIR != kForward ? NF : KS;
  uint32_t p_at[PP], q_at[QP];
  P::template places<WM>(wm, p_at);
  Q::template places<1>(wn * NF, q_at);
  // Row fragments are dealt to the waves in turn, and those behind the tile's last row are left out: every wave has its
  // share of a tile that is not full.
  const int live = (tile_rows + 15) / 16 > wm ? ((tile_rows + 15) / 16 - wm + WM - 1) / WM : 0;
  f32x4 acc[MF][NF];
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int n = 0; n < NF; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) load(s, s * kStage);
  uint32_t now = 0, next = (ST - 1) * kStage;  // buffers of this step, and of the one asked for beside it
  u32x4 fp[MF], fq[NF];
  auto read = [&](int ks) {
    const uint8_t* buf = lds + now;
#pragma unroll
    for (int n = 0; n < NF; ++n) fq[n] = Q::template frag<1>(buf + P::kBytes, q_at, n, ks);
#pragma unroll
    for (int m = 0; m < MF; ++m) fp[m] = P::template frag<WM>(buf, p_at, m, ks);
  };
  auto multiply = [&] {
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      if (DIR != kWeights && m >= live) break;
#pragma unroll
      for (int n = 0; n < NF; ++n) acc[m][n] = mfma_chunk<EL>(fq[n], fp[m], acc[m][n]);
    }
  };
  auto turn_buffers = [&] {
    next = now;
    now = now == (ST - 1) * kStage ? 0 : now + kStage;
  };
  if constexpr (TURNS) {
    const bool second = wave >= WM * WN / 2;
    wait_step<(ST - 2) * kLoads>();
    bare_barrier();
    if (second) bare_barrier();
    for (int s = 0; s < steps; ++s) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        read(ks);
        if (ks == 0) load(s + ST - 1, next);
        if (ks == KS - 1 && second) wait_step<(ST - 2) * kLoads>();
        else wait_step<63>();
        bare_barrier();
        __builtin_amdgcn_s_setprio(1);
        multiply();
        __builtin_amdgcn_s_setprio(0);
        if (ks == KS - 1 && !second) wait_step<(ST - 2) * kLoads>();
        bare_barrier();
      }
      turn_buffers();
    }
    if (!second) bare_barrier();
  } else {
    for (int s = 0; s < steps; ++s) {
      wait_step<(ST - 2) * kLoads>();
      bare_barrier();  // the step is in LDS, and every wave is done with the buffer that is filled next
      load(s + ST - 1, next);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        read(ks);
        if (DIR != kWeights) __builtin_amdgcn_s_setprio(1);
        multiply();
        if (DIR != kWeights) __builtin_amdgcn_s_setprio(0);
      }
      turn_buffers();
    }
  }
  wait_step<0>();   // no load writes LDS any more
  bare_barrier();

  // ---- out -----------------------------------------------------------------------
  // A lane has four columns of a row in each fragment.  Each wave turns its rows around in a part of LDS of its own, a
  // few at a time, so that whole lines are added to and written: 16 bytes a lane, consecutive lanes along the row.
  constexpr int WC = NF * 16;                            // columns of a wave
  constexpr int kTurnRow = WC * 4 + 16;                  // bytes of a turned row
  constexpr int kTurnMax = ST * kStage / (WM * WN) / (16 * kTurnRow);
  constexpr int TF = kTurnMax >= MF ? MF : kTurnMax >= 4 && MF % 4 == 0 ? 4 : kTurnMax >= 2 && MF % 2 == 0 ? 2 : 1;
  static_assert(kTurnMax >= 1, "a fragment's rows fit the wave's part of LDS");
  uint8_t* turn = lds + wave * (TF * 16 * kTurnRow);
  const int lane = lane_id(), i = lane & 15, g = lane >> 4;
  const int64_t base = DIR == kWeights ? static_cast<int64_t>(at.g) * p.out_rows : at.begin;
  const bool whole = p.parts == 1;
  // Values of a 16-byte piece: of the result, or of a part of the sum in fp32.
  auto rows_out = [&](auto width) {
    constexpr int V = decltype(width)::value, kLanes = WC / V, kRows = 64 / kLanes, kPieces = TF * 16 / kRows;
    const int c = lane % kLanes * V, col = wn * WC + c;
    const bool here = col < tile_cols;
    auto row_of = [&](int m0, int x) {
      const int r = x * kRows + lane / kLanes;
      return ((m0 + r / 16) * WM + wm) * 16 + r % 16;
    };
    auto place = [&](int row) { return (base + at.row0 + row) * p.cols + at.col0 + col; };
    // what is added is asked for one pass ahead
    u32x4 more[2][kPieces];
    const bool adds = whole && p.add;
    auto fetch = [&](int m0, u32x4 (&to)[kPieces]) {
      if (!adds) return;
#pragma unroll
      for (int x = 0; x < kPieces; ++x) {
        const int row = row_of(m0, x);
        const auto* from = static_cast<const uint8_t*>(p.add) + place(row) * (16 / V);
        to[x] = here && row < tile_rows ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from)) : u32x4{};
      }
    };
    fetch(0, more[0]);
#pragma unroll
    for (int m0 = 0; m0 < MF; m0 += TF) {
#pragma unroll
      for (int m = 0; m < TF; ++m)
#pragma unroll
        for (int n = 0; n < NF; ++n)
          *reinterpret_cast<f32x4*>(turn + (m * 16 + i) * kTurnRow + (n * 16 + g * 4) * 4) = acc[m0 + m][n];
      if (m0 + TF < MF) fetch(m0 + TF, more[(m0 / TF + 1) % 2]);
      asm volatile("" ::: "memory");  // the wave's other lanes read what this one wrote: LDS keeps a wave's order
#pragma unroll
      for (int x = 0; x < kPieces; ++x) {
        const int row = row_of(m0, x);
        if (!here || row >= tile_rows) continue;
        const u32x4 b = more[m0 / TF % 2][x];
        const f32x4* from = reinterpret_cast<const f32x4*>(turn + (x * kRows + lane / kLanes) * kTurnRow + c * 4);
        if constexpr (V == 4) {
          f32x4 v = from[0];
          if (adds) v += __builtin_bit_cast(f32x4, b);
          float* out = whole ? static_cast<float*>(p.out) : p.partial + at.part * p.part_stride;
          f32x4* to = reinterpret_cast<f32x4*>(out + place(row));
          if (DIR == kWeights) __builtin_nontemporal_store(v, to);
          else *to = v;
        } else {
          f32x4 v[2] = {from[0], from[1]};
          if (adds) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              v[q / 4][q % 4] += q % 2 ? __uint_as_float(b[q / 2] & 0xFFFF0000u) : bf16_bits_to_f32(b[q / 2] & 0xFFFFu);
          }
          const u32x4 o{bf16x2_bits(v[0][0], v[0][1]), bf16x2_bits(v[0][2], v[0][3]), bf16x2_bits(v[1][0], v[1][1]),
                    bf16x2_bits(v[1][2], v[1][3])};
          u32x4* to = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + place(row));
          if (DIR == kWeights) __builtin_nontemporal_store(o, to);
          else *to = o;
        }
      }
      asm volatile("" ::: "memory");
    }
  };
  if (OEL == EL_F32 || !whole) rows_out(std::integral_constant<int, 4>{});
  else rows_out(std::integral_constant<int, 8>{});
}

// Sum of the parts in order, the added tensor, one rounding.  n4: fours of values, row4 a row's; with offsets (device)
// only the rows from the first group's first to the last one's last.
template <int OEL>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ partial, int parts, int64_t part_stride,
                                                   const int32_t* __restrict__ offsets, int n_groups, int64_t row4,
                                                   int64_t n4, const void* add, void* out) {
  int64_t q0 = 0;
  if (offsets) {
    q0 = max(offsets[0], 0) * row4;
    n4 = min(n4, max(offsets[n_groups], 0) * row4);
  }
  for (int64_t q = q0 + blockIdx.x * 256ll + threadIdx.x; q < n4; q += gridDim.x * 256ll) {
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

// Workgroups of a launch: a grid dimension holds less than 2^32 threads, and larger calls are several launches.
constexpr int kMaxLaunch = 1 << 22;

template <int EL, int OEL, int DIR, int BM, int BN, int RB, int WM, int WN, int ST, int MINB, bool TURNS>
void launch(GroupGemm p, hipStream_t s) {
  for (p.first = 0; p.first < p.blocks; p.first += kMaxLaunch)
    hipLaunchKernelGGL((group_gemm_kernel<EL, OEL, DIR, BM, BN, RB, WM, WN, ST, MINB, TURNS>),
                       dim3(std::min(kMaxLaunch, p.blocks - p.first)), dim3(WM * WN * 64), 0, s, p);
}

template <int EL, int OEL, int DIR>
void launch_shape(int shape, const GroupGemm& p, hipStream_t s) {
  if (shape == kSmall) return launch<EL, OEL, DIR, 64, 64, 128, 2, 2, 3, 3, false>(p, s);
  if (shape == kNarrow) return launch<EL, OEL, DIR, 64, 128, 128, 2, 2, 3, 2, false>(p, s);
  if constexpr (EL == EL_BF16) {
    if constexpr (DIR != kWeights)
      if (shape == kFew) return launch<EL, OEL, DIR, 32, 64, 256, 1, 4, 3, 2, false>(p, s);
    if (shape == kMiddle) return launch<EL, OEL, DIR, 128, 128, 128, 2, 2, 2, 2, false>(p, s);
    if (shape == kWide) return launch<EL, OEL, DIR, 128, 256, 64, 2, 4, 3, 2, false>(p, s);
    if (DIR == kWeights) return launch<EL, OEL, DIR, 256, 256, 128, 2, 4, 2, 1, true>(p, s);
    return launch<EL, OEL, DIR, 256, 256, 64, 2, 4, 5, 1, true>(p, s);
  }
}

template <int DIR>
void launch_types(int el, int oel, int shape, const GroupGemm& p, hipStream_t s) {
  if (el == EL_F32) launch_shape<EL_F32, EL_F32, DIR>(shape, p, s);
  else if (oel == EL_F32) launch_shape<EL_BF16, EL_F32, DIR>(shape, p, s);
  else launch_shape<EL_BF16, EL_BF16, DIR>(shape, p, s);
}

Plan plan_of(int dir, int el, int oel, const GroupGemm& p) {
  return plan(dir, GroupSizes{p.n_groups, p.rows, p.w_stride, p.cols, p.red, p.out_rows}, el == EL_F32, oel == EL_F32);
}

}  // namespace

size_t group_gemm_workspace(int dir, int el, int oel, const GroupGemm& p) {
  const Plan r = plan_of(dir, el, oel, p);
  const int64_t rows = dir == kWeights ? static_cast<int64_t>(p.n_groups) * p.out_rows : p.rows;
  return r.parts > 1 ? static_cast<size_t>(rows) * p.cols * r.parts * 4 : 0;
}

hipError_t launch_group_gemm(int dir, int el, int oel, GroupGemm p, void* ws, hipStream_t s) {
  const Plan r = plan_of(dir, el, oel, p);
  if (r.blocks == 0) return hipSuccess;
  const int64_t rows = dir == kWeights ? static_cast<int64_t>(p.n_groups) * p.out_rows : p.rows;
  p.parts = r.parts;
  p.high = r.high;
  p.partial = static_cast<float*>(ws);
  p.part_stride = rows * p.cols;
  p.blocks = static_cast<int>(r.blocks);
  if (dir == kForward) launch_types<kForward>(el, oel, r.shape, p, s);
  else if (dir == kRows) launch_types<kRows>(el, oel, r.shape, p, s);
  else launch_types<kWeights>(el, oel, r.shape, p, s);
  if (r.parts > 1) {
    const int64_t n4 = rows * p.cols / 4;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((n4 + 255) / 256, 4096)));
    const int32_t* ragged = dir == kWeights ? nullptr : p.offsets;
    if (oel == EL_F32)
      hipLaunchKernelGGL(join_kernel<EL_F32>, grid, dim3(256), 0, s, p.partial, r.parts, p.part_stride, ragged,
                         p.n_groups, p.cols / 4, n4, p.add, p.out);
    else
      hipLaunchKernelGGL(join_kernel<EL_BF16>, grid, dim3(256), 0, s, p.partial, r.parts, p.part_stride, ragged,
                         p.n_groups, p.cols / 4, n4, p.add, p.out);
  }
  return hipGetLastError();
}

}  // namespace moe
