// The grouped 16-bit product on the matrix cores: BM x BN output tiles, the
// contraction in steps of 64 through LDS.  Needs operands whose rows start on
// 16-byte addresses (the plan's rule); any row count, and with LOOSE results of
// any row length and alignment.
//
// Bound by the matrix cores where the contraction is long.  256 x 256 tiles,
// eight waves of 128 x 64 (128 accumulator registers, two waves a SIMD, two
// 64 KB buffers): of the wave shapes that fit, the one whose LDS reads (192 KB
// a step at 128 bytes a cycle) stay under its products (2048 cycles); four
// waves of 128 x 128 would read a third less but the compiler then copies
// accumulators around.  8192 x 14336 x 4096 bf16: forward 710 us, dx 752, dw
// 780 (1355, 1280, 1235 TFLOP/s; the library's products timed in turn on the same
// card 612, 693 and 956 us).  128 x 128 tiles, four waves of 64 x 64,
// two blocks a compute unit, where 256 x 256 tiles would not fill the chip.
//
// Operands go from memory straight into LDS, 16 bytes a lane, through buffer
// resources that end where the operand does: what lies past a row range, a
// column range or the contraction arrives as zeros.  Two LDS buffers: a step
// computes on one while the next step's data arrives in the other.
//
// deep operand: LDS [row][64], 16-byte piece c of row r at place c ^ (r mod 8).
//   A fragment (16 rows, 8 contraction values a lane) is one 16-byte LDS read;
//   the places spread 8 rows over all banks.
// wide operand: LDS [64][cols] as in memory, 32-byte granule g of contraction
//   row k at place g ^ f(k).  A fragment is two transposing reads
//   (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 values, lane i gets column
//   i); f gives the rows of one read different banks.
#pragma once

#include <type_traits>

#include "linear.hpp"

namespace milo {

constexpr int kDepth = kLinearStep;        // contraction values per step
constexpr int kTileRsrcWord3 = 0x00020000; // raw buffer, bounds checked in bytes
constexpr int kOutside = 0x70000000;       // an offset no operand reaches, with room for a tile's offsets after it

typedef __attribute__((address_space(3))) void lds_void;

// ROWS rows (deep) or columns (wide) of one operand, staged by NW waves.
template <bool WIDE, int ROWS, int NW>
struct Operand {
  static constexpr int kLoads = ROWS * kDepth * 2 / (16 * 64 * NW);   // per lane and step
  static constexpr int kBytes = ROWS * kDepth * 2;
  int voff[kLoads];      // byte offset of each piece from the step's first element
  int piece[kLoads];     // deep: contraction index of the piece within the step

  static __device__ __forceinline__ int wide_swizzle(int k) {
    return ((k & 3) | (((k >> 3) & 3) << 2)) & (ROWS / 16 - 1);
  }

  // ld: elements between rows; cols_left: wide, columns from the tile's first to the operand's end
  __device__ __forceinline__ void init(int lane, int wave, int ld, int cols_left) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int slot = (j * NW + wave) * 64 + lane;
      if constexpr (!WIDE) {
        const int r = slot >> 3, c = (slot & 7) ^ (r & 7);
        voff[j] = r * ld * 2 + c * 16;
        piece[j] = c * 8;
      } else {
        const int k = slot / (ROWS / 8), p = slot % (ROWS / 8);
        const int c = (((p >> 1) ^ wide_swizzle(k)) << 1) | (p & 1);
        voff[j] = c * 8 < cols_left ? k * ld * 2 + c * 16 : kOutside;
        piece[j] = 0;
      }
    }
  }

  // Step k0 into LDS at dst; nothing (zeros, no traffic) unless `on`.  deep:
  // src is the tile's first row, `left` its rows inside the operand; wide: src
  // is the tile's first column of the first contraction row, `depth` the
  // contraction's length.  No branch: the loads are spread between products.
  __device__ __forceinline__ void load(const uint16_t* src, int64_t ld, int left, int depth, int k0, bool on,
                                       char* dst, int wave) const {
    if constexpr (!WIDE) {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(src + k0), 0, on ? (int)(left * ld - k0) * 2 : 0, kTileRsrcWord3);
      const bool whole = k0 + kDepth <= depth;
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + (j * NW + wave) * 1024), 16,
                                                 whole || k0 + piece[j] < depth ? voff[j] : kOutside, 0, 0, 0);
    } else {
      const int rows = depth - k0 < kDepth ? depth - k0 : kDepth;
      // `left` columns remain in the last row: the resource ends with the operand's last element
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(src + k0 * ld), 0, on ? (int)((rows - 1) * ld + left) * 2 : 0, kTileRsrcWord3);
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + (j * NW + wave) * 1024), 16, voff[j], 0, 0, 0);
    }
  }
};

// A transposing LDS read.  `restrict` tells the compiler that no load into LDS
// in flight writes what is read (the barriers see to that); without it every
// such read waits for all of them.
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
__device__ __forceinline__ s16x4 read_transposed(const lds_s16x4* __restrict__ p) {
#ifdef __HIP_DEVICE_COMPILE__
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
#else
  return s16x4{};
#endif
}

// Fragments of NF 16-wide groups starting at row (column) w0 of an LDS tile.
template <bool WIDE, int ROWS, int NF>
struct Fragments {
  int off[WIDE ? NF : 2];
  __device__ __forceinline__ void init(int lane, int w0) {
    if constexpr (!WIDE) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        off[s] = (w0 + (lane & 15)) * kDepth * 2 + (((4 * s + (lane >> 4)) ^ (lane & 7)) << 4);
    } else {
      const int i = lane & 15, k = 8 * (lane >> 4) + (i >> 2);
      const int f = ((k & 3) | (((k >> 3) & 3) << 2)) & (ROWS / 16 - 1);
#pragma unroll
      for (int t = 0; t < NF; ++t) off[t] = k * ROWS * 2 + (((w0 >> 4) + t) ^ f) * 32 + (i & 3) * 8;
    }
  }
  // group t of the step's half s (32 contraction values)
  __device__ __forceinline__ s16x8 read(const char* lds, int s, int t) const {
    if constexpr (!WIDE) {
      return *(const s16x8*)(lds + off[s] + t * 16 * kDepth * 2);
    } else {
      const char* p = lds + off[t] + s * 32 * ROWS * 2;
      const s16x4 lo = read_transposed((const lds_s16x4*)p), hi = read_transposed((const lds_s16x4*)(p + 4 * ROWS * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Block -> tile.  Blocks go to the 8 XCDs in turn; each XCD gets a run of
// consecutive full tiles, so that tiles sharing operands share its L2, and then
// a run of the short tiles (a row tile with at most half of its rows), which
// fill the last round: among the full ones they unbalanced it (8192 ragged rows
// over 8 experts x 14336 x 4096: 1033 us mixed, 985 apart).
struct TileIndex {
  int at;        // -1: none left
  bool short_;
};
__device__ __forceinline__ TileIndex xcd_order(int id, int full, int shorts) {
  const int x = id & 7;
  int i = id >> 3;
  const int nf = (full >> 3) + (x < (full & 7) ? 1 : 0), ns = (shorts >> 3) + (x < (shorts & 7) ? 1 : 0);
  const int step = gridDim.x >> 3, l = i % step, j = i / step;
  // Every other block starts with its last tile, often a short one: their
  // results' traffic then falls between the others', not all at once (SiLU,
  // gate operand and kept pre-activation on those rows: 985 us, 964 so).
  if ((l & 1) && i < nf + ns) {
    const int c = (nf + ns - l + step - 1) / step;
    i = l + (j == 0 ? c - 1 : j - 1) * step;
  }
  if (i < nf) return {x * (full >> 3) + min(x, full & 7) + i, false};
  i -= nf;
  if (i < ns) return {x * (shorts >> 3) + min(x, shorts & 7) + i, true};
  return {-1, false};
}

// dw: an expert's tiles cost as its rows do, so every XCD gets an eighth of
// each expert's tiles (`each` of them: experts in turn, the eighths rotating),
// not a run over experts.  Positions past an expert's last tile are skipped.
// Moves id to the tile it returns.
__device__ __forceinline__ TileIndex spread_order(int& id, int stride, int E, int full, int shorts) {
  const int ef = (full + 7) >> 3, es = (shorts + 7) >> 3;
  for (;; id += stride) {
    const int x = id & 7;
    int i = id >> 3;
    const bool s = i >= E * ef;
    if (s) i -= E * ef;
    const int each = s ? es : ef, all = s ? shorts : full;
    if (i >= E * each) return {-1, false};
    const int e = i / each, local = ((x + e) & 7) * each + i - e * each;
    if (local < all) return {e * all + local, s};
  }
}

// Row tiles of `rows` rows that have more than half of them, and whether a
// short one follows.
template <int BM>
__device__ __forceinline__ int full_tiles(int rows) { return (rows + BM / 2 - 1) / BM; }
template <int BM>
__device__ __forceinline__ int short_tiles(int rows) { return rows > full_tiles<BM>(rows) * BM ? 1 : 0; }

// Within an expert: bands of kBand column tiles, row tiles inside a band.
constexpr int kBand = 8;
__device__ __forceinline__ void band_order(int local, int tm, int tn, int* m, int* n) {
  const int band = local / (kBand * tm), first = band * kBand;
  const int width = tn - first < kBand ? tn - first : kBand, rest = local - first * tm;
  *m = rest / width;
  *n = first + rest % width;
}

template <int BM, int BN>
constexpr size_t tile_lds() {
  return (size_t)2 * (BM + BN) * kDepth * 2;
}

// Scheduling of one half step: its LDS reads and loads spread evenly between
// its products, so that the matrix cores never wait for the LDS or the loads'
// issue.
template <int MFMAS, int READS, int LOADS>
__device__ __forceinline__ void interleave() {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kGroups = 16, kM = MFMAS / kGroups;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    constexpr int kR = READS / kGroups, kL = LOADS / kGroups;
    if constexpr (kR > 0) __builtin_amdgcn_sched_group_barrier(0x100, kR, 0);
    else if (g < READS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, kM, 0);
    if constexpr (kL > 0) __builtin_amdgcn_sched_group_barrier(0x020, kL, 0);
    else if (g < LOADS) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
  }
#endif
}

// Every wave's loads into LDS have arrived and its LDS reads are done.  The
// barrier alone does not wait for loads into LDS: the wait is explicit.
__device__ __forceinline__ void arrived() {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#endif
  __syncthreads();
}

// Full and short row tiles before each expert's, its first row and row count, in LDS.
struct ExpertTable {
  int first[2][257], base[256], rows[256];
};

// One output tile's work: steps [first, last) of its contraction.
struct Tile {
  int e;               // -1: none left
  int base, M, D;      // span's first row; rows (columns for dw) of the output here; contraction length
  int m0, n0, split;
  int first, last;
};

// The tile at `id`, or at the block's next id that has one (id moves there).
// All values are wave-uniform scalars.
template <int MODE, int BM, int BN>
__device__ __forceinline__ Tile find_tile(const LinearArgs& a, const ExpertTable& tab, int& id) {
  const int cols = MODE == kFwd ? a.N : a.K, tn = (cols + BN - 1) / BN;
  // dw: every expert has the same row tiles
  const int fw = full_tiles<BM>(a.N), sw = short_tiles<BM>(a.N);
  const int full = (MODE == kDw ? fw : __builtin_amdgcn_readfirstlane(tab.first[0][a.E])) * tn;
  const int shorts = (MODE == kDw ? sw : __builtin_amdgcn_readfirstlane(tab.first[1][a.E])) * tn;
  Tile t;
  t.e = -1;
  const TileIndex x = MODE == kDw ? spread_order(id, gridDim.x, a.E, full * a.splits, shorts * a.splits)
                                  : xcd_order(id, full * a.splits, shorts * a.splits);
  if (x.at < 0) return t;
  const int per = x.short_ ? shorts : full;      // dw: of one expert
  int tm, local;       // row tiles of this kind of the expert, index among its tiles of this kind
  if (MODE == kDw) {
    tm = x.short_ ? sw : fw;
    t.e = x.at / (per * a.splits);
    const int in = x.at - t.e * per * a.splits;
    t.split = in / per;
    local = in - t.split * per;
  } else {
    t.split = x.at / per;
    const int at = x.at - t.split * per;
    const int* first = tab.first[x.short_ ? 1 : 0];
    const int q = at / tn, lane = threadIdx.x & 63;
    int e = -1;                                              // the last expert that starts at or before row tile q
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (64 * c >= a.E) break;
      e += __builtin_popcountll(__ballot(64 * c + lane < a.E && first[64 * c + lane] <= q));
    }
    t.e = e;
    const int f = __builtin_amdgcn_readfirstlane(first[e]);
    tm = __builtin_amdgcn_readfirstlane(first[e + 1]) - f;
    local = at - f * tn;
  }
  int mt, nt;
  band_order(local, tm, tn, &mt, &nt);
  t.base = __builtin_amdgcn_readfirstlane(tab.base[t.e]);
  const int rows = __builtin_amdgcn_readfirstlane(tab.rows[t.e]);
  t.M = MODE == kDw ? a.N : rows;
  t.D = MODE == kFwd ? a.K : MODE == kDx ? a.N : rows;
  t.m0 = (x.short_ ? full_tiles<BM>(t.M) : mt) * BM;
  t.n0 = nt * BN;
  const int all = (t.D + kDepth - 1) / kDepth, each = (all + a.splits - 1) / a.splits;
  t.first = t.split * each < all ? t.split * each : all;
  t.last = t.first + each < all ? t.first + each : all;
  return t;
}

__device__ __forceinline__ void swap_odd_even_rows(float& x, float& y) {
#ifdef __HIP_DEVICE_COMPILE__
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y),
                                                   false, false);
  const unsigned r0 = r[0], r1 = r[1];     // a bit cast of a vector's element itself reads element 0
  x = __builtin_bit_cast(float, r0);
  y = __builtin_bit_cast(float, r1);
#endif
}

template <class T>
using Packed8 = Pack<T, 8, false>;

// 8 values rounded to the 16-bit type.
template <class T>
__device__ __forceinline__ u32x4 rounded(const float* v) {
  Pack<T, 8> o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] = T::down(v[i]);
  return __builtin_bit_cast(u32x4, o);
}

// Orders a wave's LDS accesses where its lanes read what others of them wrote:
// the hardware runs a wave's LDS instructions in order, this keeps the compiler
// from moving them past each other.  No instruction.
__device__ __forceinline__ void wave_in_order() {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#endif
}

// Results of a wave for arrays of any alignment and row length: 64 rows x 64
// columns from row m, column n on, turned around in the wave's own LDS (16-byte
// piece c of row r at place c ^ (r mod 16)), so that a lane gets 8 consecutive
// columns and the epilogue's code is there once.
constexpr int kTurned = 64 * 64 * 4;
template <class T, int MODE>
__device__ __forceinline__ void finish_turned(const LinearArgs& a, int e, int base, int M, int m0, int n0, int split,
                                              char* mine, const f32x4 (*acc)[4]) {
  const int lane = threadIdx.x & 63, r0 = lane & 15, cols = MODE == kFwd ? a.N : a.K;
  wave_in_order();                         // the rows before have been read
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *(f32x4*)(mine + (16 * i + r0) * 256 + (((4 * j + (lane >> 4)) ^ r0) << 4)) = acc[i][j];
  wave_in_order();                         // all lanes' results are there
  LinearArgs to = a;
  if (a.splits > 1) {                      // this split's sums as they are
    to.out = a.part + (int64_t)split * (MODE == kDw ? (int64_t)a.E * a.N : a.rows) * cols;
    to.out_f32 = 1;
    to.act = MILO_ACT_NONE;
    to.bias = to.mul = to.residual = nullptr;
    to.pre = nullptr;
  }
  const int n = n0 + 8 * (lane & 7);
#pragma unroll 1
  for (int it = 0; it < 8; ++it) {
    const int r = 8 * it + (lane >> 3), p = 2 * (lane & 7);
    const f32x4 lo = *(const f32x4*)(mine + r * 256 + ((p ^ (r & 15)) << 4));
    const f32x4 hi = *(const f32x4*)(mine + r * 256 + (((p + 1) ^ (r & 15)) << 4));
    if (m0 + r >= M || n + 8 > cols) continue;
    const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    finish<T, MODE, 8, true>(to, e, base + (int64_t)(m0 + r), n, v);
  }
  // The piece that the last column cuts, a column at a time over all 64 rows
  // (within the loop above, piece by piece, it made the last column tile
  // 40 us longer).
  const int left = cols - n0;
  if (left > 0 && left < 64 && m0 + lane < M)
#pragma unroll 1
    for (int c = left & ~7; c < left; ++c) {
      const float v = *(const float*)(mine + lane * 256 + (((c >> 2) ^ r0) << 4) + (c & 3) * 4);
      finish<T, MODE, 1, true>(to, e, base + (int64_t)(m0 + lane), n0 + c, &v);
    }
}

constexpr int kAhead = 2;   // row groups whose epilogue operands are asked for at a time

// Persistent blocks: block b takes tiles b, b + grid, ...  The steps of all its
// tiles form one stream of loads that runs two steps ahead of the products,
// across tile borders: the next tile's operands are on their way while this
// tile's results are written.
//
// A step is used in two halves of 32 contraction values; the fragments of one
// half are read from LDS while the products of the half before run.  One
// barrier a step, between the halves: there every wave has read the last of
// the buffer (so the stream's next step may be loaded into it) and its part of
// the step after has arrived.
//
// ACT: the activation of a forward launch (MILO_ACT_NONE also stands for
// RELU), a template so that each kernel holds one activation's code.  LOOSE:
// the stream of loads stops at each tile's end, its results go through LDS.
template <class T, int MODE, int ACT, int BM, int BN, int WM, int WN, bool LOOSE = false>
__global__ void __launch_bounds__(64 * WM * WN, BM == 256 ? 1 : 2) linear_tile_kernel(LinearArgs a) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass has no gfx950 builtins; it needs the launch stub only
  constexpr int NW = WM * WN, NI = BM / WM / 16, NJ = BN / WN / 16;
  constexpr bool AW = MODE == kDw, BW = MODE != kFwd;
  extern __shared__ __align__(16) char lds[];
  __shared__ ExpertTable tab;
  typedef Operand<AW, BM, NW> OpA;
  typedef Operand<BW, BN, NW> OpB;
  constexpr int kBuf = OpA::kBytes + OpB::kBytes;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = MODE == kFwd ? a.N : a.K;
  const int64_t lda = a.lda, ldb = a.ldb;

  if (wave == 0) {
    int before[2] = {0, 0};
    for (int c = 0; c < a.E; c += 64) {
      const int e = c + lane;
      const Span p = e < a.E ? expert_span(a.offsets, e, a.rows) : Span{0, 0};
      if (e < a.E) {
        tab.base[e] = p.base;
        tab.rows[e] = p.rows;
      }
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        const int n = kind ? short_tiles<BM>(p.rows) : full_tiles<BM>(p.rows);
        int v = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int u = __shfl_up(v, d);
          if (lane >= d) v += u;
        }
        if (e < a.E) tab.first[kind][e] = before[kind] + v - n;
        before[kind] += __shfl(v, 63);
      }
    }
    if (lane == 0) {
      tab.first[0][a.E] = before[0];
      tab.first[1][a.E] = before[1];
    }
  }
  __syncthreads();

  // ---- the stream of loads
  OpA oa;
  OpB ob;
  Tile ahead;
  int ahead_id = blockIdx.x, step = 0;
  const uint16_t *pa = nullptr, *pb = nullptr;
  int lefta = 0, leftb = 0;
  auto seek = [&]() {                        // to the first tile at or after ahead_id with steps
    for (;; ahead_id += gridDim.x) {
      ahead = find_tile<MODE, BM, BN>(a, tab, ahead_id);
      if (ahead.e < 0) {
        step = 0;
        ahead.D = ahead.last = 0;
        return;
      }
      if (ahead.first < ahead.last) break;
    }
    step = ahead.first;
    pa = (const uint16_t*)a.a + (int64_t)ahead.base * lda + (AW ? (int64_t)ahead.m0 : ahead.m0 * lda);
    pb = (const uint16_t*)a.b + (MODE == kDw ? (int64_t)ahead.base * ldb : (int64_t)ahead.e * a.N * ldb) +
         (BW ? (int64_t)ahead.n0 : ahead.n0 * ldb);
    // wide: to the end of the row's last piece of 8 (rows are padded to whole pieces)
    lefta = AW ? (ahead.M - ahead.m0 + 7) & ~7 : ahead.M - ahead.m0 < BM ? ahead.M - ahead.m0 : BM;
    leftb = BW ? (cols - ahead.n0 + 7) & ~7 : cols - ahead.n0 < BN ? cols - ahead.n0 : BN;
    oa.init(lane, wave, (int)lda, ahead.M - ahead.m0);
    ob.init(lane, wave, (int)ldb, cols - ahead.n0);
  };
  auto issue = [&](int buf) {
    char* dst = lds + buf * kBuf;
    const bool on = step < ahead.last;
    oa.load(pa, lda, lefta, ahead.D, step * kDepth, on, dst, wave);
    ob.load(pb, ldb, leftb, ahead.D, step * kDepth, on, dst + OpA::kBytes, wave);
  };
  auto advance = [&]() {
    if (++step >= ahead.last && ahead.e >= 0 && !LOOSE) {
      ahead_id += gridDim.x;
      seek();
    }
  };
  oa.init(lane, wave, (int)lda, 0);
  ob.init(lane, wave, (int)ldb, 0);
  ahead.e = -1;
  auto start = [&]() {
    seek();
    issue(0);
    advance();
    issue(1);
    advance();
    arrived();
  };
  if constexpr (!LOOSE) start();

  // ---- one tile with NIX of the NI row groups of a wave
  const int wn = wave % WN * (BN / WN);
  Fragments<BW, BN, NJ> fb;
  fb.init(lane, wn);
  int buf = 0;
  auto tile = [&](const Tile& t, auto nix) {
    constexpr int NIX = decltype(nix)::value;
    const int wm = wave / WN * (NIX * 16);
    Fragments<AW, BM, NIX> fa;
    fa.init(lane, wm);
    f32x4 acc[NIX][NJ];
#pragma unroll
    for (int i = 0; i < NIX; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    s16x8 xa[2][NIX], xb[2][NJ];
    auto read = [&](int b, int h) {
      const char* la = lds + b * kBuf;
#pragma unroll
      for (int j = 0; j < NJ; ++j) xb[h][j] = fb.read(la + OpA::kBytes, h, j);
#pragma unroll
      for (int i = 0; i < NIX; ++i) xa[h][i] = fa.read(la, h, i);
    };
    auto products = [&](int h) {
#pragma unroll
      for (int i = 0; i < NIX; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = T::mfma(xb[h][j], xa[h][i], acc[i][j]);
    };
    constexpr int kReads = NIX * (AW ? 2 : 1) + NJ * (BW ? 2 : 1), kLoads = OpA::kLoads + OpB::kLoads;
    if (t.first < t.last) {
      read(buf, 0);
      for (int k = t.first; k < t.last; ++k, buf ^= 1) {
        read(buf, 1);
        products(0);
        interleave<NIX * NJ, kReads, 0>();
        arrived();
        issue(buf);
        read(buf ^ 1, 0);          // past the tile's last step: another's data, not used
        products(1);
        interleave<NIX * NJ, kReads, kLoads>();
        advance();
      }
    }

    if constexpr (LOOSE) {
      // The stream has stopped behind this tile, so that the LDS is free for
      // the results; it starts again at the block's next tile.
      static_assert(NJ == 4 && NIX % 4 == 0 && NW * kTurned <= 2 * kBuf, "64 x 64 results a wave at a time");
      arrived();
#pragma unroll
      for (int g = 0; g < NIX; g += 4)
        finish_turned<T, MODE>(a, t.e, (MODE == kDw ? 0 : t.base), t.M, t.m0 + wm + 16 * g, t.n0 + wn, t.split,
                               lds + wave * kTurned, &acc[g]);
      __syncthreads();
      return;
    }
    // ---- results.  Lane l holds row l % 16, columns 4 (l / 16) .. +3 of each
    // 16 x 16 product.  All accesses go through buffer resources that begin at
    // the tile and end with its last row, columns past the end get an offset
    // outside: no branches, so the compiler keeps many in flight.  No scalar
    // offsets here: with one, a 16-byte store's data registers were overwritten
    // by the next lane exchange before the store had read them (lanes 12..15
    // of its first word); without one the compiler knows the wait it needs.
    const int lane_row = lane & 15;
    const int rows_here = t.M - t.m0 < BM ? t.M - t.m0 : BM;
    const int64_t origin = ((MODE == kDw ? (int64_t)t.e * a.N : t.base) + (int64_t)t.m0) * cols;
    auto rsrc = [&](const void* p, int bytes) __attribute__((always_inline)) {
      return __builtin_amdgcn_make_buffer_rsrc((char*)p + origin * bytes, 0, rows_here * cols * bytes, kTileRsrcWord3);
    };
    if (a.splits > 1 || (MODE == kDw && a.out_f32)) {
      // float32 as it is: 64 contiguous bytes a row
      float* dst = (float*)a.out;
      if (a.splits > 1) dst = a.part + (int64_t)t.split * (MODE == kDw ? (int64_t)a.E * a.N : a.rows) * cols;
      const __amdgpu_buffer_rsrc_t r = rsrc(dst, 4);
      const int n = t.n0 + wn + 4 * (lane >> 4), at = ((wm + lane_row) * cols + n) * 4;
#pragma unroll
      for (int i = 0; i < NIX; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i][j]), r,
                                                 (n + 16 * j < cols ? at + 64 * j : kOutside) + 64 * i * cols, 0, 0);
      return;
    }
    // Exchanging rows of lanes between two neighbouring products gives a lane
    // 8 consecutive columns of the 32.
    const int n = t.n0 + wn + 16 * ((lane >> 4) & 1) + 8 * (lane >> 5);
    const int at = (wm + lane_row) * cols + n;
    const bool has_mul = MODE == kFwd && a.mul, has_add = MODE != kDw && a.residual;
    Pack<T, 8> bias[NJ / 2] = {};
    if (MODE == kFwd && a.bias) {
#pragma unroll
      for (int j = 0; j < NJ / 2; ++j)
        if (n + 32 * j < cols) bias[j] = load_pack<T, 8>(a.bias, (int64_t)t.e * a.N + n + 32 * j);
    }
    const __amdgpu_buffer_rsrc_t rm = rsrc(has_mul ? a.mul : a.out, 2), ra = rsrc(has_add ? a.residual : a.out, 2),
                                 rp = rsrc(MODE == kFwd && a.pre ? a.pre : a.out, 2), ro = rsrc(a.out, a.out_f32 ? 4 : 2);
#pragma unroll
    for (int q = 0; q < NIX / kAhead; ++q) {
      u32x4 mul[kAhead][NJ / 2], add[kAhead][NJ / 2];
      if (has_mul) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
          for (int j = 0; j < NJ / 2; ++j)
            mul[i][j] = __builtin_amdgcn_raw_buffer_load_b128(
                rm, (n + 32 * j < cols ? 2 * at + 64 * j : kOutside) + 32 * (kAhead * q + i) * cols, 0, 0);
      }
      if (has_add) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
          for (int j = 0; j < NJ / 2; ++j)
            add[i][j] = __builtin_amdgcn_raw_buffer_load_b128(
                ra, (n + 32 * j < cols ? 2 * at + 64 * j : kOutside) + 32 * (kAhead * q + i) * cols, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int j = 0; j < NJ / 2; ++j) {
          const int g = kAhead * q + i;
          const f32x4 lo = acc[g][2 * j], hi = acc[g][2 * j + 1];
          float v[8];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            v[c] = lo[c];
            v[4 + c] = hi[c];
            swap_odd_even_rows(v[c], v[4 + c]);
          }
          const int off = (n + 32 * j < cols ? 2 * at + 64 * j : kOutside) + 32 * g * cols;
          if constexpr (MODE == kFwd) {
            if (a.bias) add_pack(v, bias[j]);
            if (a.pre) __builtin_amdgcn_raw_buffer_store_b128(rounded<T>(v), rp, off, 0, 0);
            if (ACT != MILO_ACT_NONE) {
#pragma unroll
              for (int c = 0; c < 8; ++c) v[c] = act_value(ACT, v[c]);
            } else if (a.act == MILO_ACT_RELU) {
#pragma unroll
              for (int c = 0; c < 8; ++c) v[c] = act_value(MILO_ACT_RELU, v[c]);
            }
            if (has_mul) mul_pack(v, __builtin_bit_cast(Packed8<T>, mul[i][j]));
          }
          if (has_add) add_pack(v, __builtin_bit_cast(Packed8<T>, add[i][j]));
          if (MODE != kFwd || !a.out_f32) {
            __builtin_amdgcn_raw_buffer_store_b128(rounded<T>(v), ro, off, 0, 0);
          } else {
            const int wide = (n + 32 * j < cols ? 4 * at + 128 * j : kOutside) + 64 * g * cols;
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}), ro, wide, 0,
                                                   0);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}), ro,
                                                   wide + 16, 0, 0);
          }
        }
    }
  };

  // A tile with at most half of its rows runs at half the height: a good part
  // of the experts' last row tiles would otherwise multiply mostly nothing.
  for (int id = blockIdx.x;; id += gridDim.x) {   // find_tile may move id on
    const Tile t = find_tile<MODE, BM, BN>(a, tab, id);
    if (t.e < 0) break;
    if constexpr (LOOSE) {
      ahead_id = id;
      buf = 0;
      start();
    }
    if constexpr (NI == 8) {
      if (t.M - t.m0 <= BM / 2) {
        tile(t, std::integral_constant<int, NI / 2>());
        continue;
      }
    }
    tile(t, std::integral_constant<int, NI>());
  }
  // the loads past the last step (of nothing) have ended before the LDS is given back
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#endif
}

template <class T, int MODE, int ACT, int BM, int BN, int WM, int WN, bool LOOSE = false>
static hipError_t run_tile(const LinearArgs& a, hipStream_t st) {
  const int64_t tn = ((MODE == kFwd ? a.N : a.K) + BN - 1) / BN;
  const int64_t rows = MODE == kDw ? (int64_t)a.E * ((a.N + BM - 1) / BM)
                                   : (a.rows + BM - 1) / BM + (a.E > 1 ? a.E : 0);
  // as many blocks as run at once (one or two to a compute unit: the LDS
  // ring), a multiple of 8 so that a block's tiles stay on its XCD
  const int64_t slots = (int64_t)device_cu_count() * (BM == 256 ? 1 : 2);
  int64_t blocks = rows * tn * a.splits;
  blocks = (blocks < slots ? blocks + 7 : slots) / 8 * 8;
  if (blocks < 8) blocks = 8;
  constexpr size_t bytes = tile_lds<BM, BN>();
  const void* fn = (const void*)linear_tile_kernel<T, MODE, ACT, BM, BN, WM, WN, LOOSE>;
  if (bytes + sizeof(ExpertTable) > 65536) {
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((linear_tile_kernel<T, MODE, ACT, BM, BN, WM, WN, LOOSE>), dim3((unsigned)blocks),
                     dim3(64 * WM * WN), bytes, st, a);
  return hipGetLastError();
}

}  // namespace milo
