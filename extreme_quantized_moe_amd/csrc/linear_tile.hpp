// The grouped 16-bit product on the matrix cores: BM x BN output tiles, the
// contraction in steps of 64 through LDS.  Needs row lengths of a multiple of
// 8 elements and 16-byte aligned operands (the plan's rule); any row count.
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

#include "linear.hpp"

namespace milo {

constexpr int kDepth = 64;                 // contraction values per step
constexpr int kTileRsrcWord3 = 0x00020000; // raw buffer, bounds checked in bytes
constexpr int kOutside = 0x7FFFFFF0;       // an offset no operand reaches

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
      typedef __attribute__((address_space(3))) s16x4 lds4;
      const char* p = lds + off[t] + s * 32 * ROWS * 2;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * ROWS * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Block -> tile.  Blocks go to the 8 XCDs in turn; each XCD gets a run of
// consecutive tiles, so that tiles sharing operands share its L2.
__device__ __forceinline__ int xcd_order(int id, int total) {
  const int q = total >> 3, r = total & 7, x = id & 7, i = id >> 3;
  if (i >= q + (x < r ? 1 : 0)) return -1;
  return x * q + (x < r ? x : r) + i;
}

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

// One tile: rows m0 .. of the expert's span (or output rows of dw), columns
// n0 .., this split's share of the contraction.
template <class T, int MODE, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void tile_body(const LinearArgs& a, const TileSlot& s, int m0, int n0, int split,
                                          char* lds) {
  constexpr int NW = WM * WN, NI = BM / WM / 16, NJ = BN / WN / 16;
  constexpr bool AW = MODE == kDw, BW = MODE != kFwd;
  typedef Operand<AW, BM, NW> OpA;
  typedef Operand<BW, BN, NW> OpB;
  constexpr int kBuf = OpA::kBytes + OpB::kBytes;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = MODE == kFwd ? a.N : a.K;
  const int M = MODE == kDw ? a.N : s.span.rows;
  const int D = MODE == kFwd ? a.K : MODE == kDx ? a.N : s.span.rows;
  const int64_t lda = MODE == kFwd ? a.K : a.N, ldb = a.K;
  const uint16_t* pa = (const uint16_t*)a.a + (int64_t)s.span.base * lda + (AW ? (int64_t)m0 : m0 * lda);
  const uint16_t* pb = (const uint16_t*)a.b +
                       (MODE == kDw ? (int64_t)s.span.base * ldb : (int64_t)s.e * a.N * a.K) +
                       (BW ? (int64_t)n0 : n0 * ldb);
  const int lefta = M - m0 < BM && !AW ? M - m0 : AW ? M - m0 : BM;
  const int leftb = BW ? cols - n0 : cols - n0 < BN ? cols - n0 : BN;

  OpA oa;
  OpB ob;
  oa.init(lane, wave, (int)lda, M - m0);
  ob.init(lane, wave, (int)ldb, cols - n0);
  const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
  Fragments<AW, BM, NI> fa;
  Fragments<BW, BN, NJ> fb;
  fa.init(lane, wm);
  fb.init(lane, wn);
  f32x4 acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // This split's steps.  Step k is used in two halves of 32 contraction
  // values; the fragments of one half are read from LDS while the products of
  // the half before run.  One barrier a step, between the halves: there every
  // wave has read the last of buffer k (so step k + 2 may be loaded into it,
  // a whole step of products ahead of its use) and its part of step k + 1 has
  // arrived.
  const int all = (D + kDepth - 1) / kDepth, each = (all + a.splits - 1) / a.splits;
  const int first = split * each, last = first + each < all ? first + each : all;
  auto issue = [&](int k, int buf) {
    char* dst = lds + buf * kBuf;
    oa.load(pa, lda, lefta, D, k * kDepth, k < last, dst, wave);
    ob.load(pb, ldb, leftb, D, k * kDepth, k < last, dst + OpA::kBytes, wave);
  };
  s16x8 xa[2][NI], xb[2][NJ];
  auto read = [&](int buf, int h) {
    const char* la = lds + buf * kBuf;
#pragma unroll
    for (int j = 0; j < NJ; ++j) xb[h][j] = fb.read(la + OpA::kBytes, h, j);
#pragma unroll
    for (int i = 0; i < NI; ++i) xa[h][i] = fa.read(la, h, i);
  };
  auto products = [&](int h) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = T::mfma(xb[h][j], xa[h][i], acc[i][j]);
  };
  constexpr int kReads = NI * (AW ? 2 : 1) + NJ * (BW ? 2 : 1), kLoads = OpA::kLoads + OpB::kLoads;
  if (first < last) {
    issue(first, 0);
    issue(first + 1, 1);
    arrived();
    read(0, 0);
    int buf = 0;
    for (int k = first; k < last; ++k, buf ^= 1) {
      read(buf, 1);
      products(0);
      interleave<NI * NJ, kReads, 0>();
      arrived();
      issue(k + 2, buf);
      read(buf ^ 1, 0);          // past the last step: stale data, never used
      products(1);
      interleave<NI * NJ, kReads, kLoads>();
    }
    arrived();             // the epilogue reuses the LDS
  }

  // Lane l holds row l % 16, columns 4 (l / 16) .. +3 of each 16 x 16 product.
  // Each wave turns 64 x 64 results at a time around in its own 16 KB of LDS
  // (16-byte piece c of row r at place c ^ (r mod 16)), so that a lane gets 8
  // consecutive columns: 128-byte rows of 16-byte accesses.
  static_assert(NJ % 4 == 0 && NI % 4 == 0, "the epilogue takes 64 x 64 results at a time");
  char* mine = lds + wave * 16384;
#pragma unroll
  for (int qq = 0; qq < NI / 4 * (NJ / 4); ++qq) {
    const int q = qq / (NJ / 4), g = qq % (NJ / 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = lane & 15;
        *(f32x4*)(mine + (16 * i + r) * 256 + (((4 * j + (lane >> 4)) ^ r) << 4)) = acc[4 * q + i][4 * g + j];
      }
    const int n = n0 + wn + 64 * g + 8 * (lane & 7), mq = m0 + wm + 64 * q + (lane >> 3);
    const int64_t row = (MODE == kDw ? 0 : s.span.base) + (int64_t)mq;
    // step it of a pass: row mq + 8 it, its two 16-byte pieces
    auto lo_at = [&](int it) {
      const int r = 8 * it + (lane >> 3);
      return (f32x4*)(mine + r * 256 + (((2 * (lane & 7)) ^ (r & 15)) << 4));
    };
    auto hi_at = [&](int it) {
      const int r = 8 * it + (lane >> 3);
      return (f32x4*)(mine + r * 256 + (((2 * (lane & 7) + 1) ^ (r & 15)) << 4));
    };
    if (a.splits > 1) {
      const int64_t rows = MODE == kDw ? (int64_t)a.E * a.N : a.rows;
      float* part = a.part + (split * rows + (MODE == kDw ? (int64_t)s.e * a.N : 0) + row) * cols + n;
#pragma unroll
      for (int it = 0; it < 8; ++it)
        if (mq + 8 * it < M && n < cols) {
          *(f32x4*)(part + (int64_t)8 * it * cols) = *lo_at(it);
          *(f32x4*)(part + (int64_t)8 * it * cols + 4) = *hi_at(it);
        }
      continue;
    }
    // What the epilogue reads is asked for before the first pass: its latency
    // is paid once for the 64 x 64 results, not once a row.
    const bool has_mul = MODE == kFwd && a.mul, has_add = MODE != kDw && a.residual;
    Pack<T, 8> bias = {}, mul[8], add[8];
    if (MODE == kFwd && a.bias && n < cols) bias = load_pack<T, 8>(a.bias, (int64_t)s.e * a.N + n);
    if (has_mul) {
#pragma unroll
      for (int it = 0; it < 8; ++it)
        if (mq + 8 * it < M && n < cols) mul[it] = load_pack<T, 8>(a.mul, (row + 8 * it) * cols + n);
    }
    if (has_add) {
#pragma unroll
      for (int it = 0; it < 8; ++it)
        if (mq + 8 * it < M && n < cols) add[it] = load_pack<T, 8>(a.residual, (row + 8 * it) * cols + n);
    }
    if (MODE == kFwd && (a.bias || a.pre || a.act != MILO_ACT_NONE)) {
      // bias, kept pre-activation and activation, back into LDS: one copy of
      // the activations' code
#pragma unroll 1
      for (int it = 0; it < 8; ++it) {
        if (mq + 8 * it >= M || n >= cols) continue;
        const f32x4 lo = *lo_at(it), hi = *hi_at(it);
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        if (a.bias) add_pack<T, 8>(v, bias);
        if (a.pre) store_pack<T, 8>(a.pre, (row + 8 * it) * cols + n, v);
        if (a.act != MILO_ACT_NONE) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = act_value(a.act, v[i]);
        }
        *lo_at(it) = f32x4{v[0], v[1], v[2], v[3]};
        *hi_at(it) = f32x4{v[4], v[5], v[6], v[7]};
      }
    }
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      if (mq + 8 * it >= M || n >= cols) continue;
      const f32x4 lo = *lo_at(it), hi = *hi_at(it);
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      if (has_mul) mul_pack<T, 8>(v, mul[it]);
      if (has_add) add_pack<T, 8>(v, add[it]);
      store_out<T, 8>(a, out_at<MODE>(a, s.e, row + 8 * it, n), v);
    }
  }
}

// A row tile with at most half of its rows runs a form of half the height (a
// quarter of the experts' last tiles otherwise multiply mostly nothing).
template <class T, int MODE, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN, BM == 256 ? 1 : 2) linear_tile_kernel(LinearArgs a) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass has no gfx950 builtins; it needs the launch stub only
  extern __shared__ __align__(16) char lds[];
  static_assert(tile_lds<BM, BN>() >= (size_t)WM * WN * 16384, "the epilogue's staging fits");
  const int tn = ((MODE == kFwd ? a.N : a.K) + BN - 1) / BN;
  TileSlot s;
  int mt, nt;
  if constexpr (MODE == kDw) {
    const int tm = (a.N + BM - 1) / BM, id = xcd_order(blockIdx.x, a.E * tm * tn);
    if (id < 0) return;
    s.e = id / (tm * tn);
    s.span = expert_span(a.offsets, s.e, a.rows);
    band_order(id - s.e * tm * tn, tm, tn, &mt, &nt);
  } else {
    const int id = blockIdx.x;
    s = find_slot(a.offsets, a.E, a.rows, BM, tn, [&](int total) { return xcd_order(id, total); });
    if (s.e < 0) return;
    band_order(s.local, s.row_tiles, tn, &mt, &nt);
  }
  const int m0 = mt * BM, left = (MODE == kDw ? a.N : s.span.rows) - m0;
  if constexpr (BM == 256) {
    if (left <= BM / 2) {
      tile_body<T, MODE, BM / 2, BN, WM, WN>(a, s, m0, nt * BN, blockIdx.y, lds);
      return;
    }
  }
  tile_body<T, MODE, BM, BN, WM, WN>(a, s, m0, nt * BN, blockIdx.y, lds);
#endif
}

}  // namespace milo
