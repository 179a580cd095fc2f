// The grouped 16-bit product on 128 x 128 tiles for operands that are aligned
// to their elements only, or have row lengths that are no multiple of 8.  Such
// rows start anywhere, which loads straight into LDS do not take: a step's
// pieces of 8 values go through registers (asked for a step ahead, while the
// products of the step before run) into the same LDS layout the aligned tile
// kernels use.  Rows past an operand's end read its last row instead, since
// they feed results that are not stored; contraction values and columns past
// the end read as zeros.  Bound by the loads: 16 bytes that start on an odd
// element cost several aligned ones.  4096 x 14335 x 4097 over 8 experts forward
// 0.91 ms, dx 1.05, dw 0.97 (530, 455, 495 TFLOP/s).  For few rows, where
// copying the weights into whole rows would cost more than it saves (the plan's
// rule).
#include "linear_tile.hpp"

namespace milo {

template <bool WIDE>
struct LoosePieces {
  static constexpr int kPieces = 4;          // 128 x 64 values over 256 threads, 8 at a time
  u32x4 v[kPieces];

  // As Operand: deep: src is the tile's first row, `left` its rows; wide: src is
  // the tile's first column, `left` its columns.  The two forms are one uniform
  // branch a step: a branch at each load has them wait for each other (4096 x
  // 14335 x 4097 over 8 experts dx 1302 us with one, 1054 without).
  __device__ __forceinline__ void load(const uint16_t* src, int64_t ld, int left, int depth, int k0) {
    if constexpr (!WIDE) {
      auto rows = [&](auto piece) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          const int slot = j * 256 + threadIdx.x, r = slot >> 3;
          v[j] = piece(src + (int64_t)(r < left ? r : left - 1) * ld, k0 + (((slot & 7) ^ (r & 7)) << 3));
        }
      };
      if (k0 + kDepth <= depth) rows([&](const uint16_t* row, int k) { return load_whole(row + k); });
      else rows([&](const uint16_t* row, int k) { return load_cut(row + k, depth - k); });
    } else {
      auto rows = [&](auto piece) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          const int slot = j * 256 + threadIdx.x, k = slot >> 4, p = slot & 15;
          v[j] = piece(k0 + k, ((((p >> 1) ^ Operand<true, 128, 4>::wide_swizzle(k)) << 1) | (p & 1)) << 3);
        }
      };
      // Rows past the contraction read its last one and count as zeros.
      auto rows_to_end = [&](auto piece) {
        rows([&](int k, int c) {
          const u32x4 some = piece(src + (k < depth ? k : depth - 1) * ld, c);
          return k < depth ? some : u32x4{0, 0, 0, 0};
        });
      };
      // Columns past the end feed results that are not stored: where another
      // row of 8 or more follows the step, a piece may run on into it.
      if (left >= 128 ? k0 + kDepth <= depth : k0 + kDepth < depth && ld >= 8)
        rows([&](int k, int c) { return load_whole(src + k * ld + (c < left ? c : 0)); });
      else if (left >= 128)
        rows_to_end([&](const uint16_t* row, int c) { return load_whole(row + c); });
      else
        rows_to_end([&](const uint16_t* row, int c) { return load_cut(row + c, left - c); });
    }
  }

  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) *(u32x4*)(lds + (j * 256 + threadIdx.x) * 16) = v[j];
  }
};

template <class T, int MODE>
__global__ void __launch_bounds__(256, 2) linear_loose_kernel(LinearArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr bool AW = MODE == kDw, BW = MODE != kFwd;
  constexpr int kTile = 128, kOperand = kTile * kDepth * 2, kBuf = 2 * kOperand;
  __shared__ __align__(16) char lds[2 * kBuf];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = MODE == kFwd ? a.N : a.K, tn = (cols + kTile - 1) / kTile;
  const int split = blockIdx.y, id = blockIdx.x;
  TileSlot s;
  int mt, nt;
  if constexpr (MODE == kDw) {
    const int tm = (a.N + kTile - 1) / kTile;
    s.e = id / (tm * tn);
    s.span = expert_span(a.offsets, s.e, a.rows);
    band_order(id - s.e * tm * tn, tm, tn, &mt, &nt);
  } else {
    s = find_slot(a.offsets, a.E, a.rows, kTile, tn, [&](int) { return id; });
    if (s.e < 0) return;
    band_order(s.local, s.row_tiles, tn, &mt, &nt);
  }
  const int m0 = mt * kTile, n0 = nt * kTile;
  const int M = MODE == kDw ? a.N : s.span.rows;
  const int D = MODE == kFwd ? a.K : MODE == kDx ? a.N : s.span.rows;
  const int64_t lda = MODE == kFwd ? a.K : a.N, ldb = a.K;
  const uint16_t* pa = (const uint16_t*)a.a + (int64_t)s.span.base * lda + (AW ? (int64_t)m0 : m0 * lda);
  const uint16_t* pb = (const uint16_t*)a.b + (MODE == kDw ? (int64_t)s.span.base * ldb : (int64_t)s.e * a.N * a.K) +
                       (BW ? (int64_t)n0 : n0 * ldb);
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  Fragments<AW, kTile, 4> fa;
  Fragments<BW, kTile, 4> fb;
  fa.init(lane, wm);
  fb.init(lane, wn);
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int all = (D + kDepth - 1) / kDepth, each = (all + a.splits - 1) / a.splits;
  const int first = split * each, last = first + each < all ? first + each : all;
  LoosePieces<AW> qa;
  LoosePieces<BW> qb;
  auto load = [&](int k) {
    qa.load(pa, lda, M - m0, D, k * kDepth);
    qb.load(pb, ldb, cols - n0, D, k * kDepth);
  };
  if (first < last) load(first);
  char* buf = lds;
  for (int k = first; k < last; ++k) {
    // the other buffer was last read before the barrier of the step before
    qa.store(buf);
    qb.store(buf + kOperand);
    __syncthreads();
    if (k + 1 < last) load(k + 1);
    __builtin_amdgcn_sched_barrier(0);      // loads first: the products are what they wait behind
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s16x8 xa[4], xb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xb[i] = fb.read(buf + kOperand, h, i);
        xa[i] = fa.read(buf, h, i);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = T::mfma(xb[j], xa[i], acc[i][j]);
    }
    buf = buf == lds ? lds + kBuf : lds;
  }
  __syncthreads();
  finish_turned<T, MODE>(a, s.e, MODE == kDw ? 0 : s.span.base, M, m0 + wm, n0 + wn, split, lds + wave * kTurned, acc);
#endif
}

template <class T, int MODE>
static void run_loose(const LinearArgs& a, hipStream_t st) {
  const int64_t tn = ((MODE == kFwd ? a.N : a.K) + 127) / 128;
  const int64_t tm = MODE == kDw ? (int64_t)a.E * ((a.N + 127) / 128) : (a.rows + 127) / 128 + (a.E > 1 ? a.E : 0);
  hipLaunchKernelGGL((linear_loose_kernel<T, MODE>), dim3((unsigned)(tm * tn), (unsigned)a.splits), dim3(256), 0, st,
                     a);
}

template <class T>
static void run_loose_mode(int mode, const LinearArgs& a, hipStream_t st) {
  if (mode == kFwd) run_loose<T, kFwd>(a, st);
  else if (mode == kDx) run_loose<T, kDx>(a, st);
  else run_loose<T, kDw>(a, st);
}

int32_t launch_linear_loose(int mode, int dtype, const LinearArgs& a, hipStream_t st) {
  if (dtype == MILO_F16) run_loose_mode<F16>(mode, a, st);
  else run_loose_mode<BF16>(mode, a, st);
  return hip_status(hipGetLastError(), "linear_loose_kernel launch");
}

}  // namespace milo
