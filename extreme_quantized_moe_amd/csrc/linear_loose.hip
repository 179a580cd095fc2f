// The grouped 16-bit product on 128 x 128 tiles for operands that are aligned
// to their elements only, or have row lengths that are no multiple of 8.  Such
// rows start anywhere, which loads straight into LDS do not take: a step's
// pieces of 8 values go through registers (asked for a step ahead, while the
// products of the step before run) into the same LDS layout the aligned tile
// kernels use.  Rows past an operand's end read its last row instead, since
// they feed results that are not stored; contraction values and columns past
// the end read as zeros.  Bound by the loads' issue: 4096 x 14335 x 4097 over 8
// experts forward 0.87 ms, dx 1.1, dw 1.0 (550, 435, 480 TFLOP/s).
#include "linear_tile.hpp"

namespace milo {

template <bool WIDE>
struct LoosePieces {
  static constexpr int kPieces = 4;          // 128 x 64 values over 256 threads, 8 at a time
  u32x4 v[kPieces];

  // As Operand: deep: src is the tile's first row, `left` its rows; wide: src is
  // the tile's first column, `left` its columns.
  __device__ __forceinline__ void load(const uint16_t* src, int64_t ld, int left, int depth, int k0) {
    const bool whole = k0 + kDepth <= depth && (!WIDE || left >= 128);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int slot = j * 256 + threadIdx.x;
      if constexpr (!WIDE) {
        const int r = slot >> 3, c = k0 + (((slot & 7) ^ (r & 7)) << 3);
        const uint16_t* row = src + (int64_t)(r < left ? r : left - 1) * ld;
        v[j] = load_loose(row + c, whole ? 8 : depth - c);
      } else {
        const int k = slot >> 4, p = slot & 15;
        const int c = ((((p >> 1) ^ Operand<true, 128, 4>::wide_swizzle(k)) << 1) | (p & 1)) << 3;
        v[j] = load_loose(src + (int64_t)(k0 + k) * ld + c, whole ? 8 : k0 + k < depth ? left - c : 0);
      }
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
  // Each wave turns its 64 x 64 results around in its own 16 KB (16-byte piece
  // c of row r at place c ^ (r mod 16)), so that a lane gets 8 consecutive
  // columns and the epilogue's code is there once.
  char* mine = lds + wave * 16384;
  const int r0 = lane & 15;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *(f32x4*)(mine + (16 * i + r0) * 256 + (((4 * j + (lane >> 4)) ^ r0) << 4)) = acc[i][j];
  const int n = n0 + wn + 8 * (lane & 7);
#pragma unroll 1
  for (int it = 0; it < 8; ++it) {
    const int r = 8 * it + (lane >> 3), m = m0 + wm + r, p = 2 * (lane & 7);
    const f32x4 lo = *(const f32x4*)(mine + r * 256 + ((p ^ (r & 15)) << 4));
    const f32x4 hi = *(const f32x4*)(mine + r * 256 + (((p + 1) ^ (r & 15)) << 4));
    if (m >= M || n >= cols) continue;
    const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    const int64_t row = (MODE == kDw ? 0 : s.span.base) + (int64_t)m;
    if (a.splits > 1) {
      LinearArgs part = a;                   // this split's sums as they are
      part.out = a.part + (int64_t)split * (MODE == kDw ? (int64_t)a.E * a.N : a.rows) * cols;
      part.out_f32 = 1;
      part.act = MILO_ACT_NONE;
      part.bias = part.mul = part.residual = nullptr;
      part.pre = nullptr;
      finish_loose<T, MODE, 8>(part, s.e, row, n, cols - n, v);
    } else {
      finish_loose<T, MODE, 8>(a, s.e, row, n, cols - n, v);
    }
  }
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
