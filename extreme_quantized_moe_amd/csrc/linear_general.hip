// The grouped 16-bit product for any sizes and any element-aligned operands:
// 64 x 64 output tiles, contraction in steps of 32, staged through LDS element
// by element with every access bounded.
#include "linear.hpp"

namespace milo {

constexpr int kGenTile = 64, kGenDepth = 32, kGenStride = kGenDepth + 8;   // halves; rows stay 16-byte aligned

// The tile's part of an operand into LDS as [64][kGenStride], contraction
// contiguous.  deep: element (i, c) at src[i * ld + c]; wide: at src[c * ld + i].
template <bool WIDE>
__device__ __forceinline__ void stage(const uint16_t* __restrict__ src, int64_t ld, int count, int depth,
                                      uint16_t* lds) {
#pragma unroll
  for (int j = 0; j < kGenTile * kGenDepth / 256; ++j) {
    const int f = j * 256 + threadIdx.x;
    const int i = WIDE ? f % kGenTile : f / kGenDepth, c = WIDE ? f / kGenTile : f % kGenDepth;
    lds[i * kGenStride + c] = i < count && c < depth ? src[WIDE ? c * ld + i : i * ld + c] : (uint16_t)0;
  }
}

template <class T, int MODE>
__global__ void __launch_bounds__(256) linear_general_kernel(LinearArgs a) {
  __shared__ __align__(16) uint16_t la[kGenTile * kGenStride], lb[kGenTile * kGenStride];
  const int cols = MODE == kFwd ? a.N : a.K;
  const int ntn = (cols + kGenTile - 1) / kGenTile;
  const int id = blockIdx.x;
  TileSlot s;
  int m0, n0;
  if constexpr (MODE == kDw) {
    const int ntm = (a.N + kGenTile - 1) / kGenTile;
    s.e = id / (ntm * ntn);
    s.span = expert_span(a.offsets, s.e, a.rows);
    const int l = id - s.e * ntm * ntn;
    m0 = l / ntn * kGenTile;
    n0 = l % ntn * kGenTile;
  } else {
    s = find_slot(a.offsets, a.E, a.rows, kGenTile, ntn, [&](int) { return id; });
    if (s.e < 0) return;
    m0 = s.local / ntn * kGenTile;
    n0 = s.local % ntn * kGenTile;
  }
  // extents and first elements
  const int M = MODE == kDw ? a.N : s.span.rows;
  const int D = MODE == kFwd ? a.K : MODE == kDx ? a.N : s.span.rows;
  const int64_t lda = MODE == kFwd ? a.K : a.N, ldb = a.K;
  const uint16_t* pa = (const uint16_t*)a.a + (int64_t)s.span.base * lda;
  const uint16_t* pb = MODE == kDw ? (const uint16_t*)a.b + (int64_t)s.span.base * ldb
                                   : (const uint16_t*)a.b + (int64_t)s.e * a.N * a.K;
  constexpr bool AW = MODE == kDw, BW = MODE != kFwd;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;   // the wave's 32 x 32 quarter
  f32x4 acc[2][2] = {};
  for (int c0 = 0; c0 < D; c0 += kGenDepth) {
    stage<AW>(pa + (AW ? c0 * lda + m0 : m0 * lda + c0), lda, M - m0, D - c0, la);
    stage<BW>(pb + (BW ? c0 * ldb + n0 : n0 * ldb + c0), ldb, cols - n0, D - c0, lb);
    __syncthreads();
    s16x8 fa[2], fb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fa[i] = *(const s16x8*)(la + (wm + 16 * i + (lane & 15)) * kGenStride + 8 * (lane >> 4));
      fb[i] = *(const s16x8*)(lb + (wn + 16 * i + (lane & 15)) * kGenStride + 8 * (lane >> 4));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = T::mfma(fb[j], fa[i], acc[i][j]);
    __syncthreads();
  }
  // lane l of a 16 x 16 product holds row l % 16, columns 4 (l / 16) .. +3
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = m0 + wm + 16 * i + (lane & 15), n = n0 + wn + 16 * j + 4 * (lane >> 4) + r;
        if (m < M && n < cols) {
          const float v = acc[i][j][r];
          finish<T, MODE, 1>(a, s.e, (MODE == kDw ? 0 : s.span.base) + (int64_t)m, n, &v);
        }
      }
}

template <int MODE>
static int64_t general_blocks(const LinearArgs& a) {
  const int64_t ntn = ((MODE == kFwd ? a.N : a.K) + kGenTile - 1) / kGenTile;
  if (MODE == kDw) return a.E * (((int64_t)a.N + kGenTile - 1) / kGenTile) * ntn;
  return ((a.rows + kGenTile - 1) / kGenTile + (a.E > 1 ? a.E : 0)) * ntn;
}

template <class T>
static void run_general(int mode, const LinearArgs& a, hipStream_t st) {
  if (mode == kFwd)
    hipLaunchKernelGGL((linear_general_kernel<T, kFwd>), dim3((unsigned)general_blocks<kFwd>(a)), dim3(256), 0, st, a);
  else if (mode == kDx)
    hipLaunchKernelGGL((linear_general_kernel<T, kDx>), dim3((unsigned)general_blocks<kDx>(a)), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((linear_general_kernel<T, kDw>), dim3((unsigned)general_blocks<kDw>(a)), dim3(256), 0, st, a);
}

int32_t launch_linear_general(int mode, int dtype, const LinearArgs& a, hipStream_t st) {
  if (dtype == MILO_F16) run_general<F16>(mode, a, st);
  else run_general<BF16>(mode, a, st);
  return hip_status(hipGetLastError(), "linear_general_kernel launch");
}

}  // namespace milo
