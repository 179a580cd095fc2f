// Launches of the tile kernels of the grouped 16-bit product.
#include "linear_tile.hpp"

namespace milo {

template <class T, int MODE, int ACT>
static hipError_t run_mode(const LinearArgs& a, int kernel, hipStream_t st) {
  return kernel == kPlanTile256 ? run_tile<T, MODE, ACT, 256, 256, 2, 4>(a, st)
                                : run_tile<T, MODE, ACT, 128, 128, 2, 2>(a, st);
}

template <class T>
static hipError_t run_type(int mode, const LinearArgs& a, int kernel, hipStream_t st) {
  if (mode == kDx) return run_mode<T, kDx, MILO_ACT_NONE>(a, kernel, st);
  if (mode == kDw) return run_mode<T, kDw, MILO_ACT_NONE>(a, kernel, st);
  switch (a.act) {
    case MILO_ACT_SILU: return run_mode<T, kFwd, MILO_ACT_SILU>(a, kernel, st);
    case MILO_ACT_GELU: return run_mode<T, kFwd, MILO_ACT_GELU>(a, kernel, st);
    case MILO_ACT_GELU_TANH: return run_mode<T, kFwd, MILO_ACT_GELU_TANH>(a, kernel, st);
    default: return run_mode<T, kFwd, MILO_ACT_NONE>(a, kernel, st);
  }
}

// ---- split contraction: the partial sums of each result in split order, then
// the epilogue.  A wave takes one row, a lane 8 columns.
template <class T, int MODE, bool LOOSE>
__global__ void __launch_bounds__(256) linear_join_kernel(LinearArgs a) {
  const int cols = MODE == kFwd ? a.N : a.K;
  const int n = (blockIdx.y * 64 + (threadIdx.x & 63)) * 8, wave = threadIdx.x >> 6;
  int e;
  int64_t row;
  if (MODE == kDw) {
    const int64_t r = (int64_t)blockIdx.x * 4 + wave;
    e = (int)(r / a.N);
    row = r - (int64_t)e * a.N;
    if (e >= a.E) return;
  } else {
    const int id = blockIdx.x;
    const TileSlot s = find_slot(a.offsets, a.E, a.rows, 4, 1, [&](int) { return id; });
    if (s.e < 0 || s.local * 4 + wave >= s.span.rows) return;
    e = s.e;
    row = s.span.base + (int64_t)s.local * 4 + wave;
  }
  const int64_t one = (MODE == kDw ? (int64_t)a.E * a.N : a.rows) * cols;
  if (n + (LOOSE ? 8 : 1) <= cols) {
    const int64_t at = out_at<MODE>(a, e, row, n);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < a.splits; ++s) {
      typedef Pack<F32, 4, LOOSE> Four;
      const float* p = a.part + s * one + at;
      const Four lo = *(const Four*)p, hi = *(const Four*)(p + 4);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] += lo.v[c];
        v[4 + c] += hi.v[c];
      }
    }
    finish<T, MODE, 8, LOOSE>(a, e, row, n, v);
  }
  // the last columns where eight do not fit, one a lane
  if (LOOSE && blockIdx.y == gridDim.y - 1 && (int)(threadIdx.x & 63) < cols % 8) {
    const int c = cols / 8 * 8 + (threadIdx.x & 63);
    float v = 0.f;
    for (int s = 0; s < a.splits; ++s) v += a.part[s * one + out_at<MODE>(a, e, row, c)];
    finish<T, MODE, 1, true>(a, e, row, c, &v);
  }
}

template <class T, int MODE>
static void run_join(const LinearArgs& a, bool loose, hipStream_t st) {
  const int cols = MODE == kFwd ? a.N : a.K;
  const int64_t quads = MODE == kDw ? ((int64_t)a.E * a.N + 3) / 4 : (a.rows + 3) / 4 + (a.E > 1 ? a.E : 0);
  const dim3 grid((unsigned)quads, (unsigned)((cols + 511) / 512));
  if (loose) hipLaunchKernelGGL((linear_join_kernel<T, MODE, true>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((linear_join_kernel<T, MODE, false>), grid, dim3(256), 0, st, a);
}

template <class T>
static void run_join_mode(int mode, const LinearArgs& a, bool loose, hipStream_t st) {
  if (mode == kFwd) run_join<T, kFwd>(a, loose, st);
  else if (mode == kDx) run_join<T, kDx>(a, loose, st);
  else run_join<T, kDw>(a, loose, st);
}

int32_t launch_linear_join(int mode, int dtype, const LinearArgs& a, bool loose, hipStream_t st) {
  if (dtype == MILO_F16) run_join_mode<F16>(mode, a, loose, st);
  else run_join_mode<BF16>(mode, a, loose, st);
  return hip_status(hipGetLastError(), "linear_join_kernel launch");
}

int32_t launch_linear_tile(int mode, int dtype, const LinearArgs& a, int kernel, hipStream_t st) {
  const hipError_t e = dtype == MILO_F16 ? run_type<F16>(mode, a, kernel, st) : run_type<BF16>(mode, a, kernel, st);
  return hip_status(e, "linear_tile_kernel launch");
}

}  // namespace milo
