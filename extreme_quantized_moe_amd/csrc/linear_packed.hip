// The tile kernels for results of any alignment and row length, and copies of
// operands that loads straight into LDS cannot take.
//
// Such a load moves 16 bytes from a 16-byte boundary, so rows have to start on
// one.  An operand whose rows do not is copied once into rows of a multiple of
// 8 elements, zeros behind each row's end: 4 bytes of traffic an element, where
// the register-staged kernel pays twice a tile kernel's time a product.
#include "linear_tile.hpp"

namespace milo {

// One piece of 8 elements a thread and turn, kTurns of them in flight.
constexpr int kTurns = 4;
__global__ void __launch_bounds__(256) pack_rows_kernel(const uint16_t* __restrict__ src, int64_t rows, int len, int ld,
                                                        uint16_t* __restrict__ dst) {
  const int per = ld / 8;
  const int64_t stride = (int64_t)gridDim.x * 256, first = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t step_row = stride / per;
  const int step_col = (int)(stride - step_row * per);
  int64_t row = first / per;
  int col = (int)(first - row * per);
  while (row < rows) {
    u32x4 v[kTurns];
    int64_t at[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
      at[t] = -1;
      if (row < rows) {
        at[t] = row * ld + col * 8;
        v[t] = col * 8 + 8 <= len ? load_whole(src + row * len + col * 8)
                                   : load_cut(src + row * len + col * 8, len - col * 8);
      }
      row += step_row;
      col += step_col;
      if (col >= per) {
        col -= per;
        ++row;
      }
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t)
      if (at[t] >= 0) *(u32x4*)(dst + at[t]) = v[t];
  }
}

int32_t launch_pack_rows(const void* src, int64_t rows, int len, int ld, void* dst, hipStream_t st) {
  const int64_t want = (rows * (ld / 8) + 256 * kTurns - 1) / (256 * kTurns), most = (int64_t)device_cu_count() * 16;
  hipLaunchKernelGGL(pack_rows_kernel, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st,
                     (const uint16_t*)src, rows, len, ld, (uint16_t*)dst);
  return hip_status(hipGetLastError(), "pack_rows_kernel launch");
}

template <class T, int MODE>
static hipError_t run_packed(const LinearArgs& a, int kernel, hipStream_t st) {
  return kernel == kPlanTile256 ? run_tile<T, MODE, MILO_ACT_NONE, 256, 256, 2, 4, true>(a, st)
                                : run_tile<T, MODE, MILO_ACT_NONE, 128, 128, 2, 2, true>(a, st);
}

template <class T>
static hipError_t run_type(int mode, const LinearArgs& a, int kernel, hipStream_t st) {
  if (mode == kFwd) return run_packed<T, kFwd>(a, kernel, st);
  return mode == kDx ? run_packed<T, kDx>(a, kernel, st) : run_packed<T, kDw>(a, kernel, st);
}

int32_t launch_linear_packed(int mode, int dtype, const LinearArgs& a, int kernel, hipStream_t st) {
  const hipError_t e = dtype == MILO_F16 ? run_type<F16>(mode, a, kernel, st) : run_type<BF16>(mode, a, kernel, st);
  return hip_status(e, "linear_tile_kernel launch");
}

}  // namespace milo
