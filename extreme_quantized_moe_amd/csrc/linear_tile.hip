// Launches of the tile kernels of the grouped 16-bit product.
#include "linear_tile.hpp"

namespace milo {

template <class T, int MODE, int BM, int BN, int WM, int WN>
static hipError_t run_tile(const LinearArgs& a, hipStream_t st) {
  const int64_t tn = ((MODE == kFwd ? a.N : a.K) + BN - 1) / BN;
  const int64_t rows = MODE == kDw ? (int64_t)a.E * ((a.N + BM - 1) / BM)
                                   : (a.rows + BM - 1) / BM + (a.E > 1 ? a.E : 0);
  const int64_t blocks = (rows * tn + 7) / 8 * 8;      // a whole turn over the XCDs
  constexpr size_t bytes = tile_lds<BM, BN>();
  const void* fn = (const void*)linear_tile_kernel<T, MODE, BM, BN, WM, WN>;
  if (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((linear_tile_kernel<T, MODE, BM, BN, WM, WN>), dim3((unsigned)blocks, (unsigned)a.splits),
                     dim3(64 * WM * WN), bytes, st, a);
  return hipGetLastError();
}

template <class T, int MODE>
static hipError_t run_mode(const LinearArgs& a, int kernel, hipStream_t st) {
  return kernel == kPlanTile256 ? run_tile<T, MODE, 256, 256, 2, 4>(a, st)
                                : run_tile<T, MODE, 128, 128, 2, 2>(a, st);
}

int32_t launch_linear_tile(int mode, int dtype, const LinearArgs& a, int kernel, hipStream_t st) {
  hipError_t e;
#define RUN(T)                                             \
  (mode == kFwd ? run_mode<T, kFwd>(a, kernel, st)         \
   : mode == kDx ? run_mode<T, kDx>(a, kernel, st) : run_mode<T, kDw>(a, kernel, st))
  if (dtype == MILO_F16) e = RUN(F16);
  else e = RUN(BF16);
#undef RUN
  return hip_status(e, "linear_tile_kernel launch");
}

}  // namespace milo
