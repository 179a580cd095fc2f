// Launches of the tile kernels of the grouped 16-bit product.
#include "linear_tile.hpp"

namespace milo {

template <class T, int MODE, int ACT, int BM, int BN, int WM, int WN>
static hipError_t run_tile(const LinearArgs& a, hipStream_t st) {
  const int64_t tn = ((MODE == kFwd ? a.N : a.K) + BN - 1) / BN;
  const int64_t rows = MODE == kDw ? (int64_t)a.E * ((a.N + BM - 1) / BM)
                                   : (a.rows + BM - 1) / BM + (a.E > 1 ? a.E : 0);
  // as many blocks as run at once (one or two to a compute unit), a multiple
  // of 8 so that a block's tiles stay on its XCD
  const int64_t slots = (int64_t)device_cu_count() * (BM == 256 ? 1 : 2);
  int64_t blocks = rows * tn * a.splits;
  blocks = (blocks < slots ? blocks + 7 : slots) / 8 * 8;
  if (blocks < 8) blocks = 8;
  constexpr size_t bytes = tile_lds<BM, BN>();
  const void* fn = (const void*)linear_tile_kernel<T, MODE, ACT, BM, BN, WM, WN>;
  if (bytes + sizeof(ExpertTable) > 65536) {
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((linear_tile_kernel<T, MODE, ACT, BM, BN, WM, WN>), dim3((unsigned)blocks), dim3(64 * WM * WN),
                     bytes, st, a);
  return hipGetLastError();
}

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

int32_t launch_linear_tile(int mode, int dtype, const LinearArgs& a, int kernel, hipStream_t st) {
  const hipError_t e = dtype == MILO_F16 ? run_type<F16>(mode, a, kernel, st) : run_type<BF16>(mode, a, kernel, st);
  return hip_status(e, "linear_tile_kernel launch");
}

}  // namespace milo
