// Which kernel runs a grouped 16-bit product: chosen on the host from sizes,
// types and alignment, never from device data.
#include "linear.hpp"

namespace milo {

static bool wide_access(const LinearArgs& a) {
  const uintptr_t bits = (uintptr_t)a.a | (uintptr_t)a.b | (uintptr_t)a.bias | (uintptr_t)a.mul |
                         (uintptr_t)a.residual | (uintptr_t)a.pre | (uintptr_t)a.out;
  return a.N % 8 == 0 && a.K % 8 == 0 && bits % 16 == 0;
}

LinearPlan plan_linear(int mode, const LinearArgs& a) {
  LinearPlan p = {kPlanGeneral, 1, 0};
  if (!wide_access(a)) return p;
  if (mode == kFwd && a.rows <= 64 * (int64_t)a.E) {
    p.kernel = kPlanFew;
    return p;
  }
  const int64_t m = mode == kDw ? a.N : (a.rows + a.E - 1) / a.E, n = mode == kFwd ? a.N : a.K;
  const int64_t big = a.E * ((m + 255) / 256) * ((n + 255) / 256);
  p.kernel = big >= 256 ? kPlanTile256 : kPlanTile128;
  return p;
}

int32_t launch_linear(int mode, int dtype, const LinearArgs& a, const LinearPlan& p, hipStream_t st) {
  if (p.kernel == kPlanGeneral) return launch_linear_general(mode, dtype, a, st);
  if (p.kernel == kPlanFew) return launch_linear_few(dtype, a, st);
  return launch_linear_tile(mode, dtype, a, p.kernel, st);
}

}  // namespace milo
