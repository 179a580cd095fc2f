// Which kernels run a grouped 16-bit product: chosen on the host from sizes,
// types and alignment, never from device data.
#include "linear.hpp"

namespace milo {

// 16-byte accesses everywhere: row lengths of a multiple of 8 elements and
// 16-byte aligned arrays; anything else takes the general kernel.
static bool wide_access(const LinearArgs& a) {
  const uintptr_t bits = (uintptr_t)a.a | (uintptr_t)a.b | (uintptr_t)a.bias | (uintptr_t)a.mul |
                         (uintptr_t)a.residual | (uintptr_t)a.pre | (uintptr_t)a.out;
  return a.N % 8 == 0 && a.K % 8 == 0 && bits % 16 == 0;
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Microseconds of a tile kernel, from what its steps (64 of the contraction)
// and partial sums took on an MI355X: a step of a 256 x 256 tile 1.5; of a 128
// x 128 tile 0.71 alone on its compute unit, 1.05 with a second block beside
// it; the join of a split contraction 5, and its partial sums written and read
// at 4 TB/s.  (512 x 4096 x 4096: 49 us unsplit, 38 in two, 35 in four parts
// on 128 x 128 tiles; 8192 x 14336 x 4096: 936 us on 128 x 128, 700 on 256 x
// 256 tiles.)
static double tile_cost(int tile, int splits, int64_t tiles, int64_t steps, int64_t results, int64_t cus) {
  const int64_t work = tiles * splits;
  double step;
  int64_t rounds;
  if (tile == 256) {
    step = 1.5;
    rounds = ceil_div(work, cus);
  } else {
    step = work <= cus ? 0.71 : 1.05;
    rounds = work <= cus ? 1 : ceil_div(work, 2 * cus);
  }
  return rounds * ceil_div(steps, splits) * step + (splits > 1 ? 5 + 8e-6 * splits * results / 4 : 0);
}

LinearPlan plan_linear(int mode, const LinearArgs& a) {
  LinearPlan p = {kPlanGeneral, 1, 0};
  if (!wide_access(a)) return p;
  const int64_t rows = ceil_div(a.rows, a.E);            // of an expert, on average
  if (mode == kFwd) {
    // Few rows an expert: the weights are streamed once for every 64 rows, at
    // the memory's rate; from about 32 rows on a tile's reuse wins (4096 x
    // 4096: 32 rows 14.7 us against 16.6 on split tiles, 64 rows 22.6 against
    // 18.5).
    if (a.max_rows <= 32 || rows <= 24) {
      p.kernel = kPlanFew;
      return p;
    }
    // Few columns: 64 of a router for 4096 rows of 2048 13 us, on split tiles
    // 17; for 16384 rows 45 against 28.
    if (a.N <= 64 && (int64_t)a.rows * a.K <= 12 << 20) {
      p.kernel = kPlanNarrow;
      return p;
    }
  }
  const int64_t m = mode == kDw ? a.N : rows, n = mode == kFwd ? a.N : a.K;
  const int64_t depth = mode == kFwd ? a.K : mode == kDx ? a.N : rows, steps = ceil_div(depth, kLinearStep);
  const int64_t results = (mode == kDw ? (int64_t)a.E * a.N : a.rows) * n, cus = device_cu_count();
  double best = 0;
  for (int tile = 256; tile >= 128; tile -= 128)
    for (int splits = 1; splits <= 8 && (splits == 1 || 2 * splits <= steps); splits *= 2) {
      const int64_t tiles = a.E * ceil_div(m, tile) * ceil_div(n, tile);
      const double c = tile_cost(tile, splits, tiles, steps, results, cus);
      if (p.kernel != kPlanGeneral && c >= best) continue;
      best = c;
      p.kernel = tile == 256 ? kPlanTile256 : kPlanTile128;
      p.splits = splits;
    }
  if (p.splits > 1) p.part_bytes = (size_t)p.splits * results * sizeof(float);
  return p;
}

int32_t launch_linear(int mode, int dtype, const LinearArgs& args, const LinearPlan& p, hipStream_t st) {
  if (p.kernel == kPlanGeneral) return launch_linear_general(mode, dtype, args, st);
  if (p.kernel == kPlanFew || p.kernel == kPlanNarrow)
    return launch_linear_few(dtype, args, p.kernel == kPlanNarrow, st);
  LinearArgs a = args;
  a.splits = p.splits;
  const int32_t rc = launch_linear_tile(mode, dtype, a, p.kernel, st);
  return rc || p.splits == 1 ? rc : launch_linear_join(mode, dtype, a, st);
}

}  // namespace milo
