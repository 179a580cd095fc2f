// Which kernels run a grouped 16-bit product: chosen on the host from sizes,
// types and alignment, never from device data.
#include "linear.hpp"

namespace milo {

// 16-byte accesses everywhere: row lengths of a multiple of 8 elements and
// 16-byte aligned arrays; anything else takes the loose forms.
static bool wide_access(const LinearArgs& a) {
  const uintptr_t bits = (uintptr_t)a.a | (uintptr_t)a.b | (uintptr_t)a.bias | (uintptr_t)a.mul |
                         (uintptr_t)a.residual | (uintptr_t)a.pre | (uintptr_t)a.out;
  return a.N % 8 == 0 && a.K % 8 == 0 && bits % 16 == 0;
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Microseconds of a tile kernel, from what its steps (64 of the contraction),
// results and partial sums took on an MI355X: a step of a 256 x 256 tile 1.5,
// of a 128 x 128 tile 0.71 alone on its compute unit and 1.05 with a second
// block beside it; a tile's results 8 and 3.5 in 16 bits, 13 and 7.4 in 32
// (every compute unit writes at once); the join of a split contraction 5, and
// its reading of the partial sums 4 TB/s.  Measured: 512 x 4096 x 4096 49
// us unsplit, 38 in two, 35 in four parts on 128 x 128 tiles; 8192 x 14336 x
// 4096 936 us on 128 x 128, 700 on 256 x 256 tiles; dw of 66 experts of 1408 x
// 2048 with 31 rows on average 112 us on 128 x 128, 130 on 256 x 256 tiles, of
// 8 experts of 4096 x 14336 with 512 rows 680 and 567.
static double tile_cost(int tile, int splits, int64_t tiles, int64_t steps, int64_t results, bool wide_out,
                        int64_t cus) {
  const int64_t work = tiles * splits;
  const bool out32 = wide_out || splits > 1;
  double step, out;
  int64_t rounds;
  if (tile == 256) {
    step = 1.5;
    out = out32 ? 13 : 8;
    rounds = ceil_div(work, cus);
  } else {
    step = work <= cus ? 0.71 : 1.05;
    out = out32 ? 7.4 : 3.5;
    rounds = work <= cus ? 1 : ceil_div(work, 2 * cus);
  }
  // fewer blocks than compute units write faster each
  const double writes = rounds * out * (work < cus ? (double)work / cus : 1);
  return rounds * ceil_div(steps, splits) * step + writes + (splits > 1 ? 5 + 4e-6 * splits * results / 4 : 0);
}

LinearPlan plan_linear(int mode, const LinearArgs& a) {
  LinearPlan p = {kPlanTile128, 1, !wide_access(a), 0};
  const int64_t rows = ceil_div(a.rows, a.E);            // of an expert, on average
  if (mode == kFwd) {
    // Few rows an expert: the weights are streamed straight into the matrix
    // cores, where no expert can have many (an expert's further rows read its
    // weights again: 500 rows over 66 experts of 1408 x 2048, 305 of them one
    // expert's, 66 us, on tiles 29) and either few rows are certain (32 over 8
    // experts of 14336 x 4096: 168 us, on tiles 174), the experts are small (66
    // of 1408 x 2048, 16 rows each: 85 us, on tiles 100) or few tiles would run
    // (24 x 4096 x 4096: 13 us, on tiles 17).  Large experts take tiles (12
    // rows each of 8 x 14336 x 4096: 194 us, streamed 222), and so do odd row
    // lengths (4 rows each of 8 x 14335 x 4097: 321 us, streamed 493).
    const bool few_tiles = a.E * ceil_div(a.N, 128) < 256, small = (int64_t)a.N * a.K <= kSmallMatrixElems;
    if (rows <= 24 && a.max_rows <= 16 * kFewWalks && (few_tiles || ((a.max_rows <= 32 || small) && !p.loose))) {
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
  bool any = false;
  for (int tile = p.loose ? 128 : 256; tile >= 128; tile -= 128)
    for (int splits = 1; splits <= 8 && (splits == 1 || 2 * splits <= steps); splits *= 2) {
      const int64_t tiles = a.E * ceil_div(m, tile) * ceil_div(n, tile);
      const double c = tile_cost(tile, splits, tiles, steps, results, a.out_f32, cus);
      if (any && c >= best) continue;
      any = true;
      best = c;
      p.kernel = tile == 256 ? kPlanTile256 : kPlanTile128;
      p.splits = splits;
    }
  if (p.splits > 1) p.part_bytes = (size_t)p.splits * results * sizeof(float);
  return p;
}

int32_t launch_linear(int mode, int dtype, const LinearArgs& args, const LinearPlan& p, hipStream_t st) {
  if (p.kernel == kPlanFew || p.kernel == kPlanNarrow)
    return launch_linear_few(dtype, args, p.kernel == kPlanNarrow, p.loose, st);
  LinearArgs a = args;
  a.splits = p.splits;
  const int32_t rc = p.loose ? launch_linear_loose(mode, dtype, a, st) : launch_linear_tile(mode, dtype, a, p.kernel, st);
  return rc || p.splits == 1 ? rc : launch_linear_join(mode, dtype, a, p.loose, st);
}

}  // namespace milo
