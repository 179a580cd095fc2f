// Which kernels run a grouped 16-bit product: chosen on the host from sizes,
// types and alignment, never from device data.
#include "linear.hpp"

namespace milo {

// Rows that 16-byte accesses reach: of a multiple of 8 elements, from aligned arrays.
static bool wide_rows(int len, const void* a, const void* b = nullptr, const void* c = nullptr,
                      const void* d = nullptr, const void* e = nullptr) {
  return len % 8 == 0 && ((uintptr_t)a | (uintptr_t)b | (uintptr_t)c | (uintptr_t)d | (uintptr_t)e) % 16 == 0;
}

// Elements between the rows of a copied operand: whole 16-byte pieces, and
// where that adds little whole cache lines (a step of 64 then takes one line a
// row, not two).
static int packed_row(int len) { return len < 512 ? (len + 7) / 8 * 8 : (len + 63) / 64 * 64; }

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
// The register-staged kernel's steps took 1.2 alone and 2.0 with a second block
// beside it; a copy into whole rows its launch and 4 bytes an element at 4 TB/s.
// Measured for odd row lengths, on whole rows and register-staged: 4096 x 14335
// x 4097 over 8 experts dw 737 and 973 us, dx 1030 and 1054, forward 930 and 907;
// 512 rows of it 615 and 292 forward (the weights' copy), 420 and 395 dw; 16384
// x 1023 x 1025 dw 101 and 272; 234 x 10031 x 7544 (weights' rows whole) dx 61
// and 118.
constexpr double kCopyLaunch = 6;
static double tile_cost(int kernel, int splits, int64_t tiles, int64_t steps, int64_t results, bool wide_out,
                        int64_t cus) {
  const int64_t work = tiles * splits;
  const bool out32 = wide_out || splits > 1;
  double step, out;
  int64_t rounds;
  if (kernel == kPlanTile256) {
    step = 1.5;
    out = out32 ? 13 : 8;
    rounds = ceil_div(work, cus);
  } else {
    step = work <= cus ? 0.71 : 1.05;
    if (kernel == kPlanLoose128) step = work <= cus ? 1.2 : 2.0;
    out = out32 ? 7.4 : 3.5;
    rounds = work <= cus ? 1 : ceil_div(work, 2 * cus);
  }
  // fewer blocks than compute units write faster each
  const double writes = rounds * out * (work < cus ? (double)work / cus : 1);
  return rounds * ceil_div(steps, splits) * step + writes + (splits > 1 ? 5 + 4e-6 * splits * results / 4 : 0);
}

LinearPlan plan_linear(int mode, const LinearArgs& a) {
  // row lengths and rows of the operands
  const int len_a = mode == kFwd ? a.K : a.N, len_b = a.K, ld_a = packed_row(len_a), ld_b = packed_row(len_b);
  const int64_t rows_b = mode == kDw ? a.rows : (int64_t)a.E * a.N;
  const bool wide_a = wide_rows(len_a, a.a), wide_b = wide_rows(len_b, a.b);
  const bool wide_out = wide_rows(mode == kFwd ? a.N : a.K, a.out, a.bias, a.mul, a.residual, a.pre);
  const bool any_loose = !wide_a || !wide_b || !wide_out;
  LinearPlan p = {kPlanTile128, 1, any_loose, 0, 0, 0};
  const int64_t rows = ceil_div(a.rows, a.E);            // of an expert, on average
  if (mode == kFwd) {
    // Few rows an expert: the weights are streamed straight into the matrix
    // cores, where no expert can have many (an expert's further rows read its
    // weights again: 500 rows over 66 experts of 1408 x 2048, 305 of them one
    // expert's, 66 us, on tiles 29) and either few rows are certain (32 over 8
    // experts of 14336 x 4096: 168 us, on tiles 174), the experts are small (66
    // of 1408 x 2048, 16 rows each: 85 us, on tiles 100) or few tiles would run
    // (24 x 4096 x 4096: 13 us, on tiles 17).  Large experts take tiles (12
    // rows each of 8 x 14336 x 4096: 194 us, streamed 222), and so do rows
    // that start within a 4-byte word (4 rows each of 8 x 14335 x 4097: 318 us,
    // streamed 506; x 4098: 251 and 191).
    const bool few_tiles = a.E * ceil_div(a.N, 128) < 256, small = (int64_t)a.N * a.K <= kSmallMatrixElems;
    const bool words = a.K % 2 == 0 && ((uintptr_t)a.a | (uintptr_t)a.b) % 4 == 0;
    if (rows <= 24 && a.max_rows <= 16 * kFewWalks && (few_tiles || ((a.max_rows <= 32 || small) && words))) {
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
  const size_t a_bytes = wide_a ? 0 : whole_lines((size_t)a.rows * ld_a * 2);
  const size_t b_bytes = wide_b ? 0 : whole_lines((size_t)rows_b * ld_b * 2);
  const double copies = (wide_a ? 0 : kCopyLaunch + 5e-7 * a_bytes) + (wide_b ? 0 : kCopyLaunch + 5e-7 * b_bytes);
  double best = 0;
  bool any = false;
  for (int kernel = any_loose ? kPlanLoose128 : kPlanTile256; kernel >= kPlanTile128; --kernel)
    for (int splits = 1; splits <= 8 && (splits == 1 || 2 * splits <= steps); splits *= 2) {
      const int tile = kernel == kPlanTile256 ? 256 : 128;
      const int64_t tiles = a.E * ceil_div(m, tile) * ceil_div(n, tile);
      double c = tile_cost(kernel, splits, tiles, steps, results, a.out_f32, cus);
      if (kernel != kPlanLoose128) c += copies;
      if (any && c >= best) continue;
      any = true;
      best = c;
      p.kernel = kernel;
      p.splits = splits;
    }
  if (p.splits > 1) p.part_bytes = whole_lines((size_t)p.splits * results * sizeof(float));
  if (p.kernel != kPlanLoose128) {
    p.a_bytes = a_bytes;
    p.b_bytes = b_bytes;
    p.loose = !wide_out;
  }
  return p;
}

int32_t launch_linear(int mode, int dtype, const LinearArgs& args, const LinearPlan& p, void* workspace, bool a_packed,
                      hipStream_t st) {
  if (p.kernel == kPlanFew || p.kernel == kPlanNarrow)
    return launch_linear_few(dtype, args, p.kernel == kPlanNarrow, p.loose, st);
  LinearArgs a = args;
  a.splits = p.splits;
  a.lda = mode == kFwd ? a.K : a.N;
  a.ldb = a.K;
  char* ws = (char*)workspace;
  a.part = (float*)(ws + p.a_bytes + p.b_bytes);
  int32_t rc = MILO_OK;
  if (p.a_bytes) {
    const int len = a.lda;
    a.lda = packed_row(len);
    if (!a_packed) rc = launch_pack_rows(a.a, a.rows, len, a.lda, ws, st);
    a.a = ws;
  }
  if (p.b_bytes && !rc) {
    const int len = a.ldb;
    a.ldb = packed_row(len);
    rc = launch_pack_rows(a.b, mode == kDw ? a.rows : (int64_t)a.E * a.N, len, a.ldb, ws + p.a_bytes, st);
    a.b = ws + p.a_bytes;
  }
  if (rc) return rc;
  if (p.kernel == kPlanLoose128) rc = launch_linear_loose(mode, dtype, a, st);
  else if (p.loose) rc = launch_linear_packed(mode, dtype, a, p.kernel, st);
  else rc = launch_linear_tile(mode, dtype, a, p.kernel, st);
  return rc || p.splits == 1 ? rc : launch_linear_join(mode, dtype, a, p.loose, st);
}

}  // namespace milo
