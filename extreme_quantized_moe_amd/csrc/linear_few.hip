// The grouped 16-bit product for few rows an expert (decoding): bound by
// streaming the weights once.  A block takes 16 NT weight rows (output
// columns) of one expert; its waves share the contraction, each walking it in
// pieces of 128 with the next piece's loads in flight, straight from memory
// into matrix-core operands (no LDS on the way: a weight is used once).  Row
// counts up to 16 MT go in one walk; more rows walk again, 16 MT at a time.
// Partial sums meet in LDS in wave order.  Measured: one row of 4096 x 14336
// 19.4 us (6.1 TB/s), 32 rows over 8 experts of 14336 x 4096 160..175 us (5.4 to
// 5.9 TB/s).  Loads that pass the caches by (non-temporal) were slower: 199 us
// against 170 for 16 rows over 8 experts of 4096 x 14336.
//
// A lane's operand: row l % 16, contraction values 8 (l / 16) .. +7 of a step
// of 32: 16-byte loads, 64 contiguous bytes a row and load, four loads to 256.
// Rows of x past the expert's and columns past N are cut off by the buffer
// resources' ends: they read as zeros and cost no traffic.  LOOSE: operands
// aligned to their elements only or odd row lengths, through plain loads with
// the same bounds.
#include <algorithm>

#include "linear.hpp"

namespace milo {

constexpr int kFewRsrcWord3 = 0x00020000;
constexpr int kFewOutside = 0x7FFFFFF0;
constexpr int kFewPiece = 128;            // contraction values a wave takes at a time

template <class T, int MT, int NT, int NW, bool LOOSE>
__device__ __forceinline__ void few_rows(const LinearArgs& a, int e, int base, int m0, int rows, int n0, float* lds) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = a.K, left_n = a.N - n0 < 16 * NT ? a.N - n0 : 16 * NT;
  const int left_m = rows - m0 < 16 * MT ? rows - m0 : 16 * MT;
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((const uint16_t*)a.b + ((int64_t)e * a.N + n0) * K), 0, left_n * K * 2, kFewRsrcWord3);
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((const uint16_t*)a.a + (int64_t)(base + m0) * K), 0, left_m * K * 2, kFewRsrcWord3);
  const int at = (lane & 15) * K * 2 + (lane >> 4) * 16;   // byte offset of the lane's first piece
  f32x4 acc[MT][NT] = {};
  struct Piece {
    u32x4 w[NT][4], x[MT][4];
  };
  // LOOSE: the lane's row of a group of 16, from the lane's first value on; a
  // row past the end, whose results are not stored, reads the last one
  const int64_t n_row0 = (int64_t)e * a.N + n0, m_row0 = base + m0;
  auto row_of = [&](const void* p, int64_t row0, int group, int left) {
    const int r = group + (lane & 15);
    return (const uint16_t*)p + (row0 + (r < left ? r : left - 1)) * K + 8 * (lane >> 4);
  };
  auto load = [&](int k0, Piece& p) {
    if constexpr (LOOSE) {          // whole pieces only, no branch: all are in flight
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < 4; ++s) p.w[t][s] = load_whole(row_of(a.b, n_row0, 16 * t, left_n) + k0 + 32 * s);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int s = 0; s < 4; ++s) p.x[t][s] = load_whole(row_of(a.a, m_row0, 16 * t, left_m) + k0 + 32 * s);
      // all of them before the products of the piece before, not one by one
      // where they are used
      __builtin_amdgcn_sched_barrier(0);
      return;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const bool in = k0 + 32 * s + 8 * (lane >> 4) < K;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        p.w[t][s] = __builtin_amdgcn_raw_buffer_load_b128(rw, in ? at + (16 * t * K + k0 + 32 * s) * 2 : kFewOutside, 0, 0);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        p.x[t][s] = __builtin_amdgcn_raw_buffer_load_b128(rx, in ? at + (16 * t * K + k0 + 32 * s) * 2 : kFewOutside, 0, 0);
    }
  };
  auto use = [&](const Piece& p) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = T::mfma(__builtin_bit_cast(s16x8, p.w[j][s]), __builtin_bit_cast(s16x8, p.x[i][s]), acc[i][j]);
  };
  constexpr int kTurn = kFewPiece * NW;
  const int first = wave * kFewPiece, end = LOOSE ? K / kFewPiece * kFewPiece : K;
  if (first < end) {
    Piece p0, p1;
    load(first, p0);
    int k = first;
    for (; k + 2 * kTurn < end; k += 2 * kTurn) {
      load(k + kTurn, p1);
      use(p0);
      load(k + 2 * kTurn, p0);
      use(p1);
    }
    // the last one or two pieces: nothing is asked for past the contraction (a
    // load that is cut off whole still takes its turn)
    if (k + kTurn < end) {
      load(k + kTurn, p1);
      use(p0);
      use(p1);
    } else {
      use(p0);
    }
  }
  if (LOOSE && end < K && end / kFewPiece % NW == wave) {      // the piece that the end cuts
#pragma unroll 1
    for (int k = end; k < K; k += 32) {
      s16x8 w[NT], x[MT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
        w[t] = __builtin_bit_cast(s16x8, load_cut(row_of(a.b, n_row0, 16 * t, left_n) + k, K - k - 8 * (lane >> 4)));
#pragma unroll
      for (int t = 0; t < MT; ++t)
        x[t] = __builtin_bit_cast(s16x8, load_cut(row_of(a.a, m_row0, 16 * t, left_m) + k, K - k - 8 * (lane >> 4)));
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = T::mfma(w[j], x[i], acc[i][j]);
    }
  }
  // partial sums: lds[wave][row][16 NT columns]; lane l holds row l % 16,
  // columns 4 (l / 16) .. +3 of each product
  constexpr int kLine = 16 * NT + 4;
  __syncthreads();                                   // the previous walk's readers are done
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *(f32x4*)(lds + (wave * 16 * MT + 16 * i + (lane & 15)) * kLine + 16 * j + 4 * (lane >> 4)) = acc[i][j];
  __syncthreads();
  auto sums = [&](auto first, int at) {
    auto sum = first;
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += *(const decltype(first)*)(lds + w * 16 * MT * kLine + at);
    return sum;
  };
  for (int q = threadIdx.x; q < 16 * MT * 4 * NT; q += 64 * NW) {
    const int r = q / (4 * NT), c = q % (4 * NT) * 4;
    if (m0 + r >= rows || n0 + c + (LOOSE ? 4 : 1) > a.N) continue;
    const f32x4 sum = sums(*(const f32x4*)(lds + r * kLine + c), r * kLine + c);
    const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    finish<T, kFwd, 4, LOOSE>(a, e, (int64_t)base + m0 + r, n0 + c, v);
  }
  // the last columns where four do not fit, one a lane
  if (LOOSE && left_n % 4 != 0)
    for (int q = threadIdx.x; q < 16 * MT * 4; q += 64 * NW) {
      const int r = q / 4, c = left_n / 4 * 4 + q % 4;
      if (m0 + r >= rows || c >= left_n) continue;
      const float v = sums(lds[r * kLine + c], r * kLine + c);
      finish<T, kFwd, 1, true>(a, e, (int64_t)base + m0 + r, n0 + c, &v);
    }
}

// MT_MAX bounds the 16-row groups of one walk; an expert with fewer rows takes
// the smallest form that holds them.  Blocks along z share the walks of an
// expert that needs more than one (skewed routing: 128 rows over 66 experts of
// 1408 x 2048, 74 of them one expert's, 52 us with one block to a column
// group, 25 with one to a walk; balanced ones lose nothing to the empty blocks).
template <class T, int MT_MAX, int NT, int NW, bool LOOSE>
__global__ void __launch_bounds__(64 * NW) linear_few_kernel(LinearArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ __align__(16) float lds[NW * 16 * MT_MAX * (16 * NT + 4)];
  const int e = blockIdx.y, n0 = blockIdx.x * 16 * NT;
  const Span s = expert_span(a.offsets, e, a.rows);
  for (int m0 = 16 * MT_MAX * blockIdx.z; m0 < s.rows; m0 += 16 * MT_MAX * gridDim.z) {
    const int left = s.rows - m0;
    if (left <= 16 || MT_MAX == 1) few_rows<T, 1, NT, NW, LOOSE>(a, e, s.base, m0, s.rows, n0, lds);
    else if (left <= 32 || MT_MAX == 2) few_rows<T, MT_MAX < 2 ? 1 : 2, NT, NW, LOOSE>(a, e, s.base, m0, s.rows, n0, lds);
    else few_rows<T, MT_MAX, NT, NW, LOOSE>(a, e, s.base, m0, s.rows, n0, lds);
  }
#endif
}

// The same walk for few columns and many rows (a router): a block takes 16
// rows and 64 columns, so it is x that is streamed once and w that every
// block reads again, from the L2, which bounds it (256 blocks of 16 rows read 67
// MB of w for 16 MB of x): 4096 rows of 2048 to 64 columns 13.6 us traced alone,
// 11.3 a call among others (x alone would take 4).
template <class T, bool LOOSE>
__global__ void __launch_bounds__(512) linear_narrow_kernel(LinearArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ __align__(16) float lds[8 * 16 * (64 + 4)];
  const int id = blockIdx.x, width = (a.N + 63) / 64;
  const TileSlot s = find_slot(a.offsets, a.E, a.rows, 16, width, [&](int) { return id; });
  if (s.e < 0) return;
  few_rows<T, 1, 4, 8, LOOSE>(a, s.e, s.span.base, s.local / width * 16, s.span.rows, s.local % width * 64, lds);
#endif
}

template <class T, bool LOOSE>
static void run_few(const LinearArgs& a, hipStream_t st) {
  // With few column groups in all, eight waves share one group of 16 columns.
  // With many, four waves: two groups a block halve the traffic of x where the
  // contraction is short (66 experts of 1408 x 2048 with 4 rows: 69 us against
  // 78 with one), one group reads long rows faster (8 experts of 14336 x 4096
  // with 4 rows: 174 us against 219 with two).
  const bool wide = (int64_t)a.E * ((a.N + 31) / 32) >= 1024;
  auto walks = [&](int mt) { return std::min(kFewWalks, (a.max_rows + 16 * mt - 1) / (16 * mt)); };
#define RUN(MT, NT, NW)                                                                                         \
  hipLaunchKernelGGL((linear_few_kernel<T, MT, NT, NW, LOOSE>), dim3((a.N + 16 * NT - 1) / (16 * NT), a.E, walks(MT)), \
                     dim3(64 * NW), 0, st, a)
  const int bound = few_bound(a);
  if (bound <= 16) { if (!wide) RUN(1, 1, 8); else if (a.K >= 4096) RUN(1, 1, 4); else RUN(1, 2, 4); }
  else if (bound <= 32) { if (wide) RUN(2, 2, 4); else RUN(2, 1, 8); }
  else { if (wide) RUN(4, 2, 4); else RUN(4, 1, 8); }
#undef RUN
}

template <class T, bool LOOSE>
static void run_narrow(const LinearArgs& a, hipStream_t st) {
  const int64_t blocks = ((int64_t)(a.rows + 15) / 16 + (a.E > 1 ? a.E : 0)) * ((a.N + 63) / 64);
  hipLaunchKernelGGL((linear_narrow_kernel<T, LOOSE>), dim3((unsigned)blocks), dim3(512), 0, st, a);
}

template <class T>
static void run_any(const LinearArgs& a, bool narrow, bool loose, hipStream_t st) {
  if (narrow) { if (loose) run_narrow<T, true>(a, st); else run_narrow<T, false>(a, st); }
  else { if (loose) run_few<T, true>(a, st); else run_few<T, false>(a, st); }
}

int32_t launch_linear_few(int dtype, const LinearArgs& a, bool narrow, bool loose, hipStream_t st) {
  if (dtype == MILO_F16) run_any<F16>(a, narrow, loose, st);
  else run_any<BF16>(a, narrow, loose, st);
  return hip_status(hipGetLastError(), "linear_few_kernel launch");
}

}  // namespace milo
