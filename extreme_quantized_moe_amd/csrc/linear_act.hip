// Gradient through the epilogue of the grouped product: with
//   y = act(pre) mul + residual,  pre = x W^T + bias:
//   dpre = dy mul act'(pre),  dmul = dy act(pre),
//   dbias[e] = sum of dpre (before its rounding) over expert e's rows.
// Bound by HBM (dy, pre and mul read once, dpre and dmul written once): 8192 x
// 14336 bf16 with gate operand 210 to 222 us, 5.3 to 5.6 TB/s; with bias gradients
// of one expert 221, and 28 for the sum of its 256 row groups.  8192 x 14335 goes by
// 2 bytes an access: 257 and 350.
#include "linear.hpp"

namespace milo {

template <class T, int V, bool MUL>
__device__ __forceinline__ void act_grad_piece(int act, const Pack<T, V>& g, const Pack<T, V>& p, const Pack<T, V>& m,
                                               float* d, Pack<T, V>* dpre, Pack<T, V>* dmul) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float value;
    const float gi = T::up(g.v[i]);
    d[i] = gi * act_slope(act, T::up(p.v[i]), &value);
    if (MUL) {
      d[i] *= T::up(m.v[i]);
      dmul->v[i] = T::down(gi * value);
    }
    dpre->v[i] = T::down(d[i]);
  }
}

// In both kernels dpre and dmul may be the buffers of dy, pre or mul, so none of
// the five is `restrict`: a thread reads all it needs of an element before it
// writes there, and no other thread touches that element.

// ---- without bias gradients the experts' rows are one flat run of elements
template <class T, int V, bool MUL>
__global__ void __launch_bounds__(256) act_grad_kernel(const uint16_t* dy, const uint16_t* pre, const uint16_t* mul,
                                                       const int32_t* __restrict__ offsets, int E, int N, int rows,
                                                       int act, uint16_t* dpre, uint16_t* dmul) {
  typedef Pack<T, V> P;
  const Span s = offsets ? clip_span(offsets[0], offsets[E], rows) : Span{0, rows};
  const int64_t first = (int64_t)s.base * N / V, count = (int64_t)s.rows * N / V;   // V divides N
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const P g = ((const P*)dy)[first + i], p = ((const P*)pre)[first + i];
    P m = g, o, om;
    if (MUL) m = ((const P*)mul)[first + i];
    float d[V];
    act_grad_piece<T, V, MUL>(act, g, p, m, d, &o, &om);
    ((P*)dpre)[first + i] = o;
    if (MUL) ((P*)dmul)[first + i] = om;
  }
}

// ---- with bias gradients a block takes kActRows rows of one expert: its
// threads are 2^lg column pieces by 256 / 2^lg rows, each sums its rows in
// order, and the row groups are joined in LDS in order: part[tile][N].  A thread
// asks for kActTurns of its rows at a time, before it writes any of them.
constexpr int kActRows = 32, kActTurns = 4;

template <class T, int V, bool MUL>
__global__ void __launch_bounds__(256) act_grad_bias_kernel(const uint16_t* dy, const uint16_t* pre,
                                                            const uint16_t* mul,
                                                            const int32_t* __restrict__ offsets, int E, int N,
                                                            int rows, int act, int lg, uint16_t* dpre,
                                                            uint16_t* dmul, float* __restrict__ part) {
  typedef Pack<T, V> P;
  __shared__ float sums[256 * V];
  const int id = blockIdx.y;
  const TileSlot s = find_slot(offsets, E, rows, kActRows, 1, [&](int) { return id; });
  if (s.e < 0) return;
  const int pieces = N / V, across = 1 << lg, down = 256 >> lg;
  const int c = blockIdx.x * across + (threadIdx.x & (across - 1)), rg = threadIdx.x >> lg;
  const int r0 = s.local * kActRows;
  const int r1 = r0 + kActRows < s.span.rows ? r0 + kActRows : s.span.rows;
  float total[V];
#pragma unroll
  for (int i = 0; i < V; ++i) total[i] = 0.f;
  if (c < pieces)
    for (int r = r0 + rg; r < r1; r += kActTurns * down) {
      P g[kActTurns], p[kActTurns], m[kActTurns];
      const int64_t first = (int64_t)(s.span.base + r) * pieces + c, step = (int64_t)down * pieces;
#pragma unroll
      for (int t = 0; t < kActTurns; ++t) {
        const int64_t at = first + (r + t * down < r1 ? t : 0) * step;   // past the last row: this one again
        g[t] = ((const P*)dy)[at];
        p[t] = ((const P*)pre)[at];
        m[t] = MUL ? ((const P*)mul)[at] : g[t];
      }
#pragma unroll
      for (int t = 0; t < kActTurns; ++t) {
        if (r + t * down >= r1) break;
        float d[V];
        P o, om;
        act_grad_piece<T, V, MUL>(act, g[t], p[t], m[t], d, &o, &om);
        ((P*)dpre)[first + t * step] = o;
        if (MUL) ((P*)dmul)[first + t * step] = om;
#pragma unroll
        for (int i = 0; i < V; ++i) total[i] += d[i];
      }
    }
#pragma unroll
  for (int i = 0; i < V; ++i) sums[threadIdx.x * V + i] = total[i];
  __syncthreads();
  if (rg == 0 && c < pieces) {
    for (int k = 1; k < down; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) total[i] += sums[(threadIdx.x + k * across) * V + i];
#pragma unroll
    for (int i = 0; i < V; ++i) part[(int64_t)id * N + (int64_t)c * V + i] = total[i];
  }
}

// dbias[e][n]: expert e's tiles in order, four waves a quarter each.  A table
// that is not non-decreasing could name more tiles than there are: bounded.
__global__ void __launch_bounds__(256) bias_sum_kernel(const float* __restrict__ part,
                                                       const int32_t* __restrict__ offsets, int E, int N, int rows, int all_tiles,
                                                       float* __restrict__ dbias) {
  __shared__ float join[256];
  const int e = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int first = 0;
  const Span mine = expert_span(offsets, e, rows);
  if (offsets) {
    int before = 0;
    for (int i = lane; i < e; i += 64) {
      const Span p = clip_span(offsets[i], offsets[i + 1], rows);
      before += (p.rows + kActRows - 1) / kActRows;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) before += __shfl_xor(before, d);
    first = before;
  }
  int tiles = (mine.rows + kActRows - 1) / kActRows;
  if (first + tiles > all_tiles) tiles = first < all_tiles ? all_tiles - first : 0;
  const int n = blockIdx.x * 64 + lane;
  const int each = (tiles + 3) / 4, lo = wave * each, hi = lo + each < tiles ? lo + each : tiles;
  float sum = 0.f;
  if (n < N)
    for (int i = lo; i < hi; ++i) sum += part[(int64_t)(first + i) * N + n];
  join[threadIdx.x] = sum;
  __syncthreads();
  if (wave == 0 && n < N)
    dbias[(int64_t)e * N + n] = ((join[lane] + join[64 + lane]) + join[128 + lane]) + join[192 + lane];
}

static int64_t act_tiles(int E, int rows) { return (rows + kActRows - 1) / kActRows + (E > 1 ? E : 0); }

size_t act_grad_workspace_bytes(int E, int N, int rows) { return (size_t)act_tiles(E, rows) * N * sizeof(float); }

template <class T, int V, bool MUL>
static void run_act_grad(const void* dy, const void* pre, const void* mul, const int32_t* offsets, int E, int N,
                         int rows, int act, void* dpre, void* dmul, float* dbias, float* part, hipStream_t st) {
  const uint16_t *g = (const uint16_t*)dy, *p = (const uint16_t*)pre, *m = (const uint16_t*)mul;
  if (!dbias) {
    int64_t blocks = ((int64_t)rows * N / V + 255) / 256;
    if (blocks > 16384) blocks = 16384;
    if (blocks)
      hipLaunchKernelGGL((act_grad_kernel<T, V, MUL>), dim3((unsigned)blocks), dim3(256), 0, st, g, p, m, offsets, E,
                         N, rows, act, (uint16_t*)dpre, (uint16_t*)dmul);
    return;
  }
  const int pieces = N / V;
  // at most 64 pieces across: four row groups share a block's rows (1031 x 1403
  // at odd row lengths: 13.7 us with one group of 256 pieces, 7.6 with four)
  int lg = 0;
  while (lg < 6 && (1 << lg) < pieces) ++lg;
  if (rows)
    hipLaunchKernelGGL((act_grad_bias_kernel<T, V, MUL>),
                       dim3((unsigned)((pieces + (1 << lg) - 1) >> lg), (unsigned)act_tiles(E, rows)), dim3(256), 0,
                       st, g, p, m, offsets, E, N, rows, act, lg, (uint16_t*)dpre, (uint16_t*)dmul, part);
  hipLaunchKernelGGL(bias_sum_kernel, dim3((unsigned)((N + 63) / 64), (unsigned)E), dim3(256), 0, st, part, offsets,
                     E, N, rows, (int)act_tiles(E, rows), dbias);
}

int32_t launch_act_grad(const void* dy, const void* pre, const void* mul, const int32_t* offsets, int E, int N,
                        int rows, int dtype, int act, void* dpre, void* dmul, float* dbias, float* part,
                        hipStream_t st) {
  int bytes = access_bytes((size_t)N * 2, dy, pre, dpre, mul);
  const int more = access_bytes((size_t)N * 2, dmul);
  if (more < bytes) bytes = more;
#define RUN(T, V)                                                                                            \
  do {                                                                                                       \
    if (mul) run_act_grad<T, V, true>(dy, pre, mul, offsets, E, N, rows, act, dpre, dmul, dbias, part, st);   \
    else run_act_grad<T, V, false>(dy, pre, mul, offsets, E, N, rows, act, dpre, dmul, dbias, part, st);      \
  } while (0)
  if (dtype == MILO_F16) {
    if (bytes == 16) RUN(F16, 8); else if (bytes == 4) RUN(F16, 2); else RUN(F16, 1);
  } else {
    if (bytes == 16) RUN(BF16, 8); else if (bytes == 4) RUN(BF16, 2); else RUN(BF16, 1);
  }
#undef RUN
  return hip_status(hipGetLastError(), "act_grad_kernel launch");
}

}  // namespace milo
