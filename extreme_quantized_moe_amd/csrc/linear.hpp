// What the 16-bit grouped product kernels share: arguments, the rows of an
// expert, the tile order, the activations and the epilogue.
//
//   forward  C[p][n]    = sum_k x[p][k] w[e][n][k],   p of expert e; epilogue
//   dx       C[p][k]    = sum_n dy[p][n] w[e][n][k]
//   dw       C[e][n][k] = sum_p dy[p][n] x[p][k],     p over expert e's rows
//
// Each is C[m][n] = sum_c A[m][c] B[n][c].  An operand is "deep" where the
// contraction index c is the contiguous one in memory and "wide" where m (or
// n) is: forward deep x deep, dx deep x wide, dw wide x wide.
#pragma once

#include "half_types.hpp"

namespace milo {

enum { kFwd = 0, kDx = 1, kDw = 2 };

struct LinearArgs {
  const void* a;            // fwd: x; dx, dw: dy
  const void* b;            // fwd, dx: w; dw: x
  const int32_t* offsets;   // NULL: one expert owns every row
  const void* bias;         // each may be NULL; bias, mul, pre: forward only
  const void* mul;
  const void* residual;     // dx: the other gradient added
  void* pre;
  void* out;
  float* part;              // split contraction: partial sums
  int E, rows, N, K;
  int lda, ldb;             // elements between rows of a and b (tile kernels)
  int max_rows;             // host bound on an expert's rows (plan only)
  int act;
  int out_f32;              // out holds float32 instead of the 16-bit type
  int splits;               // parts of the contraction (1: not split)
};

// Expert e's rows [base, base + rows); the table is clipped to the buffer, so
// no table makes a kernel read or write outside it.
struct Span {
  int base, rows;
};

__device__ __forceinline__ Span clip_span(int lo, int hi, int total) {
  lo = lo < 0 ? 0 : lo > total ? total : lo;
  hi = hi < lo ? lo : hi > total ? total : hi;
  return {lo, hi - lo};
}

__device__ __forceinline__ Span expert_span(const int32_t* __restrict__ offsets, int e, int total) {
  if (!offsets) return {0, total};
  return clip_span(offsets[e], offsets[e + 1], total);
}

// Row tile `id` of `id = row_tile * width + column` when every expert's rows
// are cut into tiles of `tile_rows`: wave-uniform, no LDS, no barrier.  Up to
// 256 experts, four to a lane group.  total: number of ids over all experts.
struct TileSlot {
  int e;          // -1: past the last tile
  Span span;
  int local;      // id within the expert, 0 .. row_tiles * width - 1
  int row_tiles;  // of this expert
  int first;      // row tiles before this expert's
};

template <class Remap>
__device__ __forceinline__ TileSlot find_slot(const int32_t* __restrict__ offsets, int E, int total_rows,
                                              int tile_rows, int width, Remap remap) {
  TileSlot s;
  if (!offsets || E == 1) {
    s.span = expert_span(offsets, 0, total_rows);
    s.row_tiles = (s.span.rows + tile_rows - 1) / tile_rows;
    s.first = 0;
    s.local = remap(s.row_tiles * width);
    s.e = s.local >= 0 && s.local < s.row_tiles * width ? 0 : -1;
    return s;
  }
  const int lane = threadIdx.x & 63;
  int lo[4], n[4], incl[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int e = 64 * c + lane, ec = e < E ? e : E - 1;
    const Span p = clip_span(offsets[ec], offsets[ec + 1], total_rows);
    lo[c] = p.base;
    n[c] = e < E ? p.rows : 0;
  }
  int before = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    int v = (n[c] + tile_rows - 1) / tile_rows;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(v, d);
      if (lane >= d) v += u;
    }
    incl[c] = before + v;
    before = __shfl(incl[c], 63);
  }
  const int id = remap(__builtin_amdgcn_readfirstlane(before) * width);
  s.e = -1;
  s.span = {0, 0};
  s.local = s.row_tiles = s.first = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int tiles = (n[c] + tile_rows - 1) / tile_rows, first = incl[c] - tiles;
    const uint64_t hit = __ballot(id >= 0 && id >= first * width && id < incl[c] * width);
    if (hit) {
      const int src = __builtin_amdgcn_readfirstlane(__builtin_ctzll(hit));
      s.e = 64 * c + src;     // scalar values, so that what follows from them is scalar too
      s.span.base = __builtin_amdgcn_readlane(lo[c], src);
      s.span.rows = __builtin_amdgcn_readlane(n[c], src);
      s.first = __builtin_amdgcn_readlane(first, src);
      s.row_tiles = __builtin_amdgcn_readlane(tiles, src);
      s.local = id - s.first * width;
    }
  }
  return s;
}

// ---------------------------------------------------------------- activations
// Float32 values, a few instructions each: in the tile kernel's epilogue and in
// the activation gradient they run once per output on the vector units, 16
// lanes a cycle, with nothing else to hide behind.  Tails are computed without
// cancellation (sigmoid from exp(-|v|), the normal distribution from erfcx), down
// to results of 2^-126, which the exponential flushes to zero.  The exponential
// takes a rounded argument, so a tail's relative error grows with the argument a:
// at most 1.25 a + 10 roundings of 2^-24 for SILU (a = |v|), 1.25 a + 22 for GELU
// (a = v^2 / 2), 6.5 a + 12 for GELU_TANH, whose argument a = 2 sqrt(2/pi) |v +
// 0.044715 v^3| is itself computed.  With a < 88 that stays under a tenth of a
// 16-bit rounding (2^-15 against 2^-12 for fp16); float32 results show it, and a
// second word of the argument would cost the epilogue four more instructions a
// value.  Arguments are bounded where a product of 0 and infinity would appear.
// NaN stays NaN.
__device__ __forceinline__ float bounded(float v, float lo, float hi) { return v < lo ? lo : v > hi ? hi : v; }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhC = 0.79788456080286536f;       // sqrt(2 / pi)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

__device__ __forceinline__ float exp2_fast(float v) {
#ifdef __HIP_DEVICE_COMPILE__
  return __builtin_amdgcn_exp2f(v);
#else
  return v;
#endif
}

__device__ __forceinline__ float rcp_fast(float v) {
#ifdef __HIP_DEVICE_COMPILE__
  return __builtin_amdgcn_rcpf(v);
#else
  return v;
#endif
}

__device__ __forceinline__ float sigmoid(float v) {
  const float e = exp2_fast(-kLog2e * __builtin_fabsf(v));
  return (v < 0.f ? e : 1.f) * rcp_fast(1.f + e);
}

// Phi(v) of the normal distribution, and exp(-v^2 / 2).  With z = |v| / sqrt 2
// and t = 1 / (1 + z / 2): erfc(z) = exp(-z^2) erfcx(z), erfcx(z) / t a
// polynomial of degree 8 in t fitted for the smallest largest relative error
// on z <= 14 (4.5e-8; 1.3e-7 in float32), beyond which exp(-z^2) is zero.
__device__ __forceinline__ float normal_cdf(float v, float* exp_half_sq) {
  const float s = v * v, lo = __builtin_fmaf(v, v, -s);      // v^2 to twice the precision
  const float e = exp2_fast(__builtin_fmaf(s, -0.5f * kLog2e, lo * (-0.5f * kLog2e)));
  const float t = rcp_fast(__builtin_fmaf(__builtin_fabsf(v), 0.35355339059327376f, 1.f));
  float p = -0.05938772112131119f;
  p = __builtin_fmaf(p, t, 0.28612956404685974f);
  p = __builtin_fmaf(p, t, -0.49041667580604553f);
  p = __builtin_fmaf(p, t, 0.28174346685409546f);
  p = __builtin_fmaf(p, t, -0.029154308140277863f);
  p = __builtin_fmaf(p, t, 0.20375439524650574f);
  p = __builtin_fmaf(p, t, 0.24283479154109955f);
  p = __builtin_fmaf(p, t, 0.2824121117591858f);
  p = __builtin_fmaf(p, t, 0.2820843458175659f);
  const float h = 0.5f * e * (t * p);
  *exp_half_sq = e;
  return v < 0.f ? h : 1.f - h;
}

__device__ __forceinline__ float tanh_gelu_arg(float v) {
  return 2.f * kTanhC * __builtin_fmaf(0.044715f * v * v, v, v);
}

__device__ __forceinline__ float act_value(int act, float v) {
  float e;
  switch (act) {
    case MILO_ACT_RELU: return v < 0.f ? 0.f : v;
    case MILO_ACT_SILU: v = v < -1e3f ? -1e3f : v; return v * sigmoid(v);
    case MILO_ACT_GELU: v = v < -1e3f ? -1e3f : v; return v * normal_cdf(bounded(v, -1e3f, 1e3f), &e);
    case MILO_ACT_GELU_TANH: v = v < -1e3f ? -1e3f : v; return v * sigmoid(tanh_gelu_arg(bounded(v, -1e3f, 1e3f)));
    default: return v;
  }
}

// act(v) and act'(v); relu'(0) = 0.
__device__ __forceinline__ float act_slope(int act, float v, float* value) {
  const float b = bounded(v, -1e3f, 1e3f), w = v > b ? v : b;
  switch (act) {
    case MILO_ACT_RELU: *value = v < 0.f ? 0.f : v; return v > 0.f ? 1.f : v <= 0.f ? 0.f : v;
    case MILO_ACT_SILU: {
      const float g = sigmoid(b);
      *value = w * g;
      return g * __builtin_fmaf(b, 1.f - g, 1.f);
    }
    case MILO_ACT_GELU: {
      float e;
      const float cdf = normal_cdf(b, &e);
      *value = w * cdf;
      return __builtin_fmaf(b * kInvSqrt2Pi, e, cdf);
    }
    case MILO_ACT_GELU_TANH: {
      const float g = sigmoid(tanh_gelu_arg(b));
      *value = w * g;
      // d/dv of v g(2 u), u' = c (1 + 3 0.044715 v^2)
      return __builtin_fmaf(b * g * (1.f - g), 2.f * kTanhC * __builtin_fmaf(3.f * 0.044715f * b, b, 1.f), g);
    }
    default: *value = v; return 1.f;
  }
}

// ---------------------------------------------------------------- epilogue
// V consecutive columns of one row.  V > 1 needs every array's row length and
// address to allow V-wide accesses (the launcher's rule).  Forward: bias, the
// kept pre-activation, activation, gate operand, residual, all in float32,
// one rounding at each store.
template <int MODE>
__device__ __forceinline__ int64_t out_at(const LinearArgs& a, int e, int64_t row, int col) {
  return ((MODE == kDw ? (int64_t)e * a.N : 0) + row) * (MODE == kFwd ? a.N : a.K) + col;
}

template <class T, int V, bool LOOSE = false>
__device__ __forceinline__ Pack<T, V, LOOSE> load_pack(const void* p, int64_t at) {
  return *(const Pack<T, V, LOOSE>*)((const uint16_t*)p + at);
}

template <class T, int V, bool LOOSE>
__device__ __forceinline__ void add_pack(float* v, const Pack<T, V, LOOSE>& p) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] += T::up(p.v[i]);
}

template <class T, int V, bool LOOSE>
__device__ __forceinline__ void mul_pack(float* v, const Pack<T, V, LOOSE>& p) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] *= T::up(p.v[i]);
}

template <class T, int V, bool LOOSE = false>
__device__ __forceinline__ void store_pack(void* dst, int64_t at, const float* v) {
  Pack<T, V, LOOSE> o;
#pragma unroll
  for (int i = 0; i < V; ++i) o.v[i] = T::down(v[i]);
  *(Pack<T, V, LOOSE>*)((uint16_t*)dst + at) = o;
}

template <class T, int V, bool LOOSE = false>
__device__ __forceinline__ void store_out(const LinearArgs& a, int64_t at, const float* v) {
  if (a.out_f32) {
    constexpr int W = V < 4 ? V : 4;        // at most 16 bytes an access
#pragma unroll
    for (int p = 0; p < V / W; ++p) {
      Pack<F32, W, LOOSE> o;
#pragma unroll
      for (int i = 0; i < W; ++i) o.v[i] = v[p * W + i];
      *(Pack<F32, W, LOOSE>*)((float*)a.out + at + p * W) = o;
    }
  } else {
    store_pack<T, V, LOOSE>(a.out, at, v);
  }
}

template <class T, int MODE, int V, bool LOOSE = false>
__device__ __forceinline__ void finish(const LinearArgs& a, int e, int64_t row, int col, const float* v_in) {
  const int64_t at = out_at<MODE>(a, e, row, col);
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = v_in[i];
  if constexpr (MODE == kFwd) {
    if (a.bias) add_pack(v, load_pack<T, V, LOOSE>(a.bias, (int64_t)e * a.N + col));
    if (a.pre) store_pack<T, V, LOOSE>(a.pre, at, v);
    if (a.act != MILO_ACT_NONE) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_value(a.act, v[i]);
    }
    if (a.mul) mul_pack(v, load_pack<T, V, LOOSE>(a.mul, at));
  }
  if (MODE != kDw && a.residual) add_pack(v, load_pack<T, V, LOOSE>(a.residual, at));
  store_out<T, V, LOOSE>(a, at, v);
}

// 8 values from any element on.
__device__ __forceinline__ u32x4 load_whole(const uint16_t* src) {
  return __builtin_bit_cast(u32x4, *(const Pack<F16, 8, true>*)src);
}

// 8 values at src, of which the row (of at least one) has `left`, perhaps none:
// the others read as zeros.  Eight loads of two bytes without a branch, so that
// they are in flight together; those past the end read the row's last value.
__device__ __forceinline__ u32x4 load_cut(const uint16_t* src, int left) {
  Pack<F16, 8, true> p;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint16_t v = src[i < left ? i : left - 1];
    p.v[i] = i < left ? v : (uint16_t)0;
  }
  return __builtin_bit_cast(u32x4, p);
}

// ---------------------------------------------------------------- host side
constexpr int kLinearStep = 64;   // contraction values per step of the tile kernels

// How one product is run (host side; chosen from sizes, types and alignment).
struct LinearPlan {
  int kernel;          // kPlan*
  int splits;
  int loose;           // element-aligned arrays or odd row lengths: of any array, on the tile kernels of the results'
  size_t part_bytes;   // fp32 partial sums of a split contraction
  size_t a_bytes, b_bytes;   // copies of a and b in rows of a multiple of 8 elements (0: used as they are)
};
enum { kPlanFew = 0, kPlanNarrow, kPlanTile128, kPlanTile256, kPlanLoose128 };

// Workspace of a plan: [copy of a][copy of b][partial sums], each part 256-byte aligned.
inline size_t whole_lines(size_t bytes) { return (bytes + 255) / 256 * 256; }
inline size_t plan_bytes(const LinearPlan& p) { return p.a_bytes + p.b_bytes + p.part_bytes; }

constexpr int kFewWalks = 8;      // walks of 16 rows that blocks of the streaming kernel share

// Rows the streaming kernel plans an expert for: twice the average, or the
// caller's bound (a fuller expert walks its weights again).
inline int few_bound(const LinearArgs& a) {
  const int twice = (a.rows + a.E - 1) / a.E * 2;
  return a.E > 1 && twice < a.max_rows ? twice : a.max_rows;
}

LinearPlan plan_linear(int mode, const LinearArgs& a);
// a_packed: a's copy is in the workspace already
int32_t launch_linear(int mode, int dtype, const LinearArgs& a, const LinearPlan& p, void* workspace, bool a_packed,
                      hipStream_t st);
int32_t launch_linear_tile(int mode, int dtype, const LinearArgs& a, int kernel, hipStream_t st);
int32_t launch_linear_packed(int mode, int dtype, const LinearArgs& a, int kernel, hipStream_t st);
int32_t launch_pack_rows(const void* src, int64_t rows, int len, int ld, void* dst, hipStream_t st);
int32_t launch_linear_loose(int mode, int dtype, const LinearArgs& a, hipStream_t st);
int32_t launch_linear_join(int mode, int dtype, const LinearArgs& a, bool loose, hipStream_t st);
int32_t launch_linear_few(int dtype, const LinearArgs& a, bool narrow, bool loose, hipStream_t st);
size_t act_grad_workspace_bytes(int E, int N, int rows);
int32_t launch_act_grad(const void* dy, const void* pre, const void* mul, const int32_t* offsets, int E, int N,
                        int rows, int dtype, int act, void* dpre, void* dmul, float* dbias, float* part,
                        hipStream_t st);

}  // namespace milo
