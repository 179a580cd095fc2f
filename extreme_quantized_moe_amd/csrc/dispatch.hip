// Rows to the experts and back, and the gradients.
// [talk] = "MiLo: Efficient Quantized MoE Inference with Mixture of Low-Rank
// Compensators" (MLSys 2025 talk write-up), Background: each token activates
// a subset of the experts and its output combines theirs.
//
// pos[t * slots + j] is the row of pair (t, j) in the expert-ordered buffer,
// or a negative value for a dropped pair:
//   permute         y[pos] = x[t]
//   permute grad    dx[t] = sum_j dy[pos]          (= unpermute with weights 1)
//   unpermute       out[t] = sum_j w[t, j] y[pos]
//   unpermute grad  dy[pos] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[pos]>
// All are bound by HBM: every row is read or written once, and the kernels
// are driven by tokens, so a token's row is read once for all its slots.
// Sums run in float32 in a fixed order (slots, then lanes, then waves) and
// are rounded once.  A position at or past `rows` counts as dropped, so no
// table makes a kernel touch memory outside the buffers.  Measured (MI355X, a
// large copy runs at 4.7 TB/s): 4096 rows of 4096 bf16 values to two slots each
// 16 us and back 17 (5.9 TB/s: part of it stays in the last-level cache); 8192
// rows of 2048 over eight slots, both gradients 130 us (4.5 TB/s) and 67 (4.5).
#include "half_types.hpp"

namespace milo {

// ---- permute: a thread moves one V-wide piece of a token's row per step.
// A block holds 256 / tpt tokens, tpt = threads per token (a power of two).
// MS bounds the slots, so their positions stay in registers.
template <class T, int V, int MS>
__global__ void __launch_bounds__(256) permute_kernel(const typename T::store* __restrict__ x,
                                                      const int32_t* __restrict__ pos, int64_t tokens, int slots,
                                                      int pieces, int64_t rows, int tpt_log2,
                                                      typename T::store* __restrict__ y) {
  typedef Pack<T, V> P;
  const int tpt = 1 << tpt_log2;
  const int64_t t = (int64_t)blockIdx.x * (256 >> tpt_log2) + (threadIdx.x >> tpt_log2);
  if (t >= tokens) return;
  int64_t dst[MS];
#pragma unroll
  for (int j = 0; j < MS; ++j) dst[j] = j < slots ? pos[t * slots + j] : -1;
  const P* src = (const P*)x + t * pieces;
  for (int c = blockIdx.y * tpt + (threadIdx.x & (tpt - 1)); c < pieces; c += gridDim.y * tpt) {
    const P v = src[c];
#pragma unroll
    for (int j = 0; j < MS; ++j)
      if (dst[j] >= 0 && dst[j] < rows) ((P*)y)[dst[j] * pieces + c] = v;
  }
}

// ---- unpermute: the same shape, a weighted sum over the slots.
template <class T, int V, int MS, bool W>
__global__ void __launch_bounds__(256) unpermute_kernel(const typename T::store* __restrict__ y,
                                                        const int32_t* __restrict__ pos,
                                                        const float* __restrict__ slot_w, int64_t tokens, int slots,
                                                        int pieces, int64_t rows, int tpt_log2,
                                                        typename T::store* __restrict__ out) {
  typedef Pack<T, V> P;
  const int tpt = 1 << tpt_log2;
  const int64_t t = (int64_t)blockIdx.x * (256 >> tpt_log2) + (threadIdx.x >> tpt_log2);
  if (t >= tokens) return;
  int64_t src[MS];
  float w[MS];
#pragma unroll
  for (int j = 0; j < MS; ++j) {
    src[j] = j < slots ? pos[t * slots + j] : -1;
    w[j] = W && j < slots ? slot_w[t * slots + j] : 1.f;
  }
  for (int c = blockIdx.y * tpt + (threadIdx.x & (tpt - 1)); c < pieces; c += gridDim.y * tpt) {
    P v[MS];
#pragma unroll
    for (int j = 0; j < MS; ++j)            // every load issued before the sum
      if (src[j] >= 0 && src[j] < rows) v[j] = ((const P*)y)[src[j] * pieces + c];
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
    for (int j = 0; j < MS; ++j)
      if (src[j] >= 0 && src[j] < rows) {   // a dropped pair adds nothing, whatever its weight
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += W ? w[j] * T::up(v[j].v[i]) : T::up(v[j].v[i]);
      }
    P o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.v[i] = T::down(acc[i]);
    ((P*)out)[t * pieces + c] = o;
  }
}

// ---- unpermute gradient: WPT waves per token walk its row; each lane keeps
// one partial dot product per slot, joined over lanes (and waves) at the end.
template <class T, int V, int MS, bool W, int WPT>
__global__ void __launch_bounds__(256) unpermute_grad_kernel(
    const typename T::store* __restrict__ dout, const typename T::store* __restrict__ y,
    const int32_t* __restrict__ pos, const float* __restrict__ slot_w, int64_t tokens, int slots, int pieces,
    int64_t rows, typename T::store* __restrict__ dy, float* __restrict__ dw) {
  typedef Pack<T, V> P;
  __shared__ float part[4][MS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * (4 / WPT) + wave / WPT;
  const bool live = t < tokens;             // no early return: waves meet at a barrier
  int64_t at[MS];
  float w[MS], dot[MS];
#pragma unroll
  for (int j = 0; j < MS; ++j) {
    at[j] = live && j < slots ? pos[t * slots + j] : -1;
    w[j] = W && live && j < slots ? slot_w[t * slots + j] : 1.f;
    dot[j] = 0.f;
  }
  if (live)
    for (int c = (wave % WPT) * 64 + lane; c < pieces; c += 64 * WPT) {
      const P g = ((const P*)dout)[t * pieces + c];
      P v[MS];
#pragma unroll
      for (int j = 0; j < MS; ++j)
        if (at[j] >= 0 && at[j] < rows) v[j] = ((const P*)y)[at[j] * pieces + c];
#pragma unroll
      for (int j = 0; j < MS; ++j)
        if (at[j] >= 0 && at[j] < rows) {
          P o;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float gi = T::up(g.v[i]);
            dot[j] = __builtin_fmaf(gi, T::up(v[j].v[i]), dot[j]);
            o.v[i] = T::down(W ? w[j] * gi : gi);
          }
          ((P*)dy)[at[j] * pieces + c] = o;
        }
    }
  if (!dw) return;                          // uniform over the grid
#pragma unroll
  for (int j = 0; j < MS; ++j) {
#pragma unroll
    for (int d = 32; d; d >>= 1) dot[j] += __shfl_xor(dot[j], d);
  }
  if constexpr (WPT == 1) {
    float mine = 0.f;
#pragma unroll
    for (int j = 0; j < MS; ++j) mine = lane == j ? dot[j] : mine;
    if (live && lane < slots) dw[t * slots + lane] = mine;
  } else {
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < MS; ++j) part[wave][j] = dot[j];
    }
    __syncthreads();
    if (live && wave % WPT == 0 && lane < slots) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < WPT; ++k) sum += part[wave + k][lane];
      dw[t * slots + lane] = sum;
    }
  }
}

// ---- gradient of the routed weights (softmax, top k): one wave per token.
//   renormalized: w = softmax over the picks: dl[i] = w_i (g_i - sum_j w_j g_j)
//   plain:        w = p[picks], p = softmax over all E experts:
//                 dl[e] = p_e (g_e [e picked] - sum_j p_j g_j)
__global__ void __launch_bounds__(256) route_grad_kernel(const float* __restrict__ dslot_w,
                                                         const float* __restrict__ logits,
                                                         const int32_t* __restrict__ ids, int64_t tokens, int E,
                                                         int k, int slots, int renorm, float* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= tokens) return;
  float l[4], g[4];                          // experts lane, lane + 64, ...: up to 256
  bool pick[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int e = 64 * c + lane;
    l[c] = e < E ? logits[t * E + e] : -__builtin_inff();
    g[c] = 0.f;
    pick[c] = false;
  }
  // lane j holds pick j: the picks are one load, not one after the other
  const int my_id = lane < k ? ids[t * k + lane] : -1;
  const float my_g = lane < k ? dslot_w[t * slots + lane] : 0.f;
  for (int j = 0; j < k; ++j) {
    const int id = __shfl(my_id, j);
    const float gj = __shfl(my_g, j);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (64 * c + lane == id) {
        g[c] = gj;
        pick[c] = true;
      }
  }
  float m = -__builtin_inff();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (64 * c + lane < E && (!renorm || pick[c])) m = fmaxf(m, l[c]);
#pragma unroll
  for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  float p[4], sum = 0.f, dot = 0.f;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    p[c] = 64 * c + lane < E && (!renorm || pick[c]) ? expf(l[c] - m) : 0.f;
    sum += p[c];
    dot += pick[c] ? p[c] * g[c] : 0.f;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    sum += __shfl_xor(sum, d);
    dot += __shfl_xor(dot, d);
  }
  const float inv = 1.f / sum;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int e = 64 * c + lane;
    if (e < E) dlogits[t * E + e] = p[c] == 0.f ? 0.f : p[c] * inv * (g[c] - dot * inv);
  }
}

// ---------------------------------------------------------------- launchers
struct RowGrid {
  dim3 grid;
  int tpt_log2;
};

// Threads per token: a power of two up to 256 that covers the row's pieces.
// With few tokens the row is cut over blockIdx.y instead of walked by the
// thread, so that a decoding step's 16 rows still spread over the chip.
static RowGrid row_grid(int64_t tokens, int pieces) {
  int lg = 0;
  while (lg < 8 && (1 << lg) < pieces) ++lg;
  const int64_t gx = (tokens + (256 >> lg) - 1) / (256 >> lg);
  const int cuts = (pieces + (1 << lg) - 1) >> lg;
  int64_t gy = (4096 + gx - 1) / gx;
  if (gy > cuts) gy = cuts;
  return {dim3((unsigned)gx, (unsigned)gy), lg};
}

#define MILO_SLOTS(MS_MAX, ...)                       \
  do {                                                \
    if (slots <= 2) { constexpr int MS = 2; __VA_ARGS__; }        \
    else if (slots <= 4) { constexpr int MS = 4; __VA_ARGS__; }   \
    else if (slots <= 8) { constexpr int MS = 8; __VA_ARGS__; }   \
    else { constexpr int MS = 16; __VA_ARGS__; }      \
  } while (0)

template <class T, int V>
static void run_permute(const void* x, const int32_t* pos, int64_t tokens, int slots, int H, int64_t rows, void* y,
                        hipStream_t st) {
  typedef typename T::store S;
  const int pieces = H / V;
  const RowGrid g = row_grid(tokens, pieces);
  MILO_SLOTS(16, hipLaunchKernelGGL((permute_kernel<T, V, MS>), g.grid, dim3(256), 0, st, (const S*)x, pos, tokens,
                                    slots, pieces, rows, g.tpt_log2, (S*)y));
}

template <class T, int V, bool W>
static void run_unpermute(const void* y, const int32_t* pos, const float* w, int64_t tokens, int slots, int H,
                          int64_t rows, void* out, hipStream_t st) {
  typedef typename T::store S;
  const int pieces = H / V;
  const RowGrid g = row_grid(tokens, pieces);
  MILO_SLOTS(16, hipLaunchKernelGGL((unpermute_kernel<T, V, MS, W>), g.grid, dim3(256), 0, st, (const S*)y, pos, w,
                                    tokens, slots, pieces, rows, g.tpt_log2, (S*)out));
}

template <class T, int V, bool W>
static void run_unpermute_grad(const void* dout, const void* y, const int32_t* pos, const float* w, int64_t tokens,
                               int slots, int H, int64_t rows, void* dy, float* dw, hipStream_t st) {
  typedef typename T::store S;
  const int pieces = H / V;
  // four waves to a token while the tokens alone do not fill the chip (256
  // compute units x 8 waves) and the row is long enough to share
  if (tokens < 2048 && pieces > 64)
    MILO_SLOTS(16, hipLaunchKernelGGL((unpermute_grad_kernel<T, V, MS, W, 4>), dim3((unsigned)tokens), dim3(256), 0,
                                      st, (const S*)dout, (const S*)y, pos, w, tokens, slots, pieces, rows, (S*)dy,
                                      dw));
  else
    MILO_SLOTS(16, hipLaunchKernelGGL((unpermute_grad_kernel<T, V, MS, W, 1>), dim3((unsigned)((tokens + 3) / 4)),
                                      dim3(256), 0, st, (const S*)dout, (const S*)y, pos, w, tokens, slots, pieces,
                                      rows, (S*)dy, dw));
}

// Calls F<T, V>(args) for the type and the widest access the operands allow.
#define MILO_BY_TYPE(F, ...)                                                                       \
  do {                                                                                             \
    if (dtype == MILO_F32) { if (bytes == 16) F(F32, 4, __VA_ARGS__); else F(F32, 1, __VA_ARGS__); } \
    else if (dtype == MILO_F16) {                                                                  \
      if (bytes == 16) F(F16, 8, __VA_ARGS__); else if (bytes == 4) F(F16, 2, __VA_ARGS__);          \
      else F(F16, 1, __VA_ARGS__);                                                                 \
    } else {                                                                                       \
      if (bytes == 16) F(BF16, 8, __VA_ARGS__); else if (bytes == 4) F(BF16, 2, __VA_ARGS__);        \
      else F(BF16, 1, __VA_ARGS__);                                                                \
    }                                                                                              \
  } while (0)

static size_t elem_bytes(int dtype) { return dtype == MILO_F32 ? 4 : 2; }

// Tokens of one launch: it takes fewer than 2^32 threads, and a token up to
// 256.  (unpermute_grad takes 64 a token from 2048 on.)
constexpr int64_t kMostTokens = 1 << 23;

// run(first token, tokens) for every launch's share.
template <class Run>
static void by_launches(int64_t tokens, Run run) {
  for (int64_t t = 0; t < tokens; t += kMostTokens) run(t, tokens - t < kMostTokens ? tokens - t : kMostTokens);
}

int32_t launch_permute(const void* x, const int32_t* pos, int64_t tokens, int slots, int H, int64_t rows, int dtype,
                       void* y, hipStream_t st) {
  const int bytes = access_bytes(H * elem_bytes(dtype), x, y);
#define RUN(T, V, ...) run_permute<T, V>(__VA_ARGS__)
  by_launches(tokens, [&](int64_t t, int64_t n) {
    MILO_BY_TYPE(RUN, (const char*)x + t * H * elem_bytes(dtype), pos + t * slots, n, slots, H, rows, y, st);
  });
#undef RUN
  return hip_status(hipGetLastError(), "permute_kernel launch");
}

int32_t launch_unpermute(const void* y, const int32_t* pos, const float* w, int64_t tokens, int slots, int H,
                         int64_t rows, int dtype, void* out, hipStream_t st) {
  const int bytes = access_bytes(H * elem_bytes(dtype), y, out);
#define RUN(T, V, ...)                            \
  do {                                            \
    if (w) run_unpermute<T, V, true>(__VA_ARGS__); \
    else run_unpermute<T, V, false>(__VA_ARGS__);  \
  } while (0)
  by_launches(tokens, [&](int64_t t, int64_t n) {
    MILO_BY_TYPE(RUN, y, pos + t * slots, w ? w + t * slots : w, n, slots, H, rows,
                 (char*)out + t * H * elem_bytes(dtype), st);
  });
#undef RUN
  return hip_status(hipGetLastError(), "unpermute_kernel launch");
}

int32_t launch_unpermute_grad(const void* dout, const void* y, const int32_t* pos, const float* w, int64_t tokens,
                              int slots, int H, int64_t rows, int dtype, void* dy, float* dw, hipStream_t st) {
  const int bytes = access_bytes(H * elem_bytes(dtype), dout, y, dy);
#define RUN(T, V, ...)                                 \
  do {                                                 \
    if (w) run_unpermute_grad<T, V, true>(__VA_ARGS__); \
    else run_unpermute_grad<T, V, false>(__VA_ARGS__);  \
  } while (0)
  MILO_BY_TYPE(RUN, dout, y, pos, w, tokens, slots, H, rows, dy, dw, st);
#undef RUN
  return hip_status(hipGetLastError(), "unpermute_grad_kernel launch");
}

int32_t launch_route_grad(const float* dslot_w, const float* logits, const int32_t* ids, int64_t tokens, int E, int k,
                          int S, int renorm, float* dlogits, hipStream_t st) {
  hipLaunchKernelGGL(route_grad_kernel, dim3((unsigned)((tokens + 3) / 4)), dim3(256), 0, st, dslot_w, logits, ids,
                     tokens, E, k, k + S, renorm, dlogits);
  return hip_status(hipGetLastError(), "route_grad_kernel launch");
}

}  // namespace milo
