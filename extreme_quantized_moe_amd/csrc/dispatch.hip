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
// large copy runs at 4.7 to 4.9 TB/s): 4096 rows of 4096 bf16 values to two slots
// each 17 us and back 18 (5.9 TB/s: part of it stays in the last-level cache);
// 8192 rows of 2048 over eight slots, gradient of the way back 128 us (4.5 TB/s),
// of the way there 67 with pairs spread at random (4.5) and 86 with the few
// destinations of skewed experts (3.5: its blocks live for one token, with two
// dependent loads and a store).  Rows of 2047 values go by 2 bytes an access: there
// 132 us (2048: 61), back 69 (80), gradients 217 (143) and 66 (69).
#include "half_types.hpp"

namespace milo {

// ---- rows that no pair names, as zeros (where the caller asks for it: the
// zeros that a gradient of the experts' rows needs there).  Which they are is
// known only from the whole table, so the first blocks of a launch (Zeroing)
// each scan it for a slice of the rows, mark those it names in LDS and clear the
// others, beside the blocks that move rows: no launch and no scratch of its own.
constexpr int kSliceRows = 1 << 15;        // at most, a multiple of 32

struct Zeroing {
  int blocks, slice;                       // blocks: 0 to leave those rows as they are
  int64_t pairs;
};

template <class P>
__device__ __forceinline__ void zero_free_rows(const int32_t* __restrict__ pos, const Zeroing& z, int64_t rows,
                                               int pieces, P* __restrict__ y) {
  struct alignas(4) Four {
    int32_t v[4];
  };
  constexpr int kAhead = 8;
  __shared__ uint32_t named[kSliceRows / 32];
  const int64_t first = (int64_t)blockIdx.x * z.slice;
  const int here = rows - first < z.slice ? (int)(rows - first) : z.slice;
  for (int i = threadIdx.x; i < z.slice / 32; i += 256) named[i] = 0;
  __syncthreads();
  for (int64_t i = 4 * threadIdx.x; i < z.pairs; i += 1024 * kAhead) {
    Four f[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int64_t at = i + 1024 * a;
      if (at + 4 <= z.pairs) {
        f[a] = *(const Four*)(pos + at);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) f[a].v[c] = at + c < z.pairs ? pos[at + c] : -1;
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t r = (uint32_t)f[a].v[c] - (uint32_t)first;   // rows are at most 2^28: a negative entry is past `here`
        if (r < (uint32_t)here) atomicOr(&named[r >> 5], 1u << (r & 31));
      }
  }
  __syncthreads();
  const int lane = threadIdx.x & 63;
  for (int w = threadIdx.x >> 6; 32 * w < here; w += 4) {
    uint32_t left = ~named[w];
    if (here - 32 * w < 32) left &= (1u << (here - 32 * w)) - 1;
    for (; left; left &= left - 1) {
      const int64_t row = first + 32 * w + __builtin_ctz(left);
      for (int c = lane; c < pieces; c += 64) y[row * pieces + c] = P{};
    }
  }
}

// ---- permute: a thread moves one V-wide piece of a token's row per step.
// A block holds 256 / tpt tokens, tpt = threads per token (a power of two).
// MS bounds the slots, so their positions stay in registers.
template <class T, int V, int MS>
__global__ void __launch_bounds__(256) permute_kernel(const typename T::store* __restrict__ x,
                                                      const int32_t* __restrict__ pos, int64_t tokens, int slots,
                                                      int pieces, int64_t rows, int tpt_log2, Zeroing z,
                                                      typename T::store* __restrict__ y) {
  typedef Pack<T, V> P;
  if (blockIdx.x < z.blocks) {
    if (blockIdx.y == 0) zero_free_rows(pos, z, rows, pieces, (P*)y);
    return;
  }
  const int tpt = 1 << tpt_log2;
  const int64_t t = (int64_t)(blockIdx.x - z.blocks) * (256 >> tpt_log2) + (threadIdx.x >> tpt_log2);
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
    int64_t rows, Zeroing z, typename T::store* __restrict__ dy, float* __restrict__ dw) {
  typedef Pack<T, V> P;
  __shared__ float part[4][MS];
  if (blockIdx.x < z.blocks) {
    zero_free_rows(pos, z, rows, pieces, (P*)dy);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)(blockIdx.x - z.blocks) * (4 / WPT) + wave / WPT;
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
static void run_permute(const void* x, const int32_t* pos, int64_t tokens, int slots, int H, int64_t rows, Zeroing z,
                        void* y, hipStream_t st) {
  typedef typename T::store S;
  const int pieces = H / V;
  RowGrid g = row_grid(tokens, pieces);
  g.grid.x += z.blocks;
  MILO_SLOTS(16, hipLaunchKernelGGL((permute_kernel<T, V, MS>), g.grid, dim3(256), 0, st, (const S*)x, pos, tokens,
                                    slots, pieces, rows, g.tpt_log2, z, (S*)y));
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
                               int slots, int H, int64_t rows, Zeroing z, void* dy, float* dw, hipStream_t st) {
  typedef typename T::store S;
  const int pieces = H / V;
  // four waves to a token while the tokens alone do not fill the chip (256
  // compute units x 8 waves) and the row is long enough to share
  if (tokens < 2048 && pieces > 64)
    MILO_SLOTS(16, hipLaunchKernelGGL((unpermute_grad_kernel<T, V, MS, W, 4>), dim3((unsigned)tokens + z.blocks),
                                      dim3(256), 0, st, (const S*)dout, (const S*)y, pos, w, tokens, slots, pieces,
                                      rows, z, (S*)dy, dw));
  else
    MILO_SLOTS(16, hipLaunchKernelGGL((unpermute_grad_kernel<T, V, MS, W, 1>),
                                      dim3((unsigned)((tokens + 3) / 4) + z.blocks), dim3(256), 0, st, (const S*)dout,
                                      (const S*)y, pos, w, tokens, slots, pieces, rows, z, (S*)dy, dw));
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

// ---- all rows as zeros, 4 bytes a thread and turn behind the first ones that
// do not reach an address of 4 (2-byte types)
__global__ void __launch_bounds__(256) zero_kernel(uint16_t* __restrict__ y, int64_t halves) {
  const int64_t lead = ((uintptr_t)y & 2) ? 1 : 0, words = (halves - lead) / 2;
  uint32_t* const w = (uint32_t*)(y + lead);
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t i = first; i < words; i += (int64_t)gridDim.x * 256) w[i] = 0;
  if (first == 0 && lead) y[0] = 0;
  if (first == 0 && (halves - lead) % 2) y[halves - 1] = 0;
}

// How the rows without a pair become zeros: by the scan where the rows' own
// traffic hides most of it, else all rows at first, a launch and their bytes.
// 131072 pairs to rows of 128 values of 16 bits: 8 us without, 28 with the scan,
// 16 with the rows cleared; of 512 values 24, 32 and 37; 262144 pairs to 256
// values 24, 55 and 43; 65536 to 2048 values 56, 61 with the scan; 8192 to 4096
// values 16.7 and 16.5.  (With 512 blocks of scanning instead of 128 the gradient
// of the 2048 values took 150 us, 142 so.)
static Zeroing plan_zeroing(bool zero, int64_t tokens, int slots, int64_t rows, int H, int dtype, void* y,
                            hipStream_t st) {
  if (!zero || rows == 0) return {0, 0, 0};
  const int64_t pairs = tokens * slots, row_bytes = (int64_t)H * elem_bytes(dtype);
  int64_t slice = (rows + 127) / 128;      // 128 blocks: few readers of the table, enough to clear many rows
  slice = slice > kSliceRows ? kSliceRows : (slice + 31) / 32 * 32;
  const int64_t blocks = (rows + slice - 1) / slice;
  const double scan = 1.8e-4 * pairs * ((blocks + 127) / 128);
  const double move = 1.8e-7 * pairs * row_bytes, clear = 4 + 1.3e-7 * rows * row_bytes;
  if (pairs > 0 && scan < move + clear) return {(int)blocks, (int)slice, pairs};
  const int64_t halves = rows * row_bytes / 2, want = (halves / 2 + 255) / 256;
  hipLaunchKernelGGL(zero_kernel, dim3((unsigned)(want < 1 ? 1 : want < 16384 ? want : 16384)), dim3(256), 0, st,
                     (uint16_t*)y, halves);
  return {0, 0, 0};
}

int32_t launch_permute(const void* x, const int32_t* pos, int64_t tokens, int slots, int H, int64_t rows, int dtype,
                       bool zero, void* y, hipStream_t st) {
  const int bytes = access_bytes(H * elem_bytes(dtype), x, y);
  const Zeroing first = plan_zeroing(zero, tokens, slots, rows, H, dtype, y, st);
#define RUN(T, V, ...) run_permute<T, V>(__VA_ARGS__)
  by_launches(tokens, [&](int64_t t, int64_t n) {
    const Zeroing z = t == 0 ? first : Zeroing{0, 0, 0};
    MILO_BY_TYPE(RUN, (const char*)x + t * H * elem_bytes(dtype), pos + t * slots, n, slots, H, rows, z, y, st);
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
                              int slots, int H, int64_t rows, int dtype, bool zero, void* dy, float* dw,
                              hipStream_t st) {
  const int bytes = access_bytes(H * elem_bytes(dtype), dout, y, dy);
  const Zeroing z = plan_zeroing(zero, tokens, slots, rows, H, dtype, dy, st);
  if (tokens == 0) return hip_status(hipGetLastError(), "zero_kernel launch");
#define RUN(T, V, ...)                                 \
  do {                                                 \
    if (w) run_unpermute_grad<T, V, true>(__VA_ARGS__); \
    else run_unpermute_grad<T, V, false>(__VA_ARGS__);  \
  } while (0)
  MILO_BY_TYPE(RUN, dout, y, pos, w, tokens, slots, H, rows, z, dy, dw, st);
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
