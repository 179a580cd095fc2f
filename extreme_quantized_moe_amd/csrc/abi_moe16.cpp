// The C ABI of the 16-bit MoE operators (declared in include/milo.h):
// argument validation and kernel dispatch.  Host code only; every check runs
// before anything is enqueued.
#include "linear.hpp"

namespace milo {

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

#define MILO_FAIL(code, ...)   \
  do {                         \
    set_error(__VA_ARGS__);    \
    return (code);             \
  } while (0)

static size_t elem_size(int dtype) { return dtype == MILO_F32 ? 4 : 2; }

// Checks the dispatch operators share; rows_ptr is the expert-ordered buffer,
// tok_ptr the one in token order.
static int32_t check_dispatch(const void* tok_ptr, const void* rows_ptr, const int32_t* pos, int T, int slots, int H,
                              int num_rows, int dtype) {
  if (dtype != MILO_F16 && dtype != MILO_BF16 && dtype != MILO_F32) MILO_FAIL(MILO_ERR_ARG, "unknown dtype %d", dtype);
  if (T < 0 || T > (1 << 24) || slots < 1 || slots > 16 || H < 1 || H > (1 << 20) || num_rows < 0 ||
      num_rows > (1 << 28))
    MILO_FAIL(MILO_ERR_SHAPE, "T=%d slots=%d H=%d num_rows=%d: need 0 <= T <= 2^24, 1 <= slots <= 16, "
              "1 <= H <= 2^20, 0 <= num_rows <= 2^28", T, slots, H, num_rows);
  if (T > 0 && (!tok_ptr || !pos)) MILO_FAIL(MILO_ERR_NULL, "the token rows and pair_pos are required");
  if (T > 0 && num_rows > 0 && !rows_ptr) MILO_FAIL(MILO_ERR_NULL, "the expert-ordered rows are required");
  if (!aligned(tok_ptr, elem_size(dtype)) || !aligned(rows_ptr, elem_size(dtype)) || !aligned(pos, 4))
    MILO_FAIL(MILO_ERR_ALIGN, "a pointer is not aligned to its element");
  return MILO_OK;
}

static int32_t check_dtype16(int dtype, int out_dtype) {
  if (dtype != MILO_F16 && dtype != MILO_BF16) MILO_FAIL(MILO_ERR_ARG, "dtype %d: need MILO_F16 or MILO_BF16", dtype);
  if (out_dtype != dtype && out_dtype != MILO_F32)
    MILO_FAIL(MILO_ERR_ARG, "output type %d: need the operands' type or MILO_F32", out_dtype);
  return MILO_OK;
}

static int32_t check_groups(int E, int N, int K, int num_rows, const int32_t* offsets) {
  if (E < 1 || E > 256) MILO_FAIL(MILO_ERR_SHAPE, "num_experts=%d outside 1..256", E);
  if (N < 1 || N > 65536 || K < 1 || K > 65536) MILO_FAIL(MILO_ERR_SHAPE, "N=%d K=%d: need both in 1..65536", N, K);
  if (num_rows < 0 || num_rows > (1 << 20)) MILO_FAIL(MILO_ERR_SHAPE, "num_rows=%d outside 0..1048576", num_rows);
  if (E > 1 && !offsets) MILO_FAIL(MILO_ERR_NULL, "offsets is required with num_experts > 1");
  if (!aligned(offsets, 4)) MILO_FAIL(MILO_ERR_ALIGN, "offsets must be 4-byte aligned");
  return MILO_OK;
}

static int32_t check_workspace(size_t need, const void* ws, size_t ws_bytes) {
  if (!need) return MILO_OK;
  if (!ws || ws_bytes < need)
    MILO_FAIL(MILO_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
  if (!aligned(ws, 256)) MILO_FAIL(MILO_ERR_ALIGN, "workspace must be 256-byte aligned");
  return MILO_OK;
}

static int32_t check_act(int act) {
  if (act < MILO_ACT_NONE || act > MILO_ACT_GELU_TANH) MILO_FAIL(MILO_ERR_ARG, "unknown activation %d", act);
  return MILO_OK;
}

static int32_t check_linear(const milo_linear_desc* d) {
  if (!d) MILO_FAIL(MILO_ERR_NULL, "desc is NULL");
  int32_t rc;
  if ((rc = check_groups(d->num_experts, d->N, d->K, d->num_rows, d->offsets))) return rc;
  if ((rc = check_dtype16(d->dtype, d->out_dtype))) return rc;
  if ((rc = check_act(d->activation))) return rc;
  if (d->max_rows_per_expert < 0) MILO_FAIL(MILO_ERR_SHAPE, "max_rows_per_expert < 0");
  if (!d->w || (d->num_rows > 0 && (!d->x || !d->y))) MILO_FAIL(MILO_ERR_NULL, "x, w and y are required");
  if (!aligned(d->x, 2) || !aligned(d->w, 2) || !aligned(d->bias, 2) || !aligned(d->mul, 2) ||
      !aligned(d->residual, 2) || !aligned(d->pre, 2) || !aligned(d->y, elem_size(d->out_dtype)))
    MILO_FAIL(MILO_ERR_ALIGN, "a pointer is not aligned to its element");
  return MILO_OK;
}

static LinearArgs linear_args(const milo_linear_desc* d) {
  LinearArgs a = {};
  a.a = d->x;
  a.b = d->w;
  a.offsets = d->offsets;
  a.bias = d->bias;
  a.mul = d->mul;
  a.residual = d->residual;
  a.pre = d->pre;
  a.out = d->y;
  a.E = d->num_experts;
  a.rows = d->num_rows;
  a.max_rows = d->max_rows_per_expert > 0 && d->max_rows_per_expert < d->num_rows ? d->max_rows_per_expert
                                                                                  : d->num_rows;
  a.N = d->N;
  a.K = d->K;
  a.act = d->activation;
  a.out_f32 = d->out_dtype == MILO_F32;
  a.splits = 1;
  return a;
}

static int32_t check_linear_grad(const milo_linear_grad_desc* d) {
  if (!d) MILO_FAIL(MILO_ERR_NULL, "desc is NULL");
  int32_t rc;
  if ((rc = check_groups(d->num_experts, d->N, d->K, d->num_rows, d->offsets))) return rc;
  if ((rc = check_dtype16(d->dtype, d->dw_dtype))) return rc;
  if (d->num_rows > 0 && !d->dy && (d->dx || d->dw)) MILO_FAIL(MILO_ERR_NULL, "dy is required");
  if (d->num_rows > 0 && d->dx && !d->w) MILO_FAIL(MILO_ERR_NULL, "w is required for dx");
  if (d->num_rows > 0 && d->dw && !d->x) MILO_FAIL(MILO_ERR_NULL, "x is required for dw");
  if (!aligned(d->dy, 2) || !aligned(d->x, 2) || !aligned(d->w, 2) || !aligned(d->dx, 2) ||
      !aligned(d->dx_add, 2) || !aligned(d->dw, elem_size(d->dw_dtype)))
    MILO_FAIL(MILO_ERR_ALIGN, "a pointer is not aligned to its element");
  return MILO_OK;
}

// The two products of one gradient call; they run one after the other on the
// stream, so they share the workspace.
static LinearArgs grad_args(const milo_linear_grad_desc* d, int mode) {
  LinearArgs a = {};
  a.a = d->dy;
  a.b = mode == kDx ? d->w : d->x;
  a.offsets = d->offsets;
  a.out = mode == kDx ? d->dx : d->dw;
  a.residual = mode == kDx ? d->dx_add : nullptr;
  a.E = d->num_experts;
  a.rows = a.max_rows = d->num_rows;
  a.N = d->N;
  a.K = d->K;
  a.out_f32 = mode == kDw && d->dw_dtype == MILO_F32;
  a.splits = 1;
  return a;
}

}  // namespace milo

using namespace milo;

static int32_t run_permute(const void* x, const int32_t* pair_pos, int32_t T, int32_t slots, int32_t H,
                           int32_t num_rows, int32_t dtype, bool zero, void* y, void* stream) {
  set_error("%s", "");
  if (int32_t rc = check_dispatch(x, y, pair_pos, T, slots, H, num_rows, dtype)) return rc;
  if (zero && num_rows > 0 && !y) MILO_FAIL(MILO_ERR_NULL, "the expert-ordered rows are required");
  if (num_rows == 0 || (T == 0 && !zero)) return MILO_OK;
  return launch_permute(x, pair_pos, T, slots, H, num_rows, dtype, zero, y, (hipStream_t)stream);
}

static int32_t run_unpermute_grad(const void* dout, const void* y, const int32_t* pair_pos, const float* slot_w,
                                  int32_t T, int32_t slots, int32_t H, int32_t num_rows, int32_t dtype, bool zero,
                                  void* dy, float* dslot_w, void* stream) {
  set_error("%s", "");
  if (int32_t rc = check_dispatch(dout, y, pair_pos, T, slots, H, num_rows, dtype)) return rc;
  if ((T > 0 || zero) && num_rows > 0 && !dy) MILO_FAIL(MILO_ERR_NULL, "dy is required");
  if (!aligned(slot_w, 4) || !aligned(dslot_w, 4) || !aligned(dy, elem_size(dtype)))
    MILO_FAIL(MILO_ERR_ALIGN, "dy must be aligned to its element, slot_w and dslot_w to 4 bytes");
  if (T == 0 && !zero) return MILO_OK;
  return launch_unpermute_grad(dout, y, pair_pos, slot_w, T, slots, H, num_rows, dtype, zero, dy, dslot_w,
                               (hipStream_t)stream);
}

extern "C" {

int32_t milo_moe_permute(const void* x, const int32_t* pair_pos, int32_t T, int32_t slots, int32_t H,
                         int32_t num_rows, int32_t dtype, void* y, void* stream) {
  return run_permute(x, pair_pos, T, slots, H, num_rows, dtype, false, y, stream);
}

int32_t milo_moe_permute_zeroed(const void* x, const int32_t* pair_pos, int32_t T, int32_t slots, int32_t H,
                                int32_t num_rows, int32_t dtype, void* y, void* stream) {
  return run_permute(x, pair_pos, T, slots, H, num_rows, dtype, true, y, stream);
}

int32_t milo_moe_permute_grad(const void* dy, const int32_t* pair_pos, int32_t T, int32_t slots, int32_t H,
                              int32_t num_rows, int32_t dtype, void* dx, void* stream) {
  return milo_moe_unpermute(dy, pair_pos, nullptr, T, slots, H, num_rows, dtype, dx, stream);
}

int32_t milo_moe_unpermute(const void* y, const int32_t* pair_pos, const float* slot_w, int32_t T, int32_t slots,
                           int32_t H, int32_t num_rows, int32_t dtype, void* out, void* stream) {
  set_error("%s", "");
  if (int32_t rc = check_dispatch(out, y, pair_pos, T, slots, H, num_rows, dtype)) return rc;
  if (!aligned(slot_w, 4)) MILO_FAIL(MILO_ERR_ALIGN, "slot_w must be 4-byte aligned");
  if (T == 0) return MILO_OK;
  return launch_unpermute(y, pair_pos, slot_w, T, slots, H, num_rows, dtype, out, (hipStream_t)stream);
}

int32_t milo_moe_unpermute_grad(const void* dout, const void* y, const int32_t* pair_pos, const float* slot_w,
                                int32_t T, int32_t slots, int32_t H, int32_t num_rows, int32_t dtype, void* dy,
                                float* dslot_w, void* stream) {
  return run_unpermute_grad(dout, y, pair_pos, slot_w, T, slots, H, num_rows, dtype, false, dy, dslot_w, stream);
}

int32_t milo_moe_unpermute_grad_zeroed(const void* dout, const void* y, const int32_t* pair_pos, const float* slot_w,
                                       int32_t T, int32_t slots, int32_t H, int32_t num_rows, int32_t dtype, void* dy,
                                       float* dslot_w, void* stream) {
  return run_unpermute_grad(dout, y, pair_pos, slot_w, T, slots, H, num_rows, dtype, true, dy, dslot_w, stream);
}

int32_t milo_route_grad(const float* dslot_w, const float* logits, const int32_t* topk_ids, int32_t T, int32_t E,
                        int32_t k, int32_t S, int32_t renormalize, float* dlogits, void* stream) {
  set_error("%s", "");
  if (T < 0 || T > (1 << 24) || E < 1 || S < 0 || E + S > 256 || k < 1 || k > 8 || k > E || k + S > 16)
    MILO_FAIL(MILO_ERR_SHAPE, "T=%d E=%d k=%d S=%d: need 0 <= T <= 2^24, 1 <= k <= min(E, 8), S >= 0, "
              "E + S <= 256, k + S <= 16", T, E, k, S);
  if (T > 0 && (!dslot_w || !logits || !topk_ids || !dlogits))
    MILO_FAIL(MILO_ERR_NULL, "dslot_w, logits, topk_ids and dlogits are required");
  if (!aligned(dslot_w, 4) || !aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(dlogits, 4))
    MILO_FAIL(MILO_ERR_ALIGN, "pointers must be 4-byte aligned");
  if (T == 0) return MILO_OK;
  return launch_route_grad(dslot_w, logits, topk_ids, T, E, k, S, renormalize ? 1 : 0, dlogits, (hipStream_t)stream);
}

size_t milo_moe_linear_workspace_bytes(const milo_linear_desc* desc) {
  if (check_linear(desc) || desc->num_rows == 0) return 0;
  return plan_bytes(plan_linear(kFwd, linear_args(desc)));
}

int32_t milo_moe_linear(const milo_linear_desc* desc, void* workspace, size_t ws_bytes, void* stream) {
  set_error("%s", "");
  if (int32_t rc = check_linear(desc)) return rc;
  if (desc->num_rows == 0) return MILO_OK;
  const LinearArgs a = linear_args(desc);
  const LinearPlan p = plan_linear(kFwd, a);
  if (int32_t rc = check_workspace(plan_bytes(p), workspace, ws_bytes)) return rc;
  return launch_linear(kFwd, desc->dtype, a, p, workspace, false, (hipStream_t)stream);
}

size_t milo_moe_linear_act_grad_workspace_bytes(int32_t num_experts, int32_t N, int32_t num_rows) {
  if (num_experts < 1 || num_experts > 256 || N < 1 || N > 65536 || num_rows < 0 || num_rows > (1 << 20)) return 0;
  return act_grad_workspace_bytes(num_experts, N, num_rows);
}

int32_t milo_moe_linear_act_grad(const void* dy, const void* pre, const void* mul, const int32_t* offsets,
                                 int32_t num_experts, int32_t N, int32_t num_rows, int32_t dtype, int32_t activation,
                                 void* dpre, void* dmul, float* dbias, void* workspace, size_t ws_bytes,
                                 void* stream) {
  set_error("%s", "");
  int32_t rc;
  if ((rc = check_groups(num_experts, N, 1, num_rows, offsets))) return rc;
  if ((rc = check_dtype16(dtype, dtype))) return rc;
  if ((rc = check_act(activation))) return rc;
  if (num_rows > 0 && (!dy || !pre || !dpre)) MILO_FAIL(MILO_ERR_NULL, "dy, pre and dpre are required");
  if (num_rows > 0 && (mul != nullptr) != (dmul != nullptr)) MILO_FAIL(MILO_ERR_ARG, "mul and dmul go together");
  if (!aligned(dy, 2) || !aligned(pre, 2) || !aligned(mul, 2) || !aligned(dpre, 2) || !aligned(dmul, 2) ||
      !aligned(dbias, 4))
    MILO_FAIL(MILO_ERR_ALIGN, "a pointer is not aligned to its element");
  if (dbias && (rc = check_workspace(act_grad_workspace_bytes(num_experts, N, num_rows), workspace, ws_bytes)))
    return rc;
  return launch_act_grad(dy, pre, mul, offsets, num_experts, N, num_rows, dtype, activation, dpre, dmul, dbias,
                         (float*)workspace, (hipStream_t)stream);
}

size_t milo_moe_linear_grad_workspace_bytes(const milo_linear_grad_desc* desc) {
  if (check_linear_grad(desc)) return 0;
  size_t need = 0;
  for (int mode = kDx; mode <= kDw; ++mode) {
    const LinearArgs a = grad_args(desc, mode);
    if (!a.out || (mode == kDx && a.rows == 0)) continue;
    const size_t b = plan_bytes(plan_linear(mode, a));
    need = b > need ? b : need;
  }
  return need;
}

int32_t milo_moe_linear_grad(const milo_linear_grad_desc* desc, void* workspace, size_t ws_bytes, void* stream) {
  set_error("%s", "");
  if (int32_t rc = check_linear_grad(desc)) return rc;
  if (int32_t rc = check_workspace(milo_moe_linear_grad_workspace_bytes(desc), workspace, ws_bytes)) return rc;
  bool packed = false;                                      // dy's copy, first in both products' workspace
  for (int mode = kDx; mode <= kDw; ++mode) {
    const LinearArgs a = grad_args(desc, mode);
    if (!a.out || (mode == kDx && a.rows == 0)) continue;   // dw is written (zeros) without rows too
    const LinearPlan p = plan_linear(mode, a);
    if (int32_t rc = launch_linear(mode, desc->dtype, a, p, workspace, packed, (hipStream_t)stream)) return rc;
    packed = p.a_bytes > 0;
  }
  return MILO_OK;
}

}  // extern "C"
