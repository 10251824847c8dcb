// api.hip -- the extern "C" entry points of libmoe.so: argument validation, workspace
// carving and launch sequencing on the caller's stream.  The operations themselves are
// documented in moe.h.
#include <float.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "common.h"

namespace {

thread_local char g_err[512];

moe_status fail(moe_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

moe_status hip_status(hipError_t e, const char* where) {
  if (e == hipSuccess) return MOE_OK;
  return fail(MOE_EHIP, "%s: %s", where, hipGetErrorString(e));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
// whether the output p (if there is one) is none of the arguments o
template <typename... P>
bool apart(const void* p, P... o) { return !p || ((p != (const void*)o) && ...); }

#define REQUIRE(cond, st, ...) \
  do {                         \
    if (!(cond)) return fail(st, __VA_ARGS__); \
  } while (0)

moe_status check_dims(int32_t N, int32_t E, int32_t k) {
  REQUIRE(N >= 0, MOE_EINVAL, "N must be >= 0 (got %d)", N);
  REQUIRE(E >= 1 && E <= 1024, MOE_EINVAL, "E must be in [1, 1024] (got %d)", E);
  REQUIRE(k >= 1 && k <= E, MOE_EINVAL, "k must be in [1, E] (got k=%d, E=%d)", k, E);
  REQUIRE((int64_t)N * k <= INT32_MAX / 2, MOE_EINVAL, "N*k too large");
  return MOE_OK;
}

moe_status check_hi(int32_t H, int32_t I) {
  REQUIRE(H >= 8 && I >= 8, MOE_EINVAL, "H and I must be >= 8 (got H=%d, I=%d)", H, I);
  REQUIRE(H % 8 == 0 && I % 8 == 0, MOE_EUNSUPPORTED, "H and I must be multiples of 8 (got H=%d, I=%d)", H, I);
  return MOE_OK;
}

moe_status check_dtype(moe_dtype dt) {
  REQUIRE(dt == MOE_F32 || dt == MOE_BF16, MOE_EUNSUPPORTED, "unknown dtype %d", (int)dt);
  return MOE_OK;
}

moe_status check_plan(const moe_plan* p) {
  REQUIRE(p != nullptr, MOE_EINVAL, "plan is NULL");
  moe_status st = check_dims(p->N, p->E, p->k);
  if (st != MOE_OK) return st;
  REQUIRE(p->kind == MOE_PLAN_TOPK || p->kind == MOE_PLAN_TR || p->kind == MOE_PLAN_CAP, MOE_EINVAL,
          "unknown plan kind %d", p->kind);
  const int64_t need = moe_plan_rows_cap(p->kind, p->N, p->E, p->k, p->kind == MOE_PLAN_TOPK ? 0 : p->mtile);
  REQUIRE(need >= 0, MOE_EINVAL, "invalid plan dimensions");
  REQUIRE(p->M_cap >= need, MOE_EINVAL, "plan M_cap %d < required %lld", p->M_cap, (long long)need);
  REQUIRE(p->counts && p->offsets && p->tok_ptr, MOE_EINVAL, "plan has a NULL counts/offsets/tok_ptr array");
  REQUIRE(p->M_cap == 0 || (p->row_token && p->row_w && p->row_pair && p->tok_rows), MOE_EINVAL,
          "plan has a NULL row array");
  return MOE_OK;
}

constexpr int32_t kMaxSeqs = 1 << 20;

// (1024 threads per sequence and 64 experts: a launch takes fewer than 2^32)
moe_status check_seqs(int32_t B, int32_t E, const int32_t* seq_ptr) {
  REQUIRE(B >= 1 && B <= kMaxSeqs, MOE_EINVAL, "B must be in [1, %d] (got %d)", kMaxSeqs, B);
  REQUIRE((int64_t)B * ((E + 63) / 64) < 1 << 22, MOE_EUNSUPPORTED, "B * ceil(E / 64) must be below 2^22 (got B=%d, E=%d)",
          B, E);
  REQUIRE(seq_ptr || B == 1, MOE_EINVAL, "B > 1 needs seq_ptr");
  return MOE_OK;
}

// types and sizes of the norm calls: rdt is dt, or fp32 beside bf16
moe_status check_norm(moe_dtype dt, moe_dtype rdt, int32_t N, int32_t H) {
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  if ((st = check_dtype(rdt)) != MOE_OK) return st;
  REQUIRE(rdt == dt || rdt == MOE_F32, MOE_EUNSUPPORTED, "the residual type must be the activations' or fp32");
  REQUIRE(N >= 0, MOE_EINVAL, "N must be >= 0 (got %d)", N);
  REQUIRE(H >= 8, MOE_EINVAL, "H must be >= 8 (got %d)", H);
  REQUIRE(H % 8 == 0 && H <= 16384, MOE_EUNSUPPORTED, "H must be a multiple of 8 up to 16384 (got %d)", H);
  REQUIRE((int64_t)N * H < (int64_t)1 << 40, MOE_EUNSUPPORTED, "N*H too large");
  return MOE_OK;
}

int64_t mcap_of(const moe_plan* p) { return p->M_cap; }

// The GEMM kernels address a tensor through one buffer descriptor with 32-bit byte offsets
// (an offset of 2^31 or more marks a masked lane), so every tensor one descriptor covers must
// stay below 2 GiB: x and dOut [N,H], one expert's weight or weight-gradient matrix [I,H],
// the row-ordered activations (hcache and dH [M_cap, 2I], A and A' [M_cap, I]) and the plan's
// row arrays (4 M_cap bytes).
constexpr int64_t kDescBytes = 0x7FFFFFFF;
moe_status check_desc_sizes(moe_dtype dt, int64_t N, int64_t H, int64_t I, int64_t M_cap) {
  const int64_t es = dt == MOE_BF16 ? 2 : 4;
  REQUIRE(N * H * es <= kDescBytes, MOE_EUNSUPPORTED, "x/dout [N=%lld, H=%lld] must be < 2 GiB", (long long)N,
          (long long)H);
  REQUIRE(I * H * es <= kDescBytes, MOE_EUNSUPPORTED, "one expert's weight matrix [I=%lld, H=%lld] must be < 2 GiB",
          (long long)I, (long long)H);
  REQUIRE(M_cap * 2 * I * es <= kDescBytes, MOE_EUNSUPPORTED,
          "row activations [M_cap=%lld, 2I=%lld] must be < 2 GiB", (long long)M_cap, (long long)(2 * I));
  REQUIRE(M_cap * 4 <= kDescBytes, MOE_EUNSUPPORTED, "plan row arrays (M_cap=%lld) must be < 2 GiB",
          (long long)M_cap);
  return MOE_OK;
}

// type and sizes of the dense products: their kernels address each operand (in fp32 its three bf16
// parts) with 32-bit byte offsets
moe_status check_linear(moe_dtype dt, int32_t N, int32_t K, int32_t O) {
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  REQUIRE(N >= 0, MOE_EINVAL, "N must be >= 0 (got %d)", N);
  REQUIRE(K >= 8 && O >= 8, MOE_EINVAL, "K and O must be >= 8 (got K=%d, O=%d)", K, O);
  REQUIRE(K % 8 == 0 && O % 8 == 0, MOE_EUNSUPPORTED, "K and O must be multiples of 8 (got K=%d, O=%d)", K, O);
  // (512 threads per 16 outputs, 1024 per 32 columns of dbias: a launch takes fewer than 2^32)
  REQUIRE(O <= 1 << 26, MOE_EUNSUPPORTED, "O must be at most 2^26 (got %d)", O);
  const int64_t es = dt == MOE_F32 ? 6 : 2;
  REQUIRE((int64_t)N * K * es <= kDescBytes && (int64_t)N * O * es <= kDescBytes && (int64_t)O * K * es <= kDescBytes,
          MOE_EUNSUPPORTED, "x [N=%d, K=%d], w [O=%d, K] and out [N, O] must each be < 2 GiB (bf16; fp32: a third of it "
          "in elements)", N, K, O);
  return MOE_OK;
}

// type and sizes of the layer for a few tokens; unit: what H and I are multiples of
moe_status check_few(moe_dtype dt, int32_t N, int32_t H, int32_t I, int32_t E, int32_t k, int32_t unit) {
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  if ((st = check_dims(N, E, k)) != MOE_OK) return st;
  REQUIRE(N <= MOE_FEW_MAX_TOKENS, MOE_EUNSUPPORTED, "N must be at most %d (got %d)", MOE_FEW_MAX_TOKENS, N);
  REQUIRE(k <= MOE_FEW_MAX_K, MOE_EUNSUPPORTED, "k must be at most %d (got %d)", MOE_FEW_MAX_K, k);
  REQUIRE(H >= unit && I >= unit, MOE_EINVAL, "H and I must be >= %d (got H=%d, I=%d)", unit, H, I);
  REQUIRE(H % unit == 0 && I % unit == 0, MOE_EUNSUPPORTED, "H and I must be multiples of %d (got H=%d, I=%d)", unit, H,
          I);
  REQUIRE(H <= 1 << 20 && I <= 1 << 20, MOE_EUNSUPPORTED, "H and I must be at most 2^20 (got H=%d, I=%d)", H, I);
  return MOE_OK;
}

// the arguments that both forms of the layer for a few tokens share
moe_status check_few_args(moe_dtype dt, const void* x, const void* w_r, const void* bias, const void* wg,
                          const void* wu, const void* wd, int32_t N, int32_t H, int32_t I, int32_t E, int32_t k,
                          const void* out, const void* idx, const void* w, const void* ws, size_t ws_bytes) {
  REQUIRE(w_r && wg && wu && wd, MOE_EINVAL, "NULL weight argument");
  REQUIRE(N == 0 || (x && out && idx && w), MOE_EINVAL, "NULL x/out/topk_idx/topk_w");
  REQUIRE(N == 0 || (apart(out, x, w_r, bias, wg, wu, wd, idx, w, ws) && apart(idx, x, w_r, bias, wg, wu, wd, w, ws) &&
                     apart(w, x, w_r, bias, wg, wu, wd, ws)),
          MOE_EINVAL, "out, topk_idx and topk_w must be no other argument");
  REQUIRE(aligned16(x) && aligned16(wg) && aligned16(wu) && aligned16(wd) && aligned16(out) && aligned16(ws),
          MOE_EUNSUPPORTED, "x, weights, out and workspace must be 16-byte aligned");
  REQUIRE(aligned4(w_r) && aligned4(bias) && aligned4(idx) && aligned4(w), MOE_EUNSUPPORTED,
          "w_r, bias, topk_idx and topk_w must be 4-byte aligned");
  const size_t need = moe::layer_few_ws_bytes(dt, N, E, k, H, I);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  return MOE_OK;
}

// type and sizes of the cross entropy: descriptors of 32-bit byte offsets over x and over a piece (256
// columns at least) of dz and of w; launches of fewer than 2^32 threads
moe_status check_ce(moe_dtype dt, int32_t N, int32_t H, int32_t V) {
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  REQUIRE(N >= 0, MOE_EINVAL, "N must be >= 0 (got %d)", N);
  REQUIRE(H >= 8 && V >= 1, MOE_EINVAL, "H must be >= 8 and V >= 1 (got H=%d, V=%d)", H, V);
  REQUIRE(H % 8 == 0, MOE_EUNSUPPORTED, "H must be a multiple of 8 (got %d)", H);
  const int64_t es = dt == MOE_F32 ? 6 : 2, h = H > 256 ? H : 256;
  REQUIRE(N * h * es <= kDescBytes && 256 * (int64_t)H * es <= kDescBytes, MOE_EUNSUPPORTED,
          "x [N=%d, max(H=%d, 256)] must be < 2 GiB (bf16; fp32: a third of it in elements)", N, H);
  REQUIRE(V <= 1 << 30 && (int64_t)N * V <= (int64_t)1 << 36 && (int64_t)V * H <= (int64_t)1 << 36, MOE_EUNSUPPORTED,
          "V must be at most 2^30, N V and V H at most 2^36 (got N=%d, V=%d, H=%d)", N, V, H);
  return MOE_OK;
}

}  // namespace

namespace moe {
DevInfo dev_info() {
  static DevInfo cache[64];
  static bool have[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return DevInfo{256, 8};
  if (!have[dev]) {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
    cache[dev] = DevInfo{cus, 8};
    have[dev] = true;
  }
  return cache[dev];
}
}  // namespace moe

namespace {
hipEvent_t g_events[MOE_K_COUNT][2];
}

namespace moe {
void kernel_event(int kid, int which, hipStream_t s) {
  hipEvent_t ev = g_events[kid][which];
  if (ev) (void)hipEventRecord(ev, s);
}
}  // namespace moe

extern "C" {

const char* moe_last_error(void) { return g_err; }

moe_status moe_set_kernel_events(int32_t kernel_id, void* start_event, void* stop_event) {
  g_err[0] = 0;
  REQUIRE(kernel_id >= 0 && kernel_id < MOE_K_COUNT, MOE_EINVAL, "unknown kernel id %d", kernel_id);
  g_events[kernel_id][0] = (hipEvent_t)start_event;
  g_events[kernel_id][1] = (hipEvent_t)stop_event;
  return MOE_OK;
}

int64_t moe_plan_rows_cap(int32_t kind, int32_t N, int32_t E, int32_t k, int32_t mtile) {
  if (N < 0 || E < 1 || E > 1024 || k < 1 || k > E) return -1;
  if (kind == MOE_PLAN_TOPK) return (int64_t)N * k;
  if (kind == MOE_PLAN_TR) {
    if (mtile < 1) return -1;
    return (int64_t)N * k + (int64_t)E * (mtile / 2);
  }
  if (kind == MOE_PLAN_CAP) {  // mtile holds the capacity
    if (mtile < 0) return -1;
    const int64_t a = (int64_t)N * k, b = (int64_t)E * mtile;
    return a < b ? a : b;
  }
  return -1;
}

size_t moe_workspace_bytes(moe_op op, moe_dtype dt, int32_t N, int32_t E, int32_t k, int32_t H, int32_t I,
                           int32_t M_cap) {
  if (op == MOE_OP_ADD_RMSNORM_BWD) {  // (the limit on N k is the router's)
    if (check_norm(dt, dt, N, H) != MOE_OK) return 0;
    return moe::add_rmsnorm_bwd_ws_bytes(N, H);
  }
  if (check_dims(N, E, k) != MOE_OK) return 0;
  switch (op) {
    case MOE_OP_PERMUTE: return moe::permute_ws_bytes(N, E);
    case MOE_OP_ROUTE_TR: return moe::tr_ws_bytes(N, E);
    case MOE_OP_GEMM_FWD:
      if (check_dtype(dt) != MOE_OK || check_hi(H, I) != MOE_OK || M_cap < 0) return 0;
      return moe::gemm_fwd_ws_bytes(dt, M_cap, I);
    case MOE_OP_LAYER_BWD:
      if (check_dtype(dt) != MOE_OK || check_hi(H, I) != MOE_OK || M_cap < 0) return 0;
      return moe::layer_bwd_ws_bytes(dt, N, M_cap, H, I);
    case MOE_OP_ROUTER_BWD:
      if (check_dtype(dt) != MOE_OK || H < 1) return 0;
      return moe::router_bwd_ws_bytes(dt, N, H, E);
    case MOE_OP_ROUTER_LOGITS:
      if (check_dtype(dt) != MOE_OK || H < 1) return 0;
      return moe::router_logits_ws_bytes(dt, N, H, E);
    case MOE_OP_GEMM_FWD_MXFP8:
      if (H < 32 || I < 32 || H % 32 || I % 32 || M_cap < 0) return 0;
      return moe::gemm_fwd_mxfp8_ws_bytes(M_cap, I);
    case MOE_OP_LAYER_BWD_MXFP8:
      if (H < 32 || I < 32 || H % 32 || I % 32 || M_cap < 0) return 0;
      return moe::layer_bwd_mxfp8_ws_bytes(N, M_cap, H, I);
    case MOE_OP_LAYER_BWD_CKPT8:
      if (check_hi(H, I) != MOE_OK || I % 32 || M_cap < 0) return 0;
      return moe::layer_bwd_ckpt8_ws_bytes(N, M_cap, H, I);
    case MOE_OP_BALANCE_LOSS:  // I: the sequences
      if (check_seqs(I, E, &I) != MOE_OK) return 0;
      return moe::balance_loss_ws_bytes(N, E, I);
    case MOE_OP_LINEAR_FWD:
      if (check_linear(dt, N, H, I) != MOE_OK) return 0;
      return moe::linear_fwd_ws_bytes(dt, N, H, I);
    case MOE_OP_LINEAR_BWD:
      if (check_linear(dt, N, H, I) != MOE_OK) return 0;
      return moe::linear_bwd_ws_bytes(dt, N, H, I);
    case MOE_OP_LINEAR_CE_FWD:
      if (check_ce(dt, N, H, I) != MOE_OK) return 0;
      return moe::linear_ce_fwd_ws_bytes(dt, N, H, I);
    case MOE_OP_LINEAR_CE_BWD:
      if (check_ce(dt, N, H, I) != MOE_OK) return 0;
      return moe::linear_ce_bwd_ws_bytes(dt, N, H, I);
    case MOE_OP_LAYER_FEW:
      if (check_few(dt, N, H, I, E, k, 8) != MOE_OK) return 0;
      return moe::layer_few_ws_bytes(dt, N, E, k, H, I);
    case MOE_OP_ADD_RMSNORM_BWD: break;  // above
  }
  return 0;
}

moe_status moe_route_topk(const float* logits, const float* bias, int32_t N, int32_t E, int32_t k,
                          int32_t* topk_idx, float* topk_w, float* probs, void* stream) {
  g_err[0] = 0;
  moe_status st = check_dims(N, E, k);
  if (st != MOE_OK) return st;
  REQUIRE(N == 0 || (logits && topk_idx && topk_w), MOE_EINVAL, "NULL logits/topk_idx/topk_w");
  moe::kernel_event(MOE_K_ROUTE, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_route_topk(logits, bias, N, E, k, topk_idx, topk_w, probs, nullptr, (hipStream_t)stream);
  moe::kernel_event(MOE_K_ROUTE, 1, (hipStream_t)stream);
  return hip_status(e, "moe_route_topk");
}

moe_status moe_permute(const int32_t* topk_idx, const float* topk_w, int32_t N, int32_t E, int32_t k,
                       const moe_plan* plan, void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st = check_dims(N, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(plan->kind == MOE_PLAN_TOPK, MOE_EINVAL, "moe_permute needs a top-k plan");
  REQUIRE(plan->N == N && plan->E == E && plan->k == k, MOE_EINVAL, "plan dimensions differ from the call");
  REQUIRE(N == 0 || (topk_idx && topk_w), MOE_EINVAL, "NULL topk_idx/topk_w");
  const size_t need = moe::permute_ws_bytes(N, E);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  moe::kernel_event(MOE_K_PERMUTE, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_permute(topk_idx, topk_w, N, E, k, *plan, ws, (hipStream_t)stream);
  moe::kernel_event(MOE_K_PERMUTE, 1, (hipStream_t)stream);
  return hip_status(e, "moe_permute");
}

moe_status moe_permute_noalloc(const int32_t* topk_idx, const float* topk_w, int32_t N, int32_t E, int32_t k,
                               const moe_plan* plan, void* stream) {
  g_err[0] = 0;
  moe_status st = check_dims(N, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(plan->kind == MOE_PLAN_TOPK, MOE_EINVAL, "moe_permute_noalloc needs a top-k plan");
  REQUIRE(plan->N == N && plan->E == E && plan->k == k, MOE_EINVAL, "plan dimensions differ from the call");
  REQUIRE(N == 0 || (topk_idx && topk_w), MOE_EINVAL, "NULL topk_idx/topk_w");
  const size_t need = moe::permute_ws_bytes(N, E);
  REQUIRE(need <= moe::permute_scratch_bytes(), MOE_EUNSUPPORTED,
          "moe_permute_noalloc: N=%d, E=%d need %zu bytes of scratch, more than its fixed %zu", N, E, need,
          moe::permute_scratch_bytes());
  void* scratch = nullptr;
  hipError_t e = moe::permute_scratch(&scratch);
  if (e != hipSuccess) return hip_status(e, "moe_permute_noalloc: scratch address");
  moe::kernel_event(MOE_K_PERMUTE, 0, (hipStream_t)stream);
  e = moe::launch_permute(topk_idx, topk_w, N, E, k, *plan, scratch, (hipStream_t)stream);
  moe::kernel_event(MOE_K_PERMUTE, 1, (hipStream_t)stream);
  return hip_status(e, "moe_permute_noalloc");
}

moe_status moe_route_token_rounding(const float* logits, const float* bias, int32_t N, int32_t E, int32_t k,
                                    int32_t mtile, int32_t* topk_idx, float* topk_w, float* probs,
                                    const moe_plan* plan, void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st = check_dims(N, E, k);
  if (st != MOE_OK) return st;
  REQUIRE(mtile >= 1 && mtile <= 65536, MOE_EINVAL, "mtile must be in [1, 65536] (got %d)", mtile);
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(plan->kind == MOE_PLAN_TR && plan->mtile == mtile, MOE_EINVAL,
          "token rounding needs a plan of kind MOE_PLAN_TR with the same mtile");
  REQUIRE(plan->N == N && plan->E == E && plan->k == k, MOE_EINVAL, "plan dimensions differ from the call");
  REQUIRE(N == 0 || (logits && topk_idx && topk_w && probs), MOE_EINVAL, "NULL logits/topk_idx/topk_w/probs");
  const size_t need = moe::tr_ws_bytes(N, E);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  // the token normaliser sits right after the block histogram in the workspace
  float* tok_norm = moe::tr_tok_norm(ws, N, E);
  hipStream_t s = (hipStream_t)stream;
  moe::kernel_event(MOE_K_ROUTE, 0, s);
  hipError_t e = moe::launch_route_topk(logits, bias, N, E, k, topk_idx, topk_w, probs, tok_norm, s);
  moe::kernel_event(MOE_K_ROUTE, 1, s);
  if (e != hipSuccess) return hip_status(e, "moe_route_token_rounding/route");
  moe::kernel_event(MOE_K_ROUTE_TR_PLAN, 0, s);
  e = moe::launch_token_round(topk_idx, probs, tok_norm, nullptr, N, E, k, 0, mtile, 1, *plan, ws, s);
  moe::kernel_event(MOE_K_ROUTE_TR_PLAN, 1, s);
  return hip_status(e, "moe_route_token_rounding");
}

moe_status moe_route_capacity(const float* logits, const float* bias, int32_t N, int32_t E, int32_t k,
                              int32_t capacity, int32_t policy, int32_t* topk_idx, float* topk_w, float* probs,
                              const moe_plan* plan, void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st = check_dims(N, E, k);
  if (st != MOE_OK) return st;
  REQUIRE(capacity >= 0, MOE_EINVAL, "capacity must be >= 0 (got %d)", capacity);
  REQUIRE(policy == MOE_CAP_POSITION || policy == MOE_CAP_PROBS, MOE_EINVAL, "unknown capacity policy %d", policy);
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(plan->kind == MOE_PLAN_CAP && plan->mtile == capacity, MOE_EINVAL,
          "a capacity plan needs kind MOE_PLAN_CAP with the capacity in its mtile field");
  REQUIRE(plan->N == N && plan->E == E && plan->k == k, MOE_EINVAL, "plan dimensions differ from the call");
  REQUIRE(N == 0 || (logits && topk_idx && topk_w && probs), MOE_EINVAL, "NULL logits/topk_idx/topk_w/probs");
  const size_t need = moe::tr_ws_bytes(N, E);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  float* tok_norm = moe::tr_tok_norm(ws, N, E);
  hipStream_t s = (hipStream_t)stream;
  moe::kernel_event(MOE_K_ROUTE, 0, s);
  hipError_t e = moe::launch_route_topk(logits, bias, N, E, k, topk_idx, topk_w, probs, tok_norm, s);
  moe::kernel_event(MOE_K_ROUTE, 1, s);
  if (e != hipSuccess) return hip_status(e, "moe_route_capacity/route");
  moe::kernel_event(MOE_K_ROUTE_TR_PLAN, 0, s);
  e = moe::launch_token_round(topk_idx, probs, tok_norm, topk_w, N, E, k, 1, capacity,
                              policy == MOE_CAP_PROBS ? 1 : 0, *plan, ws, s);
  moe::kernel_event(MOE_K_ROUTE_TR_PLAN, 1, s);
  return hip_status(e, "moe_route_capacity");
}

moe_status moe_grouped_gemm_fwd(moe_dtype dt, const void* x, const void* w_gate, const void* w_up,
                                const void* w_down, int32_t H, int32_t I, const moe_plan* plan, void* hcache,
                                void* y, void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  if ((st = check_hi(H, I)) != MOE_OK) return st;
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(w_gate && w_up && w_down, MOE_EINVAL, "NULL weight argument");
  REQUIRE(plan->M_cap == 0 || (x && hcache && y), MOE_EINVAL, "NULL tensor argument");
  REQUIRE(aligned16(x) && aligned16(w_gate) && aligned16(w_up) && aligned16(w_down) && aligned16(hcache) &&
              aligned16(y) && aligned16(ws),
          MOE_EUNSUPPORTED, "tensors and workspace must be 16-byte aligned");
  if ((st = check_desc_sizes(dt, plan->N, H, I, plan->M_cap)) != MOE_OK) return st;
  const size_t need = moe::gemm_fwd_ws_bytes(dt, (int)mcap_of(plan), I);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  return hip_status(moe::launch_gemm_fwd(dt, x, w_gate, w_up, w_down, H, I, *plan, hcache, y, ws,
                                         (hipStream_t)stream),
                    "moe_grouped_gemm_fwd");
}

moe_status moe_quantize_mxfp8(moe_dtype dt, const void* src, int64_t rows, int32_t K, uint8_t* q, uint8_t* scales,
                              void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  REQUIRE(rows >= 0, MOE_EINVAL, "rows must be >= 0 (got %lld)", (long long)rows);
  REQUIRE(K >= 32 && K % 32 == 0, MOE_EUNSUPPORTED, "K must be a positive multiple of 32 (got %d)", K);
  REQUIRE(rows == 0 || (src && q && scales), MOE_EINVAL, "NULL src/q/scales");
  REQUIRE(aligned16(src) && aligned16(q), MOE_EUNSUPPORTED, "src and q must be 16-byte aligned");
  REQUIRE(rows <= ((int64_t)1 << 40) / K, MOE_EINVAL, "rows too large");
  moe::kernel_event(MOE_K_QUANT, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_quant_mxfp8(dt, src, rows, K, q, scales, (hipStream_t)stream);
  moe::kernel_event(MOE_K_QUANT, 1, (hipStream_t)stream);
  return hip_status(e, "moe_quantize_mxfp8");
}

moe_status moe_dequantize_mxfp8(moe_dtype dt, const uint8_t* q, const uint8_t* scales, int64_t rows, int32_t K,
                                void* out, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  REQUIRE(rows >= 0, MOE_EINVAL, "rows must be >= 0 (got %lld)", (long long)rows);
  REQUIRE(K >= 32 && K % 32 == 0, MOE_EUNSUPPORTED, "K must be a positive multiple of 32 (got %d)", K);
  REQUIRE(rows == 0 || (q && scales && out), MOE_EINVAL, "NULL q/scales/out");
  REQUIRE(aligned16(q) && aligned16(out), MOE_EUNSUPPORTED, "q and out must be 16-byte aligned");
  REQUIRE(rows <= ((int64_t)1 << 40) / K, MOE_EINVAL, "rows too large");
  moe::kernel_event(MOE_K_DEQUANT, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_dequant_mxfp8(dt, q, scales, rows, K, out, (hipStream_t)stream);
  moe::kernel_event(MOE_K_DEQUANT, 1, (hipStream_t)stream);
  return hip_status(e, "moe_dequantize_mxfp8");
}

moe_status moe_grouped_gemm_fwd_ckpt8(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                                      int32_t H, int32_t I, const moe_plan* plan, uint8_t* hq, uint8_t* hs, void* y,
                                      void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_hi(H, I)) != MOE_OK) return st;
  REQUIRE(I % 32 == 0, MOE_EUNSUPPORTED, "I must be a multiple of 32 (got %d)", I);
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(w_gate && w_up && w_down, MOE_EINVAL, "NULL weight argument");
  REQUIRE(plan->M_cap == 0 || (x && hq && hs && y), MOE_EINVAL, "NULL tensor argument");
  REQUIRE(aligned16(x) && aligned16(w_gate) && aligned16(w_up) && aligned16(w_down) && aligned16(hq) && aligned4(hs) &&
              aligned16(y) && aligned16(ws),
          MOE_EUNSUPPORTED, "tensors and workspace must be 16-byte aligned, hs 4-byte aligned");
  if ((st = check_desc_sizes(MOE_BF16, plan->N, H, I, plan->M_cap)) != MOE_OK) return st;
  const size_t need = moe::gemm_fwd_ws_bytes(MOE_BF16, (int)mcap_of(plan), I);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  return hip_status(moe::launch_gemm_fwd_ckpt8(x, w_gate, w_up, w_down, H, I, *plan, hq, hs, y, ws,
                                               (hipStream_t)stream),
                    "moe_grouped_gemm_fwd_ckpt8");
}

moe_status moe_layer_bwd_ckpt8(const void* dout, const void* x, const uint8_t* xs, const void* w_gate,
                               const void* w_up, const void* w_down, int32_t H, int32_t I, const moe_plan* plan,
                               const uint8_t* hq, const uint8_t* hs, void* dx, void* dw_gate, void* dw_up,
                               void* dw_down, float* ds, void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_hi(H, I)) != MOE_OK) return st;
  REQUIRE(I % 32 == 0 && (!xs || H % 32 == 0), MOE_EUNSUPPORTED,
          "I, and H where x comes as codes, must be a multiple of 32 (got H=%d, I=%d)", H, I);
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(w_gate && w_up && w_down && dw_gate && dw_up && dw_down, MOE_EINVAL, "NULL weight/gradient argument");
  REQUIRE(plan->N == 0 || (dout && x && dx), MOE_EINVAL, "NULL activation argument");
  REQUIRE(plan->M_cap == 0 || (hq && hs && ds), MOE_EINVAL, "NULL hq/hs/ds argument");
  REQUIRE(aligned16(dout) && aligned16(x) && aligned16(w_gate) && aligned16(w_up) && aligned16(w_down) &&
              aligned16(hq) && aligned4(hs) && aligned16(dx) && aligned16(dw_gate) && aligned16(dw_up) &&
              aligned16(dw_down) && aligned16(ws),
          MOE_EUNSUPPORTED, "tensors and workspace must be 16-byte aligned, hs 4-byte aligned");
  if ((st = check_desc_sizes(MOE_BF16, plan->N, H, I, plan->M_cap)) != MOE_OK) return st;
  const size_t need = moe::layer_bwd_ckpt8_ws_bytes(plan->N, (int)mcap_of(plan), H, I);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  return hip_status(moe::launch_layer_bwd_ckpt8(dout, x, xs, w_gate, w_up, w_down, H, I, *plan, hq, hs, dx, dw_gate,
                                                dw_up, dw_down, ds, ws, (hipStream_t)stream),
                    "moe_layer_bwd_ckpt8");
}

moe_status moe_grouped_gemm_fwd_mxfp8(const uint8_t* x_q, const uint8_t* x_s, const uint8_t* wg_q,
                                      const uint8_t* wg_s, const uint8_t* wu_q, const uint8_t* wu_s,
                                      const uint8_t* wd_q, const uint8_t* wd_s, int32_t H, int32_t I,
                                      const moe_plan* plan, void* hcache, void* y, void* ws, size_t ws_bytes,
                                      void* stream) {
  g_err[0] = 0;
  moe_status st;
  REQUIRE(H >= 32 && I >= 32, MOE_EINVAL, "H and I must be >= 32 (got H=%d, I=%d)", H, I);
  REQUIRE(H % 32 == 0 && I % 32 == 0, MOE_EUNSUPPORTED, "H and I must be multiples of 32 (got H=%d, I=%d)", H, I);
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(wg_q && wg_s && wu_q && wu_s && wd_q && wd_s, MOE_EINVAL, "NULL weight argument");
  REQUIRE(plan->M_cap == 0 || (x_q && x_s && hcache && y), MOE_EINVAL, "NULL tensor argument");
  REQUIRE(aligned16(x_q) && aligned16(wg_q) && aligned16(wu_q) && aligned16(wd_q) && aligned16(hcache) &&
              aligned16(y) && aligned16(ws) && ((uintptr_t)x_s & 3u) == 0 && ((uintptr_t)wg_s & 3u) == 0 &&
              ((uintptr_t)wu_s & 3u) == 0 && ((uintptr_t)wd_s & 3u) == 0,
          MOE_EUNSUPPORTED, "codes, outputs and workspace must be 16-byte aligned, scale codes 4-byte aligned");
  // the bf16 outputs bound the sizes as in the bf16 forward; the codes are half as large
  if ((st = check_desc_sizes(MOE_BF16, plan->N, H, I, plan->M_cap)) != MOE_OK) return st;
  const size_t need = moe::gemm_fwd_mxfp8_ws_bytes((int)mcap_of(plan), I);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  return hip_status(moe::launch_gemm_fwd_mxfp8(x_q, x_s, wg_q, wg_s, wu_q, wu_s, wd_q, wd_s, H, I, *plan, hcache, y,
                                               ws, (hipStream_t)stream),
                    "moe_grouped_gemm_fwd_mxfp8");
}

moe_status moe_unpermute_combine(moe_dtype dt, const void* y, int32_t H, const moe_plan* plan, const float* row_w,
                                 void* out, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  REQUIRE(H >= 8, MOE_EINVAL, "H must be >= 8 (got %d)", H);
  REQUIRE(H % 8 == 0, MOE_EUNSUPPORTED, "H must be a multiple of 8 (got %d)", H);
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(plan->N == 0 || (out && (plan->M_cap == 0 || y)), MOE_EINVAL, "NULL tensor argument");
  REQUIRE(aligned16(y) && aligned16(out), MOE_EUNSUPPORTED, "tensors must be 16-byte aligned");
  moe::kernel_event(MOE_K_COMBINE, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_combine(dt, y, H, *plan, row_w, out, (hipStream_t)stream);
  moe::kernel_event(MOE_K_COMBINE, 1, (hipStream_t)stream);
  return hip_status(e, "moe_unpermute_combine");
}

moe_status moe_layer_bwd(moe_dtype dt, const void* dout, const void* x, const void* w_gate, const void* w_up,
                         const void* w_down, int32_t H, int32_t I, const moe_plan* plan, const void* hcache,
                         void* dx, void* dw_gate, void* dw_up, void* dw_down, float* ds, void* ws, size_t ws_bytes,
                         void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  if ((st = check_hi(H, I)) != MOE_OK) return st;
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(w_gate && w_up && w_down && dw_gate && dw_up && dw_down, MOE_EINVAL, "NULL weight/gradient argument");
  REQUIRE(plan->N == 0 || (dout && x && dx), MOE_EINVAL, "NULL activation argument");
  REQUIRE(plan->M_cap == 0 || (hcache && ds), MOE_EINVAL, "NULL hcache/ds argument");
  REQUIRE(aligned16(dout) && aligned16(x) && aligned16(w_gate) && aligned16(w_up) && aligned16(w_down) &&
              aligned16(hcache) && aligned16(dx) && aligned16(dw_gate) && aligned16(dw_up) && aligned16(dw_down) &&
              aligned16(ws),
          MOE_EUNSUPPORTED, "tensors and workspace must be 16-byte aligned");
  if ((st = check_desc_sizes(dt, plan->N, H, I, plan->M_cap)) != MOE_OK) return st;
  const size_t need = moe::layer_bwd_ws_bytes(dt, plan->N, (int)mcap_of(plan), H, I);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  return hip_status(moe::launch_layer_bwd(dt, dout, x, w_gate, w_up, w_down, H, I, *plan, hcache, dx, dw_gate,
                                          dw_up, dw_down, ds, ws, (hipStream_t)stream),
                    "moe_layer_bwd");
}

moe_status moe_quantize_dx_weights_mxfp8(moe_dtype dt, const void* w_gate, const void* w_up, int32_t E, int32_t H,
                                         int32_t I, uint8_t* wt_q, uint8_t* wt_s, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  REQUIRE(E >= 1 && E <= 1024, MOE_EINVAL, "E must be in [1, 1024] (got %d)", E);
  REQUIRE(H >= 32 && I >= 32, MOE_EINVAL, "H and I must be >= 32 (got H=%d, I=%d)", H, I);
  REQUIRE(H % 32 == 0 && I % 32 == 0, MOE_EUNSUPPORTED, "H and I must be multiples of 32 (got H=%d, I=%d)", H, I);
  REQUIRE(w_gate && w_up && wt_q && wt_s, MOE_EINVAL, "NULL argument");
  REQUIRE(aligned16(wt_q), MOE_EUNSUPPORTED, "wt_q must be 16-byte aligned");
  REQUIRE((int64_t)H * 2 * I <= kDescBytes, MOE_EUNSUPPORTED, "one expert's [H=%d, 2I=%d] codes must be < 2 GiB", H,
          2 * I);
  moe::kernel_event(MOE_K_QUANT, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_quant_dx_weights(dt, w_gate, w_up, E, H, I, wt_q, wt_s, (hipStream_t)stream);
  moe::kernel_event(MOE_K_QUANT, 1, (hipStream_t)stream);
  return hip_status(e, "moe_quantize_dx_weights_mxfp8");
}

moe_status moe_layer_bwd_mxfp8(const void* dout, const void* x, const void* w_gate, const void* w_up,
                               const void* w_down, const uint8_t* wt_q, const uint8_t* wt_s, int32_t H, int32_t I,
                               const moe_plan* plan, const void* hcache, void* dx, void* dw_gate, void* dw_up,
                               void* dw_down, float* ds, void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st;
  REQUIRE(H >= 32 && I >= 32, MOE_EINVAL, "H and I must be >= 32 (got H=%d, I=%d)", H, I);
  REQUIRE(H % 32 == 0 && I % 32 == 0, MOE_EUNSUPPORTED, "H and I must be multiples of 32 (got H=%d, I=%d)", H, I);
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(w_gate && w_up && w_down && dw_gate && dw_up && dw_down && wt_q && wt_s, MOE_EINVAL,
          "NULL weight/gradient argument");
  REQUIRE(plan->N == 0 || (dout && x && dx), MOE_EINVAL, "NULL activation argument");
  REQUIRE(plan->M_cap == 0 || (hcache && ds), MOE_EINVAL, "NULL hcache/ds argument");
  REQUIRE(aligned16(dout) && aligned16(x) && aligned16(w_gate) && aligned16(w_up) && aligned16(w_down) &&
              aligned16(hcache) && aligned16(dx) && aligned16(dw_gate) && aligned16(dw_up) && aligned16(dw_down) &&
              aligned16(ws) && aligned16(wt_q) && ((uintptr_t)wt_s & 3u) == 0,
          MOE_EUNSUPPORTED, "tensors and workspace must be 16-byte aligned, wt_s 4-byte aligned");
  if ((st = check_desc_sizes(MOE_BF16, plan->N, H, I, plan->M_cap)) != MOE_OK) return st;
  REQUIRE((int64_t)H * 2 * I <= kDescBytes, MOE_EUNSUPPORTED, "one expert's [H=%d, 2I=%d] codes must be < 2 GiB", H,
          2 * I);
  const size_t need = moe::layer_bwd_mxfp8_ws_bytes(plan->N, (int)mcap_of(plan), H, I);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  return hip_status(moe::launch_layer_bwd_mxfp8(dout, x, w_gate, w_up, w_down, wt_q, wt_s, H, I, *plan, hcache, dx,
                                                dw_gate, dw_up, dw_down, ds, ws, (hipStream_t)stream),
                    "moe_layer_bwd_mxfp8");
}

moe_status moe_router_logits(moe_dtype dt, const void* x, const float* w_r, const float* bias, int32_t N,
                             int32_t H, int32_t E, float* logits, void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  REQUIRE(N >= 0, MOE_EINVAL, "N must be >= 0 (got %d)", N);
  REQUIRE(E >= 1 && E <= 1024, MOE_EINVAL, "E must be in [1, 1024] (got %d)", E);
  REQUIRE(H >= 1, MOE_EINVAL, "H must be >= 1 (got %d)", H);
  REQUIRE((int64_t)N * (H + 8) * 2 <= kDescBytes && (int64_t)(H + 1) * (N + 8) * 2 <= kDescBytes, MOE_EUNSUPPORTED,
          "N*H too large for one router call (N=%d, H=%d: the operand planes exceed 2 GiB)", N, H);
  REQUIRE(N == 0 || (x && w_r && logits), MOE_EINVAL, "NULL x/w_r/logits");
  const size_t need = moe::router_logits_ws_bytes(dt, N, H, E);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  return hip_status(moe::launch_router_logits(dt, x, w_r, bias, N, H, E, logits, ws, (hipStream_t)stream),
                    "moe_router_logits");
}

moe_status moe_router_bwd_acc(moe_dtype dt, const float* logits, const float* bias, const int32_t* topk_idx,
                              const moe_plan* plan, const float* ds, const float* dlogits_in, const void* x,
                              const float* w_r, int32_t H, const void* dx_in, void* dx_out, float* dlogits,
                              float* dw_r, float* dbias, void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_dtype(dt)) != MOE_OK) return st;
  if ((st = check_plan(plan)) != MOE_OK) return st;
  REQUIRE(H >= 1, MOE_EINVAL, "H must be >= 1 (got %d)", H);
  const int32_t N = plan->N;
  REQUIRE(N == 0 || (logits && topk_idx && dlogits), MOE_EINVAL, "NULL logits/topk_idx/dlogits");
  REQUIRE(N == 0 || plan->M_cap == 0 || ds, MOE_EINVAL, "NULL ds");
  REQUIRE(!dx_out || (dx_in && w_r), MOE_EINVAL, "dx_out needs dx_in and w_r");
  REQUIRE(!(dw_r || dbias) || N == 0 || x, MOE_EINVAL, "dw_r / dbias need x");
  REQUIRE((int64_t)N * (H + 8) * 2 <= kDescBytes && (int64_t)(H + 1) * (N + 8) * 2 <= kDescBytes, MOE_EUNSUPPORTED,
          "N*H too large for one router call (N=%d, H=%d: the operand planes exceed 2 GiB)", N, H);
  if (dx_out || dw_r || dbias) {
    const size_t need = moe::router_bwd_ws_bytes(dt, N, H, plan->E);
    REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  }
  return hip_status(moe::launch_router_bwd(dt, logits, bias, topk_idx, *plan, ds, dlogits_in, x, w_r, H, dx_in, dx_out, dlogits,
                                           dw_r, dbias, ws, (hipStream_t)stream),
                    "moe_router_bwd");
}

moe_status moe_router_bwd(moe_dtype dt, const float* logits, const float* bias, const int32_t* topk_idx,
                          const moe_plan* plan, const float* ds, const void* x, const float* w_r, int32_t H,
                          const void* dx_in, void* dx_out, float* dlogits, float* dw_r, float* dbias, void* ws,
                          size_t ws_bytes, void* stream) {
  return moe_router_bwd_acc(dt, logits, bias, topk_idx, plan, ds, nullptr, x, w_r, H, dx_in, dx_out, dlogits, dw_r,
                            dbias, ws, ws_bytes, stream);
}

moe_status moe_add_rmsnorm(moe_dtype dt, moe_dtype rdt, const void* x, const void* res, const float* w, float eps,
                           int32_t N, int32_t H, void* h, void* y, uint8_t* q, uint8_t* scales, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_norm(dt, rdt, N, H)) != MOE_OK) return st;
  REQUIRE(eps >= 0.f && eps <= FLT_MAX, MOE_EINVAL, "eps must be finite and >= 0");
  REQUIRE(!q || H % 32 == 0, MOE_EUNSUPPORTED, "an MX-FP8 output needs H a multiple of 32 (got %d)", H);
  REQUIRE(h || y || q, MOE_EINVAL, "no output requested");
  REQUIRE((q != nullptr) == (scales != nullptr), MOE_EINVAL, "q and scales are given together or not at all");
  REQUIRE(N == 0 || x, MOE_EINVAL, "NULL x");
  REQUIRE(h == nullptr || h != x || rdt == dt, MOE_EINVAL, "h can be x only where their types agree");
  REQUIRE(y == nullptr || (y != h && y != x && y != res), MOE_EINVAL, "y must not be x, res or h");
  REQUIRE(aligned16(x) && aligned16(res) && aligned16(w) && aligned16(h) && aligned16(y) && aligned16(q),
          MOE_EUNSUPPORTED, "tensors must be 16-byte aligned");
  moe::kernel_event(MOE_K_ADD_RMSNORM, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_add_rmsnorm(dt, rdt, x, res, w, eps, N, H, h, y, q, scales, (hipStream_t)stream);
  moe::kernel_event(MOE_K_ADD_RMSNORM, 1, (hipStream_t)stream);
  return hip_status(e, "moe_add_rmsnorm");
}

moe_status moe_add_rmsnorm_bwd(moe_dtype dt, moe_dtype rdt, const void* dy, const void* h, const void* dh_in,
                               const float* w, float eps, int32_t N, int32_t H, void* dh, void* dx, float* dw,
                               void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_norm(dt, rdt, N, H)) != MOE_OK) return st;
  REQUIRE(eps >= 0.f && eps <= FLT_MAX, MOE_EINVAL, "eps must be finite and >= 0");
  REQUIRE(N == 0 || (dy && h && dh), MOE_EINVAL, "NULL dy/h/dh");
  REQUIRE(N == 0 || (dh != h && dh != dy && (!dx || (dx != dh && dx != h && dx != dh_in && dx != dy))), MOE_EINVAL,
          "dh may be dh_in; it and dx must be no other argument");
  REQUIRE(aligned16(dy) && aligned16(h) && aligned16(dh_in) && aligned16(w) && aligned16(dh) && aligned16(dx) &&
              aligned16(dw) && aligned16(ws),
          MOE_EUNSUPPORTED, "tensors and workspace must be 16-byte aligned");
  if (dw) {
    const size_t need = moe::add_rmsnorm_bwd_ws_bytes(N, H);
    REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  }
  moe::kernel_event(MOE_K_ADD_RMSNORM_BWD, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_add_rmsnorm_bwd(dt, rdt, dy, h, dh_in, w, eps, N, H, dh, dx, dw, ws, (hipStream_t)stream);
  moe::kernel_event(MOE_K_ADD_RMSNORM_BWD, 1, (hipStream_t)stream);
  return hip_status(e, "moe_add_rmsnorm_bwd");
}

moe_status moe_balance_loss(const float* logits, const float* bias, const int32_t* topk_idx, const uint8_t* mask,
                            const int32_t* seq_ptr, int32_t B, int32_t N, int32_t E, int32_t k, float alpha,
                            float beta, float* loss, int32_t* counts, float* saved, void* ws, size_t ws_bytes,
                            void* stream) {
  g_err[0] = 0;
  moe_status st = check_dims(N, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_seqs(B, E, seq_ptr)) != MOE_OK) return st;
  REQUIRE(alpha - alpha == 0.f && beta - beta == 0.f, MOE_EINVAL, "alpha and beta must be finite");
  REQUIRE(N == 0 || (logits && topk_idx), MOE_EINVAL, "NULL logits/topk_idx");
  REQUIRE(loss && counts && saved, MOE_EINVAL, "NULL loss/counts/saved");
  const size_t need = moe::balance_loss_ws_bytes(N, E, B);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  REQUIRE(aligned16(ws), MOE_EUNSUPPORTED, "the workspace must be 16-byte aligned");
  moe::kernel_event(MOE_K_BALANCE, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_balance_loss(logits, bias, topk_idx, mask, seq_ptr, B, N, E, k, alpha, beta, loss, counts,
                                          saved, ws, (hipStream_t)stream);
  moe::kernel_event(MOE_K_BALANCE, 1, (hipStream_t)stream);
  return hip_status(e, "moe_balance_loss");
}

moe_status moe_balance_loss_bwd(const float* logits, const float* bias, const uint8_t* mask, const int32_t* seq_ptr,
                                int32_t B, int32_t N, int32_t E, const float* saved, const float* dloss,
                                const float* dlogits_in, float* dlogits, void* stream) {
  g_err[0] = 0;
  moe_status st = check_dims(N, E, 1);
  if (st != MOE_OK) return st;
  if ((st = check_seqs(B, E, seq_ptr)) != MOE_OK) return st;
  REQUIRE(N == 0 || (logits && saved && dlogits), MOE_EINVAL, "NULL logits/saved/dlogits");
  REQUIRE(N == 0 || (dlogits != logits && dlogits != saved), MOE_EINVAL, "dlogits must not be logits or saved");
  moe::kernel_event(MOE_K_BALANCE_BWD, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_balance_loss_bwd(logits, bias, mask, seq_ptr, B, N, E, saved, dloss, dlogits_in, dlogits,
                                              (hipStream_t)stream);
  moe::kernel_event(MOE_K_BALANCE_BWD, 1, (hipStream_t)stream);
  return hip_status(e, "moe_balance_loss_bwd");
}

moe_status moe_linear_fwd(moe_dtype dt, const void* x, const void* w, const float* bias, int32_t act, const void* res,
                          int32_t N, int32_t K, int32_t O, void* out, void* z, void* ws, size_t ws_bytes,
                          void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_linear(dt, N, K, O)) != MOE_OK) return st;
  REQUIRE(act >= MOE_ACT_NONE && act <= MOE_ACT_GELU_TANH, MOE_EINVAL, "unknown activation %d", act);
  REQUIRE(w, MOE_EINVAL, "NULL w");
  REQUIRE(N == 0 || (x && out), MOE_EINVAL, "NULL x/out");
  REQUIRE(N == 0 || (out != x && out != w && (!z || (z != out && z != x && z != w && z != res))), MOE_EINVAL,
          "out may be res; it and z must be no other argument");
  REQUIRE(aligned16(x) && aligned16(w) && aligned16(bias) && aligned16(res) && aligned16(out) && aligned16(z) &&
              aligned16(ws),
          MOE_EUNSUPPORTED, "tensors and workspace must be 16-byte aligned");
  const size_t need = moe::linear_fwd_ws_bytes(dt, N, K, O);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  moe::kernel_event(MOE_K_LINEAR, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_linear_fwd(dt, x, w, bias, act, res, N, K, O, out, z, ws, (hipStream_t)stream);
  moe::kernel_event(MOE_K_LINEAR, 1, (hipStream_t)stream);
  return hip_status(e, "moe_linear_fwd");
}

moe_status moe_linear_bwd(moe_dtype dt, const void* dout, const void* x, const void* w, const void* z, int32_t act,
                          int32_t N, int32_t K, int32_t O, void* dx, void* dw, float* dbias, void* ws, size_t ws_bytes,
                          void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_linear(dt, N, K, O)) != MOE_OK) return st;
  REQUIRE(act >= MOE_ACT_NONE && act <= MOE_ACT_GELU_TANH, MOE_EINVAL, "unknown activation %d", act);
  REQUIRE(dx || dw || dbias, MOE_EINVAL, "no gradient requested");
  REQUIRE(N == 0 || dout, MOE_EINVAL, "NULL dout");
  REQUIRE(N == 0 || act == MOE_ACT_NONE || z, MOE_EINVAL, "an activation's backward needs z");
  REQUIRE(N == 0 || !dx || w, MOE_EINVAL, "dx needs w");
  REQUIRE(N == 0 || !dw || x, MOE_EINVAL, "dw needs x");
  REQUIRE(N == 0 || ((!dx || (dx != dout && dx != x && dx != w && dx != z && dx != dw)) &&
                     (!dw || (dw != dout && dw != x && dw != w && dw != z))),
          MOE_EINVAL, "dx and dw must be no other argument");
  REQUIRE(aligned16(dout) && aligned16(x) && aligned16(w) && aligned16(z) && aligned16(dx) && aligned16(dw) &&
              aligned16(dbias) && aligned16(ws),
          MOE_EUNSUPPORTED, "tensors and workspace must be 16-byte aligned");
  const size_t need = moe::linear_bwd_ws_bytes(dt, N, K, O);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  moe::kernel_event(MOE_K_LINEAR_BWD, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_linear_bwd(dt, dout, x, w, z, act, N, K, O, dx, dw, dbias, ws, (hipStream_t)stream);
  moe::kernel_event(MOE_K_LINEAR_BWD, 1, (hipStream_t)stream);
  return hip_status(e, "moe_linear_bwd");
}

moe_status moe_linear_ce_fwd(moe_dtype dt, const void* x, const void* w, const int32_t* targets, int32_t N, int32_t H,
                             int32_t V, float z_coef, float* loss, float* lse, void* ws, size_t ws_bytes,
                             void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_ce(dt, N, H, V)) != MOE_OK) return st;
  REQUIRE(z_coef - z_coef == 0.f, MOE_EINVAL, "z_coef must be finite");
  REQUIRE(w, MOE_EINVAL, "NULL w");
  REQUIRE(N == 0 || (x && targets && loss && lse), MOE_EINVAL, "NULL x/targets/loss/lse");
  REQUIRE(N == 0 || (apart(loss, x, w, targets, lse, ws) && apart(lse, x, w, targets, ws)), MOE_EINVAL,
          "loss and lse must be no other argument");
  REQUIRE(aligned16(x) && aligned16(w) && aligned16(ws), MOE_EUNSUPPORTED, "x, w and workspace must be 16-byte aligned");
  REQUIRE(aligned4(targets) && aligned4(loss) && aligned4(lse), MOE_EUNSUPPORTED,
          "targets, loss and lse must be 4-byte aligned");
  const size_t need = moe::linear_ce_fwd_ws_bytes(dt, N, H, V);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  moe::kernel_event(MOE_K_LINEAR_CE, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_linear_ce_fwd(dt, x, w, targets, N, H, V, z_coef, loss, lse, ws, (hipStream_t)stream);
  moe::kernel_event(MOE_K_LINEAR_CE, 1, (hipStream_t)stream);
  return hip_status(e, "moe_linear_ce_fwd");
}

moe_status moe_linear_ce_bwd(moe_dtype dt, const float* dloss, const void* x, const void* w, const int32_t* targets,
                             const float* lse, int32_t N, int32_t H, int32_t V, float z_coef, void* dx, void* dw,
                             void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_ce(dt, N, H, V)) != MOE_OK) return st;
  REQUIRE(z_coef - z_coef == 0.f, MOE_EINVAL, "z_coef must be finite");
  REQUIRE(dx || dw, MOE_EINVAL, "no gradient requested");
  REQUIRE(N == 0 || (x && w && targets && lse), MOE_EINVAL, "NULL x/w/targets/lse");
  REQUIRE(apart(dw, w, ws) && (N == 0 || (apart(dx, x, w, targets, lse, dloss, dw, ws) && apart(dw, x, targets, lse, dloss))),
          MOE_EINVAL, "dx and dw must be no other argument");
  REQUIRE(aligned16(x) && aligned16(w) && aligned16(dx) && aligned16(dw) && aligned16(ws), MOE_EUNSUPPORTED,
          "x, w, dx, dw and workspace must be 16-byte aligned");
  REQUIRE(aligned4(targets) && aligned4(lse) && aligned4(dloss), MOE_EUNSUPPORTED,
          "targets, lse and dloss must be 4-byte aligned");
  const size_t need = moe::linear_ce_bwd_ws_bytes(dt, N, H, V);
  REQUIRE(ws_bytes >= need, MOE_EWORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  REQUIRE(ws != nullptr, MOE_EINVAL, "NULL workspace");
  moe::kernel_event(MOE_K_LINEAR_CE_BWD, 0, (hipStream_t)stream);
  hipError_t e =
      moe::launch_linear_ce_bwd(dt, dloss, x, w, targets, lse, N, H, V, z_coef, dx, dw, ws, (hipStream_t)stream);
  moe::kernel_event(MOE_K_LINEAR_CE_BWD, 1, (hipStream_t)stream);
  return hip_status(e, "moe_linear_ce_bwd");
}

moe_status moe_layer_few(moe_dtype dt, const void* x, const float* w_r, const float* bias, const void* w_gate,
                         const void* w_up, const void* w_down, int32_t N, int32_t H, int32_t I, int32_t E, int32_t k,
                         void* out, int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_few(dt, N, H, I, E, k, 8)) != MOE_OK) return st;
  if ((st = check_few_args(dt, x, w_r, bias, w_gate, w_up, w_down, N, H, I, E, k, out, topk_idx, topk_w, ws, ws_bytes)) !=
      MOE_OK)
    return st;
  moe::kernel_event(MOE_K_LAYER_FEW, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_layer_few(dt, x, w_r, bias, w_gate, nullptr, w_up, nullptr, w_down, nullptr, N, H, I, E, k,
                                       out, topk_idx, topk_w, ws, (hipStream_t)stream);
  moe::kernel_event(MOE_K_LAYER_FEW, 1, (hipStream_t)stream);
  return hip_status(e, "moe_layer_few");
}

moe_status moe_layer_few_mxfp8(const void* x, const float* w_r, const float* bias, const uint8_t* wg_q,
                               const uint8_t* wg_s, const uint8_t* wu_q, const uint8_t* wu_s, const uint8_t* wd_q,
                               const uint8_t* wd_s, int32_t N, int32_t H, int32_t I, int32_t E, int32_t k, void* out,
                               int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  moe_status st;
  if ((st = check_few(MOE_BF16, N, H, I, E, k, 32)) != MOE_OK) return st;
  REQUIRE(wg_s && wu_s && wd_s, MOE_EINVAL, "NULL scale codes");
  REQUIRE(aligned4(wg_s) && aligned4(wu_s) && aligned4(wd_s), MOE_EUNSUPPORTED, "scale codes must be 4-byte aligned");
  if ((st = check_few_args(MOE_BF16, x, w_r, bias, wg_q, wu_q, wd_q, N, H, I, E, k, out, topk_idx, topk_w, ws,
                           ws_bytes)) != MOE_OK)
    return st;
  REQUIRE(N == 0 || (apart(out, wg_s, wu_s, wd_s) && apart(topk_idx, wg_s, wu_s, wd_s) && apart(topk_w, wg_s, wu_s, wd_s)),
          MOE_EINVAL, "out, topk_idx and topk_w must be no other argument");
  moe::kernel_event(MOE_K_LAYER_FEW, 0, (hipStream_t)stream);
  hipError_t e = moe::launch_layer_few(MOE_BF16, x, w_r, bias, wg_q, wg_s, wu_q, wu_s, wd_q, wd_s, N, H, I, E, k, out,
                                       topk_idx, topk_w, ws, (hipStream_t)stream);
  moe::kernel_event(MOE_K_LAYER_FEW, 1, (hipStream_t)stream);
  return hip_status(e, "moe_layer_few_mxfp8");
}

}  // extern "C"
