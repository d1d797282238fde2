// C ABI of the operators beside the layer forward (declared in include/moe_ops.h):
// argument checks and launches.
#include <cmath>

#include "../../include/moe_ops.h"
#include "api_common.hpp"
#include "launch.hpp"

namespace {

using moe::current_device;
using moe::fail;
using moe::hip_status;

inline hipStream_t S(void* s) { return static_cast<hipStream_t>(s); }

bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }

size_t align_up(size_t v) { return (v + 255) & ~size_t(255); }

moe::FewDtype few_dt(moe_dtype dt) { return dt == MOE_BF16 ? moe::kFewBf16 : moe::kFewF32; }

bool float_dt(moe_dtype dt) { return dt == MOE_BF16 || dt == MOE_F32; }

int v_group(const char* fn, int group) {
  REQUIRE(group == 32 || group == 64 || group == 128, "%s: group must be 32, 64 or 128 (got %d)",
          fn, group);
  return MOE_OK;
}

int v_router(const char* fn, int T, int E, int k, int B, const int32_t* offsets) {
  REQUIRE(T >= 0 && T <= (1 << 30), "%s: T must be in [0, 2^30] (got %d)", fn, T);
  REQUIRE(E >= 1 && E <= 1024, "%s: E must be in [1, 1024] (got %d)", fn, E);
  REQUIRE(k >= 1 && k <= E && k <= 64, "%s: k must be in [1, min(E, 64)] (got %d)", fn, k);
  REQUIRE(B >= 1 && B <= 65535, "%s: B must be in [1, 65535] (got %d)", fn, B);
  REQUIRE(offsets || B == 1, "%s: B > 1 needs offsets", fn);
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_quant_weight_int4_group(const float* w, int G, int N, int K, int group, uint8_t* q,
                                float* s7, void* stream) {
  REQUIRE(w && q && s7, "moe_quant_weight_int4_group: null pointer");
  int st = v_group("moe_quant_weight_int4_group", group);
  if (st) return st;
  REQUIRE(G >= 1 && N >= 1, "moe_quant_weight_int4_group: bad G/N");
  REQUIRE(K >= group && K % group == 0,
          "moe_quant_weight_int4_group: K must be a positive multiple of group (got %d)", K);
  // one thread per word of 8 codes, fewer than 2^32 threads a launch
  REQUIRE((long long)G * N <= ((1LL << 32) - 256) / (K / 8),
          "moe_quant_weight_int4_group: G * N * K too large (at most about 2^35 weights a call)");
  REQUIRE(aligned(w, 16) && aligned(q, 16),
          "moe_quant_weight_int4_group: w and q must be 16-byte aligned");
  if ((st = current_device(nullptr))) return st;
  return hip_status(moe::launch_quant_weight_int4_group(w, G, N, K, group, q, s7, S(stream)),
                    "int4 group quant launch");
}

int moe_matvec_int4(const void* x, moe_dtype x_dt, int x_div, const uint8_t* q, const float* s7,
                    int group, const int32_t* idx, int n_slots, int G, int N, int K, int epilogue,
                    void* y, moe_dtype y_dt, void* stream) {
  REQUIRE(n_slots >= 0 && n_slots <= MOE_FEW_SLOTS_MAX,
          "moe_matvec_int4: S must be in [0, %d] (got %d; use the grouped GEMMs for more)",
          MOE_FEW_SLOTS_MAX, n_slots);
  REQUIRE(q && s7 && (n_slots == 0 || (x && y)), "moe_matvec_int4: null pointer");
  REQUIRE(float_dt(x_dt) && float_dt(y_dt), "moe_matvec_int4: dtypes must be MOE_BF16 or MOE_F32");
  int st = v_group("moe_matvec_int4", group);
  if (st) return st;
  REQUIRE(x_div >= 1 && (idx || x_div == 1),
          "moe_matvec_int4: x_div must be >= 1, and 1 without idx (got %d)", x_div);
  REQUIRE(G >= 1 && G <= 65536, "moe_matvec_int4: G must be in [1, 65536] (got %d)", G);
  REQUIRE(N >= 1 && N <= (1 << 24), "moe_matvec_int4: N must be in [1, 2^24] (got %d)", N);
  REQUIRE(K >= group && K % group == 0,
          "moe_matvec_int4: K must be a positive multiple of group (got %d)", K);
  REQUIRE(epilogue == MOE_EPI_PLAIN || epilogue == MOE_EPI_SWIGLU,
          "moe_matvec_int4: unknown epilogue %d", epilogue);
  REQUIRE(K <= (1 << 24), "moe_matvec_int4: K must be <= 2^24 (got %d)", K);
  REQUIRE(aligned(x, 16) && aligned(q, 16), "moe_matvec_int4: x and q must be 16-byte aligned");
  if (n_slots == 0) return MOE_OK;
  if ((st = current_device(nullptr))) return st;
  return hip_status(moe::launch_matvec_int4(x, few_dt(x_dt), x_div, q, s7, group, idx, n_slots, G,
                                            N, K, epilogue == MOE_EPI_SWIGLU, y, few_dt(y_dt),
                                            S(stream)),
                    "matvec launch");
}

size_t moe_ffn_int4_workspace_size(int T, int k, int d, int I) {
  if (T <= 0 || k < 1 || d < 1 || I < 1 || (long long)T * k > MOE_FEW_SLOTS_MAX) return 0;
  const size_t slots = (size_t)T * k;
  return align_up(slots * I * 6) + align_up(slots * d * 4);   // h in three parts, o
}

int moe_ffn_int4(const void* x, moe_dtype dt, const uint8_t* w13, const float* s13,
                 const uint8_t* w2, const float* s2, int group, const int32_t* topk_idx,
                 const float* topk_w, int T, int k, int E, int d, int I, void* y, void* ws,
                 size_t ws_bytes, void* stream) {
  REQUIRE(T >= 0 && k >= 1 && (long long)T * k <= MOE_FEW_SLOTS_MAX,
          "moe_ffn_int4: T >= 0, k >= 1 and T * k <= %d (got %d, %d; use moe_layer_fwd for more)",
          MOE_FEW_SLOTS_MAX, T, k);
  REQUIRE(w13 && s13 && w2 && s2 && (T == 0 || (x && y && topk_idx && topk_w && ws)),
          "moe_ffn_int4: null pointer");
  REQUIRE(float_dt(dt), "moe_ffn_int4: dt must be MOE_BF16 or MOE_F32");
  int st = v_group("moe_ffn_int4", group);
  if (st) return st;
  REQUIRE(E >= 1 && E <= 65536, "moe_ffn_int4: E must be in [1, 65536] (got %d)", E);
  REQUIRE(d >= group && d % group == 0 && I >= group && I % group == 0,
          "moe_ffn_int4: d and I must be positive multiples of group (got %d, %d)", d, I);
  REQUIRE(d <= (1 << 24) && I <= (1 << 24), "moe_ffn_int4: d and I must be <= 2^24");
  REQUIRE(aligned(x, 16) && aligned(w13, 16) && aligned(w2, 16) && aligned(ws, 16),
          "moe_ffn_int4: x, w13, w2 and ws must be 16-byte aligned");
  if (T == 0) return MOE_OK;
  const size_t need = moe_ffn_int4_workspace_size(T, k, d, I);
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "moe_ffn_int4: workspace %zu < %zu bytes", ws_bytes, need);
  if ((st = current_device(nullptr))) return st;
  const int slots = T * k;
  // h is fp32 kept as three bf16 rows a slot, the form the down product multiplies
  float* o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align_up((size_t)slots * I * 6));
  if ((st = hip_status(moe::launch_matvec_int4(x, few_dt(dt), k, w13, s13, group, topk_idx, slots,
                                               E, I, d, true, ws, moe::kFewParts, S(stream)),
                       "ffn gate/up launch")))
    return st;
  // While a workgroup per token and 16 outputs fits the chip at once, the down products are not
  // gathered by expert: a token's are joined in one kernel, without o and the combine.  One
  // token, 8 of 256 experts, 7168 x 2048 (448 workgroups): 52.5 us the whole FFN, 55.6 gathered;
  // 8 tokens, 6 of 64 experts, 1024 x 512 (512): 17.4, 22.2; 32 tokens, 2 of 8, 256 x 512 (512):
  // 13.3, 14.8.  Beyond that reading each weight once counts: 16 tokens, 1 of 64, 1024 x 512
  // (1024): 18.3, 17.5; 8 tokens, 1 of 64, 4096 x 2048 (2048): 42.7, 33.9.
  if ((long long)((d + 15) / 16) * T <= 512)
    return hip_status(moe::launch_join_int4(ws, w2, s2, group, topk_idx, topk_w, T, k, E, d, I, y,
                                            dt == MOE_BF16, S(stream)),
                      "ffn down launch");
  if ((st = hip_status(moe::launch_matvec_int4(ws, moe::kFewParts, 1, w2, s2, group, topk_idx,
                                               slots, E, d, I, false, o, moe::kFewF32, S(stream)),
                       "ffn down launch")))
    return st;
  return hip_status(moe::launch_few_combine(o, topk_idx, topk_w, T, k, E, d, y, dt == MOE_BF16,
                                            S(stream)),
                    "ffn combine launch");
}

size_t moe_balance_workspace_size(int T, int E, int B) {
  if (T < 0 || T > (1 << 30) || E < 1 || E > 1024 || B < 1 || B > 65535) return 0;
  return moe::balance_ws_bytes(T, E, B);
}

size_t moe_route_bwd_workspace_size(int T, int E) {
  if (T < 0 || T > (1 << 30) || E < 1 || E > 1024) return 0;
  return align_up((size_t)moe::route_bwd_blocks(T) * E * 4);
}

int moe_balance_loss(const float* logits, const float* bias, const int32_t* topk_idx,
                     const uint8_t* mask, const int32_t* offsets, int T, int E, int k, int B,
                     int kind, float coef, int32_t* counts, float* probs, float* grad, float* loss,
                     void* ws, size_t ws_bytes, void* stream) {
  int st = v_router("moe_balance_loss", T, E, k, B, offsets);
  if (st) return st;
  REQUIRE(((logits && topk_idx) || T == 0) && counts && probs && grad && loss && ws,
          "moe_balance_loss: null pointer");
  REQUIRE(kind == MOE_BALANCE_SWITCH || kind == MOE_BALANCE_SQUARE,
          "moe_balance_loss: unknown kind %d", kind);
  REQUIRE(std::isfinite(coef), "moe_balance_loss: coef must be finite");
  REQUIRE(aligned(ws, 16), "moe_balance_loss: ws must be 16-byte aligned");
  const size_t need = moe_balance_workspace_size(T, E, B);
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "moe_balance_loss: workspace %zu < %zu bytes", ws_bytes, need);
  if ((st = current_device(nullptr))) return st;
  return hip_status(moe::launch_balance_loss(logits, bias, topk_idx, mask, offsets, T, E, k, B,
                                             kind == MOE_BALANCE_SQUARE, coef, counts, probs, grad,
                                             loss, ws, S(stream)),
                    "balance loss launch");
}

int moe_route_bwd(const float* logits, const float* bias, const int32_t* topk_idx,
                  const float* dtopk_w, const uint8_t* mask, const int32_t* offsets,
                  const float* balance_grad, const float* dloss, int T, int E, int k, int B,
                  unsigned flags, float* dlogits, float* dbias, void* ws, size_t ws_bytes,
                  void* stream) {
  int st = v_router("moe_route_bwd", T, E, k, B, offsets);
  if (st) return st;
  REQUIRE((flags & ~MOE_ROUTE_RENORM) == 0, "moe_route_bwd: unknown route flags 0x%x", flags);
  REQUIRE((logits && dlogits) || T == 0, "moe_route_bwd: null pointer");
  REQUIRE(dtopk_w || balance_grad || T == 0, "moe_route_bwd: dtopk_w or balance_grad is needed");
  REQUIRE(!dtopk_w || topk_idx || T == 0, "moe_route_bwd: dtopk_w needs topk_idx");
  if (dbias) {
    REQUIRE(ws, "moe_route_bwd: dbias needs a workspace");
    REQUIRE(aligned(ws, 16), "moe_route_bwd: ws must be 16-byte aligned");
    const size_t need = moe_route_bwd_workspace_size(T, E);
    if (ws_bytes < need)
      return fail(MOE_ERR_WORKSPACE, "moe_route_bwd: workspace %zu < %zu bytes", ws_bytes, need);
  }
  if (T == 0 && !dbias) return MOE_OK;
  if ((st = current_device(nullptr))) return st;
  return hip_status(moe::launch_route_bwd(logits, bias, topk_idx, dtopk_w, mask, offsets,
                                          balance_grad, dloss, T, E, k, B,
                                          flags & MOE_ROUTE_RENORM, dlogits, dbias, ws, S(stream)),
                    "route backward launch");
}

}  // extern "C"
