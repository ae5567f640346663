// api_operators.cpp — the C-ABI of the operators around the block GEMM: the GEMM with an epilogue,
// the router and the whole mixture-of-experts layer.
// Validation as in api.cpp: synchronous, before anything is enqueued.
#include "api_common.hpp"

using namespace fgb_api;

namespace {

bool is_out_dtype(int d) { return d == FGB_OUT_BF16 || d == FGB_OUT_F32; }
int64_t dtype_bytes(int d) { return d == FGB_OUT_BF16 ? 2 : 4; }

// (T * top_k pairs, E experts and a row's block scales fit the kernels' tables)
bool moe_shape_ok(int64_t T, int64_t top_k, int64_t E, int64_t H, int64_t I) {
  if (T < 0 || T > fgb::kMoeMaxTokens || top_k < 1 || top_k > fgb::kMoeMaxPairs || E < 1 || E > fgb::kMoeMaxExperts)
    return false;
  if (T * top_k > fgb::kMoeMaxPairs || H <= 0 || I <= 0 || H % FGB_BLOCK || I % FGB_BLOCK) return false;
  return H <= 32768 && I <= 32768;
}

}  // namespace

extern "C" {

int fgb_w8a8_block_gemm_epilogue(const uint8_t* a_q, int64_t lda, const float* s_a, int64_t ld_sa,
                                 const uint8_t* w_q, const void* s_w, int s_w_fmt, const void* bias, int bias_dtype,
                                 int activation, const void* residual, int residual_dtype, int64_t ldr, void* y,
                                 int y_dtype, int64_t ldy, int64_t M, int64_t N, int64_t K, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  int st = validate_gemm(a_q, lda, s_a, ld_sa, w_q, s_w, s_w_fmt, y, y_dtype, ldy, M, N, K);
  if (st != FGB_OK) return st;
  if (activation < FGB_ACT_NONE || activation > FGB_ACT_SILU) return FGB_ERR_ENUM;
  if (bias && !is_out_dtype(bias_dtype)) return FGB_ERR_ENUM;
  if (residual && !is_out_dtype(residual_dtype)) return FGB_ERR_ENUM;
  if (M == 0) return FGB_OK;
  if (bias && !aligned16(bias)) return FGB_ERR_ALIGN;
  if (residual) {
    if (ldr < N) return FGB_ERR_STRIDE;
    if (!aligned16(residual) || (ldr * dtype_bytes(residual_dtype)) % 16) return FGB_ERR_ALIGN;
    // in place: every element is read and written by one thread, which needs one layout
    if (residual == y && (residual_dtype != y_dtype || ldr != ldy)) return FGB_ERR_STRIDE;
  }
  const bool decode = fgb::use_decode(M, K);
  const size_t need = decode ? fgb::decode_workspace_bytes(M, N, K) : fgb::prefill_workspace_bytes(M, N, K);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FGB_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return FGB_ERR_ALIGN;
  st = check_device();
  if (st != FGB_OK) return st;
  fgb::GemmEpiArgs a;
  static_cast<fgb::GemmArgs&>(a) =
      fgb::GemmArgs{a_q, lda, s_a, ld_sa, w_q, s_w, s_w_fmt, y, y_dtype, ldy, M, N, K, nullptr, 1};
  a.ep = fgb::Epilogue{bias, bias_dtype, activation, residual, residual_dtype, ldr};
  if (decode) return launch_status(fgb::launch_gemm_epilogue_decode(a, workspace, (hipStream_t)stream));
  return launch_status(fgb::launch_gemm_epilogue_prefill(a, workspace, (hipStream_t)stream));
}

int fgb_moe_route(const void* logits, int logits_dtype, int64_t ld, int64_t T, int32_t E, int32_t top_k, int scoring,
                  const float* select_bias, int renormalize, float scale, int32_t* ids, float* weights, void* stream) {
  if (T < 0 || T >= kMaxDim || E < 1 || E > fgb::kRouteMaxExperts) return FGB_ERR_SHAPE;
  if (top_k < 1 || top_k > E || top_k > fgb::kRouteMaxTopK) return FGB_ERR_SHAPE;
  if (!is_out_dtype(logits_dtype)) return FGB_ERR_ENUM;
  if (scoring != FGB_SCORE_SOFTMAX && scoring != FGB_SCORE_SIGMOID) return FGB_ERR_ENUM;
  if (T == 0) return FGB_OK;
  if (!logits || !ids || !weights) return FGB_ERR_NULL;
  if (ld < E) return FGB_ERR_STRIDE;
  if ((uintptr_t)logits % dtype_bytes(logits_dtype) || ((uintptr_t)select_bias & 3u) || ((uintptr_t)ids & 3u) ||
      ((uintptr_t)weights & 3u))
    return FGB_ERR_ALIGN;
  int st = check_device();
  if (st != FGB_OK) return st;
  const fgb::RouteArgs a{logits, logits_dtype, ld, T, E, top_k, scoring, select_bias, renormalize != 0, scale, ids, weights};
  return launch_status(fgb::launch_moe_route(a, (hipStream_t)stream));
}

size_t fgb_moe_ffn_workspace_bytes(int64_t T, int32_t top_k, int32_t E, int64_t H, int64_t I) {
  if (T == 0 || !moe_shape_ok(T, top_k, E, H, I)) return 0;
  return fgb::moe_ffn_workspace_bytes((int)T, top_k, E, (int)H, (int)I);
}

int fgb_moe_ffn(const uint16_t* x, int64_t ldx, const int32_t* ids, const float* weights, int32_t top_k,
                const uint8_t* w13_q, const void* s_w13, const uint8_t* w2_q, const void* s_w2, int s_w_fmt, int32_t E,
                int activation, const void* residual, int residual_dtype, int64_t ldr, void* y, int y_dtype,
                int64_t ldy, int64_t T, int64_t H, int64_t I, void* workspace, size_t workspace_bytes, void* stream) {
  if (!moe_shape_ok(T, top_k, E, H, I)) return FGB_ERR_SHAPE;
  if (s_w_fmt != FGB_SCALE_F32 && s_w_fmt != FGB_SCALE_UE8M0) return FGB_ERR_ENUM;
  if (activation != FGB_ACT_SILU && activation != FGB_ACT_GELU && activation != FGB_ACT_GELU_TANH) return FGB_ERR_ENUM;
  if (!is_out_dtype(y_dtype) || (residual && !is_out_dtype(residual_dtype))) return FGB_ERR_ENUM;
  if (T == 0) return FGB_OK;
  if (!x || !ids || !weights || !w13_q || !s_w13 || !w2_q || !s_w2 || !y) return FGB_ERR_NULL;
  if (ldx < H || ldy < H || (residual && ldr < H)) return FGB_ERR_STRIDE;
  if (!aligned16(x) || !aligned16(w13_q) || !aligned16(w2_q) || !aligned16(y) || (ldx * 2) % 16 ||
      (ldy * dtype_bytes(y_dtype)) % 16)
    return FGB_ERR_ALIGN;
  if (((uintptr_t)ids & 3u) || ((uintptr_t)weights & 3u)) return FGB_ERR_ALIGN;
  if (s_w_fmt == FGB_SCALE_F32 && (((uintptr_t)s_w13 & 3u) || ((uintptr_t)s_w2 & 3u))) return FGB_ERR_ALIGN;
  if (residual) {
    if (!aligned16(residual) || (ldr * dtype_bytes(residual_dtype)) % 16) return FGB_ERR_ALIGN;
    if (residual == y && (residual_dtype != y_dtype || ldr != ldy)) return FGB_ERR_STRIDE;
  }
  const size_t need = fgb::moe_ffn_workspace_bytes((int)T, top_k, E, (int)H, (int)I);
  if (workspace == nullptr || workspace_bytes < need) return FGB_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FGB_ERR_ALIGN;
  int st = check_device();
  if (st != FGB_OK) return st;
  const fgb::MoeArgs a{x,    ldx,        ids,      weights,        w13_q, s_w13, w2_q,    s_w2, s_w_fmt, activation,
                       residual, residual_dtype, ldr, y, y_dtype, ldy, (int)T, top_k, E, (int)H, (int)I};
  return launch_status(fgb::launch_moe_ffn(a, workspace, (hipStream_t)stream));
}

}  // extern "C"
