// api_operators.cpp — the C-ABI of the operators around the block GEMM: the GEMM with an epilogue.
// Validation as in api.cpp: synchronous, before anything is enqueued.
#include "api_common.hpp"

using namespace fgb_api;

namespace {

bool is_out_dtype(int d) { return d == FGB_OUT_BF16 || d == FGB_OUT_F32; }
int64_t dtype_bytes(int d) { return d == FGB_OUT_BF16 ? 2 : 4; }

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

}  // extern "C"
