// api_common.hpp — argument checks shared by the C-ABI's translation units: limits, alignment, the
// device check and the validation of the block GEMM's operands.
#pragma once
#include <hip/hip_runtime.h>
#include <string.h>

#include "../../include/fgb.h"
#include "internal.h"

namespace fgb_api {

constexpr int64_t kMaxDim = (int64_t)1 << 31;  // grid and index arithmetic bound
constexpr int64_t kMax32 = (int64_t)1 << 32;   // bytes addressable by a 32-bit offset
constexpr int kMaxDevices = 64;
constexpr int kMaxExperts = 65535;  // experts index grid.y in the per-expert decode kernels

// 0 = unknown, 1 = gfx950, -1 = other
inline int g_dev_ok[kMaxDevices];

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline int check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
    (void)hipGetLastError();
    return FGB_ERR_DEVICE;
  }
  if (g_dev_ok[dev] == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      (void)hipGetLastError();
      return FGB_ERR_DEVICE;
    }
    g_dev_ok[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
  }
  return g_dev_ok[dev] == 1 ? FGB_OK : FGB_ERR_DEVICE;
}

inline int launch_status(hipError_t e) { return e == hipSuccess ? FGB_OK : FGB_ERR_LAUNCH; }

// Shared validation of the GEMM operands (dense: E = 1, offsets unused).
inline int validate_gemm(const uint8_t* a_q, int64_t lda, const float* s_a, int64_t ld_sa,
                         const uint8_t* w_q, const void* s_w, int s_w_fmt, const void* y, int y_dtype,
                         int64_t ldy, int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N <= 0 || K <= 0 || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return FGB_ERR_SHAPE;
  if (N % FGB_BLOCK || K % FGB_BLOCK) return FGB_ERR_SHAPE;
  if (s_w_fmt != FGB_SCALE_F32 && s_w_fmt != FGB_SCALE_UE8M0) return FGB_ERR_ENUM;
  if (y_dtype != FGB_OUT_BF16 && y_dtype != FGB_OUT_F32) return FGB_ERR_ENUM;
  if (M == 0) return FGB_OK;
  if (!a_q || !s_a || !w_q || !s_w || !y) return FGB_ERR_NULL;
  if (lda < K || ldy < N || ld_sa < M) return FGB_ERR_STRIDE;
  const int64_t ybytes = y_dtype == FGB_OUT_BF16 ? 2 : 4;
  if (!aligned16(a_q) || !aligned16(s_a) || !aligned16(w_q) || !aligned16(s_w) || !aligned16(y))
    return FGB_ERR_ALIGN;
  if (lda % 16 || (ldy * ybytes) % 16 || (ld_sa * 4) % 16) return FGB_ERR_ALIGN;
  // the kernels address A, one expert's W and the scales with 32-bit offsets, and hold a weight
  // row's K/128 block scales in registers (K <= 32768)
  if (M * lda >= kMax32 || N * K >= kMax32 || (K / FGB_BLOCK) * ld_sa * 4 >= kMax32) return FGB_ERR_SHAPE;
  if (K > 32768) return FGB_ERR_SHAPE;
  return FGB_OK;
}

}  // namespace fgb_api
