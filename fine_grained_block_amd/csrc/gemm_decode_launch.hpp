// gemm_decode_launch.hpp — kernel choice and launches of the dense decode GEMM, for GemmArgs and for
// GemmEpiArgs (the same choice for both: the epilogue is a few operations per output).
#pragma once
#include "gemm_decode_kernels.hpp"

namespace fgb {

namespace {

template <typename Args>
hipError_t launch_decode_kernels(const Args& a, void* workspace, hipStream_t stream) {
  if (a.M <= 16 && decode_ring(a.N, a.K)) {
    const int wk = decode_small_waves(a.N, a.K);
    const dim3 grid((unsigned)(a.N / 16));
#define FGB_RING(WK, SWF, OUT)                                                                              \
  do {                                                                                                      \
    if (a.M <= 8) hipLaunchKernelGGL((gemm_decode_ring_kernel<WK, 8, 5, SWF, OUT, 0, 0, Args>), grid, dim3(64 * WK), 0, stream, a); \
    else hipLaunchKernelGGL((gemm_decode_ring_kernel<WK, 16, 4, SWF, OUT, 0, 0, Args>), grid, dim3(64 * WK), 0, stream, a);         \
  } while (0)
#define FGB_RING_WK(SWF, OUT)                  \
  do {                                         \
    if (wk == 1) FGB_RING(1, SWF, OUT);        \
    else if (wk == 2) FGB_RING(2, SWF, OUT);   \
    else if (wk == 4) FGB_RING(4, SWF, OUT);   \
    else FGB_RING(8, SWF, OUT);                \
  } while (0)
    if (a.s_w_fmt == 0) {
      if (a.y_dtype == 0) FGB_RING_WK(0, 0); else FGB_RING_WK(0, 1);
    } else {
      if (a.y_dtype == 0) FGB_RING_WK(1, 0); else FGB_RING_WK(1, 1);
    }
#undef FGB_RING_WK
#undef FGB_RING
    return hipGetLastError();
  }
  if (a.M > 16 && a.M <= 64 && ring_mid_rows(a.N, a.K)) {
    const dim3 grid((unsigned)(a.N / 16));
#define FGB_RING_MID(SWF, OUT)                                                                                   \
  do {                                                                                                           \
    if (a.M <= 32) hipLaunchKernelGGL((gemm_decode_ring_kernel<4, 32, 3, SWF, OUT, 0, 0, Args>), grid, dim3(256), 0, stream, a); \
    else hipLaunchKernelGGL((gemm_decode_ring_kernel<4, 64, 2, SWF, OUT, 0, 0, Args>), grid, dim3(256), 0, stream, a);           \
  } while (0)
    if (a.s_w_fmt == 0) {
      if (a.y_dtype == 0) FGB_RING_MID(0, 0); else FGB_RING_MID(0, 1);
    } else {
      if (a.y_dtype == 0) FGB_RING_MID(1, 0); else FGB_RING_MID(1, 1);
    }
#undef FGB_RING_MID
    return hipGetLastError();
  }
  if (a.M <= 16) {
    const int wk = decode_small_waves(a.N, a.K);
    const dim3 grid((unsigned)(a.N / 16));
#define FGB_SMALL(WK, SWF, OUT) \
  hipLaunchKernelGGL((gemm_decode_small_kernel<WK, SWF, OUT, 0, 0, 0, 1, Args>), grid, dim3(64 * WK), 0, stream, a)
#define FGB_SMALL_WK(SWF, OUT)                  \
  do {                                          \
    if (wk == 1) FGB_SMALL(1, SWF, OUT);        \
    else if (wk == 2) FGB_SMALL(2, SWF, OUT);   \
    else if (wk == 4) FGB_SMALL(4, SWF, OUT);   \
    else FGB_SMALL(8, SWF, OUT);                \
  } while (0)
    if (a.s_w_fmt == 0) {
      if (a.y_dtype == 0) FGB_SMALL_WK(0, 0); else FGB_SMALL_WK(0, 1);
    } else {
      if (a.y_dtype == 0) FGB_SMALL_WK(1, 0); else FGB_SMALL_WK(1, 1);
    }
#undef FGB_SMALL_WK
#undef FGB_SMALL
    return hipGetLastError();
  }
  {
    const int S = decode_splits(a.M, a.N, a.K);
    const int nw = mid_waves(a.M, a.N, a.K);
    const int kpw = S == 1 ? (int)(a.K / 128) : mid_kpw(a.N, a.K);
    const dim3 grid((unsigned)((a.N / (16 * nw)) * S)), block(64 * nw);
    float* ws = reinterpret_cast<float*>(workspace);
#define FGB_MID(NW_, MT_, D_, SWF, OUT) \
  hipLaunchKernelGGL((gemm_decode_mid_kernel<NW_, MT_, D_, SWF, OUT, 0, 0, Args>), grid, block, 0, stream, a, kpw, S, ws)
#define FGB_MID_MT(SWF, OUT)                                    \
  do {                                                          \
    if (a.M > 64) FGB_MID(8, 8, kMidStages, SWF, OUT);          \
    else if (a.M > 32) FGB_MID(8, 4, kMidStages, SWF, OUT);     \
    else if (nw == 2) FGB_MID(2, 2, 6, SWF, OUT);               \
    else if (nw == 4) FGB_MID(4, 2, 4, SWF, OUT);               \
    else FGB_MID(8, 2, kMidStages, SWF, OUT);                   \
  } while (0)
    if (a.s_w_fmt == 0) {
      if (a.y_dtype == 0) FGB_MID_MT(0, 0); else FGB_MID_MT(0, 1);
    } else {
      if (a.y_dtype == 0) FGB_MID_MT(1, 0); else FGB_MID_MT(1, 1);
    }
#undef FGB_MID_MT
#undef FGB_MID
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || S == 1) return err;
    if constexpr (Args::kEpilogue) return launch_splitk_reduce_epilogue(ws, S, a, stream);
    else return launch_splitk_reduce(ws, S, a.M, a.N, a.y, a.y_dtype, a.ldy, stream);
  }
}

}  // namespace

}  // namespace fgb
