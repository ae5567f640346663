// gemm_epilogue_decode.hip — decode launches of the dense block-scaled GEMM with bias, activation and
// residual in its epilogue (kernels and kernel choice of the plain GEMM).
#include "gemm_decode_launch.hpp"

namespace fgb {

hipError_t launch_gemm_epilogue_decode(const GemmEpiArgs& a, void* workspace, hipStream_t stream) {
  return launch_decode_kernels(a, workspace, stream);
}

hipError_t launch_splitk_reduce_epilogue(const float* ws, int S, const GemmEpiArgs& a, hipStream_t stream) {
  const int64_t total = a.M * (a.N / 4);
  const dim3 rgrid((unsigned)((total + 255) / 256));
  if (a.y_dtype == 0)
    hipLaunchKernelGGL(splitk_reduce_epilogue_kernel<0>, rgrid, dim3(256), 0, stream, ws, S, a);
  else
    hipLaunchKernelGGL(splitk_reduce_epilogue_kernel<1>, rgrid, dim3(256), 0, stream, ws, S, a);
  return hipGetLastError();
}

}  // namespace fgb
