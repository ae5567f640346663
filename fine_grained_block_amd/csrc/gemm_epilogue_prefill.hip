// gemm_epilogue_prefill.hip — prefill launches of the dense block-scaled GEMM with bias, activation
// and residual in its epilogue (kernels and tile choice of the plain GEMM).
#include "gemm_prefill_launch.hpp"

namespace fgb {

hipError_t launch_gemm_epilogue_prefill(const GemmEpiArgs& a, void* workspace, hipStream_t stream) {
  return launch_prefill_kernels(a, workspace, stream);
}

}  // namespace fgb
