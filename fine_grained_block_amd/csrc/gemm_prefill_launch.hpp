// gemm_prefill_launch.hpp — launches of the dense prefill GEMM, for GemmArgs and for GemmEpiArgs (the
// same tiles, column split and K slices for both), and the pieces the grouped launch shares.
#pragma once
#include "gemm_prefill_kernels.hpp"

namespace fgb {

namespace {

template <typename C, bool GROUPED, typename Args>
hipError_t launch_cfg(const Args& a, int tiles_m, hipStream_t stream) {
  const int tiles_n = (int)(a.N / C::BN);
  // grouped: tiles_m is an upper bound; a multiple of 8 workgroups gives every XCD at least its
  // share of the real tiles
  const int nwg = GROUPED ? (tiles_m * tiles_n + 7) / 8 * 8 : tiles_m * tiles_n;
  dim3 grid(nwg), block(C::THREADS);
#define FGB_LAUNCH(SWF, OUT)                                                                  \
  hipLaunchKernelGGL((gemm_prefill_kernel<C, SWF, OUT, GROUPED, 0, 0, false, Args>), grid, block, 0, stream, a, \
                     tiles_m, tiles_n)
  if (a.s_w_fmt == 0 && a.y_dtype == 0) FGB_LAUNCH(0, 0);
  else if (a.s_w_fmt == 0) FGB_LAUNCH(0, 1);
  else if (a.y_dtype == 0) FGB_LAUNCH(1, 0);
  else FGB_LAUNCH(1, 1);
#undef FGB_LAUNCH
  return hipGetLastError();
}

template <typename C>
int64_t tiles_for(int64_t M, int64_t N) { return ((M + C::BM - 1) / C::BM) * (N / C::BN); }

// The persistent form for more 256 x 256 tiles than CUs when K has at most max_kb blocks.  Dense
// (16 blocks), where the work between tiles weighs most: measured +4-7% at 12-16 blocks; at 32
// (gate+up) +2% alone but 0.5% slower inside the Llama step, and 0.2-1.5% slower at 56-144
// blocks.  Grouped (64 blocks): a one-tile launch also looks up each tile's expert when it
// starts, which the persistent form does from registers; MoE gate+up (56 blocks) +2-4%.  An even
// K-block count (a multiple of 4 with UE8M0 scales, copied four to a dword), bf16 output and
// 32-bit output offsets.
bool use_persistent(const GemmArgs& a, int64_t max_kb) {
  const int64_t KB = a.K / KBYTES, tiles = tiles_for<Big>(a.M, a.N);
  return tiles > cu_count() && KB <= max_kb && KB % 2 == 0 && (a.s_w_fmt == 0 || KB % 4 == 0) && a.y_dtype == 0 &&
         a.M * a.ldy * 2 < (int64_t(1) << 32);
}

template <typename Args>
hipError_t launch_prefill_kernels(const Args& a, void* workspace, hipStream_t stream) {
  const int S = prefill_splits(a.M, a.N, a.K);
  if (S > 1) {
    float* ws = reinterpret_cast<float*>(workspace);
    const hipError_t e = launch_prefill_slices(a, S, ws, stream);
    if (e != hipSuccess) return e;
    if constexpr (Args::kEpilogue) return launch_splitk_reduce_epilogue(ws, S, a, stream);
    else return launch_splitk_reduce(ws, S, a.M, a.N, a.y, a.y_dtype, a.ldy, stream);
  }
  if (a.N % Big::BN != 0 || a.N % Half::BN != 0)
    return launch_cfg<Narrow, false>(a, (int)((a.M + Narrow::BM - 1) / Narrow::BM), stream);
  const int64_t n_big = big_columns(a.M, a.N, a.K);
  if (n_big > 0) {
    Args b = a;
    b.N = n_big;
    const int tiles_m = (int)((b.M + Big::BM - 1) / Big::BM);
    // (the epilogue runs in the one-tile-per-workgroup kernel: 8192 x 24576 x 1536 with nothing to apply 302 us,
    // 326 with bias and silu, where the plain GEMM takes 274)
    bool launched = false;
    if constexpr (!Args::kEpilogue) {
      if (use_persistent(b, 16)) {
        // one workgroup per CU (a multiple of 8, as the XCD mapping of tiles assumes)
        const dim3 grid(cu_count() / 8 * 8);
        if (b.s_w_fmt == 0)
          hipLaunchKernelGGL((gemm_prefill_persistent_kernel<Big, 0, false>), grid, dim3(Big::THREADS), 0, stream, b,
                             tiles_m, (int)(b.N / Big::BN));
        else
          hipLaunchKernelGGL((gemm_prefill_persistent_kernel<Big, 1, false>), grid, dim3(Big::THREADS), 0, stream, b,
                             tiles_m, (int)(b.N / Big::BN));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        launched = true;
      }
    }
    if (!launched) {
      const hipError_t e = launch_cfg<Big, false>(b, tiles_m, stream);
      if (e != hipSuccess) return e;
    }
  }
  if (n_big == a.N) return hipSuccess;
  // the remaining output columns: their weight rows, block-scale rows and output columns
  Args h = a;
  h.N = a.N - n_big;
  h.w_q = a.w_q + n_big * a.K;
  h.s_w = (const uint8_t*)a.s_w + (n_big / 128) * (a.K / KBYTES) * (a.s_w_fmt == 0 ? 4 : 1);
  h.y = (uint8_t*)a.y + n_big * (a.y_dtype == 0 ? 2 : 4);
  if constexpr (Args::kEpilogue) {
    if (h.ep.bias != nullptr) h.ep.bias = (const uint8_t*)h.ep.bias + n_big * (h.ep.bias_dtype == 0 ? 2 : 4);
    if (h.ep.residual != nullptr)
      h.ep.residual = (const uint8_t*)h.ep.residual + n_big * (h.ep.residual_dtype == 0 ? 2 : 4);
  }
  return launch_cfg<Half, false>(h, (int)((h.M + Half::BM - 1) / Half::BM), stream);
}

}  // namespace

}  // namespace fgb
