// moe_route.hip — the router of a mixture of experts: for every token the top_k experts of its row of
// logits and their weights.
//
//   score    softmax: p_e = exp(l_e - max l) / sum_j exp(l_j - max l);  sigmoid: p_e = 1 / (1 + exp(-l_e))
//   select   the k largest of key_e = l_e (both scores grow with l), or of p_e + bias_e with a selection
//            bias; equal keys go to the lowest index.  A masked expert (l = -inf or NaN) is never
//            selected: a row with fewer than k open experts fills up with id -1 and weight 0.
//   weight   p_e, or p_e / (sum of the selected p) renormalized, times a scale.
//
// One wave per token, the row in registers (expert lane + 64 v in register v), so a row is read once
// and nothing but the result is written: T * (E * 2 or 4 + 8 k) bytes.  Each selection is one wave-wide
// integer maximum of order-preserving keys (four DPP steps and four lane reads) and a ballot.  The
// renormalized weights are formed relative to the largest selected term, so they neither overflow
// nor divide 0 by 0 however small the scores are.
#include <type_traits>

#include "gemm_common.hpp"
#include "internal.h"

namespace fgb {

namespace {

constexpr int RT_WAVES = 4;  // tokens per workgroup

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  auto dpp = [](uint32_t x, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, decltype(ctrl)::value, 0xF, 0xF, false);
  };
  // quad_perm [1,0,3,2], quad_perm [2,3,0,1], row_half_mirror, row_mirror: the maximum of 16 lanes
  v = max(v, dpp(v, std::integral_constant<int, 0xB1>{}));
  v = max(v, dpp(v, std::integral_constant<int, 0x4E>{}));
  v = max(v, dpp(v, std::integral_constant<int, 0x141>{}));
  v = max(v, dpp(v, std::integral_constant<int, 0x140>{}));
  const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0), b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
  const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32), d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
  return max(max(a, b), max(c, d));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// Order-preserving integer of a float (-inf and NaN are mapped to 0 by the caller).
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float sigmoid_exact(float l) {
  const float e = expf(-fabsf(l));
  return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}

template <int V, int DT>
__global__ __launch_bounds__(64 * RT_WAVES) void moe_route_kernel(RouteArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * RT_WAVES + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const float inf = __builtin_inff(), big = 3.4028234663852886e38f;
  float l[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    float x = -inf;
    if (e < p.E) {
      if constexpr (DT == 0) x = bf16_lo(gload<uint16_t>((const uint16_t*)p.logits + t * p.ld + e));
      else x = gload<float>((const float*)p.logits + t * p.ld + e);
    }
    // NaN is masked; +inf counts as the largest finite value; -0 and +0 are one value
    l[v] = x > -inf ? fminf(x, big) + 0.0f : -inf;
  }
  // softmax: the row's maximum and sum (of the open experts)
  float row_max = 0.0f, row_sum = 1.0f;
  if (p.scoring == 0 && (p.bias != nullptr || !p.renorm)) {
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) m = max(m, l[v] > -inf ? order_key(l[v]) : 0u);
    m = wave_max_u32(m);
    row_max = m ? order_value(m) : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) s += l[v] > -inf ? expf(l[v] - row_max) : 0.0f;
    row_sum = wave_sum(s);
  }
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float f = l[v];
    if (p.bias != nullptr) {
      const int e = lane + 64 * v;
      const float b = e < p.E ? gload<float>(p.bias + e) : 0.0f;
      f = (p.scoring == 0 ? expf(f - row_max) / row_sum : sigmoid_exact(f)) + b + 0.0f;
    }
    key[v] = l[v] > -inf ? order_key(f) : 0u;
  }
  // lane j keeps the j-th selection
  int my_id = -1;
  float my_l = -inf;
  for (int j = 0; j < p.top_k; ++j) {
    uint32_t best = key[0];
    int bv = 0;
    float bl = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) {
      if (key[v] > best) { best = key[v]; bv = v; bl = l[v]; }  // ties: the lower register, hence index
    }
    const uint32_t m = wave_max_u32(best);
    if (m == 0) break;  // no open expert is left
    // the lowest index among the lanes that hold the maximum
    unsigned long long hit = __ballot(best == m);
    int win = __ffsll((long long)hit) - 1;
    if (hit & (hit - 1)) {
      int low = __builtin_amdgcn_readlane(bv, win);
      for (unsigned long long h = hit & (hit - 1); h; h &= h - 1) {
        const int q = __ffsll((long long)h) - 1;
        const int w = __builtin_amdgcn_readlane(bv, q);
        if (w < low) { low = w; win = q; }
      }
    }
    const int wv = __builtin_amdgcn_readlane(bv, win);
    const float wl = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bl), win));
    if (lane == j) { my_id = win + 64 * wv; my_l = wl; }
    if (lane == win) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v == bv) key[v] = 0;
    }
  }
  // weights of the selected (lanes without one: 0)
  const bool have = my_id >= 0;
  float w = 0.0f;
  if (p.renorm) {
    const uint32_t m = wave_max_u32(have ? order_key(my_l) : 0u);
    if (m != 0) {
      const float top = order_value(m);
      if (p.scoring == 0) {
        w = have ? expf(my_l - top) : 0.0f;
      } else if (top >= 0.0f) {
        w = have ? sigmoid_exact(my_l) : 0.0f;
      } else {  // every score times exp(-top): exp(l - top) / (1 + exp(l))
        w = have ? expf(my_l - top) / (1.0f + expf(my_l)) : 0.0f;
      }
      w = w / wave_sum(w);
    }
  } else if (have) {
    w = p.scoring == 0 ? expf(my_l - row_max) / row_sum : sigmoid_exact(my_l);
  }
  if (lane < p.top_k) {
    gstore<int>(p.ids + t * p.top_k + lane, my_id);
    gstore<float>(p.weights + t * p.top_k + lane, have ? w * p.scale : 0.0f);
  }
}

template <int V>
void launch_v(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + RT_WAVES - 1) / RT_WAVES)), block(64 * RT_WAVES);
  if (a.dtype == 0) hipLaunchKernelGGL((moe_route_kernel<V, 0>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((moe_route_kernel<V, 1>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
  // registers per lane: the next power of two of ceil(E / 64)
  if (a.E <= 64) launch_v<1>(a, stream);
  else if (a.E <= 128) launch_v<2>(a, stream);
  else if (a.E <= 256) launch_v<4>(a, stream);
  else if (a.E <= 512) launch_v<8>(a, stream);
  else launch_v<16>(a, stream);
  return hipGetLastError();
}

}  // namespace fgb
