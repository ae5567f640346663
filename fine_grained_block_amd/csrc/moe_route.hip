// moe_route.hip — the router of a mixture of experts: for every token the top_k experts of its row of
// logits and their weights.
//
//   score    softmax: p_e = exp(l_e - max l) / sum_j exp(l_j - max l);  sigmoid: p_e = 1 / (1 + exp(-l_e))
//   select   the k largest of key_e = l_e (both scores grow with l), or of p_e + bias_e with a selection
//            bias; equal keys go to the lowest index.  A masked expert (l = -inf or NaN, or a NaN
//            bias) is never selected: a row with fewer than k open experts fills up with id -1 and weight 0.
//   weight   p_e, or p_e / (sum of the selected p) renormalized, times a scale.
//
// One wave per token, or 16 lanes with many tokens, the row in registers (expert lane + 64 v in register
// v), so a row is read once and nothing but the result is written: T * (E * 2 or 4 + 8 k) bytes.  Each
// selection is one integer maximum of order-preserving keys over the token's lanes (four DPP steps, and four
// lane reads for a wave) and a search for its lowest index: a few tokens are bound by that chain's
// latency, many by its instructions.  The
// renormalized weights are formed relative to the largest selected term, so they neither overflow
// nor divide 0 by 0 however small the scores are.
#include <type_traits>

#include "gemm_common.hpp"
#include "internal.h"

namespace fgb {

namespace {

constexpr int RT_WAVES = 4;  // tokens per workgroup

// f of v over each row of 16 lanes, for every lane of the row.
template <typename T, typename F>
__device__ __forceinline__ T row_reduce(T v, F f) {
  auto dpp = [](T x, auto ctrl) {
    return __builtin_bit_cast(
        T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  // quad_perm [1,0,3,2], quad_perm [2,3,0,1], row_half_mirror, row_mirror
  v = f(v, dpp(v, std::integral_constant<int, 0xB1>{}));
  v = f(v, dpp(v, std::integral_constant<int, 0x4E>{}));
  v = f(v, dpp(v, std::integral_constant<int, 0x141>{}));
  return f(v, dpp(v, std::integral_constant<int, 0x140>{}));
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = row_reduce(v, umax);
  auto row = [&](int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); };
  return max(max(row(0), row(16)), max(row(32), row(48)));
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

// Logit e of token t, for e >= E masked: NaN is masked (-inf); +inf counts as the largest finite value;
// -0 and +0 are one value.  (Loads without branches, so that a row's are in flight together.)
template <int DT>
__device__ __forceinline__ float logit(const RouteArgs& p, int64_t t, int e) {
  const float inf = __builtin_inff(), big = 3.4028234663852886e38f;
  const int64_t at = t * p.ld + min(e, p.E - 1);
  float x;
  if constexpr (DT == 0) x = bf16_lo(gload<uint16_t>((const uint16_t*)p.logits + at));
  else x = gload<float>((const float*)p.logits + at);
  return e < p.E && x > -inf ? fminf(x, big) + 0.0f : -inf;
}

// Weight of a lane's selection (0 without one).  mx and sum reduce over a token's lanes, all of which come here.
template <typename Max, typename Sum>
__device__ __forceinline__ float selected_weight(const RouteArgs& p, bool have, float l, float row_max, float row_sum,
                                                 Max mx, Sum sum) {
  if (!p.renorm) return !have ? 0.0f : (p.scoring == 0 ? expf(l - row_max) / row_sum : sigmoid_exact(l));
  const uint32_t m = mx(have ? order_key(l) : 0u);
  const float top = order_value(m);
  float w = 0.0f;
  if (have) {
    if (p.scoring == 0) w = expf(l - top);
    else if (top >= 0.0f) w = sigmoid_exact(l);
    else w = expf(l - top) / (1.0f + expf(l));  // every score times exp(-top)
  }
  const float s = sum(w);
  return m != 0 ? w / s : 0.0f;
}

template <int V, int DT>
__global__ __launch_bounds__(64 * RT_WAVES) void moe_route_kernel(RouteArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * RT_WAVES + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const float inf = __builtin_inff();
  float l[V];
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = logit<DT>(p, t, lane + 64 * v);
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
      const float b = gload<float>(p.bias + min(lane + 64 * v, p.E - 1));
      f = (p.scoring == 0 ? expf(f - row_max) / row_sum : sigmoid_exact(f)) + b + 0.0f;
    }
    key[v] = l[v] > -inf && f == f ? order_key(f) : 0u;  // (a NaN bias; its pattern would order above +inf)
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
  const bool have = my_id >= 0;
  const float w = selected_weight(p, have, my_l, row_max, row_sum, wave_max_u32, wave_sum);
  if (lane < p.top_k) {
    gstore<int>(p.ids + t * p.top_k + lane, my_id);
    gstore<float>(p.weights + t * p.top_k + lane, have ? w * p.scale : 0.0f);
  }
}

// The same for many tokens: four tokens per wave, 16 lanes each (expert sub + 16 v in register v of the
// row's lane sub), so that a selection's instructions serve four tokens.  The sums are added in the wave
// kernel's order: a token's result is the same, bit for bit, whichever kernel computes it.
template <int V, int DT>
__global__ __launch_bounds__(256) void moe_route_rows_kernel(RouteArgs p) {
  const int sub = threadIdx.x & 15;
  const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t t = row < p.T ? row : p.T - 1;  // (all lanes stay for the row reductions)
  const float inf = __builtin_inff();
  auto fadd = [](float a, float b) { return a + b; };
  float l[V];
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = logit<DT>(p, t, sub + 16 * v);
  float row_max = 0.0f, row_sum = 1.0f;
  if (p.scoring == 0 && (p.bias != nullptr || !p.renorm)) {
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) m = max(m, l[v] > -inf ? order_key(l[v]) : 0u);
    m = row_reduce(m, umax);
    row_max = m ? order_value(m) : 0.0f;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) s[v & 3] += l[v] > -inf ? expf(l[v] - row_max) : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = row_reduce(s[i], fadd);
    row_sum = (s[0] + s[1]) + (s[2] + s[3]);
  }
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float f = l[v];
    if (p.bias != nullptr) {
      const float b = gload<float>(p.bias + min(sub + 16 * v, p.E - 1));
      f = (p.scoring == 0 ? expf(f - row_max) / row_sum : sigmoid_exact(f)) + b + 0.0f;
    }
    key[v] = l[v] > -inf && f == f ? order_key(f) : 0u;  // (a NaN bias; its pattern would order above +inf)
  }
  // lane j of the row keeps the j-th selection
  int my_id = -1;
  float my_l = -inf;
  for (int j = 0; j < p.top_k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    const uint32_t m = row_reduce(best, umax);
    if (__ballot(m != 0) == 0) break;
    // this lane's lowest register that holds it, then the row's lowest index
    uint32_t at = V;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) at = key[v] == m ? v : at;
    const uint32_t mine = at < V ? 16 * at + sub : 0xFFFFu;
    const uint32_t win = row_reduce(mine, [](uint32_t a, uint32_t b) { return min(a, b); });
    if (sub == j && m != 0) { my_id = (int)win; my_l = order_value(m); }
    const uint32_t gone = mine == win ? at : V;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = gone == v ? 0u : key[v];
  }
  const bool have = my_id >= 0;
  if (p.bias != nullptr && have) my_l = logit<DT>(p, t, my_id);  // (the keys held the biased score)
  const float w = selected_weight(p, have, my_l, row_max, row_sum, [](uint32_t v) { return row_reduce(v, umax); },
                                  [&](float v) { return row_reduce(v, fadd); });
  if (row < p.T && sub < p.top_k) {
    gstore<int>(p.ids + t * p.top_k + sub, my_id);
    gstore<float>(p.weights + t * p.top_k + sub, have ? w * p.scale : 0.0f);
  }
}

// From these many tokens on the waves of one token each are bound by instruction issue and four tokens per
// wave win; below, each selection's chain of 16 registers a lane is the longer one.  Measured at 8
// of 256 experts (one token a wave, four): 1 token 3.7 and 4.8 us, 4096 5.8 and 5.2, 8191 8.6 and 6.4, 16384
// 14.2 and 9.5; with a selection bias 4096 6.6 and 7.3, 8191 10.1 and 8.6; 6 of 64 experts 4096 4.0 and 3.3,
// 16384 8.8 and 4.6.
constexpr int kManyTokens = 4096, kManyTokensBias = 6144;

template <int V>
void launch_rows(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + 15) / 16)), block(256);
  if (a.dtype == 0) hipLaunchKernelGGL((moe_route_rows_kernel<V, 0>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((moe_route_rows_kernel<V, 1>), grid, block, 0, stream, a);
}

template <int V>
void launch_v(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + RT_WAVES - 1) / RT_WAVES)), block(64 * RT_WAVES);
  if (a.dtype == 0) hipLaunchKernelGGL((moe_route_kernel<V, 0>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((moe_route_kernel<V, 1>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
  if (a.T >= (a.bias == nullptr ? kManyTokens : kManyTokensBias) && a.E <= 256 && a.top_k <= 16) {
    if (a.E <= 64) launch_rows<4>(a, stream);
    else if (a.E <= 128) launch_rows<8>(a, stream);
    else launch_rows<16>(a, stream);
    return hipGetLastError();
  }
  // registers per lane: the next power of two of ceil(E / 64)
  if (a.E <= 64) launch_v<1>(a, stream);
  else if (a.E <= 128) launch_v<2>(a, stream);
  else if (a.E <= 256) launch_v<4>(a, stream);
  else if (a.E <= 512) launch_v<8>(a, stream);
  else launch_v<16>(a, stream);
  return hipGetLastError();
}

}  // namespace fgb
