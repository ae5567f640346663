// moe_ffn.hip — a whole mixture-of-experts layer for a few tokens (T <= 64) on FP8 block weights:
//
//   y[t] = residual[t] + sum_j w[t, j] * W2[e] . Q(act(W13[e][0:I] . Q(x[t])) * (W13[e][I:2I] . Q(x[t]))),
//
// e = ids[t, j], Q the 1x128-group E4M3 quantization.
//
// What bounds it: every routed expert's 3 H I weight bytes are read once, and a token's share of
// arithmetic on them is small, so the layer runs at the rate of the weight stream (HBM).  Three
// launches:
//   prep    sorts the (token, expert) pairs by expert into 16-row tiles and quantizes each pair's row
//           of x into its tile;
//   gate+up a workgroup owns 128 columns of the intermediate of one expert: 8 waves, each streaming
//           its 16 gate rows and 16 up rows over the whole H against the expert's tiles (one
//           activation fragment serves both), so that act(gate) * up and its group's maximum stay in
//           the workgroup and the codes of the quantized product are all that is written;
//   down    a workgroup owns 32 columns of y: its 8 waves split the routed experts' K-blocks, add
//           their weighted contributions per token in LDS in a fixed order, and the workgroup adds
//           the waves' sums and the residual.  No partial sums in memory, no atomics.
// Codes lie in the workspace in the matrix instruction's operand order: tile, K-block, 16-byte half,
// lane (16 g + r holds bytes 32 g .. 32 g + 31 of row r), so a fragment is two loads of whole lines
// however the rows were gathered.  Rows of a tile past its count are neither written nor read.
// Weights are loaded as whole lines and reordered through a per-wave LDS tile (as in the decode GEMM's
// register kernel), D K-blocks in flight per wave.
#include <type_traits>

#include "epilogue.hpp"
#include "gemm_common.hpp"
#include "internal.h"
#include "quant_common.hpp"

namespace fgb {

namespace {

constexpr int kTile = 16;           // rows per activation tile
constexpr int kFrag = kTile * 128;  // bytes of a tile's K-block

// 16-byte chunk c of 128-byte row r at c ^ ((r & 7) ^ (r>>3 & 1)): conflict-free 16-row fragment reads.
__device__ __forceinline__ int swz(int row, int chunk) {
  return row * 128 + ((chunk ^ ((row & 7) ^ ((row >> 3) & 1))) << 4);
}

// The layer's group quantization: s = fl32(amax * fl32(1 / 448)), within an ulp of the activation
// quantizer's fl32(amax / 448) and one multiplication; codes E4M3(fl32(v / s)) with IEEE quotients (the
// quantizers' shorter quotient is checked for their scale only); an all-zero group has s = 0, codes +-0.
constexpr float kInvMax = 1.0f / kE4M3Max;
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s) {
  const float v = s == 0.0f ? 1.0f : s;
  return cvt_pk_e4m3<true>(c / v, d / v, cvt_pk_e4m3<false>(a / v, b / v, 0u));
}

// Workspace: the routed experts in ascending order, each with its first tile and its row count; the
// tiles' rows (token and weight); the codes and scales of x and of the gated product.  Scales are
// [tile][K-block][16 rows].
struct Space {
  int* active;         // number of routed experts
  int4* experts;       // {expert, first tile, rows, 0}
  int* row_token;      // [tiles * 16]
  float* row_weight;   // [tiles * 16]
  uint8_t* xq;
  float* xs;
  uint8_t* hq;
  float* hs;
};

int max_experts(int T, int top_k, int E) { return T * top_k < E ? T * top_k : E; }
// sum over experts of ceil(rows / 16) <= (pairs + 15 experts) / 16
int max_tiles(int T, int top_k, int E) { return T * top_k / kTile + max_experts(T, top_k, E); }

size_t layout(int T, int top_k, int E, int H, int I, uint8_t* base, Space* s) {
  const size_t tiles = (size_t)max_tiles(T, top_k, E), rows = tiles * kTile;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return base + here;
  };
  Space t;
  t.active = (int*)take(sizeof(int));
  t.experts = (int4*)take(max_experts(T, top_k, E) * sizeof(int4));
  t.row_token = (int*)take(rows * sizeof(int));
  t.row_weight = (float*)take(rows * sizeof(float));
  t.xq = take(rows * H);
  t.xs = (float*)take(rows * (H / 128) * sizeof(float));
  t.hq = take(rows * I);
  t.hs = (float*)take(rows * (I / 128) * sizeof(float));
  if (s) *s = t;
  return at;
}

// ---------------------------------------------------------------------------------------------
// prep: one workgroup per (token, choice) pair.  Every workgroup counts the pairs per expert (at most
// 1024 of each) and finds its own pair's tile and row: the tiles of the experts before its own,
// then its rank among the expert's pairs in pair order.  A pair whose expert its token has named
// already is dropped and its weight goes to the first (so a token has one row per expert).
// Workgroup 0 also writes the table of routed experts.
// ---------------------------------------------------------------------------------------------
constexpr int PREP = 256;

__global__ __launch_bounds__(PREP) void moe_prep_kernel(MoeArgs p, Space s) {
  __shared__ int sid[kMoeMaxPairs];
  __shared__ int cnt[kMoeMaxExperts];
  __shared__ int part[3][PREP / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int pair = blockIdx.x, P = p.T * p.top_k;
  for (int e = tid; e < p.E; e += PREP) cnt[e] = 0;
  for (int q = tid; q < P; q += PREP) sid[q] = gload<int>(p.ids + q);
  __syncthreads();
  // drop foreign ids and repeats (a repeat looks at the ids as they came: dropping is decided from
  // registers before any is overwritten)
  int kept[kMoeMaxPairs / PREP];
#pragma unroll
  for (int i = 0; i < kMoeMaxPairs / PREP; ++i) {
    const int q = tid + i * PREP;
    kept[i] = -1;
    if (q < P) {
      const int id = sid[q];
      bool keep = id >= 0 && id < p.E;
      for (int f = q / p.top_k * p.top_k; f < q; ++f) keep = keep && sid[f] != id;
      kept[i] = keep ? id : -1;
    }
  }
  const int first = pair / p.top_k * p.top_k;
  const int raw = sid[pair];
  float weight = 0.0f;
  if (tid == 0) {
    for (int f = pair; f < first + p.top_k; ++f)
      if (sid[f] == raw) weight += gload<float>(p.weights + f);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMoeMaxPairs / PREP; ++i) {
    const int q = tid + i * PREP;
    if (q < P) {
      sid[q] = kept[i];
      if (kept[i] >= 0) atomicAdd(&cnt[kept[i]], 1);
    }
  }
  __syncthreads();
  const int id = sid[pair];
  // rank of this pair among its expert's, tiles and routed experts before its expert
  int rank = 0, tiles = 0;
  for (int q = tid; q < pair; q += PREP) rank += sid[q] == id;
  for (int e = tid; e < id; e += PREP) tiles += (cnt[e] + kTile - 1) / kTile;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    rank += __shfl_xor(rank, d);
    tiles += __shfl_xor(tiles, d);
  }
  if (lane == 0) {
    part[0][wave] = rank;
    part[1][wave] = tiles;
  }
  if (pair == 0) {
    // the table: thread i owns experts 4 i .. 4 i + 3; an exclusive scan of (routed, tiles) over the
    // threads places them
    int c[kMoeMaxExperts / PREP], na = 0, nt = 0;
#pragma unroll
    for (int i = 0; i < kMoeMaxExperts / PREP; ++i) {
      const int e = tid * (kMoeMaxExperts / PREP) + i;
      c[i] = e < p.E ? cnt[e] : 0;
      na += c[i] > 0;
      nt += (c[i] + kTile - 1) / kTile;
    }
    int both = na + (nt << 16), inc = both;  // (at most 1024 and 1088)
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    if (lane == 63) part[2][wave] = inc;
    __syncthreads();
    int before = inc - both;
    for (int w = 0; w < wave; ++w) before += part[2][w];
    int a = before & 0xFFFF, t = before >> 16;
#pragma unroll
    for (int i = 0; i < kMoeMaxExperts / PREP; ++i) {
      if (c[i] > 0) {
        s.experts[a] = make_int4(tid * (kMoeMaxExperts / PREP) + i, t, c[i], 0);
        ++a;
        t += (c[i] + kTile - 1) / kTile;
      }
    }
    if (tid == PREP - 1) *s.active = a;
  } else {
    __syncthreads();
  }
  if (id < 0) return;
  rank = tiles = 0;
#pragma unroll
  for (int w = 0; w < PREP / 64; ++w) {
    rank += part[0][w];
    tiles += part[1][w];
  }
  const int tile = tiles + rank / kTile, row = rank % kTile;
  if (tid == 0) {
    s.row_token[tile * kTile + row] = pair / p.top_k;
    s.row_weight[tile * kTile + row] = weight;
  }
  // the row's codes: 16 lanes per 128-group, 8 values per lane, as the activation quantizer does
  const int KB = p.H / 128;
  const uint16_t* x = p.x + (int64_t)(pair / p.top_k) * p.ldx;
  uint8_t* xq = s.xq + (int64_t)tile * KB * kFrag;
  // (whole waves for the row maxima: lanes past the row repeat its first group and store nothing)
  for (int c0 = wave * 64; c0 < p.H / 8; c0 += PREP) {
    const bool in = c0 + lane < p.H / 8;
    const int c = in ? c0 + lane : lane % 16;
    const int4 v = gload_i4(x + 8 * c);
    const uint4 u = make_uint4(v.x, v.y, v.z, v.w);
    const float sc = row16_max(absmax8(u)) * kInvMax;
    const float v8[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                         bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
    if (!in) continue;
    const int kb = c / 16, k = c % 16 * 8;
    v2u w;
    w[0] = codes4(v8[0], v8[1], v8[2], v8[3], sc);
    w[1] = codes4(v8[4], v8[5], v8[6], v8[7], sc);
    gstore<v2u>(xq + kb * kFrag + (k % 32) / 16 * 1024 + (k / 32 * 16 + row) * 16 + k % 16, w);
    if (c % 16 == 0) gstore<float>(s.xs + ((int64_t)tile * KB + kb) * kTile + row, sc);
  }
}

// Product sums of one K-block.  The FP8 matrix instruction adds its 128 products at a fixed-point
// alignment: measured 1.3e-5 of the 2-norm on normal data, up to 9e-5 on rows with outliers, against
// 64-bit sums.  That vanishes in a bf16 result, but not ahead of a second quantization: codes near a
// rounding boundary flip by a whole E4M3 step, and with gate and up sums of that accuracy the layer's
// output was 2.3e-3 to 3.2e-3 of its 2-norm off (64 bits), twice its bf16 rounding of 1.7e-3, to which
// exact sums bring it back.  So there the codes are widened to bf16 (exact) and take the bf16
// instruction, whose sums of the same data measured 1e-8: twice the matrix time and two conversions
// per four codes, behind the weight stream (7168 x 2048, 32 experts, top 8: 1 token 78.1 -> 79.9 us,
// 64 tokens 269 -> 274 us).  The down products, rounded to bf16 next, take the FP8 instruction.
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
struct Wide {
  v8bf k[4];  // bytes 8 i .. 8 i + 7 of the lane's 32
};
__device__ __forceinline__ Wide widen(const int4& lo, const int4& hi) {
  const int b[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  Wide w;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b[i], 1.0f, false);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b[i], 1.0f, true);
    w.k[i / 2][i % 2 * 4 + 0] = a[0];
    w.k[i / 2][i % 2 * 4 + 1] = a[1];
    w.k[i / 2][i % 2 * 4 + 2] = c[0];
    w.k[i / 2][i % 2 * 4 + 3] = c[1];
  }
  return w;
}
__device__ __forceinline__ v4f block_sum(const Wide& a, const Wide& b) {
  v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.k[i], b.k[i], s, 0, 0, 0);
  return s;
}

struct Codes {
  v8i v;
};
__device__ __forceinline__ Codes narrow(const int4& lo, const int4& hi) {
  Codes c;
  c.v[0] = lo.x; c.v[1] = lo.y; c.v[2] = lo.z; c.v[3] = lo.w;
  c.v[4] = hi.x; c.v[5] = hi.y; c.v[6] = hi.z; c.v[7] = hi.w;
  return c;
}
__device__ __forceinline__ v4f block_sum(const Codes& a, const Codes& b) { return mfma_e4m3_16x16x128(a.v, b.v); }

template <bool WIDE>
__device__ __forceinline__ auto operand(const int4& lo, const int4& hi) {
  if constexpr (WIDE) return widen(lo, hi);
  else return narrow(lo, hi);
}

// ---------------------------------------------------------------------------------------------
// One wave's stream: NT weight tiles (16 rows each) against MT activation tiles over nk K-blocks,
// D blocks in flight in registers.
//   acc[n][m] += P * (s_a * s_w[n])   per K-block, P the block's product sums (WIDE: from bf16).
// w[n]: lane address of weight tile n at the first block (row l/8, 16-byte chunk l%8), rows 8 further
// at + 8 * pitch; a[m]: lane address of tile m's fragment; sa[m]: lane address of its row's scale;
// `scale(n, kk)` gives the weight block's scale.  Lanes whose row does not exist are given the
// addresses of one that does (the same lines: no traffic, no branch), and their results are dropped.
// Blocks past the end are clamped to the last one, so the loads in flight are the same number in
// every step.
// ---------------------------------------------------------------------------------------------
template <int NT, int MT, int D, bool WIDE, typename Scale>
__device__ __forceinline__ void stream_blocks(const uint8_t* const (&w)[NT], int64_t pitch, const uint8_t* const (&a)[MT],
                                              const float* const (&sa)[MT], int nk, uint8_t* lds,
                                              Scale scale, v4f (&acc)[NT][MT]) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wo0 = swz(lane >> 3, lane & 7), wo1 = swz((lane >> 3) + 8, lane & 7);
  const int ro0 = swz(r, 2 * g), ro1 = swz(r, 2 * g + 1);
  int4 wv[D][NT][2], av[D][MT][2];
  float sv[D][MT];
  auto load = [&](int kk, int d) {
    const int64_t wk = (int64_t)kk * 128, ak = (int64_t)kk * kFrag;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      wv[d][n][0] = gload_i4_last(w[n] + wk);
      wv[d][n][1] = gload_i4_last(w[n] + 8 * pitch + wk);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      av[d][m][0] = gload_i4(a[m] + ak);
      av[d][m][1] = gload_i4(a[m] + ak + 1024);
      sv[d][m] = gload<float>(sa[m] + kk * kTile);
    }
  };
  auto compute = [&](int kk, int d) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // (a wave's LDS operations complete in order: the reads see the writes, and the next block's
      // writes follow these reads)
      uint8_t* t = lds + n * kFrag;
      *reinterpret_cast<int4*>(t + wo0) = wv[d][n][0];
      *reinterpret_cast<int4*>(t + wo1) = wv[d][n][1];
    }
    decltype(operand<WIDE>(av[d][0][0], av[d][0][1])) af[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) af[m] = operand<WIDE>(av[d][m][0], av[d][m][1]);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint8_t* t = lds + n * kFrag;
      const int4 lo = *reinterpret_cast<const int4*>(t + ro0);
      const int4 hi = *reinterpret_cast<const int4*>(t + ro1);
      const auto wf = operand<WIDE>(lo, hi);
      const float sw = scale(n, kk);
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[n][m] += block_sum(wf, af[m]) * (sv[d][m] * sw);
    }
  };
#pragma unroll
  for (int d = 0; d < D - 1; ++d) load(min(d, nk - 1), d);
  int kk = 0;
  for (; kk + D <= nk; kk += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      load(min(kk + d + D - 1, nk - 1), (d + D - 1) % D);
      compute(kk + d, d);
    }
  }
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (kk + d < nk) compute(kk + d, d);
}

// ---------------------------------------------------------------------------------------------
// gate+up: grid (I / 128, routed experts at most), 8 waves.
// ---------------------------------------------------------------------------------------------
template <int SWF>
__global__ __launch_bounds__(512) void moe_gate_up_kernel(MoeArgs p, Space s) {
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[8][2 * kFrag];
  __shared__ float sws[2][256];      // the two weight block rows' scales (H <= 32768)
  __shared__ float amax[8][4 * kTile];
  if ((int)blockIdx.y >= gload<int>(s.active)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const v4i ex = gload<v4i>(s.experts + blockIdx.y);
  const int e = __builtin_amdgcn_readfirstlane(ex[0]), tile0 = __builtin_amdgcn_readfirstlane(ex[1]);
  const int rows = __builtin_amdgcn_readfirstlane(ex[2]);
  const int KB = p.H / 128, NB = p.I / 128, gb = blockIdx.x;
  const int64_t sw0 = ((int64_t)e * 2 * NB + gb) * KB;
  for (int k = tid; k < KB; k += 512) {
    sws[0][k] = load_sw<SWF>(p.s_w13, sw0 + k);
    sws[1][k] = load_sw<SWF>(p.s_w13, sw0 + (int64_t)NB * KB + k);
  }
  __syncthreads();
  const uint8_t* w0 = p.w13_q + ((int64_t)e * 2 * p.I + gb * 128 + wave * 16 + (lane >> 3)) * p.H + 16 * (lane & 7);
  const uint8_t* const w[2] = {w0, w0 + (int64_t)p.I * p.H};

  auto run = [&](auto mt_c) {
    constexpr int MT = decltype(mt_c)::value;
    constexpr int D = MT >= 4 ? 2 : 3;
    const uint8_t* a[MT];
    const float* sa[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int q = min(m * kTile + r, rows - 1);  // (MT = 4 may run three tiles)
      a[m] = s.xq + (int64_t)(tile0 + q / kTile) * KB * kFrag + (g * kTile + q % kTile) * 16;
      sa[m] = s.xs + (int64_t)(tile0 + q / kTile) * KB * kTile + q % kTile;
    }
    v4f acc[2][MT];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    stream_blocks<2, MT, D, true>(w, p.H, a, sa, KB, &tiles[wave][0],
                            [&](int n, int kk) { return sws[n][kk]; }, acc);
    // the gated product of this wave's 16 columns (lane: row r, columns 4 g .. 4 g + 3) and the rows'
    // maxima over the workgroup's 128 columns
    v4f h[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float v[4] = {acc[0][m][0], acc[0][m][1], acc[0][m][2], acc[0][m][3]};
      activate<4>(p.act, v);
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[m][i] = v[i] * acc[1][m][i];
        mx = fmaxf(mx, fabsf(h[m][i]));
      }
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      if (g == 0) amax[wave][m * kTile + r] = mx;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m * kTile + r < rows) {
        float mx = amax[0][m * kTile + r];
#pragma unroll
        for (int q = 1; q < 8; ++q) mx = fmaxf(mx, amax[q][m * kTile + r]);
        const float sc = mx * kInvMax;
        const uint32_t c = codes4(h[m][0], h[m][1], h[m][2], h[m][3], sc);
        uint8_t* hq = s.hq + ((int64_t)(tile0 + m) * NB + gb) * kFrag;
        gstore<uint32_t>(hq + (wave & 1) * 1024 + ((wave >> 1) * 16 + r) * 16 + 4 * g, c);
        if (wave == 0 && g == 0) gstore<float>(s.hs + ((int64_t)(tile0 + m) * NB + gb) * kTile + r, sc);
      }
    }
  };
  // (an expert has at most T <= 64 rows: four tiles)
  if (rows <= 16) run(std::integral_constant<int, 1>{});
  else if (rows <= 32) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 4>{});
}

// ---------------------------------------------------------------------------------------------
// down: grid H / 32, 8 waves.  The K-blocks of all routed experts, in expert order, are one list that
// the waves split evenly; a wave walks its share expert by expert (segments).
// ---------------------------------------------------------------------------------------------
template <int SWF, int OUT>
__global__ __launch_bounds__(512) void moe_down_kernel(MoeArgs p, Space s) {
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[8][2 * kFrag];
  extern __shared__ __attribute__((aligned(16))) float ysum[];  // [8 waves][T][32]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 32;
  const int KB = p.I / 128, NB = p.H / 128;
  float* const mine = ysum + wave * p.T * 32;
  for (int i = lane; i < p.T * 8; i += 64) *reinterpret_cast<v4f*>(mine + 4 * i) = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  const int units = gload<int>(s.active) * KB;
  const int per = (units + 7) / 8;
  int u = __builtin_amdgcn_readfirstlane(min(units, wave * per));
  const int u1 = __builtin_amdgcn_readfirstlane(min(units, (wave + 1) * per));
  while (u < u1) {
    const int si = u / KB, kb0 = u - si * KB;
    const int nk = min(min(KB - kb0, u1 - u), 64);
    const v4i ex = gload<v4i>(s.experts + si);
    const int e = __builtin_amdgcn_readfirstlane(ex[0]), tile0 = __builtin_amdgcn_readfirstlane(ex[1]);
    const int rows = __builtin_amdgcn_readfirstlane(ex[2]);
    const float swl = lane < nk ? load_sw<SWF>(p.s_w2, ((int64_t)e * NB + n0 / 128) * KB + kb0 + lane) : 0.0f;
    const uint8_t* w0 = p.w2_q + ((int64_t)e * p.H + n0 + (lane >> 3)) * p.I + (int64_t)kb0 * 128 + 16 * (lane & 7);
    const uint8_t* const w[2] = {w0, w0 + (int64_t)16 * p.I};
    auto run = [&](auto mt_c) {
      constexpr int MT = decltype(mt_c)::value;
      constexpr int D = MT >= 4 ? 2 : 3;
      const uint8_t* a[MT];
      const float* sa[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int q = min(m * kTile + r, rows - 1);
        a[m] = s.hq + ((int64_t)(tile0 + q / kTile) * KB + kb0) * kFrag + (g * kTile + q % kTile) * 16;
        sa[m] = s.hs + ((int64_t)(tile0 + q / kTile) * KB + kb0) * kTile + q % kTile;
      }
      v4f acc[2][MT];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      stream_blocks<2, MT, D, false>(w, p.I, a, sa, nk, &tiles[wave][0],
                              [&](int, int kk) {
                                return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(swl), kk));
                              }, acc);
      // (a token has one row per expert, so no two lanes add to the same sums)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m * kTile + r < rows) {
          const int row = (tile0 + m) * kTile + r;
          const int t = gload<int>(s.row_token + row);
          const float wt = gload<float>(s.row_weight + row);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            v4f* const q = reinterpret_cast<v4f*>(mine + t * 32 + n * 16 + 4 * g);
            *q += acc[n][m] * wt;
          }
        }
      }
    };
    if (rows <= 16) run(std::integral_constant<int, 1>{});
    else if (rows <= 32) run(std::integral_constant<int, 2>{});
    else run(std::integral_constant<int, 4>{});
    u += nk;
  }
  __syncthreads();
  // the waves' sums in wave order, the residual, one rounding
  for (int i = tid; i < p.T * 8; i += 512) {
    const int t = i >> 3, c = (i & 7) * 4;
    v4f sum = *reinterpret_cast<const v4f*>(ysum + t * 32 + c);
#pragma unroll
    for (int q = 1; q < 8; ++q) sum += *reinterpret_cast<const v4f*>(ysum + (q * p.T + t) * 32 + c);
    if (p.residual != nullptr) {
      float f[4];
      load_values<4>(p.residual, p.residual_dtype, (int64_t)t * p.ldr + n0 + c, f);
      sum += v4f{f[0], f[1], f[2], f[3]};
    }
    store4<OUT>(p.y, p.ldy, t, n0 + c, sum);
  }
}

}  // namespace

size_t moe_ffn_workspace_bytes(int T, int top_k, int E, int H, int I) {
  return layout(T, top_k, E, H, I, nullptr, nullptr);
}

hipError_t launch_moe_ffn(const MoeArgs& a, void* workspace, hipStream_t stream) {
  Space s;
  layout(a.T, a.top_k, a.E, a.H, a.I, reinterpret_cast<uint8_t*>(workspace), &s);
  hipLaunchKernelGGL(moe_prep_kernel, dim3((unsigned)(a.T * a.top_k)), dim3(PREP), 0, stream, a, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 up((unsigned)(a.I / 128), (unsigned)max_experts(a.T, a.top_k, a.E)), down((unsigned)(a.H / 32));
  if (a.s_w_fmt == 0) hipLaunchKernelGGL(moe_gate_up_kernel<0>, up, dim3(512), 0, stream, a, s);
  else hipLaunchKernelGGL(moe_gate_up_kernel<1>, up, dim3(512), 0, stream, a, s);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t lds = (size_t)8 * a.T * 32 * sizeof(float);
#define FGB_DOWN(SWF, OUT) hipLaunchKernelGGL((moe_down_kernel<SWF, OUT>), down, dim3(512), lds, stream, a, s)
  if (a.s_w_fmt == 0) {
    if (a.y_dtype == 0) FGB_DOWN(0, 0); else FGB_DOWN(0, 1);
  } else {
    if (a.y_dtype == 0) FGB_DOWN(1, 0); else FGB_DOWN(1, 1);
  }
#undef FGB_DOWN
  return hipGetLastError();
}

}  // namespace fgb
