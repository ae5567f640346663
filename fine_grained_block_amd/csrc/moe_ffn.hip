// moe_ffn.hip — a whole mixture-of-experts layer for a few tokens (T <= 64) on FP8 block weights:
//
//   y[t] = residual[t] + sum_j w[t, j] * W2[e] . Q(act(W13[e][0:I] . Q(x[t])) * (W13[e][I:2I] . Q(x[t]))),
//
// e = ids[t, j], Q the 1x128-group E4M3 quantization.
//
// What bounds it: every routed expert's 3 H I weight bytes are read once, and a token's share of
// arithmetic on them is small, so the layer runs at the rate of the weight stream (HBM).  Three
// launches, two for the fewest tokens, and one more each where gate+up or down is sliced:
//   prep    quantizes the rows of x and, in one more workgroup, sorts the (token, expert) pairs by
//           expert into tiles of 16 rows;
//   gate+up a workgroup owns 128 columns of the intermediate of one expert: 8 waves, each streaming
//           its 16 gate rows and 16 up rows over the whole H against the expert's tiles (one
//           activation fragment serves both), so that act(gate) * up and its group's maximum stay in
//           the workgroup and the codes of the quantized product are all that is written.  With the
//           fewest tokens each workgroup finds its expert and quantizes its rows itself, and there is
//           no prep launch;
//   down    a workgroup owns 16 or 32 columns of y: its waves split the routed experts' K-blocks, add
//           their weighted contributions per token in LDS in a fixed order, and the workgroup adds
//           the waves' sums and the residual.
// Where few experts or few columns would leave CUs idle, gate+up is sliced along K and down over the
// experts' K-blocks; their float32 partial sums are then added in slice order by a launch of their own.
// The only atomics are the integer counters of the sort, whose order moves rows within a tile and
// changes no value.
// The gated product's codes lie in the workspace in the matrix instruction's operand order: tile,
// K-block, 16-byte half, lane (16 g + r holds bytes 32 g .. 32 g + 31 of row r), so a fragment is two
// loads of whole lines.  Rows of a tile past its count are not written by gate+up and not read by down; the
// launch that adds sliced gate+up takes them along, from whatever the workspace holds into their own places.
// Weights are loaded as whole lines and reordered through a per-wave LDS tile (as in the decode GEMM's
// register kernel), several K-blocks in flight per wave.
#include <type_traits>

#include "epilogue.hpp"
#include "gemm_common.hpp"
#include "internal.h"
#include "moe_plan.hpp"
#include "quant_common.hpp"

namespace fgb {

namespace {

constexpr int kFrag = kTile * 128;  // bytes of a tile's K-block

// 16-byte chunk c of 128-byte row r at c ^ ((r & 7) ^ (r>>3 & 1)): conflict-free 16-row fragment reads.
__device__ __forceinline__ int swz(int row, int chunk) {
  return row * 128 + ((chunk ^ ((row & 7) ^ ((row >> 3) & 1))) << 4);
}

// The layer's group quantization: s = fl32(amax * fl32(1 / 448)); codes E4M3(fl32(v / s)) with IEEE quotients
// (the quantizers' shorter quotient is checked for their scale only); an all-zero group has s = 0, codes +-0.
// The product is what torch computes on the GPU for amax / 448.0 (a Python number as divisor), so the codes
// are those of the layer written in torch operations.  The activation quantizer divides: its scale is an ulp
// off in 55% of the groups, which moves bf16 values that lie on a tie between two codes, 1 in 1000, by a whole
// code.  The layer's result with the quotient was 0.3 to 2.3% of its 2-norm (64 bits, 1 to 64 tokens) off the
// one with the product, where the quantization itself is 3% off.
constexpr float kInvMax = 1.0f / kE4M3Max;
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s) {
  const float v = s == 0.0f ? 1.0f : s;
  return cvt_pk_e4m3<true>(c / v, d / v, cvt_pk_e4m3<false>(a / v, b / v, 0u));
}

// Group maxima are taken over magnitudes as bit patterns: finite values order like them and NaN lies above
// all, so a NaN makes its group's scale NaN and reaches the output (a float maximum would drop it, and the
// conversion to codes would make it finite).
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ float group_scale(uint32_t m) { return __uint_as_float(m) * kInvMax; }
// Maximum over 8 or 16 consecutive lanes, for all of them (quad_perm [1,0,3,2], quad_perm [2,3,0,1],
// row_half_mirror, row_mirror).
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  static_assert(L == 8 || L == 16, "half a DPP row or a whole one");
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
  if constexpr (L == 16) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));
  return v;
}

// Workspace: the routed experts, each with its first tile and its row count; the tiles' rows (token
// and weight); codes [T, H] and scales [T, H/128] of x; the gated product's codes and scales, the
// scales [tile][K-block][16 rows].
struct Space {
  int* active;         // number of routed experts
  int4* experts;       // {expert, first tile, rows, 0}
  int* row_token;      // [tiles * 16]
  float* row_weight;   // [tiles * 16]
  uint8_t* xq;
  float* xs;
  uint8_t* hq;
  float* hs;
  float* hf;           // [experts * T, I]: the product itself, where the down launch quantizes it
  float* gu;           // [K slices][tiles * 16][2][I]: gate and up sums, where K is sliced
  float* yp;           // [expert slices][T][H]: weighted sums, where the experts are sliced
  int rows, kper;      // tiles * 16; K-blocks per slice
};

size_t layout(int T, int top_k, int E, int H, int I, uint8_t* base, Space* s) {
  const size_t tiles = (size_t)max_tiles(T, top_k, E, H), rows = tiles * kTile;
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
  t.xq = take((size_t)T * H);
  t.xs = (float*)take((size_t)T * (H / 128) * sizeof(float));
  const bool late = use_late(T, top_k, E, H, I);
  const int ks = late ? 1 : gate_up_slices(T, top_k, E, H, I), es = down_slices(T, top_k, E, H, I);
  t.hq = take(late ? 0 : rows * I);
  t.hs = (float*)take(late ? 0 : rows * (I / 128) * sizeof(float));
  t.hf = (float*)take(late ? (size_t)max_experts(T, top_k, E) * T * I * sizeof(float) : 0);
  t.gu = (float*)take(ks > 1 ? ks * rows * 2 * I * sizeof(float) : 0);
  t.yp = (float*)take(es > 1 ? (size_t)es * T * H * sizeof(float) : 0);
  t.rows = (int)rows;
  t.kper = (H / 128 + ks - 1) / ks;
  if (s) *s = t;
  return at;
}

// ---------------------------------------------------------------------------------------------
// prep: workgroups 0 .. T-1 quantize a row of x each, workgroup T sorts the pairs: counts per expert
// (an LDS counter hands a pair its rank), an exclusive scan over the experts places the routed ones
// and their tiles.  A pair whose expert its token has named already is dropped and its weight goes
// to the first, so a token has one row per expert.
// ---------------------------------------------------------------------------------------------
constexpr int PREP = 1024;  // pairs and experts at most: one each per thread
static_assert(kMoeMaxPairs <= PREP && kMoeMaxExperts <= PREP, "one pair and one expert per thread");

// Codes of 16 consecutive values of row x (chunk c) and, from the chunk's first lane, the group's
// scale.  8 lanes share a group; whole groups are active.
__device__ __forceinline__ int4 quant_chunk(const uint16_t* x, int c, float& sc) {
  const int4 a = gload_i4(x + 16 * c), b = gload_i4(x + 16 * c + 8);
  const uint4 u = make_uint4(a.x, a.y, a.z, a.w), v = make_uint4(b.x, b.y, b.z, b.w);
  const uint32_t words[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  typedef unsigned short v2us __attribute__((ext_vector_type(2)));
  v2us m = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(v2us, words[i] & 0x7FFF7FFFu));
  sc = group_scale(lanes_max<8>((uint32_t)max(m[0], m[1]) << 16));
  int4 q;
  q.x = codes4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y), sc);
  q.y = codes4(bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w), sc);
  q.z = codes4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y), sc);
  q.w = codes4(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w), sc);
  return q;
}

__global__ __launch_bounds__(PREP) void moe_prep_kernel(MoeArgs p, Space s) {
  __shared__ int sid[kMoeMaxPairs];
  __shared__ int cnt[kMoeMaxExperts];
  __shared__ int first_tile[kMoeMaxExperts];
  __shared__ int part[PREP / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if ((int)blockIdx.x < p.T) {
    const int t = blockIdx.x;
    for (int c = tid; c < p.H / 16; c += PREP) {
      float sc;
      const int4 q = quant_chunk(p.x + (int64_t)t * p.ldx, c, sc);
      gstore<v4i>(s.xq + (int64_t)t * p.H + 16 * c, v4i{q.x, q.y, q.z, q.w});
      if (c % 8 == 0) gstore<float>(s.xs + (int64_t)t * (p.H / 128) + c / 8, sc);
    }
    return;
  }
  const int P = p.T * p.top_k;
  const int id = tid < P ? gload<int>(p.ids + tid) : -1;
  const float w = tid < P ? gload<float>(p.weights + tid) : 0.0f;
  sid[tid] = id;
  cnt[tid] = 0;
  __syncthreads();
  const int first = tid / p.top_k * p.top_k;
  bool keep = id >= 0 && id < p.E;
  for (int q = first; q < tid; ++q) keep = keep && sid[q] != id;
  const int rank = keep ? atomicAdd(&cnt[id], 1) : 0;
  __syncthreads();
  // expert tid: routed or not, its tiles; both scanned in one integer (at most 1024 and 1088)
  const int rows = cnt[tid];
  const int both = (rows > 0) + ((rows + kTile - 1) / kTile << 16);
  int inc = both;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 63) part[wave] = inc;
  __syncthreads();
  for (int q = 0; q < wave; ++q) inc += part[q];
  const int at = (inc - both) & 0xFFFF, tile = (inc - both) >> 16;
  first_tile[tid] = tile;
  if (rows > 0) s.experts[at] = make_int4(tid, tile, rows, 0);
  if (tid == PREP - 1) *s.active = inc & 0xFFFF;
  __syncthreads();
  if (keep) {
    float sum = w;  // with the weights of later pairs that name the same expert
    for (int q = tid + 1; q < first + p.top_k; ++q)
      if (sid[q] == id) sum += gload<float>(p.weights + q);
    const int row = first_tile[id] * kTile + rank;
    s.row_token[row] = tid / p.top_k;
    s.row_weight[row] = sum;
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

__device__ __forceinline__ v8i codes8(const int4& lo, const int4& hi) {
  v8i v;
  v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
  v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  return v;
}

// ---------------------------------------------------------------------------------------------
// One wave's stream: NT weight tiles (16 rows each) against MT activation tiles over nk K-blocks,
// D blocks in flight in registers.
//   acc[n][m] += P * (s_a * s_w[n])   per K-block, P the block's product sums.
// w[n]: lane address of weight tile n at the first block (row l/8, 16-byte chunk l%8), rows 8 further
// at + 8 * pitch; acts.load(kk, d) starts a block's activation loads, acts.start() runs once the first
// blocks are on their way, acts.codes(kk, d, m) and acts.scale(kk, d, m) give tile m's fragment and the
// scale of this lane's row; `scale(n, kk)` the weight block's.  Lanes whose row does not exist repeat
// one that does, and their results are dropped.  Blocks past the end are clamped to the last one, so
// the loads in flight are the same number in every step.
template <int NT, int MT, int D, typename Acts, typename Scale>
__device__ __forceinline__ void stream_blocks(const uint8_t* const (&w)[NT], int64_t pitch, Acts& acts, int nk,
                                              uint8_t* lds, Scale scale, v4f (&acc)[NT][MT]) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wo0 = swz(lane >> 3, lane & 7), wo1 = swz((lane >> 3) + 8, lane & 7);
  const int ro0 = swz(r, 2 * g), ro1 = swz(r, 2 * g + 1);
  int4 wv[D][NT][2];
  auto load = [&](int kk, int d) {
    const int64_t wk = (int64_t)kk * 128;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      wv[d][n][0] = gload_i4_last(w[n] + wk);
      wv[d][n][1] = gload_i4_last(w[n] + 8 * pitch + wk);
    }
    acts.load(kk, d);
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
    v8i af[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) af[m] = acts.codes(kk, d, m);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint8_t* t = lds + n * kFrag;
      const v8i wf = codes8(*reinterpret_cast<const int4*>(t + ro0), *reinterpret_cast<const int4*>(t + ro1));
      const float sw = scale(n, kk);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[n][m] += mfma_e4m3_16x16x128(wf, af[m]) * (acts.scale(kk, d, m) * sw);
        asm volatile("" : "+v"(acc[n][m]));
      }
    }
  };
#pragma unroll
  for (int d = 0; d < D - 1; ++d) load(min(d, nk - 1), d);
  __builtin_amdgcn_sched_barrier(0);
  acts.start();
  int kk = 0;
  for (; kk + D <= nk; kk += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      // (pinned: left to itself the scheduler sinks the loads to just before their use)
      load(min(kk + d + D - 1, nk - 1), (d + D - 1) % D);
      __builtin_amdgcn_sched_barrier(0);
      compute(kk + d, d);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (kk + d < nk) compute(kk + d, d);
}

// 16 bytes at base + lane_off + off: buffer form, scalar base and scalar offset, so that a stream of
// loads holds one address register per row.  AUX: kLastReadAux for weights (read for the last time).
template <int AUX>
__device__ __forceinline__ int4 bload16(const void* base, uint32_t lane_off, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)  // (the builtins exist in the device pass only)
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, -1, 0x00020000);
  const v4i v = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs, lane_off, off, AUX));
  return make_int4(v[0], v[1], v[2], v[3]);
#else
  return make_int4(0, 0, 0, 0);
#endif
}
__device__ __forceinline__ float bload4(const void* base, uint32_t lane_off) {
#if defined(__HIP_DEVICE_COMPILE__)
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, -1, 0x00020000);
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, lane_off, 0, 0));
#else
  return 0.0f;
#endif
}

// Barrier after LDS writes that other waves read next, without the fence that would also wait for
// every weight load in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));  // lgkmcnt(0), vmcnt and expcnt at their maxima
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------------------------
// gate+up: grid (I / 128, routed experts at most), 8 waves.
//
// The expert's activation codes go through LDS, once for the 8 waves: chunks of CH K-blocks, two
// buffers, the next chunk loaded into registers while the current one is multiplied.  (Loaded by each
// wave into registers, the activations of a popular expert's 64 rows were 2 x 4 KB per 4 KB of
// weights, and as vector-memory loads complete in order, waiting for them waited for the weight
// loads issued before them.)  In LDS, 16-byte chunk c of row r of K-block k sits at slot r ^ (c + 8 (k & 1))
// of its 16-slot group: writes of one row's 16 chunks and reads of one chunk of 16 rows both hit 16
// distinct bank groups.
// MTMAX: the most 16-row tiles an expert can have (T <= 16 MTMAX).
// ---------------------------------------------------------------------------------------------
constexpr int CH = 4;  // K-blocks per chunk and weight blocks in registers per wave

struct Routed {
  int e, tile0, rows;  // expert, its first tile, its rows; e < 0: the workgroup has none
};

// FUSED: every workgroup finds routed expert number `n` (in ascending order) and its tokens from the ids:
// a bit per expert, the n-th set bit, then the pairs that name it, in order, a token once.  `tokens`
// gets the rows' tokens.  The workgroups of column 0 write the expert's table entries for the down launch.
__device__ __forceinline__ Routed find_expert(const MoeArgs& p, const Space& s, int n, bool writes, int* sid,
                                              uint32_t* bits, int* tokens) {
  const int tid = threadIdx.x, lane = tid & 63, P = p.T * p.top_k;
  if (tid < kMoeMaxExperts / 32) bits[tid] = 0;
  for (int q = tid; q < P; q += 512) sid[q] = gload<int>(p.ids + q);
  __syncthreads();
  for (int q = tid; q < P; q += 512) {
    const int id = sid[q];
    if (id >= 0 && id < p.E) atomicOr(&bits[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
  const uint32_t word = lane < kMoeMaxExperts / 32 ? bits[lane] : 0u;
  const int count = __popc(word);
  int inc = count;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  const int active = __builtin_amdgcn_readlane(inc, 31);
  if (writes && n == 0 && tid == 0) *s.active = active;
  if (n >= active) return Routed{-1, 0, 0};
  const int w = __ffsll((long long)__ballot(inc > n && inc - count <= n)) - 1;
  uint32_t left = (uint32_t)__builtin_amdgcn_readlane((int)word, w);
  for (int skip = n - __builtin_amdgcn_readlane(inc - count, w); skip > 0; --skip) left &= left - 1;
  Routed ex{32 * w + __ffs((int)left) - 1, n * ((p.T + kTile - 1) / kTile), 0};
  for (int c = 0; c < P; c += 64) {
    const int q = c + lane;
    bool keep = q < P && sid[q] == ex.e;
    const int t = q / p.top_k;
    for (int f = t * p.top_k; keep && f < q; ++f) keep = sid[f] != ex.e;
    const unsigned long long mask = __ballot(keep);
    if (keep) {
      const int row = ex.rows + __popcll(mask & ((1ull << lane) - 1));
      tokens[row] = t;  // (all waves write the same)
      if (writes && tid < 64) {
        float sum = 0.0f;  // with the weights of later pairs of the token that name the same expert
        for (int f = q; f < (t + 1) * p.top_k; ++f)
          if (sid[f] == ex.e) sum += gload<float>(p.weights + f);
        s.row_token[ex.tile0 * kTile + row] = t;
        s.row_weight[ex.tile0 * kTile + row] = sum;
      }
    }
    ex.rows += __popcll(mask);
  }
  if (writes && tid == 0) s.experts[n] = make_int4(ex.e, ex.tile0, ex.rows, 0);
  return ex;
}

template <int SWF, int MTMAX, bool FUSED, int COLS = 128>
__global__ __launch_bounds__(512, 2) void moe_gate_up_kernel(MoeArgs p, Space s) {
  static_assert(!FUSED || MTMAX * kTile <= kFusedTokens, "few tokens");
  static_assert(COLS == 128 || (COLS == 64 && FUSED && MTMAX == 1), "half groups: quantized by the down launch");
  constexpr int CT = COLS / 16;  // column tiles; 64 columns: two waves each, splitting the K-blocks
  __shared__ __attribute__((aligned(1024))) uint8_t wtiles[8][2 * kFrag];
  __shared__ __attribute__((aligned(1024))) uint8_t atiles[2][FUSED ? 16 : CH * MTMAX * kFrag];
  __shared__ float ascale[2][CH][FUSED ? 1 : MTMAX * kTile];
  __shared__ float sws[2][256];  // the two weight block rows' scales (H <= 32768)
  __shared__ uint32_t amax[8][MTMAX * kTile];  // magnitudes
  // FUSED: the expert's rows, codes [H/128][T][128] (16-byte chunks swizzled by row) and scales [H/128][T]
  extern __shared__ __attribute__((aligned(1024))) uint8_t xrows[];
  __shared__ int sid[FUSED ? kMoeMaxPairs : 1];
  __shared__ uint32_t bits[FUSED ? kMoeMaxExperts / 32 : 1];
  __shared__ int tokens[FUSED ? kFusedTokens : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  int e, tile0, rows;
  if constexpr (FUSED) {
    const Routed ex = find_expert(p, s, blockIdx.y, blockIdx.x == 0 && blockIdx.z == 0, sid, bits, tokens);
    if (ex.e < 0) return;
    e = ex.e;
    tile0 = ex.tile0;
    rows = ex.rows;
  } else {
    // (the entry is loaded with the count, not after it: a workgroup past the count drops it)
    const int active = gload<int>(s.active);
    const v4i ex = gload<v4i>(s.experts + blockIdx.y);
    if ((int)blockIdx.y >= active) return;
    e = ex[0];
    tile0 = ex[1];
    rows = ex[2];
  }
  e = __builtin_amdgcn_readfirstlane(e);
  tile0 = __builtin_amdgcn_readfirstlane(tile0);
  rows = __builtin_amdgcn_readfirstlane(rows);
  const int KB = p.H / 128, NB = p.I / 128, gb = blockIdx.x * COLS / 128;
  // this wave's K-blocks: the workgroup's slice, or (64 columns) one half
  const int ct = wave % CT;
  const int kbeg = COLS == 64 ? wave / CT * ((KB + 1) / 2) : min((int)blockIdx.z * s.kper, KB);
  const int kend = COLS == 64 ? (wave < CT ? (KB + 1) / 2 : KB) : min(kbeg + s.kper, KB);
  // this lane's weight bytes from the expert's first: 32-bit offsets (2 I H <= 2^31), the K-block is the
  // buffer load's scalar offset
  const uint32_t wrow = (uint32_t)((blockIdx.x * COLS + ct * 16 + (lane >> 3)) * p.H + 16 * (lane & 7));
  const uint32_t up = (uint32_t)p.I * p.H, pitch8 = 8u * p.H;
  const uint32_t woff[4] = {wrow, wrow + pitch8, wrow + up, wrow + up + pitch8};
  const uint8_t* const wexp = p.w13_q + (int64_t)e * 2 * p.I * p.H;
  const int wo0 = swz(lane >> 3, lane & 7), wo1 = swz((lane >> 3) + 8, lane & 7);
  const int ro0 = swz(r, 2 * g), ro1 = swz(r, 2 * g + 1);
  uint8_t* const wt = &wtiles[wave][0];

  auto run = [&](auto mt_c) {
    constexpr int MT = decltype(mt_c)::value;
    // weights: blocks past the end repeat the last one (their scale is 0)
    int4 wv[CH][2][2];
    auto block = [&](int kk) { return max(min(kbeg + kk, kend - 1), 0); };
    auto load = [&](int kk, int d) {
#pragma unroll
      for (int i = 0; i < 4; ++i) wv[d][i / 2][i % 2] = bload16<kLastReadAux>(wexp, woff[i], (uint32_t)block(kk) * 128);
    };
    // activations: a chunk is CH * 128 contiguous bytes of each row; copy i of a thread takes 16 of them
    // (rows past the count repeat the last one)
    constexpr int RC = CH * 8, NA = MT * kTile * RC / 512, RPC = 512 / RC;  // 16-byte pieces per row, copies, rows per copy
    static_assert(NA * 512 == MT * kTile * RC && kTile % RPC == 0, "whole copies");
    int4 av[NA];
    float sv = 0.0f;
    const int ak = tid % RC / 8, ac = tid & 7, ar = tid / RC;
    uint32_t aoff[NA], soff = 0;
    const int sk = tid / (MT * kTile), sr = tid % (MT * kTile);  // scale of row sr, block sk < CH
    if constexpr (!FUSED) {
#pragma unroll
      for (int i = 0; i < NA; ++i)
        aoff[i] = (uint32_t)gload<int>(s.row_token + tile0 * kTile + min(i * RPC + ar, rows - 1)) * p.H + 16 * ac;
      soff = (uint32_t)gload<int>(s.row_token + tile0 * kTile + min(sr, rows - 1)) * KB * 4;
    }
    auto fetch = [&](int k0) {
#pragma unroll
      for (int i = 0; i < NA; ++i) av[i] = bload16<0>(s.xq, aoff[i] + block(k0 + ak) * 128, 0);
      sv = bload4(s.xs, soff + block(k0 + min(sk, CH - 1)) * 4);
    };
    float* const xscale = reinterpret_cast<float*>(xrows + p.T * p.H);
    // this lane's rows (FUSED; rows past the count repeat the last one)
    int fq[MT], flo[MT], fhi[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      fq[m] = min(m * kTile + r, rows - 1);
      flo[m] = swz(fq[m], 2 * g);
      fhi[m] = swz(fq[m], 2 * g + 1);
    }
    auto stash = [&](int k0, int buf) {
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        const int q = i * RPC + ar;
        *reinterpret_cast<int4*>(&atiles[buf][(ak * MT + q / kTile) * kFrag + (ac & 1) * 1024 +
                                              ((ac >> 1) * 16 + ((q % kTile) ^ (ac + 8 * (ak & 1)))) * 16]) = av[i];
      }
      if (sk < CH) ascale[buf][sk][sr] = kbeg + k0 + sk < kend ? sv : 0.0f;
    };
    v4f acc[2][MT];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto compute = [&](int kk, int d, int buf) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        // (a wave's LDS operations complete in order: the reads see the writes, and the next block's
        // writes follow these reads)
        *reinterpret_cast<int4*>(wt + n * kFrag + wo0) = wv[d][n][0];
        *reinterpret_cast<int4*>(wt + n * kFrag + wo1) = wv[d][n][1];
      }
      Wide wf[2];
      float sw[2];
      auto weights = [&](int n) {
        wf[n] = widen(*reinterpret_cast<const int4*>(wt + n * kFrag + ro0), *reinterpret_cast<const int4*>(wt + n * kFrag + ro1));
        sw[n] = sws[n][block(kk)];
      };
      // (one activation tile: the weight tiles are widened one after the other, which keeps the kernel
      // within the registers of two workgroups per CU)
      if constexpr (MT > 1) {
        weights(0);
        weights(1);
      }
      const uint8_t* const t = FUSED ? xrows + block(kk) * p.T * 128 : &atiles[buf][d * MT * kFrag];
      const int lo = (g * 16 + (r ^ (2 * g + 8 * (d & 1)))) * 16, hi = 1024 + (g * 16 + (r ^ (2 * g + 1 + 8 * (d & 1)))) * 16;
      auto half = [&](int m, bool second) {
        return *reinterpret_cast<const int4*>(t + (FUSED ? (second ? fhi[m] : flo[m]) : m * kFrag + (second ? hi : lo)));
      };
      int4 alo = half(0, false), ahi = half(0, true);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const Wide af = widen(alo, ahi);
        const float sa = FUSED ? (kbeg + kk < kend ? xscale[block(kk) * p.T + fq[m]] : 0.0f) : ascale[buf][d][m * kTile + r];
        if (m + 1 < MT) {
          alo = half(m + 1, false);
          ahi = half(m + 1, true);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if constexpr (MT == 1) weights(n);
          acc[n][m] += block_sum(wf[n], af) * (sa * sw[n]);
          // (the sum is due here: left alone, the compiler keeps every block's product sums to the end
          // of the chunk, in the registers that the weights in flight need)
          asm volatile("" : "+v"(acc[n][m]));
        }
      }
    };
#pragma unroll
    for (int d = 0; d < CH - 1; ++d) load(d, d);
    if constexpr (!FUSED) fetch(0);
    __builtin_amdgcn_sched_barrier(0);
    const int64_t sw0 = ((int64_t)e * 2 * NB + gb) * KB;
    for (int k = tid; k < KB; k += 512) {
      sws[0][k] = load_sw<SWF>(p.s_w13, sw0 + k);
      sws[1][k] = load_sw<SWF>(p.s_w13, sw0 + (int64_t)NB * KB + k);
    }
    if constexpr (FUSED) {
      const int c0 = COLS == 64 ? 0 : kbeg * 8, chunks = COLS == 64 ? p.H / 16 : (kend - kbeg) * 8;
      for (int i = tid; i < rows * chunks; i += 512) {
        const int q = i / chunks, c = c0 + i - q * chunks;
        float sc;
        const int4 codes = quant_chunk(p.x + (int64_t)tokens[q] * p.ldx, c, sc);
        *reinterpret_cast<int4*>(xrows + c / 8 * p.T * 128 + swz(q, c % 8)) = codes;
        if (c % 8 == 0) xscale[c / 8 * p.T + q] = sc;
      }
    } else {
      stash(0, 0);
    }
    lds_barrier();
    int buf = 0;
    for (int k0 = 0; k0 < kend - kbeg; k0 += CH) {
      if constexpr (!FUSED) fetch(k0 + CH);  // (past the end: the last block again, stashed where nothing reads it)
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < CH; ++d) {
        // (pinned: left to itself the scheduler sinks the loads to just before their use)
        load(k0 + d + CH - 1, (d + CH - 1) % CH);
        __builtin_amdgcn_sched_barrier(0);
        compute(k0 + d, d, buf);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!FUSED) {
        stash(k0 + CH, buf ^ 1);
        lds_barrier();
        buf ^= 1;
      }
    }
    if constexpr (COLS == 64) {
      // the two K halves, the gated product, float32
      v4f* const red = reinterpret_cast<v4f*>(wtiles);
      __syncthreads();  // (the weight tiles are free)
      if (wave >= CT) {
        red[(ct * 2 + 0) * 64 + lane] = acc[0][0];
        red[(ct * 2 + 1) * 64 + lane] = acc[1][0];
      }
      __syncthreads();
      if (wave < CT && r < rows) {
        const v4f gate = acc[0][0] + red[(ct * 2 + 0) * 64 + lane], u = acc[1][0] + red[(ct * 2 + 1) * 64 + lane];
        float v[4] = {gate[0], gate[1], gate[2], gate[3]};
        activate<4>(p.act, v);
        gstore<v4f>(s.hf + ((int64_t)blockIdx.y * p.T + r) * p.I + blockIdx.x * COLS + ct * 16 + 4 * g,
                    v4f{v[0] * u[0], v[1] * u[1], v[2] * u[2], v[3] * u[3]});
      }
      return;
    }
    if (gridDim.z > 1) {  // a K slice: the sums as they are
      if (COLS == 128) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (m * kTile + r < rows) {
            float* const q = s.gu + (((int64_t)blockIdx.z * s.rows + (tile0 + m) * kTile + r) * 2) * p.I + gb * 128 + wave * 16 + 4 * g;
            gstore<v4f>(q, acc[0][m]);
            gstore<v4f>(q + p.I, acc[1][m]);
          }
        }
      }
      return;
    }
    // the gated product of this wave's 16 columns (lane: row r, columns 4 g .. 4 g + 3) and the rows'
    // maxima over the workgroup's 128 columns
    v4f h[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float v[4] = {acc[0][m][0], acc[0][m][1], acc[0][m][2], acc[0][m][3]};
      activate<4>(p.act, v);
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[m][i] = v[i] * acc[1][m][i];
        mx = max(mx, magnitude(h[m][i]));
      }
      mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16));
      mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
      if (g == 0) amax[wave][m * kTile + r] = mx;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m * kTile + r < rows) {
        uint32_t mx = amax[0][m * kTile + r];
#pragma unroll
        for (int q = 1; q < 8; ++q) mx = max(mx, amax[q][m * kTile + r]);
        const float sc = group_scale(mx);
        const uint32_t c = codes4(h[m][0], h[m][1], h[m][2], h[m][3], sc);
        uint8_t* hq = s.hq + ((int64_t)(tile0 + m) * NB + gb) * kFrag;
        gstore<uint32_t>(hq + (wave & 1) * 1024 + ((wave >> 1) * 16 + r) * 16 + 4 * g, c);
        if (wave == 0 && g == 0) gstore<float>(s.hs + ((int64_t)(tile0 + m) * NB + gb) * kTile + r, sc);
      }
    }
  };
  if (MTMAX == 1 || rows <= 16) run(std::integral_constant<int, 1>{});
  else if (MTMAX == 2 || rows <= 32) run(std::integral_constant<int, MTMAX < 2 ? 1 : 2>{});
  else run(std::integral_constant<int, MTMAX < 4 ? 1 : 4>{});
}

// The sliced gate+up sums: grid (I / 128, tiles), 16 threads per row of 16, 8 columns each.  Slices in
// order, then activation, gate and quantization as above.
__global__ __launch_bounds__(256) void moe_gate_up_finish_kernel(MoeArgs p, Space s, int slices) {
  const int active = gload<int>(s.active);
  if (active == 0) return;
  const v4i last = gload<v4i>(s.experts + active - 1);
  const int tile = blockIdx.y, row = threadIdx.x >> 4, j = threadIdx.x & 15, gb = blockIdx.x, NB = p.I / 128;
  if (tile >= last[1] + (last[2] + kTile - 1) / kTile) return;
  // (a tile's rows past its count, and without the prep launch whole tiles between two experts', hold what the
  // workspace held: their results go to their own places, which nothing reads)
  const float* q = s.gu + ((int64_t)(tile * kTile + row) * 2) * p.I + gb * 128 + 8 * j;
  float gate[8], u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) gate[i] = u[i] = 0.0f;
  for (int z = 0; z < slices; ++z, q += (int64_t)s.rows * 2 * p.I) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const v4f a = gload<v4f>(q + 4 * i), b = gload<v4f>(q + p.I + 4 * i);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        gate[4 * i + k] += a[k];
        u[4 * i + k] += b[k];
      }
    }
  }
  activate<8>(p.act, gate);
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    gate[i] *= u[i];
    mx = max(mx, magnitude(gate[i]));
  }
  const float sc = group_scale(lanes_max<16>(mx));
  v2u c;
  c[0] = codes4(gate[0], gate[1], gate[2], gate[3], sc);
  c[1] = codes4(gate[4], gate[5], gate[6], gate[7], sc);
  uint8_t* hq = s.hq + ((int64_t)tile * NB + gb) * kFrag;
  gstore<v2u>(hq + (j >> 1 & 1) * 1024 + ((j >> 2) * 16 + row) * 16 + (j & 1) * 8, c);
  if (j == 0) gstore<float>(s.hs + ((int64_t)tile * NB + gb) * kTile + row, sc);
}

// The sliced weighted sums: slices in order, the residual, one rounding.
template <int OUT>
__global__ __launch_bounds__(256) void moe_down_finish_kernel(MoeArgs p, Space s, int slices) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.T * (p.H / 4)) return;
  const int t = i / (p.H / 4), n = (i - t * (p.H / 4)) * 4;
  v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int z = 0; z < slices; ++z) sum += gload<v4f>(s.yp + ((int64_t)z * p.T + t) * p.H + n);
  if (p.residual != nullptr) {
    float f[4];
    load_values(p.residual, p.residual_dtype, (int64_t)t * p.ldr + n, f);
    sum += v4f{f[0], f[1], f[2], f[3]};
  }
  store4<OUT>(p.y, p.ldy, t, n, sum);
}

// Activations of the down products: the quantized product's fragments from the workspace ...
template <int MT, int D>
struct StoredActs {
  const uint8_t* a[MT];   // lane address of tile m's fragment at the first block
  const float* sa[MT];    // and of its row's scale
  int4 av[D][MT][2];
  float sv[D][MT];
  __device__ __forceinline__ void load(int kk, int d) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      av[d][m][0] = gload_i4(a[m] + (int64_t)kk * kFrag);
      av[d][m][1] = gload_i4(a[m] + (int64_t)kk * kFrag + 1024);
      sv[d][m] = gload<float>(sa[m] + kk * kTile);
    }
  }
  __device__ __forceinline__ void start() {}
  __device__ __forceinline__ v8i codes(int, int d, int m) const { return codes8(av[d][m][0], av[d][m][1]); }
  __device__ __forceinline__ float scale(int, int d, int m) const { return sv[d][m]; }
};

// ... or the product's float32 rows, quantized by the wave for its own K-blocks: 8 lanes per 128-group,
// 16 values each; codes [block][T][128], chunks swizzled by row, and scales [block][T] in LDS.
struct LateActs {
  const float* h;  // row 0 at the first block
  int64_t pitch;
  int T, rows, nk, q;  // q: this lane's row
  uint8_t* codes_lds;
  float* scale_lds;
  __device__ __forceinline__ void load(int, int) {}
  __device__ __forceinline__ void start() {
    const int lane = threadIdx.x & 63;
    for (int i = lane >> 3; i < nk * rows; i += 8) {  // (whole 8-lane groups)
      const int kk = i / rows, row = i - kk * rows;
      const float* src = h + row * pitch + kk * 128 + 16 * (lane & 7);
      float v[16];
      uint32_t mx = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const v4f t = gload<v4f>(src + 4 * u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[4 * u + j] = t[j];
          mx = max(mx, magnitude(t[j]));
        }
      }
      const float sc = group_scale(lanes_max<8>(mx));
      int4 c;
      c.x = codes4(v[0], v[1], v[2], v[3], sc);
      c.y = codes4(v[4], v[5], v[6], v[7], sc);
      c.z = codes4(v[8], v[9], v[10], v[11], sc);
      c.w = codes4(v[12], v[13], v[14], v[15], sc);
      *reinterpret_cast<int4*>(codes_lds + kk * T * 128 + swz(row, lane & 7)) = c;
      if ((lane & 7) == 0) scale_lds[kk * T + row] = sc;
    }
  }
  __device__ __forceinline__ v8i codes(int kk, int, int) const {
    const int g = (threadIdx.x & 63) >> 4;
    const uint8_t* t = codes_lds + kk * T * 128;
    return codes8(*reinterpret_cast<const int4*>(t + swz(q, 2 * g)), *reinterpret_cast<const int4*>(t + swz(q, 2 * g + 1)));
  }
  __device__ __forceinline__ float scale(int kk, int, int) const { return scale_lds[kk * T + q]; }
};

// ---------------------------------------------------------------------------------------------
// down: grid (H / (16 NT), slices), WK waves.  The K-blocks of all routed experts, in expert order, are
// one list that the slices' waves split evenly; a wave walks its share expert by expert (segments).
// ---------------------------------------------------------------------------------------------
template <int SWF, int OUT, int MTMAX, int NT, int WK, bool LATE>
__global__ __launch_bounds__(64 * WK) void moe_down_kernel(MoeArgs p, Space s) {
  constexpr int COLS = 16 * NT;
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[WK][NT * kFrag];
  // [WK waves][T][COLS]; LATE: then the waves' codes and scales of a segment (late_codes_at, late_scales_at)
  extern __shared__ __attribute__((aligned(16))) float ysum[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * COLS;
  const int KB = p.I / 128, NB = p.H / 128;
  float* const mine = ysum + wave * p.T * COLS;
  for (int i = lane; i < p.T * (COLS / 4); i += 64) *reinterpret_cast<v4f*>(mine + 4 * i) = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // lane l holds the table entries of routed expert l (loaded with the count; entries past it are not
  // used), later ones are loaded when they come up
  const v4i table = gload<v4i>(s.experts + min(lane, min(p.T * p.top_k, p.E) - 1));
  const int units = gload<int>(s.active) * KB;
  const int part = blockIdx.y * WK + wave, per = (units + WK * (int)gridDim.y - 1) / (WK * (int)gridDim.y);
  int u = __builtin_amdgcn_readfirstlane(min(units, part * per));
  const int u1 = __builtin_amdgcn_readfirstlane(min(units, (part + 1) * per));
  while (u < u1) {
    const int si = u / KB, kb0 = u - si * KB;
    const int nk = min(min(KB - kb0, u1 - u), 64);
    int e, tile0, rows;
    if (si < 64) {
      e = __builtin_amdgcn_readlane(table[0], si);
      tile0 = __builtin_amdgcn_readlane(table[1], si);
      rows = __builtin_amdgcn_readlane(table[2], si);
    } else {
      const v4i ex = gload<v4i>(s.experts + si);
      e = __builtin_amdgcn_readfirstlane(ex[0]);
      tile0 = __builtin_amdgcn_readfirstlane(ex[1]);
      rows = __builtin_amdgcn_readfirstlane(ex[2]);
    }
    const float swl = lane < nk ? load_sw<SWF>(p.s_w2, ((int64_t)e * NB + n0 / 128) * KB + kb0 + lane) : 0.0f;
    const uint8_t* w0 = p.w2_q + ((int64_t)e * p.H + n0 + (lane >> 3)) * p.I + (int64_t)kb0 * 128 + 16 * (lane & 7);
    const uint8_t* w[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) w[n] = w0 + (int64_t)16 * n * p.I;
    auto run = [&](auto mt_c) {
      constexpr int MT = decltype(mt_c)::value;
      constexpr int D = 3;  // blocks in registers (4: 2-8% slower with one row tile, registers; 2: 5% with four)
      std::conditional_t<LATE, LateActs, StoredActs<MT, D>> acts;
      if constexpr (LATE) {
        static_assert(WK == kDownWaves, "LDS layout");
        const int seg = late_segment(p.I);
        uint8_t* const mem = reinterpret_cast<uint8_t*>(ysum + WK * p.T * COLS);
        acts.h = s.hf + (int64_t)si * p.T * p.I + kb0 * 128;
        acts.pitch = p.I;
        acts.T = p.T;
        acts.rows = rows;
        acts.nk = nk;
        acts.q = min(r, rows - 1);
        acts.codes_lds = mem + late_codes_at(wave, seg, p.T);
        acts.scale_lds = reinterpret_cast<float*>(mem + late_scales_at(wave, seg, p.T));
      } else {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int q = min(m * kTile + r, rows - 1);
          acts.a[m] = s.hq + ((int64_t)(tile0 + q / kTile) * KB + kb0) * kFrag + (g * kTile + q % kTile) * 16;
          acts.sa[m] = s.hs + ((int64_t)(tile0 + q / kTile) * KB + kb0) * kTile + q % kTile;
        }
      }
      // the rows' tokens and weights, needed at the segment's end
      int token[MT];
      float weight[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = tile0 * kTile + min(m * kTile + r, rows - 1);
        token[m] = gload<int>(s.row_token + row);
        weight[m] = gload<float>(s.row_weight + row);
      }
      v4f acc[NT][MT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      stream_blocks<NT, MT, D>(w, p.I, acts, nk, &tiles[wave][0],
                              [&](int, int kk) {
                                return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(swl), kk));
                              }, acc);
      // (a token has one row per expert, so no two lanes add to the same sums)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m * kTile + r < rows) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            v4f* const q = reinterpret_cast<v4f*>(mine + token[m] * COLS + n * 16 + 4 * g);
            *q += acc[n][m] * weight[m];
          }
        }
      }
    };
    if (MTMAX == 1 || rows <= 16) run(std::integral_constant<int, 1>{});
    else if (MTMAX == 2 || rows <= 32) run(std::integral_constant<int, MTMAX < 2 ? 1 : 2>{});
    else run(std::integral_constant<int, MTMAX < 4 ? 1 : 4>{});
    u += nk;
  }
  __syncthreads();
  // the waves' sums in wave order, the residual, one rounding
  for (int i = tid; i < p.T * (COLS / 4); i += 64 * WK) {
    const int t = i / (COLS / 4), c = i % (COLS / 4) * 4;
    v4f sum = *reinterpret_cast<const v4f*>(ysum + t * COLS + c);
#pragma unroll
    for (int q = 1; q < WK; ++q) sum += *reinterpret_cast<const v4f*>(ysum + (q * p.T + t) * COLS + c);
    if (gridDim.y > 1) {  // a slice
      gstore<v4f>(s.yp + ((int64_t)blockIdx.y * p.T + t) * p.H + n0 + c, sum);
      continue;
    }
    if (p.residual != nullptr) {
      float f[4];
      load_values(p.residual, p.residual_dtype, (int64_t)t * p.ldr + n0 + c, f);
      sum += v4f{f[0], f[1], f[2], f[3]};
    }
    store4<OUT>(p.y, p.ldy, t, n0 + c, sum);
  }
}

}  // namespace

size_t moe_ffn_workspace_bytes(int T, int top_k, int E, int H, int I) {
  return layout(T, top_k, E, H, I, nullptr, nullptr);
}

namespace {

template <int MTMAX, bool FUSED, int COLS>
void launch_gate_up(const MoeArgs& a, const Space& s, int slices, hipStream_t stream) {
  const dim3 grid((unsigned)(a.I / COLS), (unsigned)max_experts(a.T, a.top_k, a.E), (unsigned)slices), block(512);
  const size_t lds = FUSED ? (size_t)a.T * (a.H + a.H / 128 * sizeof(float)) : 0;
  if (a.s_w_fmt == 0) hipLaunchKernelGGL((moe_gate_up_kernel<0, MTMAX, FUSED, COLS>), grid, block, lds, stream, a, s);
  else hipLaunchKernelGGL((moe_gate_up_kernel<1, MTMAX, FUSED, COLS>), grid, block, lds, stream, a, s);
}

template <int MTMAX>
hipError_t launch_layer(const MoeArgs& a, const Space& s, hipStream_t stream) {
  hipError_t e;
  const bool late = use_late(a.T, a.top_k, a.E, a.H, a.I);
  // (no empty slice: kper blocks each)
  const int ks = late ? 1 : (a.H / 128 + s.kper - 1) / s.kper;
  const int es = down_slices(a.T, a.top_k, a.E, a.H, a.I);
  if (MTMAX == 1 && late) {
    launch_gate_up<1, true, 64>(a, s, 1, stream);
  } else if (MTMAX * kTile <= kFusedTokens && fused_prep(a.T, a.H)) {
    launch_gate_up<MTMAX * kTile <= kFusedTokens ? MTMAX : 1, true, 128>(a, s, ks, stream);
  } else {
    hipLaunchKernelGGL(moe_prep_kernel, dim3((unsigned)a.T + 1), dim3(PREP), 0, stream, a, s);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    launch_gate_up<MTMAX, false, 128>(a, s, ks, stream);
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (ks > 1) {
    hipLaunchKernelGGL(moe_gate_up_finish_kernel, dim3((unsigned)(a.I / 128), (unsigned)(s.rows / kTile)), dim3(256), 0,
                       stream, a, s, ks);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // (late: one activation tile, T <= 16)
  const size_t extra = late ? (size_t)late_bytes(late_segment(a.I), a.T) : 0;
#define FGB_DOWN_LATE(SWF, OUT, NT, WK, LATE)                                                                     \
  hipLaunchKernelGGL((moe_down_kernel<SWF, OUT, LATE ? 1 : MTMAX, NT, WK, LATE>), dim3((unsigned)(a.H / (16 * NT)), (unsigned)es), \
                     dim3(64 * WK), (size_t)WK * a.T * 16 * NT * sizeof(float) + extra, stream, a, s)
#define FGB_DOWN(SWF, OUT, NT, WK)                            \
  do {                                                        \
    if (MTMAX == 1 && late) FGB_DOWN_LATE(SWF, OUT, NT, WK, true); \
    else FGB_DOWN_LATE(SWF, OUT, NT, WK, false);              \
  } while (0)
#define FGB_DOWN_TYPES(NT, WK)                            \
  do {                                                    \
    if (a.s_w_fmt == 0) {                                 \
      if (a.y_dtype == 0) FGB_DOWN(0, 0, NT, WK);         \
      else FGB_DOWN(0, 1, NT, WK);                        \
    } else {                                              \
      if (a.y_dtype == 0) FGB_DOWN(1, 0, NT, WK);         \
      else FGB_DOWN(1, 1, NT, WK);                        \
    }                                                     \
  } while (0)
  // two weight tiles per wave share each activation fragment, and two tiles' bytes are in flight; one
  // where that would leave CUs without a workgroup (measured: H = 7168, 224 workgroups of 32 columns
  // 20.2 us against 448 of 16 23.6 at 1 token, 86 against 139 at 64; H = 2048, 128 workgroups of 16
  // columns 17.0 us against 64 of 32 24.5)
  if (down_wide(a.H)) FGB_DOWN_TYPES(2, kDownWaves);
  else FGB_DOWN_TYPES(1, kDownWaves);
#undef FGB_DOWN_TYPES
#undef FGB_DOWN
#undef FGB_DOWN_LATE
  e = hipGetLastError();
  if (e != hipSuccess || es == 1) return e;
  const dim3 fgrid((unsigned)((a.T * (a.H / 4) + 255) / 256));
  if (a.y_dtype == 0) hipLaunchKernelGGL(moe_down_finish_kernel<0>, fgrid, dim3(256), 0, stream, a, s, es);
  else hipLaunchKernelGGL(moe_down_finish_kernel<1>, fgrid, dim3(256), 0, stream, a, s, es);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_ffn(const MoeArgs& a, void* workspace, hipStream_t stream) {
  Space s;
  layout(a.T, a.top_k, a.E, a.H, a.I, reinterpret_cast<uint8_t*>(workspace), &s);
  if (a.T <= 16) return launch_layer<1>(a, s, stream);
  if (a.T <= 32) return launch_layer<2>(a, s, stream);
  return launch_layer<4>(a, s, stream);
}

}  // namespace fgb
