// moe_plan.hpp — which launches the few-token mixture-of-experts layer takes (moe_ffn.hip), how they are
// sliced, and the down launch's LDS behind its sums.  Plain C++: rules on sizes alone.
#pragma once
#include <stddef.h>

namespace fgb {

constexpr int kTile = 16;      // rows per activation tile
constexpr int kDownWaves = 8;  // waves per workgroup of the down launch

inline int max_experts(int T, int top_k, int E) { return T * top_k < E ? T * top_k : E; }

// Whether the gate+up workgroups find their expert and quantize its rows themselves (no prep launch).  Up
// to 16 tokens the rows' codes, T * H bytes at most, have to leave LDS for two workgroups per CU; with more
// the registers allow one only, and the limit is the time that quantizing takes.  Measured, tokens x
// experts x top_k x H x I, all launches, without and with the prep launch: 1 x 32 x 8 x 7168 x 2048 70.7
// and 73.8 us, 9 x 32 x 8 x 4096 x 2048 (36 KB) 131 and 138, 7 x 32 x 8 x 7168 x 2048 (49 KB, one workgroup
// per CU) 171 and 168; 19 x 24 x 4 x 2048 x 1408 44.0 and 45.2, 32 x 8 x 2 x 2048 x 1024 (64 KB) 26.7 and
// 27.9, 20 x 16 x 4 x 4096 x 1024 (80 KB) 58.1 and 56.1.
constexpr int kFusedTokens = 32, kFusedBytes = 39 << 10, kFusedManyBytes = 64 << 10;
inline bool fused_prep(int T, int H) {
  return T <= kFusedTokens && T * H <= (T <= kTile ? kFusedBytes : kFusedManyBytes);
}

// Whether the gated product is quantized by the down launch.  A gate+up workgroup of 128 columns (the
// quantization group) leaves half the CUs idle when one or two tokens reach only a few experts, and a CU
// takes in no more than about 16 bytes a clock whatever is in flight (128 workgroups: 5.0 TB/s with 3
// or with 7 K-blocks ahead); workgroups of 64 columns write the float32 product and every down
// workgroup quantizes all of it, which has to stay small.  Measured at 1 token (7168 x 2048, 32 experts,
// top 8): gate+up 50.2 -> 40.5 us, down 20.5 -> 22.4 us.
constexpr int kLateValues = 32 << 10, kLateBlocks = 62;
inline bool late_quant(int T, int top_k, int E, int H, int I) {
  return T <= kTile && fused_prep(T, H) && max_experts(T, top_k, E) * T * (I / 128) <= kLateValues / 128 &&
         (I / 128 < 64 ? I / 128 : 64) * T <= kLateBlocks;
}

// Few experts or a narrow layer give few workgroups, and a CU's share of the stream is bounded (above):
// then the launches are sliced over grid.z (gate+up, along K) and grid.y (down, over the experts'
// K-blocks), with float32 partial sums added in slice order by one more launch each, which costs 3 to
// 4 us: about 8 K-blocks of a gate+up workgroup's time.  Slices fill the 256 CUs (more are slower, two of
// each 16 x 8 x 2 x 7168 x 2048 67 us, four 74) and keep at least 4 K-blocks per wave.  Measured, tokens x
// experts x top_k x H x I, whole layer without and with slices: 64 x 4 x 2 x 7168 x 2048 93 and 58 us, 64 x
// 2 x 1 x 7168 x 2048 86 and 43, 16 x 4 x 2 x 4096 x 1024 36.6 and 24.7 (gate+up); 32 x 32 x 4 x 512 x 4096
// 98 and 62, 8 x 64 x 6 x 2048 x 1408 65 and 58 (down).  From 128 to 255 gate+up workgroups two slices:
// 16 x 8 x 2 x 7168 x 2048 80 and 67, 64 x 8 x 2 x 7168 x 2048 104 and 83, 24 x 8 x 2 x 4096 x 2048 55 and
// 49, 64 x 16 x 4 x 2048 x 1024 45.5 and 43.6, but with short rows and two workgroups per CU (up to 16
// tokens) 8 x 16 x 6 x 2048 x 1408 34.9 and 38.4.
inline int gate_up_slices(int T, int top_k, int E, int H, int I) {
  const int wgs = max_experts(T, top_k, E) * (I / 128), KB = H / 128;
  if (wgs >= 256 || KB < 16 || (wgs >= 128 && KB < 32 && T <= kTile)) return 1;
  int n = wgs >= 128 ? 2 : 256 / wgs;
  if (n > KB / 4) n = KB / 4;
  return n > 16 ? 16 : n;
}
inline bool down_wide(int H) { return H / 32 >= 160; }
inline int down_slices(int T, int top_k, int E, int H, int I) {
  const int wgs = H / (down_wide(H) ? 32 : 16), units = max_experts(T, top_k, E) * (I / 128);
  if (wgs > 128 || units < 8 * 12) return 1;
  int n = 256 / wgs;
  if (n > units / (8 * 4)) n = units / (8 * 4);
  return n > 16 ? 16 : n;
}
// Late quantization where its 64-column workgroups occupy the CUs, or slicing gains little (1 token, 64
// experts, top 8, 2048 x 1024: 128 workgroups 22.2 us, 4 slices 24.0; 8 experts, top 2, 4096 x 512: 16
// workgroups 20.8 us, 8 slices 16.2).
inline bool use_late(int T, int top_k, int E, int H, int I) {
  return late_quant(T, top_k, E, H, I) &&
         (max_experts(T, top_k, E) * (I / 64) >= 96 || gate_up_slices(T, top_k, E, H, I) < 4);
}

// Tiles of 16 rows: with the prep launch they are packed (sum over experts of ceil(rows / 16) <=
// (pairs + 15 experts) / 16), without it every routed expert has room for all tokens.
inline int expert_tiles(int T) { return (T + kTile - 1) / kTile; }
inline int max_tiles(int T, int top_k, int E, int H) {
  const int n = max_experts(T, top_k, E);
  return fused_prep(T, H) ? n * expert_tiles(T) : T * top_k / kTile + n;
}

// Late quantization: LDS of the down launch behind the waves' sums.  A segment is the K-blocks of one expert
// that a wave takes at a time, at most 64.  All waves' codes, [wave][K-block][T][128] bytes, then their
// scales, [wave][K-block][T] floats: 16-byte accesses to the codes lie on 16-byte boundaries whatever T and I.
constexpr int late_segment(int I) { return I / 128 < 64 ? I / 128 : 64; }
constexpr int late_codes_at(int wave, int seg, int T) { return wave * seg * T * 128; }
constexpr int late_scales_at(int wave, int seg, int T) { return (kDownWaves * 128 + wave * 4) * seg * T; }
constexpr int late_bytes(int seg, int T) { return kDownWaves * seg * T * (128 + 4); }

}  // namespace fgb
