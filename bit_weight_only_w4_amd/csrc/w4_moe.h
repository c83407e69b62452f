// Internal interface of the mixture-of-experts kernels (w4_moe*.hip).
#pragma once
#include "w4_common.h"

namespace w4 {

// One launch of an expert product.  Up: gate and up rows of one expert on the token rows of x.
// Down: rows of one expert on the rows of h.
struct MoeArgs {
  const uint8_t* packed;   // [E, N, K/2]; up: N = 2 inter, gate rows first
  const void* scales;      // [E, N, scales of K]
  const uint16_t* x;       // up: x [tokens, K]; down: the three planes of h [3, pairs, K]
  const int32_t* order;    // many tokens: the pairs sorted by expert
  const int32_t* start;    // ... and the first position of each expert, [experts + 1]
  const int32_t* ids;      // [pairs], pair = token * top_k + slot; outside [0, experts): absent
  uint16_t* h;             // up: planes of h [3, pairs, inter]
  float* part;             // down: [pairs, N]
  const float* weights;    // down with the combination: [pairs]
  float* y;                // ... and its result [tokens, N]
  uint32_t n;              // rows of one expert matrix
  uint32_t k;
  uint32_t experts;
  uint32_t pairs;
  uint32_t top_k;
  uint32_t tiles;          // row tiles of 16 rows, even; up: gate and up tiles alternate
  uint32_t qpk;            // quads (256 weights) per K group
  uint32_t qpw;            // quads per activation window, a multiple of the K groups
  uint32_t cols;           // pairs of a chunk: at most 16 per column tile (down with one tile: 4)
  uint32_t grid;           // workgroups of an expert, at most one per group of tiles
  uint32_t win_bytes;      // LDS bytes of a window: rows * qpw * 512
};

constexpr int kMoeThreads = 512;   // 8 waves
constexpr uint32_t kMoeMaxWindow = 81920;  // LDS bytes of a window
constexpr int kMoePacked = 4;      // pairs of a down chunk whose three planes share one tile

// kw K groups (1, 2, 4) in a workgroup of 8 / kw row tiles; down also: tiles (1: up to kMoePacked
// pairs a chunk, 3: up to 16, a tile per plane).
hipError_t launch_moe_up_f16(int weight, int kw, const MoeArgs& a, hipStream_t s);
hipError_t launch_moe_up_bf16(int weight, int kw, const MoeArgs& a, hipStream_t s);
hipError_t launch_moe_pair_f16(int weight, int kw, const MoeArgs& a, uint32_t tokens, hipStream_t s);
hipError_t launch_moe_pair_bf16(int weight, int kw, const MoeArgs& a, uint32_t tokens, hipStream_t s);
hipError_t launch_moe_token(int weight, int kw, const MoeArgs& a, uint32_t tokens, hipStream_t s);
hipError_t launch_moe_down(int weight, int kw, int tiles, const MoeArgs& a, hipStream_t s);
// Many tokens (the pairs sorted by expert).
hipError_t launch_moe_wide_up(int weight, int xtype, const MoeArgs& a, hipStream_t s);
hipError_t launch_moe_wide_down(int weight, const MoeArgs& a, hipStream_t s);

// The launches of a layer, chosen on its sizes before the first of them.
enum MoeKind { kMoePerPair = 0, kMoeShared = 1, kMoeSorted = 2 };
struct MoeProduct {  // of the shared products; a wave per pair: kw and qpk alone
  int kw;            // K groups
  uint32_t qpk, qpw, cols, win_bytes;  // as in MoeArgs
};
struct MoePlan {
  int kind;
  int tiles;  // shared products, down: see launch_moe_down
  MoeProduct up, down;
};
// False if a window would not fit LDS.
bool plan_moe(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k, MoePlan* out);

// The layer (arguments as w4_moe, already validated).
hipError_t launch_moe(int fmt, const MoePlan& plan, const uint16_t* x, const int32_t* ids,
                      const float* weights, const uint8_t* gate_up, const void* gate_up_scales,
                      const uint8_t* down, const void* down_scales, int64_t tokens, int64_t hidden, int64_t inter,
                      int64_t experts, int64_t top_k, float* y, void* ws, hipStream_t s);
size_t moe_workspace(int64_t pairs, int64_t hidden, int64_t inter, int64_t experts);
hipError_t launch_moe_route(const void* logits, int type, int64_t tokens, int64_t experts, int64_t top_k,
                            bool renormalize, int32_t* ids, float* weights, hipStream_t s);

}  // namespace w4
