// Mixture-of-experts layer: the router's choice, the combination of a token's experts, and the
// launch rules of the expert products (w4_moe_impl.h).
#include <algorithm>

#include "w4_moe.h"

namespace w4 {
namespace {

// Router: the top_k largest of a token's expert logits and their softmax weights.  One wave per
// token, expert i in lane i % 64, register i / 64.  A logit becomes an unsigned key that orders
// like it (-0 as +0), 0 for one that is never chosen (NaN, -inf); a round takes the largest key
// (maximum over the wave) of the lowest expert (first register, first lane of a ballot).  The
// weights are exp(v - max) over their sum, in fp32; a logit of +inf counts as its maximum's equal.
// Bound by latency: one wave's chain of top_k reductions.  Measured on MI355X: top 8 of 64, 1 token 3.7 us; of
// 256, 4096 tokens 8.0 us (2.4 MB: 0.3 TB/s).
template <int TYPE>
__device__ inline float load_logit(const void* p, size_t i) {
  if constexpr (TYPE == W4_LOGITS_F32) return reinterpret_cast<const float*>(p)[i];
  if constexpr (TYPE == W4_LOGITS_F16) return (float)reinterpret_cast<const _Float16*>(p)[i];
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

__device__ inline uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, off);
    v = o > v ? o : v;
  }
  return v;
}

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
  return v;
}

__device__ inline float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

__device__ inline float exp_from(float v, float top) { return v == top ? 1.0f : expf(v - top); }

template <int TYPE, int NV>
__global__ void __launch_bounds__(256) route_kernel(const void* __restrict__ logits, uint32_t tokens,
                                                    uint32_t experts, uint32_t top_k, int renormalize,
                                                    int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const uint32_t t = blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
  if (t >= tokens) return;
  uint32_t key[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t i = (uint32_t)lane + 64u * j;
    key[j] = 0;
    if (i < experts) {
      const float v = load_logit<TYPE>(logits, (size_t)t * experts + i) + 0.0f;
      const uint32_t u = __float_as_uint(v);
      const bool never = v != v || u == 0xFF800000u;
      key[j] = never ? 0u : u & 0x80000000u ? ~u : u ^ 0x80000000u;
    }
  }
  float all = 0.0f, top = 0.0f, mine = 0.0f;
  int mine_id = -1;
  float chosen = 0.0f;
  for (uint32_t r = 0; r < top_k; ++r) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) best = key[j] > best ? key[j] : best;
    best = wave_max(best);
    if (best == 0) break;  // nothing left to choose: the remaining slots stay absent
    if (r == 0) {
      top = key_value(best);
      if (!renormalize) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (key[j] != 0) all += exp_from(key_value(key[j]), top);
        all = wave_sum(all);
      }
    }
    int id = -1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint64_t mask = __ballot(key[j] == best);
      if (id < 0 && mask != 0) {
        const int at = __builtin_ctzll(mask);
        id = 64 * j + at;
        if (lane == at) key[j] = 0;
      }
    }
    const float w = exp_from(key_value(best), top);
    chosen += w;
    if ((uint32_t)lane == r) {
      mine = w;
      mine_id = id;
    }
  }
  if ((uint32_t)lane < top_k) {
    const float sum = renormalize ? chosen : all;
    ids[(size_t)t * top_k + lane] = mine_id;
    weights[(size_t)t * top_k + lane] = mine_id < 0 ? 0.0f : mine / sum;
  }
}

template <int TYPE>
hipError_t route_slice(const void* logits, uint32_t tokens, uint32_t experts, uint32_t top_k,
                       int renorm, int32_t* ids, float* weights, hipStream_t s) {
  const uint32_t waves = tokens < 4 ? tokens : 4;
  const dim3 grid((tokens + waves - 1) / waves), block(64 * waves);
#define W4_ROUTE(NV)                                                                              \
  if (experts <= 64 * NV) {                                                                       \
    hipLaunchKernelGGL((route_kernel<TYPE, NV>), grid, block, 0, s, logits, tokens, experts, top_k, \
                       renorm, ids, weights);                                                     \
    return hipGetLastError();                                                                     \
  }
  W4_ROUTE(1)
  W4_ROUTE(2)
  W4_ROUTE(4)
  W4_ROUTE(8)
  W4_ROUTE(16)
#undef W4_ROUTE
  return hipErrorInvalidValue;
}

// A launch's threads, 64 a token, have to number fewer than 2^32: slices of 2^25 tokens.
template <int TYPE>
hipError_t route_type(const void* logits, uint32_t tokens, uint32_t experts, uint32_t top_k,
                      int renorm, int32_t* ids, float* weights, hipStream_t s) {
  constexpr uint32_t kSlice = 1u << 25;
  constexpr size_t kBytes = TYPE == W4_LOGITS_F32 ? 4 : 2;
  for (uint32_t t = 0; t < tokens; t += kSlice) {
    const hipError_t e = route_slice<TYPE>(reinterpret_cast<const char*>(logits) + (size_t)t * experts * kBytes,
                                           std::min(kSlice, tokens - t), experts, top_k, renorm,
                                           ids + (size_t)t * top_k, weights + (size_t)t * top_k, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// y[t] = sum over slots j, in order, of weights[t, j] * part[t * top_k + j]; absent slots add
// nothing (their rows of `part` were never written), a token without experts gets zeros.  Bound by the
// latency of one load after another, so a thread has four slots' loads in flight.
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ part,
                                                      const int32_t* __restrict__ ids,
                                                      const float* __restrict__ weights, uint32_t hidden,
                                                      uint32_t experts, uint32_t top_k,
                                                      float* __restrict__ y) {
  const uint32_t t = blockIdx.y;
  const uint32_t n = blockIdx.x * 256 + threadIdx.x;
  if (n >= hidden) return;
  float v = 0.0f;
  // four slots' loads together; what an absent slot's row holds is loaded too, and left out
  for (uint32_t j0 = 0; j0 < top_k; j0 += 4) {
    float x[4], w[4];
    bool have[4];
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t p = t * top_k + min(j0 + i, top_k - 1u);
      x[i] = part[(size_t)p * hidden + n];
      w[i] = weights[p];
      have[i] = j0 + i < top_k && (uint32_t)ids[p] < experts;
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) v = have[i] ? __builtin_fmaf(w[i], x[i], v) : v;
  }
  y[(size_t)t * hidden + n] = v;
}

// Pairs sorted by expert, in pair order: workgroup e counts the valid ids below e and writes the pairs of
// e behind them, start[e] being their number.  Batches of 1024 ids, one a thread; ranks by ballots.
constexpr uint32_t kOrderThreads = 1024;

__global__ void __launch_bounds__(kOrderThreads) order_kernel(const int32_t* __restrict__ ids, uint32_t pairs,
                                                              uint32_t experts, int32_t* __restrict__ order,
                                                              int32_t* __restrict__ start) {
  __shared__ uint32_t below_s[16], match_s[2][16];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  const int e = (int)blockIdx.x;  // e == experts: the number of valid pairs alone
  uint32_t below = 0;
  for (uint32_t i = tid; i < pairs; i += kOrderThreads) {
    const int id = ids[i];
    below += id >= 0 && id < e ? 1u : 0u;
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) below += (uint32_t)__shfl_xor((int)below, off);
  if (lane == 0) below_s[wave] = below;
  __syncthreads();
  uint32_t at = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) at += below_s[w];
  if (tid == 0) start[e] = (int32_t)at;
  if ((uint32_t)e == experts) return;
  uint32_t flip = 0;
  for (uint32_t base = 0; base < pairs; base += kOrderThreads, flip ^= 1u) {
    const uint32_t i = base + tid;
    const bool match = i < pairs && ids[i] == e;
    const uint64_t mask = __ballot(match);
    if (lane == 0) match_s[flip][wave] = (uint32_t)__builtin_popcountll(mask);
    __syncthreads();  // (the other buffer is read no more when it is written again)
    uint32_t before = 0, all = 0;
#pragma unroll
    for (uint32_t w = 0; w < 16; ++w) {
      const uint32_t c = match_s[flip][w];
      before += w < wave ? c : 0u;
      all += c;
    }
    if (match)
      order[at + before + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                    __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] = (int32_t)i;
    at += all;
  }
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Workgroups of an expert (MoeArgs::grid): as many as give the experts two per CU together, what fits;
// each then walks the expert's tile groups with its loads running ahead and one window of activations.
// Measured on MI355X (32 tokens, 8 of 128 experts, 2048 x 768, MXFP4): 4 workgroups of each expert
// and direction 83.5 us, one per tile group 92.
// K groups: the fewest whose workgroups give every CU two, at most one per quad, and two quads of
// `rows` window rows for each inside the largest window.
int moe_kw(int64_t tiles, int64_t experts, int64_t k, int64_t rows) {
  const int64_t quads = (k + 255) / 256;
  int kw = 1;
  while (kw < 4 && 2 * kw <= quads && rows * 1024 * 2 * kw <= kMoeMaxWindow &&
         (tiles + 8 / kw - 1) / (8 / kw) * experts < 2 * device_cu_count())
    kw *= 2;
  return kw;
}

// Quads, window and chunk of a product over K with kw K groups: `cols` pairs a chunk of `planes`
// rows each, and as many quads a window as fit kWindowBytes: all of K if it fits, else an even number of
// quads of each K group (the loop takes two at a time), so that evening out the windows cannot pass what fits.
// Two quads of each always do: moe_kw leaves room for them in kMoeMaxWindow.
constexpr int64_t kWindowBytes = 65536;

MoeProduct moe_window(int64_t k, int kw, uint32_t cols, uint32_t planes) {
  const int64_t qpk = ((k + 255) / 256 + kw - 1) / kw;
  const int64_t rows = (int64_t)cols * planes;
  const int64_t fit = kWindowBytes / (rows * 512 * kw);
  int64_t per = qpk;
  if (per > fit) {
    const int64_t most = std::max<int64_t>(2, fit / 2 * 2);
    const int64_t windows = (qpk + most - 1) / most;
    per = ((qpk + windows - 1) / windows + 1) / 2 * 2;
  }
  MoeProduct p;
  p.kw = kw;
  p.cols = cols;
  p.qpk = (uint32_t)qpk;
  p.qpw = (uint32_t)(per * kw);
  p.win_bytes = (uint32_t)rows * p.qpw * 512u;
  return p;
}

}  // namespace

hipError_t launch_moe_route(const void* logits, int type, int64_t tokens, int64_t experts, int64_t top_k,
                            bool renormalize, int32_t* ids, float* weights, hipStream_t s) {
  const uint32_t t = (uint32_t)tokens, e = (uint32_t)experts, k = (uint32_t)top_k;
  switch (type) {
    case W4_LOGITS_F32: return route_type<W4_LOGITS_F32>(logits, t, e, k, renormalize, ids, weights, s);
    case W4_LOGITS_F16: return route_type<W4_LOGITS_F16>(logits, t, e, k, renormalize, ids, weights, s);
    case W4_LOGITS_BF16: return route_type<W4_LOGITS_BF16>(logits, t, e, k, renormalize, ids, weights, s);
  }
  return hipErrorInvalidValue;
}

// Many tokens: from three pairs an expert on where the experts fill the card without K groups (down: a workgroup has
// 128 rows).  Measured on MI355X against the kernels with K groups (us for the layer): 8 of 128 experts, 2048 x 768,
// MXFP4, at 2 / 4 / 8 / 16 pairs an expert 95 / 99 / 104 / 130 against 83 / 109 / 140 / 239; 1 of 32, 2048 x 2048,
// FP4, 68 / 72 / 74 / 93 against 58 / 68 / 78 / 140.
// Else from eight pairs on: 2 of 8, 1024 x 768, FP4, at 6 / 8 / 12 / 16 pairs 21 / 21 / 22 / 24 against 20 / 22 / 27 /
// 35; 2 of 8, 1536 x 2048, NF4, 45 / 45 / 47 / 48 against 46 / 48 / 68 / 83; 4 of 16, 1024 x 512, INT4, 21 / 21 / 21 /
// 24 against 19 / 20 / 27 / 33.  With fewer than eight experts the sorted kernels have too few workgroups for longer,
// and start at 14: at 8 / 12 / 14 / 16 / 20 pairs one expert of 2048 x 4096, INT4, 50 / 50 / 50 / 50 / 53 against 35 /
// 40 / 54 / 56 / 91; one of 4096 x 1408, MXFP4, 39 / 39 / 40 / 40 / 45 against 25 / 29 / 32 / 34 / 52; 1 of 2, 4096 x
// 2048, NF4, 61 / 63 / 65 / 66 / 66 against 40 / 53 / 63 / 73 / 76; 2 of 4, 2048 x 2048, NF4, 48 / 48 / 48 / 50 / 51
// against 44 / 48 / 50 / 74 / 82.
static bool moe_wide(int64_t pairs, int64_t experts, int64_t hidden) {
  const bool fills = 4 * (hidden / 128) * experts >= 3 * device_cu_count();
  return pairs >= (fills ? 3 : experts < 8 ? 14 : 8) * experts;
}

// The planes of h (three bf16 values per pair and row), the partial results, the sorted pairs and the
// experts' first positions among them.
size_t moe_workspace(int64_t pairs, int64_t hidden, int64_t inter, int64_t experts) {
  return align256((size_t)pairs * (size_t)inter * 6) + align256((size_t)pairs * (size_t)hidden * 4) +
         align256((size_t)pairs * 4) + ((size_t)experts + 1) * 4;
}

// Fewer pairs than experts: a wave per pair in both launches, the second combining.  Measured on MI355X
// against the shared products and their third launch (us): 8 of 128 experts, 2048 x 768, MXFP4, at 2 / 4 /
// 8 / 12 / 16 / 32 tokens 18 / 27 / 48 / 63 / 78 / 140 against 54 / 60 / 64 / 66 / 75 / 83; 4 of 64, 1536 x 1408,
// INT4, at 4 / 8 / 12 / 16 tokens 23 / 34 / 49 / 60 against 54 / 55 / 58 / 59.
// One slot a token pays up to half as many pairs as experts: 1 of 32, 2048 x 2048, FP4, at 12 / 16 / 24 tokens
// 33 / 42 / 60 against 38 / 43 / 44; 1 of 64, 1024 x 1024, INT4, at 24 / 32 / 48 26 / 33 / 46 against 30 / 31 / 32.
static bool moe_per_pair(int64_t tokens, int64_t experts, int64_t top_k) {
  const int64_t pairs = tokens * top_k;
  return tokens == 1 || (pairs < experts && (top_k > 1 || 2 * pairs <= experts));
}

bool plan_moe(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int64_t top_k, MoePlan* out) {
  const int64_t pairs = tokens * top_k;
  MoePlan p{};
  if (moe_per_pair(tokens, experts, top_k)) {
    p.kind = kMoePerPair;
    const int least = top_k > 4 ? 1 : top_k > 2 ? 2 : top_k > 1 ? 4 : 8;  // no wave without a slot ...
    // ... or without a quad (1 token, 2 of 8, 512 x 256, NF4: 9.2 against 10.2); up: then K ranges until the waves
    // number two per SIMD
    const int64_t units = inter / 16 * pairs;
    int kw = least;
    while (kw > 1 && kw > (hidden + 255) / 256) kw /= 2;
    while (kw < 8 && 2 * kw <= (hidden + 255) / 256 && units * kw < 8 * device_cu_count()) kw *= 2;
    p.up.kw = kw;
    p.up.qpk = (uint32_t)(((hidden + 255) / 256 + kw - 1) / kw);
    kw = least;
    while (kw > 1 && kw > (inter + 255) / 256) kw /= 2;
    p.down.kw = kw;
    p.down.qpk = (uint32_t)(((inter + 255) / 256 + kw - 1) / kw);
  } else if (moe_wide(pairs, experts, hidden)) {
    p.kind = kMoeSorted;
  } else {
    p.kind = kMoeShared;
    uint32_t cols = (uint32_t)std::min<int64_t>(16, tokens);
    p.up = moe_window(hidden, moe_kw(inter / 8, experts, hidden, cols), cols, 1);
    p.tiles = pairs <= 2 * experts ? 1 : 3;
    cols = (uint32_t)std::min<int64_t>(p.tiles == 1 ? kMoePacked : 16, tokens);
    p.down = moe_window(inter, moe_kw(hidden / 16, experts, inter, 3 * cols), cols, 3);
    if (p.up.win_bytes > kMoeMaxWindow || p.down.win_bytes > kMoeMaxWindow) return false;
  }
  *out = p;
  return true;
}

hipError_t launch_moe(int fmt, const MoePlan& plan, const uint16_t* x, const int32_t* ids, const float* weights,
                      const uint8_t* gate_up, const void* gate_up_scales, const uint8_t* down,
                      const void* down_scales, int64_t tokens, int64_t hidden, int64_t inter,
                      int64_t experts, int64_t top_k, float* y, void* ws, hipStream_t s) {
  const int64_t pairs = tokens * top_k;
  const int weight = fmt_weight(fmt);
  MoeArgs a{};
  auto combine = [&]() {
    hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((hidden + 255) / 256), (unsigned)tokens), dim3(256), 0, s,
                       a.part, ids, weights, (uint32_t)hidden, (uint32_t)experts, (uint32_t)top_k, y);
    return hipGetLastError();
  };
  auto set = [&](const MoeProduct& p) {
    a.qpk = p.qpk;
    a.qpw = p.qpw;
    a.cols = p.cols;
    a.win_bytes = p.win_bytes;
  };
  // the second product's operands
  auto turn_down = [&]() {
    a.packed = down;
    a.scales = down_scales;
    a.x = a.h;
    a.n = (uint32_t)hidden;
    a.k = (uint32_t)inter;
    a.tiles = (uint32_t)(hidden / 16);
    set(plan.down);
  };
  a.ids = ids;
  a.h = reinterpret_cast<uint16_t*>(ws);
  a.part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + align256((size_t)pairs * (size_t)inter * 6));
  a.experts = (uint32_t)experts;
  a.pairs = (uint32_t)pairs;
  a.top_k = (uint32_t)top_k;

  a.packed = gate_up;
  a.scales = gate_up_scales;
  a.x = x;
  a.n = (uint32_t)(2 * inter);
  a.k = (uint32_t)hidden;
  a.tiles = (uint32_t)(inter / 8);
  set(plan.up);
  if (plan.kind == kMoePerPair) {
    hipError_t e = fmt_xtype(fmt) == kF16 ? launch_moe_pair_f16(weight, plan.up.kw, a, (uint32_t)tokens, s)
                                          : launch_moe_pair_bf16(weight, plan.up.kw, a, (uint32_t)tokens, s);
    if (e != hipSuccess) return e;
    turn_down();
    a.weights = weights;
    a.y = y;
    return launch_moe_token(weight, plan.down.kw, a, (uint32_t)tokens, s);
  }
  if (plan.kind == kMoeSorted) {
    char* at = reinterpret_cast<char*>(a.part) + align256((size_t)pairs * (size_t)hidden * 4);
    int32_t* order = reinterpret_cast<int32_t*>(at);
    int32_t* start = reinterpret_cast<int32_t*>(at + align256((size_t)pairs * 4));
    hipLaunchKernelGGL(order_kernel, dim3((unsigned)experts + 1), dim3(kOrderThreads), 0, s, ids, (uint32_t)pairs,
                       (uint32_t)experts, order, start);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.order = order;
    a.start = start;
    e = launch_moe_wide_up(weight, fmt_xtype(fmt), a, s);
    if (e != hipSuccess) return e;
    turn_down();
    e = launch_moe_wide_down(weight, a, s);
    if (e != hipSuccess) return e;
    return combine();
  }
  a.grid = (uint32_t)std::max<int64_t>(1, 2 * device_cu_count() / experts);
  hipError_t e = fmt_xtype(fmt) == kF16 ? launch_moe_up_f16(weight, plan.up.kw, a, s)
                                        : launch_moe_up_bf16(weight, plan.up.kw, a, s);
  if (e != hipSuccess) return e;
  turn_down();
  e = launch_moe_down(weight, plan.down.kw, plan.tiles, a, s);
  if (e != hipSuccess) return e;
  return combine();
}

}  // namespace w4
