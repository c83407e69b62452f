// Expert products of many tokens (kernel template): chunks of up to 64 pairs of an expert (down: 32), its
// weights decoded once for all of them.
//
// The products, formats and decoders are those of w4_moe_impl.h.  A wave takes two row tiles (up: the
// gate tile and the up tile of 16 rows of h; down: 32 rows), so that each piece of activations read from
// LDS feeds two MFMAs and no sum has to leave the wave.  A workgroup's four waves share the
// chunk's activations, a quad (256 k; down: half of one) at a time, in two LDS buffers: while one is multiplied,
// the next is in registers on its way into the other, and one barrier a buffer suffices.  Two or three
// workgroups fit a CU, whose waves compute while the others' wait.  (Whole quads in the down product too would
// leave a CU one workgroup with the planes of 32 pairs; halves in the up product: 206 against 178 us for 512
// tokens, 8 of 128 experts, 2048 x 768, MXFP4.)
//   * Integer codes decode as q + 16, and an MFMA with a column of -(16 + z) takes the offset off inside each
//     step, so that sums keep the size of the result's terms.  (Taken off a block at a time, by one MFMA with
//     ones for both tiles, the layer's error at 150 tokens, 1920 x 2432, INT4A, was 1.5e-6 of the largest output
//     against 5.1e-7, for 73 us against 77.)
//   * Down: the three planes of a column are summands of one value, so their MFMAs add to the same
//     sums (a plane as a column tile of its own: 162 against 143 us
//     for 512 tokens, 4 of 64 experts, 1536 x 1408, INT4).
//   * Weights keep to the caches' ordinary policy: several chunks read them (173 against 163 us with the
//     streaming hint).
//   * The pairs come sorted by expert (order_kernel); a chunk's columns are cut to what it has, in
//     tiles of 16.
// Measured on MI355X, 512 tokens, 6 of 64 experts, 1536 x 1408, FP4: up 84 us (315 TFLOP/s), down 93 us
// (142 TFLOP/s of the layer's, 427 with the planes).  Bound by waiting, not by the matrix units: the
// registers of two row tiles in flight leave a SIMD two waves, which do not cover LDS and barrier
// latencies.
#pragma once
#include <algorithm>

#include "w4_moe_impl.h"

namespace w4 {
namespace {

constexpr int kWideWaves = 4, kWideThreads = 64 * kWideWaves;

// acc[r][t] += half H of the quads of both row tiles times the 128 k of the window, whose column tile t is NP
// planes to be added up; see quad_product.
template <int FMT, int XT, int NT, int NP, int ODD, int H>
__device__ __attribute__((always_inline)) inline void wide_product(
    float4_t (&acc)[2][NT], const MoeQuad (&d)[2], const MoeScales<FMT> (&scales)[2], uint32_t jw, uint32_t left,
    const uint8_t* wbase, uint32_t apiece, const uint32_t* tab, int lane) {
  using Sc = MoeScales<FMT>;
  constexpr int KC = is_g128(FMT) ? 128 : 64;  // weights per block
  constexpr int QH = 128 / KC;                 // blocks of a half
  constexpr int STEPS = KC / 32;
  constexpr bool kMX = FMT == kMXFP4;
  constexpr bool kTable = FMT == kNF4;
  constexpr bool kInt = is_g128(FMT);
  constexpr uint32_t SB = FMT == kINT4 || kMX ? 2 : 4;
  constexpr int kDwords = Sc::kPer == 4 ? 2 : 1;               // of scales of a half
  constexpr int kFirst = Sc::kPer == 1 ? 0 : H * kDwords;      // ... among the quad's
  const int m = lane & 15;
  const uint32_t laneoff = (uint32_t)m * 16u;
  const char* tabc = reinterpret_cast<const char*>(tab);
  const int from = (4 * m + (int)(jw >> 1)) * 4;
  // (an opaque copy: the pieces' offsets are recomputed, an operation each, not held across the loop)
  uint32_t ap = apiece;
  asm volatile("" : "+v"(ap));
  uint32_t sw[2][kDwords], wb[2][QH][STEPS];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
#pragma unroll
    for (int i = 0; i < kDwords; ++i)
      sw[r][i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)scales[r].v[ODD * Sc::kPer + kFirst + i]);
    if (left < 256u / KC * SB) {
#pragma unroll
      for (int i = 0; i < kDwords; ++i) {
        const uint32_t at = 4u * (kFirst + i);
        sw[r][i] = at + 4u <= left ? sw[r][i] : at < left ? sw[r][i] & 0xFFFFu : 0u;
      }
    }
    half_steps<FMT, H>(d[r], wb[r]);
  }
#pragma unroll
  for (int c = 0; c < QH; ++c) {
    float4_t dd[2][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) dd[r][t] = float4_t{0.f, 0.f, 0.f, 0.f};
    uint4 zcol[2];
    if constexpr (kInt) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float zn = FMT == kINT4 ? -24.0f : -16.0f - (float)((sw[r][0] >> 16) & 15u);
        const uint32_t h = XT == kF16 ? f16_bits(zn) : (__float_as_uint(zn) >> 16);
        zcol[r] = make_uint4(h | (h << 16), h | (h << 16), h | (h << 16), h | (h << 16));
      }
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      constexpr uint32_t kPieces = KC / 8;  // of a block
      const uint32_t at = (c * kPieces + s * (kMX ? 4u : 1u)) * 16u;
      const uint8_t* xp = wbase + (ap ^ at);
      uint4 xv[NT][NP];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int p = 0; p < NP; ++p) xv[t][p] = *reinterpret_cast<const uint4*>(xp + (t * NP + p) * 4096u);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint4 b1, b2;
        if constexpr (kTable) {
          uint2 tv[4];
#pragma unroll
          for (int kb = 0; kb < 4; ++kb) {
            const uint32_t addr =
                __builtin_amdgcn_perm(wb[r][c][s], laneoff, 0x0C0C0000u | ((4u + (uint32_t)kb) << 8)) >> 1;
            tv[kb] = *reinterpret_cast<const uint2*>(tabc + addr);
          }
          b1 = make_uint4(tv[0].x, tv[1].x, tv[2].x, tv[3].x);
          b2 = make_uint4(tv[0].y, tv[1].y, tv[2].y, tv[3].y);
        } else {
          b1 = decode8<FMT, XT>(wb[r][c][s]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            dd[r][t] = mfma<XT>(xv[t][p], b1, dd[r][t]);
            if constexpr (kTable) dd[r][t] = mfma<XT>(xv[t][p], b2, dd[r][t]);
            if constexpr (kInt) dd[r][t] = mfma<XT>(xv[t][p], zcol[r], dd[r][t]);
          }
      }
      if constexpr (kMX) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float sc =
              ldexpf(__uint_as_float(0x00400000u), (int)((sw[r][0] >> (16 * c + 8 * s)) & 0xFFu));
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf(dd[r][t][i], sc, acc[r][t][i]);
            dd[r][t] = float4_t{0.f, 0.f, 0.f, 0.f};
          }
        }
      }
    }
    if constexpr (!kMX) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float sc = __uint_as_float(FMT == kINT4    ? (H == 0 ? sw[r][0] << 16 : sw[r][0] & 0xFFFF0000u)
                                         : FMT == kINT4A ? sw[r][0] << 16
                                                         : sw[r][c % kDwords]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf(dd[r][t][i], sc, acc[r][t][i]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int DIR, int FMT, int XT, int NT>
struct MoeWide {
  static constexpr int KC = is_g128(FMT) ? 128 : 64;
  static constexpr uint32_t QC = 256 / KC;
  static constexpr uint32_t SB = FMT == kINT4 || FMT == kMXFP4 ? 2 : 4;
  static constexpr int NP = DIR == kUp ? 1 : 3;              // planes
  static constexpr uint32_t kBuffer = NT * NP * 16u * 256u;  // bytes of half a quad in LDS
  static constexpr uint32_t kHalves = DIR == kUp ? 2 : 1;    // halves of a buffer, and of a barrier
  static constexpr uint32_t kPieces = NT * NP;               // of a thread
  static_assert(kWideThreads == 16 * 16, "a thread takes one piece of each 16 window rows");

  // 32 rows a wave (unit `unit`) of expert e, on the chunk's pairs: `list` holds them in lanes, `have` of
  // them.  odd_sum becomes NaN if a sum of this lane's is not finite.
  static __device__ __attribute__((always_inline)) inline void run(const MoeArgs& a, int e, uint32_t unit, int list,
                                                                   uint32_t have, uint8_t* smem, const uint32_t* tab,
                                                                   float& odd_sum) {
    using Sc = MoeScales<FMT>;
    const int tid = threadIdx.x, lane = tid & 63;
    const int g = lane >> 4, m = lane & 15;
    const uint32_t units = a.tiles / 2;
    const uint32_t pitch = a.k >> 1, nblocks = a.k / KC, spitch = nblocks * SB, nchunks = a.k >> 5;
    const uint32_t nq = (a.k + 255u) / 256u;
    const bool live = unit < units;
    __amdgpu_buffer_rsrc_t rw[2], rs[2];
    uint32_t row0[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      row0[r] = DIR == kUp ? (r ? a.n >> 1 : 0u) + unit * 16u : unit * 32u + 16u * r;
      const size_t row = (size_t)e * a.n + (live ? row0[r] : 0u);
      rw[r] = make_rsrc(reinterpret_cast<const char*>(a.packed) + row * pitch, live ? 16u * pitch : 0u);
      rs[r] = make_rsrc(reinterpret_cast<const char*>(a.scales) + row * spitch, live ? 16u * spitch : 0u);
    }
    const uint32_t chunk = (uint32_t)g + 4u * (uint32_t)(m >> 3);
    const uint32_t wlane = (uint32_t)(m & 7) * pitch + chunk * 16u;
    auto load_quad = [&](uint32_t q, MoeQuad (&d)[2]) __attribute__((always_inline)) {
      const bool in = q * 8 + chunk < nchunks;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 v0 = buffer_load16(rw[r], offset_or_oob(in, wlane + q * 128u));
        const uint4 v1 = buffer_load16(rw[r], offset_or_oob(in, wlane + q * 128u + 8u * pitch));
        d[r].w[0][0] = v0.x; d[r].w[0][1] = v0.y; d[r].w[0][2] = v0.z; d[r].w[0][3] = v0.w;
        d[r].w[1][0] = v1.x; d[r].w[1][1] = v1.y; d[r].w[1][2] = v1.z; d[r].w[1][3] = v1.w;
      }
    };
    auto load_scales = [&](uint32_t q, Sc (&d)[2]) __attribute__((always_inline)) {
      const uint32_t at = (uint32_t)(lane >> 2) * spitch + (q + 2u * (uint32_t)(lane & 3)) * (QC * SB);
      const uint32_t off = offset_or_oob(q * QC < nblocks, at & ~3u);
#pragma unroll
      for (int r = 0; r < 2; ++r) load_scale_window<FMT>(d[r], rs[r], off);
    };
    const uint32_t sshift = ((uint32_t)(lane >> 2) * spitch & 2u) * 8u;

    // Activations: piece s of a thread belongs to window row 16 s + tid / 16, at position tid % 16.  Rows
    // without a pair read as zeros.
    const __amdgpu_buffer_rsrc_t rx =
        make_rsrc(a.x, (DIR == kUp ? a.pairs / a.top_k : 3u * a.pairs) * a.k * 2u);
    const uint32_t wrow = (uint32_t)tid >> 4, slot = (uint32_t)tid & 15u;
    const uint32_t xpiece = slot ^ wrow;  // in the half quad
    uint32_t xoff[kPieces];
#pragma unroll
    for (uint32_t s = 0; s < kPieces; ++s) {
      const uint32_t col = s / NP * 16u + wrow, plane = s % NP;
      const uint32_t p = (uint32_t)__shfl(list, (int)col);
      const uint32_t base = (DIR == kUp ? p / a.top_k : plane * a.pairs + p) * a.k * 2u;
      xoff[s] = offset_or_oob(col < have, base + xpiece * 16u);
    }
    uint4 xv[kHalves][kPieces];
    auto load_x = [&](uint32_t u) __attribute__((always_inline)) {  // buffer u's halves
#pragma unroll
      for (uint32_t h = 0; h < kHalves; ++h)
#pragma unroll
        for (uint32_t s = 0; s < kPieces; ++s) {
          const uint32_t at = u * kHalves + h;
          // (an offset past the buffer stays past it: the sum does not wrap)
          xv[h][s] = buffer_load16(rx, offset_or_oob(at * 16u + xpiece < a.k >> 3 && xoff[s] != kOutOfRange, xoff[s] + at * 256u));
        }
    };
    auto store_x = [&](uint32_t b) __attribute__((always_inline)) {
#pragma unroll
      for (uint32_t h = 0; h < kHalves; ++h)
#pragma unroll
        for (uint32_t s = 0; s < kPieces; ++s)
          *reinterpret_cast<uint4*>(smem + (b * kHalves + h) * kBuffer + (16u * s + wrow) * 256u + slot * 16u) =
              arranged<FMT>(xv[h][s]);
    };

    const uint32_t piece0 = FMT == kMXFP4 ? g : is_g128(FMT) ? 4 * g : 4 * (g & 1) + 2 * (g >> 1);
    const uint32_t apiece = (piece0 ^ (uint32_t)m) * 16u;
    const uint8_t* arow = smem + (uint32_t)m * 256u;

    float4_t acc[2][NT];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[r][t] = float4_t{0.f, 0.f, 0.f, 0.f};
    MoeQuad W0[2], W1[2];
    Sc held[2], next[2];
    load_x(0);
    load_scales(0, next);
    load_quad(0, W0);
    __syncthreads();  // the buffers (and the table) are free
    store_x(0);
    load_x(1);
    load_quad(1, W1);
    __syncthreads();
    auto half = [&](uint32_t q, MoeQuad (&d)[2], auto odd, auto which) __attribute__((always_inline)) {
      constexpr int ODD = decltype(odd)::value, H = decltype(which)::value;
      constexpr uint32_t B = kHalves == 2 ? ODD : H;  // the buffer multiplied
      const uint32_t u = kHalves == 2 ? q : 2u * q + H;
      if ((kHalves == 1 || H == 0) && u + 1 < 2u / kHalves * nq) {
        store_x(1u - B);
        load_x(u + 2);
      }
      const uint32_t left = (nblocks - q * QC) * SB;
      wide_product<FMT, XT, NT, NP, ODD, H>(acc, d, held, q % Sc::kQuads, left,
                                            arow + (kHalves == 2 ? 2u * B + H : B) * kBuffer, apiece, tab, lane);
      if (H == 1) load_quad(q + 2, d);
      if (kHalves == 1 || H == 1) __syncthreads();
    };
    auto step = [&](uint32_t q, MoeQuad (&d)[2], auto odd) __attribute__((always_inline)) {
      half(q, d, odd, std::integral_constant<int, 0>{});
      half(q, d, odd, std::integral_constant<int, 1>{});
    };
    for (uint32_t q = 0; q < nq; q += 2) {
      if (q % Sc::kQuads == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) place_scales<FMT>(held[r], next[r], sshift);
        load_scales(q + Sc::kQuads, next);
      }
      step(q, W0, std::integral_constant<int, 0>{});
      if (q + 1 < nq) step(q + 1, W1, std::integral_constant<int, 1>{});
    }

    auto finished = [&](float v) __attribute__((always_inline)) {
      if constexpr (FMT == kNF4) v *= 1.0f / kNf4Factor;
      watch(odd_sum, v);
      return v;
    };
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t col = 16u * t + 4u * g + i;
        const uint32_t pair = (uint32_t)__shfl(list, (int)col);
        if (live && col < have) {
          if constexpr (DIR == kUp) {
            const float gate = finished(acc[0][t][i]);
            store_h(a, pair, row0[0] + (uint32_t)m, a.n >> 1, gate, finished(acc[1][t][i]));
          } else {
#pragma unroll
            for (int r = 0; r < 2; ++r)
              a.part[(size_t)pair * a.n + row0[r] + (uint32_t)m] = finished(acc[r][t][i]);
          }
        }
      }
  }
};

// grid (groups of 4 units, experts, chunks at a time)
template <int DIR, int FMT, int XT, int NT>
__global__ void __launch_bounds__(kWideThreads, DIR == kUp && NT == 1 ? 3 : 2) moe_wide_kernel(MoeArgs a) {
  constexpr bool kTable = FMT == kNF4;
  constexpr uint32_t kCols = 16 * NT;
  __shared__ __align__(16) uint32_t tab[kTable ? kTableBytes / 4 : 4];
  extern __shared__ __align__(16) uint8_t smem[];
  const int e = (int)blockIdx.y;
  const uint32_t first = (uint32_t)a.start[e], count = (uint32_t)a.start[e + 1] - first;
  if (blockIdx.z * kCols >= count) return;
  if constexpr (kTable) fill_moe_table<XT, kWideThreads>(tab);
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t unit = blockIdx.x * kWideWaves + (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  float odd_sum = 0.0f;
  for (uint32_t c0 = blockIdx.z * kCols; c0 < count; c0 += gridDim.z * kCols) {
    const uint32_t have = min(kCols, count - c0);
    const int list = lane < have ? a.order[first + c0 + lane] : 0;
    if (NT > 3 && have > 48) {
      MoeWide<DIR, FMT, XT, NT>::run(a, e, unit, list, have, smem, tab, odd_sum);
    } else if (NT > 2 && have > 32) {
      MoeWide<DIR, FMT, XT, NT < 3 ? NT : 3>::run(a, e, unit, list, have, smem, tab, odd_sum);
    } else if (NT > 1 && have > 16) {
      MoeWide<DIR, FMT, XT, NT < 2 ? NT : 2>::run(a, e, unit, list, have, smem, tab, odd_sum);
    } else {
      MoeWide<DIR, FMT, XT, 1>::run(a, e, unit, list, have, smem, tab, odd_sum);
    }
  }
  if (__any(odd_sum != odd_sum)) {  // this wave's results once more, each by the lane that stored it
    const MoeArgs b = args_again();
    const uint32_t base = (uint32_t)b.start[blockIdx.y], pairs = (uint32_t)b.start[blockIdx.y + 1] - base;
    const uint32_t u = blockIdx.x * kWideWaves + (threadIdx.x >> 6), m = threadIdx.x & 15u;
    if (u < b.tiles / 2) {
#pragma unroll 1
      for (uint32_t c0 = blockIdx.z * kCols; c0 < pairs; c0 += gridDim.z * kCols) {
#pragma unroll 1
        for (uint32_t i = 0; i < 4u * NT; ++i) {
          const uint32_t col = c0 + 16u * (i >> 2) + 4u * ((threadIdx.x & 63u) >> 4) + (i & 3u);
          if (col >= pairs) continue;
          const uint32_t pair = (uint32_t)b.order[base + col];
          if constexpr (DIR == kUp) {
            settle_h<FMT, XT>(b, (int)blockIdx.y, pair, u * 16u + m);
          } else {
#pragma unroll 1
            for (uint32_t r = 0; r < 2; ++r) settle_part<FMT>(b, (int)blockIdx.y, pair, u * 32u + 16u * r + m);
          }
        }
      }
    }
  }
}

template <int DIR, int FMT, int XT, int NT>
hipError_t launch_moe_wide_one(const MoeArgs& a, hipStream_t s) {
  constexpr int kLds = 2 * MoeWide<DIR, FMT, XT, NT>::kHalves * MoeWide<DIR, FMT, XT, NT>::kBuffer;
  static const hipError_t raised =
      hipFuncSetAttribute(reinterpret_cast<const void*>(&moe_wide_kernel<DIR, FMT, XT, NT>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (raised != hipSuccess) return raised;
  const uint32_t groups = (a.tiles / 2 + kWideWaves - 1) / kWideWaves;
  // Chunks side by side until every CU has two workgroups, at most one more than an average expert has:
  // 16 tokens an expert of four, 2048 x 2048, NF4, 69 us without and 50 with.
  constexpr uint32_t kCols = 16 * NT;
  const uint32_t chunks = (a.pairs / a.experts + kCols - 1) / kCols + 1u;
  const uint32_t fill = (uint32_t)(2 * device_cu_count()) / (groups * a.experts);
  const uint32_t z = std::max(1u, std::min(chunks, fill));
  hipLaunchKernelGGL((moe_wide_kernel<DIR, FMT, XT, NT>), dim3(groups, a.experts, z), dim3(kWideThreads), kLds, s, a);
  return hipGetLastError();
}

// Up: 16 columns a chunk, three workgroups to a CU, up to 12 pairs an expert, else up to 64.  Measured on
// MI355X (us for the layer with 16 pairs a down chunk, 16 columns against 64): 8 of 128 experts, 2048 x 768, MXFP4, at 4 / 8 / 16 / 32
// pairs an expert 110 / 110 / 161 / 244 against 114 / 113 / 152 / 200; 4 of 64, 1536 x 1408, INT4, 77 / 83 /
// 123 / 190 against 82 / 86 / 112 / 155.  NF4, whose table takes 32 KiB: 32 columns always.
// Down: 16 pairs a chunk up to 12 pairs an expert, or where chunks of 32 would leave CUs without one; else
// 32.  Measured (16 against 32): 6 of 64, 1536 x 1408, FP4, at 24 / 48 pairs an expert 138 / 201 against 124 /
// 177; 8 of 128, 2048 x 768, MXFP4, at 16 / 32 pairs 152 / 200 against 132 / 178; 2 of 8, 1536 x 2048, NF4,
// at 16 / 32 / 64 / 128 pairs 48 / 57 / 72 / 115 against 56 / 59 / 75 / 104.
template <int DIR, int FMT, int XT>
hipError_t launch_moe_wide_cols(const MoeArgs& a, hipStream_t s) {
  if constexpr (DIR == kDown) {
    const bool fills = (uint64_t)(a.pairs / 32u) * (a.n / 128u) >= (uint64_t)device_cu_count();
    return a.pairs > 12u * a.experts && fills ? launch_moe_wide_one<DIR, FMT, XT, 2>(a, s)
                                              : launch_moe_wide_one<DIR, FMT, XT, 1>(a, s);
  } else if constexpr (FMT == kNF4) {
    return launch_moe_wide_one<DIR, FMT, XT, 2>(a, s);
  } else {
    return a.pairs <= 12u * a.experts ? launch_moe_wide_one<DIR, FMT, XT, 1>(a, s)
                                      : launch_moe_wide_one<DIR, FMT, XT, 4>(a, s);
  }
}

template <int DIR, int XT>
hipError_t launch_moe_wide_weight(int weight, const MoeArgs& a, hipStream_t s) {
  switch (weight) {
    case kNF4: return launch_moe_wide_cols<DIR, kNF4, XT>(a, s);
    case kINT4: return launch_moe_wide_cols<DIR, kINT4, XT>(a, s);
    case kFP4: return launch_moe_wide_cols<DIR, kFP4, XT>(a, s);
    case kINT4A: return launch_moe_wide_cols<DIR, kINT4A, XT>(a, s);
    case kMXFP4: return launch_moe_wide_cols<DIR, kMXFP4, XT>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace w4
