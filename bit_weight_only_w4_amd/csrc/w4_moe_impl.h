// Expert products of the mixture-of-experts layer on the matrix cores (kernel template; one
// translation unit per direction and activation type instantiates it).
//
// The layer: y[t] = sum_j w[t, j] Down_e h[t, j], h[t, j] = silu(Gate_e x[t]) (Up_e x[t]),
// e = ids[t, j], with silu(v) = v / (1 + exp(-v)).  A (token, slot) pair is a column of its expert's
// products; the up kernel writes h for every pair, the down kernel one row of partial results per
// pair, and the combine kernel adds a token's pairs in slot order, scaled by their routing weights.
//
// Which experts are in use is known on the device alone.  grid.y gives each possible expert in use
// a slot: with fewer pairs than experts slot s is pair s, whose workgroups take all pairs of the
// pair's expert if no earlier pair has it (and end otherwise); else slot s is expert s.  Every wave finds
// its expert's pairs itself, 64 ids at a time (a ballot, and a lane permutation that hands the r-th
// pair to lane r): no launch, memory or barrier for a sorted list.
//
// Inside a workgroup 8 waves are RW row units x KW K groups.  A unit is two 16-row tiles that share
// every activation fragment: a gate tile and its up tile (the product silu(g) u then needs no
// exchange), or two adjacent row tiles of the down matrix.  A wave streams its unit's quads (256
// weights of each row, two 16-byte loads per lane and tile, whole 128-byte lines) and activations
// into one of two register sets while it multiplies the other:
//   * v_mfma_f32_16x16x32, A = 16 weight rows x 32 k, B = 32 k x 16 columns, the k order inside a
//     block permuted alike on both sides (see load_quad); fp32 accumulation per scale block, then
//     acc += scale[row] * D.
//   * Weight codes are exact 16-bit values (E2M1 through the hardware conversion; q - 8 through a
//     byte -> pair LDS table, asymmetric INT4 with one more MFMA whose rows hold -(z - 8)).  NF4's codes
//     are not: they are held as two 16-bit terms, after a factor of 1.4376 (taken off the sums)
//     that leaves the two bf16 terms an rms error of 4.2e-7 over normal weights (2.5e-6 without it).
//   * h has fp32's 24 bits as three bf16 planes (the value cut after 8 bits, then the rest, then
//     what is left), which keeps bf16's range for either activation type.  The planes are
//     columns of the same product: up to five tokens' planes fill one 16-column tile, so keeping
//     24 bits costs a few tokens nothing; from six tokens on a plane is a column tile of its own.
#pragma once
#include "w4_mfma_common.h"
#include "w4_moe.h"

namespace w4 {
namespace {

constexpr int kUp = 0, kDown = 1;
constexpr float kNf4Factor = 1.4376f;

// Byte -> decoded pair table: 32 copies of each 4-byte entry, or 16 of each 8-byte NF4 entry
// (first terms, second terms), 128 bytes per entry.
template <int FMT, int XT>
__device__ inline void fill_moe_table(uint32_t* tab) {
  uint32_t v1, v2 = 0;
  if (FMT == kNF4) {
    const float c = __uint_as_float(codes_in_lanes<kNF4>()) * kNf4Factor;
    if (XT == kF16) {
      const _Float16 hi = (_Float16)c;
      v1 = f16_bits((float)hi);
      v2 = f16_bits(c - (float)hi);
    } else {
      v1 = bf16_rne_bits(c);
      v2 = bf16_rne_bits(c - __uint_as_float(v1 << 16));
    }
  } else {
    const float v = (float)((int)(threadIdx.x & 15u) - 8);
    v1 = XT == kF16 ? f16_bits(v) : (__float_as_uint(v) >> 16);
  }
  uint4* t4 = reinterpret_cast<uint4*>(tab);
  const int tid = threadIdx.x;
  const uint32_t lo1 = (uint32_t)__shfl((int)v1, (tid >> 3) & 15) << 16;
  const uint32_t lo2 = FMT == kNF4 ? (uint32_t)__shfl((int)v2, (tid >> 3) & 15) << 16 : 0u;
#pragma unroll
  for (int j = 0; j < kTableBytes / 16 / kMoeThreads; ++j) {
    const int i = tid + kMoeThreads * j;
    const int hi = __builtin_amdgcn_readfirstlane(i >> 7);
    const uint32_t p1 = (uint32_t)__builtin_amdgcn_readlane((int)v1, hi) | lo1;
    if (FMT == kNF4) {
      const uint32_t p2 = (uint32_t)__builtin_amdgcn_readlane((int)v2, hi) | lo2;
      t4[i] = make_uint4(p1, p2, p1, p2);
    } else {
      t4[i] = make_uint4(p1, p1, p1, p1);
    }
  }
}

// The four E2M1 pairs of a packed dword in memory order (high nibble first) as 16-bit pairs.  The
// conversion returns a byte's low nibble in the low half, so the nibbles are swapped first.
template <int XT>
__device__ inline uint4 e2m1_pairs(uint32_t w) {
  w = ((w >> 4) & 0x0F0F0F0Fu) | ((w << 4) & 0xF0F0F0F0u);
  if constexpr (XT == kF16) {
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3)));
  } else {
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3)));
  }
}

// The pairs of expert e in pair order: returns their number and the first of them, and in lane r
// (r < ncol <= 63) the pair of rank c0 + r, or -1.  Every lane of the wave takes part.
__device__ inline uint32_t scan_pairs(const int32_t* __restrict__ ids, uint32_t pairs, int e,
                                      uint32_t c0, uint32_t ncol, int lane, uint32_t& first, int& mine) {
  uint32_t total = 0;
  first = 0xFFFFFFFFu;
  mine = -1;
  for (uint32_t base = 0; base < pairs; base += 64) {
    const uint32_t i = base + (uint32_t)lane;
    const int id = i < pairs ? ids[i] : -1;
    const bool match = id == e;
    const uint64_t mask = __ballot(match);
    const uint32_t rank = total + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                            __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
    // lanes without a pair of this chunk send to lane 63, which is no column
    const uint32_t to = match && rank >= c0 && rank - c0 < ncol ? rank - c0 : 63u;
    const int got = __builtin_amdgcn_ds_permute((int)(to * 4u), (int)(i + 1u));
    if (lane < (int)ncol && got > 0) mine = got - 1;
    if (first == 0xFFFFFFFFu && mask != 0) first = base + (uint32_t)__builtin_ctzll(mask);
    total += (uint32_t)__builtin_popcountll(mask);
  }
  return total;
}

template <int FMT>
struct MoeQuad {
  static constexpr int QC = is_g128(FMT) ? 2 : 4;  // scale blocks (MXFP4: block pairs) per quad
  uint32_t w[2][2][4];  // [tile][load][dword]
  uint32_t s[2][QC];    // as loaded, for one D row of each tile
};

template <int DIR, int FMT, int XT, int NT, int KW>
__global__ void __launch_bounds__(kMoeThreads, 2) moe_kernel(MoeArgs a) {
  constexpr int RW = 8 / KW;
  constexpr int KC = is_g128(FMT) ? 128 : 64;  // weights per block
  constexpr int QC = 256 / KC;
  constexpr int STEPS = KC / 32;
  constexpr bool kMX = FMT == kMXFP4;
  constexpr bool kTable = FMT != kFP4 && !kMX;
  constexpr bool kSplit = FMT == kNF4;
  constexpr int SB = FMT == kINT4 || kMX ? 2 : 4;
  constexpr uint32_t kCols = DIR == kUp ? 16u * NT : NT == 1 ? (uint32_t)kMoePacked : 16u * (NT / 3);
  __shared__ __align__(16) uint32_t tab[kTable ? kTableBytes / 4 : 4];
  __shared__ float4_t red[KW > 1 ? (KW - 1) * RW * 2 * NT * 64 : 1];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rg = wave % RW, kg = wave / RW;
  const int g = lane >> 4, m = lane & 15;

  // This slot's expert.
  const bool by_pair = a.pairs < a.experts;
  const int e = by_pair ? a.ids[blockIdx.y] : (int)blockIdx.y;
  if ((uint32_t)e >= a.experts) return;

  const uint32_t pitch = a.k >> 1;
  const uint32_t nblocks = a.k / KC;
  const uint32_t spitch = nblocks * SB;
  const uint32_t unit = blockIdx.x * RW + (uint32_t)rg;
  const uint32_t live = unit < a.units ? 16u : 0u;  // a wave past the last unit reads zeros
  const uint32_t row0 = DIR == kUp ? unit * 16u : unit * 32u;
  const uint32_t row1 = DIR == kUp ? (a.n >> 1) + unit * 16u : unit * 32u + 16u;
  __amdgpu_buffer_rsrc_t rw[2], rs[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const size_t row = (size_t)e * a.n + (live ? (r ? row1 : row0) : 0u);
    rw[r] = make_rsrc(a.packed + row * pitch, live * pitch);
    rs[r] = make_rsrc(reinterpret_cast<const char*>(a.scales) + row * spitch, live * spitch);
  }

  // Weight loads of lane (g, m): load h covers rows 8 h .. 8 h + 7 with 8 lanes on the 128 bytes of
  // each row's quad: the lane's own row m when m >> 3 == h, else its partner row m ^ 8; rotating by
  // 8 lanes later gives lane (g, m) chunks g and g + 4 (16 bytes each) of row m.
  const uint32_t chunk0 = m < 8 ? g : g + 4, chunk1 = m < 8 ? g + 4 : g;
  const uint32_t wl0 = (uint32_t)(m & 7) * pitch + chunk0 * 16u;
  const uint32_t wl1 = (uint32_t)(8 + (m & 7)) * pitch + chunk1 * 16u;
  const uint32_t slane = (uint32_t)(4 * g + (m & 3)) * spitch;
  const uint32_t nchunks = a.k >> 5;

  auto load_weights = [&](uint32_t q, bool in, MoeQuad<FMT>& d) __attribute__((always_inline)) {
    const uint32_t qb = q * QC;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint4 v0 = buffer_load16_stream(rw[r], offset_or_oob(in && q * 8 + chunk0 < nchunks, wl0 + q * 128u));
      const uint4 v1 = buffer_load16_stream(rw[r], offset_or_oob(in && q * 8 + chunk1 < nchunks, wl1 + q * 128u));
      d.w[r][0][0] = v0.x; d.w[r][0][1] = v0.y; d.w[r][0][2] = v0.z; d.w[r][0][3] = v0.w;
      d.w[r][1][0] = v1.x; d.w[r][1][1] = v1.y; d.w[r][1][2] = v1.z; d.w[r][1][3] = v1.w;
      if constexpr (!is_g128(FMT) && !kMX) {
        // blocks past K hold the next row's scales here; they are zeroed when used
        const uint4 sv = buffer_load16(rs[r], offset_or_oob(in && qb < nblocks, slane + qb * SB));
        d.s[r][0] = sv.x; d.s[r][1] = sv.y; d.s[r][2] = sv.z; d.s[r][3] = sv.w;
      } else {
#pragma unroll
        for (int c = 0; c < QC; ++c) {
          const uint32_t off = offset_or_oob(in && qb + c < nblocks, slane + (qb + c) * SB);
          d.s[r][c] = FMT == kINT4A ? buffer_load32(rs[r], off) : buffer_load16bit(rs[r], off);
        }
      }
    }
  };

  const uint32_t qpk = a.qpk, q0 = (uint32_t)kg * qpk;
  MoeQuad<FMT> W0, W1;
  load_weights(q0, true, W0);
  load_weights(q0 + 1, 1 < qpk, W1);

  if constexpr (kTable) fill_moe_table<FMT, XT>(tab);
  uint32_t first, count;
  int list;
  count = scan_pairs(a.ids, a.pairs, e, 0, kCols, lane, first, list);
  // without pairs, or another slot has this expert: every wave sees the same count
  if (count == 0 || (by_pair && first != blockIdx.y)) return;
  if constexpr (kTable) __syncthreads();

  const uint32_t laneoff = kSplit ? (uint32_t)(lane & 15) * 16u : (uint32_t)(lane & 31) * 8u;
  const char* tabc = reinterpret_cast<const char*>(tab);
  // k of this lane's first weight of a block's first step, and the step's stride
  const uint32_t klane = kMX ? 8 * g : is_g128(FMT) ? 32 * g : 32 * (g & 1) + 16 * (g >> 1);
  constexpr uint32_t kstep = kMX ? 32 : 8;
  const int zsrc = 16 * (m >> 2) + (m & 3);  // lane holding the scale word of A row m
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(a.cols, (DIR == kUp ? a.pairs / a.top_k : 3u * a.pairs) * a.k * 2u);

  for (uint32_t c0 = 0; c0 < count; c0 += kCols) {
    if (c0 > 0) {
      scan_pairs(a.ids, a.pairs, e, c0, kCols, lane, first, list);
      load_weights(q0, true, W0);
      load_weights(q0 + 1, 1 < qpk, W1);
    }
    // The row of `cols` behind this lane's column of each tile, as a byte offset.
    uint32_t coff[NT];
    bool chave[NT];
    int pair[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if constexpr (DIR == kUp) {
        pair[t] = __shfl(list, 16 * t + m);
        coff[t] = (uint32_t)max(pair[t], 0) / a.top_k * a.k * 2u;
      } else {
        const int plane = NT == 1 ? m / kMoePacked : t % 3;
        pair[t] = __shfl(list, NT == 1 ? m % kMoePacked : 16 * (t / 3) + m);
        if (plane > 2) pair[t] = -1;
        coff[t] = ((uint32_t)plane * a.pairs + (uint32_t)max(pair[t], 0)) * a.k * 2u;
      }
      chave[t] = pair[t] >= 0;
    }
    auto load_cols = [&](uint32_t q, bool in, uint4 (&x)[NT][8]) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int c = 0; c < QC; ++c) {
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const uint32_t kpos = q * 256u + c * KC + klane + s * kstep;
            x[t][c * STEPS + s] = buffer_load16(rx, offset_or_oob(in && chave[t] && kpos < a.k, coff[t] + kpos * 2u));
          }
        }
      }
    };

    float4_t acc[2][NT];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[r][t] = float4_t{0.f, 0.f, 0.f, 0.f};

    auto compute = [&](uint32_t q, const MoeQuad<FMT>& d, const uint4 (&x)[NT][8]) __attribute__((always_inline)) {
      const uint32_t qb = q * QC;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t wh[2][4], wb[QC][STEPS];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t send = m < 8 ? d.w[r][1][i] : d.w[r][0][i];
          wh[0][i] = m < 8 ? d.w[r][0][i] : d.w[r][1][i];
          wh[1][i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)send, 0x128, 0xF, 0xF, false);  // row_ror:8
        }
        if constexpr (is_g128(FMT)) {
#pragma unroll
          for (int c = 0; c < QC; ++c)
#pragma unroll
            for (int s = 0; s < STEPS; ++s) wb[c][s] = wh[c][s];
        } else {
          // 64-weight blocks: chunks 2 c, 2 c + 1 of the half quad to every lane group, two dwords
          // each; MXFP4: one more swap gives step s the dwords of the 32-weight block s.
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const auto s0 = __builtin_amdgcn_permlane32_swap(wh[h][0], wh[h][2], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(wh[h][1], wh[h][3], false, false);
            wb[2 * h][0] = s0[0];
            wb[2 * h][1] = s1[0];
            wb[2 * h + 1][0] = s0[1];
            wb[2 * h + 1][1] = s1[1];
          }
          if constexpr (kMX) {
#pragma unroll
            for (int c = 0; c < QC; ++c) {
              const auto t = __builtin_amdgcn_permlane16_swap(wb[c][0], wb[c][1], false, false);
              wb[c][0] = t[0];
              wb[c][1] = t[1];
            }
          }
        }
#pragma unroll
        for (int c = 0; c < QC; ++c) {
          float4_t dd[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) dd[t] = float4_t{0.f, 0.f, 0.f, 0.f};
          uint4 zrow = make_uint4(0u, 0u, 0u, 0u);
          if constexpr (FMT == kINT4A) {
            const uint32_t word = (uint32_t)__shfl((int)d.s[r][c], zsrc);
            const float zn = (float)(8 - (int)((word >> 16) & 15u));
            const uint32_t h = XT == kF16 ? f16_bits(zn) : (__float_as_uint(zn) >> 16);
            zrow = make_uint4(h | (h << 16), h | (h << 16), h | (h << 16), h | (h << 16));
          }
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            uint4 a1, a2;
            if constexpr (!kTable) {
              a1 = e2m1_pairs<XT>(wb[c][s]);
            } else {
              uint32_t p1[4], p2[4];
#pragma unroll
              for (int kb = 0; kb < 4; ++kb) {
                const uint32_t addr =
                    __builtin_amdgcn_perm(wb[c][s], laneoff, 0x0C0C0000u | ((4u + (uint32_t)kb) << 8)) >> 1;
                if (kSplit) {
                  const uint2 tv = *reinterpret_cast<const uint2*>(tabc + addr);
                  p1[kb] = tv.x;
                  p2[kb] = tv.y;
                } else {
                  p1[kb] = *reinterpret_cast<const uint32_t*>(tabc + addr);
                }
              }
              a1 = make_uint4(p1[0], p1[1], p1[2], p1[3]);
              if (kSplit) a2 = make_uint4(p2[0], p2[1], p2[2], p2[3]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint4 bv = x[t][c * STEPS + s];
              dd[t] = mfma<XT>(a1, bv, dd[t]);
              if constexpr (kSplit) dd[t] = mfma<XT>(a2, bv, dd[t]);
              if constexpr (FMT == kINT4A) dd[t] = mfma<XT>(zrow, bv, dd[t]);
            }
            if constexpr (kMX) {
              const uint32_t sraw = __float_as_uint(e8m0_value((d.s[r][c] >> (8 * s)) & 0xFFu));
              const float sc[4] = {row_bcast<0>(sraw), row_bcast<1>(sraw), row_bcast<2>(sraw),
                                   row_bcast<3>(sraw)};
#pragma unroll
              for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf(dd[t][i], sc[i], acc[r][t][i]);
                dd[t] = float4_t{0.f, 0.f, 0.f, 0.f};
              }
            }
          }
          if constexpr (!kMX) {
            const uint32_t sraw = is_g128(FMT) ? d.s[r][c] << 16 : c > 0 && qb + c >= nblocks ? 0u : d.s[r][c];
            const float sc[4] = {row_bcast<0>(sraw), row_bcast<1>(sraw), row_bcast<2>(sraw),
                                 row_bcast<3>(sraw)};
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf(dd[t][i], sc[i], acc[r][t][i]);
          }
        }
      }
    };

    // Activations two quads ahead like the weights for one column tile; more tiles leave registers
    // for one set.
    uint4 X0[NT][8], X1[NT][8];
    load_cols(q0, true, X0);
    if constexpr (NT == 1) load_cols(q0 + 1, 1 < qpk, X1);
    for (uint32_t q = 0; q < qpk; q += 2) {
      compute(q0 + q, W0, X0);
      load_weights(q0 + q + 2, q + 2 < qpk, W0);
      if constexpr (NT == 1) {
        load_cols(q0 + q + 2, q + 2 < qpk, X0);
      } else {
        load_cols(q0 + q + 1, q + 1 < qpk, X0);
      }
      if (q + 1 < qpk) {
        if constexpr (NT == 1) {
          compute(q0 + q + 1, W1, X1);
          load_weights(q0 + q + 3, q + 3 < qpk, W1);
          load_cols(q0 + q + 3, q + 3 < qpk, X1);
        } else {
          compute(q0 + q + 1, W1, X0);
          load_weights(q0 + q + 3, q + 3 < qpk, W1);
          load_cols(q0 + q + 2, q + 2 < qpk, X0);
        }
      }
    }

    if constexpr (KW > 1) {
      if (c0 > 0) __syncthreads();  // the previous chunk's sums have been read
      if (kg > 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int t = 0; t < NT; ++t) red[((((kg - 1) * RW + rg) * 2 + r) * NT + t) * 64 + lane] = acc[r][t];
      }
      __syncthreads();
      if (kg > 0) continue;
      for (int j = 1; j < KW; ++j) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float4_t v = red[((((j - 1) * RW + rg) * 2 + r) * NT + t) * 64 + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][t][i] += v[i];
          }
      }
    }
    if constexpr (kSplit) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][t][i] *= 1.0f / kNf4Factor;
    }
    if (!live) continue;

    if constexpr (DIR == kUp) {
      const uint32_t inter = a.n >> 1;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint32_t p[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gate = acc[0][t][i];
          const float v = gate / (1.0f + expf(-gate)) * acc[1][t][i];
          const uint32_t b1 = __float_as_uint(v) & 0xFFFF0000u;
          const float r1 = __builtin_isinf(v) ? 0.0f : v - __uint_as_float(b1);
          const uint32_t b2 = __float_as_uint(r1) & 0xFFFF0000u;
          p[0][i] = b1;
          p[1][i] = b2;
          // (r1 may be the remainder of the unrounded product, a contracted multiply-subtract: cut)
          p[2][i] = __float_as_uint(r1 - __uint_as_float(b2)) & 0xFFFF0000u;
        }
        if (chave[t]) {
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) {
            const size_t at = ((size_t)pl * a.pairs + (uint32_t)pair[t]) * inter + row0 + 4u * g;
            *reinterpret_cast<uint2*>(a.h + at) =
                make_uint2(p[pl][0] >> 16 | p[pl][1], p[pl][2] >> 16 | p[pl][3]);
          }
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (NT == 1) {
          float4_t v;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v2 = __shfl(acc[r][0][i], lane + kMoePacked), v3 = __shfl(acc[r][0][i], lane + 2 * kMoePacked);
            v[i] = acc[r][0][i] + (v2 + v3);
          }
          if (m < kMoePacked && chave[0])
            *reinterpret_cast<float4_t*>(a.part + (size_t)pair[0] * a.n + (r ? row1 : row0) + 4u * g) = v;
        } else {
#pragma unroll
          for (int t = 0; t < NT; t += 3) {
            float4_t v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = acc[r][t][i] + (acc[r][t + 1][i] + acc[r][t + 2][i]);
            if (chave[t])
              *reinterpret_cast<float4_t*>(a.part + (size_t)pair[t] * a.n + (r ? row1 : row0) + 4u * g) = v;
          }
        }
      }
    }
  }
}

template <int DIR, int FMT, int XT, int NT>
hipError_t launch_moe_kw(int kw, const MoeArgs& a, uint32_t slots, hipStream_t s) {
  const uint32_t rw = 8u / (uint32_t)kw;
  const dim3 grid((a.units + rw - 1) / rw, slots, 1);
  switch (kw) {
    case 1: hipLaunchKernelGGL((moe_kernel<DIR, FMT, XT, NT, 1>), grid, dim3(kMoeThreads), 0, s, a); break;
    case 2: hipLaunchKernelGGL((moe_kernel<DIR, FMT, XT, NT, 2>), grid, dim3(kMoeThreads), 0, s, a); break;
    case 4: hipLaunchKernelGGL((moe_kernel<DIR, FMT, XT, NT, 4>), grid, dim3(kMoeThreads), 0, s, a); break;
    case 8: hipLaunchKernelGGL((moe_kernel<DIR, FMT, XT, NT, 8>), grid, dim3(kMoeThreads), 0, s, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int DIR, int XT, int NT>
hipError_t launch_moe_weight(int weight, int kw, const MoeArgs& a, uint32_t slots, hipStream_t s) {
  switch (weight) {
    case kNF4: return launch_moe_kw<DIR, kNF4, XT, NT>(kw, a, slots, s);
    case kINT4: return launch_moe_kw<DIR, kINT4, XT, NT>(kw, a, slots, s);
    case kFP4: return launch_moe_kw<DIR, kFP4, XT, NT>(kw, a, slots, s);
    case kINT4A: return launch_moe_kw<DIR, kINT4A, XT, NT>(kw, a, slots, s);
    case kMXFP4: return launch_moe_kw<DIR, kMXFP4, XT, NT>(kw, a, slots, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace w4
