// Expert products of the mixture-of-experts layer on the matrix cores (kernel template; one
// translation unit per direction and activation type instantiates it).
//
// The layer: y[t] = sum_j w[t, j] Down_e h[t, j], h[t, j] = silu(Gate_e x[t]) (Up_e x[t]),
// e = ids[t, j], with silu(v) = v / (1 + exp(-v)).  A (token, slot) pair is a column of its expert's
// products; the up kernel writes h for every pair, the down kernel one row of partial results per
// pair, and the combine kernel adds a token's pairs in slot order, scaled by their routing weights.
//
// Which experts are in use is known on the device alone.  With fewer pairs than experts (and for one token)
// a wave takes one pair (moe_pair_kernel, moe_token_kernel).  With more, the pairs of an expert share its
// weights: grid.y is the expert, whose workgroups end at once if no pair has it.  Every wave finds
// its expert's pairs itself, 64 ids at a time (a ballot, and a lane permutation that hands the r-th
// pair to lane r): no launch, memory or barrier for a sorted list.  With
// several pairs an expert, the kernels of w4_moe_wide_impl.h take over.
//
// Inside a workgroup 8 waves are RT row tiles (16 weight rows each) x KW K groups; the tiles of the
// up direction alternate between a gate tile and the up tile of the same rows.  K runs in quads (256
// weights of a row), in KW contiguous ranges.  A workgroup walks several groups of RT tiles of its
// expert, its loads running ahead across them.
//   * v_mfma_f32_16x16x32, A = 16 columns of the chunk x 32 k from LDS, B = 32 k x 16 weight rows
//     decoded in registers, the k order inside a block permuted alike on both sides.  A lane's
//     results all belong to one weight row, so the block scale is the lane's own: fp32 accumulation
//     per scale block, then acc += scale * D.
//   * A lane's weights arrive in two 16-byte loads per quad (whole 128-byte lines), two quads ahead of
//     the one being multiplied.
//   * The chunk's activations are copied into LDS once per window (all of K where it fits), 16-byte
//     pieces at position piece ^ (row mod 16): the 16 lanes that an LDS cycle serves read
//     16 different rows at one k, and the exclusive or puts them in different banks.
//   * Weight codes are exact 16-bit values, decoded without a table: E2M1 through the hardware
//     conversion, integers as q + 16 (two operations a pair) with one more MFMA whose columns
//     hold -(16 + z) taking the offset off.  The activations are put into the decoder's order on their
//     way into the window.  NF4's codes are not exact: they are held as two 16-bit terms in a byte
//     -> pair LDS table, after a factor of 1.4376 (taken off the sums) that leaves the two bf16
//     terms an rms error of 4.2e-7 over normal weights (2.5e-6 without it).
//   * h has fp32's 24 bits as three bf16 planes (the value cut after 8 bits, then the rest, then
//     what is left), which keeps bf16's range for either activation type.  The planes are rows of
//     the same product: four tokens' planes share one 16-row tile, so keeping 24 bits costs a few
//     tokens nothing; from five tokens on a plane is a tile of its own.
//   * A group's sums go through LDS, where every thread takes its share of the results: the K groups
//     are added in group order, gate meets up, and a row's values are stored side by side.
// Measured on MI355X, 32 tokens, 8 of 128 experts, 2048 x 768, MXFP4 (280 MB of weights): up 44 us (4.3 TB/s),
// down 39 us (2.4 TB/s: rows of three quads leave little to run ahead with), where a copy reaches 4.8 TB/s.
#pragma once
#include <type_traits>

#include "w4_mfma_common.h"
#include "w4_moe.h"

namespace w4 {
namespace {

constexpr int kUp = 0, kDown = 1;
constexpr float kNf4Factor = 1.4376f;
__constant__ uint32_t c_moe_nf4[16] = W4_NF4_CODE_BITS;
__constant__ uint32_t c_moe_fp4[16] = W4_FP4_CODE_BITS;

// NF4's byte -> decoded pair table: 16 copies of each 8-byte entry (first terms, second terms), lane L
// reading copy L % 16.
template <int XT, int THREADS = kMoeThreads>
__device__ inline void fill_moe_table(uint32_t* tab) {
  const float c = __uint_as_float(codes_in_lanes<kNF4>()) * kNf4Factor;
  uint32_t v1, v2;
  if (XT == kF16) {
    const _Float16 hi = (_Float16)c;
    v1 = f16_bits((float)hi);
    v2 = f16_bits(c - (float)hi);
  } else {
    v1 = bf16_rne_bits(c);
    v2 = bf16_rne_bits(c - __uint_as_float(v1 << 16));
  }
  uint4* t4 = reinterpret_cast<uint4*>(tab);
  const int tid = threadIdx.x;
  const uint32_t lo1 = (uint32_t)__shfl((int)v1, (tid >> 3) & 15) << 16;
  const uint32_t lo2 = (uint32_t)__shfl((int)v2, (tid >> 3) & 15) << 16;
#pragma unroll
  for (int j = 0; j < kTableBytes / 16 / THREADS; ++j) {
    const int i = tid + THREADS * j;
    const int hi = __builtin_amdgcn_readfirstlane(i >> 7);
    const uint32_t p1 = (uint32_t)__builtin_amdgcn_readlane((int)v1, hi) | lo1;
    const uint32_t p2 = (uint32_t)__builtin_amdgcn_readlane((int)v2, hi) | lo2;
    t4[i] = make_uint4(p1, p2, p1, p2);
  }
}

// Eight weights of a packed dword as 16-bit pairs, without a table.  Each decoder gives its own order of
// the eight, and `arranged` puts an activation piece (8 values in memory order) into that order.
//   E2M1: one conversion per byte, the low nibble (odd k) first.
//   q + 16 (integers): the nibble of each half placed in the mantissa of 16.0, two operations a pair:
//   nibbles 0, 1, 2, 3 of the halves, which are k = (1, 5), (0, 4), (3, 7), (2, 6).
template <int FMT, int XT>
__device__ inline uint4 decode8(uint32_t w) {
  if constexpr (FMT == kFP4 || FMT == kMXFP4) {
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
  } else if constexpr (XT == kF16) {  // 16.0 = 0x4C00, one unit = 1 << 6
    constexpr uint32_t kMask = 0x03C003C0u, kOne = 0x4C004C00u;
    return make_uint4(((w << 6) & kMask) | kOne, ((w << 2) & kMask) | kOne, ((w >> 2) & kMask) | kOne,
                      ((w >> 6) & kMask) | kOne);
  } else {  // 16.0 = 0x4180, one unit = 1 << 3
    constexpr uint32_t kMask = 0x00780078u, kOne = 0x41804180u;
    return make_uint4(((w << 3) & kMask) | kOne, ((w >> 1) & kMask) | kOne, ((w >> 5) & kMask) | kOne,
                      ((w >> 9) & kMask) | kOne);
  }
}

template <int FMT>
__device__ inline uint4 arranged(uint4 v) {
  if constexpr (FMT == kFP4 || FMT == kMXFP4) {
    return make_uint4(__builtin_amdgcn_alignbit(v.x, v.x, 16), __builtin_amdgcn_alignbit(v.y, v.y, 16),
                      __builtin_amdgcn_alignbit(v.z, v.z, 16), __builtin_amdgcn_alignbit(v.w, v.w, 16));
  } else if constexpr (is_g128(FMT)) {
    constexpr uint32_t kHi = 0x07060302u, kLo = 0x05040100u;  // (second, first) operand's halves
    return make_uint4(__builtin_amdgcn_perm(v.z, v.x, kHi), __builtin_amdgcn_perm(v.z, v.x, kLo),
                      __builtin_amdgcn_perm(v.w, v.y, kHi), __builtin_amdgcn_perm(v.w, v.y, kLo));
  } else {
    return v;
  }
}

// The pairs of expert e in pair order: returns their number, and in lane r (r < ncol <= 63) the pair of
// rank c0 + r, or -1.  Every lane of the wave takes part.
__device__ inline uint32_t scan_pairs(const int32_t* __restrict__ ids, uint32_t pairs, int e, uint32_t c0,
                                      uint32_t ncol, int lane, int& mine) {
  uint32_t total = 0;
  mine = -1;
  auto batch = [&](uint32_t base, int id) __attribute__((always_inline)) {
    const bool match = id == e;
    const uint64_t mask = __ballot(match);
    if (mask == 0) return;
    const uint32_t rank = total + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                            __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
    // lanes without a pair of this chunk send to lane 63, which is no column
    const uint32_t to = match && rank - c0 < ncol ? rank - c0 : 63u;
    const int got = __builtin_amdgcn_ds_permute((int)(to * 4u), (int)(base + (uint32_t)lane + 1u));
    if (lane < (int)ncol && got > 0) mine = got - 1;
    total += (uint32_t)__builtin_popcountll(mask);
  };
  // eight batches at a time: their loads are in flight together
  for (uint32_t base = 0; base < pairs; base += 512) {
    int id[8];
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint32_t i = base + 64u * b + (uint32_t)lane;
      id[b] = i < pairs ? ids[i] : -1;
    }
#pragma unroll
    for (int b = 0; b < 8; ++b) batch(base + 64u * b, id[b]);
  }
  return total;
}

// A quad of this lane's tile: load h.
struct MoeQuad {
  uint32_t w[2][4];
};

// Block scales.  The scales of 16 rows lie together in memory, a few bytes of each row per quad, so they
// are loaded for eight quads at a time: lane 4 r + p takes those of quads 2 p, 2 p + 1 of row r, and a
// quad's scales reach the 4 lanes of their row by lane permutations.  (Loaded quad by quad, each load
// touched 16 cache lines for a few bytes of each, and re-fetched them from L2 at every quad.)
template <int FMT>
struct MoeScales {
  static constexpr uint32_t kQuads = 8;
  static constexpr int kPer = FMT == kMXFP4 ? 2 : FMT == kINT4 ? 1 : FMT == kINT4A ? 2 : 4;  // dwords a quad
  // 2-byte rows: one dword more, loaded from the aligned address below and shifted into place
  static constexpr bool kShift = FMT == kMXFP4 || FMT == kINT4;
  static constexpr int kRaw = 2 * kPer + (kShift ? 1 : 0);
  uint32_t v[kRaw];
};

// A half quad's dwords as the B operands of its steps: wb[block][step] holds 8 weights of row m, k order inside
// a block permuted as the activations' pieces are read.
template <int FMT, int H>
__device__ __attribute__((always_inline)) inline void half_steps(
    const MoeQuad& d, uint32_t (&wb)[is_g128(FMT) ? 1 : 2][is_g128(FMT) ? 4 : 2]) {
  // chunks g and g + 4 of row m: lanes m < 8 hold (row m, g) in load 0 and need (row m, g + 4) of
  // lane m + 8; lanes m >= 8 hold (row m, g + 4) in load 1 and need (row m, g) of lane m - 8
  uint32_t wh[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    wh[i] = H == 0 ? (uint32_t)__builtin_amdgcn_update_dpp((int)d.w[0][i], (int)d.w[1][i], 0x118, 0xF, 0xC, false)
                   : (uint32_t)__builtin_amdgcn_update_dpp((int)d.w[1][i], (int)d.w[0][i], 0x108, 0xF, 0x3, false);
  if constexpr (is_g128(FMT)) {
#pragma unroll
    for (int s = 0; s < 4; ++s) wb[0][s] = wh[s];
  } else {
    // 64-weight blocks: chunks 2 c, 2 c + 1 of the half quad to every lane group, two dwords
    // each; MXFP4: one more swap gives step s the dwords of the 32-weight block s.
    const auto s0 = __builtin_amdgcn_permlane32_swap(wh[0], wh[2], false, false);
    const auto s1 = __builtin_amdgcn_permlane32_swap(wh[1], wh[3], false, false);
    wb[0][0] = s0[0];
    wb[0][1] = s1[0];
    wb[1][0] = s0[1];
    wb[1][1] = s1[1];
    if constexpr (FMT == kMXFP4) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const auto t = __builtin_amdgcn_permlane16_swap(wb[c][0], wb[c][1], false, false);
        wb[c][0] = t[0];
        wb[c][1] = t[1];
      }
    }
  }
}

// acc += the product of the quad held in d (B) and 256 k of the window (A).  The quad is the jw-th of the
// scales' eight, ODD its parity; `left` is the bytes of its row's scales that lie inside K; its first piece of A row r
// of column tile t stands at wbase + arow[t].
template <int FMT, int XT, int NT, int ODD>
__device__ __attribute__((always_inline)) inline void quad_product(
    float4_t (&acc)[NT], const MoeQuad& d, const MoeScales<FMT>& scales, uint32_t jw, uint32_t left,
    const uint8_t* wbase, const uint32_t (&arow)[NT], const uint32_t (&apiece)[NT], const uint32_t* tab, int lane) {
  using Sc = MoeScales<FMT>;
  constexpr int KC = is_g128(FMT) ? 128 : 64;  // weights per block
  constexpr uint32_t QC = 256 / KC;
  constexpr int STEPS = KC / 32;
  constexpr bool kMX = FMT == kMXFP4;
  constexpr bool kTable = FMT == kNF4;
  constexpr uint32_t SB = FMT == kINT4 || kMX ? 2 : 4;
  const int m = lane & 15;
  const uint32_t laneoff = (uint32_t)m * 16u;
  const char* tabc = reinterpret_cast<const char*>(tab);
  // The quad's scales of row m: from lane 4 m + (pair of quads), the quad's half of its dwords.  Those of
  // blocks past K are the next row's: zeros instead.
  const int from = (4 * m + (int)(jw >> 1)) * 4;
  uint32_t sw[Sc::kPer];
#pragma unroll
  for (int i = 0; i < Sc::kPer; ++i)
    sw[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)scales.v[ODD * Sc::kPer + i]);
  if (left < QC * SB) {
#pragma unroll
    for (int i = 0; i < Sc::kPer; ++i)
      sw[i] = 4u * i + 4u <= left ? sw[i] : 4u * i < left ? sw[i] & 0xFFFFu : 0u;
  }
  // (Opaque copies: offsets derived from these are recomputed per quad, an operation each, instead of
  // being held across the loop in registers that the loads in flight need.)
  uint32_t ap[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    ap[t] = apiece[t];
    asm volatile("" : "+v"(ap[t]));
  }
  uint32_t wb[QC][STEPS], half[2][QC / 2][STEPS];
  half_steps<FMT, 0>(d, half[0]);
  half_steps<FMT, 1>(d, half[1]);
#pragma unroll
  for (int c = 0; c < (int)QC; ++c)
#pragma unroll
    for (int s = 0; s < STEPS; ++s) wb[c][s] = half[c / (QC / 2)][c % (QC / 2)][s];
#pragma unroll
  for (int c = 0; c < (int)QC; ++c) {
    float4_t dd[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) dd[t] = float4_t{0.f, 0.f, 0.f, 0.f};
    // Integer codes decode as q + 16; a column of -(16 + z) takes the offset off (z = 8: INT4).
    uint4 zcol = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (is_g128(FMT)) {
      const float zn = FMT == kINT4 ? -24.0f : -16.0f - (float)((sw[c % Sc::kPer] >> 16) & 15u);
      const uint32_t h = XT == kF16 ? f16_bits(zn) : (__float_as_uint(zn) >> 16);
      zcol = make_uint4(h | (h << 16), h | (h << 16), h | (h << 16), h | (h << 16));
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      constexpr uint32_t kPieces = KC / 8;  // of a block
      const uint32_t at = (c * kPieces + s * (kMX ? 4u : 1u)) * 16u;
      uint4 xv[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) xv[t] = *reinterpret_cast<const uint4*>(wbase + arow[t] + (ap[t] ^ at));
      uint4 b1, b2;
      if constexpr (kTable) {
        uint2 tv[4];
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          // LDS byte address = byte * 128 + lane offset: byte * 256 + 2 * lane offset, halved
          const uint32_t addr =
              __builtin_amdgcn_perm(wb[c][s], laneoff, 0x0C0C0000u | ((4u + (uint32_t)kb) << 8)) >> 1;
          tv[kb] = *reinterpret_cast<const uint2*>(tabc + addr);
        }
        b1 = make_uint4(tv[0].x, tv[1].x, tv[2].x, tv[3].x);
        b2 = make_uint4(tv[0].y, tv[1].y, tv[2].y, tv[3].y);
      } else {
        b1 = decode8<FMT, XT>(wb[c][s]);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        dd[t] = mfma<XT>(xv[t], b1, dd[t]);
        if constexpr (kTable) dd[t] = mfma<XT>(xv[t], b2, dd[t]);
        if constexpr (is_g128(FMT)) dd[t] = mfma<XT>(xv[t], zcol, dd[t]);
      }
      if constexpr (kMX) {
        // 2^(e - 127); e = 255 gives an infinity here, and its sums are looked at again (defined_sum)
        const float sc = ldexpf(__uint_as_float(0x00400000u), (int)((sw[c >> 1] >> (16 * (c & 1) + 8 * s)) & 0xFFu));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(dd[t][i], sc, acc[t][i]);
          dd[t] = float4_t{0.f, 0.f, 0.f, 0.f};
        }
      }
    }
    if constexpr (!kMX) {
      const float sc = __uint_as_float(FMT == kINT4    ? (c == 0 ? sw[0] << 16 : sw[0] & 0xFFFF0000u)
                                       : FMT == kINT4A ? sw[c % Sc::kPer] << 16 : sw[c % Sc::kPer]);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(dd[t][i], sc, acc[t][i]);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The scales of eight quads as loaded (see MoeScales), from byte `off` of the tile's.
template <int FMT>
__device__ inline void load_scale_window(MoeScales<FMT>& d, __amdgpu_buffer_rsrc_t rs, uint32_t off) {
  if constexpr (FMT == kINT4) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, (int)off, 0, 0);
    d.v[0] = v[0];
    d.v[1] = v[1];
    d.v[2] = buffer_load32(rs, off + 8u);
  } else {
    const uint4 v = buffer_load16(rs, off);
    d.v[0] = v.x; d.v[1] = v.y; d.v[2] = v.z; d.v[3] = v.w;
    if constexpr (FMT == kMXFP4) d.v[4] = buffer_load32(rs, off + 16u);
    if constexpr (MoeScales<FMT>::kPer == 4) {
      const uint4 u = buffer_load16(rs, off + 16u);
      d.v[4] = u.x; d.v[5] = u.y; d.v[6] = u.z; d.v[7] = u.w;
    }
  }
}

// ... and moved into place; `sshift`: the bits by which a 2-byte row starts inside its first dword.
template <int FMT>
__device__ inline void place_scales(MoeScales<FMT>& held, const MoeScales<FMT>& raw, uint32_t sshift) {
#pragma unroll
  for (int i = 0; i < 2 * MoeScales<FMT>::kPer; ++i) {
    if constexpr (MoeScales<FMT>::kShift) {
      held.v[i] = __builtin_amdgcn_alignbit(raw.v[i + 1], raw.v[i], sshift);
    } else {
      held.v[i] = raw.v[i];
    }
  }
}

// h = silu(gate) up of one row and pair, as three bf16 planes.
__device__ inline void store_h(const MoeArgs& a, uint32_t pair, uint32_t row, uint32_t inter, float gate, float up) {
  const float v = gate / (1.0f + expf(-gate)) * up;
  const uint32_t b1 = __float_as_uint(v) & 0xFFFF0000u;
  const float r1 = __builtin_isinf(v) ? 0.0f : v - __uint_as_float(b1);
  const uint32_t b2 = __float_as_uint(r1) & 0xFFFF0000u;
  const float r2 = r1 - __uint_as_float(b2);  // cut: a contracted r1 may be longer
  const size_t at = (size_t)pair * inter + row, plane = (size_t)a.pairs * inter;
  a.h[at] = (uint16_t)(b1 >> 16);
  a.h[at + plane] = (uint16_t)(b2 >> 16);
  a.h[at + 2 * plane] = (uint16_t)(__float_as_uint(r2) >> 16);
}

// Sums that are not finite, computed again from the definition.  The kernels' arithmetic leaves it there:
// integer codes are taken as q + 16 with an offset taken off beside and NF4's as two terms, so an infinite operand
// meets terms of both signs (a NaN where the definition has an infinity), sums of such terms may
// overflow early, and an MXFP4 scale byte of 255 multiplies as an infinity.  A kernel marks that one of its sums
// was not finite and looks at what it stored; a wave with none passes by.  One row over k0 .. k1 - 1 in 64
// bits: code scale x, x the value whose NP planes (bf16) or one value (XT) stand in its row.
template <int FMT, int XT, int NP>
__device__ __attribute__((always_inline)) inline float defined_sum(const MoeArgs& a, int e, uint32_t row, uint32_t xrow,
                                                                   uint32_t k0, uint32_t k1) {
  constexpr uint32_t KC = FMT == kMXFP4 ? 32 : is_g128(FMT) ? 128 : 64;
  constexpr uint32_t SB = FMT == kMXFP4 ? 1 : FMT == kINT4 ? 2 : 4;
  const size_t at = (size_t)e * a.n + row;
  const uint8_t* packed = a.packed + at * (a.k >> 1);
  const char* scales = reinterpret_cast<const char*>(a.scales) + at * (a.k / KC * SB);
  const uint16_t* x = a.x + (size_t)xrow * a.k;
  const size_t plane = (size_t)a.pairs * a.k;
  double sum = 0.0;
#pragma unroll 1
  for (uint32_t k = k0; k < k1 && sum == sum; k += 8) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(packed + (k >> 1));
    const char* sp = scales + k / KC * SB;
    float scale, zero = FMT == kINT4 ? 8.0f : 0.0f;
    if constexpr (FMT == kMXFP4) {
      scale = e8m0_value(*reinterpret_cast<const uint8_t*>(sp));
    } else if constexpr (FMT == kINT4) {
      scale = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(sp) << 16);
    } else {
      const uint32_t word = *reinterpret_cast<const uint32_t*>(sp);
      scale = __uint_as_float(FMT == kINT4A ? word << 16 : word);
      if constexpr (FMT == kINT4A) zero = (float)((word >> 16) & 15u);
    }
    float v[8], code[8];
    auto halves = [&](const uint16_t* p, auto add) __attribute__((always_inline)) {
      const uint4 q = *reinterpret_cast<const uint4*>(p + k);
      const uint32_t d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) add(v[i], (d[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
    };
    if constexpr (XT == kF16) {
      halves(x, [](float& o, uint32_t b) { o = (float)__builtin_bit_cast(_Float16, (uint16_t)b); });
    } else {
      halves(x, [](float& o, uint32_t b) { o = __uint_as_float(b << 16); });
      if constexpr (NP == 3) {
        halves(x + plane, [](float& o, uint32_t b) { o += __uint_as_float(b << 16); });
        halves(x + 2 * plane, [](float& o, uint32_t b) { o += __uint_as_float(b << 16); });
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t nibble = (w >> (4 * (i ^ 1))) & 15u;  // the high nibble first
      if constexpr (is_g128(FMT)) {
        code[i] = (float)nibble - zero;
      } else {
        code[i] = __uint_as_float(FMT == kNF4 ? c_moe_nf4[nibble] : c_moe_fp4[nibble]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += (double)code[i] * scale * v[i];
  }
  return (float)sum;
}

// NaN into `odd` if v is not finite.
__device__ inline void watch(float& odd, float v) { odd = __builtin_fmaf(v, 0.0f, odd); }

// The launch's arguments read anew from memory: what looks at results again holds no register for it before.
__device__ __attribute__((always_inline)) inline MoeArgs args_again() {
  uint64_t p = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  MoeArgs a;
  __builtin_memcpy(&a, (const MoeArgs*)reinterpret_cast<const __attribute__((address_space(4))) MoeArgs*>(p), sizeof(a));
  return a;
}

// h of one row and pair, and a partial result, looked at again.  (h is not finite where gate or up is not.)
template <int FMT, int XT>
__device__ __attribute__((always_inline)) inline void settle_h(const MoeArgs& a, int e, uint32_t pair, uint32_t row) {
  const uint32_t inter = a.n >> 1;
  if ((a.h[(size_t)pair * inter + row] & 0x7F80u) != 0x7F80u) return;
  float gate = 0.0f, up = 0.0f;
#pragma unroll 1
  for (uint32_t r = 0; r < 2; ++r) {
    const float v = defined_sum<FMT, XT, 1>(a, e, r * inter + row, pair / a.top_k, 0, a.k);
    gate = r == 0 ? v : gate;
    up = v;
  }
  store_h(a, pair, row, inter, gate, up);
}

template <int FMT>
__device__ __attribute__((always_inline)) inline void settle_part(const MoeArgs& a, int e, uint32_t pair, uint32_t row) {
  float* p = a.part + (size_t)pair * a.n + row;
  if (!__builtin_isfinite(*p)) *p = defined_sum<FMT, kBF16, 3>(a, e, row, pair, 0, a.k);
}

template <int DIR, int FMT, int XT, int NT, int KW>
__global__ void __launch_bounds__(kMoeThreads, NT == 1 ? 4 : 2) moe_kernel(MoeArgs a) {
  constexpr uint32_t RT = 8 / KW;
  constexpr int KC = is_g128(FMT) ? 128 : 64;  // weights per block
  constexpr uint32_t QC = 256 / KC;
  constexpr bool kMX = FMT == kMXFP4;
  constexpr bool kTable = FMT == kNF4;
  constexpr uint32_t SB = FMT == kINT4 || kMX ? 2 : 4;
  __shared__ __align__(16) uint32_t tab[kTable ? kTableBytes / 4 : 4];
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* win = smem;                                          // the window of activations
  float* sums = reinterpret_cast<float*>(smem + a.win_bytes);  // two buffers of [8 waves][NT][4][64]

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t rt = (uint32_t)wave % RT, kg = (uint32_t)wave / RT;
  const int g = lane >> 4, m = lane & 15;

  const int e = (int)blockIdx.y;  // the expert
  if constexpr (kTable) fill_moe_table<XT>(tab);
  const uint32_t cols = a.cols;  // pairs of a chunk

  const uint32_t qpk = a.qpk;
  const uint32_t pitch = a.k >> 1;
  const uint32_t nblocks = a.k / KC;
  const uint32_t spitch = nblocks * SB;
  const uint32_t ngroups = (a.tiles + RT - 1) / RT;
  // First weight row of tile `tile` (tiles past the last: none, they read zeros).
  auto tile_rsrc = [&](const void* base, uint32_t tile, uint32_t bytes) __attribute__((always_inline)) {
    const bool live = tile < a.tiles;
    const uint32_t row0 = DIR == kUp ? (tile & 1u) * (a.n >> 1) + (tile >> 1) * 16u : tile * 16u;
    const size_t row = (size_t)e * a.n + (live ? row0 : 0u);
    return make_rsrc(reinterpret_cast<const char*>(base) + row * bytes, live ? 16u * bytes : 0u);
  };

  // The load cursor: quad lj of tile lt.
  uint32_t lt, lj;
  __amdgpu_buffer_rsrc_t rw;
  // Weight loads of lane (g, m): load h covers rows 8 h .. 8 h + 7, whole 128-byte lines with 8 lanes
  // each: the lane takes row 8 h + (m & 7), chunk (16 bytes) g + 4 (m >> 3).
  const uint32_t chunk = (uint32_t)g + 4u * (uint32_t)(m >> 3);
  const uint32_t wlane = (uint32_t)(m & 7) * pitch + chunk * 16u;
  const uint32_t nchunks = a.k >> 5;
  // The quad at the cursor (past K everything reads as zero), and the cursor's step: tiles of an even
  // number of quads, the last of an odd count left out.
  auto load_quad = [&](MoeQuad& d) __attribute__((always_inline)) {
    if (lj < qpk) {
      const uint32_t q = kg * qpk + lj;
      const bool in = q * 8 + chunk < nchunks;
      const uint4 v0 = buffer_load16_stream(rw, offset_or_oob(in, wlane + q * 128u));
      const uint4 v1 = buffer_load16_stream(rw, offset_or_oob(in, wlane + q * 128u + 8u * pitch));
      d.w[0][0] = v0.x; d.w[0][1] = v0.y; d.w[0][2] = v0.z; d.w[0][3] = v0.w;
      d.w[1][0] = v1.x; d.w[1][1] = v1.y; d.w[1][2] = v1.z; d.w[1][3] = v1.w;
    }
    if (++lj >= ((qpk + 1u) & ~1u)) {
      lj = 0;
      lt += gridDim.x * RT;
      rw = tile_rsrc(a.packed, lt, pitch);
    }
  };

  // The scale cursor, window sj (eight quads) of tile st, one window ahead of the multiplication.
  using Sc = MoeScales<FMT>;
  uint32_t st, sj;
  const uint32_t nsw = (qpk + Sc::kQuads - 1) / Sc::kQuads;
  auto load_scales = [&](Sc& d) __attribute__((always_inline)) {
    const uint32_t q = kg * qpk + sj * Sc::kQuads;
    const uint32_t at = (uint32_t)(lane >> 2) * spitch + (q + 2u * (uint32_t)(lane & 3)) * (QC * SB);
    const uint32_t off = offset_or_oob(q * QC < nblocks, at & ~3u);
    const __amdgpu_buffer_rsrc_t rs = tile_rsrc(a.scales, st, spitch);
    load_scale_window<FMT>(d, rs, off);
    if (++sj == nsw) {
      sj = 0;
      st += gridDim.x * RT;
    }
  };
  // bits by which this lane's 2-byte rows start inside their first dword (rows of every tile alike:
  // a tile starts on a multiple of 32 bytes)
  const uint32_t sshift = ((uint32_t)(lane >> 2) * spitch & 2u) * 8u;

  const uint32_t rpitch = a.qpw * 512u;  // bytes of a window row: its quads
  const uint32_t per = a.qpw / KW;       // quads of a K group per window
  // This lane's A row in each column tile, as its window offset, and its piece of a block's first
  // step with the row's exclusive or.
  uint32_t arow[NT], apiece[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint32_t last = cols - 1u;
    const uint32_t r = DIR == kUp ? min((uint32_t)(16 * t + m), last)
                       : NT == 1  ? (uint32_t)min(m >> 2, 2) * cols + min((uint32_t)(m & 3), last)
                                  : (uint32_t)t * cols + min((uint32_t)m, last);
    const uint32_t piece = kMX ? g : is_g128(FMT) ? 4 * g : 4 * (g & 1) + 2 * (g >> 1);
    arow[t] = r * rpitch + kg * per * 512u;
    apiece[t] = (piece ^ (r & 15u)) * 16u;
  }
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(a.x, (DIR == kUp ? a.pairs / a.top_k : 3u * a.pairs) * a.k * 2u);

  MoeQuad W0, W1;
  Sc held_scales, next_scales;
  float odd_sum = 0.0f;  // NaN: a sum of this thread's was not finite
  uint32_t count = 1;
  for (uint32_t c0 = 0; c0 < count; c0 += cols) {
    // The expert's pairs, before any other vector load of the chunk: loads complete in order, and what
    // waits for the ids must not wait for weights.
    int list;
    count = scan_pairs(a.ids, a.pairs, e, c0, cols, lane, list);
    if (count == 0) return;  // (every wave sees the same count)
    const uint32_t have = min(cols, count - c0);
    lt = st = blockIdx.x * RT + rt;
    lj = sj = 0;
    rw = tile_rsrc(a.packed, lt, pitch);

    // Copies the window that starts at quad j0 of each K group (`per` quads of each, one group after the
    // other) of the chunk's rows: a unit is 64 pieces (two quads) of a row, each wave takes every eighth
    // unit and keeps four in flight.  At the start of a chunk the first weights are requested behind
    // the first of these loads.
    auto load_window = [&](uint32_t j0, bool start) __attribute__((always_inline)) {
      // (opaque copies: the divisions below are recomputed by each call, not held across the loop)
      uint32_t nseg = (a.qpw + 1u) / 2u, top_k = a.top_k, pl = cols, rows = have;
      asm volatile("" : "+s"(nseg), "+s"(top_k), "+s"(rows), "+s"(pl));
      const uint32_t total = (DIR == kUp ? rows : 3u * rows) * nseg;
      uint32_t u0 = (uint32_t)wave;
      do {
        uint4 v[4];
        uint32_t at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          at[i] = 0xFFFFFFFFu;
          const uint32_t u = u0 + 8u * i;
          if (u < total) {
            const uint32_t row = u / nseg, seg = u - row * nseg;
            const uint32_t plane = DIR == kUp ? 0u : row / rows, j = DIR == kUp ? row : row - plane * rows;
            const uint32_t p = (uint32_t)__builtin_amdgcn_readlane(list, (int)j);
            const uint32_t base = (DIR == kUp ? p / top_k : plane * a.pairs + p) * a.k * 2u;
            const uint32_t r = plane * pl + j;                             // window row
            const uint32_t sl = seg * 64u + (uint32_t)lane, ql = sl >> 5;  // slot and quad in the row
            // (all of K in the window, per == qpk: quads in order; else quads past the group's last
            // belong to the next one, and are left out)
            const uint32_t gr = per == qpk ? 0u : ql / per;
            const uint32_t jq = per == qpk ? 0u : j0 + ql - gr * per;
            const uint32_t quad = per == qpk ? ql : gr * qpk + jq;
            const uint32_t kpos = quad * 256u + (((sl & 31u) ^ (r & 15u)) * 8u);
            v[i] = buffer_load16(rx, offset_or_oob(kpos < a.k && jq < qpk, base + kpos * 2u));
            if (ql < a.qpw) at[i] = r * rpitch + sl * 16u;
          }
        }
        // (the stores stand in both branches: behind a join they would wait for the weights too)
        if (start) {
          load_scales(next_scales);
          load_quad(W0);
          load_quad(W1);
          start = false;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (at[i] != 0xFFFFFFFFu) *reinterpret_cast<uint4*>(win + at[i]) = arranged<FMT>(v[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (at[i] != 0xFFFFFFFFu) *reinterpret_cast<uint4*>(win + at[i]) = arranged<FMT>(v[i]);
        }
        u0 += 32u;
      } while (u0 < total);
    };

    float4_t acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};

    // Multiply the quad held in d: quad j of this K group, at window quad wq (of this K group).
    auto compute = [&](uint32_t j, uint32_t wq, const MoeQuad& d, auto odd) __attribute__((always_inline)) {
      const uint32_t qb = (kg * qpk + j) * QC;
      const uint32_t left = qb < nblocks ? (nblocks - qb) * SB : 0u;
      quad_product<FMT, XT, NT, decltype(odd)::value>(acc, d, held_scales, j % Sc::kQuads, left, win + wq * 512u, arow, apiece, tab, lane);
    };

    // A tile's value for (row n, A row 4 g + i of column tile t): its K groups' sums, in group order.
    // Waves hold theirs as [t][i][16 g + n].
    auto tile_value = [&](const float* buf, uint32_t tile, uint32_t n, uint32_t t, uint32_t r)
                          __attribute__((always_inline)) {
      float v = 0.0f;
      const uint32_t at = (t * 4u + (r & 3u)) * 64u + (r >> 2) * 16u + n;
#pragma unroll
      for (uint32_t w = 0; w < (uint32_t)KW; ++w) v += buf[(w * RT + tile % RT) * (NT * 256u) + at];
      return kTable ? v * (1.0f / kNf4Factor) : v;
    };
    uint32_t held = 0xFFFFFFFFu;  // first quad (of each K group) of the window in LDS
    uint32_t buffer = 0;
    for (uint32_t ug = blockIdx.x; ug < ngroups; ug += gridDim.x) {
      for (uint32_t j = 0; j < qpk; j += 2) {
        const uint32_t w0 = per == qpk ? 0u : j / per * per;
        if (w0 != held) {
          __syncthreads();  // every wave is done with the old window (or has written its table entries)
          load_window(w0, held == 0xFFFFFFFFu);
          held = w0;
          __syncthreads();
        }
        if (j % Sc::kQuads == 0) {  // the next scale window: shifted into place, the one after it requested
          place_scales<FMT>(held_scales, next_scales, sshift);
          load_scales(next_scales);
        }
        compute(j, j - w0, W0, std::integral_constant<int, 0>{});
        load_quad(W0);
        if (j + 1 < qpk) compute(j + 1, j + 1 - w0, W1, std::integral_constant<int, 1>{});
        load_quad(W1);
      }

      // The group's sums into this buffer; the other one is read until the next group's barrier.
      float* buf = sums + buffer * (8u * NT * 256u);
      buffer ^= 1u;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) buf[((uint32_t)wave * NT + t) * 256u + i * 64u + lane] = acc[t][i];
        acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
      }
      __syncthreads();
      const uint32_t tile0 = ug * RT, tiles = min(RT, a.tiles - tile0);
      if constexpr (DIR == kUp) {
        const uint32_t inter = a.n >> 1, row0 = tile0 * 8u, rows = tiles * 8u;  // rows of h in this group
        for (uint32_t i = (uint32_t)tid; i < rows * have; i += kMoeThreads) {
          const uint32_t j = i / rows, row = i - j * rows, tile = row / 16u * 2u, n = row & 15u;
          const int pair = __shfl(list, (int)j);  // (rows * have is a multiple of 16: lanes 0 .. 15 take part)
          const float gate = tile_value(buf, tile, n, j / 16u, j & 15u);
          const float up = tile_value(buf, tile + 1u, n, j / 16u, j & 15u);
          watch(odd_sum, gate);
          watch(odd_sum, up);
          store_h(a, (uint32_t)pair, row0 + row, inter, gate, up);
        }
      } else {
        const uint32_t row0 = tile0 * 16u, rows = tiles * 16u;
        for (uint32_t i = (uint32_t)tid; i < rows * have; i += kMoeThreads) {
          const uint32_t j = i / rows, row = i - j * rows, tile = row / 16u, n = row & 15u;
          const int pair = __shfl(list, (int)j);  // (rows * have is a multiple of 16: lanes 0 .. 15 take part)
          float v;
          if constexpr (NT == 1) {  // planes in rows 4 p + j
            v = tile_value(buf, tile, n, 0, j) + (tile_value(buf, tile, n, 0, 4u + j) + tile_value(buf, tile, n, 0, 8u + j));
          } else {
            v = tile_value(buf, tile, n, 0, j) + (tile_value(buf, tile, n, 1, j) + tile_value(buf, tile, n, 2, j));
          }
          watch(odd_sum, v);
          a.part[(size_t)(uint32_t)pair * a.n + row0 + row] = v;
        }
      }
    }
    if (c0 + cols < count) __syncthreads();  // the window and the sums have been read
  }
  if (__any(odd_sum != odd_sum)) {  // this wave's results once more, walked as above
    const MoeArgs b = args_again();
    const uint32_t ngroups = (b.tiles + RT - 1) / RT;
    int list;
    count = 1;
#pragma unroll 1
    for (uint32_t c0 = 0; c0 < count; c0 += b.cols) {
      count = scan_pairs(b.ids, b.pairs, (int)blockIdx.y, c0, b.cols, lane, list);
      const uint32_t have = min(b.cols, count - c0);
#pragma unroll 1
      for (uint32_t ug = blockIdx.x; ug < ngroups; ug += gridDim.x) {
        constexpr uint32_t kHeight = DIR == kUp ? 8u : 16u;  // result rows of a tile
        const uint32_t tile0 = ug * RT, row0 = tile0 * kHeight, rows = min(RT, b.tiles - tile0) * kHeight;
#pragma unroll 1
        for (uint32_t i = (uint32_t)tid; i < rows * have; i += kMoeThreads) {
          const uint32_t j = i / rows, row = row0 + i - j * rows;
          const uint32_t pair = (uint32_t)__shfl(list, (int)j);
          if constexpr (DIR == kUp) {
            settle_h<FMT, XT>(b, (int)blockIdx.y, pair, row);
          } else {
            settle_part<FMT>(b, (int)blockIdx.y, pair, row);
          }
        }
      }
    }
  }
}

// The products of a few tokens, whose pairs are few beside the experts: no list of an expert's pairs and no
// window that waves share.  A wave takes one pair; tokens that share an expert read its weights
// again, mostly from L2.  SL = 8 / KW pairs side by side in a workgroup, K in KW ranges; a wave's
// window holds what it needs itself, and no barrier stands before the sums.  Measured on MI355X, 1 token, 8 of 64
// experts, 2048 x 1024, INT4: up 8.6 us (2.0 TB/s), down 7.5 us (1.2 TB/s); 5 tokens, 4 of 60, 1536 x 1408,
// NF4: 17.3 and 10.8 us.  Bound by one load's latency after another: arguments, ids, weights.

// Up: 16 rows of h of SL slots of one token; a wave multiplies its expert's gate and up tile by x.
constexpr uint32_t kPairQuads = 8;  // quads of a wave's window

template <int FMT, int XT, int KW>
__global__ void __launch_bounds__(kMoeThreads, 4) moe_pair_kernel(MoeArgs a) {
  constexpr uint32_t SL = 8 / KW;
  constexpr int KC = is_g128(FMT) ? 128 : 64;
  constexpr uint32_t QC = 256 / KC;
  constexpr bool kMX = FMT == kMXFP4;
  constexpr bool kTable = FMT == kNF4;
  constexpr uint32_t SB = FMT == kINT4 || kMX ? 2 : 4;
  using Sc = MoeScales<FMT>;
  __shared__ __align__(16) uint32_t tab[kTable ? kTableBytes / 4 : 4];
  __shared__ float sums[8][2][16];
  __shared__ __align__(16) uint8_t window[8][kPairQuads * 512];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t sl = (uint32_t)wave % SL, kg = (uint32_t)wave / SL;
  const int g = lane >> 4, m = lane & 15;
  const uint32_t rounds = (a.top_k + SL - 1) / SL;
  const uint32_t token = blockIdx.y / rounds, slot0 = (blockIdx.y - token * rounds) * SL;
  const bool have = slot0 + sl < a.top_k;
  const uint32_t pair = token * a.top_k + slot0 + sl;
  const int e = have ? a.ids[pair] : -1;

  const uint32_t qpk = a.qpk;
  const uint32_t tile = blockIdx.x, inter = a.n >> 1;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (size_t)token * a.k, a.k * 2u);
  uint8_t* win = window[wave];
  // quads j0 .. j0 + 7 of this K range, 32 pieces each
  uint4 v[kPairQuads / 2];
  auto load_window = [&](uint32_t j0) __attribute__((always_inline)) {
#pragma unroll
    for (uint32_t i = 0; i < kPairQuads / 2; ++i) {
      const uint32_t jq = j0 + 2u * i + (uint32_t)(lane >> 5), kpos = (kg * qpk + jq) * 256u + ((uint32_t)lane & 31u) * 8u;
      if (j0 + 2u * i < qpk) v[i] = buffer_load16(rx, offset_or_oob(jq < qpk && kpos < a.k, kpos * 2u));
    }
  };
  auto store_window = [&](uint32_t j0) __attribute__((always_inline)) {
#pragma unroll
    for (uint32_t i = 0; i < kPairQuads / 2; ++i)
      if (j0 + 2u * i < qpk) *reinterpret_cast<uint4*>(win + i * 1024u + (uint32_t)lane * 16u) = arranged<FMT>(v[i]);
  };
  load_window(0);  // x does not wait for the ids
  if constexpr (kTable) {
    fill_moe_table<XT>(tab);
    __syncthreads();
  }

  const uint32_t pitch = a.k >> 1;
  const uint32_t nblocks = a.k / KC;
  const uint32_t spitch = nblocks * SB;
  const uint32_t nchunks = a.k >> 5;
  const uint32_t chunk = (uint32_t)g + 4u * (uint32_t)(m >> 3);
  const uint32_t wlane = (uint32_t)(m & 7) * pitch + chunk * 16u;
  const uint32_t sshift = ((uint32_t)(lane >> 2) * spitch & 2u) * 8u;
  const uint32_t arow[1] = {0};  // every A row is x
  const uint32_t apiece[1] = {(uint32_t)(kMX ? g : is_g128(FMT) ? 4 * g : 4 * (g & 1) + 2 * (g >> 1)) * 16u};

  if ((uint32_t)e < a.experts) {
    __amdgpu_buffer_rsrc_t rw[2], rs[2];
    size_t row0[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      row0[r] = (size_t)e * a.n + (r ? inter : 0u) + tile * 16u;
      rw[r] = make_rsrc(a.packed + row0[r] * pitch, 16u * pitch);
      rs[r] = make_rsrc(reinterpret_cast<const char*>(a.scales) + row0[r] * spitch, 16u * spitch);
    }
    auto load_quad = [&](uint32_t j, MoeQuad (&d)[2]) __attribute__((always_inline)) {
      const uint32_t q = kg * qpk + j;
      const bool in = j < qpk && q * 8 + chunk < nchunks;
      const uint32_t o0 = offset_or_oob(in, wlane + q * 128u), o1 = offset_or_oob(in, wlane + q * 128u + 8u * pitch);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 v0 = buffer_load16_stream(rw[r], o0);
        const uint4 v1 = buffer_load16_stream(rw[r], o1);
        d[r].w[0][0] = v0.x; d[r].w[0][1] = v0.y; d[r].w[0][2] = v0.z; d[r].w[0][3] = v0.w;
        d[r].w[1][0] = v1.x; d[r].w[1][1] = v1.y; d[r].w[1][2] = v1.z; d[r].w[1][3] = v1.w;
      }
    };
    Sc raw[2], held[2];
    auto load_scales = [&](uint32_t j) __attribute__((always_inline)) {
      const uint32_t q = kg * qpk + j;
      const uint32_t at = (uint32_t)(lane >> 2) * spitch + (q + 2u * (uint32_t)(lane & 3)) * (QC * SB);
      const uint32_t off = offset_or_oob(j < qpk && q * QC < nblocks, at & ~3u);
#pragma unroll
      for (int r = 0; r < 2; ++r) load_scale_window<FMT>(raw[r], rs[r], off);
    };
    MoeQuad W0[2], W1[2];
    load_scales(0);
    load_quad(0, W0);
    load_quad(1, W1);
    store_window(0);
    float4_t acc[2][1] = {{float4_t{0.f, 0.f, 0.f, 0.f}}, {float4_t{0.f, 0.f, 0.f, 0.f}}};
    for (uint32_t j = 0; j < qpk; j += 2) {
      if (j > 0 && j % kPairQuads == 0) {
        load_window(j);
        store_window(j);
      }
      if (j % Sc::kQuads == 0) {  // (past the first window the scales are waited for: few ranges are so long)
        if (j > 0) load_scales(j);
#pragma unroll
        for (int r = 0; r < 2; ++r) place_scales<FMT>(held[r], raw[r], sshift);
      }
      auto product = [&](uint32_t jj, const MoeQuad (&d)[2], auto odd) __attribute__((always_inline)) {
        const uint32_t qb = (kg * qpk + jj) * QC, left = qb < nblocks ? (nblocks - qb) * SB : 0u;
#pragma unroll
        for (int r = 0; r < 2; ++r)
          quad_product<FMT, XT, 1, decltype(odd)::value>(acc[r], d[r], held[r], jj % Sc::kQuads, left,
                                                         win + (jj % kPairQuads) * 512u, arow, apiece, tab, lane);
      };
      product(j, W0, std::integral_constant<int, 0>{});
      load_quad(j + 2, W0);
      if (j + 1 < qpk) product(j + 1, W1, std::integral_constant<int, 1>{});
      load_quad(j + 3, W1);
    }
    if (lane < 16) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float s = acc[r][0][0];  // all of D's rows are alike
        if constexpr (kTable) s *= 1.0f / kNf4Factor;
        sums[wave][r][lane] = s;
      }
    }
  }
  __syncthreads();
  if (kg == 0 && lane < 16 && (uint32_t)e < a.experts) {
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (uint32_t w = 0; w < (uint32_t)KW; ++w) {
      gate += sums[w * SL + sl][0][lane];
      up += sums[w * SL + sl][1][lane];
    }
    store_h(a, pair, tile * 16u + (uint32_t)lane, inter, gate, up);
    if (!__builtin_isfinite(gate) || !__builtin_isfinite(up)) settle_h<FMT, XT>(args_again(), e, pair, tile * 16u + (uint32_t)lane);
  }
}

template <int FMT, int XT, int KW>
hipError_t launch_moe_pair_one(const MoeArgs& a, uint32_t tokens, hipStream_t s) {
  constexpr uint32_t SL = 8 / KW;
  hipLaunchKernelGGL((moe_pair_kernel<FMT, XT, KW>), dim3(a.tiles / 2, tokens * ((a.top_k + SL - 1) / SL)),
                     dim3(kMoeThreads), 0, s, a);
  return hipGetLastError();
}

template <int XT>
hipError_t launch_moe_pair_weight(int weight, int kw, const MoeArgs& a, uint32_t tokens, hipStream_t s) {
#define W4_PAIR(F)                                                                    \
  case F:                                                                             \
    return kw == 1   ? launch_moe_pair_one<F, XT, 1>(a, tokens, s)                    \
           : kw == 2 ? launch_moe_pair_one<F, XT, 2>(a, tokens, s)                    \
           : kw == 4 ? launch_moe_pair_one<F, XT, 4>(a, tokens, s)                    \
           : kw == 8 ? launch_moe_pair_one<F, XT, 8>(a, tokens, s)                    \
                     : hipErrorInvalidValue;
  switch (weight) {
    W4_PAIR(kNF4)
    W4_PAIR(kINT4)
    W4_PAIR(kFP4)
    W4_PAIR(kINT4A)
    W4_PAIR(kMXFP4)
  }
#undef W4_PAIR
  return hipErrorInvalidValue;
}

// Down, combined in the same launch: 16 rows of y of one token, each wave the product with one of the
// token's experts (SL slots at a time), scaled by its routing weight and added up in LDS in a fixed order.
// No partial results in memory and no third launch.
constexpr uint32_t kTokenQuads = 6;  // quads of a wave's window

template <int FMT, int KW>
__global__ void __launch_bounds__(kMoeThreads, 4) moe_token_kernel(MoeArgs a) {
  constexpr uint32_t SL = 8 / KW;
  constexpr int KC = is_g128(FMT) ? 128 : 64;
  constexpr uint32_t QC = 256 / KC;
  constexpr bool kMX = FMT == kMXFP4;
  constexpr bool kTable = FMT == kNF4;
  constexpr uint32_t SB = FMT == kINT4 || kMX ? 2 : 4;
  using Sc = MoeScales<FMT>;
  __shared__ __align__(16) uint32_t tab[kTable ? kTableBytes / 4 : 4];
  __shared__ float sums[8][16];
  extern __shared__ __align__(16) uint8_t smem[];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t sl = (uint32_t)wave % SL, kg = (uint32_t)wave / SL;
  const int g = lane >> 4, m = lane & 15;
  const uint32_t token = blockIdx.y;
  const bool slot_lane = (uint32_t)lane < a.top_k;
  const int id = slot_lane ? a.ids[token * a.top_k + (uint32_t)lane] : -1;
  const float weight = slot_lane ? a.weights[token * a.top_k + (uint32_t)lane] : 0.0f;
  if constexpr (kTable) {
    fill_moe_table<kBF16>(tab);
    __syncthreads();
  }

  const uint32_t qpk = a.qpk;
  const uint32_t pitch = a.k >> 1;
  const uint32_t nblocks = a.k / KC;
  const uint32_t spitch = nblocks * SB;
  const uint32_t nchunks = a.k >> 5;
  const uint32_t per = min(qpk, kTokenQuads);  // quads of a window
  uint8_t* win = smem + (uint32_t)wave * (3u * per * 512u);
  const uint32_t chunk = (uint32_t)g + 4u * (uint32_t)(m >> 3);
  const uint32_t wlane = (uint32_t)(m & 7) * pitch + chunk * 16u;
  const uint32_t sshift = ((uint32_t)(lane >> 2) * spitch & 2u) * 8u;
  const uint32_t plane = (uint32_t)min(m, 2);  // A row m is plane m (rows 3 .. 15 repeat the last)
  const uint32_t arow[1] = {plane * (per * 512u)};
  const uint32_t piece = kMX ? g : is_g128(FMT) ? 4 * g : 4 * (g & 1) + 2 * (g >> 1);
  const uint32_t apiece[1] = {(piece ^ plane) * 16u};
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, 3u * a.pairs * a.k * 2u);
  const uint32_t tile = blockIdx.x;

  float y = 0.0f;  // lanes 0 .. 15: this wave's share of row 16 tile + lane
  float odd_sum = 0.0f;  // NaN: one of its products was not finite
  for (uint32_t slot = sl; slot < a.top_k; slot += SL) {
    const int e = __builtin_amdgcn_readlane(id, (int)slot);
    if ((uint32_t)e >= a.experts) continue;
    const size_t row0 = (size_t)e * a.n + tile * 16u;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.packed + row0 * pitch, 16u * pitch);
    const __amdgpu_buffer_rsrc_t rs =
        make_rsrc(reinterpret_cast<const char*>(a.scales) + row0 * spitch, 16u * spitch);
    auto load_quad = [&](uint32_t j, MoeQuad& d) __attribute__((always_inline)) {
      const uint32_t q = kg * qpk + j;
      const bool in = j < qpk && q * 8 + chunk < nchunks;
      const uint4 v0 = buffer_load16_stream(rw, offset_or_oob(in, wlane + q * 128u));
      const uint4 v1 = buffer_load16_stream(rw, offset_or_oob(in, wlane + q * 128u + 8u * pitch));
      d.w[0][0] = v0.x; d.w[0][1] = v0.y; d.w[0][2] = v0.z; d.w[0][3] = v0.w;
      d.w[1][0] = v1.x; d.w[1][1] = v1.y; d.w[1][2] = v1.z; d.w[1][3] = v1.w;
    };
    auto load_scales = [&](uint32_t j, Sc& d) __attribute__((always_inline)) {
      const uint32_t q = kg * qpk + j;
      const uint32_t at = (uint32_t)(lane >> 2) * spitch + (q + 2u * (uint32_t)(lane & 3)) * (QC * SB);
      load_scale_window<FMT>(d, rs, offset_or_oob(j < qpk && q * QC < nblocks, at & ~3u));
    };
    const uint32_t pair = token * a.top_k + slot;

    MoeQuad W0, W1;
    Sc held, next;
    float4_t acc[1] = {float4_t{0.f, 0.f, 0.f, 0.f}};
    for (uint32_t j0 = 0; j0 < qpk; j0 += per) {
      // The window: quads j0 .. j0 + per - 1 of this K range, 32 pieces of a plane's quad
      uint4 v[3][kTokenQuads / 2];
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (uint32_t i = 0; i < kTokenQuads / 2; ++i) {
          const uint32_t ql = 2u * i + (uint32_t)(lane >> 5), jq = j0 + ql;
          const uint32_t kpos = (kg * qpk + jq) * 256u + ((((uint32_t)lane & 31u) ^ (uint32_t)p) * 8u);
          if (2u * i < per)
            v[p][i] = buffer_load16(rx, offset_or_oob(ql < per && jq < qpk && kpos < a.k,
                                                      (((uint32_t)p * a.pairs + pair) * a.k + kpos) * 2u));
        }
      auto store_window = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (uint32_t i = 0; i < kTokenQuads / 2; ++i) {
            const uint32_t ql = 2u * i + (uint32_t)(lane >> 5);
            if (2u * i < per && ql < per)
              *reinterpret_cast<uint4*>(win + ((uint32_t)p * per + 2u * i) * 512u + (uint32_t)lane * 16u) = arranged<FMT>(v[p][i]);
          }
      };
      // (the stores stand in both branches: behind a join they would wait for the weights too)
      if (j0 == 0) {
        load_scales(0, next);
        load_quad(0, W0);
        load_quad(1, W1);
        store_window();
      } else {
        store_window();
      }
      const uint32_t end = min(qpk, j0 + per);
      for (uint32_t j = j0; j < end; j += 2) {
        if (j % Sc::kQuads == 0) {
          place_scales<FMT>(held, next, sshift);
          load_scales(j + Sc::kQuads, next);
        }
        auto product = [&](uint32_t jj, const MoeQuad& d, auto odd) __attribute__((always_inline)) {
          const uint32_t qb = (kg * qpk + jj) * QC;
          quad_product<FMT, kBF16, 1, decltype(odd)::value>(acc, d, held, jj % Sc::kQuads, qb < nblocks ? (nblocks - qb) * SB : 0u,
                                      win + (jj - j0) * 512u, arow, apiece, tab, lane);
        };
        product(j, W0, std::integral_constant<int, 0>{});
        load_quad(j + 2, W0);
        if (j + 1 < end) product(j + 1, W1, std::integral_constant<int, 1>{});
        load_quad(j + 3, W1);
      }
    }
    // rows 0, 1, 2 of D are the planes' products: lanes 0 .. 15, i = 0, 1, 2
    float v = acc[0][0] + (acc[0][1] + acc[0][2]);
    if constexpr (kTable) v *= 1.0f / kNf4Factor;
    watch(odd_sum, v);
    const float w = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(weight), (int)slot));
    y = __builtin_fmaf(w, v, y);
  }
  if (lane < 16 && odd_sum != odd_sum) {  // this wave's slots and K range once more
    const MoeArgs b = args_again();
    const uint32_t wave2 = threadIdx.x >> 6, k0 = min(b.k, wave2 / SL * b.qpk * 256u);
    y = 0.0f;
#pragma unroll 1
    for (uint32_t slot = wave2 % SL; slot < b.top_k; slot += SL) {
      const uint32_t pair = blockIdx.y * b.top_k + slot;
      const int e = b.ids[pair];
      if ((uint32_t)e < b.experts)
        y = __builtin_fmaf(b.weights[pair], defined_sum<FMT, kBF16, 3>(b, e, blockIdx.x * 16u + (uint32_t)lane, pair, k0,
                                                                       min(b.k, k0 + b.qpk * 256u)), y);
    }
  }
  if (lane < 16) sums[wave][lane] = y;
  __syncthreads();
  if (tid < 16) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sums[w][tid];
    a.y[(size_t)token * a.n + tile * 16u + (uint32_t)tid] = v;
  }
}

template <int FMT, int KW>
hipError_t launch_moe_token_one(const MoeArgs& a, uint32_t tokens, hipStream_t s) {
  constexpr uint32_t kMost = 8 * 3 * kTokenQuads * 512;
  static const hipError_t raised = hipFuncSetAttribute(reinterpret_cast<const void*>(&moe_token_kernel<FMT, KW>),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, kMost);
  if (raised != hipSuccess) return raised;
  const uint32_t per = a.qpk < kTokenQuads ? a.qpk : kTokenQuads;
  hipLaunchKernelGGL((moe_token_kernel<FMT, KW>), dim3(a.tiles, tokens), dim3(kMoeThreads), 8u * 3u * per * 512u, s, a);
  return hipGetLastError();
}

template <int DIR, int FMT, int XT, int NT, int KW>
hipError_t launch_moe_one(const MoeArgs& a, hipStream_t s) {
  constexpr uint32_t RT = 8 / KW, kSums = 2 * 8 * NT * 1024;
  // the limit on dynamic LDS, raised once per instantiation and process
  static const hipError_t raised = hipFuncSetAttribute(
      reinterpret_cast<const void*>(&moe_kernel<DIR, FMT, XT, NT, KW>),
      hipFuncAttributeMaxDynamicSharedMemorySize, kMoeMaxWindow + kSums);
  if (raised != hipSuccess) return raised;
  if (a.win_bytes > kMoeMaxWindow) return hipErrorInvalidValue;
  const uint32_t ngroups = (a.tiles + RT - 1) / RT;
  hipLaunchKernelGGL((moe_kernel<DIR, FMT, XT, NT, KW>), dim3(a.grid < ngroups ? a.grid : ngroups, a.experts),
                     dim3(kMoeThreads), a.win_bytes + kSums, s, a);
  return hipGetLastError();
}

template <int DIR, int FMT, int XT, int NT>
hipError_t launch_moe_kw(int kw, const MoeArgs& a, hipStream_t s) {
  switch (kw) {
    case 1: return launch_moe_one<DIR, FMT, XT, NT, 1>(a, s);
    case 2: return launch_moe_one<DIR, FMT, XT, NT, 2>(a, s);
    case 4: return launch_moe_one<DIR, FMT, XT, NT, 4>(a, s);
  }
  return hipErrorInvalidValue;
}

template <int DIR, int XT, int NT>
hipError_t launch_moe_weight(int weight, int kw, const MoeArgs& a, hipStream_t s) {
  switch (weight) {
    case kNF4: return launch_moe_kw<DIR, kNF4, XT, NT>(kw, a, s);
    case kINT4: return launch_moe_kw<DIR, kINT4, XT, NT>(kw, a, s);
    case kFP4: return launch_moe_kw<DIR, kFP4, XT, NT>(kw, a, s);
    case kINT4A: return launch_moe_kw<DIR, kINT4A, XT, NT>(kw, a, s);
    case kMXFP4: return launch_moe_kw<DIR, kMXFP4, XT, NT>(kw, a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace w4
