// Gated block for a few tokens: h = act(x Wg^T) * (x Wu^T) in one launch that streams the packed weights once.
//
// Work layout.  A workgroup of KW waves owns 16 channels: their 16 gate rows and 16 up rows.  K runs in units of 128
// weights; wave w takes units w, w + KW, ...  The matrix cores multiply 16 tokens by 16 rows by 32 k a step
// (16x16x32), the tokens as the A operand and the weights as B, so that a lane's results share one weight row and a
// block's scale, which the lane loaded itself, is applied in fp32 without any exchange:
//   * weights: lane 16 g + m loads bytes 16 g .. 16 g + 15 of the unit's 64 bytes of gate row m and of up row m, up to
//     four units ahead of the one multiplied.  Blocks of 64: two v_permlane32_swap give every lane 8 bytes of each of
//     the unit's two blocks (16 weights from 32 (g & 1) + 16 (g >> 1)); blocks of 32: one v_permlane16_swap more (8
//     weights from 8 g of each); groups of 128: as loaded (32 weights from 32 g);
//   * tokens: the same k of token m, 16 bytes a step straight from memory (a few rows, held by the caches), one unit
//     ahead;
//   * D: lane 16 g + m holds channel m of tokens 4 g .. 4 g + 3.
// Decoding: E2M1 by the hardware's conversion; INT4 and asymmetric INT4 as q - 8 and q - z, exact small integers,
// from the bytes by integer-to-float conversions (subtracting z x instead would turn infinities into NaN); NF4 by
// a byte -> pair table in LDS with each code as the sum of two 16-bit numbers (2^-18 of itself in bf16, 2^-22 in
// fp16; one fp16 number alone would be off by as much as the result's own rounding).
// The waves' sums are added in LDS in wave order: the same call gives the same bits.
#pragma once
#include "w4_ffn.h"
#include "w4_ffn_math.h"
#include "w4_mfma_common.h"

namespace w4 {

namespace {

constexpr int kFewAhead = 4;  // units of weights in flight

// One unit of one matrix in a lane: its 16 bytes, and the scales of its row's blocks in the unit.
struct FewWeights {
  uint32_t w[4], s[2];
};

// 8 weights of a packed dword as B operand: one or (NF4) two terms.
template <int FMT, int XT>
__device__ inline void few_decode(uint32_t w, const char* tab, uint32_t lane_off, float zero, uint4 (&o)[2]) {
  if constexpr (FMT == kNF4) {
    uint32_t a[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t at = __builtin_amdgcn_perm(w, lane_off, 0x0C0C0000u | ((4u + (uint32_t)j) << 8)) >> 1;
      const uint2 v = *reinterpret_cast<const uint2*>(tab + at);
      a[j] = v.x;
      b[j] = v.y;
    }
    o[0] = make_uint4(a[0], a[1], a[2], a[3]);
    o[1] = make_uint4(b[0], b[1], b[2], b[3]);
  } else if constexpr (FMT == kFP4 || FMT == kMXFP4) {
    const uint32_t v = ((w >> 4) & 0x0F0F0F0Fu) | ((w << 4) & 0xF0F0F0F0u);
    uint32_t a[4];
    if constexpr (XT == kF16) {
      a[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 0));
      a[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 1));
      a[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 2));
      a[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 3));
    } else {
      a[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 0));
      a[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 1));
      a[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 2));
      a[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 3));
    }
    o[0] = make_uint4(a[0], a[1], a[2], a[3]);
  } else {
    const uint32_t hi = (w >> 4) & 0x0F0F0F0Fu, lo = w & 0x0F0F0F0Fu;  // weights 2 j and 2 j + 1 in byte j
    uint32_t a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float e = (float)((hi >> (8 * j)) & 0xFFu) - zero, q = (float)((lo >> (8 * j)) & 0xFFu) - zero;
      if constexpr (XT == kF16)
        a[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(e, q));
      else
        a[j] = (__float_as_uint(e) >> 16) | (__float_as_uint(q) & 0xFFFF0000u);  // small integers: exact
    }
    o[0] = make_uint4(a[0], a[1], a[2], a[3]);
  }
}

// The byte -> two-term pairs table: 256 entries of 16 copies of (first terms, second terms), 8 bytes each.
template <int XT, int THREADS>
__device__ inline void few_table(uint32_t* tab) {
  const float c = __uint_as_float(codes_in_lanes<kNF4>());
  uint32_t v1, v2;
  if constexpr (XT == kF16) {
    v1 = f16_bits(c);
    v2 = f16_bits(c - (float)__builtin_bit_cast(_Float16, (uint16_t)v1));
  } else {
    v1 = bf16_rne_bits(c);
    v2 = bf16_rne_bits(c - __uint_as_float(v1 << 16));
  }
  uint4* t4 = reinterpret_cast<uint4*>(tab);
  const int tid = threadIdx.x;
#pragma unroll 4
  for (int i = tid; i < kTableBytes / 16; i += THREADS) {  // slot i: entry i >> 3
    const int hi = i >> 7, lo = (i >> 3) & 15;
    const uint32_t p1 = (uint32_t)__shfl((int)v1, hi) | ((uint32_t)__shfl((int)v1, lo) << 16);
    const uint32_t p2 = (uint32_t)__shfl((int)v2, hi) | ((uint32_t)__shfl((int)v2, lo) << 16);
    t4[i] = make_uint4(p1, p2, p1, p2);
  }
}

template <int FMT, int XT, int NT, int KW>
__global__ void __launch_bounds__(64 * KW) gated_few_kernel(GatedFewArgs p) {
  constexpr bool kTab = FMT == kNF4, kMX = FMT == kMXFP4;
  constexpr int TERMS = kTab ? 2 : 1;
  constexpr int STEPS = is_g128(FMT) ? 4 : kMX ? 1 : 2;  // matrix steps of a scale block
  constexpr int RED = KW * 2 * NT * 64 * 16;
  __shared__ __align__(16) uint8_t smem[kTab && kTableBytes > RED ? kTableBytes : RED];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, m = lane & 15;
  const uint32_t c0 = blockIdx.x * 16u;
  const uint32_t k = p.k, pitch = k / 2, units = (k + 127) / 128;
  const uint32_t nblocks = k / (is_g128(FMT) ? 128u : 64u);
  const uint32_t spitch = nblocks * (FMT == kINT4 || kMX ? 2u : 4u);
  const uint32_t rows = min(16u, p.inter - c0);
  const size_t r0[2] = {c0, (size_t)p.inter + c0};
  __amdgpu_buffer_rsrc_t rw[2], rs[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    rw[q] = make_rsrc(p.packed + r0[q] * pitch, rows * pitch);
    rs[q] = make_rsrc(reinterpret_cast<const uint8_t*>(p.scales) + r0[q] * spitch, rows * spitch);
  }
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x, p.t * k * 2u);

  auto load_weights = [&](uint32_t u, FewWeights (&d)[2]) __attribute__((always_inline)) {
    const uint32_t at = u * 64 + g * 16;
    const uint32_t off = offset_or_oob(at < pitch, (uint32_t)m * pitch + at);
    const uint32_t so = (uint32_t)m * spitch;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 v = buffer_load16_stream(rw[q], off);
      d[q].w[0] = v.x, d[q].w[1] = v.y, d[q].w[2] = v.z, d[q].w[3] = v.w;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if constexpr (FMT == kINT4) {
        d[q].s[0] = buffer_load16bit(rs[q], offset_or_oob(u < units, so + u * 2));
      } else if constexpr (FMT == kINT4A) {
        d[q].s[0] = buffer_load32(rs[q], offset_or_oob(u < units, so + u * 4));
      } else if constexpr (kMX) {  // two bytes a 64-weight block: rows of them are 2-byte aligned
        d[q].s[0] = buffer_load16bit(rs[q], offset_or_oob(2 * u < nblocks, so + u * 4));
        d[q].s[1] = buffer_load16bit(rs[q], offset_or_oob(2 * u + 1 < nblocks, so + u * 4 + 2));
      } else {
        d[q].s[0] = buffer_load32(rs[q], offset_or_oob(2 * u < nblocks, so + u * 8));
        d[q].s[1] = buffer_load32(rs[q], offset_or_oob(2 * u + 1 < nblocks, so + u * 8 + 4));
      }
    }
  };
  uint32_t xrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xrow[t] = min((uint32_t)(16 * t + m), p.t - 1) * k;  // rows past T repeat the last
  auto load_x = [&](uint32_t u, uint4 (&x)[NT][4]) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t kk = u * 128 + (is_g128(FMT) ? 32 * g + 8 * s
                                     : kMX        ? 32 * s + 8 * g
                                                  : 64 * (s >> 1) + 32 * (g & 1) + 16 * (g >> 1) + 8 * (s & 1));
#pragma unroll
      for (int t = 0; t < NT; ++t) x[t][s] = buffer_load16(rx, offset_or_oob(kk < k, (xrow[t] + kk) * 2));
    }
  };

  float4_t acc[2][NT];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[q][t] = float4_t{0.f, 0.f, 0.f, 0.f};
  const char* tab = reinterpret_cast<const char*>(smem);
  const uint32_t lane_off = (uint32_t)m * 16u;  // twice the copy's offset, see few_decode

  auto compute = [&](const FewWeights (&d)[2], const uint4 (&x)[NT][4]) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t w[4];  // the dwords of matrix steps 0 .. 3
      float s[4];     // their scales
      float zero = 8.0f;
      if constexpr (is_g128(FMT)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = d[q].w[j];
        s[0] = __uint_as_float(d[q].s[0] << 16);
        if constexpr (FMT == kINT4A) zero = (float)((d[q].s[0] >> 16) & 15u);
      } else {
        const auto a = __builtin_amdgcn_permlane32_swap(d[q].w[0], d[q].w[2], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(d[q].w[1], d[q].w[3], false, false);
        w[0] = a[0], w[1] = b[0], w[2] = a[1], w[3] = b[1];
        if constexpr (kMX) {
          const auto e = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
          const auto f = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
          w[0] = e[0], w[1] = e[1], w[2] = f[0], w[3] = f[1];
#pragma unroll
          for (int j = 0; j < 4; ++j) s[j] = e8m0_value((d[q].s[j >> 1] >> (8 * (j & 1))) & 255u);
        } else {
          s[0] = __uint_as_float(d[q].s[0]);
          s[1] = __uint_as_float(d[q].s[1]);
        }
      }
#pragma unroll
      for (int b = 0; b < 4 / STEPS; ++b) {
        float4_t dd[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) dd[t] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
          uint4 o[2];
          few_decode<FMT, XT>(w[STEPS * b + j], tab, lane_off, zero, o);
#pragma unroll
          for (int term = 0; term < TERMS; ++term)
#pragma unroll
            for (int t = 0; t < NT; ++t) dd[t] = mfma<XT>(x[t][STEPS * b + j], o[term], dd[t]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[q][t][i] = __builtin_fmaf(dd[t][i], s[b], acc[q][t][i]);
      }
    }
  };

  // Weights first, then the table, then the tokens: what takes longest to come is asked for first.
  FewWeights d[kFewAhead][2];
  uint4 x[2][NT][4];
#pragma unroll
  for (int j = 0; j < kFewAhead; ++j) load_weights(wave + j * KW, d[j]);
  load_x(wave, x[0]);
  if constexpr (kTab) {
    few_table<XT, 64 * KW>(reinterpret_cast<uint32_t*>(smem));
    __syncthreads();
  }
  for (uint32_t u = wave; u < units; u += kFewAhead * KW) {
#pragma unroll
    for (int j = 0; j < kFewAhead; ++j) {
      const uint32_t v = u + j * KW;
      if (v < units) {  // uniform
        load_x(v + KW, x[(j + 1) & 1]);
        compute(d[j], x[j & 1]);
        load_weights(v + kFewAhead * KW, d[j]);
      }
    }
  }

  // The waves' sums: [wave][matrix][tile][lane], added by as many threads as there are results.
  __syncthreads();
  float4_t* red = reinterpret_cast<float4_t*>(smem);
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[((wave * 2 + q) * NT + t) * 64 + lane] = acc[q][t];
  __syncthreads();
  for (int at = tid; at < NT * 256; at += 64 * KW) {  // element i of lane l of tile t
    const int t = at >> 8, i = (at >> 6) & 3, l = at & 63;
    const float* f = reinterpret_cast<const float*>(red);
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      gate += f[(((w * 2 + 0) * NT + t) * 64 + l) * 4 + i];
      up += f[(((w * 2 + 1) * NT + t) * 64 + l) * 4 + i];
    }
    const uint32_t token = 16 * t + 4 * (l >> 4) + i, channel = c0 + (l & 15);
    if (token < p.t && channel < p.inter) {
      const float y = p.act == W4_ACT_SILU ? act_value<W4_ACT_SILU>(gate) : act_value<W4_ACT_GELU_TANH>(gate);
      p.h[(size_t)token * p.inter + channel] = (uint16_t)to16<XT>(y * up);
      if (p.products) {
        uint16_t* o = p.products + (size_t)token * 2 * p.inter + channel;
        o[0] = (uint16_t)to16<XT>(gate);
        o[p.inter] = (uint16_t)to16<XT>(up);
      }
    }
  }
}

template <int FMT, int XT, int NT>
hipError_t few_launch(const GatedFewArgs& a, hipStream_t s) {
  const dim3 grid((a.inter + 15) / 16);
  if ((a.k + 127) / 128 >= 16)
    gated_few_kernel<FMT, XT, NT, 8><<<grid, dim3(512), 0, s>>>(a);
  else
    gated_few_kernel<FMT, XT, NT, 4><<<grid, dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <int XT>
hipError_t few_dispatch(int weight, const GatedFewArgs& a, hipStream_t s) {
#define W4_FEW(F)                                                                    \
  case F:                                                                            \
    return a.t <= 16 ? few_launch<F, XT, 1>(a, s) : few_launch<F, XT, 2>(a, s);
  switch (weight) {
    W4_FEW(kNF4)
    W4_FEW(kINT4)
    W4_FEW(kFP4)
    W4_FEW(kINT4A)
    default: W4_FEW(kMXFP4)
  }
#undef W4_FEW
}

}  // namespace

}  // namespace w4
