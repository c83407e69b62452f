// Activations of the gated block, and what its kernels share.
//   silu(g)      = g p,  p = 1 / (1 + exp(-g));        silu'(g) = p (1 + g (1 - p))
//   gelu_tanh(g) = g / 2 (1 + tanh(v)) = g p,  p = 1 / (1 + exp(-2 v)),  v = sqrt(2/pi) (g + 0.044715 g^3);
//                  gelu_tanh'(g) = p + g 2 v' p (1 - p),  v' = sqrt(2/pi) (1 + 3 * 0.044715 g^2)
// The logistic form has no difference of near-equal numbers where tanh is close to -1.  exp and the reciprocal
// are the hardware's (a few units of 2^-24, times |g| for exp; p below 2^-126 reads 0): the results are rounded to
// 16 bits.
#pragma once
#include "w4_common.h"

namespace w4 {
namespace {

__device__ inline float logistic(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }

// 2 v(g) and its derivative.  g is held to +-30 (where p is 0 or 1 in fp32), so that g^3 stays in range and
// p (1 - p) = 0 meets a finite factor; a NaN passes.
__device__ inline float gelu_arg(float g, float* slope) {
  const float c = g > 30.0f ? 30.0f : g < -30.0f ? -30.0f : g;
  *slope = 1.5957691216057308f * (1.0f + 0.134145f * c * c);
  return 1.5957691216057308f * (c + 0.044715f * c * c * c);
}

template <int ACT>
__device__ inline float act_value(float g) {
  if constexpr (ACT == W4_ACT_SILU) {
    return g * logistic(g);
  } else {
    float d;
    return g * logistic(gelu_arg(g, &d));
  }
}

// act(g), and act'(g) in *slope.
template <int ACT>
__device__ inline float act_slope(float g, float* slope) {
  if constexpr (ACT == W4_ACT_SILU) {
    const float p = logistic(g);
    *slope = p * (1.0f + g * (1.0f - p));
    return g * p;
  } else {
    float d;
    const float p = logistic(gelu_arg(g, &d));
    *slope = p + g * (p * (1.0f - p)) * d;  // in this order: g d alone may leave the range
    return g * p;
  }
}

// 16-bit values as fp32 and back (to nearest, ties to even).
template <int XT>
__device__ inline float from16(uint32_t bits) {
  if constexpr (XT == kF16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  return __uint_as_float(bits << 16);
}
template <int XT>
__device__ inline uint32_t to16(float v) {
  if constexpr (XT == kF16) return __builtin_bit_cast(uint16_t, (_Float16)v);
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Two values as bf16 in a dword, one instruction.
__device__ inline uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), bf2));
}

// a * s and b * t, rounded to fp32 and to fp16, in a dword.
__device__ inline uint32_t scaled_pair(float a, float b, float s, float t) {
  uint32_t d;
  asm("v_fma_mixlo_f16 %0, %1, %2, 0" : "=v"(d) : "v"(a), "v"(s));
  asm("v_fma_mixhi_f16 %0, %1, %2, 0" : "+v"(d) : "v"(b), "v"(t));
  return d;
}
__device__ inline uint32_t scaled_pair(float a, float b, float s) { return scaled_pair(a, b, s, s); }

// a * s and b * t less h, rounded the same way, h the fp16 halves of a dword.
__device__ inline uint32_t rest_of_pair(float a, float b, float s, float t, uint32_t h) {
  uint32_t d;
  asm("v_fma_mixlo_f16 %0, %1, %2, -%3 op_sel_hi:[0,0,1]" : "=v"(d) : "v"(a), "v"(s), "v"(h));
  asm("v_fma_mixhi_f16 %0, %1, %2, -%3 op_sel:[0,0,1] op_sel_hi:[0,0,1]" : "+v"(d) : "v"(b), "v"(t), "v"(h));
  return d;
}
__device__ inline uint32_t rest_of_pair(float a, float b, float s, uint32_t h) { return rest_of_pair(a, b, s, s, h); }

// Two fp16 terms of a weight w = code * s: the first is rounded from code * first_term(s), which is w less 2^-10 of it,
// the second from what that leaves of w.  It leaves 2^-11 to 1.5 * 2^-10 of w: so both have the weight's sign and neither
// is 0 unless the weight is (or lies more than 2^28 below fp16's largest), and an infinite activation gives what it gives
// with the weight itself.  The second is off by at most half its step, 2^-20.4 of w.
__device__ inline float first_term(float s) { return s * (1.0f - 0x1p-10f); }

// The 16-bit terms of an NF4 code in a gated launch, two fp16 or three bf16 ones: each but the last is what is left cut
// towards zero (and one step short of it where it would be held whole), so that all have the code's sign and none is 0
// unless the code is: an infinite activation then gives what it gives with the code itself.  bf16: the sum is the code
// (24 bits); fp16: it is off by at most 2^-21 of it.
template <int XT>
__device__ inline uint32_t signed_term(float c) {
  uint32_t v;
  if constexpr (XT == kF16) {
    v = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(c, 0.0f)) & 0xFFFFu;
    if (c != 0.0f && (float)__builtin_bit_cast(_Float16, (uint16_t)v) == c) v -= 1;
  } else {
    v = __float_as_uint(c) >> 16;
    if (c != 0.0f && __uint_as_float(v << 16) == c) v -= 1;
  }
  return v;
}
template <int XT>
__device__ inline void signed_terms(float c, uint32_t& v1, uint32_t& v2, uint32_t& v3) {
  v1 = signed_term<XT>(c);
  const float r = c - from16<XT>(v1);
  if constexpr (XT == kF16) {
    v2 = to16<kF16>(r);
    v3 = 0;
  } else {
    v2 = signed_term<kBF16>(r);
    v3 = to16<kBF16>(r - __uint_as_float(v2 << 16));
  }
}

// A block's scale as fp32 from its stored form (INT4A: the low half of its word).
template <int FMT>
__device__ inline float scale_of(const void* scales, size_t i) {
  if constexpr (FMT == kNF4 || FMT == kFP4) return reinterpret_cast<const float*>(scales)[i];
  if constexpr (FMT == kINT4) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(scales)[i] << 16);
  if constexpr (FMT == kINT4A) return __uint_as_float(reinterpret_cast<const uint32_t*>(scales)[i] << 16);
  return e8m0_value(reinterpret_cast<const uint8_t*>(scales)[i]);
}
template <int FMT>
constexpr int weights_per_scale() { return is_g128(FMT) ? 128 : FMT == kMXFP4 ? 32 : 64; }

// A block's scale and what its codes' offset is (INT4 8, asymmetric INT4 its zero point).
struct BlockScale {
  float s, zero;
};
template <int FMT>
__device__ inline BlockScale block_scale(const void* scales, size_t i) {
  BlockScale b;
  b.s = scale_of<FMT>(scales, i);
  b.zero = FMT == kINT4A ? (float)((reinterpret_cast<const uint32_t*>(scales)[i] >> 16) & 15u) : 8.0f;
  return b;
}

// The fp32 codes of NF4, by the first sixteen threads of a workgroup (other formats need none).
template <int FMT>
__device__ inline void code_table(float* table) {
  constexpr uint32_t kn[16] = W4_NF4_CODE_BITS;
  if (FMT == kNF4 && threadIdx.x < 16) {
    uint32_t bits = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) bits = (int)threadIdx.x == q ? kn[q] : bits;
    table[threadIdx.x] = __uint_as_float(bits);
  }
}

// The two weights of byte j of a packed dword in fp32, code times scale, the high nibble's (the earlier k) first:
// NF4 through the table, E2M1 by the hardware's conversion, integers less their offset (exact) times the scale.
template <int FMT>
__device__ inline void decode_pair(uint32_t v, int j, const float* table, BlockScale b, float* first, float* second) {
  if constexpr (FMT == kNF4) {
    *first = table[(v >> (8 * j + 4)) & 15u] * b.s;
    *second = table[(v >> (8 * j)) & 15u] * b.s;
  } else if constexpr (FMT == kFP4 || FMT == kMXFP4) {
    const auto c = j == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 0)
                   : j == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 1)
                   : j == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 2)
                            : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 3);
    *first = c[1] * b.s;
    *second = c[0] * b.s;
  } else {
    *first = ((float)((v >> (8 * j + 4)) & 15u) - b.zero) * b.s;
    *second = ((float)((v >> (8 * j)) & 15u) - b.zero) * b.s;
  }
}

// Exponent e with s c 2^-e in [2^14, 2^15), c the largest code of the format: fp16's highest binade but one.  What lies
// within 2^28 below s c is a normal number then; smaller weights are off by at most half of fp16's smallest step, 2^-25,
// which is 2^-39 of s c at most.
template <int FMT>
__device__ inline int fold_exponent(float s) {
  constexpr float c = FMT == kNF4 ? 1.0f : FMT == kINT4 ? 8.0f : FMT == kINT4A ? 15.0f : 6.0f;
  if (!(s > 0.0f)) return 0;
  const int e = ilogbf(s);
  return e + ilogbf(ldexpf(s, -e) * c) - 14;  // (s c itself may leave the range)
}

__device__ inline float wave_max(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// The exponent of unit `unit` (of `units`) of columns from the scan's maxima, by a wave.
template <int FMT>
__device__ inline int unit_exponent(const float* parts, uint32_t nparts, uint32_t units, uint32_t unit, int lane) {
  float top = 0.0f;
  if (unit < units)
    for (uint32_t i = lane; i < nparts; i += 64) top = fmaxf(top, parts[(size_t)i * units + unit]);
  return fold_exponent<FMT>(wave_max(top));
}

}  // namespace
}  // namespace w4
