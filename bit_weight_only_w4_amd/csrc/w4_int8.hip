// 8-bit rows: the quantizer (the products are launches of the dense kernel, w4_dense.h).
//
// A row's scale is s = fp32(max|x| / 127) and its codes q = rint(x / s), ties to even, held to +-127 (a subnormal
// scale may be rounded so far down that the quotient passes 127).  The nearest integer of the exact quotient:
// c = rint(x * (1/s)) is off by at most one; the sign of x - (c +- 1/2) s, one fused multiply-add whose single
// rounding keeps the sign, then says whether the border was crossed.  A row that holds an infinity or NaN gets
// scale NaN and codes 0, so its products are NaN.
#include "w4_ffn.h"
#include "w4_ffn_math.h"

namespace w4 {
namespace {

// 8 consecutive values of a row as fp32.  TYPE 0 fp32, 1 fp16, 2 bf16.
template <int TYPE, bool ALIGNED>
__device__ inline void load8(const void* x, size_t at, uint32_t left, float (&v)[8]) {
  if constexpr (ALIGNED) {
    if constexpr (TYPE == 0) {
      const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + at);
      const float4 a = q[0], b = q[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + at);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = from16<TYPE == 1 ? kF16 : kBF16>(w[j] & 0xFFFFu);
        v[2 * j + 1] = from16<TYPE == 1 ? kF16 : kBF16>(w[j] >> 16);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if ((uint32_t)j < left) {
        if constexpr (TYPE == 0)
          v[j] = reinterpret_cast<const float*>(x)[at + j];
        else
          v[j] = from16<TYPE == 1 ? kF16 : kBF16>(reinterpret_cast<const uint16_t*>(x)[at + j]);
      }
    }
  }
}

__device__ inline int code_of(float x, float s, float inv) {
  float c = rintf(x * inv);
  const float over = __builtin_fmaf(-(c + 0.5f), s, x), under = __builtin_fmaf(-(c - 0.5f), s, x);
  const bool odd = ((int)c & 1) != 0;
  // past the upper border, or on it where the even neighbour is the upper one; the lower border alike
  c += over > 0.0f || (over == 0.0f && odd) ? 1.0f : under < 0.0f || (under == 0.0f && odd) ? -1.0f : 0.0f;
  return (int)fminf(fmaxf(c, -127.0f), 127.0f);
}

// A row by a workgroup of THREADS; HOLD chunks of 8 values stay in a thread's registers between the pass for the
// maximum and the pass that writes the codes, what is beyond them is read again.
template <int TYPE, bool ALIGNED, int THREADS, int HOLD>
__global__ void __launch_bounds__(THREADS) quantize_int8_kernel(const void* x, uint32_t k, int8_t* codes,
                                                                float* scales) {
  const size_t row = blockIdx.x, base = row * (size_t)k;
  const uint32_t chunks = (k + 7) / 8, tid = threadIdx.x;
  float v[HOLD][8];
  float top = 0.0f;
  bool bad = false;
  auto fold = [&](const float(&w)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(w[j]);
      bad |= !(a < __builtin_inff());
      top = fmaxf(top, a);
    }
  };
#pragma unroll
  for (int i = 0; i < HOLD; ++i) {
    const uint32_t ch = tid + i * THREADS;
    if (ch < chunks) {
      load8<TYPE, ALIGNED>(x, base + (size_t)ch * 8, k - ch * 8, v[i]);
      fold(v[i]);
    }
  }
  for (uint32_t ch = tid + HOLD * THREADS; ch < chunks; ch += THREADS) {
    float w[8];
    load8<TYPE, ALIGNED>(x, base + (size_t)ch * 8, k - ch * 8, w);
    fold(w);
  }
  top = bad ? __builtin_inff() : top;
  top = wave_max(top);
  if constexpr (THREADS > 64) {
    __shared__ float part[THREADS / 64];
    if ((tid & 63) == 0) part[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) top = fmaxf(top, part[i]);
  }
  bad = !(top < __builtin_inff());
  const float s = bad ? __builtin_nanf("") : top / 127.0f;
  if (tid == 0) scales[row] = s;
  const bool none = bad || s == 0.0f;
  // A subnormal s may have no reciprocal in fp32: those few rows divide in fp64, exactly decided as well (a
  // quotient of 24-bit numbers that is no border is at least 2^-33 of itself away from one).
  const bool tiny = s < 0x1p-120f;
  const float inv = 1.0f / s;
  auto put = [&](const float(&w)[8], uint32_t ch) __attribute__((always_inline)) {
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      int q = 0;
      if (!none) q = tiny ? (int)fmin(fmax(rint((double)w[j] / (double)s), -127.0), 127.0) : code_of(w[j], s, inv);
      o[j >> 2] |= ((uint32_t)q & 255u) << (8 * (j & 3));
    }
    int8_t* to = codes + base + (size_t)ch * 8;
    if constexpr (ALIGNED) {
      *reinterpret_cast<uint2*>(to) = make_uint2(o[0], o[1]);
    } else {
      for (uint32_t j = 0; j < 8 && ch * 8 + j < k; ++j) to[j] = (int8_t)(o[j >> 2] >> (8 * (j & 3)));
    }
  };
#pragma unroll
  for (int i = 0; i < HOLD; ++i) {
    const uint32_t ch = tid + i * THREADS;
    if (ch < chunks) put(v[i], ch);
  }
  for (uint32_t ch = tid + HOLD * THREADS; ch < chunks; ch += THREADS) {
    float w[8];
    load8<TYPE, ALIGNED>(x, base + (size_t)ch * 8, k - ch * 8, w);
    put(w, ch);
  }
}

template <int TYPE, bool ALIGNED>
void quantize_rows(const void* x, int64_t rows, int64_t k, int8_t* codes, float* scales, hipStream_t s) {
  if (k <= 1024)
    quantize_int8_kernel<TYPE, ALIGNED, 64, 2><<<dim3((uint32_t)rows), dim3(64), 0, s>>>(x, (uint32_t)k, codes, scales);
  else
    quantize_int8_kernel<TYPE, ALIGNED, 256, 5><<<dim3((uint32_t)rows), dim3(256), 0, s>>>(x, (uint32_t)k, codes,
                                                                                          scales);
}

template <int TYPE>
void quantize_typed(const void* x, int64_t rows, int64_t k, int8_t* codes, float* scales, hipStream_t s) {
  const bool aligned = k % 8 == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)codes % 8 == 0;
  if (aligned)
    quantize_rows<TYPE, true>(x, rows, k, codes, scales, s);
  else
    quantize_rows<TYPE, false>(x, rows, k, codes, scales, s);
}

}  // namespace

hipError_t launch_quantize_int8(int type, const void* x, int64_t rows, int64_t k, int8_t* codes, float* scales,
                                hipStream_t s) {
  if (type == 0)
    quantize_typed<0>(x, rows, k, codes, scales, s);
  else if (type == 1)
    quantize_typed<1>(x, rows, k, codes, scales, s);
  else
    quantize_typed<2>(x, rows, k, codes, scales, s);
  return hipGetLastError();
}

}  // namespace w4
