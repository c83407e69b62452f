// 8-bit rows: the quantizer (the products are launches of the dense kernel, w4_dense.h).
//
// A row's scale is s = fp32(max|x| / 127) and its codes q = rint(x / s), ties to even, held to +-127 (a subnormal
// scale may be rounded so far down that the quotient passes 127).  The nearest integer of the exact quotient:
// c = rint(x * (1/s)) is right unless x * (1/s) lies next to a border between two integers, and then off by at most one;
// the sign of x - (c +- 1/2) s, one fused multiply-add whose single rounding keeps the sign, says whether the border was
// crossed.  A row that holds an infinity or NaN gets
// scale NaN and codes 0, so its products are NaN.
#include <algorithm>
#include <type_traits>

#include "w4_ffn.h"
#include "w4_ffn_math.h"

namespace w4 {
namespace {

// 8 consecutive values of a row as fp32, zeros past the `left` that it still has.  TYPE a w4_type_t.
template <int TYPE>
__device__ inline void load8(const void* x, size_t at, uint32_t left, float (&v)[8]) {
  if constexpr (TYPE == W4_F32) {
    const float* from = reinterpret_cast<const float*>(x) + at;
    if (left >= 8) {
      __builtin_memcpy(v, from, 32);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (uint32_t)j < left ? from[j] : 0.0f;
    }
  } else {
    constexpr int XT = TYPE == W4_F16 ? kF16 : kBF16;
    const uint16_t* from = reinterpret_cast<const uint16_t*>(x) + at;
    uint16_t w[8];
    if (left >= 8) {
      __builtin_memcpy(w, from, 16);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = (uint32_t)j < left ? from[j] : (uint16_t)0;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = from16<XT>(w[j]);
  }
}

// x * (1/s) is within 127 * 2^-23 of the quotient: an integer that is nearer to it than this is the quotient's nearest too.
constexpr float kNear = 0.5f - 0x1p-15f;

// The code of x from c, the nearest integer of x * (1/s).
__device__ inline float code_at_border(float x, float s, float c) {
  const float over = __builtin_fmaf(-(c + 0.5f), s, x), under = __builtin_fmaf(-(c - 0.5f), s, x);
  const bool odd = ((int)c & 1) != 0;
  // past the upper border, or on it where the even neighbour is the upper one; the lower border alike
  return c + (over > 0.0f || (over == 0.0f && odd) ? 1.0f : under < 0.0f || (under == 0.0f && odd) ? -1.0f : 0.0f);
}

// A row by a workgroup of THREADS; HOLD chunks of 8 values stay in a thread's registers between the pass for the
// maximum and the pass that writes the codes, what is beyond them is read again.  Two or four bytes read and one written a
// value bound it (65536 x 1024 bf16 45 us, 4.5 TB/s; 4096 x 8192 26 us, 3.8 TB/s), once the border test is left to the
// few chunks that need it (with it for every value: 54 and 32 us).
template <int TYPE, int THREADS, int HOLD>
__global__ void __launch_bounds__(THREADS) quantize_int8_kernel(const void* x, uint32_t k, int8_t* codes,
                                                                float* scales) {
  const size_t row = blockIdx.x, base = row * (size_t)k;
  const uint32_t chunks = (k + 7) / 8, tid = threadIdx.x;
  float v[HOLD][8];
  uint32_t most = 0;  // the largest magnitude's bits: above every finite one for infinities and NaN
  auto fold = [&](const float(&w)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(w[j]) & 0x7FFFFFFFu);
  };
#pragma unroll
  for (int i = 0; i < HOLD; ++i) {
    const uint32_t ch = tid + i * THREADS;
    if (ch < chunks) {
      load8<TYPE>(x, base + (size_t)ch * 8, k - ch * 8, v[i]);
      fold(v[i]);
    }
  }
  for (uint32_t ch = tid + HOLD * THREADS; ch < chunks; ch += THREADS) {
    float w[8];
    load8<TYPE>(x, base + (size_t)ch * 8, k - ch * 8, w);
    fold(w);
  }
  float top = wave_max(__uint_as_float(min(most, 0x7F800000u)));
  if constexpr (THREADS > 64) {
    __shared__ float part[THREADS / 64];
    if ((tid & 63) == 0) part[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) top = fmaxf(top, part[i]);
  }
  const bool bad = !(top < __builtin_inff());
  const float s = bad ? __builtin_nanf("") : top / 127.0f;
  if (tid == 0) scales[row] = s;
  const bool none = bad || s == 0.0f;
  // A subnormal s may have no reciprocal in fp32: those few rows divide in fp64, exactly decided as well (a
  // quotient of 24-bit numbers that is no border is at least 2^-33 of itself away from one).
  const bool tiny = s < 0x1p-120f;
  const float inv = 1.0f / s;
  auto put = [&](const float(&w)[8], uint32_t ch) __attribute__((always_inline)) {
    float c[8], far = 0.0f;  // how far the quotients are from integers
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = w[j] * inv;
      c[j] = rintf(v);
      far = fmaxf(far, fabsf(v - c[j]));
    }
    if (none) {
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = 0.0f;
    } else if (tiny) {
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = (float)fmin(fmax(rint((double)w[j] / (double)s), -127.0), 127.0);
    } else if (far > kNear) {
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = code_at_border(w[j], s, c[j]);
    }
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j >> 2] |= ((uint32_t)(int)c[j] & 255u) << (8 * (j & 3));
    int8_t* to = codes + base + (size_t)ch * 8;
    if (ch * 8 + 8 <= k) {
      __builtin_memcpy(to, o, 8);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (ch * 8 + j < k) to[j] = (int8_t)(o[j >> 2] >> (8 * (j & 3)));
    }
  };
#pragma unroll
  for (int i = 0; i < HOLD; ++i) {
    const uint32_t ch = tid + i * THREADS;
    if (ch < chunks) put(v[i], ch);
  }
  for (uint32_t ch = tid + HOLD * THREADS; ch < chunks; ch += THREADS) {
    float w[8];
    load8<TYPE>(x, base + (size_t)ch * 8, k - ch * 8, w);
    put(w, ch);
  }
}

template <int TYPE>
void quantize_typed(const void* x, int64_t rows, int64_t k, int8_t* codes, float* scales, hipStream_t s) {
  auto run = [&](auto threads, auto hold) {
    constexpr int T = decltype(threads)::value, H = decltype(hold)::value;
    quantize_int8_kernel<TYPE, T, H><<<dim3((uint32_t)rows), dim3(T), 0, s>>>(x, (uint32_t)k, codes, scales);
  };
  using std::integral_constant;
  // Microseconds (bf16) with 64, 256 and 1024 threads: 4096 x 512 4.5, 6.4, 17.0; 4096 x 1536 7.9, 8.4, 18.5; 1024 x 1536
  // 5.5, 4.1, 6.3; 4096 x 2048 10.8, 10.0, 19.5; 4096 x 8192 34.8, 26.3, 30.3; 512 x 8192 18.1, 7.0, 6.3; 1 x 8192 10.5,
  // 4.5, 3.3; 1 x 1536 3.4, 2.9, 2.8.
  if (k <= 1536 && rows >= 2048)
    run(integral_constant<int, 64>{}, integral_constant<int, 3>{});
  else if (k <= 2048 || rows > 512)
    run(integral_constant<int, 256>{}, integral_constant<int, 5>{});
  else
    run(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
}

}  // namespace

hipError_t launch_quantize_int8(int type, const void* x, int64_t rows, int64_t k, int8_t* codes, float* scales,
                                hipStream_t s) {
  const int64_t most = (int64_t)1 << 23;  // a launch has fewer than 2^32 threads
  for (int64_t first = 0; first < rows; first += most) {
    const int64_t r = std::min(rows - first, most);
    const uint8_t* from = reinterpret_cast<const uint8_t*>(x) + first * k * (type == W4_F32 ? 4 : 2);
    if (type == W4_F32)
      quantize_typed<W4_F32>(from, r, k, codes + first * k, scales + first, s);
    else if (type == W4_F16)
      quantize_typed<W4_F16>(from, r, k, codes + first * k, scales + first, s);
    else
      quantize_typed<W4_BF16>(from, r, k, codes + first * k, scales + first, s);
  }
  return hipGetLastError();
}

}  // namespace w4
