// 8-bit products for a few tokens: y[t, n] = s_t s_n sum_k x[t, k] w[n, k] with the weights streamed once, straight
// into the matrix cores' registers.
//
// Work layout.  A workgroup of KW waves owns 16 rows (gated: 16 gate rows and the 16 up rows of the same channels); K
// runs in steps of 64, wave w takes steps w, w + KW, ...  One matrix step multiplies 16 tokens by 16 rows by 64 k
// (i32_16x16x64_i8): tokens are the A operand, lane 16 g + m holding 16 consecutive codes of token m, weights B, the
// same codes of row m.  Both come from memory as they are, 16 bytes a lane, kAhead steps ahead; the rows of the few
// tokens stay in the caches.  D: lane 16 g + m holds row m, tokens 4 g .. 4 g + 3.  The waves' int32 sums are added
// in LDS (exact in any order).
#pragma once
#include "w4_dense.h"

namespace w4 {
namespace {

constexpr int kAhead = 4;

template <bool GATED, int NT, int KW>
__global__ void __launch_bounds__(64 * KW) int8_few_kernel(DenseArgs p) {
  constexpr int R = GATED ? 2 : 1;
  __shared__ __align__(16) i32x4 red[KW * R * NT * 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, m = lane & 15;
  const uint32_t c0 = blockIdx.x * 16u, k = p.pitch, steps = k / 64;
  const uint32_t rows = min(16u, p.n - c0);
  __amdgpu_buffer_rsrc_t rw[R];
#pragma unroll
  for (int q = 0; q < R; ++q) rw[q] = make_rsrc(p.b + ((size_t)q * p.n + c0) * k, rows * k);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.a, p.m * k);
  const uint32_t woff = (uint32_t)m * k + 16 * g;
  uint32_t xoff[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xoff[t] = min((uint32_t)(16 * t + m), p.m - 1) * k + 16 * g;  // rows past M repeat the last

  struct Step {
    uint4 w[R], x[NT];
  };
  auto load = [&](uint32_t st, Step& d) __attribute__((always_inline)) {
    const bool have = st < steps;
#pragma unroll
    for (int q = 0; q < R; ++q) d.w[q] = buffer_load16_stream(rw[q], offset_or_oob(have, woff + st * 64));
#pragma unroll
    for (int t = 0; t < NT; ++t) d.x[t] = buffer_load16(rx, offset_or_oob(have, xoff[t] + st * 64));
  };
  i32x4 acc[R][NT];
#pragma unroll
  for (int q = 0; q < R; ++q)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[q][t] = i32x4{0, 0, 0, 0};
  Step d[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) load(wave + j * KW, d[j]);
  for (uint32_t st = wave; st < steps; st += kAhead * KW) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {  // steps past the last multiply zeros
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[q][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, d[j].x[t]),
                                                            __builtin_bit_cast(i32x4, d[j].w[q]), acc[q][t], 0, 0, 0);
      load(st + (kAhead + j) * KW, d[j]);
    }
  }
#pragma unroll
  for (int q = 0; q < R; ++q)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[((wave * R + q) * NT + t) * 64 + lane] = acc[q][t];
  __syncthreads();
  const int* f = reinterpret_cast<const int*>(red);
  for (int at = tid; at < NT * 256; at += 64 * KW) {  // element i of lane l of tile t
    const int t = at >> 8, i = (at >> 6) & 3, l = at & 63;
    const uint32_t token = 16 * t + 4 * (l >> 4) + i, n = c0 + (l & 15);
    if (token >= p.m || n >= p.n) continue;
    const float rs = p.row_scale[token];
    float v[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < KW; ++w) sum += f[(((w * R + q) * NT + t) * 64 + l) * 4 + i];
      v[q] = (float)sum * rs * p.col_scale[q * p.n + n];
    }
    auto store = [&](void* out, size_t o, float y) __attribute__((always_inline)) {
      if (p.out_type == W4_F32)
        reinterpret_cast<float*>(out)[o] = y;
      else
        reinterpret_cast<uint16_t*>(out)[o] = (uint16_t)(p.out_type == W4_F16 ? to16<kF16>(y) : to16<kBF16>(y));
    };
    if constexpr (GATED) {
      const float y = p.act == W4_ACT_SILU ? act_value<W4_ACT_SILU>(v[0]) : act_value<W4_ACT_GELU_TANH>(v[0]);
      store(p.out, (size_t)token * p.n + n, y * v[1]);
      if (p.products) {
        store(p.products, (size_t)token * 2 * p.n + n, v[0]);
        store(p.products, (size_t)token * 2 * p.n + p.n + n, v[1]);
      }
    } else {
      store(p.out, (size_t)token * p.n + n, v[0]);
    }
  }
}

template <bool GATED, int NT>
hipError_t int8_few_launch(const DenseArgs& a, hipStream_t s) {
  const dim3 grid((a.n + 15) / 16);
  if (a.pitch / 64 >= 16)
    int8_few_kernel<GATED, NT, 8><<<grid, dim3(512), 0, s>>>(a);
  else
    int8_few_kernel<GATED, NT, 4><<<grid, dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace
}  // namespace w4
