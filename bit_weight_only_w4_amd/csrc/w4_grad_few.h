// Input gradient of a 4-bit product for a few tokens: dx[t, k] = sum_n d[t, n] W_hat[n, k], the packed weights
// streamed once and decoded in registers.
//
// Work layout.  A workgroup of eight waves owns 128 columns; N runs in steps of 32 rows, wave w of split z takes every
// eighth step of the split.  The sum runs along the rows, so an operand of the matrix cores (16x16x32) needs eight
// consecutive rows of one column in a lane, while a packed dword holds eight columns of one row.  Lane 16 g + m
// therefore loads the dwords of columns 8 m .. 8 m + 7 of rows 8 g .. 8 g + 7 and runs eight products: product j has
// column 8 m + j where it says column m.  No exchange between lanes, and a lane ends with eight consecutive columns of
// tokens 4 g .. 4 g + 3.
//   * Scales: lane 16 g + m loads one, of row 8 g + (m & 7) and the column half m >> 3 (groups of 128: of the row;
//     blocks of 32: the two bytes of that half); lane r of each half row hands it to the others when row r is decoded.
//   * A weight enters as the sum of bf16 numbers, which have fp32's range, so that no common exponent is needed: MXFP4
//     one (exact), INT4 two (exact, at most 12 bits), NF4 and FP4 three (2^-21).  Every term but the last is rounded from
//     what is left less 2^-7 of it: so all have the weight's sign and none is 0 unless the weight is, and an infinite
//     gradient gives what it gives with the weight itself.  fp16 gradients are the sum of two bf16 numbers (exact); of
//     the products of terms the one below 2^-20 of the whole is left out.
//   * Bound by decoding: a weight of three terms takes some ten vector instructions, of two seven.  16 bf16 tokens of
//     28672 x 4096, in all: NF4 55 us (1.2 TB/s), FP4 46, INT4 38, MXFP4 31; small ones also by the chain of loads of a few
//     steps and the splits' sums: NF4 1536 x 8960 11.3 us (0.7 TB/s) and 1.7 for the sum.
//   * The waves' sums are added in LDS, the splits' by a second kernel, both in a fixed order.
#pragma once
#include <type_traits>

#include "w4_ffn.h"
#include "w4_ffn_math.h"
#include "w4_mfma_common.h"

namespace w4 {
namespace {

constexpr int kGradWaves = 8;

struct GradStep {
  uint32_t w[8], s;
};

template <int FMT, int XT, int NT>
__global__ void __launch_bounds__(64 * kGradWaves) grad_few_kernel(GradFewArgs p) {
  constexpr bool kMX = FMT == kMXFP4;
  constexpr int TERMS = kMX ? 1 : is_g128(FMT) ? 2 : 3;  // of a weight
  constexpr float kLess = 1.0f - 0x1p-7f;
  __shared__ __align__(16) float4_t red[kGradWaves * 8 * 64];
  __shared__ float table[FMT == kNF4 ? 16 * 64 : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, m = lane & 15;
  // Every eighth workgroup runs on one XCD: those take neighbouring columns, whose 64 bytes of a row share cache lines
  // (16 tokens FP4 28672 x 4096 49 to 47 us, 17920 x 1536 23.0 to 22.2, NF4 1536 x 8960 14.3 to 13.3).
  const uint32_t groups = (p.k + 127) / 128, share = gridDim.x / 8, rem = gridDim.x % 8, xcd = blockIdx.x % 8;
  const uint32_t wg = xcd * share + min(xcd, rem) + blockIdx.x / 8, split = wg / groups;
  const uint32_t k0 = (wg - split * groups) * 128u, k = p.k, n = p.n, pitch = k / 2;
  constexpr uint32_t G = weights_per_scale<FMT>();
  constexpr uint32_t SB = FMT == kINT4 ? 2 : kMX ? 1 : 4;
  const uint32_t spitch = k / G * SB;
  const uint32_t steps = (n + 31) / 32;
  const uint32_t first = split * p.per, last = min(first + p.per, steps);

  const bool have = k0 + 8 * m < k;
  uint32_t woff[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) woff[r] = offset_or_oob(have, (8 * g + r) * pitch + k0 / 2 + 4 * m);
  // the scale's column: of the half m >> 3 (64 columns), or of the whole group
  const uint32_t scol = is_g128(FMT) ? k0 / 128 : kMX ? k0 / 32 + 2 * (m >> 3) : k0 / 64 + (m >> 3);
  const uint32_t soff = offset_or_oob(scol * G < k, (uint32_t)(8 * g + (m & 7)) * spitch + scol * SB);
  auto load_step = [&](uint32_t st, GradStep& d) __attribute__((always_inline)) {
    const uint32_t n0 = st * 32, rows = st < last ? min(32u, n - n0) : 0u;
    const size_t at = st < last ? n0 : 0;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.packed + at * pitch, rows * pitch);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(reinterpret_cast<const uint8_t*>(p.scales) + at * spitch, rows * spitch);
#pragma unroll
    for (int r = 0; r < 8; ++r) d.w[r] = buffer_load32(rw, woff[r]);
    d.s = FMT == kINT4 || kMX ? buffer_load16bit(rs, soff) : buffer_load32(rs, soff);
  };
  // d of token m of a tile: eight rows' values, zero past N.
  auto load_d = [&](uint32_t st, uint4 (&d)[NT]) __attribute__((always_inline)) {
    const uint32_t n0 = st * 32 + 8 * g;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint16_t* row = p.d + (size_t)min((uint32_t)(16 * t + m), p.b - 1) * n;
      uint32_t v[4] = {0, 0, 0, 0};
      if (st < last && n0 + 8 <= n) {
        __builtin_memcpy(v, row + n0, 16);
      } else if (st < last) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (n0 + j < n) v[j >> 1] |= (uint32_t)row[n0 + j] << (16 * (j & 1));
      }
      d[t] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  };

  const char* codes = reinterpret_cast<const char*>(table);
  float4_t acc[NT][8];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[t][j] = float4_t{0.f, 0.f, 0.f, 0.f};

  // The scale of row r of this lane's eight (as stored), from the lane that loaded it.
  auto scale_bits = [&](uint32_t s, auto r) __attribute__((always_inline)) {
    const uint32_t lo = __float_as_uint(row_bcast<decltype(r)::value>(s));
    if constexpr (is_g128(FMT)) return lo;
    const uint32_t hi = __float_as_uint(row_bcast<8 + decltype(r)::value>(s));
    return m < 8 ? lo : hi;
  };
  auto compute = [&](const GradStep& st, const uint4 (&d)[NT]) __attribute__((always_inline)) {
    uint4 dh[NT], dl[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if constexpr (XT == kBF16) {
        dh[t] = d[t];
      } else {
        const uint32_t v[4] = {d[t].x, d[t].y, d[t].z, d[t].w};
        uint32_t a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = from16<kF16>(v[j] & 0xFFFFu), y = from16<kF16>(v[j] >> 16);
          a[j] = bf16_pair(x, y);
          // at most 3 bits; none of an infinity or NaN
          const float xl = fabsf(x) < __builtin_inff() ? x - __uint_as_float(a[j] << 16) : 0.0f;
          const float yl = fabsf(y) < __builtin_inff() ? y - __uint_as_float(a[j] & 0xFFFF0000u) : 0.0f;
          b[j] = (__float_as_uint(xl) >> 16) | (__float_as_uint(yl) & 0xFFFF0000u);
        }
        dh[t] = make_uint4(a[0], a[1], a[2], a[3]);
        dl[t] = make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
    float s[8], o[8], s1[8];  // scales, the offsets of integer codes, and the first term's scales
    auto one = [&](auto r) __attribute__((always_inline)) {
      constexpr int R = decltype(r)::value;
      const uint32_t bits = scale_bits(st.s, r);
      o[R] = 8.0f;
      if constexpr (kMX) {
        s[R] = e8m0_value((bits >> (2 * (m & 4))) & 255u);
      } else if constexpr (is_g128(FMT)) {
        s[R] = __uint_as_float(bits << 16);
        if constexpr (FMT == kINT4A) o[R] = (float)((bits >> 16) & 15u);
      } else {
        s[R] = __uint_as_float(bits);
      }
      s1[R] = TERMS > 1 ? s[R] * kLess : s[R];
    };
    one(std::integral_constant<int, 0>{});
    one(std::integral_constant<int, 1>{});
    one(std::integral_constant<int, 2>{});
    one(std::integral_constant<int, 3>{});
    one(std::integral_constant<int, 4>{});
    one(std::integral_constant<int, 5>{});
    one(std::integral_constant<int, 6>{});
    one(std::integral_constant<int, 7>{});
#pragma unroll
    for (int b = 0; b < 4; ++b) {  // byte b: columns 2 b (high nibble) and 2 b + 1
      float w[2][8];  // codes, integers less their offset
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const uint32_t v = st.w[r];
        if constexpr (FMT == kNF4) {
          // byte offsets of a code's 64 copies, then of this lane's
          const uint32_t hi = (b < 1 ? v << 4 : v >> (8 * b - 4)) & 0xF00u, lo = (b < 1 ? v << 8 : v >> (8 * b - 8)) & 0xF00u;
          w[0][r] = *reinterpret_cast<const float*>(codes + (hi | (4u * lane)));
          w[1][r] = *reinterpret_cast<const float*>(codes + (lo | (4u * lane)));
        } else {
          decode_pair<FMT>(v, b, nullptr, BlockScale{1.0f, o[r]}, &w[0][r], &w[1][r]);
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t h[4], m2[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = 2 * i;
          const float x = w[q][j], y = w[q][j + 1];
          h[i] = bf16_pair(x * s1[j], y * s1[j + 1]);
          if constexpr (TERMS > 1) {
            const float xl = __builtin_fmaf(x, s[j], -__uint_as_float(h[i] << 16));
            const float yl = __builtin_fmaf(y, s[j + 1], -__uint_as_float(h[i] & 0xFFFF0000u));
            if constexpr (TERMS == 2) {
              m2[i] = bf16_pair(xl, yl);  // exact
            } else {
              m2[i] = bf16_pair(xl * kLess, yl * kLess);
              l[i] = bf16_pair(xl - __uint_as_float(m2[i] << 16), yl - __uint_as_float(m2[i] & 0xFFFF0000u));
            }
          }
        }
        const uint4 oh = make_uint4(h[0], h[1], h[2], h[3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float4_t& c = acc[t][2 * b + q];
          if constexpr (TERMS == 3) c = mfma<kBF16>(dh[t], make_uint4(l[0], l[1], l[2], l[3]), c);
          if constexpr (TERMS > 1) {
            const uint4 om = make_uint4(m2[0], m2[1], m2[2], m2[3]);
            if constexpr (XT == kF16) c = mfma<kBF16>(dl[t], om, c);
            c = mfma<kBF16>(dh[t], om, c);
          }
          if constexpr (XT == kF16) c = mfma<kBF16>(dl[t], oh, c);
          c = mfma<kBF16>(dh[t], oh, c);
        }
      }
    }
  };
  GradStep sa, sb;
  uint4 da[NT], db[NT];
  uint32_t st = first + wave;
  load_step(st, sa);
  load_d(st, da);
  load_step(st + kGradWaves, sb);
  load_d(st + kGradWaves, db);
  if constexpr (FMT == kNF4) {
    const float c = __uint_as_float(codes_in_lanes<kNF4>());
    for (int i = wave; i < 16; i += kGradWaves) table[i * 64 + lane] = __shfl(c, i);
    __syncthreads();
  }
  for (; st < last; st += 2 * kGradWaves) {
    compute(sa, da);
    load_step(st + 2 * kGradWaves, sa);
    load_d(st + 2 * kGradWaves, da);
    if (st + kGradWaves < last) {
      compute(sb, db);
      load_step(st + 3 * kGradWaves, sb);
      load_d(st + 3 * kGradWaves, db);
    }
  }

  // A tile at a time: [wave][product][lane]; then half a token's group of eight columns a thread.
  const float* f = reinterpret_cast<const float*>(red);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) red[(wave * 8 + j) * 64 + lane] = acc[t][j];
    __syncthreads();
    const int half = tid & 1, column = (tid >> 1) & 15, token = tid >> 5;  // 16 tokens
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kGradWaves; ++w)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += f[((w * 8 + 4 * half + j) * 64 + (token >> 2) * 16 + column) * 4 + (token & 3)];
    const uint32_t row = 16 * t + token, col = k0 + 8 * column + 4 * half;
    if (row < p.b && col < k) {
      if (p.partial) {
        float* to = p.partial + ((size_t)split * p.b + row) * k + col;
        *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
        uint16_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = (uint16_t)to16<XT>(v[j]);
        __builtin_memcpy(p.dx + (size_t)row * k + col, o, 8);
      }
    }
  }
}

template <int XT>
__global__ void __launch_bounds__(256) grad_sum_kernel(const float* partial, uint16_t* dx, int64_t count, uint32_t splits) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (uint32_t s = 0; s < splits; ++s) {
    const float4 q = *reinterpret_cast<const float4*>(partial + (int64_t)s * count + i);
    v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
  }
  const uint16_t o[4] = {(uint16_t)to16<XT>(v.x), (uint16_t)to16<XT>(v.y), (uint16_t)to16<XT>(v.z),
                         (uint16_t)to16<XT>(v.w)};
  __builtin_memcpy(dx + i, o, 8);
}

template <int FMT, int XT>
hipError_t grad_few_launch(const GradFewArgs& a, uint32_t splits, hipStream_t s) {
  const dim3 grid((a.k + 127) / 128 * splits), block(64 * kGradWaves);
  if (a.b <= 16)
    grad_few_kernel<FMT, XT, 1><<<grid, block, 0, s>>>(a);
  else if (a.b <= 32)
    grad_few_kernel<FMT, XT, 2><<<grid, block, 0, s>>>(a);
  else if constexpr (grad_few_most(FMT, XT) > 32)
    grad_few_kernel<FMT, XT, 4><<<grid, block, 0, s>>>(a);
  else
    return hipErrorInvalidValue;
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const int64_t count = (int64_t)a.b * a.k;
  grad_sum_kernel<XT><<<dim3((uint32_t)((count / 4 + 255) / 256)), dim3(256), 0, s>>>(a.partial, a.dx, count, splits);
  return hipGetLastError();
}

template <int XT>
hipError_t grad_few_dispatch(int weight, const GradFewArgs& a, uint32_t splits, hipStream_t s) {
  switch (weight) {
    case kNF4: return grad_few_launch<kNF4, XT>(a, splits, s);
    case kINT4: return grad_few_launch<kINT4, XT>(a, splits, s);
    case kFP4: return grad_few_launch<kFP4, XT>(a, splits, s);
    case kINT4A: return grad_few_launch<kINT4A, XT>(a, splits, s);
    default: return grad_few_launch<kMXFP4, XT>(a, splits, s);
  }
}

}  // namespace
}  // namespace w4
