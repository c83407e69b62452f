// Input gradient of a product with frozen 4-bit weights: dx[t, k] = sum_n d[t, n] W_hat[n, k].
//
// The sum runs over the weight rows, along which a packed byte holds nothing: the weights are decoded once into
// W_hat^T rows of 16 bits in the workspace (through LDS, 64 x 64 weights a workgroup), which the dense kernel
// multiplies with d.  A weight is rounded once to d's type (2^-8 of itself in bf16, 2^-11 in fp16; fp16 with one
// exponent for the whole matrix, taken from its largest scale, so that neither large nor small weights leave its
// range).  Rows of W_hat^T are padded with zeros to whole steps of the dense kernel, and so is d where its rows do
// not end on one or are not aligned.
#include <algorithm>

#include "w4_ffn.h"
#include "w4_ffn_math.h"

namespace w4 {
namespace {

constexpr int kTile = 64;       // weights of a tile along either axis
constexpr int kMaxParts = 256;  // workgroups of the scale scan

template <int FMT>
__global__ void __launch_bounds__(256) scale_max_kernel(const void* scales, int64_t count, float* parts) {
  float top = 0.0f;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const float s = fabsf(scale_of<FMT>(scales, (size_t)i));
    top = s < __builtin_inff() ? fmaxf(top, s) : top;
  }
  __shared__ float w[4];
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) parts[blockIdx.x] = fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3]));
}

struct TransposeArgs {
  const uint8_t* packed;  // [N, K/2]
  const void* scales;
  uint16_t* wt;           // [K, NP] of d's type
  uint32_t n, k, np;
  const float* parts;     // the scan's maxima, null for bf16
  uint32_t nparts;
  int* exp;               // the exponent that they give
};

template <int FMT, int XT>
__global__ void __launch_bounds__(256) transpose_kernel(TransposeArgs p) {
  constexpr uint32_t G = weights_per_scale<FMT>();
  constexpr uint32_t kn[16] = W4_NF4_CODE_BITS;
  constexpr uint32_t kf[16] = W4_FP4_CODE_BITS;
  __shared__ float table[16];
  __shared__ uint16_t tile[kTile][kTile + 2];  // [k][n]
  const int tid = threadIdx.x;
  if (tid < 16) {
    uint32_t bits = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) bits = tid == q ? (FMT == kNF4 ? kn[q] : kf[q]) : bits;
    table[tid] = is_g128(FMT) ? (float)(tid - 8) : __uint_as_float(bits);
  }
  int f = 0;
  if constexpr (XT == kF16) {  // every wave for itself: at most 256 values
    float top = 0.0f;
    for (uint32_t i = tid & 63; i < p.nparts; i += 64) top = fmaxf(top, p.parts[i]);
    f = fold_exponent<FMT>(wave_max(top));
    if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) *p.exp = f;
  }
  __syncthreads();
  const uint32_t n0 = blockIdx.x * kTile, k0 = blockIdx.y * kTile;
  {
    const uint32_t r = tid >> 2, part = tid & 3;  // row of the tile, 16 weights of it
    const uint32_t n = n0 + r, k = k0 + part * 16;
    if (n < p.n) {
      const uint2 v = *reinterpret_cast<const uint2*>(p.packed + ((size_t)n * p.k + k) / 2);
      const size_t at = (size_t)n * (p.k / G) + k / G;
      const float s = ldexpf(scale_of<FMT>(p.scales, at), -f);
      float shift = 0.0f;
      if constexpr (FMT == kINT4A)
        shift = 8.0f - (float)((reinterpret_cast<const uint32_t*>(p.scales)[at] >> 16) & 15u);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        tile[part * 16 + j][r] = (uint16_t)to16<XT>((table[nibble(j < 8 ? v.x : v.y, j & 7)] + shift) * s);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) tile[part * 16 + j][r] = 0;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t k = (uint32_t)(tid >> 3) + 32u * i, c = tid & 7;
    uint32_t o[4];
    __builtin_memcpy(o, &tile[k][c * 8], 16);
    *reinterpret_cast<uint4*>(p.wt + (size_t)(k0 + k) * p.np + n0 + c * 8) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// d's rows padded with zeros: [B, N] -> [B, NP].
__global__ void __launch_bounds__(256) pad_kernel(const uint16_t* d, uint16_t* to, uint32_t n, uint32_t np) {
  const uint32_t c = blockIdx.x * 256 + threadIdx.x;
  if (c >= np) return;
  const size_t t = blockIdx.y;
  to[t * np + c] = c < n ? d[t * n + c] : (uint16_t)0;
}

constexpr int kFewTokens = 64;

// Splits of N for a few tokens: as many as give every CU a workgroup of 128 columns, each at least a step of 32 rows
// for each of its eight waves.
uint32_t few_splits(int64_t n, int64_t k) {
  const int64_t groups = (k + 127) / 128, rounds = ((n + 31) / 32 + 7) / 8;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(rounds, device_cu_count() / groups));
  const int64_t per = (rounds + want - 1) / want;  // rounds a split
  return (uint32_t)((rounds + per - 1) / per);
}

size_t up16(size_t v) { return (v + 15) & ~(size_t)15; }

struct GradSpace {
  uint32_t np;
  size_t wt, d, parts, exp, partial, bytes;
};
GradSpace grad_space(int64_t n, int64_t k, int64_t b) {
  GradSpace g;
  g.np = (uint32_t)((n + kTile - 1) / kTile * kTile);
  g.wt = 0;
  g.d = up16((size_t)k * g.np * 2);
  g.parts = g.d + up16((size_t)b * g.np * 2);
  g.exp = g.parts + kMaxParts * 4;
  g.partial = g.exp + 16;
  g.bytes = g.partial + up16(dense_bytes(false, b, k, (int64_t)g.np * 2));
  return g;
}

template <int FMT>
hipError_t prepare(int xt, const uint8_t* packed, const void* scales, int64_t n, int64_t k, uint8_t* ws,
                   const GradSpace& g, hipStream_t s) {
  TransposeArgs p;
  p.packed = packed;
  p.scales = scales;
  p.wt = reinterpret_cast<uint16_t*>(ws + g.wt);
  p.n = (uint32_t)n;
  p.k = (uint32_t)k;
  p.np = g.np;
  p.parts = reinterpret_cast<const float*>(ws + g.parts);
  p.exp = reinterpret_cast<int*>(ws + g.exp);
  p.nparts = 0;
  const dim3 grid(g.np / kTile, (uint32_t)(k / kTile));
  if (xt == kF16) {
    const int64_t count = n * (k / weights_per_scale<FMT>());
    p.nparts = (uint32_t)std::min<int64_t>(kMaxParts, (count + 1023) / 1024);
    scale_max_kernel<FMT><<<dim3(p.nparts), dim3(256), 0, s>>>(scales, count, reinterpret_cast<float*>(ws + g.parts));
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    transpose_kernel<FMT, kF16><<<grid, dim3(256), 0, s>>>(p);
  } else {
    transpose_kernel<FMT, kBF16><<<grid, dim3(256), 0, s>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

size_t gemm_grad_workspace(int, int64_t n, int64_t k, int64_t b) {
  if (b <= kFewTokens) {
    const uint32_t splits = few_splits(n, k);
    return splits > 1 ? up16((size_t)splits * (size_t)(b * k) * 4) : 0;
  }
  return grad_space(n, k, b).bytes;
}

hipError_t launch_gemm_grad(int fmt, const uint16_t* d, const uint8_t* packed, const void* scales, int64_t n, int64_t k,
                            int64_t b, uint16_t* dx, void* ws, hipStream_t s) {
  const int xt = fmt_xtype(fmt);
  if (b <= kFewTokens) {
    const uint32_t splits = few_splits(n, k), steps = (uint32_t)((n + 31) / 32);
    const GradFewArgs f{d, packed, scales, dx, splits > 1 ? reinterpret_cast<float*>(ws) : nullptr,
                        (uint32_t)n, (uint32_t)k, (uint32_t)b, (steps + splits - 1) / splits};
    return xt == kF16 ? launch_grad_few_f16(fmt_weight(fmt), f, splits, s)
                      : launch_grad_few_bf16(fmt_weight(fmt), f, splits, s);
  }
  const GradSpace g = grad_space(n, k, b);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  hipError_t e;
  switch (fmt_weight(fmt)) {
    case kNF4: e = prepare<kNF4>(xt, packed, scales, n, k, base, g, s); break;
    case kINT4: e = prepare<kINT4>(xt, packed, scales, n, k, base, g, s); break;
    case kFP4: e = prepare<kFP4>(xt, packed, scales, n, k, base, g, s); break;
    case kINT4A: e = prepare<kINT4A>(xt, packed, scales, n, k, base, g, s); break;
    default: e = prepare<kMXFP4>(xt, packed, scales, n, k, base, g, s); break;
  }
  if (e != hipSuccess) return e;
  if ((int64_t)g.np != n || (uintptr_t)d % 16) {
    uint16_t* pad = reinterpret_cast<uint16_t*>(base + g.d);
    pad_kernel<<<dim3((g.np + 255) / 256, (uint32_t)b), dim3(256), 0, s>>>(d, pad, (uint32_t)n, g.np);
    if (e = hipGetLastError(); e != hipSuccess) return e;
    d = pad;
  }
  DenseArgs a{};
  a.a = reinterpret_cast<const uint8_t*>(d);
  a.b = base + g.wt;
  a.m = (uint32_t)b;
  a.n = (uint32_t)k;
  a.pitch = g.np * 2;
  a.exp = xt == kF16 ? reinterpret_cast<const int*>(base + g.exp) : nullptr;
  a.partial = reinterpret_cast<uint32_t*>(base + g.partial);
  a.out = dx;
  a.out_type = xt == kF16 ? 1 : 2;
  return launch_dense(xt == kF16 ? kDenseF16 : kDenseBF16, false, a, s);
}

}  // namespace w4
