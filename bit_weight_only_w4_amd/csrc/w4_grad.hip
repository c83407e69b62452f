// Input gradient of a product with frozen 4-bit weights: dx[t, k] = sum_n d[t, n] W_hat[n, k].
//
// The sum runs over the weight rows, along which a packed byte holds nothing: the weights are decoded once into W_hat^T
// rows of 16 bits in the workspace (through LDS), which the dense kernel multiplies with d, or, where that costs less, the
// dense kernel decodes and transposes them as they arrive (PackedColumns in w4_dense_sources.h).  A weight is rounded
// once to d's type (2^-8 of itself in bf16, 2^-11 in fp16; fp16 with one exponent for the whole matrix, taken from its
// largest scale, so that neither large nor small weights leave its range).  Rows of W_hat^T are padded with zeros to whole
// steps of the dense kernel, and so is d where its rows do not end on one or are not aligned.
#include <algorithm>
#include <type_traits>

#include "w4_ffn.h"
#include "w4_ffn_math.h"

namespace w4 {
namespace {

constexpr int kTile = 64;       // weight rows of a tile
constexpr int kMaxParts = 256;  // workgroups of the scale scan

template <int FMT>
__device__ inline void scale_max(const void* scales, int64_t count, float* parts, uint32_t workgroups) {
  float top = 0.0f;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)workgroups * 256) {
    const float s = fabsf(scale_of<FMT>(scales, (size_t)i));
    top = s < __builtin_inff() ? fmaxf(top, s) : top;
  }
  __shared__ float w[4];
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) parts[blockIdx.x] = fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3]));
}

// A row of d, zeros after its end up to `np`.
__device__ inline void pad_row(const uint16_t* from, uint16_t* to, uint32_t n, uint32_t np) {
  for (uint32_t c = threadIdx.x * 8; c < np; c += 256 * 8) {
    uint32_t v[4] = {0, 0, 0, 0};
    if (c + 8 <= n) {
      __builtin_memcpy(v, from + c, 16);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j)
        if (c + j < n) v[j >> 1] |= (uint32_t)from[c + j] << (16 * (j & 1));
    }
    *reinterpret_cast<uint4*>(to + c) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// What the product that decodes the weights itself needs before it: the scales' maxima (fp16; `parts` workgroups), and d
// with whole rows in the workgroups after those.
template <int FMT>
__global__ void __launch_bounds__(256) ready_kernel(const void* scales, int64_t count, float* maxima, uint32_t parts,
                                                    const uint16_t* d, uint16_t* padded, uint32_t n, uint32_t np) {
  if (blockIdx.x >= parts) {
    const size_t t = blockIdx.x - parts;
    pad_row(d + t * n, padded + t * np, n, np);
    return;
  }
  scale_max<FMT>(scales, count, maxima, parts);
}

struct TransposeArgs {
  const uint8_t* packed;  // [N, K/2]
  const void* scales;
  uint16_t* wt;           // [K, NP] of d's type
  uint32_t n, k, np;
  const float* parts;     // the scan's maxima, null for bf16
  uint32_t nparts;
  int* exp;               // the exponent that they give
  uint32_t tiles;         // workgroups that transpose; those after them copy d
  const uint16_t* d;      // [B, N]
  uint16_t* padded;       // [B, NP]
};

// A tile of 64 rows x 256 columns a workgroup, whole cache lines of the packed rows: a thread decodes 32 columns of two
// rows, writes them to LDS as pairs along n, and stores 16 bytes of rows of W_hat^T.  In LDS column 32 part + j is at
// row 8 j + part of 40 dwords: the 64 pairs that a wave writes at once then lie in 64 banks (27.5 million weights: 17 us,
// 4 TB/s).  Neighbouring workgroups
// take neighbouring rows, whose pieces of W_hat^T are one after another.
constexpr int kColumns = 256;

template <int FMT, int XT>
__global__ void __launch_bounds__(256) transpose_kernel(TransposeArgs p) {
  constexpr uint32_t G = weights_per_scale<FMT>();
  constexpr int PITCH = 40;
  const uint32_t tid = threadIdx.x;
  if (blockIdx.x >= p.tiles) {  // a row of d, zeros after its end
    const size_t t = blockIdx.x - p.tiles;
    pad_row(p.d + t * p.n, p.padded + t * p.np, p.n, p.np);
    return;
  }
  __shared__ float table[16];
  __shared__ __align__(16) uint32_t tile[kColumns * PITCH];
  const uint32_t along = p.np / kTile;
  const uint32_t n0 = blockIdx.x % along * kTile, k0 = blockIdx.x / along * kColumns;
  const uint32_t rp = tid >> 3, part = tid & 7;  // rows n0 + 2 rp and the next, columns k0 + 32 part ..
  const uint32_t kt = k0 + 32 * part;
  uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  BlockScale s[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t n = n0 + 2 * rp + q;
    if (n < p.n && kt < p.k) {
      v[q] = *reinterpret_cast<const uint4*>(p.packed + ((size_t)n * p.k + kt) / 2);
      s[q] = block_scale<FMT>(p.scales, (size_t)n * (p.k / G) + kt / G);
    }
  }
  code_table<FMT>(table);
  if constexpr (XT == kF16) {  // every wave for itself: at most 256 values
    float top = 0.0f;
    for (uint32_t i = tid & 63; i < p.nparts; i += 64) top = fmaxf(top, p.parts[i]);
    const int f = fold_exponent<FMT>(wave_max(top));
    if (tid == 0 && blockIdx.x == 0) *p.exp = f;
    s[0].s = ldexpf(s[0].s, -f);
    s[1].s = ldexpf(s[1].s, -f);
  }
  __syncthreads();
  const uint32_t w0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, w1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float a[2], b[2];  // rows past N have scale 0 and finite codes: zeros
    decode_pair<FMT>(w0[j >> 2], j & 3, table, s[0], &a[0], &a[1]);
    decode_pair<FMT>(w1[j >> 2], j & 3, table, s[1], &b[0], &b[1]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      tile[(8 * (2 * j + q) + part) * PITCH + rp] = to16<XT>(a[q]) | (to16<XT>(b[q]) << 16);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t k = (tid >> 3) + 32u * i, c = tid & 7;
    const uint4 o = *reinterpret_cast<const uint4*>(tile + (8 * (k & 31) + (k >> 5)) * PITCH + 4 * c);
    if (k0 + k < p.k) *reinterpret_cast<uint4*>(p.wt + (size_t)(k0 + k) * p.np + n0 + c * 8) = o;
  }
}

// How many tokens take the packed weights decoded in registers (w4_grad_few.h).  Microseconds there / by the dense
// kernel decoding them itself:
//                   4096 x 4096   28672 x 4096   896 x 4864
//   32  FP4 bf16    14.0 / 15.5     37 / 47     10.7 / 15.5
//       INT4 fp16   18.0 / 19.3     58 / 55     12.6 / 19.7
//   64  FP4 bf16    19.9 / 17.9     49 / 51     15.9 / 15.6
//       INT4 fp16   26.0 / 21.8     76 / 58     18.2 / 20.0
// fp16 with NF4 or FP4 goes on to 64, though up to 15% slower there (NF4 28672 x 4096 80 / 69, 4096 x 4096 26 / 25): two
// terms keep their weights to 2^-16, the other way they are rounded to 2^-11.
int64_t few_tokens(int fmt) {
  const int w = fmt_weight(fmt);
  return fmt_xtype(fmt) == kF16 && (w == kNF4 || w == kFP4) ? 64 : 32;
}

// Splits of N for a few tokens: as many as give every CU a workgroup of 128 columns, each at least a step of 32 rows
// for each of its eight waves.  16 tokens of NF4 1536 x 8960 take 11.5 us, with twice and half as many splits 13.8 and 14.9;
// 17920 x 1536 18.9, 24.3, 21.0; 28672 x 4096 37, 39, 58.
uint32_t few_splits(int64_t n, int64_t k) {
  const int64_t groups = (k + 127) / 128, rounds = ((n + 31) / 32 + 7) / 8;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(rounds, device_cu_count() / groups));
  const int64_t per = (rounds + want - 1) / want;  // rounds a split
  return (uint32_t)((rounds + per - 1) / per);
}

size_t up16(size_t v) { return (v + 15) & ~(size_t)15; }

// Whether the product decodes and transposes the weights itself, by the estimates of both: it does so for every tile of up
// to 256 tokens, and the workgroups of a split start with steps that only decode; the other way all weights are transposed
// through memory once, 2.5 bytes each at 4 TB/s and a launch.  Microseconds, by the product / transposed first:
//   FP4 bf16   17920 x 1536: 128 tokens 28 / 40, 512 53 / 64, 1000 88 / 84, 2048 131 / 135
//              11008 x 4096: 128 33 / 58, 512 76 / 104, 2048 217 / 179
//              28672 x 4096: 80 54 / 134, 512 136 / 187, 2048 465 / 464
//              4001 x 2048: 80 19 / 22, 333 29 / 26;  4096 x 4096: 80 22 / 27, 512 38 / 36, 2048 90 / 72, 4096 128 / 118
//   NF4 bf16   28672 x 4096: 80 60 / 132, 512 148 / 188, 2048 510 / 466;  4001 x 2048: 80 22 / 23, 333 30 / 26
//   INT4 fp16  28672 x 4096: 80 59 / 152, 512 142 / 203, 2048 478 / 474;  17920 x 1536: 2048 133 / 142
bool grad_columns(int fmt, int64_t n, int64_t k, int64_t b) {
  const int64_t pitch = (n + kTile - 1) / kTile * kTile * 2;
  return b <= 2048 && dense_us(false, b, k, pitch, fmt_weight(fmt), 1) < dense_us(false, b, k, pitch, -1, 1) + 3 + (double)n * k * 2.5 / 4e6;
}

struct GradSpace {
  uint32_t np;
  size_t wt, d, parts, exp, partial, bytes;
};
GradSpace grad_space(int fmt, int64_t n, int64_t k, int64_t b) {
  GradSpace g;
  const bool columns = grad_columns(fmt, n, k, b);
  g.np = (uint32_t)((n + kTile - 1) / kTile * kTile);
  g.wt = 0;
  g.d = columns ? 0 : up16((size_t)k * g.np * 2);
  g.parts = g.d + up16((size_t)b * g.np * 2);
  g.exp = g.parts + kMaxParts * 4;
  g.partial = g.exp + 16;
  g.bytes = g.partial + up16(dense_bytes(false, b, k, (int64_t)g.np * 2, columns ? fmt_weight(fmt) : -1, 1));
  return g;
}

template <int FMT>
hipError_t prepare(int xt, const uint16_t* d, int64_t pad_rows, const uint8_t* packed, const void* scales, int64_t n,
                   int64_t k, uint8_t* ws, const GradSpace& g, hipStream_t s) {
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
  p.tiles = (uint32_t)((int64_t)(g.np / kTile) * ((k + kColumns - 1) / kColumns));
  p.d = d;
  p.padded = reinterpret_cast<uint16_t*>(ws + g.d);
  const dim3 grid(p.tiles + (uint32_t)pad_rows);
  if (xt == kF16) {
    const int64_t count = n * (k / weights_per_scale<FMT>());
    p.nparts = (uint32_t)std::min<int64_t>(kMaxParts, (count + 1023) / 1024);
    ready_kernel<FMT><<<dim3(p.nparts), dim3(256), 0, s>>>(scales, count, reinterpret_cast<float*>(ws + g.parts), p.nparts,
                                                           nullptr, nullptr, 0, 0);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    transpose_kernel<FMT, kF16><<<grid, dim3(256), 0, s>>>(p);
  } else {
    transpose_kernel<FMT, kBF16><<<grid, dim3(256), 0, s>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

size_t gemm_grad_workspace(int fmt, int64_t n, int64_t k, int64_t b) {
  if (b <= few_tokens(fmt)) {
    const uint32_t splits = few_splits(n, k);
    return splits > 1 ? up16((size_t)splits * (size_t)(b * k) * 4) : 0;
  }
  return grad_space(fmt, n, k, b).bytes;
}

hipError_t launch_gemm_grad(int fmt, const uint16_t* d, const uint8_t* packed, const void* scales, int64_t n, int64_t k,
                            int64_t b, uint16_t* dx, void* ws, hipStream_t s) {
  const int xt = fmt_xtype(fmt);
  if (b <= few_tokens(fmt)) {
    const uint32_t splits = few_splits(n, k), steps = (uint32_t)((n + 31) / 32);
    const GradFewArgs f{d, packed, scales, dx, splits > 1 ? reinterpret_cast<float*>(ws) : nullptr,
                        (uint32_t)n, (uint32_t)k, (uint32_t)b, (steps + splits - 1) / splits};
    return xt == kF16 ? launch_grad_few_f16(fmt_weight(fmt), f, splits, s)
                      : launch_grad_few_bf16(fmt_weight(fmt), f, splits, s);
  }
  const GradSpace g = grad_space(fmt, n, k, b);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  const bool pad = (int64_t)g.np != n || (uintptr_t)d % 16;
  const int64_t pr = pad ? b : 0;
  const bool columns = grad_columns(fmt, n, k, b);
  uint32_t parts = 0;
  auto ready = [&](auto format) {
    constexpr int F = decltype(format)::value;
    if (!columns) return prepare<F>(xt, d, pr, packed, scales, n, k, base, g, s);
    const int64_t count = n * (k / weights_per_scale<F>());
    parts = xt == kF16 ? (uint32_t)std::min<int64_t>(kMaxParts, (count + 1023) / 1024) : 0u;
    if (parts + pr)
      ready_kernel<F><<<dim3(parts + (uint32_t)pr), dim3(256), 0, s>>>(
          scales, count, reinterpret_cast<float*>(base + g.parts), parts, d, reinterpret_cast<uint16_t*>(base + g.d),
          (uint32_t)n, g.np);
    return hipGetLastError();
  };
  using std::integral_constant;
  hipError_t e;
  switch (fmt_weight(fmt)) {
    case kNF4: e = ready(integral_constant<int, kNF4>{}); break;
    case kINT4: e = ready(integral_constant<int, kINT4>{}); break;
    case kFP4: e = ready(integral_constant<int, kFP4>{}); break;
    case kINT4A: e = ready(integral_constant<int, kINT4A>{}); break;
    default: e = ready(integral_constant<int, kMXFP4>{}); break;
  }
  if (e != hipSuccess) return e;
  if (pad) d = reinterpret_cast<const uint16_t*>(base + g.d);
  DenseArgs a{};
  a.a = reinterpret_cast<const uint8_t*>(d);
  a.b = columns ? packed : base + g.wt;
  a.m = (uint32_t)b;
  a.n = (uint32_t)k;
  a.pitch = g.np * 2;
  a.terms = 1;
  a.exp = xt == kF16 ? reinterpret_cast<const int*>(base + g.exp) : nullptr;
  a.partial = reinterpret_cast<uint32_t*>(base + g.partial);
  a.out = dx;
  a.out_type = xt == kF16 ? 1 : 2;
  const int type = xt == kF16 ? kDenseF16 : kDenseBF16;
  if (!columns) return launch_dense(type, false, a, s);
  a.scales = scales;
  a.rows = (uint32_t)n;
  a.parts = reinterpret_cast<const float*>(base + g.parts);
  a.nparts = parts;
  a.exp_out = reinterpret_cast<int*>(base + g.exp);
  switch (fmt_weight(fmt)) {
    case kNF4: return launch_dense_columns_nf4(type, a, s);
    case kINT4: return launch_dense_columns_int4(type, a, s);
    case kFP4: return launch_dense_columns_fp4(type, a, s);
    case kINT4A: return launch_dense_columns_int4a(type, a, s);
    default: return launch_dense_columns_mxfp4(type, a, s);
  }
}

}  // namespace w4
