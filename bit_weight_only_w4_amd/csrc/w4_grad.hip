// Input gradient of a product with frozen 4-bit weights: dx[t, k] = sum_n d[t, n] W_hat[n, k].
//
// The sum runs over the weight rows, along which a packed byte holds nothing: the weights are decoded once into W_hat^T
// rows of 16 bits in the workspace (through LDS), which the dense kernel multiplies with d, or, where that costs less, the
// dense kernel decodes and transposes them as they arrive (PackedColumns in w4_dense_sources.h).  Both types of d are
// multiplied in fp16, bf16 d as d 2^-e with one e a token (exact), weights as w 2^-f with one f for each unit of 64 columns
// (128 of the integer formats), taken from its largest scale, so that neither large nor small weights leave fp16's range
// and no column suffers from another's scales.  INT4 and MXFP4 weights fit one fp16 number, the others are the sum of two
// (first_term in w4_ffn_math.h); bf16 would hold them to 2^-8 and need three.  MXFP4 with bf16 d is multiplied in bf16,
// which holds its weights whole and needs no exponents.  Rows of W_hat^T are padded with zeros to whole steps of the
// dense kernel, and so is d where its rows do not end on one or are not aligned.
#include <algorithm>
#include <type_traits>

#include "w4_ffn.h"
#include "w4_ffn_math.h"

namespace w4 {
namespace {

constexpr int kTile = 64;       // weight rows of a tile
constexpr int kMaxParts = 512;  // workgroups of the scale scan

// The largest finite scale of each unit of columns over rows [first, end), to `parts`.
template <int FMT>
__device__ inline void scale_max(const void* scales, uint32_t first, uint32_t end, uint32_t units, float* parts) {
  constexpr uint32_t PER = column_unit(FMT) / weights_per_scale<FMT>();  // scales of a row and unit
  __shared__ float part[256];
  const uint32_t tid = threadIdx.x;
  auto fold = [&](float top, uint32_t row, uint32_t unit) __attribute__((always_inline)) {
#pragma unroll
    for (uint32_t j = 0; j < PER; ++j) {
      const float s = fabsf(scale_of<FMT>(scales, ((size_t)row * units + unit) * PER + j));
      top = s < __builtin_inff() ? fmaxf(top, s) : top;
    }
    return top;
  };
  if (units > 128) {
    for (uint32_t u = tid; u < units; u += 256) {
      float top = 0.0f;
#pragma unroll 8
      for (uint32_t r = first; r < end; ++r) top = fold(top, r, u);
      parts[u] = top;
    }
    return;
  }
  const uint32_t at_once = 256 / units, u = tid % units, r0 = tid / units;  // rows at once
  float top = 0.0f;
  if (r0 < at_once) {
#pragma unroll 8
    for (uint32_t r = first + r0; r < end; r += at_once) top = fold(top, r, u);
  }
  part[tid] = top;
  __syncthreads();
  if (tid >= units) return;
  for (uint32_t j = 1; j < at_once; ++j) top = fmaxf(top, part[j * units + tid]);
  parts[tid] = top;
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

// A row of bf16 d as fp16 numbers times 2^e, zeros after its end up to `np`: e puts the row's largest into fp16's highest
// binade but one, so that all that lie within 2^28 below it are exact.  A thread keeps the first kHeld pieces of 8 between
// the pass for the largest and the one that writes (2048 rows of 17920 27 us with the scan beside it, 5.4 TB/s).
constexpr int kHeld = 4;

__device__ inline void convert_row(const uint16_t* from, uint16_t* to, int* exponent, uint32_t n, uint32_t np) {
  __shared__ uint32_t most[4];
  uint32_t held[kHeld][4], top = 0;  // the largest finite magnitude, as bits
  auto load = [&](uint32_t c, uint32_t (&v)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = 0;
    if (c + 8 <= n) {
      __builtin_memcpy(v, from + c, 16);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j)
        if (c + j < n) v[j >> 1] |= (uint32_t)from[c + j] << (16 * (j & 1));
    }
  };
  auto fold = [&](const uint32_t (&v)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = v[j] & 0x7FFFu, b = (v[j] >> 16) & 0x7FFFu;
      top = max(top, max(a < 0x7F80u ? a : 0u, b < 0x7F80u ? b : 0u));
    }
  };
  const uint32_t c0 = threadIdx.x * 8;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    load(c0 + i * 2048, held[i]);
    fold(held[i]);
  }
#pragma unroll 4
  for (uint32_t c = c0 + kHeld * 2048; c < n; c += 2048) {
    uint32_t v[4];
    load(c, v);
    fold(v);
  }
  const float m = wave_max(__uint_as_float(top << 16));
  if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = __float_as_uint(m);
  __syncthreads();
  top = max(max(most[0], most[1]), max(most[2], most[3]));
  const int e = top ? ilogbf(__uint_as_float(top)) - 14 : 0;
  if (threadIdx.x == 0) *exponent = e;
  auto put = [&](uint32_t c, const uint32_t (&v)[4]) __attribute__((always_inline)) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = to16<kF16>(ldexpf(__uint_as_float(v[j] << 16), -e)) |
             (to16<kF16>(ldexpf(__uint_as_float(v[j] & 0xFFFF0000u), -e)) << 16);
    *reinterpret_cast<uint4*>(to + c) = make_uint4(o[0], o[1], o[2], o[3]);
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (c0 + i * 2048 < np) put(c0 + i * 2048, held[i]);
#pragma unroll 2
  for (uint32_t c = c0 + kHeld * 2048; c < np; c += 2048) {
    uint32_t v[4];
    load(c, v);
    put(c, v);
  }
}

// What a product needs before it: the scales' maxima (fp16; `parts` workgroups of `per` rows each), and d with whole rows,
// bf16 as fp16 where there are exponents for it, in the workgroups after those.
struct ReadyArgs {
  const void* scales;
  float* maxima;  // [parts, units]
  uint32_t parts, per, rows, units;
  const uint16_t* d;  // [B, N]
  uint16_t* padded;   // [B, NP]
  int* row_exp;       // [B] or null
  uint32_t n, np;
};

template <int FMT>
__global__ void __launch_bounds__(256) ready_kernel(ReadyArgs p) {
  if (blockIdx.x >= p.parts) {
    const size_t t = blockIdx.x - p.parts;
    if (p.row_exp)
      convert_row(p.d + t * p.n, p.padded + t * p.np, p.row_exp + t, p.n, p.np);
    else
      pad_row(p.d + t * p.n, p.padded + t * p.np, p.n, p.np);
    return;
  }
  const uint32_t first = blockIdx.x * p.per;
  scale_max<FMT>(p.scales, first, min(first + p.per, p.rows), p.units, p.maxima + (size_t)blockIdx.x * p.units);
}

struct TransposeArgs {
  const uint8_t* packed;  // [N, K/2]
  const void* scales;
  uint16_t* wt;           // [K, NP], of two terms [K, NP / 64, 2, 64]
  uint32_t n, k, np;
  const float* parts;     // fp16: the scan's maxima [nparts, K / unit]
  uint32_t nparts;
  int* exps;              // fp16: [K], the columns' exponents that they give
  uint32_t tiles;         // workgroups that transpose; those after them copy d
  const uint16_t* d;      // [B, N]
  uint16_t* padded;       // [B, NP]
};

// A tile of 64 rows x 256 columns a workgroup, whole cache lines of the packed rows: a thread decodes 32 columns of two
// rows, writes them to LDS as pairs along n, and stores 16 bytes of rows of W_hat^T, one term after the other.  In LDS
// column 32 part + j is at row 8 j + part of 40 dwords: the 64 pairs that a wave writes at once then lie in 64 banks.
// Neighbouring workgroups take neighbouring rows, whose pieces of W_hat^T are one after another.  27.5 million weights take
// 21 us, in two terms 34 (3.7 TB/s).
constexpr int kColumns = 256;

template <int FMT, int XT>
__global__ void __launch_bounds__(256) transpose_kernel(TransposeArgs p) {
  constexpr uint32_t G = weights_per_scale<FMT>(), UNIT = column_unit(FMT);
  constexpr int TERMS = XT == kF16 ? dense_terms(FMT) : 1;
  constexpr int PITCH = 40;
  const uint32_t tid = threadIdx.x;
  if (blockIdx.x >= p.tiles) {  // a row of d, zeros after its end
    const size_t t = blockIdx.x - p.tiles;
    pad_row(p.d + t * p.n, p.padded + t * p.np, p.n, p.np);
    return;
  }
  __shared__ float table[16];
  __shared__ int exps[kColumns / UNIT];
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
  if constexpr (XT == kF16) {
    const uint32_t wave = tid >> 6;
    static_assert(kColumns / UNIT <= 4, "a wave for each unit");
    if (wave < kColumns / UNIT) {
      const int e = unit_exponent<FMT>(p.parts, p.nparts, p.k / UNIT, k0 / UNIT + wave, tid & 63);
      if ((tid & 63) == 0) exps[wave] = e;
    }
  }
  __syncthreads();
  if constexpr (XT == kF16) {
    if (n0 == 0 && k0 + tid < p.k) p.exps[k0 + tid] = exps[tid / UNIT];
    const int f = exps[32 * part / UNIT];
    s[0].s = ldexpf(s[0].s, -f);
    s[1].s = ldexpf(s[1].s, -f);
  }
  const uint32_t w0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, w1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
  for (int term = 0; term < TERMS; ++term) {
    if (term) __syncthreads();  // the first has been read
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float a[2], b[2];  // rows past N have scale 0 and finite codes: zeros
      decode_pair<FMT>(w0[j >> 2], j & 3, table, BlockScale{TERMS == 2 ? 1.0f : s[0].s, s[0].zero}, &a[0], &a[1]);
      decode_pair<FMT>(w1[j >> 2], j & 3, table, BlockScale{TERMS == 2 ? 1.0f : s[1].s, s[1].zero}, &b[0], &b[1]);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t o;
        if constexpr (TERMS == 2) {
          o = scaled_pair(a[q], b[q], first_term(s[0].s), first_term(s[1].s));
          if (term) o = rest_of_pair(a[q], b[q], s[0].s, s[1].s, o);
        } else {
          o = to16<XT>(a[q]) | (to16<XT>(b[q]) << 16);
        }
        tile[(8 * (2 * j + q) + part) * PITCH + rp] = o;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t k = (tid >> 3) + 32u * i, c = tid & 7;
      const uint4 o = *reinterpret_cast<const uint4*>(tile + (8 * (k & 31) + (k >> 5)) * PITCH + 4 * c);
      if (k0 + k < p.k)
        *reinterpret_cast<uint4*>(p.wt + ((size_t)(k0 + k) * p.np + n0) * TERMS + term * kTile + c * 8) = o;
    }
  }
}

// How many tokens take the packed weights decoded in registers (w4_grad_few.h).  Microseconds there / by the dense
// kernel decoding them itself:
//                   4864 x 896   1536 x 8960  4096 x 4096  17920 x 1536  28672 x 4096
//   33  INT4 fp16    18 / 17      19 / 20      20 / 20      30 / 26       67 / 54
//       MXFP4 bf16   16 / 13      14 / 16      16 / 15      21 / 21       39 / 45
//       INT4 bf16    17 / 17      16 / 20      18 / 20      26 / 28       49 / 57
//   64  INT4 fp16    21 / 17      23 / 22      24 / 22      34 / 26       73 / 56
//       MXFP4 bf16   18 / 14      18 / 16      20 / 17      25 / 21       44 / 47
//       MXFP4 fp16   19 / 19      20 / 22      22 / 23      29 / 29       52 / 59
//       INT4 bf16    19 / 18      20 / 22      22 / 22      29 / 30       53 / 58
//       INT4A fp16   21 / 21      23 / 30      24 / 29      34 / 39       73 / 93
//       FP4 fp16     22 / 20      25 / 27      26 / 27      39 / 36       87 / 89
//       NF4 bf16     21 / 24      23 / 32      25 / 33      35 / 48       71 / 106
// The first two have one term there and d as it is.  At 17 tokens all are faster here (INT4 fp16 28672 x 4096 51 / 53).
int64_t few_tokens(int fmt) { return grad_few_most(fmt_weight(fmt), fmt_xtype(fmt)); }

// Splits of N for a few tokens: as many as give every CU a workgroup of 128 columns, each at least a step of 32 rows
// for each of its eight waves.  16 tokens of NF4 1536 x 8960 take 13.6 us, with twice and half as many splits 16.0 and 21.4;
// 17920 x 1536 24.4, 28.7, 30.1; 28672 x 4096 54.8, 53.2, 88.4.
uint32_t few_splits(int64_t n, int64_t k) {
  const int64_t groups = (k + 127) / 128, rounds = ((n + 31) / 32 + 7) / 8;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(rounds, device_cu_count() / groups));
  const int64_t per = (rounds + want - 1) / want;  // rounds a split
  return (uint32_t)((rounds + per - 1) / per);
}

// Past the few tokens the product is made in fp16, with an exponent a unit of columns and, for bf16 gradients, a token;
// MXFP4 with bf16 gradients in bf16, which holds its weights whole and needs no exponents.
bool grad_in_fp16(int fmt) { return fmt_xtype(fmt) == kF16 || fmt_weight(fmt) != kMXFP4; }
int grad_terms(int fmt) { return grad_in_fp16(fmt) ? dense_terms(fmt_weight(fmt)) : 1; }

size_t up16(size_t v) { return (v + 15) & ~(size_t)15; }

// Whether the product decodes and transposes the weights itself, by the estimates of both: it does so for every tile of up
// to 256 tokens, and the workgroups of a split start with steps that only decode; the other way all weights are transposed
// through memory once, 2 bytes a term and 0.5 each at 4 TB/s and a launch.  Microseconds, by the product / transposed first:
//              4096 x 4096   17920 x 1536  11008 x 4096  28672 x 4096
//   NF4 bf16   80 tokens    34 / 43      62 / 70      55 / 98      109 / 286
//              512          69 / 69     108 / 121    150 / 154     276 / 400
//              2048        201 / 150    272 / 265    397 / 378     998 / 987
//   FP4 fp16   512          59 / 66      87 / 112    126 / 146     242 / 381
//              2048        162 / 141    228 / 234    352 / 355     856 / 940
//   INT4 fp16  512          41 / 42      55 / 80      78 / 94      147 / 217
//              2048         88 / 79     131 / 142    224 / 191     468 / 484
//   MXFP4 bf16 512          34 / 36      48 / 62      67 / 81      127 / 187
// Of 276 pairs of six sizes and 80 to 2048 tokens the rule's way is at most 29% slower than the other, 1% at the mean.
bool grad_columns(int fmt, int64_t n, int64_t k, int64_t b) {
  const int64_t pitch = (n + kTile - 1) / kTile * kTile * 2;
  const int w = fmt_weight(fmt), terms = grad_terms(fmt);
  return b <= 2048 && dense_us(false, b, k, pitch, w, terms) <
                          dense_us(false, b, k, pitch, -1, terms) + 3 + (double)n * k * (0.5 + 2 * terms) / 4e6;
}

struct GradSpace {
  uint32_t np;
  size_t wt, d, parts, row_exp, col_exp, partial, bytes;
};
GradSpace grad_space(int fmt, int64_t n, int64_t k, int64_t b) {
  GradSpace g;
  const bool columns = grad_columns(fmt, n, k, b);
  const int w = fmt_weight(fmt), terms = grad_terms(fmt);
  g.np = (uint32_t)((n + kTile - 1) / kTile * kTile);
  g.wt = 0;
  g.d = columns ? 0 : up16((size_t)k * g.np * 2 * terms);
  g.parts = g.d + up16((size_t)b * g.np * 2);
  g.row_exp = g.parts + up16((size_t)kMaxParts * (k / column_unit(w)) * 4);
  g.col_exp = g.row_exp + up16((size_t)b * 4);
  g.partial = g.col_exp + up16((size_t)k * 4);
  g.bytes = g.partial + up16(dense_bytes(false, b, k, (int64_t)g.np * 2, columns ? w : -1, terms));
  return g;
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
  const int w = fmt_weight(fmt);
  const bool half = grad_in_fp16(fmt), convert = half && xt == kBF16, columns = grad_columns(fmt, n, k, b);
  const bool pad = (int64_t)g.np != n || (uintptr_t)d % 16;
  ReadyArgs r{};
  r.scales = scales;
  r.maxima = reinterpret_cast<float*>(base + g.parts);
  r.rows = (uint32_t)n;
  r.units = (uint32_t)(k / column_unit(w));
  if (half) {  // at least 1024 scales a workgroup
    const int64_t want = std::min<int64_t>(kMaxParts, (n * r.units + 1023) / 1024);
    r.per = (uint32_t)((n + want - 1) / want);
    r.parts = (uint32_t)((n + r.per - 1) / r.per);
  }
  r.d = d;
  r.padded = reinterpret_cast<uint16_t*>(base + g.d);
  r.row_exp = convert ? reinterpret_cast<int*>(base + g.row_exp) : nullptr;
  r.n = (uint32_t)n;
  r.np = g.np;
  TransposeArgs t;
  t.packed = packed;
  t.scales = scales;
  t.wt = reinterpret_cast<uint16_t*>(base + g.wt);
  t.n = (uint32_t)n;
  t.k = (uint32_t)k;
  t.np = g.np;
  t.parts = r.maxima;
  t.nparts = r.parts;
  t.exps = reinterpret_cast<int*>(base + g.col_exp);
  t.tiles = (uint32_t)((int64_t)(g.np / kTile) * ((k + kColumns - 1) / kColumns));
  t.d = d;
  t.padded = r.padded;
  // d's rows are copied with the scan where they are converted or nothing is transposed, else with the transposing.
  const uint32_t with_scan = convert || (pad && columns) ? (uint32_t)b : 0u;
  const uint32_t with_tiles = pad && !convert ? (uint32_t)b : 0u;
  auto ready = [&](auto format) {
    constexpr int F = decltype(format)::value;
    if (r.parts + with_scan) ready_kernel<F><<<dim3(r.parts + with_scan), dim3(256), 0, s>>>(r);
    if (columns) return hipGetLastError();
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const dim3 grid(t.tiles + with_tiles);
    if constexpr (F == kMXFP4) {
      if (!half) {
        transpose_kernel<F, kBF16><<<grid, dim3(256), 0, s>>>(t);
        return hipGetLastError();
      }
    }
    transpose_kernel<F, kF16><<<grid, dim3(256), 0, s>>>(t);
    return hipGetLastError();
  };
  using std::integral_constant;
  hipError_t e;
  switch (w) {
    case kNF4: e = ready(integral_constant<int, kNF4>{}); break;
    case kINT4: e = ready(integral_constant<int, kINT4>{}); break;
    case kFP4: e = ready(integral_constant<int, kFP4>{}); break;
    case kINT4A: e = ready(integral_constant<int, kINT4A>{}); break;
    default: e = ready(integral_constant<int, kMXFP4>{}); break;
  }
  if (e != hipSuccess) return e;
  DenseArgs a{};
  a.a = pad || convert ? base + g.d : reinterpret_cast<const uint8_t*>(d);
  a.b = columns ? packed : base + g.wt;
  a.m = (uint32_t)b;
  a.n = (uint32_t)k;
  a.pitch = g.np * 2;
  a.terms = (uint32_t)grad_terms(fmt);
  a.row_exp = r.row_exp;
  a.col_exp = half ? t.exps : nullptr;
  a.partial = reinterpret_cast<uint32_t*>(base + g.partial);
  a.out = dx;
  a.out_type = xt == kF16 ? 1 : 2;
  const int type = half ? kDenseF16 : kDenseBF16;
  if (!columns) return launch_dense(type, false, a, s);
  a.scales = scales;
  a.rows = (uint32_t)n;
  a.parts = r.maxima;
  a.nparts = r.parts;
  a.exp_out = t.exps;
  switch (w) {
    case kNF4: return launch_dense_columns_nf4(a, s);
    case kINT4: return launch_dense_columns_int4(a, s);
    case kFP4: return launch_dense_columns_fp4(a, s);
    case kINT4A: return launch_dense_columns_int4a(a, s);
    default: return launch_dense_columns_mxfp4(type, a, s);
  }
}

}  // namespace w4
