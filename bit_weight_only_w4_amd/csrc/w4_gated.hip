// Gated feed-forward block over 4-bit weights: h = act(x Wg^T) * (x Wu^T), and the gradients of its two products.
//
// Many tokens: the dense kernel (w4_dense.h) multiplies fp16 rows with fp16 weights, which are decoded once into the
// workspace or, where they meet few tiles of tokens, by the dense kernel as they arrive.  A weight row is held as w 2^-f
// with one exponent f a row that puts its largest scale into the top of fp16's range, bf16 tokens as x 2^-e with one e a
// token; both come off exactly in the epilogue.  fp16 has 11 significant bits where bf16 has 8: INT4 and MXFP4 weights and
// bf16 tokens are exact, NF4, FP4 and asymmetric INT4 weights the sum of two fp16 numbers (first_term in w4_ffn_math.h),
// within 2^-20 of themselves; what lies more than 2^28 below its row's largest is off by at most 2^-39 of that.  One fp16
// number would be off by 2^-11, as much as the rounding of fp16 results and a quarter of bf16's; two cost twice the matrix
// instructions (4096 -> 11008, 1000 tokens of NF4: 211 us against 430).
#include <algorithm>
#include <type_traits>

#include "w4_ffn.h"
#include "w4_ffn_math.h"

namespace w4 {
namespace {

constexpr int kDecodeThreads = 256;
struct DecodeArgs {
  const uint8_t* packed;  // [N, K/2]
  const void* scales;
  uint16_t* w;   // [N, K] fp16: decoded rows, or [N, K / 64, 2, 64]: first and second terms
  float2* fold;  // [N, K / 64], in place of w: what the dense kernel takes for 64 packed weights, the scales 2^-f of
                 // their halves, for integer formats the scale 2^-f and the codes' offset
  int* w_exp;    // [N]
  uint32_t n, k;
  const uint16_t* x;  // [T, K] bf16, null: no tokens to convert
  uint16_t* xh;       // [T, K] fp16
  int* x_exp;         // [T]
  uint32_t t;
};

// Token rows to fp16, a wave each: a lane takes 8 consecutive values of every 512 and keeps those of the first kHeld
// rounds between the pass for the largest and the one that writes.
constexpr int kHeld = 4;

__device__ inline void token_row(const DecodeArgs& p, uint32_t t, int lane) {
  const uint4* src = reinterpret_cast<const uint4*>(p.x + (size_t)t * p.k);
  uint4* dst = reinterpret_cast<uint4*>(p.xh + (size_t)t * p.k);
  const uint32_t chunks = p.k / 8;
  uint32_t top = 0;  // the largest finite magnitude, as bits
  auto fold = [&](const uint4& v) __attribute__((always_inline)) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = w[j] & 0x7FFFu, b = (w[j] >> 16) & 0x7FFFu;
      top = a < 0x7F80u ? max(top, a) : top;
      top = b < 0x7F80u ? max(top, b) : top;
    }
  };
  uint4 held[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) held[j] = j * 64 + lane < chunks ? src[j * 64 + lane] : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < kHeld; ++j) fold(held[j]);
  for (uint32_t i = kHeld * 64 + lane; i < chunks; i += 64) fold(src[i]);
  const float m = wave_max(__uint_as_float(top << 16));
  const int e = m > 0.0f ? ilogbf(m) - 14 : 0;
  if (lane == 0) p.x_exp[t] = e;
  auto put = [&](uint32_t i, const uint4& v) __attribute__((always_inline)) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = to16<kF16>(ldexpf(__uint_as_float(w[j] << 16), -e)) |
             (to16<kF16>(ldexpf(__uint_as_float(w[j] & 0xFFFF0000u), -e)) << 16);
    dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
  };
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    if (j * 64 + lane < chunks) put(j * 64 + lane, held[j]);
  for (uint32_t i = kHeld * 64 + lane; i < chunks; i += 64) put(i, src[i]);
}

// The scales of weight rows for the kernel that decodes them itself, sixteen lanes a row; token rows in the first
// workgroups, whose two passes take longest (27.5 million MXFP4 weights and 1000 tokens 7 us).
constexpr int kFoldRows = kDecodeThreads / 16;

template <int FMT>
__global__ void __launch_bounds__(kDecodeThreads) fold_rows_kernel(DecodeArgs p) {
  const uint32_t before = p.x ? (p.t + kDecodeThreads / 64 - 1) / (kDecodeThreads / 64) : 0u;
  if (blockIdx.x < before) {
    const uint32_t t = blockIdx.x * (kDecodeThreads / 64) + (threadIdx.x >> 6);
    if (t < p.t) token_row(p, t, threadIdx.x & 63);
    return;
  }
  const uint32_t lane = threadIdx.x & 15, row = (blockIdx.x - before) * kFoldRows + (threadIdx.x >> 4);
  if (row >= p.n) return;  // sixteen lanes at once
  constexpr uint32_t G = weights_per_scale<FMT>();
  const uint32_t groups = p.k / G, blocks = p.k / 64;
  const size_t s0 = (size_t)row * groups;
  float top = 0.0f;
  for (uint32_t i = lane; i < groups; i += 16) {
    const float a = fabsf(scale_of<FMT>(p.scales, s0 + i));
    top = a < __builtin_inff() ? fmaxf(top, a) : top;  // infinities and NaN have no binade
  }
#pragma unroll
  for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  const int f = fold_exponent<FMT>(top);
  if (lane == 0) p.w_exp[row] = f;
  for (uint32_t i = lane; i < blocks; i += 16) {
    const BlockScale b = block_scale<FMT>(p.scales, s0 + 64 * i / G);
    float second = FMT == kINT4 || FMT == kINT4A ? b.zero : ldexpf(b.s, -f);
    if constexpr (FMT == kMXFP4) second = ldexpf(scale_of<FMT>(p.scales, s0 + 2 * i + 1), -f);
    p.fold[(size_t)row * blocks + i] = make_float2(ldexpf(b.s, -f), second);
  }
}

// Weight rows decoded, a wave each, then token rows.  A lane takes 8 consecutive weights of every 512 (so that a store
// of the wave is 1 KiB in one piece; 27.5 million weights take 20 us, in two terms, 128 bytes of each in turn, 24, and 90
// million 80, 5.1 TB/s), the first kHeld rounds with their scales
// in flight at once; the largest of these scales is the row's unless the row is longer.
template <int FMT>
__global__ void __launch_bounds__(kDecodeThreads) decode_rows_kernel(DecodeArgs p) {
  const int lane = threadIdx.x & 63;
  const uint32_t row = blockIdx.x * (kDecodeThreads / 64) + (threadIdx.x >> 6);
  constexpr uint32_t G = weights_per_scale<FMT>();
  __shared__ float table[16];
  code_table<FMT>(table);
  __syncthreads();
  if (row < p.n) {
    const uint32_t groups = p.k / G, chunks = p.k / 8;
    const size_t s0 = (size_t)row * groups;
    float top = 0.0f;
    auto fold = [&](float x) __attribute__((always_inline)) {
      const float a = fabsf(x);
      top = a < __builtin_inff() ? fmaxf(top, a) : top;  // infinities and NaN have no binade
    };
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.packed + (size_t)row * (p.k / 2));
    constexpr int TERMS = dense_terms(FMT);
    uint4* dst = reinterpret_cast<uint4*>(p.w + (size_t)row * p.k * TERMS);
    uint32_t v[kHeld];
    BlockScale s[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const uint32_t i = j * 64 + lane;
      if (i < chunks) {
        v[j] = src[i];
        s[j] = block_scale<FMT>(p.scales, s0 + i * 8 / G);
      }
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (j * 64 + lane < chunks) fold(s[j].s);
    for (uint32_t i = kHeld * 512 / G + lane; i < groups; i += 64) fold(scale_of<FMT>(p.scales, s0 + i));
    const int f = fold_exponent<FMT>(wave_max(top));
    if (lane == 0) p.w_exp[row] = f;
    auto put = [&](uint32_t i, uint32_t w, BlockScale b) __attribute__((always_inline)) {
      b.s = ldexpf(b.s, -f);
      uint32_t o[4], r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float lo, hi;
        if constexpr (TERMS == 1) {
          decode_pair<FMT>(w, j, table, b, &lo, &hi);
          o[j] = to16<kF16>(lo) | (to16<kF16>(hi) << 16);
        } else {
          decode_pair<FMT>(w, j, table, BlockScale{1.0f, b.zero}, &lo, &hi);
          o[j] = scaled_pair(lo, hi, first_term(b.s));
          r[j] = rest_of_pair(lo, hi, b.s, o[j]);
        }
      }
      if constexpr (TERMS == 1) {
        dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        const uint32_t at = i / 8 * 16 + i % 8;
        dst[at] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[at + 8] = make_uint4(r[0], r[1], r[2], r[3]);
      }
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (j * 64 + lane < chunks) put(j * 64 + lane, v[j], s[j]);
    for (uint32_t i = kHeld * 64 + lane; i < chunks; i += 64) put(i, src[i], block_scale<FMT>(p.scales, s0 + i * 8 / G));
    return;
  }
  const uint32_t t = row - p.n;
  if (p.x && t < p.t) token_row(p, t, lane);
}

size_t up16(size_t v) { return (v + 15) & ~(size_t)15; }

// Whether the dense kernel decodes the packed weights itself, by the estimates of both: it decodes them once for every tile
// of up to 256 tokens, which makes its steps up to half as long again; the other way the weights go through memory once
// more, at 2 bytes a term and 4 TB/s.  Microseconds, by the dense kernel / decoded first (two terms: NF4, FP4, asymmetric
// INT4); of 108 measured pairs the rule's way is at most 20% slower than the other (NF4), 1.5% at the mean.
//                1536 -> 8960   4096 -> 11008   8192 -> 28672
//   NF4   192      70 / 58       137 / 217       540 / 939      300  79 / 67    309 / 259  1094 / 1130
//   NF4   512     131 / 95       231 / 313      1032 / 1387    2048 297 / 236   781 / 719  3818 / 3481
//   FP4   192      56 / 58       126 / 220       503 / 934      512 110 / 94    213 / 313   961 / 1390
//   INT4  192      34 / 41        87 / 101       284 / 493      300  41 / 46    138 / 141   498 / 594
//   INT4  512      64 / 63       123 / 155       523 / 720     2048 152 / 141   388 / 370  1905 / 1812
//   MXFP4 512      57 / 59       111 / 146       466 / 697     1000  78 / 80    213 / 211   924 / 1028
//   MXFP4 2048    138 / 134      337 / 346      1660 / 1708    4096 254 / 234   681 / 637  3236 / 3119
bool gated_packed(int fmt, int64_t tokens, int64_t hidden, int64_t inter) {
  const int w = fmt_weight(fmt), terms = dense_terms(w);
  return dense_us(true, tokens, inter, 2 * hidden, w, terms) <
         dense_us(true, tokens, inter, 2 * hidden, -1, terms) + (double)(2 * inter) * hidden * (0.5 + 2 * terms) / 4e6;
}

struct GatedSpace {
  size_t w, w_exp, xh, x_exp, partial, bytes;
};
GatedSpace gated_space(int fmt, int64_t tokens, int64_t hidden, int64_t inter) {
  GatedSpace g;
  const bool packed = gated_packed(fmt, tokens, hidden, inter);
  g.w = 0;
  g.w_exp = up16(packed ? (size_t)(2 * inter) * (size_t)(hidden / 64) * 8 : (size_t)(2 * inter * hidden) * 2 * dense_terms(fmt_weight(fmt)));
  g.xh = g.w_exp + up16((size_t)(2 * inter) * 4);
  g.x_exp = g.xh;
  g.partial = g.xh;
  if (fmt_xtype(fmt) == kBF16) {
    g.x_exp = g.xh + up16((size_t)(tokens * hidden) * 2);
    g.partial = g.x_exp + up16((size_t)tokens * 4);
  }
  g.bytes = g.partial + up16(dense_bytes(true, tokens, inter, 2 * hidden, packed ? fmt_weight(fmt) : -1,
                                       dense_terms(fmt_weight(fmt))));
  return g;
}

// Gradients of g | u from that of h, element by element: six bytes read and four written a channel, which is all
// that bounds it (bf16, 4096 x 8960: 65 us, 5.6 TB/s; 4096 x 8961, whose rows are not aligned, 66).  A thread takes
// 8 channels of a row, the last one of a row what is left.
template <int XT, int ACT>
__global__ void __launch_bounds__(256) gated_grad_kernel(const uint16_t* dh, const uint16_t* pr, uint16_t* dp, int64_t first,
                                                         int64_t pieces, int64_t inter) {
  const int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x;  // piece, row-major
  if (i >= pieces) return;
  const int64_t per = (inter + 7) / 8, t = i / per, c = (i - t * per) * 8;
  const uint16_t* from = dh + t * inter + c;
  const uint16_t* gu = pr + t * 2 * inter + c;
  uint16_t* to = dp + t * 2 * inter + c;
  auto one = [&](uint16_t dv, uint16_t gv, uint16_t uv, uint16_t& og, uint16_t& ou) __attribute__((always_inline)) {
    float slope;
    const float y = act_slope<ACT>(from16<XT>(gv), &slope), f = from16<XT>(dv), u = from16<XT>(uv);
    // The slope is at most 1.13: times it first a large u, then f u of a small one, so that neither leaves the range
    // where the whole does not.
    og = (uint16_t)to16<XT>(fabsf(u) >= 1.0f ? f * (u * slope) : f * u * slope);
    ou = (uint16_t)to16<XT>(f * y);
  };
  if (c + 8 > inter) {
    for (int64_t j = 0; c + j < inter; ++j) one(from[j], gu[j], gu[inter + j], to[j], to[inter + j]);
    return;
  }
  uint16_t d[8], g[8], u[8], og[8], ou[8];
  __builtin_memcpy(d, from, 16);
  __builtin_memcpy(g, gu, 16);
  __builtin_memcpy(u, gu + inter, 16);
#pragma unroll
  for (int j = 0; j < 8; ++j) one(d[j], g[j], u[j], og[j], ou[j]);
  __builtin_memcpy(to, og, 16);
  __builtin_memcpy(to + inter, ou, 16);
}

template <int XT, int ACT>
hipError_t grad_launch(const uint16_t* dh, const uint16_t* pr, uint16_t* dp, int64_t tokens, int64_t inter,
                       hipStream_t s) {
  const int64_t pieces = tokens * ((inter + 7) / 8), most = (int64_t)1 << 31;  // a launch has fewer than 2^32 threads
  for (int64_t first = 0; first < pieces; first += most) {
    const dim3 grid((uint32_t)((std::min(pieces - first, most) + 255) / 256));
    gated_grad_kernel<XT, ACT><<<grid, dim3(256), 0, s>>>(dh, pr, dp, first, pieces, inter);
  }
  return hipGetLastError();
}

}  // namespace

// Whether the weights are streamed once past the tokens and decoded in registers (run_gated_few; no workspace).  Microseconds
// so / by the dense kernel:
//                      896 -> 4864   1536 -> 8960   4096 -> 11008  8192 -> 28672
//   64 tokens   INT4    11 / 17       18 / 27        51 / 57        142 / 170
//               FP4     11 / 23       19 / 42        52 / 98        144 / 299
//               NF4     13 / 26       24 / 53        67 / 124       229 / 354
//               MXFP4   11 / 15       21 / 24        63 / 50        173 / 157      32 tokens  36 / 50   106 / 149
//   128 tokens  INT4    15 / 17       30 / 34        67 / 61        252 / 205
//               FP4     15 / 26       37 / 42        77 / 94        277 / 369
//               NF4     19 / 33       49 / 46       107 / 111       402 / 414
//               INT4A   16 / 28       33 / 42        76 / 100       288 / 360
//               MXFP4   19 / 15       41 / 31        92 / 57        332 / 180      96 tokens  19 / 15, 41 / 31
// (a launch has up to 128 tokens in one pass: 192 tokens of NF4 91 / 70, 208 / 137.)
bool gated_few(int fmt, int64_t tokens, int64_t hidden, int64_t inter) {
  const int w = fmt_weight(fmt);
  const bool large = 2 * inter * hidden >= (int64_t)1 << 25;
  const int64_t most = w == kMXFP4 ? (large ? 32 : 64) : w == kINT4 && large ? 64 : 128;
  return tokens <= most && gated_mfma_fits(fmt, inter, hidden, tokens);
}

size_t gated_workspace(int fmt, int64_t tokens, int64_t hidden, int64_t inter) {
  return gated_few(fmt, tokens, hidden, inter) ? 0 : gated_space(fmt, tokens, hidden, inter).bytes;
}

hipError_t launch_gated(int fmt, int act, const uint16_t* x, const uint8_t* packed, const void* scales, int64_t tokens,
                        int64_t hidden, int64_t inter, uint16_t* h, uint16_t* products, void* ws, hipStream_t s) {
  const GatedSpace g = gated_space(fmt, tokens, hidden, inter);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  const bool convert = fmt_xtype(fmt) == kBF16;
  DecodeArgs d;
  d.packed = packed;
  d.scales = scales;
  d.w = reinterpret_cast<uint16_t*>(base + g.w);
  d.fold = reinterpret_cast<float2*>(base + g.w);
  d.w_exp = reinterpret_cast<int*>(base + g.w_exp);
  d.n = (uint32_t)(2 * inter);
  d.k = (uint32_t)hidden;
  d.x = convert ? x : nullptr;
  d.xh = reinterpret_cast<uint16_t*>(base + g.xh);
  d.x_exp = reinterpret_cast<int*>(base + g.x_exp);
  d.t = (uint32_t)tokens;
  const bool fold = gated_packed(fmt, tokens, hidden, inter);
  const uint32_t per = kDecodeThreads / 64, token_rows = convert ? d.t : 0;
  const dim3 grid(fold ? (token_rows + per - 1) / per + (d.n + kFoldRows - 1) / kFoldRows
                       : (d.n + token_rows + per - 1) / per);
  auto decode = [&](auto format) {
    constexpr int F = decltype(format)::value;
    if (fold)
      fold_rows_kernel<F><<<grid, dim3(kDecodeThreads), 0, s>>>(d);
    else
      decode_rows_kernel<F><<<grid, dim3(kDecodeThreads), 0, s>>>(d);
  };
  using std::integral_constant;
  switch (fmt_weight(fmt)) {
    case kNF4: decode(integral_constant<int, kNF4>{}); break;
    case kINT4: decode(integral_constant<int, kINT4>{}); break;
    case kFP4: decode(integral_constant<int, kFP4>{}); break;
    case kINT4A: decode(integral_constant<int, kINT4A>{}); break;
    default: decode(integral_constant<int, kMXFP4>{}); break;
  }
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  DenseArgs a{};
  a.a = reinterpret_cast<const uint8_t*>(convert ? d.xh : x);
  a.b = fold ? packed : reinterpret_cast<const uint8_t*>(d.w);
  a.scales = fold ? reinterpret_cast<const float*>(d.fold) : nullptr;
  a.m = (uint32_t)tokens;
  a.n = (uint32_t)inter;
  a.pitch = (uint32_t)(2 * hidden);
  a.terms = (uint32_t)dense_terms(fmt_weight(fmt));
  a.row_exp = convert ? d.x_exp : nullptr;
  a.col_exp = d.w_exp;
  a.partial = reinterpret_cast<uint32_t*>(base + g.partial);
  a.out = h;
  a.products = products;
  a.out_type = convert ? 2 : 1;
  a.act = (uint32_t)act;
  if (!fold) return launch_dense(kDenseF16, true, a, s);
  switch (fmt_weight(fmt)) {
    case kNF4: return launch_dense_nf4(a, s);
    case kFP4: return launch_dense_fp4(a, s);
    case kMXFP4: return launch_dense_mxfp4(a, s);
    case kINT4: return launch_dense_int4(a, s);
    default: return launch_dense_int4a(a, s);
  }
}

hipError_t launch_gated_grad(int xt, int act, const uint16_t* dh, const uint16_t* products, int64_t tokens,
                             int64_t inter, uint16_t* dp, hipStream_t s) {
  if (xt == kF16)
    return act == W4_ACT_SILU ? grad_launch<kF16, W4_ACT_SILU>(dh, products, dp, tokens, inter, s)
                              : grad_launch<kF16, W4_ACT_GELU_TANH>(dh, products, dp, tokens, inter, s);
  return act == W4_ACT_SILU ? grad_launch<kBF16, W4_ACT_SILU>(dh, products, dp, tokens, inter, s)
                            : grad_launch<kBF16, W4_ACT_GELU_TANH>(dh, products, dp, tokens, inter, s);
}

}  // namespace w4
