// Copies from memory to LDS for the dense kernel (w4_dense.h), and its sources of four-bit weights.
#pragma once
#include "w4_ffn.h"
#include "w4_ffn_math.h"
#include "w4_mfma_common.h"

namespace w4 {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// A raw buffer resource as four scalars (make_rsrc's form, for the copies below).
__device__ inline i32x4 dense_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  i32x4 r;
  r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
  r.y = __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
  r.z = __builtin_amdgcn_readfirstlane((int)bytes);
  r.w = 0x00020000;
  return r;
}

// Copies 16 bytes a lane from offset `off` of the resource to LDS, lane l's to `to` + 16 l (`to` uniform).  By hand,
// because the compiler makes an LDS read wait for copies that it cannot tell from the one that filled what is read;
// here the kernel's own waits say which have landed.  It has no result register; its address is read as it issues; m0
// holds nothing else (the compiler sets it right before each use of its own).  No memory clobber: copies keep their
// order to each other and to the barriers, and only to those.
__device__ inline void dense_copy(i32x4 r, const uint8_t* to, uint32_t off) {
  const uint32_t lds = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)to;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(
                   __builtin_amdgcn_readfirstlane((int)lds)),
               "v"(off), "s"(r));
}

// The same for 4 bytes a lane, and for 2 (to a dword each).
__device__ inline void dense_copy2(i32x4 r, const uint8_t* to, uint32_t off) {
  const uint32_t lds = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)to;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ushort %1, %2, 0 offen lds" ::"s"(
                   __builtin_amdgcn_readfirstlane((int)lds)),
               "v"(off), "s"(r));
}
__device__ inline void dense_copy4(i32x4 r, const uint8_t* to, uint32_t off) {
  const uint32_t lds = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)to;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(
                   __builtin_amdgcn_readfirstlane((int)lds)),
               "v"(off), "s"(r));
}

__device__ inline __amdgpu_buffer_rsrc_t dense_buffer(i32x4 r) {
  return __builtin_amdgcn_make_buffer_rsrc(
      reinterpret_cast<void*>((uint64_t)(uint32_t)r.x | ((uint64_t)(uint32_t)r.y << 32)), (short)0, r.z, r.w);
}

// B in four bits.  A source of the dense kernel's B tile writes the stage that the copies would have filled: the packed
// bytes and scales of a wave's part come to LDS of its own (which leaves the counting of loads in flight to the kernel) a
// step ahead of their use, and a quarter of them is decoded, scaled, rounded to 16 bits and written in each quarter of a
// step.  The kernel calls, a step t: copy(t) asks for its bytes; once they have landed take() reads them, and after
// settle() the next copy() may overwrite them; then look(q, i), put(stage, q, i) for quarters q and fourths i of them, each
// look() before its put() (NF4 asks the table some matrix instructions earlier).  first_steps() loads the first ones
// without LDS.

// a * s rounded to fp32 and to fp16, two of them in a dword, a in fp16 (the halves of c).
__device__ inline uint32_t scaled_halves(uint32_t c, float s) {
  uint32_t d;
  asm("v_fma_mixlo_f16 %0, %1, %2, 0 op_sel_hi:[1,0,0]" : "=v"(d) : "v"(c), "v"(s));
  asm("v_fma_mixhi_f16 %0, %1, %2, 0 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "+v"(d) : "v"(c), "v"(s));
  return d;
}
// a * s - h rounded the same way, h the fp16 halves of a dword: what a first term leaves of a product.
__device__ inline uint32_t rest_of_halves(uint32_t c, float s, uint32_t h) {
  uint32_t d;
  asm("v_fma_mixlo_f16 %0, %1, %2, -%3 op_sel_hi:[1,0,1]" : "=v"(d) : "v"(c), "v"(s), "v"(h));
  asm("v_fma_mixhi_f16 %0, %1, %2, -%3 op_sel:[1,0,1] op_sel_hi:[1,0,1]" : "+v"(d) : "v"(c), "v"(s), "v"(h));
  return d;
}

// The weights of a packed dword, two of them at a time, in fp16: code (exact) times scale, or one of the two terms that
// such a product is held in (first_term in w4_ffn_math.h).
//   * E2M1: the hardware's conversion to fp16, which takes the low nibble first: the nibbles are swapped before.
//     MXFP4's scales are powers of two, which it applies itself (NaN too).
//   * INT4: the nibbles as bytes below 0x64, which is 1024 + q in fp16, less 1024 + the offset.
//   * NF4: fp32 codes from a table in LDS, sixteen banks of it, so lanes never wait for each other.
template <int FMT, int TERMS>
struct DenseDecoder {
  uint32_t a, b;
  float s, s1;  // the scale, and the first term's
  uint32_t bias;
  float code[8];  // NF4: asked for some matrix instructions before they are used
  template <int J>
  __device__ inline void look(const float* table) {
    const uint8_t* t = reinterpret_cast<const uint8_t*>(table);
    code[2 * J] = *reinterpret_cast<const float*>(t + ((a >> (8 * J)) & 0xFFu));
    code[2 * J + 1] = *reinterpret_cast<const float*>(t + ((b >> (8 * J)) & 0xFFu));
  }
  __device__ inline void set(uint32_t w, BlockScale k) {
    s = k.s;
    s1 = TERMS == 2 ? first_term(s) : s;
    if constexpr (FMT == kFP4 || FMT == kMXFP4) {
      a = ((w >> 4) & 0x0F0F0F0Fu) | ((w & 0x0F0F0F0Fu) << 4);
    } else if constexpr (FMT == kNF4) {
      a = (w >> 2) & 0x3C3C3C3Cu;  // byte offsets of the first nibbles' codes, and of the second's
      b = (w << 2) & 0x3C3C3C3Cu;
    } else {
      const uint32_t h = (w >> 4) & 0x0F0F0F0Fu, l = w & 0x0F0F0F0Fu;
      a = __builtin_amdgcn_perm(h, l, 0x01050004u);  // codes 0 1 2 3 of this dword's eight as bytes, then 4 5 6 7
      b = __builtin_amdgcn_perm(h, l, 0x03070206u);
      const _Float16 z = (_Float16)(1024.0f + k.zero);
      bias = (uint32_t)__builtin_bit_cast(uint16_t, z) * 0x10001u;
    }
  }
  // Pair J of the dword, its term T.
  template <int J, int T>
  __device__ inline uint32_t pair() const {
    if constexpr (FMT == kMXFP4) {
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(a, s, J));
    } else if constexpr (FMT == kNF4) {
      const uint32_t h = scaled_pair(code[2 * J], code[2 * J + 1], s1);
      return T == 0 ? h : rest_of_pair(code[2 * J], code[2 * J + 1], s, h);
    } else {
      const uint32_t c = halves<J>(), h = scaled_halves(c, s1);
      return T == 0 ? h : rest_of_halves(c, s, h);
    }
  }
  // The codes of pair J as fp16 numbers.
  template <int J>
  __device__ inline uint32_t halves() const {
    if constexpr (FMT == kFP4) {
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(a, 1.0f, J));
    } else {
      typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
      const uint32_t q = __builtin_amdgcn_perm(0x64646464u, J < 2 ? a : b, J & 1 ? 0x04030402u : 0x04010400u);
      return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, q) - __builtin_bit_cast(half2_t, bias));
    }
  }
};

constexpr int kRawBytes = 64 * 16 + 64 * 4;  // a step's packed bytes and scales of a wave

// Rows of packed weights along K (w4_gated): a wave has 32 rows of the tile, a lane 32 weights of row lane / 2 in a step, in
// chunks of 8.  The scales are folded (w4_gated.hip), two numbers a step.
template <int FMT, int TERMS, int TM, int TN, int W, int STAGES>
struct PackedRows {
  static_assert(TN == 32 * W, "32 rows of B a wave");
  uint8_t* own;
  uint8_t* ring;
  const float* table;
  i32x4 rw, rs;
  uint32_t woff, soff, to, steps, half, lane;
  uint4 w;
  float s;
  uint4 ahead_w[STAGES];
  float ahead_s[STAGES];
  BlockScale scale;
  DenseDecoder<FMT, TERMS> dec;
  uint32_t made[4];

  // Rows n0 .. of the tile, gate rows first (CN of them, `nrows` exist), then up rows.
  __device__ inline void init(const DenseArgs& p, uint32_t n0, uint32_t nrows, uint32_t last, uint8_t* raw, uint8_t* stages,
                              const float* codes, int lane_, int wave) {
    constexpr uint32_t CN = TN / 2;
    own = raw + wave * kRawBytes;
    ring = stages;
    table = codes;
    steps = last / TERMS;  // of A's
    lane = (uint32_t)lane_;
    const uint32_t r = 32 * wave, up = r >= CN ? 1u : 0u, at = r - (up ? CN : 0u);
    const size_t row = (size_t)(up ? p.n : 0u) + n0 + at;
    const uint32_t rows = at < nrows ? min(32u, nrows - at) : 0u;
    rw = dense_rsrc(p.b + row * (p.pitch / 4), rows * (p.pitch / 4));
    rs = dense_rsrc(reinterpret_cast<const uint8_t*>(p.scales) + row * (p.pitch / 16), rows * (p.pitch / 16));
    const uint32_t of = lane >> 1;
    half = lane & 1u;
    woff = of * (p.pitch / 4) + half * 16;
    soff = of * (p.pitch / 16) + half * 4;
    to = (TM + r + of) * 128 + ((4u * half) ^ ((of >> 1) & 7u)) * 16;
  }
  __device__ inline void first_steps(uint32_t first) {
    const __amdgpu_buffer_rsrc_t bw = dense_buffer(rw), bs = dense_buffer(rs);
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
      const uint32_t t = (first + i) / TERMS;
      ahead_w[i] = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(bw, woff + (t < steps ? t * 32 : 0x40000000u), 0, 0));
      ahead_s[i] =
          __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(bs, soff + (t < steps ? t * 8 : 0x40000000u), 0, 0));
    }
  }
  __device__ inline void use_first(int i) {
    w = ahead_w[i];
    s = ahead_s[i];
    scales();
  }
  __device__ inline void copy(uint32_t t) {  // past the last step: from outside the buffers
    t /= TERMS;
    dense_copy(rw, own, woff + (t < steps ? t * 32 : 0x40000000u));
    dense_copy4(rs, own + 1024, soff + (t < steps ? t * 8 : 0x40000000u));
  }
  __device__ inline void take() {
    w = *reinterpret_cast<const uint4*>(own + lane * 16);
    s = *reinterpret_cast<const float*>(own + 1024 + lane * 4);
  }
  __device__ inline void scales() {
    scale = BlockScale{s, 8.0f};
    if constexpr (is_g128(FMT)) {  // the pair's first lane has the scale, its second the zero point
      const float other =
          __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(s), 0xB1, 0xF, 0xF, true));
      scale = half ? BlockScale{other, s} : BlockScale{s, other};
    }
  }
  __device__ inline void settle() {
    asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w), "+v"(s));
    scales();
  }
  template <int I>
  __device__ inline void look(int q) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    if (I == 0) dec.set(v[q], scale);
    if constexpr (FMT == kNF4) dec.template look<I>(table);
  }
  template <int I, int T>
  __device__ inline void put(uint32_t stage, int q) {
    made[I] = dec.template pair<I, T>();
    if (I == 3)
      *reinterpret_cast<uint4*>(ring + ((to + stage) ^ (uint32_t)(q * 16))) = make_uint4(made[0], made[1], made[2], made[3]);
  }
};

// Two products rounded to fp32 (with an addend) and to fp16, in a dword.
__device__ inline uint32_t fma_halves(float a, float s, float add, float b, float t, float more) {
  uint32_t d;
  asm("v_fma_mixlo_f16 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(s), "v"(add));
  asm("v_fma_mixhi_f16 %0, %1, %2, %3" : "+v"(d) : "v"(b), "v"(t), "v"(more));
  return d;
}

// Columns of packed weights (w4_gemm_grad): the sum runs along the weight rows, so a step's 64 of them, each with TN / 8
// dwords of the tile's columns, have to be transposed.  A wave has 64 / W rows, a lane 8 columns (a dword) of four rows 4 a
// .. 4 a + 3 among them; a quarter is the two columns of a byte, four weights of each, 8 bytes of a stage's row.
//   * The chunks of stage row r are keyed on (r / 2) xor (r / 8): 32 lanes write to every eighth row, and so to 8 slots; the
//     rows that a 16-lane group reads still have 8 different keys.
//   * Scales come in the format's own form: one for each row and 64 or 128 columns; fp16 takes them times 2^-f, f of a
//     unit of columns, and where TERMS is 2 a weight in its two terms.
template <int FMT, int TERMS, int TYPE, int TM, int TN, int W, int STAGES>
struct PackedColumns {
  static_assert(TN == 32 * W, "64 rows of weights in the waves of a workgroup");
  static constexpr uint32_t RPW = 64 / W;        // rows a wave
  static constexpr uint32_t DW = TN / 8;         // dwords of a row
  static constexpr uint32_t SU = TN / (is_g128(FMT) ? 128 : 64);  // scale units of a row
  static constexpr uint32_t SB = FMT == kINT4 || FMT == kMXFP4 ? 2 : 4;
  uint8_t* own;
  uint8_t* ring;
  const float* table;
  const uint8_t* packed;
  const uint8_t* scale_rows;
  uint64_t wstep, sstep;  // bytes of 64 rows
  uint32_t wbytes, sbytes;  // bytes of a row
  uint32_t woff, soff, to, n, steps, from, lane, unit, dcol, scol;
  int f;
  bool odd;  // MXFP4: the second 32 columns of a unit
  uint32_t w[4], b[4];
  uint32_t ahead_w[STAGES][4], ahead_b[STAGES][4];
  float s[4], add[4];    // w = code * s + add
  float s1[4], add1[4];  // what its first term is rounded from
  float code[8];
  uint32_t lo[2], hi[2];

  __device__ inline void init(const DenseArgs& p, uint32_t k0, uint32_t last, uint8_t* raw, uint8_t* stages,
                              const float* codes, int lane_, int wave) {
    own = raw + wave * kRawBytes;
    ring = stages;
    table = codes;
    lane = (uint32_t)lane_;
    steps = last / TERMS;  // of A's
    n = p.rows;
    wbytes = p.n / 2;
    sbytes = p.n / (is_g128(FMT) ? 128 : 64) * SB;
    wstep = (uint64_t)wbytes * 64;
    sstep = (uint64_t)sbytes * 64;
    packed = p.b;
    scale_rows = reinterpret_cast<const uint8_t*>(p.scales);
    const uint32_t first_row = RPW * wave;
    {  // the copies: 16 bytes of row lane / (DW / 4), a scale of row lane / SU
      const uint32_t r = lane / (DW / 4), c = lane % (DW / 4), k = k0 + 32 * c;
      woff = k < p.n ? (first_row + r) * wbytes + k / 2 : kOutOfRange;
      const uint32_t sr = lane / SU, u = lane % SU, ku = k0 + u * (is_g128(FMT) ? 128 : 64);
      soff = sr < RPW && ku < p.n ? (first_row + sr) * sbytes + ku / (is_g128(FMT) ? 128 : 64) * SB : kOutOfRange;
    }
    const uint32_t c = lane % DW, a = lane / DW;
    unit = c * 8 / (is_g128(FMT) ? 128 : 64);
    odd = FMT == kMXFP4 && (c * 8 / 32) % 2;
    from = (4 * a) * DW + c;  // the first of its four dwords
    dcol = (first_row + 4 * a) * wbytes + k0 / 2 + 4 * c;
    scol = (first_row + 4 * a) * sbytes + (k0 + 8 * c) / (is_g128(FMT) ? 128 : 64) * SB;
    if (k0 + 8 * c >= p.n) dcol = scol = kOutOfRange - 4 * wbytes;
    const uint32_t chunk = (first_row + 4 * a) / 8, key = (4 * (c & 1)) ^ (c & 7);
    to = (TM + 8 * c) * 128 + ((chunk ^ key) & 7u) * 16 + 8 * (a & 1);
  }
  __device__ inline i32x4 rows_of(const uint8_t* base, uint64_t step, uint32_t bytes, uint32_t t) {
    const uint32_t left = t < steps ? min(64u, n - 64 * t) : 0u;
    return dense_rsrc(base + (t < steps ? t * step : 0), left * bytes);
  }
  __device__ inline void first_steps(uint32_t first) {
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
      const __amdgpu_buffer_rsrc_t bw = dense_buffer(rows_of(packed, wstep, wbytes, (first + i) / TERMS));
      const __amdgpu_buffer_rsrc_t bs = dense_buffer(rows_of(scale_rows, sstep, sbytes, (first + i) / TERMS));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        ahead_w[i][r] = __builtin_amdgcn_raw_buffer_load_b32(bw, dcol + r * wbytes, 0, 0);
        const uint32_t so = scol + r * sbytes;
        ahead_b[i][r] = SB == 2 ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(bs, so, 0, 0)
                                : __builtin_amdgcn_raw_buffer_load_b32(bs, so, 0, 0);
      }
    }
  }
  __device__ inline void use_first(int i) {
#pragma unroll
    for (int r = 0; r < 4; ++r) w[r] = ahead_w[i][r], b[r] = ahead_b[i][r];
    scales();
  }
  __device__ inline void copy(uint32_t t) {
    t /= TERMS;
    dense_copy(rows_of(packed, wstep, wbytes, t), own, woff);
    const i32x4 rs = rows_of(scale_rows, sstep, sbytes, t);
    if constexpr (SB == 2)
      dense_copy2(rs, own + 1024, soff);
    else
      dense_copy4(rs, own + 1024, soff);
  }
  __device__ inline void take() {
    const uint32_t* v = reinterpret_cast<const uint32_t*>(own);
    const uint32_t* u = v + 256 + from / DW * SU + unit;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      w[r] = v[from + r * DW];
      b[r] = u[r * SU];
    }
  }
  __device__ inline void scales() {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float zero = 8.0f;
      if constexpr (FMT == kMXFP4)
        s[r] = e8m0_value((odd ? b[r] >> 8 : b[r]) & 255u);
      else if constexpr (is_g128(FMT))
        s[r] = __uint_as_float(b[r] << 16);
      else
        s[r] = __uint_as_float(b[r]);
      if constexpr (FMT == kINT4A) zero = (float)((b[r] >> 16) & 15u);
      if constexpr (TYPE == kDenseF16) s[r] = ldexpf(s[r], -f);
      s1[r] = TERMS == 2 ? first_term(s[r]) : s[r];
      add[r] = is_g128(FMT) ? -zero * s[r] : 0.0f;  // exact: 8 and 4 bits
      add1[r] = is_g128(FMT) ? -zero * s1[r] : 0.0f;  // exact: 18 and 4
    }
  }
  __device__ inline void settle() {
    asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]), "+v"(b[0]), "+v"(b[1]), "+v"(b[2]), "+v"(b[3]));
    scales();
  }
  // The codes of row I's byte q, the first column's and the second's.
  template <int I>
  __device__ inline void look(int q) {
    if constexpr (FMT == kNF4) {
      const uint8_t* t = reinterpret_cast<const uint8_t*>(table);
      const uint32_t v = w[I] >> (8 * q);
      code[2 * I] = *reinterpret_cast<const float*>(t + ((v >> 2) & 0x3Cu));
      code[2 * I + 1] = *reinterpret_cast<const float*>(t + ((v << 2) & 0x3Cu));
    } else if constexpr (FMT == kFP4 || FMT == kMXFP4) {
      decode_pair<FMT>(w[I], q, nullptr, BlockScale{1.0f, 0.0f}, &code[2 * I], &code[2 * I + 1]);
    } else {
      const uint32_t v = w[I] >> (8 * q);
      code[2 * I] = (float)((v >> 4) & 15u);
      code[2 * I + 1] = (float)(v & 15u);
    }
  }
  // Term T of the weights of codes a and b, of rows I - 1 and I.
  template <int I, int T>
  __device__ inline uint32_t pair(float a, float b) const {
    if constexpr (TYPE != kDenseF16) return bf16_pair(a * s[I - 1], b * s[I]);  // (MXFP4: exact)
    const uint32_t h = fma_halves(a, s1[I - 1], add1[I - 1], b, s1[I], add1[I]);
    if constexpr (T == 0) return h;
    if constexpr (is_g128(FMT))  // (the sums are exact: 12 bits)
      return rest_of_pair(__builtin_fmaf(a, s[I - 1], add[I - 1]), __builtin_fmaf(b, s[I], add[I]), 1.0f, 1.0f, h);
    return rest_of_pair(a, b, s[I - 1], s[I], h);
  }
  template <int I, int T>
  __device__ inline void put(uint32_t stage, int q) {
    if constexpr (I % 2 == 1) {
      lo[I / 2] = pair<I, T>(code[2 * I - 2], code[2 * I]);
      hi[I / 2] = pair<I, T>(code[2 * I - 1], code[2 * I + 1]);
    }
    if (I == 3) {
      uint8_t* at = ring + ((to + stage) ^ (uint32_t)(q * 16)) + 2 * q * 128;
      *reinterpret_cast<uint2*>(at) = make_uint2(lo[0], lo[1]);
      *reinterpret_cast<uint2*>(at + 128) = make_uint2(hi[0], hi[1]);
    }
  }
};

}  // namespace
}  // namespace w4
