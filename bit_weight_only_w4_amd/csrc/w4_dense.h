// Dense product of two row-major operands with K contiguous, C[m, n] = sum_k A[m, k] B[n, k], on the matrix
// cores: fp16 or bf16 (32x32x16 steps, fp32 sums) or 8-bit integers (32x32x32 steps, int32 sums, exact).  A lane's
// fragment is 16 bytes in every type, so one kernel moves bytes and only the matrix instruction differs.
//
// Work layout.  A workgroup of WM x WN waves owns a tile of TM = 32 MT WM rows of A by TN = 32 NT WN rows of B and
// walks K in steps of 128 bytes (whole cache lines: steps of 64 asked the L2 for each line twice, two thirds of the
// requests it can serve) through a ring of STAGES stages.  Both operand tiles of a step come straight from memory
// into LDS (buffer loads with the LDS destination).  One barrier a step, before its last quarter: by then a wave has
// read its last fragments of the stage, and waits for its own copies of the next one; behind it every wave finds the
// next stage whole and this one free for the copies of the step STAGES further.  A wave's fragments are a quarter
// ahead of its matrix instructions, across the barrier too.
//   * Stage layout: 128 bytes a row, the 16-byte chunk c of row r in slot c XOR (r / 2 mod 8): the sixteen rows that
//     a 16-lane group of a 128-bit LDS read takes then lie in distinct banks.
//   * A (32 rows x 32 bytes): lane 32 h + c takes row c, bytes 16 h .. 16 h + 15 of the quarter.  B the same.
//   * D (32 x 32): lane 32 h + c holds column c (a row of B), rows 8 (e / 4) + 4 h + e % 4 (register e).
//   * Gated: the B tile holds TN / 2 gate rows, then the up rows of the same channels; a wave's even column tiles
//     are gate, its odd ones the up of the same channels, so the activation and the product happen in registers.
//   * Rows past M or N and bytes past K are read at an offset outside the buffer, which gives zeros.
//   * B in four bits: a wave's packed weights and their scales come to LDS of its own a step ahead, and between the matrix
//     instructions it decodes them, scales them, rounds them to 16 bits and writes them into the stage where the copies
//     would have put them: rows of weights for the gated block (PackedRows), columns for a gradient (PackedColumns).
//
// What bounds it is the matrix cores under the card's power limit: its rate depends on the data.  4096 x 8192 x 8192: int8
// 245 to 260 us (2110 to 2240 Tops/s; the library's product 2090), fp16 1160 TFLOP/s (1250).  One wave of every SIMD waits
// while the other issues: with the copies in one burst behind the barrier, or with steps of 64 bytes, int8 took 300 us and
// more.
#pragma once
#include <type_traits>

#include "w4_ffn.h"
#include "w4_ffn_math.h"
#include "w4_mfma_common.h"

namespace w4 {

struct DensePlan {
  double us;  // the estimate
  int tile;
  uint32_t splits, per;
  uint32_t tiles, rest;  // tiles in all, and how many of the last are covered with 64 x 128 tiles by a second launch
};
DensePlan plan_dense(bool gated, int64_t m, int64_t n, int64_t pitch, int packed);
// Sets what a launch of the plan needs; false where it has too many tiles.
bool dense_prepare(const DensePlan& p, DenseArgs* a);

namespace {

// The tiles, largest first: waves along M and N, 32-row tiles of a wave along M and N, stages; how many workgroups of it
// a CU holds (LDS), and what was measured (MI355X, over twelve shapes of 1 to 4096 rows, fp16 and int8): microseconds
// a step of 128 bytes when alone on a CU and when the CU is full, and a round's start and end.
struct Tile {
  int tm, tn, fit;
  double alone, full, ends;
};
constexpr Tile kTiles[] = {{256, 256, 1, 1.85, 1.85, 5}, {128, 256, 1, 0.95, 0.95, 4.5}, {64, 128, 2, 0.34, 0.72, 3},
                           {32, 128, 2, 0.33, 0.60, 3}};
constexpr int kTileCount = 4;  // (four bits: without the last, whose waves would hold 64 rows of B)
constexpr int kRestTile = 2;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

template <int TYPE>
struct DenseAcc {
  using type = f32x16;
};
template <>
struct DenseAcc<kDenseI8> {
  using type = i32x16;
};

template <int TYPE>
__device__ inline typename DenseAcc<TYPE>::type dense_mfma(const uint4& a, const uint4& b,
                                                           typename DenseAcc<TYPE>::type c) {
  if constexpr (TYPE == kDenseF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0,
                                                   0, 0);
  else if constexpr (TYPE == kDenseBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf168_t, a), __builtin_bit_cast(bf168_t, b), c,
                                                    0, 0, 0);
  else
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0,
                                                  0);
}

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

// a * s rounded to fp32 and to fp16, two of them in a dword: a in fp16 (the halves of c) or in fp32.
__device__ inline uint32_t scaled_halves(uint32_t c, float s) {
  uint32_t d;
  asm("v_fma_mixlo_f16 %0, %1, %2, 0 op_sel_hi:[1,0,0]" : "=v"(d) : "v"(c), "v"(s));
  asm("v_fma_mixhi_f16 %0, %1, %2, 0 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "+v"(d) : "v"(c), "v"(s));
  return d;
}
__device__ inline uint32_t scaled_pair(float a, float b, float s) {
  uint32_t d;
  asm("v_fma_mixlo_f16 %0, %1, %2, 0" : "=v"(d) : "v"(a), "v"(s));
  asm("v_fma_mixhi_f16 %0, %1, %2, 0" : "+v"(d) : "v"(b), "v"(s));
  return d;
}

// The weights of a packed dword, two of them at a time, in fp16: code (exact) times scale.
//   * E2M1: the hardware's conversion to fp16, which takes the low nibble first: the nibbles are swapped before.
//     MXFP4's scales are powers of two, which it applies itself (NaN too).
//   * INT4: the nibbles as bytes below 0x64, which is 1024 + q in fp16, less 1024 + the offset.
//   * NF4: fp32 codes from a table in LDS, sixteen banks of it, so lanes never wait for each other.
template <int FMT>
struct DenseDecoder {
  uint32_t a, b;
  float s;
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
  template <int J>
  __device__ inline uint32_t pair() const {
    if constexpr (FMT == kMXFP4) {
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(a, s, J));
    } else if constexpr (FMT == kFP4) {
      return scaled_halves(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(a, 1.0f, J)), s);
    } else if constexpr (FMT == kNF4) {
      return scaled_pair(code[2 * J], code[2 * J + 1], s);
    } else {
      typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
      const uint32_t q = __builtin_amdgcn_perm(0x64646464u, J < 2 ? a : b, J & 1 ? 0x04030402u : 0x04010400u);
      return scaled_halves(
          __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, q) - __builtin_bit_cast(half2_t, bias)), s);
    }
  }
};

constexpr int kRawBytes = 64 * 16 + 64 * 4;  // a step's packed bytes and scales of a wave

// Rows of packed weights along K (w4_gated): a wave has 32 rows of the tile, a lane 32 weights of row lane / 2 in a step, in
// chunks of 8.  The scales are folded (w4_gated.hip), two numbers a step.
template <int FMT, int TM, int TN, int W, int STAGES>
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
  DenseDecoder<FMT> dec;
  uint32_t made[4];

  // Rows n0 .. of the tile, gate rows first (CN of them, `nrows` exist), then up rows.
  __device__ inline void init(const DenseArgs& p, uint32_t n0, uint32_t nrows, uint32_t last, uint8_t* raw, uint8_t* stages,
                              const float* codes, int lane_, int wave) {
    constexpr uint32_t CN = TN / 2;
    own = raw + wave * kRawBytes;
    ring = stages;
    table = codes;
    steps = last;
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
      const uint32_t t = first + i;
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
    dense_copy(rw, own, woff + (t < steps ? t * 32 : 0x40000000u));
    dense_copy4(rs, own + 1024, soff + (t < steps ? t * 8 : 0x40000000u));
  }
  __device__ inline void take() {
    w = *reinterpret_cast<const uint4*>(own + lane * 16);
    s = *reinterpret_cast<const float*>(own + 1024 + lane * 4);
  }
  __device__ inline void scales() {
    scale = BlockScale{s, 8.0f};
    if constexpr (FMT == kINT4A) {  // the pair's first lane has the scale, its second the zero point
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
  template <int I>
  __device__ inline void put(uint32_t stage, int q) {
    made[I] = dec.template pair<I>();
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
//   * Scales come in the format's own form: one for each row and 64 or 128 columns; fp16 takes them times 2^-f.
template <int FMT, int TYPE, int TM, int TN, int W, int STAGES>
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
  float s[4], add[4];
  float code[8];
  uint32_t lo[2], hi[2];

  __device__ inline void init(const DenseArgs& p, uint32_t k0, uint32_t last, int exponent, uint8_t* raw, uint8_t* stages,
                              const float* codes, int lane_, int wave) {
    own = raw + wave * kRawBytes;
    ring = stages;
    table = codes;
    lane = (uint32_t)lane_;
    steps = last;
    n = p.rows;
    f = exponent;
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
      const __amdgpu_buffer_rsrc_t bw = dense_buffer(rows_of(packed, wstep, wbytes, first + i));
      const __amdgpu_buffer_rsrc_t bs = dense_buffer(rows_of(scale_rows, sstep, sbytes, first + i));
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
      add[r] = is_g128(FMT) ? -zero * s[r] : 0.0f;  // exact: 8 and 4 bits
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
  template <int I>
  __device__ inline void put(uint32_t stage, int q) {
    if constexpr (I % 2 == 1) {
      if constexpr (TYPE == kDenseF16) {
        lo[I / 2] = fma_halves(code[2 * I - 2], s[I - 1], add[I - 1], code[2 * I], s[I], add[I]);
        hi[I / 2] = fma_halves(code[2 * I - 1], s[I - 1], add[I - 1], code[2 * I + 1], s[I], add[I]);
      } else {
        lo[I / 2] = to16<kBF16>(__builtin_fmaf(code[2 * I - 2], s[I - 1], add[I - 1])) |
                    (to16<kBF16>(__builtin_fmaf(code[2 * I], s[I], add[I])) << 16);
        hi[I / 2] = to16<kBF16>(__builtin_fmaf(code[2 * I - 1], s[I - 1], add[I - 1])) |
                    (to16<kBF16>(__builtin_fmaf(code[2 * I + 1], s[I], add[I])) << 16);
      }
    }
    if (I == 3) {
      uint8_t* at = ring + ((to + stage) ^ (uint32_t)(q * 16)) + 2 * q * 128;
      *reinterpret_cast<uint2*>(at) = make_uint2(lo[0], lo[1]);
      *reinterpret_cast<uint2*>(at + 128) = make_uint2(hi[0], hi[1]);
    }
  }
};

template <int TYPE, bool GATED, int FMT, int WM, int WN, int MT, int NT, int STAGES>
__global__ void __launch_bounds__(64 * WM * WN) dense_kernel(DenseArgs p) {
  constexpr int W = WM * WN, TM = 32 * MT * WM, TN = 32 * NT * WN;
  constexpr int ROWS = TM + TN;             // rows of a stage
  constexpr bool PACKED = FMT >= 0;         // B in four bits
  constexpr int COPIES = (PACKED ? TM : ROWS) / 8 / W;  // copies of 8 rows a wave makes for a stage
  static_assert(TM % (8 * W) == 0 && (PACKED || (GATED ? TN / 2 : TN) % (8 * W) == 0), "a round of copies fills one operand");
  static_assert(!GATED || NT % 2 == 0, "gate and up in one wave");
  __shared__ __align__(16) uint8_t ring[STAGES][ROWS * 128];
  __shared__ __align__(16) uint8_t raw[PACKED ? W * kRawBytes : 16];
  __shared__ float table[16];
  using Acc = typename DenseAcc<TYPE>::type;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 31, h = lane >> 5;

  // Every eighth workgroup runs on one XCD: those take consecutive tiles, in blocks of up to eight tiles along M and as
  // many columns of B as are in work at once, so that both operands are read by few XCDs.
  // (A launch may cover the last tiles of a larger size with its own smaller ones.)
  constexpr uint32_t CN = GATED ? TN / 2 : TN;  // channels of a tile
  const uint32_t mt = (p.m + p.bm - 1) / p.bm, nt = (p.n + p.bn - 1) / p.bn;
  const uint32_t tiles = gridDim.x, share = tiles / 8, rem = tiles % 8;
  const uint32_t xcd = blockIdx.x % 8, at = xcd * share + min(xcd, rem) + blockIdx.x / 8;
  const uint32_t sm = p.bm / TM, parts = sm * (p.bn / CN);
  const uint32_t tile = p.tile0 + at / parts, part = at % parts;
  const uint32_t band = tile / (8 * nt), in_band = tile % (8 * nt), high = min(8u, mt - 8 * band);
  const uint32_t m0 = (8 * band + in_band % high) * p.bm + part % sm * TM, n0 = in_band / high * p.bn + part / sm * CN;
  if (m0 >= p.m || n0 >= p.n) return;  // uniform; a part of a larger tile past the end

  const uint32_t nrows = min(CN, p.n - n0);
  const i32x4 ra = dense_rsrc(p.a + (size_t)m0 * p.pitch, min((uint32_t)TM, p.m - m0) * p.pitch);
  i32x4 rb{}, ru{};  // B, gated: its gate and up rows
  if constexpr (!PACKED) {
    rb = dense_rsrc(p.b + (size_t)n0 * p.pitch, nrows * p.pitch);
    ru = dense_rsrc(p.b + (size_t)(GATED ? p.n + n0 : 0) * p.pitch, GATED ? nrows * p.pitch : 0u);
  }

  // Copy j of this wave fills rows 8 (W j + wave) .. + 7 of a stage: lane l slot l % 8 of row l / 8.  Its offsets:
  uint32_t off[COPIES];
  const uint32_t mine = (((uint32_t)lane & 7u) ^ ((4u * wave + ((uint32_t)lane >> 4)) & 7u)) * 16;  // the chunk, for W even
  static_assert(W % 2 == 0, "the same chunk in every copy");
#pragma unroll
  for (int j = 0; j < COPIES; ++j) {
    const uint32_t r = 8u * (uint32_t)(W * j + wave) + ((uint32_t)lane >> 3);
    const uint32_t row = r < (uint32_t)TM ? r : (r - TM) % CN;
    const uint32_t rows = r < (uint32_t)TM ? min((uint32_t)TM, p.m - m0) : nrows;
    off[j] = row < rows ? row * p.pitch + mine : kOutOfRange - p.pitch;
  }
  const uint32_t first = blockIdx.y * p.per, steps = min(first + p.per, (p.pitch + 127) / 128);  // this split's
  // Copy j of step t; past the last step copies are made all the same, from outside the buffers, so that the number
  // of copies in flight is the same in every step.
  auto copy = [&](const uint8_t* st, uint32_t t, int j) __attribute__((always_inline)) {
    uint32_t k = t < steps ? t * 128 : 0x40000000u;
    if constexpr (TYPE == kDenseI8) k = k + mine < p.pitch ? k : 0x40000000u;  // rows may end in the middle of a step
    const uint8_t* to = st + 8 * (W * j + wave) * 128;
    if (8 * W * j < TM)  // known when compiled
      dense_copy(ra, to, off[j] + k);
    else if (!GATED || 8 * W * j < TM + (int)CN)
      dense_copy(rb, to, off[j] + k);
    else
      dense_copy(ru, to, off[j] + k);
  };

  Acc acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  const uint32_t key = ((uint32_t)c >> 1) & 7u;  // every fragment row is c modulo 32
  struct Frags {
    uint4 a[MT], b[NT];
  };
  // Quarter s of the stage at byte `st` of the ring.
  const uint32_t base = (((uint32_t)h ^ key) * 16) + c * 128;
  constexpr bool COLUMNS = PACKED && !GATED;  // B rows are keyed as PackedColumns writes them
  const uint32_t bdiff = COLUMNS ? (((uint32_t)c >> 3) & 3u) * 16 : 0u;
  auto fetch = [&](Frags& f, uint32_t at, int i) __attribute__((always_inline)) {  // fragment i of a quarter
    const int j = i - MT;
    const int row = i < MT ? 32 * (MT * wm + i)
                           : TM + (GATED ? (j & 1) * (int)CN + 32 * (NT / 2 * wn + j / 2) : 32 * (NT * wn + j));
    static_assert(!COLUMNS || NT % 2 == 0, "a B tile's parity is its column tile's");
    const uint32_t x = COLUMNS && i >= MT ? bdiff ^ (uint32_t)((j & 1) * 64) : 0u;
    const uint4 v = *reinterpret_cast<const uint4*>(&ring[0][0] + ((at ^ x) + row * 128));
    if (i < MT)
      f.a[i] = v;
    else
      f.b[j] = v;
  };
  constexpr uint32_t SIZE = ROWS * 128;
  // The copies of a step are spread over the quarters in which its stage is free, the last of this step and the first
  // ones of the next (two stages: only the first, so that they have half a step to arrive): in one burst behind the
  // barrier they kept the waves from issuing matrix instructions.
  constexpr int C3 = STAGES == 2 ? (COPIES + 1) / 2 : (COPIES + 3) / 4;  // up to the end of quarter 3, 0, 1, 2
  constexpr int C0 = STAGES == 2 ? COPIES : COPIES < 2 * C3 ? COPIES : 2 * C3;
  constexpr int C1 = COPIES < 3 * C3 ? COPIES : 3 * C3;
  using std::integral_constant;
  using Source = typename std::conditional<GATED, PackedRows<PACKED ? FMT : kFP4, TM, PACKED ? TN : 32 * W, W, STAGES>,
                                           PackedColumns<PACKED ? FMT : kFP4, TYPE, TM, PACKED ? TN : 32 * W, W, STAGES>>::type;
  Source src;
  int all = 0;  // the exponent of all of B
  if constexpr (PACKED && GATED) src.init(p, n0, nrows, steps, raw, &ring[0][0], table, lane, wave);
  if constexpr (COLUMNS) {
    if constexpr (TYPE == kDenseF16) {  // from the scan's maxima, every wave for itself
      float top = 0.0f;
      for (uint32_t i = lane; i < p.nparts; i += 64) top = fmaxf(top, p.parts[i]);
      all = fold_exponent<FMT>(wave_max(top));
      if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.exp_out = all;
    }
    src.init(p, n0, steps, all, raw, &ring[0][0], table, lane, wave);
  }
  // A quarter: after each matrix instruction one of the next quarter's fragments is requested, and a copy now and then.
  auto quarter = [&](Frags& next, uint32_t st, auto which, const Frags& f, uint32_t to, uint32_t t, auto from, auto end)
      __attribute__((always_inline)) {
    constexpr int A = decltype(from)::value, Z = decltype(end)::value, ALL = MT * NT;
    constexpr int s = decltype(which)::value;  // the quarter whose fragments are requested
    constexpr int D0 = PACKED && s == 0 ? 1 : 0;
    const uint32_t at = (base + st) ^ (uint32_t)(s * 32);
#pragma unroll
    for (int q = 0; q < ALL; ++q) {
      acc[q / NT][q % NT] = dense_mfma<TYPE>(f.a[q / NT], f.b[q % NT], acc[q / NT][q % NT]);
#pragma unroll
      for (int i = 0; i < MT + NT; ++i)
        if (i * ALL / (MT + NT) == q) fetch(next, at, i);
      if constexpr (PACKED) {
        if (D0 && q == 1) {  // the packed bytes are in registers before the next ones are asked for
          src.settle();
          src.copy(t + 1);
        }
        if constexpr (FMT == kNF4) {
          if (D0 == q) src.template look<0>(s), src.template look<1>(s);
          if (D0 + (ALL - D0) / 3 == q) {
            src.template put<0>(to, s), src.template put<1>(to, s);
            src.template look<2>(s), src.template look<3>(s);
          }
          if (D0 + 2 * (ALL - D0) / 3 == q) src.template put<2>(to, s), src.template put<3>(to, s);
        } else {
          if (D0 == q) src.template look<0>(s), src.template put<0>(to, s);
          if (D0 + (ALL - D0) / 4 == q) src.template look<1>(s), src.template put<1>(to, s);
          if (D0 + 2 * (ALL - D0) / 4 == q) src.template look<2>(s), src.template put<2>(to, s);
          if (D0 + 3 * (ALL - D0) / 4 == q) src.template look<3>(s), src.template put<3>(to, s);
        }
      }
#pragma unroll
      for (int j = A; j < Z; ++j)
        if (D0 + (j - A) * (ALL - D0) / (Z - A > 0 ? Z - A : 1) == q) copy(&ring[0][0] + to, t, j);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  Frags f0, f1;
  if constexpr (PACKED) {
    code_table<FMT>(table);
    src.first_steps(first);
    __syncthreads();  // the table
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
#pragma unroll
      for (int j = 0; j < COPIES; ++j) copy(&ring[i][0], first + i, j);
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
      src.use_first(i);
#pragma unroll
      for (int q = 0; q < (i == STAGES - 1 ? 1 : 4); ++q) {
        src.template look<0>(q), src.template put<0>(i * SIZE, q);
        src.template look<1>(q), src.template put<1>(i * SIZE, q);
        src.template look<2>(q), src.template put<2>(i * SIZE, q);
        src.template look<3>(q), src.template put<3>(i * SIZE, q);
      }
    }
    src.copy(first + STAGES);
#pragma unroll
    for (int j = 0; j < C3; ++j) copy(&ring[STAGES - 1][0], first + STAGES - 1, j);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 + C3) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
#pragma unroll
      for (int j = 0; j < (i == STAGES - 1 ? C3 : COPIES); ++j) copy(&ring[i][0], first + i, j);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((STAGES - 2) * COPIES + C3) : "memory");
  }
#pragma unroll
  for (int i = 0; i < MT + NT; ++i) fetch(f0, base, i);
  uint32_t now = 0, spare = (STAGES - 1) * SIZE;  // the step's stage, and the last step's
  for (uint32_t t = first; t < steps; ++t) {
    const uint32_t u = t + STAGES - 1;
    quarter(f1, now, integral_constant<int, 1>{}, f0, spare, u, integral_constant<int, C3>{}, integral_constant<int, C0>{});
    quarter(f0, now, integral_constant<int, 2>{}, f1, spare, u, integral_constant<int, C0>{}, integral_constant<int, C1>{});
    quarter(f1, now, integral_constant<int, 3>{}, f0, spare, u, integral_constant<int, C1>{}, integral_constant<int, COPIES>{});
    // by hand: the compiler's own barrier waits for every copy in flight
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * COPIES) : "memory");
    spare = now;
    now = now + SIZE == STAGES * SIZE ? 0 : now + SIZE;
    if constexpr (PACKED) src.take();
    quarter(f0, now, integral_constant<int, 0>{}, f1, spare, u + 1, integral_constant<int, 0>{}, integral_constant<int, C3>{});
  }
  wait_all_vector_loads();  // no copy outlives the workgroup

  // Epilogue.  16 bits: the exponents come off exactly (ldexp).  8 bits: the int32 sum is rounded to fp32 and
  // multiplied by its token's and its channel's scale, at most 2^-24 each.  16-bit results of 32 rows go through LDS
  // (the ring is free: a part of it for each wave), so that a store writes whole 16-byte pieces of a row; fp32
  // results are stored from the registers, 128 bytes a row.
  __syncthreads();
  constexpr int CT = GATED ? NT / 2 : NT;   // column tiles of an output
  constexpr int CW = 32 * CT;               // its columns in this wave
  uint16_t* stage = reinterpret_cast<uint16_t*>(&ring[0][0]) + wave * 32 * CW;
  const uint32_t nw = n0 + (uint32_t)wn * CW;  // first column
  if (p.partial) {  // a split's sums as they are; dense_sum_kernel adds them
    const uint32_t width = GATED ? 2 * p.n : p.n;
    uint32_t* plane = p.partial + (size_t)blockIdx.y * p.m * width;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t m = m0 + 32 * (MT * wm + i) + 8 * (e / 4) + 4 * h + e % 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint32_t n = nw + 32 * (GATED ? j / 2 : j) + c;
          const auto v = acc[i][j][e];  // (a value: the cast of a vector's element itself takes another one)
          if (m < p.m && n < p.n)
            plane[(size_t)m * width + (GATED && (j & 1) ? p.n : 0u) + n] = __builtin_bit_cast(uint32_t, v);
        }
      }
    return;
  }
  const void* rows_of = TYPE == kDenseI8 ? (const void*)p.row_scale : (const void*)p.row_exp;
  const void* cols_of = TYPE == kDenseI8 ? (const void*)p.col_scale : (const void*)p.col_exp;
  const i32x4 rr = dense_rsrc(reinterpret_cast<const uint32_t*>(rows_of) + m0, rows_of ? min((uint32_t)TM, p.m - m0) * 4 : 0u);
  uint32_t cv[NT];  // this lane's channels
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const uint32_t n = nw + 32 * (GATED ? j / 2 : j) + c;
    cv[j] = cols_of && n < p.n ? reinterpret_cast<const uint32_t*>(cols_of)[(GATED && (j & 1) ? p.n : 0u) + n] : 0u;
  }
  if constexpr (TYPE != kDenseI8 && !COLUMNS) all = p.exp ? *p.exp : 0;
  // One output's 32 rows from row `mw` on, in LDS, to memory.
  auto flush = [&](void* out, uint32_t pitch, uint32_t n, uint32_t nend, uint32_t mw) __attribute__((always_inline)) {
    asm volatile("" ::: "memory");  // a wave's LDS accesses keep their order; the compiler's must too
    uint16_t* o = reinterpret_cast<uint16_t*>(out);
    if (p.wide) {
      constexpr int PER = CW / 8;  // pieces a row
#pragma unroll
      for (int q = 0; q < 32 * PER / 64; ++q) {
        const int at = q * 64 + lane, r = at / PER, piece = at % PER;
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * CW + piece * 8);
        if (mw + r < p.m && n + piece * 8 < nend)
          *reinterpret_cast<uint4*>(o + (size_t)(mw + r) * pitch + n + piece * 8) = v;
      }
    } else {
#pragma unroll 4
      for (int q = 0; q < 32 * CW / 64; ++q) {
        const int at = q * 64 + lane, r = at / CW, col = at % CW;
        if (mw + r < p.m && n + col < nend) o[(size_t)(mw + r) * pitch + n + col] = stage[r * CW + col];
      }
    }
    asm volatile("" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const uint32_t mw = m0 + 32 * (MT * wm + i);
    uint32_t rv[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x4 v = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(dense_buffer(rr), (32 * (MT * wm + i) + 8 * q + 4 * h) * 4, 0, 0));
      rv[4 * q] = v.x, rv[4 * q + 1] = v.y, rv[4 * q + 2] = v.z, rv[4 * q + 3] = v.w;
    }
    auto value = [&](int j, int e) __attribute__((always_inline)) {
      if constexpr (TYPE == kDenseI8)
        return (float)acc[i][j][e] * __uint_as_float(rv[e]) * __uint_as_float(cv[j]);
      else
        return ldexpf(acc[i][j][e], (int)rv[e] + (int)cv[j] + all);
    };
    auto put = [&](int e, int j, float v) __attribute__((always_inline)) {
      stage[(8 * (e / 4) + 4 * h + e % 4) * CW + 32 * j + c] =
          (uint16_t)(p.out_type == W4_F16 ? to16<kF16>(v) : to16<kBF16>(v));
    };
    if constexpr (GATED) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
#pragma unroll
        for (int j = 0; j < CT; ++j) {
          const float g = value(2 * j, e);
          const float y = p.act == W4_ACT_SILU ? act_value<W4_ACT_SILU>(g) : act_value<W4_ACT_GELU_TANH>(g);
          put(e, j, y * value(2 * j + 1, e));
        }
      flush(p.out, p.n, nw, p.n, mw);
      if (p.products) {
#pragma unroll
        for (int half_of = 0; half_of < 2; ++half_of) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
#pragma unroll
            for (int j = 0; j < CT; ++j) put(e, j, value(2 * j + half_of, e));
          flush(p.products, 2 * p.n, nw + (half_of ? p.n : 0u), half_of ? 2 * p.n : p.n, mw);
        }
      }
    } else if (p.out_type == W4_F32) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t m = mw + 8 * (e / 4) + 4 * h + e % 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint32_t n = nw + 32 * j + c;
          if (m < p.m && n < p.n) reinterpret_cast<float*>(p.out)[(size_t)m * p.n + n] = value(j, e);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
#pragma unroll
        for (int j = 0; j < NT; ++j) put(e, j, value(j, e));
      flush(p.out, p.n, nw, p.n, mw);
    }
  }
}

// Adds the splits' sums in split order and makes of them what the epilogue above does.  V columns a thread.
template <int TYPE, bool GATED, int V>
__global__ void __launch_bounds__(256) dense_sum_kernel(DenseArgs p) {
  const uint32_t n = (blockIdx.x * 256 + threadIdx.x) * V, m = blockIdx.y;
  if (n >= p.n) return;
  using T = typename std::conditional<TYPE == kDenseI8, int, float>::type;
  const uint32_t width = GATED ? 2 * p.n : p.n;
  const size_t plane = (size_t)p.m * width;
  T sum[GATED ? 2 : 1][V] = {};
#pragma unroll
  for (int q = 0; q < (GATED ? 2 : 1); ++q) {
    const T* at = reinterpret_cast<const T*>(p.partial) + (size_t)m * width + q * p.n + n;
#pragma unroll 4
    for (uint32_t z = 0; z < p.splits; ++z) {
      T v[V];
      __builtin_memcpy(v, at + z * plane, sizeof v);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[q][i] += v[i];
    }
  }
  const float rs = TYPE == kDenseI8 ? p.row_scale[m] : 0.0f;
  const int re = TYPE == kDenseI8 ? 0 : (p.row_exp ? p.row_exp[m] : 0) + (p.exp ? *p.exp : 0);
  float v[3][V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) {
      const uint32_t c = q * p.n + n + i;
      if constexpr (TYPE == kDenseI8)
        v[q][i] = (float)sum[q][i] * rs * p.col_scale[c];
      else
        v[q][i] = ldexpf(sum[q][i], re + (p.col_exp ? p.col_exp[c] : 0));
    }
    if constexpr (GATED)
      v[2][i] = v[1][i] * (p.act == W4_ACT_SILU ? act_value<W4_ACT_SILU>(v[0][i]) : act_value<W4_ACT_GELU_TANH>(v[0][i]));
  }
  auto store = [&](void* out, size_t at, const float(&w)[V]) __attribute__((always_inline)) {
    if (p.out_type == W4_F32) {
      __builtin_memcpy(reinterpret_cast<float*>(out) + at, w, sizeof w);
    } else {
      uint16_t o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = (uint16_t)(p.out_type == W4_F16 ? to16<kF16>(w[i]) : to16<kBF16>(w[i]));
      __builtin_memcpy(reinterpret_cast<uint16_t*>(out) + at, o, sizeof o);
    }
  };
  store(p.out, (size_t)m * p.n + n, v[GATED ? 2 : 0]);
  if constexpr (GATED) {
    if (p.products) {
      store(p.products, (size_t)m * width + n, v[0]);
      store(p.products, (size_t)m * width + p.n + n, v[1]);
    }
  }
}

// One launch over `count` tiles of bm x bn channels from tile0 on.
template <int TYPE, bool GATED, int FMT, int WM, int WN, int MT, int NT, int STAGES>
hipError_t dense_launch(DenseArgs a, uint32_t tile0, uint32_t count, uint32_t bm, uint32_t bn, hipStream_t s) {
  constexpr uint32_t TM = 32 * MT * WM, CN = 32 * NT * WN / (GATED ? 2 : 1);
  a.tile0 = tile0;
  a.bm = bm;
  a.bn = bn;
  dense_kernel<TYPE, GATED, FMT, WM, WN, MT, NT, STAGES>
      <<<dim3(count * (bm / TM) * (bn / CN), a.splits), dim3(64 * WM * WN), 0, s>>>(a);
  return hipGetLastError();
}

template <int TYPE, bool GATED>
hipError_t dense_sum(const DenseArgs& a, hipStream_t s) {
  if (a.wide)
    dense_sum_kernel<TYPE, GATED, 4><<<dim3((a.n + 1023) / 1024, a.m), dim3(256), 0, s>>>(a);
  else
    dense_sum_kernel<TYPE, GATED, 1><<<dim3((a.n + 255) / 256, a.m), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <int TYPE, bool GATED, int FMT>
hipError_t dense_tiles(int tile, const DenseArgs& a, uint32_t tile0, uint32_t count, int of, hipStream_t s) {
  const uint32_t bm = kTiles[of].tm, bn = kTiles[of].tn / (GATED ? 2 : 1);
  if (tile == 0) return dense_launch<TYPE, GATED, FMT, 2, 4, 4, 2, 2>(a, tile0, count, bm, bn, s);
  if (tile == 1) return dense_launch<TYPE, GATED, FMT, 2, 4, 2, 2, 3>(a, tile0, count, bm, bn, s);
  if (tile == 2) return dense_launch<TYPE, GATED, FMT, 2, 2, 1, 2, 3>(a, tile0, count, bm, bn, s);
  if constexpr (FMT < 0) return dense_launch<TYPE, GATED, FMT, 1, 2, 1, 2, 4>(a, tile0, count, bm, bn, s);
  return hipErrorInvalidValue;
}

template <int TYPE, bool GATED, int FMT>
hipError_t dense_run(const DensePlan& p, const DenseArgs& a, hipStream_t s) {
  hipError_t e = dense_tiles<TYPE, GATED, FMT>(p.tile, a, 0, p.tiles - p.rest, p.tile, s);
  if (e == hipSuccess && p.rest)
    e = dense_tiles<TYPE, GATED, FMT>(kRestTile, a, p.tiles - p.rest, p.rest, p.tile, s);
  if (e == hipSuccess && p.splits > 1) e = dense_sum<TYPE, GATED>(a, s);
  return e;
}

}  // namespace
}  // namespace w4
