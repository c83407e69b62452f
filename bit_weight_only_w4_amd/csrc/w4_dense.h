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
//   * B of two terms (fp16, dense_terms): K is twice as long, a step of A's meets one of first and then one of second terms.
//   * B in four bits: a wave's packed weights and their scales come to LDS of its own a step ahead, and between the matrix
//     instructions it decodes them, scales them, rounds them to 16 bits and writes them into the stage where the copies
//     would have put them: rows of weights for the gated block (PackedRows), columns for a gradient (PackedColumns; both
//     in w4_dense_sources.h).
//
// What bounds it is the matrix cores under the card's power limit: its rate depends on the data.  4096 x 8192 x 8192: int8
// 245 to 260 us (2110 to 2240 Tops/s; the library's product 2090), fp16 1160 TFLOP/s (1250).  One wave of every SIMD waits
// while the other issues: with the copies in one burst behind the barrier, or with steps of 64 bytes, int8 took 300 us and
// more.
#pragma once
#include <type_traits>

#include "w4_dense_sources.h"

namespace w4 {

struct DensePlan {
  double us;  // the estimate
  int tile;
  uint32_t splits, per;
  uint32_t tiles, rest;  // tiles in all, and how many of the last are covered with 64 x 128 tiles by a second launch
};
DensePlan plan_dense(bool gated, int64_t m, int64_t n, int64_t pitch, int packed, int terms);
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

template <int V>
using I = std::integral_constant<int, V>;

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

template <int TYPE, bool GATED, int FMT, int WM, int WN, int MT, int NT, int STAGES>
__global__ void __launch_bounds__(64 * WM * WN) dense_kernel(DenseArgs p) {
  constexpr int W = WM * WN, TM = 32 * MT * WM, TN = 32 * NT * WN;
  constexpr int ROWS = TM + TN;             // rows of a stage
  constexpr bool PACKED = FMT >= 0;         // B in four bits
  constexpr int TERMS = PACKED && TYPE == kDenseF16 ? dense_terms(FMT) : 1;  // known when compiled
  constexpr int COPIES = (PACKED ? TM : ROWS) / 8 / W;  // copies of 8 rows a wave makes for a stage
  static_assert(TM % (8 * W) == 0 && (PACKED || (GATED ? TN / 2 : TN) % (8 * W) == 0),
                "a round of copies fills one operand");
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
  const uint32_t twice = PACKED ? TERMS - 1 : TYPE == kDenseI8 ? 0 : p.terms - 1;  // steps of B to one of A, as a shift
  const uint32_t bpitch = p.pitch << twice;
  i32x4 rb{}, ru{};  // B, gated: its gate and up rows
  if constexpr (!PACKED) {
    rb = dense_rsrc(p.b + (size_t)n0 * bpitch, nrows * bpitch);
    ru = dense_rsrc(p.b + (size_t)(GATED ? p.n + n0 : 0) * bpitch, GATED ? nrows * bpitch : 0u);
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
    // (outside: past 2^31, which no resource of fewer rows than a tile's reaches)
    off[j] = row < rows ? row * (r < (uint32_t)TM ? p.pitch : bpitch) + mine : 0x80000000u;
  }
  const uint32_t first = blockIdx.y * p.per, steps = min(first + p.per, (p.pitch + 127) / 128 << twice);  // this split's
  // Copy j of step t; past the last step copies are made all the same, of what is never read (mostly from outside the
  // buffers), so that the number of copies in flight is the same in every step.
  auto copy = [&](const uint8_t* st, uint32_t t, int j) __attribute__((always_inline)) {
    uint32_t k = t < steps ? (8 * W * j < TM ? t >> twice : t) * 128 : 0x40000000u;
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
  constexpr int SF = PACKED ? FMT : kFP4, SN = PACKED ? TN : 32 * W;  // (a source that is never used otherwise)
  using Source = typename std::conditional<GATED, PackedRows<SF, PACKED ? TERMS : 1, TM, SN, W, STAGES>,
                                           PackedColumns<SF, PACKED ? TERMS : 1, TYPE, TM, SN, W, STAGES>>::type;
  Source src;
  constexpr bool EXPONENTS = COLUMNS && TYPE == kDenseF16;  // of units of columns
  constexpr int UNIT = column_unit(SF);
  __shared__ int exps[EXPONENTS ? TN / UNIT : 1];
  if constexpr (PACKED && GATED) src.init(p, n0, nrows, steps, raw, &ring[0][0], table, lane, wave);
  if constexpr (COLUMNS) {
    src.init(p, n0, steps, raw, &ring[0][0], table, lane, wave);
    if constexpr (EXPONENTS) {
      static_assert(TN / UNIT <= W, "a wave for each unit");
      if (wave < TN / UNIT) {
        const int e = unit_exponent<FMT>(p.parts, p.nparts, p.n / UNIT, n0 / UNIT + wave, lane);
        if (lane == 0) exps[wave] = e;
      }
    }
  }
  // A quarter: after each matrix instruction one of the next quarter's fragments is requested, and a copy now and then.
  // What it decodes are weights of step t, of their term `of`.
  auto quarter = [&](Frags& next, uint32_t st, auto which, const Frags& f, uint32_t to, uint32_t t, auto of, auto from,
                     auto end) __attribute__((always_inline)) {
    constexpr int T = decltype(of)::value;
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
            src.template put<0, T>(to, s), src.template put<1, T>(to, s);
            src.template look<2>(s), src.template look<3>(s);
          }
          if (D0 + 2 * (ALL - D0) / 3 == q) src.template put<2, T>(to, s), src.template put<3, T>(to, s);
        } else {
          if (D0 == q) src.template look<0>(s), src.template put<0, T>(to, s);
          if (D0 + (ALL - D0) / 4 == q) src.template look<1>(s), src.template put<1, T>(to, s);
          if (D0 + 2 * (ALL - D0) / 4 == q) src.template look<2>(s), src.template put<2, T>(to, s);
          if (D0 + 3 * (ALL - D0) / 4 == q) src.template look<3>(s), src.template put<3, T>(to, s);
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
    __syncthreads();  // the table and the exponents
    if constexpr (EXPONENTS) {
      src.f = exps[src.unit];
      if (m0 == 0 && blockIdx.y == 0 && tid < TN && n0 + tid < p.n) p.exp_out[n0 + tid] = exps[tid / UNIT];
    }
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
#pragma unroll
      for (int j = 0; j < COPIES; ++j) copy(&ring[i][0], first + i, j);
    auto decode = [&](auto at, auto of) __attribute__((always_inline)) {
      constexpr int i = decltype(at)::value, T = decltype(of)::value;
      src.use_first(i);
#pragma unroll
      for (int q = 0; q < (i == STAGES - 1 ? 1 : 4); ++q) {
        src.template look<0>(q), src.template put<0, T>(i * SIZE, q);
        src.template look<1>(q), src.template put<1, T>(i * SIZE, q);
        src.template look<2>(q), src.template put<2, T>(i * SIZE, q);
        src.template look<3>(q), src.template put<3, T>(i * SIZE, q);
      }
    };
    static_assert(STAGES == 2 || STAGES == 3, "the stages decoded here");
    decode(I<0>{}, I<0>{});
    decode(I<1>{}, I<1 % TERMS>{});
    if constexpr (STAGES == 3) decode(I<2>{}, I<0>{});
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
  auto step = [&](uint32_t t, auto of) __attribute__((always_inline)) {
    const uint32_t u = t + STAGES - 1;
    using Now = I<(decltype(of)::value + STAGES - 1) % TERMS>;  // the term of step u
    using Next = I<(decltype(of)::value + STAGES) % TERMS>;
    quarter(f1, now, I<1>{}, f0, spare, u, Now{}, I<C3>{}, I<C0>{});
    quarter(f0, now, I<2>{}, f1, spare, u, Now{}, I<C0>{}, I<C1>{});
    quarter(f1, now, I<3>{}, f0, spare, u, Now{}, I<C1>{}, I<COPIES>{});
    // by hand: the compiler's own barrier waits for every copy in flight
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * COPIES) : "memory");
    spare = now;
    now = now + SIZE == STAGES * SIZE ? 0 : now + SIZE;
    if constexpr (PACKED) src.take();
    quarter(f0, now, I<0>{}, f1, spare, u + 1, Next{}, I<0>{}, I<C3>{});
  };
  for (uint32_t t = first; t < steps; t += TERMS) {  // (splits begin with a first term)
    step(t, I<0>{});
    if constexpr (TERMS == 2) step(t + 1, I<1>{});
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
  const i32x4 rr =
      dense_rsrc(reinterpret_cast<const uint32_t*>(rows_of) + m0, rows_of ? min((uint32_t)TM, p.m - m0) * 4 : 0u);
  uint32_t cv[NT];  // this lane's channels
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const uint32_t n = nw + 32 * (GATED ? j / 2 : j) + c;
    if constexpr (EXPONENTS)
      cv[j] = (uint32_t)exps[(n - n0) / UNIT];
    else
      cv[j] = cols_of && n < p.n ? reinterpret_cast<const uint32_t*>(cols_of)[(GATED && (j & 1) ? p.n : 0u) + n] : 0u;
  }
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
        return ldexpf(acc[i][j][e], (int)rv[e] + (int)cv[j]);
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
  const int re = TYPE == kDenseI8 || !p.row_exp ? 0 : p.row_exp[m];
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
