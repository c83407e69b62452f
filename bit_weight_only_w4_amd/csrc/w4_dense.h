// Dense product of two row-major operands with K contiguous, C[m, n] = sum_k A[m, k] B[n, k], on the matrix
// cores: fp16 or bf16 (32x32x16 steps, fp32 sums) or 8-bit integers (32x32x32 steps, int32 sums, exact).  A lane's
// fragment is 16 bytes in every type, so one kernel moves bytes and only the matrix instruction differs.
//
// Work layout.  A workgroup of WM x WN waves owns a tile of TM = 32 MT WM rows of A by TN = 32 NT WN rows of B and
// walks K in steps of 128 bytes.  Both operand tiles of a step come straight from memory into LDS (buffer loads
// with the LDS destination), two stages, the next one in flight while one is multiplied.
//   * Stage layout: 128 bytes a row, the 16-byte chunk c of row r in slot c XOR (r / 2 mod 8): the sixteen rows that
//     a 16-lane group of a 128-bit LDS read takes then lie in distinct banks.
//   * A (32 rows x 32 bytes): lane 32 h + c takes row c, bytes 16 h .. 16 h + 15 of the step.  B the same.
//   * D (32 x 32): lane 32 h + c holds column c (a row of B), rows 8 (e / 4) + 4 h + e % 4 (register e).
//   * Gated: the B tile holds TN / 2 gate rows, then the up rows of the same channels; a wave's even column tiles
//     are gate, its odd ones the up of the same channels, so the activation and the product happen in registers.
//   * Rows past M or N and chunks past K are read at an offset outside the buffer, which gives zeros.
#pragma once
#include "w4_ffn.h"
#include "w4_ffn_math.h"
#include "w4_mfma_common.h"

namespace w4 {
namespace {

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

__device__ inline void store_typed(void* out, size_t i, float v, uint32_t type) {
  if (type == 0)
    reinterpret_cast<float*>(out)[i] = v;
  else
    reinterpret_cast<uint16_t*>(out)[i] = (uint16_t)(type == 1 ? to16<kF16>(v) : to16<kBF16>(v));
}

template <int TYPE, bool GATED, int WM, int WN, int MT, int NT>
__global__ void __launch_bounds__(64 * WM * WN) dense_kernel(DenseArgs p) {
  constexpr int W = WM * WN, TM = 32 * MT * WM, TN = 32 * NT * WN;
  constexpr int ROWS = TM + TN;             // rows of a stage
  constexpr int COPIES = ROWS / 8 / W;      // copies of 8 rows a wave makes for a stage
  static_assert(ROWS % (8 * W) == 0 && TM % 8 == 0, "whole copies");
  static_assert(!GATED || NT % 2 == 0, "gate and up in one wave");
  __shared__ __align__(16) uint8_t st0[ROWS * 128], st1[ROWS * 128];
  using Acc = typename DenseAcc<TYPE>::type;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 31, h = lane >> 5;

  // Every eighth workgroup runs on one XCD: those take consecutive tiles, the tiles of a column of B first, so that
  // a B tile is read from memory by one XCD.
  const uint32_t mt = (p.m + TM - 1) / TM;
  const uint32_t tiles = gridDim.x, per = tiles / 8, rem = tiles % 8;
  const uint32_t xcd = blockIdx.x % 8, at = blockIdx.x / 8;
  const uint32_t tile = xcd * per + min(xcd, rem) + at;
  const uint32_t m0 = (tile % mt) * TM;
  constexpr uint32_t CN = GATED ? TN / 2 : TN;  // channels of a tile
  const uint32_t n0 = (tile / mt) * CN;

  const __amdgpu_buffer_rsrc_t ra =
      make_rsrc(p.a + (size_t)m0 * p.pitch, min((uint32_t)TM, p.m - m0) * p.pitch);
  const uint32_t nrows = min(CN, p.n - n0);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.b + (size_t)n0 * p.pitch, nrows * p.pitch);
  const __amdgpu_buffer_rsrc_t ru =
      make_rsrc(p.b + (size_t)(GATED ? p.n + n0 : 0) * p.pitch, GATED ? nrows * p.pitch : 0u);

  // Copy j of this wave fills rows 8 (W j + wave) .. + 7 of a stage: lane l slot l % 8 of row l / 8.  Its offsets:
  uint32_t off[COPIES], col[COPIES];
#pragma unroll
  for (int j = 0; j < COPIES; ++j) {
    const uint32_t r0 = 8u * (uint32_t)(W * j + wave);  // uniform
    const uint32_t r = r0 + ((uint32_t)lane >> 3);
    const uint32_t ch = ((uint32_t)lane & 7u) ^ ((r >> 1) & 7u);
    const uint32_t row = r < (uint32_t)TM ? r : (r - TM) % CN;
    const uint32_t rows = r < (uint32_t)TM ? min((uint32_t)TM, p.m - m0) : nrows;
    col[j] = ch * 16;
    off[j] = row < rows ? row * p.pitch + ch * 16 : kOutOfRange - p.pitch;
  }
  auto copy = [&](uint8_t* st, uint32_t k) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < COPIES; ++j) {
      const uint32_t r0 = 8u * (uint32_t)(W * j + wave);
      const __amdgpu_buffer_rsrc_t r = r0 < (uint32_t)TM ? ra : !GATED || r0 < (uint32_t)TM + CN ? rb : ru;
      uint32_t o = off[j] + k;
      if constexpr (TYPE == kDenseI8) o = k + col[j] < p.pitch ? o : kOutOfRange;  // rows of 64 bytes times an odd number
      asm volatile("" : "+v"(o));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          r, (__attribute__((address_space(3))) void*)(st + r0 * 128), 16, (int)o, 0, 0, 0);
    }
  };

  Acc acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  const uint32_t key = ((uint32_t)c >> 1) & 7u;  // every fragment row is c modulo 32
  auto frag = [&](const uint8_t* st, int row, int s) __attribute__((always_inline)) {
    const uint32_t slot = (uint32_t)(2 * s + h) ^ key;
    return *reinterpret_cast<const uint4*>(st + (row + c) * 128 + slot * 16);
  };
  auto multiply = [&](const uint8_t* st) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint4 a[MT], b[NT];
#pragma unroll
      for (int i = 0; i < MT; ++i) a[i] = frag(st, 32 * (MT * wm + i), s);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        b[j] = frag(st, TM + (GATED ? (j & 1) * (int)CN + 32 * (NT / 2 * wn + j / 2) : 32 * (NT * wn + j)), s);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = dense_mfma<TYPE>(a[i], b[j], acc[i][j]);
    }
  };

  // Two stages.  A stage's copies are waited for by the wave that made them, then the barrier hands the stage over;
  // a second barrier, after it is read, frees it for the copies of the step after the next.
  const uint32_t steps = (p.pitch + 127) / 128;
  auto landed = [&](bool more) __attribute__((always_inline)) {
    if (more)
      __builtin_amdgcn_s_waitcnt(0x0F70 | (COPIES & 15) | ((COPIES >> 4) << 14));  // all but the next stage's
    else
      wait_all_vector_loads();
    __syncthreads();
  };
  copy(st0, 0);
  if (steps > 1) copy(st1, 128);
  for (uint32_t t = 0; t < steps; t += 2) {
    landed(t + 1 < steps);
    multiply(st0);
    __syncthreads();
    if (t + 2 < steps) copy(st0, (t + 2) * 128);
    if (t + 1 < steps) {
      landed(t + 2 < steps);
      multiply(st1);
      __syncthreads();
      if (t + 3 < steps) copy(st1, (t + 3) * 128);
    }
  }

  // Epilogue.  16 bits: the exponents come off exactly (ldexp).  8 bits: the int32 sum is rounded to fp32 and
  // multiplied by its token's and its channel's scale, at most 2^-24 each.
#pragma unroll
  for (int i = 0; i < MT; ++i) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t m = m0 + 32 * (MT * wm + i) + 8 * (e / 4) + 4 * h + e % 4;
      if (m >= p.m) continue;
      float rs = 1.0f;
      int re = 0;
      if constexpr (TYPE == kDenseI8)
        rs = p.row_scale[m];
      else
        re = (p.row_exp ? p.row_exp[m] : 0) + (p.exp ? *p.exp : 0);
      auto value = [&](auto v, uint32_t n) __attribute__((always_inline)) {
        if constexpr (TYPE == kDenseI8)
          return (float)v * rs * p.col_scale[n];
        else
          return ldexpf(v, re + (p.col_exp ? p.col_exp[n] : 0));
      };
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (GATED) {
          if (j & 1) continue;
          const uint32_t n = n0 + 32 * (NT / 2 * wn + j / 2) + c;
          if (n >= p.n) continue;
          const float g = value(acc[i][j][e], n), u = value(acc[i][j + 1][e], p.n + n);
          const float y = p.act == W4_ACT_SILU ? act_value<W4_ACT_SILU>(g) : act_value<W4_ACT_GELU_TANH>(g);
          store_typed(p.out, (size_t)m * p.n + n, y * u, p.out_type);
          if (p.products) {
            store_typed(p.products, (size_t)m * 2 * p.n + n, g, p.out_type);
            store_typed(p.products, (size_t)m * 2 * p.n + p.n + n, u, p.out_type);
          }
        } else {
          const uint32_t n = n0 + 32 * (NT * wn + j) + c;
          if (n < p.n) store_typed(p.out, (size_t)m * p.n + n, value(acc[i][j][e], n), p.out_type);
        }
      }
    }
  }
}

template <int TYPE, bool GATED, int WM, int WN, int MT, int NT>
hipError_t dense_launch(const DenseArgs& a, hipStream_t s) {
  constexpr uint32_t TM = 32 * MT * WM, CN = 32 * NT * WN / (GATED ? 2 : 1);
  const uint64_t tiles = (uint64_t)((a.m + TM - 1) / TM) * ((a.n + CN - 1) / CN);
  if (tiles >= ((uint64_t)1 << 31)) return hipErrorInvalidValue;
  dense_kernel<TYPE, GATED, WM, WN, MT, NT><<<dim3((uint32_t)tiles), dim3(64 * WM * WN), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace
}  // namespace w4
