// Internal declarations of the gated feed-forward block, its gradients and the 8-bit products.
#pragma once
#include "w4_common.h"

namespace w4 {

// The operand types of the dense kernel (w4_dense.h).
enum DenseType { kDenseF16 = 0, kDenseBF16 = 1, kDenseI8 = 2 };

// fp16 terms that a weight of the format is the sum of in the dense kernel: integers and E2M1 times a power of two fit one
// (at most 11 bits), the others take two, which leave at most 2^-20 of a weight.
constexpr int dense_terms(int weight) { return weight == kNF4 || weight == kFP4 || weight == kINT4A ? 2 : 1; }

// Columns of W that share an exponent in a gradient's product: one scale of each row, or MXFP4's two.
constexpr int column_unit(int weight) { return weight == kINT4 || weight == kINT4A ? 128 : 64; }

// One dense product C[m, n] = sum_k A[m, k] B[n, k], both operands with K contiguous, and what becomes of it.
struct DenseArgs {
  const uint8_t* a;  // [M, pitch] rows of operand bytes, 16-byte aligned
  const uint8_t* b;  // [N, pitch]; gated: [2 N, pitch], gate rows, then up rows
  // B in four bits: b holds packed weights.  Gated: B's rows, with the folded scales [rows, K / 64, 2] of w4_gated.hip.
  // Without a gate: the weights [rows, N / 2] and their scales as they are, transposed; fp16 takes an exponent for each unit
  // of columns (column_unit) from parts.
  const void* scales;
  uint32_t rows;       // without a gate: weight rows, of which the last step of K may hold fewer than 64
  const float* parts;  // [nparts, N / unit]: maxima of the scales
  uint32_t nparts;
  int* exp_out;        // [N]: where the columns' exponents go, for dense_sum_kernel (`col_exp`)
  uint32_t m, n;     // outputs (gated: N is the width of h)
  uint32_t pitch;    // bytes of a row of A (its K elements), a multiple of 64, below 2^22
  uint32_t terms;    // B's rows in 16 bits: 1, or 2 where each 128 bytes are followed by 128 of second terms
  const float* row_scale;   // 8 bits: s[m]
  const float* col_scale;   // 8 bits: s[n]
  const int* row_exp;       // 16 bits: a row stands for its values times 2^row_exp[m]; may be null
  const int* col_exp;       // 16 bits: the same for B's rows; may be null
  void* out;         // [M, N]
  void* products;    // gated: [M, 2 N] or null
  uint32_t out_type;  // w4_type_t; fp32 for 8-bit products without a gate alone
  uint32_t act;
  uint32_t* partial;  // scratch for dense_bytes() bytes, null where that is 0
  uint32_t splits, per;  // set by launch_dense: K split over workgroups, steps of 128 bytes in a split
  uint32_t tile0, bm, bn;  // set by launch_dense: the launch covers, in its own tiles, tiles of bm x bn from tile0 on
  uint32_t wide;      // set by launch_dense: rows of the outputs are whole, aligned 16-byte pieces
};

hipError_t launch_dense(int type, bool gated, const DenseArgs& a, hipStream_t s);
// Scratch that a product of these sizes needs (its K split over workgroups): [splits, M, N or 2 N] of 4 bytes.
// `packed`: the weight format of B in four bits, else -1; `terms` of B's rows.
size_t dense_bytes(bool gated, int64_t m, int64_t n, int64_t pitch, int packed, int terms);
// The estimated time of a product, in microseconds.
double dense_us(bool gated, int64_t m, int64_t n, int64_t pitch, int packed, int terms);
// The gated product with B in four bits: A fp16.
hipError_t launch_dense_nf4(const DenseArgs& a, hipStream_t s);
hipError_t launch_dense_fp4(const DenseArgs& a, hipStream_t s);
hipError_t launch_dense_mxfp4(const DenseArgs& a, hipStream_t s);
hipError_t launch_dense_int4(const DenseArgs& a, hipStream_t s);
hipError_t launch_dense_int4a(const DenseArgs& a, hipStream_t s);
// The product with B transposed from four bits: A fp16, for MXFP4 of either type.
hipError_t launch_dense_columns_nf4(const DenseArgs& a, hipStream_t s);
hipError_t launch_dense_columns_fp4(const DenseArgs& a, hipStream_t s);
hipError_t launch_dense_columns_mxfp4(int type, const DenseArgs& a, hipStream_t s);
hipError_t launch_dense_columns_int4(const DenseArgs& a, hipStream_t s);
hipError_t launch_dense_columns_int4a(const DenseArgs& a, hipStream_t s);

// ---- gated block over 4-bit weights
bool gated_few(int fmt, int64_t tokens, int64_t hidden, int64_t inter);
size_t gated_workspace(int fmt, int64_t tokens, int64_t hidden, int64_t inter);
hipError_t launch_gated(int fmt, int act, const uint16_t* x, const uint8_t* packed, const void* scales, int64_t tokens,
                        int64_t hidden, int64_t inter, uint16_t* h, uint16_t* products, void* ws, hipStream_t s);
// The same for a few tokens, in one launch without a workspace: the fused GEMV's gated launch for one token, the MFMA
// kernel's for more (gated_mfma_fits: whether it has a launch shape).
hipError_t launch_gated_gemv_f16(int weight, const GemvGatedArgs& a, const GemvPlan& p, hipStream_t s);
hipError_t launch_gated_gemv_bf16(int weight, const GemvGatedArgs& a, const GemvPlan& p, hipStream_t s);
bool gated_mfma_fits(int fmt, int64_t inter, int64_t k, int64_t b);
hipError_t launch_gated_mfma(int fmt, const GemvGatedArgs& a, int64_t k, int64_t b, hipStream_t s);
hipError_t launch_gated_grad(int xt, int act, const uint16_t* dh, const uint16_t* products, int64_t tokens,
                             int64_t inter, uint16_t* dp, hipStream_t s);

// ---- input gradient of a 4-bit product
size_t gemm_grad_workspace(int fmt, int64_t n, int64_t k, int64_t b);
hipError_t launch_gemm_grad(int fmt, const uint16_t* d, const uint8_t* packed, const void* scales, int64_t n, int64_t k,
                            int64_t b, uint16_t* dx, void* ws, hipStream_t s);

// The same for a few tokens, without decoded rows (w4_grad_few.h), and how many those are at most (w4_grad.hip).
constexpr int grad_few_most(int weight, int xt) {
  return (weight == kINT4 && xt == kF16) || (weight == kMXFP4 && xt == kBF16) ? 32 : 64;
}
struct GradFewArgs {
  const uint16_t* d;      // [B, N]
  const uint8_t* packed;  // [N, K/2]
  const void* scales;
  uint16_t* dx;           // [B, K]
  float* partial;         // [splits, B, K] where N is split over workgroups, else null
  uint32_t n, k, b;
  uint32_t per;           // steps of 32 rows in a split
};
hipError_t launch_grad_few_f16(int weight, const GradFewArgs& a, uint32_t splits, hipStream_t s);
hipError_t launch_grad_few_bf16(int weight, const GradFewArgs& a, uint32_t splits, hipStream_t s);

// ---- 8 bits
// Products of a few tokens, without scratch (w4_int8_rows.hip); args as for launch_dense.
bool int8_few(int64_t b);
hipError_t launch_int8_rows(bool gated, const DenseArgs& a, hipStream_t s);
hipError_t launch_quantize_int8(int type, const void* x, int64_t rows, int64_t k, int8_t* codes, float* scales,
                                hipStream_t s);

}  // namespace w4
