// 8-bit products for a few tokens: rows of weights streamed past the tokens' codes, dot products of four in the vector
// unit (exact int32 sums, in any order the same).
//
// Work layout.  A wave owns R rows of weights (gated: R / 2 gate rows and the up rows of the same channels) and walks K
// in chunks of 1 KiB, 16 bytes a lane; every chunk of the tokens, from the L1, meets R rows in registers.  The four waves
// of a workgroup share the rows and take every fourth chunk each, their sums meet in LDS; rows of a KiB or less leave
// nothing to share, and each wave has its own.
//
// The weights' bytes bound it: one token, 8192 x 28672 46 us (5.1 TB/s), 151936 x 1536 42 us, 8960 x 1536 4.7 us, of which
// the launch and the wave's chain of loads and sums are 2.5.  Microseconds with the quantizer of the tokens before it (3 to
// 6), beside the dense kernel's for the same: one token 8960 x 1536 7.5 / 11.3, 1536 x 8960 8.2 / 13.4, 8192 x 8192 17.9 /
// 23.0; four tokens 9.2 / 11.4, 9.4 / 14.1, 20.0 / 23.0, 8192 x 28672 62.8 / 62.3, 151936 x 1536 61.4 / 62.0; eight tokens
// 15.0 / 11.6, 13.4 / 14.2, 28.2 / 23.4 (with eight in registers): so up to four.
#include "w4_ffn.h"
#include "w4_ffn_math.h"

namespace w4 {
namespace {

__device__ inline int dot16(const uint4& a, const uint4& b, int c) {
  c = __builtin_amdgcn_sdot4((int)a.x, (int)b.x, c, false);
  c = __builtin_amdgcn_sdot4((int)a.y, (int)b.y, c, false);
  c = __builtin_amdgcn_sdot4((int)a.z, (int)b.z, c, false);
  return __builtin_amdgcn_sdot4((int)a.w, (int)b.w, c, false);
}

template <int CTRL>
__device__ inline int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}

// Sums of V values over the wave's lanes, V a power of two up to 16: lane l ends with that of value
// (l % 16) / (16 / V).  A step adds a lane's values to those of its mirror image in 16, 8, 4 and 2 lanes; while there
// is more than one value left, each lane of such a pair goes on with half of them.
template <int V, int CTRL, int BIT>
__device__ inline int lanes_sum(const int (&v)[V], int lane) {
  if constexpr (V > 1) {
    int half[V / 2];
    const bool high = (lane & BIT) != 0;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) half[i] = (high ? v[V / 2 + i] : v[i]) + dpp<CTRL>(high ? v[i] : v[V / 2 + i]);
    if constexpr (BIT == 8) return lanes_sum<V / 2, 0x141, 4>(half, lane);
    if constexpr (BIT == 4) return lanes_sum<V / 2, 0x4E, 2>(half, lane);
    if constexpr (BIT == 2) return lanes_sum<V / 2, 0xB1, 1>(half, lane);
    return lanes_sum<V / 2, 0, 0>(half, lane);
  } else {
    int s = v[0];
    if constexpr (BIT >= 8) s += dpp<0x140>(s);  // row_mirror
    if constexpr (BIT >= 4) s += dpp<0x141>(s);  // row_half_mirror
    if constexpr (BIT >= 2) s += dpp<0x4E>(s);   // quad_perm [2,3,0,1]
    if constexpr (BIT >= 1) s += dpp<0xB1>(s);   // quad_perm [1,0,3,2]
    s += __shfl_xor(s, 16);
    return s + __shfl_xor(s, 32);
  }
}

// NB tokens (those past p.m repeat the last one and are not stored); SHARED: the workgroup's waves share rows.
template <int NB, int R, bool GATED, bool SHARED>
__global__ void __launch_bounds__(256) int8_rows_kernel(DenseArgs p) {
  constexpr int CH = GATED ? R / 2 : R;  // channels of a wave
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const uint32_t n0 = (SHARED ? blockIdx.x : blockIdx.x * 4 + wave) * CH;
  if (!SHARED && n0 >= p.n) return;
  const uint4* w[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t c = min(n0 + r % CH, p.n - 1);
    w[r] = reinterpret_cast<const uint4*>(p.b + (size_t)(GATED && r >= CH ? p.n + c : c) * p.pitch);
  }
  const uint4* x[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    x[b] = reinterpret_cast<const uint4*>(p.a + (size_t)min((uint32_t)b, p.m - 1) * p.pitch);
  int sum[R][NB] = {};
  const uint32_t chunks = p.pitch / 16;
  constexpr uint32_t step = SHARED ? 256 : 64;
#pragma unroll 2
  for (uint32_t i = (SHARED ? wave * 64 : 0) + lane; i < chunks; i += step) {
    uint4 v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = w[r][i];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint4 t = x[b][i];
#pragma unroll
      for (int r = 0; r < R; ++r) sum[r][b] = dot16(v[r], t, sum[r][b]);
    }
  }
  // A lane takes the sums of a channel and a token, gated of both products.
  constexpr int PARTS = GATED ? 2 : 1, VALUES = CH * NB;
  int mine[PARTS];
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    int v[VALUES];
#pragma unroll
    for (int i = 0; i < VALUES; ++i) v[i] = sum[q * CH + i / NB][i % NB];
    mine[q] = lanes_sum<VALUES, 0x140, 8>(v, lane);
  }
  const bool owner = lane < 16 && lane % (16 / VALUES) == 0;
  const int value = (lane & 15) / (16 / VALUES);
  if constexpr (SHARED) {
    __shared__ int part[4][PARTS][VALUES];
    if (owner)
#pragma unroll
      for (int q = 0; q < PARTS; ++q) part[wave][q][value] = mine[q];
    __syncthreads();
    if (wave || !owner) return;
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
      mine[q] = part[0][q][value] + part[1][q][value] + part[2][q][value] + part[3][q][value];
  }
  const uint32_t n = n0 + value / NB, m = value % NB;
  if (!owner || n >= p.n || m >= p.m) return;
  const float rs = p.row_scale[m];
  auto store = [&](void* out, size_t at, float v) __attribute__((always_inline)) {
    if (!GATED && p.out_type == W4_F32)
      reinterpret_cast<float*>(out)[at] = v;
    else
      reinterpret_cast<uint16_t*>(out)[at] = (uint16_t)(p.out_type == W4_F16 ? to16<kF16>(v) : to16<kBF16>(v));
  };
  float v[PARTS];
#pragma unroll
  for (int q = 0; q < PARTS; ++q) v[q] = (float)mine[q] * rs * p.col_scale[q * p.n + n];
  if constexpr (GATED) {
    store(p.out, (size_t)m * p.n + n,
          v[1] * (p.act == W4_ACT_SILU ? act_value<W4_ACT_SILU>(v[0]) : act_value<W4_ACT_GELU_TANH>(v[0])));
    if (p.products) {
      store(p.products, (size_t)m * 2 * p.n + n, v[0]);
      store(p.products, (size_t)m * 2 * p.n + p.n + n, v[1]);
    }
  } else {
    store(p.out, (size_t)m * p.n + n, v[0]);
  }
}

// Sharing rows against a wave for each, one token: 17920 x 1536 10.9 us against 12.0, 151936 x 1536 44.6 and 47.6.
template <int NB, int R, bool GATED>
hipError_t rows_launch(const DenseArgs& a, hipStream_t s) {
  constexpr uint32_t CH = GATED ? R / 2 : R;
  const uint32_t waves = (a.n + CH - 1) / CH;
  if (a.pitch > 1024)
    int8_rows_kernel<NB, R, GATED, true><<<dim3(waves), dim3(256), 0, s>>>(a);
  else
    int8_rows_kernel<NB, R, GATED, false><<<dim3((waves + 3) / 4), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

// R: 2, 4 and 8 rows took 60.4, 44.6, 46.2 us for one token of 151936 x 1536 and 62.4, 56.8, 47.6 for two, for four tokens
// 90.3 and 61.4 (2 and 4); 8.1, 8.2, 8.2 and 8.6, 9.0, 9.7 for 1536 x 8960.
template <bool GATED>
hipError_t rows_tokens(const DenseArgs& a, hipStream_t s) {
  if (a.m == 1) return rows_launch<1, 4, GATED>(a, s);
  if (a.m == 2) return rows_launch<2, 8, GATED>(a, s);
  return rows_launch<4, 4, GATED>(a, s);
}

}  // namespace

bool int8_few(int64_t b) { return b <= 4; }

hipError_t launch_int8_rows(bool gated, const DenseArgs& a, hipStream_t s) {
  return gated ? rows_tokens<true>(a, s) : rows_tokens<false>(a, s);
}

}  // namespace w4
