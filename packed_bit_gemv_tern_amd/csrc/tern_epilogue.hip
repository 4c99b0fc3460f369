// tern_epilogue.hip -- a ternary linear with what follows it in the same
// launch: bias, activation, the product with a second linear of the same shape
// (the gate and up projections of a gated feed-forward) and the residual.
//
//     v  = (s_row * (float)acc) * s_act [+ bias]        acc exact in int32
//     h  = act(v) [* v_up]
//     y  = [res +] h
//
// every product and sum one fp32 rounding.
#include <algorithm>

#include "tern_prologue.h"

namespace tern {

namespace {

constexpr uint32_t kCodeTable = 0x000100FFu;  // code byte 0, 1, 2 -> -1, 0, +1
constexpr uint32_t kZeroCodes = 0x55555555u;

__device__ __forceinline__ i32x4 decode16(uint32_t x) {
  i32x4 b;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    b[k] = (int32_t)__builtin_amdgcn_perm(kCodeTable, kCodeTable, (x >> (2 * k)) & 0x03030303u);
  return b;
}

// gelu in its tanh form, x (1 + tanh(c (x + 0.044715 x^3))) / 2 with c =
// sqrt(2 / pi), as x / (1 + e^(-2 c (...))): nothing cancels for negative x.
__device__ __forceinline__ float gelu32(float x) {
  const float cube = __fmul_rn(__fmul_rn(x, x), x);
  const float t = __fmul_rn(-1.5957691216057308f, __fadd_rn(x, __fmul_rn(0.044715f, cube)));
  return __fdiv_rn(x, __fadd_rn(1.0f, exp32(t)));
}

__device__ __forceinline__ float activate(int act, float v) { return act == 1 ? silu32(v) : act == 2 ? gelu32(v) : v; }

// y of one output: the linears' sums, row i and token m
template <int MATS>
__device__ __forceinline__ void finish(const EpilogueArgs& a, const int32_t (&sum)[MATS], int64_t m, int64_t i,
                                       int32_t z, float s_act) {
  float v[MATS];
#pragma unroll
  for (int k = 0; k < MATS; ++k) {
    const int32_t acc = (int32_t)((uint32_t)sum[k] - mul_zr(z, load_g(a.w[k].rowsum + i)));
    v[k] = epilogue(load_g(a.w[k].s_row + i), acc, s_act);
    if (a.w[k].bias) v[k] = __fadd_rn(v[k], load_g(a.w[k].bias + i));
  }
  float h = activate(a.act, v[0]);
  if constexpr (MATS == 2) h = __fmul_rn(h, v[1]);
  if (a.res) h = __fadd_rn(load_g(a.res + m * a.ldr + i), h);
  store_g(a.y + m * a.ldy + i, h);
}

// 16 activations from column j on, zeros past K.
__device__ __forceinline__ i32x4 load_q16(const int8_t* q, int64_t j, int K) {
  if (j + 16 <= K) return __builtin_bit_cast(i32x4, load16(q + j));
  i32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int d = 0; d < 16; ++d)
    if (j + d < K) v[d / 4] |= (int32_t)((uint32_t)(uint8_t)load_g(q + j + d) << (8 * (d % 4)));
  return v;
}

// RB blocks of 16 rows (of each matrix) and TB blocks of 16 tokens to a
// workgroup; its W waves take 256 columns at a time in turn, and their exact
// int32 sums meet in LDS.  v_mfma_i32_16x16x64_i8 with the weights as A: lane
// (r, g) loads the whole 16-byte chunk 4 i + g of row r, four operands of 64
// weights for four instructions; the tokens' operands are the same columns of
// token r, loaded as they lie (any order of K serves if both sides have it).
constexpr int RB = 2;
constexpr int kRedStride = 68;  // of 64 lanes' values of one register, off each other's banks

template <int W, int TB, int MATS>
__global__ __launch_bounds__(64 * W) void epilogue_rows_kernel(EpilogueArgs a, int row_tiles) {
  __shared__ int32_t red[W][MATS * RB * 4 * kRedStride];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int row0 = (blockIdx.x % row_tiles) * 16 * RB;
  const int64_t tok0 = (int64_t)(blockIdx.x / row_tiles) * 16 * TB;
  const uint8_t* wsrc[MATS][RB];
  const int8_t* qsrc[TB];
#pragma unroll
  for (int k = 0; k < MATS; ++k)
#pragma unroll
    for (int b = 0; b < RB; ++b) wsrc[k][b] = a.w[k].packed + (int64_t)min(row0 + 16 * b + r, a.N - 1) * a.ld;
#pragma unroll
  for (int t = 0; t < TB; ++t) qsrc[t] = a.q + min(tok0 + 16 * t + r, (int64_t)a.M - 1) * a.ldq;
  i32x4 acc[MATS][RB][TB];
#pragma unroll
  for (int k = 0; k < MATS; ++k)
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int t = 0; t < TB; ++t) acc[k][b][t] = i32x4{0, 0, 0, 0};
  for (int c0 = 4 * w; c0 < a.nch; c0 += 4 * W) {
    const int c = c0 + g;
    u32x4 wd[MATS][RB];
    i32x4 qa[TB][4];
#pragma unroll
    for (int k = 0; k < MATS; ++k)
#pragma unroll
      for (int b = 0; b < RB; ++b)
        wd[k][b] = c < a.nch ? load16(wsrc[k][b] + 16ll * c) : u32x4{kZeroCodes, kZeroCodes, kZeroCodes, kZeroCodes};
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int d = 0; d < 4; ++d) qa[t][d] = load_q16(qsrc[t], 64ll * c + 16 * d, a.K);
#pragma unroll
    for (int k = 0; k < MATS; ++k)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const i32x4 wb = decode16(wd[k][b][d]);
#pragma unroll
          for (int t = 0; t < TB; ++t)
            acc[k][b][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wb, qa[t][d], acc[k][b][t], 0, 0, 0);
        }
  }
  // lane (r, g), register v: row 16 b + 4 g + v, token 16 t + r
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    if (t) __syncthreads();
#pragma unroll
    for (int k = 0; k < MATS; ++k)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[w][((k * RB + b) * 4 + v) * kRedStride + lane] = acc[k][b][t][v];
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * RB * 16; o += 64 * W) {
      const int row = o % (16 * RB), tok = o / (16 * RB);
      const int64_t m = tok0 + 16 * t + tok;
      if (m >= a.M || row0 + row >= a.N) continue;
      int32_t sum[MATS];
#pragma unroll
      for (int k = 0; k < MATS; ++k) {
        sum[k] = 0;
#pragma unroll
        for (int i = 0; i < W; ++i)
          sum[k] += red[i][((k * RB + row / 16) * 4 + row % 4) * kRedStride + 16 * (row % 16 / 4) + tok];
      }
      finish<MATS>(a, sum, m, row0 + row, load_g(a.z + m), load_g(a.s_act + m));
    }
  }
}

template <int TB, int MATS>
hipError_t launch_rows(const EpilogueArgs& a, hipStream_t s) {
  constexpr int W = 8;
  const int64_t row_tiles = (a.N + 16 * RB - 1) / (16 * RB), tok_tiles = ((int64_t)a.M + 16 * TB - 1) / (16 * TB);
  hipLaunchKernelGGL((epilogue_rows_kernel<W, TB, MATS>), dim3((unsigned)(row_tiles * tok_tiles)), dim3(64 * W), 0, s,
                     a, (int)row_tiles);
  return hipGetLastError();
}

template <int MATS>
hipError_t launch_mats(const EpilogueArgs& a, hipStream_t s) {
  if (a.M <= 16) return launch_rows<1, MATS>(a, s);
  if (a.M <= 32) return launch_rows<2, MATS>(a, s);
  return launch_rows<4, MATS>(a, s);
}

}  // namespace

int64_t epilogue_work_items(const EpilogueArgs& a) {
  const int64_t row_tiles = ((int64_t)a.N + 16 * RB - 1) / (16 * RB), tb = a.M <= 16 ? 16 : a.M <= 32 ? 32 : 64;
  return mul_sat(mul_sat(row_tiles, ((int64_t)a.M + tb - 1) / tb), 512);
}

hipError_t launch_epilogue(const EpilogueArgs& a, int cus, hipStream_t s) {
  (void)cus;
  return a.w[1].packed ? launch_mats<2>(a, s) : launch_mats<1>(a, s);
}

}  // namespace tern
