// tern_norm.hip -- residual addition, root-mean-square norm and the int8
// quantisation of its result, one launch: what every ternary linear and the
// int8 head read.
//
//     h_j = x_j + res_j                                     (fp32, one rounding)
//     y_j = fp32( h_j * gain_j / sqrt(mean_j(h_j^2) + eps) )  (fp64 inside)
//     q, s_act, z of y as tern_quantize_act makes them
//
// The norm runs in fp64 between two fp32 roundings: the squares of fp32
// numbers are exact there and the order of the sum changes the last of 53
// bits only, so the codes (integers, decided at rounding borders) are in
// practice a function of the inputs alone and not of the launch shape.
// Roofline: HBM; 13 bytes per element (x, res, h, q).  The row stays in
// registers from the first load to the codes, so x and res are read once:
// 4,096 x 4,096 in 50 us, 4.3 TB/s (a copy: 4.8).  One row, 4.2 us, is the launch
// and two trips to memory.
#include "tern_prologue.h"

namespace tern {

namespace {

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

struct NormArgs {
  const float *x, *res, *gain;
  float* h;
  int8_t* q;
  float* s_act;
  int32_t* z;
  int64_t K, ldx, ldr, ldh, ldq;
  double eps;
};

// Sum of v over the workgroup's T threads, in an order of its own.
template <int T>
__device__ __forceinline__ double wg_sum(double v, double* red) {
  v = wave_sum_d(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < T / 64; ++i) v += red[i];
  return v;
}

template <int T>
__device__ __forceinline__ void wg_range(float& lo, float& hi, float (*red)[16]) {
  lo = wave_min_f(lo);
  hi = wave_max_f(hi);
  if ((threadIdx.x & 63) == 0) red[0][threadIdx.x >> 6] = lo, red[1][threadIdx.x >> 6] = hi;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < T / 64; ++i) lo = fminf(lo, red[0][i]), hi = fmaxf(hi, red[1][i]);
}

// act_code of a row's scale, with the quotient from the reciprocal and the
// division only where that lies near a border between two codes: it is off by
// at most 255 * 2^-22.
__device__ __forceinline__ int32_t row_code(float y, float s, float inv, int32_t zm) {
  const float v = y * inv;
  float c = __builtin_rintf(v);
  if (!(fabsf(v - c) < 0.4999f)) c = __builtin_rintf(__fdiv_rn(y, s));  // (also where the reciprocal overflows)
  return min(127, max(-128, (int32_t)c + zm));
}

__device__ __forceinline__ float normed(float h, double r, float gain) {
  return (float)((double)h * r * (double)gain);
}

// The row in registers: V groups of four columns per thread (K <= 4 V T).
// VEC: every row 16-byte aligned and K a multiple of 4, so a group is one
// 16-byte access; otherwise a thread's columns are T apart.
template <int T, int V, bool VEC>
__global__ __launch_bounds__(T) void norm_kernel(NormArgs a) {
  __shared__ double red_d[T / 64];
  __shared__ float red_f[2][16];
  const int t = threadIdx.x;
  const int64_t m = blockIdx.x;
  const int K = (int)a.K;
  const float* x = a.x + m * a.ldx;
  const float* res = a.res ? a.res + m * a.ldr : nullptr;
  float* h = a.h ? a.h + m * a.ldh : nullptr;
  auto col = [&](int v, int c) { return VEC ? 4 * (t + T * v) + c : t + T * (4 * v + c); };
  float val[V][4];
  double sum = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (VEC) {
      if (col(v, 0) < K) {
        f32x4 g = __builtin_bit_cast(f32x4, load16(x + col(v, 0)));
        if (res) g += __builtin_bit_cast(f32x4, load16(res + col(v, 0)));
#pragma unroll
        for (int c = 0; c < 4; ++c) val[v][c] = g[c];
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) val[v][c] = 0.0f;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = col(v, c);
        val[v][c] = j < K ? (res ? load_g(x + j) + load_g(res + j) : load_g(x + j)) : 0.0f;
      }
    }
  }
  // (the gains are on their way while the sum is joined)
  f32x4 gain[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    gain[v] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (VEC) {
      if (col(v, 0) < K) gain[v] = __builtin_bit_cast(f32x4, load16(a.gain + col(v, 0)));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) gain[v][c] = col(v, c) < K ? load_g(a.gain + col(v, c)) : 0.0f;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int c = 0; c < 4; ++c) sum = __builtin_fma((double)val[v][c], (double)val[v][c], sum);
  if (h) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (VEC) {
        f32x4 g;
#pragma unroll
        for (int c = 0; c < 4; ++c) g[c] = val[v][c];
        if (col(v, 0) < K) store_g(reinterpret_cast<f32x4*>(h + col(v, 0)), g);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (col(v, c) < K) store_g(h + col(v, c), val[v][c]);
      }
    }
  }
  sum = wg_sum<T>(sum, red_d);
  const double r = 1.0 / sqrt(sum / (double)K + a.eps);
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      val[v][c] = normed(val[v][c], r, gain[v][c]);
      lo = fminf(lo, val[v][c]);
      hi = fmaxf(hi, val[v][c]);
    }
  }
  wg_range<T>(lo, hi, red_f);
  float s;
  int32_t zm;
  act_params(lo, hi, s, zm);
  const float inv = __fdiv_rn(1.0f, s);
  int8_t* q = a.q + m * a.ldq;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (VEC) {
      uint32_t word = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) word |= ((uint32_t)row_code(val[v][c], s, inv, zm) & 0xffu) << (8 * c);
      if (col(v, 0) < K) store_g(reinterpret_cast<uint32_t*>(q + col(v, 0)), word);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (col(v, c) < K) store_g(q + col(v, c), (int8_t)row_code(val[v][c], s, inv, zm));
    }
  }
  if (t == 0) {
    store_g(a.s_act + m, s);
    store_g(a.z + m, zm);
  }
}

// Rows too long for the registers: three passes over the row, the later ones
// reading the sum again (from h where the call has one: a thread reads only
// what it wrote itself).
constexpr int kLongT = 1024;
__global__ __launch_bounds__(kLongT) void norm_long_kernel(NormArgs a) {
  __shared__ double red_d[kLongT / 64];
  __shared__ float red_f[2][16];
  const int t = threadIdx.x;
  const int64_t m = blockIdx.x;
  const float* x = a.x + m * a.ldx;
  const float* res = a.res ? a.res + m * a.ldr : nullptr;
  float* h = a.h ? a.h + m * a.ldh : nullptr;
  double sum = 0.0;
  for (int64_t j = t; j < a.K; j += kLongT) {
    const float v = res ? x[j] + res[j] : x[j];
    if (h) h[j] = v;
    sum = __builtin_fma((double)v, (double)v, sum);
  }
  sum = wg_sum<kLongT>(sum, red_d);
  const double r = 1.0 / sqrt(sum / (double)a.K + a.eps);
  auto y = [&](int64_t j) {
    const float v = h ? h[j] : res ? x[j] + res[j] : x[j];
    return normed(v, r, load_g(a.gain + j));
  };
  float lo = 0.0f, hi = 0.0f;
  for (int64_t j = t; j < a.K; j += kLongT) {
    const float v = y(j);
    lo = fminf(lo, v);
    hi = fmaxf(hi, v);
  }
  wg_range<kLongT>(lo, hi, red_f);
  float s;
  int32_t zm;
  act_params(lo, hi, s, zm);
  int8_t* q = a.q + m * a.ldq;
  for (int64_t j = t; j < a.K; j += kLongT) store_g(q + j, (int8_t)act_code(y(j), s, zm));
  if (t == 0) {
    store_g(a.s_act + m, s);
    store_g(a.z + m, zm);
  }
}

template <int T, int V>
void launch_rows(bool vec, int64_t M, const NormArgs& a, hipStream_t s) {
  if (vec)
    hipLaunchKernelGGL((norm_kernel<T, V, true>), dim3((unsigned)M), dim3(T), 0, s, a);
  else
    hipLaunchKernelGGL((norm_kernel<T, V, false>), dim3((unsigned)M), dim3(T), 0, s, a);
}

}  // namespace

int64_t rmsnorm_work_items(int64_t M) { return mul_sat(M, kLongT); }

hipError_t launch_rmsnorm_quantize(const float* x, int64_t ldx, const float* res, int64_t ldr, const float* gain,
                                   float eps, int64_t M, int64_t K, float* h, int64_t ldh, int8_t* q,
                                   int64_t ldq, float* s_act, int32_t* z, hipStream_t s) {
  const NormArgs a = {x, res, gain, h, q, s_act, z, K, ldx, ldr, ldh, ldq, (double)eps};
  auto rows16 = [&](const void* p, int64_t ld) {
    return !p || ((reinterpret_cast<uintptr_t>(p) % 16) == 0 && (M == 1 || ld % 4 == 0));
  };
  const bool vec = K % 4 == 0 && rows16(x, ldx) && rows16(res, ldr) && rows16(h, ldh) && rows16(gain, 0);
  // A few rows: as many threads as the row has groups, for the latency of one
  // row (4,096 columns: 4.2 us).  From a row per CU on: fewer, longer threads,
  // several rows per CU (512 x 4,096: 10.2 -> 8.5 us, 4,096 x 2,048: 38 -> 28,
  // 4,096 x 4,096: 58 -> 50).
  const bool many = M >= 256;
  if (K <= 1024)
    launch_rows<256, 1>(vec, M, a, s);
  else if (K <= 2048 && many)
    launch_rows<256, 2>(vec, M, a, s);
  else if (K <= 4096)
    many ? launch_rows<256, 4>(vec, M, a, s) : launch_rows<1024, 1>(vec, M, a, s);
  else if (K <= 8192)
    many ? launch_rows<512, 4>(vec, M, a, s) : launch_rows<1024, 2>(vec, M, a, s);
  else if (K <= 16384)
    launch_rows<1024, 4>(vec, M, a, s);
  else
    hipLaunchKernelGGL(norm_long_kernel, dim3((unsigned)M), dim3(kLongT), 0, s, a);
  return hipGetLastError();
}

}  // namespace tern
