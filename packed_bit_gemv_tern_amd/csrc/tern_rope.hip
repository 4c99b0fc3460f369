// tern_rope.hip -- per-head RMS norm and rotary positions of queries and keys,
// between the q/k/v linears and the cache.
//
// For a head's row x of D elements at position p, with f_i = inv_freq[i]:
//
//     n_j  = x_j * gain_j / sqrt(mean_j(x_j^2) + eps)           (without a gain: n = x)
//     a_i  = p * f_i                                            i < R / 2
//     y_i         = m (n_i cos a_i - n_(i + R/2) sin a_i)
//     y_(i + R/2) = m (n_(i + R/2) cos a_i + n_i sin a_i)
//     y_j  = n_j                                                j >= R
//
// all in fp64 with one rounding to fp32: positions reach 2^30, where an angle
// in fp32 would be off by whole turns, and what fp64 costs stays under the
// memory time.  The angles are one per (token, i) and shared by all heads.
// Roofline: HBM, 8 bytes an element: 5,270 tokens of 40 heads of 128, 216 MB, in
// 43 us, 5.0 TB/s (a copy: 4.7).  48 single tokens, 3.9 us: the launch, the token's
// sequence, the angles and the heads' rows one after the other.
#include <algorithm>

#include "tern_device.h"

namespace tern {

namespace {

constexpr int kRopeT = 256;

// sin and cos of 0 <= a < 2^31, each to 2^-44: a = k pi/2 + r by Cody and Waite's
// reduction (pi/2 in two fp64 parts; k <= 2^30.4, so what the second leaves out
// is below 2^-76), Taylor series of r in [-pi/4, pi/4] through r^13 and r^14.
__device__ __forceinline__ void sincos64(double a, double& sn, double& cs) {
  constexpr double kTwoOverPi = 0.63661977236758134308;
  constexpr double kHi = 1.57079632679489655800, kLo = 6.12323399573676603587e-17;
  const double k = __builtin_rint(a * kTwoOverPi);
  const double r = __builtin_fma(-k, kLo, __builtin_fma(-k, kHi, a));
  const double x = r * r;
  double s = 1.0 / 6227020800.0, c = -1.0 / 87178291200.0;
  s = __builtin_fma(s, x, -1.0 / 39916800.0), c = __builtin_fma(c, x, 1.0 / 479001600.0);
  s = __builtin_fma(s, x, 1.0 / 362880.0), c = __builtin_fma(c, x, -1.0 / 3628800.0);
  s = __builtin_fma(s, x, -1.0 / 5040.0), c = __builtin_fma(c, x, 1.0 / 40320.0);
  s = __builtin_fma(s, x, 1.0 / 120.0), c = __builtin_fma(c, x, -1.0 / 720.0);
  s = __builtin_fma(s, x, -1.0 / 6.0), c = __builtin_fma(c, x, 1.0 / 24.0);
  c = __builtin_fma(c, x, -0.5);
  s = __builtin_fma(s * x, r, r), c = __builtin_fma(c, x, 1.0);
  const int quarter = (int)((int64_t)k & 3);
  const double u = quarter & 1 ? c : s, v = quarter & 1 ? s : c;
  sn = quarter & 2 ? -u : u;
  cs = quarter == 1 || quarter == 2 ? -v : v;
}

// D / 8 lanes take a head's row: lane u the elements 4u .. 4u + 3 and R/2 + 4u ..
// while those are pairs, then eight unrotated ones at R + 8 (u - R/8).  A
// workgroup takes `per` groups of heads of one token (kRopeT * 8 / D heads in a
// group), from group `blockIdx.x % splits` on every splits-th.
template <int D, bool VEC>
__global__ __launch_bounds__(kRopeT) void rope_kernel(RopeArgs a, int splits) {
  constexpr int LPH = D / 8, HPG = kRopeT / LPH;  // lanes of a head, heads of a group
  __shared__ double cs[D / 2], sn[D / 2];
  __shared__ int seq;
  const int t = threadIdx.x, row = blockIdx.x / splits, part = blockIdx.x % splits;
  const int heads = a.heads[0] + a.heads[1], R = a.R, u = t % LPH;
  // the row's sequence (the first, if several claim it)
  if (t == 0) seq = a.S;
  __syncthreads();
  for (int s = t; s < a.S; s += kRopeT) {
    const int32_t r0 = load_g(a.start + s), r1 = load_g(a.start + s + 1);
    if (r0 >= 0 && r0 <= row && row < r1 && r1 <= a.rows) atomicMin(&seq, s);
  }
  __syncthreads();
  if (seq == a.S) return;
  const int32_t r0 = load_g(a.start + seq), n = load_g(a.start + seq + 1) - r0;
  const int64_t pos = (int64_t)max(load_g(a.len + seq), 0) - n + row - r0;
  if (row - r0 >= a.max_new || pos < 0) return;
  for (int i = t; i < R / 2; i += kRopeT) {
    double s, c;
    sincos64((double)pos * fabs((double)load_g(a.inv_freq + i)), s, c);
    sn[i] = (load_g(a.inv_freq + i) < 0.0f ? -s : s) * (double)a.magnitude;
    cs[i] = c * (double)a.magnitude;
  }
  __syncthreads();
  const bool pairs = 8 * u < R;
  const int e0 = pairs ? 4 * u : 8 * u, e1 = pairs ? R / 2 + 4 * u : 8 * u + 4;
  for (int h = part * HPG + t / LPH; h < heads; h += splits * HPG) {
    const bool key = h >= a.heads[0];
    const int hh = key ? h - a.heads[0] : h;
    const float* x = (key ? a.x[1] + row * a.ldx[1] : a.x[0] + row * a.ldx[0]) + (int64_t)hh * D;
    float* y = (key ? a.y[1] + row * a.ldy[1] : a.y[0] + row * a.ldy[0]) + (int64_t)hh * D;
    const float* gain = key ? a.gain[1] : a.gain[0];
    double v[2][4];
    if constexpr (VEC) {
      const f32x4 p = load_g(reinterpret_cast<const f32x4*>(x + e0)), q = load_g(reinterpret_cast<const f32x4*>(x + e1));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[0][i] = p[i], v[1][i] = q[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[0][i] = load_g(x + e0 + i), v[1][i] = load_g(x + e1 + i);
    }
    if (gain) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum = __builtin_fma(v[0][i], v[0][i], __builtin_fma(v[1][i], v[1][i], sum));
#pragma unroll
      for (int d = 1; d < LPH; d *= 2) sum += __shfl_xor(sum, d, 64);
      const double r = 1.0 / sqrt(sum / D + (double)a.eps);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[0][i] *= r * (double)load_g(gain + e0 + i);
        v[1][i] *= r * (double)load_g(gain + e1 + i);
      }
    }
    f32x4 o[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (pairs) {
        o[0][i] = (float)(v[0][i] * cs[e0 + i] - v[1][i] * sn[e0 + i]);
        o[1][i] = (float)(v[1][i] * cs[e0 + i] + v[0][i] * sn[e0 + i]);
      } else {
        o[0][i] = (float)v[0][i], o[1][i] = (float)v[1][i];
      }
    }
    if constexpr (VEC) {
      store_g(reinterpret_cast<f32x4*>(y + e0), o[0]);
      store_g(reinterpret_cast<f32x4*>(y + e1), o[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) store_g(y + e0 + i, o[0][i]), store_g(y + e1 + i, o[1][i]);
    }
  }
}

// Workgroups that share a token's heads: one for many tokens, whose angles are then
// computed once; as many as there are groups of heads (three of 16 here) for few,
// which would leave CUs idle (1 token: 3.3 us, in one workgroup 4.8; 512: 6.9 and
// 7.5; 1,024: 12.7 and 10.8; 2,048: 17.7 and 16.0).
int rope_splits(const RopeArgs& a) {
  const int per = kRopeT * 8 / a.D;
  return a.rows >= 768 ? 1 : (a.heads[0] + a.heads[1] + per - 1) / per;
}

}  // namespace

int64_t rope_work_items(const RopeArgs& a) { return mul_sat(mul_sat(a.rows, rope_splits(a)), kRopeT); }

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
  const int splits = rope_splits(a);
  bool vec = true;
  for (int i = 0; i < 2; ++i)
    if (a.heads[i])
      vec = vec && ((reinterpret_cast<uintptr_t>(a.x[i]) | reinterpret_cast<uintptr_t>(a.y[i])) & 15) == 0 &&
            (a.rows == 1 || (a.ldx[i] % 4 == 0 && a.ldy[i] % 4 == 0));
  const dim3 grid((unsigned)((int64_t)a.rows * splits));
  auto run = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(kRopeT), 0, s, a, splits); };
  if (a.D == 64)
    vec ? run(rope_kernel<64, true>) : run(rope_kernel<64, false>);
  else
    vec ? run(rope_kernel<128, true>) : run(rope_kernel<128, false>);
  return hipGetLastError();
}

}  // namespace tern
