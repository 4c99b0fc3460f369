// tern_sample.hip -- one token from each row of logits, with temperature,
// top-k, top-p, min-p and a given random number.
//
// With the row's tokens ordered by logit, the largest first (ties: the lowest
// index first), and weights w = e^((x - max) / T), the kept tokens are the
// first ones of that order that pass every filter:
//     top-k   the first k tokens;
//     top-p   the tokens whose forerunners among the first k hold less than
//             top_p of the weight of the first k;
//     min-p   the tokens with w >= min_p
// (the first token always).  The token drawn is the first one, in the order
// of the vocabulary, at which the running sum of the kept weights passes
// u * their total.
//
// Weights are computed in fp64 and summed as integers of 2^-44, so a sum is
// the same in whatever order it is taken (atomics included), and two rows
// with the same logits draw the same token.  The largest weight is 1, so
// 2^18 tokens sum to less than 2^63.
#include "tern_device.h"

namespace tern {

namespace {

constexpr int kSampleT = 1024;
constexpr double kFix = 17592186044416.0;  // 2^44

// e^x for x <= 0 (0 below -708) by Cody and Waite's reduction x = k ln 2 + r
// and the Taylor series of e^r through r^13 (|r| <= 0.347: its next term is
// 4e-18), in fp64.
__device__ __forceinline__ double exp_neg(double x) {
  if (!(x > -708.0)) return 0.0;
  constexpr double kInvLn2 = 1.4426950408889634074;
  constexpr double kHead = 0.693147180369123816490;  // ln 2 to 33 bits
  constexpr double kTail = 1.90821492927058770002e-10;
  const double k = __builtin_rint(x * kInvLn2);
  const double r = __builtin_fma(-k, kTail, __builtin_fma(-k, kHead, x));
  double p = 1.0 / 6227020800.0;
  p = __builtin_fma(p, r, 1.0 / 479001600.0);
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)k);
}

// Monotone key of a logit: larger logit, larger key; 0 for those that can
// never be drawn (-inf and NaN).  +0 and -0 compare equal and share a key.
__device__ __forceinline__ uint32_t logit_key(float x) {
  if (!(x > -__builtin_inff())) return 0;
  x += 0.0f;  // -0 -> +0
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

typedef unsigned long long u64;

struct RowParams {
  double inv_t, top_p, min_p;
  float mx, u;
  bool greedy;
  int64_t k;  // tokens of top-k (N: no limit)
};

__device__ __forceinline__ double weight_of(const RowParams& r, float x) {
  if (x == r.mx) return 1.0;  // (also where both are +inf)
  return exp_neg(((double)x - (double)r.mx) * r.inv_t);
}
__device__ __forceinline__ u64 fixed(double w) { return (u64)__builtin_rint(w * kFix); }

struct SampleLds {
  u64 mass[256];
  uint32_t count[256];
  u64 wave64[16];
  uint32_t wave32[16];
  u64 out64[2];
  uint32_t out32[4];
};

// Exclusive prefix over the workgroup of v (thread order), and the total.
__device__ __forceinline__ u64 wg_scan(u64 v, u64* wave, u64& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  u64 s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const u64 o = __shfl_up(s, d, 64);
    if (lane >= d) s += o;
  }
  __syncthreads();
  if (lane == 63) wave[w] = s;
  __syncthreads();
  u64 before = 0;
  total = 0;
  for (int i = 0; i < kSampleT / 64; ++i) {
    if (i < w) before += wave[i];
    total += wave[i];
  }
  return before + s - v;
}

// The first tokens of the order up to a border: keys above `key`, and of
// those with that key the `ties` lowest indices.
struct Border {
  uint32_t key;
  uint32_t ties;
};

// Finds the border by the 32 bits of the keys, 8 at a time from the top: of
// the tokens inside `in`, the first `want` (by count) or the first whose
// forerunners hold less than `mass` (by mass).
template <bool BY_MASS>
__device__ Border find_border(const float* x, int64_t N, const RowParams& r, Border in, uint32_t want, u64 mass,
                              SampleLds& L) {
  uint32_t prefix = 0, mask = 0, before_n = 0;
  u64 before_m = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kSampleT) L.mass[i] = 0, L.count[i] = 0;
    __syncthreads();
    for (int64_t j = threadIdx.x; j < N; j += kSampleT) {
      const float v = load_g(x + j);
      const uint32_t k = logit_key(v);
      if (k == 0 || (k & mask) != prefix || k < in.key) continue;
      const int bin = (k >> shift) & 255;
      atomicAdd(&L.count[bin], 1u);
      if (BY_MASS) atomicAdd(&L.mass[bin], fixed(weight_of(r, v)));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int bin = 255;
      uint32_t n = before_n;
      u64 m = before_m;
      for (; bin > 0; --bin) {  // the last bin that is not empty holds the border at the latest
        if (L.count[bin]) {
          const bool inside = BY_MASS ? m + L.mass[bin] >= mass : n + L.count[bin] >= want;
          if (inside) break;
        }
        n += L.count[bin];
        m += L.mass[bin];
      }
      L.out32[0] = (uint32_t)bin;
      L.out32[1] = n;
      L.out64[0] = m;
    }
    __syncthreads();
    prefix |= L.out32[0] << shift;
    mask |= 255u << shift;
    before_n = L.out32[1];
    before_m = L.out64[0];
    __syncthreads();
  }
  // tokens with the border's key: all have one weight
  Border out;
  out.key = prefix;
  const uint32_t here = L.count[prefix & 255];
  if (BY_MASS) {
    const u64 w = fixed(weight_of(r, key_logit(prefix)));
    // the i-th of them is kept where before_m + i w < mass
    const u64 need = mass > before_m ? mass - before_m : 0;
    const u64 n = w ? (need + w - 1) / w : (need ? here : 0);
    out.ties = (uint32_t)min((u64)here, n);
  } else {
    out.ties = min(here, want - before_n);
  }
  __syncthreads();
  if (prefix == in.key) out.ties = min(out.ties, in.ties);
  return out;
}

__global__ __launch_bounds__(kSampleT) void sample_kernel(SampleArgs a) {
  __shared__ SampleLds L;
  __shared__ u64 best[16];
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  const int64_t row = blockIdx.x, N = a.N;
  const float* x = a.x + row * a.ldx;

  // largest logit, its lowest index, and the tokens that can be drawn
  u64 top = 0;  // key, then the complement of the index
  uint32_t live = 0;
  for (int64_t j = t; j < N; j += kSampleT) {
    const uint32_t k = logit_key(load_g(x + j));
    live += k != 0;
    const u64 v = k ? ((u64)k << 32) | (uint32_t)~(uint32_t)j : 0;
    top = v > top ? v : top;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const u64 o = __shfl_xor(top, d, 64);
    top = o > top ? o : top;
    live += __shfl_xor(live, d, 64);
  }
  if (lane == 0) best[wv] = top, L.wave32[wv] = live;
  __syncthreads();
  live = 0;
  for (int i = 0; i < kSampleT / 64; ++i) {
    top = best[i] > top ? best[i] : top;
    live += L.wave32[i];
  }
  RowParams r;
  const float T = load_g(a.temperature + row);
  r.mx = key_logit((uint32_t)(top >> 32));
  r.greedy = !(T > 0.0f);
  r.inv_t = 1.0 / (double)T;
  r.u = load_g(a.u + row);
  const int32_t k = a.top_k ? load_g(a.top_k + row) : 0;
  r.k = k > 0 ? k : N;
  const float tp = a.top_p ? load_g(a.top_p + row) : 1.0f, mp = a.min_p ? load_g(a.min_p + row) : 0.0f;
  r.top_p = tp < 1.0f ? (double)fmaxf(tp, 0.0f) : 1.0;  // (a NaN is no filter)
  r.min_p = mp > 0.0f ? (double)fminf(mp, 1.0f) : 0.0;
  if (live == 0 || r.greedy) {
    if (t == 0) {
      store_g(a.token + row, live ? (int32_t)~(uint32_t)top : -1);
      if (a.prob) store_g(a.prob + row, live ? 1.0f : 0.0f);
      if (a.kept) store_g(a.kept + row, live ? 1 : 0);
    }
    return;
  }

  Border cut = {1u, 0xffffffffu};  // every live token
  if (r.k < (int64_t)live) cut = find_border<false>(x, N, r, cut, (uint32_t)r.k, 0, L);
  if (r.top_p < 1.0) {
    // weight of the first k: above the border, and the ties inside it
    u64 sum = 0;
    for (int64_t j = t; j < N; j += kSampleT) {
      const float v = load_g(x + j);
      const uint32_t kk = logit_key(v);
      if (kk > cut.key || (kk == cut.key && cut.ties == 0xffffffffu)) sum += fixed(weight_of(r, v));
    }
    u64 total;
    wg_scan(sum, L.wave64, total);
    if (cut.ties != 0xffffffffu) total += (u64)cut.ties * fixed(weight_of(r, key_logit(cut.key)));
    // forerunners < top_p * total, in whole units: forerunners < ceil(top_p * total)
    const double lim = r.top_p > 0.0 ? r.top_p * (double)total : 0.0;
    u64 mass = (u64)lim;
    if ((double)mass < lim) ++mass;
    if (mass == 0) mass = 1;  // the first token always
    __syncthreads();
    cut = find_border<true>(x, N, r, cut, 0, mass, L);
  }

  // kept weight, then the token at which its running sum passes u * total.
  // Thread t takes a run of the row's tokens, so that the scan is in order.
  const int64_t per = (N + kSampleT - 1) / kSampleT;
  const int64_t j0 = min(N, t * per), j1 = min(N, j0 + per);
  uint32_t ties = 0;
  for (int64_t j = j0; j < j1; ++j) ties += logit_key(load_g(x + j)) == cut.key;
  u64 all;
  uint32_t ties_before = (uint32_t)wg_scan(ties, L.wave64, all);
  auto keeps = [&](float v, uint32_t key, uint32_t& tie, double& w) {
    if (key < cut.key || key == 0) return false;
    if (key == cut.key && tie++ >= cut.ties) return false;
    w = weight_of(r, v);
    return w >= r.min_p || key == (uint32_t)(top >> 32);
  };
  u64 sum = 0;
  uint32_t kept = 0, tie = ties_before;
  for (int64_t j = j0; j < j1; ++j) {
    const float v = load_g(x + j);
    double w;
    if (keeps(v, logit_key(v), tie, w)) sum += fixed(w), ++kept;
  }
  u64 total, nkept;
  __syncthreads();
  const u64 before = wg_scan(sum, L.wave64, total);
  __syncthreads();
  wg_scan(kept, L.wave64, nkept);
  const double u = r.u > 0.0f ? fmin((double)r.u, 1.0) : 0.0;
  u64 target = (u64)(u * (double)total);
  if (target >= total) target = total - 1;
  if (before <= target && target < before + sum) {  // exactly one thread
    u64 run = before;
    tie = ties_before;
    for (int64_t j = j0; j < j1; ++j) {
      const float v = load_g(x + j);
      double w;
      if (!keeps(v, logit_key(v), tie, w)) continue;
      run += fixed(w);
      if (run > target) {
        store_g(a.token + row, (int32_t)j);
        if (a.prob) store_g(a.prob + row, (float)(w * kFix / (double)total));
        if (a.kept) store_g(a.kept + row, (int32_t)nkept);
        break;
      }
    }
  }
}

}  // namespace

int64_t sample_workspace_bytes(int64_t, int64_t) { return 0; }
int64_t sample_work_items(int64_t M, int64_t) { return M * kSampleT; }

hipError_t launch_sample(const SampleArgs& a, void*, hipStream_t s) {
  hipLaunchKernelGGL(sample_kernel, dim3((unsigned)a.M), dim3(kSampleT), 0, s, a);
  return hipGetLastError();
}

}  // namespace tern
