// tern_cache.hip -- new keys and values into the paged int8 cache.
//
// Codes are symmetric: a value is code * scale, one fp32 scale for each page,
// KV head and of K and V.  When a call's tokens reach a page,
//
//     cand   = max |x| / 127 over the page's new tokens
//     scale' = max(scale, cand)      (scale = 0 where the page holds no token yet)
//     held codes   c -> rint(c * (scale / scale'))    where scale' > scale
//     new codes    rint(x / scale'), in [-127, 127]   (0 where scale' = 0)
//
// with correctly rounded fp32 divisions and products and rint half to even,
// so the codes are a function of the inputs alone.  A held code moves by at
// most half a step each time the page's scale grows.
//
// Layouts are the attention's: K pages [token][dim], V pages [dim][token],
// so that both matrix operands read 16 contiguous codes per lane.  One
// workgroup takes one (sequence, page, head) of K or of V: it is the only
// writer of that page and head.  Roofline: HBM (5 bytes a value), and the
// launch for single tokens.
#include "tern_cache.h"

namespace tern {

namespace {

constexpr int kAppendT = 256;

__device__ __forceinline__ int32_t kv_code(float x, float s) {
  if (s == 0.0f) return 0;
  const float v = __builtin_rintf(__fdiv_rn(x, s));
  return (int32_t)fminf(127.0f, fmaxf(-127.0f, v));
}

__device__ __forceinline__ uint32_t requant4(uint32_t w, float ratio) {
  uint32_t o = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float v = __builtin_rintf(__fmul_rn((float)(int8_t)(w >> (8 * c)), ratio));
    o |= ((uint32_t)(int32_t)v & 0xffu) << (8 * c);
  }
  return o;
}

__global__ __launch_bounds__(kAppendT) void append_kernel(KvArgs a, const float* kx, int64_t ldk,
                                                          const float* vx, int64_t ldv, int chunks) {
  extern __shared__ __align__(16) uint8_t stage[];  // the new codes, in the page's own layout (V rows padded)
  __shared__ float red[kAppendT / 64];
  const int t = threadIdx.x;
  int b = blockIdx.x;
  const bool isv = b & 1;
  b >>= 1;
  const int h = b % a.H;
  b /= a.H;
  const int c = b % chunks, s = b / chunks;
  const SeqView sv = seq_view(a, s);
  const int P = 1 << a.log_p, D = a.D;
  const int64_t first = max(sv.pos0, (int64_t)0);
  const int64_t last = min(sv.len, sv.pos0 + min(sv.n, a.max_new));  // positions [first, last) are new
  const int64_t page = (first >> a.log_p) + c;
  const int64_t p0 = page << a.log_p;
  const int64_t lo = max(first, p0), hi = min(last, p0 + P);
  if (lo >= hi) return;
  const int32_t id = page_of(a, s, page);
  if (id < 0) return;
  const int held = (int)(lo - p0), n = (int)(hi - lo);
  const int64_t ld = isv ? ldv : ldk;
  const float* x = (isv ? vx : kx) + (sv.row0 + (lo - sv.pos0)) * ld + (int64_t)h * D;

  float amax = 0.0f;
  for (int i = t; i < n * D; i += kAppendT) amax = fmaxf(amax, fabsf(load_g(x + (int64_t)(i / D) * ld + i % D)));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d, 64));
  if ((t & 63) == 0) red[t >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAppendT / 64; ++i) amax = fmaxf(amax, red[i]);
  float* sp = (isv ? a.v_scale : a.k_scale) + (int64_t)id * a.H + h;
  const float was = held ? load_g(sp) : 0.0f;
  const float now = fmaxf(was, __fdiv_rn(amax, 127.0f));
  const bool grew = held && now > was;
  const float ratio = grew ? __fdiv_rn(was, now) : 1.0f;

  const int ldsv = P + 16;
  for (int i = t; i < n * D; i += kAppendT) {
    const int tok = i / D, d = i % D;
    const int32_t code = kv_code(load_g(x + (int64_t)tok * ld + d), now);
    stage[isv ? d * ldsv + held + tok : (held + tok) * D + d] = (uint8_t)code;
  }
  __syncthreads();
  uint8_t* out = (uint8_t*)(isv ? a.v : a.k) + (((int64_t)id * a.H + h) << a.log_p) * D;
  for (int u = t; u < (P * D) >> 4; u += kAppendT) {
    const int at = 16 * u;
    // tokens [t0, t1) of the unit's 16 codes (K: one token's)
    const int t0 = isv ? at & (P - 1) : at / D, t1 = isv ? t0 + 16 : t0 + 1;
    const bool any_new = t0 < held + n && t1 > held, any_old = grew && t0 < held;
    if (!any_new && !any_old) continue;
    u32x4 w = {0, 0, 0, 0};
    if (t0 < held || t1 > held + n) {
      w = load16(out + at);
      if (any_old) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t r = requant4(w[k], ratio);
          uint32_t keep = 0;  // bytes of tokens not held: left as they were
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (isv && t0 + 4 * k + e >= held) keep |= 0xffu << (8 * e);
          w[k] = (r & ~keep) | (w[k] & keep);
        }
      }
    }
    if (any_new) {
      const u32x4 nw = *reinterpret_cast<const u32x4*>(stage + (isv ? (at >> a.log_p) * ldsv + t0 : at));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t take = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tk = isv ? t0 + 4 * k + e : t0;
          if (tk >= held && tk < held + n) take |= 0xffu << (8 * e);
        }
        w[k] = (nw[k] & take) | (w[k] & ~take);
      }
    }
    store_g(reinterpret_cast<u32x4*>(out + at), w);
  }
  if (t == 0) store_g(sp, now);
}

// Pages that the new tokens of one sequence can reach.
int64_t append_chunks(const KvArgs& a) {
  const int64_t P = 1ll << a.log_p;
  return (a.max_new + P - 2) / P + 1;
}

}  // namespace

int64_t kv_append_work_items(const KvArgs& a) { return mul_sat(mul_sat(a.S * a.H, append_chunks(a)), 2 * kAppendT); }

hipError_t launch_kv_append(const KvArgs& a, const float* k, int64_t ldk, const float* v, int64_t ldv,
                            hipStream_t s) {
  const int64_t chunks = append_chunks(a);
  const size_t lds = (size_t)a.D * ((1 << a.log_p) + 16);
  hipLaunchKernelGGL(append_kernel, dim3((unsigned)(a.S * chunks * a.H * 2)), dim3(kAppendT), lds, s, a, k, ldk, v,
                     ldv, (int)chunks);
  return hipGetLastError();
}

}  // namespace tern
