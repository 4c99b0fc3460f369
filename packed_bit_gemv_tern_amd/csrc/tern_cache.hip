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
// writer of that page and head.  Roofline: HBM (5 bytes a value): three prompts
// to 2,047 tokens, 8 heads of 128, 16.1 us (a copy of as much takes 11.5).  K's
// workgroups alone take 12.2 of those and V's 14.8: most of it is each
// workgroup's chain (two trips to memory, the page's maximum, V's codes through
// LDS) and not bytes.  Single tokens: the launch and that chain, 24 tokens 5.4 us,
// 6.0 where every page's scale grows; 48 tokens after 96 held ones in pages of
// 128 10.2, and 14.2 where all of those are requantised.
#include "tern_cache.h"

namespace tern {

namespace {

constexpr int kAppendT = 256;

// rint(x / s) in [-127, 127].  The quotient is taken from the reciprocal, and
// divided only where that lies near a border between two codes: it is off by
// at most 127 * 2^-22.
__device__ __forceinline__ int32_t kv_code(float x, float s, float inv) {
  float v = x * inv, c = __builtin_rintf(v);
  if (!(fabsf(v - c) < 0.4999f)) c = __builtin_rintf(__fdiv_rn(x, s));  // (also where the reciprocal overflows)
  return (int32_t)fminf(127.0f, fmaxf(-127.0f, c));
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

// bytes [lo, hi) of four from position p on
__device__ __forceinline__ uint32_t byte_mask(int p, int lo, int hi) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (p + e >= lo && p + e < hi) m |= 0xffu << (8 * e);
  return m;
}

// A thread holds U blocks of 4 tokens x 4 dims from the maximum to the codes,
// so k and v are read once; block i of the page is tokens 4 (i / (D / 4)) and
// dims 4 (i % (D / 4)).  V goes through LDS to its transposed page: dword
// (dim, token / 4) is stored at column (token / 4) ^ (dim / 4), which keeps
// the writes, whose lanes run over the dims, off each other's banks.
template <int U>
__global__ __launch_bounds__(kAppendT) void append_kernel(KvArgs a, const float* kx, int64_t ldk, const float* vx,
                                                          int64_t ldv, int chunks, bool k16, bool v16) {
  extern __shared__ __align__(16) uint32_t stage[];  // V codes: D rows of P / 4 dwords
  __shared__ float red[kAppendT / 64];
  const int t = threadIdx.x;
  int b = blockIdx.x;
  const bool isv = b & 1;
  b >>= 1;
  const int h = b % a.H;
  b /= a.H;
  const int c = b % chunks, s = b / chunks;
  const SeqView sv = seq_view(a, s);
  const int P = 1 << a.log_p, D = a.D, log_d4 = D == 64 ? 4 : 5;
  const int64_t first = max(sv.pos0, (int64_t)0);
  const int64_t last = min(sv.len, sv.pos0 + min((int64_t)sv.n, a.max_new));  // positions [first, last) are new
  const int64_t page = (first >> a.log_p) + c;
  const int64_t p0 = page << a.log_p;
  const int64_t lo = max(first, p0), hi = min(last, p0 + P);
  if (lo >= hi) return;
  const int32_t id = page_of(a, s, page);
  const int held = (int)(lo - p0), top = (int)(hi - p0);  // tokens [held, top) of the page are new
  const int64_t ld = isv ? ldv : ldk;
  const bool x16 = isv ? v16 : k16;
  const float* x = (isv ? vx : kx) + (sv.row0 + (p0 - sv.pos0)) * ld + (int64_t)h * D;  // token 0's row (if it is one)
  const int blocks = (P * D) >> 4;

  f32x4 val[U][4];
  float amax = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = t + kAppendT * u, tok = 4 * (i >> log_d4), d = 4 * (i & ((1 << log_d4) - 1));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      val[u][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (i < blocks && tok + e >= held && tok + e < top) {
        const float* p = x + (int64_t)(tok + e) * ld + d;
        if (x16) {
          val[u][e] = __builtin_bit_cast(f32x4, load16(p));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) val[u][e][k] = load_g(p + k);
        }
      }
    }
  }
  if (id < 0) return;  // (the rows' loads were on their way meanwhile)
  float* sp = (isv ? a.v_scale : a.k_scale) + (int64_t)id * a.H + h;
  const float was = held ? load_g(sp) : 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int k = 0; k < 4; ++k) amax = fmaxf(amax, fabsf(val[u][e][k]));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d, 64));
  if ((t & 63) == 0) red[t >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAppendT / 64; ++i) amax = fmaxf(amax, red[i]);
  const float now = fmaxf(was, __fdiv_rn(amax, 127.0f));
  const bool grew = held && now > was;
  const float ratio = grew ? __fdiv_rn(was, now) : 1.0f;
  // (a scale of 0 belongs to zeros: any divisor gives their code)
  const float by = now == 0.0f ? 1.0f : now, inv = __fdiv_rn(1.0f, by);

  uint8_t* out = (uint8_t*)(isv ? a.v : a.k) + (((int64_t)id * a.H + h) << a.log_p) * D;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = t + kAppendT * u, tok = 4 * (i >> log_d4), d = 4 * (i & ((1 << log_d4) - 1));
    if (i >= blocks || tok >= top || tok + 4 <= held) continue;
    uint32_t code[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int k = 0; k < 4; ++k) code[e][k] = (uint32_t)kv_code(val[u][e][k], by, inv) & 0xffu;
    if (!isv) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (tok + e >= held && tok + e < top)
          store_g(reinterpret_cast<uint32_t*>(out + (tok + e) * D + d),
                  code[e][0] | code[e][1] << 8 | code[e][2] << 16 | code[e][3] << 24);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        stage[((d + k) << (a.log_p - 2)) + ((tok >> 2) ^ ((d >> 2) & ((P >> 2) - 1)))] =
            code[0][k] | code[1][k] << 8 | code[2][k] << 16 | code[3][k] << 24;
    }
  }
  if (t == 0) store_g(sp, now);
  if (!isv) {
    if (!grew) return;
    for (int u = t; u < (held * D) >> 4; u += kAppendT) {
      u32x4 w = load16(out + 16 * u);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = requant4(w[k], ratio);
      store_g(reinterpret_cast<u32x4*>(out + 16 * u), w);
    }
    return;
  }
  __syncthreads();
  for (int u = t; u < blocks; u += kAppendT) {
    const int d = u >> (a.log_p - 4), t0 = (16 * u) & (P - 1);  // 16 tokens of a dim
    const bool any_new = t0 < top && t0 + 16 > held, any_old = grew && t0 < held;
    if (!any_new && !any_old) continue;
    u32x4 w = {0, 0, 0, 0};
    if (t0 < held || t0 + 16 > top) w = load16(out + 16 * u);  // (tokens to keep, or to bring to the new scale)
    const int swz = (d >> 2) & ((P >> 2) - 1);
    const u32x4 nw = *reinterpret_cast<const u32x4*>(stage + (d << (a.log_p - 2)) + (((t0 >> 2) ^ swz) & ~3));
    u32x4 o;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t r = w[k];
      if (any_old) {
        const uint32_t mo = byte_mask(t0 + 4 * k, 0, held);
        r = (requant4(r, ratio) & mo) | (r & ~mo);
      }
      const uint32_t mn = byte_mask(t0 + 4 * k, held, top);
      const uint32_t fresh = (swz & 1) ? ((swz & 2) ? nw[k ^ 3] : nw[k ^ 1]) : ((swz & 2) ? nw[k ^ 2] : nw[k]);
      o[k] = (fresh & mn) | (r & ~mn);
    }
    store_g(reinterpret_cast<u32x4*>(out + 16 * u), o);
  }
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
  const size_t lds = (size_t)a.D << a.log_p;
  const dim3 grid((unsigned)(a.S * chunks * a.H * 2)), block(kAppendT);
  auto rows16 = [&](const float* p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.rows == 1 || ld % 4 == 0);
  };
  const bool k16 = rows16(k, ldk), v16 = rows16(v, ldv);
  const int U = ((a.D << a.log_p) / 16 + kAppendT - 1) / kAppendT;  // 1, 2 or 4
  if (U == 1)
    hipLaunchKernelGGL(append_kernel<1>, grid, block, lds, s, a, k, ldk, v, ldv, (int)chunks, k16, v16);
  else if (U == 2)
    hipLaunchKernelGGL(append_kernel<2>, grid, block, lds, s, a, k, ldk, v, ldv, (int)chunks, k16, v16);
  else
    hipLaunchKernelGGL(append_kernel<4>, grid, block, lds, s, a, k, ldk, v, ldv, (int)chunks, k16, v16);
  return hipGetLastError();
}

}  // namespace tern
