// tern_attn.hip -- attention over the paged int8 cache.
//
// Row r (a new token and a query head) sees the positions j <= pos_r of its
// sequence; with k_j = ks_j * ck_j, v_j = vs_j * cv_j (codes ck, cv, scales
// of the page and KV head):
//
//     s_j = scale * (q_r . k_j),  y_r = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// in one pass over the positions with the running maximum m and sum.  A
// row with no position to see is 0.
//
// Matrix form, per step of 64 positions (v_mfma_f32_16x16x32_f16, fp32
// accumulators):  S^T = K Q^T,  O^T += V^T P^T.  The codes are exact in
// fp16.  The other operand of each product is split in two fp16 numbers, hi
// + lo, 22 bits together: q after a power of two that brings the row's
// largest element under 2^9 (so that lo stays far above fp16's smallest
// numbers), and w_j = e^(s_j - m) * vs_j / 2^e <= 2^15 (e: exponent of the
// largest V scale met so far).  Errors are then those of fp32.
//
// Layout: in S^T a lane holds one query row (lane % 16) and 4 positions per
// 16 x 16 tile.  Row i of K tile t is position 16 * (i / 4) + 4 t + i % 4 of
// the step, so lane group g = lane / 16 ends up with the 16 consecutive
// positions 16 g .. 16 g + 15, which are one page's (pages hold a multiple of
// 16): its own scale, and exactly the positions it has to hold as an operand
// of the second product if a V^T operand is 16 contiguous codes of one
// dimension.  V pages are stored [dim][token] for that.  So P goes from the
// first product to the second without leaving the lane's registers, and K
// and V go from memory to registers by 16-byte loads, without LDS.
#include <algorithm>

#include "tern_cache.h"

namespace tern {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kAttnWaves = 4;
constexpr int kStep = 64;  // positions per step of a wave

struct AttnArgs {
  KvArgs kv;
  const float* q;
  float* y;
  float* part;  // per (row, head, chunk): D sums, then m and l per (row, head, chunk)
  float* part_ml;
  int64_t ldq, ldy;
  int32_t Hq, G;
  int32_t chunk, nchunk;  // positions per chunk, chunks a sequence is split into
  int32_t row_tiles;
  float scale;
};

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Eight int8 codes as fp16, exactly: 0x6400 | u is 1024 + u, u = code + 128.
__device__ __forceinline__ f16x8 codes_f16(uint32_t w0, uint32_t w1) {
  const f16x2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
  union {
    f16x2 h[4];
    f16x8 v;
  } o;
  w0 ^= 0x80808080u;
  w1 ^= 0x80808080u;
  o.h[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w0, 0x04010400u)) - bias;
  o.h[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w0, 0x04030402u)) - bias;
  o.h[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w1, 0x04010400u)) - bias;
  o.h[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w1, 0x04030402u)) - bias;
  return o.v;
}

// v = hi + lo to 22 bits (hi rounded toward zero: lo has its sign).
__device__ __forceinline__ void split2(float a, float b, f16x2& hi, f16x2& lo) {
  hi = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(a, b));
  lo = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(a - (float)hi[0], b - (float)hi[1]));
}

__device__ __forceinline__ float pow2i(int e) { return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23); }

// Maximum / sum over the four lanes that hold one query row.
__device__ __forceinline__ float max_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

constexpr float kNegInf = -__builtin_inff();

// One workgroup: one (sequence, KV head), 16 * NT rows (row i: new token i /
// G, query head i % G of the KV head's), one chunk of the positions, whose
// steps the four waves take in turn.
template <int D, int NT>
__global__ __launch_bounds__(64 * kAttnWaves, 2) void attn_kernel(AttnArgs a) {
  constexpr int KS = D / 32;  // k steps of the first product
  constexpr int DT = D / 16;  // 16-dim tiles of the output
  constexpr int LD = D + 4;
  __shared__ float so[kAttnWaves][16 * NT][LD];
  __shared__ float sml[kAttnWaves][16 * NT][2];

  const KvArgs& kv = a.kv;
  int b = blockIdx.x;
  const int h = b % kv.H;
  b /= kv.H;
  const int c = b % a.nchunk;
  b /= a.nchunk;
  const int rt = a.row_tiles - 1 - b % a.row_tiles;
  const int s = b / a.row_tiles;
  const SeqView sv = seq_view(kv, s);
  const int rows = min(sv.n, (int)kv.max_new) * a.G, row_lo = rt * 16 * NT;
  if (row_lo >= rows) return;
  // positions that some row of the tile sees: up to the last row's own
  const int64_t last_pos = sv.pos0 + min(row_lo + 16 * NT - 1, rows - 1) / a.G;
  const int64_t end = min(sv.len, last_pos + 1);
  const int64_t c0 = (int64_t)c * a.chunk;
  const int64_t c1 = c == a.nchunk - 1 ? end : min(end, c0 + a.chunk);
  // (chunk 0 always writes: it is the one that the joining pass counts on)
  if (c0 >= c1 && c > 0) return;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, g = lane >> 4;

  // the query rows, split
  f16x8 qh[NT][KS], ql[NT][KS];
  float cs[NT];     // factor of a row's scores: scale * log2(e) * the row's power of two
  int32_t pos[NT];  // last position that the row sees (-1: none)
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int r = row_lo + 16 * u + n;
    const bool live = r < rows;
    pos[u] = live ? (int32_t)max(min(sv.pos0 + r / a.G, sv.len - 1), (int64_t)-1) : -1;
    const float* q = a.q + (int64_t)(sv.row0 + (live ? r / a.G : 0)) * a.ldq +
                     (int64_t)(h * a.G + (live ? r % a.G : 0)) * D + g * (D / 4);
    float x[D / 4];
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 4; ++j) {
      x[j] = live ? load_g(q + j) : 0.0f;
      amax = fmaxf(amax, fabsf(x[j]));
    }
    amax = max_groups(amax);
    // 2^(8 - exponent): the largest element lands in [2^8, 2^9)
    const int e = min(max((int)(__builtin_bit_cast(uint32_t, amax) >> 23) - 127, -100), 120);
    const float up = pow2i(8 - e);
    cs[u] = a.scale * 1.44269504088896340736f * pow2i(e - 8);
#pragma unroll
    for (int j = 0; j < KS; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f16x2 hi, lo;
        split2(x[8 * j + 2 * i] * up, x[8 * j + 2 * i + 1] * up, hi, lo);
        qh[u][j][2 * i] = hi[0], qh[u][j][2 * i + 1] = hi[1];
        ql[u][j][2 * i] = lo[0], ql[u][j][2 * i + 1] = lo[1];
      }
    }
  }

  f32x4 o[NT][DT];
  float m[NT], l[NT];
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    m[u] = kNegInf;
    l[u] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[u][d] = {0.0f, 0.0f, 0.0f, 0.0f};
  }
  int ve = -100;  // o holds sums of code * weight * 2^(14 - ve)

  // position of the tile that every row sees: below it no mask is needed
  const int64_t all_see = min(sv.len, sv.pos0 + row_lo / a.G + 1);
  const int P = 1 << kv.log_p;
  for (int64_t j0 = c0 + kStep * wave; j0 < c1; j0 += kStep * kAttnWaves) {
    // pages of the K rows this lane loads (group n / 4) and of its own positions (group g)
    const int64_t jk = j0 + 16 * (n >> 2), jv = j0 + 16 * g;
    const int32_t idk = page_of(kv, s, jk >> kv.log_p), idv = page_of(kv, s, jv >> kv.log_p);
    // (a group outside its sequence or its cache reads page 0 and counts for nothing)
    const int8_t* kp = kv.k + ((((int64_t)max(idk, 0) * kv.H + h) << kv.log_p) + (jk & (P - 1))) * D + g * (D / 4);
    const int8_t* vp = kv.v + ((((int64_t)max(idv, 0) * kv.H + h) * D + n) << kv.log_p) + (jv & (P - 1));
    u32x4 kw[4][D / 64], vw[DT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) kw[t][i] = load16(kp + (4 * t + (n & 3)) * D + 16 * i);
#pragma unroll
    for (int d = 0; d < DT; ++d) vw[d] = load16(vp + ((int64_t)(16 * d) << kv.log_p));
    const bool here = idv >= 0 && jv < sv.len;
    const int64_t si = (int64_t)max(idv, 0) * kv.H + h;
    const float ks = here ? load_g(kv.k_scale + si) : 0.0f;
    const float vs = here ? load_g(kv.v_scale + si) : 0.0f;

    f32x4 sc[NT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int u = 0; u < NT; ++u) sc[u][t] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const f16x8 kf = codes_f16(kw[t][j / 2][2 * (j % 2)], kw[t][j / 2][2 * (j % 2) + 1]);
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          sc[u][t] = mfma(kf, qh[u][j], sc[u][t]);
          sc[u][t] = mfma(kf, ql[u][j], sc[u][t]);
        }
      }
    }

    // a larger V scale: everything summed so far moves to its power of two
    const int e_new = min((int)(__builtin_bit_cast(uint32_t, max_groups(vs)) >> 23) - 127, 120);
    if (__builtin_amdgcn_readfirstlane(e_new) > ve) {
      const int e = __builtin_amdgcn_readfirstlane(e_new);
      const float f = ve - e < -126 ? 0.0f : pow2i(ve - e);
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int d = 0; d < DT; ++d) o[u][d] *= f;
      ve = e;
    }
    const float vn = vs * pow2i(14 - ve > 127 ? 127 : 14 - ve);

    const int32_t jv32 = (int32_t)jv;
    const bool masked = j0 + kStep > all_see || __any(!here);
    f16x8 ph[NT][2], pl[NT][2];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      float p[16];
      float mx = kNegInf;
      const float f = cs[u] * ks;
#pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = sc[u][i >> 2][i & 3] * f;
      if (masked) {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = here && jv32 + i <= pos[u] ? p[i] : kNegInf;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, p[i]);
      mx = max_groups(mx);
      if (__any(mx > m[u])) {
        const float mn = fmaxf(m[u], mx);
        const float al = mn == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[u] - mn);
        m[u] = mn;
        l[u] *= al;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[u][d] *= al;
      }
      const float mu = m[u] == kNegInf ? 0.0f : m[u];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[i] = __builtin_amdgcn_exp2f(p[i] - mu);
        l[u] += p[i];
        p[i] *= vn;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f16x2 hi, lo;
          split2(p[8 * k + 2 * i], p[8 * k + 2 * i + 1], hi, lo);
          ph[u][k][2 * i] = hi[0], ph[u][k][2 * i + 1] = hi[1];
          pl[u][k][2 * i] = lo[0], pl[u][k][2 * i + 1] = lo[1];
        }
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f16x8 vf = codes_f16(vw[d][2 * k], vw[d][2 * k + 1]);
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          o[u][d] = mfma(vf, ph[u][k], o[u][d]);
          o[u][d] = mfma(vf, pl[u][k], o[u][d]);
        }
      }
    }
  }

  // join the four waves
  const float back = pow2i(max(ve - 14, -126));
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const float lt = sum_groups(l[u]);
    if (g == 0) sml[wave][16 * u + n][0] = m[u], sml[wave][16 * u + n][1] = lt;
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *reinterpret_cast<f32x4*>(&so[wave][16 * u + n][16 * d + 4 * g]) = o[u][d] * back;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * NT * D; i += 64 * kAttnWaves) {
    const int r = i / D, d = i % D;
    if (row_lo + r >= rows) break;
    float mm = kNegInf;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) mm = fmaxf(mm, sml[w][r][0]);
    float ls = 0.0f, os = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      const float f = sml[w][r][0] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(sml[w][r][0] - mm);
      ls = __builtin_fmaf(sml[w][r][1], f, ls);
      os = __builtin_fmaf(so[w][r][d], f, os);
    }
    const int64_t row = sv.row0 + (row_lo + r) / a.G;
    const int hq = h * a.G + (row_lo + r) % a.G;
    if (a.nchunk == 1) {
      store_g(a.y + row * a.ldy + (int64_t)hq * D + d, ls > 0.0f ? os / ls : 0.0f);
    } else {
      const int64_t at = (row * a.Hq + hq) * a.nchunk + c;
      store_g(a.part + at * D + d, os);
      if (d == 0) {
        store_g(a.part_ml + 2 * at, mm);
        store_g(a.part_ml + 2 * at + 1, ls);
      }
    }
  }
}

// Joins the chunks of each (row, query head): one wave each.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int hq = (int)(w % a.Hq);
  const int64_t rest = w / a.Hq;
  const int i = (int)(rest % a.kv.max_new);
  const int64_t s = rest / a.kv.max_new;
  if (s >= a.kv.S) return;
  const SeqView sv = seq_view(a.kv, (int)s);
  if (i >= sv.n) return;
  // chunks that wrote: those that start before the last position of the row's tile; the row's own
  // positions lie in these
  const int64_t end = min(sv.len, sv.pos0 + i + 1);
  const int nc = (int)min((int64_t)a.nchunk, max((end + a.chunk - 1) / a.chunk, (int64_t)1));
  const int64_t row = sv.row0 + i, at = (row * a.Hq + hq) * a.nchunk;
  float m = kNegInf;
  for (int c = 0; c < nc; ++c) m = fmaxf(m, load_g(a.part_ml + 2 * (at + c)));
  float l = 0.0f, o[D / 64];
#pragma unroll
  for (int d = 0; d < D / 64; ++d) o[d] = 0.0f;
  for (int c = 0; c < nc; ++c) {
    const float mc = load_g(a.part_ml + 2 * (at + c));
    const float f = mc == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mc - m);
    l = __builtin_fmaf(load_g(a.part_ml + 2 * (at + c) + 1), f, l);
#pragma unroll
    for (int d = 0; d < D / 64; ++d) o[d] = __builtin_fmaf(load_g(a.part + (at + c) * D + lane + 64 * d), f, o[d]);
  }
#pragma unroll
  for (int d = 0; d < D / 64; ++d)
    store_g(a.y + row * a.ldy + (int64_t)hq * D + lane + 64 * d, l > 0.0f ? o[d] / l : 0.0f);
}

int attn_tiles_per_wave(int64_t rows) { return rows <= 16 ? 1 : 2; }

}  // namespace

AttnPlan attn_plan(const KvArgs& kv, int64_t Hq, int cus) {
  AttnPlan p;
  const int64_t G = Hq / kv.H, rows = kv.max_new * G;
  p.nt = attn_tiles_per_wave(rows);
  p.row_tiles = (rows + 16 * p.nt - 1) / (16 * p.nt);
  // Chunks: enough workgroups to fill the chip a few times over, each at
  // least one step per wave.
  const int64_t most = kv.ld_table << kv.log_p;
  const int64_t len = kv.max_len > 0 ? std::min(kv.max_len, most) : most;
  const int64_t units = mul_sat(kv.S * kv.H, p.row_tiles);
  const int64_t step = kStep * kAttnWaves;
  const int64_t want = std::max<int64_t>(1, (int64_t)cus * 4 / std::max<int64_t>(1, units));
  const int64_t chunk = std::max<int64_t>(step, ((len + want - 1) / want + step - 1) / step * step);
  p.chunk = std::min<int64_t>(chunk, 1ll << 30);
  p.nchunk = std::max<int64_t>(1, (len + p.chunk - 1) / p.chunk);
  p.work_items = mul_sat(mul_sat(units, p.nchunk), 64 * kAttnWaves);
  p.join_items = p.nchunk > 1 ? mul_sat(mul_sat(kv.S * kv.max_new, Hq) / 4 + 1, 256) : 0;
  p.workspace = p.nchunk > 1 ? mul_sat((int64_t)kv.rows * Hq, p.nchunk * (kv.D + 2) * 4) : 0;
  return p;
}

hipError_t launch_attention(const KvArgs& kv, const AttnPlan& p, const float* q, int64_t ldq, int64_t Hq, float scale,
                            float* y, int64_t ldy, void* workspace, hipStream_t s) {
  AttnArgs a;
  a.kv = kv;
  a.q = q;
  a.y = y;
  a.part = static_cast<float*>(workspace);
  a.part_ml = p.nchunk > 1 ? a.part + (int64_t)kv.rows * Hq * p.nchunk * kv.D : nullptr;
  a.ldq = ldq;
  a.ldy = ldy;
  a.Hq = (int32_t)Hq;
  a.G = (int32_t)(Hq / kv.H);
  a.chunk = (int32_t)p.chunk;
  a.nchunk = (int32_t)p.nchunk;
  a.row_tiles = (int32_t)p.row_tiles;
  a.scale = scale;
  const dim3 grid((unsigned)(p.work_items / (64 * kAttnWaves))), block(64 * kAttnWaves);
  if (kv.D == 64) {
    if (p.nt == 1) hipLaunchKernelGGL((attn_kernel<64, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attn_kernel<64, 2>), grid, block, 0, s, a);
  } else {
    if (p.nt == 1) hipLaunchKernelGGL((attn_kernel<128, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attn_kernel<128, 2>), grid, block, 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.nchunk == 1) return e;
  const dim3 jgrid((unsigned)(p.join_items / 256));
  if (kv.D == 64) hipLaunchKernelGGL((attn_join_kernel<64>), jgrid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((attn_join_kernel<128>), jgrid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace tern
