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
//
// Loads: a wave issues the next step's K loads once the first product has
// read the registers, and the next V loads after the second, so 8 to 16 KB
// per wave are always in flight.  Page ids and scales of up to kWindow
// positions are fetched to LDS at once, out of the steps' way.
#include <algorithm>

#include "tern_cache.h"

namespace tern {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kAttnWaves = 4;
constexpr int kStep = 64;  // positions per step of a wave
constexpr int kWindow = 4096;  // positions whose pages are looked up at once
constexpr int kGroups = kWindow / 16;
static_assert(kGroups == 64 * kAttnWaves, "one group of 16 positions per thread");

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
  bool q16;  // query rows are 16-byte aligned
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

// Eight int8 codes as (code + 128) * 2^-24: u in the low byte of an fp16 is
// the subnormal u * 2^-24, so nothing is subtracted here.  The first product
// starts its sums at -128 times the sum of the query row instead; what that
// costs is a rounding at about twice the magnitude.  (The second product
// cannot: its sums, of many values of either sign, are small beside those of
// values + 128.)
__device__ __forceinline__ f16x8 codes_sub(uint32_t w0, uint32_t w1) {
  w0 ^= 0x80808080u;
  w1 ^= 0x80808080u;
  const u32x4 o = {__builtin_amdgcn_perm(0u, w0, 0x0c010c00u), __builtin_amdgcn_perm(0u, w0, 0x0c030c02u),
                   __builtin_amdgcn_perm(0u, w1, 0x0c010c00u), __builtin_amdgcn_perm(0u, w1, 0x0c030c02u)};
  return __builtin_bit_cast(f16x8, o);
}

// v - hi of one half of a pair: one instruction that reads the fp16 as it is.
template <bool HIGH>
__device__ __forceinline__ float minus_half(float v, f16x2 h) {
  float r;
  if constexpr (HIGH)
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r) : "v"(h), "v"(v));
  else
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r) : "v"(h), "v"(v));
  return r;
}
// v = hi + lo to 22 bits (hi rounded toward zero: lo has its sign).
__device__ __forceinline__ void split2(float a, float b, f16x2& hi, f16x2& lo) {
  hi = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(a, b));
  lo = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(minus_half<false>(a, hi), minus_half<true>(b, hi)));
}

// The value of the lane eight columns on (the other half of a packed tile).
__device__ __forceinline__ float other_half(float v) {
  return __builtin_bit_cast(float, dpp_partner<8>(__builtin_bit_cast(uint32_t, v)));
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
// steps the four waves take in turn.  PACK: 8 rows, whose high and low
// operands are the columns 0-7 and 8-15 of one matrix operand, so a product
// takes one instruction where two tiles would take two.
template <int D, int NT, bool PACK>
__global__ __launch_bounds__(64 * kAttnWaves, 2) void attn_kernel(AttnArgs a) {
  constexpr int KS = D / 32;  // k steps of the first product
  constexpr int DT = D / 16;  // 16-dim tiles of the output
  constexpr int LD = D + 4;
  constexpr int ROWS = PACK ? 8 : 16 * NT;
  static_assert(!PACK || NT == 1, "a packed tile stands alone");
  // the query operands (high and low halves, by lane), and after the last step the waves' sums of a tile
  union Share {
    f16x8 q[NT][KS][PACK ? 1 : 2][64];
    float o[kAttnWaves][16][LD];
  };
  __shared__ Share sh;
  __shared__ float sml[kAttnWaves][16 * NT][2];
  // a row's |scale| * log2(e) * powers of two, and where its sums start
  __shared__ float qfac[16 * NT], qbias[16 * NT];
  __shared__ int32_t page[kGroups];  // of a group of 16 positions (-1: none there)
  __shared__ float kscale[kGroups], vscale[kGroups];

  const KvArgs& kv = a.kv;
  int b = blockIdx.x;
  const int h = b % kv.H;
  b /= kv.H;
  const int c = b % a.nchunk;
  b /= a.nchunk;
  const int rt = a.row_tiles - 1 - b % a.row_tiles;
  const int s = b / a.row_tiles;
  const SeqView sv = seq_view(kv, s);
  const int rows = min(sv.n, (int)kv.max_new) * a.G, row_lo = rt * ROWS;
  if (row_lo >= rows) return;
  // positions that some row of the tile sees: up to the last row's own
  const int64_t last_pos = sv.pos0 + min(row_lo + ROWS - 1, rows - 1) / a.G;
  const int64_t end = min(sv.len, last_pos + 1);
  const int64_t c0 = (int64_t)c * a.chunk;
  const int64_t c1 = c == a.nchunk - 1 ? end : min(end, c0 + a.chunk);
  // (chunk 0 always writes: it is the one that the joining pass counts on)
  if (c0 >= c1 && c > 0) return;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, g = lane >> 4;
  const int nr = PACK ? n & 7 : n;  // the lane's row of a tile
  const bool low = PACK && n >= 8;  // the lane holds low operands

  // Loads in three trips to memory: the sequence; page ids and query rows;
  // scales, K and V.  Wave u prepares query tile u, for all the waves, while
  // its first K and V are under way.
  float x[D / 4];
  if (wave < NT) {
    const int r = row_lo + 16 * wave + nr;
    const bool live = r < rows;
    const float* q = a.q + (int64_t)(sv.row0 + (live ? r / a.G : 0)) * a.ldq +
                     (int64_t)(h * a.G + (live ? r % a.G : 0)) * D + g * (D / 4);
    // (a row past the last reads the sequence's first, for zeros)
    if (a.q16) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const f32x4 v = __builtin_bit_cast(f32x4, load16(q + 4 * j));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * j + i] = v[i];
      }
    } else {
#pragma unroll
      for (int j = 0; j < D / 4; ++j) x[j] = load_g(q + j);
    }
  }
  auto prepare_q = [&]() {
    const bool live = row_lo + 16 * wave + nr < rows;
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 4; ++j) {
      x[j] = live ? x[j] : 0.0f;
      amax = fmaxf(amax, fabsf(x[j]));
    }
    amax = max_groups(amax);
    // 2^(8 - exponent): the largest element lands in [2^8, 2^9); the sign of
    // the scale goes with it, so that a row's factor is not negative
    const int e = min(max((int)(__builtin_bit_cast(uint32_t, amax) >> 23) - 127, -100), 120);
    const float up = a.scale < 0.0f ? -pow2i(8 - e) : pow2i(8 - e);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      f16x8 qh, ql;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x0 = x[8 * j + 2 * i] * up, x1 = x[8 * j + 2 * i + 1] * up;
        f16x2 hi, lo;
        split2(x0, x1, hi, lo);
        qh[2 * i] = hi[0], qh[2 * i + 1] = hi[1];
        ql[2 * i] = lo[0], ql[2 * i + 1] = lo[1];
        if (PACK)
          sum += low ? (float)lo[0] + (float)lo[1] : (float)hi[0] + (float)hi[1];
        else
          sum += x0 + x1;
      }
      if constexpr (PACK) {
        sh.q[wave][j][0][lane] = low ? ql : qh;
      } else {
        sh.q[wave][j][0][lane] = qh;
        sh.q[wave][j][1][lane] = ql;
      }
    }
    sum = sum_groups(sum);
    if (g == 0) {
      qfac[16 * wave + n] = fabsf(a.scale) * 1.44269504088896340736f * pow2i(e - 8) * 16777216.0f;
      qbias[16 * wave + n] = sum * (-128.0f / 16777216.0f);
    }
  };
  int32_t pos[NT];  // last position that the row sees (-1: none)
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int r = row_lo + 16 * u + nr;
    pos[u] = r < rows ? (int32_t)max(min(sv.pos0 + r / a.G, sv.len - 1), (int64_t)-1) : -1;
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
  u32x4 kw[4][D / 64], vw[DT];
  int64_t w0 = c0;
  int steps = 0;
  // A step's K rows (this lane's are of group n / 4) and V rows (of its own
  // positions, group g).  A group without a page reads page 0 and counts for
  // nothing.
  auto load_k = [&](int st) {
    const int gr = 4 * st + (n >> 2);
    const int64_t base = (((int64_t)max(page[gr], 0) * kv.H + h) << kv.log_p) + (((int)w0 + 16 * gr) & (P - 1));
    const int8_t* kp = kv.k + (base + (n & 3)) * D + g * (D / 4);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) kw[t][i] = load16(kp + 4 * t * D + 16 * i);
  };
  auto load_v = [&](int st) {
    const int gr = 4 * st + g;
    const int8_t* vp = kv.v + ((((int64_t)max(page[gr], 0) * kv.H + h) * D + n) << kv.log_p) +
                       (((int)w0 + 16 * gr) & (P - 1));
#pragma unroll
    for (int d = 0; d < DT; ++d) vw[d] = load16(vp + ((int64_t)(16 * d) << kv.log_p));
  };
  // The pages and scales of the window at w0, and its first loads.
  auto open_window = [&]() {
    const int64_t j = w0 + 16 * (int)threadIdx.x;
    const int32_t id = j < sv.len ? page_of(kv, s, j >> kv.log_p) : -1;
    const int64_t si = (int64_t)max(id, 0) * kv.H + h;
    const float ks = load_g(kv.k_scale + si), vs = load_g(kv.v_scale + si);
    page[threadIdx.x] = id;
    __syncthreads();
    steps = (int)((min(c1 - w0, (int64_t)kWindow) + kStep - 1) / kStep);
    if (wave < steps) {
      load_k(wave);
      load_v(wave);
    }
    kscale[threadIdx.x] = id < 0 ? 0.0f : ks;
    vscale[threadIdx.x] = id < 0 ? 0.0f : vs;
  };
  open_window();
  if (wave < NT) prepare_q();
  __syncthreads();
  for (;;) {
    f32x4 sc[NT][4];
    auto scores = [&]() {
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const float b = qbias[16 * u + n];
#pragma unroll
        for (int t = 0; t < 4; ++t) sc[u][t] = {b, b, b, b};
      }
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        f16x8 q[NT][2];
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int e = 0; e < (PACK ? 1 : 2); ++e) q[u][e] = sh.q[u][j][e][lane];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const f16x8 kf = codes_sub(kw[t][j / 2][2 * (j % 2)], kw[t][j / 2][2 * (j % 2) + 1]);
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int e = 0; e < (PACK ? 1 : 2); ++e) sc[u][t] = mfma(kf, q[u][e], sc[u][t]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (PACK) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[0][t][i] += other_half(sc[0][t][i]);
      }
    };
    auto weigh_and_sum = [&](int st) {
      const int64_t j0 = w0 + kStep * st;
      const int32_t jv = (int32_t)j0 + 16 * g;
      const bool here = page[4 * st + g] >= 0;
      const float ks = kscale[4 * st + g], vs = vscale[4 * st + g];
      // a larger V scale: everything summed so far moves to its power of two
      const int e = __builtin_amdgcn_readfirstlane(
          min((int)(__builtin_bit_cast(uint32_t, max_groups(vs)) >> 23) - 127, 120));
      if (e > ve) {
        const float f = ve - e < -126 ? 0.0f : pow2i(ve - e);
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int d = 0; d < DT; ++d) o[u][d] *= f;
        ve = e;
      }
      // weights take the V scale, vn <= 2^15, with the exponential: e^(s - m)
      // vn = 2^(s' - m' + log2 vn), and sums of weights are divided by it.  A
      // scale of 0, or far below the largest, is multiplied afterwards.
      const float vn = vs * pow2i(14 - ve);
      const bool apart = vn < 0x1p-16f;
      const float lv = apart ? 0.0f : __builtin_amdgcn_logf(vn), rl = apart ? 1.0f : __builtin_amdgcn_rcpf(vn);
      const bool any_apart = __any(apart);

      const bool masked = j0 + kStep > all_see || __any(!here);
      f16x8 pb[NT][2][2];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        float f = qfac[16 * u + n] * ks;
        if (masked) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sc[u][i >> 2][i & 3] = here && jv + i <= pos[u] ? sc[u][i >> 2][i & 3] * f : kNegInf;
          f = 1.0f;
        }
        float mx = sc[u][0][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[u][i >> 2][i & 3]);
        mx = max_groups(mx * f);
        if (__any(mx > m[u])) {
          const float mn = fmaxf(m[u], mx);
          const float al = mn == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[u] - mn);
          m[u] = mn;
          l[u] *= al;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[u][d] *= al;
        }
        const float off = lv - (m[u] == kNegInf ? 0.0f : m[u]);
        float p[16], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[u][i >> 2][i & 3], f, off));
          sum += p[i];
        }
        l[u] = __builtin_fmaf(sum, rl, l[u]);
        if (any_apart) {
          const float mul = apart ? vn : 1.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] *= mul;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f16x2 hi, lo;
            split2(p[8 * k + 2 * i], p[8 * k + 2 * i + 1], hi, lo);
            if constexpr (PACK) hi = low ? lo : hi;
            pb[u][k][0][2 * i] = hi[0], pb[u][k][0][2 * i + 1] = hi[1];
            pb[u][k][1][2 * i] = lo[0], pb[u][k][1][2 * i + 1] = lo[1];
          }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const f16x8 vf = codes_f16(vw[d][2 * k], vw[d][2 * k + 1]);
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int e = 0; e < (PACK ? 1 : 2); ++e) o[u][d] = mfma(vf, pb[u][k][e], o[u][d]);
        }
    };
    // (the last step apart: a load that may or may not have been issued would
    // have every step wait for all of them)
    int st = wave;
    for (; st + kAttnWaves < steps; st += kAttnWaves) {
      asm volatile("" ::: "memory");  // (the query operands stay in LDS: held in registers they cost a wave per SIMD)
      scores();
      load_k(st + kAttnWaves);
      weigh_and_sum(st);
      load_v(st + kAttnWaves);
    }
    if (st < steps) {
      scores();
      weigh_and_sum(st);
    }
    w0 += kWindow;
    if (w0 >= c1) break;
    __syncthreads();  // (the window before has been read)
    open_window();
    __syncthreads();
  }

  // join the four waves, a tile at a time
  const float back = pow2i(max(ve - 14, -126));
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const float lt = sum_groups(l[u]);
    if (g == 0) sml[wave][16 * u + n][0] = m[u], sml[wave][16 * u + n][1] = lt;
  }
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    __syncthreads();  // (the operands, or the tile before, have been read)
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      f32x4 v = o[u][d] * back;
      if constexpr (PACK) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += other_half(v[i]);
      }
      *reinterpret_cast<f32x4*>(&sh.o[wave][n][16 * d + 4 * g]) = v;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (PACK ? 8 : 16) * D; i += 64 * kAttnWaves) {
      const int r = 16 * u + i / D, d = i % D;
      if (row_lo + r >= rows) break;
      float mm = kNegInf;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) mm = fmaxf(mm, sml[w][r][0]);
      float ls = 0.0f, os = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) {
        const float f = sml[w][r][0] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(sml[w][r][0] - mm);
        ls = __builtin_fmaf(sml[w][r][1], f, ls);
        os = __builtin_fmaf(sh.o[w][i / D][d], f, os);
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
}

// Joins the chunks of each (row, query head): a workgroup of four waves each,
// wave w the chunks w, w + 4, ...
template <int D>
__global__ __launch_bounds__(64 * kAttnWaves) void attn_join_kernel(AttnArgs a) {
  __shared__ float so[kAttnWaves][D], sml[kAttnWaves][2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int hq = (int)(blockIdx.x % a.Hq);
  const int64_t rest = blockIdx.x / a.Hq;
  const int i = (int)(rest % a.kv.max_new);
  const SeqView sv = seq_view(a.kv, (int)(rest / a.kv.max_new));
  if (i >= sv.n) return;
  // chunks that hold positions of the row (their workgroups have written)
  const int64_t end = min(sv.len, sv.pos0 + i + 1);
  const int nc = (int)min((int64_t)a.nchunk, max((end + a.chunk - 1) / a.chunk, (int64_t)1));
  const int64_t row = sv.row0 + i, at = (row * a.Hq + hq) * a.nchunk;
  // up to 64 of the wave's chunks at a time: a lane holds one chunk's m and l
  float m = kNegInf, l = 0.0f, o[D / 64];
#pragma unroll
  for (int d = 0; d < D / 64; ++d) o[d] = 0.0f;
  for (int b = wave; b < nc; b += 64 * kAttnWaves) {
    const int c = b + kAttnWaves * lane;
    const float mc = c < nc ? load_g(a.part_ml + 2 * (at + c)) : kNegInf;
    const float lc = c < nc ? load_g(a.part_ml + 2 * (at + c) + 1) : 0.0f;
    float mn = mc;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) mn = fmaxf(mn, __shfl_xor(mn, d, 64));
    mn = fmaxf(mn, m);
    if (mn == kNegInf) continue;  // (nothing seen yet)
    const float al = __builtin_amdgcn_exp2f(m - mn), f = __builtin_amdgcn_exp2f(mc - mn);
    m = mn;
    float ls = lc * f;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) ls += __shfl_xor(ls, d, 64);
    l = __builtin_fmaf(l, al, ls);
#pragma unroll
    for (int d = 0; d < D / 64; ++d) o[d] *= al;
    const int cn = min(64, (nc - b + kAttnWaves - 1) / kAttnWaves);
#pragma unroll 4
    for (int e = 0; e < cn; ++e) {
      const float fe = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), e));
#pragma unroll
      for (int d = 0; d < D / 64; ++d)
        o[d] = __builtin_fmaf(load_g(a.part + (at + b + kAttnWaves * e) * D + lane + 64 * d), fe, o[d]);
    }
  }
  if (lane == 0) sml[wave][0] = m, sml[wave][1] = l;
#pragma unroll
  for (int d = 0; d < D / 64; ++d) so[wave][lane + 64 * d] = o[d];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 64 * kAttnWaves) {
    float mm = kNegInf, ls = 0.0f, os = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) mm = fmaxf(mm, sml[w][0]);
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      const float f = sml[w][0] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(sml[w][0] - mm);
      ls = __builtin_fmaf(sml[w][1], f, ls);
      os = __builtin_fmaf(so[w][d], f, os);
    }
    store_g(a.y + row * a.ldy + (int64_t)hq * D + d, ls > 0.0f ? os / ls : 0.0f);
  }
}

constexpr int kWgPerCu = 4;

// 16-row tiles per workgroup; 0: eight rows in a packed tile.
int attn_tiles(int64_t rows) { return rows <= 8 ? 0 : rows <= 16 ? 1 : 2; }

template <int D>
void launch_tiles(int nt, dim3 grid, dim3 block, const AttnArgs& a, hipStream_t s) {
  if (nt == 0) hipLaunchKernelGGL((attn_kernel<D, 1, true>), grid, block, 0, s, a);
  else if (nt == 1) hipLaunchKernelGGL((attn_kernel<D, 1, false>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((attn_kernel<D, 2, false>), grid, block, 0, s, a);
}

}  // namespace

AttnPlan attn_plan(const KvArgs& kv, int64_t Hq, int cus) {
  AttnPlan p;
  const int64_t G = Hq / kv.H, rows = kv.max_new * G;
  p.nt = attn_tiles(rows);
  const int64_t tile = p.nt == 0 ? 8 : 16 * p.nt;
  p.row_tiles = (rows + tile - 1) / tile;
  // Chunks: enough workgroups to fill the chip a few times over, each at
  // least one step per wave.
  const int64_t most = kv.ld_table << kv.log_p;
  const int64_t len = kv.max_len > 0 ? std::min(kv.max_len, most) : most;
  const int64_t units = mul_sat(kv.S * kv.H, p.row_tiles);
  const int64_t step = kStep * kAttnWaves;
  const int64_t want = std::max<int64_t>(1, (int64_t)cus * kWgPerCu / std::max<int64_t>(1, units));
  const int64_t chunk = std::max<int64_t>(step, ((len + want - 1) / want + step - 1) / step * step);
  p.chunk = std::min<int64_t>(chunk, 1ll << 30);
  p.nchunk = std::max<int64_t>(1, (len + p.chunk - 1) / p.chunk);
  p.work_items = mul_sat(mul_sat(units, p.nchunk), 64 * kAttnWaves);
  p.join_items = p.nchunk > 1 ? mul_sat(mul_sat(kv.S * kv.max_new, Hq), 64 * kAttnWaves) : 0;
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
  a.q16 = reinterpret_cast<uintptr_t>(q) % 16 == 0 && (kv.rows == 1 || ldq % 4 == 0);
  const dim3 grid((unsigned)(p.work_items / (64 * kAttnWaves))), block(64 * kAttnWaves);
  if (kv.D == 64)
    launch_tiles<64>(p.nt, grid, block, a, s);
  else
    launch_tiles<128>(p.nt, grid, block, a, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.nchunk == 1) return e;
  const dim3 jgrid((unsigned)(p.join_items / (64 * kAttnWaves)));
  if (kv.D == 64) hipLaunchKernelGGL((attn_join_kernel<64>), jgrid, block, 0, s, a);
  else hipLaunchKernelGGL((attn_join_kernel<128>), jgrid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace tern
