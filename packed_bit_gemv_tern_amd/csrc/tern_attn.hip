// tern_attn.hip -- attention over the paged int8 cache.
//
// Row r (a new token and a query head) sees the positions j <= pos_r of its
// sequence; with k_j = ks_j * ck_j, v_j = vs_j * cv_j (codes ck, cv, scales
// of the page and KV head):
//
//     s_j = scale * (q_r . k_j),  y_r = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// in one pass over the positions with a running maximum (here the units of the
// sums) and sum.  A row with no position to see is 0.
//
// Matrix form, per step of 64 positions (v_mfma_f32_16x16x32_f16, fp32
// accumulators):  S^T = K Q^T,  O^T += V^T P^T.  The codes are exact in
// fp16.  The other operand of each product is split in two fp16 numbers, hi
// + lo, 23 bits together: q after a power of two that brings the row's
// largest element under 2^9 (so that lo stays far above fp16's smallest
// numbers), and the weights w_j = e^(s_j) vs_j 2^-R.  Errors are then those of
// fp32.
//
// Small weights are what the split has to get right: a position that takes
// nearly all of a row's softmax may hold values near 0, and pages with large V
// scales may have hardly any of it, so the weights that make up y can be far
// below the largest.  hi + lo is good to 23 bits of a weight from 2^-3 on and to
// 2^-25 below that.  With the largest weight brought to 2^9 .. 2^15 that is enough
// for a row whose largest sum ends at 2^8 or more (2^-33 of it for each
// weight).  A workgroup with other rows takes its positions again for those, in
// bands of 18 octaves of weight, each in units of its own (next_band).
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
// per wave are always in flight.  Page ids and scales of 1,024 positions
// per wave are fetched to LDS at once, out of the steps' way.
#include <algorithm>

#include "tern_cache.h"

namespace tern {

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 64;  // positions per step of a wave
constexpr int kWaves = 4;  // of a workgroup
constexpr int kJoinWaves = 4;

// n / d for 0 <= n < 2^31 by a multiplication (an integer division is some
// thirty instructions, and a workgroup begins with several).
struct FastDiv {
  uint32_t d, mul, shift;
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
  __device__ __forceinline__ uint32_t divmod(uint32_t n, uint32_t& rem) const {
    const uint32_t q = div(n);
    rem = n - q * d;
    return q;
  }
};
inline FastDiv fast_div(int64_t d) {  // d in [1, 2^31)
  FastDiv f = {(uint32_t)d, 0, 0};
  while ((1ull << f.shift) < (uint64_t)d) ++f.shift;
  f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - (uint64_t)d)) / (uint64_t)d + 1);
  return f;
}

struct AttnArgs {
  KvArgs kv;
  const float* q;
  float* y;
  float* part;  // per (row, head, chunk): D sums, then m and l per (row, head, chunk)
  float* part_ml;
  int64_t ldq, ldy;
  int32_t Hq;
  int32_t chunk, nchunk;  // positions per chunk, chunks a sequence is split into
  int32_t row_tiles;
  FastDiv by_h, by_chunks, by_tiles, by_g;  // KV heads, chunks, row tiles, query heads per KV head
  float scale;
  bool q16, y16;  // query rows, output rows are 16-byte aligned
};

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Eight int8 codes as fp16, exactly: 0x6400 | u is 1024 + u, u = code + 128.
// (Codes + 128 as subnormals, and scores that start at -128 times the sum of the
// query row, cost two instructions in five less and 1 % of the prompts' time, but
// such scores round at the size of 128 |sum q|: with one key channel far above the
// others and a query row of one sign that was 60 times as far off.)
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
// v = hi + lo, each rounded to nearest: to 23 bits while lo is normal.
__device__ __forceinline__ void split2(float a, float b, f16x2& hi, f16x2& lo) {
  hi = __builtin_convertvector(f32x2{a, b}, f16x2);
  lo = __builtin_convertvector(f32x2{minus_half<false>(a, hi), minus_half<true>(b, hi)}, f16x2);
}

// The value of the lane eight columns on (the other half of a packed tile).
__device__ __forceinline__ float other_half(float v) {
  return __builtin_bit_cast(float, dpp_partner<8>(__builtin_bit_cast(uint32_t, v)));
}

__device__ __forceinline__ float pow2i(int e) { return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23); }

// Maximum / sum over the four lanes that hold one query row.
__device__ __forceinline__ float max_groups(float v) {
  auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  v = fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
  p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
}
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

constexpr float kNegInf = -__builtin_inff();

// The elements of a query row that lane group g holds: 16 g .. 16 g + 15 of
// every 64, the operands of k steps 2 i and 2 i + 1 (8 each).
template <int D>
__device__ __forceinline__ void load_query(const AttnArgs& a, const float* q, int g, float (&x)[D / 4]) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const float* p = q + 64 * i + 16 * g;
    if (a.q16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 v = __builtin_bit_cast(f32x4, load16(p + 4 * j));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[16 * i + 4 * j + e] = v[e];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[16 * i + j] = load_g(p + j);
    }
  }
}

// The power of two that brings a query row's largest element to [2^8, 2^9),
// with the sign of the scale (so that the factor of its scores is not
// negative), and that factor: |scale| * log2(e) * the powers of two left out.
struct QueryScale {
  float up, factor;
};
template <int D>
__device__ __forceinline__ QueryScale query_scale(float scale, const float (&x)[D / 4]) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < D / 4; ++j) amax = fmaxf(amax, fabsf(x[j]));
  amax = max_groups(amax);
  const int e = min(max((int)(__builtin_bit_cast(uint32_t, amax) >> 23) - 127, -100), 120);
  const float up = scale < 0.0f ? -pow2i(8 - e) : pow2i(8 - e);
  return {up, fabsf(scale) * 1.44269504088896340736f * pow2i(e - 8)};
}
// One k step's operands, high and low.
__device__ __forceinline__ void split_query(const float (&x)[8], float up, f16x8& qh, f16x8& ql) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f16x2 hi, lo;
    split2(x[2 * i] * up, x[2 * i + 1] * up, hi, lo);
    qh[2 * i] = hi[0], qh[2 * i + 1] = hi[1];
    ql[2 * i] = lo[0], ql[2 * i + 1] = lo[1];
  }
}

// The V scale of the lane's 16 positions in a step: vs = 2^(lm + e), lm in
// [-1, 0), and 2^-lm (e = -infinity for a scale of 0).  Weights take it with
// the exponential.
struct VScale {
  float lm, e, rm;
};
__device__ __forceinline__ VScale v_scale(float vs) {
  const float mant = vs == 0.0f ? 1.0f : __builtin_amdgcn_frexp_mantf(vs);
  return {__builtin_amdgcn_logf(mant), vs == 0.0f ? kNegInf : (float)__builtin_amdgcn_frexp_expf(vs),
          __builtin_amdgcn_rcpf(mant)};
}

// What a row has summed: o holds sums of code * e^s vs in units of 2^R, l the
// sum of e^s in units of 2^L; R and L are whole numbers, so changing units
// is exact.  R grows where a weight would pass 2^15 (fp16 ends at 2^16), L where
// an e^s would pass 2^24 (in waves with a base: 1).
constexpr float kNoUnit = -3.0e38f;  // nothing summed yet (finite: differences with -infinity stay that)
constexpr float kTop = 15.0f;
constexpr float kLead = 24.0f;  // octaves that an e^s may be above L
constexpr float kDeep = 200.0f;  // R is not further below L: such weights give 0 in fp32
constexpr float kReset = 10.0f;  // a new R brings the step's largest weight to 2^9 .. 2^10
struct RowUnits {
  float R, L;
};
__device__ __forceinline__ float pow2_of(float e) {  // 2^e of a whole number, 0 below 2^-126
  return e < -126.0f ? 0.0f : pow2i((int)fminf(e, 120.0f));
}
template <int DT>
__device__ __forceinline__ void change_unit(float to, RowUnits& r, f32x4 (&o)[DT]) {
  const float al = pow2_of(r.R - to);
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] *= al;
  r.R = to;
}

// Scores beyond 2^20, of which fp32 holds too few digits for units: the row's are
// counted from a base, the largest when that was met (Far: what a wave keeps of
// it).  Scores are rounded before the base is taken off, as a plain form rounds
// them, so those near the base are exact beside it.
constexpr float kFar = 1048576.0f;
struct Far {
  float* base;  // of the wave's rows, in LDS
  bool any;     // some row has one
};
// One row's 16 scores of a step times f (units of log2), of which only the
// positions up to `last` of the lane's 16 count.
__device__ __forceinline__ void mask_scores(f32x4 (&sc)[4], float& f, int last) {
#pragma unroll
  for (int i = 0; i < 16; ++i) sc[i >> 2][i & 3] = i <= last ? sc[i >> 2][i & 3] * f : kNegInf;
  f = 1.0f;
}
__device__ __forceinline__ float largest_score(const f32x4 (&sc)[4], float f) {
  float mx = sc[0][0];
#pragma unroll
  for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[i >> 2][i & 3]);
  return mx * f;
}
// Scores (f is 1) from the row's base, a new one where they pass it by 2^20.
__device__ __forceinline__ void from_base(f32x4 (&sc)[4], RowUnits& r, const Far& far, int row) {
  const float ms = __builtin_ceilf(max_groups(largest_score(sc, 1.0f)));
  float base = far.base[row];
  if (ms - base > r.L && fabsf(ms - base) > kFar) {
    r = {fmaxf(r.R - (ms - base), kNoUnit), fmaxf(r.L - (ms - base), kNoUnit)};
    far.base[row] = base = ms;  // (the row's lanes alike)
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) sc[i >> 2][i & 3] -= base;
}
// Brings the row's units to the step.  Returns the exponent that the lane's weights
// take from the V scale (v.e; -infinity where their e^s had to be summed here).
template <int DT>
__device__ __forceinline__ float row_units(f32x4 (&sc)[4], float& f, const VScale& v, RowUnits& r, float& l,
                                           f32x4 (&o)[DT], Far& far, int row) {
  if (far.any) from_base(sc, r, far, row);
  float mx = largest_score(sc, f);
  float tl = mx + (v.lm + v.e);  // the lane's largest weight
  float t = max_groups(tl);
  float e = v.e;
  const float lead = far.any ? 0.0f : kLead;
  if (__any(t - r.R > kTop || mx - r.L > lead)) {
    float ms = __builtin_ceilf(max_groups(mx));
    if (!far.any && __any(ms - r.L > lead && fabsf(ms) > kFar)) {
      far.any = true;
      mask_scores(sc, f, 15);
      from_base(sc, r, far, row);
      mx = largest_score(sc, f);
      tl = mx + (v.lm + v.e);
      t = max_groups(tl);
      ms = __builtin_ceilf(max_groups(mx));
    }
    if (ms - r.L > lead) {
      l *= pow2_of(r.L - ms);
      r.L = ms;
    }
    change_unit(fmaxf(t - r.R > kTop ? __builtin_ceilf(t) - kReset : r.R, r.L - kDeep), r, o);
  }
  // A lane whose weights vanish beside the row's (a V scale of 0, or 2^-90 of
  // the others'): its e^s count all the same.
  const bool own = tl < r.R - 90.0f;
  if (__any(own && mx > kNegInf)) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i >> 2][i & 3], f, -r.L));
    l += own ? sum : 0.0f;
    e = own ? kNegInf : e;
  }
  return e;
}
// and their weights, as operands of the second product (high and low); returns
// the sum of their e^s in units of 2^L.
__device__ __forceinline__ float row_weights(const f32x4 (&sc)[4], float f, const VScale& v, float e, const RowUnits& r,
                                             f16x8 (&hi)[2], f16x8 (&lo)[2]) {
  const float d = e - r.R, off = v.lm + d;
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = 8 * k + 2 * i;
      const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[x >> 2][x & 3], f, off));
      const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[x >> 2][(x & 3) + 1], f, off));
      sum += p0 + p1;
      f16x2 h, r;
      split2(p0, p1, h, r);
      hi[k][2 * i] = h[0], hi[k][2 * i + 1] = h[1];
      lo[k][2 * i] = r[0], lo[k][2 * i + 1] = r[1];
    }
  return __builtin_ldexpf(sum * v.rm, (int)(-d - r.L));
}

// The row's sum of e^s, and its unit's exponent for the join.  The unit brings the
// sum to 1/2 .. 1, so that sums of values are no larger than the values (a base
// has no digits for that: there the unit is the largest e^s as it is).
__device__ __forceinline__ float whole_sum(float l, RowUnits& r, const Far& far, int row, float& m) {
  l = sum_groups(l);
  const float base = far.any ? far.base[row] : 0.0f;
  const int e = l > 0.0f && base == 0.0f ? __builtin_amdgcn_frexp_expf(l) : 0;
  r.L += (float)e;
  m = l == 0.0f ? kNegInf : base + r.L;
  return __builtin_ldexpf(l, -e);
}

// The weights that a band takes, e^s vs from 2^from up to 2^to (-infinity, and
// below: none), and a row's next one: after the first pass of all weights, from
// the border of fp16's full precision up, then 18 octaves at a time, with
// smaller units, until the sums have passed 2^8 (or 60 octaves are done): the
// rest at once.  Returns whether the row takes part.
struct Band {
  float from, to;
};
constexpr float kInf = __builtin_inff();
constexpr float kFull = -3.0f, kBand = 18.0f, kSettled = 256.0f;
static_assert(kFull + kBand == kTop, "a band's weights are those that fit its units");
template <int DT, bool PACK>
__device__ bool next_band(int pass, bool live, RowUnits& r, f32x4 (&o)[DT], Band& b) {
  float big = 0.0f;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) big = fmaxf(big, fabsf(o[d][i]));
  big = max_groups(big);
  if constexpr (PACK) big = fmaxf(big, other_half(big));
  const bool settled = !(big < kSettled);
  Band n = {kInf, kNegInf};
  if (pass == 0) {
    if (live && !settled && r.R > r.L - kDeep) {
      n = {r.R + kFull, kInf};
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
  } else if (fabsf(b.from) < kInf) {
    n = {kNegInf, b.from};
    if (!settled && pass < 4) {
      change_unit(r.R - kBand, r, o);
      n.from = r.R + kFull;
    }
  }
  b = n;
  return n.from < kInf;
}
__device__ __forceinline__ void band_scores(f32x4 (&sc)[4], float& f, const VScale& v, const Band& b, float base) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float s = sc[i >> 2][i & 3] * f - base, t = s + (v.lm + v.e);
    sc[i >> 2][i & 3] = t >= b.from && t < b.to ? s : kNegInf;
  }
  f = 1.0f;
}

// see attn_prompt_kernel
__device__ __forceinline__ int swizzle(int g) { return (0x84C0 >> (4 * g)) & 15; }

// One workgroup: one (sequence, KV head), 16 * NT rows (row i: new token i /
// G, query head i % G of the KV head's), one chunk of the positions, whose
// steps the four waves take in turn.  PACK: 8 rows, whose high and low
// operands are the columns 0-7 and 8-15 of one matrix operand, so a product
// takes one instruction where two tiles would take two.
// HBM bound for many sequences: 48 contexts to 8,192 (363 MB of codes) in 72
// us, 5.0 TB/s.  Short of that a chain bounds it: two trips to memory (the
// sequence and page ids; q, scales, K and V), 1.8 us per step of a wave, the
// join: one token on 4,099 positions 7.6 + 3.8 us (8.4 MB: 1.7 at HBM's rate),
// eight on 32,771 23.9 + 4.6 (67 MB: 14).  Rows that take another pass (next_band)
// cost it: one zero-valued position that takes the weight three more, 21.8 us
// for one token, 72 for the eight.
template <int D, int NT, bool PACK>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_kernel(AttnArgs a) {
  constexpr int W = kWaves;
  constexpr int KS = D / 32;  // k steps of the first product
  constexpr int DT = D / 16;  // 16-dim tiles of the output
  constexpr int LD = D + 4;
  constexpr int kGroups = 64 * W;         // groups of 16 positions, one per thread,
  constexpr int kWindow = 16 * kGroups;   // whose pages are looked up at once
  constexpr int ROWS = PACK ? 8 : 16 * NT;
  static_assert(!PACK || NT == 1, "a packed tile stands alone");
  // the query operands (high and low halves, by lane), and after the last step the waves' sums of a tile
  union Share {
    f16x8 q[NT][KS][PACK ? 1 : 2][64];
    float o[W][16][LD];
  };
  __shared__ Share sh;
  __shared__ float sml[W][16 * NT][2];
  __shared__ float qfac[16 * NT];  // a row's |scale| * log2(e) * powers of two
  __shared__ int32_t page[kGroups];  // of a group of 16 positions (-1: none there)
  __shared__ float kscale[kGroups];
  __shared__ VScale vscale[kGroups];
  __shared__ Band band[W][16 * NT];
  __shared__ float base[W][16 * NT];
  __shared__ int again;  // some row needs another pass

  const KvArgs& kv = a.kv;
  uint32_t h, cu, tile;
  const int s = (int)a.by_tiles.divmod(a.by_chunks.divmod(a.by_h.divmod(blockIdx.x, h), cu), tile);
  const int c = (int)cu, G = (int)a.by_g.d;
  const int rt = a.row_tiles - 1 - (int)tile;
  const int64_t c0 = (int64_t)c * a.chunk;
  // (asked for before the sequence is known: its length only says which count)
  int32_t entry = page_entry(kv, s, (c0 + 16 * (int)threadIdx.x) >> kv.log_p);
  const SeqView sv = seq_view(kv, s);
  const int rows = min(sv.n, (int)kv.max_new) * G, row_lo = rt * ROWS;
  if (row_lo >= rows) return;
  // positions that some row of the tile sees: up to the last row's own
  const int64_t last_pos = sv.pos0 + (int)a.by_g.div(min(row_lo + ROWS - 1, rows - 1));
  const int64_t end = min(sv.len, last_pos + 1);
  const int64_t c1 = c == a.nchunk - 1 ? end : min(end, c0 + a.chunk);
  // (chunk 0 always writes: it is the one that the joining pass counts on)
  if (c0 >= c1 && c > 0) return;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int nr = PACK ? n & 7 : n;  // the lane's row of a tile
  const bool low = PACK && n >= 8;  // the lane holds low operands

  // Loads in two trips to memory: the sequence and page ids; query rows, scales,
  // K and V.  The query operands are prepared by all the waves, some k
  // steps of one tile each, while the first K and V are under way.
  constexpr int PREP = NT * KS > W ? NT * KS / W : 1;  // operands per wave
  const int pu = wave * PREP / KS, pj = wave * PREP % KS;
  const bool prepares = wave * PREP < NT * KS;
  float x[D / 4];
  if (prepares) {
    const int r = row_lo + 16 * pu + nr;
    // (a row past the last reads the sequence's first, for zeros)
    uint32_t rem;
    const int i = (int)a.by_g.divmod(r < rows ? r : 0, rem);
    load_query<D>(a, a.q + (int64_t)(sv.row0 + i) * a.ldq + (int64_t)(h * G + rem) * D, g, x);
  }
  auto prepare_q = [&]() {
    const bool live = row_lo + 16 * pu + nr < rows;
#pragma unroll
    for (int j = 0; j < D / 4; ++j) x[j] = live ? x[j] : 0.0f;
    const QueryScale f = query_scale<D>(a.scale, x);
    if (g == 0 && pj == 0) qfac[16 * pu + n] = f.factor;
#pragma unroll
    for (int i = 0; i < PREP; ++i) {
      f16x8 qh, ql;
      float part[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        part[e] = x[8 * i + e];
#pragma unroll
        for (int j = 1; j < KS / PREP; ++j) part[e] = pj == j * PREP ? x[8 * (j * PREP + i) + e] : part[e];
      }
      split_query(part, f.up, qh, ql);
      if constexpr (PACK) {
        sh.q[pu][pj + i][0][lane] = low ? ql : qh;
      } else {
        sh.q[pu][pj + i][0][lane] = qh;
        sh.q[pu][pj + i][1][lane] = ql;
      }
    }
  };
  int32_t pos[NT];  // last position that the row sees (-1: none)
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int r = row_lo + 16 * u + nr;
    pos[u] = r < rows ? (int32_t)max(min(sv.pos0 + (int)a.by_g.div(r), sv.len - 1), (int64_t)-1) : -1;
  }

  f32x4 o[NT][DT];
  float l[NT];
  RowUnits units[NT];
  Far far = {base[wave], false};
  if ((int)threadIdx.x < W * 16 * NT) base[0][threadIdx.x] = 0.0f;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    units[u] = {kNoUnit, kNoUnit};
    l[u] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[u][d] = {0.0f, 0.0f, 0.0f, 0.0f};
  }

  // position of the tile that every row sees: below it no mask is needed
  const int64_t all_see = min(sv.len, sv.pos0 + (int)a.by_g.div(row_lo) + 1);
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
    const int8_t* kp = kv.k + (base + (n & 3)) * D + 16 * g;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) kw[t][i] = load16(kp + 4 * t * D + 64 * i);
  };
  auto load_v = [&](int st) {
    const int gr = 4 * st + g;
    const int8_t* vp = kv.v + ((((int64_t)max(page[gr], 0) * kv.H + h) * D + n) << kv.log_p) +
                       (((int)w0 + 16 * gr) & (P - 1));
#pragma unroll
    for (int d = 0; d < DT; ++d) vw[d] = load16(vp + ((int64_t)(16 * d) << kv.log_p));
  };
  // The pages and scales of the window at w0, and its first loads; `meanwhile`
  // is done while those are on their way.
  auto open_window = [&](auto meanwhile) {
    const int64_t j = w0 + 16 * (int)threadIdx.x;
    const int32_t id = j < sv.len ? valid_page(kv, entry) : -1;
    const int64_t si = (int64_t)max(id, 0) * kv.H + h;
    const float ks = load_g(kv.k_scale + si), vs = load_g(kv.v_scale + si);
    page[threadIdx.x] = id;
    if (threadIdx.x == 0) again = 0;
    __syncthreads();
    steps = (int)((min(c1 - w0, (int64_t)kWindow) + kStep - 1) / kStep);
    if (wave < steps) {
      load_k(wave);
      load_v(wave);
    }
    meanwhile();
    // (this waits for K and V too: loads return in order, and not every wave has some)
    kscale[threadIdx.x] = id < 0 ? 0.0f : ks;
    vscale[threadIdx.x] = v_scale(id < 0 ? 0.0f : vs);
  };
  open_window([&]() {
    if (prepares) prepare_q();
  });
  __syncthreads();
  float fac[NT];
#pragma unroll
  for (int u = 0; u < NT; ++u) fac[u] = qfac[16 * u + n];
  int pass = 0;  // over the positions (see next_band)
  for (;;) {
    f32x4 sc[NT][4];
    auto scores = [&]() {
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) sc[u][t] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        f16x8 q[NT][2];
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int e = 0; e < (PACK ? 1 : 2); ++e) q[u][e] = sh.q[u][j][e][lane];
        // (the high halves first: no instruction waits for the one before it)
        f16x8 kf[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          kf[t] = codes_f16(kw[t][j / 2][2 * (j % 2)], kw[t][j / 2][2 * (j % 2) + 1]);
#pragma unroll
          for (int u = 0; u < NT; ++u) sc[u][t] = mfma(kf[t], q[u][0], sc[u][t]);
        }
        if constexpr (!PACK) {
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int u = 0; u < NT; ++u) sc[u][t] = mfma(kf[t], q[u][1], sc[u][t]);
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
      const float ks = kscale[4 * st + g];
      const VScale v = vscale[4 * st + g];
      const bool masked = j0 + kStep > all_see || __any(!here);
      f16x8 pb[NT][2][2];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        float f = fac[u] * ks;
        if (masked || far.any) mask_scores(sc[u], f, here ? pos[u] - jv : -1);
        f16x8 hi[2], lo[2];
        if (pass == 0) {
          const float e = row_units(sc[u], f, v, units[u], l[u], o[u], far, 16 * u + n);
          l[u] += row_weights(sc[u], f, v, e, units[u], hi, lo);
        } else {
          band_scores(sc[u], f, v, band[wave][16 * u + n], far.any ? far.base[16 * u + n] : 0.0f);
          row_weights(sc[u], f, v, v.e, units[u], hi, lo);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (PACK) {
            const u32x4 a4 = __builtin_bit_cast(u32x4, hi[k]), b4 = __builtin_bit_cast(u32x4, lo[k]);
            u32x4 c4;
#pragma unroll
            for (int i = 0; i < 4; ++i) c4[i] = low ? b4[i] : a4[i];
            hi[k] = __builtin_bit_cast(f16x8, c4);
          }
          pb[u][k][0] = hi[k];
          pb[u][k][1] = lo[k];
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int d0 = 0; d0 < DT; d0 += 4) {
          f16x8 vf[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            vf[d] = codes_f16(vw[d0 + d][2 * k], vw[d0 + d][2 * k + 1]);
#pragma unroll
            for (int u = 0; u < NT; ++u) o[u][d0 + d] = mfma(vf[d], pb[u][k][0], o[u][d0 + d]);
          }
          if constexpr (!PACK) {
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
              for (int u = 0; u < NT; ++u) o[u][d0 + d] = mfma(vf[d], pb[u][k][1], o[u][d0 + d]);
          }
        }
    };
    // (the last step apart: a load that may or may not have been issued would
    // have every step wait for all of them)
    int st = wave;
    for (; st + W < steps; st += W) {
      asm volatile("" ::: "memory");  // (the query operands stay in LDS: held in registers they cost a wave per SIMD)
      scores();
      load_k(st + W);
      weigh_and_sum(st);
      load_v(st + W);
    }
    if (st < steps) {
      scores();
      weigh_and_sum(st);
    }
    w0 += kWindow;
    if (w0 >= c1) {
      bool more = false;
#pragma unroll
      for (int u = 0; u < NT; ++u) more |= next_band<DT, PACK>(pass, pos[u] >= 0, units[u], o[u], band[wave][16 * u + n]);
      if (more) again = 1;
      __syncthreads();
      if (!again) break;
      ++pass;
      w0 = c0;
    }
    entry = page_entry(kv, s, (w0 + 16 * (int)threadIdx.x) >> kv.log_p);
    __syncthreads();  // (the window before has been read)
    open_window([]() {});
    __syncthreads();
  }

  // join the waves, a tile at a time
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    float m;
    const float lt = whole_sum(l[u], units[u], far, 16 * u + n, m);
    if (g == 0) sml[wave][16 * u + n][0] = m, sml[wave][16 * u + n][1] = lt;
  }
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    if (u) __syncthreads();  // (the tile before has been read)
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      f32x4 v = o[u][d];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (PACK) v[i] += other_half(v[i]);
        v[i] = __builtin_ldexpf(v[i], (int)(units[u].R - units[u].L));
      }
      *reinterpret_cast<f32x4*>(&sh.o[wave][n][16 * d + 4 * g]) = v;
    }
    __syncthreads();
    // four dims per thread and turn
    for (int i = threadIdx.x; i < (PACK ? 8 : 16) * (D / 4); i += 64 * W) {
      const int rr = i / (D / 4), d = 4 * (i % (D / 4)), r = 16 * u + rr;
      if (row_lo + r >= rows) break;
      float mm = kNegInf;
#pragma unroll
      for (int w = 0; w < W; ++w) mm = fmaxf(mm, sml[w][r][0]);
      float ls = 0.0f;
      f32x4 os = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = sml[w][r][0] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(sml[w][r][0] - mm);
        ls = __builtin_fmaf(sml[w][r][1], f, ls);
        os += *reinterpret_cast<const f32x4*>(&sh.o[w][rr][d]) * f;
      }
      uint32_t rem;
      const int64_t row = sv.row0 + a.by_g.divmod(row_lo + r, rem), hq = h * G + rem;
      if (a.nchunk == 1) {
        float* y = a.y + row * a.ldy + hq * D + d;
        os *= ls == 0.0f ? 0.0f : 1.0f / ls;
        if (a.y16) {
          store_g(reinterpret_cast<f32x4*>(y), os);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) store_g(y + e, os[e]);
        }
      } else {
        const int64_t at = (row * a.Hq + hq) * a.nchunk + c;
        store_g(reinterpret_cast<f32x4*>(a.part + at * D + d), os);
        if (d == 0) {
          store_g(a.part_ml + 2 * at, mm);
          store_g(a.part_ml + 2 * at + 1, ls);
        }
      }
    }
  }
}

// Prompts: a workgroup of four waves takes 128 rows, a wave 32 of them over
// all positions.  Each step's 64 positions are converted to fp16 once, by all
// the waves, into one of two LDS buffers, laid out as the products read them
// (16 bytes per lane, a whole kilobyte per instruction), so a wave's 32 rows
// cost a quarter of the conversions.  Operand n of lane group g is in slot
// 16 g + (n ^ swizzle(g)): writes run over g and the low bits of n, reads
// over n, and 16-byte accesses are served sixteen lanes at a time as 0-3,
// 12-15, 20-27 and so on; these four constants keep both off each other's
// banks (4 g had half of the read cycles lost to conflicts).  The codes of the
// step after the next are on their way to registers meanwhile.  Two
// workgroups per CU: one's matrix instructions run beside the other's
// exponentials.  Bound by matrix and vector instructions, which add up: four
// products (two halves each of Q and P) where 16-bit attention takes two keep
// the matrix cores busy 53 % of the time, exponentials and conversions the
// rest.  2 x 2,048 tokens on 4,096 positions, 32 heads: 237 to 257 us on
// different cards, up to 570 TFLOP/s of the definition's products, 1,140 of
// those done (a library product of 8,192^3 in bf16: 1,250); 900 us where a
// position of value 0 takes the weight of every row (next_band).
template <int D>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_prompt_kernel(AttnArgs a) {
  constexpr int KS = D / 32, DT = D / 16, NT = 2, W = kWaves, ROWS = 16 * NT * W;
  constexpr int kGroups = 64 * W, kWindow = 16 * kGroups;
  constexpr int NP = D / 64;  // 16-code pieces of K, and of V, per thread
  __shared__ f16x8 kf[2][4][KS][64];
  __shared__ f16x8 vf[2][DT][2][64];
  __shared__ int32_t page[kGroups];
  __shared__ float kscale[kGroups];
  __shared__ VScale vscale[kGroups];
  __shared__ Band band[ROWS];
  __shared__ float base[ROWS];
  __shared__ int again;  // some row needs another pass

  const KvArgs& kv = a.kv;
  uint32_t h, cu, tile;
  const int s = (int)a.by_tiles.divmod(a.by_chunks.divmod(a.by_h.divmod(blockIdx.x, h), cu), tile);
  const int c = (int)cu, G = (int)a.by_g.d;
  const int rt = a.row_tiles - 1 - (int)tile;  // (the longest first)
  const SeqView sv = seq_view(kv, s);
  const int rows = min(sv.n, (int)kv.max_new) * G, row_lo = rt * ROWS;
  if (row_lo >= rows) return;
  const int64_t last_pos = sv.pos0 + (int)a.by_g.div(min(row_lo + ROWS - 1, rows - 1));
  const int64_t end = min(sv.len, last_pos + 1);
  const int64_t c0 = (int64_t)c * a.chunk;
  const int64_t c1 = c == a.nchunk - 1 ? end : min(end, c0 + a.chunk);
  if (c0 >= c1 && c > 0) return;

  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int slot = 16 * g + (n ^ swizzle(g));

  // (of two workgroups on a CU the second's waves go first: out of step, one's
  // products fill the other's exponentials; 261 -> 249 us)
  if ((blockIdx.x >> 8) & 1) __builtin_amdgcn_s_setprio(1);

  f16x8 qh[NT][KS], ql[NT][KS];
  float qfac[NT];
  int32_t pos[NT];
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int r = row_lo + 16 * (NT * wave + u) + n;
    const bool live = r < rows;
    uint32_t rem;
    const int i = (int)a.by_g.divmod(live ? r : 0, rem);
    pos[u] = live ? (int32_t)max(min(sv.pos0 + i, sv.len - 1), (int64_t)-1) : -1;
    float x[D / 4];
    load_query<D>(a, a.q + (int64_t)(sv.row0 + i) * a.ldq + (int64_t)(h * G + rem) * D, g, x);
#pragma unroll
    for (int j = 0; j < D / 4; ++j) x[j] = live ? x[j] : 0.0f;
    const QueryScale f = query_scale<D>(a.scale, x);
    qfac[u] = f.factor;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      float part[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) part[e] = x[8 * j + e];
      split_query(part, f.up, qh[u][j], ql[u][j]);
    }
  }

  f32x4 o[NT][DT];
  float l[NT];
  RowUnits units[NT];
  Far far = {base + 16 * NT * wave, false};
  if (t < ROWS) base[t] = 0.0f;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    units[u] = {kNoUnit, kNoUnit};
    l[u] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[u][d] = {0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int64_t all_see = min(sv.len, sv.pos0 + (int)a.by_g.div(row_lo + 16 * NT * wave) + 1);
  const int P = 1 << kv.log_p;

  // A thread's pieces of a step: K piece e is 16 dims (g' + 4 i) of position
  // 16 grp + r; V piece e is the 16 positions of group g' of one dim.  g'
  // and the low bits of the position or dim are the lane's lowest bits.
  const int pg = t & 3;
  u32x4 kraw[NP], vraw[NP];
  int64_t w0 = c0;
  auto k_piece = [&](int e, int& tok, int& i) {
    const int id = (t >> 2) + 64 * e;  // position, then the 64 dims
    tok = id & 63, i = id >> 6;
  };
  auto load_codes = [&](int st) {
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      int tok, i;
      k_piece(e, tok, i);
      const int gr = 4 * st + (tok >> 4);
      const int64_t base = (((int64_t)max(page[gr], 0) * kv.H + h) << kv.log_p) + (((int)w0 + kStep * st + tok) & (P - 1));
      kraw[e] = load16(kv.k + base * D + 64 * i + 16 * pg);
      const int d = (t >> 2) + 64 * e, gv = 4 * st + pg;
      vraw[e] = load16(kv.v + ((((int64_t)max(page[gv], 0) * kv.H + h) * D + d) << kv.log_p) +
                       (((int)w0 + 16 * gv) & (P - 1)));
    }
  };
  auto write_codes = [&](int buf) {
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      int tok, i;
      k_piece(e, tok, i);
      const int r = tok & 15, kn = 4 * (tok >> 4) + (r & 3);
      const int at = 16 * pg + (kn ^ swizzle(pg));
      kf[buf][r >> 2][2 * i][at] = codes_f16(kraw[e][0], kraw[e][1]);
      kf[buf][r >> 2][2 * i + 1][at] = codes_f16(kraw[e][2], kraw[e][3]);
      const int d = (t >> 2) + 64 * e;
      const int vt = 16 * pg + ((d & 15) ^ swizzle(pg));
      vf[buf][d >> 4][0][vt] = codes_f16(vraw[e][0], vraw[e][1]);
      vf[buf][d >> 4][1][vt] = codes_f16(vraw[e][2], vraw[e][3]);
    }
  };

  int pass = 0;  // over the positions (see next_band)
  while (w0 < c1) {
    {
      const int64_t j = w0 + 16 * t;
      const int32_t id = j < sv.len ? page_of(kv, s, j >> kv.log_p) : -1;
      const int64_t si = (int64_t)max(id, 0) * kv.H + h;
      const float ks = load_g(kv.k_scale + si), vs = load_g(kv.v_scale + si);
      __syncthreads();  // (the window before has been read)
      page[t] = id;
      if (t == 0) again = 0;
      kscale[t] = id < 0 ? 0.0f : ks;
      vscale[t] = v_scale(id < 0 ? 0.0f : vs);
      __syncthreads();
    }
    const int steps = (int)((min(c1 - w0, (int64_t)kWindow) + kStep - 1) / kStep);
    load_codes(0);
    write_codes(0);
    load_codes(min(1, steps - 1));
    for (int st = 0; st < steps; ++st) {
      const int buf = st & 1;
      // this step's operands are written; every wave is past the step before,
      // whose buffer the next step's go to
      __syncthreads();
      const int64_t j0 = w0 + kStep * st;
      const int32_t jv = (int32_t)j0 + 16 * g;
      const bool here = page[4 * st + g] >= 0;
      const float ks = kscale[4 * st + g];
      const VScale v = vscale[4 * st + g];
      const bool masked = j0 + kStep > all_see || __any(!here);
      f32x4 sc[NT][4];
      f16x8 hi[NT][2], lo[NT][2];
      // Both products: the next four operands are read while the matrix
      // instructions of these four run (sixteen; the high halves first, so
      // that none waits for the one before it).
      f16x8 fr[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) fr[0][e] = kf[buf][e][0][slot];
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[u][e] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        if (j + 1 < KS) {
#pragma unroll
          for (int e = 0; e < 4; ++e) fr[(j + 1) & 1][e] = kf[buf][e][j + 1][slot];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int u = 0; u < NT; ++u) sc[u][e] = mfma(fr[j & 1][e], qh[u][j], sc[u][e]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int u = 0; u < NT; ++u) sc[u][e] = mfma(fr[j & 1][e], ql[u][j], sc[u][e]);
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 16, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      // (after the last step: codes that no one reads)
      write_codes(buf ^ 1);
      load_codes(min(st + 2, steps - 1));
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        float f = qfac[u] * ks;
        if (masked || far.any) mask_scores(sc[u], f, here ? pos[u] - jv : -1);
        if (pass == 0) {
          const float e = row_units(sc[u], f, v, units[u], l[u], o[u], far, 16 * u + n);
          l[u] += row_weights(sc[u], f, v, e, units[u], hi[u], lo[u]);
        } else {
          band_scores(sc[u], f, v, band[16 * (NT * wave + u) + n], far.any ? far.base[16 * u + n] : 0.0f);
          row_weights(sc[u], f, v, v.e, units[u], hi[u], lo[u]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) fr[0][e] = vf[buf][e][0][slot];
#pragma unroll
      for (int x = 0; x < DT / 2; ++x) {  // four dims' tiles of one half of the positions
        const int k = x / (DT / 4), d0 = 4 * (x % (DT / 4));
        if (x + 1 < DT / 2) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            fr[(x + 1) & 1][e] = vf[buf][4 * ((x + 1) % (DT / 4)) + e][(x + 1) / (DT / 4)][slot];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int u = 0; u < NT; ++u) o[u][d0 + e] = mfma(fr[x & 1][e], hi[u][k], o[u][d0 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int u = 0; u < NT; ++u) o[u][d0 + e] = mfma(fr[x & 1][e], lo[u][k], o[u][d0 + e]);
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 1);
        __builtin_amdgcn_sched_group_barrier(0x008, 16, 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    w0 += kWindow;
    if (w0 >= c1) {
      bool more = false;
#pragma unroll
      for (int u = 0; u < NT; ++u) more |= next_band<DT, false>(pass, pos[u] >= 0, units[u], o[u], band[16 * (NT * wave + u) + n]);
      if (more) again = 1;
      __syncthreads();
      if (!again) break;
      ++pass;
      w0 = c0;
    }
  }

#pragma unroll
  for (int u = 0; u < NT; ++u) {
    float m;
    const float lt = whole_sum(l[u], units[u], far, 16 * u + n, m);
    const int r = row_lo + 16 * (NT * wave + u) + n;
    if (r >= rows) continue;
    uint32_t rem;
    const int64_t row = sv.row0 + a.by_g.divmod(r, rem), hq = h * G + rem;
    const int64_t at = (row * a.Hq + hq) * a.nchunk + c;
    const bool whole = a.nchunk == 1;
    const float f = whole ? (lt == 0.0f ? 0.0f : 1.0f / lt) : 1.0f;
    const int back = (int)(units[u].R - units[u].L);
    float* out = whole ? a.y + row * a.ldy + hq * D : a.part + at * D;
    if (!whole && g == 0) {
      store_g(a.part_ml + 2 * at, m);
      store_g(a.part_ml + 2 * at + 1, lt);
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      f32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __builtin_ldexpf(o[u][d][i] * f, back);
      if (a.y16 || !whole) {
        store_g(reinterpret_cast<f32x4*>(out + 16 * d + 4 * g), v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) store_g(out + 16 * d + 4 * g + i, v[i]);
      }
    }
  }
}

// Joins the chunks of each (row, query head): a workgroup of four waves each,
// wave w the chunks w, w + 4, ...  Two trips to memory: 3.9 us with its launch
// (32 heads of 17 chunks), 4.7 for 256 of 26.
template <int D>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_join_kernel(AttnArgs a) {
  __shared__ float so[kJoinWaves][D], sml[kJoinWaves][2];
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
  // (the first sums are asked for with their maxima; 0 where there is none)
  constexpr int kAhead = 8;
  float ahead[kAhead][D / 64];
#pragma unroll
  for (int e = 0; e < kAhead; ++e)
#pragma unroll
    for (int d = 0; d < D / 64; ++d)
      ahead[e][d] = wave + kJoinWaves * e < nc ? load_g(a.part + (at + wave + kJoinWaves * e) * D + lane + 64 * d) : 0.0f;
  for (int b = wave; b < nc; b += 64 * kJoinWaves) {
    const int c = b + kJoinWaves * lane;
    const float mc = c < nc ? load_g(a.part_ml + 2 * (at + c)) : kNegInf;
    const float lc = c < nc ? load_g(a.part_ml + 2 * (at + c) + 1) : 0.0f;
    float mn = mc;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) mn = fmaxf(mn, __shfl_xor(mn, d, 64));
    mn = fmaxf(mn, m);
    const float from = mn == kNegInf ? 0.0f : mn;  // (nothing seen yet: factors of 0)
    const float al = __builtin_amdgcn_exp2f(m - from), f = __builtin_amdgcn_exp2f(mc - from);
    m = mn;
    float ls = lc * f;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) ls += __shfl_xor(ls, d, 64);
    l = __builtin_fmaf(l, al, ls);
#pragma unroll
    for (int d = 0; d < D / 64; ++d) o[d] *= al;
    auto add = [&](int e, auto value) {
      const float fe = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), e));
#pragma unroll
      for (int d = 0; d < D / 64; ++d) o[d] = __builtin_fmaf(value(d), fe, o[d]);
    };
    const int cn = min(64, (nc - b + kJoinWaves - 1) / kJoinWaves);
    if (b == wave) {
#pragma unroll
      for (int e = 0; e < kAhead; ++e) add(e, [&](int d) { return ahead[e][d]; });
    }
#pragma unroll 4
    for (int e = b == wave ? kAhead : 0; e < cn; ++e)
      add(e, [&](int d) { return load_g(a.part + (at + b + kJoinWaves * e) * D + lane + 64 * d); });
  }
  if (lane == 0) sml[wave][0] = m, sml[wave][1] = l;
#pragma unroll
  for (int d = 0; d < D / 64; ++d) so[wave][lane + 64 * d] = o[d];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 64 * kJoinWaves) {
    float mm = kNegInf, ls = 0.0f, os = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) mm = fmaxf(mm, sml[w][0]);
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) {
      const float f = sml[w][0] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(sml[w][0] - mm);
      ls = __builtin_fmaf(sml[w][1], f, ls);
      os = __builtin_fmaf(so[w][d], f, os);
    }
    store_g(a.y + row * a.ldy + (int64_t)hq * D + d, ls == 0.0f ? 0.0f : os / ls);
  }
}

int attn_rows(AttnKind k) { return k == ATTN_PACKED ? 8 : k == ATTN_16 ? 16 : k == ATTN_32 ? 32 : 128; }

// Which kernel, by a sequence's rows per KV head.  Up to 32 the smallest tile
// that holds them (32 ragged contexts to 4,096, 8 KV heads: 8 rows 38.1 us
// packed, 38.7 by 16; 16 rows 39.6 by 16, 48.3 by 32, 45.4 by two of 8; 32 rows
// 50.1 by 32, 57.7 by two of 16; eight of 2,048, 24 rows: 18.3 by 32, 19.1 by 16).
// Beyond 128 the prompt kernel pays once it has its two workgroups on every CU
// (8 x 1,024 tokens from nothing: 176 us, 263 by 32; 4 x 512 on 4,096 226 and 266),
// the contexts are so long that they can be split for that (1,024 on 32,768:
// 889, 1,015), or they are so short that starting counts (8 x 128: 17.5, 24.5).
// Else tiles of 32 spread better (512 on 4,096: 76, 96; 4 x 256 on 4,096: 144,
// 149; up to 128 rows always: 8 x 32 on 2,048 30, 47).
AttnKind attn_kind(int64_t rows, int64_t groups, int64_t len, int cus) {
  if (rows <= 32) return rows <= 8 ? ATTN_PACKED : rows <= 16 ? ATTN_16 : ATTN_32;
  const int64_t units = mul_sat(groups, (rows + 127) / 128);
  const bool prompt = units >= 2 * cus || len > 16384 || (units >= cus && len <= 512);
  return rows > 128 && prompt ? ATTN_PROMPT : ATTN_32;
}

template <int D>
void launch_kind(AttnKind k, dim3 grid, dim3 block, const AttnArgs& a, hipStream_t s) {
  switch (k) {
    case ATTN_PACKED: hipLaunchKernelGGL((attn_kernel<D, 1, true>), grid, block, 0, s, a); break;
    case ATTN_16: hipLaunchKernelGGL((attn_kernel<D, 1, false>), grid, block, 0, s, a); break;
    case ATTN_32: hipLaunchKernelGGL((attn_kernel<D, 2, false>), grid, block, 0, s, a); break;
    case ATTN_PROMPT: hipLaunchKernelGGL((attn_prompt_kernel<D>), grid, block, 0, s, a); break;
  }
}

}  // namespace

AttnPlan attn_plan(const KvArgs& kv, int64_t Hq, int cus) {
  AttnPlan p;
  const int64_t G = Hq / kv.H, rows = kv.max_new * G;
  const int64_t most = kv.ld_table << kv.log_p;
  const int64_t len = kv.max_len > 0 ? std::min(kv.max_len, most) : most;
  p.kind = attn_kind(rows, kv.S * kv.H, len, cus);
  const int64_t tile = attn_rows(p.kind);
  p.row_tiles = (rows + tile - 1) / tile;
  const int64_t units = mul_sat(kv.S * kv.H, p.row_tiles);
  // Pieces of a context.  Together one workgroup per CU: a second round of
  // workgroups, each two trips to memory before its first product, costs more
  // than it evens out (32 ragged contexts to 4,096: whole 36 us, halves 41,
  // quarters 45; 16 to 2,048 in 1, 2, 4, 8 pieces: 18.7, 17.5, 17.6, 20.2), and
  // more than 64 pieces cost more to join (one KV head, 32,768 positions: 64
  // pieces 15.2 us, 128 17.4).  Two per CU where products count: prompts (1,024
  // rows on 32,768: 242 to 265 us, 303 with one), 32 rows and more on long contexts
  // (256 rows on 32,768: 79 in 32 pieces, 157 in 8), if that is at most 32 pieces
  // (32 rows: 25.5 in 32, 28.1 in 64).
  const bool two = p.kind == ATTN_PROMPT || (p.kind == ATTN_32 && len > 4096);
  int64_t want = cus / units;
  if (two && 2 * cus / units <= 32) want = 2 * cus / units;
  // Short ones whole, without the joining launch (512 positions: 9.4 us whole, 11.8
  // in two; 1,024 with a workgroup on half of the CUs 12.9, 15.6).
  if (len <= 512 || (len <= 1024 && units >= cus / 2) || (len <= 4096 && units >= cus)) want = 1;
  want = std::min<int64_t>(std::max<int64_t>(want, 1), 64);
  int64_t chunk = (len + want - 1) / want;
  // A batch of long contexts of single tokens is taken to be ragged, and cut finer
  // to even it out (lengths up to 8,192 over 48 sequences: 77 us, 102 whole; to
  // 16,384 over 32: 116, 131; where all are as long as the longest that costs a
  // little: 147.7, 147.3 and 187, 180).  With more rows the pieces' starts cost more
  // than that (8 x 64 rows on 8,192 each: 56 us in 4, 67 in 7).
  if (kv.S > 1 && rows <= 16 && len > 4096 && units < 4 * cus) chunk = std::min(chunk, std::max<int64_t>(1280, len / 8));
  const int64_t step = kStep * kWaves;
  chunk = std::max<int64_t>(step, (chunk + step - 1) / step * step);
  p.chunk = std::min<int64_t>(chunk, 1ll << 30);
  p.nchunk = std::max<int64_t>(1, (len + p.chunk - 1) / p.chunk);
  p.work_items = mul_sat(mul_sat(units, p.nchunk), 64 * kWaves);
  p.join_items = p.nchunk > 1 ? mul_sat(mul_sat(kv.S * kv.max_new, Hq), 64 * kJoinWaves) : 0;
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
  a.by_h = fast_div(kv.H);
  a.by_chunks = fast_div(p.nchunk);
  a.by_tiles = fast_div(p.row_tiles);
  a.by_g = fast_div(Hq / kv.H);
  a.chunk = (int32_t)p.chunk;
  a.nchunk = (int32_t)p.nchunk;
  a.row_tiles = (int32_t)p.row_tiles;
  a.scale = scale;
  auto rows16 = [&](const float* p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (kv.rows == 1 || ld % 4 == 0);
  };
  a.q16 = rows16(q, ldq);
  a.y16 = rows16(y, ldy);
  const dim3 grid((unsigned)(p.work_items / (64 * kWaves))), block(64 * kWaves), jblock(64 * kJoinWaves);
  if (kv.D == 64)
    launch_kind<64>(p.kind, grid, block, a, s);
  else
    launch_kind<128>(p.kind, grid, block, a, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.nchunk == 1) return e;
  const dim3 jgrid((unsigned)(p.join_items / jblock.x));
  if (kv.D == 64) hipLaunchKernelGGL((attn_join_kernel<64>), jgrid, jblock, 0, s, a);
  else hipLaunchKernelGGL((attn_join_kernel<128>), jgrid, jblock, 0, s, a);
  return hipGetLastError();
}

}  // namespace tern
