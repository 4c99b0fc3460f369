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
// 2^19 tokens sum to at most 2^63.
//
// Nothing is sorted but a few tokens around the cut.  A row is split in
// chunks, one workgroup each, and goes through up to four launches:
//   1. the largest logit and the number of live tokens of each chunk;
//   2. (rows with top-k or top-p) a histogram of the row, counts and weights
//      in bins of 3/64 of log2-probability below the maximum;
//   3. from the histogram every workgroup finds the bins that the cuts fall
//      in, lists the tokens of those bins, and sums the weight that its chunk
//      holds in the bins above;
//   4. one workgroup per row orders the listed tokens, fixes the cut exactly,
//      finds the chunk that the random number falls in, and walks that chunk.
// A row whose cut bins hold more than kListMax tokens is cut by the bits of its
// keys instead, by that one workgroup in up to ten passes over the row
// (slow_cut).  Many equal logits do that, and so do many close ones: a bin is
// 0.0325 T wide, so 151,936 normal logits of deviation 1.5 at T = 2 put 2,300 in
// the bin where top-p 0.9 ends, and where top-k splits a bin top-p may end in
// several.  Rows of 151,936 like that take 0.6 to 1.0 ms alone and 0.3 to 0.6 in
// batches of 8 and 96 (1,024 threads a row against 256), rows of equal logits
// 0.7 to 1.5.
//
// Times of the launches for 151,936 tokens: one row with top-k and top-p 2.9 +
// 8.2 + 5.6 + 7.9 us, each a launch and one or two trips to memory, bins and
// scans between barriers; 96 rows of mixed filters 12.4 + 22 + 20 + 17 us.  There
// the maxima run at 4.7 TB/s, and so would the histogram without its weights:
// those, some seventeen fp64 instructions a token, take 10 of its 22 us (its
// additions in LDS 2).  Not better: the steps below the maximum in fp32 with
// the rounding made up for in the series (1 us more), a series of twelve terms
// in place of the table (5 us more), tiles of 32 tokens a thread, the next tile
// ahead.
#include "tern.h"
#include "tern_device.h"

namespace tern {

namespace {

typedef unsigned long long u64;

constexpr int kT = 256;          // threads of launches 1 to 3
// Threads of launch 4.  Few rows, short chunks: one wave per SIMD, since the
// launch is a chain of short steps between barriers and four waves per SIMD
// take turns at each of them (one row: 10.0 us with 1,024 threads, 7.3 with
// 256).  Many rows, long chunks: the walk through a chunk and the ordering of
// a long list want more.
constexpr int kFinishFew = 256, kFinishMany = 1024;
constexpr int kBins = 1024;      // of 3 steps of 2^(-1/64) each; the last one holds all that is further below
constexpr uint32_t kListMax = 2048;
constexpr uint32_t kMine = kListMax;  // those that one chunk lists
constexpr int kChunkMin = 4 * kT;
constexpr int kChunkMax = 16384;
constexpr int kChunksMax = TERN_SAMPLE_MAX_N / kChunkMin;
constexpr double kFix = 17592186044416.0;  // 2^44
static_assert((kBins - 1) * 3 / 64.0 - 1 / 128.0 > 47, "the last bin's weights round to 0: 2^44 2^-47 < 1/2");

// 2^(-j / 64)
__constant__ double kExp2[64] = {
    0x1.0000000000000p+0, 0x1.fa7c1819e90d8p-1, 0x1.f50765b6e4540p-1, 0x1.efa1bee615a27p-1,
    0x1.ea4afa2a490dap-1, 0x1.e502ee78b3ff6p-1, 0x1.dfc97337b9b5fp-1, 0x1.da9e603db3285p-1,
    0x1.d5818dcfba487p-1, 0x1.d072d4a07897cp-1, 0x1.cb720dcef9069p-1, 0x1.c67f12e57d14bp-1,
    0x1.c199bdd85529cp-1, 0x1.bcc1e904bc1d2p-1, 0x1.b7f76f2fb5e47p-1, 0x1.b33a2b84f15fbp-1,
    0x1.ae89f995ad3adp-1, 0x1.a9e6b5579fdbfp-1, 0x1.a5503b23e255dp-1, 0x1.a0c667b5de565p-1,
    0x1.9c49182a3f090p-1, 0x1.97d829fde4e50p-1, 0x1.93737b0cdc5e5p-1, 0x1.8f1ae99157736p-1,
    0x1.8ace5422aa0dbp-1, 0x1.868d99b4492edp-1, 0x1.82589994cce13p-1, 0x1.7e2f336cf4e62p-1,
    0x1.7a11473eb0187p-1, 0x1.75feb564267c9p-1, 0x1.71f75e8ec5f74p-1, 0x1.6dfb23c651a2fp-1,
    0x1.6a09e667f3bcdp-1, 0x1.6623882552225p-1, 0x1.6247eb03a5585p-1, 0x1.5e76f15ad2148p-1,
    0x1.5ab07dd485429p-1, 0x1.56f4736b527dap-1, 0x1.5342b569d4f82p-1, 0x1.4f9b2769d2ca7p-1,
    0x1.4bfdad5362a27p-1, 0x1.486a2b5c13cd0p-1, 0x1.44e086061892dp-1, 0x1.4160a21f72e2ap-1,
    0x1.3dea64c123422p-1, 0x1.3a7db34e59ff7p-1, 0x1.371a7373aa9cbp-1, 0x1.33c08b26416ffp-1,
    0x1.306fe0a31b715p-1, 0x1.2d285a6e4030bp-1, 0x1.29e9df51fdee1p-1, 0x1.26b4565e27cddp-1,
    0x1.2387a6e756238p-1, 0x1.2063b88628cd6p-1, 0x1.1d4873168b9aap-1, 0x1.1a35beb6fcb75p-1,
    0x1.172b83c7d517bp-1, 0x1.1429aaea92de0p-1, 0x1.11301d0125b51p-1, 0x1.0e3ec32d3d1a2p-1,
    0x1.0b5586cf9890fp-1, 0x1.0874518759bc8p-1, 0x1.059b0d3158574p-1, 0x1.02c9a3e778061p-1};

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

// A row's place in the workspace: its histogram, list and chunks.
struct RowWs {
  u64* mass;        // kBins
  u64* list;        // kListMax: key, complement of the index
  u64* chunk_top;   // key, complement of the index, of a chunk's largest logit
  u64* chunk_mass;  // weight that a chunk holds above the cut bins, and its tokens
  uint32_t* count;  // kBins
  uint32_t* chunk_live;
  uint32_t* chunk_kept;
  uint32_t* list_n;
};

struct Launch {
  SampleArgs a;
  uint8_t* ws;
  int64_t row_bytes;
  int32_t per, chunks;  // tokens per chunk
  bool vec;             // rows are 16-byte aligned
};

__host__ __device__ inline int64_t row_ws_bytes(int64_t chunks) {
  return ((kBins + kListMax) * 8 + chunks * 16 + kBins * 4 + chunks * 8 + 4 + 255) / 256 * 256;
}

__device__ __forceinline__ RowWs row_ws(const Launch& L, int64_t row) {
  uint8_t* p = L.ws + row * L.row_bytes;
  RowWs w;
  w.mass = reinterpret_cast<u64*>(p);
  w.list = w.mass + kBins;
  w.chunk_top = w.list + kListMax;
  w.chunk_mass = w.chunk_top + L.chunks;
  w.count = reinterpret_cast<uint32_t*>(w.chunk_mass + L.chunks);
  w.chunk_live = w.count + kBins;
  w.chunk_kept = w.chunk_live + L.chunks;
  w.list_n = w.chunk_kept + L.chunks;
  return w;
}

struct Row {
  const float* x;
  double inv_t, top_p, min_p;
  u64 top;        // key and complement of the index of the first token (0: none)
  uint32_t live;  // tokens that can be drawn
  uint32_t k;     // tokens of top-k (live: no limit)
  float mx, u;
  bool greedy;
};

// v of the lane that the DPP control names (0 where there is none, or where
// the row mask leaves it out).
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 dpp64(u64 v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
  return ((u64)hi << 32) | lo;
}
// Inclusive prefix over 16 lanes (row_shr 1, 2, 4, 8), and over the wave
// (row_bcast 15 and 31 after that).
__device__ __forceinline__ u64 row_scan(u64 v) {
  v += dpp64<0x111, 0xF>(v);
  v += dpp64<0x112, 0xF>(v);
  v += dpp64<0x114, 0xF>(v);
  return v + dpp64<0x118, 0xF>(v);
}
__device__ __forceinline__ u64 wave_scan(u64 v) {
  v = row_scan(v);
  v += dpp64<0x142, 0xA>(v);
  return v + dpp64<0x143, 0xC>(v);
}
__device__ __forceinline__ u64 lane64(u64 v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return ((u64)hi << 32) | lo;
}

// Exclusive prefixes over the workgroup of a and b (thread order), and their
// totals; `wave` holds 32 words.  Every wave scans the waves' totals itself,
// one per lane: read one after the other by all the threads, they had cost
// most of the scan.
template <int T>
__device__ __forceinline__ void wg_scan2(u64& a, u64& b, u64* wave, u64& ta, u64& tb) {
  constexpr int W = T / 64;
  static_assert(W <= 16, "the waves' totals fit a DPP row");
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const u64 sa = wave_scan(a), sb = wave_scan(b);
  __syncthreads();  // (the words' last readers are past them)
  if (lane == 63) wave[w] = sa, wave[16 + w] = sb;
  __syncthreads();
  const u64 va = row_scan(lane < W ? wave[lane] : 0), vb = row_scan(lane < W ? wave[16 + lane] : 0);
  ta = lane64(va, W - 1);
  tb = lane64(vb, W - 1);
  a = sa - a + (w ? lane64(va, w - 1) : 0);
  b = sb - b + (w ? lane64(vb, w - 1) : 0);
}
template <int T>
__device__ __forceinline__ u64 wg_scan(u64 v, u64* wave, u64& total) {
  u64 none = 0, none_total;
  wg_scan2<T>(v, none, wave, total, none_total);
  return v;
}

// The row's parameters, its largest logit and live tokens from the chunks of
// launch 1 (the same on every thread; `lds` holds 32 words).
template <int T>
__device__ Row load_row(const Launch& L, const RowWs& w, int64_t row, u64* lds) {
  const SampleArgs& a = L.a;
  // (every load before the first barrier: one trip to memory)
  const float t = load_g(a.temperature + row), u = load_g(a.u + row);
  const int32_t k = a.top_k ? load_g(a.top_k + row) : 0;
  const float tp = a.top_p ? load_g(a.top_p + row) : 1.0f, mp = a.min_p ? load_g(a.min_p + row) : 0.0f;
  u64 top = 0;
  uint32_t live = 0;
  for (int c = threadIdx.x; c < L.chunks; c += T) {
    const u64 v = load_g(w.chunk_top + c);
    live += load_g(w.chunk_live + c);
    top = v > top ? v : top;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const u64 o = __shfl_xor(top, d, 64);
    top = o > top ? o : top;
    live += __shfl_xor(live, d, 64);
  }
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = top, lds[16 + (threadIdx.x >> 6)] = live;
  __syncthreads();
  const int lane = threadIdx.x & 63;
  top = lane < T / 64 ? lds[lane] : 0;
  live = lane < T / 64 ? (uint32_t)lds[16 + lane] : 0;
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) {
    const u64 o = __shfl_xor(top, d, 64);
    top = o > top ? o : top;
    live += __shfl_xor(live, d, 64);
  }
  top = lane64(top, 0);
  live = (uint32_t)__builtin_amdgcn_readlane((int)live, 0);
  Row r;
  r.x = a.x + row * a.ldx;
  r.top = top;
  r.live = live;
  r.mx = key_logit((uint32_t)(top >> 32));
  r.greedy = !(t > 0.0f);
  r.inv_t = 1.0 / (double)t;
  r.u = u;
  r.k = k > 0 && (uint32_t)k < live ? (uint32_t)k : live;
  r.top_p = tp < 1.0f ? (double)fmaxf(tp, 0.0f) : 1.0;  // (a NaN is no filter)
  r.min_p = mp > 0.0f ? (double)fminf(mp, 1.0f) : 0.0;
  return r;
}

// With v = (max - x) / T in fp64: k = rint(v 64 / ln 2), s = k ln 2 / 64 - v;
// k is monotone in x and gives the bin (three of its steps each).
struct Reduced {
  double s;
  int k;
};
constexpr int kLastStep = 3 * (kBins - 1);
__device__ __forceinline__ Reduced reduce(const Row& r, float x) {
  constexpr double kStep = 0x1.62e42fefa39efp-7, kPerUnit = 0x1.71547652b82fep+6;  // ln 2 / 64 and its inverse
  // (equal also where both are +inf; a NaN, from T = inf, counts as far below)
  const double v = x == r.mx ? 0.0 : fmin(((double)r.mx - (double)x) * r.inv_t, 700.0);
  const double k = __builtin_rint(v * kPerUnit);
  return {__builtin_fma(k, kStep, -v), (int)k};
}
__device__ __forceinline__ int bin_of(const Reduced& d) { return (int)((uint32_t)min(d.k, kLastStep) * 21846u >> 16); }
static_assert((kLastStep * 21846u >> 16) == kBins - 1 && ((kLastStep - 1) * 21846u >> 16) == kBins - 2, "k / 3");
// e^-v: the table's 2^(-(k % 64) / 64), the Taylor series of e^s through s^4
// (|s| <= 0.0055: its next term is 4e-14) and a power of two.
__device__ __forceinline__ double weight_of(const Reduced& d, const double* tab) {
  const double s = d.s;
  double p = 1.0 / 24.0;
  p = __builtin_fma(p, s, 1.0 / 6.0);
  p = __builtin_fma(p, s, 0.5);
  p = __builtin_fma(p, s, 1.0);
  p = __builtin_fma(p, s, 1.0);
  return __builtin_ldexp(p * tab[d.k & 63], -(d.k >> 6));
}
__device__ __forceinline__ double weight_of(const Row& r, const double* tab, float x) {
  return weight_of(reduce(r, x), tab);
}
// w in units of 2^-44, w <= 1: the mantissa of w 2^44 + 2^52
__device__ __forceinline__ u64 fixed(double w) {
  return __builtin_bit_cast(u64, __builtin_fma(w, kFix, 4503599627370496.0)) & 0xfffffffffffffull;
}

// U groups of four consecutive tokens per thread, all loaded at once: tokens
// j, ..., j + 4 T U - 1 of a row (-infinity, which no one counts, from j1 on).
template <int T, int U>
struct Tile {
  float v[U][4];
  __device__ __forceinline__ static int at(int j, int u) { return j + 4 * ((int)threadIdx.x + T * u); }
  __device__ __forceinline__ void load(const float* x, int j, int j1, bool vec) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = at(j, u);
      if (vec && k + 4 <= j1) {
        const f32x4 g = __builtin_bit_cast(f32x4, load16(x + k));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = g[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = k + i < j1 ? load_g(x + k + i) : -__builtin_inff();
      }
    }
  }
  // fn(index, logit) for each
  template <typename Fn>
  __device__ __forceinline__ void each(int j, Fn fn) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) fn(at(j, u) + i, v[u][i]);
  }
};

// fn(index, logit) for the tokens [j0, j1) of a row; the first tile is
// already loaded.
template <int T, int U, typename Fn>
__device__ __forceinline__ void each_token(Tile<T, U>& tile, const float* x, int j0, int j1, bool vec, Fn fn) {
  for (int j = j0; j < j1;) {
    tile.each(j, fn);
    j += 4 * T * U;
    if (j < j1) tile.load(x, j, j1, vec);
  }
}
template <int T, typename Fn>
__device__ __forceinline__ void each_token(const float* x, int j0, int j1, bool vec, Fn fn) {
  Tile<T, 1> tile;
  tile.load(x, j0, j1, vec);
  each_token<T, 1>(tile, x, j0, j1, vec, fn);
}

__device__ __forceinline__ u64 pack_token(uint32_t key, int j) { return ((u64)key << 32) | (uint32_t)~(uint32_t)j; }

// Units of weight that the forerunners of a token kept by top-p stay below:
// forerunners < top_p * total, at least one (the first token always).
__device__ __forceinline__ u64 mass_limit(double top_p, u64 total) {
  const double lim = top_p * (double)total;
  u64 n = (u64)lim;
  if ((double)n < lim) ++n;
  return n ? n : 1;
}

// ------------------------------------------------------ launch 1: maxima --

template <int U>
__global__ __launch_bounds__(kT) void top_kernel(Launch L) {
  __shared__ u64 tops[kT / 64];
  __shared__ uint32_t lives[kT / 64];
  const int c = blockIdx.x % L.chunks;
  const int64_t row = blockIdx.x / L.chunks;
  const RowWs w = row_ws(L, row);
  const float* x = L.a.x + row * L.a.ldx;
  const int j0 = c * L.per, j1 = (int)min((int64_t)(c + 1) * L.per, L.a.N);
  Tile<kT, U> tile;
  tile.load(x, j0, j1, L.vec);
  // the row's histogram and list start empty, its chunks clearing a share each
  for (int i = c * kT + threadIdx.x; i < kBins; i += L.chunks * kT) {
    store_g(w.mass + i, (u64)0);
    store_g(w.count + i, 0u);
  }
  if (c == 0 && threadIdx.x == 0) store_g(w.list_n, 0u);
  u64 top = 0;
  uint32_t live = 0;
  each_token<kT, U>(tile, x, j0, j1, L.vec, [&](int j, float x) {
    const uint32_t k = logit_key(x);
    if (!k) return;
    ++live;
    const u64 t = pack_token(k, j);
    top = t > top ? t : top;
  });
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const u64 o = __shfl_xor(top, d, 64);
    top = o > top ? o : top;
    live += __shfl_xor(live, d, 64);
  }
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top, lives[threadIdx.x >> 6] = live;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kT / 64; ++i) {
      top = tops[i] > top ? tops[i] : top;
      live += lives[i];
    }
    store_g(w.chunk_top + c, top);
    store_g(w.chunk_live + c, live);
  }
}

// --------------------------------------------------- launch 2: histogram --

__device__ __forceinline__ bool wants_bins(const Row& r) { return r.k < r.live || r.top_p < 1.0; }

// Two copies of the bins for long chunks, even and odd threads apart: a bulk of
// close logits has a wave's additions meet in few bins (96 rows of 151,936:
// 25 -> 22 us; chunks of one tile gain less than the second copy costs).
template <int U>
__global__ __launch_bounds__(kT) void histogram_kernel(Launch L) {
  constexpr int kCopies = U > 1 ? 2 : 1;
  __shared__ u64 mass[kCopies][kBins];
  __shared__ uint32_t count[kCopies][kBins];
  __shared__ double tab[64];
  __shared__ u64 red[32];
  const int c = blockIdx.x % L.chunks;
  const int64_t row = blockIdx.x / L.chunks;
  const RowWs w = row_ws(L, row);
  const int j0 = c * L.per, j1 = (int)min((int64_t)(c + 1) * L.per, L.a.N);
  Tile<kT, U> tile;
  tile.load(L.a.x + row * L.a.ldx, j0, j1, L.vec);
  const Row r = load_row<kT>(L, w, row, red);
  if (r.greedy || r.live == 0 || !wants_bins(r)) return;
  if (threadIdx.x < 64) tab[threadIdx.x] = kExp2[threadIdx.x];
#pragma unroll
  for (int e = 0; e < kCopies; ++e)
    for (int i = threadIdx.x; i < kBins; i += kT) mass[e][i] = 0, count[e][i] = 0;
  const int copy = threadIdx.x % kCopies;
  __syncthreads();
  const bool weigh = r.top_p < 1.0;
  uint32_t rest = 0;  // the last bin: no weight, and too many tokens for one counter
  each_token<kT, U>(tile, r.x, j0, j1, L.vec, [&](int, float x) {
    if (!(x > -__builtin_inff())) return;
    const Reduced d = reduce(r, x);
    const int b = bin_of(d);
    if (b == kBins - 1) {
      ++rest;
      return;
    }
    atomicAdd(&count[copy][b], 1u);
    if (weigh) atomicAdd(&mass[copy][b], fixed(weight_of(d, tab)));
  });
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) rest += __shfl_xor(rest, d, 64);
  if ((threadIdx.x & 63) == 0 && rest) atomicAdd(&count[0][kBins - 1], rest);
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kT) {
    const uint32_t n = count[0][i] + (kCopies > 1 ? count[kCopies - 1][i] : 0);
    if (!n) continue;
    atomicAdd(w.count + i, n);
    if (weigh) atomicAdd(w.mass + i, mass[0][i] + (kCopies > 1 ? mass[kCopies - 1][i] : 0));
  }
}

// ------------------------------------------------------------ the cuts --

// Where the cuts fall, from the histogram: bins below `sure` are kept (as far
// as top-k and top-p go), and the tokens of bins [p1, p2] and of bin `kbin`
// are listed to be ordered.
struct Cut {
  int sure, p1, p2, kbin;  // p1 > p2: no bins of top-p; kbin = kBins: top-k ends with a bin
  uint32_t kneed;          // tokens of bin kbin among the first k
  uint32_t rest_kept;      // tokens kept of the last bin, which holds no weight and is not listed
  u64 mass_p1, mass_k;     // weight before bin p1; before bin kbin, or of the first k
};

struct CutLds {
  u64 wave[32];
  int kb;
  uint32_t kbefore, kcount;
  u64 kmass, kbin_mass;
  int p[2];
  u64 pm[2];
};

// A thread's bins, loaded before anything waits.
template <int T>
struct Bins {
  uint32_t n[kBins / T];
  u64 m[kBins / T];
};
template <int T>
__device__ __forceinline__ Bins<T> load_bins(const Launch& L, const RowWs& w) {
  constexpr int V = kBins / T;
  Bins<T> b;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    b.n[i] = L.a.top_k || L.a.top_p ? load_g(w.count + V * threadIdx.x + i) : 0;
    b.m[i] = L.a.top_p ? load_g(w.mass + V * threadIdx.x + i) : 0;
  }
  return b;
}

template <int T>
__device__ Cut find_cut(const Row& r, const Bins<T>& bins, CutLds& S) {
  constexpr int V = kBins / T;
  Cut c;
  c.sure = kBins;
  c.p1 = 1, c.p2 = 0;
  c.kbin = kBins;
  c.kneed = c.rest_kept = 0;
  c.mass_p1 = c.mass_k = 0;
  if (!wants_bins(r)) return c;
  const uint32_t* n = bins.n;
  const u64* m = bins.m;
  u64 nb = 0, mb0 = 0, all, total;
#pragma unroll
  for (int i = 0; i < V; ++i) nb += n[i], mb0 += m[i];
  wg_scan2<T>(nb, mb0, S.wave, all, total);
  // the bin that the k-th token lies in (there is one: 1 <= k <= live)
  u64 mb = mb0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (nb < r.k && nb + n[i] >= r.k) {
      S.kb = V * (int)threadIdx.x + i;
      S.kbefore = (uint32_t)nb, S.kcount = n[i];
      S.kmass = mb, S.kbin_mass = m[i];
    }
    nb += n[i], mb += m[i];
  }
  __syncthreads();
  u64 z_lo, z_hi;  // bounds of the weight of the first k
  const int kb = S.kb;
  const uint32_t need = r.k - S.kbefore;
  const bool part = need < S.kcount && kb < kBins - 1;  // (the last bin's tokens weigh nothing)
  if (part) {
    c.kbin = kb;
    c.kneed = need;
    c.mass_k = z_lo = S.kmass;
    z_hi = S.kmass + S.kbin_mass;
    c.sure = kb;
  } else {
    c.mass_k = z_lo = z_hi = S.kmass + S.kbin_mass;
    c.sure = kb < kBins - 1 ? kb + 1 : kBins - 1;
    // (a min-p above the last bin's weights, 2^-47 at most, keeps none of its tokens)
    if (kb == kBins - 1 && !(r.min_p > 1e-14)) c.rest_kept = need;
  }
  if (r.top_p < 1.0) {
    const u64 lim[2] = {mass_limit(r.top_p, z_lo), mass_limit(r.top_p, z_hi)};
    u64 before = mb0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (before < lim[e] && before + m[i] >= lim[e]) {
          S.p[e] = V * (int)threadIdx.x + i;
          S.pm[e] = before;
        }
      before += m[i];
    }
    __syncthreads();
    c.p1 = S.p[0], c.p2 = S.p[1];
    c.mass_p1 = S.pm[0];
    c.sure = c.p1;
    c.rest_kept = 0;
  }
  return c;
}

// A logit that every token of the kept and listed bins reaches: one comparison
// passes over the others (most of a row).  Bin b ends at v = (3 b + 2.5) ln 2 /
// 64; half a step more, and two fp32 steps, are over any rounding.  Of the
// kept bins, min-p ends the last (that of -64 log2 min_p + 1/2 steps, with a
// slack of most of a bin).
__device__ __forceinline__ float cut_logit(const Row& r, const Cut& c) {
  const float steps = -64.0f * __builtin_amdgcn_logf((float)r.min_p);  // (inf: no limit)
  const int kept = min(c.sure - 1, (int)fminf(steps / 3.0f + 1.0f, (float)kBins));
  const int last = max(max(kept, c.p2), c.kbin < kBins ? c.kbin : 0);
  if (last >= kBins - 1 || !(r.mx < __builtin_inff())) return -__builtin_inff();
  const double x = (double)r.mx - (3 * last + 3) * 0x1.62e42fefa39efp-7 / r.inv_t;
  return (float)(x - 3e-7 * fabs(x));
}

__device__ __forceinline__ bool listed(const Cut& c, int b) { return (b >= c.p1 && b <= c.p2) || b == c.kbin; }

// ------------------------------------- launch 3: listed tokens and sums --

template <int U>
__global__ __launch_bounds__(kT) void gather_kernel(Launch L) {
  __shared__ double tab[64];
  __shared__ u64 red[32];
  __shared__ CutLds S;
  // listed tokens gather here first: a wave that asks memory for each one's
  // place waits for every answer
  __shared__ u64 mine[kMine];
  __shared__ uint32_t mine_n, mine_at;
  const int c = blockIdx.x % L.chunks;
  const int64_t row = blockIdx.x / L.chunks;
  const RowWs w = row_ws(L, row);
  const int j0 = c * L.per, j1 = (int)min((int64_t)(c + 1) * L.per, L.a.N);
  Tile<kT, U> tile;
  tile.load(L.a.x + row * L.a.ldx, j0, j1, L.vec);
  const Bins<kT> bins = load_bins<kT>(L, w);
  const Row r = load_row<kT>(L, w, row, red);
  if (r.greedy || r.live == 0) return;
  if (threadIdx.x < 64) tab[threadIdx.x] = kExp2[threadIdx.x];
  if (threadIdx.x == 0) mine_n = 0;
  __syncthreads();
  const Cut cut = find_cut<kT>(r, bins, S);
  const float least = cut_logit(r, cut);
  u64 sum = 0, kept = 0;
  each_token<kT, U>(tile, r.x, j0, j1, L.vec, [&](int j, float x) {
    if (!(x > -__builtin_inff() && x >= least)) return;
    const Reduced d = reduce(r, x);
    const int b = bin_of(d);
    if (b < cut.sure) {
      const double wt = weight_of(d, tab);
      if (wt >= r.min_p) {  // (the largest logit's weight is 1)
        sum += fixed(wt);
        ++kept;
      }
    } else if (listed(cut, b)) {
      const uint32_t at = atomicAdd(&mine_n, 1u);
      if (at < kMine) mine[at] = pack_token(logit_key(x), j);
    }
  });
  __syncthreads();
  const uint32_t found = mine_n;
  if (threadIdx.x == 0 && found) mine_at = atomicAdd(w.list_n, found);
  u64 total, n;
  wg_scan2<kT>(sum, kept, S.wave, total, n);
  // (where the tokens here are too many for the list, it is not read)
  for (uint32_t i = threadIdx.x; i < min(found, kMine); i += kT)
    if (mine_at + i < kListMax) store_g(w.list + mine_at + i, mine[i]);
  if (threadIdx.x == 0) {
    store_g(w.chunk_mass + c, total);
    store_g(w.chunk_kept + c, (uint32_t)n);
  }
}

// ------------------------------------------------------ launch 4: the draw --

// Tokens kept: those with key and index up to the border, and in the bins
// that are kept for sure.
struct Keep {
  u64 border;  // packed token: kept where the token's own is not less
  int sure;
};

template <int T>
struct FinishLds {
  // (the lists' place holds a chunk's tiles afterwards)
  double tab[64];
  u64 red[32];
  CutLds cut;
  u64 mass[256];
  uint32_t count[256];
  u64 tok[kListMax];         // the listed tokens, ordered
  double weight[kListMax];   // theirs
  u64 list[kListMax];        // and as they came
  uint32_t rank[kListMax];
  u64 prefix[kListMax + 1];  // weight before each, and of all
  u64 tiles[(kChunkMax + 4 * T - 1) / (4 * T)][T / 64];  // weight of a chunk's tiles, by wave
  uint32_t out32[2];
  u64 out64;
};

// The border of a row by the bits of its keys, 8 at a time from the top, a
// pass over the row for each: of the tokens down to the border `in`, the
// first `want` (BY_MASS: those whose forerunners weigh less than `mass`).
struct KeyBorder {
  uint32_t key, ties;  // tokens with larger keys, and the first `ties` of those with this one
};
template <int T, bool BY_MASS>
__device__ KeyBorder key_border(const Launch& L, const Row& r, KeyBorder in, uint32_t want, u64 mass, FinishLds<T>& F) {
  uint32_t prefix = 0, mask = 0, before_n = 0;
  u64 before_m = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += T) F.mass[i] = 0, F.count[i] = 0;
    __syncthreads();
    each_token<T>(r.x, 0, (int)L.a.N, L.vec, [&](int, float x) {
      const uint32_t k = logit_key(x);
      if (k == 0 || (k & mask) != prefix || k < in.key) return;
      const int bin = (k >> shift) & 255;
      atomicAdd(&F.count[bin], 1u);
      if (BY_MASS) atomicAdd(&F.mass[bin], fixed(weight_of(r, F.tab, x)));
    });
    __syncthreads();
    if (threadIdx.x == 0) {
      int bin = 255;
      uint32_t n = before_n;
      u64 m = before_m;
      for (; bin > 0; --bin) {
        if (F.count[bin] && (BY_MASS ? m + F.mass[bin] >= mass : n + F.count[bin] >= want)) break;
        n += F.count[bin];
        m += F.mass[bin];
      }
      F.out32[0] = (uint32_t)bin;
      F.out32[1] = n;
      F.out64 = m;
    }
    __syncthreads();
    prefix |= F.out32[0] << shift;
    mask |= 255u << shift;
    before_n = F.out32[1];
    before_m = F.out64;
    __syncthreads();
  }
  KeyBorder out;
  out.key = prefix;
  const uint32_t here = F.count[prefix & 255];
  if (BY_MASS) {
    // equal keys, equal weights: the i-th is kept where before_m + i w < mass
    const u64 w = fixed(weight_of(r, F.tab, key_logit(prefix)));
    const u64 need = mass > before_m ? mass - before_m : 0;
    out.ties = (uint32_t)min((u64)here, w ? (need + w - 1) / w : (need ? (u64)here : 0));
  } else {
    out.ties = min(here, want - before_n);
  }
  if (prefix == in.key) out.ties = min(out.ties, in.ties);
  __syncthreads();
  return out;
}

// Cuts a row of too many equal or close logits, and redoes its chunks' sums.
template <int T>
__device__ Keep slow_cut(const Launch& L, const RowWs& w, const Row& r, FinishLds<T>& F) {
  KeyBorder cut = {1u, 0xffffffffu};
  if (r.k < r.live) cut = key_border<T, false>(L, r, cut, r.k, 0, F);
  if (r.top_p < 1.0) {
    u64 sum = 0, total;
    each_token<T>(r.x, 0, (int)L.a.N, L.vec, [&](int, float x) {
      const uint32_t k = logit_key(x);
      if (k > cut.key || (k == cut.key && cut.ties == 0xffffffffu)) sum += fixed(weight_of(r, F.tab, x));
    });
    wg_scan<T>(sum, F.red, total);
    if (cut.ties != 0xffffffffu) total += (u64)cut.ties * fixed(weight_of(r, F.tab, key_logit(cut.key)));
    cut = key_border<T, true>(L, r, cut, 0, mass_limit(r.top_p, total), F);
  }
  // the index of the last tie inside: the one with ties - 1 before it
  Keep keep = {pack_token(cut.key, 0x7fffffff), 0};
  uint32_t seen = 0;
  for (int j0 = 0; j0 < (int)L.a.N && cut.ties != 0xffffffffu; j0 += 4 * T) {
    const int j1 = (int)min((int64_t)j0 + 4 * T, L.a.N);
    uint32_t mine = 0;
    each_token<T>(r.x, j0, j1, L.vec, [&](int, float x) { mine += logit_key(x) == cut.key; });
    u64 all;
    uint32_t at = seen + (uint32_t)wg_scan<T>(mine, F.red, all);
    each_token<T>(r.x, j0, j1, L.vec, [&](int j, float x) {
      if (logit_key(x) == cut.key && ++at == cut.ties) F.out64 = pack_token(cut.key, j);
    });
    seen += (uint32_t)all;
    if (seen >= cut.ties) break;
  }
  __syncthreads();
  if (cut.ties != 0xffffffffu) keep.border = F.out64;
  for (int c = 0; c < L.chunks; ++c) {
    u64 sum = 0, kept = 0;
    each_token<T>(r.x, c * L.per, (int)min((int64_t)(c + 1) * L.per, L.a.N), L.vec, [&](int j, float x) {
      const uint32_t k = logit_key(x);
      if (!k || pack_token(k, j) < keep.border) return;
      const double wt = weight_of(r, F.tab, x);
      if (wt >= r.min_p) sum += fixed(wt), ++kept;
    });
    u64 total, n;
    wg_scan<T>(sum, F.red, total);
    wg_scan<T>(kept, F.red, n);
    if (threadIdx.x == 0) {
      store_g(w.chunk_mass + c, total);
      store_g(w.chunk_kept + c, (uint32_t)n);
    }
  }
  __syncthreads();
  return keep;
}

// Orders n packed tokens, the largest first: each one's place is the number of
// larger ones, counted by as many threads as there are for a token (a bitonic
// network of 1,027 tokens took 33 us, its 66 barriers each waiting for LDS).
// `tok` is read, `sorted` written; `rank` is scratch.
template <int T>
__device__ void order_tokens(const u64* tok, uint32_t* rank, u64* sorted, int n) {
  for (int i = threadIdx.x; i < n; i += T) rank[i] = 0;
  __syncthreads();
  int log_share = 0;
  while ((2 << log_share) * n <= T) ++log_share;
  const int share = 1 << log_share;
  for (int i = threadIdx.x; i < n << log_share; i += T) {
    const int e = i >> log_share;
    const u64 me = tok[e];
    uint32_t before = 0;
#pragma unroll 8
    for (int o = i & (share - 1); o < n; o += share) before += tok[o] > me;
    if (before) atomicAdd(&rank[e], before);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += T) sorted[rank[i]] = tok[i];
  __syncthreads();
}

template <int T>
__global__ __launch_bounds__(T) void finish_kernel(Launch L) {
  constexpr int kPer = kListMax / T;   // listed tokens per thread
  constexpr int kCh = (kChunksMax + T - 1) / T;  // chunks per thread
  __shared__ u64 cmass[kChunksMax];  // a chunk's kept weight, that of its listed tokens included
  __shared__ FinishLds<T> F;
  const SampleArgs& a = L.a;
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x;
  const RowWs w = row_ws(L, row);
  // everything that the earlier launches left, loaded before anything waits
  const bool cuts = a.top_k || a.top_p;
  const Bins<T> bins = load_bins<T>(L, w);
  const uint32_t list_n = cuts ? load_g(w.list_n) : 0;
  u64 tok[kPer], chunk_mass[kCh], kept = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) tok[e] = cuts ? load_g(w.list + t + e * T) : 0;
#pragma unroll
  for (int e = 0; e < kCh; ++e) {
    const int c = t + e * T;
    chunk_mass[e] = c < L.chunks ? load_g(w.chunk_mass + c) : 0;
    kept += c < L.chunks ? load_g(w.chunk_kept + c) : 0;
  }
  if (t < 64) F.tab[t] = kExp2[t];
  const Row r = load_row<T>(L, w, row, F.red);
  if (r.greedy || r.live == 0) {
    if (t == 0) {
      store_g(a.token + row, r.live ? (int32_t)~(uint32_t)r.top : -1);
      if (a.prob) store_g(a.prob + row, r.live ? 1.0f : 0.0f);
      if (a.kept) store_g(a.kept + row, r.live ? 1 : 0);
    }
    return;
  }
  const Cut cut = find_cut<T>(r, bins, F.cut);
  Keep keep = {~0ull, cut.sure};
  float least = cut_logit(r, cut);
  const uint32_t nl = wants_bins(r) ? list_n : 0;
  // (a minimum below the last bin's weights would have to look into it)
  const bool slow = nl > kListMax || (cut.rest_kept && r.min_p > 0.0);
  if (slow) {
    __syncthreads();
    keep = slow_cut<T>(L, w, r, F);
    least = -__builtin_inff();
    kept = 0;
#pragma unroll
    for (int e = 0; e < kCh; ++e) {
      const int c = t + e * T;
      chunk_mass[e] = c < L.chunks ? load_g(w.chunk_mass + c) : 0;
      kept += c < L.chunks ? load_g(w.chunk_kept + c) : 0;
    }
  } else if (t == 0) {
    kept += cut.rest_kept;
  }
#pragma unroll
  for (int e = 0; e < kCh; ++e)
    if (t + e * T < L.chunks) cmass[t + e * T] = chunk_mass[e];
  const int n = slow ? 0 : (int)nl;
  if (n) {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (t + e * T < n) F.list[t + e * T] = tok[e];
    order_tokens<T>(F.list, F.rank, F.tok, n);
    // weights before each of them; tokens before bin kbin, and in the bins of top-p
    const int per = (n + T - 1) / T, i0 = min(n, t * per), i1 = min(n, i0 + per);
    u64 before = 0, counts = 0, all, all_counts;
    for (int i = i0; i < i1; ++i) {
      const Reduced d = reduce(r, key_logit((uint32_t)(F.tok[i] >> 32)));
      const int b = bin_of(d);
      const double wd = weight_of(d, F.tab);
      F.weight[i] = wd;
      before += fixed(wd);
      counts += (b < cut.kbin ? 1ull : 0ull) | (b <= cut.p2 ? 1ull << 32 : 0ull);
    }
    wg_scan2<T>(before, counts, F.red, all, all_counts);
    const int nk = (int)(uint32_t)all_counts, np = (int)(all_counts >> 32);
    for (int i = i0; i < i1; ++i) {
      F.prefix[i] = before;
      before += fixed(F.weight[i]);
    }
    if (t == 0) F.prefix[n] = all, F.out32[0] = 0;
    __syncthreads();
    const int kend = cut.kbin < kBins ? nk + (int)cut.kneed : n;  // listed tokens among the first k
    int end = kend;
    if (r.top_p < 1.0) {
      const u64 z = cut.kbin < kBins ? cut.mass_k + F.prefix[kend] - F.prefix[nk] : cut.mass_k;
      const u64 lim = mass_limit(r.top_p, z);
      const int most = min(np, kend);
      // (forerunners grow along the order: one last token is inside)
      for (int i = t; i < most; i += T)
        if (cut.mass_p1 + F.prefix[i] < lim && (i + 1 == most || cut.mass_p1 + F.prefix[i + 1] >= lim)) F.out32[0] = i + 1;
      __syncthreads();
      end = (int)F.out32[0];
    }
    if (end > 0) keep.border = F.tok[end - 1];
    for (int i = t; i < end; i += T) {
      if (F.weight[i] < r.min_p) continue;
      ++kept;
      atomicAdd(&cmass[~(uint32_t)F.tok[i] / (uint32_t)L.per], fixed(F.weight[i]));
    }
  }
  __syncthreads();

  // the chunk that u * total falls in (kCh consecutive ones per thread)
  u64 mine[kCh], before = 0, total, nkept;
#pragma unroll
  for (int e = 0; e < kCh; ++e) {
    mine[e] = kCh * t + e < L.chunks ? cmass[kCh * t + e] : 0;
    before += mine[e];
  }
  wg_scan2<T>(before, kept, F.red, total, nkept);
  const double u = r.u > 0.0f ? fmin((double)r.u, 1.0) : 0.0;
  u64 target = (u64)(u * (double)total);
  if (target >= total) target = total - 1;
#pragma unroll
  for (int e = 0; e < kCh; ++e) {
    if (before <= target && target < before + mine[e]) F.out32[0] = (uint32_t)(kCh * t + e), F.out64 = before;  // once
    before += mine[e];
  }
  __syncthreads();
  const int c = (int)min(F.out32[0], (uint32_t)L.chunks - 1);
  before = F.out64;

  // the tile of that chunk, four tokens per thread, and the token in it
  const int j0 = c * L.per, j1 = (int)min((int64_t)(c + 1) * L.per, a.N);
  auto weight = [&](float x, int j) {  // of token j where it is kept
    u64 f = 0;
    const uint32_t key = x >= least ? logit_key(x) : 0;
    if (key) {
      const Reduced d = reduce(r, x);
      const double wd = weight_of(d, F.tab);
      if ((bin_of(d) < keep.sure || pack_token(key, j) >= keep.border) && wd >= r.min_p) f = fixed(wd);
    }
    return f;
  };
  constexpr int kTile = 4 * T, kAtOnce = kFinishMany / T * 2;
  static_assert(2 * kListMax * sizeof(u64) >= kAtOnce * kTile * sizeof(float), "the tiles fit where tok and weight were");
  Tile<T, 1> tile;
  int at = j0;
  if (j1 - j0 > kTile) {
    // every tile's weight, several tiles loaded at once (and kept in LDS, where
    // the lists were: one copy of the code for all of them)
    float* mem = reinterpret_cast<float*>(F.tok);
    for (int jb = j0; jb < j1; jb += kAtOnce * kTile) {
      Tile<T, kAtOnce> all;
      all.load(r.x, jb, j1, L.vec);
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e)
        *reinterpret_cast<f32x4*>(mem + kTile * e + 4 * t) = f32x4{all.v[e][0], all.v[e][1], all.v[e][2], all.v[e][3]};
#pragma unroll 1
      for (int e = 0; e < kAtOnce && jb + e * kTile < j1; ++e) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(mem + kTile * e + 4 * t);
        const int j = Tile<T, 1>::at(jb + e * kTile, 0);
        u64 sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += weight(x[i], j + i);
        sum = wave_scan(sum);
        if ((t & 63) == 63) F.tiles[(jb - j0) / kTile + e][t >> 6] = sum;
      }
    }
    __syncthreads();
    for (; at + kTile < j1; at += kTile) {  // (every thread alike; the last tile needs no look)
      u64 sum = 0;
#pragma unroll
      for (int v = 0; v < T / 64; ++v) sum += F.tiles[(at - j0) / kTile][v];
      if (before + sum > target) break;
      before += sum;
    }
  }
  tile.load(r.x, at, j1, L.vec);
  u64 wt[4], sum = 0, all;
  const int me = Tile<T, 1>::at(at, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) sum += wt[i] = weight(tile.v[0][i], me + i);
  before += wg_scan<T>(sum, F.red, all);
  if (before <= target && target < before + sum) {  // one thread
    int i = 0;
#pragma unroll
    for (int e = 0; e < 3; ++e) {
      if (before + wt[e] > target) break;
      before += wt[e];
      i = e + 1;
    }
    const float x = i == 0 ? tile.v[0][0] : i == 1 ? tile.v[0][1] : i == 2 ? tile.v[0][2] : tile.v[0][3];
    store_g(a.token + row, me + i);
    if (a.prob) store_g(a.prob + row, (float)(weight_of(r, F.tab, x) * kFix / (double)total));
    if (a.kept) store_g(a.kept + row, (int32_t)nkept);
  }
}

// Tokens per chunk.  A few rows: one tile per workgroup, so that a row is read
// at once.  Where there is a histogram its workgroups all add into the row's
// bins, and beyond 256 of them that costs more than longer chunks do (top-k
// and top-p on 8 rows of 151,936: 47 us at 1,024 tokens, 35 at 2,048, 32 at
// 4,096, 37 at 8,192; without a histogram 17.8 / 19.8 / 19.8 / 25.9); many
// rows want no more than about 2,048 workgroups (64 rows: 59 us at 4,096, 57 at
// 8,192, 64 at 16,384; 96 rows: 81 at 8,192, 91 at 16,384).
int64_t tokens_per_chunk(int64_t M, int64_t N, bool cuts) {
  auto chunks = [&](int64_t per) { return mul_sat(M, (N + per - 1) / per); };
  if (chunks(kChunkMin) <= (cuts ? 256 : 1280)) return kChunkMin;
  int64_t per = 4 * kChunkMin;
  while (per < kChunkMax && chunks(per) > 2048) per *= 2;
  return per;
}
static_assert(kChunkMin == 1024, "the figures above");

template <int U>
void launch_chunks(const Launch& L, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL(top_kernel<U>, grid, dim3(kT), 0, s, L);
  if (L.a.top_k || L.a.top_p) hipLaunchKernelGGL(histogram_kernel<U>, grid, dim3(kT), 0, s, L);
  hipLaunchKernelGGL(gather_kernel<U>, grid, dim3(kT), 0, s, L);
}

}  // namespace

int64_t sample_workspace_bytes(int64_t M, int64_t N) {
  const int64_t per = tokens_per_chunk(M, N, false);  // (the more chunks of the two)
  return mul_sat(M, row_ws_bytes((N + per - 1) / per));
}
int64_t sample_work_items(int64_t M, int64_t N) {
  const int64_t per = tokens_per_chunk(M, N, false);
  return mul_sat(mul_sat(M, (N + per - 1) / per), kFinishMany);
}

hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t s) {
  Launch L;
  L.a = a;
  L.ws = static_cast<uint8_t*>(workspace);
  L.per = (int32_t)tokens_per_chunk(a.M, a.N, a.top_k || a.top_p);
  L.chunks = (int32_t)((a.N + L.per - 1) / L.per);
  L.row_bytes = row_ws_bytes(L.chunks);
  L.vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.M == 1 || a.ldx % 4 == 0);
  const dim3 grid((unsigned)(a.M * L.chunks));
  const dim3 rows((unsigned)a.M);
  if (L.per > kChunkMin) {
    launch_chunks<4>(L, grid, s);
    hipLaunchKernelGGL(finish_kernel<kFinishMany>, rows, dim3(kFinishMany), 0, s, L);
  } else {
    launch_chunks<1>(L, grid, s);
    hipLaunchKernelGGL(finish_kernel<kFinishFew>, rows, dim3(kFinishFew), 0, s, L);
  }
  return hipGetLastError();
}

}  // namespace tern
