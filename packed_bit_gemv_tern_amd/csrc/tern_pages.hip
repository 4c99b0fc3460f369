// tern_pages.hip -- the pages under the cache: which table entries hold them
// (refs[p] counts the entries that hold page p; 0: free), and moving their
// contents.
//
//   fork      dst's entries become src's, every page taken counted once more
//   truncate  entries past the kept tokens are given up, their pages counted down
//   reserve   the lowest free pages to the sequences in order; a part-filled page
//             that others hold too is left to them and copied
//   compact   the k-th lowest hole takes the k-th highest page in use
//   copy      listed pages of all layers, bytes as they are
//
// Whole numbers only, and each page's place follows from counts over the pages
// and sequences before it, not from the order in which threads arrive: results
// are the same in every run.  Ids outside [0, pages) are passed over wherever
// one is read, so no content of the tables reaches past the buffers.
// Roofline: launches and trips to memory (the tables are a few KB to a few MB) and,
// for copy, HBM: 744 pages of 128 KB, 195 MB read and written, in 42 us, 4.6 TB/s
// (a large copy: 4.7).
#include <algorithm>

#include "tern_device.h"

namespace tern {

namespace {

constexpr int kPoolT = kPoolThreads;
constexpr int kChunk = 16 * kPoolT;  // pages that one workgroup counts

__device__ __forceinline__ int64_t pages_for(int32_t tokens, int log_p) {
  return ((int64_t)max(tokens, 0) + (1 << log_p) - 1) >> log_p;
}
__device__ __forceinline__ bool is_page(const PoolArgs& p, int32_t id) { return id >= 0 && id < p.pages; }
__device__ __forceinline__ int32_t* entry(const PoolArgs& p, int64_t s, int64_t j) { return p.table + s * p.ld_table + j; }

// One entry less holds a page; a count that was 0 stays 0 (it is given back), so a
// page given up twice is free, not lost.
__device__ __forceinline__ void drop_ref(int32_t* ref) {
  if (__hip_atomic_fetch_add(ref, -1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) <= 0)
    __hip_atomic_fetch_add(ref, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Exclusive prefix of v over the workgroup's T threads, and its total.
template <int T = kPoolT>
__device__ __forceinline__ int64_t wg_prefix(int64_t v, int64_t& total, int64_t* red) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  __syncthreads();  // (red may still be read from the call before)
  if (lane == 63) red[w] = x;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < T / 64; ++i) {
    if (i < w) before += red[i];
    total += red[i];
  }
  return before + x - v;
}

// ---- fork and truncate ---------------------------------------------------

// One workgroup per pair.  A pair is passed over if its rows lie outside the
// table, if its dst is the src of any pair, or if a later pair has the same dst.
__global__ __launch_bounds__(kPoolT) void fork_kernel(PoolArgs p, const int32_t* len, const int32_t* src,
                                                      const int32_t* dst, int64_t n) {
  __shared__ int32_t bad;
  const int64_t i = blockIdx.x;
  const int32_t from = load_g(src + i), to = load_g(dst + i);
  if (threadIdx.x == 0) bad = from < 0 || from >= p.S || to < 0 || to >= p.S;
  __syncthreads();
  for (int64_t k = threadIdx.x; k < n; k += kPoolT)
    if (load_g(src + k) == to || (k > i && load_g(dst + k) == to)) bad = 1;
  __syncthreads();
  if (bad) return;
  const int64_t J = min(pages_for(load_g(len + from), p.log_p), p.ld_table);
  for (int64_t j = threadIdx.x; j < J; j += kPoolT) {
    const int32_t id = load_g(entry(p, from, j));
    if (is_page(p, id)) __hip_atomic_fetch_add(p.refs + id, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    store_g(entry(p, to, j), is_page(p, id) ? id : -1);
  }
}

__global__ __launch_bounds__(kPoolT) void truncate_kernel(PoolArgs p, const int32_t* len, const int32_t* keep) {
  const int64_t s = blockIdx.x;
  const int64_t J = min(pages_for(load_g(len + s), p.log_p), p.ld_table);
  for (int64_t j = pages_for(load_g(keep + s), p.log_p) + threadIdx.x; j < J; j += kPoolT) {
    const int32_t id = load_g(entry(p, s, j));
    if (is_page(p, id)) drop_ref(p.refs + id);
    store_g(entry(p, s, j), -1);
  }
}

// ---- reserve ---------------------------------------------------------------

// Workspace: int32 count[chunks], then int32 need[S] (reserve) or rank[pages]
// (compact).
__host__ __device__ __forceinline__ int64_t chunks_of(int64_t pages) { return (pages + kChunk - 1) / kChunk; }

// What a sequence asks for: pages past its last one, and whether the one that
// its next token goes to has to be copied (`sole`: it is held by others too,
// but they all copy it, and this sequence keeps it).
struct Need {
  int32_t copy, sole;
  int64_t fresh;
};
constexpr int32_t kNeedCopy = 1 << 30, kNeedSole = 1 << 29, kNeedNever = -1;

// The page that sequence s writes into next (-1: none that it holds already).
__device__ __forceinline__ int32_t written_page(const PoolArgs& p, const int32_t* len, const int32_t* want, int64_t s) {
  const int32_t n = max(load_g(len + s), 0), w = load_g(want + s);
  if (w <= n || (n & ((1 << p.log_p) - 1)) == 0 || pages_for(w, p.log_p) > p.ld_table) return -1;
  const int32_t id = load_g(entry(p, s, n >> p.log_p));
  return is_page(p, id) ? id : -1;
}

// Workgroups below `chunks` count the free pages of a chunk; the others take
// four sequences, one to a wave.
__global__ __launch_bounds__(kPoolT) void reserve_count_kernel(PoolArgs p, const int32_t* len, const int32_t* want,
                                                               int32_t* count, int32_t* need, int64_t chunks) {
  __shared__ int64_t red[kPoolT / 64];
  if (blockIdx.x < chunks) {
    int64_t n = 0, total;
    for (int i = 0; i < kChunk / kPoolT; ++i) {
      const int64_t id = (int64_t)blockIdx.x * kChunk + i * kPoolT + threadIdx.x;
      if (id < p.pages) n += load_g(p.refs + id) <= 0;
    }
    wg_prefix(n, total, red);
    if (threadIdx.x == 0) store_g(count + blockIdx.x, (int32_t)total);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int64_t s = ((int64_t)blockIdx.x - chunks) * (kPoolT / 64) + (threadIdx.x >> 6);
  if (s >= p.S) return;
  const int32_t n = max(load_g(len + s), 0), w = load_g(want + s);
  int32_t v = 0;
  if (w > n) {
    const int64_t j0 = pages_for(n, p.log_p), j1 = pages_for(w, p.log_p);
    if (j1 > p.ld_table) {
      v = kNeedNever;
    } else {
      v = (int32_t)(j1 - j0);
      const int32_t id = written_page(p, len, want, s);
      const int32_t held = id >= 0 ? load_g(p.refs + id) : 0;
      if (held > 1) {  // as many copies as others write into it, the last of all holders keeps it
        int64_t writers = 0;
        bool later = false;
        for (int64_t k = lane; k < p.S; k += 64)
          if (written_page(p, len, want, k) == id) ++writers, later |= k > s;
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) writers += __shfl_xor(writers, d, 64);
        later = __any(later);
        v |= writers >= held && !later ? kNeedSole : kNeedCopy;
      }
    }
  }
  if (lane == 0) store_g(need + s, v);
}

__device__ __forceinline__ Need unpack_need(int32_t v) {
  Need n;
  n.copy = v >= 0 && (v & kNeedCopy) != 0;
  n.sole = v >= 0 && (v & kNeedSole) != 0;
  n.fresh = v < 0 ? 0 : v & (kNeedSole - 1);
  return n;
}

// The sequences' needs as one running sum: those whose sum lies inside the
// free pages get theirs.  Workgroup b hands out the free pages of chunk b, the
// one with rank r (among all free pages) to the sequence that r falls into;
// workgroup 0 also writes granted, from and to of sequences that need none.
__global__ __launch_bounds__(kPoolT) void reserve_kernel(PoolArgs p, const int32_t* len, const int32_t* want,
                                                         const int32_t* count, const int32_t* need, int64_t chunks,
                                                         int32_t* granted, int32_t* from, int32_t* to) {
  __shared__ int64_t red[kPoolT / 64];
  __shared__ int32_t free_id[kChunk];
  const int t = threadIdx.x;
  int64_t before = 0, all = 0, total;  // free pages before this chunk, of all
  for (int64_t c = t; c < chunks; c += kPoolT) {
    const int64_t n = load_g(count + c);
    all += n;
    if (c < blockIdx.x) before += n;
  }
  wg_prefix(before, total, red);
  before = total;
  wg_prefix(all, total, red);
  all = total;
  // this chunk's free pages, lowest first
  int32_t mine = 0;
  const int64_t id0 = (int64_t)blockIdx.x * kChunk + (int64_t)t * (kChunk / kPoolT);
  uint32_t mask = 0;
#pragma unroll
  for (int i = 0; i < kChunk / kPoolT; ++i)
    if (id0 + i < p.pages && load_g(p.refs + id0 + i) <= 0) mask |= 1u << i, ++mine;
  int64_t at = wg_prefix(mine, total, red);
  const int64_t here = total;
#pragma unroll
  for (int i = 0; i < kChunk / kPoolT; ++i)
    if (mask >> i & 1) free_id[at++] = (int32_t)(id0 + i);
  __syncthreads();
  // sequences in order, kPoolT at a time
  int64_t run = 0;
  for (int64_t s0 = 0; s0 < p.S; s0 += kPoolT) {
    const int64_t s = s0 + t;
    const int32_t v = s < p.S ? load_g(need + s) : 0;
    const Need nd = unpack_need(v);
    const int64_t n = nd.copy + nd.fresh;
    const int64_t first = run + wg_prefix(n, total, red);
    run += total;
    if (s >= p.S) continue;
    const bool ok = v != kNeedNever && (first + n <= all || (n == 0 && !nd.sole));
    if (blockIdx.x == 0) {
      store_g(granted + s, (int32_t)ok);
      if (!(ok && nd.copy)) store_g(from + s, -1), store_g(to + s, -1);
    }
    if (!ok || first >= before + here || first + n <= before) continue;
    const int64_t j0 = pages_for(load_g(len + s), p.log_p);
    for (int64_t k = max(first, before); k < min(first + n, before + here); ++k) {
      const int32_t id = free_id[k - before];
      int64_t j = j0 + (k - first) - nd.copy;
      if (nd.copy && k == first) {
        const int32_t old = load_g(entry(p, s, j));
        __hip_atomic_fetch_add(p.refs + old, -1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // (it was above 1)
        store_g(from + s, old);
        store_g(to + s, id);
      }
      store_g(entry(p, s, j), id);
      store_g(p.refs + id, 1);
    }
  }
}

// A pool of up to kSmallPages pages and kSmallSeqs sequences in one launch of one
// workgroup: the free pages as a bitmap in LDS, the sequences' needs and their
// running sum beside it; then thread r takes the r-th page that is handed out, and
// finds its sequence and its page by bisection.  One step of 8 tokens, this against
// the two launches above: 9 sequences, 80 pages 4.3 and 6.4 us, 64 and 4,096 6.9 and
// 9.6, 256 and 15,548 8.9 and 9.6 (64 of them sharing pages 8.8 and 9.7), 256 and
// 32,768 10.0 and 9.7, 65,536 13.9 and 9.9: a chain of trips to memory either way.
constexpr int kSmallT = 1024, kSmallPages = 16384, kSmallSeqs = 2048;

// the last i < n with first[i] <= r (first[0] <= r)
__device__ __forceinline__ int last_at(const int32_t* first, int n, int32_t r) {
  int lo = 0;
  for (int d = 1 << (31 - __builtin_clz(n)); d; d >>= 1)
    if (lo + d < n && first[lo + d] <= r) lo += d;
  return lo;
}

__global__ __launch_bounds__(kSmallT) void reserve_small_kernel(PoolArgs p, const int32_t* len, const int32_t* want,
                                                                int32_t* granted, int32_t* from, int32_t* to) {
  __shared__ int64_t red[kSmallT / 64];
  __shared__ uint64_t free_bits[kSmallPages / 64];
  __shared__ int32_t free_first[kSmallPages / 64], first[kSmallSeqs], needs[kSmallSeqs];
  __shared__ int32_t writes[kSmallSeqs];
  __shared__ __attribute__((aligned(16))) struct { int32_t id, s; } sharer[kSmallSeqs];
  __shared__ int32_t handed, sharers;
  const int t = threadIdx.x, lane = t & 63, S = (int)p.S, pages = (int)p.pages, words = (pages + 63) / 64;
  // each sequence's need, as if all others kept the page it writes into (first:
  // how many hold that)
  for (int i = t; i < kSmallSeqs; i += kSmallT) sharer[i].id = -2;  // (no page)
  if (t == 0) sharers = handed = 0;
  __syncthreads();
  for (int s = t; s < S; s += kSmallT) {
    const int32_t n = max(load_g(len + s), 0), w = load_g(want + s), id = written_page(p, len, want, s);
    const int64_t j1 = pages_for(w, p.log_p);
    const int32_t held = id >= 0 ? load_g(p.refs + id) : 0;
    writes[s] = id;
    first[s] = held;
    needs[s] = w <= n ? 0 : j1 > p.ld_table ? kNeedNever : (int32_t)(j1 - pages_for(n, p.log_p)) | (held > 1 ? kNeedCopy : 0);
    if (held > 1) sharer[atomicAdd(&sharers, 1)] = {id, s};
  }
  constexpr int U = 8;  // loads in flight
  for (int i0 = 0; i0 < pages; i0 += U * kSmallT) {
    int32_t held[U];
#pragma unroll
    for (int u = 0; u < U; ++u) held[u] = load_g(p.refs + min(i0 + u * kSmallT + t, pages - 1));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = i0 + u * kSmallT + t;
      const uint64_t bits = __ballot(id < pages && held[u] <= 0);
      if (lane == 0 && id < pages) free_bits[id / 64] = bits;
    }
  }
  __syncthreads();
  int64_t all;
  const int mine = t < words ? __builtin_popcountll(free_bits[t]) : 0;
  const int64_t before = wg_prefix<kSmallT>(mine, all, red);
  if (t < words) free_first[t] = (int32_t)before;
  int64_t run = 0;
  for (int s0 = 0; s0 < S; s0 += kSmallT) {
    const int s = s0 + t;
    int32_t v = s < S ? needs[s] : 0;
    const bool shared = v > 0 && (v & kNeedCopy);
    if (__any(shared)) {  // how many write into the page, and the last that does
      const int32_t id = s < S ? writes[s] : -1;
      int writers = 0, last = 0;
      for (int k0 = 0; k0 < sharers; k0 += 8) {
#pragma unroll
        for (int k = k0; k < k0 + 8; k += 2) {
          const i32x4 w = *reinterpret_cast<const i32x4*>(&sharer[k]);
          writers += (w[0] == id) + (w[2] == id);
          last = max(last, max(w[0] == id ? w[1] : 0, w[2] == id ? w[3] : 0));
        }
      }
      if (shared && writers >= first[s] && last == s) v = (v & ~kNeedCopy) | kNeedSole;
    }
    const Need nd = unpack_need(v);
    const int64_t n = nd.copy + nd.fresh;
    int64_t total;
    const int64_t at = run + wg_prefix<kSmallT>(n, total, red);
    run += total;
    __syncthreads();  // (first is rewritten from here on, a part for each round)
    if (s < S) {
      const bool ok = v != kNeedNever && (at + n <= all || (n == 0 && !nd.sole));
      store_g(granted + s, (int32_t)ok);
      if (!(ok && nd.copy)) store_g(from + s, -1), store_g(to + s, -1);
      needs[s] = v;
      first[s] = (int32_t)min(at, (int64_t)pages);
      if (ok && n > 0) atomicMax(&handed, (int32_t)(at + n));
    }
  }
  __syncthreads();
  // (the sums of the rows that get something lie side by side from 0 on)
  for (int r = t; r < handed; r += kSmallT) {
    const int s = last_at(first, S, r), w = last_at(free_first, words, r);
    uint64_t bits = free_bits[w];
    for (int k = r - free_first[w]; k > 0; --k) bits &= bits - 1;
    const int32_t id = 64 * w + __builtin_ctzll(bits);
    const Need nd = unpack_need(needs[s]);
    const int64_t j = pages_for(load_g(len + s), p.log_p) + (r - first[s]) - nd.copy;
    if (nd.copy && r == first[s]) {
      __hip_atomic_fetch_add(p.refs + writes[s], -1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      store_g(from + s, writes[s]);
      store_g(to + s, id);
    }
    store_g(entry(p, s, j), id);
    store_g(p.refs + id, 1);
  }
}

// ---- compact -----------------------------------------------------------------

__device__ __forceinline__ void clear_moves(int32_t* from, int32_t* to, int64_t moves, int64_t i0, int64_t step) {
  for (int64_t i = i0; i < moves; i += step) store_g(from + i, -1), store_g(to + i, -1);
}

// Counts the pages in use of a chunk; clears the lists of moves.
__global__ __launch_bounds__(kPoolT) void compact_count_kernel(PoolArgs p, int32_t* count, int32_t* from, int32_t* to,
                                                               int64_t moves) {
  __shared__ int64_t red[kPoolT / 64];
  clear_moves(from, to, moves, (int64_t)blockIdx.x * kPoolT + threadIdx.x, (int64_t)gridDim.x * kPoolT);
  int64_t n = 0, total;
  for (int i = 0; i < kChunk / kPoolT; ++i) {
    const int64_t id = (int64_t)blockIdx.x * kChunk + i * kPoolT + threadIdx.x;
    if (id < p.pages) n += load_g(p.refs + id) > 0;
  }
  wg_prefix(n, total, red);
  if (threadIdx.x == 0) store_g(count + blockIdx.x, (int32_t)total);
}

// Page p with u pages in use before it: a hole (p < live) is the (p - u)-th
// from below, a page in use at or behind `live` the (live - 1 - u)-th from
// above; there are as many of one as of the other.  With T = kSmallT the workgroup
// is alone (up to kAlonePages pages), counts for itself and clears the lists too:
// compact of 9 sequences' 80 pages 6.5 us, with the launch that counts 8.9, of 64
// and 4,096 7.6 and 14.1, of 256 and 8,192 9.2 and 14.7, and 12,288 11.1 and 14.7, and
// 16,384 17.4 and 15.2.
constexpr int kAlonePages = 12 * kSmallT;
template <int T>
__global__ __launch_bounds__(T) void compact_plan_kernel(PoolArgs p, const int32_t* count, int64_t chunks,
                                                         int32_t* from, int32_t* to, int64_t moves, int32_t* rank,
                                                         int32_t* live_out) {
  constexpr bool kAlone = T == kSmallT;
  constexpr int kEach = kAlone ? kAlonePages / T : kChunk / T;
  __shared__ int64_t red[T / 64];
  const int t = threadIdx.x;
  int64_t before = 0, live = 0, total;
  const int64_t id0 = ((int64_t)blockIdx.x * T + t) * kEach;
  int32_t held[kEach] = {};
  if (p.pages > 0) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) held[i] = load_g(p.refs + min(id0 + i, p.pages - 1));
  }
  uint32_t mask = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) mask |= (uint32_t)(id0 + i < p.pages && held[i] > 0) << i;
  if constexpr (kAlone) {
    clear_moves(from, to, moves, t, T);
  } else {
    for (int64_t c = t; c < chunks; c += T) {
      const int64_t n = load_g(count + c);
      live += n;
      if (c < blockIdx.x) before += n;
    }
    wg_prefix<T>(before, total, red);
    before = total;
    wg_prefix<T>(live, total, red);
    live = total;
  }
  int64_t u = before + wg_prefix<T>(__builtin_popcount(mask), total, red);  // (its barriers also order the clearing)
  if constexpr (kAlone) live = total;
  if (blockIdx.x == 0 && t == 0) store_g(live_out, (int32_t)live);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t id = id0 + i;
    if (id >= p.pages) break;
    const bool used = mask >> i & 1;
    if (!used && id < live && id - u < moves) store_g(to + (id - u), (int32_t)id);
    if (used && id >= live) {
      const int64_t k = live - 1 - u;
      store_g(rank + id, (int32_t)k);
      if (k < moves) store_g(from + k, (int32_t)id);
    }
    u += used;
  }
}

// Entries of pages that move, and the pages' counts: workgroups below `rows`
// take a row of the table each, the others kPoolT moves.
__global__ __launch_bounds__(kPoolT) void compact_apply_kernel(PoolArgs p, const int32_t* len, const int32_t* from,
                                                               const int32_t* to, int64_t moves, const int32_t* rank,
                                                               const int32_t* live_in) {
  if (blockIdx.x >= p.S) {
    const int64_t k = ((int64_t)blockIdx.x - p.S) * kPoolT + threadIdx.x;
    if (k >= moves) return;
    const int32_t a = load_g(from + k), b = load_g(to + k);
    if (a < 0 || b < 0) return;
    store_g(p.refs + b, load_g(p.refs + a));
    store_g(p.refs + a, 0);
    return;
  }
  const int64_t s = blockIdx.x, J = min(pages_for(load_g(len + s), p.log_p), p.ld_table);
  const int32_t live = load_g(live_in);
  for (int64_t j = threadIdx.x; j < J; j += kPoolT) {
    const int32_t id = load_g(entry(p, s, j));
    if (!is_page(p, id) || id < live) continue;
    const int32_t k = load_g(rank + id);
    if (k >= 0 && k < moves && load_g(from + k) == id) store_g(entry(p, s, j), load_g(to + k));
  }
}

// ---- copy ----------------------------------------------------------------------

constexpr int kCopyU = 4;  // 16-byte loads of a thread before its first store
constexpr int64_t kCopyBytes = 16ll * kCopyU * kPoolT;

// One workgroup moves up to kCopyBytes of one page of K or V of one layer.
__global__ __launch_bounds__(kPoolT) void copy_kernel(CopyArgs a, int parts) {
  int64_t b = blockIdx.x;
  const int part = (int)(b % parts);
  b /= parts;
  const bool isv = b & 1;
  b >>= 1;
  const int l = (int)(b % a.layers);
  const int64_t i = b / a.layers;
  const int32_t from = load_g(a.from + i), to = load_g(a.to + i);
  if (from < 0 || from >= a.pages_from || to < 0 || to >= a.pages_to) return;
  const CopyLayer& L = a.layer[l];
  const int8_t* src = (isv ? L.v : L.k) + from * a.page_bytes;
  int8_t* dst = (isv ? L.v_to : L.k_to) + to * a.page_bytes;
  const int64_t at = part * kCopyBytes + 16 * threadIdx.x;
  u32x4 v[kCopyU];
#pragma unroll
  for (int u = 0; u < kCopyU; ++u)
    if (at + u * 16 * kPoolT < a.page_bytes) v[u] = load16(src + at + u * 16 * kPoolT);
#pragma unroll
  for (int u = 0; u < kCopyU; ++u)
    if (at + u * 16 * kPoolT < a.page_bytes) store_g(reinterpret_cast<u32x4*>(dst + at + u * 16 * kPoolT), v[u]);
  if (part == 0)
    for (int h = threadIdx.x; h < a.H; h += kPoolT)
      store_g((isv ? L.v_scale_to : L.k_scale_to) + (int64_t)to * a.H + h,
              load_g((isv ? L.v_scale : L.k_scale) + (int64_t)from * a.H + h));
}

int64_t seq_blocks(const PoolArgs& p) { return (p.S + kPoolT / 64 - 1) / (kPoolT / 64); }

}  // namespace

int64_t pool_workspace_bytes(const PoolArgs& p) { return 4 * (chunks_of(p.pages) + std::max(p.S, p.pages)); }

// The largest launch of any call on the pool (moves and pairs apart).
int64_t pool_work_items(const PoolArgs& p) {
  return mul_sat(chunks_of(p.pages) + p.S + (p.pages + kPoolT - 1) / kPoolT, kPoolT);
}

hipError_t launch_kv_fork(const PoolArgs& p, const int32_t* len, const int32_t* src, const int32_t* dst, int64_t n,
                          hipStream_t s) {
  hipLaunchKernelGGL(fork_kernel, dim3((unsigned)n), dim3(kPoolT), 0, s, p, len, src, dst, n);
  return hipGetLastError();
}

hipError_t launch_kv_truncate(const PoolArgs& p, const int32_t* len, const int32_t* keep, hipStream_t s) {
  hipLaunchKernelGGL(truncate_kernel, dim3((unsigned)p.S), dim3(kPoolT), 0, s, p, len, keep);
  return hipGetLastError();
}

hipError_t launch_kv_reserve(const PoolArgs& p, const int32_t* len, const int32_t* want, int32_t* granted,
                             int32_t* from, int32_t* to, void* workspace, hipStream_t s) {
  if (p.pages <= kSmallPages && p.S <= kSmallSeqs) {
    hipLaunchKernelGGL(reserve_small_kernel, dim3(1), dim3(kSmallT), 0, s, p, len, want, granted, from, to);
    return hipGetLastError();
  }
  const int64_t chunks = chunks_of(p.pages);
  int32_t* count = static_cast<int32_t*>(workspace);
  int32_t* need = count + chunks;
  hipLaunchKernelGGL(reserve_count_kernel, dim3((unsigned)(chunks + seq_blocks(p))), dim3(kPoolT), 0, s, p, len, want,
                     count, need, chunks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(reserve_kernel, dim3((unsigned)chunks), dim3(kPoolT), 0, s, p, len, want, count, need, chunks,
                     granted, from, to);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const PoolArgs& p, const int32_t* len, int32_t* from, int32_t* to, int64_t moves,
                             int32_t* live, void* workspace, hipStream_t s) {
  const int64_t chunks = chunks_of(p.pages);
  int32_t* count = static_cast<int32_t*>(workspace);
  int32_t* rank = count + chunks;
  hipError_t e;
  if (p.pages <= kAlonePages) {
    hipLaunchKernelGGL(compact_plan_kernel<kSmallT>, dim3(1), dim3(kSmallT), 0, s, p, count, chunks, from, to, moves,
                       rank, live);
  } else {
    hipLaunchKernelGGL(compact_count_kernel, dim3((unsigned)chunks), dim3(kPoolT), 0, s, p, count, from, to, moves);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(compact_plan_kernel<kPoolT>, dim3((unsigned)chunks), dim3(kPoolT), 0, s, p, count, chunks, from,
                       to, moves, rank, live);
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  // (no more than pages / 2 of the listed moves are in use)
  const int64_t apply = p.S + (std::min(moves, p.pages) + kPoolT - 1) / kPoolT;
  if (apply == 0) return hipSuccess;
  hipLaunchKernelGGL(compact_apply_kernel, dim3((unsigned)apply), dim3(kPoolT), 0, s, p, len, from, to, moves, rank,
                     live);
  return hipGetLastError();
}

static int copy_parts(int64_t page_bytes) { return (int)((page_bytes + kCopyBytes - 1) / kCopyBytes); }

int64_t kv_copy_work_items(int64_t page_bytes, int64_t n, int64_t layers) {
  return mul_sat(mul_sat(mul_sat(2 * copy_parts(page_bytes), n), layers), kPoolT);
}

hipError_t launch_kv_copy(const CopyArgs& a, hipStream_t s) {
  const int parts = copy_parts(a.page_bytes);
  hipLaunchKernelGGL(copy_kernel, dim3((unsigned)(2 * a.n * a.layers * parts)), dim3(kPoolT), 0, s, a, parts);
  return hipGetLastError();
}

}  // namespace tern
