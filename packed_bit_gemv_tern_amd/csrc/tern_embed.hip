// tern_embed.hip -- rows of the int8 embedding table (one scale per row, the
// format of the output head):
//
//     x[m][j] = (W[ids[m]][j] * s_row[ids[m]]) * scale      (fp32, in this order)
//
// and a row of zeros where ids[m] is no row of the table.  Roofline: HBM, 5
// bytes an element: 8,191 rows of 4,096 in 31 us, 5.4 TB/s (a copy: 4.7, a fill:
// 6.9; four of the five bytes are written).  One row, 1.8 us, is the launch and
// two dependent trips to memory.
#include <algorithm>

#include "tern_device.h"

namespace tern {

namespace {

constexpr int kEmbedT = 256;

// 2^lt threads take one row, a thread four columns at a time (VEC: one dword
// of codes, one 16-byte store; consecutive threads take consecutive columns, so
// every instruction of a wave covers whole lines) and U such groups before its
// first store, so that a row's codes are all asked for at once.
template <int U, bool VEC>
__global__ __launch_bounds__(kEmbedT) void embed_kernel(EmbedArgs a, int lt) {
  const int t = threadIdx.x & ((1 << lt) - 1);
  const int64_t m = (int64_t)blockIdx.x * (kEmbedT >> lt) + (threadIdx.x >> lt);
  if (m >= a.M) return;
  const int32_t id = load_g(a.ids + m);
  const bool there = id >= 0 && id < a.N;
  const int8_t* w = a.W + (int64_t)(there ? id : 0) * a.ldw;
  const float s = there ? load_g(a.s_row + id) : 0.0f, scale = there ? a.scale : 0.0f;
  float* x = a.x + m * a.ldx;
  const int64_t K = a.K, step = VEC ? 4ll << lt : 1ll << lt;
  for (int64_t j0 = VEC ? 4 * t : t; j0 < K; j0 += U * step) {
    if constexpr (VEC) {
      uint32_t c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t j = j0 + u * step;
        c[u] = there && j < K ? load_g(reinterpret_cast<const uint32_t*>(w + j)) : 0u;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t j = j0 + u * step;
        if (j >= K) break;
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(__fmul_rn((float)(int8_t)(c[u] >> (8 * i)), s), scale);
        store_g(reinterpret_cast<f32x4*>(x + j), v);
      }
    } else {
      int8_t c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t j = j0 + u * step;
        c[u] = there && j < K ? load_g(w + j) : (int8_t)0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t j = j0 + u * step;
        if (j < K) store_g(x + j, __fmul_rn(__fmul_rn((float)c[u], s), scale));
      }
    }
  }
}

// Threads per row (log2): four groups of four columns each, 16 to a whole workgroup.
int embed_lt(int64_t K) {
  int lt = 4;
  while (lt < 8 && (16ll << lt) < K) ++lt;
  return lt;
}

}  // namespace

int64_t embed_work_items(int64_t M, int64_t K) {
  const int64_t rows = kEmbedT >> embed_lt(K);
  return mul_sat(M / rows + (M % rows != 0), kEmbedT);
}

hipError_t launch_embed(const EmbedArgs& a, hipStream_t s) {
  const int lt = embed_lt(a.K);
  const bool vec = a.K % 4 == 0 && (reinterpret_cast<uintptr_t>(a.W) % 4) == 0 && a.ldw % 4 == 0 &&
                   (reinterpret_cast<uintptr_t>(a.x) % 16) == 0 && (a.M == 1 || a.ldx % 4 == 0);
  const dim3 grid((unsigned)(embed_work_items(a.M, a.K) / kEmbedT));
  if (vec)
    hipLaunchKernelGGL((embed_kernel<4, true>), grid, dim3(kEmbedT), 0, s, a, lt);
  else
    hipLaunchKernelGGL((embed_kernel<8, false>), grid, dim3(kEmbedT), 0, s, a, lt);
  return hipGetLastError();
}

}  // namespace tern
