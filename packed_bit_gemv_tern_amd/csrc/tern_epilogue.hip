// tern_epilogue.hip -- a ternary linear with what follows it in the same
// launch: bias, activation, the product with a second linear of the same shape
// (the gate and up projections of a gated feed-forward) and the residual.
//
//     v  = (s_row * (float)acc) * s_act [+ bias]        acc exact in int32
//     h  = act(v) [* v_up]
//     y  = [res +] h
//
// every product and sum one fp32 rounding.
#include <algorithm>

#include "tern_prologue.h"

namespace tern {

namespace {

constexpr uint32_t kCodeTable = 0x000100FFu;  // code byte 0, 1, 2 -> -1, 0, +1
constexpr uint32_t kZeroCodes = 0x55555555u;

__device__ __forceinline__ i32x4 decode16(uint32_t x) {
  i32x4 b;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    b[k] = (int32_t)__builtin_amdgcn_perm(kCodeTable, kCodeTable, (x >> (2 * k)) & 0x03030303u);
  return b;
}

// silu(x) = x / (1 + e^-x), and gelu in its tanh form, x (1 + tanh(c (x + 0.044715
// x^3))) / 2 with c = sqrt(2 / pi), as x / (1 + e^(-2 c (...))): nothing cancels
// for negative x.
__device__ __forceinline__ float activate(int act, float x) {
  if (act == 0) return x;
  float t = -x;
  if (act == 2) {
    const float cube = __fmul_rn(__fmul_rn(x, x), x);
    t = __fmul_rn(-1.5957691216057308f, __fadd_rn(x, __fmul_rn(0.044715f, cube)));
  }
  return __fdiv_rn(x, __fadd_rn(1.0f, exp32(t)));
}

// What an output row brings to the epilogue, of each matrix.
template <int MATS>
struct RowOps {
  int32_t rowsum[MATS];
  float s_row[MATS], bias[MATS];
};
template <int MATS>
__device__ __forceinline__ RowOps<MATS> row_ops(const EpilogueArgs& a, int64_t i) {
  RowOps<MATS> o;
#pragma unroll
  for (int k = 0; k < MATS; ++k) {
    o.rowsum[k] = load_g(a.w[k].rowsum + i);
    o.s_row[k] = load_g(a.w[k].s_row + i);
    o.bias[k] = a.w[k].bias ? load_g(a.w[k].bias + i) : 0.0f;
  }
  return o;
}

// h of one output from the linears' sums
template <int MATS>
__device__ __forceinline__ float output(const EpilogueArgs& a, const int32_t (&sum)[MATS], const RowOps<MATS>& o,
                                        int32_t z, float s_act) {
  float v[MATS];
#pragma unroll
  for (int k = 0; k < MATS; ++k) {
    v[k] = epilogue(o.s_row[k], (int32_t)((uint32_t)sum[k] - mul_zr(z, o.rowsum[k])), s_act);
    if (a.w[k].bias) v[k] = __fadd_rn(v[k], o.bias[k]);
  }
  const float h = activate(a.act, v[0]);
  return MATS == 2 ? __fmul_rn(h, v[MATS - 1]) : h;
}

// 16 activations from column j on, zeros past K.
__device__ __forceinline__ i32x4 load_q16(const int8_t* q, int64_t j, int K) {
  if (j + 16 <= K) return __builtin_bit_cast(i32x4, load16(q + j));
  i32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int d = 0; d < 16; ++d)
    if (j + d < K) v[d / 4] |= (int32_t)((uint32_t)(uint8_t)load_g(q + j + d) << (8 * (d % 4)));
  return v;
}

// RB blocks of 16 rows (of each matrix) and TB blocks of 16 tokens to a
// workgroup; its W waves take 256 columns at a time in turn, and their exact
// int32 sums meet in LDS.  v_mfma_i32_16x16x64_i8 with the weights as A: lane
// (r, g) loads the whole 16-byte chunk 4 i + g of row r, four operands of 64
// weights for four instructions; the tokens' operands are the same columns of
// token r, loaded as they lie (any order of K serves if both sides have it).
constexpr int RB = 2;
constexpr int kRedStride = 68;  // of 64 lanes' values of one register, off each other's banks

template <int W, int TB, int MATS>
__global__ __launch_bounds__(64 * W) void epilogue_rows_kernel(EpilogueArgs a, int row_tiles) {
  __shared__ int32_t red[W][MATS * RB * 4 * kRedStride];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int row0 = (blockIdx.x % row_tiles) * 16 * RB;
  const int64_t tok0 = (int64_t)(blockIdx.x / row_tiles) * 16 * TB;
  const uint8_t* wsrc[MATS][RB];
  const int8_t* qsrc[TB];
#pragma unroll
  for (int k = 0; k < MATS; ++k)
#pragma unroll
    for (int b = 0; b < RB; ++b) wsrc[k][b] = a.w[k].packed + (int64_t)min(row0 + 16 * b + r, a.N - 1) * a.ld;
#pragma unroll
  for (int t = 0; t < TB; ++t) qsrc[t] = a.q + min(tok0 + 16 * t + r, (int64_t)a.M - 1) * a.ldq;
  i32x4 acc[MATS][RB][TB];
#pragma unroll
  for (int k = 0; k < MATS; ++k)
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int t = 0; t < TB; ++t) acc[k][b][t] = i32x4{0, 0, 0, 0};
  for (int c0 = 4 * w; c0 < a.nch; c0 += 4 * W) {
    const int c = c0 + g;
    u32x4 wd[MATS][RB];
    i32x4 qa[TB][4];
#pragma unroll
    for (int k = 0; k < MATS; ++k)
#pragma unroll
      for (int b = 0; b < RB; ++b)
        wd[k][b] = c < a.nch ? load16(wsrc[k][b] + 16ll * c) : u32x4{kZeroCodes, kZeroCodes, kZeroCodes, kZeroCodes};
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int d = 0; d < 4; ++d) qa[t][d] = load_q16(qsrc[t], 64ll * c + 16 * d, a.K);
#pragma unroll
    for (int k = 0; k < MATS; ++k)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const i32x4 wb = decode16(wd[k][b][d]);
#pragma unroll
          for (int t = 0; t < TB; ++t)
            acc[k][b][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wb, qa[t][d], acc[k][b][t], 0, 0, 0);
        }
  }
  // lane (r, g), register v: row 16 b + 4 g + v, token 16 t + r
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    if (t) __syncthreads();
#pragma unroll
    for (int k = 0; k < MATS; ++k)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[w][((k * RB + b) * 4 + v) * kRedStride + lane] = acc[k][b][t][v];
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * RB * 16; o += 64 * W) {
      const int row = o % (16 * RB), tok = o / (16 * RB);
      const int64_t m = tok0 + 16 * t + tok;
      if (m >= a.M || row0 + row >= a.N) continue;
      int32_t sum[MATS];
#pragma unroll
      for (int k = 0; k < MATS; ++k) {
        sum[k] = 0;
#pragma unroll
        for (int i = 0; i < W; ++i)
          sum[k] += red[i][((k * RB + row / 16) * 4 + row % 4) * kRedStride + 16 * (row % 16 / 4) + tok];
      }
      const int64_t i = row0 + row;
      const float hid = output<MATS>(a, sum, row_ops<MATS>(a, i), load_g(a.z + m), load_g(a.s_act + m));
      store_g(a.y + m * a.ldy + i, a.res ? __fadd_rn(load_g(a.res + m * a.ldr + i), hid) : hid);
    }
  }
}

// ---- many tokens: tiles -----------------------------------------------------

typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

// A workgroup of RG x KS waves computes ROWS rows (of each matrix) x TOK tokens:
// wave (rg, ks) 64 rows (with a gate 32 of each matrix, so that its epilogue stays
// in the lane) x all the tokens over its share of K.  K is walked in stages of
// 128 columns per ks: tokens by DMA into a ring of RING LDS slots, weights
// straight to registers (no other wave of the same ks reads those rows).
template <int MATS, int RG_, int KS_, int TB_, int RING_>
struct Tile {
  static constexpr int RG = RG_, KS = KS_, TB = TB_, RING = RING_;
  static constexpr int WAVES = RG * KS, TOK = 32 * TB, ROWS = 64 * RG / MATS;
  static constexpr int DMA = TOK / 8 / RG;           // DMA instructions of a wave per stage (1 KB each)
  static constexpr int WL = 4;                       // weight loads of a wave per two stages
  static constexpr int SUB = TOK * 128, SLOT = KS * SUB;
  static constexpr int LDS = RING * SLOT > (KS > 1 ? WAVES * TB * 8192 : 0) ? RING * SLOT : WAVES * TB * 8192;
  static_assert(DMA * 8 * RG == TOK && (RING - 2) * DMA + WL < 64 && RING >= 2, "stage split");
};

template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// buffer_rsrc of values that are the same in every lane, in scalar registers.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p), hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
  return buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo), __builtin_amdgcn_readfirstlane(bytes));
}

// swizzle of a token's eight 16-byte pieces of a stage: piece p sits at p ^
// piece_swz(token), so that a 128-bit read of one piece of 8 or 16 tokens touches
// every bank once
__device__ __forceinline__ int piece_swz(int t) { return ((t >> 1) & 7) ^ ((t & 1) << 2); }

template <int MATS, typename S>
__global__ __launch_bounds__(64 * S::WAVES) __attribute__((amdgpu_waves_per_eu(2, 2)))
void epilogue_tile_kernel(EpilogueArgs a, int row_tiles, int tok_tiles) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[S::LDS];
  constexpr int TB = S::TB;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rg = w % S::RG, ks = w / S::RG;
  const int r = lane & 31, h = lane >> 5;
  const int n = gridDim.x;
  const int b = n % 8 == 0 ? (blockIdx.x % 8) * (n / 8) + blockIdx.x / 8 : blockIdx.x;
  const int row0 = (b / tok_tiles) * S::ROWS;
  const int64_t tok0 = (int64_t)(b % tok_tiles) * S::TOK;
  // first rows of the wave's two blocks of 32
  const int rows[2] = {row0 + (MATS == 2 ? 32 * rg : 64 * rg), row0 + (MATS == 2 ? 32 * rg : 64 * rg + 32)};
  __amdgpu_buffer_rsrc_t wres[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int here = min(max(a.N - rows[k], 0), 32);
    const uint8_t* base = a.w[MATS == 2 ? k : 0].packed + (here > 0 ? (int64_t)rows[k] * a.ld : 0);
    wres[k] = uniform_rsrc(base, (uint32_t)here * (uint32_t)a.ld);
  }
  const int toks = (int)min((int64_t)S::TOK, a.M - tok0);
  const uint32_t kbytes = ((uint32_t)a.K + 15) & ~15u;  // (inside ldq)
  const __amdgpu_buffer_rsrc_t qres =
      uniform_rsrc(a.q + tok0 * a.ldq, (uint32_t)((toks - 1) * a.ldq + kbytes));

  const int nst = (a.nch + 2 * S::KS - 1) / (2 * S::KS);  // stages
  // DMA: instruction i brings tokens 8 (DMA rg + i) + lane / 8, lane l the piece
  // that belongs at slot byte 16 l.  Pieces past K, tokens past M: zeros.
  uint32_t qrow[S::DMA], qcol[S::DMA];
#pragma unroll
  for (int i = 0; i < S::DMA; ++i) {
    const int t = 8 * (S::DMA * rg + i) + (lane >> 3);
    qrow[i] = t < toks ? (uint32_t)t * (uint32_t)a.ldq : kDropOffset;
    qcol[i] = 16 * ((lane & 7) ^ piece_swz(t)) + 128 * ks;
  }
  auto issue = [&](int J) {
    uint8_t* dst = lds + (J % S::RING) * S::SLOT + ks * S::SUB + 1024 * S::DMA * rg;
#pragma unroll
    for (int i = 0; i < S::DMA; ++i) {
      const uint32_t col = qcol[i] + 128u * S::KS * (uint32_t)J;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(qres, (lds_ptr_t)(dst + 1024 * i), 16,
                                               (int)(col < kbytes ? qrow[i] + col : kDropOffset), 0, 0, 0);
    }
  };
  // weights of stages 2 c and 2 c + 1: lane (r, h) chunk 2 j + h of row r
  auto load_w = [&](u32x4 (&x)[2][2], int c) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const int chunk = 2 * ((2 * c + st) * S::KS + ks) + h;
        x[st][k] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                 wres[k], (int)((uint32_t)r * (uint32_t)a.ld + 16u * chunk), 0, 0));
      }
  };
  uint32_t tofs[4];  // this lane's piece for operand d of a stage
#pragma unroll
  for (int d = 0; d < 4; ++d) tofs[d] = ks * S::SUB + r * 128 + 16 * ((4 * h + d) ^ piece_swz(r));
  auto load_tok = [&](i32x4 (&x)[TB], int J, int d) {
    const uint8_t* src = lds + (J % S::RING) * S::SLOT + tofs[d];
#pragma unroll
    for (int t = 0; t < TB; ++t) x[t] = *reinterpret_cast<const i32x4*>(src + 4096 * t);
  };
  i32x16 acc[2][TB];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[k][t][v] = 0;
  u32x4 cur[2][2], nxt[2][2];
  i32x4 tok[2][TB], wa[2][2];
  auto multiply = [&](int set) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int t = 0; t < TB; ++t)
        acc[k][t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wa[set][k], tok[set][t], acc[k][t], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2 * TB; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);              // MFMA
      if (i < TB) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
      __builtin_amdgcn_sched_group_barrier(0x002, TB == 4 ? 4 : 7, 0);  // VALU
    }
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int J = 0; J < S::RING; ++J) issue(J);
  load_w(cur, 0);
  wait_vm<0>();
  asm volatile("s_barrier" ::: "memory");
  load_tok(tok[0], 0, 0);
#pragma unroll
  for (int k = 0; k < 2; ++k) wa[0][k] = decode16(cur[0][k][0]);
  for (int c = 0; 2 * c < nst; ++c) {
    load_w(nxt, c + 1);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const int J = 2 * c + st;
#pragma unroll
      for (int d = 0; d < 3; ++d) {
        load_tok(tok[(d + 1) & 1], J, d + 1);
#pragma unroll
        for (int k = 0; k < 2; ++k) wa[(d + 1) & 1][k] = decode16(cur[st][k][d + 1]);
        multiply(d & 1);
      }
      // this wave is done with slot J; stage J + 1 has landed, mine and then everybody's
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      wait_vm<(S::RING - 2) * S::DMA + S::WL>();
      asm volatile("s_barrier" ::: "memory");
      issue(J + S::RING);
      load_tok(tok[0], J + 1, 0);
#pragma unroll
      for (int k = 0; k < 2; ++k) wa[0][k] = decode16(st == 0 ? cur[1][k][0] : nxt[0][k][0]);
      multiply(1);
    }
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int k = 0; k < 2; ++k) cur[st][k] = nxt[st][k];
  }

  // lane (r, h), block k, register 4 q + v: row rows[k] + 8 q + 4 h + v, token 32 t + r.
  // With KS > 1 the ks waves' sums meet in LDS, and each finishes the registers
  // of some q.
  wait_vm<0>();  // (the ring's last DMAs: they must not outlive the workgroup)
  if constexpr (S::KS > 1) {
    __syncthreads();
    i32x4* mine = reinterpret_cast<i32x4*>(lds) + w * TB * 512 + lane;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mine[((k * TB + t) * 4 + q) * 64] =
              i32x4{acc[k][t][4 * q], acc[k][t][4 * q + 1], acc[k][t][4 * q + 2], acc[k][t][4 * q + 3]};
    __syncthreads();
  }
  const bool yvec = (a.ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
  const bool rvec = (a.ldr & 3) == 0 && (reinterpret_cast<uintptr_t>(a.res) & 15) == 0;
  int32_t z[TB];
  float s_act[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const int64_t m = min(tok0 + 32 * t + r, (int64_t)a.M - 1);
    z[t] = load_g(a.z + m);
    s_act[t] = load_g(a.s_act + m);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (S::KS > 1 && q % S::KS != ks) continue;
#pragma unroll
    for (int k = 0; k < (MATS == 2 ? 1 : 2); ++k) {
      const int i0 = rows[k] + 8 * q + 4 * h;
      if (i0 >= a.N) continue;
      RowOps<MATS> ops[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) ops[v] = row_ops<MATS>(a, min(i0 + v, a.N - 1));
      const bool whole = i0 + 3 < a.N;
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const int64_t m = tok0 + 32 * t + r;
        if (m >= a.M) continue;
        i32x4 sum[MATS];
#pragma unroll
        for (int e = 0; e < MATS; ++e) {
          const int blk = MATS == 2 ? e : k;
          if constexpr (S::KS > 1) {
            sum[e] = i32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < S::KS; ++i)
              sum[e] += reinterpret_cast<const i32x4*>(lds)[(i * S::RG + rg) * TB * 512 +
                                                            ((blk * TB + t) * 4 + q) * 64 + lane];
          } else {
            sum[e] = i32x4{acc[blk][t][4 * q], acc[blk][t][4 * q + 1], acc[blk][t][4 * q + 2], acc[blk][t][4 * q + 3]};
          }
        }
        f32x4 res = {0.0f, 0.0f, 0.0f, 0.0f}, o;
        if (a.res) {
          const float* p = a.res + m * a.ldr + i0;
          if (rvec && whole) {
            res = load_g(reinterpret_cast<const f32x4*>(p));
          } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (i0 + v < a.N) res[v] = load_g(p + v);
          }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          int32_t one[MATS];
#pragma unroll
          for (int e = 0; e < MATS; ++e) one[e] = sum[e][v];
          o[v] = output<MATS>(a, one, ops[v], z[t], s_act[t]);
          if (a.res) o[v] = __fadd_rn(res[v], o[v]);
        }
        float* y = a.y + m * a.ldy + i0;
        if (yvec && whole) {
          store_g(reinterpret_cast<f32x4*>(y), o);
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (i0 + v < a.N) store_g(y + v, o[v]);
        }
      }
    }
  }
}

template <int MATS, typename S>
hipError_t launch_tile(const EpilogueArgs& a, hipStream_t s) {
  const int row_tiles = (a.N + S::ROWS - 1) / S::ROWS, tok_tiles = (int)(((int64_t)a.M + S::TOK - 1) / S::TOK);
  hipLaunchKernelGGL((epilogue_tile_kernel<MATS, S>), dim3((unsigned)((int64_t)row_tiles * tok_tiles)),
                     dim3(64 * S::WAVES), 0, s, a, row_tiles, tok_tiles);
  return hipGetLastError();
}

template <int TB, int MATS>
hipError_t launch_rows(const EpilogueArgs& a, hipStream_t s) {
  constexpr int W = 8;
  const int64_t row_tiles = (a.N + 16 * RB - 1) / (16 * RB), tok_tiles = ((int64_t)a.M + 16 * TB - 1) / (16 * TB);
  hipLaunchKernelGGL((epilogue_rows_kernel<W, TB, MATS>), dim3((unsigned)(row_tiles * tok_tiles)), dim3(64 * W), 0, s,
                     a, (int)row_tiles);
  return hipGetLastError();
}

template <int MATS>
hipError_t launch_mats(const EpilogueArgs& a, hipStream_t s) {
  if (a.M <= 16) return launch_rows<1, MATS>(a, s);
  if (a.M <= 32) return launch_rows<2, MATS>(a, s);
  // (the tiles' offsets within a token block are 32-bit)
  if (a.M <= 64 || 128 * a.ldq >= (1ll << 31)) return launch_rows<4, MATS>(a, s);
  if ((int64_t)((a.N * MATS + 255) / 256) * ((a.M + 127) / 128) >= 256) return launch_tile<MATS, Tile<MATS, 4, 1, 4, 4>>(a, s);
  return launch_tile<MATS, Tile<MATS, 2, 4, 2, 4>>(a, s);
}

}  // namespace

int64_t epilogue_work_items(const EpilogueArgs& a) {
  const int64_t row_tiles = ((int64_t)a.N + 16 * RB - 1) / (16 * RB), tb = a.M <= 16 ? 16 : a.M <= 32 ? 32 : 64;
  return mul_sat(mul_sat(row_tiles, ((int64_t)a.M + tb - 1) / tb), 512);
}

hipError_t launch_epilogue(const EpilogueArgs& a, int cus, hipStream_t s) {
  (void)cus;
  return a.w[1].packed ? launch_mats<2>(a, s) : launch_mats<1>(a, s);
}

}  // namespace tern
