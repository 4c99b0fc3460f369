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

// Sixteen weights of a packed dword as signed bytes, negated: code 0, 1, 2 -> +1,
// 0, -1.  v_perm_b32 takes a selector byte 0 .. 3 from its second operand, 4 .. 7
// from its first, and 8 as the sign of the second's byte 1, spread over the byte;
// so the codes at bit 2 (selectors 0, 4, 8) need no shift where the largest code
// stands for a byte of ones: nine operations, eleven for the weights themselves.
__device__ __forceinline__ i32x4 decode16(uint32_t x) {
  i32x4 b;
  const uint32_t hi = x >> 4;
  b[0] = (int32_t)__builtin_amdgcn_perm(0u, 0x00FF0001u, x & 0x03030303u);
  b[1] = (int32_t)__builtin_amdgcn_perm(0u, 0x00008001u, x & 0x0C0C0C0Cu);
  b[2] = (int32_t)__builtin_amdgcn_perm(0u, 0x00FF0001u, hi & 0x03030303u);
  b[3] = (int32_t)__builtin_amdgcn_perm(0u, 0x00008001u, hi & 0x0C0C0C0Cu);
  return b;
}

// silu(x) = x / (1 + e^-x), and gelu in its tanh form, x (1 + tanh(c (x + 0.044715
// x^3))) / 2 with c = sqrt(2 / pi), as x / (1 + e^(-2 c (...))): nothing cancels
// for negative x.
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == 0) return x;
  float t = -x;
  if constexpr (ACT == 2) {
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
    o.bias[k] = a.w[k].bias ? load_g(a.w[k].bias + i) : -0.0f;  // (adding -0 changes nothing)
  }
  return o;
}

// One output from the linears' sums (of negated weights) and the residual (-0: none).
template <int MATS, int ACT>
__device__ __forceinline__ float output(const int32_t (&sum)[MATS], const RowOps<MATS>& o, int32_t z, float s_act,
                                        float res) {
  float v[MATS];
#pragma unroll
  for (int k = 0; k < MATS; ++k) {
    const int32_t acc = (int32_t)(0u - ((uint32_t)sum[k] + mul_zr(z, o.rowsum[k])));
    v[k] = __fadd_rn(epilogue(o.s_row[k], acc, s_act), o.bias[k]);
  }
  float h = activate<ACT>(v[0]);
  if constexpr (MATS == 2) h = __fmul_rn(h, v[1]);
  return __fadd_rn(res, h);
}

// buffer_rsrc of values that are the same in every lane, in scalar registers.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p), hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
  return buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo), __builtin_amdgcn_readfirstlane(bytes));
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

// ---- few tokens: streams of K -------------------------------------------------

typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// LDS accesses of a wave's lanes on both sides stay in this order: the LDS serves a
// wave's instructions as they come, so only the compiler has to be told (no
// instruction comes of it).
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

constexpr int kRedStride = 68;  // of 64 lanes' values of one register, off each other's banks

// The sums of W waves and the epilogue: lane (r, g), register v of a block of
// both holds row 16 b + 4 g + v, token 16 t + r.
template <int W, int RB, int TB, int MATS, int ACT>
__device__ __forceinline__ void join_rows(const EpilogueArgs& a, int row0, int64_t tok0,
                                          const i32x4 (&acc)[MATS][RB][TB], int32_t* red) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  constexpr int BLOCKS = TB * MATS * RB * 4;
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int k = 0; k < MATS; ++k)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          red[(w * BLOCKS + ((t * MATS + k) * RB + b) * 4 + v) * kRedStride + lane] = acc[k][b][t][v];
  __syncthreads();
  for (int o = threadIdx.x; o < 16 * RB * 16 * TB; o += 64 * W) {
    const int row = o % (16 * RB), tok = o / (16 * RB);
    const int64_t m = tok0 + tok;
    if (m >= a.M || row0 + row >= a.N) continue;
    int32_t sum[MATS];
#pragma unroll
    for (int k = 0; k < MATS; ++k) {
      sum[k] = 0;
#pragma unroll
      for (int i = 0; i < W; ++i)
        sum[k] += red[(i * BLOCKS + ((tok / 16 * MATS + k) * RB + row / 16) * 4 + row % 4) * kRedStride +
                      16 * (row % 16 / 4) + tok % 16];
    }
    const int64_t i = row0 + row;
    const float res = a.res ? load_g(a.res + m * a.ldr + i) : -0.0f;
    store_g(a.y + m * a.ldy + i, output<MATS, ACT>(sum, row_ops<MATS>(a, i), load_g(a.z + m), load_g(a.s_act + m), res));
  }
}

// Rows whose K is no multiple of 16 may end inside a piece of 16 bytes, for up to 16
// tokens: 16 rows x 16 tokens to a workgroup of W waves, operands loaded as they lie
// (the columns behind K by the byte).  The weights of the next step are asked for
// behind this step's activations: loads return in order, so before them they would
// be waited for with them.
template <int W, int MATS, int ACT>
__global__ __launch_bounds__(64 * W) void epilogue_rows_kernel(EpilogueArgs a, int row_tiles) {
  __shared__ int32_t red[W * MATS * 4 * kRedStride];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int row0 = (blockIdx.x % row_tiles) * 16;
  const int64_t tok0 = (int64_t)(blockIdx.x / row_tiles) * 16;
  // (rows and chunks past the matrix give zeros: they meet zero activations, or are
  // not stored)
  __amdgpu_buffer_rsrc_t wres[MATS];
#pragma unroll
  for (int k = 0; k < MATS; ++k)
    wres[k] = uniform_rsrc(a.w[k].packed + (int64_t)row0 * a.ld, (uint32_t)min(a.N - row0, 16) * (uint32_t)a.ld);
  const int8_t* q = a.q + min(tok0 + r, (int64_t)a.M - 1) * a.ldq;
  i32x4 acc[MATS][1][1];
#pragma unroll
  for (int k = 0; k < MATS; ++k) acc[k][0][0] = i32x4{0, 0, 0, 0};
  auto load_w = [&](u32x4 (&x)[MATS], int c0) {
#pragma unroll
    for (int k = 0; k < MATS; ++k)
      x[k] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     wres[k], (int)(c0 + g < a.nch ? (uint32_t)r * (uint32_t)a.ld + 16u * (c0 + g) : kDropOffset), 0, 0));
  };
  u32x4 cur[MATS], nxt[MATS];
  load_w(cur, 4 * w);
  for (int c0 = 4 * w; c0 < a.nch; c0 += 4 * W) {
    i32x4 qa[4];
    const int64_t j = 64ll * (c0 + g);
    if (64 * (c0 + 4) <= a.K) {
#pragma unroll
      for (int d = 0; d < 4; ++d) qa[d] = __builtin_bit_cast(i32x4, load16(q + j + 16 * d));
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d) qa[d] = load_q16(q, j + 16 * d, a.K);
    }
    load_w(nxt, c0 + 4 * W);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < MATS; ++k) {
#pragma unroll
      for (int d = 0; d < 4; ++d)
        acc[k][0][0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(decode16(cur[k][d]), qa[d], acc[k][0][0], 0, 0, 0);
      cur[k] = nxt[k];
    }
  }
  join_rows<W, 1, 1, MATS, ACT>(a, row0, tok0, acc, red);
}

// A workgroup's W waves share K (RB blocks of 16 rows of each matrix, TB blocks of
// 16 tokens, a step 256 columns), and until the join of their exact int32 sums
// nothing else: each brings its tokens and weights by DMA to a slot of its own in
// LDS, reads them to registers, asks for the next step's and multiplies, so nobody
// waits for a barrier.  v_mfma_i32_16x16x64_i8 with the weights as A: lane (r, g) has
// the whole 16-byte chunk g of row r, four operands of 64 weights for four
// instructions, and for operand d piece d of block g of token r.  What counts is
// what L1 passes: a load instruction whose neighbouring lanes read different rows
// (the operands as they lie) gets 16 bytes a cycle, one whose four neighbours read
// 64 bytes of one row 58 (measured: 393 KB to each CU in 9.8 and 3.1 us).  So DMA
// instruction c brings 64 columns: lane 4 t + p piece p ^ swz(t) of token t, where
// the operands' reads hardly meet on a bank; weights alike.
//
// Gate and up of 12,288 x 4,096, 25 MB of weights from memory, 1, 8 and 16 tokens: 8.5,
// 8.7 and 10.1 us, of which 2.3 are the launch (operands loaded as they lie 8.1, 10.3,
// 12.3); down, 4,096 x 12,288, 8 and 64 tokens 6.3 and 11.6, with the weights in the
// last-level cache 5.0 and 11.0 (as they lie 7.4 and 17.5 there).  One slot for a wave
// and many workgroups on a CU: 7.8, 8.0 and 8.5 with the weights in the last-level
// cache, with two slots 8.7, 8.9 and 9.6, with three 9.7, 9.8 and 10.3 (not measured
// with the weights from memory).
__device__ __forceinline__ int slot_swz(int row) { return ((row >> 2) & 1) | ((row ^ (row >> 2)) & 2); }

template <int W, int RB, int TB, int MATS, int ACT>
__global__ __launch_bounds__(64 * W) void epilogue_stream_kernel(EpilogueArgs a, int row_tiles) {
  constexpr int P = 4 * TB + MATS * RB;  // DMA instructions (1 KB each) of a step
  constexpr int RED = W * TB * MATS * RB * 4 * kRedStride * 4, SLOTS = W * P * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t lds[SLOTS > RED ? SLOTS : RED];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int row0 = (blockIdx.x % row_tiles) * 16 * RB;
  const int64_t tok0 = (int64_t)(blockIdx.x / row_tiles) * 16 * TB;
  __amdgpu_buffer_rsrc_t wres[MATS];
  const int here = min(a.N - row0, 16 * RB), toks = (int)min((int64_t)16 * TB, a.M - tok0);
#pragma unroll
  for (int k = 0; k < MATS; ++k)
    wres[k] = uniform_rsrc(a.w[k].packed + (int64_t)row0 * a.ld, (uint32_t)here * (uint32_t)a.ld);
  const uint32_t kbytes = ((uint32_t)a.K + 15) & ~15u;  // (inside ldq, or K itself: shape_takes)
  const __amdgpu_buffer_rsrc_t qres =
      uniform_rsrc(a.q + tok0 * a.ldq, (uint32_t)(toks - 1) * (uint32_t)a.ldq + kbytes);
  const int lr = lane >> 2, lp = (lane & 3) ^ slot_swz(lr);
  uint32_t qrow[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) qrow[t] = 16 * t + lr < toks ? (uint32_t)(16 * t + lr) * (uint32_t)a.ldq : kDropOffset;
  uint8_t* mine = lds + w * P * 1024;
  // 256 columns from chunk c0 on; past K: zeros
  auto issue = [&](int c0) {
#pragma unroll
    for (int k = 0; k < MATS; ++k) {
      const __amdgpu_buffer_rsrc_t from = wres[k];
#pragma unroll
      for (int b = 0; b < RB; ++b)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            from, (lds_ptr_t)(mine + (k * RB + b) * 1024), 16,
            (int)(c0 + lp < a.nch ? (uint32_t)(16 * b + lr) * (uint32_t)a.ld + 16u * (c0 + lp) : kDropOffset), 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t col = 64u * (c0 + c) + 16u * lp;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(qres, (lds_ptr_t)(mine + (MATS * RB + 4 * t + c) * 1024), 16,
                                                 (int)(col < kbytes ? qrow[t] + col : kDropOffset), 0, 0, 0);
      }
    __builtin_amdgcn_sched_barrier(0);
  };
  i32x4 acc[MATS][RB][TB];
#pragma unroll
  for (int k = 0; k < MATS; ++k)
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int t = 0; t < TB; ++t) acc[k][b][t] = i32x4{0, 0, 0, 0};
  if (4 * w < a.nch) issue(4 * w);
  for (int c0 = 4 * w; c0 < a.nch; c0 += 4 * W) {
    wait_vm<0>();
    __builtin_amdgcn_sched_barrier(0);
    u32x4 wt[MATS][RB];
    i32x4 qa[TB][4];
#pragma unroll
    for (int k = 0; k < MATS; ++k)
#pragma unroll
      for (int b = 0; b < RB; ++b)
        wt[k][b] = *reinterpret_cast<const u32x4*>(mine + (k * RB + b) * 1024 + 64 * r + 16 * (g ^ slot_swz(r)));
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int d = 0; d < 4; ++d)
        qa[t][d] = *reinterpret_cast<const i32x4*>(mine + (MATS * RB + 4 * t + g) * 1024 + 64 * r + 16 * (d ^ slot_swz(r)));
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the slot has been read
    __builtin_amdgcn_sched_barrier(0);
    if (c0 + 4 * W < a.nch) issue(c0 + 4 * W);
#pragma unroll
    for (int k = 0; k < MATS; ++k)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const i32x4 wb = decode16(wt[k][b][d]);
#pragma unroll
          for (int t = 0; t < TB; ++t)
            acc[k][b][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wb, qa[t][d], acc[k][b][t], 0, 0, 0);
        }
  }
  __syncthreads();  // (slots become sums)
  join_rows<W, RB, TB, MATS, ACT>(a, row0, tok0, acc, reinterpret_cast<int32_t*>(lds));
}

// ---- many tokens: tiles -----------------------------------------------------


// A workgroup of RG x KS waves computes ROWS rows (of each matrix) x TOK tokens:
// wave (rg, ks) 64 rows (with a gate 32 of each matrix, so that its epilogue stays
// in the lane) x all the tokens over its share of K.  K is walked in stages of
// 128 columns per ks: tokens by DMA into a ring of four LDS slots, three stages
// ahead, weights as far ahead straight to registers (no other wave of the same ks
// reads those rows).  v_mfma_i32_32x32x32_i8 with the weights as A: lane (r, h) the
// columns 64 h + 16 d .. of the stage's operand d = 0 .. 3; operands come from LDS
// and are decoded one instruction group ahead.  One barrier per stage, before its
// last operand: it says that the next stage has landed and that the slot of the
// one before is free.
//
// What bounds it, gate and up of 12,288 x 4,096 for 2,048 tokens (412 Gops; a
// library's int8 product of that size alone takes 209 us): 192 us, 184 to 194 on
// different cards, 2.1 POPS (down, 4,096 x 12,288, 96 us and 2.2).  The matrix
// cores are busy in 66 % of each SIMD's cycles, and the card holds 1.5 GHz under
// them: the matrix instructions by themselves take 125 us, with the decode and the
// operands' LDS reads 134, with the loads 150; silu's 49 vector instructions per
// output would take 26 by themselves and overlap with the other workgroup's products
// in part, the 100 MB of y 15.  Two workgroups of four waves to a CU, whose products
// and epilogues fall out of step.  Steps measured: operands from the L2 per 32 tokens
// (no tiles) 740; tiles 220; fixed slots and silu without branches 209; sums
// through LDS to whole lines of y 198 (without a gate 127 -> 99); the products' waves
// ahead of those in an epilogue (s_setprio) 194; decode in nine instructions instead
// of eleven, tiles in groups 187 on that card.  Not kept (no gain): operands two groups ahead,
// weights by 64 bytes of a row and lane swaps (5 % for tiles with K split, whole
// stages lost at small K), priorities by the workgroup's place on its CU; and
// non-temporal stores of y (1 us less here, 9 more for the quantiser that reads y
// next).
template <int MATS, int RG_, int KS_, int TB_>
struct Tile {
  static constexpr int RG = RG_, KS = KS_, TB = TB_, RING = 4;
  static constexpr int WAVES = RG * KS, TOK = 32 * TB, ROWS = 64 * RG / MATS;
  static constexpr int DMA = TOK / 8 / RG;           // DMA instructions of a wave per stage (1 KB each)
  static constexpr int WL = 2;                       // weight loads of a wave per stage
  static constexpr int SUB = TOK * 128, SLOT = KS * SUB;
  static constexpr int LDS = RING * SLOT > (KS > 1 ? WAVES * TB * 8192 : 0) ? RING * SLOT : WAVES * TB * 8192;
  static_assert(DMA * 8 * RG == TOK && 2 * (DMA + WL) < 64, "stage split");
};

// swizzle of a token's eight 16-byte pieces of a stage: piece p sits at p ^
// piece_swz(token), so that a 128-bit read of one piece of 8 or 16 tokens touches
// every bank once
__device__ __forceinline__ int piece_swz(int t) { return ((t >> 1) & 7) ^ ((t & 1) << 2); }

// Tiles are numbered by groups of token tiles, all row tiles of one group before the
// next, and dealt to the XCDs in runs, so that what an XCD works on at a time is
// about as many rows as tokens and stays in its L2 (gate and up of 12,288 x 4,096,
// 8,192 tokens: all token tiles of a row tile together 792 us, by eights 752, by
// fours 747; 2,048 tokens 197, 193, 192).
constexpr int kTokGroup = 4;

template <int MATS, int ACT, typename S>
__global__ __launch_bounds__(64 * S::WAVES) __attribute__((amdgpu_waves_per_eu(2, 2)))
void epilogue_tile_kernel(EpilogueArgs a, int row_tiles, int tok_tiles) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[S::LDS];
  constexpr int TB = S::TB;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rg = w % S::RG, ks = w / S::RG;
  const int r = lane & 31, h = lane >> 5;
  const int n = gridDim.x;
  const int b = n % 8 == 0 ? (blockIdx.x % 8) * (n / 8) + blockIdx.x / 8 : blockIdx.x;
  const int group = b / (row_tiles * kTokGroup), in_group = b - group * row_tiles * kTokGroup;
  const int width = min(kTokGroup, tok_tiles - group * kTokGroup);
  const int row0 = in_group / width * S::ROWS;
  const int64_t tok0 = (int64_t)(group * kTokGroup + in_group % width) * S::TOK;
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
  auto issue = [&](int J, int slot) {
    uint8_t* dst = lds + slot * S::SLOT + ks * S::SUB + 1024 * S::DMA * rg;
#pragma unroll
    for (int i = 0; i < S::DMA; ++i) {
      const uint32_t col = qcol[i] + 128u * S::KS * (uint32_t)J;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(qres, (lds_ptr_t)(dst + 1024 * i), 16,
                                               (int)(col < kbytes ? qrow[i] + col : kDropOffset), 0, 0, 0);
    }
  };
  // weights of stage J: lane (r, h) chunk 2 j + h of row r
  auto load_w = [&](u32x4 (&x)[2], int J) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t chunk = 2 * (J * S::KS + ks) + h;
      x[k] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                           wres[k], (int)((uint32_t)r * (uint32_t)a.ld + 16u * chunk), 0, 0));
    }
  };
  uint32_t tofs[4];  // this lane's piece for operand d of a stage
#pragma unroll
  for (int d = 0; d < 4; ++d) tofs[d] = ks * S::SUB + r * 128 + 16 * ((4 * h + d) ^ piece_swz(r));
  auto load_tok = [&](i32x4 (&x)[TB], int slot, int d) {
#pragma unroll
    for (int t = 0; t < TB; ++t) x[t] = *reinterpret_cast<const i32x4*>(lds + tofs[d] + (slot * S::SLOT + 4096 * t));
  };
  i32x16 acc[2][TB];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[k][t][v] = 0;
  u32x4 wt[4][2];  // weights of stages J .. J + 3, stage j in wt[j % 4]
  i32x4 tok[2][TB], wa[2][2];
  auto multiply = [&](int set) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int t = 0; t < TB; ++t)
        acc[k][t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wa[set][k], tok[set][t], acc[k][t], 0, 0, 0);
    // issue order: the first MFMA, the next operand's LDS reads, then each MFMA
    // followed by a share of the next operand's decode
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
    __builtin_amdgcn_sched_group_barrier(0x100, TB, 0);  // LDS reads
    __builtin_amdgcn_sched_group_barrier(0x002, TB == 4 ? 3 : 5, 0);  // VALU
#pragma unroll
    for (int i = 1; i < 2 * TB; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, TB == 4 ? 3 : 5, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int J = 0; J < 3; ++J) {
    load_w(wt[J], J);
    __builtin_amdgcn_sched_barrier(0);  // (the waits below count the loads in this order)
    issue(J, J);
    __builtin_amdgcn_sched_barrier(0);
  }
  wait_vm<2 * (S::DMA + S::WL)>();  // stage 0
  asm volatile("s_barrier" ::: "memory");
  load_tok(tok[0], 0, 0);
#pragma unroll
  for (int k = 0; k < 2; ++k) wa[0][k] = decode16(wt[0][k][0]);
  // Stage J in slot `slot`.  At its barrier the loads issued behind stage J + 1's
  // DMA are, in order, the weights of J + 2, stage J + 2's DMA and the weights of J +
  // 3: the fences in multiply, and the barrier's, keep them in their places.
  auto stage = [&](int J, int slot) {
    load_w(wt[(slot + 3) % 4], J + 3);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (d == 3) {
        // stage J + 1 has landed, mine and then everybody's; everybody is done with stage J - 1
        wait_vm<S::DMA + 2 * S::WL>();
        asm volatile("s_barrier" ::: "memory");
        issue(J + 3, (slot + 3) % 4);
      }
      load_tok(tok[(d + 1) & 1], (slot + (d + 1) / 4) % 4, (d + 1) & 3);
#pragma unroll
      for (int k = 0; k < 2; ++k) wa[(d + 1) & 1][k] = decode16(wt[(slot + (d + 1) / 4) % 4][k][(d + 1) & 3]);
      multiply(d & 1);
    }
  };
  __builtin_amdgcn_s_setprio(2);
  for (int J = 0; J < nst; J += 4) {
    stage(J, 0);
    stage(J + 1, 1);
    stage(J + 2, 2);
    stage(J + 3, 3);
  }

  // Lane (r, h), block k, register 4 q + v hold row rows[k] + 8 q + 4 h + v of token
  // 32 t + r.  Stored from there, an instruction would write 32 pieces of 32
  // bytes; so the sums go through LDS (one token block at a time, with KS > 1 all
  // of them, where the ks waves' meet) to lanes that hold four rows each of the
  // same token side by side: whole lines of y and of the residual.  The four rows
  // 4 e .. of a block of 32 lie in register group q = e / 2 of half h = e % 2, and
  // there at token r ^ e, off each other's banks.
  constexpr int TC = S::KS > 1 ? TB : 1;       // token blocks in LDS at once
  constexpr int KB = MATS == 2 ? 1 : 2;        // blocks of 32 rows of y
  constexpr int PER = 8 / KB;                  // tokens of an instruction
  constexpr int ITEMS = 32 / PER / (S::KS > 1 ? 2 : 1);  // instructions of a wave and token block
  static_assert(S::KS == 1 || S::KS * ITEMS == TB * 32 / PER, "share of the ks waves");
  i32x4* sums = reinterpret_cast<i32x4*>(lds);
  auto put = [&](int t) {
    i32x4* mine = sums + (w * TC + (S::KS > 1 ? t : 0)) * 512;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mine[(k * 4 + q) * 64 + 32 * h + (r ^ (2 * q + h))] =
            i32x4{acc[k][t][4 * q], acc[k][t][4 * q + 1], acc[k][t][4 * q + 2], acc[k][t][4 * q + 3]};
  };
  const int e = lane & 7, kb = KB == 2 ? (lane >> 3) & 1 : 0;
  const int i0 = rows[kb] + 4 * e;
  const bool whole = i0 + 3 < a.N;
  const bool yvec = whole && (a.ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
  const bool rvec = whole && (a.ldr & 3) == 0 && (reinterpret_cast<uintptr_t>(a.res) & 15) == 0;
  RowOps<MATS> ops[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) ops[v] = row_ops<MATS>(a, min(i0 + v, a.N - 1));
  // token block t, instructions item0 .. of it
  auto finish = [&](int t, int item0) {
    int32_t z[ITEMS];
    float s_act[ITEMS];
    f32x4 res[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int64_t m = tok0 + 32 * t + PER * (item0 + i) + lane / (64 / PER);
      const int64_t mc = min(m, (int64_t)a.M - 1);
      z[i] = load_g(a.z + mc);
      s_act[i] = load_g(a.s_act + mc);
      res[i] = f32x4{-0.0f, -0.0f, -0.0f, -0.0f};
      if (a.res) {
        const float* p = a.res + mc * a.ldr;
        if (rvec) {
          res[i] = load_g(reinterpret_cast<const f32x4*>(p + i0));
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v) res[i][v] = load_g(p + min(i0 + v, a.N - 1));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int token = PER * (item0 + i) + lane / (64 / PER);
      const int64_t m = tok0 + 32 * t + token;
      i32x4 sum[MATS];
#pragma unroll
      for (int n = 0; n < MATS; ++n) {
        sum[n] = i32x4{0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < S::KS; ++p)
          sum[n] += sums[((p * S::RG + rg) * TC + (S::KS > 1 ? t : 0)) * 512 + ((MATS == 2 ? n : kb) * 4 + e / 2) * 64 +
                         32 * (e & 1) + (token ^ e)];
      }
      f32x4 o;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        int32_t one[MATS];
#pragma unroll
        for (int n = 0; n < MATS; ++n) one[n] = sum[n][v];
        o[v] = output<MATS, ACT>(one, ops[v], z[i], s_act[i], res[i][v]);
      }
      if (m >= a.M) continue;
      float* y = a.y + m * a.ldy + i0;
      if (yvec) {
        store_g(reinterpret_cast<f32x4*>(y), o);
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (i0 + v < a.N) store_g(y + v, o[v]);
      }
    }
  };
  __builtin_amdgcn_s_setprio(0);
  wait_vm<0>();  // the ring's last DMAs, mine and then everybody's
  __syncthreads();
  if constexpr (S::KS > 1) {
#pragma unroll
    for (int t = 0; t < TB; ++t) put(t);
    __syncthreads();
    finish(ks * TB / S::KS, ks % 2 * ITEMS);
  } else {
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      // (put writes what other lanes of the wave have read, and they read what it writes)
      wave_order();
      put(t);
      wave_order();
      finish(t, 0);
    }
  }
}

template <int MATS, int ACT, typename S>
hipError_t launch_tile(const EpilogueArgs& a, hipStream_t s) {
  const int row_tiles = (a.N + S::ROWS - 1) / S::ROWS, tok_tiles = (int)(((int64_t)a.M + S::TOK - 1) / S::TOK);
  hipLaunchKernelGGL((epilogue_tile_kernel<MATS, ACT, S>), dim3((unsigned)((int64_t)row_tiles * tok_tiles)),
                     dim3(64 * S::WAVES), 0, s, a, row_tiles, tok_tiles);
  return hipGetLastError();
}

template <int W, int RB, int TB, int MATS, int ACT>
hipError_t launch_stream(const EpilogueArgs& a, hipStream_t s) {
  const int64_t row_tiles = (a.N + 16 * RB - 1) / (16 * RB), tok_tiles = ((int64_t)a.M + 16 * TB - 1) / (16 * TB);
  hipLaunchKernelGGL((epilogue_stream_kernel<W, RB, TB, MATS, ACT>), dim3((unsigned)(row_tiles * tok_tiles)),
                     dim3(64 * W), 0, s, a, (int)row_tiles);
  return hipGetLastError();
}

template <int W, int MATS, int ACT>
hipError_t launch_rows(const EpilogueArgs& a, hipStream_t s) {
  const int64_t row_tiles = (a.N + 15) / 16, tok_tiles = ((int64_t)a.M + 15) / 16;
  hipLaunchKernelGGL((epilogue_rows_kernel<W, MATS, ACT>), dim3((unsigned)(row_tiles * tok_tiles)), dim3(64 * W), 0, s, a,
                     (int)row_tiles);
  return hipGetLastError();
}

// The shapes of a call's workgroups, rows (of both matrices together in the tiles,
// of each otherwise) x tokens, those by estimated time from few tokens to many.
enum Shape { STREAM_16, STREAM_16X32, STREAM_32, SPLIT_64, SPLIT_128, TILE_64, TILE_128, STREAM_WIDE, ROWS, SHAPES };
constexpr int kShapeRows[SHAPES] = {16, 16, 32, 64, 128, 256, 256, 64, 16};
constexpr int kShapeTokens[SHAPES] = {16, 32, 32, 64, 64, 64, 128, 16, 16};
using Split64 = Tile<1, 1, 4, 2>;
template <int MATS>
using Split128 = Tile<MATS, 2, 4, 2>;
template <int MATS>
using Tile64 = Tile<MATS, 4, 1, 2>;
template <int MATS>
using Tile128 = Tile<MATS, 4, 1, 4>;

int64_t shape_workgroups(int shape, const EpilogueArgs& a) {
  const bool tile = shape >= SPLIT_64 && shape <= TILE_128;
  const int64_t rows = kShapeRows[shape] / (tile && a.w[1].packed ? 2 : 1), tokens = kShapeTokens[shape];
  return ((a.N + rows - 1) / rows) * ((a.M + tokens - 1) / tokens);
}

// Whether pick_shape may pick the shape (up to 16 tokens: 16 or 64 rows, or ROWS;
// more: one by estimated time, or ROWS): whether a launch of it can count its threads
// (512 in STREAM_16X32 and SPLIT_128, otherwise more than 256 only where workgroups
// are few) and, but for ROWS, reach its tokens by 32-bit offsets and read them by 16
// bytes: one token's row ends at K (those of 2 to 16 could be read on to ldq, as those
// of more are, but go the same way).
bool shape_takes(int shape, const EpilogueArgs& a) {
  const bool listed = a.M <= 16 ? shape == STREAM_16 || shape == STREAM_WIDE : shape <= TILE_128;
  if (shape != ROWS && (!listed || (a.M > 1 && a.ldq >= (1 << 24)) || (a.M <= 16 && a.K % 16 != 0))) return false;
  if (shape == SPLIT_64 && a.w[1].packed) return false;  // (with a gate never the fastest)
  const int threads = shape == STREAM_16X32 || shape == SPLIT_128 ? 512 : 256;
  return shape_workgroups(shape, a) <= kMaxDispatchItems / threads;
}

// Up to 16 tokens take 16 rows to a workgroup, for the most loads in flight, or 64
// from six such workgroups per CU on, where the activations that each reads are what
// counts (weights from memory, 151,936 x 4,096: 43 and 34.5 us for one token, 67 and 42
// for 16; 32,768 rows, eight per CU: 12.6 and 10.6, 16.3 and 12.0; gate and up of 12,288
// x 12,288, three: 19.3 and 24.7, 26.3 and 26.3).  More tokens take the shape with the least estimated time:
// a start, and for each workgroup that a CU gets in turn a time with a part
// proportional to K, as measured over M = 16 .. 512 and K = 1,024 .. 12,288 (us, for
// 4,096 columns; without a gate, with one).  Both sides of some borders, weights
// from memory (600 MB of them in turn), gate and up of 12,288 x 4,096: 32 tokens in rows
// of 32 14.2, split by 128 16.3; 64: 17.0, 17.5; 96: 22.0, 30.4, tiles of 64 22.6; 128:
// 26.5, 32.6, 23.3; 256: 45, 48, tiles of 128 37.2; 512: tiles of 64 61.9, of 128 61.7;
// 1,024: 115, 102.  4,096 x 12,288 with a residual: 32 tokens in rows of 16 x 32 10.3, of
// 32 12.3; 64: 11.9, split by 128 32.5; 128: 18.5, split by 64 25.0, by 128 31.8; 192: 25.2,
// 25.4, 32.1; 256: 30.1, 25.6, 32.1; 384: 42, 47, 32.6; 512: split by 64 49, by 128 35.6,
// tiles of 64 52, of 128 75.
Shape pick_shape(const EpilogueArgs& a, int cus) {
  static constexpr double kStart[2][7] = {{3.3, 3.6, 3.3, 3, 2, 4, 2}, {3.3, 3.6, 5, 0, 2, 4, 2}};
  static constexpr double kEach[2][7] = {{0.2, 0.4, 0.1, 4, 6.5, 5.5, 9}, {0.2, 0.4, 0.6, 0, 6.5, 5.5, 9}};
  static constexpr double kTime[2][7] = {{0.95, 1.75, 2.45, 6.4, 8, 12.4, 21}, {1.2, 2.8, 2.75, 0, 9, 13.5, 24.5}};
  if (a.M <= 16) {
    const bool wide = shape_workgroups(STREAM_16, a) >= 6ll * cus || !shape_takes(STREAM_16, a);
    if (wide && shape_takes(STREAM_WIDE, a)) return STREAM_WIDE;
    return shape_takes(STREAM_16, a) ? STREAM_16 : ROWS;
  }
  const int gated = a.w[1].packed != nullptr;
  int best = ROWS;
  double least = 0;
  for (int s = STREAM_16; s <= TILE_128; ++s) {
    if (!shape_takes(s, a)) continue;
    const double turns = (double)((shape_workgroups(s, a) + cus - 1) / cus);
    const double t = kStart[gated][s] + turns * (kEach[gated][s] + kTime[gated][s] * a.K / 4096);
    if (best == ROWS || t < least) best = s, least = t;
  }
  return (Shape)best;
}

// More waves for a workgroup where workgroups are few, weights from memory: 16 rows
// from three steps of four waves on eight (4,096 x 4,096, one token: 3.8 us, four 4.6),
// from three of eight on sixteen (4,096 x 12,288: four 10.9, eight 7.3, sixteen 5.9, and
// for 16 tokens 10.9, 7.6, 8.3; gate and up of 1,024 x 1,024: 3.3, 3.2, 3.4; where a CU
// gets three, gate and up of 12,288 x 4,096, 8.5, 8.9, 12.3); 32 rows (4,096 x 12,288, 64
// tokens: 13.4, eight 11.7; 6,144 x 1,024: 4.5, 4.6; where a CU gets three, gate and up of
// 12,288 x 4,096, 17.5 and 21.5); ROWS as measured there (4,096 x 12,288 in the
// last-level cache: 8.1, eight 6.2; with two workgroups per CU 8.5, 8.9).
template <int MATS, int ACT>
hipError_t launch_act(const EpilogueArgs& a, int cus, hipStream_t s) {
  const Shape shape = pick_shape(a, cus);
  const int64_t n = shape_workgroups(shape, a);
  const bool few = n < 2ll * cus, fewer = n <= cus;
  const int steps = (a.nch + 3) / 4;
  switch (shape) {
    case STREAM_16:
      if (fewer && steps > 24) return launch_stream<16, 1, 1, MATS, ACT>(a, s);
      return few && steps > 12 ? launch_stream<8, 1, 1, MATS, ACT>(a, s) : launch_stream<4, 1, 1, MATS, ACT>(a, s);
    case STREAM_16X32: return launch_stream<8, 1, 2, MATS, ACT>(a, s);
    case STREAM_32:
      return fewer && steps > 12 ? launch_stream<8, 2, 2, MATS, ACT>(a, s) : launch_stream<4, 2, 2, MATS, ACT>(a, s);
    case SPLIT_64:
      if constexpr (MATS == 1) return launch_tile<MATS, ACT, Split64>(a, s);
      return hipErrorInvalidValue;  // (not taken with a gate)
    case SPLIT_128: return launch_tile<MATS, ACT, Split128<MATS>>(a, s);
    case TILE_64: return launch_tile<MATS, ACT, Tile64<MATS>>(a, s);
    case TILE_128: return launch_tile<MATS, ACT, Tile128<MATS>>(a, s);
    case STREAM_WIDE: return launch_stream<4, 4, 1, MATS, ACT>(a, s);
    default: return few ? launch_rows<8, MATS, ACT>(a, s) : launch_rows<4, MATS, ACT>(a, s);
  }
}

template <int MATS>
hipError_t launch_mats(const EpilogueArgs& a, int cus, hipStream_t s) {
  if (a.act == 0) return launch_act<MATS, 0>(a, cus, s);
  return a.act == 1 ? launch_act<MATS, 1>(a, cus, s) : launch_act<MATS, 2>(a, cus, s);
}

}  // namespace

bool epilogue_takes(const EpilogueArgs& a) {
  if (a.N > INT32_MAX - 255) return false;  // (rows are int32 as far as the last tile of 256 reaches)
  bool any = false;
  for (int s = STREAM_16; s < SHAPES; ++s) any = any || shape_takes(s, a);
  return any;
}

hipError_t launch_epilogue(const EpilogueArgs& a, int cus, hipStream_t s) {
  return a.w[1].packed ? launch_mats<2>(a, cus, s) : launch_mats<1>(a, cus, s);
}

}  // namespace tern
