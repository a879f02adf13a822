// Linear layer of many requests at once, each row with a low-rank adapter of its own
// choice beside the shared weight:
//   out[m] = epi(W x[m] + bias + s_a B_a (A_a x[m])),   a = index[m]
// (rows whose index names no adapter: without the last term).  x [M][K], W [N][K],
// A [L][R][K], B [L][N][R] bf16, fp32 scales, bf16 output, one rounding.
//
// lora_shrink leaves A_a x[m] in fp32, in slices of K.  Few rows (a decode step): bound by
// reading W once; lora_rows streams it and adds B (s_a A_a x[m]) to the same sums.
// Many rows: lora_tile takes the adapters' terms as further steps of K; where K is
// cut into slices, lora_join adds them.
// v = s_a A_a x, fp32, enters the products with B as three bf16 numbers whose sum it is: as one, its
// rounding would be as large as the output's own, as two (16 bits of significand) up to 2^-16 of v would be lost.
#pragma once

#include <type_traits>

#include "moe_ffn.hpp"
#include "rms_norm.hpp"

namespace mmk {

constexpr int kLoraWaves = 16, kLoraShrinkWaves = 8;
constexpr int kLoraMaxRank = 256;

struct LoraParams {
  const uint16_t* x;      // [M][K]
  const uint16_t* W;      // [N][K]
  const uint16_t* A;      // [L][R][K]
  const uint16_t* B;      // [L][N][R]
  const int* index;       // [M]
  const float* scale;     // [L]
  const uint16_t* bias;   // [N] or null
  uint16_t* out;          // [M][N]
  float* low;             // [low_slices][M][R]: parts of A x
  uint16_t* v;            // [M][3][R]: s A x, its parts
  float* acc;             // [slices][M][N]: parts of W x
  int M, N, K, R, L;
  int low_slices, low_k;  // slices of K of low_k (a multiple of 64)
  int slices;             // of acc
  int epi;
  int tiles_m, tiles_n;   // lora_tile: tiles, K in `slices` pieces of slice_steps super-steps
  int slice_steps;
  const struct LoraTileRows* tiles;  // [tiles_m]
};

// The adapters that a tile's rows (at most 256) have, in the order of their first rows,
// and which rows.
struct LoraTileRows {
  int count;
  int adapter[256];
  uint64_t rows[256][4];
};

// Super-steps of 64 values of lora_tile that the parts of an adapter of rank R take.
__device__ __forceinline__ int lora_steps(int R) { return (3 * R + 63) >> 6; }

// The adapter of row `row`, -1 for none (past the last row, or an index that names none).
__device__ __forceinline__ int lora_adapter(const LoraParams& p, int row) {
  if (row >= p.M) return -1;
  const int a = p.index[row];
  return (unsigned)a < (unsigned)p.L ? a : -1;
}

// The signs' places of a word's two bf16 set where the value is an infinity or a NaN: its exponent of ones
// carries into that place.
__device__ __forceinline__ uint32_t odd_halves(uint32_t u) { return ((u & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// The terms of chunk c (8 ranks) of B v added to `sum`; v: the row's parts [3][stride].  ODD: those only whose
// value of B is not finite.
template <bool ODD>
__device__ __forceinline__ float lora_terms(float sum, u32x4 w, const uint16_t* v, int stride, int c) {
  u32x4 part[3];
#pragma unroll
  for (int h = 0; h < 3; ++h) part[h] = *reinterpret_cast<const u32x4*>(v + h * stride + 8 * c);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    auto at = [&](const u32x4& u) { return bf16_float((uint16_t)(u[j >> 1] >> (16 * (j & 1)))); };
    if (ODD && !(odd_halves(w[j >> 1]) >> (16 * (j & 1)) & 0x8000u)) continue;
    sum = __builtin_fmaf(at(part[0]) + at(part[1]) + at(part[2]), at(w), sum);
  }
  return sum;
}

// B v of row m and column n, term by term, for sums that came out NaN: of the three parts of a v, 8 bits
// or less leave some 0, and 0 times an infinity of B is NaN where v times it is infinite.  CHUNKS: 8 ranks at a
// time (lora_rows has no registers for them).
template <bool CHUNKS>
__device__ __forceinline__ float lora_term(const LoraParams& p, int m, int n, const uint16_t* v, int stride) {
  const uint16_t* b = p.B + ((int64_t)lora_adapter(p, m) * p.N + n) * p.R;
  float sum = 0.f;
  if constexpr (CHUNKS) {
#pragma unroll 1
    for (int c = 0; c < p.R >> 3 && sum == sum; ++c)
      sum = lora_terms<false>(sum, *reinterpret_cast<const u32x4*>(b + 8 * c), v, stride, c);
  } else {
#pragma unroll 1
    for (int r = 0; r < p.R && sum == sum; ++r)
      sum = __builtin_fmaf(bf16_float(v[r]) + bf16_float(v[stride + r]) + bf16_float(v[2 * stride + r]), bf16_float(b[r]), sum);
  }
  return sum;
}

// Calls f(adapter, its lanes) for every different adapter >= 0 among a wave's lanes, in
// the order of their first lanes.
template <typename F>
__device__ __forceinline__ void each_adapter(int mine, F f) {
  uint64_t left = __ballot(mine >= 0);
  while (left) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    const uint64_t same = __ballot(mine == a);
    left &= ~same;
    f(a, same);
  }
}

// `rows` rows of an operand [rows][K] of bf16 from `base` as a buffer: zeros past the end.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const uint16_t* base, int rows, int K) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), (short)0, rows * K * 2, 0x00020000);
}

// The same rows from value `from` of the first on: the last ends where the operand's does.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t slice_buffer(const uint16_t* base, int rows, int K, int from) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), (short)0, (rows * K - from) * 2, 0x00020000);
}

// A x of the rows 16 MB y .. + 16 MB - 1 over slice x of K, for 16 RB ranks; of the
// adapters among the rows, every turns-th (blockIdx.z: ranks and turn).  The waves take every
// eighth step of 64 k, each step's loads one step ahead, and meet in LDS, added in wave
// order.  A CU by itself reads some 25 bytes per ns, so the slices, adapters and ranks
// of few rows go to many (one token, rank 16, K 8192: 4.0 us in 16 slices, 12 in one).
// Few rows: latency (16 rows of as many adapters 5.1 us, 3 MB).  Prompts: a read of x, 8192 x
// 8192 for rank 16 35 us, 3.8 TB/s.
// TURN: loaded eight lanes to a row (to_fragments): 8192 x 8192 for rank 16 43 us without, 35 with it;
// but rows of other adapters are left out, and where those are most, the MFMA's order touches few
// lines: 64 rows of 64 adapters 9.0 us without, 13.8 with it.
template <int MB, int RB, bool TURN>
__global__ void __launch_bounds__(kLoraShrinkWaves * 64) lora_shrink(LoraParams p, int turns) {
  __shared__ f32x4 red[kLoraShrinkWaves][MB * RB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  // row and chunk of a block's load j, and its two as fragments
  auto row = [&](int j) __attribute__((always_inline)) { return TURN ? 8 * j + (lane >> 3) : lx; };
  auto chunk = [&](int j) __attribute__((always_inline)) { return TURN ? lane & 7 : 4 * j + lg; };
  auto turn = [&](u32x4(&v)[2]) __attribute__((always_inline)) {
    if constexpr (TURN) to_fragments(v, red[wave][0], lane);  // (free during the products)
  };
  const int m0 = blockIdx.y * (16 * MB), rows = min(16 * MB, p.M - m0);
  const int r0 = (int)(blockIdx.z / turns) * (16 * RB), my_turn = blockIdx.z % turns;
  const int K = p.K, kbeg = blockIdx.x * p.low_k, klen = min(p.low_k, K - kbeg), steps = (klen + 63) >> 6;
  // (of a slice of a row the buffer ends where the last row's does)
  const __amdgpu_buffer_rsrc_t rx = slice_buffer(p.x + (int64_t)m0 * K + kbeg, rows, K, kbeg);
  struct Step {
    u32x4 w[RB][2], x[MB][2];
  };
  int nth = 0;
  each_adapter(lane < rows ? lora_adapter(p, m0 + lane) : -1, [&](int a, uint64_t same) {
    if (nth++ % turns != my_turn) return;
    const __amdgpu_buffer_rsrc_t rw =
        slice_buffer(p.A + ((int64_t)a * p.R + r0) * K + kbeg, min(16 * RB, p.R - r0), K, kbeg);
    uint32_t xrow[MB][2];  // (rows of other adapters are not loaded)
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int m = 16 * b + row(j);
        xrow[b][j] = (same >> m) & 1 ? (uint32_t)m * (uint32_t)K * 2u : 0x80000000u;
      }
    auto load = [&](int st, Step& t) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int c = 0; c < RB; ++c)
          t.w[c][j] = step_chunk(rw, (uint32_t)(16 * c + row(j)) * (uint32_t)K * 2u, st, chunk(j), klen, steps);
#pragma unroll
        for (int b = 0; b < MB; ++b) t.x[b][j] = step_chunk(rx, xrow[b][j], st, chunk(j), klen, steps);
      }
    };
    f32x4 acc[MB][RB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < RB; ++c) acc[b][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int st, Step& t, Step& next) __attribute__((always_inline)) {
      load(st + kLoraShrinkWaves, next);
#pragma unroll
      for (int c = 0; c < RB; ++c) turn(t.w[c]);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        turn(t.x[b]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < RB; ++c) acc[b][c] = mfma_bf16(t.x[b][j], t.w[c][j], acc[b][c]);
      }
    };
    __syncthreads();  // (what was in LDS before has been read)
    Step s0, s1;
    load(wave, s0);
    for (int st = wave; st < steps; st += 2 * kLoraShrinkWaves) {
      step(st, s0, s1);
      step(st + kLoraShrinkWaves, s1, s0);
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < RB; ++c) red[wave][b * RB + c][lane] = acc[b][c];
    __syncthreads();
    for (int i = wave; i < MB * RB; i += kLoraShrinkWaves) {
      f32x4 s = red[0][i][lane];
#pragma unroll
      for (int q = 1; q < kLoraShrinkWaves; ++q) {
        const f32x4 u = red[q][i][lane];
#pragma unroll
        for (int f = 0; f < 4; ++f) s[f] += u[f];
      }
      const int r = r0 + 16 * (i % RB) + lx;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int m = 16 * (i / RB) + 4 * lg + f;
        if (r < p.R && ((same >> m) & 1)) p.low[((int64_t)blockIdx.x * p.M + m0 + m) * p.R + r] = s[f];
      }
    }
  });
}

// v of every row, 8 ranks (a chunk) to 16 threads: each loads the sums of one slice, and their sum
// times the scale goes in its parts to put(row, chunk, parts).  Rows without an
// adapter are left out.
template <typename F>
__device__ __forceinline__ void lora_fold_all(const LoraParams& p, int64_t thread, int64_t threads, F put) {
  const int chunks = p.R >> 3, s = (int)(thread & 15);
  for (int64_t i = thread; i < (int64_t)p.M * chunks * 16; i += threads) {
    const int m = (int)((i >> 4) / chunks), c = (int)((i >> 4) - (int64_t)m * chunks);
    const int a = lora_adapter(p, m);
    f32x4 v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (s < p.low_slices) {
      const float* at = p.low + ((int64_t)s * p.M + m) * p.R + 8 * c;
      v[0] = *reinterpret_cast<const f32x4*>(at);
      v[1] = *reinterpret_cast<const f32x4*>(at + 4);
    }
#pragma unroll
    for (int d = 1; d < 16; d <<= 1)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j >> 2][j & 3] += __shfl_xor(v[j >> 2][j & 3], d);
    if (a < 0 || s > 0) continue;
    const float scale = p.scale[a];
    u32x4 part[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      split_bf16(v[j >> 1][2 * (j & 1)] * scale, [&](int h, uint16_t u) { part[h][j] = u; });
      split_bf16(v[j >> 1][2 * (j & 1) + 1] * scale, [&](int h, uint16_t u) { part[h][j] |= (uint32_t)u << 16; });
    }
    put(m, c, part);
  }
}
__device__ __forceinline__ void lora_fold_all(const LoraParams& p, int64_t thread, int64_t threads) {
  lora_fold_all(p, thread, threads, [&](int m, int c, const u32x4(&part)[3]) {
#pragma unroll
    for (int h = 0; h < 3; ++h) *reinterpret_cast<u32x4*>(p.v + ((int64_t)m * 3 + h) * p.R + 8 * c) = part[h];
  });
}

// v of every row, and the adapters of every tile of `bm` rows (0: not needed), which the first
// workgroups find.
__global__ void __launch_bounds__(256) lora_fold(LoraParams p, LoraTileRows* tiles, int bm) {
  const int finders = bm ? p.tiles_m : 0;
  if ((int)blockIdx.x >= finders) {
    lora_fold_all(p, (int64_t)(blockIdx.x - finders) * 256 + threadIdx.x, (int64_t)(gridDim.x - finders) * 256);
    return;
  }
  // one wave, four rows to a lane
  if (threadIdx.x >= 64) return;
  const int lane = threadIdx.x;
  LoraTileRows* t = tiles + blockIdx.x;
  int mine[4];
  uint64_t left[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    mine[g] = 64 * g < bm ? lora_adapter(p, (int)blockIdx.x * bm + 64 * g + lane) : -1;
    left[g] = __ballot(mine[g] >= 0);
  }
  int count = 0;
  while (left[0] | left[1] | left[2] | left[3]) {
    int a = -1;
#pragma unroll
    for (int g = 3; g >= 0; --g)
      if (left[g]) a = __builtin_amdgcn_readlane(mine[g], __builtin_ctzll(left[g]));
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint64_t same = __ballot(mine[g] == a);
      left[g] &= ~same;
      if (lane == g) t->rows[count][g] = same;
    }
    if (lane == 0) t->adapter[count] = a;
    ++count;
  }
  if (lane == 0) t->count = count;
}

// Up to 16 MB rows.  A workgroup takes a slice y of K, 16 SPW steps of 64 k, and every
// gridDim.x-th block of 16 columns.  Wave w has the slice's steps 16 i + w, i < SPW, and
// holds x there in registers for all blocks, so that W is all that it loads; each
// step's loads are issued one step ahead, across blocks.  The waves' sums of a block meet
// in LDS (two sets in turn: one barrier per block) and are added in wave order, by
// another wave for each block.
// FINISH (K in one slice): v comes into LDS first, each adapter's terms are made by a
// wave and added to the rows' sums after those of W x (so that no row's rounding depends on which wave that is,
// and with it on other rows' adapters), and the output is written.  Else lora_join_few does both,
// and v is left in memory for it.
// Bound by reading W: 16 x 28672 x 8192 96 us (4.9 TB/s), 1 x 8192 x 8192 25 (5.4), 64 x 14336 x
// 4096 26 (4.5, and 7 MB of parts).  With x read from L2 for every block the first took 150; with x
// and W loaded in the MFMA's order (see to_fragments) 99, 25 and 32.
template <int MB, int SPW, bool FINISH>
__global__ void __launch_bounds__(kLoraWaves * 64) lora_rows(LoraParams p) {
  static_assert(SPW % 2 == 0 && MB * SPW <= 8, "x in 64 registers, two steps in turn");
  __shared__ f32x4 red[2][kLoraWaves][MB][64];
  __shared__ f32x4 turn[kLoraWaves][128];
  __shared__ u32x4 v[FINISH ? 16 * MB : 1][3][kLoraMaxRank / 8];
  __shared__ f32x4 term[2][FINISH ? MB : 1][64];  // B v of rows with an adapter, in the order of red
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int lr = lane >> 3, lk = lane & 7;  // of what is loaded (to_fragments)
  const int K = p.K, steps = (K + 63) >> 6, blocks = (p.N + 15) >> 4;
  const int first = blockIdx.y * (kLoraWaves * SPW) + wave;

  struct Step {
    u32x4 w[2];
  };
  uint32_t row = (uint32_t)lr * (uint32_t)K * 2u;
  auto load = [&](int block, int i, Step& t) __attribute__((always_inline)) {
    // (opaque: the steps' offsets are not all kept in registers)
    asm volatile("" : "+v"(row));
    // (past the last block, that one again, unused)
    const int n0 = 16 * min(block, blocks - 1);
    const __amdgpu_buffer_rsrc_t rw = rows_buffer(p.W + (int64_t)n0 * K, min(16, p.N - n0), K);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      t.w[j] = step_chunk(rw, row + (uint32_t)(16 * j) * (uint32_t)K, first + kLoraWaves * i, lk, K, steps);
  };
  Step t[2];
  load(blockIdx.x, 0, t[0]);
  u32x4 x[MB][SPW][2];
  {
    const __amdgpu_buffer_rsrc_t rx = rows_buffer(p.x, p.M, K);
#pragma unroll
    for (int i = 0; i < SPW; ++i)
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          x[b][i][j] = step_chunk(rx, (uint32_t)(16 * b + 8 * j + lr) * (uint32_t)K * 2u, first + kLoraWaves * i, lk, K, steps);
#pragma unroll
    for (int i = 0; i < SPW; ++i)
#pragma unroll
      for (int b = 0; b < MB; ++b) to_fragments(x[b][i], turn[wave], lane);
  }
  // this wave's adapters (of at most 16 MB) and their rows
  int mine[MB];
  uint64_t same[MB], adapted = 0;  // (adapted: all rows with an adapter)
#pragma unroll
  for (int q = 0; q < MB; ++q) {
    mine[q] = -1;
    same[q] = 0;
  }
  if constexpr (FINISH) {
    int nth = 0;
    each_adapter(lora_adapter(p, lane), [&](int a, uint64_t s) {
      adapted |= s;
#pragma unroll
      for (int q = 0; q < MB; ++q) {
        if (nth == kLoraWaves * q + wave) {
          mine[q] = a;
          same[q] = s;
        }
      }
      ++nth;
    });
    lora_fold_all(p, threadIdx.x, kLoraWaves * 64, [&](int m, int c, const u32x4(&part)[3]) {
#pragma unroll
      for (int h = 0; h < 3; ++h) v[m][h][c] = part[h];
    });
  } else {
    lora_fold_all(p, (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * (kLoraWaves * 64) + threadIdx.x,
                  (int64_t)gridDim.x * gridDim.y * (kLoraWaves * 64));
  }

  int round = 0;
  for (int block = blockIdx.x; block < blocks; block += gridDim.x, ++round) {
    const int n0 = 16 * block;
    f32x4 acc[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < SPW; ++i) {
      if (i + 1 < SPW)
        load(block, i + 1, t[(i + 1) & 1]);
      else
        load(block + gridDim.x, 0, t[0]);
      u32x4(&w)[2] = t[i & 1].w;
      to_fragments(w, turn[wave], lane);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[b] = mfma_bf16(x[b][i][j], w[j], acc[b]);
    }
    if (FINISH && round == 0) __syncthreads();  // (v is there)
#pragma unroll
    for (int q = 0; q < MB; ++q) {
      if (!FINISH || mine[q] < 0) continue;
      const uint16_t* bw = p.B + ((int64_t)mine[q] * p.N + min(n0 + lx, p.N - 1)) * p.R;
      f32x4 d[MB];
#pragma unroll
      for (int b = 0; b < MB; ++b) d[b] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int r0 = 0; r0 < p.R; r0 += 32) {
        const int r = r0 + 8 * lg;
        u32x4 wf = {0u, 0u, 0u, 0u};
        if (r < p.R) wf = *reinterpret_cast<const u32x4*>(bw + r);
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          if (!((same[q] >> (16 * b)) & 0xffff)) continue;
          const bool have = r < p.R && ((same[q] >> (16 * b + lx)) & 1);
#pragma unroll
          for (int h = 0; h < 3; ++h) {
            u32x4 part = {0u, 0u, 0u, 0u};
            if (have) part = v[16 * b + lx][h][r >> 3];
            d[b] = mfma_bf16(part, wf, d[b]);
          }
        }
      }
      // (its rows only: 0 times what is not finite leaves other rows alone)
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        float* to = reinterpret_cast<float*>(&term[round & 1][b][lane]);
#pragma unroll
        for (int f = 0; f < 4; ++f)
          if ((same[q] >> (16 * b + 4 * lg + f)) & 1) to[f] = d[b][f];
      }
    }
    f32x4(*set)[MB][64] = red[round & 1];
#pragma unroll
    for (int b = 0; b < MB; ++b) set[wave][b][lane] = acc[b];
    __syncthreads();
    const int b = (wave - round * MB) & (kLoraWaves - 1);
    if (b >= MB) continue;
    f32x4 s = set[0][b][lane];
#pragma unroll 5
    for (int q = 1; q < kLoraWaves; ++q) {
      const f32x4 u = set[q][b][lane];
#pragma unroll
      for (int f = 0; f < 4; ++f) s[f] += u[f];
    }
    const int n = n0 + lx;
    if (n >= p.N) continue;
    if constexpr (FINISH) {
      f32x4 d = term[round & 1][b][lane];
      bool again = false;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        if (!((adapted >> (16 * b + 4 * lg + f)) & 1)) d[f] = 0.f;
        again |= d[f] != d[f] && s[f] == s[f];
      }
      if (again) {
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int m = 16 * b + 4 * lg + f;
          if (d[f] != d[f]) d[f] = lora_term<false>(p, m, n, reinterpret_cast<const uint16_t*>(v[m]), kLoraMaxRank);
        }
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) s[f] += d[f];
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int m = 16 * b + 4 * lg + f;
      if (m >= p.M) continue;
      if constexpr (FINISH)
        p.out[(int64_t)m * p.N + n] = decoder_epilogue(s[f], p.bias, p.epi, n);
      else
        p.acc[((int64_t)blockIdx.y * p.M + m) * p.N + n] = s[f];
    }
  }
}

// out = epi(sum of acc's slices + bias + B v): 64 rows by 64 columns per workgroup, 16
// rows per wave.  B is the MFMA's first operand, so a lane's sums are of one row;
// the block pair's rows of B are taken in the order that makes them 8 consecutive columns.
// Bound by the parts' bytes: 512 x 4096 in 2 slices 6.2 us.
__global__ void __launch_bounds__(256) lora_join(LoraParams p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int m0 = blockIdx.y * 64 + 16 * wave, n0 = blockIdx.x * 64;
  if (m0 >= p.M) return;
  const int m = m0 + lx;
  f32x4 acc[2][2], term[2][2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int n = n0 + 32 * c + 8 * lg;
    const float* at = p.acc + (int64_t)min(m, p.M - 1) * p.N;
    acc[c][0] = acc[c][1] = term[c][0] = term[c][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < p.slices; ++s, at += (int64_t)p.M * p.N) {
      f32x4 u[2];
      if (n + 8 <= p.N) {
        __builtin_memcpy(&u[0], at + n, 16);
        __builtin_memcpy(&u[1], at + n + 4, 16);
      } else {
#pragma unroll
        for (int f = 0; f < 8; ++f) u[f >> 2][f & 3] = at[min(n + f, p.N - 1)];
      }
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[c][f >> 2][f & 3] += u[f >> 2][f & 3];
    }
  }
  each_adapter(lane < 16 ? lora_adapter(p, m0 + lane) : -1, [&](int a, uint64_t same) {
    const bool mine = (same >> lx) & 1;
    for (int r0 = 0; r0 < p.R; r0 += 32) {
      const int r = r0 + 8 * lg;
      u32x4 wf[2][2], part[3];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = min(n0 + 32 * c + 8 * (lx >> 2) + 4 * h + (lx & 3), p.N - 1);
          wf[c][h] = u32x4{0u, 0u, 0u, 0u};
          if (r < p.R) wf[c][h] = *reinterpret_cast<const u32x4*>(p.B + ((int64_t)a * p.N + n) * p.R + r);
        }
      }
#pragma unroll
      for (int h = 0; h < 3; ++h) {
        part[h] = u32x4{0u, 0u, 0u, 0u};
        if (r < p.R && mine) part[h] = *reinterpret_cast<const u32x4*>(p.v + ((int64_t)m * 3 + h) * p.R + r);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 3; ++i) d = mfma_bf16(wf[c][h], part[i], d);
          // (0 times what is not finite: other rows' sums are left alone)
#pragma unroll
          for (int f = 0; f < 4; ++f) term[c][h][f] += mine ? d[f] : 0.f;
        }
      }
    }
  });
  if (m >= p.M) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = i >> 3, h = (i >> 2) & 1, f = i & 3, n = n0 + 32 * c + 8 * lg + 4 * h + f;
    if (term[c][h][f] != term[c][h][f] && acc[c][h][f] == acc[c][h][f] && n < p.N)
      term[c][h][f] = lora_term<true>(p, m, n, p.v + (int64_t)m * 3 * p.R, p.R);
    acc[c][h][f] += term[c][h][f];
  }
  const bool has_bias = p.epi == EPI_BIAS || p.epi == EPI_BIAS_GELU;
  const bool gelu = p.epi == EPI_GELU || p.epi == EPI_BIAS_GELU;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int n = n0 + 32 * c + 8 * lg;
    float v[8];
#pragma unroll
    for (int f = 0; f < 8; ++f) v[f] = acc[c][f >> 2][f & 3] + (has_bias ? bf16_float(p.bias[min(n + f, p.N - 1)]) : 0.f);
    if (gelu) gelu_tanh_all(v);
    uint16_t* o = p.out + (int64_t)m * p.N + n;
    if (n + 8 <= p.N) {
      const u32x4 pk = pack8(v);
      __builtin_memcpy(o, &pk, 16);
    } else {
#pragma unroll
      for (int f = 0; f < 8; ++f)
        if (n + f < p.N) o[f] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[f]));
    }
  }
}

// The same for 16 MB rows by 64 columns, which may have as many adapters as there are rows: the eight waves share these, and meet in LDS, where each finishes some
// blocks of 16 by 16.  64 x 14336, rank 64, 8 adapters 11.5 us, 24 MB (2.1 TB/s): one chain of
// index, v and B, sums and parts per workgroup.
template <int MB>
__global__ void __launch_bounds__(512) lora_join_few(LoraParams p) {
  __shared__ f32x4 red[8][MB * 4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int m0 = blockIdx.y * (16 * MB), n0 = blockIdx.x * 64;
  f32x4 acc[MB][4];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[b][q] = f32x4{0.f, 0.f, 0.f, 0.f};
  int turn = 0;
  each_adapter(lane < 16 * MB ? lora_adapter(p, m0 + lane) : -1, [&](int a, uint64_t same) {
    if ((turn++ & 7) != wave) return;
#pragma unroll 2
    for (int r0 = 0; r0 < p.R; r0 += 32) {
      const int r = r0 + 8 * lg;
      u32x4 wf[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = min(n0 + 32 * (q >> 1) + 8 * (lx >> 2) + 4 * (q & 1) + (lx & 3), p.N - 1);
        wf[q] = u32x4{0u, 0u, 0u, 0u};
        if (r < p.R) wf[q] = *reinterpret_cast<const u32x4*>(p.B + ((int64_t)a * p.N + row) * p.R + r);
      }
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        if (!((same >> (16 * b)) & 0xffff)) continue;
        const bool mine = (same >> (16 * b + lx)) & 1;
        u32x4 part[3];
#pragma unroll
        for (int h = 0; h < 3; ++h) {
          part[h] = u32x4{0u, 0u, 0u, 0u};
          if (r < p.R && mine)
            part[h] = *reinterpret_cast<const u32x4*>(p.v + ((int64_t)(m0 + 16 * b + lx) * 3 + h) * p.R + r);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 3; ++h) d = mfma_bf16(wf[q], part[h], d);
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[b][q][f] += mine ? d[f] : 0.f;
        }
      }
    }
  });
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[wave][4 * b + q][lane] = acc[b][q];
  __syncthreads();
  for (int i = wave; i < 4 * MB; i += 8) {
    // columns 32 (q / 2) + 8 lg + 4 (q % 2) + 0..3 of a lane
    const int q = i & 3, m = m0 + 16 * (i >> 2) + lx, n = n0 + 32 * (q >> 1) + 8 * lg + 4 * (q & 1);
    if (m >= p.M) continue;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    const float* at = p.acc + (int64_t)m * p.N;
    for (int s = 0; s < p.slices; ++s, at += (int64_t)p.M * p.N) {
      f32x4 u;
      if (n + 4 <= p.N) {
        __builtin_memcpy(&u, at + n, 16);
      } else {
#pragma unroll
        for (int f = 0; f < 4; ++f) u[f] = at[min(n + f, p.N - 1)];
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) sum[f] += u[f];
    }
    f32x4 term = red[0][i][lane];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      const f32x4 u = red[w][i][lane];
#pragma unroll
      for (int f = 0; f < 4; ++f) term[f] += u[f];
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      if (term[f] != term[f] && sum[f] == sum[f] && n + f < p.N)
        term[f] = lora_term<true>(p, m, n + f, p.v + (int64_t)m * 3 * p.R, p.R);
      sum[f] += term[f];
    }
    uint16_t o[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) o[f] = decoder_epilogue(sum[f], p.bias, p.epi, min(n + f, p.N - 1));
    uint16_t* to = p.out + (int64_t)m * p.N + n;
    if (n + 4 <= p.N) {
      __builtin_memcpy(to, o, 8);
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (n + f < p.N) to[f] = o[f];
    }
  }
}

// ---- many rows ---------------------------------------------------------------

// `rows` rows of an operand of `row_bytes` from row `row0` (of `have`) as a buffer.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rows(const void* base, int64_t row0, int64_t have, int rows,
                                                            uint32_t row_bytes) {
  const uint32_t n = (uint32_t)min((int64_t)rows, have - row0);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(base)) + row0 * (int64_t)row_bytes,
                                           (short)0, (int)(n * row_bytes), 0x00020000);
}

// A lane's 16 sums of the 32 x 32 block at (mb, nb): row mb + lane % 32, columns nb + 8 h + 0..7
// and + 16 (h = lane / 32).  Epilogue, one rounding.
__device__ __forceinline__ void lora_block(const LoraParams& p, float (&v)[16], int mb, int nb, int lane, bool has_bias,
                                           bool gelu) {
  int first = nb + 8 * (lane >> 5);
  asm volatile("" : "+v"(first));  // (as in q8_block)
  uint32_t bs[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  if (has_bias) {
    if (nb + 32 <= p.N) {
#pragma unroll
      for (int r = 0; r < 2; ++r) __builtin_memcpy(&bs[4 * r], p.bias + first + 16 * r, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int n = first + 16 * (i >> 2) + 2 * (i & 3);
        bs[i] = (uint32_t)p.bias[min(n, p.N - 1)] | (uint32_t)p.bias[min(n + 1, p.N - 1)] << 16;
      }
    }
  }
  // (without a bias 0 is added: sums that only some paths change spilled)
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] += __builtin_bit_cast(float, i & 1 ? bs[i >> 1] & 0xffff0000u : bs[i >> 1] << 16);
  if (gelu) gelu_tanh_all(v);
  if (nb + 32 <= p.N) {
    // (16-byte stores of 64 consecutive bytes of a row by four lanes, as in q8_block)
    u32x4 pk[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto t = __builtin_amdgcn_permlane16_swap(pack_bf16x2(v[2 * i], v[2 * i + 1]),
                                                      pack_bf16x2(v[8 + 2 * i], v[9 + 2 * i]), false, false);
      pk[0][i] = t[0];
      pk[1][i] = t[1];
    }
    int n = nb + 16 * ((lane >> 4) & 1) + 8 * (lane >> 5);
    asm volatile("" : "+v"(n));
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int m = mb + 16 * r + (lane & 15);
      if (m < p.M) __builtin_memcpy(p.out + (int64_t)m * p.N + n, &pk[r], 16);
    }
  } else if (mb + (lane & 31) < p.M) {
    uint16_t* o = p.out + (int64_t)(mb + (lane & 31)) * p.N + first;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int n = 16 * (i >> 3) + (i & 7);
      if (n < p.N - first) o[n] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]));
    }
  }
}

// Those outputs of a wave's 32 x 32 block at (mb, nb) whose row of B, of the output row's adapter, is
// not finite: the output has the class of the sum of those terms and of what is there (which the
// other terms and the epilogue gave).
__device__ __forceinline__ void lora_mark(const LoraParams& p, int mb, int nb, int lane, bool gelu) {
  const int m = mb + (lane & 31), a = lora_adapter(p, m);
  if (a < 0) return;
#pragma unroll 1
  for (int n = nb + 16 * (lane >> 5); n < min(nb + 16 * (lane >> 5) + 16, p.N); ++n) {
    const uint16_t* b = p.B + ((int64_t)a * p.N + n) * p.R;
    const uint16_t* v = p.v + (int64_t)m * 3 * p.R;
    bool odd = false;
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < p.R >> 3; ++c) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(b + 8 * c);
      if (!(odd_halves(w[0]) | odd_halves(w[1]) | odd_halves(w[2]) | odd_halves(w[3]))) continue;
      odd = true;
      sum = lora_terms<true>(sum, w, v, p.R, c);
    }
    if (!odd) continue;
    uint16_t* o = p.out + (int64_t)m * p.N + n;
    const float was = bf16_float(*o);
    if (!__builtin_isfinite(was)) sum += was;
    if (gelu) sum = gelu_tanh(sum);
    *o = __builtin_bit_cast(uint16_t, static_cast<__bf16>(sum));
  }
}

// Tiles of 64 FM rows by 64 FN columns, in the manner of gemm_q8_tile (LDS rows of 128
// bytes, here 64 k of bf16; the same rings, waits and layout, and what is mended in one belongs into the other; two
// v_mfma_f32_32x32x16_bf16 where that has one instruction).
//
// The adapters' terms are further super-steps of the same sums: for each adapter among a
// tile's rows ceil(3 R / 64) of them, in which x stands for the rows' v, part after
// part (rows of other adapters lie past the buffer's end: zeros), and W for the adapter's
// B, three times.  So a tile of one adapter of rank 16 costs one super-step more.
// Bound by issuing MFMAs and by L2: 8192^3, rank 16 870 us (864 to 921 in 60 calls; 1270 TFLOP/s; MFMAs in 75 % of a
// working CU's cycles, 10 TB/s out of L2).  Where rows start inside a 128-byte line (K not a
// multiple of 64) each copy touches two: 2047 x 3001 x 4104, rank 32 82 us, 1.27 GB out of L2 (16 TB/s).
// (A zero times an infinity or a NaN of B would be NaN in the other rows: 1 with their sign is taken
// for them, whose product has the class of theirs where v is not finite, and the outputs of the adapter's rows in
// those columns get their class at the end.)
// SPLIT: the instance for a K cut into slices; those leave their sums of W x for lora_join.
template <int FM, int FN, int SX, int SW, bool SPLIT>
__global__ void __launch_bounds__(256, SX * FM + SW * FN <= 10 ? 2 : 1) lora_tile(LoraParams p) {
  constexpr int BM = 64 * FM, BN = 64 * FN, XS = BM * 128, WS = BN * 128;
  constexpr int CX = 2 * FM, CW = 2 * FN;  // copies of 8 rows per wave and super-step
  // copies that a wait for a super-step may leave in flight: those issued after
  // the later of its own
  constexpr int kAhead = SX <= SW ? (SX - 2) * (CX + CW) : CX + (SW - 2) * (CX + CW);
  constexpr int PER = (CX + CW + 2 * FM * FN - 1) / (2 * FM * FN);  // copies per MFMA of a step
  __shared__ __attribute__((aligned(1024))) char smem[SX * XS + SW * WS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int wm = (wave >> 1) * (32 * FM), wn = (wave & 1) * (32 * FN);
  const int G = gridDim.x;
  const int wg = __builtin_amdgcn_readfirstlane(remap_workgroup(blockIdx.x, G, 1));
  const int my_units =
      __builtin_amdgcn_readfirstlane((p.tiles_m * p.tiles_n * (SPLIT ? p.slices : 1) - wg + G - 1) / G);
  const int KS = (p.K + 63) >> 6;
  // The arguments as what the compiler does not know to be the same: where they are needed
  // only from tile to tile they are loaded again, and take no scalar registers in the K loop.
  auto args = []() __attribute__((always_inline)) {
    auto* a = (__attribute__((address_space(4))) const LoraParams*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(a));
    return a;
  };

  // the lane's place in a copy: row (of 8) and chunk (of even and odd copies); opaque too
  struct Place {
    int row;
    uint32_t chunk[2];
  };
  auto place = [&]() __attribute__((always_inline)) {
    int l = lane;
    asm volatile("" : "+v"(l));
    const int row = l >> 3;
    return Place{row, {16u * (uint32_t)((l & 7) ^ (row >> 1)), 16u * (uint32_t)((l & 7) ^ (4 + (row >> 1)))}};
  };
  // the operand row of the lane in copy c
  auto row_x = [&](int c, int row) __attribute__((always_inline)) { return (uint32_t)(8 * (wave * CX + c) + row); };
  auto row_w = [&](int c, int row) __attribute__((always_inline)) {
    const int t = wave * CW + c;
    return (uint32_t)(32 * (t >> 2) + 16 * ((t >> 1) & 1) + 8 * (row >> 2) + 4 * (t & 1) + (row & 3));
  };
  uint32_t vx[CX], vw[CW];

  // Where each operand's copies are: unit (of this workgroup's), super-step and its end.
  __amdgpu_buffer_rsrc_t rx, rw;
  uint32_t bx = 0, bw = 0;  // the super-step's part of the offsets
  int xi = 0, xq = 0, xend = 0, wi = 0, wq = 0, wend = 0;
  // unit i of this workgroup: its tile and its super-steps [q0, q1)
  auto unit = [&](int i, int* tm, int* tn, int* q0, int* q1) __attribute__((always_inline)) {
    const auto* p = args();
    const int u = wg + i * G, tiles = p->tiles_m * p->tiles_n;
    const int c = SPLIT ? __builtin_amdgcn_readfirstlane(u / tiles) : 0;
    tile_coords(u - c * tiles, p->tiles_m, p->tiles_n, 4, tm, tn);
    *tm = __builtin_amdgcn_readfirstlane(*tm);
    *tn = __builtin_amdgcn_readfirstlane(*tn);
    if constexpr (SPLIT) {
      *q0 = c * p->slice_steps;
      *q1 = min(*q0 + p->slice_steps, KS);
    } else {
      *q0 = 0;
      *q1 = KS + __builtin_amdgcn_readfirstlane(p->tiles[*tm].count) * lora_steps(p->R);
    }
  };
  // offsets of super-step q: of K, the ragged last one's chunks past K out of range
  auto base = [&](int q, uint32_t row, uint32_t chunk, uint32_t K) __attribute__((always_inline)) {
    return (row * K + chunk) | (128u * (uint32_t)q + chunk < K ? 0u : 0x80000000u);
  };
  auto base_x = [&]() __attribute__((always_inline)) {
    const Place l = place();
    const uint32_t K = 2u * (uint32_t)args()->K;
#pragma unroll
    for (int c = 0; c < CX; ++c) vx[c] = base(xq, row_x(c, l.row), l.chunk[c & 1], K);
  };
  auto base_w = [&]() __attribute__((always_inline)) {
    const Place l = place();
    const uint32_t K = 2u * (uint32_t)args()->K;
#pragma unroll
    for (int c = 0; c < CW; ++c) vw[c] = base(wq, row_w(c, l.row), l.chunk[c & 1], K);
  };
  // or of an adapter: piece e of its 3 R values
  auto extra_x = [&]() __attribute__((always_inline)) {
    const auto* p = args();
    const Place l = place();
    const int ES = lora_steps(p->R), a = (xq - KS) / ES, e = (xq - KS) - a * ES;
    const uint32_t R6 = 6u * (uint32_t)p->R;
    if (e > 0) {  // the same rows, a piece further
#pragma unroll
      for (int c = 0; c < CX; ++c)
        vx[c] = vx[c] < 0x80000000u && 128u * (uint32_t)e + l.chunk[c & 1] < R6 ? vx[c] + 128u : 0x80000000u;
      return;
    }
    int tm, tn, q0, q1;
    unit(min(xi, my_units - 1), &tm, &tn, &q0, &q1);
    rx = tile_rows(p->v, (int64_t)tm * BM, p->M, BM, R6);
    const uint64_t rows = p->tiles[tm].rows[a][(8 * wave * CX) >> 6] >> ((8 * wave * CX) & 63);
#pragma unroll
    for (int c = 0; c < CX; ++c) {
      const uint32_t at = l.chunk[c & 1];
      vx[c] = at < R6 && ((rows >> (8 * c + l.row)) & 1) ? row_x(c, l.row) * R6 + at : 0x80000000u;
    }
  };
  auto extra_w = [&]() __attribute__((always_inline)) {
    const auto* p = args();
    const Place l = place();
    const int ES = lora_steps(p->R), a = (wq - KS) / ES, e = (wq - KS) - a * ES;
    const uint32_t R2 = 2u * (uint32_t)p->R;
    if (e == 0) {  // (later pieces: the same rows)
      int tm, tn, q0, q1;
      unit(min(wi, my_units - 1), &tm, &tn, &q0, &q1);
      const int64_t first = (int64_t)__builtin_amdgcn_readfirstlane(p->tiles[tm].adapter[a]) * p->N;
      rw = tile_rows(p->B, first + (int64_t)tn * BN, first + p->N, BN, R2);
    }
#pragma unroll
    for (int c = 0; c < CW; ++c) {
      const uint32_t at = 128u * (uint32_t)e + l.chunk[c & 1];
      vw[c] = at < 3 * R2 ? row_w(c, l.row) * R2 + (at < R2 ? at : at < 2 * R2 ? at - R2 : at - 2 * R2) : 0x80000000u;
    }
  };
  // (past the last unit that one again, never read)
  auto enter_x = [&]() __attribute__((always_inline)) {
    int tm, tn;
    unit(min(xi, my_units - 1), &tm, &tn, &xq, &xend);
    const auto* p = args();
    rx = tile_rows(p->x, (int64_t)tm * BM, p->M, BM, 2u * (uint32_t)p->K);
    base_x();
    bx = 128u * (uint32_t)xq;
  };
  auto enter_w = [&]() __attribute__((always_inline)) {
    int tm, tn;
    unit(min(wi, my_units - 1), &tm, &tn, &wq, &wend);
    const auto* p = args();
    rw = tile_rows(p->W, (int64_t)tn * BN, p->N, BN, 2u * (uint32_t)p->K);
    base_w();
    bw = 128u * (uint32_t)wq;
  };
  auto advance_x = [&]() __attribute__((always_inline)) {
    ++xq;
    bx += 128u;
    if (xq >= KS - 1 || xq == xend) {
      if (xq == xend) {
        ++xi;
        enter_x();
      } else if (xq == KS - 1) {
        base_x();
      } else {
        bx = 0;
        extra_x();
      }
    }
  };
  auto advance_w = [&]() __attribute__((always_inline)) {
    ++wq;
    bw += 128u;
    if (wq >= KS - 1 || wq == wend) {
      if (wq == wend) {
        ++wi;
        enter_w();
      } else if (wq == KS - 1) {
        base_w();
      } else {
        bw = 0;
        extra_w();
      }
    }
  };
  auto copy_x = [&](int c, int slot) __attribute__((always_inline)) {
    copy_to_lds(rx, smem + slot * XS + (wave * CX + c) * 1024, vx[c], bx);
  };
  auto copy_w = [&](int c, int slot) __attribute__((always_inline)) {
    copy_to_lds(rw, smem + SX * XS + slot * WS + (wave * CW + c) * 1024, vw[c], bw);
  };

  // fragments: chunks 4 s + 2 j + h of a row, j = 0, 1
  const int f0 = l32 * 128 + ((h ^ ((l32 >> 1) & 7)) << 4);
  struct Frag {
    u32x4 j[2];
  };
  auto frag = [&](int base, int s) __attribute__((always_inline)) {
    return Frag{{lds_chunk(smem + base + (f0 ^ (64 * s))), lds_chunk(smem + base + (f0 ^ (64 * s + 32)))}};
  };
  f32x16 acc[FM][FN];
  Frag x[2][FM], w[2][FN];

  auto frag_x = [&](int a, int slot, int s) __attribute__((always_inline)) {
    return frag(slot * XS + (wm + 32 * a) * 128, s);
  };
  auto frag_w = [&](int b, int slot, int s) __attribute__((always_inline)) {
    return frag(SX * XS + slot * WS + (wn + 32 * b) * 128, s);
  };
  auto multiply = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w[s][b].j[j]),
                                                              __builtin_bit_cast(bf16x8, x[s][a].j[j]), acc[a][b], 0, 0, 0);
  };

  enter_x();
  enter_w();
#pragma unroll
  for (int q = 0; q < max(SX, SW); ++q) {
    if (q > 0 && q < SW) advance_w();
    if (q > 0 && q < SX) advance_x();
    if (q < SW) {
#pragma unroll
      for (int c = 0; c < CW; ++c) copy_w(c, q);
    }
    if (q < SX) {
#pragma unroll
      for (int c = 0; c < CX; ++c) copy_x(c, q);
    }
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0((SX - 1) * CX + (SW - 1) * CW));
  order();
  __builtin_amdgcn_s_barrier();
  order();
  int xb = 0, wb = 0;  // slots of super-step q
  for (int ui = 0; ui < my_units; ++ui) {
    int tm, tn, q0, q1;
    unit(ui, &tm, &tn, &q0, &q1);
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
    // (read here and not carried over from the unit before, whose epilogue needs the registers)
#pragma unroll
    for (int a = 0; a < FM; ++a) x[0][a] = frag_x(a, xb, 0);
#pragma unroll
    for (int b = 0; b < FN; ++b) w[0][b] = frag_w(b, wb, 0);
    int left_out = 0;  // whether an adapter's B held what is not finite
    auto clean = [&](int s) __attribute__((always_inline)) {
      uint32_t any = 0;
#pragma unroll
      for (int b = 0; b < FN; ++b) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t u = w[s][b].j[i >> 2][i & 3], odd = odd_halves(u);
          const uint32_t value = (odd >> 15) * 0x7fffu;  // (all but the sign)
          w[s][b].j[i >> 2][i & 3] = (u & ~value) | (0x3f803f80u & value);
          any |= odd;
        }
      }
      left_out |= __any(any != 0);
    };
    // EXTRA: an adapter's super-step
    auto super_step = [&](auto extra) __attribute__((always_inline)) {
      constexpr bool EXTRA = decltype(extra)::value;
#ifdef MM_DEBUG_FULL_SYNC
      race_check_drain();  // every copy issued so far has landed, for every wave
      __builtin_amdgcn_s_barrier();
      order();
#endif
      if constexpr (EXTRA) clean(0);
      // step 0
#pragma unroll
      for (int a = 0; a < FM; ++a) x[1][a] = frag_x(a, xb, 1);
#pragma unroll
      for (int b = 0; b < FN; ++b) w[1][b] = frag_w(b, wb, 1);
      multiply(0);
#pragma unroll
      for (int i = 0; i < 2 * FM * FN; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);    // an MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);  // LDS reads
      }
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(kAhead));
      order();
      __builtin_amdgcn_s_barrier();
      order();
      // (their branches stand here so that each step is a block of its own to
      // the scheduler, whose groups otherwise mix the two)
      advance_w();
      advance_x();
      if constexpr (EXTRA) clean(1);
      const int xn = xb == SX - 1 ? 0 : xb + 1, wnext = wb == SW - 1 ? 0 : wb + 1;
      // step 1.  The compiler keeps the order of copies and reads: a copy after
      // each fragment, the others after those.
      auto copy = [&](int c) __attribute__((always_inline)) {
        if (c < CW)
          copy_w(c, wb);
        else
          copy_x(c - CW, xb);
      };
#pragma unroll
      for (int i = 0; i < FM + FN; ++i) {
        if (i < FM)
          x[0][i] = frag_x(i, xn, 0);
        else
          w[0][i - FM] = frag_w(i - FM, wnext, 0);
        copy(i);
      }
#pragma unroll
      for (int i = FM + FN; i < CX + CW; ++i) copy(i);
      multiply(1);
#pragma unroll
      for (int i = 0; i < FM + FN; ++i) {
        if (i < FM * FN) __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);  // two MFMAs
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);                   // a fragment
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);                   // a copy
      }
#pragma unroll
      for (int i = FM + FN; i < CX + CW; ++i) {
        if (i < FM * FN) __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
      xb = xn;
      wb = wnext;
    };
    for (int q = q0; q < min(q1, KS); ++q) super_step(std::false_type{});
    if constexpr (!SPLIT) {
      for (int q = KS; q < q1; ++q) super_step(std::true_type{});
    }

    const int m0 = tm * BM + wm, n0 = tn * BN + wn;
    if constexpr (SPLIT) {
      const int c = (wg + ui * G) / (p.tiles_m * p.tiles_n);
#pragma unroll
      for (int b = 0; b < FN; ++b)
#pragma unroll
        for (int a = 0; a < FM; ++a) {
          const int m = m0 + 32 * a + l32;
          int n = n0 + 32 * b + 8 * h;
          asm volatile("" : "+v"(n));
          if (m >= p.M) continue;
          float* o = p.acc + ((int64_t)c * p.M + m) * p.N + n;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (n + 16 * r + 8 <= p.N) {
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const f32x4 u = {acc[a][b][8 * r + 4 * f], acc[a][b][8 * r + 4 * f + 1], acc[a][b][8 * r + 4 * f + 2],
                                 acc[a][b][8 * r + 4 * f + 3]};
                __builtin_memcpy(o + 16 * r + 4 * f, &u, 16);
              }
            } else {
#pragma unroll
              for (int f = 0; f < 8; ++f)
                if (n + 16 * r + f < p.N) o[16 * r + f] = acc[a][b][8 * r + f];
            }
          }
        }
      continue;
    }
    // (the last MFMAs' results are there: the compiler does not see the reads below for what
    // they are)
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    int el = lane;  // (opaque, as in place())
    asm volatile("" : "+v"(el));
    const int epi = args()->epi;
    const bool has_bias = epi == EPI_BIAS || epi == EPI_BIAS_GELU, gelu = epi == EPI_GELU || epi == EPI_BIAS_GELU;
#pragma unroll
    for (int b = 0; b < FN; ++b)
#pragma unroll
      for (int a = 0; a < FM; ++a) {
        // (each block's sums are moved when it is their turn: taken ahead, they spilled)
        order();
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v[i]) : "a"(acc[a][b][i]));
        lora_block(p, v, m0 + 32 * a, n0 + 32 * b, el, has_bias, gelu);
      }
    if (left_out) {
      __builtin_amdgcn_s_waitcnt(0);  // (after the stores above, some of the same places)
      order();
#pragma unroll 1
      for (int i = 0; i < FM * FN; ++i) lora_mark(p, m0 + 32 * (i / FN), n0 + 32 * (i % FN), el, gelu);
    }
  }
  __builtin_amdgcn_s_waitcnt(0);  // (the copies past the last unit land before the workgroup ends)
}

}  // namespace mmk
