// Linear layer of many requests at once, each row with a low-rank adapter of its own
// choice beside the shared weight:
//   out[m] = epi(W x[m] + bias + s_a B_a (A_a x[m])),   a = index[m]
// (rows whose index names no adapter: without the last term).  x [M][K], W [N][K],
// A [L][R][K], B [L][N][R] bf16, fp32 scales, bf16 output, one rounding.
//
// lora_shrink leaves A_a x[m] in fp32, in slices of K.  Few rows (a decode step): bound by
// reading W once; lora_rows streams it and adds B (s_a A_a x[m]) to the same sums.
// Many rows: the library's tile kernels leave W x in fp32, and lora_join adds the rest.
// v = s_a A_a x enters the products with B as two bf16 numbers, high and low part, 16
// bits of significand: as one, its rounding would be as large as the output's own.
#pragma once

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
  uint16_t* v;            // [M][2][R]: s A x, high and low parts
  float* acc;             // [slices][M][N]: parts of W x
  int M, N, K, R, L;
  int low_slices, low_k;  // slices of K of low_k (a multiple of 64)
  int slices;             // of acc
  int epi;
};

// The adapter of row `row`, -1 for none (past the last row, or an index that names none).
__device__ __forceinline__ int lora_adapter(const LoraParams& p, int row) {
  if (row >= p.M) return -1;
  const int a = p.index[row];
  return (unsigned)a < (unsigned)p.L ? a : -1;
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

// A lane's piece j (0, 1) of step st of 64 k from a row at byte `row` of a buffer: chunk
// lane / 16 of 8 values.  Zeros past K; past the last step too (its base, a
// scalar, has to stay inside the buffer).
__device__ __forceinline__ u32x4 step_chunk(__amdgpu_buffer_rsrc_t buf, uint32_t row, int st, int j, int K, int steps,
                                            int lg) {
  const uint32_t off = 64 * st + 32 * j + 8 * lg < K ? row + 64u * j + 16u * (uint32_t)lg : 0x80000000u;
  return load_chunk(buf, off, 128u * (uint32_t)min(st, steps - 1));
}

// A x of the rows 16 MB y .. + 16 MB - 1 over slice x of K, for ranks 16 z .. + 15 (z the
// first part of blockIdx.z); of the adapters among the rows, every turns-th.  The waves
// take every eighth step of 64 k, each step's loads one step ahead, and meet in LDS, added in
// wave order.  A CU by itself reads some 25 bytes per ns, so the slices, adapters
// and ranks of few rows go to many (one token, rank 16, K 8192: 4.5 us in 16 slices, 12
// in one).
template <int MB>
__global__ void __launch_bounds__(kLoraShrinkWaves * 64) lora_shrink(LoraParams p, int turns) {
  __shared__ f32x4 red[kLoraShrinkWaves][MB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int m0 = blockIdx.y * (16 * MB), rows = min(16 * MB, p.M - m0);
  const int r0 = (int)(blockIdx.z / turns) * 16, my_turn = blockIdx.z % turns;
  const int K = p.K, kbeg = blockIdx.x * p.low_k, klen = min(p.low_k, K - kbeg), steps = (klen + 63) >> 6;
  // (of a slice of a row the buffer ends where the last row's does)
  const __amdgpu_buffer_rsrc_t rx = slice_buffer(p.x + (int64_t)m0 * K + kbeg, rows, K, kbeg);
  struct Step {
    u32x4 w[2], x[MB][2];
  };
  int turn = 0;
  each_adapter(lane < rows ? lora_adapter(p, m0 + lane) : -1, [&](int a, uint64_t same) {
    if (turn++ % turns != my_turn) return;
    const __amdgpu_buffer_rsrc_t rw = slice_buffer(p.A + ((int64_t)a * p.R + r0) * K + kbeg, min(16, p.R - r0), K, kbeg);
    const uint32_t row = (uint32_t)lx * (uint32_t)K * 2u;
    uint32_t xrow[MB];  // (rows of other adapters are not loaded)
#pragma unroll
    for (int b = 0; b < MB; ++b)
      xrow[b] = (same >> (16 * b + lx)) & 1 ? (uint32_t)(16 * b + lx) * (uint32_t)K * 2u : 0x80000000u;
    auto load = [&](int st, Step& t) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        t.w[j] = step_chunk(rw, row, st, j, klen, steps, lg);
#pragma unroll
        for (int b = 0; b < MB; ++b) t.x[b][j] = step_chunk(rx, xrow[b], st, j, klen, steps, lg);
      }
    };
    f32x4 acc[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int st, Step& t, Step& next) __attribute__((always_inline)) {
      load(st + kLoraShrinkWaves, next);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[b] = mfma_bf16(t.x[b][j], t.w[j], acc[b]);
    };
    Step s0, s1;
    load(wave, s0);
    for (int st = wave; st < steps; st += 2 * kLoraShrinkWaves) {
      step(st, s0, s1);
      step(st + kLoraShrinkWaves, s1, s0);
    }
    __syncthreads();  // (what was there before has been read)
#pragma unroll
    for (int b = 0; b < MB; ++b) red[wave][b][lane] = acc[b];
    __syncthreads();
    if (wave < MB) {
      f32x4 s = red[0][wave][lane];
#pragma unroll
      for (int q = 1; q < kLoraShrinkWaves; ++q) {
        const f32x4 u = red[q][wave][lane];
#pragma unroll
        for (int f = 0; f < 4; ++f) s[f] += u[f];
      }
      const int r = r0 + lx;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int m = 16 * wave + 4 * lg + f;
        if (r < p.R && ((same >> m) & 1)) p.low[((int64_t)blockIdx.x * p.M + m0 + m) * p.R + r] = s[f];
      }
    }
  });
}

// v of row m (adapter a), ranks r .. r + 7: the slices added in order, the scale, two parts.
__device__ __forceinline__ void lora_v(const LoraParams& p, int m, int a, int r, u32x4* hi, u32x4* lo) {
  f32x4 v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  const float* at = p.low + (int64_t)m * p.R + r;
#pragma unroll 4
  for (int s = 0; s < p.low_slices; ++s, at += (int64_t)p.M * p.R) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(at + 4 * h);
#pragma unroll
      for (int f = 0; f < 4; ++f) v[h][f] += u[f];
    }
  }
  const float scale = p.scale[a];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint16_t h[2], l[2];
    split_bf16(v[j >> 1][2 * (j & 1)] * scale, &h[0], &l[0]);
    split_bf16(v[j >> 1][2 * (j & 1) + 1] * scale, &h[1], &l[1]);
    (*hi)[j] = (uint32_t)h[0] | (uint32_t)h[1] << 16;
    (*lo)[j] = (uint32_t)l[0] | (uint32_t)l[1] << 16;
  }
}

// v of every row, 8 ranks per thread; rows without an adapter are left out.
__device__ __forceinline__ void lora_fold_all(const LoraParams& p, int64_t thread, int64_t threads) {
  const int chunks = p.R >> 3;
  for (int64_t i = thread; i < (int64_t)p.M * chunks; i += threads) {
    const int m = (int)(i / chunks), r = 8 * (int)(i - (int64_t)m * chunks);
    const int a = lora_adapter(p, m);
    if (a < 0) continue;
    u32x4 hi, lo;
    lora_v(p, m, a, r, &hi, &lo);
    uint16_t* v = p.v + (int64_t)m * 2 * p.R + r;
    *reinterpret_cast<u32x4*>(v) = hi;
    *reinterpret_cast<u32x4*>(v + p.R) = lo;
  }
}
__global__ void __launch_bounds__(256) lora_fold(LoraParams p) {
  lora_fold_all(p, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// Up to 16 MB rows.  A workgroup takes a slice y of K, 16 SPW steps of 64 k, and every
// gridDim.x-th block of 16 columns.  Wave w has the slice's steps 16 i + w, i < SPW, and
// holds x there in registers for all blocks, so that W is all that it loads; each
// step's loads are issued one step ahead, across blocks.  The waves' sums of a block meet
// in LDS (two sets in turn: one barrier per block) and are added in wave order, by
// another wave for each block.
// FINISH (K in one slice): v comes into LDS first, the adapters' terms join the sums
// here, each adapter on a wave, and the output is written.  Else lora_join does both,
// and v is left in memory for it.
template <int MB, int SPW, bool FINISH>
__global__ void __launch_bounds__(kLoraWaves * 64) lora_rows(LoraParams p) {
  static_assert(SPW % 2 == 0 && MB * SPW <= 8, "x in 64 registers, two steps in turn");
  __shared__ f32x4 red[2][kLoraWaves][MB][64];
  __shared__ u32x4 v[FINISH ? 16 * MB : 1][2][kLoraMaxRank / 8];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int K = p.K, steps = (K + 63) >> 6, blocks = (p.N + 15) >> 4;
  const int first = blockIdx.y * (kLoraWaves * SPW) + wave;

  struct Step {
    u32x4 w[2];
  };
  uint32_t row = (uint32_t)lx * (uint32_t)K * 2u;
  auto load = [&](int block, int i, Step& t) __attribute__((always_inline)) {
    // (opaque: the steps' offsets are not all kept in registers)
    asm volatile("" : "+v"(row));
    // (past the last block, that one again, unused)
    const int n0 = 16 * min(block, blocks - 1);
    const __amdgpu_buffer_rsrc_t rw = rows_buffer(p.W + (int64_t)n0 * K, min(16, p.N - n0), K);
#pragma unroll
    for (int j = 0; j < 2; ++j) t.w[j] = step_chunk(rw, row, first + kLoraWaves * i, j, K, steps, lg);
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
          x[b][i][j] = step_chunk(rx, (uint32_t)(16 * b + lx) * (uint32_t)K * 2u, first + kLoraWaves * i, j, K, steps, lg);
  }
  // this wave's adapters (of at most 16 MB) and their rows
  int mine[MB];
  uint64_t same[MB];
#pragma unroll
  for (int q = 0; q < MB; ++q) {
    mine[q] = -1;
    same[q] = 0;
  }
  if constexpr (FINISH) {
    int turn = 0;
    each_adapter(lora_adapter(p, lane), [&](int a, uint64_t s) {
#pragma unroll
      for (int q = 0; q < MB; ++q) {
        if (turn == kLoraWaves * q + wave) {
          mine[q] = a;
          same[q] = s;
        }
      }
      ++turn;
    });
    const int chunks = p.R >> 3;
    for (int i = threadIdx.x; i < p.M * chunks; i += kLoraWaves * 64) {
      const int m = i / chunks, c = i - m * chunks, a = lora_adapter(p, m);
      if (a >= 0) lora_v(p, m, a, 8 * c, &v[m][0][c], &v[m][1][c]);
    }
    __syncthreads();
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
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[b] = mfma_bf16(x[b][i][j], t[i & 1].w[j], acc[b]);
    }
#pragma unroll
    for (int q = 0; q < MB; ++q) {
      if (!FINISH || mine[q] < 0) continue;
      const uint16_t* bw = p.B + ((int64_t)mine[q] * p.N + min(n0 + lx, p.N - 1)) * p.R;
      for (int r0 = 0; r0 < p.R; r0 += 32) {
        const int r = r0 + 8 * lg;
        u32x4 wf = {0u, 0u, 0u, 0u};
        if (r < p.R) wf = *reinterpret_cast<const u32x4*>(bw + r);
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          if (!((same[q] >> (16 * b)) & 0xffff)) continue;
          u32x4 hi = {0u, 0u, 0u, 0u}, lo = {0u, 0u, 0u, 0u};
          if (r < p.R && ((same[q] >> (16 * b + lx)) & 1)) {
            hi = v[16 * b + lx][0][r >> 3];
            lo = v[16 * b + lx][1][r >> 3];
          }
          f32x4 d = mfma_bf16(hi, wf, f32x4{0.f, 0.f, 0.f, 0.f});
          d = mfma_bf16(lo, wf, d);
          // (0 times what is not finite: other rows' sums are left alone)
#pragma unroll
          for (int f = 0; f < 4; ++f)
            if ((same[q] >> (16 * b + 4 * lg + f)) & 1) acc[b][f] += d[f];
        }
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
__global__ void __launch_bounds__(256) lora_join(LoraParams p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int m0 = blockIdx.y * 64 + 16 * wave, n0 = blockIdx.x * 64;
  if (m0 >= p.M) return;
  const int m = m0 + lx;
  f32x4 acc[2][2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int n = n0 + 32 * c + 8 * lg;
    const float* at = p.acc + (int64_t)min(m, p.M - 1) * p.N;
    acc[c][0] = acc[c][1] = f32x4{0.f, 0.f, 0.f, 0.f};
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
      u32x4 wf[2][2], hi = {0u, 0u, 0u, 0u}, lo = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = min(n0 + 32 * c + 8 * (lx >> 2) + 4 * h + (lx & 3), p.N - 1);
          wf[c][h] = u32x4{0u, 0u, 0u, 0u};
          if (r < p.R) wf[c][h] = *reinterpret_cast<const u32x4*>(p.B + ((int64_t)a * p.N + n) * p.R + r);
        }
      }
      if (r < p.R && mine) {
        const uint16_t* v = p.v + (int64_t)m * 2 * p.R + r;
        hi = *reinterpret_cast<const u32x4*>(v);
        lo = *reinterpret_cast<const u32x4*>(v + p.R);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4 d = mfma_bf16(wf[c][h], hi, f32x4{0.f, 0.f, 0.f, 0.f});
          d = mfma_bf16(wf[c][h], lo, d);
          // (0 times what is not finite: other rows' sums are left alone)
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[c][h][f] += mine ? d[f] : 0.f;
        }
      }
    }
  });
  if (m >= p.M) return;
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

}  // namespace mmk
