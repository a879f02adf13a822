// Linear layer of many requests at once, each row with a low-rank adapter of its own
// choice beside the shared weight:
//   out[m] = epi(W x[m] + bias + s_a B_a (A_a x[m])),   a = index[m]
// (rows whose index names no adapter: without the last term).  x [M][K], W [N][K],
// A [L][R][K], B [L][N][R] bf16, fp32 scales, bf16 output, one rounding.
//
// lora_shrink leaves v[m] = A_a x[m] in fp32.  Few rows (a decode step): bound by reading
// W once; lora_rows streams it and adds B (s v) as further steps of the same sums.  Many
// rows: the library's tile kernels leave W x in fp32, and lora_join adds the rest.
// s v enters the matrix products as two bf16 numbers, high and low part, 16 bits
// of significand: one would round the adapter's term more than the output is.
#pragma once

#include "moe_ffn.hpp"
#include "rms_norm.hpp"

namespace mmk {

constexpr int kLoraWaves = 8;
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
  float* v;               // [slices][M][R]
  const float* acc;       // [M][N]: W x (lora_join)
  int M, N, K, R, L;
  int slices, kc;         // K in slices of kc (a multiple of 64)
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

// v of the rows 16 MB y .. + 16 MB - 1 over slice x of K; of the adapters among them,
// every gridDim.z-th.  The waves share the adapter's blocks of 16 ranks and, where those
// are fewer than the waves, the slice's steps of 64 k, and meet in LDS.
template <int MB>
__global__ void __launch_bounds__(kLoraWaves * 64) lora_shrink(LoraParams p) {
  __shared__ f32x4 red[kLoraWaves][MB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int m0 = blockIdx.y * (16 * MB), rows = min(16 * MB, p.M - m0);
  const int K = p.K;
  const int kbeg = blockIdx.x * p.kc, kend = min(K, kbeg + p.kc), steps = (kend - kbeg + 63) >> 6;
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(p.x) + (int64_t)m0 * K, (short)0, rows * K * 2, 0x00020000);
  bool out[2];
  uint32_t tail[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    out[j] = kbeg + 64 * (steps - 1) + 32 * j + 8 * lg >= kend;
    tail[j] = out[j] ? 0x80000000u : 0u;
  }
  const int blocks = (p.R + 15) >> 4;
  int wide = 1;  // blocks of ranks at work together
  while (wide < blocks && wide < kLoraWaves) wide *= 2;
  const int parts = kLoraWaves / wide, part = wave / wide;
  struct Step {
    u32x4 w[2], x[MB][2];
  };
  int turn = 0;
  each_adapter(lane < rows ? lora_adapter(p, m0 + lane) : -1, [&](int a, uint64_t same) {
    if (turn++ % (int)gridDim.z != (int)blockIdx.z) return;
    uint32_t xo[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
      xo[b] = (same >> (16 * b + lx)) & 1 ? (uint32_t)(16 * b + lx) * (uint32_t)K * 2u + 16u * (uint32_t)lg : 0x80000000u;
    for (int c = 0; c < blocks; c += wide) {
      const int block = c + wave % wide;
      f32x4 acc[MB];
#pragma unroll
      for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (block < blocks) {
        const uint16_t* w = p.A + ((int64_t)a * p.R + min(16 * block + lx, p.R - 1)) * K + kbeg + 8 * lg;
        auto load = [&](int st, Step& t) __attribute__((always_inline)) {
          const bool last = st == steps - 1;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            t.w[j] = *reinterpret_cast<const u32x4*>(w + (last && out[j] ? -8 * lg : 64 * st + 32 * j));
#pragma unroll
            for (int b = 0; b < MB; ++b)
              if ((same >> (16 * b)) & 0xffff)
                t.x[b][j] = load_chunk(rx, (xo[b] + 64u * j) | (last ? tail[j] : 0u), 2u * (uint32_t)kbeg + 128u * (uint32_t)st);
          }
        };
        auto step = [&](int st, Step& t, Step& next) __attribute__((always_inline)) {
          load(min(st + parts, steps - 1), next);
          const bool last = st == steps - 1;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (last && out[j]) t.w[j] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int b = 0; b < MB; ++b)
              if ((same >> (16 * b)) & 0xffff) acc[b] = mfma_bf16(t.x[b][j], t.w[j], acc[b]);
          }
        };
        if (part < steps) {
          Step s0, s1;
          load(part, s0);
          for (int st = part; st < steps; st += 2 * parts) {
            step(st, s0, s1);
            if (st + parts < steps) step(st + parts, s1, s0);
          }
        }
      }
      __syncthreads();  // (what was there before has been read)
#pragma unroll
      for (int b = 0; b < MB; ++b) red[wave][b][lane] = acc[b];
      __syncthreads();
      for (int i = threadIdx.x; i < wide * MB * 64; i += kLoraWaves * 64) {
        const int l = i & 63, b = (i >> 6) % MB, g = (i >> 6) / MB;
        const int r = 16 * (c + g) + (l & 15);
        if (r >= p.R) continue;
        f32x4 s = red[g][b][l];
        for (int q = 1; q < parts; ++q) {
          const f32x4 u = red[q * wide + g][b][l];
#pragma unroll
          for (int f = 0; f < 4; ++f) s[f] += u[f];
        }
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int m = 16 * b + 4 * (l >> 4) + f;
          if ((same >> m) & 1) p.v[((int64_t)blockIdx.x * p.M + m0 + m) * p.R + r] = s[f];
        }
      }
    }
  });
}

// s v of row m, ranks r .. r + 7, summed over the slices in order, as two bf16 fragments.
__device__ __forceinline__ void lora_low(const LoraParams& p, int m, int r, float scale, u32x4* hi, u32x4* lo) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  const float* at = p.v + (int64_t)m * p.R + r;
  for (int s = 0; s < p.slices; ++s, at += (int64_t)p.M * p.R) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(at), b = *reinterpret_cast<const f32x4*>(at + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] += a[j];
      v[4 + j] += b[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint16_t h[2], l[2];
    split_bf16(v[2 * j] * scale, &h[0], &l[0]);
    split_bf16(v[2 * j + 1] * scale, &h[1], &l[1]);
    (*hi)[j] = (uint32_t)h[0] | (uint32_t)h[1] << 16;
    (*lo)[j] = (uint32_t)l[0] | (uint32_t)l[1] << 16;
  }
}

// Up to 16 MB rows, 16 columns per workgroup.  The waves take every eighth step of 64 k,
// each step's loads one step ahead, then every eighth adapter, and meet in LDS,
// added in wave order.
template <int MB>
__global__ void __launch_bounds__(kLoraWaves * 64) lora_rows(LoraParams p) {
  __shared__ f32x4 red[kLoraWaves][MB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int n0 = blockIdx.x * 16, K = p.K, steps = (K + 63) >> 6;
  const int64_t row = min(n0 + lx, p.N - 1);
  const uint16_t* w = p.W + row * K + 8 * lg;
  const __amdgpu_buffer_rsrc_t rx =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p.x), (short)0, p.M * K * 2, 0x00020000);
  bool out[2];
  uint32_t tail[2], xo[MB];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    out[j] = 64 * (steps - 1) + 32 * j + 8 * lg >= K;
    tail[j] = out[j] ? 0x80000000u : 0u;
  }
#pragma unroll
  for (int b = 0; b < MB; ++b) xo[b] = (uint32_t)(16 * b + lx) * (uint32_t)K * 2u + 16u * (uint32_t)lg;
  struct Step {
    u32x4 w[2], x[MB][2];
  };
  auto load = [&](int st, Step& t) __attribute__((always_inline)) {
    const bool last = st == steps - 1;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      t.w[j] = *reinterpret_cast<const u32x4*>(w + (last && out[j] ? -8 * lg : 64 * st + 32 * j));
#pragma unroll
      for (int b = 0; b < MB; ++b) t.x[b][j] = load_chunk(rx, (xo[b] + 64u * j) | (last ? tail[j] : 0u), 128u * (uint32_t)st);
    }
  };
  f32x4 acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](int st, Step& t, Step& next) __attribute__((always_inline)) {
    load(min(st + kLoraWaves, steps - 1), next);
    const bool last = st == steps - 1;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (last && out[j]) t.w[j] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int b = 0; b < MB; ++b) acc[b] = mfma_bf16(t.x[b][j], t.w[j], acc[b]);
    }
  };
  if (wave < steps) {
    Step s0, s1;
    load(wave, s0);
    for (int st = wave; st < steps; st += 2 * kLoraWaves) {
      step(st, s0, s1);
      if (st + kLoraWaves < steps) step(st + kLoraWaves, s1, s0);
    }
  }
  int turn = 0;
  each_adapter(lora_adapter(p, lane), [&](int a, uint64_t same) {
    if (turn++ % kLoraWaves != wave) return;
    const float scale = p.scale[a];
    const uint16_t* bw = p.B + ((int64_t)a * p.N + row) * p.R;
    for (int r0 = 0; r0 < p.R; r0 += 32) {
      const int r = r0 + 8 * lg;
      u32x4 wf = {0u, 0u, 0u, 0u};
      if (r < p.R) wf = *reinterpret_cast<const u32x4*>(bw + r);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        if (!((same >> (16 * b)) & 0xffff)) continue;
        u32x4 hi = {0u, 0u, 0u, 0u}, lo = {0u, 0u, 0u, 0u};
        if (r < p.R && ((same >> (16 * b + lx)) & 1)) lora_low(p, 16 * b + lx, r, scale, &hi, &lo);
        // (rows without this adapter get zeros, unless it holds what is not finite:
        // only their own rows' sums are taken)
        f32x4 d = mfma_bf16(hi, wf, f32x4{0.f, 0.f, 0.f, 0.f});
        d = mfma_bf16(lo, wf, d);
#pragma unroll
        for (int f = 0; f < 4; ++f)
          if ((same >> (16 * b + 4 * lg + f)) & 1) acc[b][f] += d[f];
      }
    }
  });
#pragma unroll
  for (int b = 0; b < MB; ++b) red[wave][b][lane] = acc[b];
  __syncthreads();
  for (int i = threadIdx.x; i < MB * 64; i += kLoraWaves * 64) {
    const int l = i & 63, b = i >> 6, n = n0 + (l & 15);
    if (n >= p.N) continue;
    f32x4 s = red[0][b][l];
#pragma unroll
    for (int q = 1; q < kLoraWaves; ++q) {
      const f32x4 u = red[q][b][l];
#pragma unroll
      for (int f = 0; f < 4; ++f) s[f] += u[f];
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int m = 16 * b + 4 * (l >> 4) + f;
      if (m < p.M) p.out[(int64_t)m * p.N + n] = decoder_epilogue(s[f], p.bias, p.epi, n);
    }
  }
}

// Many rows: out = epi(acc + bias + B (s v)) for 64 rows by 256 columns per workgroup,
// 64 columns per wave.  B is the MFMA's first operand, so a lane's sums are of one row;
// the block pair's rows of B are taken in the order that makes them 8 consecutive columns.
__global__ void __launch_bounds__(256) lora_join(LoraParams p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 256 + wave * 64;
  if (n0 >= p.N) return;
  f32x4 acc[4][2][2];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int m = m0 + 16 * b + lx, n = n0 + 32 * c + 8 * lg;
      const float* at = p.acc + (int64_t)min(m, p.M - 1) * p.N;
      if (n + 8 <= p.N) {
        __builtin_memcpy(&acc[b][c][0], at + n, 16);
        __builtin_memcpy(&acc[b][c][1], at + n + 4, 16);
      } else {
#pragma unroll
        for (int f = 0; f < 8; ++f) acc[b][c][f >> 2][f & 3] = at[min(n + f, p.N - 1)];
      }
    }
  }
  each_adapter(lora_adapter(p, m0 + lane), [&](int a, uint64_t same) {
    const float scale = p.scale[a];
    for (int r0 = 0; r0 < p.R; r0 += 32) {
      const int r = r0 + 8 * lg;
      u32x4 wf[2][2];
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
      for (int b = 0; b < 4; ++b) {
        if (!((same >> (16 * b)) & 0xffff)) continue;
        const bool mine = (same >> (16 * b + lx)) & 1;
        u32x4 hi = {0u, 0u, 0u, 0u}, lo = {0u, 0u, 0u, 0u};
        if (r < p.R && mine) lora_low(p, m0 + 16 * b + lx, r, scale, &hi, &lo);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f32x4 d = mfma_bf16(wf[c][h], hi, f32x4{0.f, 0.f, 0.f, 0.f});
            d = mfma_bf16(wf[c][h], lo, d);
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[b][c][h][f] += mine ? d[f] : 0.f;
          }
        }
      }
    }
  });
  const bool has_bias = p.epi == EPI_BIAS || p.epi == EPI_BIAS_GELU;
  const bool gelu = p.epi == EPI_GELU || p.epi == EPI_BIAS_GELU;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int n = n0 + 32 * c + 8 * lg;
    float bias[8];
#pragma unroll
    for (int f = 0; f < 8; ++f) bias[f] = has_bias ? bf16_float(p.bias[min(n + f, p.N - 1)]) : 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int m = m0 + 16 * b + lx;
      if (m >= p.M) continue;
      float v[8];
#pragma unroll
      for (int f = 0; f < 8; ++f) v[f] = acc[b][c][f >> 2][f & 3] + bias[f];
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
}

}  // namespace mmk
