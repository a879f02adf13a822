// Products with 4-bit weights and group scales: out = epi(x . Wd^T + bias),
//   Wd[n][k] = (q[n][k] - z[k / G][n]) s[k / G][n],   q = 0..15, G = 32, 64, 128,
// for a few rows of bf16 activations (the decode step): bound by reading the
// weight, half a byte per value, once.
//
// Weight layout: kilobytes of 16 rows by 128 k, in the order of the MFMA
// fragments: lane (g, n) = 16 g + n of a wave loads one 16-byte chunk, whose
// 32-bit word j holds k = 32 j + 8 g .. + 7 of row n.  So a wave's load is
// one contiguous kilobyte, and word j of all lanes is the B operand of the
// MFMA over k = 32 j .. 32 j + 31.
//
// Arithmetic: a nibble becomes bf16 in one shift and one and-or: with the
// exponent of 16 and the nibble in the top mantissa bits the value is exactly
// 16 + q (two values at once: nibble p of a word's low half and nibble p of
// its high half).  The MFMAs sum x (16 + q) over a group in fp32; the group's
// sum of x comes from one more MFMA against ones; and
//   acc += s (sum x (16 + q) - (16 + z) sum x).
// Both sums are of exact products, so what the offset costs is a few roundings
// of 2^-24 of values some (16 + q) / |q - z| ~ 5 times larger than needed.
#pragma once

#include "mm_device.hpp"

namespace mmk {

struct W4Params {
  const uint16_t* x;       // [M][K] bf16
  const u32x4* W;          // [ceil(N/16)][ceil(K/128)][64 lanes]
  const uint16_t* scales;  // [groups][N] bf16
  const uint8_t* zeros;    // [groups][N] or null (8)
  const uint16_t* bias;    // [N] or null
  uint16_t* out;           // [M][N] bf16
  int M, N, K;
  int group;               // 32, 64 or 128
  int epi;
};

constexpr int kW4Waves = 8;

__device__ __forceinline__ float bf16_float(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }

// + bias, activation, one rounding
__device__ __forceinline__ uint16_t decoder_epilogue(float v, const uint16_t* bias, int epi, int n) {
  if (epi == EPI_BIAS || epi == EPI_BIAS_GELU) v += bf16_float(bias[n]);
  if (epi == EPI_GELU || epi == EPI_BIAS_GELU) v = gelu_tanh(v);
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// Output (m, n) from the definition, term by term.  The kernel's offset form
// turns an infinite activation (or a sum that overflows) into a NaN of its
// own making; those outputs, rare and never in a finite model, are computed
// again this way, which gives them their IEEE class.
__device__ __forceinline__ float w4_dot(const W4Params& p, int m, int n) {
  const int kblocks = (p.K + 127) / 128;
  const uint32_t* W = reinterpret_cast<const uint32_t*>(p.W);
  float v = 0.f;
  for (int k = 0; k < p.K; ++k) {
    const int g = (k >> 3) & 3, j = (k >> 5) & 3, e = k & 7;
    const uint32_t word = W[(((int64_t)(n >> 4) * kblocks + (k >> 7)) * 64 + 16 * g + (n & 15)) * 4 + j];
    const int q = (word >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15;
    const int64_t at = (int64_t)(k / p.group) * p.N + n;
    const float z = p.zeros ? (float)p.zeros[at] : 8.0f;
    v = __builtin_fmaf(bf16_float(p.x[(int64_t)m * p.K + k]), ((float)q - z) * bf16_float(p.scales[at]), v);
  }
  return v;
}

// MB blocks of 16 activation rows by NB blocks of 16 columns per workgroup;
// its waves take every eighth 128-k step and meet in LDS, added in wave order.
template <int MB, int NB, int G>
__global__ void __launch_bounds__(kW4Waves * 64) gemm_w4(W4Params p) {
  __shared__ f32x4 red[kW4Waves][MB * NB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int kblocks = (p.K + 127) >> 7;
  const int nblocks = (p.N + 15) >> 4;
  const int m0 = blockIdx.y * (16 * MB);
  const int b0 = blockIdx.x * NB;
  f32x4 acc[MB][NB];
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
  for (int kb = wave; kb < kblocks; kb += kW4Waves) {
    u32x4 w[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)  // (a block past N reads the last one; its sums are dropped)
      w[b] = p.W[((int64_t)min(b0 + b, nblocks - 1) * kblocks + kb) * 64 + lane];
    u32x4 x[MB][4];
#pragma unroll
    for (int a = 0; a < MB; ++a) {
      const int m = m0 + 16 * a + lx;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = kb * 128 + 32 * j + 8 * lg;
        x[a][j] = u32x4{0u, 0u, 0u, 0u};
        if (m < p.M && k < p.K) x[a][j] = *reinterpret_cast<const u32x4*>(p.x + (int64_t)m * p.K + k);
      }
    }
#pragma unroll
    for (int g = 0; g < 128 / G; ++g) {
      constexpr int JG = G / 32;  // MFMAs per group
      const int group = kb * (128 / G) + g;
      const bool live = group * G < p.K;  // (x is zero in a group past K)
      f32x4 sx[MB];
#pragma unroll
      for (int a = 0; a < MB; ++a) {
        sx[a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < JG; ++j)
          sx[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[a][g * JG + j]), ones, sx[a],
                                                          0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int n = min(16 * (b0 + b) + lx, p.N - 1);
        const int64_t at = (int64_t)(live ? group : 0) * p.N + n;
        const float s = bf16_float(p.scales[at]);
        const float off = -16.0f - (p.zeros ? (float)p.zeros[at] : 8.0f);
        f32x4 t[MB];
#pragma unroll
        for (int a = 0; a < MB; ++a) t[a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < JG; ++j) {
          const uint32_t v = w[b][g * JG + j];
          u32x4 q;
          q[0] = ((v << 3) & 0x00780078u) | 0x41804180u;
          q[1] = ((v >> 1) & 0x00780078u) | 0x41804180u;
          q[2] = ((v >> 5) & 0x00780078u) | 0x41804180u;
          q[3] = ((v >> 9) & 0x00780078u) | 0x41804180u;
#pragma unroll
          for (int a = 0; a < MB; ++a)
            t[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[a][g * JG + j]),
                                                           __builtin_bit_cast(bf16x8, q), t[a], 0, 0, 0);
        }
#pragma unroll
        for (int a = 0; a < MB; ++a)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[a][b][i] = __builtin_fmaf(s, __builtin_fmaf(off, sx[a][i], t[a][i]), acc[a][b][i]);
      }
    }
  }
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) red[wave][a * NB + b][lane] = acc[a][b];
  __syncthreads();
  for (int e = threadIdx.x; e < MB * NB * 64; e += kW4Waves * 64) {
    const int ab = e >> 6, l = e & 63;
    f32x4 v = red[0][ab][l];
#pragma unroll
    for (int q = 1; q < kW4Waves; ++q) {
      const f32x4 u = red[q][ab][l];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += u[i];
    }
    // lane l of block (a, b): rows 16 a + 4 (l / 16) + i, column 16 b + l % 16
    const int n = 16 * (b0 + ab % NB) + (l & 15);
    if (n >= p.N) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + 16 * (ab / NB) + 4 * (l >> 4) + i;
      if (m >= p.M) continue;
      float o = v[i];
      if (!__builtin_isfinite(o)) o = w4_dot(p, m, n);
      p.out[(int64_t)m * p.N + n] = decoder_epilogue(o, p.bias, p.epi, n);
    }
  }
}

// Lays out codes [N][K] (one byte each, the low four bits taken) as packed
// words, one per thread; what pads N and K is code 0.
__global__ void __launch_bounds__(256) w4_pack(const uint8_t* codes, uint32_t* packed, int N, int K, int64_t words) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= words) return;
  const int kblocks = (K + 127) / 128;
  const int64_t block = i >> 8;
  const int j = i & 3, n = (int)(block / kblocks) * 16 + ((i >> 2) & 15), g = (i >> 6) & 3;
  const int k0 = (int)(block % kblocks) * 128 + 32 * j + 8 * g;
  uint32_t w = 0u;
  if (n < N) {
    for (int e = 0; e < 8; ++e)
      if (k0 + e < K) w |= (uint32_t)(codes[(int64_t)n * K + k0 + e] & 15) << (4 * ((e >> 1) + 4 * (e & 1)));
  }
  packed[i] = w;
}

}  // namespace mmk
