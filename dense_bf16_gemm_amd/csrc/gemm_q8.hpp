// Products of e4m3 operands with row scales:
//   out[m][n] = epi(xs[m] ws[n] sum_k x[m][k] W[n][k] + bias[n]),
// x [M][K] and W [N][K] e4m3 (K contiguous), fp32 scales, bf16 output.  The
// sums are fp32; the scales are applied to the sum, then the epilogue, then
// one rounding.  v_mfma_f32_16x16x128_f8f6f4 does 65536 products and sums in
// 32 cycles of a SIMD, twice the bf16 rate.  Its lane holds 32 consecutive
// bytes of k in hardware order; any order serves as long as both operands use
// the same, so fragments are two 16-byte chunks wherever they are best read.
#pragma once

#include "gemm_w4.hpp"

namespace mmk {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Q8Params {
  const uint8_t* x;       // [M][K] e4m3
  const float* xs;        // [M]
  const uint8_t* W;       // [N][K] e4m3
  const float* ws;        // [N]
  const uint16_t* bias;   // [N] or null
  uint16_t* out;          // [M][N] bf16
  int M, N, K;
  int epi;
  int tiles_m, tiles_n;
};

__device__ __forceinline__ i32x8 join_chunks(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// (unit block scales: the instruction without scale operands)
__device__ __forceinline__ f32x4 mfma_q8(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Few rows: as gemm_w4, MB blocks of 16 rows by NB blocks of 16 columns, the
// waves taking every eighth 128-k step.
template <int MB, int NB>
__global__ void __launch_bounds__(kW4Waves * 64) gemm_q8_rows(Q8Params p) {
  __shared__ f32x4 red[kW4Waves][MB * NB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int ksteps = (p.K + 127) >> 7;
  const int m0 = blockIdx.y * (16 * MB);
  const int n0 = blockIdx.x * (16 * NB);
  f32x4 acc[MB][NB];
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int st = wave; st < ksteps; st += kW4Waves) {
    const int k = st * 128 + 16 * lg;
    i32x8 w[NB], x[MB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int n = min(n0 + 16 * b + lx, p.N - 1);
      const uint8_t* r = p.W + (int64_t)n * p.K;
      w[b] = join_chunks(k < p.K ? *reinterpret_cast<const u32x4*>(r + k) : zero,
                         k + 64 < p.K ? *reinterpret_cast<const u32x4*>(r + k + 64) : zero);
    }
#pragma unroll
    for (int a = 0; a < MB; ++a) {
      const int m = m0 + 16 * a + lx;
      const uint8_t* r = p.x + (int64_t)m * p.K;
      x[a] = join_chunks(m < p.M && k < p.K ? *reinterpret_cast<const u32x4*>(r + k) : zero,
                         m < p.M && k + 64 < p.K ? *reinterpret_cast<const u32x4*>(r + k + 64) : zero);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int a = 0; a < MB; ++a) acc[a][b] = mfma_q8(x[a], w[b], acc[a][b]);
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
    const int n = n0 + 16 * (ab % NB) + (l & 15);
    if (n >= p.N) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + 16 * (ab / NB) + 4 * (l >> 4) + i;
      if (m < p.M)
        p.out[(int64_t)m * p.N + n] = decoder_epilogue(v[i] * p.xs[m] * p.ws[n], p.bias, p.epi, n);
    }
  }
}

// Many rows: 128 x 128 tiles, four waves of 64 x 64, 128-k steps in two LDS
// buffers filled by buffer-to-LDS copies (rows past M or N, and chunks past K,
// lie past the descriptors' ends and arrive as zeros).  Chunk c of a row sits
// at position c ^ (row & 7).
__global__ void __launch_bounds__(256) gemm_q8_tile(Q8Params p) {
  __shared__ __attribute__((aligned(1024))) char smem[2][32768];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  int tm, tn;
  tile_coords(remap_workgroup(blockIdx.x, gridDim.x, 1), p.tiles_m, p.tiles_n, 8, &tm, &tn);
  const int m0 = __builtin_amdgcn_readfirstlane(tm * 128), n0 = __builtin_amdgcn_readfirstlane(tn * 128);
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const uint32_t K = (uint32_t)p.K;
  const int steps = (p.K + 127) >> 7;
  const uint32_t mrec = (uint32_t)min(p.M - m0, 128) * K, nrec = (uint32_t)min(p.N - n0, 128) * K;
  const __amdgpu_buffer_rsrc_t rx =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.x + (int64_t)m0 * p.K), (short)0, (int)mrec, 0x00020000);
  const __amdgpu_buffer_rsrc_t rw =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.W + (int64_t)n0 * p.K), (short)0, (int)nrec, 0x00020000);
  const int crow = lane >> 3;
  const uint32_t chunk = 16u * ((lane & 7) ^ crow);
  auto copy = [&](int st) __attribute__((always_inline)) {
    char* dst = smem[st & 1];
    const uint32_t k = 128u * (uint32_t)st + chunk;
    const uint32_t off = k | (k < K ? 0u : 0x80000000u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * (4 * wave + i);  // 8 rows per copy
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw, (__attribute__((address_space(3))) void*)(dst + r * 128), 16, off + (uint32_t)(r + crow) * K, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (__attribute__((address_space(3))) void*)(dst + 16384 + r * 128),
                                               16, off + (uint32_t)(r + crow) * K, 0, 0, 0);
    }
  };
  f32x4 acc[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto frag = [&](const char* rows, int row) __attribute__((always_inline)) {
    const char* r = rows + (row + lx) * 128;
    const int key = lx & 7;
    return join_chunks(*reinterpret_cast<const u32x4*>(r + 16 * (lg ^ key)),
                       *reinterpret_cast<const u32x4*>(r + 16 * ((lg + 4) ^ key)));
  };
  if (steps > 0) copy(0);
  for (int st = 0; st < steps; ++st) {
    // this wave's copies of step st have landed, then every wave's; and every
    // wave is past its reads of step st - 1
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (st + 1 < steps) copy(st + 1);
    const char* src = smem[st & 1];
    i32x8 w[4], x[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) w[b] = frag(src, wn + 16 * b);
#pragma unroll
    for (int a = 0; a < 4; ++a) x[a] = frag(src + 16384, wm + 16 * a);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[a][b] = mfma_q8(w[b], x[a], acc[a][b]);
  }
  // lane (lg, lx): column block b's columns 4 lg .. + 3 of row 16 a + lx
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int m = m0 + wm + 16 * a + lx;
    if (m >= p.M) continue;
    const float xs = p.xs[m];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + wn + 16 * b + 4 * lg + i;
        if (n < p.N)
          p.out[(int64_t)m * p.N + n] = decoder_epilogue(acc[a][b][i] * xs * p.ws[n], p.bias, p.epi, n);
      }
  }
}

}  // namespace mmk
