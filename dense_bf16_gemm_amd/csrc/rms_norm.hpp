// Residual addition and root-mean-square norm of a decoder layer's stream,
// with a bf16 or an 8-bit output, and its gradient.
//
//   h = T(x + residual)            T: the stream's type (bf16 or fp32)
//   r = 1 / sqrt(mean(h^2) + eps)  fp32, from h as stored
//   y = h r w                      w: bf16 weight
//   bf16 output: y, rounded once.  8-bit output: s = max(max|y| / 448, 2^-126),
//   q = e4m3(y / s): a row's largest value lands on e4m3's largest.
//
// One pass over memory: a row lives in its workgroup's registers between the
// sum of squares, the maximum and the output.  Bound by HBM: 7 bytes per
// element (bf16 stream, residual, 8-bit output).  4096 x 8192 takes 47.8 us, 4.9
// TB/s (a large copy reaches 4.8); one row 4 us, which is the launch, one trip to
// memory and three reductions.
#pragma once

#include "mm_device.hpp"

namespace mmk {

constexpr int kNormMaxHidden = 32768;  // 1024 threads x 4 vectors of 8

struct RmsNormParams {
  const void* x;           // [rows][ld_x]
  const void* residual;    // [rows][hidden] or null
  const uint16_t* weight;  // [hidden] bf16
  void* h;                 // [rows][hidden], written when residual is given
  void* y;                 // [rows][hidden] bf16 or e4m3
  float* stat;             // [rows]: r (bf16 output) or s (8-bit output)
  int64_t rows, ld_x;
  int hidden;
  float eps;
};

struct RmsNormGradParams {
  const uint16_t* dy;      // [rows][hidden] bf16
  const void* h;           // [rows][hidden]
  const void* dres;        // [rows][hidden] or null: the gradient that reached h past the norm
  const uint16_t* weight;
  const float* rstd;       // [rows]
  void* dh;                // [rows][hidden]
  float* part;             // [gridDim.x][hidden] sums over each workgroup's rows
  int64_t rows;
  int hidden;
};

// Eight consecutive values as stored: 16 bytes of bf16 or 32 of fp32.
template <bool F32>
struct Raw8 {
  u32x4 w[F32 ? 2 : 1];
  // (16-byte aligned rows)
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const char*>(base) + i * (F32 ? 4 : 2));
    w[0] = p[0];
    if constexpr (F32) w[1] = p[1];
  }
  __device__ __forceinline__ void clear() {
    w[0] = u32x4{0u, 0u, 0u, 0u};
    if constexpr (F32) w[1] = w[0];
  }
  __device__ __forceinline__ float operator[](int j) const {
    // (through a scalar: a bit cast of a vector's element takes element 0)
    uint32_t b;
    if constexpr (F32)
      b = w[j >> 2][j & 3];
    else
      b = j & 1 ? w[0][j >> 1] & 0xffff0000u : w[0][j >> 1] << 16;
    return __builtin_bit_cast(float, b);
  }
};

template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&v)[8]) {
  Raw8<F32> r;
  r.load(base, i);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = r[j];
}

__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&v)[8]) {
  if constexpr (F32) {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(base) + i);
    p[0] = f32x4{v[0], v[1], v[2], v[3]};
    p[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + i) = pack8(v);
  }
}

// Sum and maximum over a workgroup, the same in every thread.  The waves'
// parts meet in LDS and are added in wave order, so results do not depend on
// timing.  `slot` holds one value per wave and is not reused within a row.
__device__ __forceinline__ float block_sum(float v, float* slot) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < waves; ++w) v += slot[w];
  return v;
}
// (of the bit patterns of non-negative floats: they order as unsigned
// numbers, and a NaN lies above infinity, so it is kept)
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* slot) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0u;
  for (int w = 0; w < waves; ++w) v = max(v, slot[w]);
  return v;
}

// One row per workgroup; thread t holds vectors t, t + T, ... (VPT of them)
// of 8 values.
template <bool F32, bool Q8, int VPT>
__global__ void __launch_bounds__(1024) rms_norm(RmsNormParams p) {
  __shared__ float slot_sum[16];
  __shared__ uint32_t slot_max[16];
  const int64_t row = blockIdx.x;
  const int T = blockDim.x;
  const int vectors = p.hidden >> 3;
  float v[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * T;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (c < vectors) {
      load8<F32>(p.x, row * p.ld_x + 8 * c, v[i]);
      if (p.residual) {
        float r[8];
        load8<F32>(p.residual, row * p.hidden + 8 * c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] += r[j];
          // the norm is of h as the stream stores it
          if constexpr (!F32) v[i][j] = static_cast<float>(static_cast<__bf16>(v[i][j]));
        }
        store8<F32>(p.h, row * p.hidden + 8 * c, v[i]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(v[i][j], v[i][j], ss);
  }
  ss = block_sum(ss, slot_sum);
  // (the reciprocal root in one operation: of 1 / sqrt, rounded twice, 39 % of the rows
  // were not the nearest fp32 value, of this 28 %)
  const float rstd = rsqrtf(ss / (float)p.hidden + p.eps);
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * T;
    if (c >= vectors) continue;
    float w[8];
    load8<false>(p.weight, 8 * c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = v[i][j] * rstd * w[j];
      if constexpr (Q8) top = max(top, __builtin_bit_cast(uint32_t, v[i][j]) & 0x7fffffffu);
    }
    if constexpr (!Q8) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.y) + row * p.hidden + 8 * c) = pack8(v[i]);
  }
  if constexpr (Q8) {
    top = block_max(top, slot_max);
    float s = __builtin_bit_cast(float, top) / 448.0f;
    s = s < 0x1p-126f ? 0x1p-126f : s;  // (a NaN stays)
    // y / s: the product with 1 / s, then the remainder that it leaves, by one FMA
    // each (y - q s is exact unless it underflows).  The product alone decides
    // wrongly where a quotient lies on the border of two codes, which it often
    // does: the values have few bits.  4096 x 8192: 47.3 us with the product alone, 47.8
    // so, 50.3 with the division operator.
    const float inv = 1.0f / s;
    const float d = s > 3.4028235e38f ? 3.4028235e38f : s;  // (y / inf is 0 for a finite y)
    auto quotient = [&](float y) __attribute__((always_inline)) {
      const float q = y * inv;
      return __builtin_fmaf(__builtin_fmaf(-q, d, y), inv, q);
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * T;
      if (c >= vectors) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = quotient(v[i][j]);
      int lo = 0, hi = 0;
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[i][0], v[i][1], lo, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[i][2], v[i][3], lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[i][4], v[i][5], hi, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[i][6], v[i][7], hi, true);
      reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + row * p.hidden)[c] = uint2{(uint32_t)lo, (uint32_t)hi};
    }
    if (threadIdx.x == 0) p.stat[row] = s;
  } else {
    if (threadIdx.x == 0) p.stat[row] = rstd;
  }
}

// The gradient.  With n = h r and g = dy w:
//   dh = r (g - n mean(g n)) + dres,   dw = sum over rows of dy n.
// A workgroup takes rows b, b + G, ...; each thread keeps the same columns
// for every row, so its part of dw stays in registers (fp32) and is written
// once; rms_norm_dweight adds the workgroups' parts in order.
//
// A row's vectors are held as stored and widened where they are used, which
// keeps four vectors per thread within the 128 registers of 1024 threads.
// AHEAD (up to 512 threads): a row's loads, dres among them, are issued before the
// row before is summed, and the weight stays in registers.  8192 x 4096 bf16 with dres:
// 58.7 us (4.6 TB/s); 63.6 without AHEAD, which loads dres and the weight after the sum, on
// twice the workgroups and so with twice the parts of dw to write and add.  The
// compiler waits for most of those loads ahead of the sum all the same (around the
// branch on dres it merges registers that are being loaded with ones that are not),
// so what keeps the memory busy meanwhile are the CU's other waves.
template <bool F32, int VPT, bool AHEAD>
__global__ void __launch_bounds__(AHEAD ? 512 : 1024) rms_norm_grad(RmsNormGradParams p) {
  __shared__ float slot[2][16];
  const int T = blockDim.x;
  const int vectors = p.hidden >> 3;
  const float inv_n = 1.0f / (float)p.hidden;
  Raw8<false> w[VPT];
  float dw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * T;
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    w[i].clear();
    if (AHEAD && c < vectors) w[i].load(p.weight, 8 * c);
  }
  const bool has_dres = p.dres != nullptr;
  struct Row {
    Raw8<F32> h[VPT], dres[VPT];
    Raw8<false> dy[VPT];
    float rstd;
  };
  auto load = [&](int64_t row, Row& v) __attribute__((always_inline)) {
    v.rstd = p.rstd[row];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * T;
      if (c < vectors) {
        v.h[i].load(p.h, row * p.hidden + 8 * c);
        v.dy[i].load(p.dy, row * p.hidden + 8 * c);
        if constexpr (AHEAD) {
          if (has_dres) v.dres[i].load(p.dres, row * p.hidden + 8 * c);
        }
      } else {
        v.h[i].clear();
        v.dy[i].clear();
        if constexpr (AHEAD) v.dres[i].clear();
      }
    }
  };
  auto process = [&](int64_t row, Row& v, int turn) __attribute__((always_inline)) {
    const float r = v.rstd;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      // (in registers and widened here, not once before the loop; or, where
      // registers are short, read again)
      if constexpr (AHEAD)
        settle(w[i].w[0]);
      else if ((int)threadIdx.x + i * T < vectors)
        w[i].load(p.weight, 8 * (threadIdx.x + i * T));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = v.dy[i][j] * (v.h[i][j] * r);
        dw[i][j] += t;
        dot = __builtin_fmaf(t, w[i][j], dot);
      }
    }
    // two slot rows in turn: a wave may start the next row's sum while
    // another still reads this one's
    const float mean = block_sum(dot, slot[turn]) * inv_n;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * T;
      // (widened again, not kept across the sum)
      settle(v.dy[i].w[0]);
      settle(w[i].w[0]);
#pragma unroll
      for (int q = 0; q < (F32 ? 2 : 1); ++q) settle(v.h[i].w[q]);
      if (c >= vectors) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = r * (v.dy[i][j] * w[i][j] - v.h[i][j] * r * mean);
      if (has_dres) {
        if constexpr (!AHEAD) v.dres[i].load(p.dres, row * p.hidden + 8 * c);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += v.dres[i][j];
      }
      store8<F32>(p.dh, row * p.hidden + 8 * c, o);
    }
  };
  if constexpr (AHEAD) {
    // the next row's loads go out before this row's sum is waited for (past the
    // last, this row's again, unused: another workgroup's may be written meanwhile,
    // where dh is dres)
    Row a, b;
    const int64_t G = gridDim.x;
    load(blockIdx.x, a);
    for (int64_t row = blockIdx.x; row < p.rows; row += 2 * G) {
      load(row + G < p.rows ? row + G : row, b);
      process(row, a, 0);
      load(row + 2 * G < p.rows ? row + 2 * G : row, a);
      if (row + G < p.rows) process(row + G, b, 1);
    }
  } else {
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
      Row a;
      load(row, a);
      process(row, a, turn);
      turn ^= 1;
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * T;
    if (c < vectors) store8<true>(p.part, (int64_t)blockIdx.x * p.hidden + 8 * c, dw[i]);
  }
}

// The gradient of few rows in one launch (a second one costs the call 4 us, and
// a row per CU leaves most of a CU idle): the first workgroups sum 64 columns of
// dw each, reading dy and h for it once more, the others take one row each, as
// above.  1 x 4096 takes 2.7 us, which is latency, 512 x 8192 10 (3.4 TB/s), 2048 x 1024
// 16.6 (1 TB/s): there 16 workgroups sum the columns, whose threads have one of
// their 32 rows in flight at a time.
template <bool F32, int VPT>
__global__ void __launch_bounds__(1024) rms_norm_grad_few(RmsNormGradParams p, float* dweight) {
  __shared__ float slot[16];
  __shared__ float sums[128][64];
  const int T = blockDim.x;
  const int vectors = p.hidden >> 3;
  const int wide = (vectors + 7) >> 3;  // workgroups of columns
  if ((int)blockIdx.x < wide) {
    // 8 lanes of 8 columns by T / 8 interleaved runs of rows
    const int lane = threadIdx.x & 7, run = threadIdx.x >> 3, runs = T >> 3;
    const int c = blockIdx.x * 8 + lane;
    float dw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = 0.f;
    if (c < vectors) {
#pragma unroll 4
      for (int64_t row = run; row < p.rows; row += runs) {
        Raw8<F32> h;
        Raw8<false> dy;
        h.load(p.h, row * p.hidden + 8 * c);
        dy.load(p.dy, row * p.hidden + 8 * c);
        const float r = p.rstd[row];
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] += dy[j] * (h[j] * r);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[run][8 * lane + j] = dw[j];
    __syncthreads();
    const int col = blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x < 64 && col < p.hidden) {
      float s = 0.f;
      for (int b = 0; b < runs; ++b) s += sums[b][threadIdx.x];
      dweight[col] = s;
    }
    return;
  }
  const int64_t row = (int64_t)blockIdx.x - wide;
  const float r = p.rstd[row];
  Raw8<F32> h[VPT];
  Raw8<false> dy[VPT], w[VPT];
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * T;
    h[i].clear();
    dy[i].clear();
    w[i].clear();
    if (c < vectors) {
      h[i].load(p.h, row * p.hidden + 8 * c);
      dy[i].load(p.dy, row * p.hidden + 8 * c);
      w[i].load(p.weight, 8 * c);
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dot = __builtin_fmaf(dy[i][j] * (h[i][j] * r), w[i][j], dot);
  const float mean = block_sum(dot, slot) * (1.0f / (float)p.hidden);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * T;
    if (c >= vectors) continue;
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = r * (dy[i][j] * w[i][j] - h[i][j] * r * mean);
    if (p.dres) {
      Raw8<F32> dres;
      dres.load(p.dres, row * p.hidden + 8 * c);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += dres[j];
    }
    store8<F32>(p.dh, row * p.hidden + 8 * c, o);
  }
}

// dw[c] = sum over b of part[b][c]: 32 columns per workgroup (8 lanes of four)
// by 32 interleaved runs of b, joined in LDS in a fixed order.
__global__ void __launch_bounds__(256) rms_norm_dweight(const float* part, float* dw, int parts, int hidden) {
  __shared__ f32x4 slot[32][8];
  const int lane = threadIdx.x & 7, run = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + 4 * lane;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < hidden) {
    for (int b = run; b < parts; b += 32) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(part + (int64_t)b * hidden + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += v[j];
    }
  }
  slot[run][lane] = s;
  __syncthreads();
  if (run == 0 && c < hidden) {
    for (int b = 1; b < 32; ++b) {
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += slot[b][lane][j];
    }
    *reinterpret_cast<f32x4*>(dw + c) = s;
  }
}

}  // namespace mmk
