// Residual addition and layer norm of a decoder layer's stream, and its gradient.
//
//   h = T(x + residual)                T: the stream's type (bf16 or fp32)
//   m = mean(h),  r = 1 / sqrt(mean((h - m)^2) + eps)     fp32, from h as stored
//   y = (h - m) r w + b                w, b: bf16; one rounding
//
// The squares are of differences from the mean, a second sum over a row that is
// in registers anyway: mean(h^2) - m^2 would lose the variance of rows whose mean is
// large against their spread.
#pragma once

#include "rms_norm.hpp"
#include "wave_ops.hpp"

namespace mmk {

struct LayerNormParams {
  const void* x;           // [rows][ld_x]
  const void* residual;    // [rows][hidden] or null
  const uint16_t* weight;  // [hidden] bf16
  const uint16_t* bias;    // [hidden] bf16 or null
  void* h;                 // [rows][hidden], written when residual is given
  uint16_t* y;             // [rows][hidden] bf16
  float* mean;             // [rows]
  float* rstd;             // [rows]
  int64_t ld_x;
  int hidden;
  float eps;
};

struct LayerNormGradParams {
  const uint16_t* dy;      // [rows][hidden] bf16
  const void* h;           // [rows][hidden]
  const void* dres;        // [rows][hidden] or null: the gradient that reached h past the norm
  const uint16_t* weight;
  const float* mean;       // [rows]
  const float* rstd;       // [rows]
  void* dh;                // [rows][hidden]
  float* part;             // [gridDim.x][2][hidden] sums over each workgroup's rows
  int64_t rows;
  int hidden;
};

// Sums over a workgroup, the same in every thread: the waves' parts meet in LDS and are
// added in wave order.  `slot` holds one value per wave and is not reused within a row.
__device__ __forceinline__ float row_block_sum(float v, float* slot) {
  v = wave_sum(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < waves; ++w) v += slot[w];
  return v;
}
// Two at once.
__device__ __forceinline__ float2 row_block_sum(float2 v, float2* slot) {
  v = float2{wave_sum(v.x), wave_sum(v.y)};
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  v = float2{0.f, 0.f};
  for (int w = 0; w < waves; ++w) {
    v.x += slot[w].x;
    v.y += slot[w].y;
  }
  return v;
}

// One row per workgroup; thread t holds vectors t, t + T, ... (VPT of them)
// of 8 values, so that the row is read once and both sums run over registers.  Bound by
// HBM: 2047 x 5000 fp32 with a residual 28 us (143 MB, 5.1 TB/s); one row of 8192 3.3 us, the latency of a load and two sums.
template <bool F32, int VPT>
__global__ void __launch_bounds__(1024) layer_norm(LayerNormParams p) {
  __shared__ float slot[2][16];
  const int64_t row = blockIdx.x;
  const int T = blockDim.x;
  const int vectors = p.hidden >> 3;
  float v[VPT][8];
  float sum = 0.f;
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
    for (int j = 0; j < 8; ++j) sum += v[i][j];
  }
  const float mean = row_block_sum(sum, slot[0]) / (float)p.hidden;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if ((int)threadIdx.x + i * T >= vectors) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] -= mean;
      ss = __builtin_fmaf(v[i][j], v[i][j], ss);
    }
  }
  const float rstd = rsqrtf(row_block_sum(ss, slot[1]) / (float)p.hidden + p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * T;
    if (c >= vectors) continue;
    float w[8], b[8];
    load8<false>(p.weight, 8 * c, w);
    if (p.bias)
      load8<false>(p.bias, 8 * c, b);
    else {
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = __builtin_fmaf(v[i][j] * rstd, w[j], b[j]);
    *reinterpret_cast<u32x4*>(p.y + row * p.hidden + 8 * c) = pack8(v[i]);
  }
  if (threadIdx.x == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
}

// The gradient.  With n = (h - m) r and g = dy w:
//   dh = r (g - mean(g) - n mean(g n)) + dres,
//   dw = sum over rows of dy n,  db = sum over rows of dy.
// As rms_norm_grad: a workgroup takes rows b, b + G, ...; each thread keeps the same
// columns for every row, so its parts of dw and db stay in registers (fp32) and are
// written once; layer_norm_dparams adds the workgroups' parts in order.  AHEAD
// (up to 512 threads): a row's loads are issued before the row before is summed.
// Bound by HBM: 8192 x 4096 bf16 with dres 59 us with the parts' sum, 4.5 TB/s.
template <bool F32, int VPT, bool AHEAD>
__global__ void __launch_bounds__(AHEAD ? 512 : 1024) layer_norm_grad(LayerNormGradParams p) {
  __shared__ float2 slot[2][16];
  const int T = blockDim.x;
  const int vectors = p.hidden >> 3;
  const float inv_n = 1.0f / (float)p.hidden;
  Raw8<false> w[VPT];
  float dw[VPT][8], db[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * T;
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.f;
    w[i].clear();
    if (AHEAD && c < vectors) w[i].load(p.weight, 8 * c);
  }
  const bool has_dres = p.dres != nullptr;
  struct Row {
    Raw8<F32> h[VPT], dres[VPT];
    Raw8<false> dy[VPT];
    float mean, rstd;
  };
  auto load = [&](int64_t row, Row& v) __attribute__((always_inline)) {
    v.mean = p.mean[row];
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
        // (columns past the row: dy and w of 0 leave every sum as it is)
        v.h[i].clear();
        v.dy[i].clear();
        if constexpr (AHEAD) v.dres[i].clear();
      }
    }
  };
  auto process = [&](int64_t row, Row& v, int turn) __attribute__((always_inline)) {
    const float r = v.rstd, m = v.mean;
    float2 dot = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      // (in registers and widened here, not once before the loop; or, where
      // registers are short, read again)
      if constexpr (AHEAD)
        settle(w[i].w[0]);
      else if ((int)threadIdx.x + i * T < vectors)
        w[i].load(p.weight, 8 * (threadIdx.x + i * T));
      if ((int)threadIdx.x + i * T >= vectors) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dy = v.dy[i][j], t = dy * ((v.h[i][j] - m) * r);
        dw[i][j] += t;
        db[i][j] += dy;
        dot.x = __builtin_fmaf(dy, w[i][j], dot.x);
        dot.y = __builtin_fmaf(t, w[i][j], dot.y);
      }
    }
    // two slot rows in turn: a wave may start the next row's sum while
    // another still reads this one's
    dot = row_block_sum(dot, slot[turn]);
    const float a = dot.x * inv_n, b = dot.y * inv_n;
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
      for (int j = 0; j < 8; ++j) o[j] = r * (v.dy[i][j] * w[i][j] - a - (v.h[i][j] - m) * r * b);
      if (has_dres) {
        if constexpr (!AHEAD) v.dres[i].load(p.dres, row * p.hidden + 8 * c);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += v.dres[i][j];
      }
      store8<F32>(p.dh, row * p.hidden + 8 * c, o);
    }
  };
  if constexpr (AHEAD) {
    // (past the last row, this row's again, unused: another workgroup's may be
    // written meanwhile, where dh is dres)
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
    if (c >= vectors) continue;
    store8<true>(p.part, (int64_t)blockIdx.x * 2 * p.hidden + 8 * c, dw[i]);
    store8<true>(p.part, ((int64_t)blockIdx.x * 2 + 1) * p.hidden + 8 * c, db[i]);
  }
}

// Vectors of 8 columns that a workgroup of the kernel below sums side by side.  Measured (us,
// 2 / 4 / 8): 2048 x 1024 bf16 12.9 / 12.9 / -, 300 x 4096 bf16 8.0 / 4.7 / 4.6, 2048 x 128
// bf16 7.1 / 6.6 / -, 2048 x 8192 bf16 61.6 / 38.9 / 28.8, 2048 x 5000 fp32 - / 37.8 / 36.0,
// 2048 x 16384 bf16 - / 85 / 66.
__host__ __device__ constexpr int grad_few_lanes(int vpt) { return vpt == 1 ? 4 : 8; }

// The gradient of few rows in one launch: the first workgroups sum 8 `lanes` columns
// of dw and db each, reading dy and h for it once more, the others take one row
// each, as above.  T / lanes interleaved runs of rows per column.  A launch less and no parts
// in memory, for dy and h twice (the second time out of L2 in part): 300 x 5000 fp32 7.4 us
// (2.0 TB/s of what is needed once), 2048 x 8192 bf16 28.8 (4.7).
template <bool F32, int VPT>
__global__ void __launch_bounds__(1024) layer_norm_grad_few(LayerNormGradParams p, float* dweight, float* dbias) {
  constexpr int lanes = grad_few_lanes(VPT);
  __shared__ float2 slot[16];
  __shared__ float sums[2][64][8 * lanes];
  const int T = blockDim.x;
  const int vectors = p.hidden >> 3;
  const int wide = (vectors + lanes - 1) / lanes;  // workgroups of columns
  if ((int)blockIdx.x < wide) {
    const int lane = threadIdx.x & (lanes - 1), run = threadIdx.x / lanes, runs = T / lanes;
    const int c = blockIdx.x * lanes + lane;
    float dw[8], db[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.f;
    if (c < vectors) {
#pragma unroll 4
      for (int64_t row = run; row < p.rows; row += runs) {
        Raw8<F32> h;
        Raw8<false> dy;
        h.load(p.h, row * p.hidden + 8 * c);
        dy.load(p.dy, row * p.hidden + 8 * c);
        const float r = p.rstd[row], m = p.mean[row];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[j] += dy[j] * ((h[j] - m) * r);
          db[j] += dy[j];
        }
      }
    }
    // the runs of 16 lanes, then those sums, in a fixed order
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j] = row_sum<lanes>(dw[j]);
      db[j] = row_sum<lanes>(db[j]);
    }
    const int part = threadIdx.x >> 4, l = threadIdx.x & 15;
    if (l < lanes) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sums[0][part][8 * l + j] = dw[j];
        sums[1][part][8 * l + j] = db[j];
      }
    }
    __syncthreads();
    const int what = threadIdx.x >> 6, at = threadIdx.x & 63;
    const int col = blockIdx.x * 8 * lanes + at;
    if (what < 2 && at < 8 * lanes && col < p.hidden) {
      float s = 0.f;
#pragma unroll 8
      for (int q = 0; q < (T >> 4); ++q) s += sums[what][q][at];
      (what ? dbias : dweight)[col] = s;
    }
    return;
  }
  const int64_t row = (int64_t)blockIdx.x - wide;
  const float r = p.rstd[row], m = p.mean[row];
  Raw8<F32> h[VPT];
  Raw8<false> dy[VPT], w[VPT];
  float2 dot = {0.f, 0.f};
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
  for (int i = 0; i < VPT; ++i) {
    if ((int)threadIdx.x + i * T >= vectors) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float g = dy[i][j] * w[i][j];
      dot.x += g;
      dot.y = __builtin_fmaf(g, (h[i][j] - m) * r, dot.y);
    }
  }
  dot = row_block_sum(dot, slot);
  const float a = dot.x * (1.0f / (float)p.hidden), b = dot.y * (1.0f / (float)p.hidden);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * T;
    if (c >= vectors) continue;
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = r * (dy[i][j] * w[i][j] - a - (h[i][j] - m) * r * b);
    if (p.dres) {
      Raw8<F32> dres;
      dres.load(p.dres, row * p.hidden + 8 * c);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += dres[j];
    }
    store8<F32>(p.dh, row * p.hidden + 8 * c, o);
  }
}

// dw and db from the workgroups' parts [parts][2][hidden]: 32 columns per
// workgroup (8 lanes of four) by 32 interleaved runs, joined in LDS in a fixed
// order; blockIdx.y says which of the two.
__global__ void __launch_bounds__(256) layer_norm_dparams(const float* part, float* dweight, float* dbias, int parts,
                                                          int hidden) {
  __shared__ f32x4 slot[32][8];
  const int lane = threadIdx.x & 7, run = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + 4 * lane;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < hidden) {
#pragma unroll 4
    for (int b = run; b < parts; b += 32) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(part + ((int64_t)b * 2 + blockIdx.y) * hidden + c);
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
    *reinterpret_cast<f32x4*>((blockIdx.y ? dbias : dweight) + c) = s;
  }
}

}  // namespace mmk
