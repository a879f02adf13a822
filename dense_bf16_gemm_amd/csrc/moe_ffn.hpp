// Mixture-of-experts FFN of a few tokens (a decode step):
//   out[t] = sum over j < k of w[t][j] Wd_e (SiLU(Wg_e x[t]) * (Wu_e x[t])),  e = experts[t][j],
// where experts[t] are the k largest logits of token t (ties: the lower index) and
// w[t] their softmax, over these k or over all logits.  A logit of minus infinity
// takes no part: a token with fewer than k others has slots without an expert (-1,
// weight 0).
//
// Bound by reading the weights of the experts in use, 6 H I bytes each, once.
// Three launches: moe_route chooses and groups the tokens by expert, moe_gate_up
// leaves w SiLU(g) u, moe_down sums over experts.  The intermediate is kept as two
// bf16 numbers, high and low part, 16 bits of significand: as one, its rounding
// would add as much error to an output as the output's own.
#pragma once

#include "gemm_q8.hpp"

namespace mmk {

constexpr int kMoeTokens = 64, kMoeExperts = 512, kMoeTopK = 16;
constexpr int kMoeWaves = 8;

// Which experts are in use, in ascending order, and whose tokens: expert act[q] has
// rows start[q] .. start[q + 1] - 1, row r being token tok[r] with weight wt[r].
struct MoeTables {
  int count;  // experts in use
  int act[kMoeExperts];
  int start[kMoeExperts + 1];
  int tok[kMoeTokens * kMoeTopK];
  float wt[kMoeTokens * kMoeTopK];
};

struct MoeParams {
  const uint16_t* x;      // [T][H] bf16
  const float* logits;    // [T][E]
  const uint16_t* wg;     // [E][I][H] bf16
  const uint16_t* wu;     // [E][I][H]
  const uint16_t* wd;     // [E][H][I]
  uint16_t* out;          // [T][H] bf16
  int* experts;           // [T][k]
  float* weights;         // [T][k]
  MoeTables* tab;
  uint16_t* mid;          // [T k][2][I]: high and low parts of the intermediate
  int T, E, H, I, k;
  int renormalize;
};

// Floats as unsigned numbers of the same order; NaN above all, both zeros alike,
// minus infinity as 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f);
  if (f != f) return 0xffffffffu;
  if (f == 0.f) return 0x80000000u;
  if (b == 0xff800000u) return 0u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// One workgroup of 16 waves; a wave takes every 16th token.  VPL: logits per lane.
template <int VPL>
__global__ void __launch_bounds__(1024) moe_route(MoeParams p) {
  __shared__ uint32_t mask[kMoeExperts][2];  // the tokens of an expert
  __shared__ int first[kMoeExperts];
  __shared__ int id[kMoeTokens * kMoeTopK];
  __shared__ float share[kMoeTokens * kMoeTopK];
  __shared__ int wave_active[16], wave_rows[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < p.E; e += 1024) mask[e][0] = mask[e][1] = 0u;
  __syncthreads();
  for (int t = wave; t < p.T; t += 16) {
    uint32_t key[VPL];
    uint32_t all[VPL];
#pragma unroll
    for (int r = 0; r < VPL; ++r) {
      const int e = 64 * r + lane;
      all[r] = key[r] = e < p.E ? order_key(p.logits[(int64_t)t * p.E + e]) : 0u;
    }
    uint32_t mine = 0u, top = 0u;  // lane j: the j-th largest
    int mine_id = -1;
    for (int j = 0; j < p.k; ++j) {
      uint32_t m = key[0];
#pragma unroll
      for (int r = 1; r < VPL; ++r) m = max(m, key[r]);
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
      if (m == 0u) break;
      if (j == 0) top = m;
      int at = -1;
#pragma unroll
      for (int r = 0; r < VPL; ++r) {
        const uint64_t b = __ballot(key[r] == m);
        if (at < 0 && b) {
          const int l = __builtin_ctzll(b);
          at = 64 * r + l;
          if (lane == l) key[r] = 0u;
        }
      }
      if (lane == j) {
        mine = m;
        mine_id = at;
      }
    }
    const float peak = key_value(top);
    const float part = mine ? expf(key_value(mine) - peak) : 0.f;
    float sum = part;
    if (!p.renormalize) {
      sum = 0.f;
#pragma unroll
      for (int r = 0; r < VPL; ++r) sum += all[r] ? expf(key_value(all[r]) - peak) : 0.f;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane < p.k) {
      const int s = t * p.k + lane;
      const float w = mine ? part / sum : 0.f;
      p.experts[s] = id[s] = mine_id;
      p.weights[s] = share[s] = w;
      if (mine) atomicOr(&mask[mine_id][t >> 5], 1u << (t & 31));
    }
  }
  __syncthreads();
  // places of the experts in use and of their rows
  const int e = threadIdx.x;
  const int rows = e < p.E ? __popc(mask[e][0]) + __popc(mask[e][1]) : 0;
  const uint64_t active = __ballot(rows > 0);
  int upto = rows;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) {
    wave_active[wave] = __popcll(active);
    wave_rows[wave] = upto;
  }
  __syncthreads();
  int q = __popcll(active & ((uint64_t(1) << lane) - 1)), at = upto - rows, used = 0, total = 0;
  for (int w = 0; w < 16; ++w) {
    if (w < wave) {
      q += wave_active[w];
      at += wave_rows[w];
    }
    used += wave_active[w];
    total += wave_rows[w];
  }
  if (rows > 0) {
    p.tab->act[q] = e;
    p.tab->start[q] = at;
    first[e] = at;
  }
  if (threadIdx.x == 0) {
    p.tab->count = used;
    p.tab->start[used] = total;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < p.T * p.k; s += 1024) {
    const int x = id[s], t = s / p.k;
    if (x < 0) continue;
    const uint32_t lo = mask[x][0], hi = mask[x][1];
    const int before = t < 32 ? __popc(lo & ((1u << t) - 1u)) : __popc(lo) + __popc(hi & ((1u << (t - 32)) - 1u));
    p.tab->tok[first[x] + before] = t;
    p.tab->wt[first[x] + before] = share[s];
  }
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A float as two bf16: the high part cut, the low part rounded (2^-16 of the
// value together).  What is not finite stays in the high part.
__device__ __forceinline__ void split_bf16(float v, uint16_t* hi, uint16_t* lo) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  if ((b & 0x7f800000u) == 0x7f800000u) {
    *hi = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    *lo = 0;
    return;
  }
  *hi = (uint16_t)(b >> 16);
  *lo = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v - __builtin_bit_cast(float, b & 0xffff0000u)));
}

// SiLU(g) u, as the fused FFN has it
__device__ __forceinline__ float swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// A unit of work: 8 columns of I of one expert, gate and up rows together as the 16
// columns of an MFMA block.  The eight waves take every eighth step of 64 k, each
// step's loads one step ahead, and meet in LDS, added in wave order.
// MB: blocks of 16 tokens.
template <int MB>
__global__ void __launch_bounds__(kMoeWaves * 64) moe_gate_up(MoeParams p) {
  __shared__ float red[kMoeWaves][MB][64][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const MoeTables* tab = p.tab;
  const int cols = p.I >> 3, units = __builtin_amdgcn_readfirstlane(tab->count) * cols;
  const int H = p.H, steps = (H + 63) >> 6;
  const __amdgpu_buffer_rsrc_t rx =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p.x), (short)0, p.T * H * 2, 0x00020000);
  // chunks of the last step past H: zeros on both sides
  bool out[2];
  uint32_t tail[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    out[j] = 64 * (steps - 1) + 32 * j + 8 * lg >= H;
    tail[j] = out[j] ? 0x80000000u : 0u;
  }
  struct Step {
    u32x4 w[2], x[MB][2];
  };
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int q = __builtin_amdgcn_readfirstlane(unit / cols), c0 = 8 * (unit - q * cols);
    const int e = __builtin_amdgcn_readfirstlane(tab->act[q]), s = __builtin_amdgcn_readfirstlane(tab->start[q]);
    const int n = __builtin_amdgcn_readfirstlane(tab->start[q + 1]) - s;
    const uint16_t* w = (lx < 8 ? p.wg : p.wu) + ((int64_t)e * p.I + c0 + (lx & 7)) * H + 8 * lg;
    uint32_t xo[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
      xo[a] = 16 * a + lx < n ? (uint32_t)tab->tok[s + 16 * a + lx] * (uint32_t)H * 2u + 16u * (uint32_t)lg : 0x80000000u;
    auto load = [&](int st, Step& t) __attribute__((always_inline)) {
      const bool last = st == steps - 1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        t.w[j] = *reinterpret_cast<const u32x4*>(w + (last && out[j] ? -8 * lg : 64 * st + 32 * j));
#pragma unroll
        for (int a = 0; a < MB; ++a)
          if (16 * a < n) t.x[a][j] = load_chunk(rx, (xo[a] + 64u * j) | (last ? tail[j] : 0u), 128u * (uint32_t)st);
      }
    };
    f32x4 acc[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) acc[a] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int st, Step& t, Step& next) __attribute__((always_inline)) {
      load(min(st + kMoeWaves, steps - 1), next);
      const bool last = st == steps - 1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (last && out[j]) t.w[j] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int a = 0; a < MB; ++a)
          if (16 * a < n) acc[a] = mfma_bf16(t.x[a][j], t.w[j], acc[a]);
      }
    };
    if (wave < steps) {
      Step s0, s1;
      load(wave, s0);
      for (int st = wave; st < steps; st += 2 * kMoeWaves) {
        step(st, s0, s1);
        if (st + kMoeWaves < steps) step(st + kMoeWaves, s1, s0);
      }
    }
    __syncthreads();  // (the unit before has been read)
#pragma unroll
    for (int a = 0; a < MB; ++a) *reinterpret_cast<f32x4*>(red[wave][a][lane]) = acc[a];
    __syncthreads();
    for (int i = threadIdx.x; i < MB * 128; i += kMoeWaves * 64) {
      const int m = i >> 3, c = i & 7;
      if (m >= n) continue;
      const int a = m >> 4, l = 16 * ((m & 15) >> 2) + c, f = m & 3;
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int v = 0; v < kMoeWaves; ++v) {
        g += red[v][a][l][f];
        u += red[v][a][l + 8][f];
      }
      uint16_t hi, lo;
      split_bf16(tab->wt[s + m] * swiglu(g, u), &hi, &lo);
      uint16_t* o = p.mid + (int64_t)(s + m) * 2 * p.I + c0 + c;
      o[0] = hi;
      o[p.I] = lo;
    }
  }
}

// 16 columns of H per workgroup: the steps of 64 values of I, expert after expert,
// are dealt to the waves in equal runs.  A wave leaves an expert's sums in LDS,
// in a row per token of its own, and the waves' rows are added in wave order.
template <int MB>
__global__ void __launch_bounds__(kMoeWaves * 64) moe_down(MoeParams p) {
  __shared__ float sums[kMoeWaves][16 * MB][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const MoeTables* tab = p.tab;
  const int I = p.I, steps = (I + 63) >> 6;
  const int count = __builtin_amdgcn_readfirstlane(tab->count);
  const int64_t total = (int64_t)count * steps;
  const int lo = (int)(total * wave / kMoeWaves), hi = (int)(total * (wave + 1) / kMoeWaves);
  const int n0 = blockIdx.x * 16;
  for (int i = lane; i < 16 * MB * 16; i += 64) (&sums[wave][0][0])[i] = 0.f;
  const __amdgpu_buffer_rsrc_t rx =
      __builtin_amdgcn_make_buffer_rsrc(p.mid, (short)0, p.T * p.k * I * 4, 0x00020000);
  const int64_t row = min(n0 + lx, p.H - 1);
  bool out[2];
  uint32_t tail[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    out[j] = 64 * (steps - 1) + 32 * j + 8 * lg >= I;
    tail[j] = out[j] ? 0x80000000u : 0u;
  }
  struct Step {
    u32x4 w[2], x[MB][2][2];
  };
  // an expert and a step of its I
  struct At {
    int q, st, s, n;
    const uint16_t* w;
  };
  auto enter = [&](At& at, int q) __attribute__((always_inline)) {
    at.q = q;
    const int e = __builtin_amdgcn_readfirstlane(tab->act[q]);
    at.s = __builtin_amdgcn_readfirstlane(tab->start[q]);
    at.n = __builtin_amdgcn_readfirstlane(tab->start[q + 1]) - at.s;
    at.w = p.wd + ((int64_t)e * p.H + row) * I + 8 * lg;
  };
  auto load = [&](const At& at, Step& t) __attribute__((always_inline)) {
    const bool last = at.st == steps - 1;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      t.w[j] = *reinterpret_cast<const u32x4*>(at.w + (last && out[j] ? -8 * lg : 64 * at.st + 32 * j));
#pragma unroll
      for (int a = 0; a < MB; ++a) {
        if (16 * a >= at.n) continue;
        const uint32_t xo = 16 * a + lx < at.n
                                ? (uint32_t)(at.s + 16 * a + lx) * (uint32_t)I * 4u + 16u * (uint32_t)lg + 64u * j
                                : 0x80000000u;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          t.x[a][j][h] = load_chunk(rx, (xo + (uint32_t)(2 * I) * h) | (last ? tail[j] : 0u), 128u * (uint32_t)at.st);
      }
    }
  };
  f32x4 acc[MB];
#pragma unroll
  for (int a = 0; a < MB; ++a) acc[a] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (lo < hi) {
    At now, ahead;
    enter(now, lo / steps);
    now.st = lo - now.q * steps;
    ahead = now;
    auto advance = [&](At& at) __attribute__((always_inline)) {
      if (++at.st < steps) return;
      at.st = 0;
      enter(at, min(at.q + 1, count - 1));
    };
    auto step = [&](Step& t, Step& next) __attribute__((always_inline)) {
      advance(ahead);  // (past the last step, that of another wave or the last again: unused)
      load(ahead, next);
      const bool last = now.st == steps - 1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (last && out[j]) t.w[j] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int a = 0; a < MB; ++a) {
          if (16 * a >= now.n) continue;
          acc[a] = mfma_bf16(t.x[a][j][0], t.w[j], acc[a]);
          acc[a] = mfma_bf16(t.x[a][j][1], t.w[j], acc[a]);
        }
      }
    };
    auto leave = [&](int i) __attribute__((always_inline)) {
      if (now.st == steps - 1 || i == hi - 1) {
#pragma unroll
        for (int a = 0; a < MB; ++a) {
          if (16 * a >= now.n) continue;
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const int m = 16 * a + 4 * lg + f;
            if (m < now.n) sums[wave][tab->tok[now.s + m]][lx] += acc[a][f];
          }
          acc[a] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
      }
      advance(now);
    };
    Step s0, s1;
    load(ahead, s0);
    for (int i = lo; i < hi; i += 2) {
      step(s0, s1);
      leave(i);
      if (i + 1 < hi) {
        step(s1, s0);
        leave(i + 1);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * 16; i += kMoeWaves * 64) {
    const int t = i >> 4, n = n0 + (i & 15);
    if (n >= p.H) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kMoeWaves; ++w) v += sums[w][t][i & 15];
    p.out[(int64_t)t * p.H + n] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  }
}

}  // namespace mmk
