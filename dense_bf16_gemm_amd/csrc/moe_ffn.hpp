// Mixture-of-experts FFN of a few tokens (a decode step):
//   out[t] = sum over j < k of w[t][j] Wd_e (SiLU(Wg_e x[t]) * (Wu_e x[t])),  e = experts[t][j],
// where experts[t] are the k largest logits of token t (ties: the lower index) and
// w[t] their softmax, over these k or over all logits.  A logit of minus infinity
// takes no part: a token with fewer than k others has slots without an expert (-1,
// weight 0).
//
// Bound by reading the weights of the experts in use, 6 H I bytes each, once.
// moe_gate_up leaves w SiLU(g) u, moe_down sums over experts; what tokens an expert has
// is found by moe_route before them, or for few tokens by every workgroup of
// moe_gate_up for itself.  The intermediate is kept as two bf16 numbers, high and
// low part, 16 bits of significand: as one, its rounding would add as much error to
// an output as the output's own.
#pragma once

#include "gemm_q8.hpp"

namespace mmk {

constexpr int kMoeTokens = 64, kMoeExperts = 512, kMoeTopK = 16;
constexpr int kMoeFew = 8;  // tokens whose experts moe_gate_up chooses itself
constexpr int kMoeWaves = 8;

// The tokens of the experts in use, grouped: group g is up to 16 or 32 tokens of expert act[g]
// (experts ascending, their tokens ascending) in rows start[g] .. start[g] + rows[g] - 1,
// row r being token tok[r] with weight wt[r].
template <int N>
struct MoeGroups {
  int count;
  int act[N], start[N], rows[N];
  int tok[N];
  float wt[N];
};
typedef MoeGroups<kMoeTokens * kMoeTopK> MoeTables;

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
  float* part;            // [splits][T][H]: parts of the output
  int T, E, H, I, k;
  int renormalize;
  int splits;
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

// Chooses every token's experts and groups the tokens by expert, with a workgroup of NW
// waves (E <= 64 NW, T <= NW TPW); a wave has TPW tokens, whose steps it takes side by
// side so that their latencies overlap (61 tokens, 4 of 60 experts: 11.8 us one after the
// other).  VPL: logits per lane.  `group`: tokens to a group.  `write`: this
// workgroup writes experts and weights.
template <int VPL, int NW, int TPW, int N>
__device__ __forceinline__ void moe_choose(const MoeParams& p, MoeGroups<N>* tab, int group, bool write) {
  constexpr int kE = 64 * (VPL < NW ? VPL : NW);
  __shared__ uint32_t mask[kE][2];  // the tokens of an expert
  __shared__ int first[kE];
  __shared__ int id[N];
  __shared__ float share[N];
  __shared__ int wave_groups[NW], wave_rows[NW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < p.E; e += NW * 64) mask[e][0] = mask[e][1] = 0u;
  __syncthreads();
  uint32_t key[TPW][VPL], all[TPW][VPL];
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    const int t = wave + NW * i;
#pragma unroll
    for (int r = 0; r < VPL; ++r) {
      const int e = 64 * r + lane;
      all[i][r] = key[i][r] = t < p.T && e < p.E ? order_key(p.logits[(int64_t)t * p.E + e]) : 0u;
    }
  }
  uint32_t mine[TPW], top[TPW];  // lane j: the j-th largest
  int mine_id[TPW];
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    mine[i] = top[i] = 0u;
    mine_id[i] = -1;
  }
  for (int j = 0; j < p.k; ++j) {
    uint32_t m[TPW];
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      m[i] = key[i][0];
#pragma unroll
      for (int r = 1; r < VPL; ++r) m[i] = max(m[i], key[i][r]);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < TPW; ++i) m[i] = max(m[i], (uint32_t)__shfl_xor((int)m[i], d));
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      if (m[i] == 0u) continue;  // (none is left)
      if (j == 0) top[i] = m[i];
      int at = -1;
#pragma unroll
      for (int r = 0; r < VPL; ++r) {
        const uint64_t b = __ballot(key[i][r] == m[i]);
        if (at < 0 && b) {
          const int l = __builtin_ctzll(b);
          at = 64 * r + l;
          if (lane == l) key[i][r] = 0u;
        }
      }
      if (lane == j) {
        mine[i] = m[i];
        mine_id[i] = at;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    const int t = wave + NW * i;
    if (t >= p.T) continue;
    const float peak = key_value(top[i]);
    const float part = mine[i] ? expf(key_value(mine[i]) - peak) : 0.f;
    float sum = part;
    if (!p.renormalize) {
      sum = 0.f;
#pragma unroll
      for (int r = 0; r < VPL; ++r) sum += all[i][r] ? expf(key_value(all[i][r]) - peak) : 0.f;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane < p.k) {
      const int s = t * p.k + lane;
      const float w = mine[i] ? part / sum : 0.f;
      id[s] = mine_id[i];
      share[s] = w;
      if (write) {
        p.experts[s] = mine_id[i];
        p.weights[s] = w;
      }
      if (mine[i]) atomicOr(&mask[mine_id[i]][t >> 5], 1u << (t & 31));
    }
  }
  __syncthreads();
  // places of the groups and of their rows: sums over the experts before
  const int e = threadIdx.x;
  const int rows = e < p.E ? __popc(mask[e][0]) + __popc(mask[e][1]) : 0, groups = (rows + group - 1) / group;
  int r_upto = rows, g_upto = groups;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int r = __shfl_up(r_upto, d), g = __shfl_up(g_upto, d);
    if (lane >= d) {
      r_upto += r;
      g_upto += g;
    }
  }
  if (lane == 63) {
    wave_groups[wave] = g_upto;
    wave_rows[wave] = r_upto;
  }
  __syncthreads();
  int q = g_upto - groups, at = r_upto - rows, used = 0;
  for (int w = 0; w < NW; ++w) {
    if (w < wave) {
      q += wave_groups[w];
      at += wave_rows[w];
    }
    used += wave_groups[w];
  }
  if (rows > 0) first[e] = at;
  for (int g = 0; g < groups; ++g) {
    tab->act[q + g] = e;
    tab->start[q + g] = at + group * g;
    tab->rows[q + g] = min(group, rows - group * g);
  }
  if (threadIdx.x == 0) tab->count = used;
  __syncthreads();
  for (int s = threadIdx.x; s < p.T * p.k; s += NW * 64) {
    const int x = id[s], t = s / p.k;
    if (x < 0) continue;
    const uint32_t lo = mask[x][0], hi = mask[x][1];
    const int before = t < 32 ? __popc(lo & ((1u << t) - 1u)) : __popc(lo) + __popc(hi & ((1u << (t - 32)) - 1u));
    tab->tok[first[x] + before] = t;
    tab->wt[first[x] + before] = share[s];
  }
}

template <int VPL>
__global__ void __launch_bounds__(1024) moe_route(MoeParams p, int group) {
  moe_choose<VPL, 16, kMoeTokens / 16>(p, p.tab, group, true);
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

// A unit of work: 8 columns of I of one group, gate and up rows together as the 16
// columns of an MFMA block.  The eight waves take every eighth step of 64 k, each
// step's loads one step ahead, and meet in LDS, added in wave order.  Of an expert with
// more tokens than a group takes (16 GB) the weights are read again for each group.
// VPL > 0: up to eight tokens, each workgroup chooses their experts itself.
template <int VPL, int GB>
__global__ void __launch_bounds__(kMoeWaves * 64) moe_gate_up(MoeParams p) {
  constexpr bool kOwn = VPL > 0;
  __shared__ float red[kMoeWaves][GB][64][4];
  __shared__ MoeGroups<kOwn ? kMoeFew * kMoeTopK : 1> own;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  if constexpr (kOwn) {
    moe_choose<VPL, kMoeWaves, 1>(p, &own, 16, blockIdx.x == 0);
    __syncthreads();
    if (blockIdx.x == 0) {  // for moe_down
      const int n = p.T * p.k;
      if (threadIdx.x == 0) p.tab->count = own.count;
      for (int i = threadIdx.x; i < n; i += kMoeWaves * 64) {
        if (i < own.count) {
          p.tab->act[i] = own.act[i];
          p.tab->start[i] = own.start[i];
          p.tab->rows[i] = own.rows[i];
        }
        p.tab->tok[i] = own.tok[i];
      }
    }
  }
  auto pick = [&](auto f) __attribute__((always_inline)) {
    if constexpr (kOwn)
      return f(own);
    else
      return f(*p.tab);
  };
  const int cols = p.I >> 3, units = __builtin_amdgcn_readfirstlane(pick([](auto& t) { return t.count; })) * cols;
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
    u32x4 w[2], x[GB][2];
  };
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int q = __builtin_amdgcn_readfirstlane(unit / cols), c0 = 8 * (unit - q * cols);
    const int e = __builtin_amdgcn_readfirstlane(pick([&](auto& t) { return t.act[q]; }));
    const int s = __builtin_amdgcn_readfirstlane(pick([&](auto& t) { return t.start[q]; }));
    const int n = __builtin_amdgcn_readfirstlane(pick([&](auto& t) { return t.rows[q]; }));
    const uint16_t* w = (lx < 8 ? p.wg : p.wu) + ((int64_t)e * p.I + c0 + (lx & 7)) * H + 8 * lg;
    uint32_t xo[GB];
#pragma unroll
    for (int a = 0; a < GB; ++a) {
      const int m = 16 * a + lx;
      xo[a] = 0x80000000u;
      if (m < n) xo[a] = (uint32_t)pick([&](auto& t) { return t.tok[s + m]; }) * (uint32_t)H * 2u + 16u * (uint32_t)lg;
    }
    auto load = [&](int st, Step& t) __attribute__((always_inline)) {
      const bool last = st == steps - 1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        t.w[j] = *reinterpret_cast<const u32x4*>(w + (last && out[j] ? -8 * lg : 64 * st + 32 * j));
#pragma unroll
        for (int a = 0; a < GB; ++a)
          if (a == 0 || 16 * a < n) t.x[a][j] = load_chunk(rx, (xo[a] + 64u * j) | (last ? tail[j] : 0u), 128u * (uint32_t)st);
      }
    };
    f32x4 acc[GB];
#pragma unroll
    for (int a = 0; a < GB; ++a) acc[a] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int st, Step& t, Step& next) __attribute__((always_inline)) {
      load(min(st + kMoeWaves, steps - 1), next);
      const bool last = st == steps - 1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (last && out[j]) t.w[j] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int a = 0; a < GB; ++a)
          if (a == 0 || 16 * a < n) acc[a] = mfma_bf16(t.x[a][j], t.w[j], acc[a]);
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
    for (int a = 0; a < GB; ++a) *reinterpret_cast<f32x4*>(red[wave][a][lane]) = acc[a];
    __syncthreads();
    const int m = threadIdx.x >> 3, c = threadIdx.x & 7;
    if (m < n) {
      const int a = m >> 4, l = 16 * ((m >> 2) & 3) + c, f = m & 3;
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int v = 0; v < kMoeWaves; ++v) {
        g += red[v][a][l][f];
        u += red[v][a][l + 8][f];
      }
      uint16_t hi, lo;
      split_bf16(pick([&](auto& t) { return t.wt[s + m]; }) * swiglu(g, u), &hi, &lo);
      uint16_t* o = p.mid + (int64_t)(s + m) * 2 * p.I + c0 + c;
      o[0] = hi;
      o[p.I] = lo;
    }
  }
}

// 16 columns of H per workgroup x: the steps of 64 values of I, group after group, are
// dealt in equal runs to the waves of its gridDim.y workgroups.  A wave leaves a
// group's sums in LDS, in a row per token of its own; the waves' rows are added in wave
// order.  With more than one workgroup (few columns would leave CUs idle) moe_join
// adds their parts.  (The last workgroup to arrive could; but the fences that order
// its reads after the others' writes took 230 us, since each writes back and
// invalidates an XCD's L2.)
// TB, GB: blocks of 16 tokens in all and in a group.
template <int TB, int GB>
__global__ void __launch_bounds__(kMoeWaves * 64) moe_down(MoeParams p) {
  __shared__ float sums[kMoeWaves][16 * TB][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const MoeTables* tab = p.tab;
  const int I = p.I, steps = (I + 63) >> 6;
  const int count = __builtin_amdgcn_readfirstlane(tab->count);
  const int64_t total = (int64_t)count * steps;
  const int me = blockIdx.y * kMoeWaves + wave, all = gridDim.y * kMoeWaves;
  const int lo = (int)(total * me / all), hi = (int)(total * (me + 1) / all);
  const int n0 = blockIdx.x * 16;
  for (int i = lane; i < 16 * TB * 16; i += 64) (&sums[wave][0][0])[i] = 0.f;
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
    u32x4 w[2], x[GB][2][2];
  };
  // a group and a step of its I
  struct At {
    int q, st, s, n;
    const uint16_t* w;
    uint32_t xo[GB];
  };
  auto enter = [&](At& at, int q) __attribute__((always_inline)) {
    at.q = q;
    const int e = __builtin_amdgcn_readfirstlane(tab->act[q]);
    at.s = __builtin_amdgcn_readfirstlane(tab->start[q]);
    at.n = __builtin_amdgcn_readfirstlane(tab->rows[q]);
    at.w = p.wd + ((int64_t)e * p.H + row) * I + 8 * lg;
#pragma unroll
    for (int a = 0; a < GB; ++a)
      at.xo[a] = 16 * a + lx < at.n ? (uint32_t)(at.s + 16 * a + lx) * (uint32_t)I * 4u + 16u * (uint32_t)lg : 0x80000000u;
  };
  auto load = [&](const At& at, Step& t) __attribute__((always_inline)) {
    const bool last = at.st == steps - 1;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      t.w[j] = *reinterpret_cast<const u32x4*>(at.w + (last && out[j] ? -8 * lg : 64 * at.st + 32 * j));
#pragma unroll
      for (int a = 0; a < GB; ++a) {
        if (a > 0 && 16 * a >= at.n) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          t.x[a][j][h] =
              load_chunk(rx, (at.xo[a] + 64u * j + (uint32_t)(2 * I) * h) | (last ? tail[j] : 0u), 128u * (uint32_t)at.st);
      }
    }
  };
  f32x4 acc[GB];
#pragma unroll
  for (int a = 0; a < GB; ++a) acc[a] = f32x4{0.f, 0.f, 0.f, 0.f};
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
        for (int a = 0; a < GB; ++a) {
          if (a > 0 && 16 * a >= now.n) continue;
          acc[a] = mfma_bf16(t.x[a][j][0], t.w[j], acc[a]);
          acc[a] = mfma_bf16(t.x[a][j][1], t.w[j], acc[a]);
        }
      }
    };
    auto leave = [&](int i) __attribute__((always_inline)) {
      if (now.st == steps - 1 || i == hi - 1) {
#pragma unroll
        for (int a = 0; a < GB; ++a) {
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
  const int splits = gridDim.y;
  auto place = [&](int i, int s) __attribute__((always_inline)) {
    return ((int64_t)s * p.T + (i >> 4)) * p.H + n0 + (i & 15);
  };
  auto put = [&](int i, float v) __attribute__((always_inline)) {
    p.out[place(i, 0)] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  };
  for (int i = threadIdx.x; i < p.T * 16; i += kMoeWaves * 64) {
    if (n0 + (i & 15) >= p.H) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kMoeWaves; ++w) v += sums[w][i >> 4][i & 15];
    if (splits == 1)
      put(i, v);
    else
      p.part[place(i, blockIdx.y)] = v;
  }
}

// The output from the parts of several workgroups, added in order: four columns per thread.
__global__ void __launch_bounds__(256) moe_join(MoeParams p) {
  const int64_t n = (int64_t)p.T * p.H, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(p.part + s * n + i);
#pragma unroll
    for (int f = 0; f < 4; ++f) v[f] += u[f];
  }
  uint16_t* o = p.out + i;
  const uint32_t pk[2] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  __builtin_memcpy(o, pk, 8);
}

}  // namespace mmk
