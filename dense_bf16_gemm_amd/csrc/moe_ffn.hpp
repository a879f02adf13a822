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
// moe_gate_up for itself.  Experts of several tokens go to moe_gate_up_many, moe_down_many and
// moe_combine.  The intermediate is fp32, kept as three bf16 numbers whose sum it is, and the second
// layer multiplies each: as one, its rounding would add as much error to an output as the
// output's own; as two, 16 bits of significand, the outputs of one token of 2 of 8 experts lay 1.4e-4 from
// those of fp32 (the roundings that it turns), as three 1.1e-5.
#pragma once

#include "gemm_q8.hpp"
#include "wave_ops.hpp"

namespace mmk {

constexpr int kMoeTokens = 64, kMoeExperts = 512, kMoeTopK = 16;
constexpr int kMoeFew = 8;  // tokens whose experts moe_gate_up chooses itself
constexpr int kMoePacked = 5;  // tokens of a group whose three parts are one block of 16 rows
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
  int row[N];  // of choice t k + j, -1 for none
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
  uint16_t* mid;          // [T k][3][I]: the parts of the intermediate
  float* part;            // parts of the output: [splits][T][H], or [slices][T k][H] of each row's
  int T, E, H, I, k;
  int renormalize;
  int splits, slices;
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
    for (int i = 0; i < TPW; ++i) m[i] = wave_max(m[i]);
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
    sum = wave_sum(sum);
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
    if (x < 0) {
      tab->row[s] = -1;
      continue;
    }
    const uint32_t lo = mask[x][0], hi = mask[x][1];
    const int before = t < 32 ? __popc(lo & ((1u << t) - 1u)) : __popc(lo) + __popc(hi & ((1u << (t - 32)) - 1u));
    tab->tok[first[x] + before] = t;
    tab->wt[first[x] + before] = share[s];
    tab->row[s] = first[x] + before;
  }
}

// (latency, k dependent steps: 16 tokens, 8 of 128 experts 8.3 us, 64, 8 of 128 14.3)
template <int VPL>
__global__ void __launch_bounds__(1024) moe_route(MoeParams p, int group) {
  moe_choose<VPL, 16, kMoeTokens / 16>(p, p.tab, group, true);
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A float as the sum of three bf16: 8 bits of the significand each, cut, so that the sum is exact
// (but for what lies below 2^-126, where bf16 has fewer bits).  put(i, part i); what is not finite stays in part 0.
template <typename F>
__device__ __forceinline__ void split_bf16(float v, F put) {
  uint32_t b = __builtin_bit_cast(uint32_t, v);
  if ((b & 0x7f800000u) == 0x7f800000u) {
    put(0, __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)));
    put(1, (uint16_t)0);
    put(2, (uint16_t)0);
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    put(i, (uint16_t)(b >> 16));
    v -= __builtin_bit_cast(float, b & 0xffff0000u);
    b = __builtin_bit_cast(uint32_t, v);
  }
}

// The intermediate `v` of row `row` and column `col`, in its parts (below 2^30 values in all).
__device__ __forceinline__ void moe_leave(const MoeParams& p, int row, int col, float v) {
  const uint32_t at = (uint32_t)row * 3u * (uint32_t)p.I + (uint32_t)col;
  split_bf16(v, [&](int i, uint16_t part) __attribute__((always_inline)) { p.mid[at + (uint32_t)(i * p.I)] = part; });
}

// SiLU(g) u, as the fused FFN has it
__device__ __forceinline__ float swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// A step's 16 rows of 128 bytes are loaded with eight lanes to a row, rows lane / 8 and
// 8 + lane / 8, chunk lane % 8, and brought to the places of the MFMA's two fragments (row
// lane % 16, chunks lane / 16 and 4 + lane / 16) through 2 KiB of LDS of the wave's own.
// Loaded in those places at once, 16 neighbouring lanes touch 16 lines, which holds a CU to
// some 16 bytes a clock and the reading of weights to 5.2 TB/s.
// KEEP: the places stay in registers; else they are taken anew each time, which leaves room for more
// waves (8 tokens, 4 of 32 experts of 1024 x 512 25.1 us kept, 21.7 anew; but 61, 4 of 60 of
// 2056 x 1416, whose waves a CU holds either way, 245, 250).
template <bool KEEP = false>
__device__ __forceinline__ void to_fragments(u32x4 (&v)[2], f32x4* slot, int lane) {
  if constexpr (!KEEP) asm volatile("" : "+v"(lane));
  // (chunks of rows 2 i and 2 i + 1 keyed by i: no bank twice)
  const int at = lane ^ (lane >> 4);
  slot[at] = __builtin_bit_cast(f32x4, v[0]);
  slot[64 + (at ^ 4)] = __builtin_bit_cast(f32x4, v[1]);
  __builtin_amdgcn_wave_barrier();
  const int row = lane & 15, from = 8 * row + ((lane >> 4) ^ (row >> 1));
  v[0] = __builtin_bit_cast(u32x4, slot[from]);
  v[1] = __builtin_bit_cast(u32x4, slot[from ^ 4]);
}

// A unit of work: 8 columns of I of one group, gate and up rows together as the 16
// columns of an MFMA block.  The eight waves take every eighth step of 64 k, each
// step's loads one step ahead, and meet in LDS, added in wave order.  Of an expert with
// more tokens than a group of 16 takes the weights are read again for each group.
// VPL > 0: up to eight tokens, each workgroup chooses their experts itself.
// Bound by the weights: one token, 2 of 8 experts of 4096 x 14336, both layers 122 us (5.8 TB/s); 16
// tokens, 8 of 128 of 4096 x 1536 540 (5.8).  With w and x loaded in the MFMA's order some 10 and 50 us more.
template <int VPL>
__global__ void __launch_bounds__(kMoeWaves * 64) moe_gate_up(MoeParams p) {
  constexpr bool kOwn = VPL > 0;
  __shared__ float red[kMoeWaves][64][4];
  __shared__ f32x4 turn[kMoeWaves][128];
  __shared__ MoeGroups<kOwn ? kMoeFew * kMoeTopK : 1> own;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane >> 3, lk = lane & 7;  // of what is loaded (to_fragments)
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
        p.tab->row[i] = own.row[i];
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
  const bool out = 64 * (steps - 1) + 8 * lk >= H;
  const uint32_t tail = out ? 0x80000000u : 0u;
  struct Step {
    u32x4 w[2], x[2];
  };
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int q = __builtin_amdgcn_readfirstlane(unit / cols), c0 = 8 * (unit - q * cols);
    const int e = __builtin_amdgcn_readfirstlane(pick([&](auto& t) { return t.act[q]; }));
    const int s = __builtin_amdgcn_readfirstlane(pick([&](auto& t) { return t.start[q]; }));
    const int n = __builtin_amdgcn_readfirstlane(pick([&](auto& t) { return t.rows[q]; }));
    const int64_t wrow = ((int64_t)e * p.I + c0 + lr) * H + 8 * lk;
    const uint16_t *wg = p.wg + wrow, *wu = p.wu + wrow;
    uint32_t xo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int m = 8 * j + lr;
      xo[j] = 0x80000000u;
      if (m < n) xo[j] = (uint32_t)pick([&](auto& t) { return t.tok[s + m]; }) * (uint32_t)H * 2u + 16u * (uint32_t)lk;
    }
    auto load = [&](int st, Step& t) __attribute__((always_inline)) {
      const bool last = st == steps - 1;
      const int at = last && out ? -8 * lk : 64 * st;
      t.w[0] = *reinterpret_cast<const u32x4*>(wg + at);
      t.w[1] = *reinterpret_cast<const u32x4*>(wu + at);
#pragma unroll
      for (int j = 0; j < 2; ++j) t.x[j] = load_chunk(rx, xo[j] | (last ? tail : 0u), 128u * (uint32_t)st);
    };
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    auto step = [&](int st, Step& t, Step& next) __attribute__((always_inline)) {
      load(min(st + kMoeWaves, steps - 1), next);
      if (st == steps - 1 && out) t.w[0] = t.w[1] = u32x4{0u, 0u, 0u, 0u};
      to_fragments(t.x, turn[wave], lane);
      to_fragments(t.w, turn[wave], lane);
#pragma unroll
      for (int j = 0; j < 2; ++j) acc = mfma_bf16(t.x[j], t.w[j], acc);
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
    *reinterpret_cast<f32x4*>(red[wave][lane]) = acc;
    __syncthreads();
    const int m = threadIdx.x >> 3, c = threadIdx.x & 7;
    if (m < n) {
      const int l = 16 * (m >> 2) + c, f = m & 3;
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int v = 0; v < kMoeWaves; ++v) {
        g += red[v][l][f];
        u += red[v][l + 8][f];
      }
      moe_leave(p, s + m, c0 + c, pick([&](auto& t) { return t.wt[s + m]; }) * swiglu(g, u));
    }
  }
}

// f(i, e, row) for the chunks i of 8 values of I that a lane has of every choice of token t.
template <typename F>
__device__ __forceinline__ void moe_chunks(const MoeParams& p, int t, int lane, F f) {
  for (int j = 0; j < p.k; ++j) {
    const int e = p.experts[t * p.k + j];
    if (e < 0) break;
    const int64_t row = (int64_t)p.tab->row[t * p.k + j] * 3 * p.I;
#pragma unroll 1
    for (int i = 8 * lane; i < p.I; i += 512) f(i, e, p.mid + row + i);
  }
}

// Outputs (t, n) of a wave's lanes that came out NaN, from the definition: of the three parts of a value,
// 8 bits or less leave some 0, and 0 times an infinity of W_down is NaN where the value times it is
// infinite.  Token after token by the whole wave, first whether a value is NaN (then the outputs are), else
// one output after another.
__device__ __forceinline__ void moe_again(const MoeParams& p, int t, int n, float& v, int lane) {
  uint64_t left = __ballot(v != v);
  while (left) {
    const int lt = __builtin_amdgcn_readlane(t, __builtin_ctzll(left));
    uint64_t mine = left & __ballot(t == lt);
    left &= ~mine;
    bool nan = false;
    moe_chunks(p, lt, lane, [&](int, int, const uint16_t* x) {
      const u32x4 u = *reinterpret_cast<const u32x4*>(x);
#pragma unroll
      for (int f = 0; f < 8; ++f) nan |= (u[f >> 1] >> (16 * (f & 1)) & 0x7fffu) > 0x7f80u;
    });
    if (__any(nan)) continue;
    for (; mine; mine &= mine - 1) {
      const int l = __builtin_ctzll(mine), ln = __builtin_amdgcn_readlane(n, l);
      float sum = 0.f;
      moe_chunks(p, lt, lane, [&](int i, int e, const uint16_t* x) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p.wd + ((int64_t)e * p.H + ln) * p.I + i);
        u32x4 part[3];
#pragma unroll
        for (int h = 0; h < 3; ++h) part[h] = *reinterpret_cast<const u32x4*>(x + (int64_t)h * p.I);
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          auto at = [&](const u32x4& u) { return bf16_float((uint16_t)(u[f >> 1] >> (16 * (f & 1)))); };
          sum = __builtin_fmaf(at(part[0]) + at(part[1]) + at(part[2]), at(w), sum);
        }
      });
      sum = wave_sum(sum);
      if (lane == l) v = sum;
    }
  }
}

// The same of four columns from n on.
__device__ __forceinline__ void moe_again(const MoeParams& p, int t, int n, f32x4& v, int lane) {
  if (__ballot(v[0] + v[1] + v[2] + v[3] != v[0] + v[1] + v[2] + v[3]) == 0) return;
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    float u = v[f];
    moe_again(p, t, n + f, u, lane);
    v[f] = u;
  }
}

// 16 columns of H per workgroup x: the steps of 64 values of I, group after group, are
// dealt in equal runs to the waves of its gridDim.y workgroups.  A wave leaves a
// group's sums in LDS, in a row per token of its own; the waves' rows are added in wave
// order.  With more than one workgroup (few columns would leave CUs idle) moe_join
// adds their parts.  (The last workgroup to arrive could; but the fences that order
// its reads after the others' writes took 230 us, since each writes back and
// invalidates an XCD's L2.)  Bound by the weights, as above.  Waves that take
// every eighth step, as there, read no faster and add up more often (20, 4 of 60 experts of 1024 x 512
// 18 us, 14 in runs), and twice the waves were no faster either.
// The parts of up to kMoePacked tokens are rows of the same block (row 5 h + m: part h of token m),
// of more they are three blocks (us a call, three always / so: one token, 2 of 8 experts of 4096 x 14336
// 134.5 / 124.1, 8 tokens 502 / 457, 16, 8 of 128 of 4096 x 1536 587 / 541).
// TB: blocks of 16 tokens.
template <int TB>
__global__ void __launch_bounds__(kMoeWaves * 64) moe_down(MoeParams p) {
  __shared__ float sums[kMoeWaves][16 * TB][16];
  __shared__ f32x4 turn[kMoeWaves][128];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int lr = lane >> 3, lk = lane & 7;  // of what is loaded (to_fragments)
  const MoeTables* tab = p.tab;
  const int I = p.I, steps = (I + 63) >> 6;
  const int count = __builtin_amdgcn_readfirstlane(tab->count);
  const int64_t total = (int64_t)count * steps;
  const int me = blockIdx.y * kMoeWaves + wave, all = gridDim.y * kMoeWaves;
  const int lo = (int)(total * me / all), hi = (int)(total * (me + 1) / all);
  const int n0 = blockIdx.x * 16;
  for (int i = lane; i < 16 * TB * 16; i += 64) (&sums[wave][0][0])[i] = 0.f;
  const __amdgpu_buffer_rsrc_t rx =
      __builtin_amdgcn_make_buffer_rsrc(p.mid, (short)0, p.T * p.k * I * 6, 0x00020000);
  const bool out = 64 * (steps - 1) + 8 * lk >= I;
  const uint32_t tail = out ? 0x80000000u : 0u;
  struct Step {
    u32x4 w[2], x[3][2];  // (x: the three parts, or all in the first)
  };
  // a group and a step of its I
  struct At {
    int q, st, s, n;
    const uint16_t* w[2];
    uint32_t xo[2];
  };
  auto enter = [&](At& at, int q) __attribute__((always_inline)) {
    at.q = q;
    const int e = __builtin_amdgcn_readfirstlane(tab->act[q]);
    at.s = __builtin_amdgcn_readfirstlane(tab->start[q]);
    at.n = __builtin_amdgcn_readfirstlane(tab->rows[q]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int m = 8 * j + lr;
      at.w[j] = p.wd + ((int64_t)e * p.H + min(n0 + m, p.H - 1)) * I + 8 * lk;
      const int h = at.n > kMoePacked ? 0 : m / kMoePacked, r = m - h * kMoePacked;
      at.xo[j] = r < at.n && h < 3 ? (uint32_t)(3 * (at.s + r) + h) * (uint32_t)I * 2u + 16u * (uint32_t)lk : 0x80000000u;
    }
  };
  auto load = [&](const At& at, Step& t) __attribute__((always_inline)) {
    const bool last = at.st == steps - 1;
    auto load_x = [&](int h, int j) __attribute__((always_inline)) {
      t.x[h][j] = load_chunk(rx, (at.xo[j] + (uint32_t)(2 * I) * h) | (last ? tail : 0u), 128u * (uint32_t)at.st);
    };
    // (first: a wait that has to do for both leaves the others in flight)
    if (at.n > kMoePacked) {
#pragma unroll
      for (int h = 1; h < 3; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) load_x(h, j);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      t.w[j] = *reinterpret_cast<const u32x4*>(at.w[j] + (last && out ? -8 * lk : 64 * at.st));
      load_x(0, j);
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
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
      if (now.st == steps - 1 && out) t.w[0] = t.w[1] = u32x4{0u, 0u, 0u, 0u};
      to_fragments(t.w, turn[wave], lane);
      auto multiply = [&](int h) __attribute__((always_inline)) {
        to_fragments(t.x[h], turn[wave], lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) acc = mfma_bf16(t.x[h][j], t.w[j], acc);
      };
      multiply(0);
      if (now.n > kMoePacked) {
        multiply(1);
        multiply(2);
      }
    };
    auto leave = [&](int i) __attribute__((always_inline)) {
      if (now.st == steps - 1 || i == hi - 1) {
        if (now.n > kMoePacked) {
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const int m = 4 * lg + f;
            if (m < now.n) sums[wave][tab->tok[now.s + m]][lx] += acc[f];
          }
        } else {  // the parts' rows meet in the wave's own LDS
          float* rows = reinterpret_cast<float*>(turn[wave]);
#pragma unroll
          for (int f = 0; f < 4; ++f) rows[16 * (4 * lg + f) + lx] = acc[f];
          __builtin_amdgcn_wave_barrier();
          for (int i = lane; i < 16 * now.n; i += 64) {
            const float* r = rows + i;
            sums[wave][tab->tok[now.s + (i >> 4)]][lx] += r[0] + r[16 * kMoePacked] + r[32 * kMoePacked];
          }
          __builtin_amdgcn_wave_barrier();
        }
        acc = f32x4{0.f, 0.f, 0.f, 0.f};
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
  for (int first = wave * 64; first < p.T * 16; first += kMoeWaves * 64) {
    const int i = first + lane, t = i >> 4, n = n0 + (i & 15);
    const bool there = t < p.T && n < p.H;
    float v = 0.f;
    if (there) {
#pragma unroll
      for (int w = 0; w < kMoeWaves; ++w) v += sums[w][t][i & 15];
    }
    if (splits == 1) {
      moe_again(p, t, n, v, lane);
      if (there) p.out[(int64_t)t * p.H + n] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    } else if (there) {
      p.part[((int64_t)blockIdx.y * p.T + t) * p.H + n] = v;
    }
  }
}

// The output from the parts of several workgroups, added in order: four columns per thread.
__global__ void __launch_bounds__(256) moe_join(MoeParams p) {
  const int64_t n = (int64_t)p.T * p.H, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int splits = i < n ? p.splits : 0;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(p.part + s * n + i);
#pragma unroll
    for (int f = 0; f < 4; ++f) v[f] += u[f];
  }
  const int t = (int)(i / p.H), c = (int)(i - (int64_t)t * p.H);  // (H is a multiple of 8)
  moe_again(p, t, c, v, threadIdx.x & 63);
  if (i >= n) return;
  uint16_t* o = p.out + i;
  const uint32_t pk[2] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  __builtin_memcpy(o, pk, 8);
}

// ---- experts of several tokens -------------------------------------------------
//
// Read from L2 for every unit, the tokens' rows are as many bytes as the weights at 16
// tokens to an expert (two times as many in the second layer), which halves the rate (64
// tokens, 2 of 8 experts of 4096 x 4096: 2.8 TB/s of weights).  So here a workgroup of 16
// waves takes a run of neighbouring units, and each wave holds its part of a group's
// rows in registers until the group changes: the steps 16 i + w of 64 values, i < SPW.
// Each step's weights are loaded one step ahead, across units; the waves' sums of a unit
// meet in LDS (two sets in turn: one barrier per unit), and are added in wave order by
// another wave for each unit.  61 tokens, 4 of 60 experts of 2056 x 1416: 251 us
// in all (4.1 TB/s of rows that start inside a line), 220 of 2048 x 1408 (4.7); 64, 6 of 32 of 4096 x 2048 331 (4.9), 398 with x
// out of L2.  All SPW steps are run; those past the row's end multiply zeros (31 of 64 at 2056).

constexpr int kMoeManyWaves = 16;

// A lane's chunk of step st of 64 values from a row at byte `row` of a buffer of rows of n values;
// zeros past them, and past the last step (its base, a scalar, has to stay inside the buffer).
__device__ __forceinline__ u32x4 step_chunk(__amdgpu_buffer_rsrc_t buf, uint32_t row, int st, int chunk, int n, int steps) {
  const uint32_t off = 64 * st + 8 * chunk < n ? row + 16u * (uint32_t)chunk : 0x80000000u;
  return load_chunk(buf, off, 128u * (uint32_t)min(st, steps - 1));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t moe_rows(const uint16_t* base, int rows, int n) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), (short)0, rows * n * 2, 0x00020000);
}

// The first layer: a unit is 16 columns of I of one group, gate and up.
template <int GB, int SPW>
__global__ void __launch_bounds__(kMoeManyWaves * 64) moe_gate_up_many(MoeParams p) {
  static_assert(SPW % 2 == 0 && GB * SPW <= 8, "x in 64 registers, two steps in turn");
  __shared__ f32x4 red[2][kMoeManyWaves][2][GB][64];
  __shared__ f32x4 turn[kMoeManyWaves][128];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane >> 3, lk = lane & 7;  // of what is loaded (to_fragments)
  const MoeTables* tab = p.tab;
  const int H = p.H, steps = (H + 63) >> 6, cols = (p.I + 15) >> 4;
  const int64_t units = (int64_t)__builtin_amdgcn_readfirstlane(tab->count) * cols;
  const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
  if (u0 >= u1) return;
  struct Step {
    u32x4 w[2][2];
  };
  // where the loads are: group, column block, and the two weights' rows there
  int lq = u0 / cols, lc = u0 - lq * cols;
  __amdgpu_buffer_rsrc_t rg, ru;
  auto enter = [&]() __attribute__((always_inline)) {
    const int64_t first = (int64_t)__builtin_amdgcn_readfirstlane(tab->act[lq]) * p.I + 16 * lc;
    const int rows = min(16, p.I - 16 * lc);
    rg = moe_rows(p.wg + first * H, rows, H);
    ru = moe_rows(p.wu + first * H, rows, H);
  };
  uint32_t row = (uint32_t)lr * (uint32_t)H * 2u;
  auto load = [&](int i, Step& t) __attribute__((always_inline)) {
    // opaque: the steps' offsets are not all kept in registers; the row neither, where x leaves none
    // (6 spilled)
    int l = lane;
    if constexpr (GB * SPW == 8) {
      asm volatile("" : "+v"(l));
      row = (uint32_t)(l >> 3) * (uint32_t)H * 2u;
    } else {
      asm volatile("" : "+v"(row));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t at = row + (uint32_t)(16 * j) * (uint32_t)H;
      t.w[0][j] = step_chunk(rg, at, wave + kMoeManyWaves * i, l & 7, H, steps);
      t.w[1][j] = step_chunk(ru, at, wave + kMoeManyWaves * i, l & 7, H, steps);
    }
  };
  Step t[2];
  enter();
  load(0, t[0]);
  u32x4 x[GB][SPW][2];
  int q = -1, c = lc, s = 0, n = 0;
  for (int unit = u0; unit < u1; ++unit) {
    if (q < 0 || c == cols) {  // the next group's rows
      q = q < 0 ? lq : q + 1;
      c = unit == u0 ? c : 0;
      s = __builtin_amdgcn_readfirstlane(tab->start[q]);
      n = __builtin_amdgcn_readfirstlane(tab->rows[q]);
      const __amdgpu_buffer_rsrc_t rx = moe_rows(p.x, p.T, H);
#pragma unroll
      for (int a = 0; a < GB; ++a) {
        uint32_t xo[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int m = 16 * a + 8 * j + lr;
          xo[j] = 0x80000000u;
          if (m < n) xo[j] = (uint32_t)tab->tok[s + m] * (uint32_t)H * 2u;
        }
#pragma unroll
        for (int i = 0; i < SPW; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) x[a][i][j] = step_chunk(rx, xo[j], wave + kMoeManyWaves * i, lk, H, steps);
      }
#pragma unroll
      for (int a = 0; a < GB; ++a)
#pragma unroll
        for (int i = 0; i < SPW; ++i) to_fragments<GB == 1>(x[a][i], turn[wave], lane);
    }
    f32x4 acc[2][GB];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int a = 0; a < GB; ++a) acc[h][a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < SPW; ++i) {
      if (i + 1 < SPW) {
        load(i + 1, t[(i + 1) & 1]);
      } else {
        // (past the last unit, that one again, unused)
        if (unit + 1 < u1 && ++lc == cols) {
          lc = 0;
          ++lq;
        }
        enter();
        load(0, t[0]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4(&w)[2] = t[i & 1].w[h];
        to_fragments<GB == 1>(w, turn[wave], lane);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int a = 0; a < GB; ++a) acc[h][a] = mfma_bf16(x[a][i][j], w[j], acc[h][a]);
      }
    }
    auto set = red[(unit - u0) & 1];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int a = 0; a < GB; ++a) set[wave][h][a][lane] = acc[h][a];
    __syncthreads();
    const int c0 = 16 * c;
    ++c;
    const int a = (wave - (unit - u0) * GB) & (kMoeManyWaves - 1);
    if (a >= GB || 16 * a >= n) continue;
    f32x4 v[2] = {set[0][0][a][lane], set[0][1][a][lane]};
#pragma unroll 3
    for (int w = 1; w < kMoeManyWaves; ++w)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 u = set[w][h][a][lane];
#pragma unroll
        for (int f = 0; f < 4; ++f) v[h][f] += u[f];
      }
    // (opaque, as in load: 2 spilled)
    int l = lane;
    asm volatile("" : "+v"(l));
    if (c0 + (l & 15) >= p.I) continue;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int m = 16 * a + 4 * (l >> 4) + f;
      if (m >= n) continue;
      moe_leave(p, s + m, c0 + (l & 15), tab->wt[s + m] * swiglu(v[0][f], v[1][f]));
    }
  }
}

// The second layer: a unit is 16 columns of H of one group and slice of I (16 SPW steps), and
// leaves its sums for each of the group's rows; moe_combine adds a token's.
template <int GB, int SPW>
__global__ void __launch_bounds__(kMoeManyWaves * 64) moe_down_many(MoeParams p) {
  static_assert(GB * SPW <= 2, "x in 48 registers");
  __shared__ f32x4 red[2][kMoeManyWaves][GB][64];
  __shared__ f32x4 turn[kMoeManyWaves][128];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int lr = lane >> 3, lk = lane & 7;  // of what is loaded (to_fragments)
  const MoeTables* tab = p.tab;
  const int I = p.I, steps = (I + 63) >> 6, cols = (p.H + 15) >> 4;
  const int64_t units = (int64_t)__builtin_amdgcn_readfirstlane(tab->count) * p.slices * cols;
  const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
  if (u0 >= u1) return;
  struct Step {
    u32x4 w[2];
  };
  int lq = u0 / cols, lc = u0 - lq * cols;  // (lq, q: group and slice together)
  __amdgpu_buffer_rsrc_t rw;
  int lfirst = 0;
  auto enter = [&]() __attribute__((always_inline)) {
    const int g = lq / p.slices;
    lfirst = (lq - g * p.slices) * (kMoeManyWaves * SPW) + wave;
    const int64_t first = (int64_t)__builtin_amdgcn_readfirstlane(tab->act[g]) * p.H + 16 * lc;
    rw = moe_rows(p.wd + first * I, min(16, p.H - 16 * lc), I);
  };
  uint32_t row = (uint32_t)lr * (uint32_t)I * 2u;
  auto load = [&](int i, Step& t) __attribute__((always_inline)) {
    asm volatile("" : "+v"(row));
#pragma unroll
    for (int j = 0; j < 2; ++j)
      t.w[j] = step_chunk(rw, row + (uint32_t)(16 * j) * (uint32_t)I, lfirst + kMoeManyWaves * i, lk, I, steps);
  };
  Step t[2];
  enter();
  load(0, t[0]);
  u32x4 x[GB][SPW][3][2];
  int q = -1, c = lc, s = 0, n = 0, slice = 0;
  // `now` and `then`: the two steps in turn, now the unit's first
  auto one = [&](int unit, Step& now, Step& then) __attribute__((always_inline)) {
    if (q < 0 || c == cols) {
      q = q < 0 ? lq : q + 1;
      c = unit == u0 ? c : 0;
      const int g = q / p.slices;
      slice = q - g * p.slices;
      s = __builtin_amdgcn_readfirstlane(tab->start[g]);
      n = __builtin_amdgcn_readfirstlane(tab->rows[g]);
      const __amdgpu_buffer_rsrc_t rx = moe_rows(p.mid + (int64_t)s * 3 * I, 3 * n, I);
      const int first = slice * (kMoeManyWaves * SPW) + wave;
#pragma unroll
      for (int a = 0; a < GB; ++a) {
        uint32_t xo[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int m = 16 * a + 8 * j + lr;
          xo[j] = m < n ? (uint32_t)m * (uint32_t)I * 6u : 0x80000000u;
        }
#pragma unroll
        for (int i = 0; i < SPW; ++i)
#pragma unroll
          for (int h = 0; h < 3; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              x[a][i][h][j] = step_chunk(rx, xo[j] + (uint32_t)(2 * I) * h, first + kMoeManyWaves * i, lk, I, steps);
      }
#pragma unroll
      for (int a = 0; a < GB; ++a)
#pragma unroll
        for (int i = 0; i < SPW; ++i)
#pragma unroll
          for (int h = 0; h < 3; ++h) to_fragments<GB == 1>(x[a][i][h], turn[wave], lane);
    }
    f32x4 acc[GB];
#pragma unroll
    for (int a = 0; a < GB; ++a) acc[a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < SPW; ++i) {
      Step &used = i & 1 ? then : now, &next = i & 1 ? now : then;
      if (i + 1 < SPW) {
        load(i + 1, next);
      } else {
        if (unit + 1 < u1 && ++lc == cols) {
          lc = 0;
          ++lq;
        }
        enter();
        load(0, next);
      }
      u32x4(&w)[2] = used.w;
      to_fragments<GB == 1>(w, turn[wave], lane);
#pragma unroll
      for (int a = 0; a < GB; ++a)
#pragma unroll
        for (int h = 0; h < 3; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[a] = mfma_bf16(x[a][i][h][j], w[j], acc[a]);
    }
    auto set = red[(unit - u0) & 1];
#pragma unroll
    for (int a = 0; a < GB; ++a) set[wave][a][lane] = acc[a];
    __syncthreads();
    const int n0 = 16 * c;
    ++c;
    const int a = (wave - (unit - u0) * GB) & (kMoeManyWaves - 1);
    if (a >= GB || 16 * a >= n) return;
    f32x4 v = set[0][a][lane];
#pragma unroll 5
    for (int w = 1; w < kMoeManyWaves; ++w) {
      const f32x4 u = set[w][a][lane];
#pragma unroll
      for (int f = 0; f < 4; ++f) v[f] += u[f];
    }
    if (n0 + lx >= p.H) return;
    float* o = p.part + ((int64_t)slice * p.T * p.k + s) * p.H + n0 + lx;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int m = 16 * a + 4 * lg + f;
      if (m < n) o[(int64_t)m * p.H] = v[f];
    }
  };
  for (int unit = u0; unit < u1; ++unit) {
    one(unit, t[0], t[1]);
    // (an odd number of steps leaves the next unit's first in the other place)
    if constexpr (SPW & 1) {
      if (++unit < u1) one(unit, t[1], t[0]);
    }
  }
}

// out[t] from the rows of its choices, in their order and in that of the slices: four columns per
// thread.
__global__ void __launch_bounds__(256) moe_combine(MoeParams p) {
  const int t = blockIdx.y, n = (blockIdx.x * 256 + threadIdx.x) * 4;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < (n < p.H ? p.k : 0); ++j) {
    const int row = p.tab->row[t * p.k + j];
    if (row < 0) break;
    for (int s = 0; s < p.slices; ++s) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(p.part + ((int64_t)s * p.T * p.k + row) * p.H + n);
#pragma unroll
      for (int f = 0; f < 4; ++f) v[f] += u[f];
    }
  }
  moe_again(p, t, n, v, threadIdx.x & 63);
  if (n >= p.H) return;
  const uint32_t pk[2] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  __builtin_memcpy(p.out + (int64_t)t * p.H + n, pk, 8);
}

}  // namespace mmk
