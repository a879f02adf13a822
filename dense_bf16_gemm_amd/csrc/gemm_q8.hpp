// Products of e4m3 operands with row scales:
//   out[m][n] = epi(xs[m] ws[n] sum_k x[m][k] W[n][k] + bias[n]),
// x [M][K] and W [N][K] e4m3 (K contiguous), fp32 scales, bf16 output.  The
// scales are applied to the sum, then the epilogue, then one rounding.
//
// The sums are held in fp32 from one matrix instruction to the next.  Inside one,
// products (exact) are added as the hardware does for e4m3, aligned to the largest
// with fewer bits than fp32 keeps: against 64 bits one instruction's sum was off by
// 2^-14.8 of the sum of its products' magnitudes at the worst, and the sums of normally
// distributed operands by 1.5e-5 of their own size (K = 128 to 8192), a hundredth of the
// output's bf16 rounding.  The 16 x 16 x 32, 16 x 16 x 128 and 32 x 32 x 64 instructions do not
// differ in this.
//
// v_mfma_f32_16x16x128_f8f6f4 does 65536 products and sums in 32 cycles of a
// SIMD, twice the bf16 rate.  Its lane holds 32 consecutive bytes of k in hardware
// order; any order serves as long as both operands use the same, so fragments
// are two 16-byte chunks wherever they are best read.
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
  // K of every tile in `chunks` pieces of `chunk_steps` super-steps (the last
  // may be shorter); with more than one, each leaves its sums in `part`
  int chunks, chunk_steps;
  float* part;
};

// 16 bytes at byte `off` (the lane's) + `base` (the wave's) of a buffer, zeros
// past its end
__device__ __forceinline__ u32x4 load_chunk(__amdgpu_buffer_rsrc_t buf, uint32_t off, uint32_t base) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, off, base, 0));
}

__device__ __forceinline__ i32x8 join_chunks(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// The rows row0 .. row0 + n - 1 (of `rows`) of an operand [rows][K] as a
// buffer: what lies past the operand's last row reads as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_buffer(const uint8_t* base, int64_t row0, int rows, int n,
                                                              uint32_t K) {
  const uint32_t have = (uint32_t)min((int64_t)n, rows - row0);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base + row0 * (int64_t)K), (short)0, (int)(have * K),
                                           0x00020000);
}

// (unit block scales: the instruction without scale operands)
__device__ __forceinline__ f32x4 mfma_q8(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Few rows (a decode step): bound by reading W once.  XR rows of x (4: the
// first four of a block of 16) by NB blocks of 16 columns per workgroup; its
// waves take every WV-th 128-k step, each step's loads issued one step ahead,
// and meet in LDS, added in wave order.  A wave copies its step's tile of x,
// XR rows of 128 bytes, into LDS for itself (chunk c of row r at position c ^
// (r & 7)); the rows of W go straight to registers as fragments, chunks g and g
// + 4 of lane (g, n).  The copies go out before the loads, which arrive in
// order, so once a step's weights are there its activations are.  1 x 8192
// x 8192 takes 13.8 us (4.9 TB/s), 16 x 28672 x 8192 50.5 (4.7).
template <int XR, int NB, int WV>
__global__ void __launch_bounds__(WV * 64) gemm_q8_rows(Q8Params p) {
  constexpr int MB = XR < 16 ? 1 : XR / 16, AB = MB * NB;
  constexpr int XC = XR < 8 ? 1 : XR / 8;   // copies per step: eight rows of 128 bytes each
  constexpr int kX = 2 * XC * 1024;         // LDS bytes per wave
  constexpr int kRed = WV * AB * 1024;
  __shared__ __attribute__((aligned(1024))) char smem[WV * kX > kRed ? WV * kX : kRed];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int ksteps = (p.K + 127) >> 7;
  const int m0 = blockIdx.y * XR;
  const int n0 = blockIdx.x * (16 * NB);
  const uint32_t K = (uint32_t)p.K;
  char* xs = smem + wave * kX;

  const __amdgpu_buffer_rsrc_t rx = tile_buffer(p.x, m0, p.M, XR, K);
  const int crow = lane >> 3;
  const uint32_t chunk = 16u * (uint32_t)((lane & 7) ^ crow);
  const uint32_t tail_x = 128u * (uint32_t)(ksteps - 1) + chunk < K ? 0u : 0x80000000u;
  auto copy = [&](int st, int slot) __attribute__((always_inline)) {
    const uint32_t off = st == ksteps - 1 ? tail_x : 0u;
#pragma unroll
    for (int i = 0; i < XC; ++i)
      copy_to_lds(rx, xs + slot * (XC * 1024) + i * 1024, ((uint32_t)(8 * i + crow) * K + chunk) | off,
                  128u * (uint32_t)st);
  };
  // W: 16 rows of a block as a buffer each (rows past N repeat the last: their
  // sums are dropped); the last step's chunks past K read as zeros
  const uint32_t tail_w[2] = {128u * (uint32_t)(ksteps - 1) + 16u * (uint32_t)lg < K ? 0u : 0x80000000u,
                              128u * (uint32_t)(ksteps - 1) + 64u + 16u * (uint32_t)lg < K ? 0u : 0x80000000u};
  const __amdgpu_buffer_rsrc_t rw = tile_buffer(p.W, n0, p.N, 16 * NB, K);
  uint32_t vw[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    vw[b] = (uint32_t)(min(n0 + 16 * b + lx, p.N - 1) - n0) * K + 16u * (uint32_t)lg;
  struct Step {
    u32x4 w[NB][2];
  };
  auto load = [&](int st, Step& t) __attribute__((always_inline)) {
    const bool last = st == ksteps - 1;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) t.w[b][j] = load_chunk(rw, (vw[b] + 64u * j) | (last ? tail_w[j] : 0u), 128u * (uint32_t)st);
  };

  f32x4 acc[MB][NB];
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](int st, int slot, Step& t, Step& next) __attribute__((always_inline)) {
    const int sn = min(st + WV, ksteps - 1);
    copy(sn, slot ^ 1);
    order();  // (nothing but the loads' arrival covers the copies')
    load(sn, next);
    race_check_drain();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      arrived(t.w[b][0]);
      arrived(t.w[b][1]);
    }
    const char* xt = xs + slot * (XC * 1024);
#pragma unroll
    for (int a = 0; a < MB; ++a) {
      const int row = XR < 16 ? lx & (XR - 1) : 16 * a + lx;
      const char* r = xt + row * 128;
      const i32x8 x = join_chunks(lds_chunk(r + ((lg ^ (row & 7)) << 4)), lds_chunk(r + (((lg + 4) ^ (row & 7)) << 4)));
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = mfma_q8(x, join_chunks(t.w[b][0], t.w[b][1]), acc[a][b]);
    }
    // every read of the tile has returned before a copy into it is issued
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(63));
    order();
  };
  if (wave < ksteps) {
    // (past its last step a wave loads the last one of all again, unused: the
    // loop then has one shape.  In the built code every second step first waits for
    // most of its own loads: where the second step of a turn is left out its loads are
    // still pending at the loop's head)
    Step s0, s1;
    copy(wave, 0);
    order();
    load(wave, s0);
    for (int st = wave; st < ksteps; st += 2 * WV) {
      step(st, 0, s0, s1);
      if (st + WV < ksteps) step(st + WV, 1, s1, s0);
    }
  }

  // the copies' slots become slots of sums, once every copy has landed
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  f32x4* red = reinterpret_cast<f32x4*>(smem);
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) red[(wave * AB + a * NB + b) * 64 + lane] = acc[a][b];
  __syncthreads();
  for (int e = threadIdx.x; e < AB * 64; e += WV * 64) {
    const int ab = e >> 6, l = e & 63;
    f32x4 v = red[e];
#pragma unroll
    for (int q = 1; q < WV; ++q) {
      const f32x4 u = red[q * AB * 64 + e];
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

typedef float f32x16 __attribute__((ext_vector_type(16)));

// GELU(tanh) as t / (1 + 2^(t (c1 + c2 t^2))), c1 = -2 sqrt(2/pi) log2(e) and
// c2 = 0.044715 c1, on values independent of each other: one operation across
// all of them at a time, so that exp2's and the reciprocal's latencies overlap.
template <int N>
__device__ __forceinline__ void gelu_tanh_all(float (&v)[N]) {
  constexpr float c1 = -2.3022081983f, c2 = -0.1029432396f;
  float e[N];
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] = __builtin_fmaf(c2, v[j] * v[j], c1);
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] = __builtin_amdgcn_exp2f(v[j] * e[j]);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = v[j] * __builtin_amdgcn_rcpf(1.0f + e[j]);
}

// Scales and biases (bf16 pairs) of a lane's 16 columns of a block of 32: two
// runs of 8, at first and first + 16.  Past N the last column's stand in.
__device__ __forceinline__ void q8_scales(const Q8Params& p, int first, bool inside, bool has_bias, float (&ws)[16],
                                          uint32_t (&bs)[8]) {
  if (inside) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      __builtin_memcpy(&ws[8 * r], p.ws + first + 16 * r, 32);
      if (has_bias) __builtin_memcpy(&bs[4 * r], p.bias + first + 16 * r, 16);
    }
  } else {
    asm volatile("" : "+v"(first));  // (as in q8_block)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = first + 16 * (i >> 2) + 2 * (i & 3);
      const int u = min(n, p.N - 1), v = min(n + 1, p.N - 1);
      ws[2 * i] = p.ws[u];
      ws[2 * i + 1] = p.ws[v];
      if (has_bias) bs[i] = (uint32_t)p.bias[u] | (uint32_t)p.bias[v] << 16;
    }
  }
}

// A lane's 16 sums of the 32 x 32 block at (mb, nb): row mb + lane % 32, columns
// nb + 8 h + 0..7 and + 16 (h = lane / 32).  Scales, epilogue, one rounding.
__device__ __forceinline__ void q8_block(const Q8Params& p, float (&v)[16], float xs, const float (&ws)[16],
                                         const uint32_t (&bs)[8], int mb, int nb, int lane, bool has_bias, bool gelu) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = v[i] * xs * ws[i];
  if (has_bias) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t u = bs[i >> 1];
      v[i] += __builtin_bit_cast(float, i & 1 ? u & 0xffff0000u : u << 16);
    }
  }
  if (gelu) gelu_tanh_all(v);
  if (nb + 32 <= p.N) {
    // The odd rows of 16 lanes trade one run for the even rows' other: four
    // lanes then hold 64 consecutive bytes of one row (stores of 16 bytes into
    // 32 rows at a time took 1.5 us more per 256 x 256 tile).  The stores may
    // have any alignment: N may be odd.
    u32x4 pk[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto t = __builtin_amdgcn_permlane16_swap(pack_bf16x2(v[2 * i], v[2 * i + 1]),
                                                      pack_bf16x2(v[8 + 2 * i], v[9 + 2 * i]), false, false);
      pk[0][i] = t[0];
      pk[1][i] = t[1];
    }
    int n = nb + 16 * ((lane >> 4) & 1) + 8 * (lane >> 5);
    asm volatile("" : "+v"(n));  // (as below)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int m = mb + 16 * r + (lane & 15);
      if (m < p.M) __builtin_memcpy(p.out + (int64_t)m * p.N + n, &pk[r], 16);
    }
  } else if (mb + (lane & 31) < p.M) {
    // (opaque, or the compiler prepares the columns of all blocks in registers
    // that it does not have)
    int first = nb + 8 * (lane >> 5);
    asm volatile("" : "+v"(first));
    uint16_t* o = p.out + (int64_t)(mb + (lane & 31)) * p.N + first;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int n = 16 * (i >> 3) + (i & 7);
      if (n < p.N - first) o[n] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]));
    }
  }
}

// Many rows: persistent workgroups of four waves (2 x 2) on tiles of 64 FM
// rows by 64 FN columns; a wave's block is FM x FN MFMAs of 32 x 32 x 64
// (v_mfma_f32_32x32x64_f8f6f4: 64 cycles, twice the bf16 rate).
//
// K runs in super-steps of 128 (whole lines of both operands), two MFMA steps
// of 64 each, through SX LDS slots of x and SW of W.  During step 0 of super-step
// q the wave multiplies fragments that it read before, and reads those of step
// 1; then one wait and barrier: every wave has read all of q's slots, and q + 1
// has landed everywhere.  During step 1 it reads the first fragments of q + 1
// and issues the copies of W for q + SW and of x for q + SX into q's slots.  So no
// MFMA waits on an LDS read, and a copy has SX - 1/2 (SW - 1/2) super-steps to
// land.  256 x 256 tiles fill the LDS with 3 and 2 slots (with two each the loop
// took 458 us at 8192^3, now 415 with bias and GELU, where MFMAs issue in 65 % of
// the cycles).  What bounds the smaller tiles is the bytes in flight per
// CU, and the 10 to 13 TB/s that all of them get out of L2; those for
// products with few tiles take the LDS of a whole CU for their rings: 256 x 8192 x
// 4096 33.1 us with 128 x 128 tiles of 3 and 2 slots, 25.6 with 5 each, 20.8 with
// 128 x 64 tiles of 6 each.  The copies run on into the workgroup's next tile,
// which arrives during the epilogue.
//
// LDS rows of 128 bytes, chunk c (16 bytes) at position c ^ (row / 2 & 7): a
// fragment read of 32 rows then hits every bank once in each of its four
// cycles (with row & 7 as the key it took eight).  The
// weights are the MFMA's first operand, so a lane's 16 sums of a block belong
// to one row of x; LDS row i of a block of 32 holds the weight row 16 (i / 16) +
// 8 (i / 4 % 2) + 4 (i / 8 % 2) + i % 4, which makes those sums two runs of 8
// columns, the runs of the two lanes of a row side by side.
// SPLIT: the instance for a K cut into chunks.
template <int FM, int FN, int SX, int SW, bool SPLIT>
__global__ void __launch_bounds__(256, SX * FM + SW * FN <= 10 ? 2 : 1) gemm_q8_tile(Q8Params p) {
  constexpr int BM = 64 * FM, BN = 64 * FN, XS = BM * 128, WS = BN * 128;
  constexpr int CX = 2 * FM, CW = 2 * FN;  // copies of 8 rows per wave and super-step
  // copies that a wait for a super-step may leave in flight: those issued after
  // the later of its own
  constexpr int kAhead = SX <= SW ? (SX - 2) * (CX + CW) : CX + (SW - 2) * (CX + CW);
  constexpr int PER = (CX + CW + FM * FN - 1) / (FM * FN);  // copies (and fragment reads) per MFMA of a step
  __shared__ __attribute__((aligned(1024))) char smem[SX * XS + SW * WS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int wm = (wave >> 1) * (32 * FM), wn = (wave & 1) * (32 * FN);
  const int G = gridDim.x;
  const int wg = __builtin_amdgcn_readfirstlane(remap_workgroup(blockIdx.x, G, 1));
  // a unit of work: one tile, or one chunk of its K (chunk by chunk over all
  // tiles, so that units at work together share panels at the same k)
  const int tiles = p.tiles_m * p.tiles_n, units = SPLIT ? tiles * p.chunks : tiles;
  const int my_units = __builtin_amdgcn_readfirstlane((units - wg + G - 1) / G);
  const uint32_t K = (uint32_t)p.K;
  const int KS = (p.K + 127) >> 7;

  // Copy c of a wave fills the LDS rows 8 t + lane / 8, t = wave * CX + c, whose
  // key is 4 (t & 1) + lane / 16, so a lane's chunk is the same for every other
  // copy (CX and CW are even).
  const int crow = lane >> 3;
  uint32_t chunk[2], tail[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    chunk[e] = 16u * (uint32_t)((lane & 7) ^ (4 * e + (crow >> 1)));
    // chunks of the last super-step past K: bit 31 of the offset, past any end
    tail[e] = 128u * (uint32_t)(KS - 1) + chunk[e] < K ? 0u : 0x80000000u;
  }
  uint32_t vx[CX], vw[CW];
#pragma unroll
  for (int c = 0; c < CX; ++c) vx[c] = (uint32_t)(8 * (wave * CX + c) + crow) * K + chunk[c & 1];
#pragma unroll
  for (int c = 0; c < CW; ++c) {
    const int t = wave * CW + c;
    // LDS row i = 8 (t & 3) + crow of block t / 4
    vw[c] = (uint32_t)(32 * (t >> 2) + 16 * ((t >> 1) & 1) + 8 * (crow >> 2) + 4 * (t & 1) + (crow & 3)) * K + chunk[c & 1];
  }

  // Where each operand's copies are: tile (of this workgroup's) and super-step.
  // Those of a ragged last super-step carry `tail` in their offsets.
  const bool ragged = (K & 127u) != 0;
  __amdgpu_buffer_rsrc_t rx, rw;
  int xi = 0, xq = 0, xend = 0, wi = 0, wq = 0, wend = 0;  // unit, super-step, the unit's end
  // unit i of this workgroup: its tile and its super-steps [q0, q1)
  auto unit = [&](int i, int* tm, int* tn, int* q0, int* q1) __attribute__((always_inline)) {
    const int u = wg + i * G;
    const int c = SPLIT ? __builtin_amdgcn_readfirstlane(u / tiles) : 0;
    tile_coords(u - c * tiles, p.tiles_m, p.tiles_n, 4, tm, tn);
    *tm = __builtin_amdgcn_readfirstlane(*tm);
    *tn = __builtin_amdgcn_readfirstlane(*tn);
    *q0 = SPLIT ? c * p.chunk_steps : 0;
    *q1 = SPLIT ? min(*q0 + p.chunk_steps, KS) : KS;
  };
  auto toggle_x = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < CX; ++c) vx[c] ^= tail[c & 1];
  };
  auto toggle_w = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < CW; ++c) vw[c] ^= tail[c & 1];
  };
  // (past the last unit that one again, never read)
  auto enter_x = [&]() __attribute__((always_inline)) {
    int tm, tn;
    unit(min(xi, my_units - 1), &tm, &tn, &xq, &xend);
    rx = tile_buffer(p.x, (int64_t)tm * BM, p.M, BM, K);
  };
  auto enter_w = [&]() __attribute__((always_inline)) {
    int tm, tn;
    unit(min(wi, my_units - 1), &tm, &tn, &wq, &wend);
    rw = tile_buffer(p.W, (int64_t)tn * BN, p.N, BN, K);
  };
  auto advance_x = [&]() __attribute__((always_inline)) {
    if (ragged && xq == KS - 1) toggle_x();
    if (++xq == xend) {
      ++xi;
      enter_x();
    }
    if (ragged && xq == KS - 1) toggle_x();
  };
  auto advance_w = [&]() __attribute__((always_inline)) {
    if (ragged && wq == KS - 1) toggle_w();
    if (++wq == wend) {
      ++wi;
      enter_w();
    }
    if (ragged && wq == KS - 1) toggle_w();
  };
  auto copy_x = [&](int c, int slot) __attribute__((always_inline)) {
    copy_to_lds(rx, smem + slot * XS + (wave * CX + c) * 1024, vx[c], 128u * (uint32_t)xq);
  };
  auto copy_w = [&](int c, int slot) __attribute__((always_inline)) {
    copy_to_lds(rw, smem + SX * XS + slot * WS + (wave * CW + c) * 1024, vw[c], 128u * (uint32_t)wq);
  };

  // fragments: chunks 4 s + 2 j + h of a row, j = 0, 1
  const int f0 = l32 * 128 + ((h ^ ((l32 >> 1) & 7)) << 4);
  auto frag = [&](int base, int s) __attribute__((always_inline)) {
    return join_chunks(lds_chunk(smem + base + (f0 ^ (64 * s))), lds_chunk(smem + base + (f0 ^ (64 * s + 32))));
  };
  const bool has_bias = p.epi == EPI_BIAS || p.epi == EPI_BIAS_GELU;
  const bool gelu = p.epi == EPI_GELU || p.epi == EPI_BIAS_GELU;
  f32x16 acc[FM][FN];
  i32x8 x[2][FM], w[2][FN];

  auto frag_x = [&](int a, int slot, int s) __attribute__((always_inline)) {
    return frag(slot * XS + (wm + 32 * a) * 128, s);
  };
  auto frag_w = [&](int b, int slot, int s) __attribute__((always_inline)) {
    return frag(SX * XS + slot * WS + (wn + 32 * b) * 128, s);
  };

  enter_x();
  enter_w();
  if (ragged && xq == KS - 1) {
    toggle_x();
    toggle_w();
  }
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
#pragma unroll
  for (int a = 0; a < FM; ++a) x[0][a] = frag_x(a, 0, 0);
#pragma unroll
  for (int b = 0; b < FN; ++b) w[0][b] = frag_w(b, 0, 0);

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
    for (int q = q0; q < q1; ++q) {
#ifdef MM_DEBUG_FULL_SYNC
      race_check_drain();  // every copy issued so far has landed, for every wave
      __builtin_amdgcn_s_barrier();
      order();
#endif
      // step 0
#pragma unroll
      for (int a = 0; a < FM; ++a) x[1][a] = frag_x(a, xb, 1);
#pragma unroll
      for (int b = 0; b < FN; ++b) w[1][b] = frag_w(b, wb, 1);
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[0][b], x[0][a], acc[a][b], 0, 0, 0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < FM * FN; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);           // an MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * PER, 0);     // LDS reads
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
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[1][b], x[1][a], acc[a][b], 0, 0, 0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < FM + FN; ++i) {
        if (i < FM * FN) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // an MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);                   // a fragment
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);                   // a copy
      }
#pragma unroll
      for (int i = FM + FN; i < CX + CW; ++i) {
        if (i < FM * FN) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
      xb = xn;
      wb = wnext;
    }

    if constexpr (SPLIT) {
      // this chunk's sums, 16 bytes per lane and store
      f32x4* o = reinterpret_cast<f32x4*>(p.part) + (int64_t)(wg + ui * G) * (FM * FN * 1024) + threadIdx.x;
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[((a * FN + b) * 4 + i) * 256] =
                f32x4{acc[a][b][4 * i], acc[a][b][4 * i + 1], acc[a][b][4 * i + 2], acc[a][b][4 * i + 3]};
      continue;
    }
    const int m0 = tm * BM + wm, n0 = tn * BN + wn;
    float xs[FM];
#pragma unroll
    for (int a = 0; a < FM; ++a) xs[a] = p.xs[min(m0 + 32 * a + l32, p.M - 1)];
    const bool inside = tn * BN + BN <= p.N;
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      // (loaded a block ahead, these took registers that were not there)
      float ws[16];
      uint32_t bs[8];
      q8_scales(p, n0 + 8 * h + 32 * b, inside, has_bias, ws, bs);
      order();
#pragma unroll
      for (int a = 0; a < FM; ++a) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = acc[a][b][i];
        q8_block(p, v, xs[a], ws, bs, m0 + 32 * a, n0 + 32 * b, lane, has_bias, gelu);
      }
    }
    // (no load of the epilogue is left pending: the next tile's K loop would
    // wait for its copies in order to wait for that)
#pragma unroll
    for (int a = 0; a < FM; ++a) settle(xs[a]);
  }
  __builtin_amdgcn_s_waitcnt(0);  // (the copies past the last unit land before the workgroup ends)
}

// Second launch of a product whose K was cut: the chunks' sums of one 32 x 32
// block per wave of a tile, added in k order, then the epilogue.
template <int FM, int FN>
__global__ void __launch_bounds__(256) gemm_q8_join(Q8Params p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tiles = p.tiles_m * p.tiles_n;
  const int t = blockIdx.x / (FM * FN), ab = blockIdx.x % (FM * FN);
  int tm, tn;
  tile_coords(t, p.tiles_m, p.tiles_n, 4, &tm, &tn);
  const int mb = tm * (64 * FM) + (wave >> 1) * (32 * FM) + 32 * (ab / FN);
  const int nb = tn * (64 * FN) + (wave & 1) * (32 * FN) + 32 * (ab % FN);
  if (mb >= p.M || nb >= p.N) return;
  const bool has_bias = p.epi == EPI_BIAS || p.epi == EPI_BIAS_GELU;
  const bool gelu = p.epi == EPI_GELU || p.epi == EPI_BIAS_GELU;
  const f32x4* part = reinterpret_cast<const f32x4*>(p.part) + (int64_t)t * (FM * FN * 1024) + ab * 1024 + threadIdx.x;
  f32x4 s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = part[i * 256];
  for (int c = 1; c < p.chunks; ++c) {
    part += (int64_t)tiles * (FM * FN * 1024);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 u = part[i * 256];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] += u[j];
    }
  }
  float v[16], ws[16];
  uint32_t bs[8];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = s[i >> 2][i & 3];
  q8_scales(p, nb + 8 * (lane >> 5), nb + 32 <= p.N, has_bias, ws, bs);
  q8_block(p, v, p.xs[min(mb + (lane & 31), p.M - 1)], ws, bs, mb, nb, lane, has_bias, gelu);
}

}  // namespace mmk
