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

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kW4Waves = 8;

__device__ __forceinline__ float bf16_float(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }

// + bias, activation, one rounding
__device__ __forceinline__ uint16_t decoder_epilogue(float v, const uint16_t* bias, int epi, int n) {
  if (epi == EPI_BIAS || epi == EPI_BIAS_GELU) v += bf16_float(bias[n]);
  if (epi == EPI_GELU || epi == EPI_BIAS_GELU) v = gelu_tanh(v);
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// The constants of (a & mask) | bits as values the compiler does not know: it
// then makes one v_and_or_b32 of it, which takes no literals on this GPU, where
// of known constants it makes two instructions.
__device__ __forceinline__ void keep_in_registers(uint32_t& mask, uint32_t& bits) {
  asm volatile("" : "+s"(mask), "+v"(bits));
}
// 32 terms of output (m, n) from the definition, added to v: those of 16 bytes of W,
// its words j = 0..3 at k = 128 kb + 32 j + 8 g .. + 7.
__device__ __forceinline__ float w4_terms(const W4Params& p, int m, int n, int kb, int g, float v) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(
      p.W + ((int64_t)(n >> 4) * ((p.K + 127) / 128) + kb) * 64 + 16 * g + (n & 15));
#pragma unroll 1
  for (int j = 0; j < 4; ++j) {
    const int k = 128 * kb + 32 * j + 8 * g;
    if (k >= p.K) break;
    const int64_t at = (int64_t)(k / p.group) * p.N + n;
    const u32x4 x = *reinterpret_cast<const u32x4*>(p.x + (int64_t)m * p.K + k);
    const float s = bf16_float(p.scales[at]), z = p.zeros ? (float)p.zeros[at] : 8.0f;
    const uint32_t word = w[j];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int q = (word >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15;
      v = __builtin_fmaf(bf16_float((uint16_t)(x[e >> 1] >> (16 * (e & 1)))), ((float)q - z) * s, v);
    }
  }
  return v;
}

// Outputs (m, 16 block + 0..15) from the definition, by a whole wave: a lane gets that
// of column lane % 16, right where `wanted`.  The kernel's offset form turns an
// infinite activation (or a sum that overflows) into a NaN of its own making; outputs
// that are not finite are computed again this way, which gives them their IEEE class.
// The first pass takes only the steps with an activation or a scale that is not
// finite: they decide the class, and steps of finite terms leave it.  The second,
// where a sum of finite terms overflowed, takes every step.  A row of 16 x 28672 x
// 8192 with a NaN or an infinity somewhere takes the call from 32 to 44 us, 16 rows of NaN or
// infinities to 135 (a thread per output, term by term: 1850 and 7300).
__device__ __forceinline__ float w4_again(const W4Params& p, int m, int block, bool wanted, int lane) {
  // (opaque, or what depends on the lane alone is computed before the K loop and
  // kept in registers there)
  asm volatile("" : "+v"(lane));
  const int kblocks = (p.K + 127) / 128, n = min(16 * block + (lane & 15), p.N - 1);
  // lanes 16 i .. 16 i + 15 look at step t + i: 8 activations each, a column's scales
  auto odd = [&](int t) __attribute__((always_inline)) {
    const int kb = t + (lane >> 4);
    const u32x4 x = *reinterpret_cast<const u32x4*>(p.x + (int64_t)m * p.K + min(128 * t + 8 * lane, p.K - 8));
    bool o = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t s = p.scales[(int64_t)(min(128 * kb + 32 * j, p.K - 8) / p.group) * p.N + n];
      o |= (x[j] & 0x7f80u) == 0x7f80u || (x[j] >> 16 & 0x7f80u) == 0x7f80u || (s & 0x7f80u) == 0x7f80u;
    }
    return kb < kblocks && o;
  };
  float v = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    v = 0.f;
    for (int t = 0; t < kblocks; t += 8) {
      uint64_t steps[2] = {~uint64_t(0), ~uint64_t(0)};  // 16 bits (lanes) each
      if (pass == 0) {
        const bool o0 = odd(t), o1 = odd(t + 4);
        steps[0] = __ballot(o0);
        steps[1] = __ballot(o1);
      }
      bool done = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (done || steps[h] == 0) continue;
        for (int i = 0; i < 4; ++i, steps[h] >>= 16)
          if ((steps[h] & 0xffff) && t + 4 * h + i < kblocks) v = w4_terms(p, m, n, t + 4 * h + i, lane >> 4, v);
        // a NaN (in any of a column's four lanes) is its result
        const uint64_t nan = __ballot(v != v);
        done = !__any(wanted && !((nan | nan >> 16 | nan >> 32 | nan >> 48) >> (lane & 15) & 1));
      }
      if (done) break;
    }
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    if (!__any(wanted && __builtin_isfinite(v))) break;
  }
  return v;
}

// Where a wave's copies of the activations read (the host's tests walk them).  A
// tile is XR rows by a step (128 k; from 48 rows on a half of one, 64 k); copy i of
// it takes `chunk` (16 bytes) of `row`, at byte `offset` + (in the last step) `tail`
// of the lane + `base` of the wave from the block's first row.  The buffer ends
// with its last row: rows past that read as zeros, and so do the chunks past K,
// whose tail lies beyond any end.  `base` stays within the shortest buffer, one
// row: the hardware compares offsets with the end less the base, so the last
// step's second half, which may start past K, has its 128 bytes in `tail`.
template <int XR>
struct W4Tile {
  static constexpr bool kHalves = XR >= 48;
  static constexpr int kCopies = kHalves ? XR / 8 : XR / 4;  // of eight rows of 128 bytes, or four of 256
  // copies i and i + 4 (halves: all of one half) share the chunk, and so the tail
  static constexpr int kTails = kHalves ? 2 : kCopies < 4 ? kCopies : 4;
  static __host__ __device__ __forceinline__ int row(int i, int lane) {
    return kHalves ? 8 * i + (lane >> 3) : 4 * i + (lane >> 4);
  }
  static __host__ __device__ __forceinline__ int chunk(int i, int lane) {
    return kHalves ? (lane & 7) ^ (lane >> 3) : (lane & 15) ^ (row(i, lane) & 15);
  }
  static __host__ __device__ __forceinline__ uint32_t offset(int i, int lane, uint32_t row_bytes) {
    return (uint32_t)row(i, lane) * row_bytes + 16u * (uint32_t)chunk(i, lane);
  }
  // t: the half, or the copy (mod 4)
  static __host__ __device__ __forceinline__ uint32_t tail(int t, int lane, int K) {
    const int k = ((K + 127) / 128 - 1) * 128 + 8 * chunk(t, lane) + (kHalves ? 64 * t : 0);
    return k < K ? (kHalves ? 128u * (uint32_t)t : 0u) : 0x80000000u;
  }
  static __host__ __device__ __forceinline__ uint32_t base(int kb, int half, bool last) {
    return (uint32_t)kb * 256u + (kHalves && !last ? 128u * (uint32_t)half : 0u);
  }
};

// XR activation rows (4: the first four of a block of 16, whose others are
// never used; 16, 32, 48 or 64: 48 rows by 14336 x 4096 take 16.9 us as 48 and
// 19.5 as 64) by NB blocks of 16 columns per workgroup.  Its WV waves take
// every WV-th 128-k step, each step's loads issued one step ahead, and their
// sums meet in LDS, added in wave order.  No barrier until then: what a wave
// stages in LDS is its own.
//
// Activations: each wave copies its step's tile, XR rows of 256 bytes, from
// L2 to LDS (whole lines: fragments loaded straight into registers touch 16
// half lines each, and the products of 16 rows, bound by those, ran at 33 us
// where whole lines made it 30).  16-byte chunk c of row r sits at position
// c ^ (r & 15), so the fragment reads of 16 rows at one chunk hit 16 banks.
//
// Scales: lane (group, four columns) loads the step's, widens them with the
// offset -(16 + z), and leaves the pairs in LDS, from where the lanes of each
// column read theirs (a load per column block and group would cost more of
// the address unit than the weight does).
//
// Measured: 16 x 28672 x 8192 by groups of 128 with zeros 26.9 us, 4.6 TB/s (a
// large copy runs at 4.8); 1 x 4096 x 4096 4.4 us, where the launch and the
// one step's latency are most of it.  From 17 rows on no unit is at its limit; a step
// fetches its activations from L2 (every workgroup all of them), widens and multiplies
// in turn, and two waves per SIMD and few steps per wave do not overlap these
// fully: 64 x 14336 x 4096 takes 18.5 us against a floor of 7, with 177 MB of L2 requests
// (117 of activations; 9.6 TB/s), the vector ALU busy in 51 % of a working CU's cycles and the
// matrix units in 27; 24 x 8192 x 8192 13.6 against 7.5, 148 MB, 43 and 23 %.
//
// (16 rows: the LDS holds two workgroups, and so do the registers, of at most 128.)
template <int XR, int NB, int G, int WV>
__global__ void __launch_bounds__(WV * 64, XR == 16 ? 4 : 2) gemm_w4(W4Params p) {
  constexpr int MB = XR < 16 ? 1 : XR / 16;
  constexpr int AB = MB * NB;
  constexpr int GP = 128 / G;             // groups per step
  // HALVES: the two LDS tiles of a wave are the halves (64 k) of one step, not
  // two steps: half the LDS and half the fragment registers, which 64 rows by
  // four column blocks would not have otherwise
  using Tile = W4Tile<XR>;
  constexpr bool HALVES = Tile::kHalves;
  // a chunk: what shares one scale and one pass over the accumulators; JC
  // MFMAs, whose fragments are read JR at a time
  constexpr int JC = (HALVES && G > 64 ? 64 : G) / 32;
  constexpr int JR = HALVES ? 2 : JC;
  // The compiler would start all of a step's products at once.  Where that
  // takes more registers than there are (or than the waves of two workgroups
  // share), a column block's products wait for those BB blocks before.
  constexpr bool CALM = MB >= 3 || AB * GP > (MB == 2 ? 16 : 4);
  constexpr int BB = MB < 3 && NB > 1 ? 2 : 1;
  constexpr int XC = Tile::kCopies, XT = XC * 1024;
  // scale pairs: a column's GP * NB, in an odd number of 16-byte units (reads
  // of 16 columns then fall in 16 bank groups)
  constexpr int PB = GP * NB, SU = PB < 2 ? 1 : (PB / 2) | 1;
  constexpr int kSc = 16 * SU * 16;
  constexpr int kX = 2 * XT, kWave = kX + kSc;  // LDS bytes per wave
  constexpr int RS = AB > 8 ? WV / 2 : WV;  // waves whose sums are in LDS at once
  constexpr int kRed = RS * AB * 1024;
  __shared__ __attribute__((aligned(1024))) char smem[WV * kWave > kRed ? WV * kWave : kRed];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lx = lane & 15, lg = lane >> 4;
  const int kblocks = (p.K + 127) >> 7;
  const int nblocks = (p.N + 15) >> 4;
  const int groups = (p.K + G - 1) / G;
  const int m0 = blockIdx.y * XR;
  // neighbouring blocks on one XCD: they share the lines of the scales and zeros
  // (1 x 28672 x 8192 by groups of 32: 28.8 -> 27.8 us)
  const int b0 = remap_workgroup(blockIdx.x, gridDim.x, 1) * NB;
  char* xs = smem + wave * kX;
  char* sc = smem + WV * kX + wave * kSc;

  const uint32_t row_bytes = (uint32_t)p.K * 2u;
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(p.x + (int64_t)m0 * p.K), (short)0, (int)((uint32_t)min(p.M - m0, XR) * row_bytes),
      0x00020000);
  uint32_t voff[XC], tail[Tile::kTails];
#pragma unroll
  for (int i = 0; i < XC; ++i) {
    voff[i] = Tile::offset(i, lane, row_bytes);
    if (i < Tile::kTails) tail[i] = Tile::tail(i, lane, p.K);
  }
  // scales: lane (group sg of the step, columns sn .. sn + 3); lanes past the
  // step's groups repeat earlier ones.  The last columns' loads start early
  // enough to end with the row (N >= 4) and are shifted into place.
  const int sg = lane / (4 * NB) % GP, sq = lane % (4 * NB);
  const int sn = 16 * b0 + 4 * sq;
  const int back = max(0, sn + 4 - p.N);
  const int shift = 8 * min(back, 3);
  const uint8_t* zp = p.zeros ? p.zeros : reinterpret_cast<const uint8_t*>(p.scales);

  struct Step {
    u32x4 w[NB];
    uint64_t s;  // four bf16
    uint32_t z;
  };
  // tile: of step kb, or (HALVES) half `tile` of it
  auto copy = [&](int kb, int tile) __attribute__((always_inline)) {
    const bool last = kb == kblocks - 1;
#pragma unroll
    for (int i = 0; i < XC; ++i)
      copy_to_lds(rx, xs + tile * XT + i * 1024, voff[i] + (last ? tail[HALVES ? tile : i & 3] : 0u),
                  Tile::base(kb, tile, last));
  };
  auto load = [&](int kb, Step& t) __attribute__((always_inline)) {
    const int group = min(kb * GP + sg, groups - 1);
    const int64_t at = (int64_t)group * p.N + (sn - back);
    __builtin_memcpy(&t.s, p.scales + at, 8);
    __builtin_memcpy(&t.z, zp + at, 4);
#pragma unroll
    for (int b = 0; b < NB; ++b)  // (a block past N reads the last one; its sums are dropped)
      t.w[b] = __builtin_nontemporal_load(p.W + ((int64_t)min(b0 + b, nblocks - 1) * kblocks + kb) * 64 + lane);
  };

  f32x4 acc[MB][NB];
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
  uint32_t mask = 0x00780078u, sixteen = 0x41804180u;
  keep_in_registers(mask, sixteen);

  // Step kb, and the loads of the wave's next.  Whole steps: the next one's
  // copies go out first, in an order fixed here (loads arrive in order, so once a
  // step's weights are there its activations are: no other wait covers them).  Halves: the next step's weights go out first,
  // the copies of each half once this step's fragments of it are in registers;
  // so what a wait may leave in flight are the loads issued after its half.
  constexpr int kLoads = NB + 2;
  auto step = [&](int kb, int tile, Step& t, Step& next) __attribute__((always_inline)) {
    const int kn = min(kb + WV, kblocks - 1);
    if constexpr (HALVES) {
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(XC));
      order();
      load(kn, next);
      order();
      race_check_drain();
    } else {
      copy(kn, tile ^ 1);
      order();
      load(kn, next);
      race_check_drain();
#pragma unroll
      for (int b = 0; b < NB; ++b) arrived(t.w[b]);
    }
    // (a group past K has no activations: scale 0, whatever the last group's is)
    const uint64_t s = kb * GP + sg < groups ? t.s >> (2 * shift) : 0u;
    const uint32_t z = p.zeros ? t.z >> shift : 0x08080808u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bits = (uint32_t)(s >> (16 * i)) << 16;
      // column 4 sq + i of the workgroup's: block sq / 4, lane 4 (sq % 4) + i
      *reinterpret_cast<f32x2*>(sc + (4 * (sq & 3) + i) * (16 * SU) + (sg * NB + (sq >> 2)) * 8) =
          f32x2{__builtin_bit_cast(float, bits), -16.0f - (float)((z >> (8 * i)) & 255u)};
    }
    order();  // (a wave's LDS operations run in order)
    f32x4 so = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 4 / JR; ++r) {
      if (HALVES && r == 1) {
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(kLoads + XC));
        order();
        race_check_drain();
      }
      const char* xt = xs + (HALVES ? r : tile) * XT;
      u32x4 x[MB][JR];
#pragma unroll
      for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int j = 0; j < JR; ++j) {
          const int row = XR < 16 ? lx & (XR - 1) : 16 * a + lx;
          x[a][j] = *reinterpret_cast<const u32x4*>(
              xt + (HALVES ? row * 128 + (((4 * j + lg) ^ (row & 7)) << 4)
                           : row * 256 + (((4 * (r * JR + j) + lg) ^ (row & 15)) << 4)));
        }
      // every read of a tile has returned before a copy into it is issued
      // (whole steps: at the next one's start)
      if (HALVES || r == 4 / JR - 1) {
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(63));
        order();
        if constexpr (HALVES) copy(kn, r);
      }
#pragma unroll
      for (int c = 0; c < JR / JC; ++c) {
        const int g = (r * JR + c * JC) * 32 / G;  // the chunk's group in the step
        f32x4 sx[MB];
#pragma unroll
        for (int a = 0; a < MB; ++a) {
          sx[a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < JC; ++j)
            sx[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[a][c * JC + j]), ones, sx[a],
                                                            0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float scale, off;
          if constexpr (PB == 1) {
            const f32x2 u = *reinterpret_cast<const f32x2*>(sc + lx * (16 * SU));
            scale = u[0];
            off = u[1];
          } else {
            // two pairs per read
            const int pair = g * NB + b;
            if (pair % 2 == 0 || GP == 1) so = *reinterpret_cast<const f32x4*>(sc + lx * (16 * SU) + (pair & ~1) * 8);
            scale = so[2 * (pair & 1)];
            off = so[2 * (pair & 1) + 1];
          }
          if constexpr (CALM) {
            const int before = (b + NB - BB) % NB;
#pragma unroll
            for (int a = 0; a < MB; ++a) settle(acc[a][before]);
            settle(t.w[b]);
          }
          f32x4 d[MB];
#pragma unroll
          for (int a = 0; a < MB; ++a) d[a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < JC; ++j) {
            const uint32_t v = t.w[b][r * JR + c * JC + j];
            const u32x4 q = {((v << 3) & mask) | sixteen, ((v >> 1) & mask) | sixteen, ((v >> 5) & mask) | sixteen,
                             ((v >> 9) & mask) | sixteen};
#pragma unroll
            for (int a = 0; a < MB; ++a)
              d[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[a][c * JC + j]),
                                                             __builtin_bit_cast(bf16x8, q), d[a], 0, 0, 0);
          }
#pragma unroll
          for (int a = 0; a < MB; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[a][b][i] = __builtin_fmaf(scale, __builtin_fmaf(off, sx[a][i], d[a][i]), acc[a][b][i]);
        }
      }
    }
    order();
  };

  if (wave < kblocks) {
    // (past its last step a wave loads the last one of all again, unused: the
    // loop then has one shape, which the halves' counted waits need.  Of whole steps
    // every second one first waits, in the built code, for all of its own loads:
    // where the second step of a turn is left out its loads are still pending at
    // the loop's head)
    Step s0, s1;
    if constexpr (HALVES) {
      load(wave, s0);
      order();
      copy(wave, 0);
      copy(wave, 1);
    } else {
      copy(wave, 0);
      order();
      load(wave, s0);
    }
    for (int kb = wave; kb < kblocks; kb += 2 * WV) {
      step(kb, 0, s0, s1);
      if (kb + WV < kblocks) step(kb + WV, 1, s1, s0);
    }
  }

  // the copies' slots become slots of sums, once every copy has landed
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  f32x4* red = reinterpret_cast<f32x4*>(smem);
  auto put = [&](int place) __attribute__((always_inline)) {
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) red[(place * AB + a * NB + b) * 64 + lane] = acc[a][b];
  };
  if constexpr (RS < WV) {  // the later half of the waves hands its sums to the earlier first
    if (wave >= RS) put(wave - RS);
    __syncthreads();
    if (wave < RS) {
#pragma unroll
      for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const f32x4 u = red[(wave * AB + a * NB + b) * 64 + lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[a][b][i] += u[i];
        }
      put(wave);
    }
  } else {
    put(wave);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < AB * 64; e += WV * 64) {
    const int ab = e >> 6, l = e & 63;
    f32x4 v = red[e];
#pragma unroll
    for (int q = 1; q < RS; ++q) {
      const f32x4 u = red[q * AB * 64 + e];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += u[i];
    }
    // lane l of block (a, b): rows 16 a + 4 (l / 16) + i, column 16 b + l % 16
    const int block = b0 + ab % NB, n = 16 * block + (l & 15), mb = m0 + 16 * (ab / NB);
    uint32_t again = 0;  // which of the four are not finite
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = mb + 4 * (l >> 4) + i;
      if (n >= p.N || m >= p.M) continue;
      if (__builtin_isfinite(v[i]))
        p.out[(int64_t)m * p.N + n] = decoder_epilogue(v[i], p.bias, p.epi, n);
      else
        again |= 1u << i;
    }
    // row by row (whole waves get here: AB * 64 values, WV * 64 threads)
    for (int r = 0; __any(again != 0); ++r) {
      const bool mine = (l >> 4) == (r >> 2) && (again >> (r & 3) & 1);
      const uint64_t lanes = __ballot(mine);
      if (lanes == 0) continue;
      const bool column = (lanes | lanes >> 16 | lanes >> 32 | lanes >> 48) >> (l & 15) & 1;
      const float o = w4_again(p, mb + r, block, column, l);
      if (mine) {
        p.out[(int64_t)(mb + r) * p.N + n] = decoder_epilogue(o, p.bias, p.epi, n);
        again &= ~(1u << (r & 3));
      }
    }
  }
}

// Fewer than four columns: every output from the definition, one per thread.
__global__ void __launch_bounds__(64) gemm_w4_narrow(W4Params p) {
  const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= (int64_t)p.M * p.N) return;
  const int m = (int)(i / p.N), n = (int)(i % p.N);
  float v = 0.f;
  for (int c = 0; c < 4 * ((p.K + 127) / 128); ++c) v = w4_terms(p, m, n, c >> 2, c & 3, v);
  p.out[i] = decoder_epilogue(v, p.bias, p.epi, n);
}

// Lays out codes [N][K] (one byte each, the low four bits taken) as packed
// words, one per thread from word `first` on (256 of them make a kilobyte); what pads
// N and K is code 0.
__global__ void __launch_bounds__(256) w4_pack(const uint8_t* codes, uint32_t* packed, int N, int K, int64_t first) {
  const int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
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
