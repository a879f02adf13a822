// mm_device.hpp -- what the kernels share: vector types, epilogue codes, the
// persistent tile order and the activation.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mmk {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Epilogue codes (kernel-internal; the C ABI maps onto them).
enum : int {
  EPI_NONE = 0,
  EPI_BIAS = 1,
  EPI_GELU = 2,
  EPI_BIAS_GELU = 3,
  EPI_SWIGLU = 4,
  EPI_GLU_ID = 5
};

constexpr int kNumXcd = 8;       // MI355X: 8 accelerator dies, round-robin dispatch

// Schedule helpers, shared with the host so that it can describe the order.
__host__ __device__ inline int remap_workgroup(int b, int G, int on) {
  if (!on || G < kNumXcd) return b;
  const int per = G / kNumXcd, rem = G % kNumXcd;
  const int xcd = b % kNumXcd, local = b / kNumXcd;
  return xcd < rem ? xcd * (per + 1) + local : rem * (per + 1) + (xcd - rem) * per + local;
}

__host__ __device__ inline void tile_coords(int t, int tiles_m, int tiles_n, int group_m, int* tm,
                                            int* tn) {
  const int band = group_m * tiles_n;
  const int g = t / band;
  const int first_m = g * group_m;
  const int rows = (tiles_m - first_m) < group_m ? (tiles_m - first_m) : group_m;
  const int r = t - g * band;
  *tm = first_m + r % rows;
  *tn = r / rows;
}

__device__ __forceinline__ float gelu_tanh(float t) {
  // 0.5 t (1 + tanh z) == t / (1 + exp(-2 z)),  z = sqrt(2/pi) (t + 0.044715 t^3)
  const float z = 0.7978845608028654f * (t + 0.044715f * t * t * t);
  return t * __builtin_amdgcn_rcpf(1.0f + __expf(-2.0f * z));
}

// s_waitcnt immediate for gfx9: vmcnt in bits 3:0 and 15:14, expcnt 6:4
// (left at its maximum), lgkmcnt 11:8 (0).
constexpr int waitcnt_vm_lgkm0(int vm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4); }

// One wave-wide copy of 64 x 16 bytes from a buffer to LDS: lane l's chunk, at
// byte `off` (its own) + `base` (the wave's) of the buffer, lands at dst + 16 l;
// zeros do where `off` lies past the buffer's end.
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t buf, char* dst, uint32_t off, uint32_t base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (__attribute__((address_space(3))) void*)dst, 16, off, base, 0, 0);
}

// Marks for the compiler, no instructions.
// No memory operation moves across:
__device__ __forceinline__ void order() { asm volatile("" ::: "memory"); }
// A value is computed before this point and its uses come after it:
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void settle(f32x4& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void settle(u32x4& v) { asm volatile("" : "+v"(v)); }
// The value of a load is there before any memory operation after this point (the
// compiler may move arithmetic on it before):
__device__ __forceinline__ void arrived(u32x4 v) { asm volatile("" ::"v"(v) : "memory"); }

// Nothing, and in the race-check build (MM_DEBUG_FULL_SYNC) a wait for every
// load, copy and LDS operation of the wave: where a kernel's own waits let some
// stay in flight.
__device__ __forceinline__ void race_check_drain() {
#ifdef MM_DEBUG_FULL_SYNC
  __builtin_amdgcn_s_waitcnt(0);
  order();
#endif
}

// A 16-byte read of LDS.  The restrict parameter tells the compiler that no copy
// in flight writes what is read (the kernel's waits and barriers see to it);
// without it, it waits for every copy before reads it cannot tell apart.
__device__ __forceinline__ u32x4 lds_chunk(const char* __restrict__ p) { return *reinterpret_cast<const u32x4*>(p); }

// Two floats to a packed pair of bf16 (round to nearest even), low half
// first: one v_cvt_pk_bf16_f32 through a two-element vector conversion.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

}  // namespace mmk
