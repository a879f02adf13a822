// mm_decoder.hip -- C ABI of the decoder-layer operators (declared in
// include/mm.h): the residual addition with its RMS norm or layer norm and their
// gradients, the products with 4-bit and 8-bit weights, the linear layer with an adapter
// per row, and the mixture-of-experts FFN.  Argument checks, the choice of a
// kernel's shape, launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "mm_host.hpp"
#include "rms_norm.hpp"
#include "gemm_w4.hpp"
#include "gemm_q8.hpp"
#include "layer_norm.hpp"
#include "moe_ffn.hpp"
#include "linear_lora.hpp"

using namespace mmh;

namespace {

constexpr int64_t kLimit = int64_t(1) << 31;

// A launch takes fewer than 2^32 threads along x; longer ones go out in parts (or
// their sizes are refused before).
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;
constexpr int64_t kMaxGridY = 65535;

mm_status launch(const void* kernel, dim3 grid, int threads, void** args, void* stream, const char* what) {
  if ((int64_t)grid.x * threads > kMaxThreads)
    return fail(MM_ERR_UNSUPPORTED, std::string(what) + ": more than 2^32 - 1 threads");
  const hipError_t e = hipLaunchKernel(kernel, grid, dim3(threads), args, 0, static_cast<hipStream_t>(stream));
  if (e != hipSuccess)
    return fail(MM_ERR_HIP, std::string("hipLaunchKernel (") + what + "): " + hipGetErrorString(e));
  return MM_OK;
}

template <typename F>
const void* fn(F* kernel) {
  return reinterpret_cast<const void*>(kernel);
}

// ----------------------------------------------------------------------------
// RMS norm
// ----------------------------------------------------------------------------
mm_status check_norm_sizes(int64_t rows, int64_t hidden, mm_out_dtype dtype) {
  if (rows < 0 || hidden < 0) return fail(MM_ERR_INVALID_VALUE, "negative size");
  if (dtype != MM_OUT_BF16 && dtype != MM_OUT_F32) return fail(MM_ERR_INVALID_VALUE, "bad stream type");
  if (rows >= kLimit) return fail(MM_ERR_UNSUPPORTED, "rows must be below 2^31");
  if (hidden > mmk::kNormMaxHidden) return fail(MM_ERR_UNSUPPORTED, "hidden must be at most 32768");
  if (hidden % 8 != 0) return fail(MM_ERR_MISALIGNED, "hidden must be a multiple of 8 elements");
  return MM_OK;
}

// Threads per row and vectors of 8 per thread (1, 2 or 4).
void norm_shape(int64_t hidden, int64_t threads_wanted, int* threads, int* vpt) {
  const int64_t vectors = hidden / 8;
  int v = 1;
  while (v < 4 && threads_wanted * v < vectors) v *= 2;
  *vpt = v;
  *threads = (int)(cdiv(cdiv(vectors, v), 64) * 64);
}

template <bool F32, bool Q8>
const void* norm_kernel(int vpt) {
  switch (vpt) {
    case 1: return fn(&mmk::rms_norm<F32, Q8, 1>);
    case 2: return fn(&mmk::rms_norm<F32, Q8, 2>);
  }
  return fn(&mmk::rms_norm<F32, Q8, 4>);
}

template <bool F32>
const void* norm_grad_kernel(int vpt, int threads) {
  if (threads <= 512) return vpt == 1 ? fn(&mmk::rms_norm_grad<F32, 1, true>) : fn(&mmk::rms_norm_grad<F32, 2, true>);
  if constexpr (F32) {
    if (vpt == 4) return fn(&mmk::rms_norm_grad<F32, 4, false>);
  }
  return fn(&mmk::rms_norm_grad<F32, 2, false>);
}

mm_status norm(const void* x, int64_t ld_x, const void* residual, const void* weight, void* h, void* y, float* stat,
               int64_t rows, int64_t hidden, float eps, mm_out_dtype dtype, bool q8, void* stream) {
  mm_status s = check_norm_sizes(rows, hidden, dtype);
  if (s != MM_OK) return s;
  if (!(eps >= 0.0f)) return fail(MM_ERR_INVALID_VALUE, "eps must not be negative");
  if (rows == 0 || hidden == 0) return MM_OK;
  if (!x || !weight || !y || !stat || (residual && !h)) return fail(MM_ERR_INVALID_VALUE, "null pointer");
  if (ld_x < hidden || ld_x >= kLimit) return fail(MM_ERR_INVALID_VALUE, "rows of x must not overlap (ld_x < hidden)");
  if (ld_x % 8 != 0) return fail(MM_ERR_MISALIGNED, "ld_x must be a multiple of 8 elements");
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(y, 16) || !aligned(stat, 4) ||
      (residual && (!aligned(residual, 16) || !aligned(h, 16))))
    return fail(MM_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  const int64_t e = dtype == MM_OUT_F32 ? 4 : 2;
  const int64_t xb = ((rows - 1) * ld_x + hidden) * e, hb = rows * hidden * e;
  const int64_t yb = rows * hidden * (q8 ? 1 : 2), sb = rows * 4, wb = hidden * 2;
  const struct { const void* p; int64_t n; } in[] = {{x, xb}, {residual, hb}, {weight, wb}};
  const struct { const void* p; int64_t n; } out[] = {{residual ? h : nullptr, hb}, {y, yb}, {stat, sb}};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 3; ++i) {
      // h may be residual itself, or x (a contiguous one): each element is
      // read before it is written, by one thread
      if (o == 0 && ((i == 1 && h == residual) || (i == 0 && h == x && ld_x == hidden))) continue;
      if (overlaps(out[o].p, out[o].n, in[i].p, in[i].n))
        return fail(MM_ERR_INVALID_VALUE, "an output overlaps an input");
    }
    for (int q = 0; q < o; ++q)
      if (overlaps(out[o].p, out[o].n, out[q].p, out[q].n)) return fail(MM_ERR_INVALID_VALUE, "outputs overlap");
  }
  mmk::RmsNormParams p;
  p.weight = static_cast<const uint16_t*>(weight);
  p.ld_x = ld_x;
  p.hidden = (int)hidden;
  p.eps = eps;
  int threads, vpt;
  // Measured (us, bf16, with 256 / 512 / 1024 threads wanted): 16 x 8192 5.2 / 4.0 /
  // 3.9, 512 x 8192 10.5 / 8.3 / 8.9, 4096 x 8192 49.1 / 47.8 / 47.4, 8192 x 4096
  // without residual 24.8 / 27.0 / 26.7, 1024 x 16384 22.4 / 22.5 / 23.3.
  norm_shape(hidden, 512, &threads, &vpt);
  void* args[] = {&p};
  const void* k = dtype == MM_OUT_F32 ? (q8 ? norm_kernel<true, true>(vpt) : norm_kernel<true, false>(vpt))
                                      : (q8 ? norm_kernel<false, true>(vpt) : norm_kernel<false, false>(vpt));
  const int64_t most = kMaxThreads / threads;
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    const int64_t n = std::min(rows - r0, most);
    p.x = static_cast<const char*>(x) + r0 * ld_x * e;
    p.residual = residual ? static_cast<const char*>(residual) + r0 * hidden * e : nullptr;
    p.h = residual ? static_cast<char*>(h) + r0 * hidden * e : nullptr;
    p.y = static_cast<char*>(y) + r0 * hidden * (q8 ? 1 : 2);
    p.stat = stat + r0;
    p.rows = n;
    if ((s = launch(k, dim3((unsigned)n), threads, args, stream, "rms_norm")) != MM_OK) return s;
  }
  return MM_OK;
}

template <bool F32>
const void* norm_grad_few_kernel(int vpt) {
  return vpt == 1   ? fn(&mmk::rms_norm_grad_few<F32, 1>)
         : vpt == 2 ? fn(&mmk::rms_norm_grad_few<F32, 2>)
                    : fn(&mmk::rms_norm_grad_few<F32, 4>);
}

// Up to this many rows the gradient is one launch, whose columns' workgroups read
// dy and h again.  Measured (us, one launch / two, bf16): 16 x 4096 2.8 / 5.9, 256 x
// 4096 5.1 / 10.7, 1024 x 4096 13.1 / 19.2, 2048 x 1024 17.1 / 20.1, 2048 x 4096
// 23.3 / 22.9, 2048 x 8192 33.5 / 35.5, 4096 x 4096 42.4 / 33.2.
// A row longer than kLongRow does not fit the registers of 1024 threads together
// with its dw, and in bf16 one launch is then faster at any count: 4096 x 16392
// 189 / 267, 8192 x 32768 656 / 695 (fp32: 266 / 254, 1003 / 796).
constexpr int64_t kFewRows = 2048, kLongRow = 16384;

// Workgroups of the gradient, each with a part of dweight: as few as keep the
// memory busy.  Measured (us, 1 / 2 / 4 per CU): 4096 x 8192 fp32 112 / 118 / 133,
// 8192 x 4096 bf16 68 / 58 / 68, 8192 x 2048 bf16 54 / 37 / 40.
mm_status norm_grad_parts(int64_t rows, int64_t hidden, int64_t* parts) {
  int cus = 0;
  const mm_status s = device_cus(&cus);
  *parts = std::min<int64_t>(rows, (hidden >= 8192 ? 1 : hidden > 1024 ? 2 : 4) * (int64_t)cus);
  return s;
}

// ----------------------------------------------------------------------------
// Products with 4-bit and 8-bit weights
// ----------------------------------------------------------------------------
bool map_epilogue(mm_epilogue e, int* epi) {
  switch (e) {
    case MM_EPI_NONE: *epi = mmk::EPI_NONE; return true;
    case MM_EPI_BIAS: *epi = mmk::EPI_BIAS; return true;
    case MM_EPI_GELU_TANH: *epi = mmk::EPI_GELU; return true;
    case MM_EPI_BIAS_GELU_TANH: *epi = mmk::EPI_BIAS_GELU; return true;
  }
  return false;
}

mm_status check_product(int64_t M, int64_t N, int64_t K, const void* bias, const void* out, mm_epilogue epi_in,
                        int* epi) {
  if (M < 0 || N < 0 || K < 0) return fail(MM_ERR_INVALID_VALUE, "negative size");
  if (M >= kLimit || N >= kLimit || K >= kLimit) return fail(MM_ERR_UNSUPPORTED, "M, N and K must be below 2^31");
  if (!map_epilogue(epi_in, epi)) return fail(MM_ERR_INVALID_VALUE, "bad epilogue");
  if (M == 0 || N == 0) return MM_OK;
  if (!out) return fail(MM_ERR_INVALID_VALUE, "null output pointer");
  if (!aligned(out, 2)) return fail(MM_ERR_MISALIGNED, "out must be aligned to its element size");
  const bool need_bias = *epi == mmk::EPI_BIAS || *epi == mmk::EPI_BIAS_GELU;
  if (need_bias && !bias) return fail(MM_ERR_INVALID_VALUE, "epilogue needs a bias");
  if (need_bias && !aligned(bias, 2)) return fail(MM_ERR_MISALIGNED, "bias must be 2-byte aligned");
  const int64_t room = int64_t(1) << 60;
  if (M * K > room || N * K > room || M * N > room)
    return fail(MM_ERR_UNSUPPORTED, "an operand or the output spans 2^60 elements or more");
  if (need_bias && overlaps(out, M * N * 2, bias, N * 2))
    return fail(MM_ERR_INVALID_VALUE, "out overlaps an input");
  return MM_OK;
}

// Column blocks (1, 2 or 4 of 16 columns) per workgroup for few rows.  Each
// workgroup reads all activations for itself, which costs about `share` tenths
// of a block's weights, and the CU with the most workgroups ends last: the count
// with the least of (workgroups to a CU, rounded up) x (blocks + share) is taken.
// (A launch takes kMaxRowsGridX workgroups along x.)
constexpr int64_t kMaxRowsGridX = kMaxThreads / (mmk::kW4Waves * 64);

int column_blocks(int64_t blocks, int64_t gy, int cus, int share) {
  int best = 4;
  int64_t cost = -1;
  for (int nb = 1; nb <= 4; nb *= 2) {
    const int64_t gx = cdiv(blocks, nb);
    const int64_t c = cdiv(gx * gy, cus) * (10 * nb + share);
    if (gx <= kMaxRowsGridX && (cost < 0 || c < cost)) best = nb, cost = c;
  }
  return best;
}

template <int XR, int NB>
const void* w4_kernel(int group) {
  switch (group) {
    case 32: return fn(&mmk::gemm_w4<XR, NB, 32, mmk::kW4Waves>);
    case 64: return fn(&mmk::gemm_w4<XR, NB, 64, mmk::kW4Waves>);
  }
  return fn(&mmk::gemm_w4<XR, NB, 128, mmk::kW4Waves>);
}
template <int XR>
const void* w4_kernel(int nb, int group) {
  return nb == 1 ? w4_kernel<XR, 1>(group) : nb == 2 ? w4_kernel<XR, 2>(group) : w4_kernel<XR, 4>(group);
}
const void* w4_kernel(int rows, int nb, int group) {
  switch (rows) {
    case 4: return w4_kernel<4>(nb, group);
    case 16: return w4_kernel<16>(nb, group);
    case 32: return w4_kernel<32>(nb, group);
    case 48: return w4_kernel<48>(nb, group);
  }
  return w4_kernel<64>(nb, group);
}

template <int XR>
const void* q8_rows_kernel(int nb) {
  return nb == 1   ? fn(&mmk::gemm_q8_rows<XR, 1, mmk::kW4Waves>)
         : nb == 2 ? fn(&mmk::gemm_q8_rows<XR, 2, mmk::kW4Waves>)
                   : fn(&mmk::gemm_q8_rows<XR, 4, mmk::kW4Waves>);
}
const void* q8_rows_kernel(int rows, int nb) {
  switch (rows) {
    case 4: return q8_rows_kernel<4>(nb);
    case 16: return q8_rows_kernel<16>(nb);
    case 32: return q8_rows_kernel<32>(nb);
  }
  return q8_rows_kernel<64>(nb);
}

template <int FM, int FN, int SX, int SW>
const void* q8_tile_kernel(bool split) {
  return split ? fn(&mmk::gemm_q8_tile<FM, FN, SX, SW, true>) : fn(&mmk::gemm_q8_tile<FM, FN, SX, SW, false>);
}
const void* q8_tile_kernel(int kind, bool split) {
  switch (kind) {
    case 0: return q8_tile_kernel<4, 4, 3, 2>(split);
    case 1: return q8_tile_kernel<4, 2, 3, 4>(split);
    case 2: return q8_tile_kernel<2, 2, 3, 2>(split);
    case 3: return q8_tile_kernel<2, 2, 5, 5>(split);
  }
  return q8_tile_kernel<2, 1, 6, 6>(split);
}
const void* q8_join_kernel(int kind) {
  switch (kind) {
    case 0: return fn(&mmk::gemm_q8_join<4, 4>);
    case 1: return fn(&mmk::gemm_q8_join<4, 2>);
    case 2:
    case 3: return fn(&mmk::gemm_q8_join<2, 2>);
  }
  return fn(&mmk::gemm_q8_join<2, 1>);
}

// ----------------------------------------------------------------------------
// 8-bit products of more than kQ8Rows rows: the kind of tile, and whether K is
// cut so that few tiles fill the GPU.
// ----------------------------------------------------------------------------
constexpr int64_t kQ8Rows = 64;
constexpr int64_t kQ8MaxChunks = 8;
constexpr int64_t kQ8Cus = 256;  // of the target GPU

// A kind's cost is the time (us) of one 128-k super-step with every CU at work
// and with few (`low`); operands from HBM.  A small tile reads more per product,
// but its ring holds more super-steps (us, the kinds in turn, K whole or in the
// chunks that suit each best): 4096 x 4096 x 4096 61.6 / 70.7 / 69.3 / 81.1 / 105;
// 2048 x 3008 x 4096 44.2 / 34.3 / 39.3 / 42.2 / 45.5; 6000 x 6000 x 4096 159 /
// 157 / 151 / 176 / 236; 1024 x 4096 x 4096 38.2 / 32.9 / 32.3 / 25.4 / 32.0; 256 x 8192
// x 4096 55 / 27.5 / 26.1 / 24.3 / 20.8.
struct Q8Kind {
  int fm, fn, resident;  // tile of 64 fm x 64 fn, workgroups per CU
  double step, low;
};
constexpr Q8Kind kQ8Kinds[] = {
    {4, 4, 1, 1.72, 1.30}, {4, 2, 1, 1.12, 0.72}, {2, 2, 2, 1.12, 0.75}, {2, 2, 1, 0.66, 0.60}, {2, 1, 1, 0.52, 0.43}};

struct Q8Plan {
  int kind = 0;
  int64_t tiles_m = 0, tiles_n = 0, chunks = 1, chunk_steps = 0;
};

int64_t q8_ws_bytes(const Q8Plan& p) {
  if (p.chunks == 1) return 0;
  const Q8Kind& k = kQ8Kinds[p.kind];
  return p.tiles_m * p.tiles_n * p.chunks * k.fm * k.fn * 4096 * 4;
}

Q8Plan q8_plan(int64_t M, int64_t N, int64_t K, int64_t max_chunks) {
  const int64_t steps = cdiv(K, 128);
  Q8Plan best;
  double bc = -1.0;
  for (int kind = 0; kind < (int)std::size(kQ8Kinds); ++kind) {
    const Q8Kind& k = kQ8Kinds[kind];
    Q8Plan p;
    p.kind = kind;
    p.tiles_m = cdiv(M, 64 * k.fm);
    p.tiles_n = cdiv(N, 64 * k.fn);
    for (int64_t c = 1; c <= max_chunks; ++c) {
      p.chunk_steps = cdiv(steps, c);
      p.chunks = cdiv(steps, p.chunk_steps);
      if (p.chunks != c || (c > 1 && p.chunk_steps < 4)) continue;
      const int64_t units = p.tiles_m * p.tiles_n * c, slots = kQ8Cus * k.resident;
      const int64_t rem = units % slots;
      const double pass =
          (double)(units / slots) * k.step + (rem ? k.low + (k.step - k.low) * (double)rem / (double)slots : 0.0);
      // per pass, a start and an end worth about four super-steps
      double cost = pass * (double)(p.chunk_steps + 4);
      // the chunks' sums written and read (they stay in the cache behind L2), and
      // a second launch
      if (c > 1) cost += 2.0 * (double)q8_ws_bytes(p) / 8e6 + 3.0;
      if (bc < 0.0 || cost < bc) {
        bc = cost;
        best = p;
      }
    }
  }
  return best;
}

// ----------------------------------------------------------------------------
// Layer norm
// ----------------------------------------------------------------------------
struct Span {
  const void* p;
  int64_t n;
};

// Whether an output shares memory with an input or another output.
template <size_t I, size_t O>
bool any_overlap(const Span (&in)[I], const Span (&out)[O]) {
  for (size_t o = 0; o < O; ++o) {
    for (size_t i = 0; i < I; ++i)
      if (overlaps(out[o].p, out[o].n, in[i].p, in[i].n)) return true;
    for (size_t q = 0; q < o; ++q)
      if (overlaps(out[o].p, out[o].n, out[q].p, out[q].n)) return true;
  }
  return false;
}

template <bool F32>
const void* layer_norm_kernel(int vpt) {
  return vpt == 1 ? fn(&mmk::layer_norm<F32, 1>) : vpt == 2 ? fn(&mmk::layer_norm<F32, 2>) : fn(&mmk::layer_norm<F32, 4>);
}
template <bool F32>
const void* layer_norm_grad_kernel(int vpt, int threads) {
  if (threads <= 512)
    return vpt == 1 ? fn(&mmk::layer_norm_grad<F32, 1, true>) : fn(&mmk::layer_norm_grad<F32, 2, true>);
  return fn(&mmk::layer_norm_grad<F32, 2, false>);
}
template <bool F32>
const void* layer_norm_grad_few_kernel(int vpt) {
  return vpt == 1   ? fn(&mmk::layer_norm_grad_few<F32, 1>)
         : vpt == 2 ? fn(&mmk::layer_norm_grad_few<F32, 2>)
                    : fn(&mmk::layer_norm_grad_few<F32, 4>);
}

// Rows whose gradient is one launch, as of the RMS norm.  Measured (us, one launch / two,
// bf16): 256 x 4096 4.5 / 12.3, 1024 x 4096 11.9 / 18.5, 2048 x 1024 12.9 / 16.4, 2048 x 4096
// 20.1 / 21.3, 2048 x 8192 28.8 / 37.1, 4096 x 4096 37.2 / 31.6.
bool layer_norm_few(int64_t rows, int64_t hidden) { return rows <= kFewRows || hidden > kLongRow; }

// ----------------------------------------------------------------------------
// Linear layer with an adapter per row
// ----------------------------------------------------------------------------
// At most this many rows take the rows' kernel (us a call, so / as tiles: 64 x 14336 x 4096, rank 64
// 46.1 / 56.3, 64 x 4096 x 4096 21.4 / 27.6, 64 x 1024 x 14336 23.4 / 29.3, 33 x 3001 x 1032 17.8 / 21.8, 48 x 28672 x 8192 with as
// many adapters 129 / 137, 64 x 8192 x 8192 54.4 / 56.9; the kernel's registers hold no more).
constexpr int64_t kLoraRows = 64;

int64_t round256(int64_t n) { return cdiv(n, 256) * 256; }

struct LoraPlan {
  int mb = 0;  // blocks of 16 rows of the rows' kernel (0: tiles)
  int spw = 0;  // its steps of 64 k per wave
  int64_t slices = 1;  // of K
  bool finish = false;  // the rows' kernel writes the output
  int low_mb = 0, low_rb = 0, turns = 0;  // the adapters' first product: blocks of 16 rows, of ranks, adapters at once
  int64_t low_slices = 1, low_k = 0;  // of K there
  Q8Plan tiles;  // (mb == 0)
  int64_t low = 0, v = 0, acc = 0, tile_rows = 0;  // workspace bytes
  int64_t bytes() const { return low + v + acc + tile_rows; }
};

// The tiles of many rows: as of the 8-bit product of the same bytes, whose super-steps
// these equal.
Q8Plan lora_tile_plan(int64_t M, int64_t N, int64_t K) { return q8_plan(M, N, 2 * K, kQ8MaxChunks); }

LoraPlan lora_plan(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L) {
  LoraPlan p;
  // A x: enough workgroups to draw on every CU, K in slices of 512 or more.  Decode rows
  // may each have an adapter of their own; of prompts a block of rows has one or two.
  // Measured (us, prompts, blocks of 32 rows in 4 slices / of 64 in 256 workgroups): 2047 x 4104,
  // rank 32 10.8 / 13.0, 8192 x 8192, rank 16 42 / 44.  Slices of K (us a call of 256 columns, in 1 / 2 / 4 / 8, the rule's
  // number): 300 x 4096, rank 16 24.9 / 23.2 / 22.4 / 22.5, 8; 700 x 12288 40.0 / 34.1 / 31.0 / 31.6, 11; 1500 x 4096 28.7 / 27.4 / 28.3 /
  // 29.6, 5; 1500 x 8192, rank 128 64.7 / 52.8 / 55.3 / 61.2, 4; 6000 x 2048, rank 128 72.7 / 79.3 / 104 / 126, 1; 16000 x 4096, rank 16
  // 74.5 / 72.8 / 81.2 / 89.1, 2; farthest from the best 1500 x 2048, rank 64 27.2 / 29.1 / 32.7 / 35.2, 4.
  p.low_mb = M <= 16 ? 1 : M <= 32 || M > 64 ? 2 : 4;
  p.low_rb = M > 64 && R > 16 ? 2 : 1;
  p.turns = M <= 64 ? (int)std::min(M, L) : (int)std::min<int64_t>(2, L);
  const int64_t at_once = cdiv(M, 16 * p.low_mb) * cdiv(R, 16 * p.low_rb) * (M <= 64 ? p.turns : 1);
  const int64_t want = M <= 64 ? std::min<int64_t>(16, cdiv(512, at_once))
                               : std::max<int64_t>({1, std::min<int64_t>(4, 1024 / at_once), std::min<int64_t>(16, 256 / at_once)});
  p.low_k = std::max<int64_t>(512, cdiv(cdiv(K, want), 64) * 64);
  p.low_slices = cdiv(K, p.low_k);
  p.low = round256(p.low_slices * M * R * 4);
  p.v = round256(M * 3 * R * 2);
  if (M <= kLoraRows) {
    p.mb = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    const int64_t steps = cdiv(K, 64), most = 8 / p.mb;
    p.slices = cdiv(steps, mmk::kLoraWaves * most);
    p.spw = 2;
    while (mmk::kLoraWaves * p.spw * p.slices < steps) p.spw *= 2;
    p.finish = p.slices == 1 && p.mb < 4;
    if (!p.finish) p.acc = round256(p.slices * M * N * 4);
    return p;
  }
  p.tiles = lora_tile_plan(M, N, K);
  p.tile_rows = p.tiles.chunks == 1 ? round256(p.tiles.tiles_m * (int64_t)sizeof(mmk::LoraTileRows)) : 0;
  if (p.tiles.chunks > 1) p.acc = round256(p.tiles.chunks * M * N * 4);
  return p;
}

template <int FM, int FN, int SX, int SW>
const void* lora_tile_kernel(bool split) {
  return split ? fn(&mmk::lora_tile<FM, FN, SX, SW, true>) : fn(&mmk::lora_tile<FM, FN, SX, SW, false>);
}
const void* lora_tile_kernel(int kind, bool split) {
  switch (kind) {
    case 0: return lora_tile_kernel<4, 4, 3, 2>(split);
    case 1: return lora_tile_kernel<4, 2, 3, 4>(split);
    case 2: return lora_tile_kernel<2, 2, 3, 2>(split);
    case 3: return lora_tile_kernel<2, 2, 5, 5>(split);
  }
  return lora_tile_kernel<2, 1, 6, 6>(split);
}

const void* lora_rows_kernel(int mb, int spw, bool finish) {
  // (K in slices: as many steps as the registers hold)
  if (!finish)
    return mb == 1   ? fn(&mmk::lora_rows<1, 8, false>)
           : mb == 2 ? fn(&mmk::lora_rows<2, 4, false>)
                     : fn(&mmk::lora_rows<4, 2, false>);
  if (mb == 2) return spw == 2 ? fn(&mmk::lora_rows<2, 2, true>) : fn(&mmk::lora_rows<2, 4, true>);
  return spw == 2   ? fn(&mmk::lora_rows<1, 2, true>)
         : spw == 4 ? fn(&mmk::lora_rows<1, 4, true>)
                    : fn(&mmk::lora_rows<1, 8, true>);
}

mm_status check_lora(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L) {
  if (M < 0 || N < 0 || K < 0 || R < 0 || L < 0) return fail(MM_ERR_INVALID_VALUE, "negative size");
  if (M >= kLimit || N >= kLimit || K >= kLimit || L >= kLimit)
    return fail(MM_ERR_UNSUPPORTED, "M, N, K and the number of adapters must be below 2^31");
  if (R > mmk::kLoraMaxRank) return fail(MM_ERR_UNSUPPORTED, "rank must be at most 256");
  if (R % 8 != 0) return fail(MM_ERR_MISALIGNED, "rank must be a multiple of 8");
  if (K % 8 != 0) return fail(MM_ERR_MISALIGNED, "K must be a multiple of 8 elements");
  if (K >= (int64_t(1) << 22)) return fail(MM_ERR_UNSUPPORTED, "K must be below 2^22");
  if (N > (int64_t(1) << 27) - 16) return fail(MM_ERR_UNSUPPORTED, "N must be at most 2^27 - 16");
  // (blocks of 32 rows of A x along a grid's y; without adapters' terms there is none)
  if (M > 32 * kMaxGridY && K > 0 && R > 0 && L > 0) return fail(MM_ERR_UNSUPPORTED, "M must be at most 2^21 - 32");
  const int64_t room = int64_t(1) << 60;
  if (M > 0 && (N > room / M || K > room / M)) return fail(MM_ERR_UNSUPPORTED, "an operand spans 2^60 elements or more");
  if (L * R > 0 && (N > room / (L * R) || K > room / (L * R)))
    return fail(MM_ERR_UNSUPPORTED, "an operand spans 2^60 elements or more");
  return MM_OK;
}

// ----------------------------------------------------------------------------
// Mixture of experts
// ----------------------------------------------------------------------------
constexpr int64_t kMoeMaxWidth = int64_t(1) << 18;
constexpr int64_t kMoeTableBytes = (sizeof(mmk::MoeTables) + 255) / 256 * 256;

mm_status check_moe(int64_t T, int64_t E, int64_t H, int64_t I, int64_t k) {
  if (T < 0 || E < 0 || H < 0 || I < 0 || k < 0) return fail(MM_ERR_INVALID_VALUE, "negative size");
  if (k > E) return fail(MM_ERR_INVALID_VALUE, "top_k must not be larger than the number of experts");
  if (T > mmk::kMoeTokens) return fail(MM_ERR_UNSUPPORTED, "at most 64 tokens");
  if (E > mmk::kMoeExperts) return fail(MM_ERR_UNSUPPORTED, "at most 512 experts");
  if (k > mmk::kMoeTopK) return fail(MM_ERR_UNSUPPORTED, "top_k must be at most 16");
  if (H > kMoeMaxWidth || I > kMoeMaxWidth) return fail(MM_ERR_UNSUPPORTED, "H and I must be at most 2^18");
  if (H % 8 != 0 || I % 8 != 0) return fail(MM_ERR_MISALIGNED, "H and I must be multiples of 8 elements");
  return MM_OK;
}

const void* moe_route_kernel(int64_t E) {
  return E <= 64    ? fn(&mmk::moe_route<1>)
         : E <= 128 ? fn(&mmk::moe_route<2>)
         : E <= 256 ? fn(&mmk::moe_route<4>)
                    : fn(&mmk::moe_route<8>);
}
const void* moe_gate_up_kernel(int64_t E) {
  return E <= 64    ? fn(&mmk::moe_gate_up<1>)
         : E <= 128 ? fn(&mmk::moe_gate_up<2>)
         : E <= 256 ? fn(&mmk::moe_gate_up<4>)
                    : fn(&mmk::moe_gate_up<8>);
}

// Blocks of 16 tokens to a group there: two where an expert has 14 on the average and the
// registers hold two.  Measured (us a call, one / two; tokens, choices of experts, H x I): 16 to an expert, 64, 2 of 8,
// 4096 x 4096 203 / 178 and 64, 4 of 16, 2048 x 1024 80 / 66; 14.2, 64, 2 of 9, 4096 x 4096 220 / 198; 14, 64, 7 of 32, 2048 x 2048
// 209 / 195; but 13.3, 40, 1 of 3, 4096 x 4096 75 / 79; 12, 64, 6 of 32, 2568 x 1544 202 / 215 (of 4096 x 2048 341 / 330); 8, 64,
// 1 of 8, 4096 x 4096 160 / 171.
int moe_group_blocks(int64_t T, int64_t E, int64_t H, int64_t k) { return T * k >= 14 * E && H <= 4096 ? 2 : 1; }

// Workgroups that share 16 columns of the second layer: the number that spreads the
// columns' workgroups most evenly over the CUs, a further one for a twentieth (256 CUs: 516 workgroups
// of a layer took 66 us, 512 of them 50).
int64_t moe_splits(int64_t H) {
  const int64_t blocks = cdiv(H, 16);
  int64_t best = 1;
  double least = 0.0;
  for (int64_t s = 1; s <= 8; ++s) {
    const double c = (double)cdiv(blocks * s, 256) / (double)s * (1.0 + 0.02 * (double)(s - 1)) + (s > 1 ? 0.05 : 0.0);
    if (s == 1 || c < least) least = c, best = s;
  }
  return best;
}

// Whether experts of several tokens go to the kernels that hold the tokens' rows.  These read the rows once per
// run of columns, not for every 8 or 16 of them, but take H and I in pieces of 1024 or 2048 and a launch more.
// Measured (us a call, without / with; tokens, choices of experts, H x I), at 4 tokens to an expert and more:
//   wide: 16, 2 of 8, 4096 x 14336 505 / 456; 48, 4 of 32, 4096 x 2048 331 / 305; 64, 4 of 32, 8192 x 2048 621 / 592; but of
//     8192 x 1024 322 / 349
//   12 to an expert: 64, 6 of 32, 2048 x 2048 223 / 189; 64, 4 of 16, 4096 x 768 104 / 88; but 3 of 16 88 / 96
//   rows that start inside a line: 61, 4 of 60, 2056 x 1416 273 / 251; 64, 4 of 32 186 / 152; 33, 4 of 16 103 / 85; 17, 4 of 16
//     88 / 82; 64, 4 of 40, 2600 x 1800 322 / 265; 64, 6 of 64, 4104 x 1544 627 / 523; 64, 4 of 64, 4104 x 1032 392 / 370 and
//     1416 x 2056 311 / 306; 20, 4 of 12, 2056 x 1032 64 / 60; but with I below 1024 64, 8 of 128, 4104 x 776 578 / 592
//   others, about even: 61, 4 of 60, 2048 x 1408 221 / 219; 64, 4 of 40, 2560 x 1792 250 / 243; 32, 4 of 32, 2048 x 1408 124 / 130;
//     64, 4 of 64, 4096 x 1024 325 / 337 and 4096 x 768 252 / 280
// and below 4 to an expert: 64, 3 of 64, 2056 x 2056 365 / 382; 64, 3 of 64, 4096 x 2048 545 / 542; 32, 2 of 32, 4096 x 4096 491 / 513.
bool moe_many(int64_t T, int64_t E, int64_t H, int64_t I, int64_t k) {
  if (T <= mmk::kMoeFew || H > 8192 || T * k < 4 * E) return false;
  if (H * I >= (int64_t(1) << 23)) return true;
  return H * I >= (int64_t(1) << 21) && (T * k >= 12 * E || ((H % 64 != 0 || I % 64 != 0) && I >= 1024));
}

struct MoePlan {
  bool many = false;
  int gb = 1;  // blocks of 16 tokens to a group
  int up_spw = 0, down_spw = 0;  // steps per wave (down: the three parts of x in 48 registers)
  int64_t splits = 1, slices = 1;
  int64_t mid = 0, part = 0;  // workspace bytes, after the tables
  int64_t bytes() const { return kMoeTableBytes + mid + part; }
};

int moe_steps(int64_t n, int most) {
  int spw = 2;
  while (spw < most && mmk::kMoeManyWaves * 64 * spw < n) spw *= 2;
  return spw;
}

MoePlan moe_plan(int64_t T, int64_t E, int64_t H, int64_t I, int64_t k) {
  MoePlan p;
  p.mid = round256(T * k * I * 6);
  p.many = moe_many(T, E, H, I, k);
  if (p.many) {
    p.gb = moe_group_blocks(T, E, H, k);
    p.up_spw = moe_steps(H, 8 / p.gb);
    p.down_spw = 2 / p.gb;
    p.slices = cdiv(I, mmk::kMoeManyWaves * 64 * p.down_spw);
    p.part = round256(p.slices * T * k * H * 4);
  } else {
    p.splits = H > 0 ? moe_splits(H) : 1;
    p.part = p.splits > 1 ? round256(p.splits * T * H * 4) : 0;
  }
  return p;
}

const void* moe_gate_up_many_kernel(int gb, int spw) {
  if (gb == 2) return spw == 2 ? fn(&mmk::moe_gate_up_many<2, 2>) : fn(&mmk::moe_gate_up_many<2, 4>);
  return spw == 2   ? fn(&mmk::moe_gate_up_many<1, 2>)
         : spw == 4 ? fn(&mmk::moe_gate_up_many<1, 4>)
                    : fn(&mmk::moe_gate_up_many<1, 8>);
}
const void* moe_down_many_kernel(int gb) {
  return gb == 2 ? fn(&mmk::moe_down_many<2, 1>) : fn(&mmk::moe_down_many<1, 2>);
}

}  // namespace

extern "C" {

mm_status mm_rms_norm(const void* x, int64_t ld_x, const void* residual, const void* weight, void* h, void* y,
                      float* rstd, int64_t rows, int64_t hidden, float eps, mm_out_dtype stream_dtype, void* stream) {
  return norm(x, ld_x, residual, weight, h, y, rstd, rows, hidden, eps, stream_dtype, false, stream);
}

mm_status mm_rms_norm_q8(const void* x, int64_t ld_x, const void* residual, const void* weight, void* h, void* q,
                         float* scale, int64_t rows, int64_t hidden, float eps, mm_out_dtype stream_dtype,
                         void* stream) {
  return norm(x, ld_x, residual, weight, h, q, scale, rows, hidden, eps, stream_dtype, true, stream);
}

mm_status mm_rms_norm_backward_workspace_size(int64_t rows, int64_t hidden, int64_t* bytes) {
  if (!bytes) return fail(MM_ERR_INVALID_VALUE, "null bytes pointer");
  *bytes = 0;
  mm_status s = check_norm_sizes(rows, hidden, MM_OUT_BF16);
  if (s != MM_OK || rows == 0 || hidden == 0) return s;
  if (rows <= kFewRows) return MM_OK;
  int64_t parts = 0;
  if ((s = norm_grad_parts(rows, hidden, &parts)) != MM_OK) return s;
  *bytes = parts * hidden * 4;
  return MM_OK;
}

mm_status mm_rms_norm_backward(const void* dy, const void* h, const void* weight, const float* rstd, const void* dres,
                               void* dh, float* dweight, int64_t rows, int64_t hidden, mm_out_dtype stream_dtype,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  mm_status s = check_norm_sizes(rows, hidden, stream_dtype);
  if (s != MM_OK) return s;
  if (hidden == 0) return MM_OK;
  const bool few = rows <= kFewRows || (hidden > kLongRow && stream_dtype == MM_OUT_BF16);
  if (!dweight || (rows > 0 && (!dy || !h || !weight || !rstd || !dh || (!few && !workspace))))
    return fail(MM_ERR_INVALID_VALUE, "null pointer");
  if (!aligned(dweight, 16) || (rows > 0 && (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) ||
                                             !aligned(rstd, 4) || !aligned(dres, 16) || !aligned(dh, 16) ||
                                             !aligned(workspace, 16))))
    return fail(MM_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  const int64_t e = stream_dtype == MM_OUT_F32 ? 4 : 2, n = rows * hidden;
  if (workspace_bytes < 0) return fail(MM_ERR_INVALID_VALUE, "negative workspace size");
  if (rows > 0) {
    const struct { const void* p; int64_t n; } in[] = {{dy, n * 2}, {h, n * e}, {dres, n * e}, {weight, hidden * 2},
                                                       {rstd, rows * 4}};
    const struct { const void* p; int64_t n; } out[] = {{dh, n * e}, {dweight, hidden * 4},
                                                        {workspace, workspace_bytes}};
    for (int o = 0; o < 3; ++o) {
      for (int i = 0; i < 5; ++i) {
        if (o == 0 && i == 2 && dh == dres) continue;  // in place: read before written, by one thread
        if (overlaps(out[o].p, out[o].n, in[i].p, in[i].n))
          return fail(MM_ERR_INVALID_VALUE, "an output or the workspace overlaps an input");
      }
      for (int q = 0; q < o; ++q)
        if (overlaps(out[o].p, out[o].n, out[q].p, out[q].n))
          return fail(MM_ERR_INVALID_VALUE, "outputs or the workspace overlap");
    }
  }
  int64_t parts = 0;
  if (rows > 0) {
    if (!few && (s = norm_grad_parts(rows, hidden, &parts)) != MM_OK) return s;
    if (workspace_bytes < parts * hidden * 4)
      return fail(MM_ERR_INVALID_VALUE, "workspace smaller than mm_rms_norm_backward_workspace_size reports");
    mmk::RmsNormGradParams p;
    p.dy = static_cast<const uint16_t*>(dy);
    p.h = h;
    p.dres = dres;
    p.weight = static_cast<const uint16_t*>(weight);
    p.rstd = rstd;
    p.dh = dh;
    p.part = static_cast<float*>(workspace);
    p.rows = rows;
    p.hidden = (int)hidden;
    int threads, vpt;
    norm_shape(hidden, 512, &threads, &vpt);
    if (few) {
      threads = std::max(threads, 512);  // (for the columns' sums)
      void* args[] = {&p, &dweight};
      return launch(stream_dtype == MM_OUT_F32 ? norm_grad_few_kernel<true>(vpt) : norm_grad_few_kernel<false>(vpt),
                    dim3((unsigned)(rows + cdiv(hidden, 64))), threads, args, stream, "rms_norm gradient");
    }
    if (vpt == 4) norm_shape(hidden, 1024, &threads, &vpt);
    void* args[] = {&p};
    s = launch(stream_dtype == MM_OUT_F32 ? norm_grad_kernel<true>(vpt, threads) : norm_grad_kernel<false>(vpt, threads),
               dim3((unsigned)parts), threads, args, stream, "rms_norm gradient");
    if (s != MM_OK) return s;
  }
  const float* part = static_cast<const float*>(workspace);
  int nparts = (int)parts, hid = (int)hidden;
  void* args[] = {&part, &dweight, &nparts, &hid};
  return launch(fn(&mmk::rms_norm_dweight), dim3((unsigned)cdiv(hidden, 32)), 256, args, stream,
                "rms_norm weight gradient");
}

mm_status mm_w4_pack(const void* codes, void* packed, int64_t N, int64_t K, void* stream) {
  if (N < 0 || K < 0) return fail(MM_ERR_INVALID_VALUE, "negative size");
  if (N >= kLimit || K >= kLimit) return fail(MM_ERR_UNSUPPORTED, "N and K must be below 2^31");
  if (N == 0 || K == 0) return MM_OK;
  if (!codes || !packed) return fail(MM_ERR_INVALID_VALUE, "null pointer");
  if (!aligned(packed, 16)) return fail(MM_ERR_MISALIGNED, "packed must be 16-byte aligned");
  const int64_t words = cdiv(N, 16) * cdiv(K, 128) * 256;
  if (overlaps(packed, words * 4, codes, N * K)) return fail(MM_ERR_INVALID_VALUE, "packed overlaps codes");
  const uint8_t* c = static_cast<const uint8_t*>(codes);
  uint32_t* w = static_cast<uint32_t*>(packed);
  int n = (int)N, k = (int)K;
  const int64_t most = kMaxThreads / 256 * 256;
  for (int64_t first = 0; first < words; first += most) {
    void* args[] = {&c, &w, &n, &k, &first};
    const mm_status s = launch(fn(&mmk::w4_pack), dim3((unsigned)(std::min(words - first, most) / 256)), 256, args, stream,
                               "w4_pack");
    if (s != MM_OK) return s;
  }
  return MM_OK;
}

mm_status mm_linear_w4(const void* x, const void* W, const void* scales, const void* zeros, const void* bias,
                       void* out, int64_t M, int64_t N, int64_t K, int64_t group, mm_epilogue epilogue, void* stream) {
  int epi = 0;
  mm_status s = check_product(M, N, K, bias, out, epilogue, &epi);
  if (s != MM_OK) return s;
  if (group != 32 && group != 64 && group != 128)
    return fail(MM_ERR_UNSUPPORTED, "group must be 32, 64 or 128");
  if (M == 0 || N == 0) return MM_OK;
  if (K > 0) {
    if (!x || !W || !scales) return fail(MM_ERR_INVALID_VALUE, "null operand pointer");
    if (!aligned(x, 16) || !aligned(W, 16)) return fail(MM_ERR_MISALIGNED, "x and W must be 16-byte aligned");
    if (!aligned(scales, 2)) return fail(MM_ERR_MISALIGNED, "scales must be 2-byte aligned");
    if (K % 8 != 0) return fail(MM_ERR_MISALIGNED, "K must be a multiple of 8 elements");
    if (K > (int64_t(1) << 22)) return fail(MM_ERR_UNSUPPORTED, "K must be at most 2^22");
    const int64_t ob = M * N * 2, groups = cdiv(K, group);
    if (overlaps(out, ob, x, M * K * 2) || overlaps(out, ob, W, cdiv(N, 16) * cdiv(K, 128) * 1024) ||
        overlaps(out, ob, scales, groups * N * 2) || overlaps(out, ob, zeros, groups * N))
      return fail(MM_ERR_INVALID_VALUE, "out overlaps an input");
  }
  mmk::W4Params p;
  p.W = static_cast<const mmk::u32x4*>(W);
  p.scales = static_cast<const uint16_t*>(scales);
  p.zeros = static_cast<const uint8_t*>(zeros);
  p.bias = static_cast<const uint16_t*>(bias);
  p.N = (int)N;
  p.K = (int)K;
  p.group = (int)group;
  p.epi = epi;
  void* args[] = {&p};
  // rows m0 .. m0 + m - 1
  auto part = [&](int64_t m0, int64_t m) {
    p.x = static_cast<const uint16_t*>(x) + m0 * K;
    p.out = static_cast<uint16_t*>(out) + m0 * N;
    p.M = (int)m;
  };
  if (N < 4) {
    const int64_t most = int64_t(1) << 30;
    for (int64_t m0 = 0; m0 < M; m0 += most) {
      part(m0, std::min(M - m0, most));
      s = launch(fn(&mmk::gemm_w4_narrow), dim3((unsigned)cdiv(p.M * N, 64)), 64, args, stream, "linear_w4 narrow");
      if (s != MM_OK) return s;
    }
    return MM_OK;
  }
  const int xr = M <= 4 ? 4 : M <= 16 ? 16 : M <= 32 ? 32 : M <= 48 ? 48 : 64;
  // Measured (us, 1 / 2 / 4 column blocks): 1 x 4096 x 4096 4.1 / 5.1 / 6.7, 12 x
  // 6000 x 4096 8.7 / 6.6 / 8.7, 24 x 8192 x 8192 23.8 / 16.7 / 18.7, 10 x 11000 x
  // 4096 12.7 / 11.8 / 10.4, 64 x 14336 x 4096 39 / 26 / 20.
  const int64_t blocks = cdiv(N, 16);
  if (cdiv(blocks, 4) > kMaxRowsGridX) return fail(MM_ERR_UNSUPPORTED, "N must be at most 2^29 - 64");
  int cus = 0;
  if ((s = device_cus(&cus)) != MM_OK) return s;
  const int nb = column_blocks(blocks, cdiv(M, xr), cus, 10);
  for (int64_t m0 = 0; m0 < M; m0 += kMaxGridY * xr) {
    part(m0, std::min(M - m0, kMaxGridY * xr));
    s = launch(w4_kernel(xr, nb, (int)group), dim3((unsigned)cdiv(blocks, nb), (unsigned)cdiv(p.M, xr)),
               mmk::kW4Waves * 64, args, stream, "linear_w4");
    if (s != MM_OK) return s;
  }
  return MM_OK;
}

mm_status mm_linear_q8_workspace_size(int64_t M, int64_t N, int64_t K, int64_t* bytes) {
  if (!bytes) return fail(MM_ERR_INVALID_VALUE, "null bytes pointer");
  *bytes = 0;
  if (M < 0 || N < 0 || K < 0) return fail(MM_ERR_INVALID_VALUE, "negative size");
  if (M >= kLimit || N >= kLimit || K >= kLimit) return fail(MM_ERR_UNSUPPORTED, "M, N and K must be below 2^31");
  if (M > kQ8Rows && N > 0 && K > 0) *bytes = q8_ws_bytes(q8_plan(M, N, K, kQ8MaxChunks));
  return MM_OK;
}

mm_status mm_linear_q8(const void* x, const float* x_scale, const void* W, const float* w_scale, const void* bias,
                       void* out, int64_t M, int64_t N, int64_t K, mm_epilogue epilogue, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  int epi = 0;
  mm_status s = check_product(M, N, K, bias, out, epilogue, &epi);
  if (s != MM_OK) return s;
  if (M == 0 || N == 0) return MM_OK;
  if (!x_scale || !w_scale) return fail(MM_ERR_INVALID_VALUE, "null scale pointer");
  if (!aligned(x_scale, 4) || !aligned(w_scale, 4)) return fail(MM_ERR_MISALIGNED, "scales must be 4-byte aligned");
  const int64_t ob = M * N * 2;
  if (overlaps(out, ob, x_scale, M * 4) || overlaps(out, ob, w_scale, N * 4))
    return fail(MM_ERR_INVALID_VALUE, "out overlaps an input");
  if (K > 0) {
    if (!x || !W) return fail(MM_ERR_INVALID_VALUE, "null operand pointer");
    if (!aligned(x, 16) || !aligned(W, 16)) return fail(MM_ERR_MISALIGNED, "x and W must be 16-byte aligned");
    if (K % 16 != 0) return fail(MM_ERR_MISALIGNED, "K must be a multiple of 16 elements");
    if (K > (int64_t(1) << 22)) return fail(MM_ERR_UNSUPPORTED, "K must be at most 2^22");
    if (overlaps(out, ob, x, M * K) || overlaps(out, ob, W, N * K))
      return fail(MM_ERR_INVALID_VALUE, "out overlaps an input");
  }
  if (workspace_bytes < 0) return fail(MM_ERR_INVALID_VALUE, "negative workspace size");
  if (overlaps(workspace, workspace_bytes, out, ob) || overlaps(workspace, workspace_bytes, x, M * K) ||
      overlaps(workspace, workspace_bytes, W, N * K) || overlaps(workspace, workspace_bytes, x_scale, M * 4) ||
      overlaps(workspace, workspace_bytes, w_scale, N * 4) || overlaps(workspace, workspace_bytes, bias, N * 2))
    return fail(MM_ERR_INVALID_VALUE, "workspace overlaps an operand or the output");
  mmk::Q8Params p;
  p.x = static_cast<const uint8_t*>(x);
  p.xs = x_scale;
  p.W = static_cast<const uint8_t*>(W);
  p.ws = w_scale;
  p.bias = static_cast<const uint16_t*>(bias);
  p.out = static_cast<uint16_t*>(out);
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.epi = epi;
  void* args[] = {&p};
  // (33 to 64 rows by a wide weight: in the rows' kernel every 64 columns read the
  // activations again; 64 x 28672 x 8192 68 us there, 59 as tiles, 60 x 11000 x 4096
  // 20.2 and 19.3, 60 x 6000 x 4096 13.6 and 16.6)
  if (M <= 32 || (M <= kQ8Rows && N < 11000) || K == 0) {
    const int xr = M <= 4 ? 4 : M <= 16 ? 16 : M <= 32 ? 32 : 64;
    const int64_t blocks = cdiv(N, 16);
    if (cdiv(blocks, 4) > kMaxRowsGridX) return fail(MM_ERR_UNSUPPORTED, "N must be at most 2^29 - 64");
    // Few rows with at most two workgroups to a CU: one column block streams W
    // best (us, 1 / 2 / 4 blocks: 16 x 8192 x 8192 13.9 / 16.2 / 20.0, though 12 x
    // 6000 x 4096 9.3 / 8.6 / 12.6).  Otherwise by the shares of the CUs: 1 x 28672 x
    // 8192 41.9 / 51.9 / 48.8, 16 x 14336 x 4096 15.1 / 14.4 / 13.6, 12 x 20000 x 8192
    // 37.5 / 38.7 / 46.8, 24 x 20000 x 8192 47.0 / 42.6 / 50.0, 64 x 8192 x 8192
    // 23.2 / 18.2 / 25.2, 32 x 28672 x 8192 69.8 / 60.6 / 57.2.
    int cus = 0;
    if ((s = device_cus(&cus)) != MM_OK) return s;
    const int nb = M <= 16 && blocks <= 2 * cus ? 1 : column_blocks(blocks, cdiv(M, xr), cus, M <= 4 ? 1 : M <= 16 ? 3 : 10);
    for (int64_t m0 = 0; m0 < M; m0 += kMaxGridY * xr) {  // (more than one turn only with K == 0)
      p.x = static_cast<const uint8_t*>(x) + m0 * K;
      p.xs = x_scale + m0;
      p.out = static_cast<uint16_t*>(out) + m0 * N;
      p.M = (int)std::min(M - m0, kMaxGridY * xr);
      s = launch(q8_rows_kernel(xr, nb), dim3((unsigned)cdiv(blocks, nb), (unsigned)cdiv(p.M, xr)), mmk::kW4Waves * 64,
                 args, stream, "linear_q8 rows");
      if (s != MM_OK) return s;
    }
    return MM_OK;
  }
  const Q8Plan plan = q8_plan(M, N, K, workspace && M > kQ8Rows ? kQ8MaxChunks : 1);
  if (plan.tiles_m * plan.tiles_n * plan.chunks >= kLimit) return fail(MM_ERR_UNSUPPORTED, "more than 2^31 output tiles");
  const int64_t need = q8_ws_bytes(plan);
  if (need > 0) {
    if (workspace_bytes < need)
      return fail(MM_ERR_INVALID_VALUE, "workspace smaller than mm_linear_q8_workspace_size reports");
    if (!aligned(workspace, 16)) return fail(MM_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  }
  p.tiles_m = (int)plan.tiles_m;
  p.tiles_n = (int)plan.tiles_n;
  p.chunks = (int)plan.chunks;
  p.chunk_steps = (int)plan.chunk_steps;
  p.part = static_cast<float*>(workspace);
  int cus = 0;
  if ((s = device_cus(&cus)) != MM_OK) return s;
  const int64_t units = plan.tiles_m * plan.tiles_n * plan.chunks;
  const int64_t grid = std::min<int64_t>(units, (int64_t)cus * kQ8Kinds[plan.kind].resident);
  const bool split = plan.chunks > 1;
  s = launch(q8_tile_kernel(plan.kind, split),
             dim3((unsigned)grid), 256, args, stream, "linear_q8 tiles");
  if (s != MM_OK || !split) return s;
  const int64_t blocks = plan.tiles_m * plan.tiles_n * kQ8Kinds[plan.kind].fm * kQ8Kinds[plan.kind].fn;
  return launch(q8_join_kernel(plan.kind),
                dim3((unsigned)blocks), 256, args, stream, "linear_q8 join");
}

mm_status mm_layer_norm(const void* x, int64_t ld_x, const void* residual, const void* weight, const void* bias, void* h,
                        void* y, float* mean, float* rstd, int64_t rows, int64_t hidden, float eps,
                        mm_out_dtype stream_dtype, void* stream) {
  mm_status s = check_norm_sizes(rows, hidden, stream_dtype);
  if (s != MM_OK) return s;
  if (!(eps >= 0.0f)) return fail(MM_ERR_INVALID_VALUE, "eps must not be negative");
  if (rows == 0 || hidden == 0) return MM_OK;
  if (!x || !weight || !y || !mean || !rstd || (residual && !h)) return fail(MM_ERR_INVALID_VALUE, "null pointer");
  if (ld_x < hidden || ld_x >= kLimit) return fail(MM_ERR_INVALID_VALUE, "rows of x must not overlap (ld_x < hidden)");
  if (ld_x % 8 != 0) return fail(MM_ERR_MISALIGNED, "ld_x must be a multiple of 8 elements");
  if (!residual) h = nullptr;
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(h, 16) ||
      !aligned(y, 16))
    return fail(MM_ERR_MISALIGNED, "x, residual, weight, bias, h and y must be 16-byte aligned");
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return fail(MM_ERR_MISALIGNED, "mean and rstd must be 4-byte aligned");
  const int64_t e = stream_dtype == MM_OUT_F32 ? 4 : 2;
  const int64_t xb = ((rows - 1) * ld_x + hidden) * e, hb = rows * hidden * e;
  // h may be residual itself, or x (a contiguous one): each element is read before it is
  // written, by one thread
  const bool over_residual = h && h == residual, over_x = h && h == x && ld_x == hidden;
  const Span in[] = {{x, xb}, {residual, hb}, {weight, hidden * 2}, {bias, hidden * 2}};
  const Span out[] = {{y, rows * hidden * 2}, {mean, rows * 4}, {rstd, rows * 4}};
  const Span h_in[] = {{over_x ? nullptr : x, xb}, {over_residual ? nullptr : residual, hb}, {weight, hidden * 2},
                       {bias, hidden * 2}, out[0], out[1], out[2]};
  const Span h_out[] = {{h, hb}};
  if (any_overlap(in, out) || any_overlap(h_in, h_out))
    return fail(MM_ERR_INVALID_VALUE, "an output overlaps an input or another output");
  mmk::LayerNormParams p;
  p.weight = static_cast<const uint16_t*>(weight);
  p.bias = static_cast<const uint16_t*>(bias);
  p.ld_x = ld_x;
  p.hidden = (int)hidden;
  p.eps = eps;
  int threads, vpt;
  norm_shape(hidden, 512, &threads, &vpt);
  const void* k = stream_dtype == MM_OUT_F32 ? layer_norm_kernel<true>(vpt) : layer_norm_kernel<false>(vpt);
  void* args[] = {&p};
  const int64_t most = kMaxThreads / threads;
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    p.x = static_cast<const char*>(x) + r0 * ld_x * e;
    p.residual = residual ? static_cast<const char*>(residual) + r0 * hidden * e : nullptr;
    p.h = residual ? static_cast<char*>(h) + r0 * hidden * e : nullptr;
    p.y = static_cast<uint16_t*>(y) + r0 * hidden;
    p.mean = mean + r0;
    p.rstd = rstd + r0;
    s = launch(k, dim3((unsigned)std::min(rows - r0, most)), threads, args, stream, "layer_norm");
    if (s != MM_OK) return s;
  }
  return MM_OK;
}

mm_status mm_layer_norm_backward_workspace_size(int64_t rows, int64_t hidden, int64_t* bytes) {
  if (!bytes) return fail(MM_ERR_INVALID_VALUE, "null bytes pointer");
  *bytes = 0;
  mm_status s = check_norm_sizes(rows, hidden, MM_OUT_BF16);
  if (s != MM_OK || rows == 0 || hidden == 0 || layer_norm_few(rows, hidden)) return s;
  int64_t parts = 0;
  if ((s = norm_grad_parts(rows, hidden, &parts)) != MM_OK) return s;
  *bytes = parts * hidden * 8;
  return MM_OK;
}

mm_status mm_layer_norm_backward(const void* dy, const void* h, const void* weight, const float* mean, const float* rstd,
                                 const void* dres, void* dh, float* dweight, float* dbias, int64_t rows, int64_t hidden,
                                 mm_out_dtype stream_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  mm_status s = check_norm_sizes(rows, hidden, stream_dtype);
  if (s != MM_OK) return s;
  if (hidden == 0) return MM_OK;
  const bool few = layer_norm_few(rows, hidden);
  if (!dweight || !dbias ||
      (rows > 0 && (!dy || !h || !weight || !mean || !rstd || !dh || (!few && !workspace))))
    return fail(MM_ERR_INVALID_VALUE, "null pointer");
  if (!aligned(dweight, 16) || !aligned(dbias, 16) ||
      (rows > 0 && (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(mean, 4) ||
                    !aligned(rstd, 4) || !aligned(dres, 16) || !aligned(dh, 16) || !aligned(workspace, 16))))
    return fail(MM_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  if (workspace_bytes < 0) return fail(MM_ERR_INVALID_VALUE, "negative workspace size");
  const int64_t e = stream_dtype == MM_OUT_F32 ? 4 : 2, n = rows * hidden;
  // (dh may be dres: read before written, by one thread)
  const Span in[] = {{dy, n * 2}, {h, n * e}, {weight, hidden * 2}, {mean, rows * 4}, {rstd, rows * 4}};
  const Span out[] = {{dh, n * e}, {dweight, hidden * 4}, {dbias, hidden * 4}, {workspace, workspace_bytes}};
  const Span dres_in[] = {{dres, n * e}};
  const Span dres_out[] = {{dh == dres ? nullptr : dh, n * e}, out[1], out[2], out[3]};
  if (any_overlap(in, out) || any_overlap(dres_in, dres_out))
    return fail(MM_ERR_INVALID_VALUE, "an output or the workspace overlaps an input or another output");
  int64_t parts = 0;
  if (rows > 0) {
    if (!few && (s = norm_grad_parts(rows, hidden, &parts)) != MM_OK) return s;
    if (workspace_bytes < parts * hidden * 8)
      return fail(MM_ERR_INVALID_VALUE, "workspace smaller than mm_layer_norm_backward_workspace_size reports");
    mmk::LayerNormGradParams p;
    p.dy = static_cast<const uint16_t*>(dy);
    p.h = h;
    p.dres = dres;
    p.weight = static_cast<const uint16_t*>(weight);
    p.mean = mean;
    p.rstd = rstd;
    p.dh = dh;
    p.part = static_cast<float*>(workspace);
    p.rows = rows;
    p.hidden = (int)hidden;
    int threads, vpt;
    norm_shape(hidden, 512, &threads, &vpt);
    if (few) {
      threads = std::max(threads, 512);  // (for the columns' sums)
      void* args[] = {&p, &dweight, &dbias};
      return launch(stream_dtype == MM_OUT_F32 ? layer_norm_grad_few_kernel<true>(vpt) : layer_norm_grad_few_kernel<false>(vpt),
                    dim3((unsigned)(rows + cdiv(hidden, 8 * mmk::grad_few_lanes(vpt)))), threads, args, stream,
                    "layer_norm gradient");
    }
    if (vpt == 4) norm_shape(hidden, 1024, &threads, &vpt);
    void* args[] = {&p};
    s = launch(stream_dtype == MM_OUT_F32 ? layer_norm_grad_kernel<true>(vpt, threads)
                                          : layer_norm_grad_kernel<false>(vpt, threads),
               dim3((unsigned)parts), threads, args, stream, "layer_norm gradient");
    if (s != MM_OK) return s;
  }
  const float* part = static_cast<const float*>(workspace);
  int nparts = (int)parts, hid = (int)hidden;
  void* args[] = {&part, &dweight, &dbias, &nparts, &hid};
  return launch(fn(&mmk::layer_norm_dparams), dim3((unsigned)cdiv(hidden, 32), 2), 256, args, stream,
                "layer_norm parameter gradients");
}

mm_status mm_linear_lora_workspace_size(int64_t M, int64_t N, int64_t K, int64_t rank, int64_t adapters, int64_t* bytes) {
  if (!bytes) return fail(MM_ERR_INVALID_VALUE, "null bytes pointer");
  *bytes = 0;
  mm_status s = check_lora(M, N, K, rank, adapters);
  if (s != MM_OK || M == 0 || N == 0 || K == 0 || rank == 0 || adapters == 0) return s;
  *bytes = lora_plan(M, N, K, rank, adapters).bytes();
  return MM_OK;
}

mm_status mm_linear_lora(const void* x, const void* W, const void* A, const void* B, const int32_t* index,
                         const float* scale, const void* bias, void* out, int64_t M, int64_t N, int64_t K, int64_t rank,
                         int64_t adapters, mm_epilogue epilogue, void* workspace, int64_t workspace_bytes, void* stream) {
  int epi = 0;
  mm_status s = check_product(M, N, K, bias, out, epilogue, &epi);
  if (s != MM_OK) return s;
  if ((s = check_lora(M, N, K, rank, adapters)) != MM_OK) return s;
  if (M == 0 || N == 0) return MM_OK;
  // (no terms of an adapter: the linear layer)
  if (K == 0 || rank == 0 || adapters == 0) return mm_linear(x, W, bias, out, M, N, K, MM_NT, epilogue, stream);
  if (!x || !W || !A || !B || !index || !scale) return fail(MM_ERR_INVALID_VALUE, "null operand pointer");
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(A, 16) || !aligned(B, 16))
    return fail(MM_ERR_MISALIGNED, "x, W, A and B must be 16-byte aligned");
  if (!aligned(index, 4) || !aligned(scale, 4)) return fail(MM_ERR_MISALIGNED, "index and scale must be 4-byte aligned");
  if (workspace_bytes < 0) return fail(MM_ERR_INVALID_VALUE, "negative workspace size");
  const Span in[] = {{x, M * K * 2},        {W, N * K * 2},     {A, adapters * rank * K * 2}, {B, adapters * N * rank * 2},
                     {index, M * 4},        {scale, adapters * 4}, {bias, bias ? N * 2 : 0}};
  const Span outs[] = {{out, M * N * 2}, {workspace, workspace_bytes}};
  if (any_overlap(in, outs)) return fail(MM_ERR_INVALID_VALUE, "out or the workspace overlaps an operand or each other");
  const LoraPlan plan = lora_plan(M, N, K, rank, adapters);
  if (!workspace || workspace_bytes < plan.bytes())
    return fail(MM_ERR_INVALID_VALUE, "workspace smaller than mm_linear_lora_workspace_size reports");
  if (!aligned(workspace, 256)) return fail(MM_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  mmk::LoraParams p;
  p.x = static_cast<const uint16_t*>(x);
  p.W = static_cast<const uint16_t*>(W);
  p.A = static_cast<const uint16_t*>(A);
  p.B = static_cast<const uint16_t*>(B);
  p.index = index;
  p.scale = scale;
  p.bias = static_cast<const uint16_t*>(bias);
  p.out = static_cast<uint16_t*>(out);
  char* ws = static_cast<char*>(workspace);
  p.low = reinterpret_cast<float*>(ws);
  p.v = reinterpret_cast<uint16_t*>(ws + plan.low);
  p.acc = reinterpret_cast<float*>(ws + plan.low + plan.v);
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.R = (int)rank;
  p.L = (int)adapters;
  p.slices = (int)plan.slices;
  p.epi = epi;
  p.low_slices = (int)plan.low_slices;
  p.low_k = (int)plan.low_k;
  void* args[] = {&p};
  const int64_t row_blocks = cdiv(M, 16 * plan.low_mb);
  int turns = plan.turns;
  void* shrink_args[] = {&p, &turns};
  s = launch(plan.low_mb == 1   ? fn(&mmk::lora_shrink<1, 1, false>)
             : plan.low_mb == 4 ? fn(&mmk::lora_shrink<4, 1, false>)
             : M <= 64          ? fn(&mmk::lora_shrink<2, 1, false>)
             : plan.low_rb == 1 ? fn(&mmk::lora_shrink<2, 1, true>)
                                : fn(&mmk::lora_shrink<2, 2, true>),
             dim3((unsigned)plan.low_slices, (unsigned)row_blocks, (unsigned)(cdiv(rank, 16 * plan.low_rb) * plan.turns)),
             mmk::kLoraShrinkWaves * 64, shrink_args, stream, "linear_lora shrink");
  if (s != MM_OK) return s;
  if (plan.mb) {
    int cus = 0;
    if ((s = device_cus(&cus)) != MM_OK) return s;
    const int64_t blocks = cdiv(N, 16), each = cdiv(blocks * plan.slices, cus);
    s = launch(lora_rows_kernel(plan.mb, plan.spw, plan.finish),
               dim3((unsigned)cdiv(blocks, each), (unsigned)plan.slices), mmk::kLoraWaves * 64, args, stream,
               "linear_lora rows");
    if (s != MM_OK || plan.finish) return s;
  } else {
    const Q8Plan& t = plan.tiles;
    const bool split = t.chunks > 1;
    p.tiles_m = (int)t.tiles_m;
    p.tiles_n = (int)t.tiles_n;
    p.slices = (int)t.chunks;
    p.slice_steps = (int)t.chunk_steps;
    mmk::LoraTileRows* rows = reinterpret_cast<mmk::LoraTileRows*>(ws + plan.low + plan.v + plan.acc);
    p.tiles = rows;
    int bm = split ? 0 : 64 * kQ8Kinds[t.kind].fm;
    void* fold_args[] = {&p, &rows, &bm};
    s = launch(fn(&mmk::lora_fold),
               dim3((unsigned)((split ? 0 : t.tiles_m) + std::min<int64_t>(cdiv(M * rank * 2, 256), 1024))), 256, fold_args,
               stream, "linear_lora fold");
    if (s != MM_OK) return s;
    int cus = 0;
    if ((s = device_cus(&cus)) != MM_OK) return s;
    const int64_t units = t.tiles_m * t.tiles_n * t.chunks;
    s = launch(lora_tile_kernel(t.kind, split),
               dim3((unsigned)std::min<int64_t>(units, (int64_t)cus * kQ8Kinds[t.kind].resident)), 256, args, stream,
               "linear_lora tiles");
    if (s != MM_OK || !split) return s;
  }
  // 33 to 64 rows: all to a workgroup, which reads B once, where B is much of what is read and the columns make
  // workgroups enough; else, and for fewer rows, blocks of 16 (us a call of 64 x N x 4096 with 8 adapters, so / in blocks of
  // 16: rank 64, N 14336 46.6 / 49.2, 28672 78.8 / 81.2, 11008 40.6 / 41.5, 8192 32.4 / 30.6; rank 128, N 11008 49.4 / 54.4, 8192
  // 42.2 / 39.2; rank 16, N 14336 42.2 / 42.3, 28672 72.0 / 69.8, and with 64 adapters 87.4 / 80.3).
  // More rows: 64 by 64 where that makes a workgroup for every CU (us a call of K 4096, so / in blocks of 16 rows:
  // 1000 x 1024 34.7 / 35.4, 512 x 4096 40.5 / 44.6; but 300 x 2000 37.5 / 34.9, 100 x 4096 34.8 / 30.8).
  const int64_t groups = cdiv(N, 64);
  if (!plan.mb && groups * cdiv(M, 64) >= 256)
    return launch(fn(&mmk::lora_join), dim3((unsigned)groups, (unsigned)cdiv(M, 64)), 256, args, stream, "linear_lora join");
  const int jb = plan.mb == 4 && rank >= 64 && N >= 10240 ? 4 : 1;
  return launch(jb == 1 ? fn(&mmk::lora_join_few<1>) : fn(&mmk::lora_join_few<4>),
                dim3((unsigned)groups, (unsigned)cdiv(M, 16 * jb)), 512, args, stream, "linear_lora join");
}

mm_status mm_moe_ffn_workspace_size(int64_t tokens, int64_t experts, int64_t H, int64_t I, int64_t top_k, int64_t* bytes) {
  if (!bytes) return fail(MM_ERR_INVALID_VALUE, "null bytes pointer");
  *bytes = 0;
  const mm_status s = check_moe(tokens, experts, H, I, top_k);
  if (s != MM_OK || tokens == 0) return s;
  *bytes = moe_plan(tokens, experts, H, I, top_k).bytes();
  return MM_OK;
}

mm_status mm_moe_ffn(const void* x, const float* logits, const void* W_gate, const void* W_up, const void* W_down,
                     void* out, int32_t* experts, float* weights, int64_t tokens, int64_t n_experts, int64_t H, int64_t I,
                     int64_t top_k, int renormalize, void* workspace, int64_t workspace_bytes, void* stream) {
  const int64_t T = tokens, E = n_experts;
  mm_status s = check_moe(T, E, H, I, top_k);
  if (s != MM_OK) return s;
  if (T == 0) return MM_OK;
  if ((H > 0 && !out) || (top_k > 0 && (!logits || !experts || !weights)) || (top_k > 0 && H > 0 && I > 0 &&
      (!x || !W_gate || !W_up || !W_down)))
    return fail(MM_ERR_INVALID_VALUE, "null pointer");
  if (!aligned(x, 16) || !aligned(W_gate, 16) || !aligned(W_up, 16) || !aligned(W_down, 16))
    return fail(MM_ERR_MISALIGNED, "x and the weights must be 16-byte aligned");
  if (!aligned(logits, 4) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(out, 2))
    return fail(MM_ERR_MISALIGNED, "logits, experts, weights and out must be aligned to their element size");
  if (workspace_bytes < 0) return fail(MM_ERR_INVALID_VALUE, "negative workspace size");
  const Span in[] = {{x, T * H * 2}, {logits, T * E * 4}, {W_gate, E * I * H * 2}, {W_up, E * I * H * 2},
                     {W_down, E * I * H * 2}};
  const Span outs[] = {{out, T * H * 2}, {experts, T * top_k * 4}, {weights, T * top_k * 4}, {workspace, workspace_bytes}};
  if (any_overlap(in, outs)) return fail(MM_ERR_INVALID_VALUE, "an output or the workspace overlaps an input or another output");
  const MoePlan plan = moe_plan(T, E, H, I, top_k);
  if (!workspace || workspace_bytes < plan.bytes())
    return fail(MM_ERR_INVALID_VALUE, "workspace smaller than mm_moe_ffn_workspace_size reports");
  if (!aligned(workspace, 256)) return fail(MM_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  mmk::MoeParams p;
  p.x = static_cast<const uint16_t*>(x);
  p.logits = logits;
  p.wg = static_cast<const uint16_t*>(W_gate);
  p.wu = static_cast<const uint16_t*>(W_up);
  p.wd = static_cast<const uint16_t*>(W_down);
  p.out = static_cast<uint16_t*>(out);
  p.experts = experts;
  p.weights = weights;
  char* ws = static_cast<char*>(workspace);
  p.tab = reinterpret_cast<mmk::MoeTables*>(ws);
  p.mid = reinterpret_cast<uint16_t*>(ws + kMoeTableBytes);
  p.part = reinterpret_cast<float*>(ws + kMoeTableBytes + plan.mid);
  p.T = (int)T;
  p.E = (int)E;
  p.H = (int)H;
  p.I = (int)I;
  p.k = (int)top_k;
  p.renormalize = renormalize != 0;
  p.splits = (int)plan.splits;
  p.slices = (int)plan.slices;
  void* args[] = {&p};
  // Few tokens: every workgroup of the first layer finds their experts itself (us a call, so / by a
  // launch before: one token, 2 of 8 experts of 4096 x 14336 124.8 / 127.8, 8, 2 of 8 of 512 x 512
  // 13.2 / 15.8, 8, 8 of 512 of 1024 x 512 53.5 / 58.8); a workgroup of eight waves has one token each.
  const int64_t units = T * top_k * (I / 8);  // (at most: a group for every choice)
  const bool own = T <= mmk::kMoeFew && units > 0 && H > 0;
  int group = 16 * plan.gb;
  void* route_args[] = {&p, &group};
  if (!own && (s = launch(moe_route_kernel(E), dim3(1), 1024, route_args, stream, "moe_ffn route")) != MM_OK) return s;
  if (H == 0) return MM_OK;
  int cus = 0;
  if ((s = device_cus(&cus)) != MM_OK) return s;
  if (plan.many && units > 0) {
    s = launch(moe_gate_up_many_kernel(plan.gb, plan.up_spw), dim3((unsigned)cus), mmk::kMoeManyWaves * 64, args, stream,
               "moe_ffn gate and up");
    if (s != MM_OK) return s;
    s = launch(moe_down_many_kernel(plan.gb), dim3((unsigned)cus), mmk::kMoeManyWaves * 64, args, stream,
               "moe_ffn down");
    if (s != MM_OK) return s;
    return launch(fn(&mmk::moe_combine), dim3((unsigned)cdiv(H, 1024), (unsigned)T), 256, args, stream, "moe_ffn combine");
  }
  if (units > 0) {
    s = launch(own ? moe_gate_up_kernel(E) : fn(&mmk::moe_gate_up<0>),
               dim3((unsigned)std::min<int64_t>(units, 4 * (int64_t)cus)), mmk::kMoeWaves * 64, args, stream,
               "moe_ffn gate and up");
    if (s != MM_OK) return s;
  }
  s = launch(T <= 16 ? fn(&mmk::moe_down<1>) : fn(&mmk::moe_down<4>),
             dim3((unsigned)cdiv(H, 16), (unsigned)plan.splits), mmk::kMoeWaves * 64, args, stream, "moe_ffn down");
  if (s != MM_OK || plan.splits == 1) return s;
  return launch(fn(&mmk::moe_join), dim3((unsigned)cdiv(T * H, 1024)), 256, args, stream, "moe_ffn join");
}

}  // extern "C"
