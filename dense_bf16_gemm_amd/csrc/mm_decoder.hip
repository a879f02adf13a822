// mm_decoder.hip -- C ABI of the decoder-layer operators (declared in
// include/mm.h): the residual addition with its RMS norm and gradient, and
// the products with 4-bit and 8-bit weights.  Argument checks, the choice of
// a kernel's shape, launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "mm_host.hpp"
#include "rms_norm.hpp"
#include "gemm_w4.hpp"
#include "gemm_q8.hpp"

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

}  // extern "C"
