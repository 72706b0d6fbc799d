// zf_norm.hip -- layer norm and RMS norm over rows, with 8-bit checkpoints of
// input and output from the same pass, and their gradients.
//
// Forward, a row: mean = avg(x), var = avg((x - mean)^2) with x in registers
// (two sums, so no cancellation), y = (x - mean) rstd w + b.
// Backward, a row: xh = (x - mean) rstd, h = dy w,
//   dx = rstd (h - avg(h) - xh avg(h xh)),
// and over the rows dw = sum dy xh, db = sum dy: each group of lanes keeps its
// columns' sums in registers over the rows that it takes, a block joins its
// groups in shared memory, and a second launch adds the blocks' sums in order.
//
// Bound by HBM: a row is read once and written once.  A row lies in the
// registers of G lanes, 8 elements a lane and V times: 16 lanes for up to 128
// columns, a wave for up to 2048, a block for up to 16384; longer rows are
// read again for each of their sums.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "zf_hip_status.h"
#include "zf_rows.h"

namespace {

using namespace zf::dev;
using zf::hip_ok;
using zf::kThreads;

struct NormArgs {
  const void* x;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  Act8 x8, y8;
  int64_t x_ld, y_ld, rows;
  float eps, inv_cols;
  int32_t cols, wdt;
};

constexpr int kWaves = kThreads / 64;

// Sum over the G lanes of a row; every lane gets it.  G == kThreads: `slots`
// alternates between two sets, so one barrier a sum is enough.
template <int G>
__device__ __forceinline__ float row_sum(float x, float (*slots)[kWaves], int& turn) {
  if constexpr (G <= 64) {
    return sum_lanes<G>(x);
  } else {
    turn ^= 1;
    return sum_block<kWaves>(x, slots[turn]);
  }
}

// y of this lane's 8 elements, and the checkpoints.
template <int DT, bool LAYER>
__device__ __forceinline__ void norm_out(const NormArgs& a, int64_t i, int j, int n,
                                         const float (&x)[kChunk], float mean, float rstd) {
  if (a.x8.codes) keep8<DT>(a.x8, i, j, n, x);
  float w[kChunk], b[kChunk], y[kChunk];
  if (n > 0) {
    load8_of(a.wdt, a.w, j, n, w);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) y[k] = (LAYER ? x[k] - mean : x[k]) * rstd * w[k];
    if (a.b) {
      load8_of(a.wdt, a.b, j, n, b);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) y[k] += b[k];
    }
    const Raw<DT> r = narrow8<DT>(y);
    store_raw<DT, true>(a.y, i * a.y_ld + j, n, r);
    widen8<DT>(r, y);  // the checkpoint is of y as its type holds it
  }
  if (a.y8.codes) keep8<DT>(a.y8, i, j, n, y);
}

template <int DT, bool LAYER, int G, int V>
__global__ __launch_bounds__(kThreads) void zf_norm_kernel(NormArgs a) {
  __shared__ float slots[2][kWaves];
  int turn = 0;
  constexpr int kGroups = kThreads / G;
  const int lane = threadIdx.x % G;
  for (int64_t i = (int64_t)blockIdx.x * kGroups + threadIdx.x / G; i < a.rows;
       i += (int64_t)gridDim.x * kGroups) {
    float x[V][kChunk], s = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * G + lane) * kChunk, n = a.cols - j;
#pragma unroll
      for (int k = 0; k < kChunk; ++k) x[v][k] = 0;
      if (n > 0) load8<DT, true>(a.x, i * a.x_ld + j, n, x[v]);
    }
    float mean = 0;
    if constexpr (LAYER) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < kChunk; ++k) s += x[v][k];
      mean = row_sum<G>(s, slots, turn) * a.inv_cols;
    }
    s = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int n = a.cols - (v * G + lane) * kChunk;
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        const float d = LAYER ? x[v][k] - mean : x[v][k];
        if (!LAYER || k < n) s += d * d;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<G>(s, slots, turn) * a.inv_cols + a.eps);
    if (lane == 0) {
      a.rstd[i] = rstd;
      if constexpr (LAYER) a.mean[i] = mean;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * G + lane) * kChunk;
      norm_out<DT, LAYER>(a, i, j, a.cols - j, x[v], mean, rstd);
    }
  }
}

// Rows that do not fit in a block's registers: a pass for each sum.
template <int DT, bool LAYER>
__global__ __launch_bounds__(kThreads) void zf_norm_long(NormArgs a) {
  __shared__ float slots[2][kWaves];
  int turn = 0;
  constexpr int kSpan = kThreads * kChunk;
  for (int64_t i = blockIdx.x; i < a.rows; i += gridDim.x) {
    float x[kChunk], s = 0, mean = 0;
    if constexpr (LAYER) {
      for (int j = threadIdx.x * kChunk; j < a.cols; j += kSpan) {
        load8<DT>(a.x, i * a.x_ld + j, a.cols - j, x);
#pragma unroll
        for (int k = 0; k < kChunk; ++k) s += x[k];
      }
      mean = row_sum<kThreads>(s, slots, turn) * a.inv_cols;
    }
    s = 0;
    for (int j = threadIdx.x * kChunk; j < a.cols; j += kSpan) {
      load8<DT>(a.x, i * a.x_ld + j, a.cols - j, x);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        const float d = LAYER ? x[k] - mean : x[k];
        if (!LAYER || k < a.cols - j) s += d * d;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<kThreads>(s, slots, turn) * a.inv_cols + a.eps);
    if (threadIdx.x == 0) {
      a.rstd[i] = rstd;
      if constexpr (LAYER) a.mean[i] = mean;
    }
    for (int j0 = 0; j0 < a.cols; j0 += kSpan) {  // the 4 lanes of a group together
      const int j = j0 + threadIdx.x * kChunk;
      if (j < a.cols) load8<DT>(a.x, i * a.x_ld + j, a.cols - j, x);
      norm_out<DT, LAYER>(a, i, j, a.cols - j, x, mean, rstd);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.

struct NormGradArgs {
  const void* dy;
  const void* x;
  Act8 x8;
  const void* w;
  const float* mean;
  const float* rstd;
  void* dx;
  float* partial;  // [2][blocks][cols]: dw, db; NULL: neither is wanted
  int64_t dy_ld, x_ld, dx_ld, rows;
  float inv_cols;
  int32_t cols, wdt;
};

// 8 elements of x: KEPT from the checkpoint.
template <int DT, bool KEPT>
__device__ __forceinline__ void load_x(const NormGradArgs& a, int64_t i, int j, int n,
                                       float (&x)[kChunk]) {
  if constexpr (KEPT) {
    const u32x2 c = load_codes<true>(a.x8.codes + i * a.x8.code_ld + j, n);
    decode8(c, a.x8.scales[i * a.x8.scale_ld + j / ZF_ACT8_GROUP], x);
  } else {
    load8<DT, true>(a.x, i * a.x_ld + j, n, x);
  }
}

template <int DT, bool KEPT, bool LAYER, int G, int V>
__global__ __launch_bounds__(kThreads) void zf_norm_grad_kernel(NormGradArgs a) {
  __shared__ float slots[2][kWaves];
  int turn = 0;
  constexpr int kGroups = kThreads / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  float w[V][kChunk], dw[V][kChunk], db[V][kChunk];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int j = (v * G + lane) * kChunk, n = a.cols - j;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) w[v][k] = dw[v][k] = db[v][k] = 0;
    if (n > 0) load8_of(a.wdt, a.w, j, n, w[v]);
  }
  for (int64_t i = (int64_t)blockIdx.x * kGroups + group; i < a.rows;
       i += (int64_t)gridDim.x * kGroups) {
    float xh[V][kChunk], dy[V][kChunk], s1 = 0, s2 = 0;
    const float rstd = a.rstd[i];
    const float mean = LAYER ? a.mean[i] : 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * G + lane) * kChunk, n = a.cols - j;
      if (n > 0) {
        load8<DT, true>(a.dy, i * a.dy_ld + j, n, dy[v]);
        load_x<DT, KEPT>(a, i, j, n, xh[v]);
      } else {
#pragma unroll
        for (int k = 0; k < kChunk; ++k) dy[v][k] = xh[v][k] = 0;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int n = a.cols - (v * G + lane) * kChunk;
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        xh[v][k] = (LAYER ? xh[v][k] - mean : xh[v][k]) * rstd;
        if (k >= n) xh[v][k] = 0;  // rstd may be infinite
        dw[v][k] += dy[v][k] * xh[v][k];
        db[v][k] += dy[v][k];
        const float h = dy[v][k] * w[v][k];
        s1 += h;
        s2 += h * xh[v][k];
      }
    }
    float c1 = 0;
    if constexpr (LAYER) c1 = row_sum<G>(s1, slots, turn) * a.inv_cols;
    const float c2 = row_sum<G>(s2, slots, turn) * a.inv_cols;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * G + lane) * kChunk, n = a.cols - j;
      if (n <= 0) continue;
      float o[kChunk];
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        const float h = dy[v][k] * w[v][k];
        o[k] = rstd * ((LAYER ? h - c1 : h) - xh[v][k] * c2);
      }
      store8<DT, true>(a.dx, i * a.dx_ld + j, n, o);
    }
  }
  if (!a.partial) return;
  // the groups' sums, in order, one of the two at a time
  __shared__ float join[kGroups > 1 ? (kGroups - 1) * G * V * kChunk : 1];
  float* out = a.partial + (int64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float(&sum)[V][kChunk] = half ? db : dw;
    if constexpr (kGroups > 1) {
      __syncthreads();
      if (group > 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int k = 0; k < kChunk; ++k)
            join[(((group - 1) * V + v) * kChunk + k) * G + lane] = sum[v][k];
      }
      __syncthreads();
      if (group > 0) continue;
      for (int g = 0; g < kGroups - 1; ++g) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int k = 0; k < kChunk; ++k) sum[v][k] += join[((g * V + v) * kChunk + k) * G + lane];
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * G + lane) * kChunk, n = a.cols - j;
      if (n > 0) store8<ZF_F32>(out + (int64_t)half * gridDim.x * a.cols, j, n, sum[v]);
    }
  }
}

// Rows that do not fit in a block's registers: a pass for the two sums, one
// for dx, and the columns' sums by a launch of their own.
template <int DT, bool KEPT, bool LAYER>
__global__ __launch_bounds__(kThreads) void zf_norm_grad_long(NormGradArgs a) {
  __shared__ float slots[2][kWaves];
  int turn = 0;
  constexpr int kSpan = kThreads * kChunk;
  for (int64_t i = blockIdx.x; i < a.rows; i += gridDim.x) {
    const float rstd = a.rstd[i];
    const float mean = LAYER ? a.mean[i] : 0;
    float s1 = 0, s2 = 0, c1 = 0;
    float xh[kChunk], h[kChunk], w[kChunk];
    auto take = [&](int j, int n) {
      load8<DT>(a.dy, i * a.dy_ld + j, n, h);
      load_x<DT, KEPT>(a, i, j, n, xh);
      load8_of(a.wdt, a.w, j, n, w);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        xh[k] = k < n ? (LAYER ? xh[k] - mean : xh[k]) * rstd : 0.0f;
        h[k] *= w[k];
      }
    };
    for (int j = threadIdx.x * kChunk; j < a.cols; j += kSpan) {
      take(j, a.cols - j);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        s1 += h[k];
        s2 += h[k] * xh[k];
      }
    }
    if constexpr (LAYER) c1 = row_sum<kThreads>(s1, slots, turn) * a.inv_cols;
    const float c2 = row_sum<kThreads>(s2, slots, turn) * a.inv_cols;
    for (int j = threadIdx.x * kChunk; j < a.cols; j += kSpan) {
      take(j, a.cols - j);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) h[k] = rstd * ((LAYER ? h[k] - c1 : h[k]) - xh[k] * c2);
      store8<DT>(a.dx, i * a.dx_ld + j, a.cols - j, h);
    }
  }
}

// The columns' sums of the rows r0, r0 + gridDim.y, ..: blocks along x take
// kThreads * 8 columns.
template <int DT, bool KEPT, bool LAYER>
__global__ __launch_bounds__(kThreads) void zf_norm_grad_columns(NormGradArgs a) {
  const int j = (blockIdx.x * kThreads + threadIdx.x) * kChunk, n = a.cols - j;
  if (n <= 0) return;
  float dw[kChunk], db[kChunk], xh[kChunk], dy[kChunk];
#pragma unroll
  for (int k = 0; k < kChunk; ++k) dw[k] = db[k] = 0;
  for (int64_t i = blockIdx.y; i < a.rows; i += gridDim.y) {
    const float rstd = a.rstd[i];
    const float mean = LAYER ? a.mean[i] : 0;
    load8<DT>(a.dy, i * a.dy_ld + j, n, dy);
    load_x<DT, KEPT>(a, i, j, n, xh);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      dw[k] += dy[k] * ((LAYER ? xh[k] - mean : xh[k]) * rstd);
      db[k] += dy[k];
    }
  }
  float* out = a.partial + (int64_t)blockIdx.y * a.cols;
  store8<ZF_F32>(out, j, n, dw);
  store8<ZF_F32>(out + (int64_t)gridDim.y * a.cols, j, n, db);
}

// Adds the blocks' partial sums: 64 columns a block, its 16 waves every 16th
// of them, and the waves' sums in order.
constexpr int kJoinThreads = 1024;
struct JoinArgs {
  const float* partial;  // [2][count][cols]
  void* out[2];          // dw, db; either may be NULL
  int32_t count, cols, gdt, accumulate;
};
__global__ __launch_bounds__(kJoinThreads) void zf_norm_grad_join(JoinArgs a) {
  constexpr int W = kJoinThreads / 64;
  __shared__ float s[W][64];
  void* out = a.out[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = blockIdx.x * 64 + lane;
  const float* p = a.partial + (int64_t)blockIdx.y * a.count * a.cols + j;
  float sum = 0;
  if (j < a.cols) {
#pragma unroll 8
    for (int r = wave; r < a.count; r += W) sum += p[(int64_t)r * a.cols];
  }
  s[wave][lane] = sum;
  __syncthreads();
  if (wave > 0 || j >= a.cols) return;
#pragma unroll
  for (int w = 1; w < W; ++w) sum += s[w][lane];
  if (a.accumulate) sum += load1_of(a.gdt, out, j);
  store1_of(a.gdt, out, j, sum);
}

// ---------------------------------------------------------------------------
// Host side.

constexpr int kMostCols = kThreads * kChunk * 8;  // of a row in registers

// Blocks of the backward pass, each with a partial sum: 4 for each compute
// unit at most, and rows enough for each that the partial sums are little
// beside them.
int grad_blocks(int64_t rows, int64_t cols) {
  const int64_t groups = cols <= 128 ? 16 : cols <= 2048 ? 4 : 1;
  const int64_t want = (rows + groups * 4 - 1) / (groups * 4);
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, 1024));
}

template <typename F>
void by_shape(int64_t cols, F f) {
#define ZF_SHAPE(G, V) f(std::integral_constant<int, G>(), std::integral_constant<int, V>())
  if (cols <= 128) ZF_SHAPE(16, 1);
  else if (cols <= 512) ZF_SHAPE(64, 1);
  else if (cols <= 1024) ZF_SHAPE(64, 2);
  else if (cols <= 2048) ZF_SHAPE(64, 4);
  else if (cols <= 4096) ZF_SHAPE(256, 2);
  else if (cols <= 8192) ZF_SHAPE(256, 4);
  else ZF_SHAPE(256, 8);
#undef ZF_SHAPE
}

template <typename F>
void by_dtype(int32_t dt, F f) {
  if (dt == ZF_F32) f(std::integral_constant<int, ZF_F32>());
  else if (dt == ZF_BF16) f(std::integral_constant<int, ZF_BF16>());
  else f(std::integral_constant<int, ZF_F16>());
}

}  // namespace

extern "C" int zf_layer_norm(const zf_layer_norm_args* args, void* stream) {
  if (!args || args->reserved != 0) return ZF_EINVAL;
  const zf_layer_norm_args& p = *args;
  if (p.kind != ZF_NORM_LAYER && p.kind != ZF_NORM_RMS) return ZF_EINVAL;
  if (!row_dtype(p.dtype) || !row_dtype(p.weight_dtype)) return ZF_EDTYPE;
  if (!(p.eps >= 0) || !std::isfinite((float)p.eps)) return ZF_EINVAL;
  int rc = shape_ok(p.rows, p.cols);
  if (rc == ZF_OK) rc = rows_ok(p.x, p.dtype, p.rows, p.cols, p.x_stride);
  if (rc == ZF_OK) rc = rows_ok(p.y, p.dtype, p.rows, p.cols, p.y_stride);
  if (rc == ZF_OK && p.x8) rc = act8_ok(p.x8, p.rows, p.cols);
  if (rc == ZF_OK && p.y8) rc = act8_ok(p.y8, p.rows, p.cols);
  if (rc != ZF_OK) return rc;
  const bool layer = p.kind == ZF_NORM_LAYER;
  if (p.rows > 0 && (!p.weight || !p.rstd || (layer && !p.mean))) return ZF_EINVAL;
  if (p.x == p.y && p.rows > 1 && p.x_stride != p.y_stride) return ZF_EINVAL;
  if (!aligned_to(p.weight, p.weight_dtype) || !aligned_to(p.bias, p.weight_dtype) ||
      !aligned_to(p.rstd, ZF_F32) || (layer && !aligned_to(p.mean, ZF_F32)))
    return ZF_EALIGN;
  if (p.rows == 0) return ZF_OK;
  NormArgs a;
  a.x = p.x;
  a.w = p.weight;
  a.b = p.bias;
  a.y = p.y;
  a.mean = p.mean;
  a.rstd = p.rstd;
  a.x8 = act8_of(p.x8);
  a.y8 = act8_of(p.y8);
  a.x_ld = p.x_stride;
  a.y_ld = p.y_stride;
  a.rows = p.rows;
  a.eps = (float)p.eps;
  a.inv_cols = (float)(1.0 / (double)p.cols);
  a.cols = (int32_t)p.cols;
  a.wdt = p.weight_dtype;
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  by_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (p.cols > kMostCols) {
      const dim3 grid((uint32_t)std::min<int64_t>(p.rows, kMaxBlocks));
      if (layer) hipLaunchKernelGGL((zf_norm_long<DT, true>), grid, dim3(kThreads), 0, s, a);
      else hipLaunchKernelGGL((zf_norm_long<DT, false>), grid, dim3(kThreads), 0, s, a);
      return;
    }
    by_shape(p.cols, [&](auto g, auto v) {
      constexpr int G = decltype(g)::value, V = decltype(v)::value, per = kThreads / G;
      const dim3 grid((uint32_t)std::min<int64_t>((p.rows + per - 1) / per, kMaxBlocks));
      if (layer) hipLaunchKernelGGL((zf_norm_kernel<DT, true, G, V>), grid, dim3(kThreads), 0, s, a);
      else hipLaunchKernelGGL((zf_norm_kernel<DT, false, G, V>), grid, dim3(kThreads), 0, s, a);
    });
  });
  return hip_ok(hipGetLastError()) ? ZF_OK : ZF_EHIP;
}

extern "C" int64_t zf_layer_norm_grad_bytes(int64_t rows, int64_t cols) {
  const int rc = shape_ok(rows, cols);
  if (rc != ZF_OK) return rc;
  return (2 * (int64_t)sizeof(float) * grad_blocks(rows, cols) * cols + 15) / 16 * 16;
}

extern "C" int zf_layer_norm_grad(const zf_layer_norm_grad_args* args, void* stream) {
  if (!args || args->reserved != 0) return ZF_EINVAL;
  const zf_layer_norm_grad_args& p = *args;
  if (p.kind != ZF_NORM_LAYER && p.kind != ZF_NORM_RMS) return ZF_EINVAL;
  if (!flag(p.accumulate)) return ZF_EINVAL;
  if (!row_dtype(p.dtype) || !row_dtype(p.weight_dtype) || !row_dtype(p.grad_dtype))
    return ZF_EDTYPE;
  const bool layer = p.kind == ZF_NORM_LAYER;
  int rc = shape_ok(p.rows, p.cols);
  if (rc == ZF_OK) rc = rows_ok(p.dy, p.dtype, p.rows, p.cols, p.dy_stride);
  if (rc == ZF_OK) rc = rows_ok(p.dx, p.dtype, p.rows, p.cols, p.dx_stride);
  if (rc == ZF_OK && p.x8) rc = p.x ? ZF_EINVAL : act8_ok(p.x8, p.rows, p.cols);
  else if (rc == ZF_OK) rc = rows_ok(p.x, p.dtype, p.rows, p.cols, p.x_stride);
  if (rc != ZF_OK) return rc;
  if (p.rows > 0 && (!p.weight || !p.rstd || (layer && !p.mean))) return ZF_EINVAL;
  if (p.dx == p.dy && p.rows > 1 && p.dx_stride != p.dy_stride) return ZF_EINVAL;
  if (!aligned_to(p.weight, p.weight_dtype) || !aligned_to(p.rstd, ZF_F32) ||
      (layer && !aligned_to(p.mean, ZF_F32)) || !aligned_to(p.weight_grad, p.grad_dtype) ||
      !aligned_to(p.bias_grad, p.grad_dtype))
    return ZF_EALIGN;
  const bool sums = p.weight_grad || p.bias_grad;
  if (sums && !p.workspace) return ZF_EINVAL;
  if (sums && !aligned16(p.workspace)) return ZF_EALIGN;
  if (sums && p.workspace_size < zf_layer_norm_grad_bytes(p.rows, p.cols)) return ZF_ESIZE;
  if (!sums && p.rows == 0) return ZF_OK;
  const int blocks = p.rows > 0 ? grad_blocks(p.rows, p.cols) : 0;
  NormGradArgs a;
  a.dy = p.dy;
  a.x = p.x;
  a.x8 = act8_of(p.x8);
  a.w = p.weight;
  a.mean = p.mean;
  a.rstd = p.rstd;
  a.dx = p.dx;
  a.partial = sums ? static_cast<float*>(p.workspace) : nullptr;
  a.dy_ld = p.dy_stride;
  a.x_ld = p.x_stride;
  a.dx_ld = p.dx_stride;
  a.rows = p.rows;
  a.inv_cols = (float)(1.0 / (double)p.cols);
  a.cols = (int32_t)p.cols;
  a.wdt = p.weight_dtype;
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (p.rows > 0) {
    by_dtype(p.dtype, [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      auto kinds = [&](auto kept, auto lay) {
        constexpr bool KEPT = decltype(kept)::value, LAYER = decltype(lay)::value;
        if (p.cols > kMostCols) {
          const int span = kThreads * kChunk;
          const dim3 cols((uint32_t)((p.cols + span - 1) / span), (uint32_t)blocks);
          if (sums)  // first: dx may lie in dy's place
            hipLaunchKernelGGL((zf_norm_grad_columns<DT, KEPT, LAYER>), cols, dim3(kThreads), 0, s, a);
          const dim3 grid((uint32_t)std::min<int64_t>(p.rows, kMaxBlocks));
          hipLaunchKernelGGL((zf_norm_grad_long<DT, KEPT, LAYER>), grid, dim3(kThreads), 0, s, a);
          return;
        }
        by_shape(p.cols, [&](auto g, auto v) {
          hipLaunchKernelGGL((zf_norm_grad_kernel<DT, KEPT, LAYER, decltype(g)::value, decltype(v)::value>),
                             dim3(blocks), dim3(kThreads), 0, s, a);
        });
      };
      if (p.x8 && layer) kinds(std::true_type(), std::true_type());
      else if (p.x8) kinds(std::true_type(), std::false_type());
      else if (layer) kinds(std::false_type(), std::true_type());
      else kinds(std::false_type(), std::false_type());
    });
  }
  if (sums) {
    const JoinArgs j{static_cast<const float*>(p.workspace), {p.weight_grad, p.bias_grad}, blocks,
                     (int32_t)p.cols, p.grad_dtype, p.accumulate};
    hipLaunchKernelGGL(zf_norm_grad_join, dim3((uint32_t)((p.cols + 63) / 64), 2),
                       dim3(kJoinThreads), 0, s, j);
  }
  return hip_ok(hipGetLastError()) ? ZF_OK : ZF_EHIP;
}
