// zf_norm.hip -- layer norm and RMS norm over rows, with 8-bit checkpoints of
// input and output from the same pass.
//
// A row: mean = avg(x), var = avg((x - mean)^2) with x in registers (two sums,
// so no cancellation), y = (x - mean) rstd w + b.  Bound by HBM: a row is read
// once and written once; rows of more than 16384 elements are read again for
// each of their sums.  32768 rows of 2048 bf16 with both checkpoints (407 MB): 73.6
// us, 5.5 TB/s, where a copy reaches 6.4; 333 rows of 1000: 4.3 us, a launch's time.
// So it is for rows of 128 to 8192 that are multiples of 128 bytes: 67M bf16
// elements without checkpoints in rows of 128 to 8192 46 to 57 us.  Of 1000 they take
// 57, of 10000 67, of 40 107, of 2050 112 (and 112 with both checkpoints), of 4100
// 121: rows begin inside a line, and lanes behind a row's end idle.
//
// Stores are non-temporal.  67M bf16 elements in rows of 2048, of 1000 and of 2050:
// y alone 48.4, 57.2 and 111.4 us, with plain stores 50.5, 61.4 and 117.5; y and both
// checkpoints 73.8, 95.7 and 111.1, with plain stores 66.6, 75.3 and 112.5.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "zf_hip_status.h"
#include "zf_norm.h"

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

// y of this lane's 8 elements, and the checkpoints; n of the elements exist,
// the others of x are zero.
template <int DT, bool LAYER, bool BIAS, bool WHOLE>
__device__ __forceinline__ void norm_out(const NormArgs& a, int64_t i, int j, int n,
                                         const float (&x)[kChunk], const float (&w)[kChunk],
                                         const float (&b)[kChunk], float mean, float rstd) {
  if (a.x8.codes) keep8<DT, true, WHOLE>(a.x8, i, j, n, x);
  float y[kChunk];
#pragma unroll
  for (int k = 0; k < kChunk; ++k) {
    y[k] = (LAYER ? x[k] - mean : x[k]) * rstd * w[k];
    if constexpr (BIAS) y[k] += b[k];
  }
  const Raw<DT> r = narrow8<DT>(y);
  store_raw<DT, true, WHOLE>(a.y, i * a.y_ld + j, n, r);
  if (!a.y8.codes) return;
  widen8<DT>(r, y);  // the checkpoint is of y as its type holds it
  if (n < kChunk) {
#pragma unroll
    for (int k = 0; k < kChunk; ++k) y[k] = !WHOLE && k < n ? y[k] : 0.0f;
  }
  keep8<DT, true, WHOLE>(a.y8, i, j, n, y);
}

// Sum of the squared distances of n of 8 elements from the mean.
template <bool LAYER, bool WHOLE>
__device__ __forceinline__ float squares(const float (&x)[kChunk], int n, float mean, float s) {
  if (!LAYER || (WHOLE ? n > 0 : n >= kChunk)) {
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      const float d = LAYER ? x[k] - mean : x[k];
      s = __builtin_fmaf(d, d, s);
    }
  } else if (!WHOLE && n > 0) {
#pragma unroll
    for (int k = 0; k < kChunk - 1; ++k) {
      const float d = k < n ? x[k] - mean : 0.0f;
      s = __builtin_fmaf(d, d, s);
    }
  }
  return s;
}

// Threads of a launch: 8192 for each compute unit, 1024 where a lane holds 16
// elements.  67M bf16 elements in rows of 2048 with both checkpoints 77 us (1024
// for each 83, a row a group 84), in rows of 8192 80 us (8192 for each 82).
template <typename S>
constexpr int64_t kMostThreads = 256 * (S::V == 1 ? 8192 : 1024);

// A group of G lanes takes every so many rows; its share of the parameters
// stays in registers, and the next row is on its way while this one is worked
// on.
template <int DT, bool LAYER, bool BIAS, int T, int G, int V, bool WHOLE>
__global__ __launch_bounds__(T) void zf_norm_kernel(NormArgs a) {
  __shared__ float slots[2][1][T / 64];
  int turn = 0;
  constexpr int kGroups = T / G;
  const int lane = threadIdx.x % G;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t i = (int64_t)blockIdx.x * kGroups + threadIdx.x / G;
  Raw<DT> next[V];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * G + lane) * kChunk;
      next[v] = load_raw<DT, true, WHOLE>(a.x, row * a.x_ld + j, row < a.rows ? a.cols - j : 0);
    }
  };
  fetch(i);
  float w[V][kChunk], b[V][kChunk];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int j = (v * G + lane) * kChunk;
    load8_of<WHOLE>(a.wdt, a.w, j, a.cols - j, w[v]);
    if constexpr (BIAS) load8_of<WHOLE>(a.wdt, a.b, j, a.cols - j, b[v]);
  }
  for (; i < a.rows; i += step) {
    float x[V][kChunk], s = 0, mean = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) widen8<DT>(next[v], x[v]);
    fetch(i + step);
    if constexpr (LAYER) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < kChunk; ++k) s += x[v][k];
      mean = row_sum<G, T>(s, slots, turn) * a.inv_cols;
    }
    s = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) s = squares<LAYER, WHOLE>(x[v], a.cols - (v * G + lane) * kChunk, mean, s);
    const float rstd = 1.0f / sqrtf(row_sum<G, T>(s, slots, turn) * a.inv_cols + a.eps);
    if (lane == 0) {
      a.rstd[i] = rstd;
      if constexpr (LAYER) a.mean[i] = mean;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * G + lane) * kChunk;
      norm_out<DT, LAYER, BIAS, WHOLE>(a, i, j, a.cols - j, x[v], w[v], b[v], mean, rstd);
    }
  }
}

// Rows that do not fit in a block's registers: a pass for each sum.
template <int DT, bool LAYER, bool BIAS>
__global__ __launch_bounds__(kThreads) void zf_norm_long(NormArgs a) {
  __shared__ float slots[2][1][kThreads / 64];
  int turn = 0;
  constexpr int kSpan = kThreads * kChunk;
  for (int64_t i = blockIdx.x; i < a.rows; i += gridDim.x) {
    float x[kChunk], w[kChunk], b[kChunk], s = 0, mean = 0;
    if constexpr (LAYER) {
      for (int j = threadIdx.x * kChunk; j < a.cols; j += kSpan) {
        load8<DT>(a.x, i * a.x_ld + j, a.cols - j, x);
#pragma unroll
        for (int k = 0; k < kChunk; ++k) s += x[k];
      }
      mean = row_sum<kThreads, kThreads>(s, slots, turn) * a.inv_cols;
    }
    s = 0;
    for (int j = threadIdx.x * kChunk; j < a.cols; j += kSpan) {
      load8<DT>(a.x, i * a.x_ld + j, a.cols - j, x);
      s = squares<LAYER, false>(x, a.cols - j, mean, s);
    }
    const float rstd = 1.0f / sqrtf(row_sum<kThreads, kThreads>(s, slots, turn) * a.inv_cols + a.eps);
    if (threadIdx.x == 0) {
      a.rstd[i] = rstd;
      if constexpr (LAYER) a.mean[i] = mean;
    }
    for (int j0 = 0; j0 < a.cols; j0 += kSpan) {  // the 4 lanes of a group together
      const int j = j0 + threadIdx.x * kChunk;
      load8<DT>(a.x, i * a.x_ld + j, a.cols - j, x);
      load8_of(a.wdt, a.w, j, a.cols - j, w);
      if constexpr (BIAS) load8_of(a.wdt, a.b, j, a.cols - j, b);
      norm_out<DT, LAYER, BIAS, false>(a, i, j, a.cols - j, x, w, b, mean, rstd);
    }
  }
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
    by_flags(layer, p.bias != nullptr, [&](auto lay, auto bias) {
      constexpr bool LAYER = decltype(lay)::value, BIAS = decltype(bias)::value;
      if (p.cols > kMostCols) {
        const dim3 grid((uint32_t)std::min<int64_t>(p.rows, kMaxBlocks));
        hipLaunchKernelGGL((zf_norm_long<DT, LAYER, BIAS>), grid, dim3(kThreads), 0, s, a);
        return;
      }
      by_shape(p.cols, [&](auto shape) {
        typedef decltype(shape) S;
        constexpr int64_t per = S::T / S::G;
        const dim3 grid((uint32_t)std::min<int64_t>((p.rows + per - 1) / per, kMostThreads<S> / S::T));
        hipLaunchKernelGGL((zf_norm_kernel<DT, LAYER, BIAS, S::T, S::G, S::V, S::WHOLE>), grid,
                           dim3(S::T), 0, s, a);
      });
    });
  });
  return hip_ok(hipGetLastError()) ? ZF_OK : ZF_EHIP;
}
