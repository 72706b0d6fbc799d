// zf_norm_grad.hip -- gradients of layer norm and RMS norm, from the input or
// from its 8-bit checkpoint.
//
// With xh = (x - mean) rstd and h = dy w,
//   dx = rstd (h - avg(h) - xh avg(h xh)),
// and over the rows dw = sum dy xh, db = sum dy: each group of lanes keeps its
// columns' sums in registers over the rows that it takes, a block joins its
// groups in shared memory, and a second launch adds the blocks' sums in order.
//
// Bound by HBM: a row of dy and of x is read once and one of dx written once.
// 32768 rows of 2048 bf16 from a checkpoint (338 MB): 64.7 us, of which the join
// takes 5.9 and the pass 5.6 TB/s; 1000 rows of 1024: two launches of 6.0 and 4.8 us.
// Both for rows of whole lines: 67M elements from a checkpoint take 63 to 82 us in rows
// of 128 to 8192, 76 in rows of 1000, and 137 of 2050, 126 of 4100, 114 of 40, where rows
// begin inside a line and lanes idle.  Rows of 8193 to 16384 take 93 to 114: their
// lanes hold 16 elements in 128 registers and spill 48 to 203 of them.  Longer ones
// are read three times, 140.
//
// dx is stored non-temporally: 67M elements in rows of 2048 and 2050 from x 77.8 and
// 143.3 us, plainly 79.9 and 146.2.
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

struct NormGradArgs {
  const void* dy;
  const void* x;
  Act8 x8;
  const void* w;
  const float* mean;
  const float* rstd;
  void* dx;
  float* dw;  // the blocks' sums, [blocks][cols]; NULL: not wanted
  float* db;
  int64_t dy_ld, x_ld, dx_ld, rows;
  float inv_cols;
  int32_t cols, wdt;
};

// 8 elements of x as the registers hold them: KEPT codes and their scale.
template <int DT, bool KEPT>
struct RawX {
  Raw<DT> r;
};
template <int DT>
struct RawX<DT, true> {
  u32x2 c;
  uint32_t scale;
};
template <int DT, bool KEPT, bool NT, bool WHOLE>
__device__ __forceinline__ RawX<DT, KEPT> load_x(const NormGradArgs& a, int64_t i, int j, int n) {
  RawX<DT, KEPT> r;
  if constexpr (KEPT) {
    r.c = load_codes<NT, WHOLE>(a.x8.codes + i * a.x8.code_ld + j, n);
    r.scale = n > 0 ? a.x8.scales[i * a.x8.scale_ld + j / ZF_ACT8_GROUP] : 127u;
  } else {
    r.r = load_raw<DT, NT, WHOLE>(a.x, i * a.x_ld + j, n);
  }
  return r;
}
template <int DT, bool KEPT>
__device__ __forceinline__ void widen_x(const RawX<DT, KEPT>& r, float (&x)[kChunk]) {
  if constexpr (KEPT) decode8(r.c, r.scale, x);
  else widen8<DT>(r.r, x);
}

// x to xh, and zeros past the row's n elements, where -mean rstd may be infinite.
template <bool LAYER, bool WHOLE>
__device__ __forceinline__ void normalize(float (&x)[kChunk], int n, float mean, float rstd) {
#pragma unroll
  for (int k = 0; k < kChunk; ++k) {
    const float from = (WHOLE ? n > 0 : k < n) ? mean : 0.0f;
    x[k] = (LAYER ? x[k] - from : x[k]) * rstd;
  }
}

// A group of G lanes takes a row at a time, 8 V elements a lane; its parameters
// and the columns' sums stay in registers, and the next row is on its way while
// this one is worked on.  Rows of more than 512 elements take a block and its
// barrier instead of a wave: parameters, two columns' sums and a row's
// operands are 40 V registers beside the loads, and with V = 4 (2048 columns a
// wave) they spill.  32768 rows of 2048 from a checkpoint: 70 us with V = 1 (two
// rows at a time 80, a wave a row 90; before later steps took it to 64.7).
// Elements past the row's end have dy = 0 and xh = 0, so they add nothing (where
// rstd is not finite, the row's own elements are not either).
template <int DT, bool KEPT, bool LAYER, int T, int G, int V, bool WHOLE>
__global__ __launch_bounds__(T) void zf_norm_grad_kernel(NormGradArgs a) {
  constexpr int N = LAYER ? 2 : 1;  // sums of a row: h xh, and h
  __shared__ float slots[2][N][T / 64];
  int turn = 0;
  constexpr int kGroups = T / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t i = (int64_t)blockIdx.x * kGroups + group;
  Raw<DT> next_dy[V];
  RawX<DT, KEPT> next_x[V];
  float next_rstd, next_mean;
  auto fetch = [&](int64_t row) {
    const bool in = row < a.rows;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * G + lane) * kChunk, n = in ? a.cols - j : 0;
      next_dy[v] = load_raw<DT, true, WHOLE>(a.dy, row * a.dy_ld + j, n);
      next_x[v] = load_x<DT, KEPT, true, WHOLE>(a, row, j, n);
    }
    next_rstd = in ? a.rstd[row] : 0;
    next_mean = LAYER && in ? a.mean[row] : 0;
  };
  fetch(i);
  float w[V][kChunk], dw[V][kChunk], db[V][kChunk];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int j = (v * G + lane) * kChunk;
    load8_of<WHOLE>(a.wdt, a.w, j, a.cols - j, w[v]);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) dw[v][k] = db[v][k] = 0;
  }
  for (; i < a.rows; i += step) {
    float xh[V][kChunk], h[V][kChunk], sums[N];
    const float rstd = next_rstd, mean = next_mean;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      widen8<DT>(next_dy[v], h[v]);
      widen_x<DT, KEPT>(next_x[v], xh[v]);
    }
    fetch(i + step);
#pragma unroll
    for (int k = 0; k < N; ++k) sums[k] = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int n = a.cols - (v * G + lane) * kChunk;
      normalize<LAYER, WHOLE>(xh[v], n, mean, rstd);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        dw[v][k] = __builtin_fmaf(h[v][k], xh[v][k], dw[v][k]);
        db[v][k] += h[v][k];
        h[v][k] *= w[v][k];
        sums[0] = __builtin_fmaf(h[v][k], xh[v][k], sums[0]);
        if constexpr (LAYER) sums[N - 1] += h[v][k];
      }
    }
    row_sums<G, T, N>(sums, slots, turn);
    const float c2 = sums[0] * a.inv_cols, c1 = LAYER ? sums[N - 1] * a.inv_cols : 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (v * G + lane) * kChunk;
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        h[v][k] = rstd * __builtin_fmaf(-xh[v][k], c2, LAYER ? h[v][k] - c1 : h[v][k]);
      store8<DT, true, WHOLE>(a.dx, i * a.dx_ld + j, a.cols - j, h[v]);
    }
  }
  // the groups' sums, in order, one of the two at a time
  __shared__ float join[kGroups > 1 ? (kGroups - 1) * G * V * kChunk : 1];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float* out = half ? a.db : a.dw;
    if (!out) continue;
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
      const int j = (v * G + lane) * kChunk;
      store8<ZF_F32, false, WHOLE>(out + (int64_t)blockIdx.x * a.cols, j, a.cols - j, sum[v]);
    }
  }
}

// Rows that do not fit in a block's registers: a pass for the two sums, one
// for dx, and the columns' sums by a launch of their own.
template <int DT, bool KEPT, bool LAYER>
__global__ __launch_bounds__(kThreads) void zf_norm_grad_long(NormGradArgs a) {
  __shared__ float slots[2][2][kThreads / 64];
  int turn = 0;
  constexpr int kSpan = kThreads * kChunk;
  for (int64_t i = blockIdx.x; i < a.rows; i += gridDim.x) {
    const float rstd = a.rstd[i];
    const float mean = LAYER ? a.mean[i] : 0;
    float s1 = 0, s2 = 0;
    float xh[kChunk], h[kChunk], w[kChunk];
    auto take = [&](int j, int n) {
      load8<DT>(a.dy, i * a.dy_ld + j, n, h);
      widen_x<DT, KEPT>(load_x<DT, KEPT, false, false>(a, i, j, n), xh);
      load8_of(a.wdt, a.w, j, n, w);
      normalize<LAYER, false>(xh, n, mean, rstd);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) h[k] *= w[k];
    };
    for (int j = threadIdx.x * kChunk; j < a.cols; j += kSpan) {
      take(j, a.cols - j);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        s1 += h[k];
        s2 += h[k] * xh[k];
      }
    }
    float sums[2] = {s2, s1};
    row_sums<kThreads, kThreads, 2>(sums, slots, turn);
    const float c1 = LAYER ? sums[1] * a.inv_cols : 0, c2 = sums[0] * a.inv_cols;
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
    widen_x<DT, KEPT>(load_x<DT, KEPT, false, false>(a, i, j, n), xh);
    normalize<LAYER, false>(xh, n, mean, rstd);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      dw[k] += dy[k] * xh[k];
      db[k] += dy[k];
    }
  }
  if (a.dw) store8<ZF_F32>(a.dw + (int64_t)blockIdx.y * a.cols, j, n, dw);
  if (a.db) store8<ZF_F32>(a.db + (int64_t)blockIdx.y * a.cols, j, n, db);
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

// As the forward pass's, but for rows of 4104 to 8192, where 1024 threads leave a lane
// half as many sums: 67M bf16 elements in rows of 5120 and 8192 90 and 85 us, 512
// threads with 16 elements a lane 97 and 93.
template <typename F>
void by_grad_shape(int64_t cols, F f) {
  if (cols % kChunk != 0) {
    if (cols <= 128) f(Shape<256, 16, 1, false>());
    else if (cols <= 512) f(Shape<256, 64, 1, false>());
    else if (cols <= 2048) f(Shape<256, 256, 1, false>());
    else if (cols <= 4096) f(Shape<512, 512, 1, false>());
    else if (cols <= 8192) f(Shape<1024, 1024, 1, false>());
    else f(Shape<1024, 1024, 2, false>());
  } else if (cols <= 128) f(Shape<256, 16, 1, true>());
  else if (cols <= 512) f(Shape<256, 64, 1, true>());
  else if (cols <= 1024) f(Shape<128, 128, 1, true>());
  else if (cols <= 2048) f(Shape<256, 256, 1, true>());
  else if (cols <= 4096) f(Shape<512, 512, 1, true>());
  else if (cols <= 8192) f(Shape<1024, 1024, 1, true>());
  else f(Shape<1024, 1024, 2, true>());
}

// Blocks of the backward pass, each with a partial sum: 1024 threads for each
// compute unit (32768 rows of 2048 from a checkpoint, at the time 70 us; half or
// twice as many threads 90 and 76), and 4 rows at least for each group of lanes.
int grad_blocks(int64_t rows, int64_t cols) {
  int64_t per = 4, most = 1024;
  if (cols <= kMostCols)
    by_grad_shape(cols, [&](auto shape) {
      typedef decltype(shape) S;
      per = S::T / S::G;
      most = 256 * 1024 / S::T;
    });
  return (int)std::max<int64_t>(1, std::min<int64_t>((rows + per * 4 - 1) / (per * 4), most));
}

}  // namespace

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
  float* partial = static_cast<float*>(p.workspace);
  a.dw = p.weight_grad ? partial : nullptr;
  a.db = p.bias_grad ? partial + blocks * p.cols : nullptr;
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
      by_flags(p.x8 != nullptr, layer, [&](auto kept, auto lay) {
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
        by_grad_shape(p.cols, [&](auto shape) {
          typedef decltype(shape) S;
          hipLaunchKernelGGL((zf_norm_grad_kernel<DT, KEPT, LAYER, S::T, S::G, S::V, S::WHOLE>),
                             dim3(blocks), dim3(S::T), 0, s, a);
        });
      });
    });
  }
  if (sums) {
    const JoinArgs j{partial, {p.weight_grad, p.bias_grad}, blocks,
                     (int32_t)p.cols, p.grad_dtype, p.accumulate};
    hipLaunchKernelGGL(zf_norm_grad_join, dim3((uint32_t)((p.cols + 63) / 64), 2),
                       dim3(kJoinThreads), 0, s, j);
  }
  return hip_ok(hipGetLastError()) ? ZF_OK : ZF_EHIP;
}
