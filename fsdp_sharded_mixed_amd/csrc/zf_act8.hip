// zf_act8.hip -- activation checkpoints in 8 bits: kept from and read back to
// rows of activations (the norms keep theirs in their own pass, zf_norm.hip;
// a Linear's weight gradient reads one directly, zf_weight_grad.hip).
//
// x is kept as e4m3 of x / 2^k with one k for each 32 elements of a row, so
// that products can take the numbers exactly in 16 bits and a scale is one
// byte.  Bound by HBM: 2 + 1 + 1/32 bytes an element of bf16 each way.  8192 rows
// of 8192: kept in 35.8 us (5.7 TB/s), read back in 29.4 (6.9, the codes partly
// from the Infinity Cache; 35.5 without it).  As many elements in rows of 40 to 16384
// that are whole 8s: kept in 36 to 49, read back in 35 to 46; in rows of 2050 58 and
// 50, of 300 68 and 65.  To and from fp32 58 to 65 and 89 to
// 108 in rows of whole lines (134 MB more each way).
//
// What is read back is stored non-temporally: rows of 2048 35.5 us, plainly 37.1.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "zf_hip_status.h"
#include "zf_rows.h"

namespace {

using namespace zf::dev;
using zf::hip_ok;
using zf::kThreads;

struct Act8Args {
  Act8 a;
  void* x;
  int64_t x_ld, rows, cols;
  int32_t log_lanes;  // 2^log_lanes lanes of 8 elements to a row, 4 at least
};

// Blocks along x take the rows, as far apart as the launch has blocks there;
// blocks along y the columns that one span of lanes does not cover.
template <int DT, bool STORE>
__global__ __launch_bounds__(kThreads) void zf_act8_kernel(Act8Args a) {
  const int lanes = 1 << a.log_lanes, per = kThreads >> a.log_lanes;
  const int64_t j = ((int64_t)blockIdx.y * lanes + (threadIdx.x & (lanes - 1))) * kChunk;
  const int left = (int)min((int64_t)kChunk, a.cols - j);
  int64_t i = (int64_t)blockIdx.x * per + (threadIdx.x >> a.log_lanes);
  for (; i < a.rows; i += (int64_t)gridDim.x * per) {  // the lanes of a row together
    float v[kChunk];
    if constexpr (STORE) {
      load8<DT, true>(a.x, i * a.x_ld + j, left, v);
      keep8<DT>(a.a, i, j, left, v);
    } else {
      if (left <= 0) return;
      const u32x2 c = load_codes<true>(a.a.codes + i * a.a.code_ld + j, left);
      decode8(c, a.a.scales[i * a.a.scale_ld + j / ZF_ACT8_GROUP], v);
      store8<DT, true>(a.x, i * a.x_ld + j, left, v);
    }
  }
}

int run(const zf_act8* a, int32_t dtype, void* x, int64_t x_stride, bool store, void* stream) {
  if (!a) return ZF_EINVAL;
  if (!row_dtype(dtype)) return ZF_EDTYPE;
  int rc = shape_ok(a->rows, a->cols);
  if (rc == ZF_OK) rc = act8_ok(a, a->rows, a->cols);
  if (rc == ZF_OK) rc = rows_ok(x, dtype, a->rows, a->cols, x_stride);
  if (rc != ZF_OK) return rc;
  if (a->rows == 0) return ZF_OK;
  Act8Args k{act8_of(a), x, x_stride, a->rows, a->cols, 2};
  while (k.log_lanes < 8 && ((int64_t)kChunk << k.log_lanes) < a->cols) ++k.log_lanes;
  const int64_t span = (int64_t)kChunk << k.log_lanes, per = kThreads >> k.log_lanes;
  const dim3 grid((uint32_t)std::min<int64_t>((a->rows + per - 1) / per, kMaxBlocks),
                  (uint32_t)((a->cols + span - 1) / span));
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
#define ZF_ACT8(DT) \
  do { \
    if (store) hipLaunchKernelGGL((zf_act8_kernel<DT, true>), grid, dim3(kThreads), 0, s, k); \
    else hipLaunchKernelGGL((zf_act8_kernel<DT, false>), grid, dim3(kThreads), 0, s, k); \
  } while (0)
  if (dtype == ZF_F32) ZF_ACT8(ZF_F32);
  else if (dtype == ZF_BF16) ZF_ACT8(ZF_BF16);
  else ZF_ACT8(ZF_F16);
#undef ZF_ACT8
  return hip_ok(hipGetLastError()) ? ZF_OK : ZF_EHIP;
}

}  // namespace

extern "C" int zf_act8_store(const zf_act8* a, int32_t dtype, const void* x, int64_t x_stride,
                             void* stream) {
  return run(a, dtype, const_cast<void*>(x), x_stride, true, stream);
}

extern "C" int zf_act8_load(const zf_act8* a, int32_t dtype, void* x, int64_t x_stride,
                            void* stream) {
  return run(a, dtype, x, x_stride, false, stream);
}
