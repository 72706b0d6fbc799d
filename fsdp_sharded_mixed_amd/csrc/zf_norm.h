// zf_norm.h -- what the norms' forward and backward passes share: sums over a
// row's lanes, and the choice of a kernel by a row's length.
#pragma once
#include <type_traits>

#include "zf_rows.h"

namespace zf {
namespace dev {

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

// A row lies in the registers of G lanes, 8 elements a lane and V times: 16
// lanes for up to 128 columns, a wave for up to 2048, a block for up to 16384.
// Rows of a multiple of 8 elements (WHOLE) have kernels without the code for a
// last lane's part of 8, which is most of the others' code.
constexpr int kMostCols = kThreads * kChunk * 8;  // of a row in registers

template <typename F>
inline void by_shape(int64_t cols, F f) {
#define ZF_SHAPE(G, V, WHOLE) \
  f(std::integral_constant<int, G>(), std::integral_constant<int, V>(), std::bool_constant<WHOLE>())
  if (cols % kChunk != 0) {
    if (cols <= 128) ZF_SHAPE(16, 1, false);
    else if (cols <= 2048) ZF_SHAPE(64, 4, false);
    else ZF_SHAPE(256, 8, false);
  } else if (cols <= 128) ZF_SHAPE(16, 1, true);
  else if (cols <= 512) ZF_SHAPE(64, 1, true);
  else if (cols <= 1024) ZF_SHAPE(64, 2, true);
  else if (cols <= 2048) ZF_SHAPE(64, 4, true);
  else if (cols <= 4096) ZF_SHAPE(256, 2, true);
  else if (cols <= 8192) ZF_SHAPE(256, 4, true);
  else ZF_SHAPE(256, 8, true);
#undef ZF_SHAPE
}

template <typename F>
inline void by_dtype(int32_t dt, F f) {
  if (dt == ZF_F32) f(std::integral_constant<int, ZF_F32>());
  else if (dt == ZF_BF16) f(std::integral_constant<int, ZF_BF16>());
  else f(std::integral_constant<int, ZF_F16>());
}

template <typename F>
inline void by_flags(bool a, bool b, F f) {
  if (a && b) f(std::true_type(), std::true_type());
  else if (a) f(std::true_type(), std::false_type());
  else if (b) f(std::false_type(), std::true_type());
  else f(std::false_type(), std::false_type());
}

}  // namespace dev
}  // namespace zf
