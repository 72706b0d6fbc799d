// zf_norm.h -- what the norms' forward and backward passes share: sums over a
// row's lanes, and the choice of a kernel by a row's length.
#pragma once
#include <type_traits>

#include "zf_rows.h"

namespace zf {
namespace dev {

// N sums over the G lanes of a row in a block of T threads; every lane gets
// them.  G == T: `slots` alternates between two sets, so one barrier is enough.
template <int G, int T, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float (*slots)[N][T / 64], int& turn) {
  static_assert(G <= 64 || G == T, "lanes of a row");
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = sum_lanes<(G < 64 ? G : 64)>(x[k]);
  if constexpr (G > 64) {
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) slots[turn][k][threadIdx.x >> 6] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      x[k] = slots[turn][k][0];
#pragma unroll
      for (int w = 1; w < T / 64; ++w) x[k] += slots[turn][k][w];
    }
  }
}
template <int G, int T>
__device__ __forceinline__ float row_sum(float x, float (*slots)[1][T / 64], int& turn) {
  float one[1] = {x};
  row_sums<G, T, 1>(one, slots, turn);
  return one[0];
}

constexpr int64_t kMostCols = 16384;  // of a row in registers

// The form of a row's kernel: T threads a block, G lanes a row, V times 8
// elements a lane.  Rows of a multiple of 8 elements (WHOLE) have kernels
// without the code for a part of 8, which is most of the others' code (rows of
// 2048, a wave each: 115 us with it, 77 without); other rows have fewer forms.
template <int T_, int G_, int V_, bool WHOLE_>
struct Shape {
  static constexpr int T = T_, G = G_, V = V_;
  static constexpr bool WHOLE = WHOLE_;
};
// 512 threads with 16 elements a lane for rows of 4104 to 8192: 67M bf16 elements in
// rows of 5120 and 8192 57 and 47 us, 1024 threads 93 and 70.
template <typename F>
inline void by_shape(int64_t cols, F f) {
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
  else if (cols <= 8192) f(Shape<512, 512, 2, true>());
  else f(Shape<1024, 1024, 2, true>());
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
