// zf_weight_grad.hip -- a Linear's weight gradient from its input's 8-bit
// checkpoint: grad[o][i] = sum over tokens t of dy[t][o] x[t][i].
//
// x's numbers are e4m3 times a power of two, which 16-bit floats hold exactly,
// so the product runs on the 16-bit matrix instructions: codes become 16-bit
// numbers on their way to shared memory, one conversion instruction for two of
// them with their scale.  Products are exact and sums binary32.
//
// Both operands run along their columns in memory while the matrix
// instructions sum over tokens, so fragments are transposed on their way out
// of shared memory (ds_read_b64_tr_b16).  Where the tiles of the result are
// too few to fill the GPU, the tokens are split over blocks, whose partial
// results a second launch adds in order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "zf_hip_status.h"
#include "zf_rows.h"

namespace {

using namespace zf::dev;
using zf::hip_ok;
using zf::kThreads;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
#define ZF_LDS __attribute__((address_space(3)))

constexpr int kBK = 64;  // tokens a step

template <int BM_, int BN_, int WI, int WJ>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, kThreads = WI * WJ * 64, kWavesJ = WJ;
  static constexpr int TI = BM / WI, TJ = BN / WJ, FI = TI / 16, FJ = TJ / 16;
  static constexpr int kPBytes = kBK * BM * 2, kQBytes = kBK * BN * 2;
  static constexpr int kPPieces = kBK * BM / 8 / kThreads;   // of 8 gradients a thread
  static constexpr int kQPieces = kBK * BN / 16 / kThreads;  // of 16 codes a thread
};
typedef Tile<128, 128, 2, 2> Middle;

struct GradArgs {
  const void* dy;
  Act8 x;
  void* grad;
  float* partial;  // [splits][out][in], or NULL: one split
  int64_t dy_ld, rows, split_rows;
  int32_t out, in, tiles_in, tiles, splits, gdt, accumulate;
};

// The place of a 16-byte piece of a row in shared memory: pairs of pieces are
// permuted by the row, so that the 16 rows that an instruction reads lie in
// different banks.  Rows 4 apart (and 32) are permuted alike.
template <int PIECES>
__device__ __forceinline__ int place(int row, int piece) {
  const int turn = ((row & 3) | ((row >> 1) & 4)) & (PIECES / 2 - 1);
  return (row * PIECES + (piece ^ (2 * turn))) * 16;
}

// Two codes with their scale as 16-bit numbers of type DT.
template <int DT, bool HIGH>
__device__ __forceinline__ uint32_t decode2(uint32_t codes, float scale) {
  if constexpr (DT == ZF_BF16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, HIGH));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, HIGH));
}

template <int DT>
__device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c) {
  if constexpr (DT == ZF_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// 8 tokens from k0 + 8 (lane / 16) on of column c0 + lane % 16.
template <int PIECES>
__device__ __forceinline__ s16x8 fragment(const char* tile, int k0, int c0) {
  const int lane = threadIdx.x & 63, l = lane & 15, row = k0 + 8 * (lane >> 4) + (l >> 2);
  s16x4 half[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    half[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (ZF_LDS s16x4*)((const ZF_LDS char*)tile + place<PIECES>(row + 4 * e, c0 / 8 + ((l & 3) >> 1)) +
                        (l & 1) * 8));
  return __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7);
}

template <typename T, int DT>
__global__ __launch_bounds__(T::kThreads) void zf_weight_grad_kernel(GradArgs a) {
  __shared__ __align__(16) char shared[T::kPBytes + T::kQBytes];
  const int tid = threadIdx.x;
  const int tile = blockIdx.x % a.tiles, split = blockIdx.x / a.tiles;
  const int i0 = tile / a.tiles_in * T::BM, j0 = tile % a.tiles_in * T::BN;
  const int64_t first = split * a.split_rows, end = min(first + a.split_rows, a.rows);
  const int wave = tid >> 6, wi = wave / T::kWavesJ * T::TI, wj = wave % T::kWavesJ * T::TJ;

  u32x4 p[T::kPPieces], q[T::kQPieces];
  float scale[T::kQPieces];
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int h = 0; h < T::kPPieces; ++h) {
      const int k = h * T::kThreads + tid, c = i0 + k % (T::BM / 8) * 8;
      const int64_t t = t0 + k / (T::BM / 8);
      p[h] = (u32x4){0, 0, 0, 0};
      if (t < end && c < a.out) p[h] = load_raw<ZF_BF16>(a.dy, t * a.dy_ld + c, a.out - c).w[0];
    }
#pragma unroll
    for (int h = 0; h < T::kQPieces; ++h) {
      const int k = h * T::kThreads + tid, c = j0 + k % (T::BN / 16) * 16;
      const int64_t t = t0 + k / (T::BN / 16);
      q[h] = (u32x4){0, 0, 0, 0};
      scale[h] = 1;
      if (t >= end || c >= a.in) continue;
      const uint8_t* from = a.x.codes + t * a.x.code_ld + c;
      if (c + 16 <= a.in) {
        q[h] = load_any<false, u32x4_any>(from);
      } else {
        const u32x2 lo = load_codes(from, min(8, a.in - c));
        const u32x2 hi = c + 8 < a.in ? load_codes(from + 8, a.in - c - 8) : (u32x2){0, 0};
        q[h] = (u32x4){lo.x, lo.y, hi.x, hi.y};
      }
      scale[h] = __uint_as_float((uint32_t)a.x.scales[t * a.x.scale_ld + c / ZF_ACT8_GROUP] << 23);
    }
  };
  auto put = [&]() {
#pragma unroll
    for (int h = 0; h < T::kPPieces; ++h) {
      const int k = h * T::kThreads + tid;
      *reinterpret_cast<u32x4*>(shared + place<T::BM / 8>(k / (T::BM / 8), k % (T::BM / 8))) = p[h];
    }
#pragma unroll
    for (int h = 0; h < T::kQPieces; ++h) {
      const int k = h * T::kThreads + tid, row = k / (T::BN / 16), piece = k % (T::BN / 16) * 2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const u32x4 x = {decode2<DT, false>(q[h][e * 2], scale[h]), decode2<DT, true>(q[h][e * 2], scale[h]),
                         decode2<DT, false>(q[h][e * 2 + 1], scale[h]),
                         decode2<DT, true>(q[h][e * 2 + 1], scale[h])};
        *reinterpret_cast<u32x4*>(shared + T::kPBytes + place<T::BN / 8>(row, piece + e)) = x;
      }
    }
  };

  f32x4 acc[T::FI][T::FJ];
#pragma unroll
  for (int i = 0; i < T::FI; ++i)
#pragma unroll
    for (int j = 0; j < T::FJ; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
  if (first < end) fetch(first);
  for (int64_t t = first; t < end; t += kBK) {
    __syncthreads();
    put();
    __syncthreads();
    if (t + kBK < end) fetch(t + kBK);
#pragma unroll
    for (int k = 0; k < kBK; k += 32) {
      s16x8 fp[T::FI], fq[T::FJ];
#pragma unroll
      for (int i = 0; i < T::FI; ++i) fp[i] = fragment<T::BM / 8>(shared, k, wi + i * 16);
#pragma unroll
      for (int j = 0; j < T::FJ; ++j) fq[j] = fragment<T::BN / 8>(shared + T::kPBytes, k, wj + j * 16);
#pragma unroll
      for (int i = 0; i < T::FI; ++i)
#pragma unroll
        for (int j = 0; j < T::FJ; ++j) acc[i][j] = mma<DT>(fq[j], fp[i], acc[i][j]);
    }
  }

  // acc[i][j][r]: row l, columns 4 g + r of a 16 x 16 square
  const int lane = tid & 63, l = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < T::FI; ++i)
#pragma unroll
    for (int j = 0; j < T::FJ; ++j) {
      const int o = i0 + wi + i * 16 + l, c = j0 + wj + j * 16 + g * 4;
      if (o >= a.out) continue;
      const int64_t at = (int64_t)o * a.in + c;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (c + r >= a.in) break;
        float v = acc[i][j][r];
        if (a.partial) {
          a.partial[(int64_t)split * a.out * a.in + at + r] = v;
        } else {
          if (a.accumulate) v += load1_of(a.gdt, a.grad, at + r);
          store1_of(a.gdt, a.grad, at + r, v);
        }
      }
    }
}

// Adds the splits' partial results in order.
struct JoinArgs {
  const float* partial;
  void* grad;
  int64_t size;
  int32_t splits, gdt, accumulate;
};
__global__ __launch_bounds__(kThreads) void zf_weight_grad_join(JoinArgs a) {
  const int64_t step = (int64_t)gridDim.x * kThreads * kChunk;
  for (int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kChunk; e < a.size; e += step) {
    const int n = (int)min((int64_t)kChunk, a.size - e);
    float sum[kChunk], x[kChunk];
#pragma unroll
    for (int k = 0; k < kChunk; ++k) sum[k] = 0;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      load8<ZF_F32>(a.partial + s * a.size, e, n, x);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) sum[k] += x[k];
    }
    if (a.accumulate) {
      load8_of(a.gdt, a.grad, e, n, x);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) sum[k] += x[k];
    }
    if (a.gdt == ZF_F32) store8<ZF_F32>(a.grad, e, n, sum);
    else if (a.gdt == ZF_BF16) store8<ZF_BF16>(a.grad, e, n, sum);
    else store8<ZF_F16>(a.grad, e, n, sum);
  }
}

struct Plan {
  int32_t tiles_out, tiles_in, splits;
  int64_t split_rows, bytes;
};

int plan(int64_t rows, int64_t out, int64_t in, Plan& g) {
  int rc = shape_ok(rows, in);
  if (rc == ZF_OK) rc = shape_ok(0, out);
  if (rc != ZF_OK) return rc;
  typedef Middle T;
  const int64_t tiles_out = (out + T::BM - 1) / T::BM, tiles_in = (in + T::BN - 1) / T::BN;
  const int64_t tiles = tiles_out * tiles_in, steps = (rows + kBK - 1) / kBK;
  if (tiles > kMaxBlocks) return ZF_ESIZE;
  // blocks for two rounds of the compute units, of 4 steps at least
  int64_t splits = std::min((512 + tiles - 1) / tiles, (steps + 3) / 4);
  splits = std::max<int64_t>(splits, 1);
  const int64_t per = std::max<int64_t>((steps + splits - 1) / splits, 1);
  g.tiles_out = (int32_t)tiles_out;
  g.tiles_in = (int32_t)tiles_in;
  g.split_rows = per * kBK;
  g.splits = (int32_t)std::max<int64_t>((steps + per - 1) / per, 1);
  g.bytes = g.splits > 1 ? (g.splits * out * in * 4 + 15) / 16 * 16 : 0;
  return ZF_OK;
}

}  // namespace

extern "C" int64_t zf_weight_grad_bytes(int64_t rows, int64_t out_features, int64_t in_features) {
  Plan g;
  const int rc = plan(rows, out_features, in_features, g);
  return rc != ZF_OK ? rc : g.bytes;
}

extern "C" int zf_weight_grad(const zf_weight_grad_args* args, void* stream) {
  if (!args || args->reserved != 0 || !flag(args->accumulate)) return ZF_EINVAL;
  const zf_weight_grad_args& p = *args;
  if (!valid_dtype(p.dtype) || !row_dtype(p.grad_dtype)) return ZF_EDTYPE;
  Plan g;
  int rc = plan(p.rows, p.out_features, p.in_features, g);
  if (rc == ZF_OK) rc = rows_ok(p.dy, p.dtype, p.rows, p.out_features, p.dy_stride);
  if (rc == ZF_OK) rc = act8_ok(p.x8, p.rows, p.in_features);
  if (rc != ZF_OK) return rc;
  if (!p.grad || (g.bytes > 0 && !p.workspace)) return ZF_EINVAL;
  if (!aligned_to(p.grad, p.grad_dtype) || !aligned16(p.workspace)) return ZF_EALIGN;
  if (p.workspace_size < g.bytes) return ZF_ESIZE;
  if (p.rows == 0 && p.accumulate) return ZF_OK;
  GradArgs a;
  a.dy = p.dy;
  a.x = act8_of(p.x8);
  a.grad = p.grad;
  a.partial = g.splits > 1 ? static_cast<float*>(p.workspace) : nullptr;
  a.dy_ld = p.dy_stride;
  a.rows = p.rows;
  a.split_rows = g.split_rows;
  a.out = (int32_t)p.out_features;
  a.in = (int32_t)p.in_features;
  a.tiles_in = g.tiles_in;
  a.tiles = g.tiles_out * g.tiles_in;
  a.splits = g.splits;
  a.gdt = p.grad_dtype;
  a.accumulate = p.accumulate;
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const dim3 grid((uint32_t)a.tiles * (uint32_t)g.splits);
  if (p.dtype == ZF_BF16)
    hipLaunchKernelGGL((zf_weight_grad_kernel<Middle, ZF_BF16>), grid, dim3(Middle::kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((zf_weight_grad_kernel<Middle, ZF_F16>), grid, dim3(Middle::kThreads), 0, s, a);
  if (g.splits > 1) {
    const JoinArgs j{a.partial, p.grad, p.out_features * p.in_features, g.splits, p.grad_dtype,
                     p.accumulate};
    const int64_t blocks = (j.size + kThreads * kChunk - 1) / (kThreads * kChunk);
    hipLaunchKernelGGL(zf_weight_grad_join, dim3((uint32_t)std::min<int64_t>(blocks, kMaxBlocks)),
                       dim3(kThreads), 0, s, j);
  }
  return hip_ok(hipGetLastError()) ? ZF_OK : ZF_EHIP;
}
