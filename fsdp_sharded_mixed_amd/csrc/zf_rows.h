// zf_rows.h -- pieces shared by the kernels that work on rows of activations
// (norms, checkpoints, embedding, weight gradients): 8 elements a lane at any
// alignment, the 8-bit checkpoint's codes and scales, reductions over lanes.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "zf_device.h"
#include "zf_internal.h"

namespace zf {
namespace dev {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Wide accesses at any element's address: rows of activations and parameters
// inside a flat buffer keep their element's alignment only.  gfx950 takes
// global loads and stores of 8 and 16 bytes there (unaligned access mode,
// which the HSA runtime sets), so there is one path, not one an alignment.
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

constexpr int kChunk = 8;  // consecutive elements of a lane
// Blocks of a launch along x: a launch holds fewer than 2^32 threads there,
// so kernels walk further rows in steps of the grid.
constexpr int64_t kMaxBlocks = 1 << 22;

template <int DT>
constexpr int kElem = DT == ZF_F32 ? 4 : 2;

inline int elem_bytes(int32_t dt) { return dt == ZF_F32 ? 4 : 2; }

template <bool NT, typename V>
__device__ __forceinline__ V load_any(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load(static_cast<const V*>(p));
  else return *static_cast<const V*>(p);
}
template <bool NT, typename V>
__device__ __forceinline__ void store_any(void* p, V x) {
  if constexpr (NT) __builtin_nontemporal_store(x, static_cast<V*>(p));
  else *static_cast<V*>(p) = x;
}

template <int DT>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
  if constexpr (DT == ZF_F32) return static_cast<const float*>(base)[i];
  else return widen1<DT>(static_cast<const uint16_t*>(base)[i]);
}
// A binary32 value about to be rounded to fp16.  The compiler otherwise joins
// a product and its rounding into one v_fma_mixlo_f16, which skips binary32's
// rounding: results would depend on which code it joins.
__device__ __forceinline__ float settled(float x) {
  asm("" : "+v"(x));
  return x;
}
template <int DT>
__device__ __forceinline__ uint16_t narrow(float x) {
  return narrow1<DT>(DT == ZF_F16 ? settled(x) : x);
}
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if constexpr (DT == ZF_BF16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
  else
    return (uint32_t)narrow<DT>(a) | (uint32_t)narrow<DT>(b) << 16;
}
template <int DT>
__device__ __forceinline__ void store1(void* base, int64_t i, float x) {
  if constexpr (DT == ZF_F32) static_cast<float*>(base)[i] = x;
  else static_cast<uint16_t*>(base)[i] = narrow<DT>(x);
}

// 8 elements of type DT from element i on as the registers hold them; n of
// them exist (all, if 8 or more; none, if 0 or less), the others read as zero.
// WHOLE: all or none exist, as in rows of a multiple of 8 elements.
template <int DT>
struct Raw {
  u32x4 w[DT == ZF_F32 ? 2 : 1];
};
template <int DT, bool NT = false, bool WHOLE = false>
__device__ __forceinline__ Raw<DT> load_raw(const void* base, int64_t i, int n) {
  const char* p = static_cast<const char*>(base) + i * kElem<DT>;
  Raw<DT> r;
  if (n >= kChunk) {
    r.w[0] = load_any<NT, u32x4_any>(p);
    if constexpr (DT == ZF_F32) r.w[1] = load_any<NT, u32x4_any>(p + 16);
    return r;
  }
  r.w[0] = (u32x4){0, 0, 0, 0};
  if constexpr (DT == ZF_F32) r.w[1] = (u32x4){0, 0, 0, 0};
  if (WHOLE || n <= 0) return r;
  // 4, 2 and 1 of them, as the bits of n say
  if constexpr (DT == ZF_F32) {
    u32x2 two = {0, 0};
    uint32_t one = 0;
    if (n & 4) r.w[0] = load_any<NT, u32x4_any>(p);
    if (n & 2) two = load_any<NT, u32x2_any>(p + (n & 4) * 4);
    if (n & 1) one = load_any<NT, uint32_t>(p + (n & 6) * 4);
    const u32x4 rest = n & 2 ? (u32x4){two.x, two.y, one, 0} : (u32x4){one, 0, 0, 0};
    if (n & 4) r.w[1] = rest;
    else r.w[0] = rest;
  } else {
    u32x2 four = {0, 0};
    uint32_t two = 0, one = 0;
    if (n & 4) four = load_any<NT, u32x2_any>(p);
    if (n & 2) two = load_any<NT, u32_any>(p + (n & 4) * 2);
    if (n & 1) one = load_any<NT, uint16_t>(p + (n & 6) * 2);
    const u32x2 rest = n & 2 ? (u32x2){two, one} : (u32x2){one, 0};
    r.w[0] = n & 4 ? (u32x4){four.x, four.y, rest.x, rest.y} : (u32x4){rest.x, rest.y, 0, 0};
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void widen8(const Raw<DT>& r, float (&v)[kChunk]) {
#pragma unroll
  for (int k = 0; k < kChunk; ++k) {
    if constexpr (DT == ZF_F32) v[k] = __uint_as_float(r.w[k >> 2][k & 3]);
    else v[k] = (k & 1) ? hi16<DT>(r.w[0][k >> 1]) : lo16<DT>(r.w[0][k >> 1]);
  }
}
template <int DT>
__device__ __forceinline__ Raw<DT> narrow8(const float (&v)[kChunk]) {
  Raw<DT> r;
#pragma unroll
  for (int k = 0; k < kChunk; k += 2) {
    if constexpr (DT == ZF_F32) {
      r.w[k >> 2][k & 3] = __float_as_uint(v[k]);
      r.w[k >> 2][(k & 3) + 1] = __float_as_uint(v[k + 1]);
    } else {
      r.w[0][k >> 1] = narrow2<DT>(v[k], v[k + 1]);
    }
  }
  return r;
}
template <int DT, bool NT = false, bool WHOLE = false>
__device__ __forceinline__ void store_raw(void* base, int64_t i, int n, const Raw<DT>& r) {
  char* p = static_cast<char*>(base) + i * kElem<DT>;
  if (n >= kChunk) {
    store_any<NT, u32x4_any>(p, r.w[0]);
    if constexpr (DT == ZF_F32) store_any<NT, u32x4_any>(p + 16, r.w[1]);
    return;
  }
  if (WHOLE || n <= 0) return;
  if constexpr (DT == ZF_F32) {
    const u32x4 rest = n & 4 ? r.w[1] : r.w[0];
    if (n & 4) store_any<NT, u32x4_any>(p, r.w[0]);
    if (n & 2) store_any<NT, u32x2_any>(p + (n & 4) * 4, (u32x2){rest.x, rest.y});
    if (n & 1) store_any<NT, uint32_t>(p + (n & 6) * 4, n & 2 ? rest.z : rest.x);
  } else {
    const u32x2 rest = n & 4 ? (u32x2){r.w[0].z, r.w[0].w} : (u32x2){r.w[0].x, r.w[0].y};
    if (n & 4) store_any<NT, u32x2_any>(p, (u32x2){r.w[0].x, r.w[0].y});
    if (n & 2) store_any<NT, u32_any>(p + (n & 4) * 2, rest.x);
    if (n & 1) store_any<NT, uint16_t>(p + (n & 6) * 2, (uint16_t)(n & 2 ? rest.y : rest.x));
  }
}
template <int DT, bool NT = false, bool WHOLE = false>
__device__ __forceinline__ void load8(const void* base, int64_t i, int n, float (&v)[kChunk]) {
  widen8<DT>(load_raw<DT, NT, WHOLE>(base, i, n), v);
}
template <int DT, bool NT = false, bool WHOLE = false>
__device__ __forceinline__ void store8(void* base, int64_t i, int n, const float (&v)[kChunk]) {
  store_raw<DT, NT, WHOLE>(base, i, n, narrow8<DT>(v));
}

// The same with the type known at run time (parameters: once a row or less).
template <bool WHOLE = false>
__device__ __forceinline__ void load8_of(int32_t dt, const void* base, int64_t i, int n,
                                         float (&v)[kChunk]) {
  if (dt == ZF_F32) load8<ZF_F32, false, WHOLE>(base, i, n, v);
  else if (dt == ZF_BF16) load8<ZF_BF16, false, WHOLE>(base, i, n, v);
  else load8<ZF_F16, false, WHOLE>(base, i, n, v);
}
__device__ __forceinline__ float load1_of(int32_t dt, const void* base, int64_t i) {
  return dt == ZF_F32 ? load1<ZF_F32>(base, i)
                      : dt == ZF_BF16 ? load1<ZF_BF16>(base, i) : load1<ZF_F16>(base, i);
}
__device__ __forceinline__ void store1_of(int32_t dt, void* base, int64_t i, float x) {
  if (dt == ZF_F32) store1<ZF_F32>(base, i, x);
  else if (dt == ZF_BF16) store1<ZF_BF16>(base, i, x);
  else store1<ZF_F16>(base, i, x);
}

// ---------------------------------------------------------------------------
// The checkpoint's numbers.  A group of 32 elements lies in 4 neighbouring
// lanes of 8.  Scales are powers of two, so x / 2^k and code * 2^k are exact
// (but for what underflows far below e4m3's least step) and the only rounding
// is the conversion's, to nearest even.

constexpr int kScaleLeast = 27;  // k = -100: every number stays normal in bf16

// A condition that hardly any wave meets: a branch around its code, instead of
// both sides and selects.
__device__ __forceinline__ bool rare(bool x) { return __builtin_expect(__any(x), 0) && x; }

// Magnitude bits of 8 elements' largest; FINITE: without infinities and NaN.
template <bool FINITE>
__device__ __forceinline__ uint32_t amax8(const float (&v)[kChunk]) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kChunk; ++k) {
    const uint32_t a = __float_as_uint(v[k]) & 0x7FFFFFFFu;
    m = max(m, FINITE && a >= 0x7F800000u ? 0u : a);
  }
  return m;
}
// The largest over each 4 neighbouring lanes (quad_perm 1 0 3 2 and 2 3 0 1).
__device__ __forceinline__ uint32_t max_quad(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));
}
// The scale's byte: k + 127 with k the least integer from -100 on for which
// the magnitude is at most 448 2^k = 1.75 * 2^(k + 8).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int b = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(b, kScaleLeast);
}
// 8 codes of finite elements with their group's scale.  At the largest scale
// of the type DT (f16 k = 8, else 120) the magnitudes end below 256 2^k, which
// the type does not hold: codes end at 240 there.
template <int DT>
__device__ __forceinline__ u32x2 encode8(const float (&v)[kChunk], uint32_t scale) {
  const float inv = __uint_as_float((254u - scale) << 23);
  float s[kChunk];
#pragma unroll
  for (int k = 0; k < kChunk; ++k) s[k] = v[k] * inv;
  if (rare(scale == (DT == ZF_F16 ? 135u : 247u))) {
#pragma unroll
    for (int k = 0; k < kChunk; ++k) s[k] = fminf(fmaxf(s[k], -240.0f), 240.0f);
  }
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(s[h * 4], s[h * 4 + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(s[h * 4 + 2], s[h * 4 + 3], w, true);
    c[h] = (uint32_t)w;
  }
  return c;
}
__device__ __forceinline__ void decode8(u32x2 c, uint32_t scale, float (&v)[kChunk]) {
  const float s = __uint_as_float(scale << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[h], s, false);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[h], s, true);
    v[h * 4] = a.x;
    v[h * 4 + 1] = a.y;
    v[h * 4 + 2] = b.x;
    v[h * 4 + 3] = b.y;
  }
}

struct Act8 {
  uint8_t* codes;
  uint8_t* scales;
  int64_t code_ld, scale_ld;
};

// 8 codes, of which n exist, as load_raw and store_raw take elements.
template <bool NT = false, bool WHOLE = false>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int n) {
  if (n >= kChunk) return load_any<NT, u32x2_any>(p);
  uint32_t four = 0, two = 0, one = 0;
  if (WHOLE || n <= 0) return (u32x2){0, 0};
  if (n & 4) four = load_any<NT, u32_any>(p);
  if (n & 2) two = load_any<NT, u16_any>(p + (n & 4));
  if (n & 1) one = load_any<NT, uint8_t>(p + (n & 6));
  const uint32_t rest = n & 2 ? two | one << 16 : one;
  return n & 4 ? (u32x2){four, rest} : (u32x2){rest, 0};
}
template <bool NT = false, bool WHOLE = false>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, u32x2 c) {
  if (n >= kChunk) {
    store_any<NT, u32x2_any>(p, c);
    return;
  }
  if (WHOLE || n <= 0) return;
  const uint32_t rest = n & 4 ? c.y : c.x;
  if (n & 4) store_any<NT, u32_any>(p, c.x);
  if (n & 2) store_any<NT, u16_any>(p + (n & 4), (uint16_t)rest);
  if (n & 1) store_any<NT, uint8_t>(p + (n & 6), (uint8_t)(n & 2 ? rest >> 16 : rest));
}

// Keeps this lane's 8 elements of row i from column j on, of which n exist;
// the others are zero.  All 4 lanes of a group call it together.
template <int DT, bool NT = false, bool WHOLE = false>
__device__ __forceinline__ void keep8(const Act8& a, int64_t i, int64_t j, int n,
                                      const float (&v)[kChunk]) {
  uint32_t top = amax8<false>(v);
  const bool odd = top >= 0x7F800000u;  // infinities or NaN among them
  if (rare(odd)) top = amax8<true>(v);
  const uint32_t scale = scale_byte(max_quad(top));
  if (n <= 0) return;
  u32x2 c = encode8<DT>(v, scale);
  if (rare(odd)) {
#pragma unroll
    for (int k = 0; k < kChunk; ++k)
      if (nonfinite(v[k])) c[k >> 2] = (c[k >> 2] & ~(0xFFu << (k & 3) * 8)) | 0x7Fu << (k & 3) * 8;
  }
  store_codes<NT, WHOLE>(a.codes + i * a.code_ld + j, n, c);
  if ((j & (ZF_ACT8_GROUP - 1)) == 0)
    a.scales[i * a.scale_ld + j / ZF_ACT8_GROUP] = (uint8_t)scale;
}

// ---------------------------------------------------------------------------
// Sums over G neighbouring lanes (16 or 64; every lane ends with the same
// bits).

template <int CTRL>
__device__ __forceinline__ float add_dpp(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
// By lane permutations of the vector unit alone: quads, the mirrored half of 8
// and of 16 lanes, then rows of 16 and halves of the wave swapped between two
// copies.  (Through shared memory, as __shfl_xor goes, a sum waits six times.)
template <int G>
__device__ __forceinline__ float sum_lanes(float x) {
  static_assert(G == 16 || G == 64, "a row of lanes or a wave");
  x = add_dpp<0xB1>(x);   // quad_perm 1 0 3 2
  x = add_dpp<0x4E>(x);   // quad_perm 2 3 0 1
  x = add_dpp<0x141>(x);  // row_half_mirror
  x = add_dpp<0x140>(x);  // row_mirror
  if constexpr (G == 64) {
    const uint32_t u = __float_as_uint(x);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const uint32_t w = __float_as_uint(x);
    const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    x = __uint_as_float(q[0]) + __uint_as_float(q[1]);
  }
  return x;
}

// ---------------------------------------------------------------------------
// Argument checks.

inline bool row_dtype(int32_t d) { return d == ZF_F16 || d == ZF_BF16 || d == ZF_F32; }
inline bool aligned_to(const void* p, int32_t dt) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(elem_bytes(dt) - 1)) == 0;
}
inline bool flag(int32_t f) { return f == 0 || f == 1; }

// A row-major matrix: rows in [0, ZF_MAX_ROWS], cols in [1, ZF_MAX_COLS].
inline int shape_ok(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return ZF_EINVAL;
  return rows > ZF_MAX_ROWS || cols > ZF_MAX_COLS ? ZF_ESIZE : ZF_OK;
}
// Its rows; a stride's product with the rows must fit an offset in bytes.
inline int rows_ok(const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t stride) {
  if (rows > 1 && stride < cols) return ZF_EINVAL;
  if (rows > 0 && !p) return ZF_EINVAL;
  if (!aligned_to(p, dt)) return ZF_EALIGN;
  if (rows > 1 && stride > ZF_MAX_STRIDE) return ZF_ESIZE;
  return ZF_OK;
}
inline int act8_ok(const zf_act8* a, int64_t rows, int64_t cols) {
  if (!a || a->rows != rows || a->cols != cols) return ZF_EINVAL;
  const int64_t groups = (cols + ZF_ACT8_GROUP - 1) / ZF_ACT8_GROUP;
  if (rows > 0 && (!a->codes || !a->scales)) return ZF_EINVAL;
  if (rows > 1 && (a->code_stride < cols || a->scale_stride < groups)) return ZF_EINVAL;
  if (rows > 1 && (a->code_stride > ZF_MAX_STRIDE || a->scale_stride > ZF_MAX_STRIDE)) return ZF_ESIZE;
  return ZF_OK;
}
inline Act8 act8_of(const zf_act8* a) {
  if (!a) return Act8{nullptr, nullptr, 0, 0};
  return Act8{static_cast<uint8_t*>(a->codes), static_cast<uint8_t*>(a->scales), a->code_stride,
              a->scale_stride};
}

}  // namespace dev
}  // namespace zf
