// zf_ortho.hip -- orthogonalisation of a batch of matrices by Newton-Schulz
// products (the update of the Muon optimizer), and its C entry points.
//
// Mathematics.  For G (R x C), m = min(R, C), n = max(R, C):
//   X = G / (|G|_F + eps)          (transposed if R > C, so X is m x n)
//   A = X X^T;  B = b A + c A A;  X <- a X + B X         `steps` times.
// Each step maps every singular value s of X to a s + b s^3 + c s^5 and
// keeps the singular vectors; the coefficients drive (0, 1] towards 1.
//
// Precision.  The products run on the matrix cores with fp16 operands and
// fp32 sums.  fp16 holds 11 bits where bf16 holds 8, at the same rate; the
// operands are multiplied by 2^10 first, because the elements of a
// normalised m x n matrix are near 1/sqrt(m n), which nears fp16's smallest
// normal number (2^-14) at 16K x 16K, and none passes 64 = 65536 / 2^10 for
// coefficients that keep the singular values below that.  Three parts of the
// iteration stay in 32 bits, because rounding them is what costs accuracy:
//   - the linear term a X (its rounding would drown small singular values);
//   - the diagonal of A and of B (B's is near -2.7 once the singular values
//     near 1, where the rest of a row is near 1/sqrt(m): half a step of fp16
//     there is 1e-3), so a product of two such matrices S = diag(D) + O is
//     O O + (D_i + D_j) O_ij + D_i^2 on the diagonal.
// Measured in |.|_F against 64 bits over flat, low-rank-plus-noise and 1/i
// spectra: 3e-4 to 9e-4 (all three parts in fp16: 3e-4 to 4e-3; bf16
// throughout: 1e-2 to 3e-2).  A result in more bits than bf16 gets three
// products instead of one: every operand is the sum of two fp16 numbers,
// hi + lo * 2^-11, and hi hi + hi lo + lo hi holds about 22 bits.
#include "zf_ortho.h"

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "zf_device.h"
#include "zf_hip_status.h"

namespace {

using namespace zf::dev;
using zf::DevState;
using zf::hip_ok;
using zf::kThreads;
using zf::ns::Group;
using zf::ns::kPad;
using zf::ns::Layout;
using zf::ns::Mat;
using zf::ns::MuonIo;

typedef _Float16 f16;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr float kScale = 1024.0f;           // of every 16-bit operand
constexpr float kUnscale2 = 1.0f / (1024.0f * 1024.0f);
constexpr float kLo = 2048.0f;              // lo halves: 2^11 more

// hi and lo halves of x.
__device__ __forceinline__ f16 hi_of(float x) { return (f16)(x * kScale); }
__device__ __forceinline__ f16 lo_of(float x, f16 hi) {
  return (f16)((x * kScale - (float)hi) * kLo);
}
__device__ __forceinline__ float value_of(f16 hi, f16 lo) {
  return ((float)hi + (float)lo * (1.0f / kLo)) * (1.0f / kScale);
}

// ---------------------------------------------------------------------------
// The table of matrices travels by value, a chunk a launch, into the
// workspace, so that a captured call carries it.
constexpr int kTableChunk = 16;
struct TableArgs {
  Mat* to;
  int32_t count;
  Mat m[kTableChunk];
};

__global__ __launch_bounds__(64) void zf_ns_table(TableArgs a) {
  static_assert(sizeof(Mat) % 8 == 0, "copied in words");
  const uint64_t* s = reinterpret_cast<const uint64_t*>(a.m);
  uint64_t* d = reinterpret_cast<uint64_t*>(a.to);
  for (int i = threadIdx.x; i < a.count * (int)(sizeof(Mat) / 8); i += 64) d[i] = s[i];
}

// The matrix whose blocks hold block b: the last one that starts at or
// before it.
template <int32_t Mat::*FIRST>
__device__ __forceinline__ const Mat* find(const Mat* table, int count, int b) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table[mid].*FIRST <= b) lo = mid;
    else hi = mid - 1;
  }
  return table + lo;
}

struct Common {
  char* ws;
  const Mat* table;       // the group's matrices
  int32_t count;
  const DevState* st;     // the Muon step's skip flag, or NULL
  double* inv;            // 1 / (|G|_F + eps), by slot
  double* partials;       // squared-norm partials
};

template <typename T>
__device__ __forceinline__ T* at(const Common& c, int64_t offset) {
  return reinterpret_cast<T*>(c.ws + offset);
}

// ---------------------------------------------------------------------------
// Load: the matrix (or the Muon step's momentum update) into X in 32 bits,
// with zero padding, and one squared-norm partial (64 bits) per 64 x 64 tile.
constexpr int kTile = 64;

struct LoadArgs {
  Common c;
  MuonIo io;
};

template <int SRC>  // ZF_F16, ZF_BF16, ZF_F32, or 0: the Muon step
__device__ __forceinline__ float load1(const LoadArgs& a, const Mat& m, float gs, int64_t r,
                                       int64_t c) {
  if constexpr (SRC == 0) {
    const int64_t p = m.flat + r * m.src_ld + c;
    const float g = a.io.sums[p] * gs;
    const float mm = a.io.mu * a.io.momentum[p] + g;
    a.io.momentum[p] = mm;
    return a.io.nesterov ? g + a.io.mu * mm : mm;
  } else if constexpr (SRC == ZF_F32) {
    return static_cast<const float*>(m.src)[r * m.src_ld + c];
  } else {
    return widen1<SRC>(static_cast<const uint16_t*>(m.src)[r * m.src_ld + c]);
  }
}

template <int SRC>
__global__ __launch_bounds__(kThreads) void zf_ns_load(LoadArgs a) {
  if (a.c.st && a.c.st->skipped) return;
  const Mat& m = *find<&Mat::load0>(a.c.table, a.c.count, blockIdx.x);
  const int tile = blockIdx.x - m.load0, tiles_n = m.np / kTile;
  const int i0 = tile / tiles_n * kTile, j0 = tile % tiles_n * kTile;
  const float gs = SRC == 0 ? a.c.st->gs : 0.0f;
  __shared__ float s[kTile][kTile + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double ss = 0.0;
#pragma unroll 4
  for (int k = wave; k < kTile; k += kThreads / 64) {
    // a wave reads 64 elements along the source's rows
    const int i = m.tall ? i0 + lane : i0 + k, j = m.tall ? j0 + k : j0 + lane;
    float v = 0.0f;
    if (i < m.m && j < m.n) v = load1<SRC>(a, m, gs, m.tall ? j : i, m.tall ? i : j);
    ss += (double)v * (double)v;
    if (m.tall) s[lane][k] = v;
    else s[k][lane] = v;
  }
  uint32_t unused = 0;
  block_reduce(ss, unused);  // synchronises: the tile is whole
  if (threadIdx.x == 0) a.c.partials[m.part + tile] = ss;
  float* x = at<float>(a.c, m.x);
#pragma unroll 4
  for (int k = wave; k < kTile; k += kThreads / 64)
    x[(int64_t)(i0 + k) * m.np + j0 + lane] = s[k][lane];
}

// The inverse norm of every matrix of the group: its partials in a fixed
// order, one block a matrix.
struct NormArgs {
  Common c;
  double eps;
};

__global__ __launch_bounds__(kThreads) void zf_ns_norm(NormArgs a) {
  if (a.c.st && a.c.st->skipped) return;
  const Mat& m = a.c.table[blockIdx.x];
  const int64_t tiles = (int64_t)(m.mp / kTile) * (m.np / kTile);
  double ss = 0.0;
  for (int64_t i = threadIdx.x; i < tiles; i += kThreads) ss += a.c.partials[m.part + i];
  uint32_t unused = 0;
  block_reduce(ss, unused);
  if (threadIdx.x == 0) a.c.inv[m.slot] = 1.0 / (sqrt(ss) + a.eps);
}

// ---------------------------------------------------------------------------
// The 16-bit operands of the first step from X and the inverse norm.
template <int PRODUCTS>
__global__ __launch_bounds__(kThreads) void zf_ns_prep(Common c) {
  if (c.st && c.st->skipped) return;
  const Mat& m = *find<&Mat::load0>(c.table, c.count, blockIdx.x);
  const int tile = blockIdx.x - m.load0, tiles_n = m.np / kTile;
  const int i0 = tile / tiles_n * kTile, j0 = tile % tiles_n * kTile;
  const double inv = c.inv[m.slot];
  __shared__ float s[kTile][kTile + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float* x = at<float>(c, m.x);
  f16* h = at<f16>(c, m.h);
  f16* t = at<f16>(c, m.t[0]);
  f16* hl = at<f16>(c, m.h + m.lo_x);
  f16* tl = at<f16>(c, m.t[0] + m.lo_x);
#pragma unroll 4
  for (int k = wave; k < kTile; k += kThreads / 64) {
    const int64_t p = (int64_t)(i0 + k) * m.np + j0 + lane;
    const float v = (float)((double)x[p] * inv);
    s[k][lane] = v;
    h[p] = hi_of(v);
    if constexpr (PRODUCTS == 3) hl[p] = lo_of(v, hi_of(v));
  }
  __syncthreads();
#pragma unroll 4
  for (int k = wave; k < kTile; k += kThreads / 64) {
    const int64_t p = (int64_t)(j0 + k) * m.mp + i0 + lane;
    const float v = s[lane][k];
    t[p] = hi_of(v);
    if constexpr (PRODUCTS == 3) tl[p] = lo_of(v, hi_of(v));
  }
}

// ---------------------------------------------------------------------------
// The products.  One kernel, four uses; every operand is stored with the
// summed axis contiguous (a symmetric matrix is its own transpose, and X is
// kept in both orientations), so C_ij = sum_k P[i][k] Q[j][k]:
//   kGram   A = X X^T         P = Q = X,       lower tiles, mirrored
//   kPoly   B = b A + c A A   P = Q = A,       lower tiles, mirrored
//   kApply  X <- a X + B X    P = B, Q = X^T
//   kLast   the same, written to the destination
enum Mode { kGram, kPoly, kApply, kLast };

struct GemmArgs {
  Common c;
  MuonIo io;
  float ca, cb, cc;
  int32_t turn;      // which transpose buffer holds X
  int32_t first;     // X is not normalised yet
};

constexpr int kBM = 128, kBK = 64;
constexpr int kLd = kBK + 8;  // LDS row stride in elements

template <int DST>
__device__ __forceinline__ void store1(const GemmArgs& a, const Mat& m, int64_t r, int64_t c,
                                       float o) {
  if constexpr (DST == ZF_F32) {
    static_cast<float*>(m.dst)[r * m.dst_ld + c] = o;
  } else {
    static_cast<uint16_t*>(m.dst)[r * m.dst_ld + c] = narrow1<DST>(o);
  }
}

// W <- W dec - rate O and the 16-bit parameter.
template <int PDT>  // 0: no 16-bit copy
__device__ __forceinline__ void update1(const GemmArgs& a, const Mat& m, int64_t r, int64_t c,
                                        float o) {
  const int64_t p = m.flat + r * m.dst_ld + c;
  const float w = a.io.master[p] * a.io.dec - m.rate * o;
  a.io.master[p] = w;
  if constexpr (PDT != 0) static_cast<uint16_t*>(a.io.params)[p] = narrow1<PDT>(w);
}

template <int MODE, int PRODUCTS, int DST, bool MUON>
__global__ __launch_bounds__(kThreads) void zf_ns_gemm(GemmArgs a) {
  if (a.c.st && a.c.st->skipped) return;
  constexpr bool SYM = MODE == kGram || MODE == kPoly;
  const Mat& m = SYM ? *find<&Mat::tri0>(a.c.table, a.c.count, blockIdx.x)
                     : *find<&Mat::app0>(a.c.table, a.c.count, blockIdx.x);
  int ti, tj;
  if constexpr (SYM) {
    const int b = blockIdx.x - m.tri0;
    ti = (int)((sqrtf(8.0f * (float)b + 1.0f) - 1.0f) * 0.5f);
    while ((ti + 1) * (ti + 2) / 2 <= b) ++ti;
    while (ti * (ti + 1) / 2 > b) --ti;
    tj = b - ti * (ti + 1) / 2;
  } else {
    const int b = blockIdx.x - m.app0, tiles_m = (m.mp + kBM - 1) / kBM;
    ti = b % tiles_m;
    tj = b / tiles_m;
  }
  const int mp = m.mp, np = m.np;
  const int64_t k_len = MODE == kGram ? np : mp;
  const int rows_p = mp, rows_q = SYM ? mp : np;
  const int64_t off_p = MODE == kGram ? m.h : MODE == kPoly ? m.a : m.b;
  const int64_t off_q = SYM ? off_p : m.t[a.turn];
  const int64_t lo_p = MODE == kGram ? m.lo_x : m.lo_s;
  const int64_t lo_q = MODE == kPoly ? m.lo_s : m.lo_x;
  const int i0 = ti * kBM, j0 = tj * kBM;

  __shared__ union {
    f16 k[2][kBM][kLd];
    float c[kBM][kBM + 1];
  } s;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wi = (wave >> 1) * 64, wj = (wave & 1) * 64;
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};

  // a thread copies 4 pieces of 8 elements of each operand per step; rows
  // past the padding are read from the last one and never stored
  const int lr = threadIdx.x >> 3, lc = (threadIdx.x & 7) * 8;
#pragma unroll 1
  for (int pass = 0; pass < PRODUCTS; ++pass) {
    // three products: hi lo, lo hi, (scaled down), hi hi
    const int64_t dp = (PRODUCTS == 3 && pass == 1) ? lo_p : 0;
    const int64_t dq = (PRODUCTS == 3 && pass == 0) ? lo_q : 0;
    const f16* p = at<f16>(a.c, off_p + dp);
    const f16* q = at<f16>(a.c, off_q + dq);
    if (PRODUCTS == 3 && pass == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = acc[i][j] * (1.0f / kLo);
    }
    for (int64_t k0 = 0; k0 < k_len; k0 += kBK) {
      f16x8 vp[4], vq[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int64_t rp = min(i0 + lr + h * 32, rows_p - 1);
        const int64_t rq = min(j0 + lr + h * 32, rows_q - 1);
        vp[h] = *reinterpret_cast<const f16x8*>(p + rp * k_len + k0 + lc);
        vq[h] = *reinterpret_cast<const f16x8*>(q + rq * k_len + k0 + lc);
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        *reinterpret_cast<f16x8*>(&s.k[0][lr + h * 32][lc]) = vp[h];
        *reinterpret_cast<f16x8*>(&s.k[1][lr + h * 32][lc]) = vq[h];
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < kBK; kk += 32) {
        f16x8 fp[4], fq[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          fp[i] = *reinterpret_cast<f16x8*>(&s.k[0][wi + i * 16 + (lane & 15)][kk + (lane >> 4) * 8]);
          fq[i] = *reinterpret_cast<f16x8*>(&s.k[1][wj + i * 16 + (lane & 15)][kk + (lane >> 4) * 8]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fp[i], fq[j], acc[i][j], 0, 0, 0);
      }
    }
  }

  // the tile into shared memory: the result goes out along either axis
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        s.c[wi + i * 16 + (lane >> 4) * 4 + r][wj + j * 16 + (lane & 15)] = acc[i][j][r] * kUnscale2;
  __syncthreads();

  const int col = threadIdx.x & (kBM - 1), row0 = threadIdx.x / kBM;
  constexpr int kRows = kThreads / kBM;
  if constexpr (SYM) {
    const f16* o = at<f16>(a.c, m.a);
    const f16* ol = at<f16>(a.c, m.a + m.lo_s);
    const float* da = at<float>(a.c, m.da);
    f16* out = at<f16>(a.c, MODE == kGram ? m.a : m.b);
    f16* outl = at<f16>(a.c, (MODE == kGram ? m.a : m.b) + m.lo_s);
    float* diag = at<float>(a.c, MODE == kGram ? m.da : m.db);
    for (int r = row0; r < kBM; r += kRows) {
      const int i = i0 + r, j = j0 + col;
      if (i >= mp || j >= mp) continue;
      const int64_t p = (int64_t)i * mp + j;
      float v = s.c[r][col];
      if constexpr (MODE == kPoly) {
        if (i == j) {
          const float d = da[i];
          v = a.cb * d + a.cc * (v + d * d);
        } else {
          const float x = value_of(o[p], PRODUCTS == 3 ? ol[p] : (f16)0);
          v = a.cb * x + a.cc * (v + (da[i] + da[j]) * x);
        }
      }
      if (i == j) {
        diag[i] = v;
        v = 0.0f;
      }
      s.c[r][col] = v;
      out[p] = hi_of(v);
      if constexpr (PRODUCTS == 3) outl[p] = lo_of(v, hi_of(v));
    }
    if (ti == tj) return;
    __syncthreads();
    for (int r = row0; r < kBM; r += kRows) {
      const int i = j0 + r, j = i0 + col;  // the mirrored tile
      if (i >= mp || j >= mp) continue;
      const int64_t p = (int64_t)i * mp + j;
      const float v = s.c[col][r];
      out[p] = hi_of(v);
      if constexpr (PRODUCTS == 3) outl[p] = lo_of(v, hi_of(v));
    }
  } else {
    float* x = at<float>(a.c, m.x);
    const float* db = at<float>(a.c, m.db);
    const double inv = a.first ? a.c.inv[m.slot] : 1.0;
    f16* h = at<f16>(a.c, m.h);
    f16* hl = at<f16>(a.c, m.h + m.lo_x);
    f16* t = at<f16>(a.c, m.t[a.turn ^ 1]);
    f16* tl = at<f16>(a.c, m.t[a.turn ^ 1] + m.lo_x);
    for (int r = row0; r < kBM; r += kRows) {
      const int i = i0 + r, j = j0 + col;
      if (i >= mp || j >= np) continue;
      const int64_t p = (int64_t)i * np + j;
      const float v = (a.ca + db[i]) * (float)((double)x[p] * inv) + s.c[r][col];
      s.c[r][col] = v;
      if constexpr (MODE == kApply) {
        x[p] = v;
        h[p] = hi_of(v);
        if constexpr (PRODUCTS == 3) hl[p] = lo_of(v, hi_of(v));
      } else if (!m.tall && i < m.m && j < m.n) {
        if constexpr (MUON) update1<DST>(a, m, i, j, v);
        else store1<DST>(a, m, i, j, v);
      }
    }
    if (MODE == kLast && !m.tall) return;
    __syncthreads();
    for (int r = row0; r < kBM; r += kRows) {
      const int j = j0 + r, i = i0 + col;
      if (i >= mp || j >= np) continue;
      const float v = s.c[col][r];
      if constexpr (MODE == kApply) {
        const int64_t p = (int64_t)j * mp + i;
        t[p] = hi_of(v);
        if constexpr (PRODUCTS == 3) tl[p] = lo_of(v, hi_of(v));
      } else if (i < m.m && j < m.n) {
        if constexpr (MUON) update1<DST>(a, m, j, i, v);
        else store1<DST>(a, m, j, i, v);
      }
    }
  }
}

template <int MODE, int PRODUCTS>
void launch_inner(int blocks, hipStream_t s, const GemmArgs& a) {
  hipLaunchKernelGGL((zf_ns_gemm<MODE, PRODUCTS, 0, false>), dim3(blocks), dim3(kThreads), 0, s, a);
}

template <int PRODUCTS>
void launch_last(int blocks, hipStream_t s, int32_t dst, bool muon, const GemmArgs& a) {
#define ZF_LAST(D, MU) \
  hipLaunchKernelGGL((zf_ns_gemm<kLast, PRODUCTS, D, MU>), dim3(blocks), dim3(kThreads), 0, s, a)
  if (muon) {
    if (!a.io.params) ZF_LAST(0, true);
    else if (dst == ZF_BF16) ZF_LAST(ZF_BF16, true);
    else ZF_LAST(ZF_F16, true);
  } else if (dst == ZF_BF16) {
    ZF_LAST(ZF_BF16, false);
  } else if (dst == ZF_F16) {
    ZF_LAST(ZF_F16, false);
  } else {
    ZF_LAST(ZF_F32, false);
  }
#undef ZF_LAST
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Matrices are worked on in groups whose buffers share one region, so that
// the workspace of a large model stays bounded: a group closes at this many
// padded elements.
constexpr int64_t kGroupElements = 1ll << 28;
constexpr int64_t kMaxSide = 1ll << 20;

}  // namespace

zf_ns_params zf::ns::defaults() {
  zf_ns_params p;
  p.steps = 5;
  p.products = 0;
  p.a = 3.4445;
  p.b = -4.7750;
  p.c = 2.0315;
  p.eps = 1e-7;
  return p;
}

int zf::ns::check_params(const zf_ns_params& p) {
  if (p.steps < 1 || p.steps > ZF_NS_MAX_STEPS) return ZF_EINVAL;
  if (p.products != 0 && p.products != 1 && p.products != 3) return ZF_EINVAL;
  if (!std::isfinite(p.a) || !std::isfinite(p.b) || !std::isfinite(p.c)) return ZF_EINVAL;
  if (!(p.eps >= 0.0) || !std::isfinite(p.eps)) return ZF_EINVAL;
  return ZF_OK;
}

int zf::ns::products_of(const zf_ns_params& p, int32_t dst_dtype) {
  if (p.products != 0) return p.products;
  return dst_dtype == ZF_BF16 ? 1 : 3;
}

bool zf::ns::layout(const Shape* shapes, int64_t count, int products, Layout& out) {
  out.mats.resize((size_t)count);
  out.groups.clear();
  int64_t partials = 0, region = 0, used = 0, elements = 0;
  Group g{0, 0, 0, 0, 0};
  int64_t load = 0, tri = 0, app = 0;
  const int halves = products == 3 ? 2 : 1;
  auto close = [&]() {
    g.load_blocks = (int32_t)load;
    g.tri_blocks = (int32_t)tri;
    g.app_blocks = (int32_t)app;
    out.groups.push_back(g);
    region = std::max(region, used);
    g = Group{g.first + g.count, 0, 0, 0, 0};
    used = elements = load = tri = app = 0;
  };
  auto take = [&](int64_t bytes) {
    const int64_t o = used;
    used += round_up(bytes, 256);
    return o;
  };
  for (int64_t k = 0; k < count; ++k) {
    const int64_t rows = shapes[k].rows, cols = shapes[k].cols;
    if (rows > kMaxSide || cols > kMaxSide) return false;
    Mat& m = out.mats[(size_t)k];
    m = Mat{};
    m.tall = rows > cols;
    m.m = (int32_t)std::min(rows, cols);
    m.n = (int32_t)std::max(rows, cols);
    m.mp = (int32_t)round_up(m.m, kPad);
    m.np = (int32_t)round_up(m.n, kPad);
    const int64_t mn = (int64_t)m.mp * m.np, mm = (int64_t)m.mp * m.mp;
    if (g.count > 0 && elements + mn > kGroupElements) close();
    m.slot = (int32_t)k;
    m.src_ld = m.dst_ld = cols;
    m.lo_x = round_up(mn * 2, 256);
    m.lo_s = round_up(mm * 2, 256);
    m.x = take(mn * 4);
    m.h = take(m.lo_x * halves);
    m.t[0] = take(m.lo_x * halves);
    m.t[1] = take(m.lo_x * halves);
    m.a = take(m.lo_s * halves);
    m.b = take(m.lo_s * halves);
    m.da = take((int64_t)m.mp * 4);
    m.db = take((int64_t)m.mp * 4);
    const int64_t tm = (m.mp + kBM - 1) / kBM, tn = (m.np + kBM - 1) / kBM;
    const int64_t tiles = (int64_t)(m.mp / kTile) * (m.np / kTile);
    m.part = partials;
    partials += tiles;
    m.load0 = (int32_t)load;
    m.tri0 = (int32_t)tri;
    m.app0 = (int32_t)app;
    load += tiles;
    tri += tm * (tm + 1) / 2;
    app += tm * tn;
    if (load > 0x7FFFFFFF) return false;
    elements += mn;
    ++g.count;
  }
  if (g.count > 0) close();
  int64_t at = 0;
  out.table = at;
  at += round_up(count * (int64_t)sizeof(Mat), 256);
  out.inv = at;
  at += round_up(count * 8, 256);
  out.partials = at;
  at += round_up(partials * 8, 256);
  for (Mat& m : out.mats)
    for (int64_t* o : {&m.x, &m.h, &m.t[0], &m.t[1], &m.a, &m.b, &m.da, &m.db}) *o += at;
  out.bytes = at + region;
  return true;
}

int zf::ns::enqueue(const Layout& l, const zf_ns_params& p, int products, int32_t src_dtype,
                    int32_t dst_dtype, const MuonIo* io, char* ws, hipStream_t s) {
  Mat* table = reinterpret_cast<Mat*>(ws + l.table);
  for (size_t k = 0; k < l.mats.size(); k += kTableChunk) {
    TableArgs t;
    t.to = table + k;
    t.count = (int32_t)std::min<size_t>(kTableChunk, l.mats.size() - k);
    for (int i = 0; i < t.count; ++i) t.m[i] = l.mats[k + i];
    hipLaunchKernelGGL(zf_ns_table, dim3(1), dim3(64), 0, s, t);
    if (!hip_ok(hipGetLastError())) return ZF_EHIP;
  }
  for (const Group& g : l.groups) {
    Common c;
    c.ws = ws;
    c.table = table + g.first;
    c.count = g.count;
    c.st = io ? io->st : nullptr;
    c.inv = reinterpret_cast<double*>(ws + l.inv);
    c.partials = reinterpret_cast<double*>(ws + l.partials);

    LoadArgs la;
    la.c = c;
    la.io = io ? *io : MuonIo{};
    const dim3 load(g.load_blocks), block(kThreads);
    if (io) hipLaunchKernelGGL(zf_ns_load<0>, load, block, 0, s, la);
    else if (src_dtype == ZF_F32) hipLaunchKernelGGL(zf_ns_load<ZF_F32>, load, block, 0, s, la);
    else if (src_dtype == ZF_BF16) hipLaunchKernelGGL(zf_ns_load<ZF_BF16>, load, block, 0, s, la);
    else hipLaunchKernelGGL(zf_ns_load<ZF_F16>, load, block, 0, s, la);
    if (!hip_ok(hipGetLastError())) return ZF_EHIP;
    NormArgs na;
    na.c = c;
    na.eps = p.eps;
    hipLaunchKernelGGL(zf_ns_norm, dim3(g.count), block, 0, s, na);
    if (!hip_ok(hipGetLastError())) return ZF_EHIP;
    if (products == 3) hipLaunchKernelGGL(zf_ns_prep<3>, load, block, 0, s, c);
    else hipLaunchKernelGGL(zf_ns_prep<1>, load, block, 0, s, c);
    if (!hip_ok(hipGetLastError())) return ZF_EHIP;

    GemmArgs ga;
    ga.c = c;
    ga.io = la.io;
    ga.ca = (float)p.a;
    ga.cb = (float)p.b;
    ga.cc = (float)p.c;
    for (int k = 0; k < p.steps; ++k) {
      ga.turn = k & 1;
      ga.first = k == 0;
      const bool last = k + 1 == p.steps;
      if (products == 3) {
        launch_inner<kGram, 3>(g.tri_blocks, s, ga);
        launch_inner<kPoly, 3>(g.tri_blocks, s, ga);
        if (last) launch_last<3>(g.app_blocks, s, dst_dtype, io != nullptr, ga);
        else launch_inner<kApply, 3>(g.app_blocks, s, ga);
      } else {
        launch_inner<kGram, 1>(g.tri_blocks, s, ga);
        launch_inner<kPoly, 1>(g.tri_blocks, s, ga);
        if (last) launch_last<1>(g.app_blocks, s, dst_dtype, io != nullptr, ga);
        else launch_inner<kApply, 1>(g.app_blocks, s, ga);
      }
      if (!hip_ok(hipGetLastError())) return ZF_EHIP;
    }
  }
  return ZF_OK;
}

// ---------------------------------------------------------------------------
// zf_orthogonalize

namespace {

bool valid_any(int32_t d) { return d == ZF_F16 || d == ZF_BF16 || d == ZF_F32; }

int ortho_layout(const zf_matrix* mats, int64_t count, int32_t dst_dtype,
                 const zf_ns_params* params, Layout& l, zf_ns_params& p, int& products) {
  if (count < 0 || (count > 0 && !mats)) return ZF_EINVAL;
  if (!valid_any(dst_dtype)) return ZF_EDTYPE;
  if (count > ZF_ORTHO_MAX_MATRICES) return ZF_ESIZE;
  p = params ? *params : zf::ns::defaults();
  const int rc = zf::ns::check_params(p);
  if (rc != ZF_OK) return rc;
  products = zf::ns::products_of(p, dst_dtype);
  std::vector<zf::ns::Shape> shapes((size_t)count);
  for (int64_t k = 0; k < count; ++k) {
    if (mats[k].rows < 1 || mats[k].cols < 1) return ZF_EINVAL;
    shapes[(size_t)k] = {mats[k].rows, mats[k].cols};
  }
  return zf::ns::layout(shapes.data(), count, products, l) ? ZF_OK : ZF_ESIZE;
}

bool aligned(const void* p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == ZF_F32 ? 3u : 1u)) == 0;
}

}  // namespace

extern "C" int64_t zf_orthogonalize_bytes(const zf_matrix* mats, int64_t count, int32_t dst_dtype,
                                          const zf_ns_params* params) {
  try {
    Layout l;
    zf_ns_params p;
    int products = 1;
    const int rc = ortho_layout(mats, count, dst_dtype, params, l, p, products);
    return rc == ZF_OK ? l.bytes : rc;
  } catch (const std::bad_alloc&) {
    return ZF_ENOMEM;
  }
}

extern "C" int zf_orthogonalize(const zf_matrix* mats, int64_t count, int32_t src_dtype,
                                int32_t dst_dtype, const zf_ns_params* params, void* workspace,
                                int64_t workspace_size, void* stream) {
  try {
    if (!valid_any(src_dtype)) return ZF_EDTYPE;
    Layout l;
    zf_ns_params p;
    int products = 1;
    const int rc = ortho_layout(mats, count, dst_dtype, params, l, p, products);
    if (rc != ZF_OK) return rc;
    for (int64_t k = 0; k < count; ++k) {
      const zf_matrix& z = mats[k];
      if (!z.src || !z.dst) return ZF_EINVAL;
      if (z.rows > 1 && (z.src_stride < z.cols || z.dst_stride < z.cols)) return ZF_EINVAL;
      if (!aligned(z.src, src_dtype) || !aligned(z.dst, dst_dtype)) return ZF_EALIGN;
      Mat& m = l.mats[(size_t)k];
      m.src = z.src;
      m.dst = z.dst;
      m.src_ld = z.src_stride;
      m.dst_ld = z.dst_stride;
    }
    if (count == 0) return ZF_OK;
    if (!workspace) return ZF_EINVAL;
    if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return ZF_EALIGN;
    if (workspace_size < l.bytes) return ZF_ESIZE;
    (void)hipGetLastError();
    return zf::ns::enqueue(l, p, products, src_dtype, dst_dtype, nullptr,
                           static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
  } catch (const std::bad_alloc&) {
    return ZF_ENOMEM;
  }
}
