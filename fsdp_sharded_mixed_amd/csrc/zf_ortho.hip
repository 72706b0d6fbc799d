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
// iteration keep more bits, because rounding them is what costs accuracy:
//   - the linear term a X: a singular value that starts small grows by a
//     every step, to 485 times its size in five, and an error of X anywhere
//     grows with it.  X is kept as two fp16 numbers, hi + lo * 2^-11, about
//     22 bits; the products take hi, the term both, in 32 bits;
//   - the diagonal of A and of B (B's is near -2.7 once the singular values
//     near 1, where the rest of a row is near 1/sqrt(m): half a step of fp16
//     there is 1e-3), so a product of two such matrices S = diag(D) + O is
//     O O + (D_i + D_j) O_ij + D_i^2 on the diagonal.
// A product B X with errors E in B and d in X is off by E X + B d; both shrink
// with the singular value they fall on, X's as it is and B's as its square, so
// neither outgrows it.  Taken apart, (D + O) X keeps that only if D multiplies
// what O does, hi: the step is a lo + (a + D) hi + O hi while small singular
// values still grow.  In the last two steps, where most of a + D + O is D,
// D takes lo too: (a + D) X + O hi.  Where sums are short, in shared memory
// and for short sides of one tile, lo goes through the product as well,
// (a + D + O) X: with few singular values a lo alone costs up to 2e-3 (1 x 77:
// 1.4e-3 against 1e-4).
// Measured in |.|_F against 64 bits, over flat, low-rank, low-rank-plus-noise,
// 1/i and log-uniform spectra, sparse matrices and rows of different scales:
// 5e-5 to 2e-3, up to 3e-3 for short sides under 32 (with 14 bits of X in the
// linear term and lo times a + D throughout, one strong direction comes to
// 5e-3 to 4e-2; bf16 throughout: 1e-2 to 3e-2).  A result in more bits than
// bf16 gets three products instead of one: every operand is the sum of two fp16
// numbers, hi + lo * 2^-11, and hi hi + hi lo + lo hi holds about 22 bits: 1e-6, 5e-6
// for short sides under 32, and 1e-4 for one strong direction, as the
// iteration in 32-bit arithmetic has there.
#include "zf_ortho.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

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

// Everything between the load and the result is in units of 2^-10 ("scaled"):
// a 16-bit operand holds the scaled value rounded, products of two need one
// factor 2^-10.  Multiplications by powers of two are exact, so the factors
// go wherever they cost least; the vector unit, at 4 cycles an instruction,
// is what an epilogue waits for.
constexpr float kScale = 1024.0f, kUnscale = 1.0f / 1024.0f;
constexpr float kLo = 2048.0f;              // lo halves: 2^11 more
constexpr int kLast = 2;                    // steps that the singular values end in

// (x - hi) kLo; the difference is exact either way, and this way takes two
// instructions
__device__ __forceinline__ f16 rest_of(float x, f16 hi) {
  return (f16)__builtin_fmaf((float)hi, -kLo, x * kLo);
}
__device__ __forceinline__ float join(f16 hi, f16 lo) {
  return __builtin_fmaf((float)lo, 1.0f / kLo, (float)hi);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// The table of matrices travels by value, a chunk a launch, into the
// workspace, so that a captured call carries it.
constexpr int kTableChunk = 16;
struct TableArgs {
  Mat* to;
  int32_t count;
  Mat m[kTableChunk];
};

constexpr size_t kArgBytes = 4096;  // of a launch

__global__ __launch_bounds__(64) void zf_ns_table(TableArgs a) {
  static_assert(sizeof(TableArgs) <= kArgBytes, "arguments of a launch");
  static_assert(sizeof(Mat) % 8 == 0, "copied in words");
  const uint64_t* s = reinterpret_cast<const uint64_t*>(a.m);
  uint64_t* d = reinterpret_cast<uint64_t*>(a.to);
  for (int i = threadIdx.x; i < a.count * (int)(sizeof(Mat) / 8); i += 64) d[i] = s[i];
}

// The matrices of a launch: a table in the workspace, and, for a launch of a
// few, the matrices themselves among the arguments, where they are one scalar
// load away instead of a chain of them.
constexpr int kFirsts = 64, kByValue = 8;
struct Common {
  char* ws;
  const Mat* table;       // the group's matrices
  int32_t count;
  int32_t load_tiles;
  const DevState* st;     // the Muon step's skip flag, or NULL
  double* inv;            // 1 / (|G|_F + eps), by slot
  double* partials;       // squared-norm partials
  double eps;
  int32_t firsts[kFirsts];  // each matrix's first block in this launch, INT32_MAX past the last
  Mat m[kByValue];          // count <= kByValue
};

// The matrix that holds block b of the launch: the last one that starts at
// or before it.
template <typename F>
__device__ __forceinline__ const Mat& find(const Common& c, int b, F first) {
  if (c.count <= kByValue) {
    int k = 0;
#pragma unroll
    for (int j = 1; j < kByValue; ++j) k += c.firsts[j] <= b ? 1 : 0;
    return c.m[k];
  }
  if (c.count <= kFirsts) {
    int k = 0;
#pragma unroll
    for (int j = 1; j < kFirsts; ++j) k += c.firsts[j] <= b ? 1 : 0;
    return c.table[k];
  }
  int lo = 0, hi = c.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first(c.table[mid]) <= b) lo = mid;
    else hi = mid - 1;
  }
  return c.table[lo];
}
__device__ __forceinline__ const Mat& find_load(const Common& c, int b) {
  return find(c, b, [](const Mat& m) { return m.load0; });
}

template <typename T>
__device__ __forceinline__ T* at(const Common& c, int64_t offset) {
  return reinterpret_cast<T*>(c.ws + offset);
}

// ---------------------------------------------------------------------------
// The squared norm, one partial (64 bits) for 4096 padded elements, however
// many a block takes; the Muon step's momentum update on the way.  A stream: 122M weights with momentum 261 us, 12 bytes
// each, 5.6 TB/s.
constexpr int kTile = 64, kLoadTiles = 4;  // tiles of a block, if there are many

struct LoadArgs {
  Common c;
  MuonIo io;
};
static_assert(sizeof(LoadArgs) <= kArgBytes, "arguments of a launch");

// Whether 8 elements at a multiple of 8 of any row lie at a multiple of 16
// bytes.
template <int SRC>
__device__ __forceinline__ bool wide_loads(const Mat& m) {
  if constexpr (SRC == 0) return ((m.flat | m.src_ld) & 3) == 0;
  else if constexpr (SRC == ZF_F32)
    return ((reinterpret_cast<uintptr_t>(m.src) | (uintptr_t)(m.src_ld * 4)) & 15) == 0;
  else return ((reinterpret_cast<uintptr_t>(m.src) | (uintptr_t)(m.src_ld * 2)) & 15) == 0;
}

// Elements (r, c .. c + 7) of the matrix, zeros past its last column.  SRC:
// ZF_F16, ZF_BF16, ZF_F32, or 0: the Muon step's U, from the momentum that it
// updates first (FIRST) or has updated.
template <int SRC, bool FIRST>
__device__ __forceinline__ void load8(const LoadArgs& a, const Mat& m, float gs, bool wide,
                                      int64_t r, int c, int cols, float (&v)[8]) {
  const int64_t p = r * m.src_ld + c;
  const int n = cols - c;
  if constexpr (SRC == 0) {
    float* mom = a.io.momentum + m.flat + p;
    const float* sums = a.io.sums + m.flat + p;
    const bool with_g = FIRST || a.io.nesterov;
    float g[8];
    if (wide && n >= 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 x = reinterpret_cast<const f32x4*>(mom)[h];
        f32x4 y = {0, 0, 0, 0};
        if (with_g) y = reinterpret_cast<const f32x4*>(sums)[h];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[h * 4 + e] = x[e], g[h * 4 + e] = y[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = e < n ? mom[e] : 0.0f;
        g[e] = e < n && with_g ? sums[e] : 0.0f;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g[e] = g[e] * gs;
      if constexpr (FIRST) v[e] = a.io.mu * v[e] + g[e];
    }
    if constexpr (FIRST) {
      if (wide && n >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          reinterpret_cast<f32x4*>(mom)[h] =
              (f32x4){v[h * 4], v[h * 4 + 1], v[h * 4 + 2], v[h * 4 + 3]};
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < n) mom[e] = v[e];
      }
    }
    if (a.io.nesterov) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = g[e] + a.io.mu * v[e];
    }
  } else if constexpr (SRC == ZF_F32) {
    const float* x = static_cast<const float*>(m.src) + p;
    if (wide && n >= 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 y = reinterpret_cast<const f32x4*>(x)[h];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[h * 4 + e] = y[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < n ? x[e] : 0.0f;
    }
  } else {
    const uint16_t* x = static_cast<const uint16_t*>(m.src) + p;
    if (wide && n >= 8) {
      const u32x4 y = *reinterpret_cast<const u32x4*>(x);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[2 * e] = lo16<SRC>(y[e]), v[2 * e + 1] = hi16<SRC>(y[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < n ? widen1<SRC>(x[e]) : 0.0f;
    }
  }
}

// A block takes load_tiles * 4096 elements of the rows one after another
// (padded to multiples of 64), a thread 8 neighbours at a time: this walks
// them, 2048 elements of the block a step.
struct Walk {
  int64_t r;
  int c, width;
  __device__ __forceinline__ Walk(int64_t first, int padded) : width(padded) {
    r = first / width;  // the same for the block
    c = (int)(first - r * width) + threadIdx.x * 8;
    wrap();
  }
  __device__ __forceinline__ void wrap() {
    while (c >= width) c -= width, ++r;
  }
  __device__ __forceinline__ void next() {
    c += kThreads * 8;
    wrap();
  }
};

template <int SRC>
__global__ __launch_bounds__(kThreads) void zf_ns_load(LoadArgs a) {
  if (a.c.st && a.c.st->skipped) return;
  const Mat& m = find_load(a.c, blockIdx.x);
  const int block = blockIdx.x - m.load0;
  const float gs = SRC == 0 ? a.c.st->gs : 0.0f;
  const bool wide = wide_loads<SRC>(m);
  const int rows = m.tall ? m.n : m.m, cols = m.tall ? m.m : m.n;
  const int steps = a.c.load_tiles * 2;
  Walk w((int64_t)block * a.c.load_tiles * 4096, m.tall ? m.mp : m.np);
  double ss[kLoadTiles] = {};
#pragma unroll
  for (int t = 0; t < kLoadTiles * 2; ++t, w.next()) {
    if (t >= steps) break;
    if (w.r >= rows || w.c >= cols) continue;
    float v[8];
    load8<SRC, true>(a, m, gs, wide, w.r, w.c, cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss[t / 2] += (double)v[e] * (double)v[e];
  }
  constexpr int kWaves = kThreads / 64;
  __shared__ double sum[kLoadTiles][kWaves];
#pragma unroll
  for (int k = 0; k < kLoadTiles; ++k) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) ss[k] = ss[k] + __shfl_xor(ss[k], off, 64);
    if ((threadIdx.x & 63) == 0) sum[k][threadIdx.x >> 6] = ss[k];
    if (k + 1 == a.c.load_tiles) break;
  }
  __syncthreads();
  const int k = threadIdx.x, tile = block * a.c.load_tiles + k;
  if (k < a.c.load_tiles && tile < (m.mp / kTile) * (m.np / kTile)) {
    double t = sum[k][0];
#pragma unroll
    for (int x = 1; x < kWaves; ++x) t = t + sum[k][x];
    a.c.partials[m.part + tile] = t;
  }
}

// The inverse norm of a matrix from its partials, in an order that depends on
// its shape alone; valid in every thread.
__device__ __forceinline__ double inverse_norm(const Common& c, const Mat& m) {
  const int64_t parts = (int64_t)(m.mp / kTile) * (m.np / kTile);
  double ss = 0.0;
  for (int64_t i = threadIdx.x; i < parts; i += kThreads) ss += c.partials[m.part + i];
  uint32_t unused = 0;
  block_reduce(ss, unused);
  __shared__ double total;
  if (threadIdx.x == 0) total = 1.0 / (sqrt(ss) + c.eps);
  __syncthreads();
  return total;
}

// The inverse norm of every matrix of the group, one block a matrix, unless
// the blocks of the next launch take it themselves (own_norm).
__global__ __launch_bounds__(kThreads) void zf_ns_norm(Common c) {
  if (c.st && c.st->skipped) return;
  const Mat& m = c.count <= kByValue ? c.m[blockIdx.x] : c.table[blockIdx.x];
  const double inv = inverse_norm(c, m);
  if (threadIdx.x == 0) c.inv[m.slot] = inv;
}

// X in 16-bit halves from the matrix and its inverse norm, transposed if the
// matrix is tall (by tiles of 64 x 64), with zero padding.  Non-temporal
// stores: 143 -> 85 us for a layer of hidden 2048.  Two such layers from bf16
// take 225 us, 6 bytes an element at 3.2 TB/s; from momenta and sums 364 us,
// 12 at 4.0.
template <int SRC, bool OWN_NORM>
__global__ __launch_bounds__(kThreads) void zf_ns_prep(LoadArgs a) {
  if (a.c.st && a.c.st->skipped) return;
  const Mat& m = find_load(a.c, blockIdx.x);
  const int block = blockIdx.x - m.load0, tiles_n = m.np / kTile;
  const int tiles = m.mp / kTile * tiles_n;
  const float gs = SRC == 0 ? a.c.st->gs : 0.0f;
  double inv = kScale;
  if constexpr (OWN_NORM) inv *= inverse_norm(a.c, m);
  else inv *= a.c.inv[m.slot];
  const bool wide = wide_loads<SRC>(m);
  f16* hp = at<f16>(a.c, m.h[0]);
  f16* lp = at<f16>(a.c, m.l[0]);
  // 8 values at (i, j) in whole lines that this kernel does not read back
  auto put = [&](int64_t i, int j, const float (&v)[8]) {
    f16x8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = i < m.m && j + e < m.n ? (float)((double)v[e] * inv) : 0.0f;
      hi[e] = (f16)x;
      lo[e] = rest_of(x, hi[e]);
    }
    const int64_t p = i * m.ldx + j;
    __builtin_nontemporal_store(hi, reinterpret_cast<f16x8*>(hp + p));
    __builtin_nontemporal_store(lo, reinterpret_cast<f16x8*>(lp + p));
  };
  if (!m.tall) {
    Walk w((int64_t)block * a.c.load_tiles * 4096, m.np);
#pragma unroll 2
    for (int t = 0; t < a.c.load_tiles * 2; ++t, w.next()) {
      if (w.r >= m.mp) break;
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (w.r < m.m && w.c < m.n) load8<SRC, false>(a, m, gs, wide, w.r, w.c, m.n, v);
      put(w.r, w.c, v);
    }
    return;
  }
  __shared__ float s[kTile][kTile + 1];
#pragma unroll 1
  for (int t = 0; t < a.c.load_tiles; ++t) {
    const int tile = block * a.c.load_tiles + t;
    if (tile >= tiles) break;
    const int i0 = tile / tiles_n * kTile, j0 = tile % tiles_n * kTile;
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = threadIdx.x + h * kThreads, r = j0 + k / 8, c = i0 + k % 8 * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[h][e] = 0.0f;
      if (r < m.n && c < m.m) load8<SRC, false>(a, m, gs, wide, r, c, m.m, v[h]);
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = threadIdx.x + h * kThreads;
#pragma unroll
      for (int e = 0; e < 8; ++e) s[k % 8 * 8 + e][k / 8] = v[h][e];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = threadIdx.x + h * kThreads;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[h][e] = s[k / 8][k % 8 * 8 + e];
      put(i0 + k / 8, j0 + k % 8 * 8, v[h]);
    }
  }
}

void launch_prep(int32_t src, bool own_norm, dim3 grid, hipStream_t s, const LoadArgs& a) {
#define ZF_PREP(S) \
  do { \
    if (own_norm) hipLaunchKernelGGL((zf_ns_prep<S, true>), grid, dim3(kThreads), 0, s, a); \
    else hipLaunchKernelGGL((zf_ns_prep<S, false>), grid, dim3(kThreads), 0, s, a); \
  } while (0)
  if (src == 0) ZF_PREP(0);
  else if (src == ZF_F32) ZF_PREP(ZF_F32);
  else if (src == ZF_BF16) ZF_PREP(ZF_BF16);
  else ZF_PREP(ZF_F16);
#undef ZF_PREP
}

// ---------------------------------------------------------------------------
// The products.
//
// C_ij = sum_k P[i][k] Q(k, j) over a BM x BN tile by WI x WJ waves, 64 of
// the summed axis a step.  P is stored with the summed axis contiguous; so
// is Q where it is a symmetric matrix or X^T (X itself, read by rows); where
// Q is X (the application), its rows run along j and the fragments are
// transposed on their way out of shared memory (ds_read_b64_tr_b16).
//
// What bounds it: the matrix cores, if they are fed.  A 256 x 256 tile needs
// 32 bytes a cycle of a CU from the second-level cache at their full rate
// (128 x 128: 64), and its 8 waves of 128 x 64 read 48 KiB of shared memory
// per 1024 cycles.  Loads go from global to shared memory directly (no
// registers), into two buffers in turn (of 64 KiB for 256 x 256); a step's barrier stands
// between its two halves, so that the fragments of the next half are read
// while the matrix cores work on this one, and a buffer's loads are on their
// way for a whole step.  The 16-byte pieces of a row lie permuted by the row
// number, which keeps every read free of bank conflicts (counter
// SQ_LDS_BANK_CONFLICT: 0).  fp16 operands, 16x16x32 instructions.
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define ZF_LDS __attribute__((address_space(3)))
typedef __amdgpu_buffer_rsrc_t Rsrc;

constexpr int kBK = 64;

// A buffer of n bytes; loads past its end return nothing.
__device__ __forceinline__ uint32_t extent(int64_t bytes) {
  return bytes <= 0 ? 0u : bytes > 0x7FFFFFFFll ? 0x7FFFFFFFu : (uint32_t)bytes;
}
// An address that is the same for the whole wave, as the compiler must know:
// a buffer's descriptor otherwise takes a loop over the lanes at every load.
__device__ __forceinline__ const f16* uniform(const f16* p) {
  const uint64_t x = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return reinterpret_cast<const f16*>((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ Rsrc rsrc(const f16* base, uint32_t n) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<f16*>(base), 0, n, 0x00020000);
}

template <int BM_, int BN_, int WI, int WJ, int BUFFERS>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, kWaves = WI * WJ, kThreads = kWaves * 64;
  static constexpr int TI = BM / WI, TJ = BN / WJ, FI = TI / 16, FJ = TJ / 16;
  static constexpr int kWavesJ = WJ, kBuffers = BUFFERS;
  static constexpr int kPBytes = BM * kBK * 2, kQBytes = BN * kBK * 2;
  static constexpr int kBuf = (BM + BN) * kBK;  // elements of one buffer
  static constexpr int kRows = kThreads / 8;    // rows that a load of all threads covers
  static constexpr int kChunks = BN / 8;        // 16-byte pieces of a row of X
  static constexpr int kRowsX = kThreads / kChunks;
  // consecutive symmetric tiles of one XCD, as many as it works on at a time
  // (0.25 to 3 percent less time than runs of 8 along the rows)
  static constexpr int kRun = BM == 256 ? 16 : 32;
  // a square of 64 x 64 results goes out by the waves that hold it
  static constexpr int kSquareI = TI < 64 ? 64 / TI : 1, kSquareJ = TJ < 64 ? 64 / TJ : 1;
  static constexpr int kSquareWaves = kSquareI * kSquareJ;
  static_assert(BM % kRows == 0 && BN % kRows == 0 && kRows % 8 == 0 && kRowsX % 16 == 0, "tile");
  static_assert((TI % 64 == 0 || 64 % TI == 0) && (TJ == 64 || 64 % TJ == 0), "squares");
  // for a wave at (wi, wj) of the tile: its square's place in shared memory
  // and its own share of the square
  static __device__ __forceinline__ int square_of(int wi, int wj) {
    return wi / (TI < 64 ? 64 : TI) * (BN / 64) + wj / 64;
  }
  static __device__ __forceinline__ int share_of(int wi, int wj) {
    return wi % 64 / (TI < 64 ? TI : 64) * kSquareJ + wj % 64 / TJ;
  }
};

// The operands of one tile.  XQ: Q is X, rows along j.
template <typename T, bool XQ>
struct Operands {
  Rsrc p, q;
  uint32_t np, nq;
  const f16* x;     // XQ: X at column j0
  int64_t ld;       // elements of a row of P, Q or X
  int64_t ldp;
  int64_t skip;     // XQ: columns of X before j0
  int k_len, vp, vq, rowp, rowq;
  int rp, rq[T::FJ];  // shared-memory byte offsets of this lane's fragments

  // rows_p, rows_q: rows of P and Q from this tile's first on (XQ: rows_q is
  // the tile's first column j0)
  __device__ __forceinline__ Operands(const f16* pp, int64_t p_ld, int rows_p, const f16* qq,
                                      int64_t q_ld, int rows_q, int len) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wi = wave / T::kWavesJ * T::TI, wj = wave % T::kWavesJ * T::TJ;
    const int l = lane & 15, g = lane >> 4;
    pp = uniform(pp);
    qq = uniform(qq);
    k_len = __builtin_amdgcn_readfirstlane(len);
    ldp = __builtin_amdgcn_readfirstlane((int)p_ld);
    ld = __builtin_amdgcn_readfirstlane((int)q_ld);
    rows_p = __builtin_amdgcn_readfirstlane(rows_p);
    rows_q = __builtin_amdgcn_readfirstlane(rows_q);
    np = extent(rows_p * ldp * 2);
    p = rsrc(pp, np);
    const int r = tid >> 3, c = (tid & 7) ^ (r & 7);
    vp = (int)(r * ldp * 2) + c * 16;
    rowp = (int)(T::kRows * ldp * 2);
    rp = (wi + l) * (kBK * 2) + ((g ^ (l & 7)) * 16);
    if constexpr (XQ) {
      x = qq;
      skip = rows_q;
      const int rx = tid / T::kChunks, cx = (tid % T::kChunks) ^ (2 * turn(rx));
      vq = (int)(rx * ld * 2) + cx * 16;
      rowq = (int)(T::kRowsX * ld * 2);
      const int row = 8 * g + (l >> 2);
#pragma unroll
      for (int f = 0; f < T::FJ; ++f)
        rq[f] = T::kPBytes + row * (T::BN * 2) +
                ((((wj + 16 * f) / 8 + ((l & 3) >> 1)) ^ (2 * turn(row))) * 16) + (l & 1) * 8;
    } else {
      nq = extent(rows_q * ld * 2);
      q = rsrc(qq, nq);
      vq = (int)(r * ld * 2) + c * 16;
      rowq = (int)(T::kRows * ld * 2);
      rq[0] = T::kPBytes + (wj + l) * (kBK * 2) + ((g ^ (l & 7)) * 16);
    }
  }
  // the permutation of a row of X: pairs of pieces, as many as a row has
  static __device__ __forceinline__ int turn(int r) {
    return ((r & 3) | ((r >> 1) & 4)) & (T::kChunks / 2 - 1);
  }
};

template <typename T>
struct Frags {
  f16x8 p[T::FI], q[T::FJ];
};

// One load of 16 bytes a lane from global to shared memory, at byte
// lane_at + at of a buffer of n bytes.  The hardware compares lane_at with
// n - at, which must not wrap.  (The compiler's
// pass over the host code does not know the 16-byte form.)
__device__ __forceinline__ void to_shared(Rsrc from, uint32_t n, ZF_LDS char* to, int lane_at,
                                          uint32_t at) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (ZF_LDS void*)to, 16, lane_at, min(at, n), 0, 0);
#endif
}

// Loads of step k into `buf`.  Past the end of the summed axis they read
// other rows of the operand, or (past its end) nothing; no one uses them.
template <typename T, bool XQ>
__device__ __forceinline__ void fetch(const Operands<T, XQ>& o, int k, f16* __restrict buf) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  ZF_LDS char* b = (ZF_LDS char*)(buf) + wave * 1024;
#pragma unroll
  for (int h = 0; h < T::BM / T::kRows; ++h)
    to_shared(o.p, o.np, b + h * T::kThreads * 16, o.vp, k * (kBK * 2) + h * o.rowp);
  b += T::kPBytes;
  if constexpr (XQ) {
    // 64 rows of X; the last column tile may end past the row, inside the
    // next one or (in the last row) past the 64 rows, which reads nothing
    const int k0 = k * kBK;
    const uint32_t n = k0 < o.k_len ? extent((kBK * o.ld - o.skip) * 2) : 0;
    const Rsrc q = rsrc(o.x + k0 * o.ld, n);
#pragma unroll
    for (int h = 0; h < kBK / T::kRowsX; ++h)
      to_shared(q, n, b + h * T::kThreads * 16, o.vq, h * o.rowq);
  } else {
#pragma unroll
    for (int h = 0; h < T::BN / T::kRows; ++h)
      to_shared(o.q, o.nq, b + h * T::kThreads * 16, o.vq, k * (kBK * 2) + h * o.rowq);
  }
}

// Fragments of half kk of a step.
template <typename T, bool XQ>
__device__ __forceinline__ void read(const Operands<T, XQ>& o, const f16* __restrict buf,
                                     Frags<T>& f, int kk) {
  const char* b = reinterpret_cast<const char*>(buf);
  if constexpr (XQ) {
#pragma unroll
    for (int j = 0; j < T::FJ; ++j) {
      const ZF_LDS char* q = (const ZF_LDS char*)(b) + o.rq[j] + kk * 32 * T::BN * 2;
      s16x4 half[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        half[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZF_LDS s16x4*)(q + e * 4 * T::BN * 2));
      f.q[j] = __builtin_bit_cast(
          f16x8, __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
  } else {
#pragma unroll
    for (int j = 0; j < T::FJ; ++j)
      f.q[j] = *reinterpret_cast<const f16x8*>(b + (o.rq[0] ^ (kk * 64)) + j * 16 * kBK * 2);
  }
#pragma unroll
  for (int i = 0; i < T::FI; ++i)
    f.p[i] = *reinterpret_cast<const f16x8*>(b + (o.rp ^ (kk * 64)) + i * 16 * kBK * 2);
}

// acc[i][j] holds 4 consecutive i for one j (XQ: 4 consecutive j for one i).
template <typename T, bool XQ>
__device__ __forceinline__ void multiply(const Frags<T>& f, f32x4 (&acc)[T::FI][T::FJ]) {
#pragma unroll
  for (int i = 0; i < T::FI; ++i)
#pragma unroll
    for (int j = 0; j < T::FJ; ++j)
      acc[i][j] = XQ ? __builtin_amdgcn_mfma_f32_16x16x32_f16(f.q[j], f.p[i], acc[i][j], 0, 0, 0)
                     : __builtin_amdgcn_mfma_f32_16x16x32_f16(f.p[i], f.q[j], acc[i][j], 0, 0, 0);
}

// The order within a half: one shared-memory read, one load, then a share of
// the matrix instructions, again and again (8192^2 x 4096: 1117 TFLOP/s; the
// compiler's own order 1012, reads first 1106).
template <typename T, bool XQ, int LOADS>
__device__ __forceinline__ void interleave() {
  constexpr int reads = T::FI + (XQ ? 2 : 1) * T::FJ, mma = T::FI * T::FJ;
#pragma unroll
  for (int k = 0; k < reads; ++k) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    if (k < LOADS) __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x8, mma / reads, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x8, mma % reads, 0);
}

template <typename T, bool XQ>
__device__ __forceinline__ void half0(const Operands<T, XQ>& o, const f16* __restrict cur,
                                      Frags<T>& a, Frags<T>& b, f32x4 (&acc)[T::FI][T::FJ]) {
  read(o, cur, b, 1);
  multiply<T, XQ>(a, acc);
  interleave<T, XQ, 0>();
}

template <typename T, bool XQ>
__device__ __forceinline__ void half1(const Operands<T, XQ>& o, int k, f16* __restrict cur,
                                      const f16* __restrict nxt, Frags<T>& a, Frags<T>& b,
                                      f32x4 (&acc)[T::FI][T::FJ]) {
  fetch(o, k, cur);
  read(o, nxt, a, 0);
  multiply<T, XQ>(b, acc);
  interleave<T, XQ, T::BM / T::kRows + (XQ ? kBK / T::kRowsX : T::BN / T::kRows)>();
}

// Every load to shared memory has arrived and every read of it is done, for
// all waves (the barrier alone does not wait for loads to shared memory).
__device__ __forceinline__ void arrive() {
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __syncthreads();
}

// The same for all but the wave's last N loads.
template <int N>
__device__ __forceinline__ void arrive_but() {
  static_assert(N < 64, "the counter's range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <typename T, bool XQ>
__device__ __forceinline__ void one_step(const Operands<T, XQ>& o, int k, f16* __restrict next,
                                         const f16* __restrict cur,
                                         f32x4 (&acc)[T::FI][T::FJ]) {
  Frags<T> a, b;
  fetch(o, k, next);
  read(o, cur, a, 0);
  read(o, cur, b, 1);
  multiply<T, XQ>(a, acc);
  multiply<T, XQ>(b, acc);
}

template <typename T, bool XQ>
__device__ __forceinline__ void product(const Operands<T, XQ>& o, f16* shared,
                                        f32x4 (&acc)[T::FI][T::FJ]) {
  const int steps = o.k_len / kBK;
  if constexpr (T::kBuffers == 2) {
    f16 *s0 = shared, *s1 = shared + T::kBuf;
    Frags<T> a, b;
    fetch(o, 0, s0);
    arrive();
    fetch(o, 1, s1);
    read(o, s0, a, 0);
    int t = 0;
    for (; t + 2 <= steps; t += 2) {
      half0(o, s0, a, b, acc);
      arrive();
      half1(o, t + 2, s0, s1, a, b, acc);
      half0(o, s1, a, b, acc);
      arrive();
      half1(o, t + 3, s1, s0, a, b, acc);
    }
    if (t < steps) {
      half0(o, s0, a, b, acc);
      multiply<T, XQ>(b, acc);
    }
  } else {
    // few blocks, so latency counts: loads run kBuffers - 1 steps ahead
    constexpr int ahead = T::kBuffers - 1;
#pragma unroll
    for (int t = 0; t < ahead; ++t) fetch(o, t, shared + t * T::kBuf);
    for (int t = 0; t < steps; t += T::kBuffers) {
#pragma unroll
      for (int u = 0; u < T::kBuffers; ++u) {
        if (t + u >= steps) break;
        arrive_but<(ahead - 1) * (T::BM / T::kRows + (XQ ? kBK / T::kRowsX : T::BN / T::kRows))>();
        one_step(o, t + u + ahead, shared + (u + ahead) % T::kBuffers * T::kBuf,
                 shared + u * T::kBuf, acc);
      }
    }
  }
  arrive();  // shared memory is free again
}

struct GemmArgs {
  Common c;
  MuonIo io;
  float ca, cb, cc;   // kPoly: ca I + cb S + cc S S
  int32_t in0, in1, out;  // symmetric matrices (kApply: in0)
  int32_t turn;       // which X
  int32_t early;      // kApply, one product: small singular values still grow
};
static_assert(sizeof(GemmArgs) <= kArgBytes, "arguments of a launch");

// Blocks go to the 8 XCDs in turn; each XCD takes runs of `run` consecutive
// tiles, which share rows of their operands in its cache.
__device__ __forceinline__ int tile_index(int run) {
  const int b = blockIdx.x, whole = gridDim.x / (8 * run) * (8 * run);
  if (b >= whole) return b;
  const int x = b & 7, k = b >> 3;
  return (k / run * 8 + x) * run + k % run;
}

constexpr int kApplyRun = 8;  // of the application: a column of tiles of X

__device__ __forceinline__ int row_of(int b) {  // of place b in a triangle by rows
  int i = (int)((sqrtf(8.0f * (float)b + 1.0f) - 1.0f) * 0.5f);
  while ((i + 1) * (i + 2) / 2 <= b) ++i;
  while (i * (i + 1) / 2 > b) --i;
  return i;
}

// Tile b of the lower triangle of rows x rows tiles, in squares of SUPER x
// SUPER: neighbours share rows and columns.
template <int SUPER>
__device__ __forceinline__ void tri_tile(int b, int rows, int& ti, int& tj) {
  const int i0 = row_of(b) / SUPER * SUPER;  // rows before a row of squares come first
  const int o = b - i0 * (i0 + 1) / 2, h = min(SUPER, rows - i0), square = o / (h * SUPER);
  const int r = o - square * h * SUPER;
  if (square * SUPER < i0) {
    ti = i0 + r % h;
    tj = square * SUPER + r / h;
  } else {
    const int i = row_of(r);
    ti = i0 + i;
    tj = i0 + r - i * (i + 1) / 2;
  }
}

constexpr int kCus = 256;
constexpr int kBig = 0, kMiddle = 1, kLittle = 2;  // places of the tile sizes in the tables
typedef Tile<256, 256, 2, 4, 2> Big;
typedef Tile<128, 128, 2, 2, 2> Middle;
typedef Tile<64, 64, 2, 2, 4> Little;

// The waves of a square of results may read what the others wrote.
template <typename T>
__device__ __forceinline__ void square_ready() {
  if constexpr (T::kSquareWaves == 1) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  } else {
    __syncthreads();
  }
}

__device__ __forceinline__ f16x4 halves(const float (&v)[4]) {
  return (f16x4){(f16)v[0], (f16)v[1], (f16)v[2], (f16)v[3]};
}
__device__ __forceinline__ f16x4 rests(const float (&v)[4], f16x4 h) {
  return (f16x4){rest_of(v[0], h[0]), rest_of(v[1], h[1]), rest_of(v[2], h[2]),
                 rest_of(v[3], h[3])};
}

// Entry (i, j) of a product of two symmetric matrices diag(D) + O, from the
// sum over the 16-bit parts (times 2^20), the scaled parts o0, o1 of either,
// and their diagonals: D0_i O1_ij + O0_ij D1_j + sum, scaled; on the diagonal
// D0_i D1_i + sum.  POLY (both the same matrix S): ca I + cb S + cc S S.
template <bool POLY>
__device__ __forceinline__ float combine(float sum, float o0, float o1, float d0i, float d1j,
                                         bool on, float ca, float cb, float cc) {
  if constexpr (POLY) {
    if (on) return (ca + d1j * (cb + cc * d1j)) * kScale + cc * kUnscale * sum;
    return __builtin_fmaf(o0, __builtin_fmaf(cc, d0i + d1j, cb), cc * kUnscale * sum);
  } else {
    if (on) return __builtin_fmaf(d0i * d1j, kScale, sum * kUnscale);
    return __builtin_fmaf(d0i, o1, __builtin_fmaf(o0, d1j, sum * kUnscale));
  }
}

// D_i X_ij + sum, X_ij from its two halves.  One product: the products take
// the upper half alone, so the lower one gets `rest` instead of D_i.
template <int PRODUCTS>
__device__ __forceinline__ float linear(f16 hi, f16 lo, float d, float rest, float sum) {
  if constexpr (PRODUCTS > 1) return __builtin_fmaf(d, join(hi, lo), sum);
  return __builtin_fmaf(rest * (1.0f / kLo), (float)lo, __builtin_fmaf(d, (float)hi, sum));
}

// x, without its element r if this piece is the one on the diagonal.
__device__ __forceinline__ f16x8 off_diagonal(f16x8 x, bool on, int r) {
  u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (on && r >> 1 == k) w[k] &= r & 1 ? 0xFFFFu : 0xFFFF0000u;
  return __builtin_bit_cast(f16x8, w);
}

// Three products instead of one: hi lo + lo hi, scaled down, + hi hi.  Two: P
// hi alone, Q's both halves.
template <typename T, bool XQ, int PRODUCTS, typename F>
__device__ __forceinline__ void products(F operands, f16* shared,
                                         f32x4 (&acc)[T::FI][T::FJ]) {
#pragma unroll
  for (int i = 0; i < T::FI; ++i)
#pragma unroll
    for (int j = 0; j < T::FJ; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
#pragma unroll 1
  for (int pass = 0; pass < PRODUCTS; ++pass) {
    if (PRODUCTS > 1 && pass == PRODUCTS - 1) {
#pragma unroll
      for (int i = 0; i < T::FI; ++i)
#pragma unroll
        for (int j = 0; j < T::FJ; ++j) acc[i][j] = acc[i][j] * (1.0f / kLo);
    }
    product(operands(PRODUCTS == 3 && pass == 1, PRODUCTS > 1 && pass == 0), shared, acc);
  }
}

// Symmetric results, lower tiles only, written to both places:
//   kGram  S_out = X X^T
//   kPoly  S_out = ca I + cb S + cc S S, S = S_in0
//   kMul   S_out = S_in0 S_in1 (which commute: polynomials of one matrix)
// A symmetric matrix is diag(D) + O, with O in 16 bits.
// Two layers of hidden 2048 / intermediate 8192 (14 matrices), a symmetric
// result counted once: kGram 310 us, 785 TFLOP/s; kPoly and kMul 128 us, 675.
// The main loops alone take 250 and 78 us; the rest is the epilogue's traffic
// and the last round of blocks, which is partly empty.  1024 x 1024: 8.6 us
// each, a launch and the latency of 16 steps.
enum Mode { kGram, kPoly, kMul };

template <typename T, int SIZE, int MODE, int PRODUCTS>
__global__ __launch_bounds__(T::kThreads, 2) void zf_ns_sym(GemmArgs a) {
  if (a.c.st && a.c.st->skipped) return;
  __shared__ __align__(16) f16 shared[T::kBuf * T::kBuffers];
  const int w = tile_index(T::kRun);
  const Mat& m = find(a.c, w, [](const Mat& x) { return x.tri0[SIZE]; });
  int ti, tj;
  tri_tile<4>(w - m.tri0[SIZE], (m.mp + T::BM - 1) / T::BM, ti, tj);
  const int mp = m.mp, i0 = ti * T::BM, j0 = tj * T::BN;
  const int64_t ld = MODE == kGram ? m.ldx : m.lds;
  const int len = MODE == kGram ? m.np : mp;

  f32x4 acc[T::FI][T::FJ];
  products<T, false, PRODUCTS>(
      [&](bool lo_p, bool lo_q) {
        const int64_t p = MODE == kGram ? (lo_p ? m.l[a.turn] : m.h[a.turn])
                                        : (lo_p ? m.sl[a.in0] : m.s[a.in0]);
        const int64_t q = MODE == kGram ? (lo_q ? m.l[a.turn] : m.h[a.turn])
                                        : (lo_q ? m.sl[a.in1] : m.s[a.in1]);
        return Operands<T, false>(at<f16>(a.c, p) + i0 * ld, ld, mp - i0,
                                  at<f16>(a.c, q) + j0 * ld, ld, mp - j0, len);
      },
      shared, acc);

  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = i0 + wave / T::kWavesJ * T::TI, wj = j0 + wave % T::kWavesJ * T::TJ;
  const f16* o0 = at<f16>(a.c, m.s[a.in0]);
  const f16* o1 = at<f16>(a.c, m.s[a.in1]);
  const f16* r0 = at<f16>(a.c, m.sl[a.in0]);
  const f16* r1 = at<f16>(a.c, m.sl[a.in1]);
  const float* d0 = at<float>(a.c, m.d[a.in0]);
  const float* d1 = at<float>(a.c, m.d[a.in1]);
  f16* out = at<f16>(a.c, m.s[a.out]);
  f16* rest = at<f16>(a.c, m.sl[a.out]);
  float* diag = at<float>(a.c, m.d[a.out]);
  // 64 x 64 sums at a time through shared memory (row j, 16-byte piece c at
  // c ^ (j & 7)) into values by rows of whole 128-byte lines; the values'
  // 16-bit halves then take the sums' place (row j, piece c at c ^ 2 (j & 3))
  // and go out along the other axis, transposed on the way
  constexpr int E = 8 / T::kSquareWaves;  // lines of 8 rows a wave takes
  const int e0 = T::share_of(wi - i0, wj - j0) * E;
  ZF_LDS char* square = (ZF_LDS char*)(shared) + T::square_of(wi - i0, wj - j0) * 16384;
  const int ri = (wi - i0) % 64, rj = (wj - j0) % 64;  // this wave's place in its square
  static_assert(T::kBuf * T::kBuffers * 2 >= T::kWaves / T::kSquareWaves * 16384, "squares of 64 fit");
  const int row = lane >> 3, c = lane & 7;
#pragma unroll
  for (int q = 0; q < (T::FI + 3) / 4; ++q) {
    const int si = wi - ri + q * 64, sj = wj - rj;  // the square
    const bool in = si < mp && sj < mp;
    const int64_t p0 = (int64_t)(sj + e0 * 8 + row) * m.lds + si + c * 8;
    float di[8], dj[E];
    if (MODE != kGram && in) {
#pragma unroll
      for (int r = 0; r < 8; ++r) di[r] = d0[si + c * 8 + r];
#pragma unroll
      for (int e = 0; e < E; ++e) dj[e] = d1[sj + (e0 + e) * 8 + row];
    }
#pragma unroll
    for (int f = 0; f < (T::FI < 4 ? T::FI : 4); ++f)
#pragma unroll
      for (int fj = 0; fj < T::FJ; ++fj)
        *(ZF_LDS f32x4*)(square + (rj + fj * 16 + l) * 256 +
                         ((ri / 4 + f * 4 + g) ^ (l & 7)) * 16) = acc[q * 4 + f][fj];
    square_ready<T>();
    if (si == sj && in && lane / (E * 8) == e0 / E) {  // the diagonal, before its place is reused
      const float sum = *(const ZF_LDS float*)(square + lane * 256 +
                                               ((lane >> 2) ^ (lane & 7)) * 16 + (lane & 3) * 4);
      float v = sum * kUnscale;
      if constexpr (MODE != kGram)
        v = combine<MODE == kPoly>(sum, 0.0f, 0.0f, d0[si + lane], d1[si + lane], true, a.ca, a.cb,
                                   a.cc);
      diag[si + lane] = v * kUnscale;
    }
    f16x8 low[E];
    constexpr int kBatch = E < 4 ? E : 4;  // lines whose loads are on their way together
#pragma unroll
    for (int eb = 0; eb < E; eb += kBatch) {
      if (!in) break;
      f16x8 x0[kBatch], x1[kBatch], y0[kBatch], y1[kBatch];
      if constexpr (MODE != kGram) {
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int64_t p = p0 + (int64_t)(eb + e) * 8 * m.lds;
          x0[e] = *reinterpret_cast<const f16x8*>(o0 + p);
          if constexpr (MODE == kMul) x1[e] = *reinterpret_cast<const f16x8*>(o1 + p);
          if constexpr (PRODUCTS == 3) {
            y0[e] = *reinterpret_cast<const f16x8*>(r0 + p);
            if constexpr (MODE == kMul) y1[e] = *reinterpret_cast<const f16x8*>(r1 + p);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int j = (e0 + eb + e) * 8 + row;  // in the square
        ZF_LDS char* line = square + j * 256;
        float v[8], sum[8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const f32x4 x = *(const ZF_LDS f32x4*)(line + ((2 * c + t) ^ row) * 16);
#pragma unroll
          for (int r = 0; r < 4; ++r) sum[t * 4 + r] = x[r];
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if constexpr (MODE == kGram) {
            v[r] = sum[r] * kUnscale;
          } else {
            const float a0 = PRODUCTS == 3 ? join(x0[e][r], y0[e][r]) : (float)x0[e][r];
            float a1 = a0;
            if constexpr (MODE == kMul)
              a1 = PRODUCTS == 3 ? join(x1[e][r], y1[e][r]) : (float)x1[e][r];
            v[r] = combine<MODE == kPoly>(sum[r], a0, a1, di[r], dj[eb + e], false, a.ca, a.cb, a.cc);
          }
        }
        f16x8 hi;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          hi[r] = (f16)v[r];
          if constexpr (PRODUCTS == 3) low[eb + e][r] = rest_of(v[r], hi[r]);
        }
        if (si == sj) {
          hi = off_diagonal(hi, c == e0 + eb + e, row);
          if constexpr (PRODUCTS == 3)
            low[eb + e] = off_diagonal(low[eb + e], c == e0 + eb + e, row);
        }
        const int64_t p = p0 + (int64_t)(eb + e) * 8 * m.lds;
        *reinterpret_cast<f16x8*>(out + p) = hi;
        if constexpr (PRODUCTS == 3) *reinterpret_cast<f16x8*>(rest + p) = low[eb + e];
        *(ZF_LDS f16x8*)(line + (c ^ (2 * (row & 3))) * 16) = hi;
      }
    }
#pragma unroll
    for (int half = 0; half < (PRODUCTS == 3 ? 2 : 1); ++half) {
      if (half == 1) {
        square_ready<T>();
#pragma unroll
        for (int e = 0; e < E; ++e)
          *(ZF_LDS f16x8*)(square + ((e0 + e) * 8 + row) * 256 + (c ^ (2 * (row & 3))) * 16) =
              low[e];
      }
      square_ready<T>();
      if (ti == tj || !in) continue;  // on the diagonal both places lie in this tile
#pragma unroll
      for (int k = 0; k < E; ++k) {
        // 16 lines of 32 values: in each group of 16 lanes, source lane (row
        // e, piece k) hands over 4 values along i, and lane l receives those
        // of i = l along j
        const int ib = (e0 + k) / 2, jb = (e0 + k) % 2 * 32 + 8 * g;
        s16x4 x[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
          x[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (ZF_LDS s16x4*)(square + (jb + 4 * t + (l >> 2)) * 256 +
                              ((ib * 2 + ((l & 3) >> 1)) ^ (2 * (l >> 2))) * 16 + (l & 1) * 8));
        const int64_t p = (int64_t)(si + ib * 16 + l) * m.lds + sj + jb;
        *reinterpret_cast<f16x8*>((half ? rest : out) + p) = __builtin_bit_cast(
            f16x8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
    square_ready<T>();
  }
}

// A wave's 64 x 64 results at (i0, j0) of X, from shared memory (scaled, laid
// out as in zf_ns_apply), to the destination, whose rows run along j, or for
// a tall matrix along i: 64 neighbours an instruction, at any alignment.
// Lines first .. first + count - 1 of it (rows of the destination).  DST is
// the result's type; MUON: W <- W dec - rate (result), and the 16-bit
// parameters of type DST (0: none).
template <int DST, bool MUON>
__device__ __forceinline__ void write_square(const GemmArgs& a, const Mat& m,
                                             const ZF_LDS float* square, int i0, int j0, int first,
                                             int count) {
  const int lane = threadIdx.x & 63;
  const int rows = min(m.tall ? m.n - j0 : m.m - i0, 64);
  const int cols = m.tall ? m.m - i0 : m.n - j0;
  const int64_t at = (int64_t)(m.tall ? j0 : i0) * m.dst_ld + (m.tall ? i0 : j0) + lane;
  if (lane >= cols) return;
  const float rate = m.rate * kUnscale;
  constexpr int kBatch = 8;  // rows whose loads are on their way together
  for (int k = first; k < min(rows, first + count); k += kBatch) {
    float v[kBatch], w[kBatch];
    if (m.tall) {
#pragma unroll
      for (int e = 0; e < kBatch; e += 4) {
        const f32x4 x = *(const ZF_LDS f32x4*)(square + lane * 64 + (((k + e) / 4) ^ (lane & 7)) * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[e + r] = x[r];
      }
    } else {
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        v[e] = square[(k + e) * 64 + ((lane >> 2) ^ e) * 4 + (lane & 3)];  // k: a multiple of 8
    }
    if constexpr (MUON) {
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        w[e] = k + e < rows ? a.io.master[m.flat + at + (k + e) * m.dst_ld] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      if (k + e >= rows) break;
      const int64_t p = at + (k + e) * m.dst_ld;
      if constexpr (MUON) {
        const float x = w[e] * a.io.dec - rate * v[e];
        a.io.master[m.flat + p] = x;
        if constexpr (DST != 0) static_cast<uint16_t*>(a.io.params)[m.flat + p] = narrow1<DST>(x);
      } else if constexpr (DST == ZF_F32) {
        static_cast<float*>(m.dst)[p] = v[e] * kUnscale;
      } else {
        static_cast<uint16_t*>(m.dst)[p] = narrow1<DST>(v[e] * kUnscale);
      }
    }
  }
}

// The same for the Muon step where rows of the weights keep 16-byte alignment:
// 4 rows of 64 weights an instruction, 32 rows on their way together (a row
// an instruction, 8 together: 602 us instead of 344 for the last product of
// 71M weights, where the others, without 6 bytes an element, take 241).
template <int DST, int LINES>
__device__ __forceinline__ void update_square(const GemmArgs& a, const Mat& m,
                                              const ZF_LDS float* square, int i0, int j0,
                                              int first) {
  const int lane = threadIdx.x & 63, r = lane >> 4, c = lane & 15;
  const int rows = min(m.tall ? m.n - j0 : m.m - i0, 64);
  const int cols = m.tall ? m.m - i0 : m.n - j0;
  if (c * 4 >= cols) return;
  const int64_t at = m.flat + (int64_t)(m.tall ? j0 : i0) * m.dst_ld + (m.tall ? i0 : j0) + c * 4;
  const float rate = m.rate * kUnscale;
  constexpr int kBatch = LINES < 32 ? LINES / 4 : 8;
#pragma unroll 1
  for (int k = first + r; k < first + LINES; k += 4 * kBatch) {
    f32x4 w[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      w[e] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(
          a.io.master + at + min(k + 4 * e, rows - 1) * m.dst_ld));
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int row = k + 4 * e;
      if (row >= rows) break;
      f32x4 v;
      if (m.tall) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          v[t] = square[(c * 4 + t) * 64 + ((row >> 2) ^ ((c * 4 + t) & 7)) * 4 + (row & 3)];
      } else {
        v = *(const ZF_LDS f32x4*)(square + row * 64 + (c ^ (row & 7)) * 4);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = w[e][t] * a.io.dec - rate * v[t];
      const int64_t p = at + row * m.dst_ld;
      __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(a.io.master + p));
      if constexpr (DST != 0) {
        const u32x2 q = {pack2<DST>(v[0], v[1]), pack2<DST>(v[2], v[3])};
        __builtin_nontemporal_store(
            q, reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.io.params) + p));
      }
    }
  }
}

// X <- S X with S = S_in0: D_i X_ij from both halves of X, and O X; LAST:
// into the destination, or W <- W dec - rate (S X).
// The same two layers: 590 us, 820 TFLOP/s; the main loop alone 414 us, the
// rest is 8 bytes an element in and out after it (14 with Muon's weights).
// Starting the XCDs or the blocks apart from each other, so that these do not
// come at once, gains nothing: rows of X leave the second-level caches.
template <typename T, int SIZE, bool LAST, int PRODUCTS, int DST, bool MUON>
__global__ __launch_bounds__(T::kThreads, 2) void zf_ns_apply(GemmArgs a) {
  if (a.c.st && a.c.st->skipped) return;
  __shared__ __align__(16) f16 shared[T::kBuf * T::kBuffers];
  const int w = tile_index(kApplyRun);
  const Mat& m = find(a.c, w, [](const Mat& x) { return x.app0[SIZE]; });
  const int b = w - m.app0[SIZE], tiles_m = (m.mp + T::BM - 1) / T::BM;
  const int ti = b % tiles_m, tj = b / tiles_m;
  const int mp = m.mp, np = m.np, i0 = ti * T::BM, j0 = tj * T::BN;

  f32x4 acc[T::FI][T::FJ];
  products<T, true, PRODUCTS>(
      [&](bool lo_p, bool lo_q) {
        const int64_t p = lo_p ? m.sl[a.in0] : m.s[a.in0];
        const int64_t q = lo_q ? m.l[a.turn] : m.h[a.turn];
        return Operands<T, true>(at<f16>(a.c, p) + (int64_t)i0 * m.lds, m.lds, mp - i0,
                                 at<f16>(a.c, q) + j0, m.ldx, j0, mp);
      },
      shared, acc);

  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = i0 + wave / T::kWavesJ * T::TI, wj = j0 + wave % T::kWavesJ * T::TJ;
  const f16* h = at<f16>(a.c, m.h[a.turn]);
  const f16* lo = at<f16>(a.c, m.l[a.turn]);
  f16* h1 = at<f16>(a.c, m.h[a.turn ^ 1]);
  f16* lo1 = at<f16>(a.c, m.l[a.turn ^ 1]);
  const float* d = at<float>(a.c, m.d[a.in0]);
  constexpr int E = 8 / T::kSquareWaves;  // lines of 8 rows a wave takes
  const int e0 = T::share_of(wi - i0, wj - j0) * E;
  ZF_LDS float* square = (ZF_LDS float*)(shared) + T::square_of(wi - i0, wj - j0) * 4096;
  const int ri = (wi - i0) % 64, rj = (wj - j0) % 64;  // this wave's place in its square
  static_assert(T::kBuf * T::kBuffers * 2 >= T::kWaves / T::kSquareWaves * 16384, "squares of 64 fit");
#pragma unroll
  for (int q = 0; q < (T::FI + 3) / 4; ++q) {
    // 64 x 64 of O X to shared memory, and back by rows of whole 128-byte
    // lines: the 16-byte piece c of row i lies at piece c ^ (i & 7)
    const int si = wi - ri + q * 64, sj = wj - rj;
    const bool in = si < mp && sj < np;
    const int row = lane >> 3, c = lane & 7;
    const int64_t p0 = (int64_t)(si + e0 * 8 + row) * m.ldx + sj + c * 8;
    f16x8 x[E], y[E];
    float di[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (!in) break;
      x[e] = *reinterpret_cast<const f16x8*>(h + p0 + (int64_t)e * 8 * m.ldx);
      y[e] = *reinterpret_cast<const f16x8*>(lo + p0 + (int64_t)e * 8 * m.ldx);
      di[e] = d[si + (e0 + e) * 8 + row];
    }
#pragma unroll
    for (int f = 0; f < (T::FI < 4 ? T::FI : 4); ++f)
#pragma unroll
      for (int fj = 0; fj < T::FJ; ++fj)
        *(ZF_LDS f32x4*)(square + (ri + f * 16 + l) * 64 +
                         ((rj / 4 + fj * 4 + g) ^ (l & 7)) * 4) = acc[q * 4 + f][fj];
    square_ready<T>();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (!in) break;
      ZF_LDS float* s = square + ((e0 + e) * 8 + row) * 64;
      f16x8 hi, rest;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        ZF_LDS f32x4* piece = (ZF_LDS f32x4*)(s + ((2 * c + t) ^ row) * 4);
        f32x4 v = *piece * kUnscale;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[r] = linear<PRODUCTS>(x[e][t * 4 + r], y[e][t * 4 + r], di[e],
                                  a.early ? a.ca : di[e], v[r]);
          if constexpr (!LAST) {
            hi[t * 4 + r] = (f16)v[r];
            rest[t * 4 + r] = rest_of(v[r], hi[t * 4 + r]);
          }
        }
        if constexpr (LAST) *piece = v;
      }
      if constexpr (!LAST) {
        *reinterpret_cast<f16x8*>(h1 + p0 + (int64_t)e * 8 * m.ldx) = hi;
        *reinterpret_cast<f16x8*>(lo1 + p0 + (int64_t)e * 8 * m.ldx) = rest;
      }
    }
    square_ready<T>();
    if constexpr (LAST) {
      bool wide = false;
      if constexpr (MUON) {
        wide = ((m.flat | m.dst_ld) & 3) == 0;
        if (in && wide) update_square<DST, E * 8>(a, m, square, si, sj, e0 * 8);
      }
      if (in && !wide) write_square<DST, MUON>(a, m, square, si, sj, e0 * 8, E * 8);
      square_ready<T>();
    }
  }
}

template <int MODE, int PRODUCTS>
void launch_sym(const Group& g, int size, hipStream_t s, const GemmArgs& a) {
  const dim3 grid(g.tri_blocks[size]);
  if (size == kBig)
    hipLaunchKernelGGL((zf_ns_sym<Big, kBig, MODE, PRODUCTS>), grid, dim3(Big::kThreads), 0, s, a);
  else if (size == kMiddle)
    hipLaunchKernelGGL((zf_ns_sym<Middle, kMiddle, MODE, PRODUCTS>), grid, dim3(Middle::kThreads),
                       0, s, a);
  else
    hipLaunchKernelGGL((zf_ns_sym<Little, kLittle, MODE, PRODUCTS>), grid, dim3(Little::kThreads),
                       0, s, a);
}

template <bool LAST, int PRODUCTS, int DST, bool MUON>
void launch_apply(const Group& g, int size, hipStream_t s, const GemmArgs& a) {
  const dim3 grid(g.app_blocks[size]);
  if constexpr (PRODUCTS == 2) {  // short sides of one tile
    hipLaunchKernelGGL((zf_ns_apply<Little, kLittle, LAST, PRODUCTS, DST, MUON>),
                       dim3(g.app_blocks[kLittle]), dim3(Little::kThreads), 0, s, a);
  } else if (size == kBig)
    hipLaunchKernelGGL((zf_ns_apply<Big, kBig, LAST, PRODUCTS, DST, MUON>), grid,
                       dim3(Big::kThreads), 0, s, a);
  else if (size == kMiddle)
    hipLaunchKernelGGL((zf_ns_apply<Middle, kMiddle, LAST, PRODUCTS, DST, MUON>), grid,
                       dim3(Middle::kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((zf_ns_apply<Little, kLittle, LAST, PRODUCTS, DST, MUON>), grid,
                       dim3(Little::kThreads), 0, s, a);
}

template <int PRODUCTS>
void launch_last(const Group& g, int size, hipStream_t s, int32_t dst, bool muon,
                 const GemmArgs& a) {
  if (muon) {
    if (!a.io.params) launch_apply<true, PRODUCTS, 0, true>(g, size, s, a);
    else if (dst == ZF_BF16) launch_apply<true, PRODUCTS, ZF_BF16, true>(g, size, s, a);
    else launch_apply<true, PRODUCTS, ZF_F16, true>(g, size, s, a);
  } else if (dst == ZF_BF16) {
    launch_apply<true, PRODUCTS, ZF_BF16, false>(g, size, s, a);
  } else if (dst == ZF_F16) {
    launch_apply<true, PRODUCTS, ZF_F16, false>(g, size, s, a);
  } else {
    launch_apply<true, PRODUCTS, ZF_F32, false>(g, size, s, a);
  }
}

// The iteration of one group.  Two steps may run as a pair on the m x m side
// (X_2 = Q_2 Q_1 X with A_2 = Q_1 A Q_1), which touches the long side once for
// both and costs no more products when n = m: five single steps take 20 m^3 +
// 15 m^2 (n - m) operations, every pair 3 m^2 (n - m) less.  A pair sees the
// small singular values through their squares, which A's rounding drowns, so
// pairs and single steps take turns.
//   Three products: 2, 1, 2, as exact as single steps but for short sides
// under 32 (7 x 1198: 3e-6 against 1.5e-6).
//   One product: 2, 1, 1, 1, for short sides of kPairSide and more: errors up to
// 1.5e-3 at 64 to 600, as with single steps, but 1.7e-3 at 48, 2.0e-3 at 32 and
// 5e-3 at 11, where single steps keep 1.6e-3.  A later pair costs accuracy at
// any size: with 2, 1, 2 half of the directions strong come to 3.2e-3 at 600 x
// 600 (single steps 1.0e-3).  Single steps throughout are 11 percent slower for
// two layers of hidden 2048, 2, 1, 2 is 10 percent faster.
// The number of products and the short side decide, so that a matrix's result
// does not depend on the others of the call.
template <int PRODUCTS, int APPLY>
int iterate(const Group& g, const Mat* mats, const zf_ns_params& p, int sym, int app, int32_t dst,
            bool muon, hipStream_t s, GemmArgs a) {
  auto firsts = [&](int32_t (*of)(const Mat&, int), int size) {
    for (int k = 0; k < kFirsts; ++k) a.c.firsts[k] = k < g.count ? of(mats[k], size) : INT32_MAX;
  };
  const auto tri = [](const Mat& m, int size) { return m.tri0[size]; };
  const auto along = [](const Mat& m, int size) { return m.app0[size]; };
  a.turn = 0;
  bool pair = g.pairs;
  for (int k = 0; k < p.steps;) {
    const int n = pair && k + 2 <= p.steps - (PRODUCTS == 3 ? 0 : kLast) ? 2 : 1;
    pair = PRODUCTS == 3 && n == 1;
    a.ca = (float)p.a;
    a.cb = (float)p.b;
    a.cc = (float)p.c;
    auto op = [&](int in0, int in1, int out) {
      a.in0 = in0;
      a.in1 = in1;
      a.out = out;
    };
    firsts(tri, sym);
    op(0, 0, 0);
    launch_sym<kGram, PRODUCTS>(g, sym, s, a);  // 0 = A
    op(0, 0, 1);
    launch_sym<kPoly, PRODUCTS>(g, sym, s, a);  // 1 = Q
    if (n == 2) {
      op(1, 0, 2);
      launch_sym<kMul, PRODUCTS>(g, sym, s, a);   // 2 = Q A
      op(1, 2, 0);
      launch_sym<kMul, PRODUCTS>(g, sym, s, a);   // 0 = Q Q A: the next A
      op(0, 0, 2);
      launch_sym<kPoly, PRODUCTS>(g, sym, s, a);  // 2 = the next Q
      op(2, 1, 0);
      launch_sym<kMul, PRODUCTS>(g, sym, s, a);   // 0 = their product
    }
    a.in0 = n == 2 ? 0 : 1;
    a.early = k + kLast < p.steps;
    if (n == 2) a.ca *= a.ca;
    firsts(along, app);
    k += n;
    if (k == p.steps) launch_last<APPLY>(g, app, s, dst, muon, a);
    else launch_apply<false, APPLY, ZF_F32, false>(g, app, s, a);
    a.turn ^= 1;
    if (!hip_ok(hipGetLastError())) return ZF_EHIP;
  }
  return ZF_OK;
}

// The tile size for a launch of n[kBig] tiles of 256 x 256 (one block a CU),
// n[kMiddle] of 128 x 128 or n[kLittle] of 64 x 64 (two a CU): whichever takes
// the least time, counted in rounds over the 256 CUs.  A full round takes 68,
// 37 and 14 us at 2048 x 2048, 44, 26 and 9.6 at 1024 x 1024; one that is
// nearly empty about half of that.
int tile_size(const int32_t (&n)[3]) {
  const int slots[3] = {kCus, 2 * kCus, 2 * kCus};
  const double round[3] = {1.76, 1.0, 0.375};
  double least = 0.0;
  int best = kBig;
  for (int z = 0; z < 3; ++z) {
    const double part = (double)(n[z] % slots[z]) / slots[z];
    const double cost = round[z] * (n[z] / slots[z] + (part > 0.0 ? 0.5 + 0.5 * part : 0.0));
    if (z == 0 || cost < least) {
      least = cost;
      best = z;
    }
  }
  return best;
}

// ---------------------------------------------------------------------------
// Small matrices: the whole iteration in one block, X and one symmetric
// matrix in shared memory, one launch for all of them.  Such a matrix would
// spend its time in launches (128 x 128: 20 of them, 190 us); here a step is
// three products between barriers (58 us, with three products for each 98).
// Each of the 8 waves takes a block of 2 x
// CJ tiles of 16 x 16 of X (2 x 4 of S, both triangles: cheaper than
// mirroring one), so that a fragment read from shared memory serves several
// tiles; tiles past the last one are computed again (no branches) and not
// stored, and waves without a tile only wait.  Bound by the instructions
// around the products, two waves of 4 cycles each on a SIMD, and the barriers.
constexpr int kSmallPad = 32;              // sides padded to this
constexpr int kSmallThreads = 512, kSmallWaves = 8;
constexpr int kSmallShared = 147456;       // bytes of X and S
constexpr int kSmallSide = 128;            // longest short side
constexpr int kSmallByValue = 12;          // matrices that travel as arguments

struct SmallArgs {
  const Mat* table;         // or NULL: the matrices are m[]
  const DevState* st;       // the Muon step's skip flag, or NULL
  MuonIo io;
  float ca, cb, cc;
  double eps;
  int32_t steps, src, dst;  // types; src 0: the Muon step
  Mat m[kSmallByValue];
};
static_assert(sizeof(SmallArgs) <= kArgBytes, "arguments of a launch");

// Waves along the short side (each takes 2 tiles of it), the rest along the
// long one.
__host__ __device__ inline int small_waves_i(int mp) { return mp <= 32 ? 1 : mp <= 64 ? 2 : 4; }

// A thread's elements k = tid, tid + 512, ... of the matrix, walked by row
// and column.
struct SmallWalk {
  int r, c, dr, dc, cols;
  __device__ __forceinline__ explicit SmallWalk(int columns) : cols(columns) {
    r = threadIdx.x / cols;
    c = threadIdx.x % cols;
    dr = kSmallThreads / cols;
    dc = kSmallThreads % cols;
  }
  __device__ __forceinline__ void next() {
    r += dr;
    c += dc;
    if (c >= cols) c -= cols, ++r;
  }
  __device__ __forceinline__ void skip();  // kSmallBatch elements
};
constexpr int kSmallBatch = 32;  // elements of a thread whose loads are on their way together

__device__ __forceinline__ void SmallWalk::skip() {
  const int k = r * cols + c + kSmallBatch * kSmallThreads;
  r = k / cols;
  c = k % cols;
}

// The next kSmallBatch elements of the walk, from memory (the type decides
// outside the loop, so that the loads do not wait for each other); FIRST: the
// Muon step's momentum update on the way.  Zeros past the last row.
template <bool FIRST>
__device__ __forceinline__ void small_batch(const SmallArgs& a, const Mat& m, SmallWalk w,
                                            int rows, float (&v)[kSmallBatch]) {
  auto each = [&](auto f) {
    SmallWalk at = w;
#pragma unroll
    for (int e = 0; e < kSmallBatch; ++e, at.next())
      f(e, min(at.r, rows - 1) * m.src_ld + at.c, at.r < rows);
  };
  if (a.src == 0) {
    const float gs = a.st->gs;
    const float* sums = a.io.sums + m.flat;
    float* momentum = a.io.momentum + m.flat;
    float g[kSmallBatch];
    each([&](int e, int64_t p, bool) { v[e] = momentum[p], g[e] = sums[p]; });
    each([&](int e, int64_t p, bool in) {
      g[e] = g[e] * gs;
      if constexpr (FIRST) {
        v[e] = a.io.mu * v[e] + g[e];
        if (in) momentum[p] = v[e];
      }
      if (a.io.nesterov) v[e] = g[e] + a.io.mu * v[e];
    });
  } else if (a.src == ZF_F32) {
    each([&](int e, int64_t p, bool) { v[e] = static_cast<const float*>(m.src)[p]; });
  } else {
    uint16_t x[kSmallBatch];
    each([&](int e, int64_t p, bool) { x[e] = static_cast<const uint16_t*>(m.src)[p]; });
#pragma unroll
    for (int e = 0; e < kSmallBatch; ++e)
      v[e] = a.src == ZF_BF16 ? widen1<ZF_BF16>(x[e]) : widen1<ZF_F16>(x[e]);
  }
  each([&](int e, int64_t, bool in) { v[e] = in ? v[e] : 0.0f; });
}

__device__ __forceinline__ void small_store(const SmallArgs& a, const Mat& m, int64_t r, int64_t c,
                                            float v) {
  const int64_t p = r * m.dst_ld + c;
  void* out = m.dst;
  int64_t q = p;
  if (a.src == 0) {
    q = m.flat + p;
    v = a.io.master[q] * a.io.dec - m.rate * v;
    a.io.master[q] = v;
    out = a.io.params;
    if (!out) return;
  }
  if (a.dst == ZF_F32) static_cast<float*>(out)[q] = v;
  else static_cast<uint16_t*>(out)[q] = a.dst == ZF_BF16 ? narrow1<ZF_BF16>(v) : narrow1<ZF_F16>(v);
}

template <int CJ, int PRODUCTS>
__global__ __launch_bounds__(kSmallThreads) void zf_ns_small(SmallArgs a) {
  if (a.st && a.st->skipped) return;
  const Mat& m = a.table ? a.table[blockIdx.x] : a.m[blockIdx.x];
  const int mp = (m.m + kSmallPad - 1) / kSmallPad * kSmallPad;
  const int np = (m.n + kSmallPad - 1) / kSmallPad * kSmallPad;
  // row strides that put 16 rows' pieces in different banks
  const int lx = np + 8, ls = mp + 8;
  __shared__ __align__(16) f16 shared[kSmallShared / 2];
  __shared__ __align__(16) float diag[kSmallSide];
  __shared__ double sum[kSmallWaves];
  f16* xh = shared;
  f16* xl = xh + mp * lx;
  f16* sh = xl + mp * lx;
  f16* sl = sh + mp * ls;
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rows = m.tall ? m.n : m.m, cols = m.tall ? m.m : m.n;

  // one batch of a thread's elements stays in registers until the norm is
  // known; a matrix of more is read twice
  float v[kSmallBatch];
  const SmallWalk start(cols);
  double ss = 0.0;
  for (SmallWalk w = start; w.r < rows; w.skip()) {
    small_batch<true>(a, m, w, rows, v);
#pragma unroll
    for (int e = 0; e < kSmallBatch; ++e) ss += (double)v[e] * (double)v[e];
  }
  for (int k = tid; k < mp * lx / 4; k += kSmallThreads)
    reinterpret_cast<f32x4*>(xh)[k] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) ss = ss + __shfl_xor(ss, off, 64);
  if (lane == 0) sum[wave] = ss;
  __syncthreads();
  ss = sum[0];
#pragma unroll
  for (int w = 1; w < kSmallWaves; ++w) ss = ss + sum[w];
  const double inv = 1.0 / (sqrt(ss) + a.eps) * kScale;
  const bool once = rows * cols <= kSmallBatch * kSmallThreads;
  for (SmallWalk w = start; w.r < rows; w.skip()) {
    if (!once) small_batch<false>(a, m, w, rows, v);
    SmallWalk to = w;
#pragma unroll
    for (int e = 0; e < kSmallBatch; ++e, to.next()) {
      if (to.r >= rows) continue;
      const float x = (float)((double)v[e] * inv);
      const int p = m.tall ? to.c * lx + to.r : to.r * lx + to.c;
      const f16 h = (f16)x;
      xh[p] = h;
      xl[p] = rest_of(x, h);
    }
  }
  __syncthreads();

  const int tm = mp / 16, tn = np / 16, waves_i = small_waves_i(mp);
  const int i0 = wave % waves_i * 2, js = wave / waves_i * 4, jx = wave / waves_i * CJ;

  // S = P P^T for P of `len` columns and row stride ld; finish(i, j, diagonal
  // tile, sums) turns the sums (times 2^20) of (i .. i + 3, j) into values
  const bool holds_s = i0 < tm && js < tm, holds_x = i0 < tm && jx < tn;
  auto symmetric = [&](const f16* ph, const f16* pl, int ld, int len, auto finish) {
    f32x4 acc[2][4], low[2][4];
    int pi[2], pj[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) pi[i] = (min(i0 + i, tm - 1) * 16 + l) * ld + 8 * g;
#pragma unroll
    for (int j = 0; j < 4; ++j) pj[j] = (min(js + j, tm - 1) * 16 + l) * ld + 8 * g;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = low[i][j] = (f32x4){0, 0, 0, 0};
    for (int k = holds_s ? 0 : len; k < len; k += 32) {
      f16x8 x[2], y[4], xr[2], yr[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = *reinterpret_cast<const f16x8*>(ph + pi[i] + k);
        if constexpr (PRODUCTS == 3) xr[i] = *reinterpret_cast<const f16x8*>(pl + pi[i] + k);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = *reinterpret_cast<const f16x8*>(ph + pj[j] + k);
        if constexpr (PRODUCTS == 3) yr[j] = *reinterpret_cast<const f16x8*>(pl + pj[j] + k);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[i], y[j], acc[i][j], 0, 0, 0);
          if constexpr (PRODUCTS == 3) {
            low[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[i], yr[j], low[i][j], 0, 0, 0);
            low[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xr[i], y[j], low[i][j], 0, 0, 0);
          }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i0 + i >= tm || js + j >= tm) continue;
        const int ii = (i0 + i) * 16 + 4 * g, jj = (js + j) * 16 + l;
        if constexpr (PRODUCTS == 3) acc[i][j] = acc[i][j] + low[i][j] * (1.0f / kLo);
        finish(ii, jj, i0 + i == js + j, acc[i][j]);
      }
    __syncthreads();  // every read of the old S is done
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i0 + i >= tm || js + j >= tm) continue;
        // (i, j) goes to (j, i): S is symmetric, and this way in one piece
        const int ii = (i0 + i) * 16 + 4 * g, jj = (js + j) * 16 + l;
        float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        if (i0 + i == js + j) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (ii + r != jj) continue;
            diag[jj] = v[r] * kUnscale;
            v[r] = 0.0f;
          }
        }
        const f16x4 h = halves(v);
        *reinterpret_cast<f16x4*>(sh + jj * ls + ii) = h;
        if constexpr (PRODUCTS == 3) *reinterpret_cast<f16x4*>(sl + jj * ls + ii) = rests(v, h);
      }
    __syncthreads();
  };

#pragma unroll 1
  for (int step = 0; step < a.steps; ++step) {
    symmetric(xh, xl, lx, np, [&](int, int, bool, f32x4& v) { v = v * kUnscale; });
    symmetric(sh, sl, ls, mp, [&](int i, int j, bool diagonal, f32x4& v) {
      const float dj = diag[j];
      const f32x4 di = *reinterpret_cast<const f32x4*>(diag + i);
      const f16x4 h = *reinterpret_cast<const f16x4*>(sh + j * ls + i);
      f16x4 w = h;
      if constexpr (PRODUCTS == 3) w = *reinterpret_cast<const f16x4*>(sl + j * ls + i);
      float sum[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = PRODUCTS == 3 ? join(h[r], w[r]) : (float)h[r];
        sum[r] = v[r];
        v[r] = combine<true>(sum[r], e, e, di[r], dj, false, a.ca, a.cb, a.cc);
      }
      if (diagonal) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (i + r == j) v[r] = combine<true>(sum[r], 0.0f, 0.0f, di[r], dj, true, a.ca, a.cb, a.cc);
      }
    });
    const bool last = step + 1 == a.steps;
    f32x4 acc[2][CJ], low[2][CJ];
    int pi[2], pj[CJ];
#pragma unroll
    for (int i = 0; i < 2; ++i) pi[i] = (min(i0 + i, tm - 1) * 16 + l) * ls + 8 * g;
#pragma unroll
    for (int j = 0; j < CJ; ++j)
      pj[j] = (8 * g + (l >> 2)) * lx + min(jx + j, tn - 1) * 16 + 4 * (l & 3);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < CJ; ++j) acc[i][j] = low[i][j] = (f32x4){0, 0, 0, 0};
    auto turned = [&](const f16* x) {
      const s16x4 h0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZF_LDS s16x4*)(x));
      const s16x4 h1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZF_LDS s16x4*)(x + 4 * lx));
      return __builtin_bit_cast(f16x8, __builtin_shufflevector(h0, h1, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    for (int k = holds_x ? 0 : mp; k < mp; k += 32) {
      f16x8 x[CJ], xr[CJ], y[2], yr[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        y[i] = *reinterpret_cast<const f16x8*>(sh + pi[i] + k);
        if constexpr (PRODUCTS == 3) yr[i] = *reinterpret_cast<const f16x8*>(sl + pi[i] + k);
      }
#pragma unroll
      for (int j = 0; j < CJ; ++j) {
        x[j] = turned(xh + pj[j] + k * lx);
        xr[j] = turned(xl + pj[j] + k * lx);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[j], y[i], acc[i][j], 0, 0, 0);
          if constexpr (PRODUCTS == 3)
            low[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[j], yr[i], low[i][j], 0, 0, 0);
          low[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xr[j], y[i], low[i][j], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!holds_x) break;
      const int ii = min(i0 + i, tm - 1) * 16 + l;
      const float di = diag[ii];
#pragma unroll
      for (int j = 0; j < CJ; ++j) {
        const int p = ii * lx + min(jx + j, tn - 1) * 16 + 4 * g;
        const f16x4 h = *reinterpret_cast<const f16x4*>(xh + p);
        const f16x4 w = *reinterpret_cast<const f16x4*>(xl + p);
        acc[i][j] = acc[i][j] + low[i][j] * (1.0f / kLo);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][r] = __builtin_fmaf(di, join(h[r], w[r]), acc[i][j][r] * kUnscale);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < CJ; ++j) {
        if (i0 + i >= tm || jx + j >= tn) continue;
        const int ii = (i0 + i) * 16 + l, jj = (jx + j) * 16 + 4 * g;
        const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        if (last) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (ii < m.m && jj + r < m.n)
              small_store(a, m, m.tall ? jj + r : ii, m.tall ? ii : jj + r, v[r] * kUnscale);
        } else {
          const f16x4 h = halves(v);
          *reinterpret_cast<f16x4*>(xh + ii * lx + jj) = h;
          *reinterpret_cast<f16x4*>(xl + ii * lx + jj) = rests(v, h);
        }
      }
    __syncthreads();
  }
}

// Tiles along the long side that each wave would take, or 0 for a matrix too
// large for a block.
int small_tiles(int64_t m, int64_t n) {
  if (m > kSmallSide || n > 4096) return 0;
  const int64_t mp = (m + kSmallPad - 1) / kSmallPad * kSmallPad;
  const int64_t np = (n + kSmallPad - 1) / kSmallPad * kSmallPad;
  if (mp * (np + 8 + mp + 8) * 4 > kSmallShared) return 0;
  const int64_t along = kSmallWaves / small_waves_i((int)mp);
  const int64_t tiles = (np / 16 + along - 1) / along;
  return tiles <= 8 ? (int)tiles : 0;
}

template <int PRODUCTS>
void launch_small(const Layout& l, hipStream_t s, const SmallArgs& a) {
  const dim3 grid(l.small_count), block(kSmallThreads);
  if (l.small_tiles <= 1) hipLaunchKernelGGL((zf_ns_small<1, PRODUCTS>), grid, block, 0, s, a);
  else if (l.small_tiles <= 4)
    hipLaunchKernelGGL((zf_ns_small<4, PRODUCTS>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((zf_ns_small<8, PRODUCTS>), grid, block, 0, s, a);
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Matrices are worked on in groups whose buffers share one region, so that
// the workspace of a large model stays bounded: a group closes at this many
// padded elements.
constexpr int64_t kGroupElements = 1ll << 28;
constexpr int64_t kMaxSide = 1ll << 20;
// Partials that every block of the next launch sums by itself, where blocks
// are few: two a thread, a microsecond, against four for a launch of their
// own.  (With many blocks that microsecond comes again and again: 8 layers of
// hidden 1024, 120 -> 167 us.)
constexpr int64_t kOwnNorm = 512;

constexpr int kPairSide = 64;  // shortest side of pairs with one product

// Classes of matrices: one product by single steps (short sides of one tile)
// or a pair first, three products, held in shared memory.
enum { kSingle, kPairs, kThree, kHeld, kClasses };
static_assert(kPairSide <= Little::BM, "short sides of one tile");

int small_tiles_of(const zf::ns::Shape& s) {
  return small_tiles(std::min(s.rows, s.cols), std::max(s.rows, s.cols));
}

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

bool zf::ns::layout(const Shape* shapes, int64_t count, int products, int32_t thin, Layout& out) {
  out.mats.resize((size_t)count);
  out.groups.clear();
  out.shortest = INT32_MAX;
  int64_t partials = 0, region = 0, used = 0, elements = 0;
  Group g{};
  int64_t load = 0, tri[3] = {}, app[3] = {}, all_blocks = 0;
  auto close = [&]() {
    // tiles a block takes: one while that leaves CUs without a block
    g.load_tiles = load >= 4096 ? kLoadTiles : 1;
    g.own_norm = g.load_tiles == 1;
    int64_t blocks = 0;
    for (int32_t k = g.first; k < g.first + g.count; ++k) {
      Mat& m = out.mats[(size_t)k];
      const int64_t tiles = (int64_t)(m.mp / kTile) * (m.np / kTile);
      if (tiles > kOwnNorm) g.own_norm = 0;
      m.part = partials;
      partials += tiles;
      m.load0 = (int32_t)blocks;
      blocks += (tiles + g.load_tiles - 1) / g.load_tiles;
    }
    g.load_blocks = (int32_t)blocks;
    for (int z = 0; z < 3; ++z) {
      g.tri_blocks[z] = (int32_t)tri[z];
      g.app_blocks[z] = (int32_t)app[z];
      tri[z] = app[z] = 0;
    }
    all_blocks += g.app_blocks[kLittle];
    out.groups.push_back(g);
    region = std::max(region, used);
    const int32_t next = g.first + g.count;
    g = Group{};
    g.first = next;
    used = elements = load = 0;
  };
  auto take = [&](int64_t bytes) {
    const int64_t o = used;
    used += round_up(bytes, 256);
    return o;
  };
  auto class_of = [&](const Shape& s) {
    if (small_tiles_of(s) > 0) return kHeld;
    const int64_t m = std::min(s.rows, s.cols), n = std::max(s.rows, s.cols);
    // one block walks a thin matrix's whole sum: 16 x 16384 takes 490 us with
    // three products instead of 295, 16 x 262144 6.5 ms instead of 3.7
    if (products == 3 || (m <= thin && n <= kCus * kPad)) return kThree;
    return m >= kPairSide ? kPairs : kSingle;
  };
  int64_t of_class[kClasses] = {};
  for (int64_t k = 0; k < count; ++k) {
    if (shapes[k].rows > kMaxSide || shapes[k].cols > kMaxSide) return false;
    ++of_class[class_of(shapes[k])];
  }
  const int64_t large = count - of_class[kHeld];
  out.small_first = (int32_t)large;
  out.small_count = (int32_t)of_class[kHeld];
  out.small_tiles = 0;
  int64_t placed = 0;
  for (int c = 0; c < kClasses; ++c) for (int64_t k = 0; of_class[c] > 0 && k < count; ++k) {
    if (class_of(shapes[k]) != c) continue;
    const int64_t rows = shapes[k].rows, cols = shapes[k].cols;
    Mat& m = out.mats[(size_t)placed++];
    m = Mat{};
    m.slot = (int32_t)k;
    m.src_ld = m.dst_ld = cols;
    m.tall = rows > cols;
    m.m = (int32_t)std::min(rows, cols);
    m.n = (int32_t)std::max(rows, cols);
    m.mp = (int32_t)round_up(m.m, kPad);
    m.np = (int32_t)round_up(m.n, kPad);
    if (c == kHeld) {
      out.small_tiles = std::max(out.small_tiles, small_tiles_of(shapes[k]));
      continue;
    }
    out.shortest = std::min(out.shortest, m.m);
    m.ldx = m.np;
    m.lds = m.mp;
    const int64_t mn = (int64_t)m.mp * m.ldx, mm = (int64_t)m.mp * m.lds;
    if (g.count > 0 && (g.kind != c || elements + mn > kGroupElements)) close();
    g.kind = c;
    g.products = c == kThree ? 3 : 1;
    g.pairs = c != kSingle;
    // what the rounding left of X: an operand of the products if there are
    // three, else used by its own tile alone, in place
    for (int z = 0; z < 2; ++z) {
      m.h[z] = take(mn * 2);
      m.l[z] = z == 0 || g.products == 3 ? take(mn * 2) : m.l[0];
    }
    for (int z = 0; z < 3; ++z) {
      m.s[z] = take(mm * 2);
      m.sl[z] = g.products == 3 ? take(mm * 2) : m.s[z];
      m.d[z] = take((int64_t)m.mp * 4);
    }
    const int64_t tiles = (int64_t)(m.mp / kTile) * (m.np / kTile);
    if (tiles > 0x7FFFFFFF) return false;
    load += tiles;  // blocks follow when the group is whole
    const int side[3] = {Big::BM, Middle::BM, Little::BM};
    for (int z = 0; z < 3; ++z) {
      const int64_t tm = (m.mp + side[z] - 1) / side[z], tn = (m.np + side[z] - 1) / side[z];
      m.tri0[z] = (int32_t)tri[z];
      m.app0[z] = (int32_t)app[z];
      tri[z] += tm * (tm + 1) / 2;
      app[z] += tm * tn;
    }
    if (load > 0x7FFFFFFF) return false;
    elements += mn;
    ++g.count;
  }
  if (g.count > 0) close();
  out.one_round = all_blocks <= kCus;
  int64_t at = 0;
  out.table = at;
  at += round_up(count * (int64_t)sizeof(Mat), 256);
  out.inv = at;
  at += round_up(count * 8, 256);
  out.partials = at;
  at += round_up(partials * 8, 256);
  for (Mat& m : out.mats) {
    for (int z = 0; z < 2; ++z) m.h[z] += at, m.l[z] += at;
    for (int z = 0; z < 3; ++z) m.s[z] += at, m.sl[z] += at, m.d[z] += at;
  }
  out.bytes = at + region;
  return true;
}

int zf::ns::enqueue(const Layout& l, const zf_ns_params& p, int small_products, int32_t src_dtype,
                    int32_t dst_dtype, const MuonIo* io, char* ws, hipStream_t s) {
  Mat* table = reinterpret_cast<Mat*>(ws + l.table);
  // a few small matrices, and a few large ones, go as arguments and need no
  // table
  const bool by_value = l.small_count <= kSmallByValue;
  size_t tabled = l.mats.size() - (by_value ? l.small_count : 0);
  if (by_value && tabled <= kByValue) tabled = 0;
  for (size_t k = 0; k < tabled; k += kTableChunk) {
    TableArgs t;
    t.to = table + k;
    t.count = (int32_t)std::min<size_t>(kTableChunk, tabled - k);
    for (int i = 0; i < t.count; ++i) t.m[i] = l.mats[k + i];
    hipLaunchKernelGGL(zf_ns_table, dim3(1), dim3(64), 0, s, t);
    if (!hip_ok(hipGetLastError())) return ZF_EHIP;
  }
  if (l.small_count > 0) {
    SmallArgs a;
    a.table = by_value ? nullptr : table + l.small_first;
    for (int k = 0; by_value && k < l.small_count; ++k) a.m[k] = l.mats[l.small_first + k];
    a.st = io ? io->st : nullptr;
    a.io = io ? *io : MuonIo{};
    a.ca = (float)p.a;
    a.cb = (float)p.b;
    a.cc = (float)p.c;
    a.eps = p.eps;
    a.steps = p.steps;
    a.src = io ? 0 : src_dtype;
    a.dst = dst_dtype;
    if (small_products == 3) launch_small<3>(l, s, a);
    else launch_small<1>(l, s, a);
    if (!hip_ok(hipGetLastError())) return ZF_EHIP;
  }
  for (const Group& g : l.groups) {
    LoadArgs la;
    Common& c = la.c;
    c.ws = ws;
    c.table = table + g.first;
    c.count = g.count;
    c.load_tiles = g.load_tiles;
    c.st = io ? io->st : nullptr;
    c.inv = reinterpret_cast<double*>(ws + l.inv);
    c.partials = reinterpret_cast<double*>(ws + l.partials);
    c.eps = p.eps;
    for (int k = 0; k < kFirsts; ++k)
      c.firsts[k] = k < g.count ? l.mats[g.first + k].load0 : INT32_MAX;
    for (int k = 0; k < kByValue && k < g.count; ++k) c.m[k] = l.mats[g.first + k];
    la.io = io ? *io : MuonIo{};
    const dim3 load(g.load_blocks), block(kThreads);
    const int32_t src = io ? 0 : src_dtype;
    if (src == 0) hipLaunchKernelGGL(zf_ns_load<0>, load, block, 0, s, la);
    else if (src == ZF_F32) hipLaunchKernelGGL(zf_ns_load<ZF_F32>, load, block, 0, s, la);
    else if (src == ZF_BF16) hipLaunchKernelGGL(zf_ns_load<ZF_BF16>, load, block, 0, s, la);
    else hipLaunchKernelGGL(zf_ns_load<ZF_F16>, load, block, 0, s, la);
    if (!g.own_norm) hipLaunchKernelGGL(zf_ns_norm, dim3(g.count), block, 0, s, c);
    launch_prep(src, g.own_norm, load, s, la);
    if (!hip_ok(hipGetLastError())) return ZF_EHIP;

    GemmArgs ga;
    ga.c = c;
    ga.io = la.io;
    const int sym = tile_size(g.tri_blocks);
    const int app = g.kind == kSingle ? kLittle : tile_size(g.app_blocks);
    const auto run = g.kind == kThree ? iterate<3, 3> : g.kind == kPairs ? iterate<1, 1> : iterate<1, 2>;
    const int rc = run(g, l.mats.data() + g.first, p, sym, app, dst_dtype, io != nullptr, s, ga);
    if (rc != ZF_OK) return rc;
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
  return zf::ns::layout(shapes.data(), count, products, 0, l) ? ZF_OK : ZF_ESIZE;
}

// Two results in one place, or a result in another matrix's place, which
// launches in no given order would mix.  (Partial overlaps are the caller's.)
bool distinct(const zf_matrix* mats, int64_t count) {
  std::vector<std::pair<const void*, int64_t>> at((size_t)count);
  for (int64_t k = 0; k < count; ++k) at[(size_t)k] = {mats[k].dst, k};
  std::sort(at.begin(), at.end());
  for (int64_t k = 1; k < count; ++k)
    if (at[(size_t)k].first == at[(size_t)k - 1].first) return false;
  for (int64_t k = 0; k < count; ++k) {
    const std::pair<const void*, int64_t> src(mats[k].src, 0);
    const auto z = std::lower_bound(at.begin(), at.end(), src);
    if (z != at.end() && z->first == mats[k].src && z->second != k) return false;
  }
  return true;
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
    }
    if (!distinct(mats, count)) return ZF_EINVAL;
    for (Mat& m : l.mats) {
      const zf_matrix& z = mats[m.slot];
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
