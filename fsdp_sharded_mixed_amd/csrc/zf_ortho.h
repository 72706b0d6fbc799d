// zf_ortho.h -- the Newton-Schulz engine shared by zf_orthogonalize and the
// Muon step: the work layout of a batch of matrices in a device workspace,
// and the sequence of launches over it.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <vector>

#include "zf.h"
#include "zf_internal.h"

namespace zf {
namespace ns {

// The work layout.  A matrix of R x C is iterated on its short side: X is
// m x n with m = min(R, C), n = max(R, C), the transpose of the matrix when
// R > C ("tall").  Both sides are padded with zeros to multiples of kPad, so
// that no load of the products needs a range check along the summed axis.
constexpr int kPad = 64;

// One matrix: where its data come from and where its buffers lie (byte
// offsets into the workspace).
struct Mat {
  const void* src;        // zf_orthogonalize: the matrix, row stride src_ld
  void* dst;              // zf_orthogonalize: the result, row stride dst_ld
  int64_t src_ld, dst_ld; // the Muon step: both = cols
  int64_t flat;           // the Muon step: offset in the padded flat arrays
  int64_t h[2], l[2];     // fp16 [mp][ldx]: X * 2^10 rounded, and what the
                          // rounding left; two buffers in turn (one product:
                          // l in place)
  int64_t s[3], sl[3];    // fp16 [mp][lds]: symmetric matrices off the
                          // diagonal, rounded, and what that left
  int64_t d[3];           // fp32 [mp]: their diagonals
  int64_t part;           // its first squared-norm partial
  int32_t m, n, mp, np;
  int32_t ldx, lds;       // row strides of X and of the symmetric matrices
  int32_t tall, slot;     // slot: its place in the call
  float rate;             // the Muon step: lr * scale
  int32_t load0;          // its first block in the launches of its group,
  int32_t tri0[3], app0[3];  // by tile size
};

// Launches of one group of matrices [first, first + count).
struct Group {
  int32_t first, count;
  int32_t load_tiles;     // 64 x 64 tiles a block of the load takes
  int32_t kind;           // its matrices' class
  int32_t products;       // 1 or 3
  int32_t pairs;          // steps in pairs on the short side
  int32_t own_norm;       // few enough partials for every block to sum them
  int32_t load_blocks, tri_blocks[3], app_blocks[3];
};

struct Layout {
  std::vector<Mat> mats;      // Mat.slot: the matrix's place in the call
  std::vector<Group> groups;
  int32_t small_first = 0, small_count = 0;  // matrices held in shared memory,
  int32_t small_tiles = 0;                   // and the most tiles of a wave
  // the others' X lie in one round of blocks, where every launch is mostly
  // latency, and their shortest side
  bool one_round = true;
  int32_t shortest = INT32_MAX;
  int64_t table = 0, inv = 0, partials = 0;  // byte offsets
  int64_t bytes = 0;
};

struct Shape {
  int64_t rows, cols;
};

// Plans the buffers of `count` matrices; products: 1, or 3 with the second
// 16-bit halves; thin: with one product, a matrix with a side of at most this
// takes three all the same, unless it is too long.  false: a size out of
// range.
bool layout(const Shape* shapes, int64_t count, int products, int32_t thin, Layout& out);

// Products a call computes: the caller's choice, or by the result's type.
int products_of(const zf_ns_params& p, int32_t dst_dtype);
// ZF_OK, or ZF_EINVAL for parameters out of range.
int check_params(const zf_ns_params& p);
zf_ns_params defaults();

// What the Muon step reads and writes beside the products.
struct MuonIo {
  const float* sums;
  float* master;
  float* momentum;
  void* params;           // or NULL
  const DevState* st;
  float mu, dec;
  int32_t nesterov, param_dtype;
};

// Enqueues the orthogonalisation of every matrix of `l` on `s`.  io == NULL:
// from Mat.src (src_dtype) to Mat.dst (dst_dtype); else the Muon update.
// small_products: of the matrices held in shared memory.
int enqueue(const Layout& l, const zf_ns_params& p, int small_products, int32_t src_dtype,
            int32_t dst_dtype, const MuonIo* io, char* ws, hipStream_t s);

}  // namespace ns
}  // namespace zf
