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
//
// Bound by the matrix cores where the result is large: 16384 tokens, 8192 x 2048,
// bf16 added to fp32: 448 to 507 us, by the card and its clock, 1228 to 1084
// TFLOP/s (the library's product of 16-bit operands, without decoding or adding, on
// the cards where this takes 456 to 472 us: 462 to 485; its best, 8192^3, 1385
// TFLOP/s).  Where it is small, by a stage's instructions, of which one wave a SIMD
// issues one in four cycles: 0.28 us a stage and block, for 128 cycles of products.
// 16384 tokens, 256 x 1024: 23.5 to 26 us, the join 4.1 of them (the library's 98);
// 333 tokens, 777 x 1000: 8.6.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "zf_hip_status.h"
#include "zf_rows.h"

namespace {

using namespace zf::dev;
using zf::hip_ok;
using zf::kThreads;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
#define ZF_LDS __attribute__((address_space(3)))

// A stage is 32 tokens; kStages of them lie in shared memory in turn, the loads of
// three on their way.  Six or eight in tiles of 64 x 128: no faster (333 of 776 x
// 1008 7.5, 7.5 and 7.8 us; 16384 of 256 x 1024 28.7, 29.8 and 29.9).
constexpr int kStages = 4, kDepth = 32;

template <int BM_, int BN_, int WI, int WJ>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, kThreads = WI * WJ * 64, kWavesJ = WJ;
  static constexpr int TI = BM / WI, TJ = BN / WJ, FI = TI / 16, FJ = TJ / 16;
  static constexpr int kShared = kStages * kDepth * (BM + BN) * 2;  // operands, or squares of results
  static constexpr int kSquare = TI < 64 ? TI : 64;  // rows of a square of results, 64 columns wide
  static_assert(kShared >= WI * WJ * kSquare * 256, "squares fit");
  static_assert(TJ % 64 == 0 && TI % kSquare == 0, "squares");
};
typedef Tile<64, 128, 2, 2> Little;
typedef Tile<128, 128, 2, 2> Middle;
typedef Tile<256, 256, 2, 4> Big;
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef __amdgpu_buffer_rsrc_t Rsrc;

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

// Results leave by whole lines: a wave's squares of 64 x 64 (or 32 x 64) go to
// shared memory (16-byte pieces permuted by the row, for the banks) and out
// again 8 columns a lane, with one piece of code for every type.
// acc[i][j][r] is row l, column 4 g + r of a 16 x 16 square.
template <typename T>
__device__ __forceinline__ void write_tile(const GradArgs& a, const f32x4 (&acc)[T::FI][T::FJ], char* shared,
                                           int i0, int j0, int split) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  ZF_LDS float* square = (ZF_LDS float*)shared + wave * T::kSquare * 64;
  float* partial = a.partial ? a.partial + (int64_t)split * a.out * a.in : nullptr;
  const int32_t gdt = partial ? (int32_t)ZF_F32 : a.gdt;
  void* to = partial ? partial : a.grad;
  const bool add = a.accumulate && !partial;
  const int c = lane & 7;
#pragma unroll
  for (int q = 0; q < T::TI / T::kSquare * (T::TJ / 64); ++q) {
    const int qi = q / (T::TJ / 64), qj = q % (T::TJ / 64);
    const int j = j0 + wave % T::kWavesJ * T::TJ + qj * 64 + c * 8, n = a.in - j;
#pragma unroll
    for (int f = 0; f < T::kSquare / 16; ++f)
#pragma unroll
      for (int fj = 0; fj < 4; ++fj)
        *(ZF_LDS f32x4*)(square + (f * 16 + l) * 64 + ((fj * 4 + g) ^ (l & 7)) * 4) =
            acc[qi * (T::kSquare / 16) + f][qj * 4 + fj];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int o0 = i0 + wave / T::kWavesJ * T::TI + qi * T::kSquare;
#pragma unroll 1
    for (int r = lane >> 3; r < T::kSquare; r += 8) {
      if (o0 + r >= a.out || n <= 0) break;
      const int64_t at = (int64_t)(o0 + r) * a.in + j;
      float v[kChunk], old[kChunk];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 x = *(ZF_LDS f32x4*)(square + r * 64 + ((2 * c + h) ^ (r & 7)) * 4);
        v[h * 4] = x.x;
        v[h * 4 + 1] = x.y;
        v[h * 4 + 2] = x.z;
        v[h * 4 + 3] = x.w;
      }
      if (add) {
        load8_of(gdt, to, at, n, old);
#pragma unroll
        for (int k = 0; k < kChunk; ++k) v[k] += old[k];
      }
      if (gdt == ZF_F32) store8<ZF_F32>(to, at, n, v);
      else if (gdt == ZF_BF16) store8<ZF_BF16>(to, at, n, v);
      else store8<ZF_F16>(to, at, n, v);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// Blocks go to the 8 XCDs in turn.  Each XCD takes runs of consecutive places,
// as many as it works on at a time, and consecutive places form squares of 8 x
// 8 tiles, which share rows of their operands in its cache; the splits follow
// one another.
struct Place {
  int i, j, split;
  __device__ __forceinline__ explicit Place(const GradArgs& a) {
    const int all = gridDim.x, run = min(max(all / 8, 1), 64), whole = all / (8 * run) * (8 * run);
    int b = blockIdx.x;
    if (b < whole) b = (b / 8 / run * 8 + b % 8) * run + b / 8 % run;
    split = b / a.tiles;
    b -= split * a.tiles;
    const int i8 = b / (8 * a.tiles_in) * 8, h = min(8, a.tiles / a.tiles_in - i8);
    b -= i8 * a.tiles_in;
    const int j8 = b / (8 * h) * 8, w = min(8, a.tiles_in - j8);
    b -= j8 * h;
    i = i8 + b / w;
    j = j8 + b % w;
  }
};

// Where a matrix's next kStages stages lie: the address of their first row in this
// tile's columns, and the rows that are left.  Loads past the matrix's end give
// zeros (in shared memory too), so tokens behind the last one add nothing; loads
// past a row's end give elements of columns that are not written.  A turn of
// kStages has one buffer, so that a stage computes no addresses: with one for
// each stage, its scalar arithmetic is a third of a small tile's instructions.
struct Walk {
  const char* at;
  int64_t ld;          // bytes of a stride
  int32_t left, tail;  // rows; bytes of a row from here on
  uint32_t n;          // bytes of the turn's buffer

  __device__ __forceinline__ Walk(const void* base, int64_t row, int64_t rows, int64_t row_bytes, int64_t skip,
                                  int64_t width) {
    at = static_cast<const char*>(base) + row * row_bytes + skip;
    left = (int32_t)rows;
    ld = row_bytes;
    tail = (int32_t)(width - skip);
    n = extent();
  }
  __device__ __forceinline__ uint32_t extent() const {
    const int32_t rows = min(left, kStages * kDepth);
    return rows > 0 ? (uint32_t)(rows - 1) * (uint32_t)ld + (uint32_t)tail : 0u;
  }
  __device__ __forceinline__ Rsrc buffer() const {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), 0, n, 0x00020000);
  }
  __device__ __forceinline__ void turn() {
    at += kStages * kDepth * ld;
    left -= kStages * kDepth;
    n = extent();
  }
};
// An offset that all lanes share, clamped: the hardware compares a lane's own
// offset with n less the shared one, which must not wrap.
__device__ __forceinline__ int within(uint32_t at, uint32_t n) { return (int)min(at, n); }

// (The compiler's pass over the host code does not know the 16-byte form.)
__device__ __forceinline__ void to_shared(Rsrc from, ZF_LDS char* to, int lane_at, int at) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (ZF_LDS void*)to, 16, lane_at, at, 0, 0);
#endif
}

// DIRECT: operands in whole 16-byte pieces.  Gradients then go from global to
// shared memory directly; otherwise through registers, as the codes do.
template <typename T, int DT, bool DIRECT>
struct Pipe {
  static constexpr int kPBytes = kDepth * T::BM * 2, kQBytes = kDepth * T::BN * 2;
  static constexpr int kBuf = kPBytes + kQBytes;
  static constexpr int kPRows = T::kThreads / (T::BM / 8);   // rows that a load of all threads covers
  static constexpr int kPLoads = kDepth / kPRows;
  static_assert(kPRows % 16 == 0, "the rows of a lane's loads are permuted alike");
  static_assert(T::kThreads / (T::BN / 16) == kDepth, "16 codes a thread");
  static constexpr int kLoads = kPLoads + 2;  // of a thread and stage
  static constexpr int kInFlight = DIRECT ? 2 + 2 * kLoads : 63;  // see stage()

  Walk p, q, s;  // gradients, codes, scales
  int vp, vq, vs, wp, wq, rp, rq;
  int prow, qrow;
  const char *gp, *gq, *gs, *p_end, *q_end;  // !DIRECT: this lane's pieces, the matrices' ends

  // What a thread has of a stage in registers.
  struct Held {
    u32x4 c;
    uint32_t scale;
    u32x4 g[DIRECT ? 1 : kPLoads];
  };

  __device__ __forceinline__ Pipe(const GradArgs& a, int i0, int j0, int64_t first, int64_t rows)
      : p(a.dy, first, rows, a.dy_ld * 2, (int64_t)i0 * 2, (int64_t)a.out * 2),
        q(a.x.codes, first, rows, a.x.code_ld, j0, a.in),
        s(a.x.scales, first, rows, a.x.scale_ld, j0 / ZF_ACT8_GROUP, (a.in + ZF_ACT8_GROUP - 1) / ZF_ACT8_GROUP) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & 15, g = lane >> 4;
    // shared memory is filled in order, so a lane loads the piece that belongs
    // at its place
    prow = tid / (T::BM / 8);
    qrow = tid / (T::BN / 16);
    const int at = place<T::BM / 8>(prow, tid % (T::BM / 8)) % (T::BM * 2), piece = tid % (T::BN / 16);
    wq = kPBytes + place<T::BN / 8>(qrow, piece * 2);
    if constexpr (DIRECT) {
      vp = prow * (int)p.ld + at;
      vq = qrow * (int)q.ld + piece * 16;
      vs = qrow * (int)s.ld + piece * 16 / ZF_ACT8_GROUP;
    } else {
      const int64_t row = first + prow, column = min(j0 + piece * 16, a.in - 1);
      wp = tid * 16;
      gp = static_cast<const char*>(a.dy) + (row * a.dy_ld + i0) * 2 + at;
      gq = reinterpret_cast<const char*>(a.x.codes) + (first + qrow) * a.x.code_ld + j0 + piece * 16;
      gs = reinterpret_cast<const char*>(a.x.scales) + (first + qrow) * a.x.scale_ld + column / ZF_ACT8_GROUP;
      p_end = static_cast<const char*>(a.dy) + ((a.rows - 1) * a.dy_ld + a.out) * 2;
      q_end = reinterpret_cast<const char*>(a.x.codes) + (a.rows - 1) * a.x.code_ld + a.in;
    }
    const int frow = 8 * g + (l >> 2), half = (l & 3) >> 1, wi = wave / T::kWavesJ * T::TI,
              wj = wave % T::kWavesJ * T::TJ;
    rp = place<T::BM / 8>(frow, wi / 8 + half) + (l & 1) * 8;
    rq = kPBytes + place<T::BN / 8>(frow, wj / 8 + half) + (l & 1) * 8;
  }

  // the turn's next kStages stages
  __device__ __forceinline__ void turn() {
    if constexpr (DIRECT) {
      p.turn();
      q.turn();
      s.turn();
    }
  }
  // gradients of the turn's stage e into `buf`
  __device__ __forceinline__ void fetch_p(char* __restrict buf, int e) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Rsrc from = p.buffer();
    ZF_LDS char* to = (ZF_LDS char*)buf + wave * 1024;
#pragma unroll
    for (int h = 0; h < kPLoads; ++h)
      to_shared(from, to + h * T::kThreads * 16, vp, within((e * kDepth + h * kPRows) * (uint32_t)p.ld, p.n));
  }
  // codes of the turn's stage e (!DIRECT: codes and gradients of the next stage)
  // into registers.  INSIDE: none of the stage's pieces ends past its matrix, and
  // all its tokens are there.
  template <bool INSIDE>
  __device__ __forceinline__ void fetch(Held& r, int e) {
    if constexpr (DIRECT) {
      r.c = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
          q.buffer(), vq, within(e * kDepth * (uint32_t)q.ld, q.n), 0));
      r.scale = __builtin_amdgcn_raw_buffer_load_b8(s.buffer(), vs, within(e * kDepth * (uint32_t)s.ld, s.n), 0);
    } else if constexpr (INSIDE) {
#pragma unroll
      for (int h = 0; h < kPLoads; ++h) r.g[h] = load_any<false, u32x4_any>(gp + h * kPRows * p.ld);
      r.c = load_any<false, u32x4_any>(gq);
      r.scale = *reinterpret_cast<const uint8_t*>(gs);
      advance();
    } else {
      // A piece that ends past its row holds the next row's first elements, for
      // columns that are not written; only one that ends past the matrix is
      // loaded in parts.  Tokens behind the last one are zeros.
#pragma unroll
      for (int h = 0; h < kPLoads; ++h) {
        r.g[h] = (u32x4){0, 0, 0, 0};
        const char* at = gp + h * kPRows * p.ld;
        const bool in = prow + h * kPRows < p.left;
        if (in && at + 16 <= p_end) r.g[h] = load_any<false, u32x4_any>(at);
        if (rare(in && at + 16 > p_end))
          r.g[h] = load_raw<ZF_BF16>(at, 0, (int)max((p_end - at) / 2, (int64_t)0)).w[0];
      }
      r.c = (u32x4){0, 0, 0, 0};
      r.scale = 127;
      const bool in = qrow < q.left;
      if (in) r.scale = *reinterpret_cast<const uint8_t*>(gs);
      if (in && gq + 16 <= q_end) r.c = load_any<false, u32x4_any>(gq);
      if (rare(in && gq + 16 > q_end)) {
        const int n = (int)max(q_end - gq, (int64_t)0);
        const uint8_t* at = reinterpret_cast<const uint8_t*>(gq);
        const u32x2 lo = load_codes(at, min(8, n)), hi = load_codes(at + 8, n - 8);
        r.c = (u32x4){lo.x, lo.y, hi.x, hi.y};
      }
      advance();
    }
  }
  __device__ __forceinline__ void advance() {
    gp += kDepth * p.ld;
    gq += kDepth * q.ld;
    gs += kDepth * s.ld;
    p.left -= kDepth;
    q.left -= kDepth;
  }
  // codes as 16-bit numbers (!DIRECT: and gradients) into `buf`
  __device__ __forceinline__ void put(char* __restrict buf, const Held& r) const {
    const float scale = __uint_as_float(r.scale << 23);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const u32x4 x = {decode2<DT, false>(r.c[e * 2], scale), decode2<DT, true>(r.c[e * 2], scale),
                       decode2<DT, false>(r.c[e * 2 + 1], scale), decode2<DT, true>(r.c[e * 2 + 1], scale)};
      *(ZF_LDS u32x4*)((ZF_LDS char*)buf + (wq ^ (e * 16))) = x;
    }
    if constexpr (!DIRECT) {
#pragma unroll
      for (int h = 0; h < kPLoads; ++h)
        *(ZF_LDS u32x4*)((ZF_LDS char*)buf + wp + h * T::kThreads * 16) = r.g[h];
    }
  }
  // Fragment f of 8 tokens a lane.  Its pieces lie at the first one's place ^ 32
  // f: those bits of the piece's number are zero in the first (a wave's columns
  // begin at a multiple of 32, 64 or 128).
  template <int COLS>
  __device__ __forceinline__ s16x8 read(const char* __restrict buf, int first, int f) const {
    const ZF_LDS char* at = (const ZF_LDS char*)buf + (first ^ (f * 32));
    s16x4 half[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      half[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZF_LDS s16x4*)(at + e * 4 * COLS * 2));
    return __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static_assert((T::BM / 8) % (2 * T::FI) == 0 && (T::BN / 8) % (2 * T::FJ) == 0, "fragments' pieces");
};

// Loads before this stay before those after it, so that a wait that leaves the
// last N loads on their way knows which those are.
__device__ __forceinline__ void loads_in_order() { __builtin_amdgcn_sched_barrier(0x38F); }

// All but the wave's last N loads have arrived and its accesses of shared
// memory are done, for all waves.
template <int N>
__device__ __forceinline__ void arrive() {
  static_assert(N < 64, "the counter's range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Stage k = e (mod kStages), whose fragments p and q are in registers: its products, while the
// next stage's fragments are read from `next`, the codes of stage k + 2 are
// written to `fill` and the gradients of stage k + 4 are on their way to the
// buffer `left` that stage k has left (!DIRECT: gradients go as the codes do).
// Loads are on their way for two stages (to registers) or three.
template <bool INSIDE, typename T, int DT, bool DIRECT>
__device__ __forceinline__ void stage(Pipe<T, DT, DIRECT>& o, const char* __restrict next, char* __restrict fill,
                                      char* __restrict left, s16x8 (&p)[T::FI], const s16x8 (&q)[T::FJ],
                                      s16x8 (&q_next)[T::FJ], typename Pipe<T, DT, DIRECT>::Held& held,
                                      f32x4 (&acc)[T::FI][T::FJ], int e) {
  typedef Pipe<T, DT, DIRECT> P;
  // stage k + 1 is complete: its gradients were followed by the codes of the
  // same stage and by all loads of two more
  arrive<P::kInFlight>();
  if constexpr (T::BM == 256) __builtin_amdgcn_sched_barrier(0);  // products stay in their stage
  // fragments' places are computed anew in each stage: registers that hold them
  // would be spilled
  int rp = o.rp, rq = o.rq;
  asm volatile("" : "+v"(rp), "+v"(rq));
  if constexpr (DIRECT) {
    o.fetch_p(left, e);
    loads_in_order();
  }
#pragma unroll
  for (int i = 0; i < T::FI; ++i) {
#pragma unroll
    for (int j = 0; j < T::FJ; ++j) acc[i][j] = mma<DT>(q[j], p[i], acc[i][j]);
    p[i] = o.template read<T::BM>(next, rp, i);
#pragma unroll
    for (int j = i; j < T::FJ; j += T::FI) q_next[j] = o.template read<T::BN>(next, rq, j);
  }
  o.put(fill, held);
  o.template fetch<INSIDE>(held, e);
  if constexpr (DIRECT) {
    // the order: gradients' loads; a row of products and the reads that may
    // follow it, again and again; the codes' conversion with the last rows
    __builtin_amdgcn_sched_group_barrier(0x20, P::kPLoads, 0);
#pragma unroll
    for (int i = 0; i < T::FI; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, T::FJ, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
      for (int j = i; j < T::FJ; j += T::FI) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      if (i >= T::FI - 2) __builtin_amdgcn_sched_group_barrier(0x2, 6, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x200, 2, 0);
    __builtin_amdgcn_sched_group_barrier(0x20, 2, 0);
  }
}

template <typename T, int DT, bool DIRECT>
__global__ __launch_bounds__(T::kThreads, 2) void zf_weight_grad_kernel(GradArgs a) {
  typedef Pipe<T, DT, DIRECT> P;
  __shared__ __align__(16) char shared[T::kShared];
  char *s0 = shared, *s1 = s0 + P::kBuf, *s2 = s1 + P::kBuf, *s3 = s2 + P::kBuf;
  const Place at(a);
  const int i0 = at.i * T::BM, j0 = at.j * T::BN, split = at.split;
  const int64_t first = split * a.split_rows, end = min(first + a.split_rows, a.rows);
  const int stages = (int)((end - first + kDepth - 1) / kDepth);
  f32x4 acc[T::FI][T::FJ];
#pragma unroll
  for (int i = 0; i < T::FI; ++i)
#pragma unroll
    for (int j = 0; j < T::FJ; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
  P o(a, i0, j0, first, end - first);
  typename P::Held h0, h1;
  s16x8 p[T::FI], qa[T::FJ], qb[T::FJ];
  if constexpr (DIRECT) {
    o.fetch_p(s0, 0);
    o.fetch_p(s1, 1);
  }
  o.template fetch<false>(h0, 0);
  o.template fetch<false>(h1, 1);
  o.put(s0, h0);
  o.put(s1, h1);
  arrive<0>();
  if constexpr (DIRECT) o.fetch_p(s2, 2);
  loads_in_order();
  o.template fetch<false>(h0, 2);
  loads_in_order();
  if constexpr (DIRECT) o.fetch_p(s3, 3);
  loads_in_order();
  o.template fetch<false>(h1, 3);
  loads_in_order();
#pragma unroll
  for (int i = 0; i < T::FI; ++i) p[i] = o.template read<T::BM>(s0, o.rp, i);
#pragma unroll
  for (int j = 0; j < T::FJ; ++j) qa[j] = o.template read<T::BN>(s0, o.rq, j);
  int k = 0;
  auto turn = [&](auto inside) {
    constexpr bool INSIDE = decltype(inside)::value;
    o.turn();
    stage<INSIDE, T, DT>(o, s1, s2, s0, p, qa, qb, h0, acc, 0);
    stage<INSIDE, T, DT>(o, s2, s3, s1, p, qb, qa, h1, acc, 1);
    stage<INSIDE, T, DT>(o, s3, s0, s2, p, qa, qb, h0, acc, 2);
    stage<INSIDE, T, DT>(o, s0, s1, s3, p, qb, qa, h1, acc, 3);
    k += kStages;
  };
  if constexpr (!DIRECT) {
    // loads without looking at ends while the turn's further stages are the
    // split's, and their tile's columns end inside the matrices: rows at least as
    // long as the tile is wide end a row before the last, any others 128 before
    // (4096 tokens of 2049 x 2047: 84.9 us, with looking 101.3)
    const int64_t before = a.dy_ld >= T::BM && a.x.code_ld >= T::BN ? 1 : 128;
    const int64_t inside = min(end, a.rows - before) - first;
#pragma unroll 1
    while ((k + 2 * kStages) * kDepth <= inside) turn(std::true_type());
  }
  // stages past the last one are zeros
#pragma unroll 1
  while (k < stages) turn(std::false_type());
  arrive<0>();
  write_tile<T>(a, acc, shared, i0, j0, split);
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

enum Form { kBig, kMiddle, kLittle };
struct Plan {
  Form form;
  int32_t splits;
  int64_t split_rows;
  int64_t most_splits;  // of any form, for as many tokens or fewer
};

// The tokens are split where a form's tiles leave places of the GPU free, into
// parts of `least` at least.
int64_t splits_of(int64_t rows, int64_t tiles, int64_t places, int64_t least) {
  return std::max<int64_t>(1, std::min(places / tiles, rows / least));
}
// Microseconds of a form: rounds of blocks, each of `stage` for 32 tokens and
// `more` before and after them; with splits a second launch that reads the
// partial results at 5 TB/s.
double cost(int64_t rows, int64_t size, int64_t tiles, int64_t splits, int64_t places, double stage, double more) {
  const double rounds = (double)((tiles * splits + places - 1) / places);
  const double join = splits > 1 ? 4.0 + (double)(splits * size) * 4 / 5e6 : 0;
  return rounds * ((double)((rows + splits * kDepth - 1) / (splits * kDepth)) * stage + more) + join;
}

// WHOLE: operands in whole 16-byte pieces.
int plan(int64_t rows, int64_t out, int64_t in, bool whole, Plan& g) {
  int rc = shape_ok(rows, in);
  if (rc == ZF_OK) rc = shape_ok(0, out);
  if (rc != ZF_OK) return rc;
  auto tiles_of = [&](int64_t bm, int64_t bn) { return ((out + bm - 1) / bm) * ((in + bn - 1) / bn); };
  const int64_t big = tiles_of(Big::BM, Big::BN), middle = tiles_of(Middle::BM, Middle::BN);
  const int64_t little = tiles_of(Little::BM, Little::BN);
  if (middle > kMaxBlocks) return ZF_ESIZE;
  // A compute unit holds one block of 256 x 256 or two of 128 x 128; blocks of 64 x
  // 128 are best alone.  8192 tokens of 2048 x 2048: 84 us in large tiles, 89 in
  // middle ones; 16384 of 1024 x 1024: 56, 52 and 73 in little ones; 333 of 776 x
  // 1008: 9.8 in middle ones, 7.3 in little ones, and 333 of 777 x 1000 12.6 and 9.2.
  // Middle tiles have parts of 1024 tokens at least (4096 of 1024 x 1024: parts of
  // 512 30.8 us, of 1024 29.9, of 4096 50), little ones of 512 (2048 of 512 x 512:
  // 12.4, parts of 1024 15.0); without whole pieces a stage takes longer, and 256
  // are enough (1000 tokens of 128 x 40 in little tiles: 11.1 us, of 512 15.9).
  const int64_t sb = splits_of(rows, big, 256, 1024), sm = splits_of(rows, middle, 512, whole ? 1024 : 256),
                sl = splits_of(rows, little, 256, whole ? 512 : 256);
  const double cb = cost(rows, out * in, big, sb, 256, 0.92, 10),
               cm = cost(rows, out * in, middle, sm, 512, 0.57, 5),
               cl = cost(rows, out * in, little, sl, 256, 0.30, 3.5);
  g.form = cl < cm ? kLittle : kMiddle;
  if (whole && cb < std::min(cl, cm)) g.form = kBig;
  const int64_t stages = (rows + kDepth - 1) / kDepth, splits = g.form == kBig ? sb : g.form == kMiddle ? sm : sl;
  const int64_t per = std::max<int64_t>((stages + splits - 1) / splits, 1);
  g.split_rows = per * kDepth;
  g.most_splits = std::max({sm, sl, whole ? sb : 1});
  g.splits = (int32_t)std::max<int64_t>((stages + per - 1) / per, 1);
  return ZF_OK;
}
int64_t partial_bytes(const Plan& g, int64_t out, int64_t in) {
  return g.most_splits > 1 ? (g.most_splits * out * in * 4 + 15) / 16 * 16 : 0;
}

// Whole 16-byte pieces at 16-byte alignment, and a turn's rows within an offset of
// 31 bits: a turn's buffer is kStages * kDepth - 1 strides and a row long, and a row
// is no longer than its stride.
constexpr int64_t kTurnStride = ((int64_t)1 << 31) / (kStages * kDepth);  // bytes
bool whole_pieces(const GradArgs& a) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.x.codes);
  return (at & 15) == 0 && ((a.dy_ld | a.out) & 7) == 0 && ((a.x.code_ld | a.in) & 15) == 0 &&
         a.dy_ld * 2 < kTurnStride && a.x.code_ld < kTurnStride && a.x.scale_ld < kTurnStride;
}

template <typename T, bool DIRECT>
void launch(GradArgs a, int32_t dtype, hipStream_t s) {
  a.tiles_in = (a.in + T::BN - 1) / T::BN;
  a.tiles = a.tiles_in * ((a.out + T::BM - 1) / T::BM);
  const dim3 grid((uint32_t)a.tiles * (uint32_t)a.splits), block(T::kThreads);
  if (dtype == ZF_BF16) hipLaunchKernelGGL((zf_weight_grad_kernel<T, ZF_BF16, DIRECT>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((zf_weight_grad_kernel<T, ZF_F16, DIRECT>), grid, block, 0, s, a);
}

}  // namespace

extern "C" int64_t zf_weight_grad_bytes(int64_t rows, int64_t out_features, int64_t in_features) {
  int64_t most = 0;
  for (bool whole : {false, true}) {
    Plan g;
    const int rc = plan(rows, out_features, in_features, whole, g);
    if (rc != ZF_OK) return rc;
    most = std::max(most, partial_bytes(g, out_features, in_features));
  }
  return most;
}

extern "C" int zf_weight_grad(const zf_weight_grad_args* args, void* stream) {
  if (!args || args->reserved != 0 || !flag(args->accumulate)) return ZF_EINVAL;
  const zf_weight_grad_args& p = *args;
  if (!valid_dtype(p.dtype) || !row_dtype(p.grad_dtype)) return ZF_EDTYPE;
  const int64_t most = zf_weight_grad_bytes(p.rows, p.out_features, p.in_features);
  int rc = most < 0 ? (int)most : ZF_OK;
  if (rc == ZF_OK) rc = rows_ok(p.dy, p.dtype, p.rows, p.out_features, p.dy_stride);
  if (rc == ZF_OK) rc = act8_ok(p.x8, p.rows, p.in_features);
  if (rc != ZF_OK) return rc;
  GradArgs a;
  a.dy = p.dy;
  a.x = act8_of(p.x8);
  a.grad = p.grad;
  a.dy_ld = p.dy_stride;
  if (p.rows <= 1) {  // strides of a single row are not looked at
    a.dy_ld = (p.out_features + 7) / 8 * 8;
    a.x.code_ld = (p.in_features + 15) / 16 * 16;
    a.x.scale_ld = 0;
  }
  a.rows = p.rows;
  a.out = (int32_t)p.out_features;
  a.in = (int32_t)p.in_features;
  a.gdt = p.grad_dtype;
  a.accumulate = p.accumulate;
  const bool whole = whole_pieces(a);
  Plan g;
  rc = plan(p.rows, p.out_features, p.in_features, whole, g);
  if (rc != ZF_OK) return rc;
  const int64_t need = g.splits > 1 ? most : 0;  // a call without splits takes any
  if (!p.grad || (need > 0 && !p.workspace)) return ZF_EINVAL;
  if (!aligned_to(p.grad, p.grad_dtype) || !aligned16(p.workspace)) return ZF_EALIGN;
  if (p.workspace_size < need) return ZF_ESIZE;
  if (p.rows == 0 && p.accumulate) return ZF_OK;
  a.splits = g.splits;
  a.split_rows = g.split_rows;
  a.partial = g.splits > 1 ? static_cast<float*>(p.workspace) : nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (g.form == kBig) launch<Big, true>(a, p.dtype, s);
  else if (g.form == kMiddle) whole ? launch<Middle, true>(a, p.dtype, s) : launch<Middle, false>(a, p.dtype, s);
  else whole ? launch<Little, true>(a, p.dtype, s) : launch<Little, false>(a, p.dtype, s);
  if (g.splits > 1) {
    const JoinArgs j{a.partial, p.grad, p.out_features * p.in_features, g.splits, p.grad_dtype,
                     p.accumulate};
    const int64_t blocks = (j.size + kThreads * kChunk - 1) / (kThreads * kChunk);
    hipLaunchKernelGGL(zf_weight_grad_join, dim3((uint32_t)std::min<int64_t>(blocks, kMaxBlocks)),
                       dim3(kThreads), 0, s, j);
  }
  return hip_ok(hipGetLastError()) ? ZF_OK : ZF_EHIP;
}
