// zf_embedding.hip -- the embedding lookup with scaling and its gradient.
//
// The gradient of row v is scale times the sum of dout[t] over the tokens t
// with ids[t] = v.  Tokens are sorted by id (stable, so a row's tokens stay in
// order), the sorted positions are cut into spans of equal length, and a group
// of lanes adds its span's rows of dout in registers, writing a row of the
// gradient where its run of equal ids ends.  A run that a span cuts leaves
// partial sums, which a last launch adds in order.  So no float is added
// atomically, and a token that fills a tenth of the batch takes as many groups
// as it needs.
//
// Bound by HBM: dout is read once, each touched row written (or read and
// written) once.  The sort moves 16 bytes a token and pass.  Where the
// gradient is stored, the rows without tokens are cleared by blocks of the
// first launch, beside the sort's first pass.
//
// 32768 tokens by word frequency, 2048 columns of bf16 added to an fp32 table of
// 40960 rows (296 MB at least): 97 us, of which the runs' sums take 69, the sort
// 22 in four launches (its passes wait for memory, with 32 blocks) and the join of
// cut runs 10.  1000 tokens of 1024: 16.7 us, three launches of 4-6 each.  The
// lookup of 32768 rows of 2048 from fp32: 46 us, 4.7 TB/s of what it cannot do
// without; rows that come again are read again, from the caches.
// Stored instead of added: 65536 tokens of 2048 into a bf16 table of 32000 rows 119 to
// 139 us by the kind of ids (62 at the rate of a copy), 131072 of 64 into 50000 rows of
// fp32 112 to 136 (5): the first count takes 36 and 52 of them instead of 5, since
// every clearing block reads all ids.
// The lookup stores non-temporally: 32768 rows of 2048 bf16 with ids that are even
// over 40960 rows 39.9 us, plainly 46.3; of 2049 49.6 and 63.8.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "zf_hip_status.h"
#include "zf_rows.h"

namespace {

using namespace zf::dev;
using zf::hip_ok;
using zf::kThreads;

// ids as keys: one outside the vocabulary becomes vocab, the last one.
__device__ __forceinline__ uint32_t key_of(const void* ids, bool wide, int64_t t, uint32_t vocab) {
  const uint64_t v = wide ? static_cast<const uint64_t*>(ids)[t]
                          : (uint64_t) static_cast<const uint32_t*>(ids)[t];
  return v < vocab ? (uint32_t)v : vocab;
}

// ---------------------------------------------------------------------------
// Lookup.

struct LookupArgs {
  const void* ids;
  const void* table;
  void* out;
  int64_t out_ld, tokens, cols;
  float scale;
  uint32_t vocab;
  int32_t wide, log_lanes;
};

// A group of lanes takes kTogether tokens at a time, their rows on their way
// together.  32768 tokens of 2048 bf16 columns: one at a time 31.4 us, two 31.5,
// four 32.6; 8192 of 4096 fp32 columns, all different: 52.8, 50.7 and 49.2.
constexpr int kTogether = 2;
template <int TDT, int DT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void zf_embedding_kernel(LookupArgs a) {
  const int lanes = 1 << a.log_lanes, per = kThreads >> a.log_lanes;
  const int64_t j = ((int64_t)blockIdx.y * lanes + (threadIdx.x & (lanes - 1))) * kChunk;
  const int n = (int)min((int64_t)kChunk, a.cols - j);
  if (n <= 0) return;
  const int64_t step = (int64_t)gridDim.x * per;
  int64_t t = (int64_t)blockIdx.x * per + (threadIdx.x >> a.log_lanes);
  for (; t < a.tokens; t += step * kTogether) {
    Raw<TDT> r[kTogether];
    uint32_t v[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
      v[u] = t + u * step < a.tokens ? key_of(a.ids, a.wide, t + u * step, a.vocab) : a.vocab;
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
      r[u] = load_raw<TDT, false, WHOLE>(a.table, (int64_t)v[u] * a.cols + j, v[u] < a.vocab ? n : 0);
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      if (t + u * step >= a.tokens) break;
      float x[kChunk];
      widen8<TDT>(r[u], x);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) x[k] = v[u] < a.vocab ? x[k] * a.scale : 0.0f;
      store8<DT, true, WHOLE>(a.out, (t + u * step) * a.out_ld + j, n, x);
    }
  }
}

// ---------------------------------------------------------------------------
// Sort of the tokens by id: by 9 bits or fewer a pass, from the lowest.  Up to
// 4096 tokens are sorted by one block in shared memory, all passes in one launch.
// For more, a block takes 1024 consecutive tokens (more where that would be
// over kSortBlocks blocks), a wave consecutive parts of them; a pass needs how many of
// each digit every block holds, which a launch of its own counts (counted while
// the pass before writes, by atomics: 6 us more for 32768 tokens, since many
// tokens are the same, and 3 less for the launch).

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortBlocks = 1024;
constexpr int kBins = 512;
constexpr int kSmall = 4096;

struct SortArgs {
  const void* ids;
  uint32_t* keys[2];
  uint32_t* places[2];
  uint32_t* counts;  // [blocks][bins]
  uint32_t* cut;     // cleared for the runs: how many of them spans cut
  void* grad;        // to clear, or NULL
  int64_t tokens, cols;
  int64_t clear_rows;  // rows of the table that a clearing block looks after
  uint32_t vocab;
  int32_t wide, blocks, items, bits, passes, gdt;
};

__device__ __forceinline__ uint32_t digit(uint32_t key, int pass, int bits) {
  return key >> (pass * bits) & ((1u << bits) - 1);
}

// Rows of the gradient that no token of the batch has become zero.
__device__ __forceinline__ void clear_rows(const SortArgs& a, int block) {
  extern __shared__ uint32_t seen[];
  const int64_t r0 = block * a.clear_rows;
  const int64_t rows = min(a.clear_rows, (int64_t)a.vocab - r0);
  if (rows <= 0) return;
  const int words = (int)((rows + 31) / 32);
  for (int k = threadIdx.x; k < words; k += kSortThreads) seen[k] = 0;
  __syncthreads();
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < a.tokens; t += kSortThreads) {
    const int64_t r = (int64_t)key_of(a.ids, a.wide, t, a.vocab) - r0;
    if (r >= 0 && r < rows) atomicOr(&seen[r >> 5], 1u << (r & 31));
  }
  __syncthreads();
  const int eb = a.gdt == ZF_F32 ? 4 : 2;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t r = wave; r < rows; r += kSortWaves) {
    if (seen[r >> 5] >> (r & 31) & 1) continue;
    char* p = static_cast<char*>(a.grad) + (r0 + r) * a.cols * eb;
    const int64_t bytes = a.cols * eb;
    for (int64_t k = lane * 16; k < bytes; k += 64 * 16) {
      if (k + 16 <= bytes) {
        store_any<true, u32x4_any>(p + k, (u32x4){0, 0, 0, 0});
      } else {
        for (int64_t e = k; e < bytes; e += 2) *reinterpret_cast<uint16_t*>(p + e) = 0;
      }
    }
  }
}

// One pass over this block's n tokens: place(i, to) is called for token i of
// the block with its place `to` among all tokens, in order for equal digits.
// Thread d < bins brings the tokens of smaller blocks and of all blocks with
// digit d; all_blocks false: they are this block's own.
struct SortShared {
  uint32_t at[kSortWaves][kBins];
  uint32_t waves[kBins / 64];
};
template <typename D, typename P>
__device__ __forceinline__ void sort_pass(SortShared& s, int bits, int n, int per_wave, bool all_blocks,
                                          uint32_t total, uint32_t before, D digit_of, P place) {
  const int bins = 1 << bits, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int i0 = wave * per_wave, i1 = min(i0 + per_wave, n);
  for (int k = lane; k < bins; k += 64) s.at[wave][k] = 0;
  __syncthreads();
  for (int i = i0 + lane; i < i1; i += 64) atomicAdd(&s.at[wave][digit_of(i)], 1u);
  __syncthreads();
  if (!all_blocks && tid < bins) {
    for (int w = 0; w < kSortWaves; ++w) total += s.at[w][tid];
  }
  // a digit's first place: all smaller digits, then this one in the blocks
  // before, then in the waves before
  uint32_t upto = total;
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t x = __shfl_up(upto, off, 64);
    if (lane >= off) upto += x;
  }
  if (tid < kBins && lane == 63) s.waves[wave] = upto;
  __syncthreads();
  if (tid < bins) {
    uint32_t first = upto - total + before;
    for (int w = 0; w < wave; ++w) first += s.waves[w];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t x = s.at[w][tid];
      s.at[w][tid] = first;
      first += x;
    }
  }
  __syncthreads();
  volatile uint32_t* mine = s.at[wave];
  for (int r = i0; r < i1; r += 64) {  // the wave's lanes together
    const int i = r + lane;
    const bool in = i < i1;
    const uint32_t d = in ? digit_of(i) : 0;
    uint64_t same = __ballot(in);
    for (int b = 0; b < bits; ++b) {
      const uint64_t one = __ballot(d >> b & 1);
      same &= (d >> b & 1) ? one : ~one;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    const uint32_t to = in ? mine[d] + rank : 0;
    __builtin_amdgcn_wave_barrier();
    if (in && rank == 0) mine[d] = to + (uint32_t)__popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (in) place(i, to);
  }
}

// Up to kSmall tokens: block 0 sorts them, the others clear.
__global__ __launch_bounds__(kSortThreads) void zf_sort_small(SortArgs a) {
  if (blockIdx.x > 0) return clear_rows(a, blockIdx.x - 1);
  __shared__ SortShared s;
  __shared__ uint32_t keys[2][kSmall], places[2][kSmall];
  const int n = (int)a.tokens, per_wave = (n + kSortThreads - 1) / kSortThreads * 64;
  if (n == 0) return;  // nothing to sort, and no workspace
  if (threadIdx.x == 0) *a.cut = 0;
  for (int t = threadIdx.x; t < n; t += kSortThreads) {
    keys[0][t] = key_of(a.ids, a.wide, t, a.vocab);
    places[0][t] = t;
  }
  __syncthreads();
  for (int p = 0; p < a.passes; ++p) {
    const int from = p & 1;
    sort_pass(s, a.bits, n, per_wave, false, 0, 0, [&](int i) { return digit(keys[from][i], p, a.bits); },
              [&](int i, uint32_t to) {
                keys[from ^ 1][to] = keys[from][i];
                places[from ^ 1][to] = places[from][i];
              });
    __syncthreads();
  }
  for (int t = threadIdx.x; t < n; t += kSortThreads) {
    a.keys[(a.passes - 1) & 1][t] = keys[a.passes & 1][t];
    a.places[(a.passes - 1) & 1][t] = places[a.passes & 1][t];
  }
}

// Pass `pass` reads the ids or what the pass before it wrote.
__device__ __forceinline__ uint32_t key_in(const SortArgs& a, int pass, int64_t t) {
  return pass == 0 ? key_of(a.ids, a.wide, t, a.vocab) : a.keys[(pass + 1) & 1][t];
}

__global__ __launch_bounds__(kSortThreads) void zf_sort_count(SortArgs a, int pass) {
  if ((int)blockIdx.x >= a.blocks) return clear_rows(a, blockIdx.x - a.blocks);
  __shared__ uint32_t count[kBins];
  const int bins = 1 << a.bits;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.cut = 0;
  for (int k = threadIdx.x; k < bins; k += kSortThreads) count[k] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * a.items, t1 = min(t0 + a.items, a.tokens);
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kSortThreads)
    atomicAdd(&count[digit(key_in(a, pass, t), pass, a.bits)], 1u);
  __syncthreads();
  for (int k = threadIdx.x; k < bins; k += kSortThreads)
    a.counts[(int64_t)blockIdx.x * bins + k] = count[k];
}

__global__ __launch_bounds__(kSortThreads) void zf_sort_pass(SortArgs a, int pass) {
  __shared__ SortShared s;
  const int bins = 1 << a.bits;
  const uint32_t* places = a.places[(pass + 1) & 1];
  const int64_t t0 = (int64_t)blockIdx.x * a.items;
  const int n = (int)min((int64_t)a.items, a.tokens - t0);
  uint32_t total = 0, before = 0;
  if ((int)threadIdx.x < bins) {
#pragma unroll 8
    for (int b = 0; b < a.blocks; ++b) {
      const uint32_t x = a.counts[(int64_t)b * bins + threadIdx.x];
      total += x;
      before += b < (int)blockIdx.x ? x : 0;
    }
  }
  sort_pass(s, a.bits, n, a.items / kSortWaves, true, total, before,
            [&](int i) { return digit(key_in(a, pass, t0 + i), pass, a.bits); },
            [&](int i, uint32_t to) {
              a.keys[pass & 1][to] = key_in(a, pass, t0 + i);
              a.places[pass & 1][to] = pass == 0 ? (uint32_t)(t0 + i) : places[t0 + i];
            });
}

// ---------------------------------------------------------------------------
// Sums of the runs.

struct RunArgs {
  const uint32_t* keys;
  const uint32_t* places;
  const void* dout;
  void* grad;
  float* partial;   // [spans][2][cols]: of a run that began before its span, and of one that goes on after it
  uint32_t* cut;    // [1 + spans]: how many runs begin in a span and go on after it, and in which
  int64_t dout_ld, tokens, cols, spans;
  float scale;
  uint32_t vocab;
  int32_t log_lanes, length, gdt, accumulate;
};

// The sum's row of the gradient; `old` is what it held.
template <int GDT, bool WHOLE = false>
__device__ __forceinline__ void write_row(const RunArgs& a, uint32_t v, int64_t j, int n, const Raw<GDT>& old,
                                          const float (&sum)[kChunk]) {
  float x[kChunk], o[kChunk];
#pragma unroll
  for (int k = 0; k < kChunk; ++k) x[k] = sum[k] * a.scale;
  if (a.accumulate) {
    widen8<GDT>(old, o);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) x[k] += o[k];
  }
  store8<GDT, false, WHOLE>(a.grad, (int64_t)v * a.cols + j, n, x);
}
template <int GDT, bool WHOLE = false>
__device__ __forceinline__ Raw<GDT> old_row(const RunArgs& a, uint32_t v, int64_t j, int n) {
  return load_raw<GDT, true, WHOLE>(a.grad, (int64_t)v * a.cols + j, a.accumulate ? n : 0);
}

// A group of lanes adds the rows of a span, kU of them and, where runs end,
// the rows that they are added to on their way together.
//
// WAVE: groups are whole waves, which hold keys and places a lane each and read
// them as scalars, so that a row's address and every branch are the wave's.  Such
// a group also takes the rest of a run that begins in its span and ends in the
// next one, whose group leaves it out; only runs over three spans and more are
// cut.  (32768 tokens by word frequency, 2048 columns added to fp32: spans of 32,
// cut at both ends, 75 us and 13 for the join of 700 cut runs.)
constexpr int kU = 4, kLongest = 16;
static_assert(2 * kLongest + kU < 64, "a wave holds two spans and what is read behind them");
template <int DT, int GDT, bool WHOLE, bool WAVE>
__global__ __launch_bounds__(kThreads) void zf_run_sums(RunArgs a) {
  const int lanes = 1 << a.log_lanes, per = kThreads >> a.log_lanes, lane = threadIdx.x & 63;
  const int64_t j = ((int64_t)blockIdx.y * lanes + (threadIdx.x & (lanes - 1))) * kChunk;
  const int n = (int)min((int64_t)kChunk, a.cols - j);
  if (!WAVE && n <= 0) return;
  int group = threadIdx.x >> a.log_lanes;
  if constexpr (WAVE) group = __builtin_amdgcn_readfirstlane(group);
  const uint32_t none = a.vocab + 1;  // the key of no token
  int64_t span = (int64_t)blockIdx.x * per + group;
  for (; span < a.spans; span += (int64_t)gridDim.x * per) {
    const int64_t p0 = span * a.length;
    const int count = (int)min((int64_t)a.length, a.tokens - p0);
    uint32_t held_key = none, held_place = 0;
    if constexpr (WAVE) {  // of this span and the next one, and the key behind them
      if (lane <= 2 * a.length && p0 + lane < a.tokens) {
        held_key = a.keys[p0 + lane];
        held_place = a.places[p0 + lane];
      }
    }
    auto key_at = [&](int i) -> uint32_t {
      if constexpr (WAVE) return __builtin_amdgcn_readlane(held_key, i);
      else return p0 + i < a.tokens ? a.keys[p0 + i] : none;
    };
    auto place_at = [&](int i) -> uint32_t {
      if constexpr (WAVE) return __builtin_amdgcn_readlane(held_place, i);
      else return a.places[p0 + i];
    };
    const uint32_t key0 = key_at(0);
    bool head = p0 > 0 && a.keys[p0 - 1] == key0;
    int begin = 0, stop = count;
    if constexpr (WAVE) {
      const uint32_t last = key_at(count - 1);
      if (key_at(count) == last && !(head && key0 == last) && key_at(2 * count) != last)
        stop += __builtin_ctzll(~(__ballot(held_key == last) >> count));
      if (head && key_at(count) != key0 && (p0 == a.length || a.keys[p0 - a.length - 1] != key0)) {
        begin = __builtin_ctzll(~__ballot(held_key == key0));
        head = false;
      }
    }
    float sum[kChunk];
#pragma unroll
    for (int k = 0; k < kChunk; ++k) sum[k] = 0;
    for (int i = begin; i < stop; i += kU) {
      Raw<DT> r[kU];
      Raw<GDT> old[kU];
      uint32_t key[kU + 1];
#pragma unroll
      for (int u = 0; u <= kU; ++u) key[u] = key_at(i + u);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (key[u] >= a.vocab || i + u >= stop) break;
        r[u] = load_raw<DT, true, WHOLE>(a.dout, (int64_t)place_at(i + u) * a.dout_ld + j, n);
        if (key[u] != key[u + 1]) old[u] = old_row<GDT, WHOLE>(a, key[u], j, n);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (key[u] >= a.vocab || i + u >= stop) break;
        float x[kChunk];
        widen8<DT>(r[u], x);
#pragma unroll
        for (int k = 0; k < kChunk; ++k) sum[k] += x[k];
        const bool ends = key[u] != key[u + 1], tail = !ends && i + u + 1 == stop;
        if (!ends && !tail) continue;
        if (head || tail) {
          store8<ZF_F32, false, WHOLE>(a.partial + (span * 2 + (head ? 0 : 1)) * a.cols, j, n, sum);
          if (!head && j == 0) a.cut[1 + atomicAdd(a.cut, 1u)] = (uint32_t)span;
        } else {
          write_row<GDT, WHOLE>(a, key[u], j, n, old[u], sum);
        }
        head = false;
#pragma unroll
        for (int k = 0; k < kChunk; ++k) sum[k] = 0;
      }
    }
  }
}

// Runs that spans cut (in any order: each has its row): a block adds a run's
// partial sums, every 8th to each of 8 rows of 32 lanes of 8 columns, then the 8
// in order.
template <int GDT>
__global__ __launch_bounds__(kThreads) void zf_run_join(RunArgs a) {
  constexpr int kLanes = 32, kRows = kThreads / kLanes;
  __shared__ float s[kRows][kChunk][kLanes];
  const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
  const int64_t j = ((int64_t)blockIdx.y * kLanes + lane) * kChunk;
  const int n = (int)min((int64_t)kChunk, a.cols - j);
  const uint32_t count = *a.cut;
  for (uint32_t c = blockIdx.x; c < count; c += gridDim.x) {
    const int64_t span = a.cut[1 + c], p1 = (span + 1) * a.length;
    const uint32_t key = a.keys[p1];
    const Raw<GDT> old = old_row<GDT>(a, key, j, row == 0 ? n : 0);
    float sum[kChunk];
#pragma unroll
    for (int k = 0; k < kChunk; ++k) sum[k] = 0;
    constexpr int kAhead = 4;
    for (int64_t q = span + row;; q += kAhead * kRows) {
      bool in[kAhead];
      Raw<ZF_F32> part[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {  // a span belongs to the run if it begins with its key
        const int64_t c = q + u * kRows;
        in[u] = c == span || (c < a.spans && a.keys[c * a.length] == key);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t c = q + u * kRows;
        part[u] = load_raw<ZF_F32>(a.partial, (c * 2 + (c == span ? 1 : 0)) * a.cols + j, in[u] ? n : 0);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        float x[kChunk];
        widen8<ZF_F32>(part[u], x);
#pragma unroll
        for (int k = 0; k < kChunk; ++k) sum[k] += x[k];
      }
      if (!in[kAhead - 1]) break;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kChunk; ++k) s[row][k][lane] = sum[k];
    __syncthreads();
    if (row == 0) {
#pragma unroll
      for (int r = 1; r < kRows; ++r)
#pragma unroll
        for (int k = 0; k < kChunk; ++k) sum[k] += s[r][k][lane];
      write_row<GDT>(a, key, j, n, old, sum);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.

// 2^log lanes of 8 columns, up to a block.
int log_lanes_of(int64_t cols) {
  int log = 0;
  while (log < 8 && ((int64_t)kChunk << log) < cols) ++log;
  return log;
}

struct GradPlan {
  int32_t blocks, items, bits, passes, length;
  int64_t spans, clear_blocks, clear_rows;
  int64_t keys, places, counts, cut, partial, bytes;  // offsets; enough for fewer tokens too
};

GradPlan grad_plan(int64_t tokens, int64_t vocab, int64_t cols) {
  GradPlan g;
  int width = 1;
  while (vocab >> width) ++width;
  g.passes = (width + 8) / 9;
  g.bits = (width + g.passes - 1) / g.passes;
  const int64_t all = (int64_t)kSortBlocks * kSortThreads;
  g.items = (int32_t)(std::max<int64_t>(1, (tokens + all - 1) / all) * kSortThreads);
  g.blocks = (int32_t)((tokens + g.items - 1) / g.items);
  // Spans of 16 tokens, of 8 where those would be under 2048 waves (16384 tokens of
  // 1024 columns: 46.5 us, in spans of 8 48.7).  Spans of 24: 98 us become 92 for
  // 32768 tokens of 2048 columns with ids even over their logarithm, but 129 become
  // 133 for even ids, and 97 become 104 for shuffled ids by word frequency.
  const int log = log_lanes_of(cols);
  const int64_t waves = std::max<int64_t>(1, ((int64_t)1 << log) / 64);
  const int64_t short_spans = (2048 + waves - 1) / waves * (kLongest / 8);  // the most of 8 tokens
  g.length = kLongest;
  if (tokens / g.length * waves < 2048) g.length = 8;
  g.spans = (tokens + g.length - 1) / g.length;
  const int64_t most_spans = g.length == 8 ? g.spans : std::max(g.spans, short_spans);
  // up to 512 clearing blocks, of 16384 elements and more, with a bit of shared
  // memory a row (32 KiB at most)
  g.clear_blocks = std::max<int64_t>(1, std::min<int64_t>(512, vocab * cols >> 14));
  g.clear_blocks = std::max<int64_t>(g.clear_blocks, (vocab + (1 << 18) - 1) >> 18);
  g.clear_rows = (vocab + g.clear_blocks - 1) / g.clear_blocks;
  auto place = [&](int64_t n) {
    const int64_t at = g.bytes;
    g.bytes += (n + 255) / 256 * 256;
    return at;
  };
  g.bytes = 0;
  g.keys = place(tokens * 8);
  g.places = place(tokens * 8);
  const int64_t most_blocks = std::min<int64_t>((tokens + kSortThreads - 1) / kSortThreads, kSortBlocks);
  g.counts = place(tokens > kSmall ? most_blocks * 4 << g.bits : 0);
  g.cut = place(tokens > 0 ? (1 + most_spans) * 4 : 0);
  g.partial = place(most_spans > 1 ? most_spans * 2 * cols * 4 : 0);
  return g;
}

int sizes_ok(int64_t tokens, int64_t vocab, int64_t cols) {
  const int rc = shape_ok(tokens, cols);
  if (rc != ZF_OK) return rc;
  if (vocab < 1) return ZF_EINVAL;
  return vocab > ZF_MAX_ROWS ? ZF_ESIZE : ZF_OK;
}

int ids_ok(const void* ids, int32_t id_bytes, int64_t tokens) {
  if (id_bytes != 4 && id_bytes != 8) return ZF_EINVAL;
  if (tokens > 0 && !ids) return ZF_EINVAL;
  return (reinterpret_cast<uintptr_t>(ids) & (uintptr_t)(id_bytes - 1)) == 0 ? ZF_OK : ZF_EALIGN;
}

}  // namespace

extern "C" int zf_embedding(const zf_embedding_args* args, void* stream) {
  if (!args) return ZF_EINVAL;
  const zf_embedding_args& p = *args;
  if (!row_dtype(p.table_dtype) || !row_dtype(p.dtype)) return ZF_EDTYPE;
  int rc = sizes_ok(p.tokens, p.vocab, p.cols);
  if (rc == ZF_OK) rc = ids_ok(p.ids, p.id_bytes, p.tokens);
  if (rc == ZF_OK) rc = rows_ok(p.out, p.dtype, p.tokens, p.cols, p.out_stride);
  if (rc != ZF_OK) return rc;
  if (p.tokens > 0 && !p.table) return ZF_EINVAL;
  if (!aligned_to(p.table, p.table_dtype)) return ZF_EALIGN;
  if (p.tokens == 0) return ZF_OK;
  const LookupArgs a{p.ids, p.table, p.out, p.out_stride, p.tokens, p.cols, p.scale,
                     (uint32_t)p.vocab, p.id_bytes == 8, log_lanes_of(p.cols)};
  const int64_t per = kThreads >> a.log_lanes, span = (int64_t)kChunk << a.log_lanes;
  const bool whole = p.cols % kChunk == 0;
  // a block for each set of rows up to 2048 blocks, then several sets a block
  int64_t blocks = (p.tokens + per - 1) / per;
  if (blocks > 2048) blocks = std::max<int64_t>(2048, (blocks + kTogether - 1) / kTogether);
  const dim3 grid((uint32_t)std::min<int64_t>(blocks, kMaxBlocks), (uint32_t)((p.cols + span - 1) / span));
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
#define ZF_LOOKUP(T, D) \
  do { \
    if (whole) hipLaunchKernelGGL((zf_embedding_kernel<T, D, true>), grid, dim3(kThreads), 0, s, a); \
    else hipLaunchKernelGGL((zf_embedding_kernel<T, D, false>), grid, dim3(kThreads), 0, s, a); \
  } while (0)
#define ZF_LOOKUP_TO(T) \
  do { \
    if (p.dtype == ZF_F32) ZF_LOOKUP(T, ZF_F32); \
    else if (p.dtype == ZF_BF16) ZF_LOOKUP(T, ZF_BF16); \
    else ZF_LOOKUP(T, ZF_F16); \
  } while (0)
  if (p.table_dtype == ZF_F32) ZF_LOOKUP_TO(ZF_F32);
  else if (p.table_dtype == ZF_BF16) ZF_LOOKUP_TO(ZF_BF16);
  else ZF_LOOKUP_TO(ZF_F16);
#undef ZF_LOOKUP_TO
#undef ZF_LOOKUP
  return hip_ok(hipGetLastError()) ? ZF_OK : ZF_EHIP;
}

extern "C" int64_t zf_embedding_grad_bytes(int64_t tokens, int64_t vocab, int64_t cols) {
  const int rc = sizes_ok(tokens, vocab, cols);
  return rc != ZF_OK ? rc : grad_plan(tokens, vocab, cols).bytes;
}

extern "C" int zf_embedding_grad(const zf_embedding_grad_args* args, void* stream) {
  if (!args || args->reserved != 0 || !flag(args->accumulate)) return ZF_EINVAL;
  const zf_embedding_grad_args& p = *args;
  if (!row_dtype(p.dtype) || !row_dtype(p.grad_dtype)) return ZF_EDTYPE;
  int rc = sizes_ok(p.tokens, p.vocab, p.cols);
  if (rc == ZF_OK) rc = ids_ok(p.ids, p.id_bytes, p.tokens);
  if (rc == ZF_OK) rc = rows_ok(p.dout, p.dtype, p.tokens, p.cols, p.dout_stride);
  if (rc != ZF_OK) return rc;
  if (!p.grad) return ZF_EINVAL;
  if (!aligned_to(p.grad, p.grad_dtype) || !aligned16(p.workspace)) return ZF_EALIGN;
  const GradPlan g = grad_plan(p.tokens, p.vocab, p.cols);
  if (p.tokens > 0 && !p.workspace) return ZF_EINVAL;
  if (p.workspace_size < g.bytes) return ZF_ESIZE;
  if (p.tokens == 0 && p.accumulate) return ZF_OK;
  char* ws = static_cast<char*>(p.workspace);
  SortArgs so;
  so.ids = p.ids;
  for (int k = 0; k < 2; ++k) {
    so.keys[k] = reinterpret_cast<uint32_t*>(ws + g.keys) + k * p.tokens;
    so.places[k] = reinterpret_cast<uint32_t*>(ws + g.places) + k * p.tokens;
  }
  so.counts = reinterpret_cast<uint32_t*>(ws + g.counts);
  so.cut = reinterpret_cast<uint32_t*>(ws + g.cut);
  so.grad = p.grad;
  so.tokens = p.tokens;
  so.cols = p.cols;
  so.clear_rows = g.clear_rows;
  so.vocab = (uint32_t)p.vocab;
  so.wide = p.id_bytes == 8;
  so.blocks = g.blocks;
  so.items = g.items;
  so.bits = g.bits;
  so.passes = g.passes;
  so.gdt = p.grad_dtype;
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const int64_t clear = p.accumulate ? 0 : g.clear_blocks;
  const uint32_t bits = clear ? (uint32_t)((g.clear_rows + 31) / 32 * 4) : 0;
  if (p.tokens <= kSmall) {
    hipLaunchKernelGGL(zf_sort_small, dim3((uint32_t)(1 + clear)), dim3(kSortThreads), bits, s, so);
  } else {
    for (int pass = 0; pass < g.passes; ++pass) {
      const int64_t more = pass == 0 ? clear : 0;
      hipLaunchKernelGGL(zf_sort_count, dim3((uint32_t)(g.blocks + more)), dim3(kSortThreads), more ? bits : 0,
                         s, so, pass);
      hipLaunchKernelGGL(zf_sort_pass, dim3(g.blocks), dim3(kSortThreads), 0, s, so, pass);
    }
  }
  if (p.tokens > 0) {
    RunArgs r;
    r.keys = so.keys[(g.passes - 1) & 1];
    r.places = so.places[(g.passes - 1) & 1];
    r.dout = p.dout;
    r.grad = p.grad;
    r.partial = reinterpret_cast<float*>(ws + g.partial);
    r.cut = so.cut;
    r.dout_ld = p.dout_stride;
    r.tokens = p.tokens;
    r.cols = p.cols;
    r.spans = g.spans;
    r.scale = p.scale;
    r.vocab = (uint32_t)p.vocab;
    r.log_lanes = log_lanes_of(p.cols);
    r.length = g.length;
    r.gdt = p.grad_dtype;
    r.accumulate = p.accumulate;
    const int64_t per = kThreads >> r.log_lanes, span = (int64_t)kChunk << r.log_lanes;
    const dim3 grid((uint32_t)std::min<int64_t>((g.spans + per - 1) / per, kMaxBlocks),
                    (uint32_t)((p.cols + span - 1) / span));
    const bool whole = p.cols % kChunk == 0;
    const dim3 join((uint32_t)std::min<int64_t>(g.spans - 1, 1024), (uint32_t)((p.cols + 255) / 256));
#define ZF_RUNS(D, G) \
  do { \
    if (!whole) hipLaunchKernelGGL((zf_run_sums<D, G, false, false>), grid, dim3(kThreads), 0, s, r); \
    else if (r.log_lanes < 6) hipLaunchKernelGGL((zf_run_sums<D, G, true, false>), grid, dim3(kThreads), 0, s, r); \
    else hipLaunchKernelGGL((zf_run_sums<D, G, true, true>), grid, dim3(kThreads), 0, s, r); \
    if (g.spans > 1) hipLaunchKernelGGL(zf_run_join<G>, join, dim3(kThreads), 0, s, r); \
  } while (0)
#define ZF_RUNS_TO(D) \
  do { \
    if (p.grad_dtype == ZF_F32) ZF_RUNS(D, ZF_F32); \
    else if (p.grad_dtype == ZF_BF16) ZF_RUNS(D, ZF_BF16); \
    else ZF_RUNS(D, ZF_F16); \
  } while (0)
    if (p.dtype == ZF_F32) ZF_RUNS_TO(ZF_F32);
    else if (p.dtype == ZF_BF16) ZF_RUNS_TO(ZF_BF16);
    else ZF_RUNS_TO(ZF_F16);
#undef ZF_RUNS_TO
#undef ZF_RUNS
  }
  return hip_ok(hipGetLastError()) ? ZF_OK : ZF_EHIP;
}
