// zf_muon.hip -- the sharded mixed-precision step with Muon for chosen
// matrices and AdamW for everything else, and its C entry points.
//
// The step's front half (fixed-order sums, overflow, norm, finish) is
// zf_shard_step's own, with the sums kept in fp32; the matrices then go
// through the Newton-Schulz engine (zf_ortho.hip), whose first kernel does
// the momentum update and whose last product writes the decayed weights and
// the 16-bit copy, and the complement of the matrices goes through one AdamW
// kernel over ranges.  A skipped step's kernels return at once.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "zf_device.h"
#include "zf_hip_status.h"
#include "zf_internal.h"
#include "zf_ortho.h"

namespace {
constexpr uint64_t kMuonMagic = 0x7a665f6d756f6e31ull;  // "zf_muon1"

struct Range {
  int64_t lo, hi;
};
}  // namespace

struct zf_muon {
  uint64_t magic;
  zf_plan plan;
  std::vector<zf::ns::Shape> shapes;
  std::vector<int64_t> flat;   // each matrix's first element
  std::vector<Range> rest;     // the elements AdamW updates, in order
};

namespace {

using namespace zf::dev;
using zf::DevState;
using zf::hip_ok;
using zf::kThreads;

// ---------------------------------------------------------------------------
// AdamW over ranges [lo, hi) of the flat arrays, from fp32 sums: a block
// takes 256 quads from a range's first aligned quad on, a thread
// one quad; a quad that the range covers in part goes element by element.
// A stream like zf_pass2, for the few parameters Muon leaves: 168M of them
// take 892 us, 30 bytes each, 5.6 TB/s.
constexpr int kRangeMax = 64;
struct RangeArgs {
  const float* sums;
  float* master;
  float* m;
  float* v;
  void* out;
  const DevState* st;
  zf::UpdateConsts uc;
  int32_t count;
  Range r[kRangeMax];
  int64_t first_tile[kRangeMax];
};

template <int PDT>  // 0: no 16-bit copy
__global__ __launch_bounds__(kThreads) void zf_muon_rest(RangeArgs a) {
  if (a.st->skipped) return;
  const int64_t b = blockIdx.x;
  int k = 0;
  for (int j = 1; j < a.count; ++j) k += a.first_tile[j] <= b ? 1 : 0;
  const int64_t lo = a.r[k].lo, hi = a.r[k].hi;
  const int64_t q = lo / kQuad + (b - a.first_tile[k]) * kThreads + threadIdx.x;
  const int64_t e0 = q * kQuad;
  if (e0 >= hi) return;
  Coef c;
  c.gs = a.st->gs;
  c.bc1 = a.st->bc1;
  c.bc2 = a.st->bc2;
  c.dec = a.uc.dec; c.b1 = a.uc.b1; c.c1 = a.uc.c1; c.b2 = a.uc.b2; c.c2 = a.uc.c2;
  c.lrf = a.uc.lrf; c.ef = a.uc.ef;
  if (e0 >= lo && e0 + kQuad <= hi) {
    const f32x4 acc = ldq32(a.sums, q);
    f32x4 p = ldq32<true>(a.master, q), m = ldq32<true>(a.m, q), v = ldq32<true>(a.v, q);
    float pp[4] = {p.x, p.y, p.z, p.w}, mm[4] = {m.x, m.y, m.z, m.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) adamw1(c, acc[i], pp[i], mm[i], vv[i]);
    stq32_nt(a.master, q, (f32x4){pp[0], pp[1], pp[2], pp[3]});
    stq32_nt(a.m, q, (f32x4){mm[0], mm[1], mm[2], mm[3]});
    stq32_nt(a.v, q, (f32x4){vv[0], vv[1], vv[2], vv[3]});
    if constexpr (PDT != 0)
      stq16_nt(a.out, q, (u32x2){pack2<PDT>(pp[0], pp[1]), pack2<PDT>(pp[2], pp[3])});
    return;
  }
  for (int64_t e = e0 < lo ? lo : e0; e < e0 + kQuad && e < hi; ++e) {
    float pe = a.master[e], me = a.m[e], ve = a.v[e];
    adamw1(c, a.sums[e], pe, me, ve);
    a.master[e] = pe;
    a.m[e] = me;
    a.v[e] = ve;
    if constexpr (PDT != 0) static_cast<uint16_t*>(a.out)[e] = narrow1<PDT>(pe);
  }
}

int enqueue_rest(const zf_muon* mu, const zf_hparams* hp, const zf_step_args* args,
                 const float* sums, hipStream_t s) {
  for (size_t at = 0; at < mu->rest.size(); at += kRangeMax) {
    RangeArgs a;
    a.sums = sums;
    a.master = args->master;
    a.m = args->exp_avg;
    a.v = args->exp_avg_sq;
    a.out = args->params;
    a.st = static_cast<const DevState*>(args->state);
    a.uc = zf::update_consts(hp);
    a.count = (int32_t)std::min<size_t>(kRangeMax, mu->rest.size() - at);
    int64_t tiles = 0;
    for (int i = 0; i < kRangeMax; ++i) {
      a.r[i] = i < a.count ? mu->rest[at + i] : Range{0, 0};
      a.first_tile[i] = tiles;
      if (i < a.count) {
        const int64_t quads = (a.r[i].hi + kQuad - 1) / kQuad - a.r[i].lo / kQuad;
        tiles += (quads + kThreads - 1) / kThreads;
      }
    }
    // a plan's own limit (its update pass has smaller tiles) keeps this in
    // a grid's range
    const dim3 grid((uint32_t)tiles), block(kThreads);
    if (!args->params) hipLaunchKernelGGL(zf_muon_rest<0>, grid, block, 0, s, a);
    else if (args->param_dtype == ZF_BF16)
      hipLaunchKernelGGL(zf_muon_rest<ZF_BF16>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(zf_muon_rest<ZF_F16>, grid, block, 0, s, a);
    if (!hip_ok(hipGetLastError())) return ZF_EHIP;
  }
  return ZF_OK;
}

constexpr int32_t kThin = 32;  // longest short side of a thin matrix

bool valid(const zf_muon* m) { return m && m->magic == kMuonMagic; }

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

// The workspace: the plan's own, the fp32 sums where the plan keeps none,
// the engine's.
struct Places {
  int64_t sums, engine, bytes;
};

Places places(const zf_muon* m, const zf::ns::Layout& l) {
  const zf_plan_summary& sm = m->plan.summary;
  Places p;
  int64_t at = up256(sm.workspace_bytes);
  p.sums = m->plan.ws_rs_offset;
  if (p.sums < 0 && sm.policy != 2) {
    p.sums = at;
    at += up256(sm.psi_pad * 4);
  }
  p.engine = at;
  p.bytes = at + l.bytes;
  return p;
}

int muon_layout(const zf_muon* m, const zf_ns_params* params, zf::ns::Layout& l, zf_ns_params& p) {
  p = params ? *params : zf::ns::defaults();
  const int rc = zf::ns::check_params(p);
  if (rc != ZF_OK) return rc;
  const int64_t n = (int64_t)m->shapes.size();
  // A thin matrix takes three products where the caller leaves the choice:
  // one is least exact there, and a tall one's updates are large under
  // ZF_MUON_SCALE_ROWS, 1 / sqrt(m) of the rate beside the 0.2 of
  // ZF_MUON_SCALE_RMS.  (The shape decides, not the rule: the workspace is
  // asked for before the rule is known.)
  if (!zf::ns::layout(m->shapes.data(), n, p.products ? p.products : 1, p.products ? 0 : kThin, l))
    return ZF_ESIZE;
  // Beside a thin one the others of a plan that fits in a round of blocks take
  // three products too, which is quicker than launches of their own: 300 x 700
  // and 1293 x 4 take 193 us together, apart 110 with one product and 145 with
  // three.
  if (p.products == 0 && l.one_round && l.shortest <= kThin)
    if (!zf::ns::layout(m->shapes.data(), n, 3, 0, l)) return ZF_ESIZE;
  return ZF_OK;
}

}  // namespace

extern "C" int zf_muon_plan(const zf_plan* plan, const int64_t* segments, int64_t n,
                            zf_muon** out) {
  if (!out) return ZF_EINVAL;
  *out = nullptr;
  if (!valid_plan(plan) || !segments || n < 1) return ZF_EINVAL;
  if (n > (int64_t)plan->segs.size()) return ZF_EINVAL;
  zf_muon* m = nullptr;
  try {
    std::vector<bool> chosen(plan->segs.size(), false);
    for (int64_t i = 0; i < n; ++i) {
      const int64_t k = segments[i];
      if (k < 0 || k >= (int64_t)plan->segs.size() || chosen[k]) return ZF_EINVAL;
      const zf_segment& sg = plan->segs[k];
      if (sg.dim0 < 1 || sg.numel % sg.dim0 != 0) return ZF_EINVAL;
      chosen[k] = true;
    }
    m = new zf_muon();
    m->magic = kMuonMagic;
    m->plan = *plan;
    // in the flat's order, which is the segments' own
    int64_t at = 0;
    for (size_t k = 0; k < plan->segs.size(); ++k) {
      if (!chosen[k]) continue;
      const zf_segment& sg = plan->segs[k];
      const int64_t lo = plan->seg_at[k];
      m->shapes.push_back({sg.dim0, sg.numel / sg.dim0});
      m->flat.push_back(lo);
      if (lo > at) m->rest.push_back({at, lo});
      at = lo + sg.numel;
    }
    if (at < plan->summary.psi_pad) m->rest.push_back({at, plan->summary.psi_pad});
    zf::ns::Layout l;
    if (!zf::ns::layout(m->shapes.data(), (int64_t)m->shapes.size(), 3, 0, l)) {
      delete m;
      return ZF_ESIZE;
    }
  } catch (const std::bad_alloc&) {
    delete m;
    return ZF_ENOMEM;
  }
  *out = m;
  return ZF_OK;
}

extern "C" void zf_muon_free(zf_muon* muon) {
  if (!valid(muon)) return;
  muon->magic = 0;
  delete muon;
}

extern "C" int64_t zf_muon_workspace_bytes(const zf_muon* muon, const zf_ns_params* params) {
  if (!valid(muon)) return ZF_EINVAL;
  try {
    zf::ns::Layout l;
    zf_ns_params p;
    const int rc = muon_layout(muon, params, l, p);
    return rc == ZF_OK ? places(muon, l).bytes : rc;
  } catch (const std::bad_alloc&) {
    return ZF_ENOMEM;
  }
}

extern "C" int zf_muon_step(const zf_muon* muon, const zf_hparams* hp,
                            const zf_muon_hparams* mhp, const zf_step_args* args, void* stream) {
  if (!valid(muon) || !hp || !mhp || !args) return ZF_EINVAL;
  if (!(mhp->momentum >= 0.0 && mhp->momentum < 1.0)) return ZF_EINVAL;
  if (mhp->nesterov != 0 && mhp->nesterov != 1) return ZF_EINVAL;
  if (mhp->scale_rule != ZF_MUON_SCALE_ROWS && mhp->scale_rule != ZF_MUON_SCALE_RMS)
    return ZF_EINVAL;
  if (!valid_dtype(args->param_dtype)) return ZF_EDTYPE;
  void* const bufs[] = {args->state, args->master, args->exp_avg, args->exp_avg_sq};
  for (void* b : bufs) {
    if (!b) return ZF_EINVAL;
    if (!aligned16(b)) return ZF_EALIGN;
  }
  const zf_plan_summary& sm = muon->plan.summary;
  if (!args->grad_shards && (sm.policy == 2 || args->grads_reduced)) return ZF_EINVAL;
  try {
    zf::ns::Layout l;
    zf_ns_params p;
    int rc = muon_layout(muon, &mhp->ns, l, p);
    if (rc != ZF_OK) return rc;
    const Places at = places(muon, l);
    if (!args->workspace) return ZF_EINVAL;
    if (!aligned16(args->workspace)) return ZF_EALIGN;
    if (args->workspace_size < at.bytes) return ZF_ESIZE;
    char* ws = static_cast<char*>(args->workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);

    // sums, overflow, norm and finish; checks the rest of the arguments
    // before it enqueues anything
    zf_step_args front = *args;
    if (!front.grad_shards) front.grad_shards = reinterpret_cast<float*>(ws + at.sums);
    rc = zf::step_enqueue(&muon->plan, hp, &front, stream, false, false);
    if (rc != ZF_OK) return rc;

    for (zf::ns::Mat& m : l.mats) {
      const zf::ns::Shape& sh = muon->shapes[m.slot];
      const double scale = mhp->scale_rule == ZF_MUON_SCALE_RMS
                               ? 0.2 * std::sqrt((double)std::max(sh.rows, sh.cols))
                               : std::sqrt(std::max(1.0, (double)sh.rows / (double)sh.cols));
      m.flat = muon->flat[m.slot];
      m.rate = (float)(mhp->lr * scale);
    }
    zf::ns::MuonIo io;
    io.sums = front.grad_shards;
    io.master = args->master;
    io.momentum = args->exp_avg;
    io.params = args->params;
    io.st = static_cast<const DevState*>(args->state);
    io.mu = (float)mhp->momentum;
    io.dec = (float)(1.0 - mhp->lr * mhp->weight_decay);
    io.nesterov = mhp->nesterov;
    io.param_dtype = args->param_dtype;
    // matrices held in shared memory take three products unless the caller
    // chose: 98 us for a small MLP instead of 58, and its weights are as exact
    // as in 32-bit arithmetic
    rc = zf::ns::enqueue(l, p, p.products ? p.products : 3, ZF_F32, args->param_dtype, &io,
                         ws + at.engine, s);
    if (rc != ZF_OK) return rc;
    rc = enqueue_rest(muon, hp, args, front.grad_shards, s);
    if (rc != ZF_OK) return rc;
    if (args->phase_events && args->phase_events[3] &&
        !hip_ok(hipEventRecord(static_cast<hipEvent_t>(args->phase_events[3]), s)))
      return ZF_EHIP;
    return ZF_OK;
  } catch (const std::bad_alloc&) {
    return ZF_ENOMEM;
  }
}
