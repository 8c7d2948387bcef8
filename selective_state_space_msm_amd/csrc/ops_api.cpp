// C ABI of the block operators: argument checks, workspace layout, launches.  Every check
// happens before anything is enqueued; nothing here allocates device memory.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>

#include <hip/hip_runtime_api.h>

#include "../../include/msm.h"
#include "ops_internal.h"

namespace {

using msm::DeltaArgs;

constexpr int64_t kLim = (int64_t)1 << 40;
constexpr int64_t kGridX = ((int64_t)1 << 31) - 1;
constexpr int64_t kGridY = 65535;
constexpr int64_t kSegmentLeast = 8;   // chunks of a segment at least

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }
size_t elem_bytes(msm_dtype io) { return io == MSM_BF16 ? 2 : 4; }
msm_status status_of(hipError_t e) { return e == hipSuccess ? MSM_OK : MSM_ERR_LAUNCH; }

struct Range {
  uintptr_t lo, hi;
};
Range rng(const void* p, size_t bytes) {
  return p ? Range{(uintptr_t)p, (uintptr_t)p + bytes} : Range{0, 0};
}
bool overlaps(Range a, Range b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}
bool any_overlap(const Range* outs, int nout, const Range* ins, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlaps(outs[i], ins[j])) return true;
    for (int j = i + 1; j < nout; ++j)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// ---- gated delta rule ----

struct DeltaShape {
  int64_t tokens, nseq, L, NT, nslots, nsegs, Hk, H, K, V, VP;
  int KP, C, seg_len;
};

// Chunks of a segment, 0 for none.  Segments cost 2.2 to 2.5 times a walk's work, so they pay where whole
// sequences would leave two thirds of the 256 CUs without a workgroup (Bt = 1, L = 65536, H = 16,
// V = 128: 32 workgroups, 3.8 ms whole and 1.03 ms in segments); there are enough then for one a CU.
// Packed sequences are seldom alike and the longest decides, so there half of the CUs is the bound
// (8191 fp32 tokens in 9 sequences, H = 6, V = 80: segments of 8 chunks 70 + 77 us, of 11, which leave
// no second round of workgroups, 88 + 86 us).
int delta_segment(const DeltaShape& s, bool packed) {
  const int64_t blocks = s.H * ceil_div(s.VP, 64);  // workgroups of a sequence
  if (s.nseq * blocks > (packed ? 128 : 80)) return 0;
  int64_t len = ceil_div(s.nslots * blocks, 256);
  if (len < kSegmentLeast) len = kSegmentLeast;
  return s.nslots >= 3 * len * (packed ? 1 : s.nseq) ? (int)len : 0;
}

// Sizes of a call; packed: Bt sequences in L rows together.
msm_status delta_shape(int64_t Bt, int64_t L, int64_t Hk, int64_t H, int64_t K, int64_t V,
                       msm_dtype io, bool packed, DeltaShape* s) {
  if (io != MSM_F32 && io != MSM_BF16) return MSM_ERR_UNSUPPORTED;
  if (Bt < 1 || L < 1 || Hk < 1 || H < 1 || K < 1 || V < 1 || H % Hk != 0) return MSM_ERR_INVALID_ARG;
  if (K > msm::kDeltaMaxK) return MSM_ERR_UNSUPPORTED;
  if (Bt > kGridX || L > kGridX || H > kGridY || V > ((int64_t)1 << 20)) return MSM_ERR_INVALID_ARG;
  s->tokens = packed ? L : Bt * L;
  if (s->tokens > kGridX || s->tokens * H > kLim || Bt * H > kGridX) return MSM_ERR_INVALID_ARG;
  s->nseq = Bt;
  s->L = packed ? 0 : L;
  s->Hk = Hk;
  s->H = H;
  s->K = K;
  s->V = V;
  s->VP = ceil_div(V, 32) * 32;
  s->KP = msm::delta_padded_k(K);
  s->C = msm::delta_chunk(io == MSM_BF16, s->KP);
  s->NT = packed ? 1 : ceil_div(L, s->C);
  s->nslots = packed ? L / s->C + Bt : Bt * s->NT;
  if (s->nslots > kGridX) return MSM_ERR_INVALID_ARG;
  s->seg_len = delta_segment(*s, packed);
  s->nsegs = s->seg_len == 0 ? 0 : (packed ? s->nslots / s->seg_len + Bt : Bt * s->NT / s->seg_len + Bt);
  if (s->nsegs * H > kGridX) return MSM_ERR_INVALID_ARG;
  // the rows of a chunk are addressed with 32-bit byte offsets
  const int64_t es = io == MSM_BF16 ? 2 : 4, widest = Hk * K > H * V ? Hk * K : H * V;
  if (s->C * widest * es >= ((int64_t)1 << 31)) return MSM_ERR_UNSUPPORTED;
  return MSM_OK;
}

// The same for whole sequences.  Their launches have a workgroup of 256 threads for every chunk, and
// for every sequence (or segment) and head, in one dimension, which holds fewer than 2^32 threads;
// past that a launch may run short without an error.
constexpr int64_t kGroups256 = ((int64_t)1 << 24) - 1;
msm_status delta_sequences(int64_t Bt, int64_t L, int64_t Hk, int64_t H, int64_t K, int64_t V,
                           msm_dtype io, bool packed, DeltaShape* s) {
  const msm_status st = delta_shape(Bt, L, Hk, H, K, V, io, packed, s);
  if (st != MSM_OK) return st;
  const int64_t walks = s->nsegs > s->nseq ? s->nsegs : s->nseq;
  return s->nslots > kGroups256 || walks * H > kGroups256 ? MSM_ERR_UNSUPPORTED : MSM_OK;
}

struct DeltaLayout {
  size_t vec, T, P, kq, segS, segF, M, S, dS, E, dV, pred, dots, total;
};

DeltaLayout delta_layout(const DeltaShape& s, msm_dtype io, bool bwd) {
  const size_t n = (size_t)(s.nslots * s.H), C = (size_t)s.C, KP = (size_t)s.KP, VP = (size_t)s.VP;
  // blocks of 32 x 32 on and below the diagonal
  const size_t mat = n * (1024 * (C / 32) * (C / 32 + 1) / 2) * 3 * 2;
  DeltaLayout l{};
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes);
    return here;
  };
  l.vec = take(n * 5 * C * 4);
  l.T = take(mat);
  l.P = take(mat);
  l.kq = take((size_t)(s.nslots * s.Hk) * 2 * msm::delta_in_planes(io == MSM_BF16) * C * KP * 2);
  l.segS = take((size_t)(s.nsegs * s.H) * KP * VP * 4);
  l.segF = take((size_t)(s.nsegs * s.H) * KP * KP * 4);
  if (bwd) {
    l.M = take(mat);
    l.S = take(n * KP * VP * 4);
    l.dS = take(n * KP * VP * 4);
    l.E = take(n * C * VP * 4);
    l.dV = take(n * C * VP * 4);
    l.pred = take(n * C * VP * 4);
    l.dots = take(n * (VP / 16) * 4 * C * 4);
  }
  l.total = at;
  return l;
}

DeltaArgs delta_args(const DeltaShape& s, const DeltaLayout& l, msm_dtype io, const void* q,
                     const void* k, const void* v, const float* g, const float* beta,
                     const int32_t* off, const float* S0, float scale, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  DeltaArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.off = off;
  a.S0 = S0;
  a.vec = reinterpret_cast<float*>(ws + l.vec);
  a.T = ws + l.T;
  a.P = ws + l.P;
  a.kq = ws + l.kq;
  a.segS = reinterpret_cast<float*>(ws + l.segS);
  a.segF = reinterpret_cast<float*>(ws + l.segF);
  a.nsegs = s.nsegs;
  a.seg_len = s.seg_len;
  a.M = ws + l.M;
  a.S = reinterpret_cast<float*>(ws + l.S);
  a.dS = reinterpret_cast<float*>(ws + l.dS);
  a.E = reinterpret_cast<float*>(ws + l.E);
  a.dV = reinterpret_cast<float*>(ws + l.dV);
  a.pred = reinterpret_cast<float*>(ws + l.pred);
  a.dots = reinterpret_cast<float*>(ws + l.dots);
  a.tokens = s.tokens;
  a.nseq = s.nseq;
  a.L = s.L;
  a.NT = s.NT;
  a.nslots = s.nslots;
  a.Hk = s.Hk;
  a.H = s.H;
  a.K = s.K;
  a.V = s.V;
  a.VP = s.VP;
  a.scale = scale;
  a.vec_k = s.K * (int64_t)elem_bytes(io) % 16 == 0 && aligned(q, 16) && aligned(k, 16);
  a.kq_direct = a.vec_k && io == MSM_BF16;
  return a;
}

typedef hipError_t (*DeltaLaunch)(const DeltaArgs&, hipStream_t);

DeltaLaunch delta_launch(bool bwd, msm_dtype io, int KP) {
  static const DeltaLaunch table[2][2][4] = {
      {{msm::launch_delta_fwd_0_32, msm::launch_delta_fwd_0_64, msm::launch_delta_fwd_0_128,
        msm::launch_delta_fwd_0_256},
       {msm::launch_delta_fwd_1_32, msm::launch_delta_fwd_1_64, msm::launch_delta_fwd_1_128,
        msm::launch_delta_fwd_1_256}},
      {{msm::launch_delta_bwd_0_32, msm::launch_delta_bwd_0_64, msm::launch_delta_bwd_0_128,
        msm::launch_delta_bwd_0_256},
       {msm::launch_delta_bwd_1_32, msm::launch_delta_bwd_1_64, msm::launch_delta_bwd_1_128,
        msm::launch_delta_bwd_1_256}}};
  return table[bwd][io == MSM_BF16][KP == 32 ? 0 : (KP == 64 ? 1 : (KP == 128 ? 2 : 3))];
}

// ---- layer norm ----

msm_status norm_check(int64_t rows, int64_t D, msm_dtype io) {
  if (io != MSM_F32 && io != MSM_BF16) return MSM_ERR_UNSUPPORTED;
  if (rows < 1 || D < 1 || rows > kGridX || D > ((int64_t)1 << 30)) return MSM_ERR_INVALID_ARG;
  if (rows * D > ((int64_t)1 << 50)) return MSM_ERR_INVALID_ARG;
  return MSM_OK;
}

// Workgroups of the backward: each leaves 8 D bytes of column sums, so few enough that they stay
// small beside the rows, and enough to fill the GPU.
int64_t norm_groups(int64_t rows, const msm::NormShape& f) {
  if (f.NV == 0) return rows < 64 ? rows : 64;
  const int64_t threads = msm::norm_threads(f.T, f.NV), in_flight = threads / f.T;
  const int64_t g = ceil_div(rows, 2 * in_flight), most = f.T == 256 ? 256 : 512;
  return g > most ? most : g;
}

size_t norm_bwd_bytes(int64_t rows, int64_t D, msm_dtype io) {
  // for either way of reading the rows (it depends on the arrays' alignment)
  int64_t most = 1;
  const int pers[2] = {1, io == MSM_BF16 ? 8 : 4};
  for (int per : pers) {
    const int64_t g = norm_groups(rows, msm::norm_shape(D, per));
    if (g > most) most = g;
  }
  return align_up((size_t)most * 8 * (size_t)D);
}

// ---- clipping ----

struct ClipPlan {
  int64_t batches, parts;
  int groups;  // workgroups of a launch
};

ClipPlan clip_plan(int64_t count) {
  ClipPlan p;
  p.batches = ceil_div(count, msm::kClipTensors);
  if (p.batches < 1) p.batches = 1;
  int64_t g = msm::kClipPartials / p.batches;
  p.groups = (int)(g < 64 ? 64 : (g > 1024 ? 1024 : g));
  p.parts = p.batches * p.groups;
  return p;
}

msm_status clip_check(const void* const* src, const int64_t* numel, const int32_t* dtypes,
                      int64_t count) {
  if (count < 0 || count > ((int64_t)1 << 24)) return MSM_ERR_INVALID_ARG;
  if (count > 0 && (!src || !numel || !dtypes)) return MSM_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    if (dtypes[i] != MSM_F32 && dtypes[i] != MSM_BF16) return MSM_ERR_UNSUPPORTED;
    if (numel[i] < 0 || numel[i] > kLim || (numel[i] > 0 && !src[i])) return MSM_ERR_INVALID_ARG;
    if (!aligned(src[i], dtypes[i] == MSM_BF16 ? 2 : 4)) return MSM_ERR_INVALID_ARG;
  }
  return MSM_OK;
}

// Memory of a call: what it reads, or what it writes (and perhaps reads).
struct Extent {
  uintptr_t lo, hi;
  bool written;
};

// Nothing that is written may overlap anything else: the gradients (apart from one that is scaled in
// place, which is its own output), the outputs, the norm and the workspace, in the order of their
// addresses.
msm_status clip_overlaps(const void* const* src, void* const* dst, const int64_t* numel,
                         const int32_t* dtypes, int64_t count, bool in_place, const float* norm,
                         const void* workspace, size_t workspace_bytes) {
  constexpr int64_t kHere = 514;  // of an ordinary call; longer lists go to the heap
  Extent here[kHere];
  const int64_t most = (dst ? 2 : 1) * count + 2;
  std::unique_ptr<Extent[]> heap(most > kHere ? new (std::nothrow) Extent[most] : nullptr);
  if (most > kHere && !heap) return MSM_ERR_WORKSPACE;
  Extent* const e = most > kHere ? heap.get() : here;
  int64_t n = 0;
  const auto add = [&](const void* p, size_t bytes, bool written) {
    if (bytes) e[n++] = Extent{(uintptr_t)p, (uintptr_t)p + bytes, written};
  };
  for (int64_t i = 0; i < count; ++i) {
    const size_t bytes = (size_t)numel[i] * (dtypes[i] == MSM_BF16 ? 2 : 4);
    const bool own = dst ? dst[i] == src[i] : in_place;
    add(src[i], bytes, own);
    if (dst && !own) add(dst[i], bytes, true);
  }
  add(norm, sizeof(float), true);
  add(workspace, workspace_bytes, true);
  std::sort(e, e + n, [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
  uintptr_t end = 0, end_written = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (e[i].lo < (e[i].written ? end : end_written)) return MSM_ERR_INVALID_ARG;
    if (e[i].hi > end) end = e[i].hi;
    if (e[i].written && e[i].hi > end_written) end_written = e[i].hi;
  }
  return MSM_OK;
}

// Tensors [i0, i0 + count) as a launch's table; false when their chunks outnumber 2^31.
bool clip_batch(const void* const* src, void* const* dst, const int64_t* numel,
                const int32_t* dtypes, int64_t i0, int count, msm::ClipBatch* b) {
  int64_t chunks = 0;
  b->count = count;
  for (int i = 0; i < count; ++i) {
    b->src[i] = src[i0 + i];
    b->dst[i] = dst ? dst[i0 + i] : const_cast<void*>(src[i0 + i]);
    b->n[i] = numel[i0 + i];
    b->bf16[i] = dtypes[i0 + i] == MSM_BF16;
    b->first[i] = (uint32_t)chunks;
    chunks += ceil_div(numel[i0 + i], msm::kClipChunk);
    if (chunks > kGridX) return false;
  }
  b->first[count] = (uint32_t)chunks;
  return true;
}

msm_status clip_sums(const void* const* src, const int64_t* numel, const int32_t* dtypes,
                     int64_t count, const ClipPlan& plan, double* part, hipStream_t s) {
  for (int64_t k = 0; k < plan.batches; ++k) {
    const int64_t i0 = k * msm::kClipTensors, left = count - i0;
    msm::ClipBatch b;
    clip_batch(src, nullptr, numel, dtypes, i0, (int)(left < msm::kClipTensors ? left : msm::kClipTensors), &b);
    const hipError_t e = msm::launch_clip_sum(b, part + k * plan.groups, plan.groups, s);
    if (e != hipSuccess) return MSM_ERR_LAUNCH;
  }
  return MSM_OK;
}

}  // namespace

extern "C" {

size_t msm_delta_rule_fwd_workspace_bytes(int64_t Bt, int64_t L, int64_t Hk, int64_t H, int64_t K,
                                          int64_t V, int32_t packed, msm_dtype io) {
  DeltaShape s;
  if (delta_sequences(Bt, L, Hk, H, K, V, io, packed != 0, &s) != MSM_OK) return 0;
  return delta_layout(s, io, false).total;
}

size_t msm_delta_rule_bwd_workspace_bytes(int64_t Bt, int64_t L, int64_t Hk, int64_t H, int64_t K,
                                          int64_t V, int32_t packed, msm_dtype io) {
  DeltaShape s;
  if (delta_sequences(Bt, L, Hk, H, K, V, io, packed != 0, &s) != MSM_OK) return 0;
  return delta_layout(s, io, true).total;
}

msm_status msm_delta_rule_fwd(const void* q, const void* k, const void* v, const float* g,
                              const float* beta, const int32_t* seq_offsets, const float* S0,
                              void* o, float* last_S, int64_t Bt, int64_t L, int64_t Hk, int64_t H,
                              int64_t K, int64_t V, float scale, msm_dtype io, void* workspace,
                              size_t workspace_bytes, void* stream) {
  DeltaShape s;
  const msm_status st = delta_sequences(Bt, L, Hk, H, K, V, io, seq_offsets != nullptr, &s);
  if (st != MSM_OK) return st;
  if (!q || !k || !v || !g || !beta || !o || !isfinite(scale)) return MSM_ERR_INVALID_ARG;
  const DeltaLayout l = delta_layout(s, io, false);
  if (!workspace || workspace_bytes < l.total) return MSM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MSM_ERR_INVALID_ARG;
  const size_t es = elem_bytes(io), t = (size_t)s.tokens, state = (size_t)(Bt * H * K * V) * 4;
  const size_t nk = t * Hk * K * es, nv = t * H * V * es, ng = t * H * 4;
  const Range ins[] = {rng(q, nk),  rng(k, nk),  rng(v, nv), rng(g, ng), rng(beta, ng),
                       rng(S0, state), rng(seq_offsets, (size_t)(Bt + 1) * 4)};
  const Range outs[] = {rng(o, nv), rng(last_S, state), rng(workspace, l.total)};
  if (any_overlap(outs, 3, ins, 7)) return MSM_ERR_INVALID_ARG;
  DeltaArgs a = delta_args(s, l, io, q, k, v, g, beta, seq_offsets, S0, scale, workspace);
  a.o = o;
  a.last_S = last_S;
  return status_of(delta_launch(false, io, s.KP)(a, static_cast<hipStream_t>(stream)));
}

msm_status msm_delta_rule_bwd(const void* q, const void* k, const void* v, const float* g,
                              const float* beta, const int32_t* seq_offsets, const float* S0,
                              const void* do_, const float* dlast_S, void* dq, void* dk, void* dv,
                              float* dg, float* dbeta, float* dS0, int64_t Bt, int64_t L,
                              int64_t Hk, int64_t H, int64_t K, int64_t V, float scale,
                              msm_dtype io, void* workspace, size_t workspace_bytes,
                              void* stream) {
  DeltaShape s;
  const msm_status st = delta_sequences(Bt, L, Hk, H, K, V, io, seq_offsets != nullptr, &s);
  if (st != MSM_OK) return st;
  if (!q || !k || !v || !g || !beta || !do_ || !dq || !dk || !dv || !dg || !dbeta || !isfinite(scale))
    return MSM_ERR_INVALID_ARG;
  const DeltaLayout l = delta_layout(s, io, true);
  if (!workspace || workspace_bytes < l.total) return MSM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MSM_ERR_INVALID_ARG;
  const size_t es = elem_bytes(io), t = (size_t)s.tokens, state = (size_t)(Bt * H * K * V) * 4;
  const size_t nk = t * Hk * K * es, nv = t * H * V * es, ng = t * H * 4;
  const Range ins[] = {rng(q, nk),     rng(k, nk),     rng(v, nv),
                       rng(g, ng),     rng(beta, ng),  rng(S0, state),
                       rng(do_, nv),   rng(dlast_S, state),
                       rng(seq_offsets, (size_t)(Bt + 1) * 4)};
  const Range outs[] = {rng(dq, nk), rng(dk, nk),    rng(dv, nv),       rng(dg, ng),
                        rng(dbeta, ng), rng(dS0, state), rng(workspace, l.total)};
  if (any_overlap(outs, 7, ins, 9)) return MSM_ERR_INVALID_ARG;
  DeltaArgs a = delta_args(s, l, io, q, k, v, g, beta, seq_offsets, S0, scale, workspace);
  a.do_ = do_;
  a.vec_v = V * (int64_t)es % 16 == 0 && aligned(do_, 16);
  a.dlast_S = dlast_S;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dS0 = dS0;
  return status_of(delta_launch(true, io, s.KP)(a, static_cast<hipStream_t>(stream)));
}

msm_status msm_delta_rule_step(const void* q, const void* k, const void* v, const float* g,
                               const float* beta, float* S, void* o, int64_t Bt, int64_t Hk,
                               int64_t H, int64_t K, int64_t V, float scale, msm_dtype io,
                               void* stream) {
  DeltaShape s;
  const msm_status st = delta_shape(Bt, 1, Hk, H, K, V, io, false, &s);
  if (st != MSM_OK) return st;
  if (!q || !k || !v || !g || !beta || !S || !o || !isfinite(scale)) return MSM_ERR_INVALID_ARG;
  const size_t es = elem_bytes(io), t = (size_t)Bt, state = (size_t)(Bt * H * K * V) * 4;
  const size_t nk = t * Hk * K * es, nv = t * H * V * es, ng = t * H * 4;
  const Range ins[] = {rng(q, nk), rng(k, nk), rng(v, nv), rng(g, ng), rng(beta, ng)};
  const Range outs[] = {rng(o, nv), rng(S, state)};
  if (any_overlap(outs, 2, ins, 5)) return MSM_ERR_INVALID_ARG;
  msm::DeltaStepArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.S = S;
  a.o = o;
  a.Bt = Bt;
  a.Hk = Hk;
  a.H = H;
  a.K = K;
  a.V = V;
  a.scale = scale;
  return status_of(msm::launch_delta_step(a, io == MSM_BF16, static_cast<hipStream_t>(stream)));
}

msm_status msm_layer_norm_fwd(const void* x, const float* weight, const float* bias, void* y,
                              float* mean, float* rstd, int64_t rows, int64_t D, float eps,
                              msm_dtype io, void* stream) {
  const msm_status st = norm_check(rows, D, io);
  if (st != MSM_OK) return st;
  if (!x || !y || !(eps >= 0.f) || !isfinite(eps)) return MSM_ERR_INVALID_ARG;
  const size_t n = (size_t)(rows * D) * elem_bytes(io), nd = (size_t)D * 4, nr = (size_t)rows * 4;
  const Range ins[] = {rng(x, n), rng(weight, nd), rng(bias, nd)};
  const Range outs[] = {rng(y, n), rng(mean, nr), rng(rstd, nr)};
  if (any_overlap(outs, 3, ins, 3)) return MSM_ERR_INVALID_ARG;
  msm::NormArgs a{};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.D = D;
  a.eps = eps;
  a.vec = D * (int64_t)elem_bytes(io) % 16 == 0 && aligned(x, 16) && aligned(y, 16);
  return status_of(msm::launch_norm_fwd(a, io == MSM_BF16, static_cast<hipStream_t>(stream)));
}

size_t msm_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t D, msm_dtype io) {
  return norm_check(rows, D, io) == MSM_OK ? norm_bwd_bytes(rows, D, io) : 0;
}

msm_status msm_layer_norm_bwd(const void* x, const float* weight, const void* dy,
                              const float* mean, const float* rstd, void* dx, float* dweight,
                              float* dbias, int64_t rows, int64_t D, msm_dtype io,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const msm_status st = norm_check(rows, D, io);
  if (st != MSM_OK) return st;
  if (!x || !dy || !mean || !rstd || !dx) return MSM_ERR_INVALID_ARG;
  const bool cols = dweight || dbias;
  const size_t need = cols ? norm_bwd_bytes(rows, D, io) : 0;
  if (cols && (!workspace || workspace_bytes < need)) return MSM_ERR_WORKSPACE;
  if (cols && !aligned(workspace, 16)) return MSM_ERR_INVALID_ARG;
  const size_t n = (size_t)(rows * D) * elem_bytes(io), nd = (size_t)D * 4, nr = (size_t)rows * 4;
  const Range ins[] = {rng(x, n), rng(weight, nd), rng(dy, n), rng(mean, nr), rng(rstd, nr)};
  const Range outs[] = {rng(dx, n), rng(dweight, nd), rng(dbias, nd), rng(workspace, need)};
  if (any_overlap(outs, 4, ins, 5)) return MSM_ERR_INVALID_ARG;
  msm::NormArgs a{};
  a.x = x;
  a.weight = weight;
  a.dy = dy;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.part = cols ? static_cast<float*>(workspace) : nullptr;
  a.rows = rows;
  a.D = D;
  a.vec = D * (int64_t)elem_bytes(io) % 16 == 0 && aligned(x, 16) && aligned(dy, 16) && aligned(dx, 16);
  a.groups = (int32_t)norm_groups(rows, msm::norm_shape(D, a.vec ? (io == MSM_BF16 ? 8 : 4) : 1));
  return status_of(msm::launch_norm_bwd(a, io == MSM_BF16, static_cast<hipStream_t>(stream)));
}

size_t msm_grad_norm_workspace_bytes(int64_t count) {
  if (count < 0 || count > ((int64_t)1 << 24)) return 0;
  return align_up((size_t)clip_plan(count).parts * sizeof(double));
}

msm_status msm_grad_norm(const void* const* grads, const int64_t* numel, const int32_t* dtypes,
                         int64_t count, float* norm, void* workspace, size_t workspace_bytes,
                         void* stream) {
  msm_status st = clip_check(grads, numel, dtypes, count);
  if (st != MSM_OK) return st;
  if (!norm) return MSM_ERR_INVALID_ARG;
  const ClipPlan plan = clip_plan(count);
  if (!workspace || workspace_bytes < (size_t)plan.parts * sizeof(double)) return MSM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MSM_ERR_INVALID_ARG;
  st = clip_overlaps(grads, nullptr, numel, dtypes, count, false, norm, workspace, plan.parts * sizeof(double));
  if (st != MSM_OK) return st;
  msm::ClipBatch b;
  for (int64_t k = 0; k < plan.batches; ++k) {
    const int64_t i0 = k * msm::kClipTensors, left = count - i0;
    if (!clip_batch(grads, nullptr, numel, dtypes, i0, (int)(left < msm::kClipTensors ? left : msm::kClipTensors), &b))
      return MSM_ERR_INVALID_ARG;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  st = clip_sums(grads, numel, dtypes, count, plan, part, s);
  if (st != MSM_OK) return st;
  return status_of(msm::launch_clip_norm(part, plan.parts, norm, s));
}

msm_status msm_grad_clip(const void* const* grads, void* const* out, const int64_t* numel,
                         const int32_t* dtypes, int64_t count, float max_norm, float eps,
                         float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  msm_status st = clip_check(grads, numel, dtypes, count);
  if (st != MSM_OK) return st;
  if (!norm || !(max_norm >= 0.f) || !(eps >= 0.f)) return MSM_ERR_INVALID_ARG;
  if (out) {
    for (int64_t i = 0; i < count; ++i) {
      const size_t es = dtypes[i] == MSM_BF16 ? 2 : 4;
      if (numel[i] > 0 && (!out[i] || !aligned(out[i], es))) return MSM_ERR_INVALID_ARG;
    }
  }
  const ClipPlan plan = clip_plan(count);
  if (!workspace || workspace_bytes < (size_t)plan.parts * sizeof(double)) return MSM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MSM_ERR_INVALID_ARG;
  st = clip_overlaps(grads, out, numel, dtypes, count, true, norm, workspace, plan.parts * sizeof(double));
  if (st != MSM_OK) return st;
  msm::ClipBatch b;
  for (int64_t k = 0; k < plan.batches; ++k) {
    const int64_t i0 = k * msm::kClipTensors, left = count - i0;
    if (!clip_batch(grads, out, numel, dtypes, i0, (int)(left < msm::kClipTensors ? left : msm::kClipTensors), &b))
      return MSM_ERR_INVALID_ARG;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  st = clip_sums(grads, numel, dtypes, count, plan, part, s);
  if (st != MSM_OK) return st;
  const bool joined = plan.parts > msm::kClipPartials;  // too many for every launch to read
  if (joined && msm::launch_clip_norm(part, plan.parts, norm, s) != hipSuccess) return MSM_ERR_LAUNCH;
  for (int64_t k = plan.batches - 1; k >= 0; --k) {  // the tensors read last first
    const int64_t i0 = k * msm::kClipTensors, left = count - i0;
    clip_batch(grads, out, numel, dtypes, i0, (int)(left < msm::kClipTensors ? left : msm::kClipTensors), &b);
    const hipError_t e = msm::launch_clip_scale(b, joined ? nullptr : part, plan.parts, joined || k == 0 ? norm : nullptr, max_norm, eps, plan.groups, s);
    if (e != hipSuccess) return MSM_ERR_LAUNCH;
  }
  return MSM_OK;
}

}  // extern "C"
