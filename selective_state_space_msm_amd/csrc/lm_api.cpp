// C ABI of the embedding, the block norm and the linear cross entropy: argument checks, workspace
// layout, launches.  Every check happens before anything is enqueued; nothing here allocates
// device memory.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "../../include/msm.h"
#include "lm_internal.h"
#include "ops_check.h"

namespace {

using namespace msm::check;

constexpr int64_t kMost = ((int64_t)1 << 31) - 1;
bool known(msm_dtype t) { return t == MSM_F32 || t == MSM_BF16; }

struct Take {
  size_t at = 0;
  size_t operator()(size_t bytes) {
    const size_t here = at;
    at += align_up(bytes);
    return here;
  }
};

// ---- embedding ----

msm_status embed_check(int64_t tokens, int64_t V, int64_t D, msm_dtype table, msm_dtype io) {
  if (!known(table) || !known(io)) return MSM_ERR_UNSUPPORTED;
  if (tokens < 1 || V < 1 || D < 1 || tokens > kMost || V >= kMost || D > ((int64_t)1 << 24)) return MSM_ERR_INVALID_ARG;
  if (tokens * D > ((int64_t)1 << 48) || V * D > ((int64_t)1 << 48)) return MSM_ERR_INVALID_ARG;
  return MSM_OK;
}

struct EmbedLayout {
  size_t key[2], pos[2], hist, part[2], total;
  int waves, per, bits, passes;
};

EmbedLayout embed_layout(int64_t tokens, int64_t V, int64_t D) {
  EmbedLayout l{};
  int bits = 1;
  while (((int64_t)1 << bits) <= V) ++bits;  // keys are 0 ... V
  l.passes = (bits + msm::kEmbedMostBits - 1) / msm::kEmbedMostBits;
  l.bits = (bits + l.passes - 1) / l.passes;
  // at most 256 wavefronts: a workgroup of the second launch reads all of their counts
  int64_t per = ceil_div(ceil_div(tokens, 256), 64) * 64;
  if (per < 256) per = 256;
  l.per = (int)per;
  l.waves = (int)ceil_div(tokens, per);
  Take take;
  for (int i = 0; i < 2; ++i) {
    l.key[i] = take((size_t)tokens * 4);
    l.pos[i] = take((size_t)tokens * 4);
  }
  l.hist = take(((size_t)l.waves << l.bits) * 4);
  l.part[0] = take((size_t)(tokens / msm::kEmbedRun) * D * 4);
  l.part[1] = take((size_t)(tokens / msm::kEmbedRun / msm::kEmbedRun) * D * 4);
  l.total = take.at;
  return l;
}

// ---- block norm ----

msm_status block_norm_check(int64_t rows, int64_t D, msm_dtype io) {
  if (!known(io)) return MSM_ERR_UNSUPPORTED;
  if (rows < 1 || D < 1 || rows > kMost || D > ((int64_t)1 << 30)) return MSM_ERR_INVALID_ARG;
  if (rows * D > ((int64_t)1 << 50)) return MSM_ERR_INVALID_ARG;
  return MSM_OK;
}

// Workgroups of the backward: each leaves 8 D bytes of column sums, so few enough that they stay
// small beside the rows, and enough to fill the GPU.
int64_t block_norm_groups(int64_t rows, int64_t D, msm_dtype io) {
  const msm::BlockNormShape f = msm::block_norm_shape(D, true, io == MSM_BF16);
  if (f.T == 0) return rows < 64 ? rows : 64;
  const int64_t in_flight = f.T <= 64 ? 256 / f.T : 1, g = ceil_div(rows, 2 * in_flight);
  const int waves = f.T / 64, held = f.E == 4 ? 16 : 8;  // of a row; that a CU's registers hold
  const int64_t most = f.T <= 64 ? 512 : 256 * (waves < held ? held / waves : 1);
  return g > most ? most : g;
}

struct BlockNormLayout {
  size_t part, row_mean, total;
};
BlockNormLayout block_norm_layout(int64_t rows, int64_t D, msm_dtype io) {
  BlockNormLayout l{};
  Take take;
  l.part = take((size_t)block_norm_groups(rows, D, io) * 8 * (size_t)D);
  if (msm::block_norm_shape(D, true, io == MSM_BF16).T == 0) l.row_mean = take((size_t)rows * 4);
  l.total = take.at;
  return l;
}

// ---- linear cross entropy ----

struct XentLayout {
  size_t count, map, inverse, rows, xp, wp, stat, at_target, g, dx_sum, rest, sort, words, marks, lost, total;
  EmbedLayout sorted;  // from `sort` on
  int64_t DP, DQ, piece, piece_packed;
  int planes, splits;
  bool direct, few;
  int tile;
};

constexpr int64_t kXentMost = (int64_t)1 << 22;       // T V at most 2^37: 2^23 tiles of 128, 2^15 rounds of 256 workgroups
constexpr size_t kXentPiece = (size_t)256 << 20;      // bytes of a piece's g, and of its packed weights
constexpr size_t kXentUnaligned = (size_t)16 << 20;   // bytes of weights packed for their address alone

msm_status xent_check(int64_t T, int64_t V, int64_t D, msm_dtype io) {
  if (!known(io)) return MSM_ERR_UNSUPPORTED;
  if (T < 1 || V < 1 || D < 1) return MSM_ERR_INVALID_ARG;
  if (T > kXentMost || V > kXentMost || D > ((int64_t)1 << 16) || T * V > ((int64_t)1 << 37)) return MSM_ERR_UNSUPPORTED;
  return MSM_OK;
}

int64_t rows_of(size_t bytes, size_t row, int64_t V) {
  int64_t n = (int64_t)(bytes / row) / 256 * 256;
  const int64_t all = ceil_div(V, 256) * 256;
  if (n < 256) n = 256;
  return n < all ? n : all;
}

// The product of dx sums over the vocabulary and has few tiles where T and D are small: its sum is
// split until the tiles fill the GPU twice (rows without a target leave tiles without work) or a split
// has fewer than 8 steps of 64.
int xent_splits(int64_t T, int64_t D, int64_t piece, int planes) {
  const int64_t b = msm::xent_tile(D, T, piece, planes), slots = b == 256 || (planes > 1 && b == 128) ? 256 : 512;
  const int64_t tiles = ceil_div(D, b) * ceil_div(T, b);
  if (tiles > slots * 3 / 4) return 1;
  int64_t n = 2 * slots / tiles;
  if (n > piece / 512) n = piece / 512;
  return (int)(n < 1 ? 1 : (n > 32 ? 32 : n));
}

XentLayout xent_layout(int64_t T, int64_t V, int64_t D, msm_dtype io, bool bwd) {
  XentLayout l{};
  l.planes = io == MSM_BF16 ? 1 : 3;
  l.DP = ceil_div(D, 64) * 64;
  l.DQ = ceil_div(D, 4) * 4;
  l.direct = io == MSM_BF16 && D % 8 == 0;  // if the weights are aligned, too
  const size_t row_w = (size_t)l.DP * 2 * l.planes, row_g = (size_t)T * 2 * l.planes;
  l.piece = bwd ? rows_of(kXentPiece, row_g, V) : ceil_div(V, 256) * 256;
  l.piece_packed = rows_of(l.direct ? kXentUnaligned : kXentPiece, row_w, V);
  if (l.piece_packed > l.piece) l.piece_packed = l.piece;
  if (!l.direct) l.piece = l.piece_packed;
  Take take;
  if (!bwd && T <= msm::kXentFew) {
    l.xp = take((size_t)ceil_div(D, 32) * ceil_div(T, 16) * 1024 * l.planes);
    l.stat = take((size_t)msm::kXentFewGroups * T * 8);
    l.at_target = take((size_t)T * 4);
    l.few = true;
    l.total = take.at;
    return l;
  }
  l.count = take(4);
  l.map = take((size_t)T * 4);
  l.inverse = take((size_t)T * 4);
  l.rows = take((size_t)T * sizeof(msm::XentRow));
  l.xp = take((size_t)T * row_w);
  l.wp = take((size_t)l.piece_packed * row_w);
  if (bwd) {
    l.g = take((size_t)l.piece * row_g);
    l.splits = xent_splits(T, D, l.piece, l.planes);
    l.dx_sum = take((size_t)l.splits * T * l.DQ * 4);
    l.rest = take((size_t)T * 4);
    if (l.planes == 1) {
      l.sorted = embed_layout(T, V, 0);
      l.sort = take(l.sorted.total);
      l.words = take((size_t)V * sizeof(msm::XentPlaces));
      l.marks = take((size_t)msm::xent_marks(V));
      l.lost = take((size_t)(T * l.DQ + 256) * 4);  // a tile's columns behind the last row
    }
  } else {
    // pairs of sums of half a tile of the vocabulary, a piece at a time
    int64_t pairs = 0;
    for (int64_t piece : {l.piece, l.piece_packed}) {
      const int64_t half = msm::xent_tile(piece < V ? piece : V, T, D, l.planes) / 2, n = 2 * (ceil_div(V, 2 * half) + ceil_div(V, piece));
      if (n > pairs) pairs = n;
    }
    l.stat = take((size_t)pairs * T * 8);
    l.at_target = take((size_t)T * 4);
  }
  l.total = take.at;
  return l;
}

msm::XentArgs xent_args(const XentLayout& l, const void* x, const void* w, const int64_t* targets, int64_t T, int64_t V,
                        int64_t D, float scale, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  msm::XentArgs a{};
  a.x = x;
  a.w = w;
  a.targets = targets;
  a.count = reinterpret_cast<int32_t*>(ws + l.count);
  a.map = reinterpret_cast<int32_t*>(ws + l.map);
  a.inverse = l.few ? nullptr : reinterpret_cast<int32_t*>(ws + l.inverse);
  a.rows = reinterpret_cast<msm::XentRow*>(ws + l.rows);
  a.xp = ws + l.xp;
  a.wp = ws + l.wp;
  a.stat = reinterpret_cast<float*>(ws + l.stat);
  a.at_target = reinterpret_cast<float*>(ws + l.at_target);
  a.g = ws + l.g;
  a.dx_sum = reinterpret_cast<float*>(ws + l.dx_sum);
  a.rest = reinterpret_cast<float*>(ws + l.rest);
  a.splits = l.splits;
  a.T = T;
  a.V = V;
  a.D = D;
  a.DP = l.DP;
  a.DQ = l.DQ;
  a.w_direct = l.direct && aligned(w, 16);
  a.piece = a.w_direct ? l.piece : l.piece_packed;
  a.tile = msm::xent_tile(a.piece < V ? a.piece : V, T, D, l.planes);
  a.scale = scale;
  a.planes = l.planes;
  return a;
}

}  // namespace

extern "C" {

msm_status msm_embed_fwd(const int64_t* ids, const void* table, void* y, int64_t tokens, int64_t V, int64_t D,
                         float scale, msm_dtype table_io, msm_dtype io, void* stream) {
  const msm_status st = embed_check(tokens, V, D, table_io, io);
  if (st != MSM_OK) return st;
  if (!ids || !table || !y || !isfinite(scale)) return MSM_ERR_INVALID_ARG;
  if (!aligned(ids, 8) || !aligned(table, elem_bytes(table_io)) || !aligned(y, elem_bytes(io))) return MSM_ERR_INVALID_ARG;
  const Range ins[] = {rng(ids, (size_t)tokens * 8), rng(table, (size_t)(V * D) * elem_bytes(table_io))};
  const Range outs[] = {rng(y, (size_t)(tokens * D) * elem_bytes(io))};
  if (any_overlap(outs, 1, ins, 2)) return MSM_ERR_INVALID_ARG;
  msm::EmbedArgs a{};
  a.ids = ids;
  a.table = table;
  a.y = y;
  a.tokens = tokens;
  a.V = V;
  a.D = D;
  a.scale = scale;
  return status_of(msm::launch_embed_fwd(a, table_io == MSM_BF16, io == MSM_BF16, static_cast<hipStream_t>(stream)));
}

size_t msm_embed_bwd_workspace_bytes(int64_t tokens, int64_t V, int64_t D) {
  return embed_check(tokens, V, D, MSM_F32, MSM_F32) == MSM_OK ? embed_layout(tokens, V, D).total : 0;
}

msm_status msm_embed_bwd(const int64_t* ids, const void* dy, void* dtable, int64_t tokens, int64_t V, int64_t D,
                         float scale, msm_dtype table_io, msm_dtype io, void* workspace, size_t workspace_bytes,
                         void* stream) {
  const msm_status st = embed_check(tokens, V, D, table_io, io);
  if (st != MSM_OK) return st;
  if (!ids || !dy || !dtable || !isfinite(scale)) return MSM_ERR_INVALID_ARG;
  if (!aligned(ids, 8) || !aligned(dtable, elem_bytes(table_io)) || !aligned(dy, elem_bytes(io))) return MSM_ERR_INVALID_ARG;
  const EmbedLayout l = embed_layout(tokens, V, D);
  if (!workspace || workspace_bytes < l.total) return MSM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MSM_ERR_INVALID_ARG;
  const Range ins[] = {rng(ids, (size_t)tokens * 8), rng(dy, (size_t)(tokens * D) * elem_bytes(io))};
  const Range outs[] = {rng(dtable, (size_t)(V * D) * elem_bytes(table_io)), rng(workspace, l.total)};
  if (any_overlap(outs, 2, ins, 2)) return MSM_ERR_INVALID_ARG;
  char* ws = static_cast<char*>(workspace);
  msm::EmbedArgs a{};
  a.ids = ids;
  a.dy = dy;
  a.dtable = dtable;
  for (int i = 0; i < 2; ++i) {
    a.key[i] = reinterpret_cast<uint32_t*>(ws + l.key[i]);
    a.pos[i] = reinterpret_cast<uint32_t*>(ws + l.pos[i]);
    a.part[i] = reinterpret_cast<float*>(ws + l.part[i]);
  }
  if (tokens < msm::kEmbedDeep) a.part[1] = nullptr;
  a.hist = reinterpret_cast<uint32_t*>(ws + l.hist);
  a.tokens = tokens;
  a.V = V;
  a.D = D;
  a.scale = scale;
  a.waves = l.waves;
  a.per = l.per;
  a.bits = l.bits;
  a.passes = l.passes;
  return status_of(msm::launch_embed_bwd(a, table_io == MSM_BF16, io == MSM_BF16, static_cast<hipStream_t>(stream)));
}

msm_status msm_block_norm_fwd(const void* r, const float* weight, const void* o, const float* post_weight, const void* z,
                              void* r_out, void* y, float* rstd, float* post_rstd, int64_t rows, int64_t D, float scale,
                              float eps, msm_dtype io, void* stream) {
  const msm_status st = block_norm_check(rows, D, io);
  if (st != MSM_OK) return st;
  if (!r || !y || !isfinite(scale) || !(eps >= 0.f) || !isfinite(eps)) return MSM_ERR_INVALID_ARG;
  if (o ? !r_out : (r_out || z || post_weight || post_rstd)) return MSM_ERR_INVALID_ARG;
  const size_t es = elem_bytes(io), n = (size_t)(rows * D) * es, nd = (size_t)D * 4, nr = (size_t)rows * 4;
  if (!aligned(r, es) || !aligned(o, es) || !aligned(z, es) || !aligned(r_out, es) || !aligned(y, es)) return MSM_ERR_INVALID_ARG;
  // the residual stream may be updated in place: a row's elements are read before they are written
  const Range ins[] = {rng(r_out == r ? nullptr : r, n), rng(weight, nd), rng(o, n), rng(post_weight, nd), rng(z, n)};
  const Range outs[] = {rng(r_out, n), rng(y, n), rng(rstd, nr), rng(post_rstd, nr)};
  if (any_overlap(outs, 4, ins, 5)) return MSM_ERR_INVALID_ARG;
  msm::BlockNormArgs a{};
  a.r = r;
  a.o = o;
  a.z = z;
  a.weight = weight;
  a.post_weight = post_weight;
  a.r_out = r_out;
  a.y = y;
  a.rstd = rstd;
  a.post_rstd = post_rstd;
  a.rows = rows;
  a.D = D;
  a.scale = scale;
  a.eps = eps;
  return status_of(msm::launch_block_norm_fwd(a, io == MSM_BF16, static_cast<hipStream_t>(stream)));
}

size_t msm_block_norm_bwd_workspace_bytes(int64_t rows, int64_t D, msm_dtype io) {
  return block_norm_check(rows, D, io) == MSM_OK ? block_norm_layout(rows, D, io).total : 0;
}

msm_status msm_block_norm_bwd(const void* r_out, const void* dy, const float* rstd, const float* weight, const void* o,
                              const float* post_rstd, const float* post_weight, const void* z, const void* dr_out,
                              void* dr, void* do_, void* dz, float* dweight, float* dpost_weight, int64_t rows, int64_t D,
                              float scale, msm_dtype io, void* workspace, size_t workspace_bytes, void* stream) {
  const msm_status st = block_norm_check(rows, D, io);
  if (st != MSM_OK) return st;
  if (!r_out || !dy || !rstd || !dr || !isfinite(scale)) return MSM_ERR_INVALID_ARG;
  if (o ? (!post_rstd || !do_ || !z != !dz) : (post_rstd || post_weight || z || do_ || dz || dpost_weight)) return MSM_ERR_INVALID_ARG;
  const size_t es = elem_bytes(io), n = (size_t)(rows * D) * es, nd = (size_t)D * 4, nr = (size_t)rows * 4;
  for (const void* q : {r_out, dy, o, z, dr_out, (const void*)dr, (const void*)do_, (const void*)dz})
    if (!aligned(q, es)) return MSM_ERR_INVALID_ARG;
  const bool cols = dweight || dpost_weight;
  const BlockNormLayout l = block_norm_layout(rows, D, io);
  if (!workspace || workspace_bytes < l.total) return MSM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MSM_ERR_INVALID_ARG;
  const Range ins[] = {rng(r_out, n), rng(dy, n), rng(rstd, nr), rng(weight, nd), rng(o, n), rng(post_rstd, nr),
                       rng(post_weight, nd), rng(z, n), rng(dr_out, n)};
  const Range outs[] = {rng(dr, n), rng(do_, n), rng(dz, n), rng(dweight, nd), rng(dpost_weight, nd), rng(workspace, l.total)};
  if (any_overlap(outs, 6, ins, 9)) return MSM_ERR_INVALID_ARG;
  msm::BlockNormArgs a{};
  a.r_out = const_cast<void*>(r_out);
  a.dy = dy;
  a.rstd = const_cast<float*>(rstd);
  a.weight = weight;
  a.o = o;
  a.post_rstd = const_cast<float*>(post_rstd);
  a.post_weight = post_weight;
  a.z = z;
  a.dr_out = dr_out;
  a.dr = dr;
  a.do_ = do_;
  a.dz = dz;
  a.dweight = dweight;
  a.dpost_weight = dpost_weight;
  char* ws = static_cast<char*>(workspace);
  a.part = cols ? reinterpret_cast<float*>(ws + l.part) : nullptr;
  a.row_mean = reinterpret_cast<float*>(ws + l.row_mean);
  a.rows = rows;
  a.D = D;
  a.scale = scale;
  a.groups = (int32_t)block_norm_groups(rows, D, io);
  return status_of(msm::launch_block_norm_bwd(a, io == MSM_BF16, static_cast<hipStream_t>(stream)));
}

size_t msm_linear_cross_entropy_fwd_workspace_bytes(int64_t T, int64_t V, int64_t D, msm_dtype io) {
  return xent_check(T, V, D, io) == MSM_OK ? xent_layout(T, V, D, io, false).total : 0;
}

msm_status msm_linear_cross_entropy_fwd(const void* x, const void* weight, const int64_t* targets, float* loss, float* lse,
                                        int64_t T, int64_t V, int64_t D, float scale, msm_dtype io, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  const msm_status st = xent_check(T, V, D, io);
  if (st != MSM_OK) return st;
  const size_t es = elem_bytes(io);
  if (!x || !weight || !targets || !loss || !isfinite(scale)) return MSM_ERR_INVALID_ARG;
  if (!aligned(x, es) || !aligned(weight, es) || !aligned(targets, 8)) return MSM_ERR_INVALID_ARG;
  const XentLayout l = xent_layout(T, V, D, io, false);
  if (!workspace || workspace_bytes < l.total) return MSM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MSM_ERR_INVALID_ARG;
  const size_t nt = (size_t)T * 4;
  const Range ins[] = {rng(x, (size_t)(T * D) * es), rng(weight, (size_t)(V * D) * es), rng(targets, (size_t)T * 8)};
  const Range outs[] = {rng(loss, nt), rng(lse, nt), rng(workspace, l.total)};
  if (any_overlap(outs, 3, ins, 3)) return MSM_ERR_INVALID_ARG;
  msm::XentArgs a = xent_args(l, x, weight, targets, T, V, D, scale, workspace);
  a.loss = loss;
  a.lse = lse;
  return status_of(msm::launch_xent_fwd(a, io == MSM_BF16, static_cast<hipStream_t>(stream)));
}

size_t msm_linear_cross_entropy_bwd_workspace_bytes(int64_t T, int64_t V, int64_t D, msm_dtype io) {
  return xent_check(T, V, D, io) == MSM_OK ? xent_layout(T, V, D, io, true).total : 0;
}

msm_status msm_linear_cross_entropy_bwd(const void* x, const void* weight, const int64_t* targets, const float* lse,
                                        const float* dloss, const float* dlse, void* dx, void* dweight, int64_t T,
                                        int64_t V, int64_t D, float scale, msm_dtype io, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  const msm_status st = xent_check(T, V, D, io);
  if (st != MSM_OK) return st;
  const size_t es = elem_bytes(io);
  if (!x || !weight || !targets || !lse || !dloss || !dx || !isfinite(scale)) return MSM_ERR_INVALID_ARG;
  if (!aligned(x, es) || !aligned(weight, es) || !aligned(targets, 8) || !aligned(dx, es) || !aligned(dweight, es))
    return MSM_ERR_INVALID_ARG;
  const XentLayout l = xent_layout(T, V, D, io, true);
  if (!workspace || workspace_bytes < l.total) return MSM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MSM_ERR_INVALID_ARG;
  const size_t nt = (size_t)T * 4, nx = (size_t)(T * D) * es, nw = (size_t)(V * D) * es;
  const Range ins[] = {rng(x, nx), rng(weight, nw), rng(targets, (size_t)T * 8), rng(lse, nt), rng(dloss, nt), rng(dlse, nt)};
  const Range outs[] = {rng(dx, nx), rng(dweight, nw), rng(workspace, l.total)};
  if (any_overlap(outs, 3, ins, 6)) return MSM_ERR_INVALID_ARG;
  msm::XentArgs a = xent_args(l, x, weight, targets, T, V, D, scale, workspace);
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss;
  a.dlse = dlse;
  a.dx = dx;
  a.dw = dweight;
  msm::EmbedArgs sort{};
  if (dweight && l.planes == 1) {
    char* const ws = static_cast<char*>(workspace);
    for (int i = 0; i < 2; ++i) {
      sort.key[i] = reinterpret_cast<uint32_t*>(ws + l.sort + l.sorted.key[i]);
      sort.pos[i] = reinterpret_cast<uint32_t*>(ws + l.sort + l.sorted.pos[i]);
    }
    sort.hist = reinterpret_cast<uint32_t*>(ws + l.sort + l.sorted.hist);
    sort.ids = targets;
    sort.tokens = T;
    sort.V = V;
    sort.waves = l.sorted.waves;
    sort.per = l.sorted.per;
    sort.bits = l.sorted.bits;
    sort.passes = l.sorted.passes;
    a.key = sort.key[(sort.passes - 1) & 1];
    a.pos = sort.pos[(sort.passes - 1) & 1];
    a.words = reinterpret_cast<msm::XentPlaces*>(ws + l.words);
    a.marks = reinterpret_cast<uint8_t*>(ws + l.marks);
    a.clear = (int64_t)(l.marks - l.words) + msm::xent_marks(V);
    sort.dtable = a.words;
    sort.rows = a.inverse;
    a.lost = reinterpret_cast<float*>(ws + l.lost);
    a.log_run = 5;  // one more as the tokens quadruple: a frequent word has few runs, and a run few places
    while ((int64_t)1 << (2 * a.log_run) < T) ++a.log_run;
  }
  return status_of(msm::launch_xent_bwd(a, sort, io == MSM_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
