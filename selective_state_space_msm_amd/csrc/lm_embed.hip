// Token embedding (gfx950): y_t = scale table[id_t], and its gradient
// dtable[v] = scale sum over {t: id_t = v} of dy_t.  Ids outside [0, V) give a row of zeros and take
// no part in the gradient.
//
// The forward is a copy: bound by HBM (rows read, y written), or by the launch for a few tokens (16384
// tokens, D = 2048, fp32 to bf16: 25 us, repeated rows from the caches; 256 tokens, D = 4096: 3.2 us).
//
// The gradient reads dy once and writes dtable once, most of its rows zero.  Tokens are sorted by id
// (stable, digits of up to 9 bits), so that a vocabulary row's places stand side by side in the order
// of the batch, and every row is summed in that order without atomics.  A frequent token has
// thousands of places (of log-uniform ids over 65536, the first has 6% of them): aligned runs of 32
// places that belong to one row are summed beforehand, and from 8192 places on runs of 32 such sums
// again, so that a row adds at most 62 places, 62 sums of 32 and one sum per 1024 places (those in fp64);
// of fewer places it adds up to 255 sums of 32.  Where several threads share 16 bytes of a row, what each
// has summed is joined in fp32, at most 32 sums.
//
// A sorting pass is two launches: every wavefront counts the digits of its own places, then each
// workgroup finds its wavefronts' first positions from the counts of all (at most 256 wavefronts,
// so there is no launch for a scan) and moves the places.  Ranks among 64 places come from ballots
// over the digit's bits.  Up to 4096 places are sorted by one workgroup in LDS.
//
// 16384 tokens of 65536, D = 2048, bf16: 115 us, of which the four sorting launches, which write the
// zeros meanwhile, take 55, the runs 19 and the rows that have tokens 36.  2047 tokens of 1003,
// D = 129, fp32: 18.5 us in three launches.
#include "lm_internal.h"
#include "ops_row.hpp"

namespace msm {
namespace {

constexpr int kBins = 1 << kEmbedMostBits;
constexpr int64_t kMostGroups = (int64_t)1 << 20;

// ---- forward ----

// A thread makes 16 bytes of y.
template <typename TB, typename IO>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const EmbedArgs p, int64_t pieces) {
  constexpr int VEC = Chunk<IO>::VEC, TV = Chunk<TB>::VEC;
  const int64_t all = p.tokens * pieces;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t t = quotient(i, pieces), c = (i - t * pieces) * VEC, n = p.D - c;
    const int64_t id = p.ids[t];
    float x[VEC > TV ? VEC : TV];
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = 0.f;
    if (id >= 0 && id < p.V) {
      if constexpr (VEC >= TV) {
#pragma unroll
        for (int e = 0; e < VEC; e += TV) {
          Chunk<TB> r;
          r.zero();
          if (n > e) r.load(p.table, id * p.D + c + e, n - e);
          r.get(x + e);
        }
      } else {  // 16 bytes of fp32 from 8 of bf16
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (e < n) x[e] = io<TB>::widen(io<TB>::load(p.table, id * p.D + c + e));
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] *= p.scale;
    Chunk<IO> out;
    out.set(x);
    out.store(p.y, t * p.D + c, n);
  }
}

// ---- zeros ----

// Where the vocabulary outnumbers the tokens most rows of dtable are zero.  They are written while few
// workgroups sort: launch `at` of `of` of the sort fills its share of dtable, by the workgroups behind the
// sorting ones, and only the rows that have tokens are written again.  (With the zeros written row by row
// behind the sort: 136 us for 16384 tokens of 65536, D = 2048, bf16; 114 us this way.)
struct Fill {
  int64_t bytes;  // of dtable, 0: nothing to fill
  int at, of;
};
template <int THREADS>
__device__ __forceinline__ void fill_share(const EmbedArgs& p, const Fill& f, int first, int groups) {
  const int64_t units = (f.bytes + 15) / 16, lo = units * f.at / f.of, hi = units * (f.at + 1) / f.of;
  char* const to = static_cast<char*>(p.dtable);
  for (int64_t i = lo + (int64_t)(blockIdx.x - first) * THREADS + threadIdx.x; i < hi; i += (int64_t)(groups - first) * THREADS) {
    if (i * 16 + 16 <= f.bytes)
      *reinterpret_cast<u32x4_any*>(to + i * 16) = u32x4{0, 0, 0, 0};
    else
      for (int64_t b = i * 16; b < f.bytes; b += 2) *reinterpret_cast<uint16_t*>(to + b) = 0;
  }
}

// ---- sorting ----

__device__ __forceinline__ uint32_t key_of(const EmbedArgs& p, int64_t i) {
  const int64_t id = p.ids[i];
  return id >= 0 && id < p.V ? (uint32_t)id : (uint32_t)p.V;
}

// Lanes whose digit is this lane's, among the lanes that take part.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits, bool on) {
  uint64_t same = __ballot(on);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((digit >> b) & 1);
    same &= (digit >> b) & 1 ? set : ~set;
  }
  return same;
}

// Counts of a wavefront's digits, in its own bins.
__device__ __forceinline__ void count_digit(uint32_t* bins, uint32_t digit, int bits, bool on, int lane) {
  const uint64_t same = same_digit(digit, bits, on);
  if (on && (same & ((1ull << lane) - 1)) == 0) bins[digit] += __popcll(same);
}
// The place of this lane's digit, after which the wavefront's bins stand behind its places.
__device__ __forceinline__ uint32_t take_place(uint32_t* bins, uint32_t digit, int bits, bool on, int lane) {
  const uint64_t same = same_digit(digit, bits, on), below = same & ((1ull << lane) - 1);
  const uint32_t first = on ? bins[digit] : 0;
  if (on && below == 0) bins[digit] = first + __popcll(same);
  return first + __popcll(below);
}

// A wavefront works alone on its bins: LDS answers its accesses in order, the compiler must not reorder them.
__device__ __forceinline__ void wave_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

constexpr int kSortWaves = 8;
constexpr int kAhead = 4;  // loads of 64 places in flight

// pass 0 reads the ids, later ones what the pass before left
template <bool FIRST>
__device__ __forceinline__ void place_of(const EmbedArgs& p, int pass, int64_t i, uint32_t* key, uint32_t* pos) {
  if constexpr (FIRST) {
    *key = key_of(p, i);
    *pos = p.rows ? (uint32_t)p.rows[i] : (uint32_t)i;
  } else {
    *key = p.key[(pass - 1) & 1][i];
    *pos = p.pos[(pass - 1) & 1][i];
  }
}

template <bool FIRST>
__global__ __launch_bounds__(64 * kSortWaves) void embed_count_kernel(const EmbedArgs p, int pass, int sorting, const Fill f) {
  if ((int)blockIdx.x >= sorting) return fill_share<64 * kSortWaves>(p, f, sorting, gridDim.x);
  __shared__ uint32_t lds[kSortWaves][kBins];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nb = 1 << p.bits;
  const int64_t w = (int64_t)blockIdx.x * kSortWaves + wave;
  uint32_t* bins = lds[wave];
  for (int b = lane; b < nb; b += 64) bins[b] = 0;
  wave_order();
  for (int64_t k = 0; k < p.per; k += 64 * kAhead) {
    uint32_t key[kAhead], pos;
    bool on[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t i = w * p.per + k + 64 * j + lane;
      on[j] = w < p.waves && k + 64 * j < p.per && i < p.tokens;
      key[j] = 0;
      if (on[j]) place_of<FIRST>(p, pass, i, &key[j], &pos);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      count_digit(bins, (key[j] >> (pass * p.bits)) & (nb - 1), p.bits, on[j], lane);
      wave_order();
    }
  }
  if (w < p.waves)
    for (int b = lane; b < nb; b += 64) p.hist[w * nb + b] = bins[b];
}

// Exclusive sums of one value a thread over a workgroup of N threads, N <= 1024.
template <int N>
__device__ __forceinline__ uint32_t exclusive_sum(uint32_t v, uint32_t* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t s = v;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const uint32_t o = __shfl_up(s, m, 64);
    if (lane >= m) s += o;
  }
  if (lane == 63) lds[wave] = s;
  __syncthreads();
  uint32_t before = 0;
  for (int i = 0; i < wave; ++i) before += lds[i];
  return before + s - v;
}

template <bool FIRST>
__global__ __launch_bounds__(64 * kSortWaves) void embed_move_kernel(const EmbedArgs p, int pass, int sorting, const Fill f) {
  if ((int)blockIdx.x >= sorting) return fill_share<64 * kSortWaves>(p, f, sorting, gridDim.x);
  static_assert(64 * kSortWaves == kBins, "a thread for every bin");
  __shared__ uint32_t lds[kSortWaves][kBins];
  __shared__ uint32_t sums[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nb = 1 << p.bits, b = threadIdx.x;
  const int64_t w0 = (int64_t)blockIdx.x * kSortWaves;
  // this thread's bin: what stands before the workgroup's wavefronts, and in all
  uint32_t before = 0, total = 0;
  if (b < nb) {
    int64_t w = 0;
    for (; w + 32 <= p.waves; w += 32) {
      uint32_t c[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) c[j] = p.hist[(w + j) * nb + b];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        before += w + j < w0 ? c[j] : 0;
        total += c[j];
      }
    }
    for (; w < p.waves; ++w) {
      const uint32_t c = p.hist[w * nb + b];
      before += w < w0 ? c : 0;
      total += c;
    }
  }
  uint32_t at = exclusive_sum<kBins>(total, sums) + before;
  if (b < nb)
    for (int j = 0; j < kSortWaves; ++j) {
      lds[j][b] = at;
      if (w0 + j < p.waves) at += p.hist[(w0 + j) * nb + b];
    }
  __syncthreads();
  const int64_t w = w0 + wave;
  if (w >= p.waves) return;
  uint32_t* bins = lds[wave];
  for (int64_t k = 0; k < p.per; k += 64 * kAhead) {
    uint32_t key[kAhead], pos[kAhead];
    bool on[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t i = w * p.per + k + 64 * j + lane;
      on[j] = k + 64 * j < p.per && i < p.tokens;
      key[j] = pos[j] = 0;
      if (on[j]) place_of<FIRST>(p, pass, i, &key[j], &pos[j]);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t to = take_place(bins, (key[j] >> (pass * p.bits)) & (nb - 1), p.bits, on[j], lane);
      wave_order();
      if (on[j]) {
        p.key[pass & 1][to] = key[j];
        p.pos[pass & 1][to] = pos[j];
      }
    }
  }
}

// All passes in one workgroup, for up to kEmbedSmall places: a place's rank among its wavefront's is kept
// from the counting to the moving.
constexpr int kSmallWaves = 16;
__global__ __launch_bounds__(64 * kSmallWaves) void embed_sort_small_kernel(const EmbedArgs p, const Fill f) {
  if (blockIdx.x > 0) return fill_share<64 * kSmallWaves>(p, f, 1, gridDim.x);
  constexpr int kSteps = kEmbedSmall / (64 * kSmallWaves);
  __shared__ uint32_t keys[2][kEmbedSmall];
  __shared__ uint16_t places[2][kEmbedSmall];
  __shared__ uint32_t lds[kSmallWaves][kBins];
  __shared__ uint32_t sums[kSmallWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nb = 1 << p.bits, b = threadIdx.x;
  const int n = (int)p.tokens, steps = (n + kSmallWaves * 64 - 1) / (kSmallWaves * 64);
  for (int i = threadIdx.x; i < n; i += 64 * kSmallWaves) {
    keys[0][i] = key_of(p, i);
    places[0][i] = (uint16_t)i;
  }
  uint32_t* bins = lds[wave];
  for (int pass = 0; pass < p.passes; ++pass) {
    const int from = pass & 1, shift = pass * p.bits;
    uint32_t key[kSteps], rank[kSteps];
    for (int j = lane; j < nb; j += 64) bins[j] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = (wave * steps + k) * 64 + lane;
      const bool on = k < steps && i < n;
      key[k] = on ? keys[from][i] : 0;
      if (k < steps) rank[k] = take_place(bins, (key[k] >> shift) & (nb - 1), p.bits, on, lane);
      wave_order();
    }
    __syncthreads();
    uint32_t total = 0;
    if (b < nb)
      for (int j = 0; j < kSmallWaves; ++j) total += lds[j][b];
    uint32_t at = exclusive_sum<64 * kSmallWaves>(total, sums);
    if (b < nb)
      for (int j = 0; j < kSmallWaves; ++j) {
        const uint32_t c = lds[j][b];
        lds[j][b] = at;
        at += c;
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = (wave * steps + k) * 64 + lane;
      if (k < steps && i < n) {
        const uint32_t to = bins[(key[k] >> shift) & (nb - 1)] + rank[k];
        keys[from ^ 1][to] = key[k];
        places[from ^ 1][to] = places[from][i];
      }
    }
    __syncthreads();
  }
  const int last = p.passes & 1, out = (p.passes - 1) & 1;
  for (int i = threadIdx.x; i < n; i += 64 * kSmallWaves) {
    p.key[out][i] = keys[last][i];
    p.pos[out][i] = p.rows ? (uint32_t)p.rows[places[last][i]] : places[last][i];
  }
}

// ---- sums ----

// x += 16 bytes of the rows pos[i0 ... i1) of dy, eight of them in flight
template <typename IO>
__device__ __forceinline__ void add_places(const EmbedArgs& p, const uint32_t* pos, int64_t i0, int64_t i1, int64_t c,
                                           float (&x)[Chunk<IO>::VEC]) {
  constexpr int VEC = Chunk<IO>::VEC, N = 8;
  const int by = Chunk<IO>::short_by(c, p.D);
  for (int64_t i = i0; i < i1; i += N) {
    Chunk<IO> r[N];
    uint32_t at[N];
#pragma unroll
    for (int j = 0; j < N; ++j) at[j] = i + j < i1 ? pos[i + j] : 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      r[j].zero();
      if (i + j < i1) r[j].load_row(p.dy, (int64_t)at[j] * p.D, c, p.D);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float v[VEC];
      r[j].get_row(v, by);
      if (i + j < i1)
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] += v[e];
    }
  }
}

// x += sums j0 ... j1 of a level, four in flight
template <int VEC, typename F>
__device__ __forceinline__ void add_sums(const float* part, int64_t j0, int64_t j1, int64_t D, int64_t c, F (&x)[VEC]) {
  constexpr int N = 4;
  for (int64_t j = j0; j < j1; j += N) {
    Chunk<float> r[N][VEC / 4];
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int e = 0; e < VEC / 4; ++e) {
        r[k][e].zero();
        if (j + k < j1 && c + 4 * e < D) r[k][e].load(part, (j + k) * D + c + 4 * e, D - c - 4 * e);
      }
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (j + k < j1)
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] += __uint_as_float(r[k][e / 4].raw[e % 4]);
  }
}

// Threads of a workgroup over 16-byte pieces of a row, blockIdx.y the 256 of them: where there are few,
// `parts` threads share a piece, and what each has summed is joined in their order.
struct Share {
  int part, parts;
  int64_t q;  // the piece
  bool on;
};
__device__ __forceinline__ Share share_of(int64_t pieces) {
  const int64_t left = pieces - (int64_t)blockIdx.y * 256;
  const int here = (int)(left < 256 ? left : 256), t = threadIdx.x;
  const int parts = here > 128 ? 1 : (256 / here < 32 ? 256 / here : 32);
  return Share{t / here, parts, (int64_t)blockIdx.y * 256 + t % here, t < here * parts};
}
// Share number `part` of a list
__device__ __forceinline__ int64_t cut(int64_t a, int64_t b, const Share& s, int part) {
  return a + (b - a) * part / s.parts;
}
// x of the first thread of each piece: the sum of all its threads'.  `lds` holds 256 VEC floats; its barriers
// are for the whole workgroup.
template <int VEC>
__device__ __forceinline__ void join_shares(const Share& s, int64_t pieces, float (&x)[VEC], float* lds) {
  if (s.parts == 1) return;
  const int64_t left = pieces - (int64_t)blockIdx.y * 256;
  const int here = (int)(left < 256 ? left : 256);
  __syncthreads();  // the join before has been read
#pragma unroll
  for (int e = 0; e < VEC; ++e) lds[threadIdx.x * VEC + e] = x[e];
  __syncthreads();
  if (s.on && s.part == 0)
    for (int k = 1; k < s.parts; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[e] += lds[(threadIdx.x + k * here) * VEC + e];
}

// Sums of the runs [32 k, 32 k + 32) of places that belong to one vocabulary row.
template <typename IO>
__global__ __launch_bounds__(256) void embed_run_kernel(const EmbedArgs p, int64_t runs, int64_t pieces) {
  constexpr int VEC = Chunk<IO>::VEC;
  __shared__ float lds[256 * VEC];
  const uint32_t *key = p.key[(p.passes - 1) & 1], *pos = p.pos[(p.passes - 1) & 1];
  const Share s = share_of(pieces);
  const int64_t c = s.q * VEC;
  for (int64_t k = blockIdx.x; k < runs; k += gridDim.x) {
    const int64_t i0 = k * kEmbedRun, i1 = i0 + kEmbedRun;
    if (key[i0] != key[i1 - 1] || key[i0] >= p.V) continue;
    float x[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = 0.f;
    if (s.on) add_places<IO>(p, pos, cut(i0, i1, s, s.part), cut(i0, i1, s, s.part + 1), c, x);
    join_shares<VEC>(s, pieces, x, lds);
    if (s.on && s.part == 0)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (c + e < p.D) p.part[0][k * p.D + c + e] = x[e];
  }
}

// The same over 32 runs of one vocabulary row, a thread a column.
__global__ __launch_bounds__(256) void embed_run2_kernel(const EmbedArgs p, int64_t runs) {
  const uint32_t* key = p.key[(p.passes - 1) & 1];
  for (int64_t k = blockIdx.x; k < runs; k += gridDim.x) {
    const int64_t i0 = k * kEmbedRun * kEmbedRun;
    if (key[i0] != key[i0 + kEmbedRun * kEmbedRun - 1] || key[i0] >= p.V) continue;
    for (int64_t c = (int64_t)blockIdx.y * 256 + threadIdx.x; c < p.D; c += gridDim.y * 256) {
      float x = 0.f;
#pragma unroll 8
      for (int j = 0; j < kEmbedRun; ++j) x += p.part[0][(k * kEmbedRun + j) * p.D + c];
      p.part[1][k * p.D + c] = x;
    }
  }
}

constexpr int kBusy = 8;      // a row of more places has a workgroup of its own
constexpr int kMostRows = 64;
// Vocabulary rows of a workgroup: more where a row has few pieces.
__host__ __device__ constexpr int rows_of(int64_t pieces) { return pieces <= 32 ? kMostRows : 8; }

// The first of the places lo ... hi whose key is v or more, found by a wavefront: 64 probes a round.
__device__ __forceinline__ int64_t first_place(const uint32_t* key, int64_t lo, int64_t hi, int64_t v) {
  const int lane = threadIdx.x & 63;
  while (lo < hi) {
    const int64_t step = (hi - lo + 63) / 64, at = lo + lane * step;
    const int below = __popcll(__ballot(at < hi && (int64_t)key[at < hi ? at : lo] < v));
    if (below == 0) return lo;
    const int64_t end = lo + below * step;
    lo += (below - 1) * step + 1;
    hi = end < hi ? end : hi;
  }
  return lo;
}

// first[r]: the first place of row v0 + r or of what comes after it, r = 0 ... rows, by a workgroup.
// Its barriers close what was read of `first` before; `ends` holds two words, `near` the positions of
// the first 256 places.
__device__ __forceinline__ void first_places(const uint32_t* key, const uint32_t* pos, int64_t tokens, int64_t v0, int rows,
                                             uint32_t* first, uint32_t* ends, uint32_t* near) {
  const int wave = threadIdx.x >> 6;
  __syncthreads();
  if (wave < 2) {
    const int64_t e = first_place(key, 0, tokens, v0 + wave * rows);
    if ((threadIdx.x & 63) == 0) ends[wave] = (uint32_t)e;
  }
  __syncthreads();
  const int64_t lo = ends[0], hi = ends[1], n = hi - lo;
  if (threadIdx.x < n) near[threadIdx.x] = pos[lo + threadIdx.x];
  if (n < 256) {
    const int t = threadIdx.x;
    if (t <= n) {  // place t ends the rows before its own, n ends them all
      const int64_t from = t == 0 ? 0 : (int64_t)key[lo + t - 1] - v0 + 1;
      const int64_t to = t == n ? rows : (int64_t)key[lo + t] - v0;
      for (int64_t r = from; r <= to; ++r) first[r] = (uint32_t)(lo + t);
    }
  } else {
    for (int r = threadIdx.x; r <= rows; r += 256) {
      int64_t a = lo, b = hi;
      while (a < b) {
        const int64_t mid = (a + b) / 2;
        if ((int64_t)key[mid] < v0 + r)
          a = mid + 1;
        else
          b = mid;
      }
      first[r] = (uint32_t)a;
    }
  }
  __syncthreads();
}

template <typename TB, int VEC>
__device__ __forceinline__ void store_row(const EmbedArgs& p, int64_t v, int64_t c, float (&x)[VEC]) {
  constexpr int TV = Chunk<TB>::VEC;
  const int64_t at = v * p.D + c, n = p.D - c;
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] *= p.scale;
  if constexpr (VEC >= TV) {
#pragma unroll
    for (int e = 0; e < VEC; e += TV) {
      Chunk<TB> out;
      out.set(x + e);
      if (n > e) out.store(p.dtable, at + e, n - e);
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < n) io<TB>::store(p.dtable, at + e, x[e]);
  }
}

// The row of the places i0 ... i1, more than kBusy, by a workgroup.
template <typename TB, typename IO>
__device__ __forceinline__ void busy_row(const EmbedArgs& p, const Share& s, int64_t pieces, const uint32_t* pos, int64_t v, int64_t i0,
                                         int64_t i1, float* lds) {
  constexpr int VEC = Chunk<IO>::VEC;
  const int64_t c = s.q * VEC;
  float x[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = 0.f;
  const auto places = [&](int64_t a, int64_t b) { add_places<IO>(p, pos, cut(a, b, s, s.part), cut(a, b, s, s.part + 1), c, x); };
  const auto sums = [&](const float* part, int64_t a, int64_t b, auto& y) {
    add_sums<VEC>(part, cut(a, b, s, s.part), cut(a, b, s, s.part + 1), p.D, c, y);
  };
  if (!s.on) {
  } else if (i1 - i0 < 2 * kEmbedRun) {
    places(i0, i1);
  } else {
    constexpr int R = kEmbedRun;
    const int64_t j0 = (i0 + R - 1) / R, j1 = i1 / R;  // whole runs
    const int64_t m0 = (j0 + R - 1) / R, m1 = j1 / R;  // whole runs of runs
    places(i0, j0 * R);
    if (p.part[1] && m0 < m1) {
      sums(p.part[0], j0, m0 * R, x);
      double wide[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) wide[e] = x[e];
      sums(p.part[1], m0, m1, wide);
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[e] = (float)wide[e];
      sums(p.part[0], m1 * R, j1, x);
    } else {
      sums(p.part[0], j0, j1, x);
    }
    places(j1 * R, i1);
  }
  join_shares<VEC>(s, pieces, x, lds);
  if (s.on && s.part == 0) store_row<TB, VEC>(p, v, c, x);
}

// 16 bytes of a row of up to kBusy places; at(j): the position of place j.
template <typename TB, typename IO, typename At>
__device__ __forceinline__ void light_row(const EmbedArgs& p, int64_t v, int64_t c, int count, const At& at) {
  constexpr int VEC = Chunk<IO>::VEC;
  float x[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = 0.f;
  if (count > 0) {
    const int by = Chunk<IO>::short_by(c, p.D);
    Chunk<IO> in[kBusy];
#pragma unroll
    for (int j = 0; j < kBusy; ++j) {
      in[j].zero();
      if (j < count) in[j].load_row(p.dy, (int64_t)at(j) * p.D, c, p.D);
    }
#pragma unroll
    for (int j = 0; j < kBusy; ++j) {
      float y[VEC];
      in[j].get_row(y, by);
      if (j < count)
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] += y[e];
    }
  }
  store_row<TB, VEC>(p, v, c, x);
}

// All rows.  The first `busy` workgroups each look at one place in kBusy: a row of more places holds at
// least one of these, and the workgroup of the first of them has the row.  The others take some rows each:
// one batch of loads a row.  (With the busy rows among the others, the workgroup of the first rows took 16 of
// them one after another: 500 us of 543 for 16384 tokens of 65536, D = 2048, bf16.)
template <typename TB, typename IO>
__global__ __launch_bounds__(256) void embed_rows_kernel(const EmbedArgs p, int64_t pieces, int64_t busy) {
  constexpr int VEC = Chunk<IO>::VEC;
  __shared__ uint32_t first[kMostRows + 1], ends[2], near[256];
  __shared__ float lds[256 * VEC];
  const uint32_t *key = p.key[(p.passes - 1) & 1], *pos = p.pos[(p.passes - 1) & 1];
  const int each = rows_of(pieces);
  const int64_t groups = (p.V + each - 1) / each;
  const Share s = share_of(pieces);
  for (int64_t g = blockIdx.x; g < busy + groups; g += gridDim.x) {
    if (g < busy) {
      const int64_t at = g * kBusy, v = key[at];
      if (v >= p.V) continue;
      // the row's workgroup is an earlier one
      if (at >= kBusy && key[at - kBusy] == v) continue;
      __syncthreads();
      if (threadIdx.x < 128) {
        const int64_t e = first_place(key, 0, p.tokens, v + (threadIdx.x >> 6));
        if ((threadIdx.x & 63) == 0) ends[threadIdx.x >> 6] = (uint32_t)e;
      }
      __syncthreads();
      const int64_t i0 = ends[0], i1 = ends[1];
      if (i1 - i0 > kBusy) busy_row<TB, IO>(p, s, pieces, pos, v, i0, i1, lds);
      continue;
    }
    const int64_t v0 = (g - busy) * each;
    first_places(key, pos, p.tokens, v0, each, first, ends, near);
    const int rows = (int)(p.V - v0 < each ? p.V - v0 : each);
    // this workgroup's pieces of the rows, in 32 bits
    const int64_t q0 = (int64_t)blockIdx.y * 256;
    const uint32_t here = (uint32_t)(pieces - q0 < 256 ? pieces - q0 : 256), all = rows * here;
    for (uint32_t k = threadIdx.x; k < all; k += 256) {
      const uint32_t r = k / here;
      const int64_t i0 = first[r];
      const int count = (int)(first[r + 1] - i0);
      if (count > kBusy) continue;
      light_row<TB, IO>(p, v0 + r, (q0 + (k - r * here)) * VEC, count, [&](int j) {
        const int64_t at = i0 + j - ends[0];
        return at < 256 ? near[at] : pos[i0 + j];
      });
    }
  }
}

// The rows that have tokens, where the others are filled already: a workgroup takes those whose first
// place is among its kBusy places.
template <typename TB, typename IO>
__global__ __launch_bounds__(256) void embed_present_kernel(const EmbedArgs p, int64_t pieces) {
  constexpr int VEC = Chunk<IO>::VEC, W = 2 * kBusy;
  constexpr uint32_t kNone = 0xffffffffu;  // no key: V is below it
  __shared__ uint32_t near_key[W + 1], near_pos[W];
  __shared__ float lds[256 * VEC];
  const uint32_t *key = p.key[(p.passes - 1) & 1], *pos = p.pos[(p.passes - 1) & 1];
  const Share s = share_of(pieces);
  const int64_t q0 = (int64_t)blockIdx.y * 256, groups = (p.tokens + kBusy - 1) / kBusy;
  const uint32_t here = (uint32_t)(pieces - q0 < 256 ? pieces - q0 : 256);
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
    const int64_t i0 = g * kBusy;
    __syncthreads();  // the places before have been read
    if (threadIdx.x <= W) {  // near_key[i + 1] is place i's
      const int64_t i = i0 + (int)threadIdx.x - 1;
      near_key[threadIdx.x] = i >= 0 && i < p.tokens ? key[i] : kNone;
      if (threadIdx.x > 0) near_pos[threadIdx.x - 1] = i < p.tokens ? pos[i] : 0;
    }
    __syncthreads();
    // places of the row that starts at place i, kBusy + 1 for more than kBusy, 0: none starts there
    const auto count_of = [&](int i) {
      const uint32_t v = near_key[i + 1];
      if (v == near_key[i] || v >= (uint32_t)p.V) return 0;
      int n = 1;
      while (n <= kBusy && i + n < W && near_key[i + 1 + n] == v) ++n;
      return n;
    };
    for (uint32_t k = threadIdx.x; k < kBusy * here; k += 256) {
      const int i = (int)(k / here), count = count_of(i);
      if (count == 0 || count > kBusy) continue;
      light_row<TB, IO>(p, near_key[i + 1], (q0 + (k - i * here)) * VEC, count, [&](int j) { return near_pos[i + j]; });
    }
    for (int i = 0; i < kBusy; ++i) {
      if (count_of(i) <= kBusy) continue;
      const int64_t v = near_key[i + 1];
      busy_row<TB, IO>(p, s, pieces, pos, v, i0 + i, first_place(key, i0 + i, p.tokens, v + 1), lds);
    }
  }
}

unsigned groups_of(int64_t n) { return (unsigned)(n < 1 ? 1 : (n < kMostGroups ? n : kMostGroups)); }

// Workgroups that fill `bytes` beside a sort of `of` launches
unsigned fill_groups(int64_t bytes, int of) {
  const int64_t n = (bytes / of + 65535) / 65536;
  return (unsigned)(n < 1024 ? n : 1024);
}

template <bool FIRST>
hipError_t sort_pass(const EmbedArgs& a, int pass, int64_t fill, hipStream_t s) {
  const int sorting = (a.waves + kSortWaves - 1) / kSortWaves, of = 2 * a.passes;
  const dim3 grid(sorting + fill_groups(fill, of)), block(64 * kSortWaves);
  hipLaunchKernelGGL(embed_count_kernel<FIRST>, grid, block, 0, s, a, pass, sorting, Fill{fill, 2 * pass, of});
  hipLaunchKernelGGL(embed_move_kernel<FIRST>, grid, block, 0, s, a, pass, sorting, Fill{fill, 2 * pass + 1, of});
  return hipGetLastError();
}

template <typename TB, typename IO>
hipError_t fwd(const EmbedArgs& a, hipStream_t s) {
  const int64_t pieces = (a.D + Chunk<IO>::VEC - 1) / Chunk<IO>::VEC;
  hipLaunchKernelGGL((embed_fwd_kernel<TB, IO>), dim3(groups_of((a.tokens * pieces + 255) / 256)), dim3(256), 0, s, a, pieces);
  return hipGetLastError();
}

hipError_t sort_all(const EmbedArgs& a, int64_t fill, hipStream_t s) {
  if (a.tokens <= kEmbedSmall) {
    hipLaunchKernelGGL(embed_sort_small_kernel, dim3(1 + fill_groups(fill, 1)), dim3(64 * kSmallWaves), 0, s, a, Fill{fill, 0, 1});
    return hipGetLastError();
  }
  hipError_t e = sort_pass<true>(a, 0, fill, s);
  for (int pass = 1; pass < a.passes && e == hipSuccess; ++pass) e = sort_pass<false>(a, pass, fill, s);
  return e;
}

template <typename TB, typename IO>
hipError_t bwd(const EmbedArgs& a, hipStream_t s) {
  const int64_t pieces = (a.D + Chunk<IO>::VEC - 1) / Chunk<IO>::VEC, each = rows_of(pieces);
  const unsigned slices = (unsigned)((pieces + 255) / 256);
  const bool sparse = a.V >= a.tokens;
  const hipError_t e = sort_all(a, sparse ? a.V * a.D * io<TB>::es : 0, s);
  if (e != hipSuccess) return e;
  if (a.tokens >= 2 * kEmbedRun) {
    const int64_t runs = a.tokens / kEmbedRun;
    hipLaunchKernelGGL((embed_run_kernel<IO>), dim3(groups_of(runs), slices), dim3(256), 0, s, a, runs, pieces);
    if (a.part[1]) {
      const int64_t runs2 = runs / kEmbedRun;
      hipLaunchKernelGGL(embed_run2_kernel, dim3(groups_of(runs2), slices), dim3(256), 0, s, a, runs2);
    }
  }
  if (sparse) {
    hipLaunchKernelGGL((embed_present_kernel<TB, IO>), dim3(groups_of((a.tokens + kBusy - 1) / kBusy), slices), dim3(256), 0, s, a, pieces);
  } else {
    const int64_t busy = a.tokens > kBusy ? (a.tokens + kBusy - 1) / kBusy : 0;
    hipLaunchKernelGGL((embed_rows_kernel<TB, IO>), dim3(groups_of(busy + (a.V + each - 1) / each), slices), dim3(256), 0, s, a, pieces, busy);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_fwd(const EmbedArgs& a, int table_bf16, int io_bf16, hipStream_t s) {
  if (table_bf16) return io_bf16 ? fwd<bf16_storage, bf16_storage>(a, s) : fwd<bf16_storage, float>(a, s);
  return io_bf16 ? fwd<float, bf16_storage>(a, s) : fwd<float, float>(a, s);
}
hipError_t launch_embed_sort(const EmbedArgs& a, int64_t fill, hipStream_t s) { return sort_all(a, fill, s); }
hipError_t launch_embed_bwd(const EmbedArgs& a, int table_bf16, int io_bf16, hipStream_t s) {
  if (table_bf16) return io_bf16 ? bwd<bf16_storage, bf16_storage>(a, s) : bwd<bf16_storage, float>(a, s);
  return io_bf16 ? bwd<float, bf16_storage>(a, s) : bwd<float, float>(a, s);
}

}  // namespace msm
