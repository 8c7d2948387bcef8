// Cross entropy of a linear layer over a vocabulary, without keeping its logits (gfx950).
//   l_tv = scale x_t . W_v,  lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l_t,target(t)
//   g_tv = scale ((dloss_t + dlse_t) exp(l_tv - lse_t) - dloss_t [v = target(t)])
//   dx = g W,  dW = g^T x
//
// All of it is matrix products: 2 T V D operations forward, 6 T V D backward (the logits again, dx,
// dW), on bf16 matrix cores.  The forward's tiles end in the largest logit and the sum of
// exponentials of their columns; the backward takes the vocabulary in pieces, and a piece's g is all
// of the logits that is ever in memory.
//
// One product kernel serves all three: C[m][n] = sum_k A[m][k] B[n][k], C tiles of 256 x 256 (128 x 128
// and 64 x 64 where these are few), 64 values of k at a time through LDS, the loads of a later step
// issued between the present step's products.  A and B are each either rows of k ("rows": k is contiguous in
// memory) or k rows ("columns": m or n is contiguous), which is read transposed out of LDS.  m is
// always the index that is contiguous in the result, as a lane's accumulators hold four consecutive
// m of one n: logits are made as [v][t], so that the sums over v stay within a lane's registers but
// for two exchanges; dx as [d][t] and dW as [d][v], stored four values at a time.
//
// bf16 inputs are multiplied as they are; g is rounded to bf16 for the products with W and x.  What the
// target's entry, most of a row's g, loses by that is added to dx and to dweight in fp32 (without it
// dweight of 8192 tokens of 65536, D = 2048, was off by 2.2e-3 of its size from its values in 32 bits); the other
// entries' errors, of at most 2^-8 and either sign, are summed over many small terms.  fp32 values are cut into three bf16 parts, and the six products that matter are
// summed, g too.  Rows without a target are left out of all products: the rows that
// take part are gathered in front, and what the others hold is never multiplied.
//
// 7780 of 8192 tokens take part, 65536 words, D = 2048, bf16: forward 1602 to 1682 us (1242 to 1304 TFLOP/s over
// those rows, the products alone 1306 over whole tiles in a run of 1680), backward 5115 to 5270 (1189 to 1225); a
// library product of 8192^3 reaches 1200 to 1240.  What bounds the products is the clock under matrix load (1.85 to
// 2.05 GHz) and the matrix units, busy 61 to 70% of it.  16 tokens, D = 4096: 100 us, 5.4 TB/s of weights.  fp32,
// 1000 of 1999 tokens of 10007, D = 513, backward: 278 to 290 us, six bf16 products for each of fp32.
#include "lm_internal.h"
#include "ops_row.hpp"

namespace msm {
namespace {

// ---- parts ----
// fp32 values in three bf16 parts: the first 8 bits, the next 8 rounded, what is left (exact).  The products
// of parts that are left out (second times third, third times third) are then of either sign and below 2^-23
// of a product; with all parts cut off they would all have the product's sign and make logits too small.
// The first part is not rounded, so the largest finite values stay finite.
__device__ __forceinline__ void cut3(float x0, float x1, uint32_t (&w)[3]) {
  const uint32_t u0 = __float_as_uint(x0), u1 = __float_as_uint(x1);
  w[0] = pack_hi(u0, u1);
  x0 -= __uint_as_float(u0 & 0xffff0000u);
  x1 -= __uint_as_float(u1 & 0xffff0000u);
#pragma unroll
  for (int q = 1; q < 3; ++q) {
    const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x0)), hi = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x1));
    w[q] = lo | (hi << 16);
    x0 -= __uint_as_float(lo << 16);
    x1 -= __uint_as_float(hi << 16);
  }
}
template <int P>
__device__ __forceinline__ Part<P> parts_of(const float (&x)[8]) {
  if constexpr (P == 1) {
    return split<1>(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]});
  } else {
    Part<3> r;
    u32x4 w[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t c[3];
      cut3(x[2 * i], x[2 * i + 1], c);
#pragma unroll
      for (int q = 0; q < 3; ++q) w[q][i] = c[q];
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) r.p[q] = __builtin_bit_cast(bf16x8, w[q]);
    return r;
  }
}

// ---- rows that take part ----

// The targets in order, and the places of their rows in xp (`gathered`: the rows that take part in front), for up
// to kXentRanked rows: a row's place is the number of rows before it, counted by a wavefront.  Workgroup `group` of
// `groups` takes its share, and of clearing the words' places.
template <int THREADS>
__device__ __forceinline__ void order_targets(const XentArgs& p, int group, int groups, bool gathered) {
  __shared__ uint32_t keys[kXentRanked];
  const int lane = threadIdx.x & 63, T = (int)p.T;
  for (int64_t i = (int64_t)group * THREADS + threadIdx.x; i < p.clear / 16; i += (int64_t)groups * THREADS)
    reinterpret_cast<u32x4*>(p.words)[i] = u32x4{0, 0, 0, 0};
  const uint32_t none = (uint32_t)p.V;
  for (int t = threadIdx.x; t < T; t += THREADS) {
    const int64_t id = p.targets[t];
    keys[t] = id >= 0 && id < p.V ? (uint32_t)id : none;
  }
  __syncthreads();
  for (int row = group * (THREADS / 64) + threadIdx.x / 64; row < T; row += groups * (THREADS / 64)) {
    const uint32_t own = keys[row];
    int before = 0, live = 0;
#pragma unroll 4
    for (int t = lane; t < T; t += 64) {
      const uint32_t other = keys[t];
      before += other < own + (t < row);  // V + 1 is below 2^32
      live += t < row && other != none;
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
      before += __shfl_xor(before, m, 64);
      live += __shfl_xor(live, m, 64);
    }
    if (lane == 0) {
      p.key[before] = own;
      p.pos[before] = (uint32_t)(gathered ? live : row);
    }
  }
}

// Their places in order, by one workgroup; the others put the targets in order, if that is asked for.
__global__ __launch_bounds__(1024) void xent_rows_kernel(const XentArgs p) {
  if (blockIdx.x > 0) return order_targets<1024>(p, blockIdx.x - 1, gridDim.x - 1, true);
  __shared__ int sums[2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int base = 0, turn = 0;
  for (int64_t t0 = 0; t0 < p.T; t0 += 1024, turn ^= 1) {
    const int64_t t = t0 + threadIdx.x;
    const int64_t target = t < p.T ? p.targets[t] : -1;
    const bool on = target >= 0 && target < p.V;
    const uint64_t set = __ballot(on);
    if (lane == 0) sums[turn][wave] = __popcll(set);
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < 16; ++i) {
      before += i < wave ? sums[turn][i] : 0;
      all += sums[turn][i];
    }
    const int at = base + before + __popcll(set & ((1ull << lane) - 1));
    if (t < p.T) p.inverse[t] = on ? at : -1;
    if (on) {
      XentRow r;
      r.target = (int32_t)target;
      r.lse = p.dloss ? p.lse[t] : 0.f;
      r.dloss = p.dloss ? p.dloss[t] : 0.f;
      r.both = r.dloss + (p.dlse ? p.dlse[t] : 0.f);
      p.map[at] = (int32_t)t;
      p.rows[at] = r;
    }
    base += all;
  }
  if (threadIdx.x == 0) *p.count = base;
}

// bf16 parts of rows, in rows of DP elements with zeros behind the D of the source; `map`: places
// of the rows in the source, `count` of them (null: n rows as they come).
template <typename IO>
__global__ __launch_bounds__(256) void xent_pack_kernel(const void* src, const int32_t* map, const int32_t* count,
                                                        int64_t n, int64_t D, int64_t DP, int64_t plane, uint16_t* dst) {
  constexpr int P = io<IO>::es == 2 ? 1 : 3;
  const int64_t chunks = DP / 8, all = (count ? (int64_t)*count : n) * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t row = quotient(i, chunks), c = (i - row * chunks) * 8, left = D - c;
    const int64_t at = (map ? (int64_t)map[row] : row) * D + c;
    constexpr int VEC = Chunk<IO>::VEC;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; e += VEC) {
      Chunk<IO> r;
      r.zero();
      if (left > e) r.load(src, at + e, left - e);
      r.get(x + e);
    }
    store_parts(dst + row * DP + c, plane, parts_of<P>(x));
  }
}

// Few rows stay where they are, those that are left out as zeros: their places need no launch of their own,
// and the first piece of w, if it is packed, goes along (a
// forward of 348 rows of 105, D = 45, bf16: 25.6 us with launches of their own, 19.5 with one).
template <typename IO>
__global__ __launch_bounds__(256) void xent_gather_kernel(const XentArgs p, int64_t w_rows) {
  constexpr int P = io<IO>::es == 2 ? 1 : 3, VEC = Chunk<IO>::VEC;
  if (p.words) order_targets<256>(p, blockIdx.x, gridDim.x, false);
  const int64_t chunks = p.DP / 8, of_x = p.T * chunks, all = of_x + w_rows * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const bool is_x = i < of_x;
    const int64_t at = is_x ? i : i - of_x, row = quotient(at, chunks), c = (at - row * chunks) * 8, left = p.D - c;
    bool on = true;
    if (is_x) {
      const int64_t target = p.targets[row];
      on = target >= 0 && target < p.V;
      if (c == 0) {
        XentRow r{0.f, 0.f, 0.f, -1};
        if (on) {
          r.target = (int32_t)target;
          r.lse = p.dloss ? p.lse[row] : 0.f;
          r.dloss = p.dloss ? p.dloss[row] : 0.f;
          r.both = r.dloss + (p.dlse ? p.dlse[row] : 0.f);
        }
        p.rows[row] = r;
        p.inverse[row] = on ? (int32_t)row : -1;
        if (row == 0) *p.count = (int32_t)p.T;
      }
    }
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; e += VEC) {
      Chunk<IO> r;
      r.zero();
      if (on && left > e) r.load(is_x ? p.x : p.w, row * p.D + c + e, left - e);
      r.get(x + e);
    }
    uint16_t* const to = static_cast<uint16_t*>(is_x ? p.xp : p.wp) + row * p.DP + c;
    store_parts(to, (is_x ? p.T : p.piece) * p.DP, parts_of<P>(x));
  }
}

// ---- what the targets' g lost, for dweight ----
// g is held in bf16, and its entry of the target may be off by half a step the same way for all tokens of a word;
// a rare word's gradient is that of its few targets.  So what these entries lost is made up for: a word's sum of
// rest x over its tokens, in fp32 and in the order of the batch, is added to dweight's product before that is
// rounded.  The tokens are put in the order of their targets; a word's places are summed in aligned runs, which the
// product's end adds up, so that a frequent word is not one long sum.
// 7780 of 8192 tokens, 65536 words, D = 2048: 1.3% of the backward (5048 and 5115 us), of which the order of the
// targets takes 28 and the sums 46.  As a second product with the targets' rests, in the registers of the
// first, it took 4%, and 1.7 times the time of the whole where few words have all tokens (16000 tokens of 300, D = 700:
// 283 us, this way 206, without it 167).

// A wavefront takes the sums that start among kLostPlaces places, for the words v0 ... v1 and 64 times eight columns.
// It reads 64 places at once, one of them a lane's; most sums end among them.
constexpr int kLostPlaces = 4;
struct LostShare {
  uint32_t v0, v1;
  unsigned groups;  // workgroups over the places, and as many again for every 512 columns
  unsigned all;     // workgroups; 0: nothing of this
};
__device__ __forceinline__ void sum_lost(const XentArgs& p, const LostShare& share) {
  const unsigned slice = blockIdx.x / share.groups;
  const int lane = threadIdx.x & 63, T = (int)p.T, i0 = uniform((int)((blockIdx.x - slice * share.groups) * 4 + threadIdx.x / 64)) * kLostPlaces;
  if (i0 >= T) return;
  const int64_t c = ((int64_t)slice * 64 + lane) * 8;
  const uint16_t* const xp = static_cast<const uint16_t*>(p.xp) + (c < p.DQ ? c : 0);
  struct Places {
    uint32_t key;
    int row;
    float lost;
  };
  const auto in = [&](uint32_t v) { return v >= share.v0 && v < share.v1; };
  const auto read = [&](int i) {
    const bool there = i + lane < T;
    Places w{there ? p.key[i + lane] : ~0u, there ? (int)p.pos[i + lane] : 0, 0.f};
    if (in(w.key)) w.lost = p.rest[w.row];
    return w;
  };
  const uint32_t before = i0 > 0 ? p.key[i0 - 1] : ~0u;
  const Places here = read(i0);
  if ((__ballot(in(here.key)) & ((1u << kLostPlaces) - 1)) == 0) return;
  float x[8];
  // its places u ... n, N of them with their loads in flight together
  const auto some = [&](auto N, const Places& w, int u) {
    constexpr int kN = decltype(N)::value;
    Chunk<bf16_storage> r[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) r[k].load(xp, (int64_t)__builtin_amdgcn_readlane(w.row, u + k) * p.DP, 8);
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const float f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w.lost), u + k));
      float y[8];
      r[k].get(y);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(f, y[e], x[e]);
    }
  };
  const auto add = [&](const Places& w, int u, int n) {
    for (; u + 16 <= n; u += 16) some(std::integral_constant<int, 16>{}, w, u);
    for (; u + 4 <= n; u += 4) some(std::integral_constant<int, 4>{}, w, u);
    for (; u < n; ++u) some(std::integral_constant<int, 1>{}, w, u);
  };
  for (int s = 0; s < kLostPlaces; ++s) {
    const int i = i0 + s;
    const uint32_t v = (uint32_t)__builtin_amdgcn_readlane((int)here.key, s), behind = (uint32_t)__builtin_amdgcn_readlane((int)here.key, s + 1);
    const bool first = (s == 0 ? before : (uint32_t)__builtin_amdgcn_readlane((int)here.key, s - 1)) != v;
    if (!in(v)) continue;  // nor is it behind the last place
    if (slice == 0 && lane == 0) {
      if (first) {
        p.words[v].first = i;
        p.marks[v / 16] = 1;
      }
      if (behind != v) p.words[v].end = i + 1;
    }
    if (!first && (i & ((1 << p.log_run) - 1)) != 0) continue;
    const int run_end = ((i >> p.log_run) + 1) << p.log_run;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    // the word's places stand side by side
    int n = s + __popcll(__ballot(here.key == v && lane >= s && i0 + lane < run_end));
    add(here, s, n);
    for (int j = i0 + 64; n == 64 && j < run_end; j += 64) {
      const Places w = read(j);
      n = __popcll(__ballot(w.key == v && j + lane < run_end));
      add(w, 0, n);
    }
    float* const to = p.lost + i * p.DQ + c;
#pragma unroll
    for (int e = 0; e < 8; e += 4)
      if (c + e < p.DQ) *reinterpret_cast<f32x4*>(to + e) = f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]};
  }
}

// ---- the product kernel ----

enum class Fetch { kRows, kCols };
enum class Ends { kStats, kGrad, kDx, kDw };

struct ProductArgs {
  const uint16_t *a, *b;
  int64_t lda, ldb;        // elements between rows
  int64_t plane_a, plane_b;
  int32_t M, N, K;         // valid sizes
  const int32_t* count_n;  // or null: fewer n
  const int32_t* count_k;  // or null: fewer k
  // ends
  const XentRow* rows;
  float scale;
  int32_t v0;              // first vocabulary row of the piece
  int32_t tile0;           // first tile of the vocabulary in stat
  int64_t T;
  float* stat;
  float* at_target;
  uint16_t* g;
  int64_t ldg, plane_g;
  float* dx_sum;
  int64_t ld_dx, plane_dx;
  int32_t first;           // of the pieces
  int32_t splits;          // of k, over gridDim.z
  float* rest;             // what the target's g lost to bf16
  void* dw;
  int64_t ld_dw;
  const XentPlaces* words;  // bf16: what is to be added to dweight
  const uint8_t* marks;     // words and marks of the piece
  const float* lost;
  int64_t ld_lost;
  int32_t log_run;
};

// A step's tile of an operand, of one plane: R rows of KS k (64 or 32: 128 or 64 bytes), or KS k rows of R
// elements.  16-byte units are swizzled so that the reads below spread over all banks: unit u of row r lies
// at u ^ swz_row(r); transposed, the pair of units u of row k at u ^ swz<R>(k).
template <int KS>
__device__ __forceinline__ int swz_row(int r) {
  if constexpr (KS == 64) return r & 7;
  return ((((r >> 2) ^ (r >> 3)) & 1) << 1) | ((r >> 3) & 1);
}
template <int R>
__device__ __forceinline__ int swz(int k) {
  if constexpr (R >= 128) return (k & 3) | ((k >> 1) & 4);
  return ((k >> 1) & 1) | ((k >> 2) & 2);  // rows of 128 bytes: four pairs of units
}

// Its loads by a wavefront.
template <Fetch F, int R, int NW, int KS>
struct Loader {
  static constexpr int kLoads = R * KS / 512 / NW;  // of 1024 bytes each
  uint32_t off[kLoads];
  int c8;

  // first: the tile's first row (kRows) or column (kCols), n: rows or columns there are
  __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int32_t first, int32_t n) {
    if constexpr (F == Fetch::kRows) {
      constexpr int per = KS / 8, rows = 64 / per;  // lanes of a row, rows of a load
      c8 = ((lane % per) ^ swz_row<KS>(lane / per)) * 8;
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        off[i] = (uint32_t)(((wave * kLoads + i) * rows + lane / per) * ld + c8) * 2;
    } else {
      constexpr int per = R / 8, rows = 64 / per;
      c8 = 0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int k = (wave * kLoads + i) * rows + lane / per, s = lane % per;
        const int col = (((s >> 1) ^ swz<R>(k)) * 2 + (s & 1)) * 8;
        off[i] = first + col < n ? (uint32_t)(k * ld + col) * 2 : kOutside;
      }
    }
  }
  // What a step's loads need.  base: the operand's plane; rows (kRows) or columns (kCols) from `first`
  // on, k from k0 on, K in all; nothing is loaded where there is no step.
  struct Step {
    u32x4 rsrc;
    uint32_t outside;  // of this lane's k
  };
  __device__ __forceinline__ Step step(const uint16_t* base, int64_t ld, int32_t first, int32_t n, int32_t k0, int32_t K,
                                       bool there) const {
    const int32_t left = (F == Fetch::kRows ? n - first : K - k0), most = F == Fetch::kRows ? R : KS;
    const int32_t rows = left < most ? left : most;
    const uint16_t* at = F == Fetch::kRows ? base + (int64_t)first * ld + k0 : base + (int64_t)k0 * ld + first;
    // the last row ends with the operand's own last element that a load may take
    const int64_t bytes = rows <= 0 || !there ? 0 : ((int64_t)rows * ld - (F == Fetch::kRows ? k0 : first)) * 2;
    return Step{rsrc_words((const void*)uniform((int64_t)(uintptr_t)at), (uint32_t)uniform((int)bytes)),
                F == Fetch::kRows && k0 + c8 >= K ? kOutside : 0u};
  }
  __device__ __forceinline__ void load(const Step& s, int i, int wave, lds_parts to) const {
    load_lds(s.rsrc, (MSM_LDS void*)(to + (wave * kLoads + i) * 512), off[i] | s.outside);
  }
};

// A wavefront's factors of 16 rows each, for the 32 k number kk of a step.
template <Fetch F, int R, int KS>
struct Reader {
  int lane, first;  // first: the wavefront's first row in the tile
  __device__ __forceinline__ bf16x8 read(lds_cparts tile, int i, int kk) const {
    if constexpr (F == Fetch::kRows) {
      const int row = first + i * 16 + (lane & 15);
      return *(const MSM_LDS bf16x8*)(tile + row * KS + (((lane >> 4) + 4 * kk) ^ swz_row<KS>(lane & 15)) * 8);
    } else {
      const int m = lane & 15, k = 32 * kk + 8 * (lane >> 4) + (m >> 2);
      const lds_cparts p = tile + k * R + (((first / 16 + i) ^ swz<R>(k)) * 16) + 4 * (m & 3);
      return read_tr(p, p + 4 * R);
    }
  }
};

// Waits until all but the last N loads of each wavefront have landed.
template <int N>
__device__ __forceinline__ void sync_but() {
  static_assert(N < 64, "vmcnt has 6 bits");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
  __syncthreads();
  __builtin_amdgcn_sched_barrier(0);
}

// Where a workgroup's tile is.  Workgroups go round the 8 XCDs one by one, so number i of an XCD is i * 8
// + XCD; an XCD takes blocks of 8 x 4 tiles, whose operands its L2 shares, and the XCDs stand rm x 8 / rm
// side by side, moved on by one from round to round of n, so that a last block of m is not always the same
// XCDs'.  (All m of one n after another, as the grid counts, the forward reads the whole of W for every 256
// tokens, 8.6 GB for 8192 of 65536, D = 2048: 2.09 ms there, 1.93 in blocks.)  Few tiles would leave XCDs
// without a block: there an XCD takes whole rows or columns of tiles, of the side that has more, where these
// go round the XCDs evenly enough (the logits of an fp32
// backward at 1999 tokens of 10007, D = 513: 94 and 91 us).
struct Place {
  int m, n;
};
__host__ __device__ inline int xcds_m(int tm, int tn, bool wide) {
  if (tm * (int64_t)tn < (wide ? 256 : 2048)) return 0;
  return tm <= 8 ? 1 : (tn <= 4 ? 8 : (tn <= 8 ? 4 : 2));
}
__device__ __forceinline__ Place place_of(int tm, int tn, bool wide) {
  const int rm = xcds_m(tm, tn, wide), at = blockIdx.y * gridDim.x + blockIdx.x;
  if (rm == 0) {
    const bool by_m = tm >= tn;
    const int large = by_m ? tm : tn, small = by_m ? tn : tm;
    if ((large + 7) / 8 * 64 > large * 9) return Place{at % tm, at / tm};
    const int i = at / 8, l = i / small * 8 + at % 8, r = i % small;
    return by_m ? Place{l, r} : Place{r, l};
  }
  const int rounds_m = (tm + 8 * rm - 1) / (8 * rm), round = blockIdx.y, round_n = round / rounds_m;
  const int xcd = (blockIdx.x + round_n) % 8, i = blockIdx.x / 8;
  return Place{((round % rounds_m) * rm + xcd % rm) * 8 + i % 8, (round_n * (8 / rm) + xcd / rm) * 4 + i / 8};
}

// WM x WN wavefronts of MT x NT tiles of 16 x 16; S stages of a step each in LDS.
template <typename IO, int WM, int WN, int MT, int NT, int S, Fetch FA, Fetch FB, Ends END>
__global__ __launch_bounds__(64 * WM * WN) void product_kernel(const ProductArgs p) {
  constexpr int BM = WM * MT * 16, BN = WN * NT * 16, NW = WM * WN, P = io<IO>::es == 2 ? 1 : 3;
  constexpr int KS = P == 1 ? 64 : 32, kA = BM * KS, kB = BN * KS;
  using LA = Loader<FA, BM, NW, KS>;
  using LB = Loader<FB, BN, NW, KS>;
  constexpr int kLoads = LA::kLoads + LB::kLoads;  // of a plane
  __shared__ __attribute__((aligned(16))) uint16_t lds[S * P * (kA + kB)];
  const int N = p.count_n ? uniform(*p.count_n) : p.N, K = p.count_k ? uniform(*p.count_k) : p.K;
  if (N <= 0) return;  // no row takes part: there are no tiles to divide among the XCDs
  const Place at = place_of((p.M + BM - 1) / BM, (N + BN - 1) / BN, BM == 256);
  const int32_t m0 = at.m * BM, n0 = at.n * BN;
  if (m0 >= p.M || n0 >= N) return;  // fewer rows than the grid was made for among these
  const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6)), wm = wave % WM, wn = wave / WM;
  const lds_parts tiles = (lds_parts)lds;
  // one of the wavefront's columns has a sum to be added: asked here, with the count of k, so that the end need not wait
  bool marked = false;
  if constexpr (END == Ends::kDw && P == 1) {
    const int first = n0 / 16 + wn * NT;
    marked = (reinterpret_cast<const uint32_t*>(p.marks)[first / 4] >> (first % 4 * 8) & (NT == 4 ? ~0u : (1u << (8 * NT % 32)) - 1)) != 0;
  }
  LA la;
  LB lb;
  la.init(wave, lane, p.lda, m0, p.M);
  lb.init(wave, lane, p.ldb, n0, N);
  const Reader<FA, BM, KS> ra{lane, wm * MT * 16};
  const Reader<FB, BN, KS> rb{lane, wn * NT * 16};
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = zero4();
  int k_first = 0, k_end = (K + KS - 1) / KS;
  if constexpr (END == Ends::kDx) {
    const int all = k_end, z = blockIdx.z;
    k_first = (int)((int64_t)all * z / p.splits);
    k_end = (int)((int64_t)all * (z + 1) / p.splits);
  }
  const int steps = k_end - k_first;
  typename LA::Step sa[P];
  typename LB::Step sb[P];
  int k = k_first, at_send = 0;  // the step to be loaded next, and its stage
  lds_parts to = tiles;
  const auto next = [&] {
#pragma unroll
    for (int q = 0; q < P; ++q) {
      sa[q] = la.step(p.a + q * p.plane_a, p.lda, m0, p.M, k * KS, K, k < k_end);
      sb[q] = lb.step(p.b + q * p.plane_b, p.ldb, n0, N, k * KS, K, k < k_end);
    }
    to = tiles + at_send * P * (kA + kB);
    at_send = at_send + 1 == S ? 0 : at_send + 1;
    ++k;
  };
  const auto load = [&](int i) {
    const int q = i / kLoads, j = i % kLoads;
    const lds_parts plane = to + q * (kA + kB);
    if (j < LA::kLoads)
      la.load(sa[q], j, wave, plane);
    else
      lb.load(sb[q], j - LA::kLoads, wave, plane + kA);
  };
  if (steps > 0) {
#pragma unroll
    for (int s = 0; s < (P == 1 ? S - 1 : S); ++s) {
      next();
#pragma unroll
      for (int i = 0; i < P * kLoads; ++i) load(i);
    }
  }
  // Loads go out one by one between the products: all of them right behind the barrier hold the wavefronts
  // up for as long as the CU takes to accept them, 64 KB half a step (bf16 forward at 8192 tokens of 65536,
  // D = 2048: 1833 us, one by one 1710).
  if constexpr (P == 1) {
    // The loads of S - 1 steps ahead; factors are read one tile of rows ahead; a wavefront that has its factors
    // goes before one that is still loading (backward at 8192 tokens of 65536, D = 2048: 5301 us, without the
    // priorities, and 5167).
    static_assert(kLoads <= 2 * MT, "a load between the products of each tile of rows");
    int stage = 0;
    for (int s = 0; s < steps; ++s) {
      sync_but<(S - 2) * kLoads>();
      next();
      const lds_cparts ta = tiles + stage * (kA + kB), tb = ta + kA;
      stage = stage + 1 == S ? 0 : stage + 1;
      bf16x8 b[2][NT], a[2];
#pragma unroll
      for (int j = 0; j < NT; ++j) b[0][j] = rb.read(tb, j, 0);
      a[0] = ra.read(ta, 0, 0);
#pragma unroll
      for (int it = 0; it < 2 * MT; ++it) {
        const int kk = it / MT, i = it % MT;
        if (it + 1 < 2 * MT) a[(it + 1) & 1] = ra.read(ta, (it + 1) % MT, (it + 1) / MT);
        if (kk == 0 && i >= MT - NT) b[1][i - (MT - NT)] = rb.read(tb, i - (MT - NT), 1);
        if (it < kLoads) load(it);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[it & 1], b[kk][j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  } else {
    // Three planes a step, each loaded once for the six products of parts (three loads of an operand where
    // six products of one plane each take six).  A step's factors are read during the products of the step
    // before, into the other set of registers: at the barrier before step s those of s are in registers,
    // s + 1 has landed, s + 2 may be on its way, and s + 3 goes where s was.
    static_assert(S == 3, "the stages in use and on their way");
    struct Factors {
      bf16x8 a[3][MT], b[3][NT];
    } f0, f1;
    int at_read = 0;
    constexpr int kReads = 3 * (MT + NT);
    const auto read = [&](Factors& f, int i) {
      const lds_cparts st = tiles + at_read * P * (kA + kB) + i / (MT + NT) * (kA + kB);
      const int j = i % (MT + NT);
      if (j < MT)
        f.a[i / (MT + NT)][j] = ra.read(st, j, 0);
      else
        f.b[i / (MT + NT)][j - MT] = rb.read(st + kA, j - MT, 0);
    };
    // The product of the first parts has a sum of its own: each term that is added to a sum rounds it, and
    // the five small products would round the large sum five times as often for nothing (gradients at 192
    // tokens of 610, D = 1776: 2.5e-6 off in one sum, 1.0e-6 in two; plain fp32 products 9.5e-7).
    constexpr int pairs[6][2] = {{2, 0}, {1, 1}, {0, 2}, {1, 0}, {0, 1}, {0, 0}};
    f32x4 low[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) low[i][j] = zero4();
    const auto step = [&](const Factors& now, Factors& then) {
      sync_but<P * kLoads>();
      next();
      at_read = at_read + 1 == S ? 0 : at_read + 1;
#pragma unroll
      for (int q = 0; q < 6; ++q) {
#pragma unroll
        for (int i = q * kReads / 6; i < (q + 1) * kReads / 6; ++i) read(then, i);
#pragma unroll
        for (int i = q * P * kLoads / 6; i < (q + 1) * P * kLoads / 6; ++i) load(i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            f32x4& to = q == 5 ? acc[i][j] : low[i][j];
            to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now.a[pairs[q][0]][i], now.b[pairs[q][1]][j], to, 0, 0, 0);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    if (steps > 0) {
      sync_but<(S - 1) * P * kLoads>();
#pragma unroll
      for (int i = 0; i < kReads; ++i) read(f0, i);
    }
    int s = 0;
    for (; s + 1 < steps; s += 2) {
      step(f0, f1);
      step(f1, f0);
    }
    if (s < steps) step(f0, f1);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] += low[i][j];
  }
  // the last step's loads, of nothing, still write zeros: not into LDS that is another workgroup's by then
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  // accumulator r of a lane: m = 4 (lane / 16) + r, n = lane % 16 of its tile
  const int ml = m0 + wm * MT * 16 + 4 * (lane >> 4);
  // the tile's rows of C end inside it, or one of the wavefront's columns has its target there: seldom, so
  // the ordinary way asks nothing of a value
  const bool ends = m0 + BM > p.M;
  if constexpr (END == Ends::kStats) {
    const float to2 = p.scale * kLog2e;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = n0 + wn * NT * 16 + j * 16 + (lane & 15);
      const int target = n < N ? p.rows[n].target - p.v0 - m0 : -1;
      if (__any(target >= 0 && target < BM)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (ml - m0 + i * 16 + r == target) p.at_target[n] = acc[i][j][r] * to2;
      }
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] *= to2;
      if (ends) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = ml + i * 16 + r < p.M ? acc[i][j][r] : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, acc[i][j][r]);
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      // nothing but minus infinity: a sum of 0; plus infinity among them: a sum of infinity
      const float from = fabsf(top) == INFINITY ? 0.f : top;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum += exp2_fast(acc[i][j][r] - from);
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      if (lane < 16 && n < N) {
        float* to = p.stat + (((int64_t)p.tile0 + at.m * WM + wm) * p.T + n) * 2;
        to[0] = top;  // in units of log 2
        to[1] = sum;
      }
    }
  } else if constexpr (END == Ends::kGrad) {
    const float to2 = p.scale * kLog2e;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = n0 + wn * NT * 16 + j * 16 + (lane & 15);
      XentRow row{0.f, 0.f, 0.f, -1};
      if (n < N) row = p.rows[n];
      const int target = row.target - p.v0 - m0;
      const float both = row.both * p.scale, lse2 = row.lse * kLog2e;
      // l - lse is rounded where it is small, not where its two terms are; in front of a g in bf16 one
      // operation less is worth more
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][r] = both * exp2_fast(P == 1 ? fmaf(acc[i][j][r], to2, -lse2) : fmaf(acc[i][j][r], p.scale, -row.lse) * kLog2e);
      if (__any(target >= 0 && target < BM)) {
        const float minus = row.dloss * p.scale;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (ml - m0 + i * 16 + r == target) {
              acc[i][j][r] -= minus;
              if constexpr (P == 1) p.rest[n] = acc[i][j][r] - (float)(__bf16)acc[i][j][r];
            }
      }
      if (__any(row.target < 0)) {  // left out but in its place: its zeros times an infinite weight are none
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = row.target < 0 ? 0.f : acc[i][j][r];
      }
      if (ends) {  // the products' k behind the piece
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = ml + i * 16 + r < p.M ? acc[i][j][r] : 0.f;
      }
      if (n >= N) continue;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint16_t* to = p.g + n * p.ldg + ml + i * 16;
        if constexpr (P == 1) {
          typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<bf16x4*>(to) = bf16x4{(__bf16)acc[i][j][0], (__bf16)acc[i][j][1], (__bf16)acc[i][j][2], (__bf16)acc[i][j][3]};
        } else {
          uint32_t lo[3], hi[3];
          cut3(acc[i][j][0], acc[i][j][1], lo);
          cut3(acc[i][j][2], acc[i][j][3], hi);
#pragma unroll
          for (int q = 0; q < 3; ++q) *reinterpret_cast<uint2*>(to + q * p.plane_g) = uint2{lo[q], hi[q]};
        }
      }
    }
  } else if constexpr (END == Ends::kDx) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = n0 + wn * NT * 16 + j * 16 + (lane & 15);
      if (n >= N) continue;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = ml + i * 16;
        if (m >= p.ld_dx) continue;
        f32x4* to = reinterpret_cast<f32x4*>(p.dx_sum + blockIdx.z * p.plane_dx + n * p.ld_dx + m);
        *to = p.first ? acc[i][j] : *to + acc[i][j];
      }
    }
  } else {
    if constexpr (P == 1) {
      // The products' own registers end here, behind the wait states that a matrix instruction's result needs: with sums
      // added to them the compiler moves them about inside the products' loop (64 tokens of 7178, D = 6656: 48 us, and 46).
      asm volatile("s_nop 15\n\ts_nop 15" : "+v"(acc[0][0]));
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) asm volatile("" : "+v"(acc[i][j]));
      // Before the first store, as a load's wait is also for the stores before it, and with several words' loads in flight.
      if (marked) {
        constexpr int kAtOnce = BM == 256 ? 2 : NT;  // of NT, what the registers hold
        XentPlaces places[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int n = n0 + wn * NT * 16 + j * 16 + (lane & 15);
          places[j] = n < N ? p.words[n] : XentPlaces{0, 0};
        }
        // (columns behind a row's end are the next row's, or what follows the last row, and are not stored)
        const float* const lost = p.lost + ml;
#pragma unroll
        for (int j0 = 0; j0 < NT; j0 += kAtOnce) {
          f32x4 x[kAtOnce][MT];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
            for (int i = 0; i < MT; ++i) x[j][i] = zero4();
            if (places[j0 + j].end > 0)
#pragma unroll
              for (int i = 0; i < MT; ++i) x[j][i] = *reinterpret_cast<const f32x4*>(lost + places[j0 + j].first * p.ld_lost + i * 16);
          }
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i][j0 + j] += x[j][i];
            for (int at = ((places[j0 + j].first >> p.log_run) + 1) << p.log_run; at < places[j0 + j].end; at += 1 << p.log_run)  // further runs
#pragma unroll
              for (int i = 0; i < MT; ++i) acc[i][j0 + j] += *reinterpret_cast<const f32x4*>(lost + at * p.ld_lost + i * 16);
          }
        }
      }
    }
    const bool whole = p.ld_dw % 4 == 0 && ((uintptr_t)p.dw & 15) == 0;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = n0 + wn * NT * 16 + j * 16 + (lane & 15);
      if (n >= N) continue;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = ml + i * 16;
        const int64_t to = ((int64_t)p.v0 + n) * p.ld_dw + m;
        const f32x4 c = acc[i][j];
        if (whole && m < p.M) {
          if constexpr (P == 1) {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<bf16x4*>(static_cast<uint16_t*>(p.dw) + to) = bf16x4{(__bf16)c[0], (__bf16)c[1], (__bf16)c[2], (__bf16)c[3]};
          } else {
            *reinterpret_cast<f32x4*>(static_cast<float*>(p.dw) + to) = c;
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (m + r < p.M) io<IO>::store(p.dw, to + r, c[r]);
        }
      }
    }
  }
}

// ---- few rows ----
// Log-probabilities of up to 32 tokens: the weights are read once, from memory into registers in the
// matrix cores' layout (lane l: row l % 16, eight k from 8 (l / 16) on).  The tokens are brought into that
// order beforehand, 1 KB for 32 k of 16 tokens: read as they are, 16 rows a power of two apart at the same k,
// they come from one channel of L2 (16 tokens of 65536, D = 4096, bf16: 145 us).  Bound by HBM.  A workgroup
// takes 16 vocabulary rows at a time and its wavefronts a part of k each.
constexpr int kFewWaves = 16;  // of a workgroup
constexpr int kFewHeld = 8;    // pieces of 32 k that a wavefront holds
// Wavefronts of a tile: as few as hold all of its k, so that short rows do not leave wavefronts idle (28
// tokens of 96399, D = 141, bf16: 50 us with all 16 on a tile, 32 with one).
__host__ __device__ constexpr int few_waves(int pieces) {
  int n = 1;
  while (n < kFewWaves && pieces > n * kFewHeld) n *= 2;
  return n;
}

// Joins the largest logit (in units of log 2) and the sum of exponentials of another set of columns.
__device__ __forceinline__ void join_sums(float& top, float& sum, float top2, float sum2) {
  const float m = fmaxf(top, top2);
  // minus infinity: a sum of 0; plus infinity: of infinity (a finite logit's sum is 1 at least); NaN stays
  const float from = fabsf(m) == INFINITY ? 0.f : m;
  sum = sum * exp2_fast(top - from) + sum2 * exp2_fast(top2 - from);
  top = m;
}

// Eight values, in the parts that are multiplied; the first n belong to the row, the others are zero.
template <typename IO>
struct Eight {
  static constexpr int P = io<IO>::es == 2 ? 1 : 3;
  Chunk<IO> raw[8 / Chunk<IO>::VEC];
  __device__ __forceinline__ void load(const void* p, int64_t at, int64_t n) {
#pragma unroll
    for (int i = 0; i < 8 / Chunk<IO>::VEC; ++i) {
      const int64_t left = n - i * Chunk<IO>::VEC;
      raw[i].zero();
      if (left > 0) raw[i].load(p, at + i * Chunk<IO>::VEC, left);
    }
  }
  __device__ __forceinline__ Part<P> parts() const {
    if constexpr (P == 1) {
      Part<1> r;
      r.p[0] = __builtin_bit_cast(bf16x8, raw[0].raw);
      return r;
    } else {
      float x[8];
      raw[0].get(x);
      raw[1].get(x + 4);
      return parts_of<3>(x);
    }
  }
};

// xp: [part][32 k][16 tokens] of 64 lanes' eight values; zeros behind the rows' ends and the last token.
template <typename IO>
__global__ __launch_bounds__(256) void xent_few_pack_kernel(const XentArgs p, int pieces, int groups) {
  const int i = blockIdx.x * 256 + threadIdx.x, lane = i & 63, j = (i >> 6) % groups, c = (i >> 6) / groups;
  if (c >= pieces) return;
  const int64_t t = j * 16 + (lane & 15), k = c * 32 + 8 * (lane >> 4);
  Eight<IO> x;
  x.load(p.x, (t < p.T ? t : 0) * p.D + k, t < p.T ? p.D - k : 0);
  store_parts(static_cast<uint16_t*>(p.xp) + (int64_t)i * 8, pieces * groups * 512, x.parts());
}

// A barrier for what passes through LDS alone: loads from memory stay in flight over it.
__device__ __forceinline__ void sync_lds_only() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// HOLD: a wavefront's pieces of k, at most kFewHeld, have their tokens in registers throughout (x is p.x),
// and a tile's weights are loaded during the tile before; else the tokens are read again for every tile, in
// the matrix cores' order (x is p.xp).  16 tokens of 65536, D = 4096, bf16: 93 and 116 us.
// (fp32 tokens in three parts do not fit the registers: 16 of 65536, D = 4096, 264 us, 4.1 TB/s; 17 to 32 bf16
// tokens spill 28 to 40 bytes a thread: 20 of 65536 118 us.)
template <typename IO, int NT, bool HOLD, bool ALL>
__global__ __launch_bounds__(64 * kFewWaves) void xent_few_kernel(const XentArgs p, int tiles) {
  constexpr int kAhead = HOLD ? kFewHeld : kFewHeld / (NT * (io<IO>::es / 2));  // what the registers hold
  constexpr int P = Eight<IO>::P;
  __shared__ f32x4 sums[2][kFewWaves][NT][64];
  const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
  const int k8 = 8 * (lane >> 4);
  // `kw` wavefronts share a tile's k, the others have tiles of their own; this wavefront's pieces of 32 k
  const int pieces = (int)((p.D + 31) / 32), whole = (int)(p.D / 32), kw = ALL ? kFewWaves : few_waves(pieces), side = kFewWaves / kw;
  const int each = (pieces + kw - 1) / kw, c0 = wave % kw * each, c1 = c0 + each < pieces ? c0 + each : pieces, own = wave / kw;
  const bf16x8* const xs = static_cast<const bf16x8*>(p.xp) + lane;
  // the threads join the parts, each one value of some tiles: token t, row 4 g + r of the tile
  constexpr int kCells = NT * 256, kTurns = 64 * kFewWaves / kCells;
  const int cell = threadIdx.x % kCells, t = cell / 256 * 16 + (cell & 15), g = (cell >> 4) & 3, r = (cell >> 6) & 3;
  const bool joins = t < p.T;
  const int64_t target = joins ? p.targets[t] : -1;
  float top = -INFINITY, sum = 0.f;
  int turn = 0;
  Eight<IO> w[kAhead];
  Part<P> x[kAhead][NT];
  const auto fetch = [&](int c, int tile) {  // kAhead pieces of a tile's rows
    const int64_t row = (int64_t)tile * 16 + (lane & 15), w_at = (row < p.V ? row : p.V - 1) * p.D + k8;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (c + u < c1 && c + u < whole) w[u].load(p.w, w_at + (int64_t)(c + u) * 32, 8);
      else if (c + u < c1) w[u].load(p.w, w_at + (int64_t)(c + u) * 32, p.D - (int64_t)(c + u) * 32 - k8);
      if constexpr (!HOLD)
        if (c + u < c1)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < P; ++q) {
              x[u][j].p[q] = __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0});
              if (j * 16 + (lane & 15) < p.T) x[u][j].p[q] = xs[((q * pieces + c + u) * NT + j) * 64];  // no bytes for no token
            }
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads in flight first: by itself the compiler keeps two or three
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int64_t k = (int64_t)(c0 + u) * 32 + k8, token = j * 16 + (lane & 15);
        Eight<IO> v;
        v.load(p.x, (token < p.T ? token : 0) * p.D + k, c0 + u < c1 && token < p.T ? p.D - k : 0);
        x[u][j] = v.parts();
      }
    if ((int)blockIdx.x * side < tiles) fetch(c0, blockIdx.x * side + own);
  }
  const int stride = gridDim.x * side;
  for (int tile = blockIdx.x * side; tile < tiles; tile += stride, turn ^= 1) {
    f32x4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = zero4();
    for (int c = c0; c < c1; c += kAhead) {
      if constexpr (!HOLD) fetch(c, tile + own);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c + u < c1) {
          const Part<P> a = w[u].parts();
#pragma unroll
          for (int j = 0; j < NT; ++j) mma(acc[j], a, x[u][j]);
        }
    }
    if constexpr (HOLD) {
      __builtin_amdgcn_sched_barrier(0);
      if (tile + stride < tiles) fetch(c0, tile + stride + own);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) sums[turn][wave][j][lane] = acc[j];
    sync_lds_only();  // and what was read two tiles ago may be written
    for (int sub = threadIdx.x / kCells; joins && sub < side; sub += kTurns) {
      float l = 0.f;
      if constexpr (ALL) {
#pragma unroll
        for (int i = 0; i < kFewWaves; ++i) l += sums[turn][i][cell / 256][g * 16 + (cell & 15)][r];
      } else {
        for (int i = 0; i < kw; ++i) l += sums[turn][sub * kw + i][cell / 256][g * 16 + (cell & 15)][r];
      }
      const int64_t v = (int64_t)(tile + sub) * 16 + 4 * g + r;
      if (v < p.V) {
        l *= p.scale * kLog2e;
        if (v == target) p.at_target[t] = l;
        join_sums(top, sum, l, l == l ? 1.f : l);
      }
    }
  }
  __syncthreads();
  // one pair of sums a token from its threads
  constexpr int kThreads = 16 * kTurns;  // of a token
  float* all = reinterpret_cast<float*>(sums);
  if (joins) {
    const int at = t * kThreads + (threadIdx.x / kCells) * 16 + g * 4 + r;
    all[at * 2] = top;
    all[at * 2 + 1] = sum;
  }
  __syncthreads();
  if (threadIdx.x < p.T) {
    top = -INFINITY;
    sum = 0.f;
    for (int i = 0; i < kThreads; ++i) join_sums(top, sum, all[(threadIdx.x * kThreads + i) * 2], all[(threadIdx.x * kThreads + i) * 2 + 1]);
    float* to = p.stat + ((int64_t)blockIdx.x * p.T + threadIdx.x) * 2;
    to[0] = top;
    to[1] = sum;
  }
}

int few_groups(const XentArgs& a) {
  const int side = kFewWaves / few_waves((int)((a.D + 31) / 32)), n = (int)(((a.V + 15) / 16 + side - 1) / side);
  return n < kXentFewGroups ? n : kXentFewGroups;
}

template <typename IO, int NT>
hipError_t few(const XentArgs& a, hipStream_t s) {
  const int pieces = (int)((a.D + 31) / 32), tiles = (int)((a.V + 15) / 16), groups = few_groups(a);
  const bool all = few_waves(pieces) == kFewWaves;
  const dim3 block(64 * kFewWaves);
  if constexpr (io<IO>::es == 2) {
    if (pieces <= kFewWaves * kFewHeld) {
      if (all)
        hipLaunchKernelGGL((xent_few_kernel<IO, NT, true, true>), dim3(groups), block, 0, s, a, tiles);
      else
        hipLaunchKernelGGL((xent_few_kernel<IO, NT, true, false>), dim3(groups), block, 0, s, a, tiles);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((xent_few_pack_kernel<IO>), dim3((pieces * NT + 3) / 4), dim3(256), 0, s, a, pieces, NT);
  if constexpr (io<IO>::es == 4)
    if (!all) {
      hipLaunchKernelGGL((xent_few_kernel<IO, NT, false, false>), dim3(groups), block, 0, s, a, tiles);
      return hipGetLastError();
    }
  static_assert(io<IO>::es == 4 || few_waves(kFewWaves * kFewHeld + 1) == kFewWaves, "bf16 rows that are not held take all wavefronts");
  hipLaunchKernelGGL((xent_few_kernel<IO, NT, false, true>), dim3(groups), block, 0, s, a, tiles);
  return hipGetLastError();
}

// lse and loss of a row from its tiles' largest logits and sums, by W wavefronts of a workgroup of 4: one
// for many rows, four for few (16 rows of 1024 tiles: 9.5 us by one, 4.8 by four).
template <int W>
__global__ __launch_bounds__(256) void xent_join_kernel(const XentArgs p, int64_t tiles) {
  __shared__ float others[2][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = threadIdx.x % (64 * W);
  for (int64_t t = (int64_t)blockIdx.x * (4 / W) + wave / W; t < p.T; t += (int64_t)gridDim.x * (4 / W)) {
    int64_t n = t;
    if (p.inverse)
      n = p.inverse[t];
    else if (p.targets[t] < 0 || p.targets[t] >= p.V)
      n = -1;
    float top = -INFINITY, sum = 0.f;
    if (n >= 0) {
#pragma unroll 4
      for (int64_t i = part; i < tiles; i += 64 * W) {
        const float2 s = *reinterpret_cast<const float2*>(p.stat + (i * p.T + n) * 2);
        join_sums(top, sum, s.x, s.y);
      }
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const float top2 = __shfl_xor(top, d, 64), sum2 = __shfl_xor(sum, d, 64);
        join_sums(top, sum, top2, sum2);
      }
    }
    if constexpr (W > 1) {
      __syncthreads();  // the row before has been read
      if (lane == 0) {
        others[0][wave] = top;
        others[1][wave] = sum;
      }
      __syncthreads();
      for (int i = 1; i < W; ++i)
        if (wave == 0) join_sums(top, sum, others[0][i], others[1][i]);
    }
    if (part == 0) {
      const float lse = n < 0 ? 0.f : (top + log2f(sum)) * kLn2;
      // the target's logit is taken from the largest as both were compared, before lse rounds: 0 for the largest
      p.loss[t] = n < 0 ? 0.f : (top - p.at_target[n] + log2f(sum)) * kLn2;
      if (p.lse) p.lse[t] = lse;
    }
  }
}

// The end of a piece: its words' sums for dweight, by the first workgroups (a launch of their own costs 39 tokens of
// 1391, D = 318, 5 us of 32).  Behind the last piece the others make dx from the sums over all pieces, of every split;
// zero for the rows that are left out.  With bf16 g, what the target's g lost to its rounding is made up for
// here: it is most of a row's g as a rule, and its rounding alone had dx off by 1.65 times the rounding of
// the result (2.8e-3 for 1.7e-3 of its size; 8192 tokens of 65536, D = 2048).
template <typename IO>
__global__ __launch_bounds__(256) void xent_end_kernel(const XentArgs p, const LostShare share) {
  constexpr int VEC = Chunk<IO>::VEC;
  if constexpr (io<IO>::es == 2)
    if (blockIdx.x < share.all) return sum_lost(p, share);
  const int64_t pieces = (p.D + VEC - 1) / VEC, all = p.T * pieces;
  for (int64_t i = (int64_t)(blockIdx.x - share.all) * 256 + threadIdx.x; i < all; i += (int64_t)(gridDim.x - share.all) * 256) {
    const int64_t t = quotient(i, pieces), c = (i - t * pieces) * VEC;
    const int n = p.inverse[t];
    float x[VEC];
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      f32x4 v = zero4();
      if (n >= 0 && c + e < p.DQ) {
        const float* from = p.dx_sum + n * p.DQ + c + e;
        v = *reinterpret_cast<const f32x4*>(from);
#pragma unroll 8
        for (int z = 1; z < p.splits; ++z) v += *reinterpret_cast<const f32x4*>(from + z * (p.T * p.DQ));
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) x[e + r] = v[r];
    }
    if constexpr (io<IO>::es == 2) {
      if (n >= 0) {
        const float rest = p.rest[n];
        float w[VEC];
        Chunk<IO> r;
        r.load(p.w, p.rows[n].target * p.D + c, p.D - c);
        r.get(w);
        if (rest != 0.f)  // nor is a weight multiplied that may be infinite
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[e] = fmaf(rest, w[e], x[e]);
      }
    }
    Chunk<IO> out;
    out.set(x);
    out.store(p.dx, t * p.D + c, p.D - c);
  }
}

constexpr int64_t kMostGroups = (int64_t)1 << 20;
unsigned groups_of(int64_t n) { return (unsigned)(n < 1 ? 1 : (n < kMostGroups ? n : kMostGroups)); }

template <typename IO, Fetch FA, Fetch FB, Ends END>
hipError_t product(const ProductArgs& a, int tile, hipStream_t s) {
  const int b = tile, tm = (a.M + b - 1) / b, tn = (a.N + b - 1) / b, rm = xcds_m(tm, tn, tile == 256);
  const int64_t all = (int64_t)((tm + 7) / 8 * 8) * ((tn + 7) / 8 * 8), rounds = rm == 0 ? 1 : (int64_t)((tm + 8 * rm - 1) / (8 * rm)) * ((tn + 32 / rm - 1) / (32 / rm));
  const dim3 grid(rm == 0 ? (unsigned)all : 256u, (unsigned)rounds, END == Ends::kDx ? (unsigned)a.splits : 1u);
  if constexpr (io<IO>::es == 4) {
    if (tile == 128)
      hipLaunchKernelGGL((product_kernel<IO, 2, 4, 4, 2, 3, FA, FB, END>), grid, dim3(512), 0, s, a);
    else
      hipLaunchKernelGGL((product_kernel<IO, 2, 2, 2, 2, 3, FA, FB, END>), grid, dim3(256), 0, s, a);
  } else {
    if (tile == 256)
      hipLaunchKernelGGL((product_kernel<IO, 2, 4, 8, 4, 2, FA, FB, END>), grid, dim3(512), 0, s, a);
    else if (tile == 128)
      hipLaunchKernelGGL((product_kernel<IO, 2, 2, 4, 4, 2, FA, FB, END>), grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((product_kernel<IO, 2, 2, 2, 2, 5, FA, FB, END>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

template <typename IO>
hipError_t pack(const void* src, const int32_t* map, const int32_t* count, int64_t n, const XentArgs& a, int64_t plane,
                void* dst, hipStream_t s) {
  hipLaunchKernelGGL((xent_pack_kernel<IO>), dim3(groups_of((n * (a.DP / 8) + 255) / 256)), dim3(256), 0, s, src, map, count, n,
                     a.D, a.DP, plane, static_cast<uint16_t*>(dst));
  return hipGetLastError();
}

// The rows that take part, gathered, and the left side's operand of a piece (the first one of few rows is
// packed with them).
template <typename IO>
hipError_t gather(const XentArgs& a, hipStream_t s) {
  if (a.T <= kXentPlaced) {
    const int64_t first = a.w_direct ? 0 : (a.V < a.piece ? a.V : a.piece);
    hipLaunchKernelGGL((xent_gather_kernel<IO>), dim3(groups_of(((a.T + first) * (a.DP / 8) + 255) / 256)), dim3(256), 0, s, a, first);
    return hipGetLastError();
  }
  const unsigned order = a.words && a.T <= kXentRanked ? (unsigned)((a.T + 15) / 16) : 0;
  hipLaunchKernelGGL(xent_rows_kernel, dim3(1 + order), dim3(1024), 0, s, a);
  return pack<IO>(a.x, a.map, a.count, a.T, a, a.T * a.DP, a.xp, s);
}
template <typename IO>
hipError_t weights(const XentArgs& a, int64_t v0, int64_t n, ProductArgs* g, hipStream_t s) {
  const char* at = static_cast<const char*>(a.w) + v0 * a.D * io<IO>::es;
  g->plane_a = 0;
  if (a.w_direct) {
    g->a = reinterpret_cast<const uint16_t*>(at);
    g->lda = a.D;
    return hipSuccess;
  }
  g->a = static_cast<const uint16_t*>(a.wp);
  g->lda = a.DP;
  g->plane_a = a.piece * a.DP;
  if (v0 == 0 && a.T <= kXentPlaced) return hipSuccess;
  return pack<IO>(at, nullptr, nullptr, n, a, a.piece * a.DP, a.wp, s);
}

// lse and loss
hipError_t join(const XentArgs& a, int64_t tiles, hipStream_t s) {
  if (a.T <= 512)
    hipLaunchKernelGGL(xent_join_kernel<4>, dim3(groups_of(a.T)), dim3(256), 0, s, a, tiles);
  else
    hipLaunchKernelGGL(xent_join_kernel<1>, dim3(groups_of((a.T + 3) / 4)), dim3(256), 0, s, a, tiles);
  return hipGetLastError();
}

template <typename IO>
hipError_t fwd(const XentArgs& a, hipStream_t s) {
  if (a.T <= kXentFew) {
    const hipError_t e = a.T <= 16 ? few<IO, 1>(a, s) : few<IO, 2>(a, s);
    return e != hipSuccess ? e : join(a, few_groups(a), s);
  }
  hipError_t e = gather<IO>(a, s);
  const int64_t part = a.tile / 2;  // vocabulary rows of a pair of sums
  int64_t tiles = 0;
  for (int64_t v0 = 0; v0 < a.V && e == hipSuccess; v0 += a.piece) {
    const int64_t n = a.V - v0 < a.piece ? a.V - v0 : a.piece;
    ProductArgs g{};
    e = weights<IO>(a, v0, n, &g, s);
    if (e != hipSuccess) break;
    g.b = static_cast<const uint16_t*>(a.xp);
    g.ldb = a.DP;
    g.plane_b = a.T * a.DP;
    g.M = (int32_t)n;
    g.N = (int32_t)a.T;
    g.K = (int32_t)a.D;
    g.count_n = a.count;
    g.rows = a.rows;
    g.scale = a.scale;
    g.v0 = (int32_t)v0;
    g.tile0 = (int32_t)tiles;
    g.T = a.T;
    g.stat = a.stat;
    g.at_target = a.at_target;
    e = product<IO, Fetch::kRows, Fetch::kRows, Ends::kStats>(g, a.tile, s);
    tiles += (n + 2 * part - 1) / (2 * part) * 2;
  }
  return e != hipSuccess ? e : join(a, tiles, s);
}

template <typename IO>
hipError_t bwd(const XentArgs& a, const EmbedArgs& sort, hipStream_t s) {
  constexpr bool bf16 = io<IO>::es == 2;
  hipError_t e = gather<IO>(a, s);
  if (bf16 && a.words && a.T > kXentRanked && e == hipSuccess) e = launch_embed_sort(sort, a.clear, s);
  for (int64_t v0 = 0; v0 < a.V && e == hipSuccess; v0 += a.piece) {
    const int64_t n = a.V - v0 < a.piece ? a.V - v0 : a.piece;
    ProductArgs g{};
    e = weights<IO>(a, v0, n, &g, s);
    if (e != hipSuccess) break;
    const uint16_t* w = g.a;
    const int64_t ldw = g.lda, plane_w = g.plane_a;
    g.b = static_cast<const uint16_t*>(a.xp);
    g.ldb = a.DP;
    g.plane_b = a.T * a.DP;
    g.M = (int32_t)n;
    g.N = (int32_t)a.T;
    g.K = (int32_t)a.D;
    g.count_n = a.count;
    g.rows = a.rows;
    g.scale = a.scale;
    g.v0 = (int32_t)v0;
    g.g = static_cast<uint16_t*>(a.g);
    g.ldg = a.piece;
    g.plane_g = a.T * a.piece;
    g.rest = a.rest;
    e = product<IO, Fetch::kRows, Fetch::kRows, Ends::kGrad>(g, xent_tile(n, a.T, a.D, a.planes), s);
    if (e != hipSuccess) break;
    ProductArgs x{};
    x.a = w;
    x.lda = ldw;
    x.plane_a = plane_w;
    x.b = static_cast<const uint16_t*>(a.g);
    x.ldb = a.piece;
    x.plane_b = a.T * a.piece;
    x.M = (int32_t)a.D;
    x.N = (int32_t)a.T;
    x.K = (int32_t)n;
    x.count_n = a.count;
    x.dx_sum = a.dx_sum;
    x.ld_dx = a.DQ;
    x.plane_dx = a.T * a.DQ;
    x.splits = a.splits;
    x.first = v0 == 0;
    e = product<IO, Fetch::kCols, Fetch::kRows, Ends::kDx>(x, xent_tile(a.D, a.T, n, a.planes), s);
    if (e != hipSuccess) break;
    const bool last = v0 + n == a.V;
    LostShare share{(uint32_t)v0, (uint32_t)(v0 + n), (unsigned)((a.T + 4 * kLostPlaces - 1) / (4 * kLostPlaces)), 0};
    if (a.words) share.all = share.groups * (unsigned)((a.DQ + 511) / 512);
    const unsigned of_dx = last ? groups_of((a.T * ((a.D * io<IO>::es + 15) / 16) + 255) / 256) : 0;
    if (share.all + of_dx > 0) {
      hipLaunchKernelGGL((xent_end_kernel<IO>), dim3(share.all + of_dx), dim3(256), 0, s, a, share);
      e = hipGetLastError();
    }
    if (e != hipSuccess || !a.dw) continue;
    ProductArgs d{};
    d.a = static_cast<const uint16_t*>(a.xp);
    d.lda = a.DP;
    d.plane_a = a.T * a.DP;
    d.b = static_cast<const uint16_t*>(a.g);
    d.ldb = a.piece;
    d.plane_b = a.T * a.piece;
    d.M = (int32_t)a.D;
    d.N = (int32_t)n;
    d.K = (int32_t)a.T;
    d.count_k = a.count;
    d.v0 = (int32_t)v0;
    d.dw = a.dw;
    d.ld_dw = a.D;
    d.words = a.words + v0;
    d.marks = a.marks + v0 / 16;
    d.lost = a.lost;
    d.ld_lost = a.DQ;
    d.log_run = a.log_run;
    e = product<IO, Fetch::kCols, Fetch::kCols, Ends::kDw>(d, xent_tile(a.D, n, a.T, a.planes), s);
  }
  return e;
}

}  // namespace

hipError_t launch_xent_fwd(const XentArgs& a, int io_bf16, hipStream_t s) {
  return io_bf16 ? fwd<bf16_storage>(a, s) : fwd<float>(a, s);
}
hipError_t launch_xent_bwd(const XentArgs& a, const EmbedArgs& sort, int io_bf16, hipStream_t s) {
  return io_bf16 ? bwd<bf16_storage>(a, sort, s) : bwd<float>(a, sort, s);
}

}  // namespace msm
