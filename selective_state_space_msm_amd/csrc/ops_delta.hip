// Chunked gated delta rule (gfx950): forward and backward.
//
// Per sequence and value head, with a state S (K x V), decay a_t = exp(g_t) and write strength
// beta_t:
//   e_t = v_t - a_t S_{t-1}^T k_t,  S_t = a_t S_{t-1} + beta_t k_t e_t^T,  o_t = scale S_t^T q_t.
// Over a chunk of C tokens with G_i = sum_{j<=i} g_j and D_ij = exp(G_i - G_j) the errors solve
// a unit lower triangular system, and everything else is matrix products:
//   T  = (I + stril(D K K^T) diag(beta))^-1           E  = T (V - e^G (K S0)),  U = beta E
//   O  = scale e^G (Q S0) + P U                       P  = scale tril(D Q K^T)
//   S1 = e^{G_C} S0 + K^T (e^{G_C - G} U)
// The backward, given dO and dS1, walks the chunks in reverse:
//   W  = P^T dO + e^{G_C - G} (K dS1)                 dV = T^T (beta W)
//   Y  = W - stril(D K K^T)^T dV                      dbeta_i = Y_i . E_i
//   dS0 = e^{G_C} dS1 + Q^T (scale e^G dO) - K^T (e^G dV)
//   dQ = scale e^G (dO S0^T) + X K                    X  = scale tril(D dO U^T)
//   dK = e^{G_C - G} (U dS1^T) - e^G (dV S0^T) + X^T Q + (Z + Z^T) K,   Z = -stril(D dV U^T)
// The gradient of g_t gathers every path through the decay of token t: from a write before t (or
// S0) to a read at or after t (or S1),
//   dg_t = sum_{i >= t > j} N_ij + sum_{i >= t} r_i + sum_{j < t} w_j + e^{G_C} <S0, dS1>,
//   N = P o (dO U^T) - stril(D K K^T) o (dV U^T),  r_i = dO_i . (scale e^G Q S0)_i - dV_i . (e^G K S0)_i,
//   w_j = U_j . (e^{G_C - G} K dS1)_j.
// (The scaling symmetry of the recurrence gives the shorter dg_t = sum_{i >= t} (dO_i . O_i - dV_i . V_i)
// + <S1, dS1>, but its terms do not shrink with the decay and cancel: under strong decay it loses
// two digits against this sum.)
//
// The kernels, each built for one I/O type and padded key size (this file is compiled once per
// pair):
//   prep     one workgroup per chunk and head: decays, Gram matrices, the triangular inverse
//   scan     one workgroup per sequence (or segment of one), head and 64 columns of V, chunk after
//            chunk; the state stays in registers
//   segment, join   the states that segments start from, where sequences are cut
//   rev      the walk backwards for the adjoint of the state
//   grad     one workgroup per chunk and key head: dQ, dK and the sums for dbeta and dg
// The products run on the bf16 matrix unit over values cut into parts of 8 bits (ops_delta.hpp):
// one part for a bf16 input and three for an fp32 value, which keeps its 24 bits, also where the
// result is then rounded to bf16: two parts there, 16 bits, took 10% off the forward's time at Bt=4
// L=4096 H=32 and 5% off the packed backward's, but moved about one result in 200 to its
// bf16 neighbour.
// The card's fp32 matrix unit reaches 154 TFLOP/s, its bf16 unit 1240:
// even the six products of three parts by three are faster there.
#include <type_traits>

#include "ops_delta.hpp"

namespace msm {
namespace {

constexpr int KP = MSM_KP;
constexpr int C = delta_chunk(MSM_IO_BF16, KP);
constexpr int NB = KP / 32;       // blocks of 32 state rows
constexpr int CB = C / 32;        // blocks of 32 tokens
constexpr int UK = KP / 8;        // 16-byte units of a row of keys
constexpr int kIn = MSM_IO_BF16 ? 1 : 3;        // parts of an input
constexpr int TP = 3;                           // parts of an fp32 value
constexpr int kRows = C * KP;                   // elements of a plane of keys
using TriM = Tri<C>;
constexpr int kTri = TP * TriM::kPlane;         // elements of a chunk matrix
constexpr int kVec = 5 * C;
constexpr int kDots = 4 * C;
constexpr int kWavesScan = 4;     // wavefronts of a scan workgroup, 16 columns each
#if MSM_IO_BF16
using IO = io<bf16_storage>;
using elem = uint16_t;
#else
using IO = io<float>;
using elem = float;
#endif

__device__ __forceinline__ float exp_of(double x) { return exp2_fast((float)(x * 1.4426950408889634)); }

// ---- prep ----------------------------------------------------------------------------------

// Inverse of the unit lower triangular I + Ms diag(beta) (Ms C x C in LDS, entries below the
// diagonal) into Ti.  Wavefront w inverts diagonal block w of 16 by forward substitution, a column per lane;
// block column j of the inverse then follows downwards, T_ij = -T_ii sum_k M_ik T_kj, its blocks
// staying in wavefront j's registers as right factors.  Substitution in blocks keeps the error
// of a triangular solve; products of powers of M would not.
constexpr int LDM = C + 4;
__device__ __forceinline__ void invert(const MSM_LDS float* Ms, const MSM_LDS float* beta, MSM_LDS float* Ti, int wave, int lane) {
  constexpr int B16 = C / 16;
  const int n = lane & 15, j = lane >> 4;
  if (wave < B16) {
    float x[16], bx[16];
    const MSM_LDS float* M = Ms + (16 * wave) * LDM + 16 * wave;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == n ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < i; ++k) s = fmaf(-M[i * LDM + k], bx[k], s);
      x[i] = s;
      bx[i] = s * beta[16 * wave + i];
    }
    if (j == 0)
#pragma unroll
      for (int i = 0; i < 16; ++i) Ti[(16 * wave + i) * LDM + 16 * wave + n] = x[i];
  }
  __syncthreads();
  if (wave < B16) {
    f32x4 t, bt[B16];  // a block of the inverse, and those above it times beta
#pragma unroll
    for (int r = 0; r < 4; ++r)
      bt[0][r] = Ti[(16 * wave + 4 * j + r) * LDM + 16 * wave + n] * beta[16 * wave + 4 * j + r];
#pragma unroll
    for (int d = 1; d < B16; ++d) {
      const int i = wave + d;
      if (i < B16) {
        f32x4 acc = zero4();
#pragma unroll
        for (int e = 0; e < d; ++e) {
          const f32x4 a = *(const MSM_LDS f32x4*)(Ms + (16 * i + n) * LDM + 16 * (wave + e) + 4 * j);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], bt[e][r], acc, 0, 0, 0);
        }
        const f32x4 a = *(const MSM_LDS f32x4*)(Ti + (16 * i + n) * LDM + 16 * i + 4 * j);
        t = zero4();
#pragma unroll
        for (int r = 0; r < 4; ++r) t = __builtin_amdgcn_mfma_f32_16x16x4f32(-a[r], acc[r], t, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          Ti[(16 * i + 4 * j + r) * LDM + 16 * wave + n] = t[r];
          bt[d][r] = t[r] * beta[16 * i + 4 * j + r];
        }
      }
    }
  }
  __syncthreads();
}

// KS columns from c0 of the chunk's rows of keys or queries, on their way into swizzled LDS planes;
// rows and columns past the chunk's are zero.  With `ws` the planes also go to memory, for kernels
// that then load them into LDS unchanged: fp32 inputs in their parts, and rows that cannot be read 16
// bytes at a time.
template <int THREADS, int KS>
struct RawRows {
  static constexpr int U = KS / 8, N = C * U / THREADS;
  static_assert(C * U % THREADS == 0, "whole passes");
  f32x4 a[N][2];
  static __device__ __forceinline__ int row(int u) { return u / U; }
  static __device__ __forceinline__ int unit(int u) { return (u % U) ^ swizzle<U>(u / U); }
  __device__ __forceinline__ void fetch(__amdgpu_buffer_rsrc_t r, uint32_t stride, int K, bool vec, int c0, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = tid + i * THREADS, c = c0 + unit(u) * 8;
      const uint32_t at = row(u) * stride + c * IO::es;
      if (vec) {
        a[i][0] = bload4(r, c < K ? at : kOutside);
        if (!MSM_IO_BF16) a[i][1] = bload4(r, c + 4 < K ? at + 16 : kOutside);
      } else {
        uint32_t x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const auto v = IO::bload(r, c + e < K ? at + e * IO::es : kOutside, 0);
          x[e] = __builtin_bit_cast(uint32_t, v);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (MSM_IO_BF16) {
            a[i][0][e] = __uint_as_float(x[2 * e] | (x[2 * e + 1] << 16));
          } else {
            a[i][0][e] = __uint_as_float(x[e]);
            a[i][1][e] = __uint_as_float(x[4 + e]);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void put(lds_parts lds, uint16_t* ws, int c0, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = tid + i * THREADS;
      Part<kIn> s;
      if constexpr (kIn == 1)
        s.p[0] = __builtin_bit_cast(bf16x8, a[i][0]);
      else
        s = split<kIn>(a[i][0], a[i][1]);
      store_parts(lds + u * 8, C * KS, s);
      if (ws) store_parts(ws + row(u) * KP + (((c0 / 8) + unit(u)) ^ swizzle<UK>(row(u))) * 8, kRows, s);
    }
  }
};

// The parts of a chunk matrix from LDS rows of LDM floats into its blocks, 16 bytes a plane and
// thread.
__device__ __forceinline__ void write_tri(uint16_t* to, const MSM_LDS float* from, int tid) {
  for (int u = tid; u < C * C / 8; u += 256) {
    const int row = u / (C / 8), c = (u % (C / 8)) * 8;
    if (c / 32 > row / 32) continue;
    const f32x4 a = *(const MSM_LDS f32x4*)(from + row * LDM + c), b = *(const MSM_LDS f32x4*)(from + row * LDM + c + 4);
    store_parts(to + TriM::at(row, c), TriM::kPlane, split<TP>(a, b));
  }
}

// Key columns that prep stages at a time: 64 at least, so that their planes go to memory in whole
// 128-byte lines (32 columns of fp32 keys of 128: 93 us and a slower scan after it, 313 us; 64: 90, 297).
constexpr int prep_columns() {
  int ks = KP;
  while (ks > 32 && 2 * kIn * C * ks * 2 > 50 * 1024) ks /= 2;
  return ks;
}

// Bound by the latency of its steps (load, Gram products, inverse, store), so the LDS is kept to 53 KB
// for three workgroups a CU (fp32 keys of 128: 67 KB for two): wide rows are staged some columns at a
// time, and the inverse and the outgoing matrices take the place of the keys and queries once the
// Gram products are done.  Bt=4 L=4096 H=32 K=128 bf16: 112 us, 312 MB written (the chunk matrices in
// their parts); 170 us with 100 KB, one workgroup a CU.  Bt=4 L=2048 H=16 K=128 fp32, backward: 90 us;
// 120 us with whole rows, 117 KB.
template <bool BWD>
__global__ __launch_bounds__(256) void prep_kernel(const DeltaArgs p) {
  constexpr int KS = prep_columns();
  constexpr int kMat = C * LDM * 4, kKeys = 2 * kIn * C * KS * 2, kMats = 2 * kMat;
  __shared__ __attribute__((aligned(16))) char lds_kq[kKeys > kMats ? kKeys : kMats];
  __shared__ __attribute__((aligned(16))) float lds_m[C * LDM];
  __shared__ double Gd[C];
  __shared__ float bt[C];
  const lds_parts Ks = (lds_parts)lds_kq, Qs = Ks + kIn * C * KS;
  MSM_LDS float* const Ms = (MSM_LDS float*)lds_m;
  MSM_LDS float* const Ti = (MSM_LDS float*)lds_kq;
  MSM_LDS float* const Pl = Ti + C * LDM;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, j = lane >> 4;
  const int64_t slot = blockIdx.x, h = blockIdx.y;
  const ChunkRows ch = chunk_rows<C>(p, slot);
  if (ch.n == 0) return;
  const uint32_t group = (uint32_t)p.H / (uint32_t)p.Hk;
  const int64_t sh = slot * p.H + h, hk = uniform((int)((uint32_t)h / group));
  const uint32_t stride = (uint32_t)(p.Hk * p.K * IO::es);
  uint16_t* ws = p.kq_direct || h != hk * group ? nullptr : static_cast<uint16_t*>(p.kq) + (slot * p.Hk + hk) * 2 * kIn * kRows;
  float gl = 0.f, b = 0.f;
  constexpr int B16 = C / 16, kTiles = B16 * B16 / 4;
  constexpr int kLight = B16 - 1;  // the wavefront with the fewest Gram tiles takes the decays
  if (wave == kLight && lane < ch.n) {
    gl = p.g[(ch.row0 + lane) * p.H + h];
    b = p.beta[(ch.row0 + lane) * p.H + h];
  }
  const auto rk = head_rsrc(p.k, ch.row0, p.Hk, hk, p.K, IO::es, ch.n), rq = head_rsrc(p.q, ch.row0, p.Hk, hk, p.K, IO::es, ch.n);
  RawRows<256, KS> kr, qr;
  kr.fetch(rk, stride, (int)p.K, p.vec_k, 0, tid);
  qr.fetch(rq, stride, (int)p.K, p.vec_k, 0, tid);
  // Gram tiles of the kept blocks; 16 x 16, a wavefront's share of them in its registers
  f32x4 kk[kTiles], qk[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) kk[i] = qk[i] = zero4();
#pragma unroll 1
  for (int c0 = 0; c0 < KP; c0 += KS) {
    if (c0 > 0) __syncthreads();  // the columns before have been read
    kr.put(Ks, ws, c0, tid);
    qr.put(Qs, ws ? ws + kIn * kRows : nullptr, c0, tid);
    if (c0 + KS < KP) {
      kr.fetch(rk, stride, (int)p.K, p.vec_k, c0 + KS, tid);
      qr.fetch(rq, stride, (int)p.K, p.vec_k, c0 + KS, tid);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int t = 4 * i + wave, mt = t / B16, nt = t % B16;
      if (nt <= mt) {
#pragma unroll
        for (int b = 0; b < KS / 32; ++b) {
          const auto B = load_row<KS / 8, kIn>(Ks, 16 * nt + n, 32 * b + 8 * j, C * KS);
          mma(kk[i], load_row<KS / 8, kIn>(Ks, 16 * mt + n, 32 * b + 8 * j, C * KS), B);
          mma(qk[i], load_row<KS / 8, kIn>(Qs, 16 * mt + n, 32 * b + 8 * j, C * KS), B);
        }
      }
    }
  }
  if (wave == kLight) {
    // running sum of the log decay in fp64: its differences keep fp32 accuracy.  exp(-1e4) is 0
    // already; below it the sum would lose the decays that follow (a decay of minus infinity, or
    // of the lowest float, resets the state)
    double G = gl < -1e4f ? -1e4 : (double)gl;
#pragma unroll
    for (int m = 1; m < C; m *= 2) {
      const double up = __shfl_up(G, m, 64);
      if (lane >= m) G += up;
    }
    const double last = __shfl(G, C - 1, 64);
    if (lane < C) {
      Gd[lane] = G;
      bt[lane] = b;
      float* vec = p.vec + sh * kVec;
      vec[lane] = exp_of(G);
      vec[C + lane] = exp_of(last - G);
      vec[2 * C + lane] = b;
      reinterpret_cast<double*>(vec + 3 * C)[lane] = G;
    }
  }
  __syncthreads();  // keys and queries have been read
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const int t = 4 * i + wave, mt = t / B16, nt = t % B16;
    if (nt / 2 > mt / 2) continue;  // no block is kept there
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * mt + 4 * j + r, col = 16 * nt + n;
      const float D = col <= row ? exp_of(Gd[row] - Gd[col]) : 0.f;
      const float m = col < row ? D * kk[i][r] : 0.f;
      Ms[row * LDM + col] = m;
      Pl[row * LDM + col] = col <= row ? p.scale * D * qk[i][r] : 0.f;
      if (nt > mt) Ti[row * LDM + col] = 0.f;  // the inverse leaves blocks above the diagonal alone
    }
  }
  __syncthreads();
  write_tri(static_cast<uint16_t*>(p.P) + sh * kTri, Pl, tid);
  if (BWD) write_tri(static_cast<uint16_t*>(p.M) + sh * kTri, Ms, tid);
  invert(Ms, (const MSM_LDS float*)bt, Ti, wave, lane);
  write_tri(static_cast<uint16_t*>(p.T) + sh * kTri, Ti, tid);
}

// ---- scan ----------------------------------------------------------------------------------

// A matrix of 16 columns held by a wavefront: rows in blocks of 32 (see ops_delta.hpp).
template <int BLOCKS>
struct Cols {
  f32x4 t[BLOCKS][2];
};

template <int BLOCKS>
__device__ __forceinline__ Cols<BLOCKS> zero_cols() {
  Cols<BLOCKS> x;
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) x.t[b][0] = x.t[b][1] = zero4();
  return x;
}

// f(b, t, r, row) for every value a lane holds; row is the lane's row less 8 j.
template <int BLOCKS, class F>
__device__ __forceinline__ void each(F f) {
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) f(b, t, r, 32 * b + 4 * t + r);
}

// fp32 columns through a resource whose rows are `stride` bytes apart; `at` is this lane's first
// row and column.
template <int BLOCKS>
__device__ __forceinline__ Cols<BLOCKS> load_cols(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t stride) {
  Cols<BLOCKS> x;
  each<BLOCKS>([&](int b, int t, int r, int row) { x.t[b][t][r] = io<float>::bload(rs, at + row * stride, 0); });
  return x;
}
template <int BLOCKS>
__device__ __forceinline__ void store_cols(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t stride, const Cols<BLOCKS>& x) {
  each<BLOCKS>([&](int b, int t, int r, int row) { io<float>::bstore(rs, at + row * stride, 0, x.t[b][t][r]); });
}

// The chunk's rows of v, o or do: raw I/O elements between load and use.
struct RawCols {
  IO::raw v[8 * CB];
  __device__ __forceinline__ void fetch(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t stride) {
    each<CB>([&](int b, int t, int r, int row) { v[8 * b + 4 * t + r] = IO::bload(rs, at + row * stride, 0); });
  }
  __device__ __forceinline__ Cols<CB> widen() const {
    Cols<CB> x;
    each<CB>([&](int b, int t, int r, int) { x.t[b][t][r] = IO::widen(v[8 * b + 4 * t + r]); });
    return x;
  }
};
__device__ __forceinline__ void store_out(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t stride, const Cols<CB>& x) {
  each<CB>([&](int b, int t, int r, int row) { IO::bstore(rs, at + row * stride, 0, x.t[b][t][r]); });
}

// Left factor rows of a tile with permuted row numbering: row 32 b + 8 (m / 4) + 4 t + m % 4 for
// lane m.
__device__ __forceinline__ int perm_row(int b, int t, int lane) {
  const int m = lane & 15;
  return 32 * b + 8 * (m >> 2) + 4 * t + (m & 3);
}

// Accumulators of all tiles of a chunk's 16 columns, in the order the tile sets below have.
__device__ __forceinline__ f32x4 (&tiles(Cols<CB>& c))[2 * CB] { return reinterpret_cast<f32x4(&)[2 * CB]>(c); }

// Left factors of a product with keys or queries over 32 state rows: all tokens of the chunk.
struct RowTiles {
  Part<kIn> a[2 * CB];
  __device__ __forceinline__ void load(lds_cparts lds, int b, int lane, int j) {
#pragma unroll
    for (int i = 0; i < 2 * CB; ++i) a[i] = load_row<UK, kIn>(lds, perm_row(i / 2, i % 2, lane), 32 * b + 8 * j, kRows);
  }
};

// Left factors of a product with a chunk matrix (or its transpose) over one block of tokens.
template <int NA, bool TRANS>
struct TriTiles {
  Part<NA> a[CB][2 * CB];
  __device__ __forceinline__ void load(lds_cparts lds, int lane, int j) {
#pragma unroll
    for (int b = 0; b < CB; ++b)
#pragma unroll
      for (int i = 0; i < 2 * CB; ++i) {
        const int rb = i / 2, t = i % 2;
        if (!TRANS && b <= rb) a[b][i] = load_row<4, NA>(lds + TriM::block(rb, b), perm_row(0, t, lane), 8 * j, TriM::kPlane);
        if (TRANS && b >= rb) a[b][i] = load_col<4, NA>(lds + TriM::block(b, rb), 8 * j, 4 * t, 8, lane, TriM::kPlane);
      }
  }
  template <int N>
  __device__ __forceinline__ void mma(Cols<CB>& c, const Part<N> (&B)[CB]) const {
    f32x4(&x)[2 * CB] = tiles(c);
#pragma unroll
    for (int b = 0; b < CB; ++b)
#pragma unroll
      for (int sum = Terms<NA, N>::kMost - 1; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < NA; ++i)
          if (Terms<NA, N>::in(sum, i))
#pragma unroll
            for (int k = 0; k < 2 * CB; ++k)
              if (TRANS ? b >= k / 2 : b <= k / 2)
                x[k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[b][k].p[i], B[b].p[sum - i], x[k], 0, 0, 0);
  }
};

// Left factors of a state update: 32 rows of K^T or Q^T over one block of tokens.
struct ColTiles {
  Part<kIn> a[CB][2];
  __device__ __forceinline__ void load(lds_cparts lds, int b, int lane, int j) {
#pragma unroll
    for (int rb = 0; rb < CB; ++rb)
#pragma unroll
      for (int t = 0; t < 2; ++t) a[rb][t] = load_col<UK, kIn>(lds, 32 * rb + 8 * j, 32 * b + 4 * t, 8, lane, kRows);
  }
  template <int N>
  __device__ __forceinline__ void mma(f32x4 (&c)[2], const Part<N> (&B)[CB]) const {
#pragma unroll
    for (int rb = 0; rb < CB; ++rb) mma_tiles(c, a[rb], B[rb]);
  }
};

template <int N>
__device__ __forceinline__ void split_all(Part<N> (&B)[CB], const Cols<CB>& x) {
#pragma unroll
  for (int b = 0; b < CB; ++b) B[b] = split<N>(x.t[b][0], x.t[b][1]);
}

// Everything a chunk's 16-column walks share, loaded straight into LDS by all wavefronts.
constexpr int kPasses = C * UK / (64 * kWavesScan);  // of a plane of keys
static_assert(C * UK % (64 * kWavesScan) == 0, "whole passes");

// Passes of a wavefront over N planes of a chunk matrix; LDS holds whole rounds of all wavefronts.
constexpr int tri_rounds(int n) { return (n * TriM::kPlane / 512 + kWavesScan - 1) / kWavesScan; }
constexpr int tri_lds(int n) { return tri_rounds(n) * kWavesScan * 512; }

struct KeyRows {  // LDS
  uint16_t k[kIn * kRows], q[kIn * kRows];
  float ev[256];  // e^G, e^(G_C - G), beta: 3 C floats
};
// An array as a walk meets it: the address of the present chunk's part, the bytes to the next
// one's, and the extent of a part of `rows` rows, rows * per_row + rest (0 rows: nothing, which
// reads as zeros).  A walk's step is one block of code without branches, whose products then cover
// its loads and their address arithmetic.
struct Stream {
  const char* at;
  int64_t step;
  int32_t per_row, rest;
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(int rows) const {
    return make_rsrc_u32(at, (uint32_t)uniform(rows > 0 ? rows * per_row + rest : 0));
  }
  // the same for load_lds, and for a whole chunk's part, whatever its rows
  __device__ __forceinline__ u32x4 words(int rows) const {
    return rsrc_words(at, (uint32_t)uniform(rows > 0 ? rows * per_row + rest : 0));
  }
  __device__ __forceinline__ u32x4 whole(int rows, uint32_t bytes) const {
    return rsrc_words(at, (uint32_t)uniform(rows > 0 ? (int)bytes : 0));
  }
  __device__ __forceinline__ void next(int dir) { at += dir > 0 ? step : -step; }
};
// One head of a token array (rows, heads, size), from row `row`.
__device__ __forceinline__ Stream head_stream(const void* base, int64_t row, int64_t heads, int64_t h, int64_t size) {
  const char* at = static_cast<const char*>(base) + ((row * heads + h) * size) * IO::es;
  return Stream{reinterpret_cast<const char*>(uniform((int64_t)at)), uniform(C * heads * size * IO::es),
                (int32_t)(heads * size * IO::es), (int32_t)(-(heads - 1) * size * IO::es)};
}
// Parts of `bytes` for every slot and head.
__device__ __forceinline__ Stream slot_stream(const void* base, int64_t slot, int64_t heads, int64_t h, int64_t bytes) {
  const char* at = static_cast<const char*>(base) + (slot * heads + h) * bytes;
  return Stream{reinterpret_cast<const char*>(uniform((int64_t)at)), uniform(heads * bytes), 0, (int32_t)bytes};
}

template <int N>
__device__ __forceinline__ void load_tri(lds_parts lds, const Stream& s, int rows, int wave, int lane) {
  const auto r = s.whole(rows, N * TriM::kPlane * 2);
#pragma unroll
  for (int i = 0; i < tri_rounds(N); ++i) {
    const int pass = i * kWavesScan + wave;
    load_lds(r, lds + pass * 512, lane * 16 + pass * 1024);
  }
}

// Keys, queries and row factors on their way into LDS: from q and k, or from their planes in the
// workspace.
struct Keys {
  Stream k, q, ev;
  uint32_t at[kPasses];  // offsets of this thread's units
  __device__ __forceinline__ Keys(const DeltaArgs& p, int64_t row, int64_t slot, int64_t h, int64_t hk, int tid) {
    if (p.kq_direct) {
      k = head_stream(p.k, row, p.Hk, hk, p.K);
      q = head_stream(p.q, row, p.Hk, hk, p.K);
    } else {
      k = slot_stream(p.kq, slot, p.Hk, hk, 2 * kIn * kRows * 2);
      k.rest = kIn * kRows * 2;
      q = k;
      q.at += kIn * kRows * 2;
    }
    ev = slot_stream(p.vec, slot, p.H, h, kVec * 4);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int u = tid + i * 64 * kWavesScan, row_ = u / UK, c = ((u % UK) ^ swizzle<UK>(row_)) * 8;
      at[i] = !p.kq_direct ? u * 16 : (c < p.K ? (uint32_t)(row_ * p.Hk * p.K + c) * IO::es : kOutside);
    }
  }
  // piece `part` of `parts`: the loads are issued between a step's products
  __device__ __forceinline__ void load(MSM_LDS KeyRows& l, int rows, int wave, int lane, int part, int parts) const {
    const u32x4 rk = k.words(rows), rq = q.words(rows);
#pragma unroll
    for (int x = 0; x < kIn * kPasses; ++x) {
      if (x * parts / (kIn * kPasses) != part) continue;
      const int n = x / kPasses, i = x % kPasses;
      load_lds(rk, l.k + n * kRows + (i * kWavesScan + wave) * 512, at[i] + n * kRows * 2);
      load_lds(rq, l.q + n * kRows + (i * kWavesScan + wave) * 512, at[i] + n * kRows * 2);
    }
    // every wavefront brings the same values: cheaper than a branch
    if (part == 0) load_lds(ev.whole(rows, 3 * C * 4), (MSM_LDS void*)l.ev, lane * 16);
  }
  __device__ __forceinline__ void next(int dir) {
    k.next(dir);
    q.next(dir);
    ev.next(dir);
  }
};

// LDS of the walks: two chunks' worth where the 160 KB allow, so that the next chunk's loads run
// under the present one's products.
constexpr size_t kLdsMost = 160 * 1024 - 512;
template <bool BWD>
struct ScanChunk {
  KeyRows r;
  uint16_t t[tri_lds(TP)];
  uint16_t p[BWD ? 8 : tri_lds(TP)];
};
struct Nothing {};

// LDS reads stay on their side of this point; arithmetic and memory reads may pass.  The products
// read their left factors one step ahead, and without it the reads would sink to their uses.
__device__ __forceinline__ void hold_lds() { __builtin_amdgcn_sched_barrier(0x1F); }

// Asks for N times one MFMA followed by VALU other vector instructions: an MFMA occupies the matrix
// unit for 16 cycles and the issue port for 4, so up to three instructions fit under it.
template <int N, int VALU>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
  }
}

// This wavefront's place in a walk.
struct Walk {
  int tid, wave, lane, n, j, vb, col, len, chunks;
  bool on, last;  // columns there are; the sequence's last segment
  int64_t seg;    // segment and head: place of a segment's states
  int64_t s, h, hk, row0, slot0;
  uint32_t vstride, wstride, vat, wat, sat, sbytes;
  __device__ __forceinline__ Walk(const DeltaArgs& p) {
    tid = threadIdx.x;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    lane = tid & 63;
    n = lane & 15;
    j = lane >> 4;
    const uint32_t H = (uint32_t)p.H, group = H / (uint32_t)p.Hk;  // 32-bit: 64-bit division leaves the scalar unit
    const int si = uniform((int)(blockIdx.x / H)), hi = uniform((int)(blockIdx.x - (uint32_t)si * H));
    seg = blockIdx.x;
    h = hi;
    hk = uniform((int)((uint32_t)hi / group));
    vb = blockIdx.y * kWavesScan + wave;
    col = vb * 16 + n;
    on = vb * 16 < p.VP;
    const SegRows r = seg_rows<C>(p, si);
    s = r.s;
    len = (int)r.len;
    chunks = (len + C - 1) / C;
    last = r.last;
    row0 = r.row0;
    slot0 = r.slot0;
    vstride = (uint32_t)(p.H * p.V * IO::es);
    wstride = (uint32_t)(p.VP * 4);
    vat = col < p.V ? 8 * j * vstride + col * IO::es : kOutside;  // v, o, do, dv
    wat = on ? 8 * j * wstride + col * 4 : kOutside;              // columns of the workspace
    sat = col < p.V ? (8 * j * (uint32_t)p.V + col) * 4 : kOutside;  // states
    sbytes = (uint32_t)(p.K * p.V * 4);
  }
  // rows of a chunk, none past either end
  __device__ __forceinline__ int rows(int c) const {
    const int left = len - c * C, most = left < C ? left : C;
    return c < 0 ? 0 : (most > 0 ? most : 0);
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t state(const float* base, const DeltaArgs& p) const {
    return make_rsrc_u32(base + (s * p.H + h) * p.K * p.V, sbytes);
  }
};

// Arrays that a scan step writes, or none (forward or backward).
struct ScanOut {
  Stream o, S, pred, E;
  float* dots;
};

// One chunk of a walk.  fetch(part) issues piece `part` of NB of the next chunk's loads.
template <bool BWD, class F>
__device__ __forceinline__ void scan_chunk(F fetch, const DeltaArgs& p, const Walk& w, const MSM_LDS ScanChunk<BWD>& l, Cols<NB>& S,
                                           Cols<CB> R, const Cols<CB>& dO, const ScanOut& out, int rows) {
  const int lane = w.lane, j = w.j, n = w.n;
  const MSM_LDS float* eG = l.r.ev + 8 * j;           // this lane's rows of the chunk's row factors
  const MSM_LDS float* eK = l.r.ev + C + 8 * j;
  const MSM_LDS float* bt = l.r.ev + 2 * C + 8 * j;
  const float last = l.r.ev[C - 1];           // decay over the whole chunk

  if (BWD) store_cols<NB>(out.S.rsrc(rows), w.wat, w.wstride, S);
  // products with the state: predictions K S and readouts Q S
  Cols<CB> KS = zero_cols<CB>(), O = zero_cols<CB>();
  RowTiles fk[2], fq[2];
  TriTiles<TP, false> ft;
  TriTiles<TP, false> fp;
  fk[0].load(l.r.k, 0, lane, j);
  fq[0].load(l.r.q, 0, lane, j);
  Part<TP> sb = split<TP>(S.t[0][0], S.t[0][1]);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (b + 1 < NB) {
      fk[(b + 1) & 1].load(l.r.k, b + 1, lane, j);
      fq[(b + 1) & 1].load(l.r.q, b + 1, lane, j);
    } else {
      ft.load(l.t, lane, j);
    }
    fetch(b);
    hold_lds();
    mma_tiles(tiles(KS), fk[b & 1].a, sb);
    mma_tiles(tiles(O), fq[b & 1].a, sb);
    if (b + 1 < NB) sb = split<TP>(S.t[(b + 1) % NB][0], S.t[(b + 1) % NB][1]);
    interleave<4 * CB * TP, 3>();
  }
  // errors of the chunk: E = T (V - e^G K S)
  each<CB>([&](int b, int t, int r, int row) {
    const float x = eG[row];
    KS.t[b][t][r] *= x;
    R.t[b][t][r] -= KS.t[b][t][r];
    O.t[b][t][r] *= x * p.scale;
  });
  if (BWD) store_cols<CB>(out.pred.rsrc(rows), w.wat, w.wstride, KS);
  Part<TP> B[CB];
  split_all(B, R);
  Cols<CB> U = zero_cols<CB>();
  ColTiles fc[2];
  if constexpr (!BWD) fp.load(l.p, lane, j);
  fc[0].load(l.r.k, 0, lane, j);
  hold_lds();
  ft.mma(U, B);
  if (BWD) store_cols<CB>(out.E.rsrc(rows), w.wat, w.wstride, U);
  each<CB>([&](int b, int t, int r, int row) { U.t[b][t][r] *= bt[row]; });
  if constexpr (BWD) {
    // rows of dO . (scale e^G Q S0) over this wavefront's columns
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i < 8 * CB ? O.t[(i / 8) % CB][(i / 4) % 2][i % 4] * dO.t[(i / 8) % CB][(i / 4) % 2][i % 4] : 0.f;
    const float sum = sum_rows16(x, lane);
    if (w.on && n < 8 * CB) out.dots[32 * (n / 8) + 8 * j + n % 8] = sum;
  } else {
    split_all(B, U);
    fp.mma(O, B);
    store_out(out.o.rsrc(rows), w.vat, w.vstride, O);
  }
  // state after the chunk
  each<CB>([&](int b, int t, int r, int row) { U.t[b][t][r] *= eK[row]; });
  split_all(B, U);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (b + 1 < NB) fc[(b + 1) & 1].load(l.r.k, b + 1, lane, j);
    hold_lds();
#pragma unroll
    for (int t = 0; t < 2; ++t) S.t[b][t] *= last;
    fc[b & 1].mma(S.t[b], B);
  }
}

// A wavefront owns all rows of 16 columns of the state, 2 x NB tiles in its registers: the columns
// are independent, so no state passes between wavefronts, and an accumulator's layout is that of a
// right factor with its rows permuted, so a product's result is the next one's factor without a
// trip through LDS.  Keys, queries and chunk matrices are left factors, shared by the four
// wavefronts in LDS and loaded there a chunk ahead.  Sequential in the chunks, hence bound by a
// chunk's chain of products (K S, T R, K^T U and the two of O) at one wavefront a SIMD: Bt=4 L=4096
// H=32 K=V=128 bf16, 256 workgroups: 271 us for 64 chunks, 855 TFLOP/s of matrix products (69% of
// what a large one reaches).  BWD stores what the backward needs and leaves O out: 297 us at
// Bt=4 L=2048 H=16 fp32, where 128 workgroups leave half of the CUs idle.
template <bool BWD>
__global__ __launch_bounds__(64 * kWavesScan) void scan_kernel(const DeltaArgs p) {
  constexpr bool kTwo = 2 * sizeof(ScanChunk<BWD>) <= kLdsMost;
  __shared__ __attribute__((aligned(16))) ScanChunk<BWD> lds0;
  __shared__ __attribute__((aligned(16))) std::conditional_t<kTwo, ScanChunk<BWD>, Nothing> lds1;
  auto& l0 = (MSM_LDS ScanChunk<BWD>&)lds0;
  auto& l1 = (MSM_LDS std::conditional_t<kTwo, ScanChunk<BWD>, Nothing>&)lds1;
  const Walk w(p);
  if (w.s < 0) return;  // no segment here
  Cols<NB> S = zero_cols<NB>();
  if (p.seg_len > 0)
    S = load_cols<NB>(make_rsrc_u32(p.segS + w.seg * KP * p.VP, (uint32_t)(KP * p.VP * 4)), w.wat, w.wstride);
  else if (p.S0)
    S = load_cols<NB>(w.state(p.S0, p), w.sat, (uint32_t)(p.V * 4));
  Keys keys(p, w.row0, w.slot0, w.h, w.hk, w.tid);
  Stream st = slot_stream(p.T, w.slot0, p.H, w.h, kTri * 2), sp = slot_stream(p.P, w.slot0, p.H, w.h, kTri * 2);
  Stream sv = head_stream(p.v, w.row0, p.H, w.h, p.V), sd = head_stream(p.do_, w.row0, p.H, w.h, p.V);
  ScanOut out;
  out.o = head_stream(p.o, w.row0, p.H, w.h, p.V);
  out.S = slot_stream(p.S, w.slot0, p.H, w.h, KP * p.VP * 4);
  out.pred = slot_stream(p.pred, w.slot0, p.H, w.h, C * p.VP * 4);
  out.E = slot_stream(p.E, w.slot0, p.H, w.h, C * p.VP * 4);
  out.dots = p.dots + ((w.slot0 * p.H + w.h) * (p.VP / 16) + w.vb) * kDots;
  const int64_t dots_step = p.H * (p.VP / 16) * kDots;
  RawCols v, d;
  // the chunk that the streams stand at, in NB pieces
  const auto fetch = [&](MSM_LDS ScanChunk<BWD>& l, int rows, int part) {
    keys.load(l.r, rows, w.wave, w.lane, part, NB);
    if (part == NB - 1) {
      load_tri<TP>(l.t, st, rows, w.wave, w.lane);
      if constexpr (!BWD) load_tri<TP>(l.p, sp, rows, w.wave, w.lane);
      v.fetch(sv.rsrc(rows), w.vat, w.vstride);
      if (BWD) d.fetch(sd.rsrc(rows), w.vat, w.vstride);
      keys.next(1);
      st.next(1);
      sp.next(1);
      sv.next(1);
      sd.next(1);
    }
  };
  const auto fetch_all = [&](MSM_LDS ScanChunk<BWD>& l, int rows) {
#pragma unroll
    for (int part = 0; part < NB; ++part) fetch(l, rows, part);
  };
  const auto done = [&]() {
    out.o.next(1);
    out.S.next(1);
    out.pred.next(1);
    out.E.next(1);
    out.dots += dots_step;
  };
  if constexpr (kTwo) {
    const auto step = [&](MSM_LDS ScanChunk<BWD>& here, MSM_LDS ScanChunk<BWD>& next, int c) {
      sync_loads();  // `here` is loaded, and nothing reads `next` any more
      const Cols<CB> R = v.widen(), dO = d.widen();
      const int rows = w.rows(c + 1);
      scan_chunk<BWD>([&](int part) { fetch(next, rows, part); }, p, w, here, S, R, dO, out, w.rows(c));
      done();
    };
    fetch_all(l0, w.rows(0));
    int c = 0;
    for (; c + 1 < w.chunks; c += 2) {
      step(l0, l1, c);
      step(l1, l0, c + 1);
    }
    if (c < w.chunks) step(l0, l1, c);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // the last step's empty loads still write to LDS
  } else {
    for (int c = 0; c < w.chunks; ++c) {
      sync_lds();
      fetch_all(l0, w.rows(c));
      sync_loads();
      scan_chunk<BWD>([](int) {}, p, w, l0, S, v.widen(), d.widen(), out, w.rows(c));
      done();
    }
  }
  if (w.on && w.last && p.last_S) store_cols<NB>(w.state(p.last_S, p), w.sat, (uint32_t)(p.V * 4), S);
}

// ---- segments ------------------------------------------------------------------------------
//
// A walk is sequential in the chunks, so few heads and sequences leave most of the GPU idle.  Then
// sequences are cut into segments of seg_len chunks.  A segment maps the state affinely, S -> F S + G:
// one walk over all segments at once finds G (from a zero state) and F (from the identity, with V
// zero, as K more columns), a short second kernel runs through the segments' maps, and the walk
// proper starts every segment from its state.  That is 2.2 to 2.5 times the work, the segments' maps
// at a higher rate than the walk's: Bt=1 L=65536 H=16 K=V=128 bf16 in 8 or 9 segments a head, 476 us
// (1040 TFLOP/s of matrix products, 84% of a large product's), 22 us, and 528 us for the walk, against
// 3.8 ms for the walk of whole sequences.

struct StateChunk {
  uint16_t k[kIn * kRows];
  float ev[256];
  uint16_t t[tri_lds(TP)];
};

__global__ __launch_bounds__(64 * kWavesScan) void segment_kernel(const DeltaArgs p) {
  __shared__ __attribute__((aligned(16))) StateChunk lds0;
  __shared__ __attribute__((aligned(16))) StateChunk lds1;
  auto& l0 = (MSM_LDS StateChunk&)lds0;
  auto& l1 = (MSM_LDS StateChunk&)lds1;
  const Walk w(p);
  if (w.s < 0 || w.last) return;  // nobody starts from the last segment's state
  const int lane = w.lane, j = w.j;
  const int unit = w.col - (int)p.VP;  // column of the identity
  Cols<NB> S;
  each<NB>([&](int b, int t, int r, int row) { S.t[b][t][r] = row + 8 * j == unit ? 1.f : 0.f; });
  Keys keys(p, w.row0, w.slot0, w.h, w.hk, w.tid);
  Stream st = slot_stream(p.T, w.slot0, p.H, w.h, kTri * 2), sv = head_stream(p.v, w.row0, p.H, w.h, p.V);
  RawCols v;
  const auto fetch = [&](MSM_LDS StateChunk& l, int rows) {
    const u32x4 rk = keys.k.words(rows);
#pragma unroll
    for (int x = 0; x < kIn * kPasses; ++x)
      load_lds(rk, l.k + x / kPasses * kRows + (x % kPasses * kWavesScan + w.wave) * 512,
               keys.at[x % kPasses] + x / kPasses * kRows * 2);
    load_lds(keys.ev.whole(rows, 3 * C * 4), (MSM_LDS void*)l.ev, lane * 16);
    load_tri<TP>(l.t, st, rows, w.wave, lane);
    v.fetch(sv.rsrc(rows), w.vat, w.vstride);
    keys.next(1);
    st.next(1);
    sv.next(1);
  };
  const auto step = [&](MSM_LDS StateChunk& l, MSM_LDS StateChunk& next, int c) {
    sync_loads();
    Cols<CB> R = v.widen(), KS = zero_cols<CB>(), U = zero_cols<CB>();
    fetch(next, w.rows(c + 1));
    const MSM_LDS float* eG = l.ev + 8 * j;
    const MSM_LDS float* eK = l.ev + C + 8 * j;
    const MSM_LDS float* bt = l.ev + 2 * C + 8 * j;
    RowTiles fk[2];
    TriTiles<TP, false> ft;
    fk[0].load(l.k, 0, lane, j);
    Part<TP> sb = split<TP>(S.t[0][0], S.t[0][1]);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b + 1 < NB)
        fk[(b + 1) & 1].load(l.k, b + 1, lane, j);
      else
        ft.load(l.t, lane, j);
      hold_lds();
      mma_tiles(tiles(KS), fk[b & 1].a, sb);
      if (b + 1 < NB) sb = split<TP>(S.t[(b + 1) % NB][0], S.t[(b + 1) % NB][1]);
      interleave<2 * CB * TP, 3>();
    }
    each<CB>([&](int b, int t, int r, int row) { R.t[b][t][r] = fmaf(-eG[row], KS.t[b][t][r], R.t[b][t][r]); });
    Part<TP> B[CB];
    split_all(B, R);
    ColTiles fc[2];
    fc[0].load(l.k, 0, lane, j);
    hold_lds();
    ft.mma(U, B);
    each<CB>([&](int b, int t, int r, int row) { U.t[b][t][r] *= bt[row] * eK[row]; });
    split_all(B, U);
    const float last = l.ev[C - 1];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b + 1 < NB) fc[(b + 1) & 1].load(l.k, b + 1, lane, j);
      hold_lds();
#pragma unroll
      for (int t = 0; t < 2; ++t) S.t[b][t] *= last;
      fc[b & 1].mma(S.t[b], B);
    }
  };
  fetch(l0, w.rows(0));
  int c = 0;
  for (; c + 1 < w.chunks; c += 2) {
    step(l0, l1, c);
    step(l1, l0, c + 1);
  }
  if (c < w.chunks) step(l0, l1, c);
  __builtin_amdgcn_s_waitcnt(0x0F70);
  if (w.on)
    store_cols<NB>(make_rsrc_u32(p.segS + w.seg * KP * p.VP, (uint32_t)(KP * p.VP * 4)), w.wat, w.wstride, S);
  else if (unit < KP)
    store_cols<NB>(make_rsrc_u32(p.segF + w.seg * KP * KP, (uint32_t)(KP * KP * 4)), (8 * j * KP + unit) * 4, KP * 4, S);
}

// Runs through a sequence's segments: every segment's G makes room for the state it starts from.
// A workgroup has 16 columns, a wavefront 32 rows of them; the state passes between them through
// LDS, and the next segment's map is fetched while the present one is applied.  Bound by the latency
// of that fetch, 2.5 us a segment; one wavefront with all rows took 12 us.
__global__ __launch_bounds__(64 * NB) void join_kernel(const DeltaArgs p) {
  constexpr int LDJ = 17;
  __shared__ float state[2][KP * LDJ];
  const int rb = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 15, j = lane >> 4;
  const uint32_t H = (uint32_t)p.H;
  const int64_t s = uniform((int)(blockIdx.x / H)), h = uniform((int)(blockIdx.x % H));
  const int col = blockIdx.y * 16 + n, row0 = 32 * rb + 8 * j;
  const SeqSegs q = seq_segs<C>(p, s);
  Cols<1> S = zero_cols<1>();
  if (p.S0)
    S = load_cols<1>(make_rsrc_u32(p.S0 + (s * p.H + h) * p.K * p.V, (uint32_t)(p.K * p.V * 4)),
                     col < p.V ? (row0 * (uint32_t)p.V + col) * 4 : kOutside, (uint32_t)(p.V * 4));
  const uint32_t at = (uint32_t)(row0 * p.VP + col) * 4, stride = (uint32_t)(p.VP * 4);
  f32x4 F[NB][2][2];
  const auto fetch = [&](int64_t g) {
    const auto rf = make_rsrc_u32(p.segF + ((q.first + g) * p.H + h) * KP * KP, g + 1 < q.count ? (uint32_t)(KP * KP * 4) : 0u);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t i = (uint32_t)(perm_row(rb, t, lane) * KP + 32 * b + 8 * j) * 4;
        F[b][t][0] = bload4(rf, i);
        F[b][t][1] = bload4(rf, i + 16);
      }
  };
  fetch(0);
  for (int64_t g = 0; g < q.count; ++g) {
    const auto rs = make_rsrc_u32(p.segS + ((q.first + g) * p.H + h) * KP * p.VP, (uint32_t)(KP * p.VP * 4));
    const bool more = g + 1 < q.count;  // nobody starts from the last segment's end
    Cols<1> next = zero_cols<1>();
    if (more) next = load_cols<1>(rs, at, stride);
    store_cols<1>(rs, at, stride, S);
    if (!more) break;
    float* lds = state[g & 1];
    each<1>([&](int, int t, int r, int row) { lds[(row0 + row) * LDJ + n] = S.t[0][t][r]; });
    Part<TP> f[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t) f[b][t] = split<TP>(F[b][t][0], F[b][t][1]);
    fetch(g + 1);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      f32x4 x[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i / 4][i % 4] = lds[(32 * b + 8 * j + i) * LDJ + n];
      mma_tiles(next.t[0], f[b], split<TP>(x[0], x[1]));
    }
    S = next;
  }
}

// ---- rev -----------------------------------------------------------------------------------

struct RevTri {
  uint16_t t[tri_lds(TP)], p[tri_lds(TP)], m[tri_lds(TP)];
};

struct RevOut {
  Stream dv, dV, dS;
  float* dots;
};

// p_used and tm_used are called when this wavefront has read P, and T and M, for the last time.
template <class FP, class FT>
__device__ __forceinline__ void rev_chunk(FP p_used, FT tm_used, const DeltaArgs& p, const Walk& w, const MSM_LDS KeyRows& l, const MSM_LDS RevTri& x3,
                                          Cols<NB>& S, Cols<CB> dO, const Cols<CB>& Er, const Cols<CB>& pred,
                                          const RevOut& out, int rows) {
  const int lane = w.lane, j = w.j, n = w.n;
  const MSM_LDS float* eG = l.ev + 8 * j;
  const MSM_LDS float* eK = l.ev + C + 8 * j;
  const MSM_LDS float* bt = l.ev + 2 * C + 8 * j;
  const float last = l.ev[C - 1];
  // the adjoint after this chunk, kept for the gradients of q and k
  store_cols<NB>(out.dS.rsrc(rows), w.wat, w.wstride, S);
  // W = e^{G_C - G} (K dS) + P^T dO
  Cols<CB> W = zero_cols<CB>();
  RowTiles fk[2];
  TriTiles<TP, true> f3[2];
  fk[0].load(l.k, 0, lane, j);
  Part<TP> sb = split<TP>(S.t[0][0], S.t[0][1]);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (b + 1 < NB)
      fk[(b + 1) & 1].load(l.k, b + 1, lane, j);
    else
      f3[0].load(x3.p, lane, j);
    hold_lds();
    mma_tiles(tiles(W), fk[b & 1].a, sb);
    if (b + 1 < NB) sb = split<TP>(S.t[(b + 1) % NB][0], S.t[(b + 1) % NB][1]);
  }
  float uw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) uw[i] = 0.f;
  each<CB>([&](int b, int t, int r, int row) {
    W.t[b][t][r] *= eK[row];
    uw[8 * b + 4 * t + r] = bt[row] * Er.t[b][t][r] * W.t[b][t][r];
  });
  Part<kIn> dOB[CB];
  split_all(dOB, dO);
  f3[1].load(x3.t, lane, j);
  hold_lds();
  p_used();
  f3[0].mma(W, dOB);
  // dV = T^T (beta W)
  Cols<CB> dV = zero_cols<CB>(), x;
  Part<TP> B[CB];
  each<CB>([&](int b, int t, int r, int row) { x.t[b][t][r] = W.t[b][t][r] * bt[row]; });
  split_all(B, x);
  f3[0].load(x3.m, lane, j);
  hold_lds();
  f3[1].mma(dV, B);
  // Y = W - stril(D K K^T)^T dV
  each<CB>([&](int b, int t, int r, int) { x.t[b][t][r] = -dV.t[b][t][r]; });
  split_all(B, x);
  ColTiles fq[2], fc[2];
  fq[0].load(l.q, 0, lane, j);
  fc[0].load(l.k, 0, lane, j);
  hold_lds();
  tm_used();
  f3[0].mma(W, B);
  float ye[16], dp[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) ye[i] = dp[i] = 0.f;
  each<CB>([&](int b, int t, int r, int) {
    ye[8 * b + 4 * t + r] = W.t[b][t][r] * Er.t[b][t][r];
    dp[8 * b + 4 * t + r] = dV.t[b][t][r] * pred.t[b][t][r];
  });
  float* dots = out.dots;
  const float sy = sum_rows16(ye, lane), sp = sum_rows16(dp, lane), sw = sum_rows16(uw, lane);
  if (w.on && n < 8 * CB) {
    const int row = 32 * (n / 8) + 8 * j + n % 8;
    dots[C + row] = sy;
    dots[2 * C + row] = sp;
    dots[3 * C + row] = sw;
  }
  store_cols<CB>(out.dV.rsrc(rows), w.wat, w.wstride, dV);
  store_out(out.dv.rsrc(rows), w.vat, w.vstride, dV);
  // dS0 = e^{G_C} dS1 + Q^T (scale e^G dO) - K^T (e^G dV)
  Part<TP> BQ[CB];
  each<CB>([&](int b, int t, int r, int row) {
    dO.t[b][t][r] *= eG[row] * p.scale;
    dV.t[b][t][r] *= -eG[row];
  });
  split_all(BQ, dO);
  split_all(B, dV);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (b + 1 < NB) {
      fq[(b + 1) & 1].load(l.q, b + 1, lane, j);
      fc[(b + 1) & 1].load(l.k, b + 1, lane, j);
    }
    hold_lds();
#pragma unroll
    for (int t = 0; t < 2; ++t) S.t[b][t] *= last;
    fq[b & 1].mma(S.t[b], BQ);
    fc[b & 1].mma(S.t[b], B);
  }
}

// Split and layout as the scan's; per chunk it has six products where the scan has three (W from two,
// dV, Y, dS0 from two) and three chunk matrices.  These have one buffer each in LDS, filled again as
// soon as every wavefront has read it; keys and queries have two where the LDS allows.  Bound like the
// scan: 327 us at Bt=4 L=2048 H=16 K=V=128 fp32 (128 workgroups), 499 us for 16384 packed tokens, H=16
// bf16, the longest sequence's 72 chunks at 6.9 us.
template <bool kTwo>
__global__ __launch_bounds__(64 * kWavesScan) void rev_kernel(const DeltaArgs p) {
  __shared__ __attribute__((aligned(16))) KeyRows lds0;
  __shared__ __attribute__((aligned(16))) std::conditional_t<kTwo, KeyRows, Nothing> lds1;
  __shared__ __attribute__((aligned(16))) RevTri lds_tri;
  auto& l0 = (MSM_LDS KeyRows&)lds0;
  auto& l1 = (MSM_LDS std::conditional_t<kTwo, KeyRows, Nothing>&)lds1;
  auto& x3 = (MSM_LDS RevTri&)lds_tri;
  const Walk w(p);
  Cols<NB> S = zero_cols<NB>();  // the adjoint of the state
  if (p.dlast_S) S = load_cols<NB>(w.state(p.dlast_S, p), w.sat, (uint32_t)(p.V * 4));
  const int64_t end = w.chunks - 1, row = w.row0 + end * C, slot = w.slot0 + end;
  Keys keys(p, row, slot, w.h, w.hk, w.tid);
  Stream st = slot_stream(p.T, slot, p.H, w.h, kTri * 2), sp = slot_stream(p.P, slot, p.H, w.h, kTri * 2);
  Stream sm = slot_stream(p.M, slot, p.H, w.h, kTri * 2), sd = head_stream(p.do_, row, p.H, w.h, p.V);
  Stream sE = slot_stream(p.E, slot, p.H, w.h, C * p.VP * 4), spred = slot_stream(p.pred, slot, p.H, w.h, C * p.VP * 4);
  RevOut out;
  out.dv = head_stream(p.dv, row, p.H, w.h, p.V);
  out.dV = slot_stream(p.dV, slot, p.H, w.h, C * p.VP * 4);
  out.dS = slot_stream(p.dS, slot, p.H, w.h, KP * p.VP * 4);
  out.dots = p.dots + ((slot * p.H + w.h) * (p.VP / 16) + w.vb) * kDots;
  RawCols d;
  Cols<CB> Er, pred;
  const auto fetch_keys = [&](auto& l, int rows) {
    keys.load(l, rows, w.wave, w.lane, 0, 1);
    keys.next(-1);
  };
  const auto fetch_cols = [&](int rows) {
    d.fetch(sd.rsrc(rows), w.vat, w.vstride);
    Er = load_cols<CB>(sE.rsrc(rows), w.wat, w.wstride);
    pred = load_cols<CB>(spred.rsrc(rows), w.wat, w.wstride);
    for (Stream* x : {&sd, &sE, &spred}) x->next(-1);
  };
  const auto fetch_p = [&](int rows) {
    load_tri<TP>(x3.p, sp, rows, w.wave, w.lane);
    sp.next(-1);
  };
  const auto fetch_tm = [&](int rows) {
    load_tri<TP>(x3.t, st, rows, w.wave, w.lane);
    load_tri<TP>(x3.m, sm, rows, w.wave, w.lane);
    st.next(-1);
    sm.next(-1);
  };
  const auto step = [&](auto& here, int c) {
    const int rows = w.rows(c), before = w.rows(c - 1);
    const Cols<CB> dO = d.widen(), E0 = Er, pred0 = pred;
    fetch_cols(before);
    rev_chunk(
        [&] {
          sync_lds();
          fetch_p(before);
        },
        [&] {
          sync_lds();
          fetch_tm(before);
        },
        p, w, here, x3, S, dO, E0, pred0, out, rows);
    for (Stream* x : {&out.dv, &out.dV, &out.dS}) x->next(-1);
    out.dots -= p.H * (p.VP / 16) * kDots;
  };
  fetch_cols(w.rows(w.chunks - 1));
  fetch_p(w.rows(w.chunks - 1));
  fetch_tm(w.rows(w.chunks - 1));
  if constexpr (kTwo) {
    fetch_keys(l0, w.rows(w.chunks - 1));
    int c = w.chunks - 1;
    for (; c > 0; c -= 2) {
      sync_loads();
      fetch_keys(l1, w.rows(c - 1));
      step(l0, c);
      sync_loads();
      fetch_keys(l0, w.rows(c - 2));
      step(l1, c - 1);
    }
    if (c == 0) {
      sync_loads();
      step(l0, c);
    }
  } else {
    for (int c = w.chunks - 1; c >= 0; --c) {
      sync_lds();
      fetch_keys(l0, w.rows(c));
      sync_loads();
      step(l0, c);
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // empty loads past the first chunk still write to LDS
  if (w.on && p.dS0) store_cols<NB>(w.state(p.dS0, p), w.sat, (uint32_t)(p.V * 4), S);
}

// ---- grad ----------------------------------------------------------------------------------

// Wavefronts: two a SIMD hide each other's loads, but the fp32 parts of eight would not fit.
constexpr int kWavesGrad = KP == 256 || (KP == 128 && MSM_IO_BF16) ? 8 : 4;
constexpr int kTilesGrad = KP / 16 > kWavesGrad ? KP / 16 / kWavesGrad : 1;      // 16-key tiles a wavefront
constexpr int MT = C / 16;                                                      // 16-token tiles
constexpr int VB = MSM_IO_BF16 ? 64 : 32;                                       // columns staged at a time
constexpr int LDV = VB + 8, LDT = C + 8;
constexpr int PW = kWavesGrad >= 2 * MT ? 2 : 1, PT = MT / PW;  // wavefronts for a row of token pairs, tiles each

// All chunks at once.  A wavefront accumulates kTilesGrad tiles of 16 keys of dQ and dK over the value
// heads that share them and, with others, the token pairs dO U^T and dV U^T; states and their adjoints
// are read from memory straight into the factors' registers, once each, while columns of dO, dV and U
// pass through LDS, all of them fetched one step ahead.  Bound by issue at one (fp32) or two (bf16)
// wavefronts a SIMD, 4 vector instructions a matrix one, most of them cutting fp32 values into parts,
// and by its 256 registers: 360 us at Bt=4 L=2048 H=16 K=V=128 fp32 (393 TFLOP/s of matrix products),
// 578 us for 16384 packed tokens, 8 key heads, H=16 bf16 (336 TFLOP/s, 196 bytes spilled; with two
// parts a factor 510 us, and 784 us then with four wavefronts and loads at their uses).
__global__ __launch_bounds__(64 * kWavesGrad) void grad_kernel(const DeltaArgs p) {
  constexpr int THREADS = 64 * kWavesGrad;
  constexpr int kStage = (kIn + 2 * TP) * C * LDV, kPair = 2 * TP * C * LDT;
  __shared__ __attribute__((aligned(16))) uint16_t lds_k[kIn * kRows];
  __shared__ __attribute__((aligned(16))) uint16_t lds_q[kIn * kRows];
  // first the staged columns of dO, dV and U, then the token-pair matrices X and Z + Z^T
  __shared__ __attribute__((aligned(16))) uint16_t lds_buf[kStage > kPair ? kStage : kPair];
  __shared__ __attribute__((aligned(16))) float ev[3 * C];
  __shared__ double Gd[C];
  __shared__ float inner[kWavesGrad];  // <S0, dS1> over a wavefront's keys
  __shared__ float rowsum[MT][C];  // sums of N_ij over a tile of columns
  __shared__ float across[MT][C];  // sums of N_ij over a tile of rows i >= t and all j < t
  const lds_parts Ks = (lds_parts)lds_k, Qs = (lds_parts)lds_q, buf = (lds_parts)lds_buf;
  const lds_parts dOs = buf, dVs = buf + kIn * C * LDV, Us = dVs + TP * C * LDV;
  const lds_parts Xs = buf, Zs = buf + TP * C * LDT;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, j = lane >> 4;
  const int64_t slot = blockIdx.x, hk = blockIdx.y, group = (uint32_t)p.H / (uint32_t)p.Hk;
  const ChunkRows ch = chunk_rows<C>(p, slot);
  if (ch.n == 0) return;
  const int64_t at = (ch.row0 * p.Hk + hk) * p.K;
  const uint32_t stride = (uint32_t)(p.Hk * p.K * IO::es);
  {
    RawRows<THREADS, KP> kr, qr;
    kr.fetch(head_rsrc(p.k, ch.row0, p.Hk, hk, p.K, IO::es, ch.n), stride, (int)p.K, p.vec_k, 0, tid);
    qr.fetch(head_rsrc(p.q, ch.row0, p.Hk, hk, p.K, IO::es, ch.n), stride, (int)p.K, p.vec_k, 0, tid);
    kr.put(Ks, nullptr, 0, tid);
    qr.put(Qs, nullptr, 0, tid);
  }
  const int tile0 = wave * kTilesGrad;           // this wavefront's key tiles
  const bool keys = tile0 * 16 < KP;
  // token pairs: 16-row tile `prow`, its 16-column tiles ppart, ppart + PW, ...
  const int prow = wave % MT, ppart = wave / MT;
  const bool pairs = ppart < PW;

  f32x4 dq[MT][kTilesGrad], dk[MT][kTilesGrad];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < kTilesGrad; ++t) dq[m][t] = dk[m][t] = zero4();

  for (int64_t gh = 0; gh < group; ++gh) {
    const int64_t h = hk * group + gh, sh = slot * p.H + h;
    const float evv = tid < 3 * C ? p.vec[sh * kVec + tid] : 0.f;
    const double gv = tid < C ? reinterpret_cast<const double*>(p.vec + sh * kVec + 3 * C)[tid] : 0.0;
    // sums over the columns for dbeta and dg: the last wavefront's, a token a lane
    double db = 0, after = 0, before = 0;
    if (wave == kWavesGrad - 1 && lane < C) {
      const float* dots = p.dots + sh * (p.VP / 16) * kDots;
#pragma unroll 4
      for (int b = 0; b < (int)(p.VP / 16); ++b, dots += kDots) {
        after += (double)dots[lane] - (double)dots[2 * C + lane];
        db += dots[C + lane];
        before += dots[3 * C + lane];
      }
    }
    f32x4 a1[kTilesGrad][MT], a2[kTilesGrad][MT], a3[kTilesGrad][MT], X[PT], Z[PT];
#pragma unroll
    for (int m = 0; m < PT; ++m) X[m] = Z[m] = zero4();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int t = 0; t < kTilesGrad; ++t) a1[t][m] = a2[t][m] = a3[t][m] = zero4();
    }
    const auto rdo = head_rsrc(p.do_, ch.row0, p.H, h, p.V, IO::es, ch.n);
    const auto rdv = make_rsrc_u32(p.dV + sh * C * p.VP, (uint32_t)(C * p.VP * 4));
    const auto re = make_rsrc_u32(p.E + sh * C * p.VP, (uint32_t)(C * p.VP * 4));
    const auto rs0 = make_rsrc_u32(p.S + sh * KP * p.VP, (uint32_t)(KP * p.VP * 4));
    const auto rs1 = make_rsrc_u32(p.dS + sh * KP * p.VP, (uint32_t)(KP * p.VP * 4));
    // columns and states are fetched one step ahead; both come from memory, where a step's loads
    // would take longer than its products
    constexpr int kUnits = (C * VB / 8 + THREADS - 1) / THREADS;
    f32x4 st[kUnits][6], ss[kTilesGrad][4];
    const auto fetch_cols = [&](int v0) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int u = tid + i * THREADS, row = u / (VB / 8), c = v0 + (u % (VB / 8)) * 8;
        const uint32_t o = (uint32_t)(row * p.H * p.V + c) * IO::es;
        const bool in = C * VB / 8 % THREADS == 0 || row < C;
        if (p.vec_v) {
          st[i][0] = bload4(rdo, in && c < p.V ? o : kOutside);
          if (!MSM_IO_BF16) st[i][1] = bload4(rdo, in && c + 4 < p.V ? o + 16 : kOutside);
        } else {
          uint32_t x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[e] = __builtin_bit_cast(uint32_t, IO::bload(rdo, in && c + e < p.V ? o + e * IO::es : kOutside, 0));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            st[i][0][e] = __uint_as_float(MSM_IO_BF16 ? x[2 * e] | (x[2 * e + 1] << 16) : x[e]);
            st[i][1][e] = __uint_as_float(x[4 + e]);
          }
        }
        const uint32_t w = in && c < p.VP ? (uint32_t)(row * p.VP + c) * 4 : kOutside;
        st[i][2] = bload4(rdv, w);
        st[i][3] = bload4(rdv, w + 16);
        st[i][4] = bload4(re, w);
        st[i][5] = bload4(re, w + 16);
      }
    };
    const auto put_cols = [&]() {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int u = tid + i * THREADS, row = u / (VB / 8), c = (u % (VB / 8)) * 8;
        if (C * VB / 8 % THREADS != 0 && row >= C) continue;
        Part<kIn> o;
        if constexpr (kIn == 1)
          o.p[0] = __builtin_bit_cast(bf16x8, st[i][0]);
        else
          o = split<kIn>(st[i][0], st[i][1]);
        const float beta = ev[2 * C + row];
        store_parts(dOs + row * LDV + c, C * LDV, o);
        store_parts(dVs + row * LDV + c, C * LDV, split<TP>(st[i][2], st[i][3]));
        store_parts(Us + row * LDV + c, C * LDV, split<TP>(st[i][4] * beta, st[i][5] * beta));
      }
    };
    const auto fetch_states = [&](int v) {
#pragma unroll
      for (int t = 0; t < kTilesGrad; ++t) {
        const uint32_t i = keys && v < p.VP ? (uint32_t)((16 * (tile0 + t) + n) * p.VP + v + 8 * j) * 4 : kOutside;
        ss[t][0] = bload4(rs0, i);
        ss[t][1] = bload4(rs0, i + 16);
        ss[t][2] = bload4(rs1, i);
        ss[t][3] = bload4(rs1, i + 16);
      }
    };
    float dot = 0.f;  // <S0, dS1>
    fetch_cols(0);
    fetch_states(0);
    __syncthreads();  // the head before has been read
    if (tid < 3 * C) ev[tid] = evv;
    if (tid < C) Gd[tid] = gv;
    for (int v0 = 0; v0 < p.VP; v0 += VB) {
      __syncthreads();  // ev is there; the previous columns have been used
      put_cols();
      fetch_cols(v0 + VB);
      __syncthreads();
#pragma unroll
      for (int b = 0; b < VB / 32; ++b) {
        if (v0 + 32 * b >= p.VP) break;
        Part<TP> s0[kTilesGrad], s1[kTilesGrad];
#pragma unroll
        for (int t = 0; t < kTilesGrad; ++t) {
          s0[t] = split<TP>(ss[t][0], ss[t][1]);
          s1[t] = split<TP>(ss[t][2], ss[t][3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) dot = fmaf(ss[t][0][i], ss[t][2][i], fmaf(ss[t][1][i], ss[t][3][i], dot));
        }
        fetch_states(v0 + 32 * b + 32);
        if (keys) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int e = (16 * m + n) * LDV + 32 * b + 8 * j;
            const auto fo = load_ld<kIn>(dOs + e, C * LDV);
            const auto fv = load_ld<TP>(dVs + e, C * LDV);
            const auto fu = load_ld<TP>(Us + e, C * LDV);
#pragma unroll
            for (int t = 0; t < kTilesGrad; ++t) {
              mma(a1[t][m], fo, s0[t]);
              mma(a2[t][m], fv, s0[t]);
              mma(a3[t][m], fu, s1[t]);
            }
          }
        }
        if (pairs) {
          const int e = (16 * prow + n) * LDV + 32 * b + 8 * j;
          const auto fo = load_ld<kIn>(dOs + e, C * LDV);
          const auto fv = load_ld<TP>(dVs + e, C * LDV);
#pragma unroll
          for (int i = 0; i < PT; ++i) {
            const int m = ppart + PW * i;
            if (m > prow) continue;
            const auto fu = load_ld<TP>(Us + (16 * m + n) * LDV + 32 * b + 8 * j, C * LDV);
            mma(X[i], fo, fu);
            mma(Z[i], fv, fu);
          }
        }
      }
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) dot += __shfl_xor(dot, m, 64);
    if (lane == 0) inner[wave] = dot;
    __syncthreads();  // the staged columns have been used
    float N[PT][4];  // running sums of N along the rows of a tile
    if (pairs) {
#pragma unroll
      for (int i = 0; i < PT; ++i) {
        const int m = ppart + PW * i;
        f32x4 qk = zero4(), kk = zero4();
        if (m <= prow) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const auto B = load_row<UK, kIn>(Ks, 16 * m + n, 32 * b + 8 * j, kRows);
            mma(qk, load_row<UK, kIn>(Qs, 16 * prow + n, 32 * b + 8 * j, kRows), B);
            mma(kk, load_row<UK, kIn>(Ks, 16 * prow + n, 32 * b + 8 * j, kRows), B);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * prow + 4 * j + r, c = 16 * m + n;
          const float D = c <= row ? exp_of(Gd[row] - Gd[c]) : 0.f;
          const float x = c <= row ? p.scale * D * X[i][r] : 0.f, z = c < row ? -D * Z[i][r] : 0.f;
          store_parts1<TP>(Xs + row * LDT + c, C * LDT, x);
          if (c <= row) {
            store_parts1<TP>(Zs + row * LDT + c, C * LDT, z);
            store_parts1<TP>(Zs + c * LDT + row, C * LDT, z);
          }
          float sum = c < row ? x * qk[r] + z * kk[r] : 0.f;
          sum += dpp<0x111>(sum);  // row_shr: from the lanes before in the group, zero past its start
          sum += dpp<0x112>(sum);
          sum += dpp<0x114>(sum);
          sum += dpp<0x118>(sum);
          N[i][r] = sum;
          if (n == 15) rowsum[m][row] = sum;
        }
      }
    }
    __syncthreads();
    if (pairs) {
      // a pair (row, c) lies across t = c + 1 and on, up to t = row
#pragma unroll
      for (int i = 0; i < PT; ++i) {
        const int m = ppart + PW * i;
        float below = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * prow + 4 * j + r;
          float sum = N[i][r];
#pragma unroll
          for (int k = 0; k < MT; ++k)
            if (k < m) sum += rowsum[k][row];
          if (16 * m + n < row) below += sum;
        }
        below += __shfl_xor(below, 16, 64);
        below += __shfl_xor(below, 32, 64);
        if (j == 0) across[prow][16 * m + n] = below;
      }
    }
    __syncthreads();
    if (wave == kWavesGrad - 1 && lane < C) {
      // running sums of the decay's gradient
#pragma unroll
      for (int m = 1; m < C; m *= 2) {
        const double dn = __shfl_down(after, m, 64), up = __shfl_up(before, m, 64);
        if (lane + m < C) after += dn;
        if (lane >= m) before += up;
      }
      double through = 0;
#pragma unroll
      for (int i = 0; i < kWavesGrad; ++i) through += inner[i];
      double dg = after + through * ev[C - 1];
      const double up = __shfl_up(before, 1, 64);
      if (lane > 0) {
        dg += up;
#pragma unroll
        for (int m = 0; m < MT; ++m)
          if (16 * m + 15 >= lane) dg += across[m][lane - 1];
      }
      if (lane < ch.n) {
        p.dg[(ch.row0 + lane) * p.H + h] = (float)dg;
        p.dbeta[(ch.row0 + lane) * p.H + h] = (float)db;
      }
    }
    if (keys) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = ev[16 * m + 4 * j + r], y = ev[C + 16 * m + 4 * j + r];
#pragma unroll
          for (int t = 0; t < kTilesGrad; ++t) {
            dq[m][t][r] = fmaf(x * p.scale, a1[t][m][r], dq[m][t][r]);
            dk[m][t][r] += y * a3[t][m][r] - x * a2[t][m][r];
          }
        }
#pragma unroll
      for (int b = 0; b < CB; ++b)
#pragma unroll
        for (int t = 0; t < kTilesGrad; ++t) {
          const auto kt = load_col<UK, kIn>(Ks, 32 * b + 8 * j, 16 * (tile0 + t), 4, lane, kRows);
          const auto qt = load_col<UK, kIn>(Qs, 32 * b + 8 * j, 16 * (tile0 + t), 4, lane, kRows);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (m / 2 >= b)
              mma(dq[m][t], load_ld<TP>(Xs + (16 * m + n) * LDT + 32 * b + 8 * j, C * LDT), kt);
            mma(dk[m][t], load_ld<TP>(Zs + (16 * m + n) * LDT + 32 * b + 8 * j, C * LDT), kt);
            if (m / 2 <= b)
              mma(dk[m][t], load_col_ld<TP>(Xs + (32 * b + 8 * j) * LDT, LDT, 16 * m, lane, C * LDT), qt);
          }
        }
    }
  }
  if (keys) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < kTilesGrad; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * m + 4 * j + r, c = 16 * (tile0 + t) + n;
          if (row < ch.n && c < p.K) {
            const int64_t i = at + row * p.Hk * p.K + c;
            IO::store(p.dq, i, dq[m][t][r]);
            IO::store(p.dk, i, dk[m][t][r]);
          }
        }
  }
}

dim3 scan_grid(int64_t walks, int64_t H, int64_t columns) {
  return dim3((unsigned)(walks * H), (unsigned)((columns / 16 + kWavesScan - 1) / kWavesScan));
}

// The forward walk, in segments where the call is laid out for them.
template <bool BWD>
hipError_t walk(const DeltaArgs& a, hipStream_t s) {
  const dim3 block(64 * kWavesScan);
  if (a.seg_len > 0) {
    hipLaunchKernelGGL(segment_kernel, scan_grid(a.nsegs, a.H, a.VP + KP), block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)(a.nseq * a.H), (unsigned)(a.VP / 16)), dim3(64 * NB), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(scan_kernel<BWD>, scan_grid(a.seg_len > 0 ? a.nsegs : a.nseq, a.H, a.VP), block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t MSM_DELTA_NAME(fwd, MSM_IO_BF16, MSM_KP)(const DeltaArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(prep_kernel<false>, dim3((unsigned)a.nslots, (unsigned)a.H), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? walk<false>(a, s) : e;
}

hipError_t MSM_DELTA_NAME(bwd, MSM_IO_BF16, MSM_KP)(const DeltaArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(prep_kernel<true>, dim3((unsigned)a.nslots, (unsigned)a.H), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  e = walk<true>(a, s);
  if (e != hipSuccess) return e;
  DeltaArgs whole = a;  // the walk back is not cut
  whole.seg_len = 0;
  hipLaunchKernelGGL(rev_kernel<2 * sizeof(KeyRows) + sizeof(RevTri) <= kLdsMost>, scan_grid(a.nseq, a.H, a.VP),
                     dim3(64 * kWavesScan), 0, s, whole);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(grad_kernel, dim3((unsigned)a.nslots, (unsigned)a.Hk), dim3(64 * kWavesGrad), 0, s, a);
  return hipGetLastError();
}

}  // namespace msm
