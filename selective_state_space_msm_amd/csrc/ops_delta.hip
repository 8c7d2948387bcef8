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
// Four kernels, each built for one I/O type and padded key size (this file is compiled once
// per pair):
//   prep   one workgroup per chunk and head: decays, Gram matrices, the triangular inverse
//   scan   one workgroup per sequence, head and 64 columns of V, chunk after chunk; S stays in
//          registers, each wavefront owning all K rows of 16 columns
//   rev    the same walk backwards for dS
//   grad   one workgroup per chunk and key head: dQ, dK and the sums for dbeta and dg
#include "ops_delta.hpp"

namespace msm {
namespace {

#if MSM_IO_BF16
using Math = MathBF16;
#else
using Math = MathF32;
#endif
constexpr int KP = MSM_KP;
constexpr int C = delta_chunk(MSM_IO_BF16, KP);
constexpr int NB = KP / 32;       // blocks of 32 state rows
constexpr int CB = C / 32;        // blocks of 32 tokens
constexpr int LDT = C + Math::pad;
constexpr int UK = KP / Math::kPer;                 // 16-byte units of a row of keys
constexpr int UT = 32 / Math::kPer;                 // and of a row of a chunk matrix's blocks
using TriM = Tri<Math, C>;
constexpr int TP = Math::kPlanes;
constexpr int kVec = 5 * C;
constexpr int kDots = 4 * C + 4;
constexpr int kWavesScan = 4;     // wavefronts of a scan workgroup, 16 columns each
using E = Math::elem;
using TE = Math::telem;
template <int N>
using Part = Math::Part<N>;

__device__ __forceinline__ float exp_of(double x) { return exp2_fast((float)(x * 1.4426950408889634)); }

// ---- prep ----------------------------------------------------------------------------------

// Inverse of the unit lower triangular I + Ms (C x C in LDS, entries below the diagonal) into
// Ti.  Wavefront w inverts diagonal block w of 16 by forward substitution, a column per lane;
// block column j of the inverse then follows downwards, T_ij = -T_ii sum_k M_ik T_kj, its blocks
// staying in wavefront j's registers as right factors.  Substitution in blocks keeps the error
// of a triangular solve; products of powers of M would not.
constexpr int LDM = C + 4;
__device__ __forceinline__ void invert(const float* Ms, float* Ti, int wave, int lane) {
  constexpr int B16 = C / 16;
  const int n = lane & 15, j = lane >> 4;
  if (wave < B16) {
    float x[16];
    const float* M = Ms + (16 * wave) * LDM + 16 * wave;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == n ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < i; ++k) s = fmaf(-M[i * LDM + k], x[k], s);
      x[i] = s;
    }
    if (j == 0)
#pragma unroll
      for (int i = 0; i < 16; ++i) Ti[(16 * wave + i) * LDM + 16 * wave + n] = x[i];
  }
  __syncthreads();
  if (wave < B16) {
    f32x4 t[B16];
#pragma unroll
    for (int r = 0; r < 4; ++r) t[0][r] = Ti[(16 * wave + 4 * j + r) * LDM + 16 * wave + n];
#pragma unroll
    for (int d = 1; d < B16; ++d) {
      const int i = wave + d;
      if (i < B16) {
        f32x4 acc = zero4();
#pragma unroll
        for (int e = 0; e < d; ++e) {
          const f32x4 a = *reinterpret_cast<const f32x4*>(Ms + (16 * i + n) * LDM + 16 * (wave + e) + 4 * j);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], t[e][r], acc, 0, 0, 0);
        }
        const f32x4 a = *reinterpret_cast<const f32x4*>(Ti + (16 * i + n) * LDM + 16 * i + 4 * j);
        t[d] = zero4();
#pragma unroll
        for (int r = 0; r < 4; ++r) t[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(-a[r], acc[r], t[d], 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) Ti[(16 * i + 4 * j + r) * LDM + 16 * wave + n] = t[d][r];
      }
    }
  }
  __syncthreads();
}

// Keys and queries of a chunk into LDS.
template <int THREADS>
__device__ __forceinline__ void stage_two(E* Ks, E* Qs, __amdgpu_buffer_rsrc_t rk, __amdgpu_buffer_rsrc_t rq,
                                          uint32_t stride, int K, bool vec, int tid) {
  using Stage = RowStage<Math, KP, C, THREADS>;
  if (vec) {
    Stage k, q;
    k.fetch(rk, stride, K, tid);
    q.fetch(rq, stride, K, tid);
    k.put(Ks, tid);
    q.put(Qs, tid);
  } else {
    Stage::by_element(Ks, rk, stride, K, tid);
    Stage::by_element(Qs, rq, stride, K, tid);
  }
}

template <bool BWD>
__global__ __launch_bounds__(256) void prep_kernel(const DeltaArgs p) {
  __shared__ __attribute__((aligned(16))) E Ks[C * KP];
  __shared__ __attribute__((aligned(16))) E Qs[C * KP];
  __shared__ __attribute__((aligned(16))) float Ms[C * LDM];
  __shared__ __attribute__((aligned(16))) float Ti[C * LDM];
  __shared__ double Gd[C];
  __shared__ float bt[C];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, j = lane >> 4;
  const int64_t slot = blockIdx.x, h = blockIdx.y;
  const ChunkRows ch = chunk_rows<C>(p, slot);
  if (ch.n == 0) return;
  const int64_t sh = slot * p.H + h, hk = h / (p.H / p.Hk);
  const auto rk = head_rsrc(p.k, ch.row0, p.Hk, hk, p.K, Math::es, ch.n);
  const auto rq = head_rsrc(p.q, ch.row0, p.Hk, hk, p.K, Math::es, ch.n);
  stage_two<256>(Ks, Qs, rk, rq, (uint32_t)(p.Hk * p.K * Math::es), (int)p.K, p.vec_k, tid);
  if (wave == 0) {
    // running sum of the log decay in fp64: its differences keep fp32 accuracy
    const bool on = lane < ch.n;
    const int64_t i = (ch.row0 + lane) * p.H + h;
    float gl = on ? p.g[i] : 0.f;
    // exp(-1e4) is 0 already; below it the sum would lose the decays that follow (a decay of
    // minus infinity, or of the lowest float, resets the state)
    gl = gl < -1e4f ? -1e4f : gl;
    double G = (double)gl;
    const float b = on ? p.beta[i] : 0.f;
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
  __syncthreads();
  // Gram tiles on and below the diagonal; 16 x 16, one wavefront each
  TE* Pg = static_cast<TE*>(p.P) + sh * TP * TriM::kPlane;
  TE* Mg = BWD ? static_cast<TE*>(p.M) + sh * TP * TriM::kPlane : nullptr;
  for (int t = wave; t < (C / 16) * (C / 16); t += 4) {
    const int mt = t / (C / 16), nt = t % (C / 16);
    if (nt / 2 > mt / 2) continue;  // no block is kept there
    f32x4 kk = zero4(), qk = zero4();
    if (nt <= mt) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const auto B = load_row<Math, UK, 1>(Ks, 16 * nt + n, 32 * b + 8 * j, 0);
        Math::mma(kk, load_row<Math, UK, 1>(Ks, 16 * mt + n, 32 * b + 8 * j, 0), B);
        Math::mma(qk, load_row<Math, UK, 1>(Qs, 16 * mt + n, 32 * b + 8 * j, 0), B);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * mt + 4 * j + r, col = 16 * nt + n;
      const float D = col <= row ? exp_of(Gd[row] - Gd[col]) : 0.f;
      const float m = col < row ? D * kk[r] : 0.f;
      Ms[row * LDM + col] = m * bt[col];
      Math::store1<TP>(Pg + TriM::at(row, col), TriM::kPlane, col <= row ? p.scale * D * qk[r] : 0.f);
      if (BWD) Math::store1<TP>(Mg + TriM::at(row, col), TriM::kPlane, m);
    }
  }
  __syncthreads();
  invert(Ms, Ti, wave, lane);
  TE* Tg = static_cast<TE*>(p.T) + sh * TP * TriM::kPlane;
  for (int u = tid; u < C * C / 8; u += 256) {
    const int row = u / (C / 8), c = (u % (C / 8)) * 8;
    if (c / 32 > row / 32) continue;
    f32x4 a = zero4(), b = zero4();
    if (c / 16 <= row / 16) {  // blocks above the diagonal were not written
      a = *reinterpret_cast<const f32x4*>(Ti + row * LDM + c);
      b = *reinterpret_cast<const f32x4*>(Ti + row * LDM + c + 4);
    }
    if constexpr (Math::bf16) {
      Math::store_planes<TP>(Tg + TriM::at(row, c), TriM::kPlane, a, b);
    } else {
      *reinterpret_cast<f32x4*>(Tg + TriM::at(row, c)) = a;
      *reinterpret_cast<f32x4*>(Tg + TriM::at(row, c + 4)) = b;
    }
  }
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
using IO = io<Math::storage>;
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

// c += left x B for a left factor of keys or queries, 32 state rows per block.
template <int N>
__device__ __forceinline__ void mma_rows(Cols<CB>& c, const E* lds, int b, const Part<N>& B, int lane, int j) {
#pragma unroll
  for (int rb = 0; rb < CB; ++rb)
#pragma unroll
    for (int t = 0; t < 2; ++t)
      Math::mma(c.t[rb][t], load_row<Math, UK, 1>(lds, perm_row(rb, t, lane), 32 * b + 8 * j, 0), B);
}
// c += (chunk matrix) B, or its transpose
template <int NA, int NB_>
__device__ __forceinline__ void mma_tri(Cols<CB>& c, const TE* lds, const Part<NB_> (&B)[CB], int lane, int j) {
#pragma unroll
  for (int rb = 0; rb < CB; ++rb)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int b = 0; b <= rb; ++b)
        Math::mma(c.t[rb][t], load_row<Math, UT, NA>(lds + TriM::block(rb, b), perm_row(0, t, lane), 8 * j, TriM::kPlane), B[b]);
}
template <int NA, int NB_>
__device__ __forceinline__ void mma_tri_t(Cols<CB>& c, const TE* lds, const Part<NB_> (&B)[CB], int lane, int j) {
#pragma unroll
  for (int rb = 0; rb < CB; ++rb)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int b = rb; b < CB; ++b)
        Math::mma(c.t[rb][t], load_col<Math, UT, NA>(lds + TriM::block(b, rb), 8 * j, 4 * t, 8, lane, TriM::kPlane), B[b]);
}
template <int N>
__device__ __forceinline__ void split_all(Part<N> (&B)[CB], const Cols<CB>& x) {
#pragma unroll
  for (int b = 0; b < CB; ++b) B[b] = Math::split<N>(x.t[b][0], x.t[b][1]);
}

// What a chunk needs, fetched while the chunk before it is computed.
template <int TRIS, int PLANES2>
struct ChunkFetch {
  static constexpr int THREADS = 64 * kWavesScan;
  RowStage<Math, KP, C, THREADS> k, q;
  TriStage<Math, C, TP, THREADS> t;
  TriStage<Math, C, PLANES2, THREADS> p;
  TriStage<Math, C, TP, THREADS> m;
  float ev;
  __device__ __forceinline__ void fetch(const DeltaArgs& a, int64_t sh, int64_t row0, int64_t hk, int rows, int tid) {
    if (a.vec_k) {
      const uint32_t stride = (uint32_t)(a.Hk * a.K * Math::es);
      k.fetch(head_rsrc(a.k, row0, a.Hk, hk, a.K, Math::es, rows), stride, (int)a.K, tid);
      q.fetch(head_rsrc(a.q, row0, a.Hk, hk, a.K, Math::es, rows), stride, (int)a.K, tid);
    }
    t.fetch(TriStage<Math, C, TP, THREADS>::rsrc(a.T, sh, TP), tid);
    if constexpr (TRIS > 1) p.fetch(TriStage<Math, C, PLANES2, THREADS>::rsrc(a.P, sh, TP), tid);
    if constexpr (TRIS > 2) m.fetch(TriStage<Math, C, TP, THREADS>::rsrc(a.M, sh, TP), tid);
    ev = io<float>::bload(make_rsrc_u32(a.vec + sh * kVec, 3 * C * 4), tid * 4, 0);
  }
  __device__ __forceinline__ void put(const DeltaArgs& a, E* Ks, E* Qs, TE* Ts, TE* Ps, TE* Ms, float* evs, int64_t row0,
                                      int64_t hk, int rows, int tid) const {
    if (a.vec_k) {
      k.put(Ks, tid);
      q.put(Qs, tid);
    } else {
      const uint32_t stride = (uint32_t)(a.Hk * a.K * Math::es);
      RowStage<Math, KP, C, THREADS>::by_element(Ks, head_rsrc(a.k, row0, a.Hk, hk, a.K, Math::es, rows), stride, (int)a.K, tid);
      RowStage<Math, KP, C, THREADS>::by_element(Qs, head_rsrc(a.q, row0, a.Hk, hk, a.K, Math::es, rows), stride, (int)a.K, tid);
    }
    t.put(Ts, tid);
    if constexpr (TRIS > 1) p.put(Ps, tid);
    if constexpr (TRIS > 2) m.put(Ms, tid);
    if (tid < 3 * C) evs[tid] = ev;
  }
};

template <bool BWD>
__global__ __launch_bounds__(64 * kWavesScan) void scan_kernel(const DeltaArgs p) {
  constexpr int THREADS = 64 * kWavesScan;
  // parts of what the output is made of; the backward needs the state's share of it to fp32 and
  // the chunk's own share not at all
  constexpr int OP = BWD ? TP : Math::kOutParts;
  using Fetch = ChunkFetch<BWD ? 1 : 2, OP>;
  __shared__ __attribute__((aligned(16))) E Ks[C * KP];
  __shared__ __attribute__((aligned(16))) E Qs[C * KP];
  __shared__ __attribute__((aligned(16))) TE Ts[TriStage<Math, C, TP, THREADS>::kLds];
  __shared__ __attribute__((aligned(16))) TE Ps[BWD ? 8 : TriStage<Math, C, OP, THREADS>::kLds];
  __shared__ __attribute__((aligned(16))) float ev[3 * C];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, j = lane >> 4;
  const int64_t s = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
  const int vb = blockIdx.y * kWavesScan + wave, col = vb * 16 + n;
  const bool on = vb * 16 < p.VP;
  const SeqRows seq = seq_rows<C>(p, s);
  const uint32_t vstride = (uint32_t)(p.H * p.V * Math::es), wstride = (uint32_t)(p.VP * 4);
  const uint32_t vat = col < p.V ? 8 * j * vstride + col * Math::es : kOutside;   // v, o, do
  const uint32_t wat = on ? 8 * j * wstride + col * 4 : kOutside;                 // workspace columns
  const uint32_t sat = col < p.V ? (8 * j * (uint32_t)p.V + col) * 4 : kOutside;  // states
  const uint32_t sbytes = (uint32_t)(p.K * p.V * 4);

  Cols<NB> S = zero_cols<NB>();
  if (p.S0) S = load_cols<NB>(make_rsrc_u32(p.S0 + (s * p.H + h) * p.K * p.V, sbytes), sat, (uint32_t)(p.V * 4));

  const int64_t chunks = (seq.len + C - 1) / C;
  Fetch next;
  RawCols vnext, dnext;
  const auto fetch = [&](int64_t c) {
    const int64_t row0 = seq.row0 + c * C, left = seq.len - c * C;
    const int rows = (int)(left < C ? left : C);
    next.fetch(p, (seq.slot0 + c) * p.H + h, row0, hk, rows, tid);
    vnext.fetch(head_rsrc(p.v, row0, p.H, h, p.V, Math::es, rows), vat, vstride);
    if (BWD) dnext.fetch(head_rsrc(p.do_, row0, p.H, h, p.V, Math::es, rows), vat, vstride);
  };
  if (chunks > 0) fetch(0);
  for (int64_t c = 0; c < chunks; ++c) {
    const int64_t row0 = seq.row0 + c * C, sh = (seq.slot0 + c) * p.H + h;
    const int rows = (int)(seq.len - c * C < C ? seq.len - c * C : C);
    __syncthreads();  // the last chunk's reads are done
    next.put(p, Ks, Qs, Ts, Ps, nullptr, ev, row0, hk, rows, tid);
    Cols<CB> R = vnext.widen(), dO;
    if (BWD) dO = dnext.widen();
    __syncthreads();
    if (c + 1 < chunks) fetch(c + 1);
    if (!on) continue;
    const float* eG = ev + 8 * j;           // this lane's rows of the chunk's row factors
    const float* eK = ev + C + 8 * j;
    const float* bt = ev + 2 * C + 8 * j;
    const float last = ev[C - 1];           // decay over the whole chunk
    const auto rows_ws = [&](float* base) { return make_rsrc_u32(base + sh * C * p.VP, (uint32_t)(C * p.VP * 4)); };

    if (BWD) store_cols<NB>(make_rsrc_u32(p.S + sh * KP * p.VP, (uint32_t)(KP * p.VP * 4)), wat, wstride, S);
    // products with the state: predictions K S and readouts Q S
    Cols<CB> KS = zero_cols<CB>(), O = zero_cols<CB>();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const auto B = Math::split<TP>(S.t[b][0], S.t[b][1]);
      mma_rows(KS, Ks, b, B, lane, j);
      mma_rows(O, Qs, b, Math::first<OP>(B), lane, j);
    }
    // errors of the chunk: E = T (V - e^G K S)
    each<CB>([&](int b, int t, int r, int row) {
      const float x = eG[row];
      KS.t[b][t][r] *= x;
      R.t[b][t][r] -= KS.t[b][t][r];
      O.t[b][t][r] *= x * p.scale;
    });
    if (BWD) store_cols<CB>(rows_ws(p.pred), wat, wstride, KS);
    Part<TP> B[CB];
    split_all(B, R);
    Cols<CB> U = zero_cols<CB>();
    mma_tri<TP>(U, Ts, B, lane, j);
    if (BWD) store_cols<CB>(rows_ws(p.E), wat, wstride, U);
    each<CB>([&](int b, int t, int r, int row) { U.t[b][t][r] *= bt[row]; });
    if constexpr (BWD) {
      // rows of dO . (scale e^G Q S0) over this wavefront's columns
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = i < 8 * CB ? O.t[(i / 8) % CB][(i / 4) % 2][i % 4] * dO.t[(i / 8) % CB][(i / 4) % 2][i % 4] : 0.f;
      const float sum = sum_rows16(x, lane);
      if (n < 8 * CB) p.dots[(sh * (p.VP / 16) + vb) * kDots + 32 * (n / 8) + 8 * j + n % 8] = sum;
    } else {
      Part<OP> UO[CB];
      split_all(UO, U);
      mma_tri<OP>(O, Ps, UO, lane, j);
      store_out(head_rsrc(p.o, row0, p.H, h, p.V, Math::es, rows), vat, vstride, O);
    }
    // state after the chunk
    each<CB>([&](int b, int t, int r, int row) { U.t[b][t][r] *= eK[row]; });
    split_all(B, U);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 a = S.t[b][t] * last;
#pragma unroll
        for (int rb = 0; rb < CB; ++rb)
          Math::mma(a, load_col<Math, UK, 1>(Ks, 32 * rb + 8 * j, 32 * b + 4 * t, 8, lane, 0), B[rb]);
        S.t[b][t] = a;
      }
  }
  if (on && p.last_S)
    store_cols<NB>(make_rsrc_u32(p.last_S + (s * p.H + h) * p.K * p.V, sbytes), sat, (uint32_t)(p.V * 4), S);
}

// ---- rev -----------------------------------------------------------------------------------

__global__ __launch_bounds__(64 * kWavesScan) void rev_kernel(const DeltaArgs p) {
  constexpr int THREADS = 64 * kWavesScan;
  constexpr int kTri = TriStage<Math, C, TP, THREADS>::kLds;
  __shared__ __attribute__((aligned(16))) E Ks[C * KP];
  __shared__ __attribute__((aligned(16))) E Qs[C * KP];
  __shared__ __attribute__((aligned(16))) TE Ts[kTri];
  __shared__ __attribute__((aligned(16))) TE Ps[kTri];
  __shared__ __attribute__((aligned(16))) TE Ms[kTri];
  __shared__ __attribute__((aligned(16))) float ev[3 * C];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, j = lane >> 4;
  const int64_t s = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
  const int vb = blockIdx.y * kWavesScan + wave, col = vb * 16 + n;
  const bool on = vb * 16 < p.VP;
  const SeqRows seq = seq_rows<C>(p, s);
  const uint32_t vstride = (uint32_t)(p.H * p.V * Math::es), wstride = (uint32_t)(p.VP * 4);
  const uint32_t vat = col < p.V ? 8 * j * vstride + col * Math::es : kOutside;
  const uint32_t wat = on ? 8 * j * wstride + col * 4 : kOutside;
  const uint32_t sat = col < p.V ? (8 * j * (uint32_t)p.V + col) * 4 : kOutside;
  const uint32_t sbytes = (uint32_t)(p.K * p.V * 4);

  Cols<NB> S = zero_cols<NB>();  // the adjoint of the state
  if (p.dlast_S) S = load_cols<NB>(make_rsrc_u32(p.dlast_S + (s * p.H + h) * p.K * p.V, sbytes), sat, (uint32_t)(p.V * 4));

  const int64_t chunks = (seq.len + C - 1) / C;
  ChunkFetch<3, TP> next;
  RawCols dnext;
  const auto fetch = [&](int64_t c) {
    const int64_t row0 = seq.row0 + c * C, left = seq.len - c * C;
    const int rows = (int)(left < C ? left : C);
    next.fetch(p, (seq.slot0 + c) * p.H + h, row0, hk, rows, tid);
    dnext.fetch(head_rsrc(p.do_, row0, p.H, h, p.V, Math::es, rows), vat, vstride);
  };
  if (chunks > 0) fetch(chunks - 1);
  for (int64_t c = chunks - 1; c >= 0; --c) {
    const int64_t row0 = seq.row0 + c * C, sh = (seq.slot0 + c) * p.H + h;
    const int rows = (int)(seq.len - c * C < C ? seq.len - c * C : C);
    __syncthreads();
    next.put(p, Ks, Qs, Ts, Ps, Ms, ev, row0, hk, rows, tid);
    Cols<CB> dO = dnext.widen();
    __syncthreads();
    const auto rows_ws = [&](float* base) { return make_rsrc_u32(base + sh * C * p.VP, (uint32_t)(C * p.VP * 4)); };
    const Cols<CB> Er = load_cols<CB>(rows_ws(p.E), wat, wstride);
    const Cols<CB> pred = load_cols<CB>(rows_ws(p.pred), wat, wstride);
    const uint32_t state_ws = (uint32_t)(KP * p.VP * 4);
    const Cols<NB> S0 = load_cols<NB>(make_rsrc_u32(p.S + sh * KP * p.VP, state_ws), wat, wstride);
    if (c > 0) fetch(c - 1);
    if (!on) continue;
    const float* eG = ev + 8 * j;
    const float* eK = ev + C + 8 * j;
    const float* bt = ev + 2 * C + 8 * j;
    const float last = ev[C - 1];

    // the adjoint after this chunk, kept for the gradients of q and k
    store_cols<NB>(make_rsrc_u32(p.dS + sh * KP * p.VP, state_ws), wat, wstride, S);
    // W = e^{G_C - G} (K dS) + P^T dO
    Cols<CB> W = zero_cols<CB>();
#pragma unroll
    for (int b = 0; b < NB; ++b) mma_rows(W, Ks, b, Math::split<TP>(S.t[b][0], S.t[b][1]), lane, j);
    float uw[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) uw[i] = 0.f;
    each<CB>([&](int b, int t, int r, int row) {
      W.t[b][t][r] *= eK[row];
      uw[8 * b + 4 * t + r] = bt[row] * Er.t[b][t][r] * W.t[b][t][r];
    });
    Part<1> dOB[CB];
    split_all(dOB, dO);
    mma_tri_t<TP>(W, Ps, dOB, lane, j);
    // dV = T^T (beta W)
    Cols<CB> dV = zero_cols<CB>(), x;
    Part<TP> B[CB];
    each<CB>([&](int b, int t, int r, int row) { x.t[b][t][r] = W.t[b][t][r] * bt[row]; });
    split_all(B, x);
    mma_tri_t<TP>(dV, Ts, B, lane, j);
    // Y = W - stril(D K K^T)^T dV
    each<CB>([&](int b, int t, int r, int) { x.t[b][t][r] = -dV.t[b][t][r]; });
    split_all(B, x);
    mma_tri_t<TP>(W, Ms, B, lane, j);
    float ye[16], dp[16], dot = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ye[i] = dp[i] = 0.f;
    each<CB>([&](int b, int t, int r, int) {
      ye[8 * b + 4 * t + r] = W.t[b][t][r] * Er.t[b][t][r];
      dp[8 * b + 4 * t + r] = dV.t[b][t][r] * pred.t[b][t][r];
    });
    each<NB>([&](int b, int t, int r, int) { dot = fmaf(S0.t[b][t][r], S.t[b][t][r], dot); });
    dot *= last;
    float* dots = p.dots + (sh * (p.VP / 16) + vb) * kDots;
    const float sy = sum_rows16(ye, lane), sp = sum_rows16(dp, lane), sw = sum_rows16(uw, lane);
    if (n < 8 * CB) {
      const int row = 32 * (n / 8) + 8 * j + n % 8;
      dots[C + row] = sy;
      dots[2 * C + row] = sp;
      dots[3 * C + row] = sw;
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) dot += __shfl_xor(dot, m, 64);
    if (lane == 0) dots[4 * C] = dot;
    store_cols<CB>(rows_ws(p.dV), wat, wstride, dV);
    store_out(head_rsrc(p.dv, row0, p.H, h, p.V, Math::es, rows), vat, vstride, dV);
    // dS0 = e^{G_C} dS1 + Q^T (scale e^G dO) - K^T (e^G dV)
    Part<TP> BQ[CB];
    each<CB>([&](int b, int t, int r, int row) {
      dO.t[b][t][r] *= eG[row] * p.scale;
      dV.t[b][t][r] *= -eG[row];
    });
    split_all(BQ, dO);
    split_all(B, dV);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 a = S.t[b][t] * last;
#pragma unroll
        for (int rb = 0; rb < CB; ++rb) {
          Math::mma(a, load_col<Math, UK, 1>(Qs, 32 * rb + 8 * j, 32 * b + 4 * t, 8, lane, 0), BQ[rb]);
          Math::mma(a, load_col<Math, UK, 1>(Ks, 32 * rb + 8 * j, 32 * b + 4 * t, 8, lane, 0), B[rb]);
        }
        S.t[b][t] = a;
      }
  }
  if (on && p.dS0)
    store_cols<NB>(make_rsrc_u32(p.dS0 + (s * p.H + h) * p.K * p.V, sbytes), sat, (uint32_t)(p.V * 4), S);
}

// ---- grad ----------------------------------------------------------------------------------

constexpr int GP = Math::kGradParts;  // parts that the gradients of q and k are made of
constexpr int kWavesGrad = KP == 256 ? 8 : 4;
constexpr int kTilesGrad = KP / 16 / kWavesGrad > 0 ? KP / 16 / kWavesGrad : 1;  // 16-key tiles a wavefront
constexpr int MT = C / 16;                                                      // 16-token tiles
constexpr int VB = 64;                                                          // columns staged at a time
constexpr int LDV = VB + Math::pad;

__global__ __launch_bounds__(64 * kWavesGrad) void grad_kernel(const DeltaArgs p) {
  constexpr int THREADS = 64 * kWavesGrad;
  constexpr int kStage = (1 + 2 * TP) * C * LDV, kPair = 2 * GP * C * LDT;
  __shared__ __attribute__((aligned(16))) E Ks[C * KP];
  __shared__ __attribute__((aligned(16))) E Qs[C * KP];
  // first the staged columns of dO, dV and U, then the token-pair matrices X and Z + Z^T
  __shared__ __attribute__((aligned(16))) TE buf[kStage > kPair ? kStage : kPair];
  __shared__ __attribute__((aligned(16))) float ev[3 * C];
  __shared__ double Gd[C];
  __shared__ float across[MT][C];  // sums of N_ij over a tile of rows i >= t and all j < t
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, j = lane >> 4;
  const int64_t slot = blockIdx.x, hk = blockIdx.y, group = p.H / p.Hk;
  const ChunkRows ch = chunk_rows<C>(p, slot);
  if (ch.n == 0) return;
  const int64_t at = (ch.row0 * p.Hk + hk) * p.K;
  stage_two<THREADS>(Ks, Qs, head_rsrc(p.k, ch.row0, p.Hk, hk, p.K, Math::es, ch.n),
                     head_rsrc(p.q, ch.row0, p.Hk, hk, p.K, Math::es, ch.n), (uint32_t)(p.Hk * p.K * Math::es),
                     (int)p.K, p.vec_k, tid);
  E* dOs = reinterpret_cast<E*>(buf);
  TE* dVs = buf + C * LDV;
  TE* Us = dVs + TP * C * LDV;
  TE* Xs = buf;
  TE* Zs = buf + GP * C * LDT;
  const int tile0 = wave * kTilesGrad;           // this wavefront's key tiles
  const bool keys = tile0 * 16 < KP;
  const bool pairs = wave < MT;                  // this wavefront's row of token pairs

  f32x4 dq[MT][kTilesGrad], dk[MT][kTilesGrad];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < kTilesGrad; ++t) dq[m][t] = dk[m][t] = zero4();

  for (int64_t gh = 0; gh < group; ++gh) {
    const int64_t h = hk * group + gh, sh = slot * p.H + h;
    __syncthreads();
    for (int i = tid; i < 3 * C; i += THREADS) ev[i] = p.vec[sh * kVec + i];
    for (int i = tid; i < C; i += THREADS) Gd[i] = reinterpret_cast<const double*>(p.vec + sh * kVec + 3 * C)[i];
    f32x4 a1[MT][kTilesGrad], a2[MT][kTilesGrad], a3[MT][kTilesGrad], X[MT], Z[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      X[m] = Z[m] = zero4();
#pragma unroll
      for (int t = 0; t < kTilesGrad; ++t) a1[m][t] = a2[m][t] = a3[m][t] = zero4();
    }
    const auto rdo = head_rsrc(p.do_, ch.row0, p.H, h, p.V, Math::es, ch.n);
    const auto rdv = make_rsrc_u32(p.dV + sh * C * p.VP, (uint32_t)(C * p.VP * 4));
    const auto re = make_rsrc_u32(p.E + sh * C * p.VP, (uint32_t)(C * p.VP * 4));
    for (int64_t v0 = 0; v0 < p.VP; v0 += VB) {
      __syncthreads();  // ev is there; the previous columns have been used
      for (int u = tid; u < C * VB / 8; u += THREADS) {
        const int row = u / (VB / 8), c = (u % (VB / 8)) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dOs[row * LDV + c + i] = (E)IO::bload(rdo, v0 + c + i < p.V ? (uint32_t)(row * p.H * p.V + v0 + c + i) * Math::es : kOutside, 0);
        const uint32_t w = v0 + c < p.VP ? (uint32_t)(row * p.VP + v0 + c) * 4 : kOutside;
        const f32x4 a = __builtin_bit_cast(f32x4, bload16(rdv, w)), b = __builtin_bit_cast(f32x4, bload16(rdv, w + 16));
        const f32x4 d = __builtin_bit_cast(f32x4, bload16(re, w)) * ev[2 * C + row];
        const f32x4 e = __builtin_bit_cast(f32x4, bload16(re, w + 16)) * ev[2 * C + row];
        Math::store_planes<TP>(dVs + row * LDV + c, C * LDV, a, b);
        Math::store_planes<TP>(Us + row * LDV + c, C * LDV, d, e);
      }
      __syncthreads();
#pragma unroll
      for (int b = 0; b < VB / 32; ++b) {
        if (v0 + 32 * b >= p.VP) break;
        if (keys) {
          Part<1> fo[MT];
          Part<GP> fv[MT], fu[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int e = (16 * m + n) * LDV + 32 * b + 8 * j;
            fo[m] = Math::load<1>(dOs + e, 0);
            fv[m] = Math::load<GP>(dVs + e, C * LDV);
            fu[m] = Math::load<GP>(Us + e, C * LDV);
          }
#pragma unroll
          for (int t = 0; t < kTilesGrad; ++t) {
            const int64_t i = (sh * KP + 16 * (tile0 + t) + n) * p.VP + v0 + 32 * b + 8 * j;
            const auto s0 = Math::split<GP>(*reinterpret_cast<const f32x4*>(p.S + i), *reinterpret_cast<const f32x4*>(p.S + i + 4));
            const auto s1 = Math::split<GP>(*reinterpret_cast<const f32x4*>(p.dS + i), *reinterpret_cast<const f32x4*>(p.dS + i + 4));
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              Math::mma(a1[m][t], fo[m], s0);
              Math::mma(a2[m][t], fv[m], s0);
              Math::mma(a3[m][t], fu[m], s1);
            }
          }
        }
        if (pairs) {
          const int e = (16 * wave + n) * LDV + 32 * b + 8 * j;
          const auto fo = Math::load<1>(dOs + e, 0);
          const auto fv = Math::load<TP>(dVs + e, C * LDV);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (m > wave) continue;
            const auto fu = Math::load<TP>(Us + (16 * m + n) * LDV + 32 * b + 8 * j, C * LDV);
            Math::mma(X[m], fo, fu);
            Math::mma(Z[m], fv, fu);
          }
        }
      }
    }
    __syncthreads();  // the staged columns have been used
    if (pairs) {
      float carry[4] = {0.f, 0.f, 0.f, 0.f};  // N's row sums over the tiles before
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 qk = zero4(), kk = zero4();
        if (m <= wave) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const auto B = load_row<Math, UK, 1>(Ks, 16 * m + n, 32 * b + 8 * j, 0);
            Math::mma(qk, load_row<Math, UK, 1>(Qs, 16 * wave + n, 32 * b + 8 * j, 0), B);
            Math::mma(kk, load_row<Math, UK, 1>(Ks, 16 * wave + n, 32 * b + 8 * j, 0), B);
          }
        }
        float below = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * wave + 4 * j + r, c = 16 * m + n;
          const float D = c <= row ? exp_of(Gd[row] - Gd[c]) : 0.f;
          const float x = c <= row ? p.scale * D * X[m][r] : 0.f, z = c < row ? -D * Z[m][r] : 0.f;
          Math::store1<GP>(Xs + row * LDT + c, C * LDT, x);
          if (c <= row) {
            Math::store1<GP>(Zs + row * LDT + c, C * LDT, z);
            Math::store1<GP>(Zs + c * LDT + row, C * LDT, z);
          }
          // running sum of N along the row; a pair (row, c) lies across t = c + 1 and on
          float sum = c < row ? x * qk[r] + z * kk[r] : 0.f;
          sum += dpp<0x111>(sum);  // row_shr: from the lanes before in the group, zero past its start
          sum += dpp<0x112>(sum);
          sum += dpp<0x114>(sum);
          sum += dpp<0x118>(sum);
          sum += carry[r];
          carry[r] = __shfl(sum, lane | 15, 64);
          if (c < row) below += sum;
        }
        below += __shfl_xor(below, 16, 64);
        below += __shfl_xor(below, 32, 64);
        if (j == 0) across[wave][16 * m + n] = below;
      }
    }
    __syncthreads();
    if (tid < C) {
      // sums over the columns, then the running sums of the decay's gradient
      const float* dots = p.dots + sh * (p.VP / 16) * kDots;
      double db = 0, after = 0, before = 0, through = 0;
      for (int64_t b = 0; b < p.VP / 16; ++b, dots += kDots) {
        after += (double)dots[tid] - (double)dots[2 * C + tid];
        db += dots[C + tid];
        before += dots[3 * C + tid];
        through += dots[4 * C];
      }
#pragma unroll
      for (int m = 1; m < C; m *= 2) {
        const double dn = __shfl_down(after, m, 64), up = __shfl_up(before, m, 64);
        if (tid + m < C) after += dn;
        if (tid >= m) before += up;
      }
      double dg = after + through;
      const double up = __shfl_up(before, 1, 64);
      if (tid > 0) {
        dg += up;
#pragma unroll
        for (int m = 0; m < MT; ++m)
          if (16 * m + 15 >= tid) dg += across[m][tid - 1];
      }
      if (tid < ch.n) {
        p.dg[(ch.row0 + tid) * p.H + h] = (float)dg;
        p.dbeta[(ch.row0 + tid) * p.H + h] = (float)db;
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
            dq[m][t][r] = fmaf(x * p.scale, a1[m][t][r], dq[m][t][r]);
            dk[m][t][r] += y * a3[m][t][r] - x * a2[m][t][r];
          }
        }
#pragma unroll
      for (int b = 0; b < CB; ++b)
#pragma unroll
        for (int t = 0; t < kTilesGrad; ++t) {
          const auto kt = load_col<Math, UK, 1>(Ks, 32 * b + 8 * j, 16 * (tile0 + t), 4, lane, 0);
          const auto qt = load_col<Math, UK, 1>(Qs, 32 * b + 8 * j, 16 * (tile0 + t), 4, lane, 0);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (m / 2 >= b)
              Math::mma(dq[m][t], Math::load<GP>(Xs + (16 * m + n) * LDT + 32 * b + 8 * j, C * LDT), kt);
            Math::mma(dk[m][t], Math::load<GP>(Zs + (16 * m + n) * LDT + 32 * b + 8 * j, C * LDT), kt);
            if (m / 2 <= b)
              Math::mma(dk[m][t], Math::load_t<GP>(Xs + (32 * b + 8 * j) * LDT, LDT, C * LDT, lane, 16 * m, 4), qt);
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
            static_cast<E*>(p.dq)[i] = Math::narrow(dq[m][t][r]);
            static_cast<E*>(p.dk)[i] = Math::narrow(dk[m][t][r]);
          }
        }
  }
}

dim3 scan_grid(const DeltaArgs& a) {
  return dim3((unsigned)(a.nseq * a.H), (unsigned)((a.VP / 16 + kWavesScan - 1) / kWavesScan));
}

}  // namespace

hipError_t MSM_DELTA_NAME(fwd, MSM_IO_BF16, MSM_KP)(const DeltaArgs& a, hipStream_t s) {
  const dim3 chunks((unsigned)a.nslots, (unsigned)a.H);
  hipLaunchKernelGGL(prep_kernel<false>, chunks, dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(scan_kernel<false>, scan_grid(a), dim3(64 * kWavesScan), 0, s, a);
  return hipGetLastError();
}

hipError_t MSM_DELTA_NAME(bwd, MSM_IO_BF16, MSM_KP)(const DeltaArgs& a, hipStream_t s) {
  const dim3 chunks((unsigned)a.nslots, (unsigned)a.H);
  hipLaunchKernelGGL(prep_kernel<true>, chunks, dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(scan_kernel<true>, scan_grid(a), dim3(64 * kWavesScan), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(rev_kernel, scan_grid(a), dim3(64 * kWavesScan), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(grad_kernel, dim3((unsigned)a.nslots, (unsigned)a.Hk), dim3(64 * kWavesGrad), 0, s, a);
  return hipGetLastError();
}

}  // namespace msm
