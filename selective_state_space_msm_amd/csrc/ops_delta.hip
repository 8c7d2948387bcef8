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
constexpr int LD = KP + Math::pad;
constexpr int LDT = C + Math::pad;
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

template <bool BWD>
__global__ __launch_bounds__(256) void prep_kernel(const DeltaArgs p) {
  __shared__ __attribute__((aligned(16))) E Ks[C * LD];
  __shared__ __attribute__((aligned(16))) E Qs[C * LD];
  __shared__ __attribute__((aligned(16))) float Ms[C * LDM];
  __shared__ __attribute__((aligned(16))) float Ti[C * LDM];
  __shared__ double Gd[C];
  __shared__ float bt[C];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, j = lane >> 4;
  const int64_t slot = blockIdx.x, h = blockIdx.y;
  const ChunkRows ch = chunk_rows<C>(p, slot);
  if (ch.n == 0) return;
  const int64_t sh = slot * p.H + h, hk = h / (p.H / p.Hk), stride = p.Hk * p.K;
  const int64_t at = (ch.row0 * p.Hk + hk) * p.K;
  stage_rows<Math, KP, C, LD, 256>(Ks, static_cast<const E*>(p.k) + at, stride, ch.n, (int)p.K, p.vec_k, tid);
  stage_rows<Math, KP, C, LD, 256>(Qs, static_cast<const E*>(p.q) + at, stride, ch.n, (int)p.K, p.vec_k, tid);
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
  TE* Pg = static_cast<TE*>(p.P) + sh * TP * C * C;
  TE* Mg = BWD ? static_cast<TE*>(p.M) + sh * TP * C * C : nullptr;
  for (int t = wave; t < (C / 16) * (C / 16); t += 4) {
    const int mt = t / (C / 16), nt = t % (C / 16);
    f32x4 kk = zero4(), qk = zero4();
    if (nt <= mt) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const auto B = Math::load<1>(Ks + (16 * nt + n) * LD + 32 * b + 8 * j, 0);
        Math::mma(kk, Math::load<1>(Ks + (16 * mt + n) * LD + 32 * b + 8 * j, 0), B);
        Math::mma(qk, Math::load<1>(Qs + (16 * mt + n) * LD + 32 * b + 8 * j, 0), B);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * mt + 4 * j + r, col = 16 * nt + n;
      const float D = col <= row ? exp_of(Gd[row] - Gd[col]) : 0.f;
      const float m = col < row ? D * kk[r] : 0.f;
      Ms[row * LDM + col] = m * bt[col];
      Math::store1<TP>(Pg + row * C + col, C * C, col <= row ? p.scale * D * qk[r] : 0.f);
      if (BWD) Math::store1<TP>(Mg + row * C + col, C * C, m);
    }
  }
  __syncthreads();
  invert(Ms, Ti, wave, lane);
  TE* Tg = static_cast<TE*>(p.T) + sh * TP * C * C;
  for (int u = tid; u < C * C / 8; u += 256) {
    const int row = u / (C / 8), c = (u % (C / 8)) * 8;
    f32x4 a = zero4(), b = zero4();
    if (c / 16 <= row / 16) {  // blocks above the diagonal were not written
      a = *reinterpret_cast<const f32x4*>(Ti + row * LDM + c);
      b = *reinterpret_cast<const f32x4*>(Ti + row * LDM + c + 4);
    }
    Math::store_planes<TP>(Tg + row * C + c, C * C, a, b);
  }
}

// ---- scan ----------------------------------------------------------------------------------

// A matrix of 16 columns held by a wavefront: rows in blocks of 32 (see ops_delta.hpp).
template <int BLOCKS>
struct Cols {
  f32x4 t[BLOCKS][2];
};

// Rows of this lane: row0 + 8 j + 4 s + r of every 32-row block.
template <class IO, int BLOCKS>
__device__ __forceinline__ Cols<BLOCKS> load_cols(const IO* base, int64_t stride, int rows, bool col_ok, int j) {
  Cols<BLOCKS> x;
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 32 * b + 8 * j + 4 * s + r;
        float v = 0.f;
        if (col_ok && row < rows) {
          if constexpr (sizeof(IO) == 2)
            v = MathBF16::widen(base[row * stride]);
          else
            v = base[row * stride];
        }
        x.t[b][s][r] = v;
      }
  return x;
}

// Left factor rows of a tile with permuted row numbering: row 32 b + 8 (m / 4) + 4 s + m % 4 for
// lane m.
__device__ __forceinline__ int perm_row(int b, int s, int lane) {
  const int m = lane & 15;
  return 32 * b + 8 * (m >> 2) + 4 * s + (m & 3);
}

template <bool BWD>
__global__ __launch_bounds__(64 * kWavesScan) void scan_kernel(const DeltaArgs p) {
  constexpr int THREADS = 64 * kWavesScan;
  // parts of what the output is made of; the backward needs the state's share of it to fp32 and
  // the chunk's own share not at all
  constexpr int OP = BWD ? TP : Math::kOutParts;
  __shared__ __attribute__((aligned(16))) E Ks[C * LD];
  __shared__ __attribute__((aligned(16))) E Qs[C * LD];
  __shared__ __attribute__((aligned(16))) TE Ts[TP * C * LDT];
  __shared__ __attribute__((aligned(16))) TE Ps[BWD ? 8 : OP * C * LDT];
  __shared__ __attribute__((aligned(16))) float ev[3 * C];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, j = lane >> 4;
  const int64_t s = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
  const int64_t vb = (int64_t)blockIdx.y * kWavesScan + wave, col = vb * 16 + n;
  const bool on = vb * 16 < p.VP, col_ok = col < p.V;
  const SeqRows seq = seq_rows<C>(p, s);
  const int64_t state = ((s * p.H + h) * p.K) * p.V + col;

  Cols<NB> S;
  if (p.S0)
    S = load_cols<float, NB>(p.S0 + state, p.V, (int)p.K, col_ok, j);
  else
#pragma unroll
    for (int b = 0; b < NB; ++b) S.t[b][0] = S.t[b][1] = zero4();

  const int64_t chunks = (seq.len + C - 1) / C;
  for (int64_t c = 0; c < chunks; ++c) {
    const int64_t row0 = seq.row0 + c * C, sh = (seq.slot0 + c) * p.H + h;
    const int rows = (int)(seq.len - c * C < C ? seq.len - c * C : C);
    const int64_t at = (row0 * p.Hk + hk) * p.K;
    __syncthreads();  // the last chunk's reads are done
    stage_rows<Math, KP, C, LD, THREADS>(Ks, static_cast<const E*>(p.k) + at, p.Hk * p.K, rows, (int)p.K, p.vec_k, tid);
    stage_rows<Math, KP, C, LD, THREADS>(Qs, static_cast<const E*>(p.q) + at, p.Hk * p.K, rows, (int)p.K, p.vec_k, tid);
    stage_planes<Math, C, LDT, TP, THREADS>(Ts, static_cast<const TE*>(p.T) + sh * TP * C * C, tid);
    if constexpr (!BWD) stage_planes<Math, C, LDT, OP, THREADS>(Ps, static_cast<const TE*>(p.P) + sh * TP * C * C, tid);
    for (int i = tid; i < 3 * C; i += THREADS) ev[i] = p.vec[sh * kVec + i];
    __syncthreads();
    if (!on) continue;
    const float* eG = ev + 8 * j;           // this lane's rows of the chunk's row factors
    const float* eK = ev + C + 8 * j;
    const float* bt = ev + 2 * C + 8 * j;
    const float last = ev[C - 1];           // decay over the whole chunk

    Cols<CB> R = load_cols<E, CB>(static_cast<const E*>(p.v) + (row0 * p.H + h) * p.V + col, p.H * p.V, rows, col_ok, j);
    if (BWD) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            p.S[(sh * KP + 32 * b + 8 * j + 4 * t + r) * p.VP + col] = S.t[b][t][r];
    }
    // products with the state: predictions K S and readouts Q S
    Cols<CB> KS, O;
#pragma unroll
    for (int b = 0; b < CB; ++b) KS.t[b][0] = KS.t[b][1] = O.t[b][0] = O.t[b][1] = zero4();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const auto B = Math::split<TP>(S.t[b][0], S.t[b][1]);
      const auto BO = Math::first<OP>(B);
#pragma unroll
      for (int rb = 0; rb < CB; ++rb)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int e = perm_row(rb, t, lane) * LD + 32 * b + 8 * j;
          Math::mma(KS.t[rb][t], Math::load<1>(Ks + e, 0), B);
          Math::mma(O.t[rb][t], Math::load<1>(Qs + e, 0), BO);
        }
    }
    // errors of the chunk: E = T (V - e^G K S)
    Part<TP> RB[CB];
#pragma unroll
    for (int b = 0; b < CB; ++b) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = eG[32 * b + 4 * t + r];
          R.t[b][t][r] = fmaf(-x, KS.t[b][t][r], R.t[b][t][r]);
          O.t[b][t][r] *= x * p.scale;
          if (BWD) p.pred[(sh * C + 32 * b + 8 * j + 4 * t + r) * p.VP + col] = x * KS.t[b][t][r];
        }
      RB[b] = Math::split<TP>(R.t[b][0], R.t[b][1]);
    }
    Cols<CB> U;  // first E, then U = beta E
#pragma unroll
    for (int rb = 0; rb < CB; ++rb)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 a = zero4();
#pragma unroll
        for (int b = 0; b <= rb; ++b)
          Math::mma(a, Math::load<TP>(Ts + perm_row(rb, t, lane) * LDT + 32 * b + 8 * j, C * LDT), RB[b]);
        U.t[rb][t] = a;
      }
    if (BWD) {
#pragma unroll
      for (int b = 0; b < CB; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            p.E[(sh * C + 32 * b + 8 * j + 4 * t + r) * p.VP + col] = U.t[b][t][r];
    }
#pragma unroll
    for (int b = 0; b < CB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) U.t[b][t][r] *= bt[32 * b + 4 * t + r];
    if (BWD) {
      // rows of dO . (scale e^G Q S0) over this wavefront's columns
      const Cols<CB> dO = load_cols<E, CB>(static_cast<const E*>(p.do_) + (row0 * p.H + h) * p.V + col, p.H * p.V, rows, col_ok, j);
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = i < 8 * CB ? O.t[(i / 8) % CB][(i / 4) % 2][i % 4] * dO.t[(i / 8) % CB][(i / 4) % 2][i % 4] : 0.f;
      const float sum = sum_rows16(x, lane);
      if (n < 8 * CB) p.dots[(sh * (p.VP / 16) + vb) * kDots + 32 * (n / 8) + 8 * j + n % 8] = sum;
    } else {
      Part<OP> UO[CB];
#pragma unroll
      for (int b = 0; b < CB; ++b) UO[b] = Math::split<OP>(U.t[b][0], U.t[b][1]);
#pragma unroll
      for (int rb = 0; rb < CB; ++rb)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int b = 0; b <= rb; ++b)
            Math::mma(O.t[rb][t], Math::load<OP>(Ps + perm_row(rb, t, lane) * LDT + 32 * b + 8 * j, C * LDT), UO[b]);
      E* op = static_cast<E*>(p.o) + (row0 * p.H + h) * p.V + col;
#pragma unroll
      for (int b = 0; b < CB; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 32 * b + 8 * j + 4 * t + r;
            if (col_ok && row < rows) op[row * p.H * p.V] = Math::narrow(O.t[b][t][r]);
          }
    }
    // state after the chunk
#pragma unroll
    for (int b = 0; b < CB; ++b) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) U.t[b][t][r] *= eK[32 * b + 4 * t + r];
      RB[b] = Math::split<TP>(U.t[b][0], U.t[b][1]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 a = S.t[b][t] * last;
#pragma unroll
        for (int rb = 0; rb < CB; ++rb)
          Math::mma(a, Math::load_t<1>(Ks + (32 * rb + 8 * j) * LD, LD, 0, lane, 32 * b + 4 * t, 8), RB[rb]);
        S.t[b][t] = a;
      }
  }
  if (on && col_ok && p.last_S) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 32 * b + 8 * j + 4 * t + r;
          if (row < p.K) p.last_S[state + row * p.V] = S.t[b][t][r];
        }
  }
}

// ---- rev -----------------------------------------------------------------------------------

__global__ __launch_bounds__(64 * kWavesScan) void rev_kernel(const DeltaArgs p) {
  constexpr int THREADS = 64 * kWavesScan;
  __shared__ __attribute__((aligned(16))) E Ks[C * LD];
  __shared__ __attribute__((aligned(16))) E Qs[C * LD];
  __shared__ __attribute__((aligned(16))) TE Ts[TP * C * LDT];
  __shared__ __attribute__((aligned(16))) TE Ps[TP * C * LDT];
  __shared__ __attribute__((aligned(16))) TE Ms[TP * C * LDT];
  __shared__ __attribute__((aligned(16))) float ev[3 * C];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, j = lane >> 4;
  const int64_t s = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
  const int64_t vb = (int64_t)blockIdx.y * kWavesScan + wave, col = vb * 16 + n;
  const bool on = vb * 16 < p.VP, col_ok = col < p.V;
  const SeqRows seq = seq_rows<C>(p, s);
  const int64_t state = ((s * p.H + h) * p.K) * p.V + col;

  Cols<NB> S;  // the adjoint of the state
  if (p.dlast_S)
    S = load_cols<float, NB>(p.dlast_S + state, p.V, (int)p.K, col_ok, j);
  else
#pragma unroll
    for (int b = 0; b < NB; ++b) S.t[b][0] = S.t[b][1] = zero4();

  const int64_t chunks = (seq.len + C - 1) / C;
  for (int64_t c = chunks - 1; c >= 0; --c) {
    const int64_t row0 = seq.row0 + c * C, sh = (seq.slot0 + c) * p.H + h;
    const int rows = (int)(seq.len - c * C < C ? seq.len - c * C : C);
    const int64_t at = (row0 * p.Hk + hk) * p.K;
    __syncthreads();
    stage_rows<Math, KP, C, LD, THREADS>(Ks, static_cast<const E*>(p.k) + at, p.Hk * p.K, rows, (int)p.K, p.vec_k, tid);
    stage_rows<Math, KP, C, LD, THREADS>(Qs, static_cast<const E*>(p.q) + at, p.Hk * p.K, rows, (int)p.K, p.vec_k, tid);
    stage_planes<Math, C, LDT, TP, THREADS>(Ts, static_cast<const TE*>(p.T) + sh * TP * C * C, tid);
    stage_planes<Math, C, LDT, TP, THREADS>(Ps, static_cast<const TE*>(p.P) + sh * TP * C * C, tid);
    stage_planes<Math, C, LDT, TP, THREADS>(Ms, static_cast<const TE*>(p.M) + sh * TP * C * C, tid);
    for (int i = tid; i < 3 * C; i += THREADS) ev[i] = p.vec[sh * kVec + i];
    __syncthreads();
    if (!on) continue;
    const float* eG = ev + 8 * j;
    const float* eK = ev + C + 8 * j;
    const float* bt = ev + 2 * C + 8 * j;
    const float last = ev[C - 1];
    const int64_t vat = (row0 * p.H + h) * p.V + col;
    Cols<CB> dO = load_cols<E, CB>(static_cast<const E*>(p.do_) + vat, p.H * p.V, rows, col_ok, j);
    const Cols<CB> Er = load_cols<float, CB>(p.E + sh * C * p.VP + col, p.VP, C, true, j);

    // the adjoint after this chunk, kept for the gradients of q and k, and <S0, dS1>
    float dot = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t i = (sh * KP + 32 * b + 8 * j + 4 * t + r) * p.VP + col;
          p.dS[i] = S.t[b][t][r];
          dot = fmaf(p.S[i], S.t[b][t][r], dot);
        }
    dot *= last;

    // W = e^{G_C - G} (K dS) + P^T dO
    Cols<CB> W;
#pragma unroll
    for (int b = 0; b < CB; ++b) W.t[b][0] = W.t[b][1] = zero4();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const auto B = Math::split<TP>(S.t[b][0], S.t[b][1]);
#pragma unroll
      for (int rb = 0; rb < CB; ++rb)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          Math::mma(W.t[rb][t], Math::load<1>(Ks + perm_row(rb, t, lane) * LD + 32 * b + 8 * j, 0), B);
    }
    Part<1> dOB[CB];
    float uw[16];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uw[8 * b + 4 * t + r] = 0.f;
          if (b < CB) {
            f32x4& w = W.t[b % CB][t];
            w[r] *= eK[32 * b + 4 * t + r];
            uw[8 * b + 4 * t + r] = bt[32 * b + 4 * t + r] * Er.t[b % CB][t][r] * w[r];
          }
        }
#pragma unroll
    for (int b = 0; b < CB; ++b) dOB[b] = Math::split<1>(dO.t[b][0], dO.t[b][1]);
#pragma unroll
    for (int rb = 0; rb < CB; ++rb)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int b = rb; b < CB; ++b)
          Math::mma(W.t[rb][t], Math::load_t<TP>(Ps + (32 * b + 8 * j) * LDT, LDT, C * LDT, lane, 32 * rb + 4 * t, 8), dOB[b]);
    // dV = T^T (beta W)
    Part<TP> B[CB];
    Cols<CB> dV;
#pragma unroll
    for (int b = 0; b < CB; ++b) {
      f32x4 x[2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[t][r] = W.t[b][t][r] * bt[32 * b + 4 * t + r];
      B[b] = Math::split<TP>(x[0], x[1]);
    }
#pragma unroll
    for (int rb = 0; rb < CB; ++rb)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 a = zero4();
#pragma unroll
        for (int b = rb; b < CB; ++b)
          Math::mma(a, Math::load_t<TP>(Ts + (32 * b + 8 * j) * LDT, LDT, C * LDT, lane, 32 * rb + 4 * t, 8), B[b]);
        dV.t[rb][t] = a;
      }
    // Y = W - stril(D K K^T)^T dV
#pragma unroll
    for (int b = 0; b < CB; ++b) B[b] = Math::split<TP>(-dV.t[b][0], -dV.t[b][1]);
#pragma unroll
    for (int rb = 0; rb < CB; ++rb)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int b = rb; b < CB; ++b)
          Math::mma(W.t[rb][t], Math::load_t<TP>(Ms + (32 * b + 8 * j) * LDT, LDT, C * LDT, lane, 32 * rb + 4 * t, 8), B[b]);
    {
      const Cols<CB> pred = load_cols<float, CB>(p.pred + sh * C * p.VP + col, p.VP, C, true, j);
      float x[16], y[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int b = (i / 8) % CB, t = (i / 4) % 2, r = i % 4;
        x[i] = i < 8 * CB ? W.t[b][t][r] * Er.t[b][t][r] : 0.f;
        y[i] = i < 8 * CB ? dV.t[b][t][r] * pred.t[b][t][r] : 0.f;
      }
      float* dots = p.dots + (sh * (p.VP / 16) + vb) * kDots;
      const float sx = sum_rows16(x, lane), sy = sum_rows16(y, lane), sw = sum_rows16(uw, lane);
      if (n < 8 * CB) {
        dots[C + 32 * (n / 8) + 8 * j + n % 8] = sx;
        dots[2 * C + 32 * (n / 8) + 8 * j + n % 8] = sy;
        dots[3 * C + 32 * (n / 8) + 8 * j + n % 8] = sw;
      }
#pragma unroll
      for (int m = 1; m < 64; m *= 2) dot += __shfl_xor(dot, m, 64);
      if (lane == 0) dots[4 * C] = dot;
    }
    E* dvp = static_cast<E*>(p.dv) + vat;
#pragma unroll
    for (int b = 0; b < CB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 32 * b + 8 * j + 4 * t + r;
          p.dV[(sh * C + row) * p.VP + col] = dV.t[b][t][r];
          if (col_ok && row < rows) dvp[row * p.H * p.V] = Math::narrow(dV.t[b][t][r]);
        }
    // dS0 = e^{G_C} dS1 + Q^T (scale e^G dO) - K^T (e^G dV)
    Part<TP> BQ[CB];
#pragma unroll
    for (int b = 0; b < CB; ++b) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = eG[32 * b + 4 * t + r];
          dO.t[b][t][r] *= x * p.scale;
          dV.t[b][t][r] *= -x;
        }
      BQ[b] = Math::split<TP>(dO.t[b][0], dO.t[b][1]);
      B[b] = Math::split<TP>(dV.t[b][0], dV.t[b][1]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 a = S.t[b][t] * last;
#pragma unroll
        for (int rb = 0; rb < CB; ++rb) {
          Math::mma(a, Math::load_t<1>(Qs + (32 * rb + 8 * j) * LD, LD, 0, lane, 32 * b + 4 * t, 8), BQ[rb]);
          Math::mma(a, Math::load_t<1>(Ks + (32 * rb + 8 * j) * LD, LD, 0, lane, 32 * b + 4 * t, 8), B[rb]);
        }
        S.t[b][t] = a;
      }
  }
  if (on && col_ok && p.dS0) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 32 * b + 8 * j + 4 * t + r;
          if (row < p.K) p.dS0[state + row * p.V] = S.t[b][t][r];
        }
  }
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
  __shared__ __attribute__((aligned(16))) E Ks[C * LD];
  __shared__ __attribute__((aligned(16))) E Qs[C * LD];
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
  stage_rows<Math, KP, C, LD, THREADS>(Ks, static_cast<const E*>(p.k) + at, p.Hk * p.K, ch.n, (int)p.K, p.vec_k, tid);
  stage_rows<Math, KP, C, LD, THREADS>(Qs, static_cast<const E*>(p.q) + at, p.Hk * p.K, ch.n, (int)p.K, p.vec_k, tid);
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
    for (int64_t v0 = 0; v0 < p.VP; v0 += VB) {
      __syncthreads();  // ev is there; the previous columns have been used
      for (int u = tid; u < C * VB / 8; u += THREADS) {
        const int row = u / (VB / 8), c = (u % (VB / 8)) * 8;
        const E* src = static_cast<const E*>(p.do_) + ((ch.row0 + row) * p.H + h) * p.V + v0 + c;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dOs[row * LDV + c + i] = (row < ch.n && v0 + c + i < p.V) ? src[i] : E(0);
        f32x4 a = zero4(), b = zero4(), d = zero4(), e = zero4();
        if (v0 + c < p.VP) {
          const int64_t w = (sh * C + row) * p.VP + v0 + c;
          a = *reinterpret_cast<const f32x4*>(p.dV + w);
          b = *reinterpret_cast<const f32x4*>(p.dV + w + 4);
          d = *reinterpret_cast<const f32x4*>(p.E + w) * ev[2 * C + row];
          e = *reinterpret_cast<const f32x4*>(p.E + w + 4) * ev[2 * C + row];
        }
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
            const auto B = Math::load<1>(Ks + (16 * m + n) * LD + 32 * b + 8 * j, 0);
            Math::mma(qk, Math::load<1>(Qs + (16 * wave + n) * LD + 32 * b + 8 * j, 0), B);
            Math::mma(kk, Math::load<1>(Ks + (16 * wave + n) * LD + 32 * b + 8 * j, 0), B);
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
          const auto kt = Math::load_t<1>(Ks + (32 * b + 8 * j) * LD, LD, 0, lane, 16 * (tile0 + t), 4);
          const auto qt = Math::load_t<1>(Qs + (32 * b + 8 * j) * LD, LD, 0, lane, 16 * (tile0 + t), 4);
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
