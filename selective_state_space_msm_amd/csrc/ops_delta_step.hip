// One token of the gated delta rule for a batch of sequences (gfx950):
//   e = v - a S^T k,  S <- a S + beta k e^T,  o = scale S^T q,  a = exp(g),
// with the states (Bt, H, K, V), fp32, updated in place.
//
// Every state element is read and written once and enters four multiply-adds: the step is bound
// by HBM.  Both readings of the old state are taken in one pass, since
//   o = scale (a S_old^T q + (k . q) beta e),
// so a workgroup loads its K x (LC VEC) columns once into registers, forms the partial sums of
// S^T k and S^T q over its rows, joins them through LDS, and writes the new state from the
// registers.  LC lanes share a row of the tile with 16-byte loads (VEC = 4); V that is not a
// multiple of 4, or unaligned states, take one column per lane.  256 sequences, H=32, K=V=128 (1.08 GB):
// 203 us, 5.3 TB/s, what a copy reaches; one sequence, H=16: 4.4 us, a launch's length.
#include "ops_delta.hpp"

namespace msm {
namespace {

template <typename IO, int VEC, int LC, int RPT>
__global__ __launch_bounds__(256) void delta_step_kernel(const DeltaStepArgs p, int64_t first) {
  using T = io<IO>;
  constexpr int RG = 256 / LC;          // rows of the tile in flight; row = rg + RG i
  __shared__ float ks[RG * RPT], qs[RG * RPT];
  __shared__ float part[4][2][LC * VEC];
  __shared__ float kq[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cl = tid % LC, rg = tid / LC;
  const int64_t bh = first + blockIdx.x, b = bh / p.H, h = bh - b * p.H, hk = h / (p.H / p.Hk);
  const int64_t col = ((int64_t)blockIdx.y * LC + cl) * VEC;
  const bool on = col < p.V;
  const int K = (int)p.K;
  float* S = p.S + bh * p.K * p.V + col;

  float st[RPT][VEC];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int row = rg + RG * i;
#pragma unroll
    for (int c = 0; c < VEC; ++c) st[i][c] = 0.f;
    if (on && row < K) {
      if constexpr (VEC == 4) {
        const f32x4 x = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + row * p.V));
#pragma unroll
        for (int c = 0; c < VEC; ++c) st[i][c] = x[c];
      } else {
        st[i][0] = S[row * p.V];
      }
    }
  }
  float prod = 0.f;
  for (int i = tid; i < RG * RPT; i += 256) {
    const bool in = i < K;
    const float kv = in ? T::widen(T::load(p.k, (b * p.Hk + hk) * p.K + i)) : 0.f;
    const float qv = in ? T::widen(T::load(p.q, (b * p.Hk + hk) * p.K + i)) : 0.f;
    ks[i] = kv;
    qs[i] = qv;
    prod = fmaf(kv, qv, prod);
  }
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) prod += __shfl_xor(prod, m, 64);
  if (lane == 0) kq[wave] = prod;
  const float a = exp2_fast(p.g[bh] * kLog2e), beta = p.beta[bh];
  float v[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) v[c] = on ? T::widen(T::load(p.v, bh * p.V + col + c)) : 0.f;
  __syncthreads();
  float sk[VEC], sq[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) sk[c] = sq[c] = 0.f;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const float kv = ks[rg + RG * i], qv = qs[rg + RG * i];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      sk[c] = fmaf(kv, st[i][c], sk[c]);
      sq[c] = fmaf(qv, st[i][c], sq[c]);
    }
  }
#pragma unroll
  for (int m = LC; m < 64; m *= 2)
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      sk[c] += __shfl_xor(sk[c], m, 64);
      sq[c] += __shfl_xor(sq[c], m, 64);
    }
  if (lane < LC)
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      part[wave][0][cl * VEC + c] = sk[c];
      part[wave][1][cl * VEC + c] = sq[c];
    }
  __syncthreads();
  const float dot = (kq[0] + kq[1]) + (kq[2] + kq[3]);
  float w[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    const int x = cl * VEC + c;
    const float pk = (part[0][0][x] + part[1][0][x]) + (part[2][0][x] + part[3][0][x]);
    const float pq = (part[0][1][x] + part[1][1][x]) + (part[2][1][x] + part[3][1][x]);
    w[c] = beta * fmaf(-a, pk, v[c]);
    if (on && rg == 0) T::store(p.o, bh * p.V + col + c, p.scale * fmaf(a, pq, dot * w[c]));
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int row = rg + RG * i;
    if (on && row < K) {
      const float kv = ks[row];
      if constexpr (VEC == 4) {
        f32x4 x;
#pragma unroll
        for (int c = 0; c < VEC; ++c) x[c] = fmaf(kv, w[c], a * st[i][c]);
        __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(S + row * p.V));
      } else {
        S[row * p.V] = fmaf(kv, w[0], a * st[i][0]);
      }
    }
  }
}

template <typename IO, int VEC, int LC, int RPT>
hipError_t go(const DeltaStepArgs& a, hipStream_t s) {
  // 2^24 workgroups of 256 would be 2^32 threads, more than a dimension of a launch may have
  constexpr int64_t kMost = (int64_t)1 << 23;
  for (int64_t first = 0, all = a.Bt * a.H; first < all; first += kMost) {
    const int64_t left = all - first;
    const dim3 grid((unsigned)(left < kMost ? left : kMost), (unsigned)((a.V + LC * VEC - 1) / (LC * VEC)));
    hipLaunchKernelGGL((delta_step_kernel<IO, VEC, LC, RPT>), grid, dim3(256), 0, s, a, first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename IO, int VEC>
hipError_t pick(const DeltaStepArgs& a, hipStream_t s) {
  // 8 lanes a row (128-byte pieces) while 16 would leave CUs without a workgroup
  const int64_t wide = a.Bt * a.H * ((a.V + 16 * VEC - 1) / (16 * VEC));
  if (wide < 512) {
    if (a.K <= 64) return go<IO, VEC, 8, 2>(a, s);
    if (a.K <= 128) return go<IO, VEC, 8, 4>(a, s);
    return go<IO, VEC, 8, 8>(a, s);
  }
  if (a.K <= 64) return go<IO, VEC, 16, 4>(a, s);
  if (a.K <= 128) return go<IO, VEC, 16, 8>(a, s);
  return go<IO, VEC, 16, 16>(a, s);
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepArgs& a, int io_bf16, hipStream_t s) {
  const bool vec = a.V % 4 == 0 && ((uintptr_t)a.S & 15) == 0;
  if (io_bf16) return vec ? pick<bf16_storage, 4>(a, s) : pick<bf16_storage, 1>(a, s);
  return vec ? pick<float, 4>(a, s) : pick<float, 1>(a, s);
}

}  // namespace msm
