// Layer norm over the last dimension (gfx950), forward and backward.
//   y  = (x - mean) rstd w + b,  rstd = 1 / sqrt(var + eps), var = mean of (x - mean)^2
//   dx = rstd (u - mean(u) - xh mean(u xh)),  u = dy w, xh = (x - mean) rstd
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both passes are bound by HBM: x is read once and y written once (forward), x and dy read once
// and dx written once (backward).  A row is held in the registers of T threads, NV pieces of
// VEC elements each, so mean and variance are two exact passes over registers; T is the
// smallest of 4, 16, 64 and 256 that needs at most 4 pieces (256 threads take up to 16), which
// keeps lanes busy on short rows.  The backward walks rows with a fixed grid: every thread owns
// its columns and keeps their dw and db sums in registers over all rows of its workgroup; the
// workgroups' sums are joined by a second kernel in a fixed order.  Longer rows are walked in
// loops over memory.  16384 x 4096 bf16: forward 56 us (4.8 TB/s), backward 81 us with its join
// (5.0 TB/s); a copy reaches 5.15 TB/s.
#include <type_traits>

#include "ops_delta.hpp"

namespace msm {

NormShape norm_shape(int64_t D, int per) {
  for (int T = 4; T <= 64; T *= 4)
    for (int NV = 1; NV <= 4; NV *= 2)
      if (D <= (int64_t)T * per * NV) return NormShape{T, NV};
  for (int NV = 2; NV <= 16; NV *= 2)
    if (D <= (int64_t)256 * per * NV) return NormShape{256, NV};
  return NormShape{256, 0};
}

namespace {

// Workgroups of the forward: eight for every CU, more than its registers hold at once.
constexpr int64_t kNormGroups = 2048;

// Sum over the T threads of a row, the same value in each of them.
// With 256 threads the sum of each wavefront passes through `lds`, which the next sum must not be
// (a later one may: a thread that writes there has passed the barrier in between).
template <int T>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  constexpr int W = T < 64 ? T : 64;
#pragma unroll
  for (int m = W / 2; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  if constexpr (T == 256) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  }
  return v;
}
template <int T>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* lds) {
  constexpr int W = T < 64 ? T : 64;
#pragma unroll
  for (int m = W / 2; m > 0; m >>= 1) {
    a += __shfl_xor(a, m, 64);
    b += __shfl_xor(b, m, 64);
  }
  if constexpr (T == 256) {
    if ((threadIdx.x & 63) == 0) {
      lds[(threadIdx.x >> 6) & 3] = a;
      lds[4 + ((threadIdx.x >> 6) & 3)] = b;
    }
    __syncthreads();
    a = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    b = (lds[4] + lds[5]) + (lds[6] + lds[7]);
  }
}

// VEC elements between their load and their use.
template <typename IO, int VEC>
struct Piece {
  std::conditional_t<VEC == 1, typename io<IO>::raw, u32x4> raw;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (VEC == 1)
      raw = io<IO>::load(p, i);
    else
      raw = *reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + i * io<IO>::es);
  }
  __device__ __forceinline__ void zero() { raw = {}; }
  __device__ __forceinline__ void get(float (&x)[VEC]) const {
    if constexpr (VEC == 1) {
      x[0] = io<IO>::widen(raw);
    } else if constexpr (io<IO>::es == 2) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[2 * c] = __uint_as_float(raw[c] << 16);
        x[2 * c + 1] = __uint_as_float(raw[c] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = __uint_as_float(raw[c]);
    }
  }
};
template <typename IO, int VEC>
__device__ __forceinline__ void store_piece(void* p, int64_t i, const float (&x)[VEC]) {
  using T = io<IO>;
  if constexpr (VEC == 1) {
    T::store(p, i, x[0]);
  } else if constexpr (T::es == 2) {
    u32x4 w;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x[2 * c]));
      const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x[2 * c + 1]));
      w[c] = lo | (hi << 16);
    }
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = w;
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i) = f32x4{x[0], x[1], x[2], x[3]};
  }
}
// fp32 parameters of a piece (vector loads: their address is a multiple of VEC elements)
template <int VEC>
__device__ __forceinline__ void load_param(const float* p, int64_t i, float other, float (&x)[VEC]) {
#pragma unroll
  for (int c = 0; c < VEC; ++c) x[c] = p ? p[i + c] : other;
}

// A workgroup walks several rows with its columns' weight and bias in registers: read again for
// every row they would be four times the bytes of a bf16 row.  The next row's loads are issued
// before the present one is reduced.
template <typename IO, int VEC, int T, int NV>
__global__ __launch_bounds__(256) void norm_fwd_kernel(const NormArgs p) {
  __shared__ float lds[8];
  constexpr int RW = 256 / T;  // rows in flight
  const int t = threadIdx.x % T;
  const int64_t step = (int64_t)gridDim.x * RW;
  int64_t row = (int64_t)blockIdx.x * RW + threadIdx.x / T;
  if (row >= p.rows) return;  // whole groups of T lanes (for T = 256 the workgroup): no sum crosses groups
  float w[NV][VEC], b[NV][VEC];
  Piece<IO, VEC> next[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = ((int64_t)i * T + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[i][e] = b[i][e] = 0.f;
    next[i].zero();
    if (c < p.D) {
      load_param<VEC>(p.weight, c, 1.f, w[i]);
      load_param<VEC>(p.bias, c, 0.f, b[i]);
      next[i].load(p.x, row * p.D + c);
    }
  }
  const float inv = 1.f / (float)p.D;
  for (; row < p.rows; row += step) {
    float x[NV][VEC];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * T + t) * VEC;
      next[i].get(x[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum += x[i][e];
      if (c < p.D && row + step < p.rows) next[i].load(p.x, (row + step) * p.D + c);
    }
    const float mean = row_sum<T>(sum, lds) * inv;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * T + t) * VEC;
      if (c < p.D)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x[i][e] -= mean;
          sq = fmaf(x[i][e], x[i][e], sq);
        }
    }
    const float rstd = 1.f / sqrtf(row_sum<T>(sq, lds + 4) * inv + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * T + t) * VEC;
      if (c < p.D) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[i][e] = fmaf(x[i][e] * rstd, w[i][e], b[i][e]);
        store_piece<IO, VEC>(p.y, row * p.D + c, x[i]);
      }
    }
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
}

// Sum over a workgroup, the same value in each thread.  `lds` must not be the next sum's.
__device__ __forceinline__ double wide_sum(double v, double* lds) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// Workgroups of a walk over rows: 2^24 of 256 threads would be 2^32 threads, more than a launch has.
constexpr int64_t kLoopGroups = (int64_t)1 << 20;

// Rows too long for the registers, or too long to be held in pieces of one element: three walks over
// a row, the later ones from cache.  A thread's own sum has up to D / 256 terms, 2^22 of them, so the
// sums are fp64: in fp32 the roundings of equal terms all go one way (the mean of 2^22 times 1.1 was
// off by 1e-4).
template <typename IO>
__global__ __launch_bounds__(256) void norm_fwd_loop_kernel(const NormArgs p) {
  using T = io<IO>;
  __shared__ double lds[8];
  const double inv = 1. / (double)p.D;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t at = row * p.D;
    double sum = 0;
    for (int64_t c = threadIdx.x; c < p.D; c += 256) sum += (double)T::widen(T::load(p.x, at + c));
    const float mean = (float)(wide_sum(sum, lds) * inv);
    double sq = 0;
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      const double d = T::widen(T::load(p.x, at + c)) - mean;
      sq = fma(d, d, sq);
    }
    const float rstd = 1.f / sqrtf((float)(wide_sum(sq, lds + 4) * inv) + p.eps);
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      const float d = (T::widen(T::load(p.x, at + c)) - mean) * rstd;
      T::store(p.y, at + c, fmaf(d, p.weight ? p.weight[c] : 1.f, p.bias ? p.bias[c] : 0.f));
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
}

// BS threads, BS / T rows in flight.  The rows' pieces of x and dy are fetched one row ahead.  At
// the end the workgroup joins its threads' column sums and leaves one pair of D sums.
template <typename IO, int VEC, int T, int NV, int BS>
__global__ __launch_bounds__(BS) void norm_bwd_kernel(const NormArgs p) {
  constexpr int RW = BS / T;
  constexpr int kGroup = T > 64 ? T : 64;  // threads whose column sums a wavefront (or row) has joined
  constexpr int NG = BS / kGroup;
  __shared__ float lds[2][T == 256 ? RW : 1][8];
  int turn = 0;
  __shared__ float cols[NG > 1 ? NG : 1][NG > 1 ? T * VEC : 1];
  const int t = threadIdx.x % T, rg = threadIdx.x / T;
  const float inv = 1.f / (float)p.D;
  const int64_t step = (int64_t)gridDim.x * RW;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
  Piece<IO, VEC> nx[NV], ny[NV];
  int64_t row = (int64_t)blockIdx.x * RW + rg;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = ((int64_t)i * T + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[i][e] = dw[i][e] = db[i][e] = 0.f;
    nx[i].zero();
    ny[i].zero();
    if (c < p.D) {
      load_param<VEC>(p.weight, c, 1.f, w[i]);
      if (row < p.rows) {
        nx[i].load(p.x, row * p.D + c);
        ny[i].load(p.dy, row * p.D + c);
      }
    }
  }
  // every thread takes part in every pass (the sums of a 256-thread row meet at barriers); a row
  // past the end adds nothing
  for (int64_t first = (int64_t)blockIdx.x * RW; first < p.rows; first += step, row += step) {
    const bool on = row < p.rows;
    const float mean = on ? p.mean[row] : 0.f, rstd = on ? p.rstd[row] : 0.f;
    float x[NV][VEC], u[NV][VEC];
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * T + t) * VEC;
      const bool in = on && c < p.D;
      float dy[VEC];
      nx[i].get(x[i]);
      ny[i].get(dy);
      if (c < p.D && row + step < p.rows) {
        nx[i].load(p.x, (row + step) * p.D + c);
        ny[i].load(p.dy, (row + step) * p.D + c);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x[i][e] = in ? (x[i][e] - mean) * rstd : 0.f;
        dy[e] = in ? dy[e] : 0.f;
        u[i][e] = dy[e] * w[i][e];
        a += u[i][e];
        b = fmaf(u[i][e], x[i][e], b);
        dw[i][e] = fmaf(dy[e], x[i][e], dw[i][e]);
        db[i][e] += dy[e];
      }
    }
    row_sum2<T>(a, b, lds[turn][T == 256 ? rg : 0]);
    turn ^= 1;
    a *= inv;
    b *= inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * T + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[i][e] = rstd * (u[i][e] - a - x[i][e] * b);
      if (on && c < p.D) store_piece<IO, VEC>(p.dx, row * p.D + c, x[i]);
    }
  }
  if (!p.part) return;
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float(&v)[VEC] = which ? db[i] : dw[i];
#pragma unroll
      for (int e = 0; e < VEC; ++e)
#pragma unroll
        for (int m = T; m < 64; m *= 2) v[e] += __shfl_xor(v[e], m, 64);
      if constexpr (NG > 1) {
        __syncthreads();  // the last round has been read
        if (T >= 64 || (threadIdx.x & 63) < T)
#pragma unroll
          for (int e = 0; e < VEC; ++e) cols[threadIdx.x / kGroup][t * VEC + e] = v[e];
        __syncthreads();
        for (int k = threadIdx.x; k < T * VEC; k += BS) {
          float s = 0.f;
#pragma unroll
          for (int g = 0; g < NG; ++g) s += cols[g][k];
          const int64_t c = (int64_t)i * T * VEC + k;
          if (c < p.D) part[which * p.D + c] = s;
        }
      } else {
        const int64_t c = ((int64_t)i * T + t) * VEC;
        if (c < p.D)
#pragma unroll
          for (int e = 0; e < VEC; ++e) part[which * p.D + c + e] = v[e];
      }
    }
  }
}

template <typename IO>
__global__ __launch_bounds__(256) void norm_bwd_loop_kernel(const NormArgs p) {
  using T = io<IO>;
  __shared__ double lds[8];
  const double inv = 1. / (double)p.D;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t at = row * p.D;
    const float mean = p.mean[row], rstd = p.rstd[row];
    double sa = 0, sb = 0;  // fp64 as in the forward
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      const float u = T::widen(T::load(p.dy, at + c)) * (p.weight ? p.weight[c] : 1.f);
      sa += (double)u;
      sb = fma((double)u, (double)((T::widen(T::load(p.x, at + c)) - mean) * rstd), sb);
    }
    const float a = (float)(wide_sum(sa, lds) * inv), b = (float)(wide_sum(sb, lds + 4) * inv);
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      const float u = T::widen(T::load(p.dy, at + c)) * (p.weight ? p.weight[c] : 1.f);
      const float xh = (T::widen(T::load(p.x, at + c)) - mean) * rstd;
      T::store(p.dx, at + c, rstd * (u - a - xh * b));
    }
  }
}

// Column sums of the rows of a group, for rows that the loop kernel walked: a thread per column, in
// fp64 as a group may have millions of rows.
template <typename IO>
__global__ __launch_bounds__(256) void norm_cols_kernel(const NormArgs p) {
  using T = io<IO>;
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.D) return;
  double dw = 0, db = 0;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float dy = T::widen(T::load(p.dy, row * p.D + c));
    dw = fma((double)dy, (double)((T::widen(T::load(p.x, row * p.D + c)) - p.mean[row]) * p.rstd[row]), dw);
    db += (double)dy;
  }
  p.part[(int64_t)blockIdx.y * 2 * p.D + c] = (float)dw;
  p.part[(int64_t)blockIdx.y * 2 * p.D + p.D + c] = (float)db;
}

// Joins the column sums of all parts in fp64: CL columns a workgroup, 256 / CL threads a column.
template <int CL>
__global__ __launch_bounds__(256) void norm_join_kernel(const NormArgs p, int64_t parts) {
  __shared__ double lds[2][256];
  constexpr int TH = 256 / CL;
  const int cl = threadIdx.x % CL, k = threadIdx.x / CL;
  const int64_t c = (int64_t)blockIdx.x * CL + cl;
  double dw = 0, db = 0;
  if (c < p.D)
    for (int64_t g = k; g < parts; g += TH) {
      dw += p.part[g * 2 * p.D + c];
      db += p.part[g * 2 * p.D + p.D + c];
    }
  lds[0][threadIdx.x] = dw;
  lds[1][threadIdx.x] = db;
#pragma unroll
  for (int h = TH / 2; h > 0; h /= 2) {
    __syncthreads();
    if (k < h) {
      lds[0][threadIdx.x] += lds[0][threadIdx.x + h * CL];
      lds[1][threadIdx.x] += lds[1][threadIdx.x + h * CL];
    }
  }
  if (k == 0 && c < p.D) {
    if (p.dweight) p.dweight[c] = (float)lds[0][threadIdx.x];
    if (p.dbias) p.dbias[c] = (float)lds[1][threadIdx.x];
  }
}

// Fewer columns a workgroup while that takes more of them to fill the GPU; for the widest rows a
// thread a column, as D / 16 workgroups of 256 would pass the 2^32 threads of a launch.
hipError_t join(const NormArgs& a, int64_t parts, hipStream_t s) {
  if (a.D >= (1 << 22))
    hipLaunchKernelGGL(norm_join_kernel<256>, dim3((unsigned)((a.D + 255) / 256)), dim3(256), 0, s, a, parts);
  else if (a.D >= 4096)
    hipLaunchKernelGGL(norm_join_kernel<16>, dim3((unsigned)((a.D + 15) / 16)), dim3(256), 0, s, a, parts);
  else
    hipLaunchKernelGGL(norm_join_kernel<4>, dim3((unsigned)((a.D + 3) / 4)), dim3(256), 0, s, a, parts);
  return hipGetLastError();
}

template <typename IO, int VEC, int T, int NV>
hipError_t go_fwd(const NormArgs& a, hipStream_t s) {
  const int64_t all = (a.rows + 256 / T - 1) / (256 / T);
  const dim3 grid((unsigned)(all < kNormGroups ? all : kNormGroups));
  hipLaunchKernelGGL((norm_fwd_kernel<IO, VEC, T, NV>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}
template <typename IO, int VEC, int T, int NV>
hipError_t go_bwd(const NormArgs& a, hipStream_t s) {
  constexpr int BS = norm_threads(T, NV);
  hipLaunchKernelGGL((norm_bwd_kernel<IO, VEC, T, NV, BS>), dim3((unsigned)a.groups), dim3(BS), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  return join(a, a.groups, s);
}

template <typename IO, int VEC, bool BWD>
hipError_t pick(const NormArgs& a, hipStream_t s) {
  const NormShape f = norm_shape(a.D, VEC);
#define MSM_NORM(TT, NN) \
  if (f.T == TT && f.NV == NN) return BWD ? go_bwd<IO, VEC, TT, NN>(a, s) : go_fwd<IO, VEC, TT, NN>(a, s);
  MSM_NORM(4, 1) MSM_NORM(4, 2) MSM_NORM(4, 4) MSM_NORM(16, 2) MSM_NORM(16, 4) MSM_NORM(64, 2)
  MSM_NORM(64, 4) MSM_NORM(256, 2) MSM_NORM(256, 4) MSM_NORM(256, 8) MSM_NORM(256, 16)
#undef MSM_NORM
  const dim3 grid((unsigned)(a.rows < kLoopGroups ? a.rows : kLoopGroups));
  if (!BWD) {
    hipLaunchKernelGGL((norm_fwd_loop_kernel<IO>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((norm_bwd_loop_kernel<IO>), grid, dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  hipLaunchKernelGGL((norm_cols_kernel<IO>), dim3((unsigned)((a.D + 255) / 256), (unsigned)a.groups),
                     dim3(256), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  return join(a, a.groups, s);
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, int io_bf16, hipStream_t s) {
  if (io_bf16) return a.vec ? pick<bf16_storage, 8, false>(a, s) : pick<bf16_storage, 1, false>(a, s);
  return a.vec ? pick<float, 4, false>(a, s) : pick<float, 1, false>(a, s);
}
hipError_t launch_norm_bwd(const NormArgs& a, int io_bf16, hipStream_t s) {
  if (io_bf16) return a.vec ? pick<bf16_storage, 8, true>(a, s) : pick<bf16_storage, 1, true>(a, s);
  return a.vec ? pick<float, 4, true>(a, s) : pick<float, 1, true>(a, s);
}

}  // namespace msm
