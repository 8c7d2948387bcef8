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
// loops over memory.
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
template <int T>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  constexpr int W = T < 64 ? T : 64;
#pragma unroll
  for (int m = W / 2; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  if constexpr (T == 256) {
    __syncthreads();  // the previous sum has been read
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
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
      lds[threadIdx.x >> 6] = a;
      lds[4 + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    a = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    b = (lds[4] + lds[5]) + (lds[6] + lds[7]);
  }
}

template <typename IO, int VEC>
__device__ __forceinline__ void load_piece(const void* p, int64_t i, float (&x)[VEC]) {
  using T = io<IO>;
  if constexpr (VEC == 1) {
    x[0] = T::widen(T::load(p, i));
  } else if constexpr (T::es == 2) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[2 * c] = __uint_as_float(w[c] << 16);
      x[2 * c + 1] = __uint_as_float(w[c] & 0xffff0000u);
    }
  } else {
    const f32x4 w = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = w[c];
  }
}
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
  float w[NV][VEC], b[NV][VEC], next[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = ((int64_t)i * T + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) next[i][e] = w[i][e] = b[i][e] = 0.f;
    if (c < p.D) {
      load_param<VEC>(p.weight, c, 1.f, w[i]);
      load_param<VEC>(p.bias, c, 0.f, b[i]);
      load_piece<IO, VEC>(p.x, row * p.D + c, next[i]);
    }
  }
  const float inv = 1.f / (float)p.D;
  for (; row < p.rows; row += step) {
    float x[NV][VEC];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * T + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x[i][e] = next[i][e];
        sum += x[i][e];
      }
      if (c < p.D && row + step < p.rows) load_piece<IO, VEC>(p.x, (row + step) * p.D + c, next[i]);
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
    const float rstd = 1.f / sqrtf(row_sum<T>(sq, lds) * inv + p.eps);
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

// Rows too long for the registers: three walks over the row, the later ones from cache.
template <typename IO>
__global__ __launch_bounds__(256) void norm_fwd_loop_kernel(const NormArgs p) {
  using T = io<IO>;
  __shared__ float lds[8];
  const int64_t at = (int64_t)blockIdx.x * p.D;
  float sum = 0.f;
  for (int64_t c = threadIdx.x; c < p.D; c += 256) sum += T::widen(T::load(p.x, at + c));
  const float inv = 1.f / (float)p.D;
  const float mean = row_sum<256>(sum, lds) * inv;
  float sq = 0.f;
  for (int64_t c = threadIdx.x; c < p.D; c += 256) {
    const float d = T::widen(T::load(p.x, at + c)) - mean;
    sq = fmaf(d, d, sq);
  }
  const float rstd = 1.f / sqrtf(row_sum<256>(sq, lds) * inv + p.eps);
  for (int64_t c = threadIdx.x; c < p.D; c += 256) {
    const float d = (T::widen(T::load(p.x, at + c)) - mean) * rstd;
    T::store(p.y, at + c, fmaf(d, p.weight ? p.weight[c] : 1.f, p.bias ? p.bias[c] : 0.f));
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[blockIdx.x] = mean;
    if (p.rstd) p.rstd[blockIdx.x] = rstd;
  }
}

template <typename IO, int VEC, int T, int NV>
__global__ __launch_bounds__(256) void norm_bwd_kernel(const NormArgs p) {
  __shared__ float lds[8];
  constexpr int RW = 256 / T;  // rows in flight in the workgroup
  const int t = threadIdx.x % T, rg = threadIdx.x / T;
  const float inv = 1.f / (float)p.D;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = ((int64_t)i * T + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[i][e] = dw[i][e] = db[i][e] = 0.f;
    if (c < p.D) load_param<VEC>(p.weight, c, 1.f, w[i]);
  }
  for (int64_t row = (int64_t)blockIdx.x * RW + rg; row < p.rows; row += (int64_t)gridDim.x * RW) {
    float x[NV][VEC], dy[NV][VEC];
    const float mean = p.mean[row], rstd = p.rstd[row];
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * T + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x[i][e] = mean;
        dy[i][e] = 0.f;
      }
      if (c < p.D) {
        load_piece<IO, VEC>(p.x, row * p.D + c, x[i]);
        load_piece<IO, VEC>(p.dy, row * p.D + c, dy[i]);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x[i][e] = (x[i][e] - mean) * rstd;
        const float u = dy[i][e] * w[i][e];
        a += u;
        b = fmaf(u, x[i][e], b);
        dw[i][e] = fmaf(dy[i][e], x[i][e], dw[i][e]);
        db[i][e] += dy[i][e];
      }
    }
    row_sum2<T>(a, b, lds);
    a *= inv;
    b *= inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * T + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[i][e] = rstd * (fmaf(dy[i][e], w[i][e], -a) - x[i][e] * b);
      if (c < p.D) store_piece<IO, VEC>(p.dx, row * p.D + c, x[i]);
    }
  }
  if (!p.part) return;
  // one pair of column sums a wavefront, or a workgroup when its rows are that wide
  constexpr int PW = T == 256 ? 1 : 4;
  float* part = p.part + ((int64_t)blockIdx.x * PW + (T == 256 ? 0 : threadIdx.x >> 6)) * 2 * p.D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = ((int64_t)i * T + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e)
#pragma unroll
      for (int m = T; m < 64; m *= 2) {
        dw[i][e] += __shfl_xor(dw[i][e], m, 64);
        db[i][e] += __shfl_xor(db[i][e], m, 64);
      }
    if (c < p.D && (T >= 64 || (threadIdx.x & 63) < T))
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        part[c + e] = dw[i][e];
        part[p.D + c + e] = db[i][e];
      }
  }
}

template <typename IO>
__global__ __launch_bounds__(256) void norm_bwd_loop_kernel(const NormArgs p) {
  using T = io<IO>;
  __shared__ float lds[8];
  const float inv = 1.f / (float)p.D;
  const int64_t at = (int64_t)blockIdx.x * p.D;
  const float mean = p.mean[blockIdx.x], rstd = p.rstd[blockIdx.x];
  float a = 0.f, b = 0.f;
  for (int64_t c = threadIdx.x; c < p.D; c += 256) {
    const float u = T::widen(T::load(p.dy, at + c)) * (p.weight ? p.weight[c] : 1.f);
    a += u;
    b = fmaf(u, (T::widen(T::load(p.x, at + c)) - mean) * rstd, b);
  }
  row_sum2<256>(a, b, lds);
  a *= inv;
  b *= inv;
  for (int64_t c = threadIdx.x; c < p.D; c += 256) {
    const float u = T::widen(T::load(p.dy, at + c)) * (p.weight ? p.weight[c] : 1.f);
    const float xh = (T::widen(T::load(p.x, at + c)) - mean) * rstd;
    T::store(p.dx, at + c, rstd * (u - a - xh * b));
  }
}

// Column sums of the rows of a group, for rows that the loop kernel walked: a thread per column.
template <typename IO>
__global__ __launch_bounds__(256) void norm_cols_kernel(const NormArgs p) {
  using T = io<IO>;
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.D) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float dy = T::widen(T::load(p.dy, row * p.D + c));
    dw = fmaf(dy, (T::widen(T::load(p.x, row * p.D + c)) - p.mean[row]) * p.rstd[row], dw);
    db += dy;
  }
  p.part[(int64_t)blockIdx.y * 2 * p.D + c] = dw;
  p.part[(int64_t)blockIdx.y * 2 * p.D + p.D + c] = db;
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

hipError_t join(const NormArgs& a, int64_t parts, hipStream_t s) {
  if (a.D >= 4096)
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
  hipLaunchKernelGGL((norm_bwd_kernel<IO, VEC, T, NV>), dim3((unsigned)a.groups), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  return join(a, (int64_t)a.groups * (T == 256 ? 1 : 4), s);
}

template <typename IO, int VEC, bool BWD>
hipError_t pick(const NormArgs& a, hipStream_t s) {
  const NormShape f = norm_shape(a.D, VEC);
#define MSM_NORM(TT, NN) \
  if (f.T == TT && f.NV == NN) return BWD ? go_bwd<IO, VEC, TT, NN>(a, s) : go_fwd<IO, VEC, TT, NN>(a, s);
  MSM_NORM(4, 1) MSM_NORM(4, 2) MSM_NORM(4, 4) MSM_NORM(16, 2) MSM_NORM(16, 4) MSM_NORM(64, 2)
  MSM_NORM(64, 4) MSM_NORM(256, 2) MSM_NORM(256, 4) MSM_NORM(256, 8) MSM_NORM(256, 16)
#undef MSM_NORM
  if (!BWD) {
    hipLaunchKernelGGL((norm_fwd_loop_kernel<IO>), dim3((unsigned)a.rows), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((norm_bwd_loop_kernel<IO>), dim3((unsigned)a.rows), dim3(256), 0, s, a);
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
