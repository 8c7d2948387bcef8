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
// loops over memory.  16384 x 4096 bf16: forward 56 us (4.8 TB/s), backward 79 us with its join
// (5.1 TB/s); a copy reaches 5.15 TB/s.
#include "ops_row.hpp"

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

// Joins the column sums of all parts in fp64: CL columns a workgroup, 256 / CL threads a column, eight
// parts of each in flight.  An XCD has columns side by side, so that a line of a part is in one L2, not in
// several.  (1000 parts of 2048 columns: 8.5 us, one part at a time and workgroups round the XCDs 22.)
template <int CL>
__global__ __launch_bounds__(256) void norm_join_kernel(const NormArgs p, int64_t parts) {
  __shared__ double lds[2][256];
  constexpr int TH = 256 / CL;
  const int cl = threadIdx.x % CL, k = threadIdx.x / CL;
  const int64_t c = ((int64_t)(blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8) * CL + cl;
  double dw = 0, db = 0;
  if (c < p.D) {
    int64_t g = k;
    for (; g + 7 * TH < parts; g += 8 * TH) {
      float w[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] = p.part[(g + i * TH) * 2 * p.D + c];
        b[i] = p.part[(g + i * TH) * 2 * p.D + p.D + c];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw += w[i];
        db += b[i];
      }
    }
    for (; g < parts; g += TH) {
      dw += p.part[g * 2 * p.D + c];
      db += p.part[g * 2 * p.D + p.D + c];
    }
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

}  // namespace

// Fewer columns a workgroup while that takes more of them to fill the GPU; for the widest rows a
// thread a column, as D / 16 workgroups of 256 would pass the 2^32 threads of a launch.
hipError_t launch_norm_join(const NormArgs& a, int64_t parts, hipStream_t s) {
  const int64_t cl = a.D >= (1 << 22) ? 256 : (a.D >= 4096 ? 16 : 4);
  const dim3 grid((unsigned)((a.D + 8 * cl - 1) / (8 * cl) * 8));  // as many on each XCD
  if (cl == 256)
    hipLaunchKernelGGL(norm_join_kernel<256>, grid, dim3(256), 0, s, a, parts);
  else if (cl == 16)
    hipLaunchKernelGGL(norm_join_kernel<16>, grid, dim3(256), 0, s, a, parts);
  else
    hipLaunchKernelGGL(norm_join_kernel<4>, grid, dim3(256), 0, s, a, parts);
  return hipGetLastError();
}

namespace {

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
  return launch_norm_join(a, a.groups, s);
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
  return launch_norm_join(a, a.groups, s);
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
