// The norms after a block and before the next one, fused with the block's gate, its residual
// scale and the residual sum (gfx950), forward and backward.
//   q = 1 / sqrt(mean(o^2) + eps),  oh = o q,  a = oh pw
//   r' = r + scale a silu(z)                    (held in the I/O type; without o, r' = r)
//   p = 1 / sqrt(mean(r'^2) + eps),  rh = r' p,  y = rh w
//   u = dy w,        G  = dr' + p (u - rh mean(u rh)) = dr,          dw  = sum over rows of dy rh
//   c = scale G silu(z),  v = c pw,  do = q (v - oh mean(v oh)),     dpw = sum over rows of c oh
//   dz = scale G a silu'(z)
//
// Both passes are bound by HBM: o, z, r read and r', y written (forward), o, z, r', dy, dr' read
// and dr, do, dz written (backward), each once.  A row lives in the registers of T threads, E
// elements each, and the next row's loads are issued before the present one is reduced.  A piece
// of a row is 16 bytes also where rows begin at odd addresses (the hardware takes unaligned
// 16-byte accesses); only a row's last piece may be taken element by element.  The backward's
// column sums stay in registers over 64 rows of a thread, in LDS over the others, and the workgroups'
// are joined by a second kernel in a fixed order.  Rows past the registers are walked in memory with fp64 sums.
// 16384 x 4096, bf16, with block and gate: forward 134 us (5.0 TB/s), backward 206 to 210 (5.2 TB/s); a
// copy of 1 GiB reaches 5.1.  4095 x 1001, fp32, no gate: backward 26 us (3.8 TB/s).
#include "lm_internal.h"
#include "ops_internal.h"
#include "ops_row.hpp"

namespace msm {
namespace {

// Sum over the threads of a row, the same value in each: T of them, or (T = 0) the workgroup.  Then `lds`
// must not be the next sum's (the one after it may use it: a thread that writes there has passed the
// barrier in between).
template <int T>
__device__ __forceinline__ float group_sum(float v, float* lds) {
  constexpr int W = T == 0 ? 64 : T;
#pragma unroll
  for (int m = W / 2; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  if constexpr (T == 0) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
    for (unsigned i = 0; i < blockDim.x / 64; ++i) v += lds[i];
  }
  return v;
}

// 1 / sqrt(sum / D + eps), rounded once: what a row's statistic is off by, the whole row is.
__device__ __forceinline__ float rstd_of(double sum, double inv, float eps) {
  return (float)(1. / sqrt(sum * inv + (double)eps));
}

constexpr int64_t kRowGroups = 2048;
// Rows that a thread of the backward adds up in one fp32 sum, before that is added to those of the rows before:
// 1024 rows of equal terms in one sum were off by 9e-6 of it.
constexpr int kRowsOfSum = 64;

// G threads to a row, 256 / G rows a workgroup; G = 0: a row for the workgroup, of up to MOST threads.
template <typename IO, int G, int E, int MOST>
__global__ __launch_bounds__(MOST) void block_norm_fwd_kernel(const BlockNormArgs p) {
  constexpr int VEC = Chunk<IO>::VEC, NV = E / VEC, RW = G == 0 ? 1 : MOST / (G == 0 ? 1 : G);
  __shared__ float lds[2][G == 0 ? MOST / 64 : 1];
  int turn = 0;
  const int T = G == 0 ? blockDim.x : G, t = G == 0 ? threadIdx.x : threadIdx.x % (G == 0 ? 1 : G);
  const int64_t step = (int64_t)gridDim.x * RW;
  int64_t row = (int64_t)blockIdx.x * RW + (G == 0 ? 0 : threadIdx.x / (G == 0 ? 1 : G));
  if (row >= p.rows) return;  // whole rows leave: no sum crosses rows
  float w[NV][VEC], pw[NV][VEC];
  Chunk<IO> no[NV], nz[NV], nr[NV];
  const bool block = p.o != nullptr, gate = p.z != nullptr;
  const auto fetch = [&](int i, int64_t at) {
    const int64_t c = ((int64_t)i * T + t) * VEC, n = p.D - c;
    if (n <= 0) return;
    nr[i].load_row(p.r, at, c, p.D);
    if (block) no[i].load_row(p.o, at, c, p.D);
    if (gate) nz[i].load_row(p.z, at, c, p.D);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = ((int64_t)i * T + t) * VEC;
    nr[i].zero();
    no[i].zero();
    nz[i].zero();
    fetch(i, row * p.D);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = p.weight && c + e < p.D ? p.weight[c + e] : 1.f;
      pw[i][e] = p.post_weight && c + e < p.D ? p.post_weight[c + e] : 1.f;
    }
  }
  const double inv = 1. / (double)p.D;
  for (; row < p.rows; row += step) {
    float x[NV][VEC], f[NV][VEC];
    const int64_t at = row * p.D, next = (row + step) * p.D;
    const bool more = row + step < p.rows;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int by = Chunk<IO>::short_by(((int64_t)i * T + t) * VEC, p.D);
      nr[i].get_row(x[i], by);
      if (block) {
        no[i].get_row(f[i], by);
#pragma unroll
        for (int e = 0; e < VEC; ++e) q = fmaf(f[i][e], f[i][e], q);
        if (gate) {
          float z[VEC];
          nz[i].get_row(z, by);
#pragma unroll
          for (int e = 0; e < VEC; ++e) f[i][e] *= silu_f(z[e]);
        }
      }
      if (more) fetch(i, next);
    }
    if (block) {
      q = rstd_of(group_sum<G>(q, lds[turn]), inv, p.eps);
      turn ^= 1;
      const float qs = q * p.scale;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t c = ((int64_t)i * T + t) * VEC, n = p.D - c;
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[i][e] = fmaf(f[i][e] * qs, pw[i][e], x[i][e]);
        Chunk<IO> held;
        held.set(x[i]);
        held.get(x[i]);
        if (n > 0) held.store(p.r_out, at + c, n);
        // past the row's end the inputs are zero, but a gate of zero keeps them so
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s = fmaf(x[i][e], x[i][e], s);
    const float rstd = rstd_of(group_sum<G>(s, lds[turn]), inv, p.eps);
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = ((int64_t)i * T + t) * VEC, n = p.D - c;
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[i][e] = x[i][e] * rstd * w[i][e];
      Chunk<IO> out;
      out.set(x[i]);
      if (n > 0) out.store(p.y, at + c, n);
    }
    if (t == 0) {
      if (p.rstd) p.rstd[row] = rstd;
      if (p.post_rstd) p.post_rstd[row] = q;
    }
  }
}

template <typename IO, int G, int E, int MOST>
__global__ __launch_bounds__(MOST) void block_norm_bwd_kernel(const BlockNormArgs p) {
  constexpr int VEC = Chunk<IO>::VEC, NV = E / VEC, RW = G == 0 ? 1 : MOST / (G == 0 ? 1 : G);
  constexpr int NG = G == 0 ? 1 : MOST / 64;  // wavefronts whose column sums are joined
  __shared__ float lds[2][G == 0 ? MOST / 64 : 1];
  __shared__ float cols[NG][G == 0 ? 1 : G * VEC];
  int turn = 0;
  const int T = G == 0 ? blockDim.x : G, t = G == 0 ? threadIdx.x : threadIdx.x % (G == 0 ? 1 : G);
  const float inv = 1.f / (float)p.D;
  const int64_t step = (int64_t)gridDim.x * RW;
  const bool block = p.o != nullptr, gate = p.z != nullptr, residual = p.dr_out != nullptr;
  float w[NV][VEC], pw[NV][VEC], dw[NV][VEC], dpw[NV][VEC];
  // a thread's own sums of up to kRowsOfSum rows each; in registers they would push the rows' out (131072 x 4096,
  // bf16: 2180 us, and 1532 this way; 1510 with one sum over all rows)
  __shared__ float whole[2 * E * MOST];
  const auto kept = [&](int which, int i, int e) -> float& { return whole[((which * NV + i) * VEC + e) * MOST + threadIdx.x]; };
  Chunk<IO> ny[NV], nr[NV], nd[NV], no[NV], nz[NV];
  int64_t row = (int64_t)blockIdx.x * RW + (G == 0 ? 0 : threadIdx.x / (G == 0 ? 1 : G));
  const auto fetch = [&](int i, int64_t at) {
    const int64_t c = ((int64_t)i * T + t) * VEC, n = p.D - c;
    if (n <= 0) return;
    ny[i].load_row(p.dy, at, c, p.D);
    nr[i].load_row(p.r_out, at, c, p.D);
    if (residual) nd[i].load_row(p.dr_out, at, c, p.D);
    if (block) no[i].load_row(p.o, at, c, p.D);
    if (gate) nz[i].load_row(p.z, at, c, p.D);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = ((int64_t)i * T + t) * VEC;
    ny[i].zero();
    nr[i].zero();
    nd[i].zero();
    no[i].zero();
    nz[i].zero();
    if (row < p.rows) fetch(i, row * p.D);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = p.weight && c + e < p.D ? p.weight[c + e] : 1.f;
      pw[i][e] = p.post_weight && c + e < p.D ? p.post_weight[c + e] : 1.f;
      dw[i][e] = dpw[i][e] = kept(0, i, e) = kept(1, i, e) = 0.f;
    }
  }
  while (row < p.rows) {
    for (int left = kRowsOfSum; left > 0 && row < p.rows; --left, row += step) {  // whole rows leave: no sum crosses rows
      const int64_t at = row * p.D, next = (row + step) * p.D;
      const bool more = row + step < p.rows;
      const float rstd = p.rstd[row], q = block ? p.post_rstd[row] : 0.f;
      float u[NV][VEC], h[NV][VEC], g[NV][VEC], o[NV][VEC], z[NV][VEC];
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int by = Chunk<IO>::short_by(((int64_t)i * T + t) * VEC, p.D);
        ny[i].get_row(u[i], by);
        nr[i].get_row(h[i], by);
        nd[i].get_row(g[i], by);
        no[i].get_row(o[i], by);
        nz[i].get_row(z[i], by);
        if (more) fetch(i, next);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          h[i][e] *= rstd;
          dw[i][e] = fmaf(u[i][e], h[i][e], dw[i][e]);
          u[i][e] *= w[i][e];
          a = fmaf(u[i][e], h[i][e], a);
        }
      }
      a = group_sum<G>(a, lds[turn]) * inv;
      turn ^= 1;
      float b = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t c = ((int64_t)i * T + t) * VEC, n = p.D - c;
        Chunk<IO> out;
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[i][e] = fmaf(rstd, u[i][e] - h[i][e] * a, g[i][e]);
        out.set(g[i]);
        if (n > 0) out.store(p.dr, at + c, n);
        if (!block) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          o[i][e] *= q;
          g[i][e] *= p.scale;
        }
        if (gate) {
          float dz[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const Logistic l = logistic_f(z[i][e]);
            dz[e] = g[i][e] * (o[i][e] * pw[i][e]) * (l.s * fmaf(z[i][e], l.sc, 1.f));
            g[i][e] *= z[i][e] * l.s;
          }
          out.set(dz);
          if (n > 0) out.store(p.dz, at + c, n);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          dpw[i][e] = fmaf(g[i][e], o[i][e], dpw[i][e]);
          g[i][e] *= pw[i][e];
          b = fmaf(g[i][e], o[i][e], b);
        }
      }
      if (!block) continue;
      b = group_sum<G>(b, lds[turn]) * inv;
      turn ^= 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t c = ((int64_t)i * T + t) * VEC, n = p.D - c;
        Chunk<IO> out;
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[i][e] = q * (g[i][e] - o[i][e] * b);
        out.set(g[i]);
        if (n > 0) out.store(p.do_, at + c, n);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        kept(0, i, e) += dw[i][e];
        kept(1, i, e) += dpw[i][e];
        dw[i][e] = dpw[i][e] = 0.f;
      }
  }
  if (!p.part) return;
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float(&v)[VEC] = which ? dpw[i] : dw[i];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = kept(which, i, e);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
#pragma unroll
        for (int m = G == 0 ? 64 : G; m < 64; m *= 2) v[e] += __shfl_xor(v[e], m, 64);
      if constexpr (NG > 1) {
        __syncthreads();  // the last round has been read
        if ((threadIdx.x & 63) < G)
#pragma unroll
          for (int e = 0; e < VEC; ++e) cols[threadIdx.x / 64][t * VEC + e] = v[e];
        __syncthreads();
        for (int k = threadIdx.x; k < G * VEC; k += MOST) {
          float s = 0.f;
#pragma unroll
          for (int g = 0; g < NG; ++g) s += cols[g][k];
          const int64_t c = (int64_t)i * T * VEC + k;
          if (c < p.D) part[which * p.D + c] = s;
        }
      } else {
        const int64_t c = ((int64_t)i * T + t) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (c + e < p.D) part[which * p.D + c + e] = v[e];
      }
    }
  }
}

// ---- rows past the registers: walks over memory, sums in fp64 as a thread's own may be long ----

constexpr int64_t kLoopGroups = (int64_t)1 << 20;  // 2^24 workgroups of 256 would be 2^32 threads

template <typename IO>
__device__ __forceinline__ float at_of(const void* p, int64_t i) {
  return io<IO>::widen(io<IO>::load(p, i));
}

template <typename IO>
__global__ __launch_bounds__(256) void block_norm_fwd_loop_kernel(const BlockNormArgs p) {
  __shared__ double lds[8];
  const double inv = 1. / (double)p.D;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t at = row * p.D;
    const void* r = p.r;
    float q = 0.f;
    double s = 0;
    if (p.o) {
      for (int64_t c = threadIdx.x; c < p.D; c += 256) {
        const double v = at_of<IO>(p.o, at + c);
        s = fma(v, v, s);
      }
      q = rstd_of(wide_sum(s, lds), inv, p.eps);
      s = 0;
      for (int64_t c = threadIdx.x; c < p.D; c += 256) {
        float f = at_of<IO>(p.o, at + c) * (q * p.scale);
        if (p.z) f *= silu_f(at_of<IO>(p.z, at + c));
        io<IO>::store(p.r_out, at + c, fmaf(f, p.post_weight ? p.post_weight[c] : 1.f, at_of<IO>(p.r, at + c)));
        const double v = at_of<IO>(p.r_out, at + c);
        s = fma(v, v, s);
      }
      r = p.r_out;
    } else {
      for (int64_t c = threadIdx.x; c < p.D; c += 256) {
        const double v = at_of<IO>(p.r, at + c);
        s = fma(v, v, s);
      }
    }
    const float rstd = rstd_of(wide_sum(s, lds + 4), inv, p.eps);
    for (int64_t c = threadIdx.x; c < p.D; c += 256)
      io<IO>::store(p.y, at + c, at_of<IO>(r, at + c) * rstd * (p.weight ? p.weight[c] : 1.f));
    if (threadIdx.x == 0) {
      if (p.rstd) p.rstd[row] = rstd;
      if (p.post_rstd) p.post_rstd[row] = q;
    }
    if (!p.o) __syncthreads();  // the one sum of a row: the next row's uses the same words
  }
}

// G of an element, from the row's mean(u rh)
template <typename IO>
__device__ __forceinline__ float residual_grad(const BlockNormArgs& p, int64_t i, int64_t c, float rstd, float mean) {
  const float h = at_of<IO>(p.r_out, i) * rstd, u = at_of<IO>(p.dy, i) * (p.weight ? p.weight[c] : 1.f);
  return fmaf(rstd, u - h * mean, p.dr_out ? at_of<IO>(p.dr_out, i) : 0.f);
}

template <typename IO>
__global__ __launch_bounds__(256) void block_norm_bwd_loop_kernel(const BlockNormArgs p) {
  __shared__ double lds[8];
  const double inv = 1. / (double)p.D;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t at = row * p.D;
    const float rstd = p.rstd[row];
    double s = 0;
    for (int64_t c = threadIdx.x; c < p.D; c += 256)
      s = fma((double)(at_of<IO>(p.dy, at + c) * (p.weight ? p.weight[c] : 1.f)), (double)(at_of<IO>(p.r_out, at + c) * rstd), s);
    const float a = (float)(wide_sum(s, lds) * inv);
    if (threadIdx.x == 0) p.row_mean[row] = a;
    const float q = p.o ? p.post_rstd[row] : 0.f;
    s = 0;
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      const float g = residual_grad<IO>(p, at + c, c, rstd, a);
      if (!p.o) {
        io<IO>::store(p.dr, at + c, g);
        continue;
      }
      float f = p.scale * g;
      const float oh = at_of<IO>(p.o, at + c) * q, pw = p.post_weight ? p.post_weight[c] : 1.f;
      if (p.z) {
        const float z = at_of<IO>(p.z, at + c);
        const Logistic l = logistic_f(z);
        io<IO>::store(p.dz, at + c, f * (oh * pw) * (l.s * fmaf(z, l.sc, 1.f)));
        f *= z * l.s;
      }
      s = fma((double)(f * pw), (double)oh, s);
    }
    if (!p.o) {
      __syncthreads();
      continue;
    }
    const float b = (float)(wide_sum(s, lds + 4) * inv);
    for (int64_t c = threadIdx.x; c < p.D; c += 256) {
      const float g = residual_grad<IO>(p, at + c, c, rstd, a);
      float f = p.scale * g;
      if (p.z) f *= silu_f(at_of<IO>(p.z, at + c));
      const float oh = at_of<IO>(p.o, at + c) * q;
      io<IO>::store(p.do_, at + c, q * (f * (p.post_weight ? p.post_weight[c] : 1.f) - oh * b));
      io<IO>::store(p.dr, at + c, g);
    }
  }
}

template <typename IO>
__global__ __launch_bounds__(256) void block_norm_cols_kernel(const BlockNormArgs p) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.D) return;
  double dw = 0, dpw = 0;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const int64_t i = row * p.D + c;
    const float rstd = p.rstd[row];
    dw = fma((double)at_of<IO>(p.dy, i), (double)(at_of<IO>(p.r_out, i) * rstd), dw);
    if (p.o) {
      float f = p.scale * residual_grad<IO>(p, i, c, rstd, p.row_mean[row]);
      if (p.z) f *= silu_f(at_of<IO>(p.z, i));
      dpw = fma((double)f, (double)(at_of<IO>(p.o, i) * p.post_rstd[row]), dpw);
    }
  }
  p.part[(int64_t)blockIdx.y * 2 * p.D + c] = (float)dw;
  p.part[(int64_t)blockIdx.y * 2 * p.D + p.D + c] = (float)dpw;
}

hipError_t join(const BlockNormArgs& a, hipStream_t s) {
  NormArgs n{};
  n.part = a.part;
  n.D = a.D;
  n.dweight = a.dweight;
  n.dbias = a.dpost_weight;
  return launch_norm_join(n, a.groups, s);
}

// Threads that a workgroup has at most where a row has T, more than a wavefront.
constexpr int most_threads(int T) { return T > 512 ? 1024 : (T > 256 ? 512 : 256); }
// Whether some width has this shape (a shape is the same for all widths of (64 k, 64 k + 64]).
constexpr bool shape_of_some(bool bwd, bool bf16, int G, int E, int most) {
  for (int64_t D = 64; block_norm_shape(D, bwd, bf16).T > 0; D += 64) {
    const BlockNormShape f = block_norm_shape(D, bwd, bf16);
    if (f.E == E && (G > 0 ? f.T == G : f.T > 64 && most_threads(f.T) == most)) return true;
  }
  return false;
}
// Whether pick below has a kernel for every width that has a shape.
constexpr bool all_picked(bool bwd, bool bf16) {
  for (int64_t D = 64; block_norm_shape(D, bwd, bf16).T > 0; D += 64) {
    const BlockNormShape f = block_norm_shape(D, bwd, bf16);
    if (!(f.E == 8 || (f.E == 4 && !bf16) || (f.E == 16 && f.T > 64))) return false;
  }
  return true;
}

template <typename IO, int G, int E, int MOST>
hipError_t go(const BlockNormArgs& a, int threads, bool bwd, hipStream_t s) {
  constexpr int RW = G == 0 ? 1 : MOST / (G == 0 ? 1 : G);
  constexpr bool bf16 = io<IO>::es == 2, of_fwd = shape_of_some(false, bf16, G, E, MOST), of_bwd = shape_of_some(true, bf16, G, E, MOST);
  const dim3 block(G == 0 ? threads : MOST);
  if (!bwd) {
    if constexpr (of_fwd) {
      const int64_t all = (a.rows + RW - 1) / RW;
      hipLaunchKernelGGL((block_norm_fwd_kernel<IO, G, E, MOST>), dim3((unsigned)(all < kRowGroups ? all : kRowGroups)), block, 0, s, a);
      return hipGetLastError();
    }
    return hipErrorInvalidValue;
  }
  if constexpr (of_bwd) {
    hipLaunchKernelGGL((block_norm_bwd_kernel<IO, G, E, MOST>), dim3((unsigned)a.groups), block, 0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || !a.part ? e : join(a, s);
  }
  return hipErrorInvalidValue;
}

template <typename IO, int E>
hipError_t go_wide(const BlockNormArgs& a, int threads, bool bwd, hipStream_t s) {
  if (threads <= 64) return hipErrorInvalidValue;
  const int most = most_threads(threads);
  if (most == 1024) return go<IO, 0, E, 1024>(a, threads, bwd, s);
  return most == 512 ? go<IO, 0, E, 512>(a, threads, bwd, s) : go<IO, 0, E, 256>(a, threads, bwd, s);
}

template <typename IO>
hipError_t pick(const BlockNormArgs& a, bool bwd, hipStream_t s) {
  static_assert(all_picked(false, io<IO>::es == 2) && all_picked(true, io<IO>::es == 2), "a kernel for every width");
  const BlockNormShape f = block_norm_shape(a.D, bwd, io<IO>::es == 2);
#define MSM_ROWS(GG, EE) \
  if (f.T == GG && f.E == EE) return go<IO, GG, EE, 256>(a, GG, bwd, s);
  MSM_ROWS(16, 8) MSM_ROWS(32, 8) MSM_ROWS(64, 8)
  if constexpr (io<IO>::es == 4) {
    MSM_ROWS(16, 4) MSM_ROWS(32, 4) MSM_ROWS(64, 4)
#undef MSM_ROWS
    if (f.E == 4) return go_wide<IO, 4>(a, f.T, bwd, s);
  }
  if (f.E == 8) return go_wide<IO, 8>(a, f.T, bwd, s);
  if (f.E == 16) return go_wide<IO, 16>(a, f.T, bwd, s);
  const dim3 grid((unsigned)(a.rows < kLoopGroups ? a.rows : kLoopGroups));
  if (!bwd) {
    hipLaunchKernelGGL((block_norm_fwd_loop_kernel<IO>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((block_norm_bwd_loop_kernel<IO>), grid, dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  hipLaunchKernelGGL((block_norm_cols_kernel<IO>), dim3((unsigned)((a.D + 255) / 256), (unsigned)a.groups), dim3(256), 0, s, a);
  e = hipGetLastError();
  return e != hipSuccess ? e : join(a, s);
}

}  // namespace

hipError_t launch_block_norm_fwd(const BlockNormArgs& a, int io_bf16, hipStream_t s) {
  return io_bf16 ? pick<bf16_storage>(a, false, s) : pick<float>(a, false, s);
}
hipError_t launch_block_norm_bwd(const BlockNormArgs& a, int io_bf16, hipStream_t s) {
  return io_bf16 ? pick<bf16_storage>(a, true, s) : pick<float>(a, true, s);
}

}  // namespace msm
