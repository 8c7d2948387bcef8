// Global 2-norm of many gradient tensors, and clipping by it (gfx950).
//   norm = sqrt(sum of squares over all tensors),  y = x min(1, max_norm / (norm + eps))
//
// Bound by HBM: every gradient is read once for the norm and once more for the scaling.  The
// tensors' addresses and sizes travel in the kernel arguments, kClipTensors of them a launch,
// so nothing is copied to the device first and a launch can be captured.  Tensors are cut into
// chunks of kClipChunk elements; a workgroup walks chunks at a fixed stride and leaves one
// partial sum.  Squares are summed in fp64: at HBM's rate its cost is hidden, it cannot overflow,
// and the order is fixed.  The scaling kernel joins the partial sums itself, in a fixed
// order (2048 of them come from L2 in about the time a launch takes; above 4096 tensors there are
// more, and one launch joins them first: 2^18 tensors in 2048 launches took 128 ms with a join in
// each), and walks the chunks from the last to the first: the gradients that the norm read last are still in the last-level cache.
// 24 layers of 2048, 606 MB of bf16: 320 us for the 1.82 GB that are read twice and written once
// (5.7 TB/s with the cache's part; a copy reaches 5.15; the norm alone 114 us, 5.3 TB/s), 330 us with
// twice the workgroups; small tensors are bound by the launches and the host's lists.
#include "ops_delta.hpp"

namespace msm {
namespace {

// The tensor of a chunk: the last one that starts at or before it.
__device__ __forceinline__ int tensor_of(const ClipBatch& b, uint32_t chunk) {
  int lo = 0, hi = b.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__device__ __forceinline__ double square(float x) { return (double)x * (double)x; }

// Calls use(i, piece) for the pieces of PER elements that fill n from the start on, a thread's own at
// i, with kDeep of them fetched before the first is used, and returns where they end: at four
// workgroups a CU one load a thread is less than HBM's latency asks for.
constexpr int kDeep = 4;
template <int PER, class T, class F>
__device__ __forceinline__ int walk(const T* x, int n, F use) {
  constexpr int kStep = 256 * PER;
  int i = 0;
  for (; i + kDeep * kStep <= n; i += kDeep * kStep) {
    u32x4 w[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) w[d] = *reinterpret_cast<const u32x4*>(x + i + d * kStep + PER * threadIdx.x);
#pragma unroll
    for (int d = 0; d < kDeep; ++d) use(i + d * kStep + PER * threadIdx.x, w[d]);
  }
  for (; i + kStep <= n; i += kStep)
    use(i + PER * threadIdx.x, *reinterpret_cast<const u32x4*>(x + i + PER * threadIdx.x));
  return i;
}

__global__ __launch_bounds__(256) void clip_sum_kernel(const ClipBatch b, double* part) {
  __shared__ double lds[4];
  const uint32_t chunks = b.first[b.count];
  double sum = 0;
  for (uint32_t ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    const int t = tensor_of(b, ch);
    const int64_t at = (int64_t)(ch - b.first[t]) * kClipChunk;
    const int n = (int)(b.n[t] - at < kClipChunk ? b.n[t] - at : kClipChunk);
    double s0 = 0, s1 = 0;
    if (b.bf16[t]) {
      const uint16_t* x = static_cast<const uint16_t*>(b.src[t]) + at;
      int i = 0;
      if (((uintptr_t)x & 15) == 0)
        i = walk<8>(x, n, [&](int, const u32x4& w) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            s0 += square(__uint_as_float(w[c] << 16));
            s1 += square(__uint_as_float(w[c] & 0xffff0000u));
          }
        });
      for (i += threadIdx.x; i < n; i += 256) s0 += square(__uint_as_float((uint32_t)x[i] << 16));
    } else {
      const float* x = static_cast<const float*>(b.src[t]) + at;
      int i = 0;
      if (((uintptr_t)x & 15) == 0)
        i = walk<4>(x, n, [&](int, const u32x4& u) {
          const f32x4 w = __builtin_bit_cast(f32x4, u);
          s0 += square(w[0]) + square(w[1]);
          s1 += square(w[2]) + square(w[3]);
        });
      for (i += threadIdx.x; i < n; i += 256) s0 += square(x[i]);
    }
    sum += s0 + s1;
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ float norm_of(const double* part, int64_t parts, double* lds) {
  double sum = 0;
  for (int64_t i = threadIdx.x; i < parts; i += 256) sum += part[i];
  return (float)sqrt(block_sum(sum, lds));
}

__global__ __launch_bounds__(256) void clip_norm_kernel(const double* part, int64_t parts, float* norm) {
  __shared__ double lds[4];
  const float x = norm_of(part, parts, lds);
  if (threadIdx.x == 0) *norm = x;
}

__global__ __launch_bounds__(256) void clip_scale_kernel(const ClipBatch b, const double* part,
                                                         int64_t parts, float* norm,
                                                         float max_norm, float eps) {
  __shared__ double lds[4];
  const float total = part ? norm_of(part, parts, lds) : *norm;
  if (part && norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  // a NaN norm makes the coefficient NaN, and with it every gradient
  const float c = max_norm / (total + eps), coef = c > 1.f ? 1.f : c;
  const uint32_t chunks = b.first[b.count];
  for (uint32_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    const uint32_t ch = chunks - 1 - k;
    const int t = tensor_of(b, ch);
    if (coef == 1.f && b.dst[t] == b.src[t]) continue;
    const int64_t at = (int64_t)(ch - b.first[t]) * kClipChunk;
    const int n = (int)(b.n[t] - at < kClipChunk ? b.n[t] - at : kClipChunk);
    if (b.bf16[t]) {
      const uint16_t* x = static_cast<const uint16_t*>(b.src[t]) + at;
      __bf16* y = static_cast<__bf16*>(b.dst[t]) + at;
      int i = 0;
      if ((((uintptr_t)x | (uintptr_t)y) & 15) == 0)
        i = walk<8>(x, n, [&](int to, const u32x4& w) {
          bf16x8 o;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            o[2 * q] = static_cast<__bf16>(__uint_as_float(w[q] << 16) * coef);
            o[2 * q + 1] = static_cast<__bf16>(__uint_as_float(w[q] & 0xffff0000u) * coef);
          }
          __builtin_nontemporal_store(o, reinterpret_cast<bf16x8*>(y + to));
        });
      for (i += threadIdx.x; i < n; i += 256)
        y[i] = static_cast<__bf16>(__uint_as_float((uint32_t)x[i] << 16) * coef);
    } else {
      const float* x = static_cast<const float*>(b.src[t]) + at;
      float* y = static_cast<float*>(b.dst[t]) + at;
      int i = 0;
      if ((((uintptr_t)x | (uintptr_t)y) & 15) == 0)
        i = walk<4>(x, n, [&](int to, const u32x4& w) {
          __builtin_nontemporal_store(__builtin_bit_cast(f32x4, w) * coef, reinterpret_cast<f32x4*>(y + to));
        });
      for (i += threadIdx.x; i < n; i += 256) y[i] = x[i] * coef;
    }
  }
}

}  // namespace

hipError_t launch_clip_sum(const ClipBatch& b, double* part, int groups, hipStream_t s) {
  hipLaunchKernelGGL(clip_sum_kernel, dim3((unsigned)groups), dim3(256), 0, s, b, part);
  return hipGetLastError();
}
hipError_t launch_clip_norm(const double* part, int64_t parts, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(256), 0, s, part, parts, norm);
  return hipGetLastError();
}
hipError_t launch_clip_scale(const ClipBatch& b, const double* part, int64_t parts, float* norm,
                             float max_norm, float eps, int groups, hipStream_t s) {
  hipLaunchKernelGGL(clip_scale_kernel, dim3((unsigned)groups), dim3(256), 0, s, b, part, parts,
                     norm, max_norm, eps);
  return hipGetLastError();
}

}  // namespace msm
