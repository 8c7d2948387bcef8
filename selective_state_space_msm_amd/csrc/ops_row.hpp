// Rows held in the registers of a group of threads: their pieces, and sums over a row (gfx950).
#pragma once

#include <type_traits>

#include "ops_delta.hpp"

namespace msm {

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

// Sum over a workgroup of 256 threads, the same value in each.  `lds` must not be the next sum's.
__device__ __forceinline__ double wide_sum(double v, double* lds) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// a / b for a >= 0, b > 0: in 32 bits where both are that small (a quarter of the instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// 16 bytes of a row that may begin at any element's address (the hardware takes unaligned 16-byte
// accesses).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Elements [i, i + VEC) of an array, of which the first n belong to the row (the others read zero).
template <typename IO>
struct Chunk {
  static constexpr int VEC = 16 / io<IO>::es;
  u32x4 raw;
  __device__ __forceinline__ void zero() { raw = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const void* p, int64_t i, int64_t n) {
    if (n >= VEC) {
      raw = *reinterpret_cast<const u32x4_any*>(static_cast<const char*>(p) + i * io<IO>::es);
    } else {
      raw = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < VEC - 1; ++e)
        if (e < n) {
          if constexpr (io<IO>::es == 2)
            raw[e / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[i + e] << (16 * (e & 1));
          else
            raw[e] = static_cast<const uint32_t*>(p)[i + e];
        }
    }
  }
  // Elements [c, c + VEC) of a row of D that starts at element i.  A row's last piece, where it is short and
  // not the only one, is taken as the 16 bytes that end the row: one load like the others, whose first
  // short_by(c, D) elements get() leaves out, so that nothing waits for it before it is used.  (Element by
  // element the wavefront waits where it loads: 30000 rows of 500, bf16, block norm backward: 135 us, and 56 this way.)
  static __device__ __forceinline__ int short_by(int64_t c, int64_t D) { return c > 0 && c < D && D - c < VEC ? (int)(VEC - (D - c)) : 0; }
  __device__ __forceinline__ void load_row(const void* p, int64_t i, int64_t c, int64_t D) {
    const int by = short_by(c, D);
    load(p, i + c - by, by ? VEC : D - c);
  }
  __device__ __forceinline__ void get_row(float* x, int by) const {
    Chunk<IO> r = *this;
    if (by) {
      const int s = by * io<IO>::es * 8;
      uint64_t lo = raw[0] | (uint64_t)raw[1] << 32, hi = raw[2] | (uint64_t)raw[3] << 32;
      if (s >= 64) {
        lo = hi >> (s - 64);
        hi = 0;
      } else {
        lo = lo >> s | hi << (64 - s);
        hi >>= s;
      }
      r.raw = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
    r.get(x);
  }
  __device__ __forceinline__ void get(float* x) const {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (io<IO>::es == 2) {
        x[2 * c] = __uint_as_float(raw[c] << 16);
        x[2 * c + 1] = __uint_as_float(raw[c] & 0xffff0000u);
      } else {
        x[c] = __uint_as_float(raw[c]);
      }
    }
  }
  // rounds x to the I/O type
  __device__ __forceinline__ void set(const float* x) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (io<IO>::es == 2) {
        const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x[2 * c]));
        const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x[2 * c + 1]));
        raw[c] = lo | (hi << 16);
      } else {
        raw[c] = __float_as_uint(x[c]);
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i, int64_t n) const {
    if (n >= VEC) {
      *reinterpret_cast<u32x4_any*>(static_cast<char*>(p) + i * io<IO>::es) = raw;
    } else {
#pragma unroll
      for (int e = 0; e < VEC - 1; ++e)
        if (e < n) {
          if constexpr (io<IO>::es == 2)
            static_cast<uint16_t*>(p)[i + e] = (uint16_t)(raw[e / 2] >> (16 * (e & 1)));
          else
            static_cast<uint32_t*>(p)[i + e] = raw[e];
        }
    }
  }
};

}  // namespace msm
