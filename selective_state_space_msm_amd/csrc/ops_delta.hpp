// Matrix-core building blocks of the chunked gated delta rule (gfx950, wave64).
//
// Every product here has the shape (rows x 32) times (32 x 16): its right factor is a matrix
// of 16 columns that a wavefront keeps in registers, as an earlier product left it.  In the
// accumulator layout of the 16x16 MFMAs lane l holds column l & 15 and four consecutive rows of
// group l >> 4.  Two accumulator tiles therefore give a lane eight values along the rows, which
// is exactly what it has to supply as the right factor of a product that sums over those rows,
// provided both factors number the summed index alike.  Rows are numbered in blocks of 32:
//   row(block, tile s, group j, register r) = 32 block + 8 j + 4 s + r,
// so the eight values are eight consecutive rows and the left factor's are eight consecutive
// elements in memory.  A chain of products (state -> prediction -> error -> state) then never
// moves its right factors between lanes.
#pragma once

#include "msm_device.hpp"
#include "msm_lanes.hpp"
#include "ops_internal.h"

namespace msm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// Upper halves of two words, the first one's in the low half.
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// ---- fp32 arithmetic: v_mfma_f32_16x16x4_f32, exact fp32 products ----
struct MathF32 {
  using elem = float;   // I/O elements, also what LDS holds of them
  using telem = float;  // elements of chunk matrices
  using storage = float;
  static constexpr int es = 4;
  static constexpr int bf16 = 0;
  static constexpr int kPlanes = 1;
  static constexpr int kOutParts = 1;
  static constexpr int kGradParts = 1;
  template <int N>
  struct Part {
    float v[8];
  };
  static constexpr int kPer = 4;  // elements of a 16-byte unit
  static constexpr int pad = 4;   // elements added to a padded LDS row
  static __device__ __forceinline__ float widen(float x) { return x; }
  static __device__ __forceinline__ float narrow(float x) { return x; }

  // eight consecutive elements of `planes` row-major planes
  template <int N>
  static __device__ __forceinline__ Part<N> load(const float* p, int) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return Part<N>{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
  }
  // transposed: eight consecutive rows of one column.  `row` is the first row's address and
  // `col` the column of this lane
  template <int N>
  static __device__ __forceinline__ Part<N> load_t(const float* row, int ld, int, int lane,
                                                   int tile_col, int spread) {
    const int m = lane & 15;
    const float* c = row + tile_col + spread * (m >> 2) + (m & 3);
    Part<N> a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a.v[i] = c[i * ld];
    return a;
  }
  template <int N>
  static __device__ __forceinline__ Part<N> load_sw(const float* row, int unit, int sw, int) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(row + (unit ^ sw) * 4);
    const f32x4 b = *reinterpret_cast<const f32x4*>(row + ((unit + 1) ^ sw) * 4);
    return Part<N>{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
  }
  template <int U, int N>
  static __device__ __forceinline__ Part<N> load_sw_t(const float* lds, int row0, int c, int spread, int lane, int) {
    const int m = lane & 15, col = c + spread * (m >> 2);
    Part<N> a;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // swizzle<U> of row0 + i with row0 a multiple of 8
      const int sw = U >= 16 ? (((i & 3) << 2) | ((row0 >> 3) & 3))
                             : (U == 8 ? ((((i >> 1) & 1) << 2) | ((row0 >> 3) & 3)) : ((row0 >> 3) & 3));
      a.v[i] = lds[(row0 + i) * U * 4 + ((col / 4) ^ sw) * 4 + (m & 3)];
    }
    return a;
  }
  template <int N>
  static __device__ __forceinline__ Part<N> split(const f32x4& a, const f32x4& b) {
    return Part<N>{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
  }
  // the leading N parts
  template <int N, int NA>
  static __device__ __forceinline__ Part<N> first(const Part<NA>& a) {
    return Part<N>{{a.v[0], a.v[1], a.v[2], a.v[3], a.v[4], a.v[5], a.v[6], a.v[7]}};
  }
  template <int N>
  static __device__ __forceinline__ void store_planes(float* p, int, const f32x4& a, const f32x4& b) {
    *reinterpret_cast<f32x4*>(p) = a;
    *reinterpret_cast<f32x4*>(p + 4) = b;
  }
  template <int N>
  static __device__ __forceinline__ void store1(float* p, int, float x) {
    *p = x;
  }
  template <int NA, int NB>
  static __device__ __forceinline__ void mma(f32x4& c, const Part<NA>& a, const Part<NB>& b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
  }
};

// ---- bf16 inputs, fp32 everything between: v_mfma_f32_16x16x32_bf16 on split values ----
// A value is cut into bf16 parts by truncation, x = hi + mid + lo with 8 significant bits each:
// three parts hold all 24 bits of an fp32 value, two parts 16.  A product of n-part factors
// keeps the terms whose parts' places add up to less than n: inputs (one part) times a
// three-part value are 3 MFMAs and two three-part values 6, to fp32 accuracy, against the 16
// times slower fp32 MFMA.  Infinities leave NaN in the lower parts.
struct MathBF16 {
  using elem = uint16_t;
  using telem = uint16_t;
  using storage = bf16_storage;
  static constexpr int es = 2;
  static constexpr int bf16 = 1;
  static constexpr int kPlanes = 3;
  static constexpr int kOutParts = 2;   // the output is rounded to bf16: 16 bits carry it
  static constexpr int kGradParts = 2;  // likewise the gradients of q and k
  template <int N>
  struct Part {
    bf16x8 p[N];
  };
  static constexpr int kPer = 8;
  static constexpr int pad = 8;
  static __device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
  static __device__ __forceinline__ uint16_t narrow(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
  }

  template <int N>
  static __device__ __forceinline__ Part<N> load(const uint16_t* p, int plane) {
    Part<N> a;
#pragma unroll
    for (int i = 0; i < N; ++i) a.p[i] = *reinterpret_cast<const bf16x8*>(p + i * plane);
    return a;
  }
  // ds_read_b64_tr_b16: the 16 lanes of a group read a block of 4 rows x 16 columns, lane i row
  // i / 4 and four consecutive columns from column chunk i % 4, and receive it transposed, lane i
  // the four rows of column i.  The chunks are `spread` columns apart.
  template <int N>
  static __device__ __forceinline__ Part<N> load_t(const uint16_t* row, int ld, int plane, int lane,
                                                   int tile_col, int spread) {
    typedef __attribute__((address_space(3))) s16x4* lds4;
    const int i = lane & 15;
    const uint16_t* c = row + (i >> 2) * ld + tile_col + spread * (i & 3);
    Part<N> a;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      struct {
        s16x4 lo, hi;
      } v;
      v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(c + n * plane));
      v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(c + n * plane + 4 * ld));
      a.p[n] = __builtin_bit_cast(bf16x8, v);
    }
    return a;
  }
  template <int N>
  static __device__ __forceinline__ Part<N> load_sw(const uint16_t* row, int unit, int sw, int plane) {
    return load<N>(row + (unit ^ sw) * 8, plane);
  }
  template <int U, int N>
  static __device__ __forceinline__ Part<N> load_sw_t(const uint16_t* lds, int row0, int c, int spread, int lane,
                                                      int plane) {
    typedef __attribute__((address_space(3))) s16x4* lds4;
    const int i = lane & 15, row = row0 + (i >> 2), col = c + spread * (i & 3);
    const int sw = U >= 16 ? (((i >> 2) << 2) | ((row0 >> 3) & 3))
                           : (U == 8 ? (((i >> 3) << 2) | ((row0 >> 3) & 3)) : ((row0 >> 3) & 3));
    const uint16_t* p = lds + row * U * 8 + ((col / 8) ^ sw) * 8 + col % 8;
    Part<N> a;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      struct {
        s16x4 lo, hi;
      } v;
      v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + n * plane));
      v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + n * plane + 4 * U * 8));
      a.p[n] = __builtin_bit_cast(bf16x8, v);
    }
    return a;
  }
  template <int N>
  static __device__ __forceinline__ Part<N> split(const f32x4& a, const f32x4& b) {
    float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    Part<N> o;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u0 = __float_as_uint(x[2 * i]), u1 = __float_as_uint(x[2 * i + 1]);
        w[i] = pack_hi(u0, u1);
        if (n + 1 < N) {
          x[2 * i] -= __uint_as_float(u0 & 0xffff0000u);
          x[2 * i + 1] -= __uint_as_float(u1 & 0xffff0000u);
        }
      }
      o.p[n] = __builtin_bit_cast(bf16x8, w);
    }
    return o;
  }
  template <int N, int NA>
  static __device__ __forceinline__ Part<N> first(const Part<NA>& a) {
    Part<N> o;
#pragma unroll
    for (int n = 0; n < N; ++n) o.p[n] = a.p[n];
    return o;
  }
  template <int N>
  static __device__ __forceinline__ void store_planes(uint16_t* p, int plane, const f32x4& a,
                                                      const f32x4& b) {
    const Part<N> s = split<N>(a, b);
#pragma unroll
    for (int n = 0; n < N; ++n) *reinterpret_cast<bf16x8*>(p + n * plane) = s.p[n];
  }
  template <int N>
  static __device__ __forceinline__ void store1(uint16_t* p, int plane, float x) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t u = __float_as_uint(x);
      p[n * plane] = (uint16_t)(u >> 16);
      x -= __uint_as_float(u & 0xffff0000u);
    }
  }
  template <int NA, int NB>
  static __device__ __forceinline__ void mma(f32x4& c, const Part<NA>& a, const Part<NB>& b) {
    constexpr int NM = NA > NB ? NA : NB;
#pragma unroll
    for (int sum = NM - 1; sum >= 0; --sum)  // smallest terms first
#pragma unroll
      for (int i = 0; i < NA; ++i)
        if (sum - i >= 0 && sum - i < NB)
          c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[sum - i], c, 0, 0, 0);
  }
};

// ---- sequences and their chunks ----
// Uniform batches: sequence s is rows s L ...; its chunk c has slot s NT + c.  Packed batches:
// off[] bounds the sequences and sequence s starts at slot floor(off[s] / C) + s.  A sequence of
// rows [a, b) has ceil((b - a) / C) <= floor(b / C) - floor(a / C) + 1 chunks, so slots never
// collide, no prefix sum over the lengths is needed, and nslots = floor(tokens / C) + nseq
// bounds them all.  Offsets are clamped to the arrays, so that wrong ones cannot reach outside.
struct SeqRows {
  int64_t row0, len, slot0;
};

template <int C>
__device__ __forceinline__ SeqRows seq_rows(const DeltaArgs& p, int64_t s) {
  if (!p.off) return SeqRows{s * p.L, p.L, s * p.NT};
  int64_t a = p.off[s], b = p.off[s + 1];
  a = a < 0 ? 0 : (a > p.tokens ? p.tokens : a);
  b = b < a ? a : (b > p.tokens ? p.tokens : b);
  return SeqRows{a, b - a, a / C + s};
}

// First row and number of rows of the chunk in a slot (0 rows: no chunk there).
struct ChunkRows {
  int64_t row0;
  int n;
};

template <int C>
__device__ __forceinline__ ChunkRows chunk_rows(const DeltaArgs& p, int64_t slot) {
  int64_t s;
  if (!p.off) {
    s = slot / p.NT;
  } else {
    int64_t lo = 0, hi = p.nseq;  // the last sequence whose first slot is at or before this one
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (seq_rows<C>(p, mid).slot0 <= slot)
        lo = mid;
      else
        hi = mid;
    }
    s = lo;
  }
  const SeqRows r = seq_rows<C>(p, s);
  const int64_t at = (slot - r.slot0) * C;
  if (at < 0 || at >= r.len) return ChunkRows{0, 0};
  const int64_t left = r.len - at;
  return ChunkRows{r.row0 + at, (int)(left < C ? left : C)};
}

// ---- LDS layout ----
// Rows of U 16-byte units without padding; unit u of row r lies at position u ^ swizzle<U>(r).
// The readers below take 16 rows 8 (m / 4) + m % 4 (+ 4 s) at one unit, or 4 consecutive rows
// times 4 consecutive units: either way the swizzle spreads the 16 addresses over all banks.
// It depends on row bits 0, 1, 3 and 4 alone, so a lane's swizzle is the same in all its reads.
template <int U>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (U == 4) return (r >> 3) & 3;
  if constexpr (U == 8) return (((r >> 1) & 1) << 2) | ((r >> 3) & 3);
  return ((r & 3) << 2) | ((r >> 3) & 3);
}

// Left factor of a product over 32 columns from column c (a multiple of 8) of a row.
template <class M, int U, int N, typename TE>
__device__ __forceinline__ typename M::template Part<N> load_row(const TE* lds, int row, int c, int plane) {
  return M::template load_sw<N>(lds + row * U * M::kPer, c / M::kPer, swizzle<U>(row), plane);
}
// The same transposed: eight consecutive rows from row0, of the column this lane supplies: lane m
// has column c + spread (m / 4) + m % 4.
template <class M, int U, int N, typename TE>
__device__ __forceinline__ typename M::template Part<N> load_col(const TE* lds, int row0, int c, int spread,
                                                                 int lane, int plane) {
  return M::template load_sw_t<U, N>(lds, row0, c, spread, lane, plane);
}

// ---- staging ----
constexpr uint32_t kOutside = 0x80000000u;  // an offset past any resource: reads zero, writes nothing

__device__ __forceinline__ u32x4 bload16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// The rows of one head of a chunk: (rows, heads, size) arrays, `stride` bytes from row to row and
// `bytes` of each row.  Rows past the chunk read as zero and are never written.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t head_rsrc(const void* base, int64_t row0, int64_t heads, int64_t h,
                                                             int64_t size, int es, int rows) {
  const char* p = static_cast<const char*>(base) + ((row0 * heads + h) * size) * es;
  return make_rsrc(p, rows > 0 ? ((rows - 1) * heads + 1) * size * es : 0);
}

// q or k rows of a chunk, on their way from memory to swizzled LDS rows of KP elements; rows and
// columns past the chunk's are zero.
template <class M, int KP, int C, int THREADS>
struct RowStage {
  static constexpr int U = KP / M::kPer, N = (C * U + THREADS - 1) / THREADS;
  static_assert(C * U % THREADS == 0, "whole passes");
  u32x4 w[N];

  static __device__ __forceinline__ uint32_t offset(int i, int tid, uint32_t stride, int K) {
    const int u = tid + i * THREADS, row = u / U, c = ((u % U) ^ swizzle<U>(row)) * M::kPer;
    return c < K ? row * stride + c * M::es : kOutside;
  }
  __device__ __forceinline__ void fetch(__amdgpu_buffer_rsrc_t r, uint32_t stride, int K, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = bload16(r, offset(i, tid, stride, K));
  }
  __device__ __forceinline__ void put(typename M::elem* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(lds + (tid + i * THREADS) * M::kPer) = w[i];
  }
  // rows that cannot be read 16 bytes at a time
  static __device__ __forceinline__ void by_element(typename M::elem* lds, __amdgpu_buffer_rsrc_t r,
                                                    uint32_t stride, int K, int tid) {
    using T = io<typename M::storage>;
    for (int u = tid; u < C * KP; u += THREADS) {
      const int row = u / KP, c = u % KP;
      const auto x = T::bload(r, c < K ? row * stride + c * M::es : kOutside, 0);
      lds[row * KP + ((c / M::kPer) ^ swizzle<U>(row)) * M::kPer + c % M::kPer] = (typename M::elem)x;
    }
  }
};

// Chunk matrices (lower triangular, C x C) are kept as their 32 x 32 blocks on and below the
// diagonal, (0,0), (1,0), (1,1), each in swizzled rows, in memory as in LDS; planes follow each
// other.
template <class M, int C>
struct Tri {
  static constexpr int U = 32 / M::kPer, kBlock = 32 * 32, kPlane = kBlock * (C / 32) * (C / 32 + 1) / 2;
  static __device__ __forceinline__ int block(int rb, int kb) { return (rb * (rb + 1) / 2 + kb) * kBlock; }
  // place of an element on or below the block diagonal
  static __device__ __forceinline__ int at(int row, int col) {
    const int r = row & 31, c = col & 31;
    return block(row >> 5, col >> 5) + r * 32 + ((c / M::kPer) ^ swizzle<U>(r)) * M::kPer + c % M::kPer;
  }
};

// `PLANES` planes of a chunk matrix on their way from memory to LDS.
template <class M, int C, int PLANES, int THREADS>
struct TriStage {
  static constexpr int kUnits = PLANES * Tri<M, C>::kPlane / M::kPer;
  static constexpr int N = (kUnits + THREADS - 1) / THREADS;
  static constexpr int kLds = N * THREADS * M::kPer;  // elements of LDS, whole passes
  u32x4 w[N];
  __device__ __forceinline__ void fetch(__amdgpu_buffer_rsrc_t r, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = bload16(r, (tid + i * THREADS) * 16);
  }
  __device__ __forceinline__ void put(typename M::telem* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(lds + (tid + i * THREADS) * M::kPer) = w[i];
  }
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t sh, int planes) {
    constexpr int es = (int)sizeof(typename M::telem);
    return make_rsrc_u32(static_cast<const char*>(base) + sh * planes * Tri<M, C>::kPlane * es,
                         PLANES * Tri<M, C>::kPlane * es);
  }
};

// Sums of 16 register values over the 16 lanes of a group: lane l ends with the sum of value
// l & 15 (pairings as in reduce_scatter32).
__device__ __forceinline__ float sum_rows16(float (&v)[16], int lane) {
  rs_dpp<0x140, 8, 8>(v, lane);  // row_mirror
  rs_dpp<0x141, 4, 4>(v, lane);  // row_half_mirror
  rs_dpp<0x4E, 2, 2>(v, lane);   // quad_perm [2,3,0,1]
  rs_dpp<0xB1, 1, 1>(v, lane);   // quad_perm [1,0,3,2]
  return v[0];
}

}  // namespace msm
