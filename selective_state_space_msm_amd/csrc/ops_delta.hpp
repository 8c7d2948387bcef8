// Matrix-core building blocks of the chunked gated delta rule (gfx950, wave64).
//
// Every product here has the shape (rows x 32) times (32 x 16) on v_mfma_f32_16x16x32_bf16: its
// right factor is a matrix of 16 columns that a wavefront keeps in registers, as an earlier
// product left it.  In the accumulator layout lane l holds column l & 15 and four consecutive
// rows of group l >> 4.  Two accumulator tiles therefore give a lane eight values along the
// rows, which is exactly what it has to supply as the right factor of a product that sums over
// those rows, provided both factors number the summed index alike.  Rows are numbered in blocks
// of 32:
//   row(block, tile t, group j, register r) = 32 block + 8 j + 4 t + r,
// so the eight values are eight consecutive rows and the left factor's are eight consecutive
// elements in memory.  A chain of products (state -> prediction -> error -> state) then never
// moves its right factors between lanes.
//
// Values are cut into bf16 parts by truncation, x = hi + mid + lo with 8 significant bits each:
// three parts hold all 24 bits of an fp32 value, and a bf16 input is one part.  A product of an
// NA-part and an NB-part factor keeps the terms whose places add up to less than the larger
// count: an input times a three-part value is 3 MFMAs, exact, and two three-part values are 6,
// without what is below 2^-20 of a term (a sum of 64 products is off by 6e-8 of its size, an
// fp32 sum by 1.5e-7); the fp32 MFMA, 16 times slower per product, would take 2.7 times as long
// as the 6.  Infinities leave NaN in the lower parts.
#pragma once

#include "msm_device.hpp"
#include "msm_lanes.hpp"
#include "ops_internal.h"

namespace msm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Pointers to shared memory keep their address space: the compiler then knows which arrays a load
// into LDS can touch, and need not wait for it before reading the others.
#define MSM_LDS __attribute__((address_space(3)))
typedef MSM_LDS uint16_t* lds_parts;
typedef const MSM_LDS uint16_t* lds_cparts;

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// Upper halves of two words, the first one's in the low half.
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Eight values of a factor, in N parts.
template <int N>
struct Part {
  bf16x8 p[N];
};

template <int N>
__device__ __forceinline__ Part<N> split(const f32x4& a, const f32x4& b) {
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
template <int N>
__device__ __forceinline__ void store_parts(lds_parts p, int plane, const Part<N>& s) {
#pragma unroll
  for (int n = 0; n < N; ++n) *(MSM_LDS bf16x8*)(p + n * plane) = s.p[n];
}
template <int N>
__device__ __forceinline__ void store_parts(uint16_t* p, int plane, const Part<N>& s) {
#pragma unroll
  for (int n = 0; n < N; ++n) *(bf16x8*)(p + n * plane) = s.p[n];
}
template <int N, class Ptr>
__device__ __forceinline__ void store_parts1(Ptr p, int plane, float x) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint32_t u = __float_as_uint(x);
    p[n * plane] = (uint16_t)(u >> 16);
    x -= __uint_as_float(u & 0xffff0000u);
  }
}

// The terms of a product, smallest first: term i takes part term_a(i) of the left factor and
// term_b(i) of the right one.
template <int NA, int NB>
struct Terms {
  static constexpr int kMost = NA > NB ? NA : NB;
  static constexpr bool in(int sum, int i) { return i < NA && sum - i >= 0 && sum - i < NB; }
};
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& c, const Part<NA>& a, const Part<NB>& b) {
#pragma unroll
  for (int sum = Terms<NA, NB>::kMost - 1; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (Terms<NA, NB>::in(sum, i))
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[sum - i], c, 0, 0, 0);
}
// The same for several tiles with one right factor, tile after tile within a term, so that
// neighbouring MFMAs do not wait for each other's accumulator.
template <int NT, int NA, int NB>
__device__ __forceinline__ void mma_tiles(f32x4 (&c)[NT], const Part<NA> (&a)[NT], const Part<NB>& b) {
#pragma unroll
  for (int sum = Terms<NA, NB>::kMost - 1; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (Terms<NA, NB>::in(sum, i))
#pragma unroll
        for (int t = 0; t < NT; ++t)
          c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t].p[i], b.p[sum - i], c[t], 0, 0, 0);
}

// ---- LDS layout ----
// Rows of U 16-byte units (8 bf16 parts) without padding; unit u of row r lies at position
// u ^ swizzle<U>(r).  The readers below take 16 rows 8 (m / 4) + m % 4 (+ 4 t) at one unit, or 4
// consecutive rows times 4 consecutive units: either way the swizzle spreads the 16 addresses
// over all banks.  It depends on row bits 0, 1, 3 and 4 alone, so a lane's swizzle is the same
// in all its reads.
template <int U>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (U == 4) return (r >> 3) & 3;
  if constexpr (U == 8) return (((r >> 1) & 1) << 2) | ((r >> 3) & 3);
  return ((r & 3) << 2) | ((r >> 3) & 3);
}

// Left factor over 32 columns: eight consecutive elements from column c (a multiple of 8) of a row.
template <int U, int N>
__device__ __forceinline__ Part<N> load_row(lds_cparts lds, int row, int c, int plane) {
  const lds_cparts p = lds + row * U * 8 + ((c / 8) ^ swizzle<U>(row)) * 8;
  Part<N> a;
#pragma unroll
  for (int n = 0; n < N; ++n) a.p[n] = *(const MSM_LDS bf16x8*)(p + n * plane);
  return a;
}

// A value that all lanes share, in scalar registers: resources built from it need no loop over
// the lanes' values.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)x);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)x >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ bf16x8 read_tr(lds_cparts lo, lds_cparts hi) {
  struct {
    s16x4 lo, hi;
  } v;
  v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MSM_LDS s16x4*)(lo));
  v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MSM_LDS s16x4*)(hi));
  return __builtin_bit_cast(bf16x8, v);
}
// The same transposed: eight consecutive rows from row0 (a multiple of 8) of the column this lane
// supplies, column c + spread (m / 4) + m % 4 for lane m of its group.  ds_read_b64_tr_b16: the 16
// lanes of a group read a block of 4 rows x 16 columns, lane i row i / 4 and four consecutive
// columns from chunk i % 4, and receive it transposed, lane i the four rows of column i.
template <int U, int N>
__device__ __forceinline__ Part<N> load_col(lds_cparts lds, int row0, int c, int spread, int lane, int plane) {
  const int i = lane & 15, row = row0 + (i >> 2), col = c + spread * (i & 3);
  const lds_cparts p = lds + row * U * 8 + ((col / 8) ^ swizzle<U>(row)) * 8 + col % 8;
  Part<N> a;
#pragma unroll
  for (int n = 0; n < N; ++n) a.p[n] = read_tr(p + n * plane, p + n * plane + 4 * U * 8);
  return a;
}
// Transposed from rows of `ld` elements.
template <int N>
__device__ __forceinline__ Part<N> load_col_ld(lds_cparts row0, int ld, int c, int lane, int plane) {
  const int i = lane & 15;
  const lds_cparts p = row0 + (i >> 2) * ld + c + 4 * (i & 3);
  Part<N> a;
#pragma unroll
  for (int n = 0; n < N; ++n) a.p[n] = read_tr(p + n * plane, p + n * plane + 4 * ld);
  return a;
}
template <int N>
__device__ __forceinline__ Part<N> load_ld(lds_cparts p, int plane) {
  Part<N> a;
#pragma unroll
  for (int n = 0; n < N; ++n) a.p[n] = *(const MSM_LDS bf16x8*)(p + n * plane);
  return a;
}

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
  // int32 arithmetic: offsets are below 2^31
  int64_t a = p.off[s], b = p.off[s + 1];
  a = a < 0 ? 0 : (a > p.tokens ? p.tokens : a);
  b = b < a ? a : (b > p.tokens ? p.tokens : b);
  return SeqRows{uniform(a), uniform(b - a), uniform((int)((uint32_t)a / C)) + s};
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
    s = uniform((int)((uint32_t)slot / (uint32_t)p.NT));
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

// Segments of a sequence: seg_len chunks each, numbered over all sequences as chunks are, sequence s
// from floor(slot0 / seg_len) + s on.  Without segments (seg_len 0) a sequence is one.
struct SeqSegs {
  int64_t first, count;
};
template <int C>
__device__ __forceinline__ SeqSegs seq_segs(const DeltaArgs& p, int64_t s) {
  if (p.seg_len == 0) return SeqSegs{s, 1};
  const SeqRows r = seq_rows<C>(p, s);
  const uint32_t M = (uint32_t)p.seg_len, chunks = (uint32_t)((r.len + C - 1) / C);
  const int count = uniform((int)((chunks + M - 1) / M));
  const int first = uniform((int)((uint32_t)r.slot0 / M));
  return SeqSegs{first + s, count < 1 ? 1 : count};
}

// Rows and first slot of a segment; s < 0 where there is none.
struct SegRows {
  int64_t s, row0, len, slot0;
  bool last;
};
template <int C>
__device__ __forceinline__ SegRows seg_rows(const DeltaArgs& p, int seg) {
  int64_t s = seg, g = 0;
  if (p.seg_len > 0) {
    int lo = 0, hi = (int)p.nseq;  // the last sequence whose first segment is at or before this one
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (seq_segs<C>(p, mid).first <= seg)
        lo = mid;
      else
        hi = mid;
    }
    s = uniform(lo);
  }
  const SeqSegs q = seq_segs<C>(p, s);
  const SeqRows r = seq_rows<C>(p, s);
  g = seg - q.first;
  if (g < 0 || g >= q.count) return SegRows{-1, 0, 0, 0, false};
  if (p.seg_len == 0) return SegRows{s, r.row0, r.len, r.slot0, true};
  const int64_t rows = (int64_t)p.seg_len * C, left = r.len - g * rows;
  return SegRows{s, r.row0 + g * rows, left < rows ? left : rows, r.slot0 + g * p.seg_len, g + 1 == q.count};
}

// ---- memory ----
constexpr uint32_t kOutside = 0x80000000u;  // an offset past any resource: reads zero, writes nothing

__device__ __forceinline__ u32x4 bload16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ f32x4 bload4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// The rows of one head of a chunk in a (rows, heads, size) array.  Rows past the chunk read as zero
// and are never written.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t head_rsrc(const void* base, int64_t row0, int64_t heads, int64_t h,
                                                             int64_t size, int es, int rows) {
  const char* p = static_cast<const char*>(base) + ((row0 * heads + h) * size) * es;
  return make_rsrc(p, rows > 0 ? ((rows - 1) * heads + 1) * size * es : 0);
}

// One pass of a wavefront from memory into LDS, 64 units of 16 bytes, without registers between
// (buffer_load ... lds, at m0 plus 16 bytes a lane); `lds` is the same for the whole wavefront.
// Written as assembly: before an LDS read that it cannot tell apart from the built-in's target
// the compiler waits for the load, also where the target is the other buffer, and so for the
// memory latency that the second buffer is there to hide.  It has no result register; sync_loads
// waits for it by hand, and waits that the compiler counts for other loads only get longer.
// The compiler does not look into it for wait states either, so it brings its own: a load needs 5
// after a vector instruction's write of a scalar register that it reads (the resource's extent, often
// a v_readfirstlane), 1 after m0's write.  The move to m0 is one of them and s_nop 3 the other four.
__device__ __forceinline__ void load_lds(u32x4 r, MSM_LDS void* lds, uint32_t off) {
#ifdef __HIP_DEVICE_COMPILE__
  const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)lds);
  // m0 is named as changed; the compiler, which reserves it, warns that it would not save it, and need
  // not: no kernel here has another use of it
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(r) : "m0");
#pragma clang diagnostic pop
#endif
}
// The resource of make_rsrc_u32 in its four words.
__device__ __forceinline__ u32x4 rsrc_words(const void* base, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, bytes, 0x00020000u};
}

// Barriers of the walks.  A barrier by itself is no obstacle to the scheduler's moving loads from
// memory into LDS across it, so both sides are closed.  After sync_loads every wavefront's
// load_lds have landed: each waits for its own first.
__device__ __forceinline__ void sync_lds() {
  __builtin_amdgcn_sched_barrier(0);
  __syncthreads();
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void sync_loads() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __syncthreads();
  __builtin_amdgcn_sched_barrier(0);
}

// Chunk matrices (lower triangular, C x C) are kept as their 32 x 32 blocks on and below the
// diagonal, (0,0), (1,0), (1,1), each in swizzled rows, in memory as in LDS; planes follow each
// other.
template <int C>
struct Tri {
  static constexpr int U = 4, kBlock = 32 * 32, kPlane = kBlock * (C / 32) * (C / 32 + 1) / 2;
  static __device__ __forceinline__ int block(int rb, int kb) { return (rb * (rb + 1) / 2 + kb) * kBlock; }
  // place of an element on or below the block diagonal
  static __device__ __forceinline__ int at(int row, int col) {
    const int r = row & 31, c = col & 31;
    return block(row >> 5, col >> 5) + r * 32 + ((c / 8) ^ swizzle<U>(r)) * 8 + c % 8;
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
