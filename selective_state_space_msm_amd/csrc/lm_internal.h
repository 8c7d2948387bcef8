// Internal interface between the C-ABI layer (lm_api.cpp) and the kernels of the operators at a
// language model's ends and between its blocks: embedding, block norm, linear cross entropy.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace msm {

// ---- embedding ----

struct EmbedArgs {
  const int64_t* ids;  // (tokens,)
  const void* table;   // (V, D) table type
  void* y;             // (tokens, D) I/O type
  const void* dy;      // backward
  void* dtable;        // (V, D) table type
  // workspace of the backward
  uint32_t* key[2];    // (tokens,) ids, V for the positions without a token
  uint32_t* pos[2];    // (tokens,) their positions
  uint32_t* hist;      // [wavefronts][bins]
  float* part[2];      // sums of 32 and of 1024 places of the sorted list, D each
  int64_t tokens, V, D;
  float scale;
  int32_t waves, per;  // wavefronts of a sorting pass and their places (a multiple of 64)
  int32_t bits;        // of a digit
  int32_t passes;
  const int32_t* rows; // what a sorted position is to be given as, null: as it is
};

constexpr int kEmbedMostBits = 9;      // of a digit: 512 bins
constexpr int kEmbedSmall = 4096;      // places that one workgroup sorts in LDS
constexpr int kEmbedDeep = 8192;       // places from which there are sums of the second level
constexpr int kEmbedRun = 32;          // places of a sum of the first level, and sums of the second
hipError_t launch_embed_fwd(const EmbedArgs& a, int table_bf16, int io_bf16, hipStream_t s);
hipError_t launch_embed_bwd(const EmbedArgs& a, int table_bf16, int io_bf16, hipStream_t s);
// The sort alone, stable, into key and pos [(passes - 1) & 1]; clears `fill` bytes at dtable.
hipError_t launch_embed_sort(const EmbedArgs& a, int64_t fill, hipStream_t s);

// ---- block norm ----

struct BlockNormArgs {
  const void* r;             // (rows, D) I/O type
  const void* o;             // or null
  const void* z;             // or null
  const float* weight;       // (D,) or null (ones)
  const float* post_weight;  // (D,) or null (ones)
  void* r_out;               // written by the forward when o is given, read by the backward
  void* y;
  float* rstd;
  float* post_rstd;
  const void* dy;            // backward
  const void* dr_out;        // or null
  void* dr;
  void* do_;
  void* dz;
  float* dweight;
  float* dpost_weight;
  float* part;               // [groups][2][D] column sums, or null
  float* row_mean;           // (rows,) of the first reduction, for rows past the registers
  int64_t rows, D;
  float scale, eps;
  int32_t groups;
};

// T threads hold a row, E elements each: 16, 32 or 64, or as many wavefronts as it takes; T = 0: the row is
// walked in memory.  E leaves the registers room for enough wavefronts: a backward's fp32 row has five arrays in
// flight and five in use, 256 registers a thread with 16 elements and 92 with 4 (16384 x 4096: 589 and 396 us;
// 4095 x 1001: 43 and 28), with 8 in 128 (4000 x 6000: 358 and 283); up to 512 columns a wavefront a row, which
// has no barriers (50000 x 400: 129, with 4 elements 134).  In bf16 16 elements are two loads an array, and fewer
// barriers for the same work (16384 x 4096, backward: 205 us, with 8 elements 257; 7098 x 2240: 77 and 106); up
// to 1024 columns 8 (20000 x 1000: 99 with 16, 81).  A forward has three arrays: 8 elements (20000 x 1000: bf16
// 55 with 16, 44, fp32 89 and 80; 50000 x 200: bf16 41 and 29, fp32 57 and 38).
struct BlockNormShape {
  int T, E;
};
constexpr BlockNormShape block_norm_shape(int64_t D, bool bwd, bool bf16) {
  if (D > (bwd ? 8192 : 16384)) return BlockNormShape{0, 0};
  const int E = !bwd ? (D <= 8192 ? 8 : 16) : (bf16 ? (D <= 1024 ? 8 : 16) : (D <= 256 || (D > 512 && D <= 4096) ? 4 : 8));
  for (int T = 16; T <= 64; T *= 2)
    if (D <= (int64_t)T * E) return BlockNormShape{T, E};
  return BlockNormShape{(int)((D + 64 * E - 1) / (64 * E)) * 64, E};
}
hipError_t launch_block_norm_fwd(const BlockNormArgs& a, int io_bf16, hipStream_t s);
hipError_t launch_block_norm_bwd(const BlockNormArgs& a, int io_bf16, hipStream_t s);

// ---- linear cross entropy ----

// What a row that takes part needs in the epilogues.
struct XentRow {
  float lse, both, dloss;  // both: dloss + dlse
  int32_t target;
};

// A word's places among the targets in order.
struct XentPlaces {
  int32_t first, end;
};

struct XentArgs {
  const void* x;           // (T, D) I/O type
  const void* w;           // (V, D)
  const int64_t* targets;  // (T,)
  float* loss;             // (T,) forward
  float* lse;              // (T,) written by the forward (may be null there), read by the backward
  const float* dloss;      // (T,) backward
  const float* dlse;       // (T,) or null
  void* dx;                // (T, D)
  void* dw;                // (V, D) or null
  // workspace
  int32_t* count;          // rows that take part
  int32_t* map;            // (T,) their places in x
  int32_t* inverse;        // (T,) and back, -1 for a row that is left out; null: rows as they come
  XentRow* rows;           // (T,)
  void* xp;                // [planes][T][DP] bf16 parts of the rows that take part
  void* wp;                // [planes][piece][DP] the same of a piece of w, where w is not read directly
  float* stat;             // forward: [tiles of the vocabulary][T][2] largest logit, sum of exponentials
  float* at_target;        // forward: (T,) logit of the target, in units of log 2
  void* g;                 // backward: [planes][T][piece] gradient of a piece's logits
  float* dx_sum;           // backward: [splits][T][DQ]
  float* rest;             // backward, bf16: (T,) what the target's g lost to its rounding
  uint32_t* key;           // and with dw: (T,) the targets in order, V for rows that are left out
  uint32_t* pos;           // (T,) their places in xp
  XentPlaces* words;       // (V,) each word's places among these, 0, 0: none; null: nothing of this is asked for
  uint8_t* marks;          // for 16 words a byte: one of them has places
  float* lost;             // (T, DQ) sums of rest x over a word's places in one run, at the first of them
  int64_t T, V, D, DP, DQ, piece;
  float scale;
  int32_t planes;          // 1, or 3 for fp32
  int32_t w_direct;
  int32_t tile;            // side of the forward's tiles
  int32_t splits;          // of the vocabulary's pieces in the product of dx
  int32_t log_run;         // of the places of a run
  int64_t clear;           // bytes of words and marks, which follow each other
};
constexpr int kXentFew = 32;         // rows that the forward takes without tiles
constexpr int kXentPlaced = 512;     // rows that stay in their places, also those that are left out
// Bytes of the marks: four at a time are read, and a piece begins at a multiple of 256 words.
constexpr int64_t xent_marks(int64_t V) { return (V + 255) / 256 * 16; }
constexpr int kXentRanked = 4096;    // rows whose targets are put in order by counting
constexpr int kXentFewGroups = 256;  // workgroups it takes them with at most: one a CU
// Side of the tiles of an M x N product over K.  256 or 128 by rounds of the 256 CUs (one workgroup a CU, or
// two of the smaller tiles), a small tile taking a quarter of a large one's work at 0.8 of its rate; not 256
// where the tiles' ends are the work (64 tokens, 7178 x 6656, bf16: dW in 49 us, in tiles of 128 45).  64 where 128 leaves CUs idle:
// its five stages hide what two of 128 wait for (64 tokens of 7178, D = 6656, bf16: logits in 100 us, in tiles of 64 38).  Three planes
// of an fp32 tile fill the LDS at 128.
constexpr int xent_tile(int64_t M, int64_t N, int64_t K, int planes) {
  const int64_t large = ((M + 255) / 256) * ((N + 255) / 256), small = ((M + 127) / 128) * ((N + 127) / 128);
  if (planes > 1) return small >= 192 ? 128 : 64;
  if (K > 512 && (large + 255) / 256 * 8 <= (small + 511) / 512 * 5) return 256;
  return small >= 384 ? 128 : 64;
}
hipError_t launch_xent_fwd(const XentArgs& a, int io_bf16, hipStream_t s);
// sort: of the targets, for bf16 with dw and more than kXentRanked rows
hipError_t launch_xent_bwd(const XentArgs& a, const EmbedArgs& sort, int io_bf16, hipStream_t s);

}  // namespace msm
