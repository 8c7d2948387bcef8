// Internal interface between the C-ABI layer of the block operators (ops_api.cpp) and their
// kernels: the gated delta rule, layer norm, and the gradient norm with clipping.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace msm {

// ---- gated delta rule ----

constexpr int kDeltaMaxK = 256;  // key size a state may have (rows of S)

// Tokens per chunk: 64, but 32 where a chunk of fp32 keys and queries of the largest padded size,
// in their three parts, would not fit the 160 KB of LDS.
constexpr int delta_chunk(int io_bf16, int KP) { return (!io_bf16 && KP == 256) ? 32 : 64; }
// Key size padded to a size the kernels are built for.
constexpr int delta_padded_k(int64_t K) { return K <= 32 ? 32 : (K <= 64 ? 64 : (K <= 128 ? 128 : 256)); }
// bf16 planes that q and k are kept in: as they are, or fp32 in three parts.
constexpr int delta_in_planes(int io_bf16) { return io_bf16 ? 1 : 3; }

struct DeltaArgs {
  const void* q;        // (tokens, Hk, K) I/O dtype
  const void* k;
  const void* v;        // (tokens, H, V)
  const float* g;       // (tokens, H) log decay
  const float* beta;    // (tokens, H)
  const int32_t* off;   // (nseq + 1,) first row of each packed sequence, or null (uniform)
  const float* S0;      // (nseq, H, K, V) or null (zero)
  void* o;              // (tokens, H, V)
  float* last_S;        // (nseq, H, K, V) or null
  const void* do_;      // backward
  const float* dlast_S;
  void* dq;
  void* dk;
  void* dv;
  float* dg;
  float* dbeta;
  float* dS0;
  // workspace; sh = slot * H + head numbers the chunks
  float* vec;           // [sh][5 C]: e^G, e^(G_last - G), beta, G as doubles
  void* T;              // [sh][3 planes][blocks] inverse of the chunk's unit lower system
  void* P;              // [sh][3 planes][blocks] scale D tril(Q K^T)
  void* M;              // [sh][3 planes][blocks] D stril(K K^T)            (backward)
  void* kq;             // [slot][Hk][2][planes][C][KP] k and q as LDS holds them, unless kq_direct
  float* S;             // [sh][KP][VP] state before the chunk          (backward)
  float* dS;            // [sh][KP][VP] adjoint of the state after it   (backward)
  float* E;             // [sh][C][VP] prediction errors                (backward)
  float* dV;            // [sh][C][VP] gradient of v                    (backward)
  float* pred;          // [sh][C][VP] what the state before the chunk predicts (backward)
  float* dots;          // [sh][VP / 16][4 C] row sums over 16 columns (backward)
  float* segS;          // [segment][H][KP][VP] a segment's end state from zero, then its start
  float* segF;          // [segment][H][KP][KP] its map of the state
  int64_t tokens;       // rows of the token arrays
  int64_t nseq, L;      // uniform: nseq sequences of L tokens
  int64_t NT;           // uniform: chunks per sequence
  int64_t nslots;
  int64_t nsegs;        // segments at most
  int32_t seg_len;      // chunks of a segment, 0: sequences are walked whole
  int64_t Hk, H, K, V, VP;
  float scale;
  int32_t vec_k;        // rows of q and k can be read 16 bytes at a time
  int32_t kq_direct;    // and they need no conversion
  int32_t vec_v;        // rows of do can be read 16 bytes at a time
};

struct DeltaStepArgs {
  const void* q;        // (Bt, Hk, K)
  const void* k;
  const void* v;        // (Bt, H, V)
  const float* g;       // (Bt, H)
  const float* beta;
  float* S;             // (Bt, H, K, V), updated in place
  void* o;              // (Bt, H, V)
  int64_t Bt, Hk, H, K, V;
  float scale;
};

// One launch per stage; io_bf16 and the padded key size select the build.
#define MSM_DELTA_NAME_(stage, io, kp) launch_delta_##stage##_##io##_##kp
#define MSM_DELTA_NAME(stage, io, kp) MSM_DELTA_NAME_(stage, io, kp)
#define MSM_DELTA_DECL(io, kp)                                                         \
  hipError_t MSM_DELTA_NAME(fwd, io, kp)(const DeltaArgs& a, hipStream_t s);            \
  hipError_t MSM_DELTA_NAME(bwd, io, kp)(const DeltaArgs& a, hipStream_t s);
MSM_DELTA_DECL(0, 32)
MSM_DELTA_DECL(0, 64)
MSM_DELTA_DECL(0, 128)
MSM_DELTA_DECL(0, 256)
MSM_DELTA_DECL(1, 32)
MSM_DELTA_DECL(1, 64)
MSM_DELTA_DECL(1, 128)
MSM_DELTA_DECL(1, 256)
#undef MSM_DELTA_DECL

hipError_t launch_delta_step(const DeltaStepArgs& a, int io_bf16, hipStream_t s);

// ---- layer norm ----

struct NormArgs {
  const void* x;        // (rows, D) I/O dtype
  const float* weight;  // (D,) or null (ones)
  const float* bias;    // (D,) or null (zeros)
  void* y;
  float* mean;          // (rows,) written by the forward (may be null there), read by the backward
  float* rstd;
  const void* dy;       // backward
  void* dx;
  float* dweight;       // (D,) or null
  float* dbias;         // (D,) or null
  float* part;          // workspace: [groups][2][D] column sums of each workgroup's rows
  int64_t rows, D;
  float eps;
  int32_t groups;       // workgroups of the backward
  int32_t vec;          // rows can be read and written 16 bytes at a time
};

// How a row is spread over threads: T threads hold NV pieces of `vec` elements each; NV = 0
// means the row does not fit the registers and is walked in loops.
struct NormShape {
  int T, NV;
};
NormShape norm_shape(int64_t D, int per);
// Threads of a backward workgroup: two wide rows side by side where the registers allow two
// wavefronts a SIMD.  At 16384 x 4096 bf16, 256 workgroups of 512 threads take 81 us, 512 of 256
// threads 84 us (1024: 105 us, their column sums are as many bytes as an eighth of the rows), and
// 256 of 1024 threads 131 us, their barriers holding 16 wavefronts together.
constexpr int norm_threads(int T, int NV) { return T == 256 && NV <= 4 ? 512 : 256; }
hipError_t launch_norm_fwd(const NormArgs& a, int io_bf16, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, int io_bf16, hipStream_t s);
// dweight and dbias (either may be null) from `parts` pairs of column sums at `part`
hipError_t launch_norm_join(const NormArgs& a, int64_t parts, hipStream_t s);

// ---- gradient norm and clipping ----

constexpr int kClipTensors = 128;            // tensors whose addresses travel in one launch (3.7 KB of arguments)
constexpr int kClipChunk = 16384;            // elements a workgroup takes at a time
constexpr int kClipPartials = 2048;          // partial sums aimed at over all launches

struct ClipBatch {
  const void* src[kClipTensors];
  void* dst[kClipTensors];
  int64_t n[kClipTensors];
  uint32_t first[kClipTensors + 1];          // first chunk of each tensor
  uint8_t bf16[kClipTensors];
  int32_t count;
};

hipError_t launch_clip_sum(const ClipBatch& b, double* part, int groups, hipStream_t s);
hipError_t launch_clip_norm(const double* part, int64_t parts, float* norm, hipStream_t s);
// part null: `norm` holds the norm already; else it is joined from the parts, and written if non-null
hipError_t launch_clip_scale(const ClipBatch& b, const double* part, int64_t parts, float* norm,
                             float max_norm, float eps, int groups, hipStream_t s);

}  // namespace msm
