// ssm_delta_internal.h -- parameters of the gated delta rule shared by the C
// entry points (ssm_api.cu) and its kernels (ssm_delta_step.cu: token by token;
// ssm_delta_prep.cu, ssm_delta_tc.cu, ssm_delta_grad.cu: chunk by chunk). Not
// part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

constexpr int kDeltaChunk = 64;        // tokens per chunk
constexpr int kMaxShared = 224 * 1024;  // dynamic, beside 3 KB of static shared memory
constexpr float kDeltaQkEps = 1e-6f;   // |x|^2 + eps under the unit-length scaling

struct DeltaParams {
  int batch, nheads, nkheads, headdim, dstate;
  int64_t seqlen;
  int softplus, beta_sigmoid, qk_norm;
  float scale;
  const void* q;         // (batch, seqlen, nkheads, dstate) io
  const void* k;         // (batch, seqlen, nkheads, dstate) io
  const void* v;         // (batch, seqlen, nheads, headdim) io
  const void* dt;        // (batch, seqlen, nheads) io
  const void* beta;      // (batch, seqlen, nheads) io
  const float* A;        // (nheads)
  const float* dt_bias;  // (nheads) or null
  const float* h0;       // (batch, nheads, headdim, dstate) or null
  void* y;               // (batch, seqlen, nheads, headdim) io or null
  float* h_last;         // (batch, nheads, headdim, dstate) or null
};

// Lets a kernel take kMaxShared: one limit for every launch, so that calls from
// several threads cannot lower it under one another.
template <typename K>
inline cudaError_t allow_shared(K* kern) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
}

// dstate values of the token-by-token kernel (any headdim, fp32 or bf16 io).
bool delta_step_dstate_supported(int dstate);
cudaError_t launch_delta_step(const DeltaParams& p, bool bf16, cudaStream_t stream);

// ---- chunk by chunk (bf16 io) ---------------------------------------------
// Per (batch row, chunk, key head) the workspace holds k and q as fp16 tiles,
// every row scaled by a power of two, in blocks of 64 tokens x 64 columns with
// the 128-byte swizzle; per (batch row, chunk,
// head) a block of per-token factors and the 64 x 64 tiles of the chunk.
enum DeltaScal {       // arrays of 64 floats in a head block; the forward pass reads the first seven
  kScSk = 0,           // e^G kmul: S k16 -> the decayed prediction of v
  kScU = 1,            // beta 2^-t: (T16 R) -> u
  kScKend = 2,         // kmul e^(G_end - G): u -> its weight in the end state
  kScK = 3,            // kmul: k = kmul k16
  kScSq = 4,           // e^G qmul: S q16 -> y
  kScP = 5,            // qmul 2^-p: (P16 u) -> y
  kScEnd = 6,          // [0]: e^G_end; [1], [2]: the largest e^(G_end - G) of either half, at least 1;
                       // [3], [4]: 1 where a half has a log decay below kStrongDecay;
                       // [5]: 1 where rows went token by token (set by the walk)
  kScT = 7,            // 2^-t: (T16 R) -> r
  kScBeta = 8,
  kScGhi = 9,          // the running log decay, high and low part
  kScGlo = 10,
  kScKn = 11,          // unit-length factor of k
  kScQn = 12,          // unit-length factor of q, times the readout scale
  kScRatio = 13,       // beta over its floored value (delta_beta_floor)
  kScCount = 14,
};
// The backward pass takes a token's dbeta from its dv = beta du, so there T and dU
// meet a beta of at least 2^-26 (r is then off by less than its own rounding), and dv
// is scaled back afterwards.
constexpr float kBetaFloor = 1.f / 67108864.f;
// From here on a decay's gradient, about e^g of the terms that suffix sums make it
// of (2^-24 each), comes from the pairs of tokens on either side (ssm_delta_grad.cu).
// Suffix sums leave a head's dA off by 5e-4 at e^-5, 4e-3 at e^-8 and all of it at
// e^-16, the pairs 1e-6 at any decay. A head and chunk with such a decay takes about 11 us more of
// an SM: from e^-4 on, ordinary layers would pay 15 us of 450 for a few of them.
constexpr float kStrongDecay = -5.f;
// A row of T or P stands under one scale too. With unit-length keys and beta below 1 its
// entries are alike; a chunk whose keys differ by 2^16 in length, or with a beta of 2^10,
// or whose T grows to 2^20 goes token by token: its first kScSk is NaN, and the walks
// find a value that is not finite in every row.
constexpr float kOddKeys = 65536.f, kOddBeta = 1024.f, kOddT = 1048576.f;
// A lower triangular 64 x 64 fp16 tile: its ten 16 x 16 blocks (i, j <= i),
// column of blocks by column, 512 bytes each, as 2 x 2 core matrices of eight
// rows of 16 bytes (the tensor cores' layout without a swizzle; any eight rows
// at one column lie in eight bank groups).
constexpr int kDeltaTri = 10 * 512;
__host__ __device__ constexpr int delta_tri_block(int i, int j) {
  return j * 2048 - 256 * j * (j - 1) + (i - j) * 512;
}
// The same of a transposed tile (upper triangular), row of blocks j of block
// column i: a step over 16 rows of the original reaches its columns 0 .. i.
__host__ __device__ constexpr int delta_tri_block_t(int i, int j) { return 256 * i * (i + 1) + j * 512; }
constexpr int kDeltaScalFwd = 7 * kDeltaChunk * 4, kDeltaScalBwd = kScCount * kDeltaChunk * 4;
// A head block: T hi, T lo, P hi, then the factors; for the backward pass T and P
// hi and lo, the factors, and the same four tiles transposed.
constexpr int kDeltaHeadFwd = 3 * kDeltaTri + kDeltaScalFwd;
constexpr int kDeltaLoadBwd = 4 * kDeltaTri + kDeltaScalBwd;  // what either walk reads
constexpr int kDeltaHeadBwd = kDeltaLoadBwd + 4 * kDeltaTri;

struct DeltaChunkParams {
  DeltaParams d;
  int nchunks;
  int head_bytes;        // kDeltaHeadFwd or kDeltaHeadBwd
  unsigned char* ws_kq;  // (batch, nchunks, nkheads) x [k16 tile | q16 tile]
  unsigned char* ws_head;  // (batch, nchunks, nheads) x head block
  uint64_t wait_limit_ns;
  int test_stall;
  int blocks, stages;    // 16-row blocks of the state and tile stages per CTA (set by the launch)
  // backward only
  const uint16_t* dy;    // (batch, seqlen, nheads, headdim)
  const float* dh_last;  // or null
  float* ws_state;       // (batch, nchunks, nheads, headdim x dstate): state after each chunk, in fragments
  uint16_t* ws_state16;  // (..., headdim, dstate): before each chunk, bf16
  uint16_t* ws_dstate16; // ... its adjoint after each chunk, bf16
  float* ws_end;         // (batch, nchunks, nheads, headdim/16, 2): <state, adjoint> after each chunk
  float* ws_first;       // (batch, nheads, headdim/16, 2): ... before the first, with an initial state
  uint16_t* ws_r;        // (batch, seqlen, nheads, headdim): v minus the state's prediction
  uint16_t* ws_rlo;      // what r's rounding leaves, in chunks with a strong decay (either half)
  uint16_t* ws_dvlo;     // ... dv's
  float* ws_doto;        // (batch, nchunks, nheads, headdim/16, 64): dy.y over 16 rows
  float* ws_dotv;        //   ... dv.v
  float* ws_doth;        //   ... e^(G_end - G) r . dS k, in chunks with a strong decay
  float* ws_dotb;        //   ... dv.r, before dv is scaled back to the token's own beta
  double* ws_part;       // (batch, nchunks, nheads, 2): partial dA, ddt_bias
  uint16_t *dq, *dk, *dv, *ddt, *dbeta;
  float *dA, *ddt_bias, *dh0;
};

cudaError_t launch_delta_prep(const DeltaChunkParams& p, bool bwd, cudaStream_t stream);
// The walk over the chunks (bwd: it keeps what the gradients need), and in reverse.
bool delta_chunk_supported(int dstate, int headdim);
cudaError_t launch_delta_fwd(const DeltaChunkParams& p, bool bwd, cudaStream_t stream);
cudaError_t launch_delta_rev(const DeltaChunkParams& p, cudaStream_t stream);
cudaError_t launch_delta_grad(const DeltaChunkParams& p, cudaStream_t stream);
// Whether a bounded wait gave up since the last call (synchronises the stream).
cudaError_t delta_chunk_status(cudaStream_t stream, int* timed_out);

}  // namespace ssm
