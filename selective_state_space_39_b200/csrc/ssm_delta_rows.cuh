// ssm_delta_rows.cuh -- what the two walks over the chunks of the gated delta
// rule share (ssm_delta_tc.cu): the shared-memory plan and its copies, a warp's
// 16 rows of the state and of the chunk's matrices as accumulator-shaped
// fragments, bounded waits.
#pragma once

#include <algorithm>

#include "ssm_delta.cuh"

namespace ssm {

namespace {

constexpr int kC = kDeltaChunk;

static __device__ int g_delta_timeout;  // set by a CTA that gave up a bounded wait

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

constexpr int kMaxStages = 4;
constexpr int kMaxBlocks = 8;  // 16-row blocks per CTA

// Shared memory: `stages` x [k/q tiles | head blocks], then per 16-row block two
// buffers of `tiles` column tiles (64 tokens x 16 columns).
constexpr int kCol = kC * 32;  // bytes of a column tile
struct Layout {
  int kq, head, head_off, heads, stage;  // bytes; heads of a CTA
};
// `blocks` 16-row blocks per CTA out of heads of `per_head` blocks each; the
// bytes from head_off of every head block (the walk back starts at the factors).
__host__ __device__ inline Layout layout(int dstate, int blocks, int per_head, int head_bytes,
                                         int head_off) {
  Layout l;
  l.head_off = head_off;
  l.kq = 2 * kC * dstate * 2;
  l.head = head_bytes;
  l.heads = per_head % blocks == 0 ? 1
            : blocks % per_head == 0 ? blocks / per_head
                                     : (blocks + per_head - 2) / per_head + 1;
  l.stage = (l.kq + l.heads * l.head + 1023) / 1024 * 1024;  // the swizzle's period
  return l;
}

// Byte offset of the lane's row in a fragment load (ldmatrix, stmatrix) of 16
// tokens of a column tile.
__device__ __forceinline__ uint32_t lane_col(int lane) {
  return col_at((lane & 7) + ((lane & 16) >> 1), (lane >> 3) & 1);
}

// x *= per-row factors (rows g and g + 8)
template <int T>
__device__ __forceinline__ void scale_rows(float (&x)[T][4], float f0, float f1) {
#pragma unroll
  for (int j = 0; j < T; ++j) {
    const float2 a = mul2(make_float2(x[j][0], x[j][1]), make_float2(f0, f0));
    const float2 b = mul2(make_float2(x[j][2], x[j][3]), make_float2(f1, f1));
    x[j][0] = a.x; x[j][1] = a.y;
    x[j][2] = b.x; x[j][3] = b.y;
  }
}
// x *= per-token factors (columns)
template <int T>
__device__ __forceinline__ void scale_cols(float (&x)[T][4], const float* f, int lane) {
#pragma unroll
  for (int j = 0; j < T; ++j) {
    const float2 c = *reinterpret_cast<const float2*>(f + 8 * j + 2 * (lane & 3));
    const float2 a = mul2(make_float2(x[j][0], x[j][1]), c);
    const float2 b = mul2(make_float2(x[j][2], x[j][3]), c);
    x[j][0] = a.x; x[j][1] = a.y;
    x[j][2] = b.x; x[j][3] = b.y;
  }
}
template <int T>
__device__ __forceinline__ void add_tiles(float (&x)[T][4], const float (&y)[T][4]) {
#pragma unroll
  for (int j = 0; j < T; ++j) {
    const float2 a = add2(make_float2(x[j][0], x[j][1]), make_float2(y[j][0], y[j][1]));
    const float2 b = add2(make_float2(x[j][2], x[j][3]), make_float2(y[j][2], y[j][3]));
    x[j][0] = a.x; x[j][1] = a.y;
    x[j][2] = b.x; x[j][3] = b.y;
  }
}
// The 16 columns of a column tile [token][p] as fp32 accumulator-shaped values
// [p][token], tokens t0 .. t0 + 8 T - 1.
template <int T>
__device__ __forceinline__ void load_rows(float (&x)[T][4], uint32_t tile, int t0, uint32_t lc) {
#pragma unroll
  for (int jp = 0; jp < T / 2; ++jp) {
    uint32_t r[4];
    ldsm4t(r, tile + (t0 + 16 * jp) * 32 + lc);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = 2 * jp + (q >> 1), e = (q & 1) * 2;
      x[j][e] = bf16_lo(r[q]);
      x[j][e + 1] = bf16_hi(r[q]);
    }
  }
}

// Accumulator-shaped values [p][token] of tokens t0 .. -> bf16 rows of a column
// tile, and (after it) those rows to global memory, 32 bytes a token.
template <int T>
__device__ __forceinline__ void stage_rows(const float (&x)[T][4], uint32_t tile, int t0, uint32_t lc) {
#pragma unroll
  for (int jp = 0; jp < T / 2; ++jp) {
    uint32_t r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = 2 * jp + (q >> 1), e = (q & 1) * 2;
      r[q] = pack_bf16x2(x[j][e], x[j][e + 1]);
    }
    stsm4t(tile + (t0 + 16 * jp) * 32 + lc, r);
  }
  __syncwarp();
}
template <int T>
__device__ __forceinline__ void store_rows(uint32_t tile, int t0, uint16_t* out, size_t out_stride,
                                           int valid, int lane) {
#pragma unroll
  for (int it = 0; it < T / 2; ++it) {
    const int tk = t0 + it * 16 + (lane >> 1), u = lane & 1;
    uint4 w;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(tile + col_at(tk, u))
                 : "memory");
    if (tk < valid) *reinterpret_cast<uint4*>(out + (size_t)tk * out_stride + u * 8) = w;
  }
}

// What rounding to bf16 leaves of the values.
template <int T>
__device__ __forceinline__ void rest_of(float (&x)[T][4]) {
#pragma unroll
  for (int j = 0; j < T; ++j)
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const uint32_t r = pack_bf16x2(x[j][q], x[j][q + 1]);
      x[j][q] -= bf16_lo(r);
      x[j][q + 1] -= bf16_hi(r);
    }
}

// Asynchronous copy of tokens t0 .. t0 + 8 T - 1 of 16 columns into a column
// tile; tokens from `valid` on become zero. src: the chunk's first token.
template <int T>
__device__ __forceinline__ void fetch_rows(uint32_t tile, const uint16_t* src, size_t stride, int t0,
                                           int valid, int lane) {
#pragma unroll
  for (int it = 0; it < T / 2; ++it) {
    const int tk = t0 + it * 16 + (lane >> 1), u = lane & 1;
    const bool in = tk < valid;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tile + col_at(tk, u)),
                 "l"(src + (in ? (size_t)tk * stride : 0) + u * 8), "r"(in ? 16 : 0)
                 : "memory");
  }
}

// Per-token dot products of x and y over the warp's 16 rows -> out[8 T].
template <int T>
__device__ __forceinline__ void row_dots(const float (&x)[T][4], const float (&y)[T][4],
                                         float* out, int lane) {
#pragma unroll
  for (int j = 0; j < T; ++j) {
    float a = fmaf(x[j][0], y[j][0], x[j][2] * y[j][2]);
    float b = fmaf(x[j][1], y[j][1], x[j][3] * y[j][3]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (lane < 4) *reinterpret_cast<float2*>(out + 8 * j + 2 * lane) = make_float2(a, b);
  }
}

// The warp's 16 rows of NS columns of a state of N columns (zero without src).
template <int N, int NS>
__device__ __forceinline__ void load_state(float (&s)[NS / 8][4], const float* src, int lane) {
  const float* r0 = src + (lane >> 2) * N + 2 * (lane & 3);
#pragma unroll
  for (int j = 0; j < NS / 8; ++j) {
    const float2 z = make_float2(0.f, 0.f);
    const float2 a = src ? *reinterpret_cast<const float2*>(r0 + 8 * j) : z;
    const float2 b = src ? *reinterpret_cast<const float2*>(r0 + 8 * N + 8 * j) : z;
    s[j][0] = a.x; s[j][1] = a.y; s[j][2] = b.x; s[j][3] = b.y;
  }
}
template <int N, int NS>
__device__ __forceinline__ void store_state(const float (&s)[NS / 8][4], float* dst, int lane) {
  float* r0 = dst + (lane >> 2) * N + 2 * (lane & 3);
#pragma unroll
  for (int j = 0; j < NS / 8; ++j) {
    *reinterpret_cast<float2*>(r0 + 8 * j) = make_float2(s[j][0], s[j][1]);
    *reinterpret_cast<float2*>(r0 + 8 * N + 8 * j) = make_float2(s[j][2], s[j][3]);
  }
}
// The warp's part of a state for the walk back, whose warps hold the same
// fragments: fragment by fragment, 512 contiguous bytes of a tile (row-major
// stores, 32 bytes of a row at a time, took longer than the chunk's arithmetic).
template <int NS>
__device__ __forceinline__ void store_tiles(const float (&s)[NS / 8][4], float* dst, int lane) {
#pragma unroll
  for (int j = 0; j < NS / 8; ++j)
    *reinterpret_cast<float4*>(dst + (j * 32 + lane) * 4) =
        make_float4(s[j][0], s[j][1], s[j][2], s[j][3]);
}
// Such a part, asynchronously into shared memory (a lane reads what it copied),
// and <s, it> (all lanes).
template <int NS>
__device__ __forceinline__ void fetch_tiles(uint32_t to, const float* src, int lane) {
#pragma unroll
  for (int j = 0; j < NS / 8; ++j)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + (j * 32 + lane) * 16),
                 "l"(src + (j * 32 + lane) * 4)
                 : "memory");
}
template <int NS>
__device__ __forceinline__ float tiles_dot(const float (&s)[NS / 8][4], const float* tiles, int lane) {
  float2 d0 = make_float2(0.f, 0.f), d1 = d0;
#pragma unroll
  for (int j = 0; j < NS / 8; ++j) {
    const float4 v = *reinterpret_cast<const float4*>(tiles + (j * 32 + lane) * 4);
    d0 = fma2(make_float2(s[j][0], s[j][1]), make_float2(v.x, v.y), d0);
    d1 = fma2(make_float2(s[j][2], s[j][3]), make_float2(v.z, v.w), d1);
  }
  float d = (d0.x + d0.y) + (d1.x + d1.y);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  return d;
}
// The rows as bf16, row-major (for the products of ssm_delta_grad.cu, whose
// results are bf16): through shared memory (rows of NS + 8 values), whole rows
// of NS values to global memory.
template <int N, int NS>
__device__ __forceinline__ void store_state16(const float (&s)[NS / 8][4], uint32_t rows, uint16_t* dst,
                                              int lane) {
  constexpr int kRow = (NS + 8) * 2;
  const uint32_t at = rows + ((lane & 7) + (lane & 8)) * kRow + (lane >> 4) * 16;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < NS / 8; j += 2)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at + j * 16),
                 "r"(pack_bf16x2(s[j][0], s[j][1])), "r"(pack_bf16x2(s[j][2], s[j][3])),
                 "r"(pack_bf16x2(s[j + 1][0], s[j + 1][1])), "r"(pack_bf16x2(s[j + 1][2], s[j + 1][3]))
                 : "memory");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16 * NS / 8; i += 32) {
    const int row = (i + lane) / (NS / 8), u = (i + lane) % (NS / 8);
    uint4 w;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(rows + row * kRow + u * 16)
                 : "memory");
    *reinterpret_cast<uint4*>(dst + (size_t)row * N + u * 8) = w;
  }
}

// ---------------------------------------------------------------- the CTA ----
// SP warps share a block of 16 rows (SP = 2: half of dstate each).
struct Cta {
  int b, kh, rb0, active, h0, nheads;  // row blocks of this CTA in its key head's group
};
__device__ __forceinline__ Cta cta_of(const DeltaChunkParams& p) {
  const DeltaParams& d = p.d;
  Cta c;
  const int pb = d.headdim / 16, group = d.nheads / d.nkheads * pb;
  const int slices = (group + p.blocks - 1) / p.blocks;
  const int bk = blockIdx.x / slices, sl = blockIdx.x - bk * slices;
  c.b = bk / d.nkheads;
  c.kh = bk - c.b * d.nkheads;
  c.rb0 = sl * p.blocks;
  c.active = min(p.blocks, group - c.rb0);
  const int first = c.rb0 / pb;
  c.nheads = (c.rb0 + c.active - 1) / pb - first + 1;
  c.h0 = c.kh * (d.nheads / d.nkheads) + first;
  return c;
}

// One thread: issues the copies of chunk c into stage st.
__device__ __forceinline__ void issue(const DeltaChunkParams& p, const Cta& t, const Layout& l,
                                      unsigned char* smem, uint64_t* full, int c, int st) {
  const DeltaParams& d = p.d;
  const size_t bc = (size_t)t.b * p.nchunks + c;
  unsigned char* base = smem + (size_t)st * l.stage;
  mbar_arrive_expect_tx(&full[st], (uint32_t)(l.kq + t.nheads * l.head));
  bulk_load(smem_u32(base), p.ws_kq + (bc * d.nkheads + t.kh) * (size_t)l.kq, l.kq, &full[st]);
  for (int i = 0; i < t.nheads; ++i)
    bulk_load(smem_u32(base + l.kq + i * l.head),
              p.ws_head + (bc * d.nheads + t.h0 + i) * (size_t)p.head_bytes + l.head_off, l.head,
              &full[st]);
}

// Both warps of a pair reach this; false for both if either's wait ran out.
__device__ __forceinline__ bool pair_and(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void pair_sync(int id) {
  asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory");
}
// The chunk's tiles and the warp's own column tiles are there.
__device__ __forceinline__ bool wait_stage(uint64_t* bar, uint32_t parity, uint64_t limit) {
  cp_async_wait_group<0>();
  const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit));
  __syncwarp();
  return ok;
}
// A wait ran out at step s: note it, and leave only when the copies already
// issued have landed (or that wait, too, has run out).
__device__ __forceinline__ void give_up(const DeltaChunkParams& p, uint64_t* full, int s) {
  if ((threadIdx.x & 31) == 0) atomicExch(&g_delta_timeout, 1);
  for (int i = s; i < s + p.stages && i < p.nchunks; ++i)
    mbar_wait_bounded(&full[i % p.stages], (uint32_t)((i / p.stages) & 1), p.wait_limit_ns);
}

// Whether a wait of this file's kernels ran out since the last call.
cudaError_t timeout_status(cudaStream_t stream, int* timed_out) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  const int zero = 0;
  e = cudaMemcpyFromSymbol(timed_out, g_delta_timeout, sizeof(int));
  if (e != cudaSuccess || !*timed_out) return e;
  return cudaMemcpyToSymbol(g_delta_timeout, &zero, sizeof(int));
}

}  // namespace
}  // namespace ssm
