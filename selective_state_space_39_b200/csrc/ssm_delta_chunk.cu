// ssm_delta_chunk.cu -- the gated delta rule chunk by chunk (bf16 io, sm_100a):
// the forward pass over the chunks and, for the gradients, the reverse pass.
//
// Per head, with the operands of ssm_delta_prep.cu and the state S (headdim x
// dstate) entering a chunk:
//   R = V - (e^G K) S^T,  r = T R,  u = beta r
//   Y = (e^G Q) S^T + P u
//   S <- e^G_end S + u^T (e^(G_end - G) K)
// and in reverse, dS being the adjoint of the state after the chunk:
//   dU = P^T dY + e^(G_end - G) K dS^T,  dV = dR = T^T (beta dU)
//   dS <- e^G_end dS + dY^T (e^G Q) - dR^T (e^G K)
// The rows of S (one per output column p) never meet, so a warp owns 16 of
// them for the whole sequence: S^T lies in its accumulators (16 x dstate fp32),
// is turned into A fragments in registers, and r, u and the products stay
// there too. With few rows in all, two warps share 16 rows, half of dstate
// each: they exchange their parts of S K and S Q through shared memory (one
// barrier of the two per chunk), take r and u in full and half the tokens of y,
// which shortens the chain from chunk to chunk. A CTA takes neighbouring rows
// of the heads that share one key head. The tiles of a chunk come by two bulk
// copies (k and q; T, P and the factors of the CTA's heads), issued a stage
// ahead by whichever warp is the last to finish with the stage's old tiles, so
// no warp waits for another; a warp fetches its own columns of v (dy, r) by
// 16-byte asynchronous copies one chunk ahead, zero-filled past the end.
//
// Precision: the state path (S K, T R, S's update, and the reverse
// counterparts) takes fp32 operands as two fp16 pieces (ssm_delta.cuh), so the
// carried state, dh0 and the gate gradients keep fp32's accuracy; y, rounded
// to bf16, takes one fp16 piece of S, u and P (2^-12 each).
#include <stdlib.h>

#include <algorithm>

#include "ssm_delta.cuh"

namespace ssm {

namespace {

constexpr int kC = kDeltaChunk;

__device__ int g_delta_timeout;  // set by a CTA that gave up a bounded wait

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
  int kq, head, heads, tiles, stage;  // bytes; heads of a CTA; column tiles
};
// `blocks` 16-row blocks per CTA out of heads of `per_head` blocks each.
__host__ __device__ inline Layout layout(int dstate, int blocks, int per_head, int tiles,
                                         int head_bytes) {
  Layout l;
  l.kq = 2 * kC * dstate * 2;
  l.head = head_bytes;
  l.heads = per_head % blocks == 0 ? 1
            : blocks % per_head == 0 ? blocks / per_head
                                     : (blocks + per_head - 2) / per_head + 1;
  l.tiles = tiles;
  l.stage = l.kq + l.heads * l.head;
  return l;
}

// Pairs of neighbouring tiles += A times their B fragments. The accumulators of
// one piece are all visited before the next piece's, so that no MMA waits for
// the one before it.
template <int T, int P>
__device__ __forceinline__ void mma_tiles(float (&acc)[T][4], const uint32_t (&a)[4],
                                          const uint32_t (&b)[P][4], int t0 = 0) {
#pragma unroll
  for (int j = 0; j < P; ++j) {
    mma_f16(acc[t0 + 2 * j], a, b[j][0], b[j][1]);
    mma_f16(acc[t0 + 2 * j + 1], a, b[j][2], b[j][3]);
  }
}

// Lane's row/unit offsets of the two fragment loads (see swz):
//   nt: B rows are n          tr: B rows are k (transposing load)
struct LaneMap {
  int nt_row, nt_unit, tr_row, tr_unit;
  uint32_t nt_tri, tr_tri;  // the same inside a block of a triangular tile
  uint32_t nt_col;          // and of a column tile
};
__device__ __forceinline__ LaneMap lane_map(int lane) {
  LaneMap m;
  m.nt_row = (lane & 7) + ((lane & 16) >> 1);
  m.nt_unit = (lane >> 3) & 1;
  m.tr_row = (lane & 7) + (lane & 8);
  m.tr_unit = lane >> 4;
  m.nt_tri = tri_at(m.nt_row, m.nt_unit);
  m.tr_tri = tri_at(m.tr_row, m.tr_unit);
  m.nt_col = col_at(m.nt_row, m.nt_unit);
  return m;
}

// acc[16 x 8 TT tokens] += x[16 x 64 tokens] B over a triangular tile, x as two
// pieces, B as one or two. TR false: B[n][k], blocks n >= k, the accumulators
// holding the tokens from 16 jp0 on; true: B[k][n] (TT = 8, jp0 = 0).
template <bool TR, bool XLO, bool BLO, int TT>
__device__ __forceinline__ void tri_product(float (&acc)[TT][4], const float (&x)[8][4], float s0,
                                            float s1, uint32_t bhi, uint32_t blo, int jp0,
                                            const LaneMap& m) {
#pragma unroll
  for (int kt = 0; kt < 4; ++kt) {
    uint32_t hi[4], lo[4];
    if (XLO)
      split_a(x[2 * kt], x[2 * kt + 1], s0, s1, hi, lo);
    else
      half_a(x[2 * kt], x[2 * kt + 1], s0, s1, hi);
    uint32_t bh[TT / 2][4], bl[TT / 2][4];
#pragma unroll
    for (int jj = 0; jj < TT / 2; ++jj) {
      const int jp = jp0 + jj;
      if (TR ? jp > kt : jp < kt) continue;  // warp-uniform
      const uint32_t at = TR ? delta_tri_block(kt, jp) + m.tr_tri : delta_tri_block(jp, kt) + m.nt_tri;
      if (TR) {
        ldsm4t(bh[jj], bhi + at);
        if (BLO) ldsm4t(bl[jj], blo + at);
      } else {
        ldsm4(bh[jj], bhi + at);
        if (BLO) ldsm4(bl[jj], blo + at);
      }
    }
#pragma unroll
    for (int piece = 0; piece < 3; ++piece) {
      if ((piece == 1 && !XLO) || (piece == 2 && !BLO)) continue;
#pragma unroll
      for (int jj = 0; jj < TT / 2; ++jj) {
        const int jp = jp0 + jj;
        if (TR ? jp > kt : jp < kt) continue;
        const uint32_t(&a)[4] = piece == 1 ? lo : hi;
        const uint32_t(&b)[4] = piece == 2 ? bl[jj] : bh[jj];
        mma_f16(acc[2 * jj], a, b[0], b[1]);
        mma_f16(acc[2 * jj + 1], a, b[2], b[3]);
      }
    }
  }
}

// s[16 x NS] += x[16 x 64 tokens] tile[64 tokens x N], columns from 8 u0 on, x
// as two pieces.
template <int N, int NS>
__device__ __forceinline__ void state_product(float (&s)[NS / 8][4], const float (&x)[8][4],
                                              float s0, float s1, uint32_t tile, int u0,
                                              const LaneMap& m) {
#pragma unroll
  for (int kt = 0; kt < 4; ++kt) {
    uint32_t hi[4], lo[4];
    split_a(x[2 * kt], x[2 * kt + 1], s0, s1, hi, lo);
#pragma unroll
    for (int jn = 0; jn < NS / 16; jn += 2) {
      uint32_t b[2][4];
      ldsm4t(b[0], tile + kq_at(16 * kt + m.tr_row, u0 + 2 * jn + m.tr_unit));
      ldsm4t(b[1], tile + kq_at(16 * kt + m.tr_row, u0 + 2 * jn + 2 + m.tr_unit));
      mma_tiles(s, hi, b, 2 * jn);
      mma_tiles(s, lo, b, 2 * jn);
    }
  }
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
template <int T>
__device__ __forceinline__ void zero(float (&x)[T][4]) {
#pragma unroll
  for (int j = 0; j < T; ++j) x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.f;
}
// The warp's tiles out of all eight: the half `hf` of them when TT is 4.
template <int TT>
__device__ __forceinline__ void own(float (&d)[TT][4], const float (&x)[8][4], int hf) {
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) d[j][q] = TT == 8 ? x[j][q] : (hf ? x[4 + (j & 3)][q] : x[j & 3][q]);
}

// The 16 columns of a column tile [token][p] as fp32 accumulator-shaped values
// [p][token], tokens t0 .. t0 + 8 T - 1.
template <int T>
__device__ __forceinline__ void load_rows(float (&x)[T][4], uint32_t tile, int t0, const LaneMap& m) {
#pragma unroll
  for (int jp = 0; jp < T / 2; ++jp) {
    uint32_t r[4];
    ldsm4t(r, tile + (t0 + 16 * jp) * 32 + m.nt_col);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = 2 * jp + (q >> 1), e = (q & 1) * 2;
      x[j][e] = bf16_lo(r[q]);
      x[j][e + 1] = bf16_hi(r[q]);
    }
  }
}

// Accumulator-shaped values [p][token] of tokens t0 .. -> bf16 rows of a column
// tile, then to global memory (32 bytes a token).
template <int T>
__device__ __forceinline__ void store_rows(const float (&x)[T][4], uint32_t tile, int t0,
                                           uint16_t* out, size_t out_stride, int valid, int lane,
                                           const LaneMap& m) {
#pragma unroll
  for (int jp = 0; jp < T / 2; ++jp) {
    uint32_t r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = 2 * jp + (q >> 1), e = (q & 1) * 2;
      r[q] = pack_bf16x2(x[j][e], x[j][e + 1]);
    }
    stsm4t(tile + (t0 + 16 * jp) * 32 + m.nt_col, r);
  }
  __syncwarp();
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

// The carried rows: s = true value / inv, inv a power of two per row.
template <int N, int NS>
__device__ __forceinline__ void load_state(float (&s)[NS / 8][4], const float* src, float& inv0,
                                           float& inv1, int lane) {
  if (!src) {
    zero(s);
    inv0 = inv1 = 1.f;
    return;
  }
  const float* r0 = src + (lane >> 2) * N + 2 * (lane & 3);
#pragma unroll
  for (int j = 0; j < NS / 8; ++j) {
    const float2 a = *reinterpret_cast<const float2*>(r0 + 8 * j);
    const float2 b = *reinterpret_cast<const float2*>(r0 + 8 * N + 8 * j);
    s[j][0] = a.x; s[j][1] = a.y; s[j][2] = b.x; s[j][3] = b.y;
  }
  float m0, m1;
  row_max(s, m0, m1);
  const RowScale a = row_scale<6>(exponent_of(m0)), b = row_scale<6>(exponent_of(m1));
  scale_rows(s, a.s, b.s);
  inv0 = a.inv;
  inv1 = b.inv;
}
template <int N, int NS>
__device__ __forceinline__ void store_state(const float (&s)[NS / 8][4], float* dst, float inv0,
                                            float inv1, int lane) {
  float* r0 = dst + (lane >> 2) * N + 2 * (lane & 3);
#pragma unroll
  for (int j = 0; j < NS / 8; ++j) {
    *reinterpret_cast<float2*>(r0 + 8 * j) = mul2(make_float2(s[j][0], s[j][1]), make_float2(inv0, inv0));
    *reinterpret_cast<float2*>(r0 + 8 * N + 8 * j) =
        mul2(make_float2(s[j][2], s[j][3]), make_float2(inv1, inv1));
  }
}
// The rows as bf16 (for products whose results are bf16).
template <int N, int NS>
__device__ __forceinline__ void store_state16(const float (&s)[NS / 8][4], uint16_t* dst, float inv0,
                                              float inv1, int lane) {
  uint16_t* r0 = dst + (lane >> 2) * N + 2 * (lane & 3);
#pragma unroll
  for (int j = 0; j < NS / 8; ++j) {
    *reinterpret_cast<uint32_t*>(r0 + 8 * j) = pack_bf16x2(s[j][0] * inv0, s[j][1] * inv0);
    *reinterpret_cast<uint32_t*>(r0 + 8 * N + 8 * j) = pack_bf16x2(s[j][2] * inv1, s[j][3] * inv1);
  }
}
// <s, src> over the warp's part of the state, src fp32 (all lanes).
template <int N, int NS>
__device__ __forceinline__ float state_dot(const float (&s)[NS / 8][4], const float* src, float inv0,
                                           float inv1, int lane) {
  const float* r0 = src + (lane >> 2) * N + 2 * (lane & 3);
  float2 d0 = make_float2(0.f, 0.f), d1 = d0;
#pragma unroll
  for (int j = 0; j < NS / 8; ++j) {
    d0 = fma2(make_float2(s[j][0], s[j][1]), *reinterpret_cast<const float2*>(r0 + 8 * j), d0);
    d1 = fma2(make_float2(s[j][2], s[j][3]), *reinterpret_cast<const float2*>(r0 + 8 * N + 8 * j), d1);
  }
  float d = (d0.x + d0.y) * inv0 + (d1.x + d1.y) * inv1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  return d;
}
// Decays the state and brings it under the scale of max(state, terms of
// largest exponents e0, e1): the sum of 64 terms of k rows below 2 then stays
// below 2^15.
struct NewScale {
  float s0, s1;
};
template <int T>
__device__ __forceinline__ NewScale rescale(float (&s)[T][4], float& inv0, float& inv1,
                                            uint32_t e0, uint32_t e1, float end) {
  float m0, m1;
  row_max(s, m0, m1);
  const RowScale a = row_scale<6>(max(e0, exponent_of(m0 * inv0)));
  const RowScale b = row_scale<6>(max(e1, exponent_of(m1 * inv1)));
  // 2^100: a row that is all zero has no exponent of its own
  scale_rows(s, end * fminf(inv0 * a.s, 1.2676506e30f), end * fminf(inv1 * b.s, 1.2676506e30f));
  inv0 = a.inv;
  inv1 = b.inv;
  NewScale n;
  n.s0 = a.s;
  n.s1 = b.s;
  return n;
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
  const uint32_t heads = (uint32_t)(t.nheads * l.head);
  mbar_arrive_expect_tx(&full[st], (uint32_t)l.kq + heads);
  bulk_load(smem_u32(base), p.ws_kq + (bc * d.nkheads + t.kh) * (size_t)l.kq, l.kq, &full[st]);
  bulk_load(smem_u32(base + l.kq), p.ws_head + (bc * d.nheads + t.h0) * (size_t)p.head_bytes, heads,
            &full[st]);
}

// The warp is done with a stage: true in the lane that is to refill it, lane 0
// of the last of the CTA's warps.
__device__ __forceinline__ bool last_of(unsigned* count, unsigned warps) {
  __syncwarp();
  if ((threadIdx.x & 31) != 0) return false;
  __threadfence_block();
  const bool last = atomicAdd(count, 1u) == warps - 1;
  if (last) {
    *count = 0;
    __threadfence_block();
    fence_async_smem();  // reads of the old tiles before the copies over them
  }
  return last;
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
template <int SP>
__device__ __forceinline__ bool wait_stage(uint64_t* bar, uint32_t parity, uint64_t limit,
                                           int pair_id) {
  cp_async_wait_group<0>();  // the warp's own column tiles (visible after the barriers below)
  bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit));
  __syncwarp();
  if (SP == 2) ok = pair_and(pair_id, ok);
  return ok;
}
// A wait ran out at step s: note it, and leave only when the copies already
// issued have landed (or that wait, too, has run out).
__device__ __forceinline__ void give_up(const DeltaChunkParams& p, uint64_t* full, int s) {
  if ((threadIdx.x & 31) == 0) atomicExch(&g_delta_timeout, 1);
  for (int i = s; i < s + p.stages && i < p.nchunks; ++i)
    mbar_wait_bounded(&full[i % p.stages], (uint32_t)((i / p.stages) & 1), p.wait_limit_ns);
}

// x += the partner warp's x, through shared memory (after scaling to true values)
template <int T>
__device__ __forceinline__ void put_tiles(const float (&x)[T][4], float* buf, int lane) {
#pragma unroll
  for (int j = 0; j < T; ++j)
    *reinterpret_cast<float4*>(buf + (j * 32 + lane) * 4) =
        make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
}
template <int T>
__device__ __forceinline__ void add_from(float (&x)[T][4], const float* buf, int lane) {
#pragma unroll
  for (int j = 0; j < T; ++j) {
    const float4 v = *reinterpret_cast<const float4*>(buf + (j * 32 + lane) * 4);
    x[j][0] += v.x; x[j][1] += v.y; x[j][2] += v.z; x[j][3] += v.w;
  }
}

template <int N, int SP, bool BWD>
__global__ void __launch_bounds__(256, 1) delta_fwd_kernel(const __grid_constant__ DeltaChunkParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ unsigned count[kMaxStages];
  constexpr int NS = N / SP, TT = 8 / SP;  // the warp's columns of the state, token tiles of y
  constexpr int kTris = BWD ? 4 : 3;
  const DeltaParams& d = p.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = warp / SP, hf = SP == 2 ? warp & 1 : 0;
  const int pb = d.headdim / 16;
  const Cta t = cta_of(p);
  const Layout l = layout(N, p.blocks, pb, BWD ? 2 : 1, BWD ? kDeltaHeadBwd : kDeltaHeadFwd);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      count[i] = 0;
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages && s < p.nchunks; ++s)
      if (!(p.test_stall && s == 0 && blockIdx.x == 0))  // its data never arrives
        issue(p, t, l, smem, full, s, s);
  }
  if (blk >= t.active) return;
  const unsigned warps = (unsigned)t.active * SP;

  const LaneMap m = lane_map(lane);
  const int rb = t.rb0 + blk, hx = rb / pb;                  // row block in the group, its head
  const int h = t.kh * (d.nheads / d.nkheads) + hx, pw = (rb - hx * pb) * 16;
  const size_t state_at = (((size_t)t.b * d.nheads + h) * d.headdim + pw) * N + hf * NS;
  const size_t vs = (size_t)d.nheads * d.headdim;
  const int u0 = hf * (NS / 8), tk = hf * 32;                // first column unit, first token of y
  constexpr int kTiles = BWD ? 2 : 1;  // v, dy
  unsigned char* cols = smem + (size_t)p.stages * l.stage;
  const uint32_t col0 = smem_u32(cols) + blk * 2 * kTiles * kCol;
  float* xbuf = reinterpret_cast<float*>(cols + p.blocks * 2 * kTiles * kCol) + warp * 12 * 128;
  const float* xoth = xbuf + (hf ? -12 * 128 : 12 * 128);
  float S[NS / 8][4], inv0, inv1;
  const size_t col_at = (size_t)t.b * d.seqlen * vs + (size_t)h * d.headdim + pw;
  auto fetch = [&](int c) {  // the pair's warps fetch half the tokens each
    const int valid = (int)min((int64_t)kC, d.seqlen - (int64_t)c * kC);
    const size_t at = col_at + (size_t)c * kC * vs;
    const uint32_t to = col0 + (c & 1) * kTiles * kCol;
    fetch_rows<TT>(to, static_cast<const uint16_t*>(d.v) + at, vs, tk, valid, lane);
    if (BWD) fetch_rows<TT>(to + kCol, p.dy + at, vs, tk, valid, lane);
    cp_async_commit_group();
  };
  fetch(0);
  load_state<N, NS>(S, d.h0 ? d.h0 + state_at : nullptr, inv0, inv1, lane);

  for (int c = 0; c < p.nchunks; ++c) {
    const int st = c % p.stages;
    const size_t st_at = (((size_t)t.b * p.nchunks + c) * d.nheads + h) * ((size_t)d.headdim * N) +
                         (size_t)pw * N + hf * NS;
    if (BWD) store_state16<N, NS>(S, p.ws_state16 + st_at, inv0, inv1, lane);
    if (!wait_stage<SP>(&full[st], (uint32_t)((c / p.stages) & 1), p.wait_limit_ns, 1 + blk)) {
      give_up(p, full, c);
      return;
    }
    const int64_t t0 = (int64_t)c * kC;
    const int valid = (int)min((int64_t)kC, d.seqlen - t0);
    if (c + 1 < p.nchunks) fetch(c + 1);  // the other buffer: this chunk's predecessor is done with it
    unsigned char* base = smem + (size_t)st * l.stage;
    unsigned char* head = base + l.kq + (h - t.h0) * l.head;
    const uint32_t ks = smem_u32(base), qs = ks + l.kq / 2;
    const uint32_t th = smem_u32(head), tl = th + kDeltaTri, ph = tl + kDeltaTri, pl = ph + kDeltaTri;
    const float* sc = reinterpret_cast<const float*>(head + kTris * kDeltaTri);
    const uint32_t vrow = col0 + (c & 1) * kTiles * kCol;

    // ---- S K^T and S Q^T
    float x[8][4], o[8][4], y[TT][4];
    zero(x);
    zero(o);
#pragma unroll
    for (int kt = 0; kt < NS / 16; ++kt) {
      uint32_t hi[4], lo[4];
      pieces_a(S[2 * kt], S[2 * kt + 1], hi, lo);
      uint32_t bk[4][4], bq[4][4];
#pragma unroll
      for (int jp = 0; jp < 4; ++jp) {
        const uint32_t at = kq_at(16 * jp + m.nt_row, u0 + 2 * kt + m.nt_unit);
        ldsm4(bk[jp], ks + at);
        ldsm4(bq[jp], qs + at);
      }
      mma_tiles(x, hi, bk);
      mma_tiles(o, hi, bq);
      mma_tiles(x, lo, bk);
      if (BWD) mma_tiles(o, lo, bq);
    }
    scale_rows(x, inv0, inv1);
    own<TT>(y, o, hf);
    scale_rows(y, inv0, inv1);
    if (SP == 2) {
      float other[TT][4];
      own<TT>(other, o, hf ^ 1);
      scale_rows(other, inv0, inv1);
      put_tiles(x, xbuf, lane);
      put_tiles(other, xbuf + 8 * 128, lane);
      pair_sync(1 + blk);
      add_from(x, xoth, lane);
      add_from(y, xoth + 8 * 128, lane);
    }
    scale_cols(y, sc + kScSq * kC + tk, lane);

    // ---- R = V - ..., r = T R, u = beta r
    scale_cols(x, sc + kScSk * kC, lane);
    float u[8][4];
    load_rows(u, vrow, 0, m);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[j][q] = u[j][q] - x[j][q];
        u[j][q] = 0.f;
      }
    float m0, m1;
    row_max(x, m0, m1);
    RowScale r0 = row_scale(exponent_of(m0)), r1 = row_scale(exponent_of(m1));
    tri_product<false, true, true>(u, x, r0.s, r1.s, th, tl, 0, m);
    scale_rows(u, r0.inv, r1.inv);
    if (BWD) {
      scale_cols(u, sc + kScT * kC, lane);
      if (SP == 2) pair_sync(1 + blk);  // the partner has read its rows of v
      float rr[TT][4];
      own<TT>(rr, u, hf);
      store_rows(rr, vrow, tk, p.ws_r + col_at + t0 * vs, vs, valid, lane, m);
      scale_cols(u, sc + kScBeta * kC, lane);
    } else {
      scale_cols(u, sc + kScU * kC, lane);
    }

    // ---- Y += P u
    float w[TT][4];
    zero(w);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) x[j][q] = u[j][q];
    scale_cols(x, sc + kScK * kC, lane);
    row_max(x, m0, m1);
    r0 = row_scale(exponent_of(m0));
    r1 = row_scale(exponent_of(m1));
    tri_product<false, BWD, BWD>(w, x, r0.s, r1.s, ph, pl, hf * 2, m);
    scale_rows(w, r0.inv, r1.inv);
    scale_cols(w, sc + kScP * kC + tk, lane);
    add_tiles(y, w);
    if (BWD) {
      load_rows(w, vrow + kCol, tk, m);
      row_dots(w, y, p.ws_doto + ((((size_t)t.b * p.nchunks + c) * d.nheads + h) * pb + pw / 16) * kC + tk,
               lane);
    } else if (d.y) {
      if (SP == 2) pair_sync(1 + blk);  // the partner has read its rows of v
      store_rows(y, vrow, tk, static_cast<uint16_t*>(d.y) + col_at + t0 * vs, vs, valid, lane, m);
    }

    // ---- S <- e^G_end S + u^T (e^(G_end - G) K)
    scale_cols(u, sc + kScKend * kC, lane);
    row_max(u, m0, m1);
    const NewScale n = rescale(S, inv0, inv1, exponent_of(m0), exponent_of(m1), sc[kScEnd * kC]);
    state_product<N, NS>(S, u, n.s0, n.s1, ks, u0, m);
    if (BWD) store_state<N, NS>(S, p.ws_state + st_at, inv0, inv1, lane);
    if (last_of(&count[st], warps) && c + p.stages < p.nchunks)
      issue(p, t, l, smem, full, c + p.stages, st);
  }
  if (!BWD && d.h_last)
    store_state<N, NS>(S, d.h_last + state_at, inv0, inv1, lane);
}

template <int N, int SP>
__global__ void __launch_bounds__(256, 1) delta_rev_kernel(const __grid_constant__ DeltaChunkParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ unsigned count[kMaxStages];
  constexpr int NS = N / SP, TT = 8 / SP;
  const DeltaParams& d = p.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = warp / SP, hf = SP == 2 ? warp & 1 : 0;
  const int pb = d.headdim / 16;
  const Cta t = cta_of(p);
  const Layout l = layout(N, p.blocks, pb, 3, kDeltaHeadBwd);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      count[i] = 0;
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages && s < p.nchunks; ++s)
      issue(p, t, l, smem, full, p.nchunks - 1 - s, s);
  }
  if (blk >= t.active) return;
  const unsigned warps = (unsigned)t.active * SP;

  const LaneMap m = lane_map(lane);
  const int rb = t.rb0 + blk, hx = rb / pb;
  const int h = t.kh * (d.nheads / d.nkheads) + hx, pw = (rb - hx * pb) * 16;
  const size_t state_at = (((size_t)t.b * d.nheads + h) * d.headdim + pw) * N + hf * NS;
  const size_t vs = (size_t)d.nheads * d.headdim;
  const int u0 = hf * (NS / 8), tk = hf * 32;
  constexpr int kTiles = 3;  // v, dy, r
  unsigned char* cols = smem + (size_t)p.stages * l.stage;
  const uint32_t col0 = smem_u32(cols) + blk * 2 * kTiles * kCol;
  float* xbuf = reinterpret_cast<float*>(cols + p.blocks * 2 * kTiles * kCol) + warp * 8 * 128;
  const float* xoth = xbuf + (hf ? -8 * 128 : 8 * 128);
  float S[NS / 8][4], inv0, inv1;  // the adjoint of the state
  const size_t col_at = (size_t)t.b * d.seqlen * vs + (size_t)h * d.headdim + pw;
  auto fetch = [&](int c) {
    const int valid = (int)min((int64_t)kC, d.seqlen - (int64_t)c * kC);
    const size_t at = col_at + (size_t)c * kC * vs;
    const uint32_t to = col0 + (c & 1) * kTiles * kCol;
    fetch_rows<TT>(to, static_cast<const uint16_t*>(d.v) + at, vs, tk, valid, lane);
    fetch_rows<TT>(to + kCol, p.dy + at, vs, tk, valid, lane);
    fetch_rows<TT>(to + 2 * kCol, p.ws_r + at, vs, tk, valid, lane);
    cp_async_commit_group();
  };
  fetch(p.nchunks - 1);
  load_state<N, NS>(S, p.dh_last ? p.dh_last + state_at : nullptr, inv0, inv1, lane);

  for (int s = 0; s < p.nchunks; ++s) {
    const int st = s % p.stages, c = p.nchunks - 1 - s;
    const size_t bch = ((size_t)t.b * p.nchunks + c) * d.nheads + h;
    const size_t part = (size_t)pw * N + hf * NS, st_at = bch * ((size_t)d.headdim * N) + part;
    {
      const float dot = state_dot<N, NS>(S, p.ws_state + st_at, inv0, inv1, lane);
      if (lane == 0) {
        p.ws_end[(bch * pb + pw / 16) * 2 + hf] = dot;
        if (SP == 1) p.ws_end[(bch * pb + pw / 16) * 2 + 1] = 0.f;
      }
    }
    store_state16<N, NS>(S, p.ws_dstate16 + st_at, inv0, inv1, lane);
    if (c > 0) {  // the next state on its way from DRAM: 16 rows, 128 bytes per prefetch
      const float* nx = p.ws_state + (bch - d.nheads) * ((size_t)d.headdim * N) + part;
#pragma unroll
      for (int i = 0; i < 16 * NS / 32; i += 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(nx + (size_t)((i + lane) / (NS / 32)) * N +
                                                      (i + lane) % (NS / 32) * 32));
    }
    if (!wait_stage<SP>(&full[st], (uint32_t)((s / p.stages) & 1), p.wait_limit_ns, 1 + blk)) {
      give_up(p, full, s);
      return;
    }
    const int64_t t0 = (int64_t)c * kC;
    const int valid = (int)min((int64_t)kC, d.seqlen - t0);
    if (c > 0) fetch(c - 1);  // the other buffer: this chunk's predecessor is done with it
    unsigned char* base = smem + (size_t)st * l.stage;
    unsigned char* head = base + l.kq + (h - t.h0) * l.head;
    const uint32_t ks = smem_u32(base), qs = ks + l.kq / 2;
    const uint32_t th = smem_u32(head), tl = th + kDeltaTri, ph = tl + kDeltaTri, pl = ph + kDeltaTri;
    const float* sc = reinterpret_cast<const float*>(head + 4 * kDeltaTri);
    const uint32_t vrow = col0 + (c & 1) * kTiles * kCol;
    const size_t dot_at = (bch * pb + pw / 16) * kC + tk;

    // ---- dU = P^T dY + e^(G_end - G) K dS^T
    float x[8][4], u[8][4], w[8][4];
    zero(x);
#pragma unroll
    for (int kt = 0; kt < NS / 16; ++kt) {
      uint32_t hi[4], lo[4];
      pieces_a(S[2 * kt], S[2 * kt + 1], hi, lo);
      uint32_t bk[4][4];
#pragma unroll
      for (int jp = 0; jp < 4; ++jp)
        ldsm4(bk[jp], ks + kq_at(16 * jp + m.nt_row, u0 + 2 * kt + m.nt_unit));
      mma_tiles(x, hi, bk);
      mma_tiles(x, lo, bk);
    }
    scale_rows(x, inv0, inv1);
    if (SP == 2) {
      put_tiles(x, xbuf, lane);
      pair_sync(1 + blk);
    }
    load_rows(w, vrow + kCol, 0, m);  // dY
    scale_cols(w, sc + kScP * kC, lane);
    float m0, m1;
    row_max(w, m0, m1);
    RowScale r0 = row_scale(exponent_of(m0)), r1 = row_scale(exponent_of(m1));
    zero(u);
    tri_product<true, true, true>(u, w, r0.s, r1.s, ph, pl, 0, m);
    scale_rows(u, r0.inv, r1.inv);
    scale_cols(u, sc + kScK * kC, lane);
    if (SP == 2) add_from(x, xoth, lane);
    scale_cols(x, sc + kScKend * kC, lane);
    add_tiles(u, x);
    {
      float a[TT][4], r[TT][4];
      own<TT>(a, u, hf);
      load_rows(r, vrow + 2 * kCol, tk, m);
      row_dots(a, r, p.ws_dotu + dot_at, lane);
    }

    // ---- dR = T^T (beta dU) = dV
    scale_cols(u, sc + kScU * kC, lane);
    row_max(u, m0, m1);
    r0 = row_scale(exponent_of(m0));
    r1 = row_scale(exponent_of(m1));
    zero(x);
    tri_product<true, true, true>(x, u, r0.s, r1.s, th, tl, 0, m);
    scale_rows(x, r0.inv, r1.inv);
    {
      float a[TT][4], r[TT][4];
      own<TT>(a, x, hf);
      load_rows(r, vrow, tk, m);  // v: only these tokens' rows
      row_dots(a, r, p.ws_dotv + dot_at, lane);
      __syncwarp();
      store_rows(a, vrow, tk, p.dv + col_at + t0 * vs, vs, valid, lane, m);
    }

    // ---- dS <- e^G_end dS + dY^T (e^G Q) - dR^T (e^G K)
    load_rows(w, vrow + kCol, 0, m);
    scale_cols(w, sc + kScSq * kC, lane);
    scale_cols(x, sc + kScSk * kC, lane);
    scale_rows(x, -1.f, -1.f);
    float n0, n1;
    row_max(w, m0, m1);
    row_max(x, n0, n1);
    const NewScale n = rescale(S, inv0, inv1, max(exponent_of(m0), exponent_of(n0)),
                               max(exponent_of(m1), exponent_of(n1)), sc[kScEnd * kC]);
    state_product<N, NS>(S, w, n.s0, n.s1, qs, u0, m);
    state_product<N, NS>(S, x, n.s0, n.s1, ks, u0, m);
    if (last_of(&count[st], warps) && s + p.stages < p.nchunks)
      issue(p, t, l, smem, full, c - p.stages, st);
  }
  if (p.dh0) store_state<N, NS>(S, p.dh0 + state_at, inv0, inv1, lane);
}

// The largest number of 16-row blocks per CTA that leaves two stages, halved
// while the grid then still is no larger than the SMs (each CTA fills one);
// pairs of warps per block when they fit four or fewer blocks.
template <typename K1, typename K2>
cudaError_t run(K1* one, K2* two, DeltaChunkParams& p, int tiles, int head_bytes, int tiles_x,
                cudaStream_t stream) {
  const int per_head = p.d.headdim / 16, group = p.d.nheads / p.d.nkheads * per_head;
  const int64_t groups = (int64_t)p.d.batch * p.d.nkheads;
  const int most = 225 * 1024;
  // column tiles and the pairs' exchange buffers, beside the stages
  auto extra = [&](int blocks, int sp) {
    return blocks * 2 * tiles * kCol + (sp == 2 ? blocks * 2 * tiles_x * 512 : 0);
  };
  auto stages_of = [&](int blocks, int sp) {
    return std::min(kMaxStages, (most - extra(blocks, sp)) /
                                    layout(p.d.dstate, blocks, per_head, tiles, head_bytes).stage);
  };
  auto ctas = [&](int blocks) { return groups * ((group + blocks - 1) / blocks); };
  int blocks = kMaxBlocks;
  while (blocks > 1 && (blocks / 2 >= group || stages_of(blocks, 1) < 2 || ctas(blocks / 2) <= 148))
    blocks /= 2;
  const char* force = getenv("SSM_DELTA_BLOCKS");
  if (force && *force) blocks = atoi(force);
  int sp = blocks <= 4 && stages_of(blocks, 2) >= 2 ? 2 : 1;
  const char* fsp = getenv("SSM_DELTA_SP");
  if (fsp && *fsp) sp = atoi(fsp);
  p.blocks = blocks;
  p.stages = stages_of(blocks, sp);
  if (p.stages < 1) return cudaErrorInvalidValue;
  const int bytes = layout(p.d.dstate, blocks, per_head, tiles, head_bytes).stage * p.stages +
                    extra(blocks, sp);
  const unsigned grid = (unsigned)ctas(blocks);
  auto go = [&](auto* kern) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kern<<<grid, blocks * sp * 32, bytes, stream>>>(p);
    return cudaGetLastError();
  };
  return sp == 2 ? go(two) : go(one);
}

template <int N, bool BWD>
cudaError_t fwd(DeltaChunkParams& p, cudaStream_t stream) {
  return run(delta_fwd_kernel<N, 1, BWD>, delta_fwd_kernel<N, 2, BWD>, p, BWD ? 2 : 1,
             BWD ? kDeltaHeadBwd : kDeltaHeadFwd, 12, stream);
}
template <int N>
cudaError_t rev(DeltaChunkParams& p, cudaStream_t stream) {
  return run(delta_rev_kernel<N, 1>, delta_rev_kernel<N, 2>, p, 3, kDeltaHeadBwd, 8, stream);
}

}  // namespace

bool delta_chunk_supported(int dstate, int headdim) {
  return (dstate == 64 || dstate == 128) && headdim % 16 == 0 && headdim >= 16;
}

cudaError_t launch_delta_chunk_fwd(const DeltaChunkParams& pin, bool bwd, cudaStream_t stream) {
  DeltaChunkParams p = pin;
  if (bwd) return p.d.dstate == 64 ? fwd<64, true>(p, stream) : fwd<128, true>(p, stream);
  return p.d.dstate == 64 ? fwd<64, false>(p, stream) : fwd<128, false>(p, stream);
}

cudaError_t launch_delta_chunk_rev(const DeltaChunkParams& pin, cudaStream_t stream) {
  DeltaChunkParams p = pin;
  return p.d.dstate == 64 ? rev<64>(p, stream) : rev<128>(p, stream);
}

cudaError_t delta_chunk_status(cudaStream_t stream, int* timed_out) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  const int zero = 0;
  e = cudaMemcpyFromSymbol(timed_out, g_delta_timeout, sizeof(int));
  if (e != cudaSuccess || !*timed_out) return e;
  return cudaMemcpyToSymbol(g_delta_timeout, &zero, sizeof(int));
}

}  // namespace ssm
