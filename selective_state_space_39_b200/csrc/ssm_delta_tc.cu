// ssm_delta_tc.cu -- the gated delta rule chunk by chunk on the fifth-generation
// tensor cores (tcgen05; bf16 io, sm_100a): the forward pass over the chunks,
// and the same walk for the gradients (BWD: it keeps the states, r and dy.y).
//
// Per head, with the operands of ssm_delta_prep.cu and the state S (headdim x
// dstate) entering a chunk:
//   R = V - (e^G K) S^T,  r = T R,  u = beta r
//   Y = (e^G Q) S^T + P u
//   S <- e^G_end S + u^T (e^(G_end - G) K)
// All products have the state's rows (output columns p) as their M axis, so
// that none of them ever meets another row: a CTA takes up to 128 rows (eight
// 16-row blocks of heads that share a key head), a warp 16 of them. S^T, r^T
// and u^T are the A operands, written to tensor memory as two fp16 pieces per
// fp32 value under a power-of-two scale per row; k, q (swizzled 64-column
// blocks) and T, P (core matrices on and below the diagonal, so that a step
// over 16 tokens multiplies only the tokens after it) are the B operands in
// shared memory. A warp reads its accumulators as 16 x 256-bit fragments, the
// layout of its v and y rows too, so scales, maxima and sums over a row are
// shuffles of a quad. S itself stays in fp32 registers: the tensor cores add
// up only the chunk's contribution.
//
// A chunk is a chain S -> K S -> R -> T R -> u -> K^T u -> S of three products,
// each issued by whichever warp is the last to have written its rows (no warp
// waits to issue), and answered by one mbarrier; Q S, P u and the writing of Y
// run beside the chain. With two heads in a CTA T and P products are taken for
// both heads on all rows, and a row reads its own head's columns.
//
// Tensor memory (512 columns): 0 S pieces, then u's pieces for P; 128 K S, R's
// pieces, u's pieces for K^T; 192 Q S; 256 T R per head, then K^T u; 384 P u
// per head.
#include <stdlib.h>

#include "ssm_delta_rows.cuh"
#include "ssm_tc.cuh"

namespace ssm {

namespace {

constexpr int kTmemCols = 512;
constexpr uint32_t kTmS = 0, kTmX = 128, kTmO = 192, kTmU = 256, kTmY = 384;
constexpr int kTcHeads = 2;  // heads per CTA, at most

// 64 accumulator columns of the warp's 16 lanes.
__device__ __forceinline__ void tm_load(uint32_t addr, float (&x)[8][4]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
  tc::wait_ld();
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) x[j][q] = __uint_as_float(r[4 * j + q]);
}
// 64 fp16 columns (32 columns of tensor memory) of the warp's 16 lanes.
__device__ __forceinline__ void tm_store(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Eight tiles under row scales s0, s1 as pieces at hi and (LO) lo.
template <bool LO>
__device__ __forceinline__ void tm_pieces(const float (*x)[4], float s0, float s1, uint32_t hi_at,
                                          uint32_t lo_at) {
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    split2(x[j][0], x[j][1], s0, hi[2 * j], lo[2 * j]);
    split2(x[j][2], x[j][3], s1, hi[2 * j + 1], lo[2 * j + 1]);
  }
  tm_store(hi_at, hi);
  if (LO) tm_store(lo_at, lo);
}

// D (128 rows x n) += A (16 columns of k in tensor memory) B.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint64_t b, int n, int b_mn, bool acc) {
  const uint32_t idesc = (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// D = X (pieces at hi, lo: dstate columns) tile^T, the tile's rows being D's columns.
template <int N, bool LO>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t a, uint32_t tile) {
#pragma unroll
  for (int piece = 0; piece < (LO ? 2 : 1); ++piece)
#pragma unroll
    for (int ks = 0; ks < N / 16; ++ks)
      mma(d, a + piece * (N / 2) + 8 * ks,
          tc::sdesc(tile + (ks / 4) * (kC * 128) + (ks % 4) * 32, 16, 1024), kC, 0, piece + ks > 0);
}
// D (rows x dstate) = X (64 tokens, pieces at a and a + 32) tile.
template <int N>
__device__ __forceinline__ void mma_tokens(uint32_t d, uint32_t a, uint32_t tile) {
#pragma unroll
  for (int piece = 0; piece < 2; ++piece)
#pragma unroll
    for (int ks = 0; ks < kC / 16; ++ks)
      mma(d, a + piece * 32 + 8 * ks, tc::sdesc(tile + ks * 2048, kC * 128, 1024), N, 1,
          piece + ks > 0);
}
// D (rows x 64 tokens) = X (64 tokens, pieces at a, a + 32) tri^T, the lower
// triangular tile in one or two pieces; a step over 16 tokens reaches the
// columns from those tokens on.
template <bool XLO, bool BLO>
__device__ __forceinline__ void mma_tri(uint32_t d, uint32_t a, uint32_t hi, uint32_t lo) {
#pragma unroll
  for (int piece = 0; piece < 3; ++piece) {
    if ((piece == 1 && !XLO) || (piece == 2 && !BLO)) continue;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      const uint32_t at = (piece == 2 ? lo : hi) + delta_tri_block(kt, kt);
      // core matrices: 128 bytes to the next eight columns, 256 to the next eight rows
      const uint64_t b = (uint64_t)((at >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 16) |
                         ((uint64_t)(256 >> 4) << 32) | ((uint64_t)1 << 46);
      mma(d + 16 * kt, a + (piece == 1 ? 32 : 0) + 8 * kt, b, kC - 16 * kt, 0, piece + kt > 0);
    }
  }
}

// The warp's rows are written to tensor memory: true in lane 0 of the last warp.
__device__ __forceinline__ bool wrote_last(unsigned* count, unsigned warps) {
  tc::wait_st();
  tc::fence_before_sync();
  __syncwarp();
  if ((threadIdx.x & 31) != 0) return false;
  __threadfence_block();
  const bool last = atomicAdd(count, 1u) == warps - 1;
  if (last) {
    *count = 0;
    __threadfence_block();
    tc::fence_after_sync();
  }
  return last;
}
__device__ __forceinline__ bool wait_mma(uint64_t* bar, uint32_t parity, uint64_t limit) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit));
  tc::fence_after_sync();
  return ok;
}

// mbarriers: K S, Q S, T R, K^T u, P u, and the one that drains a failed CTA
enum { kBarK, kBarQ, kBarT, kBarU, kBarP, kBarDrain, kBars };
// warps that have written: S, R, u for K^T, u for P
enum { kCntS, kCntR, kCntU, kCntP, kCnts };

template <int N, bool BWD>
__global__ void __launch_bounds__(256, 1) delta_tc_kernel(const __grid_constant__ DeltaChunkParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], bars[kBars];
  __shared__ unsigned count[kMaxStages], written[kCnts];
  __shared__ uint32_t slot;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int kTris = BWD ? 4 : 3, kTiles = BWD ? 2 : 1;
  const DeltaParams& d = p.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pb = d.headdim / 16;
  const Cta t = cta_of(p);
  const Layout l = layout(N, p.blocks, pb, kTiles, BWD ? kDeltaHeadBwd : kDeltaHeadFwd);
  const unsigned warps = (unsigned)t.active;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      count[i] = 0;
    }
    for (int i = 0; i < kBars; ++i) mbar_init(&bars[i], i == kBarDrain ? warps : 1u);
    for (int i = 0; i < kCnts; ++i) written[i] = 0;
    fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(&slot, kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = slot;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages && s < p.nchunks; ++s)
      if (!(p.test_stall && s == 0 && blockIdx.x == 0))  // its data never arrives
        issue(p, t, l, smem, full, s, s);
  }

  if (warp < t.active) {
    const uint32_t row = tm + ((uint32_t)(32 * (warp & 3) + 16 * (warp >> 2)) << 16);
    const LaneMap m = lane_map(lane);
    const int rb = t.rb0 + warp, hx = rb / pb;  // row block in the group, its head
    const int h = t.kh * (d.nheads / d.nkheads) + hx, pw = (rb - hx * pb) * 16;
    const uint32_t hcol = (uint32_t)(h - t.h0) * kC;  // the head's columns of U and Y
    const size_t state_at = (((size_t)t.b * d.nheads + h) * d.headdim + pw) * N;
    const size_t vs = (size_t)d.nheads * d.headdim;
    unsigned char* cols = smem + (size_t)p.stages * l.stage;
    const uint32_t col0 = smem_u32(cols) + warp * 2 * kTiles * kCol;
    const size_t col_at0 = (size_t)t.b * d.seqlen * vs + (size_t)h * d.headdim + pw;
    auto fetch = [&](int c) {
      const int valid = (int)min((int64_t)kC, d.seqlen - (int64_t)c * kC);
      const size_t at = col_at0 + (size_t)c * kC * vs;
      const uint32_t to = col0 + (c & 1) * kTiles * kCol;
      fetch_rows<8>(to, static_cast<const uint16_t*>(d.v) + at, vs, 0, valid, lane);
      if (BWD) fetch_rows<8>(to + kCol, p.dy + at, vs, 0, valid, lane);
      cp_async_commit_group();
    };
    fetch(0);
    float S[N / 8][4], inv0, inv1;  // the state's rows (true values), the inverse of its pieces' scale
    load_state<N, N>(S, d.h0 ? d.h0 + state_at : nullptr, inv0, inv1, lane);
    scale_rows(S, inv0, inv1);
    bool ok = true;
    // the state's pieces, and by the last warp the products of chunk c that need them
    auto put_state = [&](int c) {
      float m0, m1;
      row_max(S, m0, m1);
      const RowScale a = row_scale(exponent_of(m0)), b = row_scale(exponent_of(m1));
      inv0 = a.inv;
      inv1 = b.inv;
#pragma unroll
      for (int i = 0; i < N / 64; ++i)
        tm_pieces<true>(&S[8 * i], a.s, b.s, row + kTmS + 32 * i, row + kTmS + N / 2 + 32 * i);
      if (wrote_last(&written[kCntS], warps)) {
        const int st = c % p.stages;
        // without its tiles the chunk's products are not issued, and every wait for them runs out
        if (mbar_wait_bounded(&full[st], (uint32_t)((c / p.stages) & 1), p.wait_limit_ns)) {
          const uint32_t ks = smem_u32(smem + (size_t)st * l.stage);
          mma_state<N, true>(tm + kTmX, tm + kTmS, ks);
          tc::commit(&bars[kBarK]);
          mma_state<N, BWD>(tm + kTmO, tm + kTmS, ks + l.kq / 2);
          tc::commit(&bars[kBarQ]);
        }
      }
      __syncwarp();
    };
    put_state(0);

    int c = 0;
    for (; c < p.nchunks; ++c) {
      const int st = c % p.stages;
      const uint32_t par = (uint32_t)(c & 1);
      const size_t bch = ((size_t)t.b * p.nchunks + c) * d.nheads + h;
      const size_t st_at = bch * ((size_t)d.headdim * N) + (size_t)pw * N;
      ok = wait_stage<1>(&full[st], (uint32_t)((c / p.stages) & 1), p.wait_limit_ns, 0);
      if (!ok) break;
      const int64_t t0 = (int64_t)c * kC;
      const int valid = (int)min((int64_t)kC, d.seqlen - t0);
      if (c + 1 < p.nchunks) fetch(c + 1);
      unsigned char* base = smem + (size_t)st * l.stage;
      unsigned char* head = base + l.kq + (h - t.h0) * l.head;
      const uint32_t ks = smem_u32(base), heads = ks + l.kq;
      const float* sc = reinterpret_cast<const float*>(head + kTris * kDeltaTri);
      const uint32_t vrow = col0 + (c & 1) * kTiles * kCol;

      // ---- R = V - (e^G K) S^T; T R
      float x[8][4], u[8][4], y[8][4];
      ok = wait_mma(&bars[kBarK], par, p.wait_limit_ns);
      if (!ok) break;
      tm_load(row + kTmX, x);
      scale_rows(x, -inv0, -inv1);
      scale_cols(x, sc + kScSk * kC, lane);
      load_rows(u, vrow, 0, m);
      add_tiles(x, u);
      float m0, m1;
      row_max(x, m0, m1);
      RowScale r0 = row_scale(exponent_of(m0)), r1 = row_scale(exponent_of(m1));
      tm_pieces<true>(x, r0.s, r1.s, row + kTmX, row + kTmX + 32);
      if (wrote_last(&written[kCntR], warps)) {
        for (int i = 0; i < t.nheads; ++i)
          mma_tri<true, true>(tm + kTmU + i * kC, tm + kTmX, heads + i * l.head,
                              heads + i * l.head + kDeltaTri);
        tc::commit(&bars[kBarT]);
      }
      __syncwarp();

      // ---- meanwhile the readout of the entering state
      ok = wait_mma(&bars[kBarQ], par, p.wait_limit_ns);
      if (!ok) break;
      tm_load(row + kTmO, y);
      scale_rows(y, inv0, inv1);
      scale_cols(y, sc + kScSq * kC, lane);
      if (BWD) store_state16<N, N>(S, p.ws_state16 + st_at, 1.f, 1.f, lane);

      // ---- u = beta T R; K^T (e^(G_end - G) u)
      ok = wait_mma(&bars[kBarT], par, p.wait_limit_ns);
      if (!ok) break;
      tm_load(row + kTmU + hcol, u);
      scale_rows(u, r0.inv, r1.inv);
      if (BWD) {
        scale_cols(u, sc + kScT * kC, lane);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) x[j][q] = u[j][q];
        scale_cols(x, sc + kScBeta * kC, lane);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) x[j][q] = u[j][q];
        scale_cols(x, sc + kScU * kC, lane);
      }
      if (BWD)
        store_rows(u, vrow, 0, p.ws_r + col_at0 + t0 * vs, vs, valid, lane, m);
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) u[j][q] = x[j][q];
      scale_cols(u, sc + kScKend * kC, lane);
      row_max(u, m0, m1);
      r0 = row_scale(exponent_of(m0));
      r1 = row_scale(exponent_of(m1));
      tm_pieces<true>(u, r0.s, r1.s, row + kTmX, row + kTmX + 32);
      if (wrote_last(&written[kCntU], warps)) {
        mma_tokens<N>(tm + kTmU, tm + kTmX, ks);
        tc::commit(&bars[kBarU]);
      }
      __syncwarp();

      // ---- P u
      scale_cols(x, sc + kScK * kC, lane);
      row_max(x, m0, m1);
      const RowScale w0 = row_scale(exponent_of(m0)), w1 = row_scale(exponent_of(m1));
      tm_pieces<BWD>(x, w0.s, w1.s, row + kTmS, row + kTmS + 32);
      if (wrote_last(&written[kCntP], warps)) {
        for (int i = 0; i < t.nheads; ++i)
          mma_tri<BWD, BWD>(tm + kTmY + i * kC, tm + kTmS, heads + i * l.head + 2 * kDeltaTri,
                            heads + i * l.head + 3 * kDeltaTri);
        tc::commit(&bars[kBarP]);
      }
      __syncwarp();

      // ---- S <- e^G_end S + K^T u, and its pieces for the next chunk
      const float end = sc[kScEnd * kC];
      ok = wait_mma(&bars[kBarU], par, p.wait_limit_ns);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < N / 64; ++i) {
        tm_load(row + kTmU + 64 * i, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float(&s)[4] = S[8 * i + j];
          const float2 a = fma2(make_float2(s[0], s[1]), make_float2(end, end),
                                mul2(make_float2(x[j][0], x[j][1]), make_float2(r0.inv, r0.inv)));
          const float2 b = fma2(make_float2(s[2], s[3]), make_float2(end, end),
                                mul2(make_float2(x[j][2], x[j][3]), make_float2(r1.inv, r1.inv)));
          s[0] = a.x; s[1] = a.y; s[2] = b.x; s[3] = b.y;
        }
      }
      ok = wait_mma(&bars[kBarP], par, p.wait_limit_ns);  // the columns of the pieces are free
      if (!ok) break;
      if (c + 1 < p.nchunks) put_state(c + 1);
      if (BWD) store_state<N, N>(S, p.ws_state + st_at, 1.f, 1.f, lane);

      // ---- Y
      tm_load(row + kTmY + hcol, x);
      scale_rows(x, w0.inv, w1.inv);
      scale_cols(x, sc + kScP * kC, lane);
      add_tiles(y, x);
      if (BWD) {
        load_rows(x, vrow + kCol, 0, m);
        row_dots(x, y, p.ws_doto + (bch * pb + pw / 16) * kC, lane);
      } else if (d.y) {
        store_rows(y, vrow, 0, static_cast<uint16_t*>(d.y) + col_at0 + t0 * vs, vs, valid, lane, m);
      }
      if (last_of(&count[st], warps) && c + p.stages < p.nchunks)
        issue(p, t, l, smem, full, c + p.stages, st);
      __syncwarp();
    }
    if (ok) {
      if (!BWD && d.h_last) store_state<N, N>(S, d.h_last + state_at, 1.f, 1.f, lane);
    } else {
      // leave when this warp's products and the CTA's copies have ended, or that wait has run out too
      if (lane == 0) tc::commit(&bars[kBarDrain]);
      mbar_wait_bounded(&bars[kBarDrain], 0, p.wait_limit_ns);
      give_up(p, full, c);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tm, kTmemCols);
}

// The largest number of row blocks per CTA (one CTA fills an SM) of at most two
// heads and two stages, halved while the grid then still is no larger than the
// SMs: the chain is shorter with fewer warps per scheduler.
template <int N, bool BWD>
cudaError_t run(DeltaChunkParams p, cudaStream_t stream) {
  const int per_head = p.d.headdim / 16, group = p.d.nheads / p.d.nkheads * per_head;
  const int64_t groups = (int64_t)p.d.batch * p.d.nkheads;
  const int tiles = BWD ? 2 : 1, head_bytes = BWD ? kDeltaHeadBwd : kDeltaHeadFwd;
  auto lay = [&](int blocks) { return layout(N, blocks, per_head, tiles, head_bytes); };
  auto extra = [&](int blocks) { return blocks * 2 * tiles * kCol + 1024; };
  auto stages_of = [&](int blocks) {
    return std::min(kMaxStages, (225 * 1024 - extra(blocks)) / lay(blocks).stage);
  };
  auto ctas = [&](int blocks) { return groups * ((group + blocks - 1) / blocks); };
  int blocks = kMaxBlocks;
  while (blocks > 1 && (blocks / 2 >= group || lay(blocks).heads > kTcHeads || stages_of(blocks) < 2 ||
                        ctas(blocks / 2) <= 148))
    blocks /= 2;
  const char* force = getenv("SSM_DELTA_BLOCKS");
  if (force && *force && lay(atoi(force)).heads <= kTcHeads && stages_of(atoi(force)) >= 2) blocks = atoi(force);
  p.blocks = blocks;
  p.stages = stages_of(blocks);
  if (p.stages < 2) return cudaErrorInvalidValue;
  const int bytes = lay(blocks).stage * p.stages + extra(blocks);
  const cudaError_t e = cudaFuncSetAttribute(delta_tc_kernel<N, BWD>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  delta_tc_kernel<N, BWD><<<(unsigned)ctas(blocks), blocks * 32, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_tc(const DeltaChunkParams& p, bool bwd, cudaStream_t stream) {
  if (bwd) return p.d.dstate == 64 ? run<64, true>(p, stream) : run<128, true>(p, stream);
  return p.d.dstate == 64 ? run<64, false>(p, stream) : run<128, false>(p, stream);
}

cudaError_t delta_tc_status(cudaStream_t stream, int* timed_out) {
  return timeout_status(stream, timed_out);
}

}  // namespace ssm
