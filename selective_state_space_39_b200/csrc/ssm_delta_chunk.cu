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

#include "ssm_delta_rows.cuh"

namespace ssm {

namespace {

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
  if (!getenv("SSM_DELTA_OLD")) return launch_delta_tc(pin, bwd, stream);
  DeltaChunkParams p = pin;
  if (bwd) return p.d.dstate == 64 ? fwd<64, true>(p, stream) : fwd<128, true>(p, stream);
  return p.d.dstate == 64 ? fwd<64, false>(p, stream) : fwd<128, false>(p, stream);
}

cudaError_t launch_delta_chunk_rev(const DeltaChunkParams& pin, cudaStream_t stream) {
  DeltaChunkParams p = pin;
  return p.d.dstate == 64 ? rev<64>(p, stream) : rev<128>(p, stream);
}

cudaError_t delta_chunk_status(cudaStream_t stream, int* timed_out) {
  int tc = 0;
  cudaError_t e = delta_tc_status(stream, &tc);
  if (e == cudaSuccess) e = timeout_status(stream, timed_out);
  *timed_out |= tc;
  return e;
}

}  // namespace ssm
