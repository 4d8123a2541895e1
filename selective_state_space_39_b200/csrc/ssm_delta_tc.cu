// ssm_delta_tc.cu -- the gated delta rule chunk by chunk on the fifth-generation
// tensor cores (tcgen05; bf16 io, sm_100a): the walk over the chunks, alone or
// for the gradients (BWD: it keeps the states, r and dy.y), and the walk back.
//
// Per head, with the operands of ssm_delta_prep.cu and the state S (headdim x
// dstate) entering a chunk:
//   R = V - (e^G K) S^T,  r = T R,  u = beta r
//   Y = (e^G Q) S^T + P u
//   S <- e^G_end S + u^T (e^(G_end - G) K)
// and back, dS being the adjoint of the state after the chunk:
//   dU = P^T dY + e^(G_end - G) K dS^T,  dV = dR = T^T (beta dU)
//   dS <- e^G_end dS + dY^T (e^G Q) - dR^T (e^G K)
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
// A chunk is a chain S -> K S -> R -> T R -> u -> K^T u -> S of three products;
// Q S, P u and the writing of Y run beside it. One warp issues the copies and
// the products: the row warps tell it by mbarriers that an operand is written,
// it tells them by commits that a product is done. With up to four row blocks
// two warps share one (half the tokens and half of dstate each; they compare
// row maxima through shared memory), which halves the arithmetic on the chain;
// with more blocks one warp takes a block, the registers of its two warpgroups
// raised at the issuing warpgroup's expense. With two heads in a CTA the T and
// P products are taken for both heads on all rows, and a row reads its own
// head's columns.
//
// Precision: everything on the state's path is a product of two pieces per
// operand (k and q are exact in one; lo lo is left out), so the carried state,
// dh0 and the gate gradients keep fp32's accuracy; for y, rounded to bf16, one
// fp16 piece (2^-12) of S, u and P is taken: beside its rounding y is off by
// that of its terms, which shows where they cancel (a second piece of P is 5 KB
// more per chunk and head; the backward pass, which sums dy . y, has it). Rows
// whose values one scale does not hold go token by token (walk_tokens).
//
// Bound: the chain of a chunk (products, commits, tensor memory loads, row maxima,
// splitting), in every head at once: 8192 tokens of 32 heads of 128, dstate 128
// take 312 us, 2.4 us per chunk (128 CTAs of 32 rows); 4 x 4096 tokens of 64 heads of 64: 265 us, 4.1 us per
// chunk (128 CTAs of 128 rows; tensor pipe 27 % busy, DRAM 2.4 TB/s). For the
// backward pass, 2 x 2048 tokens of 32 heads of 128: 129 us, and 147 us back; both
// move a state per chunk (2.6 TB/s).
//
// Tensor memory (512 columns), forward: 0 S pieces, then u's pieces for P; 128 K S, R's
// pieces, u's pieces for K^T; 192 Q S; 256 T R per head, then K^T u; 384 P u
// per head. Back: 0 dS pieces; 128 K dS, dU's pieces, dR's pieces; 192 dY's
// pieces, for P^T, then for Q^T; 256 P^T dY per head, then the sum for dS; 384
// T^T dU per head.
#include "ssm_delta_rows.cuh"
#include "ssm_tc.cuh"

namespace ssm {

namespace {

constexpr int kTmemCols = 512;
constexpr uint32_t kTmS = 0, kTmX = 128, kTmO = 192, kTmU = 256, kTmY = 384;
constexpr int kTcHeads = 2;  // heads per CTA, at most

// 8 T accumulator columns of the warp's 16 lanes.
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
__device__ __forceinline__ void tm_load(uint32_t addr, float (&x)[4][4]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
  tc::wait_ld();
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) x[j][q] = __uint_as_float(r[4 * j + q]);
}
// 8 T fp16 columns (4 T columns of tensor memory) of the warp's 16 lanes.
__device__ __forceinline__ void tm_store(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_store(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// T tiles under row scales s0, s1 as pieces at hi and (LO) lo.
template <bool LO, int T>
__device__ __forceinline__ void tm_pieces(const float (*x)[4], float s0, float s1, uint32_t hi_at,
                                          uint32_t lo_at) {
  uint32_t hi[2 * T], lo[2 * T];
#pragma unroll
  for (int j = 0; j < T; ++j) {
    split2(x[j][0], x[j][1], s0, hi[2 * j], lo[2 * j]);
    split2(x[j][2], x[j][3], s1, hi[2 * j + 1], lo[2 * j + 1]);
  }
  tm_store(hi_at, hi);
  if (LO) tm_store(lo_at, lo);
}

// ------------------------------------------------------- the issuing warp ----
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// D (128 rows x n) += A (16 columns of k in tensor memory) B, the descriptor of
// B as its two words.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi,
                                    uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ constexpr uint32_t idesc(int n, int b_mn) {  // fp16, fp32 sums, M = 128
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
// Upper word of a descriptor: the distance of eight-row groups, version 1, swizzle.
constexpr uint32_t kDescSw = (1024u >> 4) | (1u << 14) | (2u << 29);  // 128-byte swizzle
constexpr uint32_t kDescTri = (256u >> 4) | (1u << 14);               // core matrices

// D = X (pieces at a, a + dstate / 2) tile^T, the tile's rows being D's columns.
template <int N, bool LO>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t a, uint32_t tile) {
  const uint32_t b = (tile >> 4) | (1u << 16);
#pragma unroll
  for (int piece = 0; piece < (LO ? 2 : 1); ++piece)
#pragma unroll
    for (int ks = 0; ks < N / 16; ++ks)
      mma(d, a + piece * (N / 2) + 8 * ks, b + (ks / 4) * (kC * 128 / 16) + (ks % 4) * 2, kDescSw,
          idesc(kC, 0), piece + ks > 0);
}
// D (rows x dstate) = X (64 tokens, pieces at a and a + 32) tile.
template <int N>
__device__ __forceinline__ void mma_tokens(uint32_t d, uint32_t a, uint32_t tile, bool acc = false) {
  const uint32_t b = (tile >> 4) | ((uint32_t)(kC * 128 / 16) << 16);  // to the next 64 columns
#pragma unroll
  for (int piece = 0; piece < 2; ++piece)
#pragma unroll
    for (int ks = 0; ks < kC / 16; ++ks)
      mma(d, a + piece * 32 + 8 * ks, b + ks * 128, kDescSw, idesc(N, 1), acc || piece + ks > 0);
}
// D (rows x 64 tokens) = X (64 tokens, pieces at a, a + 32) tri^T, the lower
// triangular tile in one or two pieces (`lo` after `hi`); a step over 16 tokens
// reaches the columns from those tokens on.
template <bool XLO, bool BLO>
__device__ __forceinline__ void mma_tri(uint32_t d, uint32_t a, uint32_t tri) {
  const uint32_t b = (tri >> 4) | ((128u >> 4) << 16);  // to the next eight columns
#pragma unroll
  for (int piece = 0; piece < 3; ++piece) {
    if ((piece == 1 && !XLO) || (piece == 2 && !BLO)) continue;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
      mma(d + 16 * kt, a + (piece == 1 ? 32 : 0) + 8 * kt,
          b + (delta_tri_block(kt, kt) + (piece == 2 ? kDeltaTri : 0)) / 16, kDescTri,
          idesc(kC - 16 * kt, 0), piece + kt > 0);
  }
}

// D (rows x 64 tokens) = X (64 tokens, pieces at a, a + 32) tri, from the tile's
// transpose in two pieces; a step over 16 rows of tri reaches its columns up to
// them (the last step reaches all, and goes first).
__device__ __forceinline__ void mma_tri_t(uint32_t d, uint32_t a, uint32_t tri_t) {
  const uint32_t b = (tri_t >> 4) | ((128u >> 4) << 16);
#pragma unroll
  for (int piece = 0; piece < 3; ++piece)
#pragma unroll
    for (int kt = 3; kt >= 0; --kt)
      mma(d, a + (piece == 1 ? 32 : 0) + 8 * kt,
          b + (delta_tri_block_t(kt, 0) + (piece == 2 ? kDeltaTri : 0)) / 16, kDescTri,
          idesc(16 * kt + 16, 0), piece > 0 || kt < 3);
}

// mbarriers of a CTA. Products done, forward: K S, Q S, T R, K^T u, P u; back: K
// dS, P^T dY, T^T dU, the sum for dS. Operands written by the row warps,
// forward: S, R, u for K^T, u for P; back: dS, dY for P^T, dU, dR and dY for dS.
// A failed CTA's drain.
enum { kBarK, kBarQ, kBarT, kBarU, kBarP, kPutS, kPutR, kPutU, kPutP, kBarDrain, kBars };

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// The warp's part of an operand is in tensor memory.
__device__ __forceinline__ void wrote(uint64_t* bar) {
  tc::wait_st();
  tc::fence_before_sync();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit));
  tc::fence_after_sync();
  return ok;
}

template <int N, bool BWD>
__device__ __forceinline__ void issue_loop(const DeltaChunkParams& p, const Cta& t, const Layout& l,
                                           unsigned char* smem, uint64_t* full, uint64_t* freed,
                                           uint64_t* bars, uint32_t tm) {
  if (elect_one()) {
    for (int s = 0; s < p.stages && s < p.nchunks; ++s)
      if (!(p.test_stall && s == 0 && blockIdx.x == 0))  // its data never arrives
        issue(p, t, l, smem, full, s, s);
  }
  __syncwarp();
  const uint32_t s0 = smem_u32(smem);
  bool ok = true;
  int c = 0, st = 0, prev = 0;
  uint32_t fpar = 0, ppar = 0;  // parities of this and the previous chunk's stage
  for (; c < p.nchunks; ++c) {
    const uint32_t par = (uint32_t)(c & 1);
    const uint32_t ks = s0 + (uint32_t)(st * l.stage), heads = ks + (uint32_t)l.kq;
    ok = wait_warp(&full[st], fpar, p.wait_limit_ns) && wait_warp(&bars[kPutS], par, p.wait_limit_ns);
    if (!ok) break;
    if (elect_one()) {
      mma_state<N, true>(tm + kTmX, tm + kTmS, ks);
      tc::commit(&bars[kBarK]);
      mma_state<N, BWD>(tm + kTmO, tm + kTmS, ks + (uint32_t)(l.kq / 2));
      tc::commit(&bars[kBarQ]);
    }
    __syncwarp();
    ok = wait_warp(&bars[kPutR], par, p.wait_limit_ns);
    if (!ok) break;
    if (elect_one()) {
      mma_tri<true, true>(tm + kTmU, tm + kTmX, heads);
      if (t.nheads > 1) mma_tri<true, true>(tm + kTmU + kC, tm + kTmX, heads + (uint32_t)l.head);
      tc::commit(&bars[kBarT]);
    }
    __syncwarp();
    // the row warps are done with the previous chunk: refill its stage
    if (c > 0 && c - 1 + p.stages < p.nchunks) {
      ok = wait_warp(&freed[prev], ppar, p.wait_limit_ns);
      if (!ok) break;
      if (elect_one()) {
        fence_async_smem();
        issue(p, t, l, smem, full, c - 1 + p.stages, prev);
      }
      __syncwarp();
    }
    ok = wait_warp(&bars[kPutU], par, p.wait_limit_ns);
    if (!ok) break;
    if (elect_one()) {
      mma_tokens<N>(tm + kTmU, tm + kTmX, ks);
      tc::commit(&bars[kBarU]);
    }
    __syncwarp();
    ok = wait_warp(&bars[kPutP], par, p.wait_limit_ns);
    if (!ok) break;
    if (elect_one()) {
      mma_tri<BWD, BWD>(tm + kTmY, tm + kTmS, heads + 2 * kDeltaTri);
      if (t.nheads > 1)
        mma_tri<BWD, BWD>(tm + kTmY + kC, tm + kTmS, heads + (uint32_t)l.head + 2 * kDeltaTri);
      tc::commit(&bars[kBarP]);
    }
    __syncwarp();
    prev = st;
    ppar = fpar;
    if (++st == p.stages) {
      st = 0;
      fpar ^= 1u;
    }
  }
  if (!ok) {  // leave when the products and copies in flight have ended, or that wait has run out too
    if (elect_one()) tc::commit(&bars[kBarDrain]);
    __syncwarp();
    mbar_wait_bounded(&bars[kBarDrain], 0, p.wait_limit_ns);
    give_up(p, full, c);
  }
}

// Largest magnitudes of the rows over both warps of a pair. The pair's barriers
// have no limit of their own: both warps come to every one of them, also after
// a wait that ran out (they go on to the end of the chunk), and leave together
// by the vote.
__device__ __forceinline__ void put_max(float m0, float m1, float* mine, int lane) {
  if ((lane & 3) == 0) {
    mine[lane >> 2] = m0;
    mine[8 + (lane >> 2)] = m1;
  }
}
__device__ __forceinline__ void get_max(float& m0, float& m1, const float* other, int lane) {
  m0 = max_nan(m0, other[lane >> 2]);
  m1 = max_nan(m1, other[8 + (lane >> 2)]);
}

constexpr int kRowWarps = 8, kTcThreads = kRowWarps * 32 + 128;

// ---- rows that the pieces do not hold --------------------------------------
// A row's pieces stand under one scale for the chunk's 64 tokens and hold 2^-40 of the
// largest. A value that is not finite, or one so large that it leaves the others too few
// bits, must not reach the tokens before it, nor those behind a decay that forgets it: the
// 16 rows then take the chunk token by token in fp32, in the fragments they hold the
// state in. (A row whose state has a NaN is NaN from there on either way.)
//
// Whether a row has values too small beside its largest m: neighbours both below 2^-24
// of it (16 bits left), or a single one below 2^-32. Exact zeros need no bits.
__device__ __forceinline__ bool too_small(float a, float b, float m) {
  const float both = fmaxf(a, b), pair = m * 0x1p-24f, one = m * 0x1p-32f;
  return (both < pair && both > 0.f) || (a < one && a > 0.f) || (b < one && b > 0.f);
}
// What a residual x = v - (its decayed prediction) stands for: it may well be small where
// v is not, and where v is zero (a masked token) and the prediction decayed, it is the
// state, of largest magnitude s.
__device__ __forceinline__ float size_of(float x, float v, float s) {
  return v != 0.f ? fmaxf(fabsf(x), fabsf(v)) : (x != 0.f ? s : 0.f);
}
// By the residuals alone first (of this lane), a third of the instructions: hardly a
// chunk has one.
template <int T>
__device__ __forceinline__ bool maybe_wide(const float (&x)[T][4], float m0, float m1) {
  float both0 = m0, both1 = m1, one0 = m0, one1 = m1;
#pragma unroll
  for (int j = 0; j < T; ++j) {
    both0 = fminf(both0, fmaxf(fabsf(x[j][0]), fabsf(x[j][1])));
    both1 = fminf(both1, fmaxf(fabsf(x[j][2]), fabsf(x[j][3])));
    one0 = fminf(one0, fminf(fabsf(x[j][0]), fabsf(x[j][1])));
    one1 = fminf(one1, fminf(fabsf(x[j][2]), fabsf(x[j][3])));
  }
  return both0 < m0 * 0x1p-24f || both1 < m1 * 0x1p-24f || one0 < m0 * 0x1p-32f || one1 < m1 * 0x1p-32f;
}
template <int T>
__device__ __forceinline__ bool wide_rows(bool maybe, const float (&x)[T][4], const float (&v)[T][4], float m0,
                                          float m1, float s0, float s1) {
  if (!__any_sync(0xffffffffu, maybe)) return false;
  bool wide = false;
#pragma unroll
  for (int j = 0; j < T; ++j) {
    wide |= too_small(size_of(x[j][0], v[j][0], s0), size_of(x[j][1], v[j][1], s0), m0);
    wide |= too_small(size_of(x[j][2], v[j][2], s1), size_of(x[j][3], v[j][3], s1), m1);
  }
  return __any_sync(0xffffffffu, wide);
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
// The sums of both warps of a pair, six values a lane (mine, other: their places for 16
// floats in three buffers, kRowWarps * 16 apart): two of rows g and g + 8, four of all.
template <int SP>
__device__ __forceinline__ void pair_sum(float (&r)[8], float* mine, const float* other, int id, int lane) {
  if (SP == 1) return;
  constexpr int kNext = kRowWarps * 16;
  pair_sync(id);  // the buffers' last readers are done
  if ((lane & 3) == 0) {
    mine[lane >> 2] = r[0];
    mine[8 + (lane >> 2)] = r[1];
    mine[kNext + (lane >> 2)] = r[2];
    mine[kNext + 8 + (lane >> 2)] = r[3];
  }
  if (lane < 4) mine[2 * kNext + lane] = lane == 0 ? r[4] : (lane == 1 ? r[5] : (lane == 2 ? r[6] : r[7]));
  pair_sync(id);
  r[0] += other[lane >> 2];
  r[1] += other[8 + (lane >> 2)];
  r[2] += other[kNext + (lane >> 2)];
  r[3] += other[kNext + 8 + (lane >> 2)];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[4 + i] += other[2 * kNext + i];
}

// Rows g and g + 8 of 16 (pw: the first) and the warp's columns, through chunk c: y (BWD:
// r and dy . y), and the state S [NS / 8][4] from before the chunk to after it. Both
// warps of a pair.
template <int N, int SP, bool BWD>
__device__ __noinline__ void walk_tokens(const DeltaChunkParams& p, int b, int h, int pw, int c, int id,
                                         float* mine, const float* other, float* state) {
  constexpr int NS = N / SP;
  const DeltaParams& d = p.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hf = SP == 2 ? (warp >> 2) & 1 : 0, kh = h / (d.nheads / d.nkheads);
  const int64_t t0 = (int64_t)c * kC;
  const int valid = (int)min((int64_t)kC, d.seqlen - t0);
  const size_t bch = ((size_t)b * p.nchunks + c) * d.nheads + h;
  const float A = d.A[h], bias = d.dt_bias ? d.dt_bias[h] : 0.f;
  float s[NS / 8][4];
#pragma unroll
  for (int j = 0; j < NS / 8; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) s[j][q] = state[4 * j + q];
  if (BWD && lane == 0)
    reinterpret_cast<float*>(p.ws_head + bch * (size_t)p.head_bytes + 4 * kDeltaTri)[kScEnd * kC + 5] = 1.f;
#pragma unroll 1
  for (int t = 0; t < valid; ++t) {
    const size_t row = (size_t)b * d.seqlen + t0 + t;
    const uint16_t* kr = static_cast<const uint16_t*>(d.k) + (row * d.nkheads + kh) * N + hf * NS + 2 * (lane & 3);
    const uint16_t* qr = static_cast<const uint16_t*>(d.q) + (row * d.nkheads + kh) * N + hf * NS + 2 * (lane & 3);
    float r[8] = {};  // S k, S q of both rows; k.k, q.q, k.q
    uint32_t kv[NS / 8];
#pragma unroll
    for (int j = 0; j < NS / 8; ++j) {
      kv[j] = *reinterpret_cast<const uint32_t*>(kr + 8 * j);
      const uint32_t qv = *reinterpret_cast<const uint32_t*>(qr + 8 * j);
      const float k0 = bf16_lo(kv[j]), k1 = bf16_hi(kv[j]), q0 = bf16_lo(qv), q1 = bf16_hi(qv);
      r[0] = fmaf(s[j][0], k0, fmaf(s[j][1], k1, r[0]));
      r[1] = fmaf(s[j][2], k0, fmaf(s[j][3], k1, r[1]));
      r[2] = fmaf(s[j][0], q0, fmaf(s[j][1], q1, r[2]));
      r[3] = fmaf(s[j][2], q0, fmaf(s[j][3], q1, r[3]));
      r[4] = fmaf(k0, k0, fmaf(k1, k1, r[4]));
      r[5] = fmaf(q0, q0, fmaf(q1, q1, r[5]));
      r[6] = fmaf(k0, q0, fmaf(k1, q1, r[6]));
    }
#pragma unroll
    for (int i = 0; i < 7; ++i) r[i] = quad_sum(r[i]);
    pair_sum<SP>(r, mine, other, id, lane);
    const float kn = d.qk_norm ? rsqrtf(r[4] + kDeltaQkEps) : 1.f;
    const float qn = (d.qk_norm ? rsqrtf(r[5] + kDeltaQkEps) : 1.f) * d.scale;
    const float step = delta_step_size(bf16_to_f32(static_cast<const uint16_t*>(d.dt)[row * d.nheads + h]) + bias,
                                       d.softplus);
    const float a = expf(step * A);
    const float beta = delta_beta(bf16_to_f32(static_cast<const uint16_t*>(d.beta)[row * d.nheads + h]),
                                  d.beta_sigmoid);
    const size_t at = (row * d.nheads + h) * d.headdim + pw + (lane >> 2);
    const uint16_t* v = static_cast<const uint16_t*>(d.v) + at;
    const float r0 = bf16_to_f32(v[0]) - a * kn * r[0], r1 = bf16_to_f32(v[8]) - a * kn * r[1];
    const float w0 = beta * r0 * kn, w1 = beta * r1 * kn;
    const float y0 = qn * fmaf(a, r[2], w0 * r[6]), y1 = qn * fmaf(a, r[3], w1 * r[6]);
#pragma unroll
    for (int j = 0; j < NS / 8; ++j) {
      const float k0 = bf16_lo(kv[j]), k1 = bf16_hi(kv[j]);
      s[j][0] = fmaf(w0, k0, a * s[j][0]);
      s[j][1] = fmaf(w0, k1, a * s[j][1]);
      s[j][2] = fmaf(w1, k0, a * s[j][2]);
      s[j][3] = fmaf(w1, k1, a * s[j][3]);
    }
    if (BWD) {
      float dot = fmaf(bf16_to_f32(p.dy[at]), y0, bf16_to_f32(p.dy[at + 8]) * y1);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (hf == 0 && lane == 0) p.ws_doto[(bch * (d.headdim / 16) + pw / 16) * kC + t] = dot;
    }
    uint16_t* out = BWD ? p.ws_r : static_cast<uint16_t*>(d.y);
    if (hf == 0 && (lane & 3) == 0 && out) {
      out[at] = f32_to_bf16(BWD ? r0 : y0);
      out[at + 8] = f32_to_bf16(BWD ? r1 : y1);
    }
  }
  if (BWD && hf == 0)
    for (int t = valid + lane; t < kC; t += 32) p.ws_doto[(bch * (d.headdim / 16) + pw / 16) * kC + t] = 0.f;
#pragma unroll
  for (int j = 0; j < NS / 8; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) state[4 * j + q] = s[j][q];
  if (SP == 2) pair_sync(id);  // the buffers are free
}

// SP warps share a block of 16 rows (BWD: two).
template <int N, int SP, bool BWD>
__global__ void __launch_bounds__(kTcThreads, 1)
    delta_tc_kernel(const __grid_constant__ DeltaChunkParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], freed[kMaxStages], bars[kBars];
  __shared__ float maxima[3][kRowWarps][16];  // a buffer per use in a chunk
  __shared__ uint32_t slot;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int NS = N / SP, TT = 8 / SP;  // the warp's part of dstate, its token tiles
  constexpr int kTris = BWD ? 4 : 3, kTiles = BWD ? 2 : 1;
  const DeltaParams& d = p.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pb = d.headdim / 16;
  const Cta t = cta_of(p);
  const Layout l = layout(N, p.blocks, pb, BWD ? kDeltaLoadBwd : kDeltaHeadFwd, 0);
  if (threadIdx.x == 0) {
    const uint32_t warps = (uint32_t)t.active * SP;
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&freed[i], warps);
    }
    for (int i = 0; i < kBars; ++i)
      mbar_init(&bars[i], (i >= kPutS && i <= kPutP) ? warps : 1u);
    fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(&slot, kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = __shfl_sync(0xffffffffu, slot, 0);
  chain_go();
  chain_wait();

  // a block's warps lie in one warpgroup column (warp % 4), which fixes the
  // tensor memory lanes they reach
  const int blk = SP == 2 ? warp & 3 : warp, hf = SP == 2 ? (warp >> 2) & 1 : 0;
  if (warp >= kRowWarps) {
    // 256 x 232 + 128 x 40 registers: what the 384 threads were launched with (168 each)
    if (SP == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == kRowWarps) issue_loop<N, BWD>(p, t, l, smem, full, freed, bars, tm);
  } else {
    if (SP == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    if (blk < t.active) {
      const uint32_t row = tm + ((uint32_t)(32 * (warp & 3) + (SP == 1 ? 16 * (warp >> 2) : 0)) << 16);
      const uint32_t lc = lane_col(lane);
      const int rb = t.rb0 + blk, hx = rb / pb;  // row block in the group, its head
      const int h = t.kh * (d.nheads / d.nkheads) + hx, pw = (rb - hx * pb) * 16;
      const int tk = 32 * hf, tcol = 32 * hf;  // first token and its column of an accumulator
      const uint32_t hcol = (uint32_t)(h - t.h0) * kC + tcol;  // the head's columns of U and Y
      const size_t part = (size_t)pw * N + hf * NS;
      const size_t state_at = ((size_t)t.b * d.nheads + h) * ((size_t)d.headdim * N) + part;
      const size_t vs = (size_t)d.nheads * d.headdim;
      const uint32_t col0 = smem_u32(smem + (size_t)p.stages * l.stage) + blk * 2 * kTiles * kCol;
      const size_t col_at0 = (size_t)t.b * d.seqlen * vs + (size_t)h * d.headdim + pw;
      float* const mx = &maxima[0][warp][0];
      const float* const ox = &maxima[0][warp ^ 4][0];
      // BWD: the warp's rows of the state on their way out
      const uint32_t out16 = smem_u32(smem + (size_t)p.stages * l.stage) + p.blocks * 2 * kTiles * kCol +
                             (blk * SP + hf) * 16 * (NS + 8) * 2;
      auto fetch = [&](int c) {  // the warp's tokens of its block's columns
        const int valid = (int)min((int64_t)kC, d.seqlen - (int64_t)c * kC);
        const size_t at = col_at0 + (size_t)c * kC * vs;
        const uint32_t to = col0 + (c & 1) * kTiles * kCol;
        fetch_rows<TT>(to, static_cast<const uint16_t*>(d.v) + at, vs, tk, valid, lane);
        if (BWD) fetch_rows<TT>(to + kCol, p.dy + at, vs, tk, valid, lane);
        cp_async_commit_group();
      };
      fetch(0);
      float S[NS / 8][4], inv0 = 1.f, inv1 = 1.f;  // the state's rows, the inverse of its pieces' scale
      float big0 = 0.f, big1 = 0.f;  // its largest magnitudes, NaN where it has one
      load_state<N, NS>(S, d.h0 ? d.h0 + state_at : nullptr, lane);
      auto meet = [&](float& m0, float& m1, int use) {
        if (SP == 1) return;
        put_max(m0, m1, mx + use * kRowWarps * 16, lane);
        pair_sync(1 + (warp & 3));
        get_max(m0, m1, ox + use * kRowWarps * 16, lane);
      };
      // the state's pieces, unless a wait has run out in either warp
      auto put_state = [&](bool ok) {
        float m0, m1;
        row_max(S, m0, m1);
        if (SP == 2) {
          put_max(m0, m1, mx, lane);
          ok = pair_and(1 + (warp & 3), ok);
          get_max(m0, m1, ox, lane);
        }
        if (!ok) return false;
        big0 = m0;
        big1 = m1;
        const RowScale a = row_scale(exponent_of(m0)), b = row_scale(exponent_of(m1));
        inv0 = a.inv;
        inv1 = b.inv;
        constexpr int G = NS / 8 < 8 ? NS / 8 : 8;  // tiles per store
#pragma unroll
        for (int i = 0; i < NS / 8; i += G)
          tm_pieces<true, G>(&S[i], a.s, b.s, row + kTmS + hf * (NS / 2) + 4 * i,
                             row + kTmS + N / 2 + hf * (NS / 2) + 4 * i);
        wrote(&bars[kPutS]);
        return true;
      };
      bool ok = put_state(true);
      int st = 0;
      uint32_t fpar = 0;
      for (int c = 0; ok && c < p.nchunks; ++c) {
        const uint32_t par = (uint32_t)(c & 1);
        const size_t bch = ((size_t)t.b * p.nchunks + c) * d.nheads + h;
        const size_t st_at = bch * ((size_t)d.headdim * N) + part;
        const int64_t t0 = (int64_t)c * kC;
        const int valid = (int)min((int64_t)kC, d.seqlen - t0);
        unsigned char* head = smem + (size_t)st * l.stage + l.kq + (h - t.h0) * l.head;
        const float* sc = reinterpret_cast<const float*>(head + kTris * kDeltaTri);
        const uint32_t vrow = col0 + (c & 1) * kTiles * kCol;

        // ---- R = V - (e^G K) S^T; T R
        float x[TT][4], u[TT][4], y[TT][4];
        ok = wait_stage(&full[st], fpar, p.wait_limit_ns);
        ok = wait_warp(&bars[kBarK], par, ok ? p.wait_limit_ns : 0) && ok;
        tm_load(row + kTmX + tcol, x);
        load_rows(u, vrow, tk, lc);
        scale_rows(x, -inv0, -inv1);
        scale_cols(x, sc + kScSk * kC + tk, lane);
        add_tiles(x, u);
        float m0, m1;
        row_max(x, m0, m1);
        meet(m0, m1, 1);
        RowScale r0 = row_scale(exponent_of(m0)), r1 = row_scale(exponent_of(m1));
        tm_pieces<true, TT>(x, r0.s, r1.s, row + kTmX + tcol / 2, row + kTmX + 32 + tcol / 2);
        wrote(&bars[kPutR]);

        // (the backward pass has no registers to keep R and V longer: 483 us for 456; the
        // forward pass alone gains by it: 8192 tokens of 32 heads 393 us, not 397)
        bool wide = BWD && wide_rows(maybe_wide(x, m0, m1), x, u, m0, m1, big0, big1);

        // ---- meanwhile the next chunk's v, and the readout of the entering state
        if (c + 1 < p.nchunks) fetch(c + 1);
        ok = wait_warp(&bars[kBarQ], par, ok ? p.wait_limit_ns : 0) && ok;
        tm_load(row + kTmO + tcol, y);
        scale_rows(y, inv0, inv1);
        scale_cols(y, sc + kScSq * kC + tk, lane);
        if (BWD) store_state16<N, NS>(S, out16, p.ws_state16 + st_at, lane);

        // ---- u = beta T R; K^T (e^(G_end - G) u)
        if (!BWD) wide = wide_rows(maybe_wide(x, m0, m1), x, u, m0, m1, big0, big1);
        ok = wait_warp(&bars[kBarT], par, ok ? p.wait_limit_ns : 0) && ok;
        tm_load(row + kTmU + hcol, x);
        scale_rows(x, r0.inv, r1.inv);
        if (BWD) {  // r leaves by the rows of v
          scale_cols(x, sc + kScT * kC + tk, lane);
          stage_rows(x, vrow, tk, lc);
          if (sc[kScEnd * kC + 3] + sc[kScEnd * kC + 4] != 0.f) {  // and its rest, by the state's rows
#pragma unroll
            for (int j = 0; j < TT; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q) u[j][q] = x[j][q];
            rest_of(u);
            __syncwarp();
            stage_rows(u, out16 - tk * 32, tk, lc);
            store_rows<TT>(out16 - tk * 32, tk, p.ws_rlo + col_at0 + t0 * vs, vs, valid, lane);
          }
        }
        scale_cols(x, sc + (BWD ? kScBeta : kScU) * kC + tk, lane);
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) u[j][q] = x[j][q];
        scale_cols(u, sc + kScKend * kC + tk, lane);
        // one scale serves u's pieces for K^T and for P: e^(G_end - G) is at most
        // `most`, 1 unless a log decay is positive
        const float most = fmaxf(sc[kScEnd * kC + 1], sc[kScEnd * kC + 2]);
        scale_cols(x, sc + kScK * kC + tk, lane);
        row_max(x, m0, m1);
        m0 = wide ? __uint_as_float(0x7FFFFFFFu) : m0 * most;
        m1 = wide ? m0 : m1 * most;
        meet(m0, m1, 2);
        const bool alone = __any_sync(0xffffffffu, (not_finite(m0) && big0 == big0) || (not_finite(m1) && big1 == big1));
        r0 = row_scale(exponent_of(m0));
        r1 = row_scale(exponent_of(m1));
        tm_pieces<true, TT>(u, r0.s, r1.s, row + kTmX + tcol / 2, row + kTmX + 32 + tcol / 2);
        wrote(&bars[kPutU]);

        // ---- P u
        tm_pieces<BWD, TT>(x, r0.s, r1.s, row + kTmS + tcol / 2, row + kTmS + 32 + tcol / 2);
        wrote(&bars[kPutP]);
        if (BWD) store_rows<TT>(vrow, tk, p.ws_r + col_at0 + t0 * vs, vs, valid, lane);

        // ---- S <- e^G_end S + K^T u, and its pieces for the next chunk
        const float end = sc[kScEnd * kC];
        ok = wait_warp(&bars[kBarU], par, ok ? p.wait_limit_ns : 0) && ok;
        constexpr int G = NS / 8 < 8 ? NS / 8 : 8;  // tiles per load
        if (alone) {
          float s[NS / 2];
#pragma unroll
          for (int i = 0; i < NS / 2; ++i) s[i] = S[i / 4][i % 4];
          walk_tokens<N, SP, BWD>(p, t.b, h, pw, c, 1 + (warp & 3), mx, ox, s);
#pragma unroll
          for (int i = 0; i < NS / 2; ++i) S[i / 4][i % 4] = s[i];
        } else {
#pragma unroll
          for (int i = 0; i < NS / 8; i += G) {
            float ds[G][4];
            tm_load(row + kTmU + hf * NS + 8 * i, ds);
#pragma unroll
            for (int j = 0; j < G; ++j) {
              float(&s)[4] = S[i + j];
              const float2 a = fma2(make_float2(s[0], s[1]), make_float2(end, end),
                                    mul2(make_float2(ds[j][0], ds[j][1]), make_float2(r0.inv, r0.inv)));
              const float2 b = fma2(make_float2(s[2], s[3]), make_float2(end, end),
                                    mul2(make_float2(ds[j][2], ds[j][3]), make_float2(r1.inv, r1.inv)));
              s[0] = a.x; s[1] = a.y; s[2] = b.x; s[3] = b.y;
            }
          }
        }
        ok = wait_warp(&bars[kBarP], par, ok ? p.wait_limit_ns : 0) && ok;  // the columns of the pieces are free
        const RowScale w0 = r0, w1 = r1;
        const uint32_t ycol = row + kTmY + hcol;
        if (c + 1 < p.nchunks) ok = put_state(ok);
        if (!ok) break;
        if (BWD) store_tiles<NS>(S, p.ws_state + (st_at - part) + (size_t)pw * N + hf * 16 * NS, lane);

        // ---- Y
        if (!alone) {
          tm_load(ycol, x);
          scale_rows(x, w0.inv, w1.inv);
          scale_cols(x, sc + kScP * kC + tk, lane);
          add_tiles(y, x);
          if (BWD) {
            load_rows(x, vrow + kCol, tk, lc);
            row_dots(x, y, p.ws_doto + (bch * pb + pw / 16) * kC + tk, lane);
          } else if (d.y) {
            stage_rows(y, vrow, tk, lc);
            store_rows<TT>(vrow, tk, static_cast<uint16_t*>(d.y) + col_at0 + t0 * vs, vs, valid, lane);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&freed[st]);
        if (++st == p.stages) {
          st = 0;
          fpar ^= 1u;
        }
      }
      if (!ok) {
        if (lane == 0) atomicExch(&g_delta_timeout, 1);
      } else if (!BWD && d.h_last) {
        store_state<N, NS>(S, d.h_last + state_at, lane);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tm, kTmemCols);
}

// The issuing warp of the walk back; step s is chunk nchunks - 1 - s.
template <int N>
__device__ __forceinline__ void issue_back(const DeltaChunkParams& p, const Cta& t, const Layout& l,
                                           unsigned char* smem, uint64_t* full, uint64_t* freed,
                                           uint64_t* bars, uint32_t tm) {
  if (elect_one()) {
    for (int s = 0; s < p.stages && s < p.nchunks; ++s)
      issue(p, t, l, smem, full, p.nchunks - 1 - s, s);
  }
  __syncwarp();
  const uint32_t s0 = smem_u32(smem);
  bool ok = true;
  int s = 0, st = 0, prev = 0;
  uint32_t fpar = 0, ppar = 0;
  for (; s < p.nchunks; ++s) {
    const uint32_t par = (uint32_t)(s & 1);
    const uint32_t ks = s0 + (uint32_t)(st * l.stage);
    const uint32_t tiles = ks + (uint32_t)l.kq + (uint32_t)kDeltaScalBwd;  // T^T hi, lo, P^T hi, lo
    ok = wait_warp(&full[st], fpar, p.wait_limit_ns) && wait_warp(&bars[kPutS], par, p.wait_limit_ns);
    if (!ok) break;
    if (elect_one()) {
      mma_state<N, true>(tm + kTmX, tm + kTmS, ks);
      tc::commit(&bars[kBarK]);
    }
    __syncwarp();
    ok = wait_warp(&bars[kPutP], par, p.wait_limit_ns);
    if (!ok) break;
    if (elect_one()) {
      mma_tri_t(tm + kTmU, tm + kTmO, tiles + 2 * kDeltaTri);
      if (t.nheads > 1) mma_tri_t(tm + kTmU + kC, tm + kTmO, tiles + (uint32_t)l.head + 2 * kDeltaTri);
      tc::commit(&bars[kBarQ]);
    }
    __syncwarp();
    ok = wait_warp(&bars[kPutU], par, p.wait_limit_ns);
    if (!ok) break;
    if (elect_one()) {
      mma_tri_t(tm + kTmY, tm + kTmX, tiles);
      if (t.nheads > 1) mma_tri_t(tm + kTmY + kC, tm + kTmX, tiles + (uint32_t)l.head);
      tc::commit(&bars[kBarT]);
    }
    __syncwarp();
    if (s > 0 && s - 1 + p.stages < p.nchunks) {
      ok = wait_warp(&freed[prev], ppar, p.wait_limit_ns);
      if (!ok) break;
      if (elect_one()) {
        fence_async_smem();
        issue(p, t, l, smem, full, p.nchunks - (s + p.stages), prev);
      }
      __syncwarp();
    }
    ok = wait_warp(&bars[kPutR], par, p.wait_limit_ns);
    if (!ok) break;
    if (elect_one()) {
      mma_tokens<N>(tm + kTmU, tm + kTmO, ks + (uint32_t)(l.kq / 2));
      mma_tokens<N>(tm + kTmU, tm + kTmX, ks, true);
      tc::commit(&bars[kBarU]);
    }
    __syncwarp();
    prev = st;
    ppar = fpar;
    if (++st == p.stages) {
      st = 0;
      fpar ^= 1u;
    }
  }
  if (!ok) {
    if (elect_one()) tc::commit(&bars[kBarDrain]);
    __syncwarp();
    mbar_wait_bounded(&bars[kBarDrain], 0, p.wait_limit_ns);
    give_up(p, full, s);
  }
}

// The same back, for the 16 rows' whole sequence over what the walk left of it: everything
// that the walk writes, from dh_last on. (Chunk by chunk inside the walk, as forward, it
// cost the walk 8 % where no row needs it: 158 us for 2 x 2048 tokens of 32 heads of 128.)
template <int N>
__device__ __noinline__ void walk_back_tokens(const DeltaChunkParams& p, int b, int h, int pw, int id, float* mine,
                                              const float* other) {
  constexpr int NS = N / 2;
  const DeltaParams& d = p.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hf = (warp >> 2) & 1, kh = h / (d.nheads / d.nkheads), pb = d.headdim / 16;
  const float A = d.A[h], bias = d.dt_bias ? d.dt_bias[h] : 0.f;
  const size_t state_at = ((size_t)b * d.nheads + h) * ((size_t)d.headdim * N) + (size_t)pw * N + hf * NS;
  float s[NS / 8][4];
  load_state<N, NS>(s, p.dh_last ? p.dh_last + state_at : nullptr, lane);
  // a token's columns of k and q, its S k (of both rows; here dS k), k.k, q.q, k.q, and gates
  uint32_t kv[NS / 8], qv[NS / 8];
  float r[8], kn, qn, a, beta;
  auto token = [&](size_t row) {
    const size_t from = (row * d.nkheads + kh) * N + hf * NS + 2 * (lane & 3);
    const uint16_t *kr = static_cast<const uint16_t*>(d.k) + from, *qr = static_cast<const uint16_t*>(d.q) + from;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = 0.f;
#pragma unroll
    for (int j = 0; j < NS / 8; ++j) {
      kv[j] = *reinterpret_cast<const uint32_t*>(kr + 8 * j);
      qv[j] = *reinterpret_cast<const uint32_t*>(qr + 8 * j);
      const float k0 = bf16_lo(kv[j]), k1 = bf16_hi(kv[j]), q0 = bf16_lo(qv[j]), q1 = bf16_hi(qv[j]);
      r[0] = fmaf(s[j][0], k0, fmaf(s[j][1], k1, r[0]));
      r[1] = fmaf(s[j][2], k0, fmaf(s[j][3], k1, r[1]));
      r[4] = fmaf(k0, k0, fmaf(k1, k1, r[4]));
      r[5] = fmaf(q0, q0, fmaf(q1, q1, r[5]));
      r[6] = fmaf(k0, q0, fmaf(k1, q1, r[6]));
    }
#pragma unroll
    for (int i = 0; i < 7; ++i) r[i] = quad_sum(r[i]);
    pair_sum<2>(r, mine, other, id, lane);
    kn = d.qk_norm ? rsqrtf(r[4] + kDeltaQkEps) : 1.f;
    qn = (d.qk_norm ? rsqrtf(r[5] + kDeltaQkEps) : 1.f) * d.scale;
    const size_t at = row * d.nheads + h;
    a = expf(delta_step_size(bf16_to_f32(static_cast<const uint16_t*>(d.dt)[at]) + bias, d.softplus) * A);
    beta = delta_beta(bf16_to_f32(static_cast<const uint16_t*>(d.beta)[at]), d.beta_sigmoid);
  };
  auto rows_sum = [&](float x) {  // over the 16 rows
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };
#pragma unroll 1
  for (int c = p.nchunks - 1; c >= 0; --c) {
    const int64_t t0 = (int64_t)c * kC;
    const int valid = (int)min((int64_t)kC, d.seqlen - t0);
    const size_t bch = ((size_t)b * p.nchunks + c) * d.nheads + h, dot_at = (bch * pb + pw / 16) * kC;
    const float* sc = reinterpret_cast<const float*>(p.ws_head + bch * (size_t)p.head_bytes + 4 * kDeltaTri);
    const bool strong = sc[kScEnd * kC + 3] + sc[kScEnd * kC + 4] != 0.f, whole = sc[kScEnd * kC + 5] == 0.f;
    {  // dS after the chunk, its product with the state
      const float* after = p.ws_state + bch * ((size_t)d.headdim * N) + (size_t)pw * N + hf * 16 * NS;
      uint16_t* out = p.ws_dstate16 + bch * ((size_t)d.headdim * N) + (size_t)(pw + (lane >> 2)) * N + hf * NS +
                      2 * (lane & 3);
      const float dot = tiles_dot<NS>(s, after, lane);
      if (lane == 0) p.ws_end[(bch * pb + pw / 16) * 2 + hf] = dot;
#pragma unroll
      for (int j = 0; j < NS / 8; ++j) {
        *reinterpret_cast<uint32_t*>(out + 8 * j) = pack_bf16x2(s[j][0], s[j][1]);
        *reinterpret_cast<uint32_t*>(out + 8 * N + 8 * j) = pack_bf16x2(s[j][2], s[j][3]);
      }
    }
    if (strong) {  // r . e^(G_end - G) dS k
      float e = 1.f;
#pragma unroll 1
      for (int t = valid - 1; t >= 0; --t) {
        const size_t row = (size_t)b * d.seqlen + t0 + t, at = (row * d.nheads + h) * d.headdim + pw + (lane >> 2);
        token(row);
        float r0 = bf16_to_f32(p.ws_r[at]), r1 = bf16_to_f32(p.ws_r[at + 8]);
        if (whole) {
          r0 += bf16_to_f32(p.ws_rlo[at]);
          r1 += bf16_to_f32(p.ws_rlo[at + 8]);
        }
        const float dot = rows_sum(e * kn * fmaf(r[0], r0, r[1] * r1));
        if (hf == 0 && lane == 0) p.ws_doth[dot_at + t] = dot;
        e *= a;
      }
    }
    if (hf == 0)
      for (int t = valid + lane; t < kC; t += 32) p.ws_doth[dot_at + t] = p.ws_dotb[dot_at + t] = p.ws_dotv[dot_at + t] = 0.f;
#pragma unroll 1
    for (int t = valid - 1; t >= 0; --t) {
      const size_t row = (size_t)b * d.seqlen + t0 + t, at = (row * d.nheads + h) * d.headdim + pw + (lane >> 2);
      token(row);
      const uint16_t* v = static_cast<const uint16_t*>(d.v) + at;
      const float y0 = bf16_to_f32(p.dy[at]) * qn, y1 = bf16_to_f32(p.dy[at + 8]) * qn;
      const float u0 = kn * fmaf(y0, r[6], r[0]), u1 = kn * fmaf(y1, r[6], r[1]);  // the adjoint of u
      const float v0 = beta * u0, v1 = beta * u1;
      const float db = rows_sum(fmaf(u0, bf16_to_f32(p.ws_r[at]), u1 * bf16_to_f32(p.ws_r[at + 8]))) *
                       delta_beta_floor(beta);
      const float dv = rows_sum(fmaf(v0, bf16_to_f32(v[0]), v1 * bf16_to_f32(v[8])));
      if (hf == 0 && lane == 0) {
        p.ws_dotb[dot_at + t] = db;
        p.ws_dotv[dot_at + t] = dv;
      }
      if (hf == 0 && (lane & 3) == 0) {
        const uint16_t h0 = f32_to_bf16(v0), h1 = f32_to_bf16(v1);
        p.dv[at] = h0;
        p.dv[at + 8] = h1;
        if (strong) {
          p.ws_dvlo[at] = f32_to_bf16(v0 - bf16_to_f32(h0));
          p.ws_dvlo[at + 8] = f32_to_bf16(v1 - bf16_to_f32(h1));
        }
      }
      const float w0 = v0 * kn, w1 = v1 * kn;
#pragma unroll
      for (int j = 0; j < NS / 8; ++j) {
        const float k0 = bf16_lo(kv[j]), k1 = bf16_hi(kv[j]), q0 = bf16_lo(qv[j]), q1 = bf16_hi(qv[j]);
        s[j][0] = a * fmaf(-w0, k0, fmaf(y0, q0, s[j][0]));
        s[j][1] = a * fmaf(-w0, k1, fmaf(y0, q1, s[j][1]));
        s[j][2] = a * fmaf(-w1, k0, fmaf(y1, q0, s[j][2]));
        s[j][3] = a * fmaf(-w1, k1, fmaf(y1, q1, s[j][3]));
      }
    }
  }
  if (p.dh0) store_state<N, NS>(s, p.dh0 + state_at, lane);
  if (d.h0) {
    float z[NS / 8][4], dot = 0.f;
    load_state<N, NS>(z, d.h0 + state_at, lane);
#pragma unroll
    for (int j = 0; j < NS / 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) dot = fmaf(z[j][q], s[j][q], dot);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) p.ws_first[(((size_t)b * d.nheads + h) * pb + pw / 16) * 2 + hf] = dot;
  }
}

// Two warps share a block of 16 rows; up to four blocks.
template <int N>
__global__ void __launch_bounds__(kTcThreads, 1)
    delta_back_kernel(const __grid_constant__ DeltaChunkParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], freed[kMaxStages], bars[kBars];
  __shared__ float maxima[4][kRowWarps][16];
  __shared__ uint32_t slot;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int NS = N / 2, TT = 4, kTiles = 3;  // column tiles: v, dy, r
  const DeltaParams& d = p.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pb = d.headdim / 16;
  const Cta t = cta_of(p);
  const Layout l = layout(N, p.blocks, pb, kDeltaLoadBwd, 4 * kDeltaTri);
  if (threadIdx.x == 0) {
    const uint32_t warps = (uint32_t)t.active * 2;
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&freed[i], warps);
    }
    for (int i = 0; i < kBars; ++i)
      mbar_init(&bars[i], (i >= kPutS && i <= kPutP) ? warps : 1u);
    fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(&slot, kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = __shfl_sync(0xffffffffu, slot, 0);
  chain_go();
  chain_wait();

  const int blk = warp & 3, hf = (warp >> 2) & 1;
  if (warp >= kRowWarps) {
    if (warp == kRowWarps) issue_back<N>(p, t, l, smem, full, freed, bars, tm);
  } else {
    if (blk < t.active) {
      const uint32_t row = tm + ((uint32_t)(32 * blk) << 16);
      const uint32_t lc = lane_col(lane);
      const int rb = t.rb0 + blk, hx = rb / pb;
      const int h = t.kh * (d.nheads / d.nkheads) + hx, pw = (rb - hx * pb) * 16;
      const int tk = 32 * hf, tcol = 32 * hf;
      const uint32_t hcol = (uint32_t)(h - t.h0) * kC + tcol;
      const size_t part = (size_t)pw * N + hf * NS;
      const size_t state_at = ((size_t)t.b * d.nheads + h) * ((size_t)d.headdim * N) + part;
      const size_t vs = (size_t)d.nheads * d.headdim;
      const uint32_t col0 = smem_u32(smem + (size_t)p.stages * l.stage) + blk * 2 * kTiles * kCol;
      const size_t col_at0 = (size_t)t.b * d.seqlen * vs + (size_t)h * d.headdim + pw;
      float* const mx = &maxima[0][warp][0];
      const float* const ox = &maxima[0][warp ^ 4][0];
      // the state after the chunk, for its product with dS; dS on its way out
      float* const after = reinterpret_cast<float*>(smem + (size_t)p.stages * l.stage +
                                                    p.blocks * 2 * kTiles * kCol) + (blk * 2 + hf) * 16 * NS;
      const uint32_t out16 = smem_u32(smem + (size_t)p.stages * l.stage) + p.blocks * 2 * kTiles * kCol +
                             p.blocks * 2 * 16 * NS * 4 + (blk * 2 + hf) * 16 * (NS + 8) * 2;
      auto fetch = [&](int c) {
        fetch_tiles<NS>(smem_u32(after), p.ws_state + (((size_t)t.b * p.nchunks + c) * d.nheads + h) *
                                                          ((size_t)d.headdim * N) + (size_t)pw * N +
                                             hf * 16 * NS, lane);
        const int valid = (int)min((int64_t)kC, d.seqlen - (int64_t)c * kC);
        const size_t at = col_at0 + (size_t)c * kC * vs;
        const uint32_t to = col0 + (c & 1) * kTiles * kCol;
        fetch_rows<TT>(to, static_cast<const uint16_t*>(d.v) + at, vs, tk, valid, lane);
        fetch_rows<TT>(to + kCol, p.dy + at, vs, tk, valid, lane);
        fetch_rows<TT>(to + 2 * kCol, p.ws_r + at, vs, tk, valid, lane);
        cp_async_commit_group();
      };
      fetch(p.nchunks - 1);
      float S[NS / 8][4], inv0 = 1.f, inv1 = 1.f;  // the rows of dS
      load_state<N, NS>(S, p.dh_last ? p.dh_last + state_at : nullptr, lane);
      auto meet = [&](float& m0, float& m1, int use) {
        put_max(m0, m1, mx + use * kRowWarps * 16, lane);
        pair_sync(1 + blk);
        get_max(m0, m1, ox + use * kRowWarps * 16, lane);
      };
      auto put_state = [&](bool ok) {
        float m0, m1;
        row_max(S, m0, m1);
        put_max(m0, m1, mx, lane);
        ok = pair_and(1 + blk, ok);
        get_max(m0, m1, ox, lane);
        if (!ok) return false;
        const RowScale a = row_scale(exponent_of(m0)), b = row_scale(exponent_of(m1));
        inv0 = a.inv;
        inv1 = b.inv;
        constexpr int G = NS / 8 < 8 ? NS / 8 : 8;
#pragma unroll
        for (int i = 0; i < NS / 8; i += G)
          tm_pieces<true, G>(&S[i], a.s, b.s, row + kTmS + hf * (NS / 2) + 4 * i,
                             row + kTmS + N / 2 + hf * (NS / 2) + 4 * i);
        wrote(&bars[kPutS]);
        return true;
      };
      bool ok = put_state(true), strong = false;  // a strong decay in the chunk
      bool alone = false;  // a row has met a value that the pieces do not hold
      int st = 0;
      uint32_t fpar = 0;
      for (int s = 0; ok && s < p.nchunks; ++s) {
        const int c = p.nchunks - 1 - s;
        const uint32_t par = (uint32_t)(s & 1);
        const size_t bch = ((size_t)t.b * p.nchunks + c) * d.nheads + h;
        const size_t st_at = bch * ((size_t)d.headdim * N) + part;
        const size_t dot_at = (bch * pb + pw / 16) * kC + tk;
        const int64_t t0 = (int64_t)c * kC;
        const int valid = (int)min((int64_t)kC, d.seqlen - t0);
        const float* sc = reinterpret_cast<const float*>(smem + (size_t)st * l.stage + l.kq +
                                                         (h - t.h0) * l.head);
        const uint32_t vrow = col0 + (c & 1) * kTiles * kCol;

        // ---- dY for P^T
        float x[TT][4], u[TT][4], y[TT][4], m0, m1;
        ok = wait_stage(&full[st], fpar, p.wait_limit_ns);
        load_rows(y, vrow + kCol, tk, lc);
        scale_cols(y, sc + kScP * kC + tk, lane);
        row_max(y, m0, m1);
        meet(m0, m1, 1);
        RowScale r0 = row_scale(exponent_of(m0)), r1 = row_scale(exponent_of(m1));
        tm_pieces<true, TT>(y, r0.s, r1.s, row + kTmO + tcol / 2, row + kTmO + 32 + tcol / 2);
        wrote(&bars[kPutP]);
        const float top0 = m0, top1 = m1;
        const bool whole = sc[kScEnd * kC + 5] == 0.f;  // r has a rest in every row
        strong = sc[kScEnd * kC + 3] + sc[kScEnd * kC + 4] != 0.f;
        if (strong && whole) {
          fetch_rows<TT>(out16 - tk * 32, p.ws_rlo + col_at0 + t0 * vs, vs, tk, valid, lane);
          cp_async_commit_group();
        }

        // ---- dU = P^T dY + e^(G_end - G) K dS^T
        ok = wait_warp(&bars[kBarK], par, ok ? p.wait_limit_ns : 0) && ok;
        tm_load(row + kTmX + tcol, x);
        scale_rows(x, inv0, inv1);
        scale_cols(x, sc + kScKend * kC + tk, lane);
        const bool maybe = maybe_wide(y, top0, top1);
        if (strong) {
#pragma unroll
          for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) y[j][q] = x[j][q];
        }
        ok = wait_warp(&bars[kBarQ], par, ok ? p.wait_limit_ns : 0) && ok;
        tm_load(row + kTmU + hcol, u);
        scale_rows(u, r0.inv, r1.inv);
        scale_cols(u, sc + kScK * kC + tk, lane);
        add_tiles(u, x);
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) x[j][q] = u[j][q];
        scale_cols(x, sc + kScU * kC + tk, lane);
        row_max(x, m0, m1);
        meet(m0, m1, 2);
        alone |= not_finite(m0) || not_finite(m1);
        r0 = row_scale(exponent_of(m0));
        r1 = row_scale(exponent_of(m1));
        tm_pieces<true, TT>(x, r0.s, r1.s, row + kTmX + tcol / 2, row + kTmX + 32 + tcol / 2);
        wrote(&bars[kPutU]);

        // ---- meanwhile: the next chunk's rows, dS for the gradients, <S, dS>
        const float dot = tiles_dot<NS>(S, after, lane);
        if (lane == 0) p.ws_end[(bch * pb + pw / 16) * 2 + hf] = dot;
        if (strong) {  // r . e^(G_end - G) dS k
          cp_async_wait_group<0>();
          __syncwarp();
          load_rows(x, vrow + 2 * kCol, tk, lc);
          if (whole) {
            load_rows(u, out16 - tk * 32, tk, lc);
            add_tiles(x, u);
          }
          row_dots(x, y, p.ws_doth + dot_at, lane);
        }
        __syncwarp();
        if (c > 0) fetch(c - 1);
        store_state16<N, NS>(S, out16, p.ws_dstate16 + st_at, lane);
        bool wide = false;
        if (__any_sync(0xffffffffu, maybe)) {
          load_rows(y, vrow + kCol, tk, lc);
          scale_cols(y, sc + kScP * kC + tk, lane);
          wide = wide_rows(true, y, y, top0, top1, 0.f, 0.f);
        }
        load_rows(y, vrow + kCol, tk, lc);
        scale_cols(y, sc + kScSq * kC + tk, lane);

        // ---- dV = dR = T^T (beta dU); dY and -dR under one scale for the sum of dS
        ok = wait_warp(&bars[kBarT], par, ok ? p.wait_limit_ns : 0) && ok;
        tm_load(row + kTmY + hcol, x);
        scale_rows(x, r0.inv, r1.inv);
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) u[j][q] = -x[j][q];
        scale_cols(u, sc + kScSk * kC + tk, lane);
        float n0, n1;
        row_max(y, n0, n1);
        row_max(u, m0, m1);
        m0 = wide ? __uint_as_float(0x7FFFFFFFu) : max_nan(m0, n0);
        m1 = wide ? m0 : max_nan(m1, n1);
        meet(m0, m1, 3);
        alone |= not_finite(m0) || not_finite(m1);
        r0 = row_scale(exponent_of(m0));
        r1 = row_scale(exponent_of(m1));
        tm_pieces<true, TT>(y, r0.s, r1.s, row + kTmO + tcol / 2, row + kTmO + 32 + tcol / 2);
        tm_pieces<true, TT>(u, r0.s, r1.s, row + kTmX + tcol / 2, row + kTmX + 32 + tcol / 2);
        wrote(&bars[kPutR]);
        load_rows(u, vrow + 2 * kCol, tk, lc);
        row_dots(x, u, p.ws_dotb + dot_at, lane);
        scale_cols(x, sc + kScRatio * kC + tk, lane);
        load_rows(u, vrow, tk, lc);
        row_dots(x, u, p.ws_dotv + dot_at, lane);
        __syncwarp();
        stage_rows(x, vrow, tk, lc);
        store_rows<TT>(vrow, tk, p.dv + col_at0 + t0 * vs, vs, valid, lane);
        if (strong) {
          rest_of(x);
          __syncwarp();
          stage_rows(x, vrow, tk, lc);
          store_rows<TT>(vrow, tk, p.ws_dvlo + col_at0 + t0 * vs, vs, valid, lane);
        }
        // ---- dS <- e^G_end dS + dY^T (e^G Q) - dR^T (e^G K), and its pieces for the next chunk
        const float end = sc[kScEnd * kC];
        ok = wait_warp(&bars[kBarU], par, ok ? p.wait_limit_ns : 0) && ok;
        constexpr int G = NS / 8 < 8 ? NS / 8 : 8;
#pragma unroll
        for (int i = 0; i < NS / 8; i += G) {
          float ds[G][4];
          tm_load(row + kTmU + hf * NS + 8 * i, ds);
#pragma unroll
          for (int j = 0; j < G; ++j) {
            float(&q)[4] = S[i + j];
            const float2 a = fma2(make_float2(q[0], q[1]), make_float2(end, end),
                                  mul2(make_float2(ds[j][0], ds[j][1]), make_float2(r0.inv, r0.inv)));
            const float2 b = fma2(make_float2(q[2], q[3]), make_float2(end, end),
                                  mul2(make_float2(ds[j][2], ds[j][3]), make_float2(r1.inv, r1.inv)));
            q[0] = a.x; q[1] = a.y; q[2] = b.x; q[3] = b.y;
          }
        }
        if (c > 0) ok = put_state(ok);
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&freed[st]);
        if (++st == p.stages) {
          st = 0;
          fpar ^= 1u;
        }
      }
      ok = pair_and(1 + blk, ok);  // the pair stays together
      if (!ok) {
        if (lane == 0) atomicExch(&g_delta_timeout, 1);
      } else if (__any_sync(0xffffffffu, alone)) {
        walk_back_tokens<N>(p, t.b, h, pw, 1 + blk, mx, ox);
        strong = false;
      } else if (p.dh0) {
        store_state<N, NS>(S, p.dh0 + state_at, lane);
      }
      if (ok && d.h0 && strong) {  // <S, dS> before the first token
        float s[NS / 8][4], dot = 0.f;
        load_state<N, NS>(s, d.h0 + state_at, lane);
#pragma unroll
        for (int j = 0; j < NS / 8; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) dot = fmaf(s[j][q], S[j][q], dot);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) p.ws_first[(((size_t)t.b * d.nheads + h) * pb + pw / 16) * 2 + hf] = dot;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tm, kTmemCols);
}

// The largest number of row blocks per CTA (one CTA fills an SM) of at most two
// heads and two stages, halved while the grid then still is no larger than the
// SMs: the chain is shorter with fewer warps per scheduler. Whole calls with 1, 2,
// 4 and 8 blocks: 8192 tokens of 32 heads of 128 (256, 128, 64, 32 CTAs) 688, 388,
// 395, 534 us; 4 x 4096 of 64 heads of 64 (1024 .. 128 CTAs) 1295, 845, 548, 489.
// `one`: the kernel of one warp per block, taken above four blocks; null where
// there is none.
// block_bytes: shared memory per row block beside its column tiles.
template <int N, typename K>
cudaError_t run(K* one, K* two, DeltaChunkParams p, int tiles, int head_bytes, int block_bytes,
                cudaStream_t stream) {
  const int per_head = p.d.headdim / 16, group = p.d.nheads / p.d.nkheads * per_head;
  const int64_t groups = (int64_t)p.d.batch * p.d.nkheads;
  auto lay = [&](int blocks) { return layout(N, blocks, per_head, head_bytes, 0); };
  auto extra = [&](int blocks) { return blocks * (2 * tiles * kCol + block_bytes) + 1024; };
  auto stages_of = [&](int blocks) {
    return std::min(kMaxStages, (kMaxShared - extra(blocks)) / lay(blocks).stage);
  };
  auto ctas = [&](int blocks) { return groups * ((group + blocks - 1) / blocks); };
  int blocks = one ? kMaxBlocks : 4;
  while (blocks > 1 && (blocks / 2 >= group || lay(blocks).heads > kTcHeads || stages_of(blocks) < 2 ||
                        ctas(blocks / 2) <= 148))
    blocks /= 2;
  p.blocks = blocks;
  p.stages = stages_of(blocks);
  if (p.stages < 2) return cudaErrorInvalidValue;
  const int bytes = lay(blocks).stage * p.stages + extra(blocks);
  K* kern = blocks <= 4 ? two : one;
  const cudaError_t e = allow_shared<K>(kern);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3((unsigned)ctas(blocks)), kTcThreads, bytes, stream, p);
}
template <int N, bool BWD>
cudaError_t fwd(const DeltaChunkParams& p, cudaStream_t stream) {
  constexpr int state16 = 2 * 16 * (N / 2 + 8) * 2;
  if constexpr (BWD)
    return run<N, void(DeltaChunkParams)>(nullptr, delta_tc_kernel<N, 2, true>, p, 2, kDeltaLoadBwd,
                                          state16, stream);
  else
    return run<N>(delta_tc_kernel<N, 1, false>, delta_tc_kernel<N, 2, false>, p, 1, kDeltaHeadFwd, 0,
                  stream);
}
template <int N>
cudaError_t rev(const DeltaChunkParams& p, cudaStream_t stream) {
  return run<N, void(DeltaChunkParams)>(nullptr, delta_back_kernel<N>, p, 3, kDeltaLoadBwd,
                                        2 * 16 * ((N / 2) * 4 + (N / 2 + 8) * 2), stream);
}

}  // namespace

bool delta_chunk_supported(int dstate, int headdim) {
  return (dstate == 64 || dstate == 128) && headdim % 16 == 0 && headdim >= 16;
}

cudaError_t launch_delta_fwd(const DeltaChunkParams& p, bool bwd, cudaStream_t stream) {
  if (bwd) return p.d.dstate == 64 ? fwd<64, true>(p, stream) : fwd<128, true>(p, stream);
  return p.d.dstate == 64 ? fwd<64, false>(p, stream) : fwd<128, false>(p, stream);
}

cudaError_t launch_delta_rev(const DeltaChunkParams& p, cudaStream_t stream) {
  return p.d.dstate == 64 ? rev<64>(p, stream) : rev<128>(p, stream);
}

cudaError_t delta_chunk_status(cudaStream_t stream, int* timed_out) {
  return timeout_status(stream, timed_out);
}

}  // namespace ssm
