// ssm_delta_grad.cu -- gradients of the gated delta rule that need no further
// walk over the sequence (bf16 io, sm_100a): dq, dk, dbeta, ddt, dA, ddt_bias
// from each chunk's entering state S, the adjoint dS of its leaving state, and
// the residuals r, dR = dv of the two passes over the chunks.
//
// With W_ij = (dy_i . u_j) e^(G_i - G_j) (j <= i) and
// N_ij = -(dv_i . u_j) e^(G_i - G_j) (j < i):
//   dq_i = e^(G_i) S dy_i + sum_j W_ij k_j
//   dk_j = e^(G_end - G_j) dS u_j - e^(G_j) S dv_j + sum_i W_ij q_i + sum_i (N + N^T)_ji k_i
//   dbeta_j = dv_j . r_j / beta_j  (beta_j at least 2^-26)
// (dv_j is beta_j times the adjoint of u_j, all its later uses included, so nothing
// is left to subtract) and, since a decay scales every later use of the state, the log decays'
// gradients need no matrix at all:
//   dg_t = sum_(i >= t in the chunk) (dy_i . y_i - dv_i . v_i) + <S_end, dS_end>
// whose row products the two passes took in fp32. After a strong decay (kStrongDecay)
// that sum is all cancellation, so there dg_t is taken from what passes over it,
//   dg_t = sum_(j < t <= i) e^(G_i - G_j) [(dy_i . u_j)(q_i . k_j) - (dv_i . u_j)(k_i . k_j)]
//        + sum_(i >= t) e^(G_i) [dy_i . S q_i - dv_i . S k_i]
//        + sum_(j < t) e^(G_end - G_j) u_j . dS k_j + e^(G_end) <S, dS>,
// every term with its decay, added up without a difference: row sums of a block's
// pairs for the tokens of its rows, column sums for those of its columns. r and dv
// then come as two bf16 pieces (2^-16); S and dS stay one, for they matter only to the
// chunk's first and last tokens: the first one's dg is <S_end, dS_end> of the chunk
// before, and the walk back takes the parts with dS in fp32. The same serves tokens
// whose suffix sum is lost in the products of far larger tokens behind them. One CTA per chunk and key
// head adds its value heads in order, so dq and dk are written once, through
// x / |x| when q and k were scaled to unit length. Operands are bf16 (q, k, dy
// exactly; S, dS, r, dv and the weights rounded once), sums fp32: the outputs
// are bf16 themselves (dq, dk: 3.0e-3 from the exact ones in the 2-norm, dbeta,
// whose r is rounded once, 2.3e-3; 1.7e-3 of it the last rounding). <S_end, dS_end> comes from the reverse pass, in fp32.
//
// One CTA of sixteen warps fills an SM's shared memory: a warp takes 16 tokens
// by a quarter of the columns; the head's tiles come by asynchronous copies,
// the states' while the weights are computed, the next head's while the last
// products run. Two warps without weights take the gates meanwhile.
//
// 2 x 2048 tokens, 32 heads of 128 on 16 key heads, dstate 128: 132 us for
// 25.8 GFLOP and 300 MB, and about 11 us for a round of heads with strong decays.
// Bound: the phases of a head (copies, weights, products with the states,
// products with the weights) follow one another with all warps: tensor pipe 32 %
// busy, DRAM 34 %. It was 176 us with the gates after the products, 148 with dy
// and dv meeting S one after the other and the weights stored element by element,
// 137 with k k^T and its column sums for dbeta.
#include "ssm_delta.cuh"

namespace ssm {

namespace {

constexpr int kC = kDeltaChunk;
constexpr int kThreads = 512;
constexpr int kGateWarp = 12;     // and the next: row blocks 0 and 1, columns behind them
constexpr int kWs = kC * 2 + 16;  // row stride (bytes) of the 64 x 64 tiles

struct GradLayout {
  int xs, ps;  // row strides (bytes) of the dstate-wide and headdim-wide tiles
  int k, q, s, ds, dy, r, dr, w1, w2, ns, dots, f, bytes;  // over w1 .. dots: the rests of r and dv
};
enum {
  kfGhi, kfGlo, kfBeta, kfKn, kfQn, kfLk, kfLq, kfRow,
  // of strong_gates: the tokens' parts with the entering state and with dS (a quarter of
  // dstate each), row sums by column block, column sums by row block,
  // the pairs inside a token's own block; the warps' parts of <S, dS>
  kfIn, kfOut = kfIn + 4, kfRows = kfOut + 4, kfCols = kfRows + 3, kfOwn = kfCols + 4, kfSum, kfCount
};

__host__ __device__ inline GradLayout grad_layout(int N, int P) {
  GradLayout g;
  g.xs = N * 2 + 16;
  g.ps = P * 2 + 16;
  int at = 0;
  g.k = at; at += kC * g.xs;
  g.q = at; at += kC * g.xs;
  g.s = at; at += P * g.xs;
  g.ds = at; at += P * g.xs;
  g.dy = at; at += kC * g.ps;
  g.r = at; at += kC * g.ps;
  g.dr = at; at += kC * g.ps;
  g.w1 = at; at += kC * kWs;
  g.w2 = at; at += kC * kWs;
  g.ns = at; at += kC * kWs;
  g.dots = at; at += 3 * (P / 16) * kC * 4;
  at = at - g.w1 < 2 * kC * g.ps ? g.w1 + 2 * kC * g.ps : at;
  g.f = at; at += kfCount * kC * 4;
  g.bytes = at;
  return g;
}

// 16-byte asynchronous copy, zeros where `in` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
// <t, x> over a warp's quarter of dstate, rows r0 and r0 + 8 of a k or q tile (all lanes of a quad)
template <int T>
__device__ __forceinline__ void rows_dot(const float (&t)[T][4], const unsigned char* x, int xs, int r0,
                                         int part, int lane, float& d0, float& d1) {
  d0 = d1 = 0.f;
#pragma unroll
  for (int j = 0; j < T; ++j) {
    const int at = (part * T + j) * 16 + (lane & 3) * 4;
    const uint32_t x0 = *reinterpret_cast<const uint32_t*>(x + r0 * xs + at);
    const uint32_t x1 = *reinterpret_cast<const uint32_t*>(x + (r0 + 8) * xs + at);
    d0 = fmaf(bf16_lo(x0), t[j][0], fmaf(bf16_hi(x0), t[j][1], d0));
    d1 = fmaf(bf16_lo(x1), t[j][2], fmaf(bf16_hi(x1), t[j][3], d1));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    d0 += __shfl_xor_sync(0xffffffffu, d0, o);
    d1 += __shfl_xor_sync(0xffffffffu, d1, o);
  }
}

// The 64 gate threads: dg of the thread's token as a suffix sum over the chunk. so, sv:
// the token's dy.y and dv.v; end, prev: a lane's part of <S, dS> after and before the
// chunk, which is the first token's dg (`first`: there is no prev). lost: the sum is small
// beside its terms, and they are 2^11 times those of the tokens before this one, whose
// size dg is of (a value far above theirs stands at this one or behind it). terms: the
// sum of their magnitudes.
__device__ __forceinline__ float suffix_sum(float so, float sv, float end, float prev, bool first, double* R,
                                            int gt, float& terms, bool& lost) {
  const int lane = gt & 31;
  float* const f = reinterpret_cast<float*>(R + 1);
  float before = terms = fabsf(so) + fabsf(sv);
  // in 64 bits: the terms cancel
  double sum = (double)so - (double)sv, all = end;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_down_sync(0xffffffffu, sum, o);
    const float t = __shfl_down_sync(0xffffffffu, terms, o), b = __shfl_up_sync(0xffffffffu, before, o);
    if (lane + o < 32) {
      sum += up;
      terms += t;
    }
    if (lane >= o) before = fmaxf(before, b);
    all += __shfl_xor_sync(0xffffffffu, all, o);
    prev += __shfl_xor_sync(0xffffffffu, prev, o);
  }
  if (gt == 32) {
    R[0] = sum;
    f[0] = terms;
  }
  if (gt == 31) f[1] = before;
  before = __shfl_up_sync(0xffffffffu, before, 1);
  asm volatile("bar.sync 1, 64;" ::: "memory");
  if (gt < 32) {
    sum += R[0];
    terms += f[0];
  } else {
    before = lane ? fmaxf(before, f[1]) : f[1];
  }
  float dg = (float)(sum + all);
  // (so written that NaN counts)
  lost = gt > 0 ? !(terms <= before * 0x1p11f) && !(fabsf(dg) >= terms * 0x1p-11f)
                : first && !(fabsf(dg) >= terms * 0x1p-11f);
  if (gt == 0 && !first) dg = prev;
  return dg;
}

// The 64 gate threads: ddt of the thread's token from dg, and the chunk's parts of dA
// and ddt_bias. `first`: the sequence's first token; `in`: a token of the sequence;
// raw, A: its step before softplus, its head's A.
__device__ __forceinline__ void write_gates(const DeltaChunkParams& p, double* R, float dg, int gt,
                                            size_t gate_at, size_t bch, bool first, bool in, float raw,
                                            float A) {
  const DeltaParams& d = p.d;
  // the first token's decay has nothing to act on without an initial state
  if (!d.h0 && first) dg = 0.f;
  double dA = 0.0, dbias = 0.0;
  if (in) {
    const float step = delta_step_size(raw, d.softplus);
    const float sig = (d.softplus && raw <= kSoftplusCut) ? 1.f / (1.f + expf(-raw)) : 1.f;
    const float ddt = dg * A * sig;
    if (step * A < kStrongDecay) R[6] = 1.0;  // the chunk has work for strong_gates
    dA = (double)dg * step;
    dbias = ddt;
    p.ddt[gate_at] = f32_to_bf16(ddt);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    dA += __shfl_xor_sync(0xffffffffu, dA, o);
    dbias += __shfl_xor_sync(0xffffffffu, dbias, o);
  }
  if ((gt & 31) == 0) {
    R[2 + 2 * (gt >> 5)] = dA;
    R[2 + 2 * (gt >> 5) + 1] = dbias;
  }
  asm volatile("bar.sync 1, 64;" ::: "memory");
  if (gt < 2) p.ws_part[bch * 2 + gt] = R[2 + gt] + R[4 + gt];
}

// Whether a head has a strong decay in the chunk.
__device__ __forceinline__ bool strong_head(const DeltaChunkParams& p, size_t bch) {
  const float* sc = reinterpret_cast<const float*>(p.ws_head + bch * (size_t)p.head_bytes + 4 * kDeltaTri);
  return sc[kScEnd * kC + 3] + sc[kScEnd * kC + 4] != 0.f;
}

// The gates of such a head, or of one with lost suffix sums, over what write_gates left:
// dg of the tokens behind a strong decay, or lost, from the pairs on either side. (Without
// a strong decay r and dv are one bf16 piece: 3e-3 of the pairs' sum.) All threads of the
// CTA, k and q in place; its own function at the kernel's end, so that neither its registers nor its
// instructions meet the others' products (inside the loop over the heads: 138 us in
// place of 131 for the kernel where no decay is strong).
template <int N>
__device__ __noinline__ void strong_gates(const DeltaChunkParams& p, unsigned char* smem, int h) {
  constexpr int LPR = N / 8;
  const DeltaParams& d = p.d;
  const int P = d.headdim, sl = P / 16;
  const GradLayout g = grad_layout(N, P);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int mi = warp & 3, part = warp >> 2;
  const int c = blockIdx.x, b = blockIdx.z;
  const int64_t t0 = (int64_t)c * kC;
  const int valid = (int)min((int64_t)kC, d.seqlen - t0);
  const size_t bch = ((size_t)b * p.nchunks + c) * d.nheads + h, row0 = (size_t)b * d.seqlen + t0;
  float* F = reinterpret_cast<float*>(smem + g.f);
  const uint32_t sm = smem_u32(smem);
  const int a_row = lane & 15, a_u = lane >> 4;
  const int nt_row = (lane & 7) + ((lane & 16) >> 1), nt_u = (lane >> 3) & 1;
  const int r0 = mi * 16 + (lane >> 2), r1 = r0 + 8;
  const int gt = tid - kGateWarp * 32;
  const bool gate = gt >= 0 && gt < kC;
  const size_t gate_at = (row0 + gt) * d.nheads + h;
  float* const red = F + kfSum * kC;
  const float* sc = reinterpret_cast<const float*>(p.ws_head + bch * (size_t)p.head_bytes + 4 * kDeltaTri);
  const bool strong = strong_head(p, bch), whole = strong && sc[kScEnd * kC + 5] == 0.f;  // r, dv in two pieces
  if (tid < 5 * kC) {
    const int w = tid / kC, i = tid % kC;
    const int from = w == 0 ? kScGhi : (w == 1 ? kScGlo : (w == 2 ? kScBeta : (w == 3 ? kScKn : kScQn)));
    F[w * kC + i] = sc[from * kC + i];
  }
  for (int i = tid; i < kC * (P / 8); i += kThreads) {
    const int row = i / (P / 8), u = i % (P / 8);
    const size_t from = ((row0 + (row < valid ? row : 0)) * d.nheads + h) * P + u * 8;
    const uint32_t to = sm + row * g.ps + u * 16;
    copy16(to + g.dy, p.dy + from, row < valid);
    copy16(to + g.r, p.ws_r + from, row < valid);
    copy16(to + g.dr, p.dv + from, row < valid);
    copy16(to + g.w1, p.ws_rlo + from, row < valid && whole);
    copy16(to + g.w1 + kC * g.ps, p.ws_dvlo + from, row < valid && whole);
  }
  for (int j = tid; j < P * LPR; j += kThreads) {
    const uint32_t to = sm + (j / LPR) * g.xs + (j % LPR) * 16;
    copy16(to + g.s, p.ws_state16 + bch * ((size_t)P * N) + (size_t)j * 8, true);
    copy16(to + g.ds, p.ws_dstate16 + bch * ((size_t)P * N) + (size_t)j * 8, true);
  }
  cp_async_commit_group();
  // a gate thread's operands meanwhile: its token's row products, <S_end, dS_end> and
  // <S, dS> before the chunk, which is the first token's dg
  float so = 0.f, sv = 0.f, out = 0.f, end = 0.f, before = 0.f, raw = 0.f, A = 0.f;
  if (gate) {
    A = d.A[h];
    if (gt < valid)
      raw = bf16_to_f32(static_cast<const uint16_t*>(d.dt)[gate_at]) + (d.dt_bias ? d.dt_bias[h] : 0.f);
    for (int i = 0; i < sl; ++i) {
      const size_t at = (bch * sl + i) * kC + gt;
      so += p.ws_doto[at];
      sv += p.ws_dotv[at];
      if (strong) out += p.ws_doth[at];
    }
    const float* prev = c > 0 ? p.ws_end + (bch - d.nheads) * 2 * sl
                              : p.ws_first + ((size_t)b * d.nheads + h) * 2 * sl;
    if (lane < 2 * sl) {
      end = p.ws_end[bch * 2 * sl + lane];
      if (c > 0 || (d.h0 && strong)) before = prev[lane];
    }
  }
  cp_async_wait_group<0>();
  __syncthreads();
  {  // e^G (dy . S q - dv . S k), a quarter of dstate
    constexpr int T = N / 32;
    const int tr_row = (lane & 7) + (lane & 8), tr_u = lane >> 4;
    float t[T][4] = {}, x[T][4] = {};
    for (int kt = 0; kt < P / 16; ++kt) {
      uint32_t a[4], e[4];
      ldsm4(a, sm + g.dy + (mi * 16 + a_row) * g.ps + (2 * kt + a_u) * 16);
      ldsm4(e, sm + g.dr + (mi * 16 + a_row) * g.ps + (2 * kt + a_u) * 16);
#pragma unroll
      for (int j = 0; j < T / 2; ++j) {
        uint32_t bb[4];
        ldsm4t(bb, sm + g.s + (16 * kt + tr_row) * g.xs + (part * T + 2 * j + tr_u) * 16);
        mma_bf16(t[2 * j], a, bb[0], bb[1]);
        mma_bf16(t[2 * j + 1], a, bb[2], bb[3]);
        mma_bf16(x[2 * j], e, bb[0], bb[1]);
        mma_bf16(x[2 * j + 1], e, bb[2], bb[3]);
      }
    }
    float i0, i1, v0, v1;
    rows_dot<T>(t, smem + g.q, g.xs, r0, part, lane, i0, i1);
    rows_dot<T>(x, smem + g.k, g.xs, r0, part, lane, v0, v1);
    if ((lane & 3) == 0) {
      F[(kfIn + part) * kC + r0] = ex2_approx(F[kfGhi * kC + r0] + F[kfGlo * kC + r0]) *
                                   (F[kfQn * kC + r0] * i0 - F[kfKn * kC + r0] * v0);
      F[(kfIn + part) * kC + r1] = ex2_approx(F[kfGhi * kC + r1] + F[kfGlo * kC + r1]) *
                                   (F[kfQn * kC + r1] * i1 - F[kfKn * kC + r1] * v1);
    }
  }
  if (!strong) {  // e^(G_end - G) u . dS k, a quarter of dstate (else the walk back took it)
    constexpr int T = N / 32;
    const int tr_row = (lane & 7) + (lane & 8), tr_u = lane >> 4;
    float t[T][4] = {};
    for (int kt = 0; kt < P / 16; ++kt) {
      uint32_t a[4];
      ldsm4(a, sm + g.r + (mi * 16 + a_row) * g.ps + (2 * kt + a_u) * 16);
#pragma unroll
      for (int j = 0; j < T / 2; ++j) {
        uint32_t bb[4];
        ldsm4t(bb, sm + g.ds + (16 * kt + tr_row) * g.xs + (part * T + 2 * j + tr_u) * 16);
        mma_bf16(t[2 * j], a, bb[0], bb[1]);
        mma_bf16(t[2 * j + 1], a, bb[2], bb[3]);
      }
    }
    float o0, o1;
    rows_dot<T>(t, smem + g.k, g.xs, r0, part, lane, o0, o1);
    if ((lane & 3) == 0) {
      const float gh = F[kfGhi * kC + kC - 1], gl = F[kfGlo * kC + kC - 1];
      F[(kfOut + part) * kC + r0] = ex2_approx((gh - F[kfGhi * kC + r0]) + (gl - F[kfGlo * kC + r0])) *
                                    F[kfBeta * kC + r0] * F[kfKn * kC + r0] * o0;
      F[(kfOut + part) * kC + r1] = ex2_approx((gh - F[kfGhi * kC + r1]) + (gl - F[kfGlo * kC + r1])) *
                                    F[kfBeta * kC + r1] * F[kfKn * kC + r1] * o1;
    }
  }
  {  // <S, dS>
    float s = 0.f;
    for (int j = tid; j < P * LPR; j += kThreads) {
      const int at = (j / LPR) * g.xs + (j % LPR) * 16;
      const uint4 a = *reinterpret_cast<const uint4*>(smem + g.s + at);
      const uint4 b = *reinterpret_cast<const uint4*>(smem + g.ds + at);
      const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s = fmaf(bf16_lo(x[i]), bf16_lo(y[i]), fmaf(bf16_hi(x[i]), bf16_hi(y[i]), s));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) red[warp] = s;
  }
  if (part <= mi) {
    float wv[2][4] = {}, xv[2][4] = {}, qk[2][4] = {}, kk[2][4] = {};
    const uint32_t a_at = (mi * 16 + a_row) * g.ps + a_u * 16, b_at = (16 * part + nt_row) * g.ps + nt_u * 16;
    for (int kt = 0; kt < P / 16; ++kt) {
      uint32_t a[4], e[4], el[4], b[4], bl[4];
      ldsm4(a, sm + g.dy + a_at + kt * 32);
      ldsm4(e, sm + g.dr + a_at + kt * 32);
      ldsm4(el, sm + g.w1 + kC * g.ps + a_at + kt * 32);
      ldsm4(b, sm + g.r + b_at + kt * 32);
      ldsm4(bl, sm + g.w1 + b_at + kt * 32);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        mma_bf16(wv[y], a, bl[2 * y], bl[2 * y + 1]);
        mma_bf16(wv[y], a, b[2 * y], b[2 * y + 1]);
        mma_bf16(xv[y], el, b[2 * y], b[2 * y + 1]);
        mma_bf16(xv[y], e, bl[2 * y], bl[2 * y + 1]);
        mma_bf16(xv[y], e, b[2 * y], b[2 * y + 1]);
      }
    }
#pragma unroll
    for (int kt = 0; kt < N / 16; ++kt) {
      uint32_t a[4], e[4], b[4];
      ldsm4(a, sm + g.q + (mi * 16 + a_row) * g.xs + (2 * kt + a_u) * 16);
      ldsm4(e, sm + g.k + (mi * 16 + a_row) * g.xs + (2 * kt + a_u) * 16);
      ldsm4(b, sm + g.k + (16 * part + nt_row) * g.xs + (2 * kt + nt_u) * 16);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        mma_bf16(qk[y], a, b[2 * y], b[2 * y + 1]);
        mma_bf16(kk[y], e, b[2 * y], b[2 * y + 1]);
      }
    }
    const int l4 = lane & 3;
    float f[2][2][2];  // [column half y][row r0, r1][column]
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = x ? r1 : r0, j = 16 * part + 8 * y + 2 * l4 + q;
          const float gm = ex2_approx((F[kfGhi * kC + i] - F[kfGhi * kC + j]) +
                                      (F[kfGlo * kC + i] - F[kfGlo * kC + j]));
          const float w = F[kfQn * kC + i] * qk[y][2 * x + q] * wv[y][2 * x + q] -
                          F[kfKn * kC + i] * kk[y][2 * x + q] * xv[y][2 * x + q];
          f[y][x][q] = j < i ? gm * F[kfBeta * kC + j] * F[kfKn * kC + j] * w : 0.f;
        }
    if (part < mi) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float s = (f[0][x][0] + f[0][x][1]) + (f[1][x][0] + f[1][x][1]);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (l4 == 0) F[(kfRows + part) * kC + (x ? r1 : r0)] = s;
      }
    }
    // the block's own tokens: what a row has before each column
    float c[2][2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float before = 0.f;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float s = f[y][x][0] + f[y][x][1];
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          const float up = __shfl_up_sync(0xffffffffu, s, o, 4);
          if (l4 >= o) s += up;
        }
        const float up = __shfl_up_sync(0xffffffffu, s, 1, 4);
        c[y][x][0] = l4 ? before + up : before;
        c[y][x][1] = c[y][x][0] + f[y][x][0];
        before += __shfl_sync(0xffffffffu, s, 3, 4);
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int j = 16 * part + 8 * y + 2 * l4 + q;
        float s = part < mi ? f[y][0][q] + f[y][1][q]
                            : (r0 >= j ? c[y][0][q] : 0.f) + (r1 >= j ? c[y][1][q] : 0.f);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane < 4) F[(part < mi ? kfCols + mi : kfOwn) * kC + j] = s;
      }
  }
  __syncthreads();
  if (gate) {
    // sums over rows from the token on and over columns before it, in its block of 16
    // and, of the parts with the states, in the chunk; totals of whole blocks
    const int K = gt >> 4, l16 = gt & 15;
    float* const tot = red + kThreads / 32;  // [2 K + J]: rows of block K by column block J; in, out, sizes
    float rs = 0.f, cs = 0.f, in = 0.f;
#pragma unroll
    for (int J = 0; J < 3; ++J) {
      float r = J < K ? F[(kfRows + J) * kC + gt] : 0.f;
      rs += r;
      if (J < 2) {
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
        if (l16 == 0) tot[2 * K + J] = r;
      }
    }
#pragma unroll
    for (int I = 1; I < 4; ++I) cs += I > K ? F[(kfCols + I) * kC + gt] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) in += F[(kfIn + i) * kC + gt];
    out *= F[kfBeta * kC + gt];
    if (!strong) {
#pragma unroll
      for (int i = 0; i < 4; ++i) out += F[(kfOut + i) * kC + gt];
    }
    float size_in = fabsf(in), size_out = fabsf(out);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float up = __shfl_up_sync(0xffffffffu, out, o), down = __shfl_down_sync(0xffffffffu, in, o);
      const float up2 = __shfl_up_sync(0xffffffffu, size_out, o);
      const float down2 = __shfl_down_sync(0xffffffffu, size_in, o);
      if (lane >= o) {
        out += up;
        size_out += up2;
      }
      if (lane + o < 32) {
        in += down;
        size_in += down2;
      }
      if (o < 16) {
        const float u = __shfl_up_sync(0xffffffffu, cs, o, 16), w = __shfl_down_sync(0xffffffffu, rs, o, 16);
        if (l16 >= o) cs += u;
        if (l16 + o < 16) rs += w;
      }
    }
    if (gt == 31) {
      tot[9] = out;
      tot[11] = size_out;
    }
    if (gt == 32) {
      tot[8] = in;
      tot[10] = size_in;
    }
    out = __shfl_up_sync(0xffffffffu, out, 1);  // the tokens before this one
    size_out = __shfl_up_sync(0xffffffffu, size_out, 1);
    cs = __shfl_up_sync(0xffffffffu, cs, 1);
    if (lane == 0) out = size_out = 0.f;
    if (l16 == 0) cs = 0.f;
    double* R = reinterpret_cast<double*>(F + kfRow * kC);
    float terms;
    bool lost;
    float dg = suffix_sum(so, sv, end, before, c == 0 && !strong, R, gt, terms, lost);
    const bool behind = delta_step_size(raw, d.softplus) * A < kStrongDecay;
    if (gt < valid && (lost || behind)) {
      float s = (F[kfOwn * kC + gt] + rs) + (cs + (in + out));
      float size = fabsf(F[kfOwn * kC + gt]) + fabsf(rs) + fabsf(cs) + size_in + size_out;
      if (K == 1) s += tot[4] + tot[6];  // rows of blocks behind, columns of blocks before
      if (K == 2) s += tot[6] + tot[7];
      s += K < 2 ? tot[8] : tot[9];
      size += K < 2 ? tot[10] : tot[11];
      float ss = 0.f;
      for (int i = 0; i < kThreads / 32; ++i) ss += red[i];
      ss *= sc[kScEnd * kC];
      // a lost sum only where the pairs are better: 2^-9 of their terms, it 2^-20 of its
      if (!behind && size + fabsf(ss) >= terms * 0x1p-11f) lost = false;
      if ((lost || behind) && (gt > 0 || (c == 0 && !strong))) dg = s + ss;
    }
    write_gates(p, R, dg, gt, gate_at, bch, t0 + gt == 0, gt < valid, raw, A);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) delta_grad_kernel(const __grid_constant__ DeltaChunkParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int T = N / 32;  // n-tiles of a warp's quarter of dstate
  const DeltaParams& d = p.d;
  const int P = d.headdim;
  const GradLayout g = grad_layout(N, P);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int mi = warp & 3, part = warp >> 2;
  const int c = blockIdx.x, kh = blockIdx.y, b = blockIdx.z;
  const int rep = d.nheads / d.nkheads;
  const int64_t t0 = (int64_t)c * kC;
  const int valid = (int)min((int64_t)kC, d.seqlen - t0);
  const size_t bc = (size_t)b * p.nchunks + c;
  const size_t row0 = (size_t)b * d.seqlen + t0;
  float* F = reinterpret_cast<float*>(smem + g.f);
  const uint32_t sm = smem_u32(smem);
  // fragment addressing: A rows (m) with k contiguous; B rows n (nt); rows k (tr)
  const int a_row = lane & 15, a_u = lane >> 4;
  const int nt_row = (lane & 7) + ((lane & 16) >> 1), nt_u = (lane >> 3) & 1;
  const int tr_row = (lane & 7) + (lane & 8), tr_u = lane >> 4;
  const int r0 = mi * 16 + (lane >> 2), r1 = r0 + 8;
  chain_go();
  chain_wait();

  if (tid < 2) reinterpret_cast<double*>(F + kfRow * kC)[6 + tid] = 0.0;

  // ---- raw k and q
  constexpr int LPR = N / 8;
#pragma unroll
  for (int i = tid; i < 2 * kC * LPR; i += kThreads) {
    const int w = i / (kC * LPR), j = i % (kC * LPR), row = j / LPR, u = j % LPR;
    const uint16_t* src = static_cast<const uint16_t*>(w ? d.q : d.k) +
                          ((row0 + (row < valid ? row : 0)) * d.nkheads + kh) * N + u * 8;
    copy16(sm + (w ? g.q : g.k) + row * g.xs + u * 16, src, row < valid);
  }

  // ---- a head's tiles on their way: factors, row products and the rows of dy, r
  // and dv first, then the states; the gates' operands into registers
  const int gt = tid - kGateWarp * 32;  // the token of a gate thread
  const bool gate = gt >= 0 && gt < kC;
  const int sl = P / 16;  // at most 8
  uint16_t dt_raw = 0, beta_raw = 0;
  float A_h = 0.f, bias_h = 0.f, end = 0.f, prev = 0.f;
  auto load = [&](int hx) {
    const int h = kh * rep + hx;
    const size_t bch = bc * d.nheads + h;
    const float* sc = reinterpret_cast<const float*>(p.ws_head + bch * (size_t)p.head_bytes +
                                                     4 * kDeltaTri);
    if (tid < 5 * 16) {  // Ghi, Glo, beta, kn, qn
      const int w = tid >> 4, u = tid & 15;
      const int from = w == 0 ? kScGhi : (w == 1 ? kScGlo : (w == 2 ? kScBeta : (w == 3 ? kScKn : kScQn)));
      copy16(sm + g.f + (w * kC + u * 4) * 4, sc + from * kC + u * 4, true);
    }
    if (tid < 3 * 16 * sl) {
      const int w = tid / (16 * sl), u = tid - w * 16 * sl;
      const float* src = (w == 0 ? p.ws_dotb : (w == 1 ? p.ws_doto : p.ws_dotv)) + bch * sl * kC;
      copy16(sm + g.dots + tid * 16, src + u * 4, true);
    }
    {  // half a warp per row of headdim (at most 16 units), two rows per thread and tensor
      const int u = lane & 15;
#pragma unroll
      for (int w = 0; w < 3; ++w) {
        const uint16_t* src = (w == 0 ? p.dy : (w == 1 ? p.ws_r : p.dv)) + (row0 * d.nheads + h) * P + u * 8;
        const uint32_t to = sm + (w == 0 ? g.dy : (w == 1 ? g.r : g.dr)) + u * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 32 * i + 2 * warp + (lane >> 4);
          if (u < P / 8)
            copy16(to + row * g.ps, src + (size_t)(row < valid ? row : 0) * d.nheads * P, row < valid);
        }
      }
    }
    cp_async_commit_group();
    {
      const size_t at = bch * ((size_t)P * N) + tid * 8;
      for (int j = tid; j < P * LPR; j += kThreads) {
        const uint32_t to = sm + (j / LPR) * g.xs + (j % LPR) * 16;
        copy16(to + g.s, p.ws_state16 + at + (size_t)(j - tid) * 8, true);
        copy16(to + g.ds, p.ws_dstate16 + at + (size_t)(j - tid) * 8, true);
      }
    }
    cp_async_commit_group();
    if (gate) {
      // <S_end, dS_end>, over the reverse pass's warps
      end = lane < 2 * sl ? p.ws_end[bch * 2 * sl + lane] : 0.f;
      prev = c > 0 && lane < 2 * sl ? p.ws_end[(bch - d.nheads) * 2 * sl + lane] : 0.f;
      A_h = d.A[h];
      bias_h = d.dt_bias ? d.dt_bias[h] : 0.f;
      if (gt < valid) {
        dt_raw = static_cast<const uint16_t*>(d.dt)[(row0 + gt) * d.nheads + h];
        beta_raw = static_cast<const uint16_t*>(d.beta)[(row0 + gt) * d.nheads + h];
      }
    }
  };

  float tq[T][4] = {}, tk[T][4] = {};
  load(0);
  for (int hx = 0; hx < rep; ++hx) {
    const int h = kh * rep + hx;
    const size_t bch = bc * d.nheads + h;
    const size_t gate_at = (row0 + gt) * d.nheads + h;  // of a gate thread
    cp_async_wait_group<1>();
    __syncthreads();

    if (hx == 0) {  // 1 / (|x|^2 + eps) of every k and q row
      const int row = tid >> 3, l8 = tid & 7;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float ss = 0.f;
#pragma unroll
        for (int u = l8; u < LPR; u += 8) {
          const uint4 raw = *reinterpret_cast<const uint4*>(smem + (w ? g.q : g.k) + row * g.xs + u * 16);
          const uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            ss = fmaf(bf16_lo(v[j]), bf16_lo(v[j]), fmaf(bf16_hi(v[j]), bf16_hi(v[j]), ss));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (l8 == 0) F[(w ? kfLq : kfLk) * kC + row] = d.qk_norm ? 1.f / (ss + kDeltaQkEps) : 0.f;
      }
    }

    // ---- the gates, one token per thread of two warps that have no weights below
    if (gate) {
      const float* dots = reinterpret_cast<const float*>(smem + g.dots) + gt;
      double* R = reinterpret_cast<double*>(F + kfRow * kC);
      float so = 0.f, sv = 0.f;
      for (int i = 0; i < sl; ++i) {
        so += dots[(sl + i) * kC];
        sv += dots[(2 * sl + i) * kC];
      }
      float terms;
      bool lost;
      const float dg = suffix_sum(so, sv, end, prev, c == 0, R, gt, terms, lost);
      if (lost && gt < valid && (d.h0 || t0 + gt > 0)) R[7] = 1.0;  // ... of every head
      if (gt < valid) {
        float db = 0.f;
        for (int i = 0; i < sl; ++i) db += dots[i * kC];
        db /= delta_beta_floor(F[kfBeta * kC + gt]);
        if (d.beta_sigmoid) {
          const float be = delta_beta(bf16_to_f32(beta_raw), 1);
          db *= be * (1.f - be);
        }
        p.dbeta[gate_at] = f32_to_bf16(db);
      }
      write_gates(p, R, dg, gt, gate_at, bch, t0 + gt == 0, gt < valid, bf16_to_f32(dt_raw) + bias_h, A_h);
    }

    // ---- dy r^T and dv r^T -> W, N + N^T: rows of block mi, columns of block `part`
    if (part <= mi) {
      float wv[2][4] = {}, xv[2][4] = {};
#pragma unroll 4
      for (int kt = 0; kt < P / 16; ++kt) {
        uint32_t a[4], e[4], bb[4];
        ldsm4(a, sm + g.dy + (mi * 16 + a_row) * g.ps + (2 * kt + a_u) * 16);
        ldsm4(e, sm + g.dr + (mi * 16 + a_row) * g.ps + (2 * kt + a_u) * 16);
        ldsm4(bb, sm + g.r + (16 * part + nt_row) * g.ps + (2 * kt + nt_u) * 16);
        mma_bf16(wv[0], a, bb[0], bb[1]);
        mma_bf16(wv[1], a, bb[2], bb[3]);
        mma_bf16(xv[0], e, bb[0], bb[1]);
        mma_bf16(xv[1], e, bb[2], bb[3]);
      }
      const float gh[2] = {F[kfGhi * kC + r0], F[kfGhi * kC + r1]};
      const float gl[2] = {F[kfGlo * kC + r0], F[kfGlo * kC + r1]};
      const float kn[2] = {F[kfKn * kC + r0], F[kfKn * kC + r1]};
      const float qn[2] = {F[kfQn * kC + r0], F[kfQn * kC + r1]};
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int j0 = 16 * part + 8 * y + 2 * (lane & 3);
        const float2 ch = *reinterpret_cast<const float2*>(F + kfGhi * kC + j0);
        const float2 cl = *reinterpret_cast<const float2*>(F + kfGlo * kC + j0);
        const float2 cb = *reinterpret_cast<const float2*>(F + kfBeta * kC + j0);
        const float2 ck = *reinterpret_cast<const float2*>(F + kfKn * kC + j0);
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // rows r0, r1: an 8 x 8 matrix each
          const int i = x ? r1 : r0;
          float w[2], n[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int j = j0 + q;
            const float gm = j <= i ? ex2_approx((gh[x] - (q ? ch.y : ch.x)) + (gl[x] - (q ? cl.y : cl.x)))
                                    : 0.f;
            const float gb = gm * (q ? cb.y : cb.x);
            w[q] = j <= i ? gb * wv[y][2 * x + q] : 0.f;
            n[q] = j < i ? -gb * xv[y][2 * x + q] : 0.f;
          }
          const int at = i * kWs + j0 * 2;
          *reinterpret_cast<uint32_t*>(smem + g.w1 + at) = pack_bf16x2(w[0] * ck.x, w[1] * ck.y);
          *reinterpret_cast<uint32_t*>(smem + g.w2 + at) = pack_bf16x2(w[0] * qn[x], w[1] * qn[x]);
          // N and its mirror image; a matrix on the diagonal holds both
          const uint32_t lo = pack_bf16x2(n[0] * ck.x, n[1] * ck.y);
          const uint32_t up = transpose8(pack_bf16x2(n[0] * kn[x], n[1] * kn[x]));
          if (part < mi || x > y) {
            const int jt = 16 * part + 8 * y + (lane >> 2), it = 16 * mi + 8 * x + 2 * (lane & 3);
            *reinterpret_cast<uint32_t*>(smem + g.ns + at) = lo;
            *reinterpret_cast<uint32_t*>(smem + g.ns + jt * kWs + it * 2) = up;
          } else if (x == y) {
            *reinterpret_cast<uint32_t*>(smem + g.ns + at) = lo | up;
          }
        }
      }
    }
    cp_async_wait_group<0>();
    __syncthreads();

    // ---- dq += e^G dy S + W k;  dk += beta e^(G_end - G) r dS - e^G dv S + W^T q + (N + N^T) k
    const float g0 = F[kfGhi * kC + r0], l0 = F[kfGlo * kC + r0];
    const float g1 = F[kfGhi * kC + r1], l1 = F[kfGlo * kC + r1];
    const float ge = F[kfGhi * kC + kC - 1], le = F[kfGlo * kC + kC - 1];
    const float D0 = ex2_approx(g0 + l0), D1 = ex2_approx(g1 + l1);
    const float E0 = ex2_approx((ge - g0) + (le - l0)) * F[kfBeta * kC + r0];
    const float E1 = ex2_approx((ge - g1) + (le - l1)) * F[kfBeta * kC + r1];
    {
      float t[T][4] = {}, x[T][4] = {};
#pragma unroll 2
      for (int kt = 0; kt < P / 16; ++kt) {
        uint32_t a[4], e[4];
        ldsm4(a, sm + g.dy + (mi * 16 + a_row) * g.ps + (2 * kt + a_u) * 16);
        ldsm4(e, sm + g.dr + (mi * 16 + a_row) * g.ps + (2 * kt + a_u) * 16);
#pragma unroll
        for (int j = 0; j < T / 2; ++j) {
          uint32_t bb[4];
          ldsm4t(bb, sm + g.s + (16 * kt + tr_row) * g.xs + (part * T + 2 * j + tr_u) * 16);
          mma_bf16(t[2 * j], a, bb[0], bb[1]);
          mma_bf16(t[2 * j + 1], a, bb[2], bb[3]);
          mma_bf16(x[2 * j], e, bb[0], bb[1]);
          mma_bf16(x[2 * j + 1], e, bb[2], bb[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tq[j][q] = fmaf(q < 2 ? D0 : D1, t[j][q], tq[j][q]);
          tk[j][q] = fmaf(q < 2 ? -D0 : -D1, x[j][q], tk[j][q]);
        }
    }
    {
      float t[T][4] = {};
#pragma unroll 4
      for (int kt = 0; kt < P / 16; ++kt) {
        uint32_t a[4];
        ldsm4(a, sm + g.r + (mi * 16 + a_row) * g.ps + (2 * kt + a_u) * 16);
#pragma unroll
        for (int j = 0; j < T / 2; ++j) {
          uint32_t bb[4];
          ldsm4t(bb, sm + g.ds + (16 * kt + tr_row) * g.xs + (part * T + 2 * j + tr_u) * 16);
          mma_bf16(t[2 * j], a, bb[0], bb[1]);
          mma_bf16(t[2 * j + 1], a, bb[2], bb[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) tk[j][q] = fmaf(q < 2 ? E0 : E1, t[j][q], tk[j][q]);
    }
    if (hx + 1 < rep) {  // rows, states and factors are read: the next head's, meanwhile
      __syncthreads();
      load(hx + 1);
    }
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      uint32_t a[4], e[4], f[4];
      ldsm4(a, sm + g.w1 + (mi * 16 + a_row) * kWs + (2 * kt + a_u) * 16);
      ldsm4t(e, sm + g.w2 + (16 * kt + nt_row) * kWs + (2 * mi + nt_u) * 16);
      ldsm4(f, sm + g.ns + (mi * 16 + a_row) * kWs + (2 * kt + a_u) * 16);
#pragma unroll
      for (int j = 0; j < T / 2; ++j) {
        uint32_t bk[4], bq[4];
        ldsm4t(bk, sm + g.k + (16 * kt + tr_row) * g.xs + (part * T + 2 * j + tr_u) * 16);
        ldsm4t(bq, sm + g.q + (16 * kt + tr_row) * g.xs + (part * T + 2 * j + tr_u) * 16);
        if (kt <= mi) {
          mma_bf16(tq[2 * j], a, bk[0], bk[1]);
          mma_bf16(tq[2 * j + 1], a, bk[2], bk[3]);
        }
        if (kt >= mi) {
          mma_bf16(tk[2 * j], e, bq[0], bq[1]);
          mma_bf16(tk[2 * j + 1], e, bq[2], bq[3]);
        }
        mma_bf16(tk[2 * j], f, bk[0], bk[1]);
        mma_bf16(tk[2 * j + 1], f, bk[2], bk[3]);
      }
    }

  }

  // ---- through x / |x| (dx = n (t - x (x . t) / |x|^2)), then bf16 rows
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float d0, d1;
    rows_dot<T>(w ? tq : tk, smem + (w ? g.q : g.k), g.xs, r0, part, lane, d0, d1);
    if ((lane & 3) == 0) {  // over the weights' tiles, which are free
      float* D = reinterpret_cast<float*>(smem + g.w1) + (4 * w + part) * kC;
      D[r0] = d0;
      D[r1] = d1;
    }
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const unsigned char* x = smem + (w ? g.q : g.k);
    const float n0 = F[(w ? kfQn : kfKn) * kC + r0], n1 = F[(w ? kfQn : kfKn) * kC + r1];
    const float* D = reinterpret_cast<const float*>(smem + g.w1) + 4 * w * kC;
    const float e0 = F[(w ? kfLq : kfLk) * kC + r0] *
                     (D[r0] + D[kC + r0] + D[2 * kC + r0] + D[3 * kC + r0]);
    const float e1 = F[(w ? kfLq : kfLk) * kC + r1] *
                     (D[r1] + D[kC + r1] + D[2 * kC + r1] + D[3 * kC + r1]);
    uint16_t* dst = w ? p.dq : p.dk;
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const int at = (part * T + j) * 16 + (lane & 3) * 4;
      const uint32_t x0 = *reinterpret_cast<const uint32_t*>(x + r0 * g.xs + at);
      const uint32_t x1 = *reinterpret_cast<const uint32_t*>(x + r1 * g.xs + at);
      const float(&t)[4] = w ? tq[j] : tk[j];
      if (r0 < valid)
        *reinterpret_cast<uint32_t*>(dst + ((row0 + r0) * d.nkheads + kh) * N + at / 2) =
            pack_bf16x2(n0 * (t[0] - bf16_lo(x0) * e0), n0 * (t[1] - bf16_hi(x0) * e0));
      if (r1 < valid)
        *reinterpret_cast<uint32_t*>(dst + ((row0 + r1) * d.nkheads + kh) * N + at / 2) =
            pack_bf16x2(n1 * (t[2] - bf16_lo(x1) * e1), n1 * (t[3] - bf16_hi(x1) * e1));
    }
  }

  // ---- the heads with strong decays
  double* const R = reinterpret_cast<double*>(F + kfRow * kC);
  const bool lost = R[7] != 0.0;
  if (R[6] == 0.0 && !lost) return;
  __syncthreads();
  for (int hx = 0; hx < rep; ++hx)
    if (lost || strong_head(p, bc * d.nheads + kh * rep + hx)) {
      strong_gates<N>(p, smem, kh * rep + hx);
      __syncthreads();
    }
}

// dA, ddt_bias: the chunks' sums of one head, in a fixed order.
__global__ void __launch_bounds__(128) delta_grad_reduce(const DeltaChunkParams p) {
  __shared__ double sh[2][128];
  const int64_t rows = (int64_t)p.d.batch * p.nchunks;
  const int nheads = p.d.nheads;
  chain_wait();
  const int h = blockIdx.x, tid = threadIdx.x;
  double a = 0.0, s = 0.0;
  for (int64_t i = tid; i < rows; i += 128) {
    a += p.ws_part[(i * nheads + h) * 2];
    s += p.ws_part[(i * nheads + h) * 2 + 1];
  }
  sh[0][tid] = a;
  sh[1][tid] = s;
  __syncthreads();
  for (int o = 64; o > 0; o >>= 1) {
    if (tid < o) {
      sh[0][tid] += sh[0][tid + o];
      sh[1][tid] += sh[1][tid + o];
    }
    __syncthreads();
  }
  if (tid == 0) {
    if (p.dA) p.dA[h] = (float)sh[0][0];
    if (p.ddt_bias) p.ddt_bias[h] = (float)sh[1][0];
  }
}

template <int N>
cudaError_t launch(const DeltaChunkParams& p, cudaStream_t stream) {
  const int bytes = grad_layout(N, p.d.headdim).bytes;
  cudaError_t e = allow_shared(delta_grad_kernel<N>);
  if (e != cudaSuccess) return e;
  e = launch_chained(delta_grad_kernel<N>, dim3(p.nchunks, p.d.nkheads, p.d.batch), kThreads, bytes,
                     stream, p);
  if (e != cudaSuccess || (!p.dA && !p.ddt_bias)) return e;
  return launch_chained(delta_grad_reduce, dim3(p.d.nheads), 128, 0, stream, p);
}

}  // namespace

cudaError_t launch_delta_grad(const DeltaChunkParams& p, cudaStream_t stream) {
  return p.d.dstate == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace ssm
