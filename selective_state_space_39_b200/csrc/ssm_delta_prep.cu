// ssm_delta_prep.cu -- what the chunk kernels of the gated delta rule need of
// each chunk of 64 tokens, before any state is known (bf16 io, sm_100a).
//
// With G_i the running log decay inside the chunk, k and q of unit length and
//   M_ij = (k_i . k_j) e^(G_i - G_j)  (j < i),   P_ij = (q_i . k_j) e^(G_i - G_j)  (j <= i)
// the chunk's residuals r (u = beta r) solve (I + M diag(beta)) r = v - e^G S k,
// so the kernel writes T = (I + M diag(beta))^-1, P, and the per-token factors
// (DeltaScal). T is inverted block by block: the eight 8 x 8 diagonal blocks by
// forward substitution (one column per lane, fp32), then
//   T_10 = -T_11 (L_10 T_00) over blocks of 8, of 16 and of 32 rows,
// the products as tf32 MMAs of two pieces (21 bits; the rest of fp32's range
// needs no scale). k and q are written as fp16 rows scaled by a power of two
// (exact for every element within 2^14 of the row's largest), T as two fp16
// pieces and P as one (two for the backward pass), each row under its own
// power-of-two scale; only blocks on and below the diagonal are kept. G is
// summed in fp64 and kept as two floats: differences of G stay exact to fp32
// even after a token with a decay of e^-100 (log decays are cut there: the
// factor is below the smallest fp32 either way).
//
// One CTA takes a chunk of a key head and up to four of its value heads: the
// fp16 rows, k k^T and q k^T (fp16 MMAs) are shared by the heads. Below the
// diagonal blocks the decay is a product of a row's and a column's factor
// around the start of the row's block, e^(G_i - G_s) e^(G_s - G_j), neither
// above 1 where no decay is; inside them it is taken from the difference itself.
//
// Bound: the latencies of about 1900 instructions per warp and head, at four CTAs
// per SM (issue slots 53 % busy, tensor pipe 20 %, DRAM 2.3 TB/s): 219 us for
// 4 x 4096 tokens, 64 heads on 16 key heads, dstate 128 (500 MB of DRAM
// traffic); five CTAs of 96 registers took 233. 8192 tokens of 32 heads: 77 us; for
// the backward pass, 2 x 2048 tokens of 32 heads: 46 us.
#include "ssm_delta.cuh"

namespace ssm {

namespace {

constexpr int kC = kDeltaChunk;
constexpr int kThreads = 128;
constexpr int kHeads = 4;        // value heads per CTA, at most
// The fp32 matrix of a head: rows of kLs floats, in which the rows with bit 2 set
// swap the two quads of every eight columns. MMA operands (rows or columns along a
// quad), float2 fragments and float4 rows then all meet every bank once.
constexpr int kLs = kC + 8;
constexpr float kMinLogDecay = -100.f;

template <int N>
struct PrepSmem {
  static constexpr int kTile = kC * N * 2;
  static constexpr int kL = kC * kLs * 4;                  // L, then T, of one head
  static constexpr int kKK = 20 * 512;                     // k k^T, in fragments
  static constexpr int kA = 2 * kTile > kL + kKK ? 2 * kTile : kL + kKK;  // over the k/q tiles
  static constexpr int kScal = 2 * kDeltaScalBwd;          // of two heads
  static constexpr int kTok = 4 * kC * 4;
  static constexpr int kCols = 2 * 3 * kC * 4;             // column factors per row block
  static constexpr int kBytes = kA + kScal + kTok + kCols + 64;
};

// tf32 MMA of two-piece fp32 operands: d += a b, hi lo cross terms included.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tf32_pieces(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// d[16 x 16] = A[16 x n] B[n x 16] over k0 <= n < k1, both in the matrix.
__device__ __forceinline__ void block_product(float (&d)[2][4], const float* A, const float* B,
                                              int k0, int k1, int lane) {
  const int g = lane >> 2, t = lane & 3, flip = g & 4;
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int q = 0; q < 4; ++q) d[n][q] = 0.f;
#pragma unroll 2
  for (int k = k0; k < k1; k += 8) {
    uint32_t ah[4], al[4];
    tf32_pieces(A[g * kLs + k + t + flip], ah[0], al[0]);
    tf32_pieces(A[(g + 8) * kLs + k + t + flip], ah[1], al[1]);
    tf32_pieces(A[g * kLs + k + t + 4 - flip], ah[2], al[2]);
    tf32_pieces(A[(g + 8) * kLs + k + t + 4 - flip], ah[3], al[3]);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      uint32_t bh0, bl0, bh1, bl1;
      tf32_pieces(B[(k + t) * kLs + 8 * n + g], bh0, bl0);
      tf32_pieces(B[(k + t + 4) * kLs + 8 * n + (g ^ 4)], bh1, bl1);
      mma_tf32(d[n], al, bh0, bh1);
      mma_tf32(d[n], ah, bl0, bl1);
      mma_tf32(d[n], ah, bh0, bh1);
    }
  }
}
// d[8 x 8] = A B, 8 x 8 blocks of the matrix (rows 8 .. 15 of the MMA are empty).
__device__ __forceinline__ void small_product(float (&d)[4], const float* A, const float* B, int lane) {
  const int g = lane >> 2, t = lane & 3, flip = g & 4;
  uint32_t ah[4] = {}, al[4] = {}, bh0, bl0, bh1, bl1;
  tf32_pieces(A[g * kLs + t + flip], ah[0], al[0]);
  tf32_pieces(A[g * kLs + t + 4 - flip], ah[2], al[2]);
  tf32_pieces(B[t * kLs + g], bh0, bl0);
  tf32_pieces(B[(t + 4) * kLs + (g ^ 4)], bh1, bl1);
  d[0] = d[1] = d[2] = d[3] = 0.f;
  mma_tf32(d, al, bh0, bh1);
  mma_tf32(d, ah, bl0, bl1);
  mma_tf32(d, ah, bh0, bh1);
}
__device__ __forceinline__ void block_store(const float (&d)[2][4], float* D, float sign, int lane) {
  const int g = lane >> 2, col = (2 * (lane & 3)) ^ (g & 4);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    *reinterpret_cast<float2*>(D + g * kLs + 8 * n + col) =
        make_float2(sign * d[n][0], sign * d[n][1]);
    *reinterpret_cast<float2*>(D + (g + 8) * kLs + 8 * n + col) =
        make_float2(sign * d[n][2], sign * d[n][3]);
  }
}

template <int N, bool BWD>
__global__ void __launch_bounds__(kThreads, 4) delta_prep_kernel(const DeltaChunkParams p, const int heads) {
  chain_go();
  extern __shared__ __align__(128) unsigned char smem[];
  using Sm = PrepSmem<N>;
  constexpr int LPR = N / 8;       // lanes (16-byte units) per row
  constexpr int RPW = 32 / LPR;    // rows per warp and step
  unsigned char* tiles = smem;
  float* L = reinterpret_cast<float*>(smem);
  float* scal = reinterpret_cast<float*>(smem + Sm::kA);
  float* tok = reinterpret_cast<float*>(smem + Sm::kA + Sm::kScal);  // kmul qmul kn qn
  float* cols = tok + 4 * kC;  // [row block 1..3][P, L] x 64
  float* rows_s = cols;      // T's row scales, once the column factors are spent
  double* carry = reinterpret_cast<double*>(smem + Sm::kA + Sm::kScal + Sm::kTok + Sm::kCols);
  const DeltaParams& d_ = p.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, b = blockIdx.z;
  const int rep = d_.nheads / d_.nkheads, subs = (rep + heads - 1) / heads;
  const int kh = blockIdx.y / subs, sub = blockIdx.y - kh * subs;
  const int64_t t0 = (int64_t)c * kC;
  const int valid = (int)min((int64_t)kC, d_.seqlen - t0);
  const size_t bc = (size_t)b * p.nchunks + c;

  // ---- k and q rows: largest magnitude, length, fp16 rows
  unsigned char* kq_out = p.ws_kq + (bc * d_.nkheads + kh) * (size_t)(2 * Sm::kTile);
  constexpr int IT = kC / (4 * RPW);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint16_t* src = static_cast<const uint16_t*>(w ? d_.q : d_.k) +
                          (((size_t)b * d_.seqlen + t0) * d_.nkheads + kh) * N;
    uint4 raw[IT];
    const int u = lane % LPR, row0 = warp * RPW + lane / LPR;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int row = it * 4 * RPW + row0;
      raw[it] = row < valid ? *reinterpret_cast<const uint4*>(src + (size_t)row * d_.nkheads * N + u * 8)
                            : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int row = it * 4 * RPW + row0;
      const uint32_t r4[4] = {raw[it].x, raw[it].y, raw[it].z, raw[it].w};
      uint32_t m2 = 0;  // magnitudes of bf16 pairs order like integers
      float2 s2 = make_float2(0.f, 0.f), f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m2 = __vmaxu2(m2, r4[i] & 0x7FFF7FFFu);
        f[i] = make_float2(bf16_lo(r4[i]), bf16_hi(r4[i]));
        s2 = fma2(f[i], f[i], s2);
      }
      float ss = s2.x + s2.y;
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) {
        m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
      }
      // s = 2^-e brings the largest magnitude to [1, 2); its inverse goes into kmul
      uint32_t e = max(m2 & 0xFFFFu, m2 >> 16) >> 7;
      e = e < 1u ? 1u : (e > 253u ? 253u : e);
      const float s = __uint_as_float((254u - e) << 23), inv = __uint_as_float(e << 23);
      uint4 out;
      uint32_t* o4 = &out.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = mul2(f[i], make_float2(s, s));
        o4[i] = h2_bits(__floats2half2_rn(v.x, v.y));
      }
      const uint32_t at = kq_at(row, u);
      *reinterpret_cast<uint4*>(tiles + w * Sm::kTile + at) = out;
      if (sub == 0) *reinterpret_cast<uint4*>(kq_out + w * Sm::kTile + at) = out;
      if (u == 0) {
        const float len = d_.qk_norm ? 1.f / sqrtf(ss + kDeltaQkEps) : 1.f;
        const float sc = w ? d_.scale : 1.f;
        tok[w * kC + row] = len * inv * sc;
        tok[(2 + w) * kC + row] = len * sc;
      }
    }
  }

  __syncthreads();

  // ---- k k^T and q k^T: warp w takes rows 16 w .. 16 w + 15, columns up to them
  float kk[8][4] = {}, qk[8][4] = {};
  {
    const uint32_t ks = smem_u32(tiles), qs = ks + Sm::kTile;
#pragma unroll
    for (int kt = 0; kt < N / 16; ++kt) {
      uint32_t ak[4], aq[4];
      const int ar = warp * 16 + (lane & 15), au = 2 * kt + (lane >> 4);
      ldsm4(ak, ks + kq_at(ar, au));
      ldsm4(aq, qs + kq_at(ar, au));
#pragma unroll
      for (int jp = 0; jp < 4; ++jp) {
        if (jp > warp) continue;
        uint32_t bb[4];
        ldsm4(bb, ks + kq_at(16 * jp + (lane & 7) + ((lane & 16) >> 1), 2 * kt + ((lane >> 3) & 1)));
        mma_f16(kk[2 * jp], ak, bb[0], bb[1]);
        mma_f16(kk[2 * jp + 1], ak, bb[2], bb[3]);
        mma_f16(qk[2 * jp], aq, bb[0], bb[1]);
        mma_f16(qk[2 * jp + 1], aq, bb[2], bb[3]);
      }
    }
  }
  // each warp keeps its part of k k^T in shared memory, out of its registers
  __syncthreads();  // the k/q tiles are free
  float4* kk_at = reinterpret_cast<float4*>(smem + Sm::kL) + warp * (warp + 1) * 32 + lane;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j <= 2 * warp + 1) kk_at[j * 32] = make_float4(kk[j][0], kk[j][1], kk[j][2], kk[j][3]);

  const int nh = min(heads, rep - sub * heads);
  const int r0 = warp * 16 + (lane >> 2), r1 = r0 + 8;
  constexpr int kTiles = BWD ? 4 : 3;
  for (int x = 0; x < nh; ++x) {
    __syncthreads();  // the previous head's matrix and factors are free

    // ---- gates of two heads: two warps per head, one token per thread
    if ((x & 1) == 0) {
      const int xg = x + (warp >> 1), i = tid & 63;
      double g = 0.0;
      float beta = 0.f;
      bool strong = false;
      if (xg < nh && i < valid) {
        const int h = kh * rep + sub * heads + xg;
        const size_t at = ((size_t)b * d_.seqlen + t0 + i) * d_.nheads + h;
        const float raw = bf16_to_f32(static_cast<const uint16_t*>(d_.dt)[at]) +
                          (d_.dt_bias ? d_.dt_bias[h] : 0.f);
        float gf = delta_step_size(raw, d_.softplus) * d_.A[h];
        strong = gf < kStrongDecay;
        gf = gf < kMinLogDecay ? kMinLogDecay : gf;
        g = (double)gf * 1.4426950408889634;  // log2 units
        beta = delta_beta(bf16_to_f32(static_cast<const uint16_t*>(d_.beta)[at]), d_.beta_sigmoid);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, g, o);
        if (lane >= o) g += up;
      }
      if ((warp & 1) == 0 && lane == 31) carry[warp >> 1] = g;
      __syncthreads();
      if (warp & 1) g += carry[warp >> 1];
      float* sc = scal + (warp >> 1) * (kDeltaScalBwd / 4);
      const float hi = (float)g;
      if (BWD) {
        strong = __any_sync(0xffffffffu, strong);
        if (xg < nh && lane == 0) {
          sc[kScEnd * kC + 3 + (warp & 1)] = strong ? 1.f : 0.f;
          sc[kScEnd * kC + 5] = 0.f;
        }
        const float use = delta_beta_floor(beta);
        if (xg < nh) sc[kScRatio * kC + i] = use == beta ? 1.f : beta / use;
        beta = use;
      }
      if (xg < nh) {
        sc[kScGhi * kC + i] = hi;
        sc[kScGlo * kC + i] = (float)(g - (double)hi);
        sc[kScBeta * kC + i] = beta;
      }
      __syncthreads();
      if (xg < nh) {
        const float ehi = sc[kScGhi * kC + kC - 1], elo = sc[kScGlo * kC + kC - 1];
        if (!d_.qk_norm || !d_.beta_sigmoid) {
          // the longest and the shortest key (those of zeros aside), and a large beta
          const float len = tok[i], odd = fabsf(sc[kScBeta * kC + i]) >= kOddBeta ? INFINITY : len;
          const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(odd));
          const uint32_t least = __reduce_min_sync(0xffffffffu, __float_as_uint(len > 0x1p-110f ? len : INFINITY));
          if (lane == 0) {
            sc[kScEnd * kC + 8 + (warp & 1)] = __uint_as_float(most);
            sc[kScEnd * kC + 10 + (warp & 1)] = __uint_as_float(least);
          }
        }
        const float lo = sc[kScGlo * kC + i];
        const float D = ex2_approx(hi + lo), E = ex2_approx((ehi - hi) + (elo - lo));
        sc[kScSk * kC + i] = D * tok[i];
        sc[kScKend * kC + i] = tok[i] * E;
        sc[kScK * kC + i] = tok[i];
        sc[kScSq * kC + i] = D * tok[kC + i];
        if (i == 0) sc[kScEnd * kC] = ex2_approx(ehi + elo);
        // (1 where no decay is above 1)
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(E, 1.f)));
        if (lane == 0) sc[kScEnd * kC + 1 + (warp & 1)] = __uint_as_float(most);
        sc[kScKn * kC + i] = tok[2 * kC + i];
        sc[kScQn * kC + i] = tok[3 * kC + i];
      }
      __syncthreads();
    }
    unsigned char* tri = p.ws_head + (bc * d_.nheads + kh * rep + sub * heads + x) * (size_t)p.head_bytes;
    float* sc = scal + (x & 1) * (kDeltaScalBwd / 4);
    const float gh0 = sc[kScGhi * kC + r0], gl0 = sc[kScGlo * kC + r0];
    const float gh1 = sc[kScGhi * kC + r1], gl1 = sc[kScGlo * kC + r1];
    const float km0 = tok[r0], km1 = tok[r1];

    // ---- column factors of the row blocks 1 .. 3, and each row's own
    for (int i = tid; i < 3 * kC; i += kThreads) {
      const int I = i / kC + 1, j = i & (kC - 1);
      const float f = ex2_approx((sc[kScGhi * kC + 16 * I] - sc[kScGhi * kC + j]) +
                                 (sc[kScGlo * kC + 16 * I] - sc[kScGlo * kC + j]));
      cols[(I - 1) * 2 * kC + j] = f;
      cols[((I - 1) * 2 + 1) * kC + j] = f * tok[j] * sc[kScBeta * kC + j];
    }
    const float a0 = ex2_approx((gh0 - sc[kScGhi * kC + 16 * warp]) + (gl0 - sc[kScGlo * kC + 16 * warp]));
    const float a1 = ex2_approx((gh1 - sc[kScGhi * kC + 16 * warp]) + (gl1 - sc[kScGlo * kC + 16 * warp]));
    __syncthreads();

    // ---- L = M diag(beta) and P on the warp's 16 rows
    float pv[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q) pv[j][q] = 0.f;
      if (j > 2 * warp + 1) continue;
      const int col = 8 * j + 2 * (lane & 3);
      const float4 kkj = kk_at[j * 32];
      float lv[4];
      if (j < 2 * warp) {
        const float2 cp = *reinterpret_cast<const float2*>(cols + (warp - 1) * 2 * kC + col);
        const float2 cl = *reinterpret_cast<const float2*>(cols + ((warp - 1) * 2 + 1) * kC + col);
        pv[j][0] = qk[j][0] * cp.x * a0;
        pv[j][1] = qk[j][1] * cp.y * a0;
        pv[j][2] = qk[j][2] * cp.x * a1;
        pv[j][3] = qk[j][3] * cp.y * a1;
        lv[0] = kkj.x * cl.x * (a0 * km0);
        lv[1] = kkj.y * cl.y * (a0 * km0);
        lv[2] = kkj.z * cl.x * (a1 * km1);
        lv[3] = kkj.w * cl.y * (a1 * km1);
      } else {
        const float2 ch = *reinterpret_cast<const float2*>(sc + kScGhi * kC + col);
        const float2 cl = *reinterpret_cast<const float2*>(sc + kScGlo * kC + col);
        const float2 cb = *reinterpret_cast<const float2*>(sc + kScBeta * kC + col);
        const float2 ck = *reinterpret_cast<const float2*>(tok + col);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int cc = col + (q & 1), row = q < 2 ? r0 : r1;
          const float gm = ex2_approx(((q < 2 ? gh0 : gh1) - ((q & 1) ? ch.y : ch.x)) +
                                      ((q < 2 ? gl0 : gl1) - ((q & 1) ? cl.y : cl.x)));
          if (cc <= row) pv[j][q] = qk[j][q] * gm;
          lv[q] = cc < row ? (q < 2 ? (q ? kkj.y : kkj.x) : (q == 3 ? kkj.w : kkj.z)) * gm * (q < 2 ? km0 : km1) *
                                 ((q & 1) ? ck.y * cb.y : ck.x * cb.x)
                           : 0.f;
        }
      }
      const int at = col ^ (r0 & 4);
      *reinterpret_cast<float2*>(L + r0 * kLs + at) = make_float2(lv[0], lv[1]);
      *reinterpret_cast<float2*>(L + r1 * kLs + at) = make_float2(lv[2], lv[3]);
    }
    float m0, m1;
    row_max(pv, m0, m1);
    const RowScale s0 = row_scale(exponent_of(m0)), s1 = row_scale(exponent_of(m1));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j > 2 * warp + 1) continue;
      uint32_t hi0, lo0, hi1, lo1;
      split2(pv[j][0], pv[j][1], s0.s, hi0, lo0);
      split2(pv[j][2], pv[j][3], s1.s, hi1, lo1);
      // a store of the warp is a whole core matrix: 128 bytes
      unsigned char* ph = tri + 2 * kDeltaTri + delta_tri_block(warp, j >> 1) + (lane & 3) * 4;
      const uint32_t a0 = tri_at(lane >> 2, j & 1), a1 = tri_at((lane >> 2) + 8, j & 1);
      *reinterpret_cast<uint32_t*>(ph + a0) = hi0;
      *reinterpret_cast<uint32_t*>(ph + a1) = hi1;
      if (BWD) {
        *reinterpret_cast<uint32_t*>(ph + kDeltaTri + a0) = lo0;
        *reinterpret_cast<uint32_t*>(ph + kDeltaTri + a1) = lo1;
        // P^T: an 8 x 8 matrix and its place are both transposed
        unsigned char* pt = tri + kDeltaLoadBwd + 2 * kDeltaTri + delta_tri_block_t(warp, j >> 1) +
                            tri_at((j & 1) * 8 + (lane >> 2), 0) + (lane & 3) * 4;
        *reinterpret_cast<uint32_t*>(pt) = transpose8(hi0);
        *reinterpret_cast<uint32_t*>(pt + 128) = transpose8(hi1);
        *reinterpret_cast<uint32_t*>(pt + kDeltaTri) = transpose8(lo0);
        *reinterpret_cast<uint32_t*>(pt + kDeltaTri + 128) = transpose8(lo1);
      }
    }
    if ((lane & 3) == 0) {
      sc[kScP * kC + r0] = tok[kC + r0] * s0.inv;
      sc[kScP * kC + r1] = tok[kC + r1] * s1.inv;
    }
    __syncwarp();

    // ---- T, the diagonal block of the warp's rows: its 8 x 8 diagonal blocks by
    // forward substitution (eight lanes each, a column per lane; lanes 16 .. 31
    // repeat lanes 0 .. 15), then the block below them
    {
      float* Ld = L + (warp * 16) * kLs + warp * 16;
      float* Lb = Ld + ((lane >> 3) & 1) * (8 * kLs + 8);
      const int col = lane & 7;
      float xs[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float acc0 = i == col ? 1.f : 0.f, acc1 = 0.f;
#pragma unroll
        for (int j = 0; j < i; j += 4) {
          const float4 l = *reinterpret_cast<const float4*>(Lb + i * kLs + (j ^ (i & 4)));
          acc0 = fmaf(-l.x, xs[j], acc0);
          if (j + 1 < i) acc1 = fmaf(-l.y, xs[j + 1], acc1);
          if (j + 2 < i) acc0 = fmaf(-l.z, xs[j + 2], acc0);
          if (j + 3 < i) acc1 = fmaf(-l.w, xs[j + 3], acc1);
        }
        xs[i] = acc0 + acc1;
      }
      __syncwarp();
      if (lane < 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) Lb[i * kLs + (col ^ (i & 4))] = xs[i];
      }
      __syncwarp();
      float e[4];
      float* Lo = Ld + 8 * kLs;
      float2* to = reinterpret_cast<float2*>(Lo + (lane >> 2) * kLs + ((2 * (lane & 3)) ^ ((lane >> 2) & 4)));
      small_product(e, Lo, Ld, lane);
      __syncwarp();
      *to = make_float2(e[0], e[1]);
      __syncwarp();
      small_product(e, Lo + 8, Lo, lane);
      __syncwarp();
      *to = make_float2(-e[0], -e[1]);
    }
    __syncthreads();

    // ---- T_10, T_32 (warps 1 and 3), then the 32 x 32 block below the diagonal
    float d[2][4];
    if (warp & 1) {
      float* Lo = L + (warp * 16) * kLs + (warp - 1) * 16;
      block_product(d, Lo, L + (warp - 1) * 16 * kLs + (warp - 1) * 16, 0, 16, lane);
      __syncwarp();
      block_store(d, Lo, 1.f, lane);
      __syncwarp();
      block_product(d, L + (warp * 16) * kLs + warp * 16, Lo, 0, 16, lane);
      __syncwarp();
      block_store(d, Lo, -1.f, lane);
    }
    __syncthreads();
    const int bi = warp >> 1, bj = warp & 1;  // this warp's 16 x 16 of the 32 x 32 block
    float* Lba = L + 32 * kLs;
    block_product(d, Lba + bi * 16 * kLs, L + bj * 16, bj * 16, 32, lane);  // T_01 = 0
    __syncthreads();
    block_store(d, Lba + bi * 16 * kLs + bj * 16, 1.f, lane);
    __syncthreads();
    block_product(d, L + (32 + bi * 16) * kLs + 32, Lba + bj * 16, 0, 16 * bi + 16, lane);
    __syncthreads();
    block_store(d, Lba + bi * 16 * kLs + bj * 16, -1.f, lane);
    __syncthreads();

    // ---- T's rows as two pieces: half of every 16-column block per thread
    {
      const int row = warp * 16 + (lane & 15), half = lane >> 4;
      const float* Lr = L + row * kLs + half * 8;
      float4 v[4][2];
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > warp) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          v[j][i] = *reinterpret_cast<const float4*>(Lr + j * 16 + ((4 * i) ^ (row & 4)));
          m = fmaxf(m, fmaxf(fmaxf(fabsf(v[j][i].x), fabsf(v[j][i].y)),
                             fmaxf(fabsf(v[j][i].z), fabsf(v[j][i].w))));
        }
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
      if (m >= kOddT) sc[kScSk * kC] = __uint_as_float(0x7FFFFFFFu);
      const RowScale s = row_scale(exponent_of(m));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > warp) continue;
        uint4 hi, lo;
        split2(v[j][0].x, v[j][0].y, s.s, hi.x, lo.x);
        split2(v[j][0].z, v[j][0].w, s.s, hi.y, lo.y);
        split2(v[j][1].x, v[j][1].y, s.s, hi.z, lo.z);
        split2(v[j][1].z, v[j][1].w, s.s, hi.w, lo.w);
        unsigned char* at = tri + delta_tri_block(warp, j) + tri_at(row & 15, half);
        *reinterpret_cast<uint4*>(at) = hi;
        *reinterpret_cast<uint4*>(at + kDeltaTri) = lo;
      }
      if (half == 0) {
        sc[kScU * kC + row] = sc[kScBeta * kC + row] * s.inv;
        sc[kScT * kC + row] = s.inv;
        if (BWD) sc[kScBeta * kC + row] *= sc[kScRatio * kC + row];
        rows_s[row] = s.s;
      }
    }
    if (tid == 0 && (!d_.qk_norm || !d_.beta_sigmoid)) {
      const float* e = sc + kScEnd * kC + 8;
      if (fmaxf(e[0], e[1]) > fminf(e[2], e[3]) * kOddKeys) sc[kScSk * kC] = __uint_as_float(0x7FFFFFFFu);
    }
    __syncthreads();
    if (BWD) {  // T^T: column `row` of T, eight rows of a block at a time
      const int row = tid >> 1, half = tid & 1;
      for (int i = row / 16; i < 4; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = i * 16 + half * 8 + 2 * q;
          const int at = row ^ (r & 4);  // r and r + 1 swap alike
          pieces2(L[r * kLs + at] * rows_s[r], L[(r + 1) * kLs + at] * rows_s[r + 1], hi[q], lo[q]);
        }
        unsigned char* at = tri + kDeltaLoadBwd + delta_tri_block_t(i, row / 16) + tri_at(row & 15, half);
        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + kDeltaTri) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }

    // ---- the factors
    const uint4* ss = reinterpret_cast<const uint4*>(sc);
    for (int i = tid; i < (BWD ? kDeltaScalBwd : kDeltaScalFwd) / 16; i += kThreads)
      reinterpret_cast<uint4*>(tri + kTiles * kDeltaTri)[i] = ss[i];
  }
}

template <int N, bool BWD>
cudaError_t launch(const DeltaChunkParams& p, cudaStream_t stream) {
  auto* kern = delta_prep_kernel<N, BWD>;
  const cudaError_t e = allow_shared(kern);
  if (e != cudaSuccess) return e;
  // heads per CTA, halved while the grid then still fits the SMs at once (2 x 203
  // tokens of 8 heads on 4 key heads: 13.9 us with two heads per CTA, 11.2 with one)
  const int rep = p.d.nheads / p.d.nkheads;
  auto ctas = [&](int heads) {
    return (int64_t)p.nchunks * p.d.batch * p.d.nkheads * ((rep + heads - 1) / heads);
  };
  int heads = rep < kHeads ? rep : kHeads;
  while (heads > 1 && ctas(heads / 2) <= 4 * 148) heads /= 2;
  const dim3 grid(p.nchunks, p.d.nkheads * ((rep + heads - 1) / heads), p.d.batch);
  kern<<<grid, kThreads, PrepSmem<N>::kBytes, stream>>>(p, heads);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_prep(const DeltaChunkParams& p, bool bwd, cudaStream_t stream) {
  if (p.d.dstate == 64) return bwd ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  return bwd ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
}

}  // namespace ssm
