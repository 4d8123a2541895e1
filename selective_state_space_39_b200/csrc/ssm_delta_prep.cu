// ssm_delta_prep.cu -- what the chunk kernels of the gated delta rule need of
// each chunk of 64 tokens, before any state is known (bf16 io, sm_100a).
//
// With G_i the running log decay inside the chunk, k and q of unit length and
//   M_ij = (k_i . k_j) e^(G_i - G_j)  (j < i),   P_ij = (q_i . k_j) e^(G_i - G_j)  (j <= i)
// the chunk's residuals r (u = beta r) solve (I + M diag(beta)) r = v - e^G S k,
// so the kernel writes T = (I + M diag(beta))^-1 (forward substitution in fp32,
// one column per thread), P, and the per-token factors (DeltaScal). k and q are
// written as fp16 rows scaled by a power of two (exact for every element
// within 2^14 of the row's largest), T as two fp16 pieces and P as one (two for
// the backward pass), each row under its own power-of-two scale. G is summed
// in fp64 and kept as two floats: differences of G stay exact to fp32 even
// after a token with a decay of e^-100 (log decays are cut there: the factor is
// below the smallest fp32 either way).
//
// One CTA takes a chunk of a key head and two of its value heads: k k^T and
// q k^T (fp16 MMAs) are shared by the heads.
#include "ssm_delta.cuh"

namespace ssm {

namespace {

constexpr int kC = kDeltaChunk;
constexpr int kThreads = 128;
constexpr int kHeads = 2;        // value heads per CTA
constexpr int kLs = kC + 4;      // row stride (floats) of the fp32 matrices
constexpr float kMinLogDecay = -100.f;

// 8 bf16 values of a unit -> fp32
__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(u[i]);
    f[2 * i + 1] = bf16_hi(u[i]);
  }
}

template <int N>
struct PrepSmem {
  static constexpr int kTile = kC * N * 2;
  static constexpr int kA = 2 * kTile > 4 * kDeltaTile ? 2 * kTile : 4 * kDeltaTile;
  static constexpr int kL = kHeads * kC * kLs * 4;
  static constexpr int kScal = kHeads * kDeltaScalBytes;
  static constexpr int kTok = 4 * kC * 4;
  static constexpr int kBytes = kA + kL + kScal + kTok + 64;
};

template <int N, bool BWD>
__global__ void __launch_bounds__(kThreads) delta_prep_kernel(const DeltaChunkParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  using Sm = PrepSmem<N>;
  constexpr int RB = N * 2;        // bytes of a k/q row
  constexpr int LPR = N / 8;       // lanes (16-byte units) per row
  constexpr int RPW = 32 / LPR;    // rows per warp and step
  unsigned char* tiles = smem;
  float* Lm = reinterpret_cast<float*>(smem + Sm::kA);
  float* scal = reinterpret_cast<float*>(smem + Sm::kA + Sm::kL);
  float* tok = reinterpret_cast<float*>(smem + Sm::kA + Sm::kL + Sm::kScal);  // kmul qmul kn qn
  double* carry = reinterpret_cast<double*>(smem + Sm::kA + Sm::kL + Sm::kScal + Sm::kTok);
  const DeltaParams& d = p.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, b = blockIdx.z;
  const int rep = d.nheads / d.nkheads, subs = (rep + kHeads - 1) / kHeads;
  const int kh = blockIdx.y / subs, sub = blockIdx.y - kh * subs;
  const int64_t t0 = (int64_t)c * kC;
  const int valid = (int)min((int64_t)kC, d.seqlen - t0);
  const size_t bc = (size_t)b * p.nchunks + c;

  // ---- k and q rows: largest magnitude, length, fp16 rows
  unsigned char* kq_out = p.ws_kq + (bc * d.nkheads + kh) * (size_t)(2 * Sm::kTile);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint16_t* src = static_cast<const uint16_t*>(w ? d.q : d.k);
#pragma unroll
    for (int it = 0; it < kC / (4 * RPW); ++it) {
      const int row = it * 4 * RPW + warp * RPW + lane / LPR, u = lane % LPR;
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (row < valid)
        raw = *reinterpret_cast<const uint4*>(
            src + (((size_t)b * d.seqlen + t0 + row) * d.nkheads + kh) * N + u * 8);
      float f[8];
      unpack8(raw, f);
      float m = 0.f, ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m = fmaxf(m, fabsf(f[i]));
        ss = fmaf(f[i], f[i], ss);
      }
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
      }
      // s = 2^-e brings the largest magnitude to [1, 2); its inverse goes into kmul
      uint32_t e = exponent_of(m);
      e = e < 1u ? 1u : (e > 253u ? 253u : e);
      const float s = __uint_as_float((254u - e) << 23), inv = __uint_as_float(e << 23);
      uint4 out;
      uint32_t* o4 = &out.x;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o4[i] = h2_bits(__floats2half2_rn(f[2 * i] * s, f[2 * i + 1] * s));
      const uint32_t at = swz<RB>(row, u);
      *reinterpret_cast<uint4*>(tiles + w * Sm::kTile + at) = out;
      if (sub == 0) *reinterpret_cast<uint4*>(kq_out + w * Sm::kTile + at) = out;
      if (u == 0) {
        const float len = d.qk_norm ? 1.f / sqrtf(ss + kDeltaQkEps) : 1.f;
        const float sc = w ? d.scale : 1.f;
        tok[w * kC + row] = len * inv * sc;
        tok[(2 + w) * kC + row] = len * sc;
      }
    }
  }

  // ---- gates: two warps per head, one token per thread
  const int hl = warp >> 1;                    // head of this half of the CTA
  const int h = kh * rep + sub * kHeads + hl;  // may lie past the group's end
  const int nh = min(kHeads, rep - sub * kHeads);
  {
    const int i = tid & 63;
    double g = 0.0;
    float beta = 0.f;
    if (hl < nh && i < valid) {
      const size_t at = ((size_t)b * d.seqlen + t0 + i) * d.nheads + h;
      const float raw = bf16_to_f32(static_cast<const uint16_t*>(d.dt)[at]) +
                        (d.dt_bias ? d.dt_bias[h] : 0.f);
      float gf = delta_step_size(raw, d.softplus) * d.A[h];
      gf = gf < kMinLogDecay ? kMinLogDecay : gf;
      g = (double)gf * 1.4426950408889634;  // log2 units
      beta = delta_beta(bf16_to_f32(static_cast<const uint16_t*>(d.beta)[at]), d.beta_sigmoid);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, g, o);
      if (lane >= o) g += up;
    }
    if ((warp & 1) == 0 && lane == 31) carry[hl] = g;
    __syncthreads();
    if (warp & 1) g += carry[hl];
    float* sc = scal + hl * (kDeltaScalBytes / 4);
    const float hi = (float)g;
    sc[kScGhi * kC + i] = hi;
    sc[kScGlo * kC + i] = (float)(g - (double)hi);
    sc[kScBeta * kC + i] = beta;
    __syncthreads();
    const float ehi = sc[kScGhi * kC + kC - 1], elo = sc[kScGlo * kC + kC - 1];
    const float lo = sc[kScGlo * kC + i];
    const float D = ex2_approx(hi + lo), E = ex2_approx((ehi - hi) + (elo - lo));
    sc[kScSk * kC + i] = D * tok[i];
    sc[kScKend * kC + i] = tok[i] * E;
    sc[kScK * kC + i] = tok[i];
    sc[kScSq * kC + i] = D * tok[kC + i];
    sc[kScEnd * kC + i] = ex2_approx(ehi + elo);
    sc[kScKn * kC + i] = tok[2 * kC + i];
    sc[kScQn * kC + i] = tok[3 * kC + i];
  }

  // ---- k k^T and q k^T: warp w takes rows 16 w .. 16 w + 15, columns up to them
  float kk[8][4] = {}, qk[8][4] = {};
  {
    const uint32_t ks = smem_u32(tiles), qs = ks + Sm::kTile;
#pragma unroll
    for (int kt = 0; kt < N / 16; ++kt) {
      uint32_t ak[4], aq[4];
      const int ar = warp * 16 + (lane & 15), au = 2 * kt + (lane >> 4);
      ldsm4(ak, ks + swz<RB>(ar, au));
      ldsm4(aq, qs + swz<RB>(ar, au));
#pragma unroll
      for (int jp = 0; jp < 4; ++jp) {
        if (jp > warp) continue;
        uint32_t bb[4];
        ldsm4(bb, ks + swz<RB>(16 * jp + (lane & 7) + ((lane & 16) >> 1), 2 * kt + ((lane >> 3) & 1)));
        mma_f16(kk[2 * jp], ak, bb[0], bb[1]);
        mma_f16(kk[2 * jp + 1], ak, bb[2], bb[3]);
        mma_f16(qk[2 * jp], aq, bb[0], bb[1]);
        mma_f16(qk[2 * jp + 1], aq, bb[2], bb[3]);
      }
    }
  }
  __syncthreads();  // the k/q tiles are free: P is staged over them

  const int r0 = warp * 16 + (lane >> 2), r1 = r0 + 8;
#pragma unroll
  for (int x = 0; x < kHeads; ++x) {
    if (x >= nh) break;
    float* sc = scal + x * (kDeltaScalBytes / 4);
    float* L = Lm + x * kC * kLs;
    unsigned char* pst = tiles + x * 2 * kDeltaTile;
    const float gh0 = sc[kScGhi * kC + r0], gl0 = sc[kScGlo * kC + r0];
    const float gh1 = sc[kScGhi * kC + r1], gl1 = sc[kScGlo * kC + r1];
    const float km0 = tok[r0], km1 = tok[r1];
    float pv[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q) pv[j][q] = 0.f;
      if (j > 2 * warp + 1) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = 8 * j + 2 * (lane & 3) + (q & 1), row = q < 2 ? r0 : r1;
        const float gm = ex2_approx(((q < 2 ? gh0 : gh1) - sc[kScGhi * kC + col]) +
                                    ((q < 2 ? gl0 : gl1) - sc[kScGlo * kC + col]));
        if (col <= row) pv[j][q] = qk[j][q] * gm;
        L[row * kLs + col] = col < row ? kk[j][q] * gm * (q < 2 ? km0 : km1) * tok[col] *
                                             sc[kScBeta * kC + col]
                                       : 0.f;
      }
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
      const uint32_t a0 = swz<128>(r0, j) + (lane & 3) * 4, a1 = swz<128>(r1, j) + (lane & 3) * 4;
      *reinterpret_cast<uint32_t*>(pst + a0) = hi0;
      *reinterpret_cast<uint32_t*>(pst + a1) = hi1;
      if (BWD) {
        *reinterpret_cast<uint32_t*>(pst + kDeltaTile + a0) = lo0;
        *reinterpret_cast<uint32_t*>(pst + kDeltaTile + a1) = lo1;
      }
    }
    if ((lane & 3) == 0) {
      sc[kScP * kC + r0] = tok[kC + r0] * s0.inv;
      sc[kScP * kC + r1] = tok[kC + r1] * s1.inv;
    }
  }
  __syncthreads();

  // ---- T = (I + L)^-1: column `col` of head hl per thread
  const int col = tid & 63;
  float xs[kC];
  if (hl < nh) {
    const float* L = Lm + hl * kC * kLs;
    // columns 32.. are zero above row 32: the second warp starts there
    if ((warp & 1) == 0) {
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        float acc = i == col ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; j += 4) {
          const float4 l = *reinterpret_cast<const float4*>(L + i * kLs + j);
          acc = fmaf(-l.x, xs[j], acc);
          if (j + 1 < i) acc = fmaf(-l.y, xs[j + 1], acc);
          if (j + 2 < i) acc = fmaf(-l.z, xs[j + 2], acc);
          if (j + 3 < i) acc = fmaf(-l.w, xs[j + 3], acc);
        }
        xs[i] = acc;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) xs[i] = 0.f;
#pragma unroll
      for (int i = 32; i < kC; ++i) {
        float acc = i == col ? 1.f : 0.f;
#pragma unroll
        for (int j = 32; j < i; j += 4) {
          const float4 l = *reinterpret_cast<const float4*>(L + i * kLs + j);
          acc = fmaf(-l.x, xs[j], acc);
          if (j + 1 < i) acc = fmaf(-l.y, xs[j + 1], acc);
          if (j + 2 < i) acc = fmaf(-l.z, xs[j + 2], acc);
          if (j + 3 < i) acc = fmaf(-l.w, xs[j + 3], acc);
        }
        xs[i] = acc;
      }
    }
  }
  __syncthreads();
  if (hl < nh) {
    float* L = Lm + hl * kC * kLs;
#pragma unroll
    for (int i = 0; i < kC; ++i) L[i * kLs + col] = xs[i];
  }
  __syncthreads();
  if (hl < nh) {  // thread: one row, its scale and its two pieces
    const int row = tid & 63;
    const float* L = Lm + hl * kC * kLs + row * kLs;
    float* sc = scal + hl * (kDeltaScalBytes / 4);
    unsigned char* out = p.ws_head + (bc * d.nheads + h) * (size_t)p.head_bytes + kDeltaScalBytes;
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < kC; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(L + j);
      m = fmaxf(fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
    }
    const RowScale s = row_scale(exponent_of(m));
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      uint4 hi, lo;
      const float4 v0 = *reinterpret_cast<const float4*>(L + u * 8);
      const float4 v1 = *reinterpret_cast<const float4*>(L + u * 8 + 4);
      split2(v0.x, v0.y, s.s, hi.x, lo.x);
      split2(v0.z, v0.w, s.s, hi.y, lo.y);
      split2(v1.x, v1.y, s.s, hi.z, lo.z);
      split2(v1.z, v1.w, s.s, hi.w, lo.w);
      const uint32_t at = swz<128>(row, u);
      *reinterpret_cast<uint4*>(out + at) = hi;
      *reinterpret_cast<uint4*>(out + kDeltaTile + at) = lo;
    }
    sc[kScU * kC + row] = sc[kScBeta * kC + row] * s.inv;
    sc[kScT * kC + row] = s.inv;
  }
  __syncthreads();

  // ---- P and the factors
  constexpr int kPBytes = (BWD ? 2 : 1) * kDeltaTile;
  for (int x = 0; x < nh; ++x) {
    unsigned char* out = p.ws_head +
                         (bc * d.nheads + kh * rep + sub * kHeads + x) * (size_t)p.head_bytes;
    const uint4* ps = reinterpret_cast<const uint4*>(tiles + x * 2 * kDeltaTile);
    uint4* po = reinterpret_cast<uint4*>(out + kDeltaScalBytes + 2 * kDeltaTile);
    for (int i = tid; i < kPBytes / 16; i += kThreads) po[i] = ps[i];
    const uint4* ss = reinterpret_cast<const uint4*>(scal + x * (kDeltaScalBytes / 4));
    for (int i = tid; i < (kScQn + 1) * kC * 4 / 16; i += kThreads)
      reinterpret_cast<uint4*>(out)[i] = ss[i];
  }
}

template <int N, bool BWD>
cudaError_t launch(const DeltaChunkParams& p, cudaStream_t stream) {
  auto* kern = delta_prep_kernel<N, BWD>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             PrepSmem<N>::kBytes);
  if (e != cudaSuccess) return e;
  const int rep = p.d.nheads / p.d.nkheads, subs = (rep + kHeads - 1) / kHeads;
  kern<<<dim3(p.nchunks, p.d.nkheads * subs, p.d.batch), kThreads, PrepSmem<N>::kBytes, stream>>>(
      p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_prep(const DeltaChunkParams& p, bool bwd, cudaStream_t stream) {
  if (p.d.dstate == 64) return bwd ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  return bwd ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
}

}  // namespace ssm
