// ssm_delta_step.cu -- sm_100a kernel of the gated delta rule, token by token:
// the decode step (one token on a carried state) and the scan of short or
// fp32 sequences, any headdim.
//
// Per batch b, head h, row p of the head's state (fp32, dstate wide):
//   S <- a S,  u = beta (v[p] - S . k),  S <- S + u k,  y[p] = S . q
// Both products are taken on the decayed state in one pass, S . q after the
// update being S . q + u (k . q). Rows are independent: eight lanes hold one
// row (dstate / 8 values each, 16-byte accesses of which the eight lanes take
// 128 contiguous bytes), so a warp holds four rows and the dot products need
// three shuffles. k and q come from L1 after their first use; their lengths
// are summed per row beside the two products.
//
// Bound, one token: the state's read and write (268 MB for 64 x 64 heads x 64
// x 128, bf16 io: 44.8 us = 6.0 TB/s; a variant with the next token's operands
// in registers, half the warps per SM, took 71 us). Bound, many tokens: the
// chain of one token (three shuffles, u and the update); operands are loaded
// up to 16 tokens ahead, the gates (exp, log1p, sigmoid) taken eight tokens at
// a time, one per lane.
#include "ssm_delta.cuh"

namespace ssm {

namespace {

constexpr int kLanes = 8;  // lanes per state row

// Four values of a lane as they lie in memory.
template <typename IOT>
struct Quad;
template <>
struct Quad<float> {
  float4 w;
  __device__ void load(const float* p) { w = *reinterpret_cast<const float4*>(p); }
  __device__ void get(float2 (&f)[2]) const {
    f[0] = make_float2(w.x, w.y);
    f[1] = make_float2(w.z, w.w);
  }
};
template <>
struct Quad<uint16_t> {
  uint2 w;
  __device__ void load(const uint16_t* p) { w = *reinterpret_cast<const uint2*>(p); }
  __device__ void get(float2 (&f)[2]) const {
    f[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
    f[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
  }
};

// One token on the lane's part of a row; returns y[p] (all eight lanes).
template <typename IOT, int U>
__device__ __forceinline__ float one_token(float2 (&s)[2 * U], const Quad<IOT> (&k)[U],
                                           const Quad<IOT> (&q)[U], float v, float a, float beta,
                                           int qk_norm, float scale) {
  float2 sk = make_float2(0.f, 0.f), sq = sk, kq = sk, kk = sk, qq = sk;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float2 kf[2], qf[2];
    k[i].get(kf);
    q[i].get(qf);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      sk = fma2(s[2 * i + j], kf[j], sk);
      sq = fma2(s[2 * i + j], qf[j], sq);
      kq = fma2(kf[j], qf[j], kq);
      kk = fma2(kf[j], kf[j], kk);
      qq = fma2(qf[j], qf[j], qq);
    }
  }
  float r[5] = {sk.x + sk.y, sq.x + sq.y, kq.x + kq.y, kk.x + kk.y, qq.x + qq.y};
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 5; ++j) r[j] += __shfl_xor_sync(0xffffffffu, r[j], o);
  }
  float kr = 1.f, qr = scale;
  if (qk_norm) {
    kr = rsqrtf(r[3] + kDeltaQkEps);
    qr = scale * rsqrtf(r[4] + kDeltaQkEps);
  }
  const float u = beta * (v - a * kr * r[0]);
  const float w = u * kr;  // weight of the raw k
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float2 kf[2];
    k[i].get(kf);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      s[2 * i + j] = fma2(make_float2(w, w), kf[j], mul2(make_float2(a, a), s[2 * i + j]));
  }
  return qr * fmaf(a, r[1], w * r[2]);
}

// ONE: a single token (fewer registers, more state bytes in flight). Otherwise
// D tokens' operands are held ahead.
template <typename IOT, int N, bool ONE>
__global__ void __launch_bounds__(256) delta_step_kernel(const DeltaParams p) {
  using IO = Io<IOT>;
  constexpr int U = N / 32;  // units of four values per lane
  constexpr int D = ONE ? 1 : (int)(sizeof(IOT) == 2 ? 16 : 8) / U;
  const int l8 = threadIdx.x & (kLanes - 1);
  const int64_t rows = (int64_t)p.batch * p.nheads * p.headdim;
  const int64_t row_raw = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / kLanes;
  if (row_raw - ((threadIdx.x & 31) / kLanes) >= rows) return;  // warp-uniform
  const bool live = row_raw < rows;
  const uint32_t row = (uint32_t)(live ? row_raw : rows - 1);  // at most 2^31 rows
  const uint32_t bh = row / (uint32_t)p.headdim;
  const int pp = (int)(row - bh * (uint32_t)p.headdim);
  const uint32_t b = bh / (uint32_t)p.nheads;
  const int h = (int)(bh - b * (uint32_t)p.nheads);
  const int kh = h / (p.nheads / p.nkheads);
  const size_t L = ONE ? 1 : (size_t)p.seqlen;

  const IOT* q = static_cast<const IOT*>(p.q) + (b * L * p.nkheads + kh) * N + l8 * 4;
  const IOT* k = static_cast<const IOT*>(p.k) + (b * L * p.nkheads + kh) * N + l8 * 4;
  const IOT* v = static_cast<const IOT*>(p.v) + (b * L * p.nheads + h) * p.headdim + pp;
  const IOT* dt = static_cast<const IOT*>(p.dt) + b * L * p.nheads + h;  // token 0's
  const IOT* be = static_cast<const IOT*>(p.beta) + b * L * p.nheads + h;
  IOT* y = static_cast<IOT*>(p.y) + (b * L * p.nheads + h) * p.headdim + pp;
  const size_t qs = (size_t)p.nkheads * N, vs = (size_t)p.nheads * p.headdim;

  float2 s[2 * U];
  if (p.h0) {
    const float4* src = reinterpret_cast<const float4*>(p.h0 + (size_t)row * N) + l8;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float4 f = src[i * kLanes];
      s[2 * i] = make_float2(f.x, f.y);
      s[2 * i + 1] = make_float2(f.z, f.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * U; ++i) s[i] = make_float2(0.f, 0.f);
  }
  const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;

  Quad<IOT> kn[D][U], qn[D][U];
  float vn[D];
  auto fetch = [&](int j) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      kn[j][i].load(k + i * kLanes * 4);
      qn[j][i].load(q + i * kLanes * 4);
    }
    vn[j] = IO::load(v);
    k += qs; q += qs; v += vs;
  };
  // the gates of eight tokens at a time, one token per lane of the row
  float raw_dt = 0.f, raw_be = 0.f, a8 = 0.f, b8 = 0.f;
  auto fetch_gates = [&](size_t t) {
    const size_t at = (t + l8 < L ? t + l8 : L - 1) * p.nheads;
    raw_dt = IO::load(dt + at);
    raw_be = IO::load(be + at);
  };
  if (L > 0) fetch_gates(0);
#pragma unroll
  for (int j = 0; j < D; ++j)
    if (j < (int64_t)L) fetch(j);
  for (size_t t0 = 0; t0 < L; t0 += D) {
#pragma unroll
    for (int j = 0; j < D; ++j) {
      if (t0 + j >= L) break;
      const int j8 = (int)((t0 + j) & (kLanes - 1));
      if (j8 == 0) {
        a8 = expf(delta_step_size(raw_dt + bias, p.softplus) * A);
        b8 = delta_beta(raw_be, p.beta_sigmoid);
        if (!ONE && t0 + j + kLanes < L) fetch_gates(t0 + j + kLanes);
      }
      const float a = __shfl_sync(0xffffffffu, a8, j8, kLanes);
      const float beta = __shfl_sync(0xffffffffu, b8, j8, kLanes);
      const float out = one_token<IOT, U>(s, kn[j], qn[j], vn[j], a, beta, p.qk_norm, p.scale);
      if (!ONE && t0 + j + D < L) fetch(j);
      if (p.y && live && l8 == 0) IO::store(y, out);
      y += vs;
    }
  }
  if (p.h_last && live) {
    float4* dst = reinterpret_cast<float4*>(p.h_last + (size_t)row * N) + l8;
#pragma unroll
    for (int i = 0; i < U; ++i)
      dst[i * kLanes] = make_float4(s[2 * i].x, s[2 * i].y, s[2 * i + 1].x, s[2 * i + 1].y);
  }
}

template <typename IOT, int N>
cudaError_t launch_n(const DeltaParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.batch * p.nheads * p.headdim;
  // small problems spread over the SMs in smaller blocks
  const int threads = rows * kLanes < 148 * 256 ? 64 : 256;
  const unsigned blocks = (unsigned)((rows * kLanes + threads - 1) / threads);
  if (p.seqlen == 1)
    delta_step_kernel<IOT, N, true><<<blocks, threads, 0, stream>>>(p);
  else
    delta_step_kernel<IOT, N, false><<<blocks, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename IOT>
cudaError_t launch_io(const DeltaParams& p, cudaStream_t stream) {
  switch (p.dstate) {
    case 32: return launch_n<IOT, 32>(p, stream);
    case 64: return launch_n<IOT, 64>(p, stream);
    case 128: return launch_n<IOT, 128>(p, stream);
    case 256: return launch_n<IOT, 256>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

bool delta_step_dstate_supported(int dstate) {
  return dstate == 32 || dstate == 64 || dstate == 128 || dstate == 256;
}

cudaError_t launch_delta_step(const DeltaParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_io<uint16_t>(p, stream) : launch_io<float>(p, stream);
}

}  // namespace ssm
