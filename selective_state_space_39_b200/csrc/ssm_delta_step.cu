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
// x 128). Bound, many tokens: the chain of one token (two shuffle reductions
// and the update); the next token's operands are loaded one token ahead.
#include "ssm_delta.cuh"

namespace ssm {

namespace {

constexpr int kLanes = 8;  // lanes per state row

template <typename IOT, int N>
__global__ void __launch_bounds__(256) delta_step_kernel(const DeltaParams p) {
  using IO = Io<IOT>;
  constexpr int U = N / 32;  // units of four values per lane
  const int l8 = threadIdx.x & (kLanes - 1);
  const int64_t rows = (int64_t)p.batch * p.nheads * p.headdim;
  const int64_t row_raw = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / kLanes;
  if (row_raw - ((threadIdx.x & 31) / kLanes) >= rows) return;  // warp-uniform
  const bool live = row_raw < rows;
  const int64_t row = live ? row_raw : rows - 1;
  const uint32_t bh = (uint32_t)(row / p.headdim);
  const int pp = (int)(row - (int64_t)bh * p.headdim);
  const uint32_t b = bh / (uint32_t)p.nheads;
  const int h = (int)(bh - b * (uint32_t)p.nheads);
  const int kh = h / (p.nheads / p.nkheads);
  const size_t L = (size_t)p.seqlen;

  const IOT* q = static_cast<const IOT*>(p.q) + (b * L * p.nkheads + kh) * N + l8 * 4;
  const IOT* k = static_cast<const IOT*>(p.k) + (b * L * p.nkheads + kh) * N + l8 * 4;
  const IOT* v = static_cast<const IOT*>(p.v) + (b * L * p.nheads + h) * p.headdim + pp;
  const IOT* dt = static_cast<const IOT*>(p.dt) + b * L * p.nheads + h;
  const IOT* be = static_cast<const IOT*>(p.beta) + b * L * p.nheads + h;
  IOT* y = static_cast<IOT*>(p.y) + (b * L * p.nheads + h) * p.headdim + pp;
  const size_t qs = (size_t)p.nkheads * N, vs = (size_t)p.nheads * p.headdim;

  float4 s[U];
  if (p.h0) {
    const float4* src = reinterpret_cast<const float4*>(p.h0 + row * N) + l8;
#pragma unroll
    for (int i = 0; i < U; ++i) s[i] = src[i * kLanes];
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;

  float4 kn[U], qn[U];
  float vn = 0.f, dn = 0.f, bn = 0.f;
  auto fetch = [&]() {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      kn[i] = IO::load4(k + i * kLanes * 4);
      qn[i] = IO::load4(q + i * kLanes * 4);
    }
    vn = IO::load(v);
    dn = IO::load(dt);
    bn = IO::load(be);
    k += qs; q += qs; v += vs; dt += p.nheads; be += p.nheads;
  };
  if (L > 0) fetch();
  for (size_t t = 0; t < L; ++t) {
    float4 kc[U], qc[U];
#pragma unroll
    for (int i = 0; i < U; ++i) { kc[i] = kn[i]; qc[i] = qn[i]; }
    const float vc = vn;
    const float a = expf(delta_step_size(dn + bias, p.softplus) * A);
    const float beta = delta_beta(bn, p.beta_sigmoid);
    if (t + 1 < L) fetch();
    float r[5] = {0.f, 0.f, 0.f, 0.f, 0.f};  // S.k, S.q, k.q, k.k, q.q
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float ss[4] = {s[i].x, s[i].y, s[i].z, s[i].w};
      const float kk[4] = {kc[i].x, kc[i].y, kc[i].z, kc[i].w};
      const float qq[4] = {qc[i].x, qc[i].y, qc[i].z, qc[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[0] = fmaf(ss[j], kk[j], r[0]);
        r[1] = fmaf(ss[j], qq[j], r[1]);
        r[2] = fmaf(kk[j], qq[j], r[2]);
        r[3] = fmaf(kk[j], kk[j], r[3]);
        r[4] = fmaf(qq[j], qq[j], r[4]);
      }
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) {
#pragma unroll
      for (int j = 0; j < 5; ++j) r[j] += __shfl_xor_sync(0xffffffffu, r[j], o);
    }
    float kr = 1.f, qr = p.scale;
    if (p.qk_norm) {
      kr = 1.f / sqrtf(r[3] + kDeltaQkEps);
      qr = p.scale / sqrtf(r[4] + kDeltaQkEps);
    }
    const float u = beta * (vc - a * kr * r[0]);
    const float w = u * kr;  // weight of the raw k
#pragma unroll
    for (int i = 0; i < U; ++i) {
      s[i].x = fmaf(w, kc[i].x, a * s[i].x);
      s[i].y = fmaf(w, kc[i].y, a * s[i].y);
      s[i].z = fmaf(w, kc[i].z, a * s[i].z);
      s[i].w = fmaf(w, kc[i].w, a * s[i].w);
    }
    if (p.y && live && l8 == 0) IO::store(y, qr * fmaf(a, r[1], w * r[2]));
    y += vs;
  }
  if (p.h_last && live) {
    float4* dst = reinterpret_cast<float4*>(p.h_last + row * N) + l8;
#pragma unroll
    for (int i = 0; i < U; ++i) dst[i * kLanes] = s[i];
  }
}

template <typename IOT>
cudaError_t launch_io(const DeltaParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.batch * p.nheads * p.headdim;
  // small problems spread over the SMs in smaller blocks
  const int threads = rows * kLanes < 148 * 256 ? 64 : 256;
  const unsigned blocks = (unsigned)((rows * kLanes + threads - 1) / threads);
  switch (p.dstate) {
    case 32: delta_step_kernel<IOT, 32><<<blocks, threads, 0, stream>>>(p); break;
    case 64: delta_step_kernel<IOT, 64><<<blocks, threads, 0, stream>>>(p); break;
    case 128: delta_step_kernel<IOT, 128><<<blocks, threads, 0, stream>>>(p); break;
    case 256: delta_step_kernel<IOT, 256><<<blocks, threads, 0, stream>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

bool delta_step_dstate_supported(int dstate) {
  return dstate == 32 || dstate == 64 || dstate == 128 || dstate == 256;
}

cudaError_t launch_delta_step(const DeltaParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_io<uint16_t>(p, stream) : launch_io<float>(p, stream);
}

}  // namespace ssm
