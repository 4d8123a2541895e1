// ssm_norm.cu -- sm_100a kernels of the norm before and after a block: RMSNorm
// over groups of a row, with the residual sum before it and the SiLU gate on
// either side of it fused in.
//
//   h = residual + residual_scale x   (or h = x)
//   u = h SiLU(z)  (gate first)  or  u = h
//   n = u / sqrt(mean(u^2) + eps),  y = n w  (gate last: y = n w SiLU(z))
// and, with t = dn w, dn = dy (gate last: dy SiLU(z)):
//   du = (t - n mean(t n)) / sqrt(mean(u^2) + eps),  dw = sum over rows of dn n
//
// One pass over the data: a group of T threads holds a row group in registers
// (up to kMaxVecs units of 16 bytes of io per thread; longer rows are read
// twice), sums the squares (backward: and t u) in fp32 by shuffles, and writes
// the results. T is the power of two that leaves a thread about two units, so
// rows of one head's width take 8 or 16 lanes and a warp holds several. dw is
// summed in registers over the rows a block takes, in shared memory over its
// row groups and over the blocks by a second kernel, always in the same order.
//
// Bound: memory traffic (forward: x, z, residual in, y, h out; backward: h,
// dy, z, dh in, dx, dz, dresidual out).
#include <algorithm>

#include "ssm_device.cuh"
#include "ssm_norm_internal.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = Io<T>::load(p);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(u[i]);
      f[2 * i + 1] = bf16_hi(u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    Io<T>::store(p, f[0]);
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  }
}

// sigmoid: MUFU approximations for bf16 io (2^-22 relative), exact functions for fp32
template <typename IOT>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(IOT) == 2)
    return rcp_approx(1.f + ex2_approx(-z * kLog2e));
  else
    return 1.f / (1.f + expf(-z));
}

// Sums over the T threads of a row group (T a power of two; above a warp
// through shared memory, one slot per warp and value).
template <int K>
__device__ __forceinline__ void group_sum(float (&v)[K], int T, float* sh) {
  const int top = T < 32 ? T : 32;
  for (int o = 1; o < top; o <<= 1) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if (T > 32) {
    const int warp = threadIdx.x >> 5, per = T >> 5, first = warp / per * per;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < K; ++i) sh[warp * K + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float s = 0.f;
      for (int q = 0; q < per; ++q) s += sh[(first + q) * K + i];
      v[i] = s;
    }
  }
}

template <typename IOT, typename RT, int V, int M, bool FIT>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormParams p, int T) {
  __shared__ float sh[32];
  const int per_block = blockDim.x / T, t = threadIdx.x % T;
  const int64_t total = p.rows * p.groups;
  const int64_t r_raw = (int64_t)blockIdx.x * per_block + threadIdx.x / T;
  const bool live = r_raw < total;
  const int64_t r = live ? r_raw : total - 1;
  const size_t base = (size_t)r * p.width;  // rows are contiguous, so their groups are too
  const int wbase = (int)(r % p.groups) * p.width;
  const IOT* x = static_cast<const IOT*>(p.x) + base;
  const RT* res = p.residual ? static_cast<const RT*>(p.residual) + base : nullptr;
  const IOT* z = p.gate ? static_cast<const IOT*>(p.z) + base : nullptr;

  auto value = [&](int at, float(&u)[V], float(&g)[V], bool store) {
    load_vec<IOT, V>(x + at, u);
    if (res) {
      float q[V];
      load_vec<RT, V>(res + at, q);
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] = fmaf(p.residual_scale, u[i], q[i]);
      if (store && live) store_vec<RT, V>(static_cast<RT*>(p.h_out) + base + at, u);
    }
    if (p.gate) {
      load_vec<IOT, V>(z + at, g);
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] *= sigmoid<IOT>(g[i]);
      if (p.gate == kGateFirst) {
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] *= g[i];
      }
    }
  };

  float u[M][V], g[M][V];
  float ss[1] = {0.f};
  if (FIT) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int at = (m * T + t) * V;
      if (at >= p.width) break;
      value(at, u[m], g[m], true);
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if ((m * T + t) * V >= p.width) break;
#pragma unroll
      for (int i = 0; i < V; ++i) ss[0] = fmaf(u[m][i], u[m][i], ss[0]);
    }
  } else {
    for (int at = t * V; at < p.width; at += T * V) {
      value(at, u[0], g[0], false);
#pragma unroll
      for (int i = 0; i < V; ++i) ss[0] = fmaf(u[0][i], u[0][i], ss[0]);
    }
  }
  group_sum<1>(ss, T, sh);
  const float inv = 1.f / sqrtf(ss[0] / (float)p.width + p.eps);

  auto finish = [&](int at, float(&uu)[V], const float(&gg)[V]) {
    float w[V];
    load_vec<float, V>(p.w + wbase + at, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      uu[i] = uu[i] * inv * w[i];
      if (p.gate == kGateLast) uu[i] *= gg[i];
    }
    if (live) store_vec<IOT, V>(static_cast<IOT*>(p.y) + base + at, uu);
  };
  if (FIT) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int at = (m * T + t) * V;
      if (at >= p.width) break;
      finish(at, u[m], g[m]);
    }
  } else {
    for (int at = t * V; at < p.width; at += T * V) {
      value(at, u[0], g[0], true);
      finish(at, u[0], g[0]);
    }
  }
}

// Grid: (slices, groups). A block takes rows slice, slice + slices, ... of its
// row slots in turn, so that a thread's columns stay the same.
template <typename IOT, typename RT, int V, int M, bool FIT>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormParams p, int T) {
  extern __shared__ float dws[];  // dw sums of the block's row groups
  __shared__ float sh[64];
  const int per_block = blockDim.x / T, t = threadIdx.x % T, slot = threadIdx.x / T;
  const int group = blockIdx.y, wbase = group * p.width;
  float acc[FIT ? M : 1][V];
#pragma unroll
  for (int m = 0; m < (FIT ? M : 1); ++m)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[m][i] = 0.f;
  if (!FIT && p.dw)
    for (int i = threadIdx.x; i < p.width; i += blockDim.x) dws[i] = 0.f;

  const int64_t step = (int64_t)gridDim.x * per_block;
  for (int64_t r0 = (int64_t)blockIdx.x * per_block; r0 < p.rows; r0 += step) {
    const bool live = r0 + slot < p.rows;
    const int64_t r = live ? r0 + slot : p.rows - 1;
    const size_t base = ((size_t)r * p.groups + group) * p.width;
    const RT* h = static_cast<const RT*>(p.h) + base;
    const IOT* dy = static_cast<const IOT*>(p.dy) + base;
    const IOT* z = p.gate ? static_cast<const IOT*>(p.z) + base : nullptr;

    // u, t = dn w; sums of u^2 and t u
    float ss[2] = {0.f, 0.f};
    float hv[M][V], dv[M][V], zv[M][V];
    auto sums = [&](int at, const float(&hh)[V], const float(&dd)[V], const float(&zz)[V]) {
      float w[V];
      load_vec<float, V>(p.w + wbase + at, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float u = hh[i], dn = dd[i];
        if (p.gate) {
          const float g = zz[i] * sigmoid<IOT>(zz[i]);
          if (p.gate == kGateFirst) u *= g; else dn *= g;
        }
        ss[0] = fmaf(u, u, ss[0]);
        ss[1] = fmaf(dn * w[i], u, ss[1]);
      }
    };
    auto fetch = [&](int at, float(&hh)[V], float(&dd)[V], float(&zz)[V]) {
      load_vec<RT, V>(h + at, hh);
      load_vec<IOT, V>(dy + at, dd);
      if (p.gate) load_vec<IOT, V>(z + at, zz);
    };
    if (FIT) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int at = (m * T + t) * V;
        if (at >= p.width) break;
        fetch(at, hv[m], dv[m], zv[m]);
      }
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int at = (m * T + t) * V;
        if (at >= p.width) break;
        sums(at, hv[m], dv[m], zv[m]);
      }
    } else {
      for (int at = t * V; at < p.width; at += T * V) {
        fetch(at, hv[0], dv[0], zv[0]);
        sums(at, hv[0], dv[0], zv[0]);
      }
    }
    group_sum<2>(ss, T, sh);
    const float inv = 1.f / sqrtf(ss[0] / (float)p.width + p.eps);
    const float c = ss[1] * inv / (float)p.width;  // mean(t n)

    auto finish = [&](int at, const float(&hh)[V], const float(&dd)[V], const float(&zz)[V],
                      float(&sum)[V]) {
      float w[V], dh[V], dzv[V], extra[V];
      load_vec<float, V>(p.w + wbase + at, w);
      if (p.dh) load_vec<RT, V>(static_cast<const RT*>(p.dh) + base + at, extra);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float sg = 0.f, g = 1.f;
        if (p.gate) {
          sg = sigmoid<IOT>(zz[i]);
          g = zz[i] * sg;
        }
        const float u = p.gate == kGateFirst ? hh[i] * g : hh[i];
        const float dn = p.gate == kGateLast ? dd[i] * g : dd[i];
        const float n = u * inv;
        const float du = inv * (dn * w[i] - n * c);
        if (live) sum[i] = fmaf(dn, n, sum[i]);
        const float dg = p.gate == kGateFirst ? du * hh[i] : dd[i] * n * w[i];
        dzv[i] = dg * sg * (1.f + zz[i] * (1.f - sg));
        dh[i] = p.gate == kGateFirst ? du * g : du;
        if (p.dh) dh[i] += extra[i];
      }
      if (!live) return;
      if (p.gate) store_vec<IOT, V>(static_cast<IOT*>(p.dz) + base + at, dzv);
      if (p.dresidual) store_vec<RT, V>(static_cast<RT*>(p.dresidual) + base + at, dh);
#pragma unroll
      for (int i = 0; i < V; ++i) dh[i] *= p.residual_scale;
      store_vec<IOT, V>(static_cast<IOT*>(p.dx) + base + at, dh);
    };
    if (FIT) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int at = (m * T + t) * V;
        if (at >= p.width) break;
        finish(at, hv[m], dv[m], zv[m], acc[m]);
      }
    } else {  // one row at a time (T = the block): the columns' sums live in shared memory
      for (int at = t * V; at < p.width; at += T * V) {
        fetch(at, hv[0], dv[0], zv[0]);
        float sum[V];
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = p.dw ? dws[at + i] : 0.f;
        finish(at, hv[0], dv[0], zv[0], sum);
        if (p.dw) {
#pragma unroll
          for (int i = 0; i < V; ++i) dws[at + i] = sum[i];
        }
      }
    }
  }
  if (!p.dw) return;
  float* out = p.ws + (size_t)blockIdx.x * p.dim + wbase;
  if (FIT) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int at = (m * T + t) * V;
      if (at >= p.width) break;
#pragma unroll
      for (int i = 0; i < V; ++i) dws[slot * p.width + at + i] = acc[m][i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.width; i += blockDim.x) {
    float s = 0.f;
    for (int q = 0; q < (FIT ? per_block : 1); ++q) s += dws[q * p.width + i];
    out[i] = s;
  }
}

// dw: 32 columns per block, the slices' sums by 8 warps in a fixed order.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* part, int slices, int dim,
                                                      float* dw) {
  __shared__ float sh[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < dim) {
#pragma unroll 4
    for (int i = warp; i < slices; i += 8) s += part[(size_t)i * dim + col];
  }
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < dim) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sh[i][lane];
    dw[col] = s;
  }
}

struct Shape {
  int V, T, M, threads;  // M units per thread; 0: the row is read twice
};
Shape shape(const NormParams& p, int types, bool vec, int max_m) {
  Shape s;
  s.V = vec ? (types == 2 ? 4 : 8) : 1;
  const int units = (p.width + s.V - 1) / s.V;
  s.T = 8;
  while (s.T < 512 && s.T * 2 < units) s.T *= 2;
  const int m = (units + s.T - 1) / s.T;
  s.M = m <= 1 ? 1 : m <= 2 ? 2 : m <= 4 ? 4 : m <= max_m ? max_m : 0;
  s.threads = std::max(s.T, kThreads);
  return s;
}

template <typename IOT, typename RT, int V>
cudaError_t fwd_m(const NormParams& p, const Shape& s, cudaStream_t stream) {
  const int64_t per = s.threads / s.T, blocks = (p.rows * p.groups + per - 1) / per;
  const unsigned g = (unsigned)blocks;
  switch (s.M) {
    case 1: norm_fwd_kernel<IOT, RT, V, 1, true><<<g, s.threads, 0, stream>>>(p, s.T); break;
    case 2: norm_fwd_kernel<IOT, RT, V, 2, true><<<g, s.threads, 0, stream>>>(p, s.T); break;
    case 4: norm_fwd_kernel<IOT, RT, V, 4, true><<<g, s.threads, 0, stream>>>(p, s.T); break;
    default: norm_fwd_kernel<IOT, RT, V, 1, false><<<g, s.threads, 0, stream>>>(p, s.T); break;
  }
  return cudaGetLastError();
}

template <typename K>
cudaError_t run_bwd(K* kern, const NormParams& p, const Shape& s, cudaStream_t stream) {
  const int slices = norm_bwd_slices(p.rows, p.dim, p.groups);
  const size_t bytes = p.dw ? (size_t)(s.M ? s.threads / s.T : 1) * p.width * 4 : 0;
  if (bytes > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
  }
  kern<<<dim3(slices, p.groups), s.threads, bytes, stream>>>(p, s.T);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.dw) return e;
  norm_dw_kernel<<<(p.dim + 31) / 32, 256, 0, stream>>>(p.ws, slices, p.dim, p.dw);
  return cudaGetLastError();
}

template <typename IOT, typename RT, int V>
cudaError_t bwd_m(const NormParams& p, const Shape& s, cudaStream_t stream) {
  switch (s.M) {
    case 1: return run_bwd(norm_bwd_kernel<IOT, RT, V, 1, true>, p, s, stream);
    case 2: return run_bwd(norm_bwd_kernel<IOT, RT, V, 2, true>, p, s, stream);
    case 4: return run_bwd(norm_bwd_kernel<IOT, RT, V, 4, true>, p, s, stream);
    default: {
      Shape one = s;
      one.T = one.threads = 512;  // one row per block
      return run_bwd(norm_bwd_kernel<IOT, RT, V, 1, false>, p, one, stream);
    }
  }
}

}  // namespace

int norm_bwd_slices(int64_t rows, int dim, int groups) {
  // about eight blocks per SM over the groups, at least four rows a slice
  const int64_t want = std::max<int64_t>(1, (148 * 8) / groups);
  const int64_t most = std::max<int64_t>(1, rows / 4);
  (void)dim;
  return (int)std::min<int64_t>(want, most);
}

cudaError_t launch_norm_fwd(const NormParams& p, int types, bool vec, cudaStream_t stream) {
  const Shape s = shape(p, types, vec, 4);
  if (types == 2) return vec ? fwd_m<float, float, 4>(p, s, stream) : fwd_m<float, float, 1>(p, s, stream);
  if (types == 1) return vec ? fwd_m<uint16_t, float, 8>(p, s, stream) : fwd_m<uint16_t, float, 1>(p, s, stream);
  return vec ? fwd_m<uint16_t, uint16_t, 8>(p, s, stream) : fwd_m<uint16_t, uint16_t, 1>(p, s, stream);
}

cudaError_t launch_norm_bwd(const NormParams& p, int types, bool vec, cudaStream_t stream) {
  const Shape s = shape(p, types, vec, 4);
  if (types == 2) return vec ? bwd_m<float, float, 4>(p, s, stream) : bwd_m<float, float, 1>(p, s, stream);
  if (types == 1) return vec ? bwd_m<uint16_t, float, 8>(p, s, stream) : bwd_m<uint16_t, float, 1>(p, s, stream);
  return vec ? bwd_m<uint16_t, uint16_t, 8>(p, s, stream) : bwd_m<uint16_t, uint16_t, 1>(p, s, stream);
}

}  // namespace ssm
