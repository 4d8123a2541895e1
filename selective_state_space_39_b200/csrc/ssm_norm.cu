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
// (up to four 16-byte units of io per thread; the backward pass of bf16 rows up
// to two; longer rows are read twice), sums the squares (backward: and t u) in
// fp32 by shuffles, and writes the results. T is the power of two that leaves a
// thread one or two units, so rows of one head's width take 8 lanes and a warp
// holds several. Rows that are no whole units, or lie off 16-byte boundaries,
// are read two values per thread. The backward pass keeps 296 blocks, each
// walking over its rows with the next row's loads in flight, sums dw in
// registers over them, in shared memory over its row groups and over the
// blocks by a second kernel, always in the same order.
//
// Bound: memory traffic (forward: x, z, residual in, y, h out; backward: h,
// dy, z, dh in, dx, dz, dresidual out). Measured, calls in a row: forward with an
// fp32 residual, 16384 x 4096 bf16, 124 us = 6.5 TB/s (119 us in a graph's
// replay, whose last writes partly stay in L2); gated backward of 131072 x 128
// bf16, 41 us = 4.1 TB/s, the sigmoid and its derivative beside the loads; 1000 x
// 1537 fp32 backward, 19 us, 16 of it the latency of a few rows.
#include <algorithm>
#include <type_traits>

#include "ssm_chain.cuh"
#include "ssm_device.cuh"
#include "ssm_norm_internal.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;
// Shared memory of the widest group's dw sums: the limit of every launch that needs more
// than 48 KB, so that calls from several threads cannot lower it under one another.
constexpr int kMaxNormShared = (kNormMaxWidth + 1) * 4;

// V values of type T as they lie in memory: 16-byte units, or (V = 2) two values
// loaded one by one, the second only where `left`, the values up to the row's
// end, has it.
template <typename T, int V>
struct Raw {
  static constexpr int kWords = V == 2 ? 2 : V * (int)sizeof(T) / 4;
  uint32_t w[kWords];
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p, int left) {
  Raw<T, V> r;
  if constexpr (V == 2) {
    using W = std::conditional_t<sizeof(T) == 2, uint16_t, uint32_t>;
    r.w[0] = reinterpret_cast<const W*>(p)[0];
    r.w[1] = left > 1 ? reinterpret_cast<const W*>(p)[1] : 0;
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, V>::kWords; i += 4) {
      const uint4 v = *(reinterpret_cast<const uint4*>(p) + i / 4);
      r.w[i] = v.x; r.w[i + 1] = v.y; r.w[i + 2] = v.z; r.w[i + 3] = v.w;
    }
  }
  return r;
}
// Values are held as pairs for the packed fp32 instructions.
template <int V>
struct Pairs {
  static constexpr int n = V / 2;
  float2 f[n];
};
template <typename T, int V>
__device__ __forceinline__ Pairs<V> unpack(const Raw<T, V>& r) {
  Pairs<V> p;
  if constexpr (V == 2) {
    p.f[0] = sizeof(T) == 2 ? make_float2(bf16_lo(r.w[0]), bf16_lo(r.w[1]))
                            : make_float2(__uint_as_float(r.w[0]), __uint_as_float(r.w[1]));
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p.f[i] = make_float2(bf16_lo(r.w[i]), bf16_hi(r.w[i]));
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      p.f[i] = make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
  }
  return p;
}
template <typename T, int V>
__device__ __forceinline__ Pairs<V> load_pairs(const T* p, int left) {
  return unpack<T, V>(load_raw<T, V>(p, left));
}
template <typename T, int V>
__device__ __forceinline__ void store_pairs(T* p, const Pairs<V>& v, int left) {
  if constexpr (V == 2) {
    Io<T>::store(p, v.f[0].x);
    if (left > 1) Io<T>::store(p + 1, v.f[0].y);
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(v.f[0].x, v.f[0].y), pack_bf16x2(v.f[1].x, v.f[1].y),
                   pack_bf16x2(v.f[2].x, v.f[2].y), pack_bf16x2(v.f[3].x, v.f[3].y));
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; i += 2)
      *reinterpret_cast<float4*>(p + 2 * i) =
          make_float4(v.f[i].x, v.f[i].y, v.f[i + 1].x, v.f[i + 1].y);
  }
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// sigmoid: MUFU approximations for bf16 io (2^-22 relative), exact functions for fp32
template <typename IOT>
__device__ __forceinline__ float2 sigmoid(float2 z) {
  if constexpr (sizeof(IOT) == 2)
    return make_float2(rcp_approx(1.f + ex2_approx(-z.x * kLog2e)),
                       rcp_approx(1.f + ex2_approx(-z.y * kLog2e)));
  else
    return make_float2(1.f / (1.f + expf(-z.x)), 1.f / (1.f + expf(-z.y)));
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

template <typename IOT, typename RT, int V, int M, bool FIT, int GATE>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormParams p, int T) {
  __shared__ float sh[32];
  using P = Pairs<V>;
  const int per_block = blockDim.x / T, t = threadIdx.x % T;
  const int64_t total = p.rows * p.groups;
  const int64_t r_raw = (int64_t)blockIdx.x * per_block + threadIdx.x / T;
  const bool live = r_raw < total;
  const int64_t r = live ? r_raw : total - 1;
  const size_t base = (size_t)r * p.width;  // rows are contiguous, so their groups are too
  const int wbase = p.groups == 1 ? 0 : (int)(r % p.groups) * p.width;
  const IOT* x = static_cast<const IOT*>(p.x) + base;
  const RT* res = p.residual ? static_cast<const RT*>(p.residual) + base : nullptr;
  const IOT* z = GATE ? static_cast<const IOT*>(p.z) + base : nullptr;

  // u (the normed value) and the gate's value where it comes last
  auto value = [&](int at, const Raw<IOT, V>& xr, const Raw<RT, V>& rr, const Raw<IOT, V>& zr, P& u,
                   P& g, bool store) {
    u = unpack<IOT, V>(xr);
    if (res) {
      const P q = unpack<RT, V>(rr);
#pragma unroll
      for (int i = 0; i < P::n; ++i) u.f[i] = fma2(both(p.residual_scale), u.f[i], q.f[i]);
      if (store && live) store_pairs<RT, V>(static_cast<RT*>(p.h_out) + base + at, u, p.width - at);
    }
    if (GATE) {
      g = unpack<IOT, V>(zr);
#pragma unroll
      for (int i = 0; i < P::n; ++i) {
        g.f[i] = mul2(g.f[i], sigmoid<IOT>(g.f[i]));
        if (GATE == kGateFirst) u.f[i] = mul2(u.f[i], g.f[i]);
      }
    }
  };
  auto square = [](const P& u, float2& s) {
#pragma unroll
    for (int i = 0; i < P::n; ++i) s = fma2(u.f[i], u.f[i], s);
  };

  P u[M], g[M];
  float2 s2 = make_float2(0.f, 0.f);
  if (FIT) {
    Raw<IOT, V> xr[M], zr[M];
    Raw<RT, V> rr[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int at = (m * T + t) * V;
      if (at >= p.width) break;
      xr[m] = load_raw<IOT, V>(x + at, p.width - at);
      if (res) rr[m] = load_raw<RT, V>(res + at, p.width - at);
      if (GATE) zr[m] = load_raw<IOT, V>(z + at, p.width - at);
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int at = (m * T + t) * V;
      if (at >= p.width) break;
      value(at, xr[m], rr[m], zr[m], u[m], g[m], true);
      square(u[m], s2);
    }
  } else {
    for (int at = t * V; at < p.width; at += T * V) {
      Raw<RT, V> rr;
      Raw<IOT, V> zr;
      if (res) rr = load_raw<RT, V>(res + at, p.width - at);
      if (GATE) zr = load_raw<IOT, V>(z + at, p.width - at);
      value(at, load_raw<IOT, V>(x + at, p.width - at), rr, zr, u[0], g[0], false);
      square(u[0], s2);
    }
  }
  float ss[1] = {s2.x + s2.y};
  group_sum<1>(ss, T, sh);
  const float inv = 1.f / sqrtf(ss[0] / (float)p.width + p.eps);

  auto finish = [&](int at, P& uu, const P& gg) {
    const P w = load_pairs<float, V>(p.w + wbase + at, p.width - at);
#pragma unroll
    for (int i = 0; i < P::n; ++i) {
      uu.f[i] = mul2(mul2(uu.f[i], both(inv)), w.f[i]);
      if (GATE == kGateLast) uu.f[i] = mul2(uu.f[i], gg.f[i]);
    }
    if (live) store_pairs<IOT, V>(static_cast<IOT*>(p.y) + base + at, uu, p.width - at);
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
      Raw<RT, V> rr;
      Raw<IOT, V> zr;
      if (res) rr = load_raw<RT, V>(res + at, p.width - at);
      if (GATE) zr = load_raw<IOT, V>(z + at, p.width - at);
      value(at, load_raw<IOT, V>(x + at, p.width - at), rr, zr, u[0], g[0], true);
      finish(at, u[0], g[0]);
    }
  }
}

// Grid: (slices, groups). A block takes row slots slice, slice + slices, ... in
// turn, so that a thread's columns stay the same; the next rows' data are
// loaded before the present ones are finished.
template <typename IOT, typename RT, int V, int M, bool FIT, int GATE>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormParams p, int T) {
  chain_go();
  extern __shared__ float dws[];  // dw sums of the block's row groups
  __shared__ float sh[64];
  using P = Pairs<V>;
  const int per_block = blockDim.x / T, t = threadIdx.x % T, slot = threadIdx.x / T;
  const int group = blockIdx.y, wbase = group * p.width;
  P acc[FIT ? M : 1];
#pragma unroll
  for (int m = 0; m < (FIT ? M : 1); ++m)
#pragma unroll
    for (int i = 0; i < P::n; ++i) acc[m].f[i] = make_float2(0.f, 0.f);
  if (!FIT && p.dw)
    for (int i = threadIdx.x; i <= p.width; i += blockDim.x) dws[i] = 0.f;

  struct Row {
    Raw<RT, V> h;
    Raw<IOT, V> dy, z;
  };
  auto load = [&](size_t base, int at, Row& r) {
    r.h = load_raw<RT, V>(static_cast<const RT*>(p.h) + base + at, p.width - at);
    r.dy = load_raw<IOT, V>(static_cast<const IOT*>(p.dy) + base + at, p.width - at);
    if (GATE) r.z = load_raw<IOT, V>(static_cast<const IOT*>(p.z) + base + at, p.width - at);
  };
  // the gate's sigmoid; adds u^2 and t u
  auto sums = [&](int at, const Row& r, P& sg, float2& uu, float2& tu) {
    const P w = load_pairs<float, V>(p.w + wbase + at, p.width - at);
    const P h = unpack<RT, V>(r.h), dn = unpack<IOT, V>(r.dy);
    P z;
    if (GATE) z = unpack<IOT, V>(r.z);
#pragma unroll
    for (int i = 0; i < P::n; ++i) {
      float2 u = h.f[i], d = dn.f[i];
      if (GATE) {
        sg.f[i] = sigmoid<IOT>(z.f[i]);
        const float2 g = mul2(z.f[i], sg.f[i]);
        if (GATE == kGateFirst) u = mul2(u, g); else d = mul2(d, g);
      }
      uu = fma2(u, u, uu);
      tu = fma2(mul2(d, w.f[i]), u, tu);
    }
  };
  auto finish = [&](size_t base, int at, const Row& r, const P& sg, float inv, float c, bool live,
                    P& sum) {
    const P h = unpack<RT, V>(r.h), dy = unpack<IOT, V>(r.dy);
    const P w = load_pairs<float, V>(p.w + wbase + at, p.width - at);
    P extra, dh, dz, z;
    if (GATE) z = unpack<IOT, V>(r.z);
    if (p.dh) extra = load_pairs<RT, V>(static_cast<const RT*>(p.dh) + base + at, p.width - at);
#pragma unroll
    for (int i = 0; i < P::n; ++i) {
      const float2 g = GATE ? mul2(z.f[i], sg.f[i]) : both(1.f);
      const float2 u = GATE == kGateFirst ? mul2(h.f[i], g) : h.f[i];
      const float2 dn = GATE == kGateLast ? mul2(dy.f[i], g) : dy.f[i];
      const float2 n = mul2(u, both(inv));
      const float2 du = mul2(both(inv), fma2(n, both(-c), mul2(dn, w.f[i])));
      if (live) sum.f[i] = fma2(dn, n, sum.f[i]);
      if (GATE) {
        const float2 dg = GATE == kGateFirst ? mul2(du, h.f[i]) : mul2(mul2(dy.f[i], n), w.f[i]);
        // SiLU'(z) = s (1 + z (1 - s))
        const float2 one_s = fma2(sg.f[i], both(-1.f), both(1.f));
        dz.f[i] = mul2(dg, mul2(sg.f[i], fma2(z.f[i], one_s, both(1.f))));
      }
      dh.f[i] = GATE == kGateFirst ? mul2(du, g) : du;
      if (p.dh) dh.f[i] = add2(dh.f[i], extra.f[i]);
    }
    if (!live) return;
    if (GATE) store_pairs<IOT, V>(static_cast<IOT*>(p.dz) + base + at, dz, p.width - at);
    if (p.dresidual) store_pairs<RT, V>(static_cast<RT*>(p.dresidual) + base + at, dh, p.width - at);
#pragma unroll
    for (int i = 0; i < P::n; ++i) dh.f[i] = mul2(dh.f[i], both(p.residual_scale));
    store_pairs<IOT, V>(static_cast<IOT*>(p.dx) + base + at, dh, p.width - at);
  };
  auto base_of = [&](int64_t r0) {
    const int64_t r = r0 + slot < p.rows ? r0 + slot : p.rows - 1;
    return ((size_t)r * p.groups + group) * p.width;
  };

  const int64_t step = (int64_t)gridDim.x * per_block;
  Row row[M];
  if (FIT) {
    const size_t base = base_of((int64_t)blockIdx.x * per_block);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int at = (m * T + t) * V;
      if (at >= p.width) break;
      load(base, at, row[m]);
    }
  }
  for (int64_t r0 = (int64_t)blockIdx.x * per_block; r0 < p.rows; r0 += step) {
    const bool live = r0 + slot < p.rows;
    const size_t base = base_of(r0);
    float2 uu = make_float2(0.f, 0.f), tu = uu;
    P sg[M];
    if (FIT) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int at = (m * T + t) * V;
        if (at >= p.width) break;
        sums(at, row[m], sg[m], uu, tu);
      }
    } else {
      for (int at = t * V; at < p.width; at += T * V) {
        load(base, at, row[0]);
        sums(at, row[0], sg[0], uu, tu);
      }
    }
    Row next[M];
    if (FIT && r0 + step < p.rows) {
      const size_t nb = base_of(r0 + step);
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int at = (m * T + t) * V;
        if (at >= p.width) break;
        load(nb, at, next[m]);
      }
    }
    float ss[2] = {uu.x + uu.y, tu.x + tu.y};
    group_sum<2>(ss, T, sh);
    const float inv = 1.f / sqrtf(ss[0] / (float)p.width + p.eps);
    const float c = ss[1] * inv / (float)p.width;  // mean(t n)
    if (FIT) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int at = (m * T + t) * V;
        if (at >= p.width) break;
        finish(base, at, row[m], sg[m], inv, c, live, acc[m]);
        row[m] = next[m];
      }
    } else {  // one row at a time (T = the block): the columns' sums live in shared memory
      for (int at = t * V; at < p.width; at += T * V) {
        load(base, at, row[0]);
        float2 a = make_float2(0.f, 0.f), b = a;
        sums(at, row[0], sg[0], a, b);
        if (p.dw) {
#pragma unroll
          for (int i = 0; i < P::n; ++i)
            acc[0].f[i] = make_float2(dws[at + 2 * i], dws[at + 2 * i + 1]);
        }
        finish(base, at, row[0], sg[0], inv, c, live, acc[0]);
        if (p.dw) {
#pragma unroll
          for (int i = 0; i < P::n; ++i) {
            dws[at + 2 * i] = acc[0].f[i].x;
            dws[at + 2 * i + 1] = acc[0].f[i].y;
          }
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
      for (int i = 0; i < P::n; ++i) {
        dws[slot * p.width + at + 2 * i] = acc[m].f[i].x;
        if (at + 2 * i + 1 < p.width) dws[slot * p.width + at + 2 * i + 1] = acc[m].f[i].y;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.width; i += blockDim.x) {
    float s = 0.f;
    for (int q = 0; q < (FIT ? per_block : 1); ++q) s += dws[q * p.width + i];
    out[i] = s;
  }
}

// dw: 32 columns per block, the slices' sums by 32 warps in a fixed order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const NormParams p) {
  __shared__ float sh[32][33];
  const float* part = p.ws;
  const int slices = p.slices, dim = p.dim;
  float* dw = p.dw;
  chain_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < dim) {
#pragma unroll 8
    for (int i = warp; i < slices; i += 32) s += part[(size_t)i * dim + col];
  }
  sh[warp][lane] = s;
  __syncthreads();
  s = sh[lane][warp];  // column `warp` of the block, summed across the lanes
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32 + warp < dim) dw[blockIdx.x * 32 + warp] = s;
}

struct Shape {
  int V, T, M, threads;  // M units per thread; 0: the row is read twice
};
Shape shape(const NormParams& p, int types, bool vec) {
  Shape s;
  s.V = vec ? (types == 2 ? 4 : 8) : 2;
  const int units = (p.width + s.V - 1) / s.V;
  s.T = 8;
  while (s.T < 512 && s.T * 2 < units) s.T *= 2;
  const int m = (units + s.T - 1) / s.T;
  s.M = m <= 1 ? 1 : m <= 2 ? 2 : m <= 4 ? 4 : 0;
  s.threads = std::max(s.T, kThreads);
  return s;
}

template <typename IOT, typename RT, int V, int GATE>
cudaError_t fwd_m(const NormParams& p, const Shape& s, cudaStream_t stream) {
  const int64_t per = s.threads / s.T, blocks = (p.rows * p.groups + per - 1) / per;
  const unsigned g = (unsigned)blocks;
  switch (s.M) {
    case 1: norm_fwd_kernel<IOT, RT, V, 1, true, GATE><<<g, s.threads, 0, stream>>>(p, s.T); break;
    case 2: norm_fwd_kernel<IOT, RT, V, 2, true, GATE><<<g, s.threads, 0, stream>>>(p, s.T); break;
    case 4: norm_fwd_kernel<IOT, RT, V, 4, true, GATE><<<g, s.threads, 0, stream>>>(p, s.T); break;
    default: norm_fwd_kernel<IOT, RT, V, 1, false, GATE><<<g, s.threads, 0, stream>>>(p, s.T); break;
  }
  return cudaGetLastError();
}

template <typename K>
cudaError_t run_bwd(K* kern, NormParams p, const Shape& s, cudaStream_t stream) {
  p.slices = norm_bwd_slices(p.rows, p.groups);
  const size_t bytes = p.dw ? ((size_t)(s.M ? s.threads / s.T : 1) * p.width + 1) * 4 : 0;
  if (bytes > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxNormShared);
    if (e != cudaSuccess) return e;
  }
  kern<<<dim3(p.slices, p.groups), s.threads, bytes, stream>>>(p, s.T);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.dw) return e;
  return launch_chained(norm_dw_kernel, dim3((p.dim + 31) / 32), 1024, 0, stream, p);
}

template <typename IOT, typename RT, int V, int GATE>
cudaError_t bwd_m(const NormParams& p, const Shape& s, cudaStream_t stream) {
  switch (s.M) {
    case 1: return run_bwd(norm_bwd_kernel<IOT, RT, V, 1, true, GATE>, p, s, stream);
    case 2: return run_bwd(norm_bwd_kernel<IOT, RT, V, 2, true, GATE>, p, s, stream);
    case 4:
      // four units of eight values and their gradients do not fit the registers
      if constexpr (V < 8) return run_bwd(norm_bwd_kernel<IOT, RT, V, 4, true, GATE>, p, s, stream);
      [[fallthrough]];
    default: {
      Shape one = s;
      one.M = 0;
      one.T = one.threads = 512;  // one row per block, read twice
      return run_bwd(norm_bwd_kernel<IOT, RT, V, 1, false, GATE>, p, one, stream);
    }
  }
}

template <bool BWD, typename IOT, typename RT, int V>
cudaError_t gated(const NormParams& p, const Shape& s, cudaStream_t st) {
  switch (p.gate) {
    case kGateFirst:
      return BWD ? bwd_m<IOT, RT, V, kGateFirst>(p, s, st) : fwd_m<IOT, RT, V, kGateFirst>(p, s, st);
    case kGateLast:
      return BWD ? bwd_m<IOT, RT, V, kGateLast>(p, s, st) : fwd_m<IOT, RT, V, kGateLast>(p, s, st);
    default:
      return BWD ? bwd_m<IOT, RT, V, kGateNone>(p, s, st) : fwd_m<IOT, RT, V, kGateNone>(p, s, st);
  }
}
template <bool BWD>
cudaError_t typed(const NormParams& p, int types, bool vec, cudaStream_t st) {
  const Shape s = shape(p, types, vec);
  if (types == 2) return vec ? gated<BWD, float, float, 4>(p, s, st) : gated<BWD, float, float, 2>(p, s, st);
  if (types == 1)
    return vec ? gated<BWD, uint16_t, float, 8>(p, s, st) : gated<BWD, uint16_t, float, 2>(p, s, st);
  return vec ? gated<BWD, uint16_t, uint16_t, 8>(p, s, st)
             : gated<BWD, uint16_t, uint16_t, 2>(p, s, st);
}

}  // namespace

int norm_bwd_slices(int64_t rows, int groups) {
  // two blocks per SM over the groups (131072 rows of 128, gated: 38.9 us; four
  // 41.2, eight 46.8 us), at least two rows a slice
  const int64_t want = std::max<int64_t>(1, (148 * 2) / groups);
  const int64_t most = std::max<int64_t>(1, rows / 2);
  return (int)std::min<int64_t>(want, most);
}

cudaError_t launch_norm_fwd(const NormParams& p, int types, bool vec, cudaStream_t stream) {
  return typed<false>(p, types, vec, stream);
}

cudaError_t launch_norm_bwd(const NormParams& p, int types, bool vec, cudaStream_t stream) {
  return typed<true>(p, types, vec, stream);
}

}  // namespace ssm
