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
// there too. Warps share only the tiles that a producer warp copies ahead
// (one bulk copy each for k/q and for T, P and the factors, one per row of
// v), through full/empty mbarriers; nothing else synchronises them.
//
// Precision: the state path (S K, T R, S's update, and the reverse
// counterparts) takes fp32 operands as two fp16 pieces (ssm_delta.cuh), so the
// carried state, dh0 and the gate gradients keep fp32's accuracy; y, rounded
// to bf16, takes one fp16 piece of S, u and P (2^-12 each).
#include <mutex>

#include "ssm_delta.cuh"

namespace ssm {

namespace {

constexpr int kC = kDeltaChunk;

__device__ int g_delta_timeout;  // set by a CTA that gave up a bounded wait

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

constexpr int kMaxStages = 4;

struct Layout {
  int kq, head, rows, row_stride, tiles, stage;  // bytes; `tiles` row tiles of v's shape
};
__host__ __device__ inline Layout layout(int dstate, int warps, int tiles, int head_load) {
  Layout l;
  l.kq = 2 * kC * dstate * 2;
  l.head = head_load;
  l.row_stride = warps * 32 + 16;  // 16 bytes of skew between rows
  l.rows = kC * l.row_stride;
  l.tiles = tiles;
  l.stage = l.kq + l.head + tiles * l.rows;
  return l;
}

// acc += A (two pieces) B^T, B tile rows = n (k contiguous): pairs jp of n-tiles
template <bool LO>
__device__ __forceinline__ void mma_pair(float (&a0)[4], float (&a1)[4], const uint32_t (&hi)[4],
                                         const uint32_t (&lo)[4], const uint32_t (&b)[4],
                                         bool trans_order) {
  (void)trans_order;
  mma_f16(a0, hi, b[0], b[1]);
  mma_f16(a1, hi, b[2], b[3]);
  if (LO) {
    mma_f16(a0, lo, b[0], b[1]);
    mma_f16(a1, lo, b[2], b[3]);
  }
}

// Lane's row/unit offsets of the two fragment loads (see swz):
//   nt: B rows are n          tr: B rows are k (transposing load)
struct LaneMap {
  int nt_row, nt_unit, tr_row, tr_unit;
};
__device__ __forceinline__ LaneMap lane_map(int lane) {
  LaneMap m;
  m.nt_row = (lane & 7) + ((lane & 16) >> 1);
  m.nt_unit = (lane >> 3) & 1;
  m.tr_row = (lane & 7) + (lane & 8);
  m.tr_unit = lane >> 4;
  return m;
}

// acc[16 x 64] += x[16 x 64 tokens] B over the triangle of a 64 x 64 tile, x as
// two pieces, B as one or two. TR false: B[n][k], n >= k blocks; true: B[k][n].
template <bool TR, bool XLO, bool BLO>
__device__ __forceinline__ void tri_product(float (&acc)[8][4], const float (&x)[8][4], float s0,
                                            float s1, uint32_t bhi, uint32_t blo,
                                            const LaneMap& m) {
#pragma unroll
  for (int kt = 0; kt < 4; ++kt) {
    uint32_t hi[4], lo[4];
    if (XLO)
      split_a(x[2 * kt], x[2 * kt + 1], s0, s1, hi, lo);
    else
      half_a(x[2 * kt], x[2 * kt + 1], s0, s1, hi);
#pragma unroll
    for (int jp = 0; jp < 4; ++jp) {
      if (TR ? jp > kt : jp < kt) continue;
      uint32_t b[4];
      if (TR)
        ldsm4t(b, bhi + swz<128>(16 * kt + m.tr_row, 2 * jp + m.tr_unit));
      else
        ldsm4(b, bhi + swz<128>(16 * jp + m.nt_row, 2 * kt + m.nt_unit));
      mma_pair<XLO>(acc[2 * jp], acc[2 * jp + 1], hi, lo, b, TR);
      if (BLO) {
        if (TR)
          ldsm4t(b, blo + swz<128>(16 * kt + m.tr_row, 2 * jp + m.tr_unit));
        else
          ldsm4(b, blo + swz<128>(16 * jp + m.nt_row, 2 * kt + m.nt_unit));
        mma_pair<false>(acc[2 * jp], acc[2 * jp + 1], hi, lo, b, TR);
      }
    }
  }
}

// s[16 x N] += x[16 x 64 tokens] tile[64 tokens x N], x as two pieces.
template <int N>
__device__ __forceinline__ void state_product(float (&s)[N / 8][4], const float (&x)[8][4],
                                              float s0, float s1, uint32_t tile,
                                              const LaneMap& m) {
#pragma unroll
  for (int kt = 0; kt < 4; ++kt) {
    uint32_t hi[4], lo[4];
    split_a(x[2 * kt], x[2 * kt + 1], s0, s1, hi, lo);
#pragma unroll
    for (int jn = 0; jn < N / 16; ++jn) {
      uint32_t b[4];
      ldsm4t(b, tile + swz<N * 2>(16 * kt + m.tr_row, 2 * jn + m.tr_unit));
      mma_pair<true>(s[2 * jn], s[2 * jn + 1], hi, lo, b, true);
    }
  }
}

template <int N>
__device__ __forceinline__ void scale_state(float (&s)[N / 8][4], float f0, float f1) {
#pragma unroll
  for (int j = 0; j < N / 8; ++j) {
    s[j][0] *= f0; s[j][1] *= f0;
    s[j][2] *= f1; s[j][3] *= f1;
  }
}

// x *= per-token factor (columns) and per-row factors
__device__ __forceinline__ void scale_cols(float (&x)[8][4], const float* f, float f0, float f1,
                                           int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 c = *reinterpret_cast<const float2*>(f + 8 * j + 2 * (lane & 3));
    x[j][0] *= c.x * f0; x[j][1] *= c.y * f0;
    x[j][2] *= c.x * f1; x[j][3] *= c.y * f1;
  }
}

// The warp's 16 columns of a row tile [token][p] as fp32 accumulator-shaped
// values [p][token]; tokens from `valid` on read as zero.
__device__ __forceinline__ void load_rows(float (&x)[8][4], uint32_t tile, int stride, int valid,
                                          int lane, const LaneMap& m) {
#pragma unroll
  for (int jp = 0; jp < 4; ++jp) {
    uint32_t r[4];
    ldsm4t(r, tile + (16 * jp + m.nt_row) * stride + m.nt_unit * 16);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = 2 * jp + (q >> 1), e = (q & 1) * 2, col = 8 * j + 2 * (lane & 3);
      x[j][e] = col < valid ? bf16_lo(r[q]) : 0.f;
      x[j][e + 1] = col + 1 < valid ? bf16_hi(r[q]) : 0.f;
    }
  }
}

// Accumulator-shaped values [p][token] -> bf16 rows of the warp's 16 columns
// in shared memory, then to global memory (32 bytes per token).
__device__ __forceinline__ void store_rows(const float (&x)[8][4], uint32_t tile, int stride,
                                           uint16_t* out, size_t out_stride, int valid, int lane,
                                           const LaneMap& m) {
#pragma unroll
  for (int jp = 0; jp < 4; ++jp) {
    uint32_t r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = 2 * jp + (q >> 1), e = (q & 1) * 2;
      r[q] = pack_bf16x2(x[j][e], x[j][e + 1]);
    }
    stsm4t(tile + (16 * jp + m.nt_row) * stride + m.nt_unit * 16, r);
  }
  __syncwarp();
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int tk = it * 16 + (lane >> 1), u = lane & 1;
    uint4 w;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(tile + tk * stride + u * 16)
                 : "memory");
    if (tk < valid) *reinterpret_cast<uint4*>(out + (size_t)tk * out_stride + u * 8) = w;
  }
}

// Per-token dot products of x and y over the warp's 16 rows -> out[64].
__device__ __forceinline__ void row_dots(const float (&x)[8][4], const float (&y)[8][4],
                                         float* out, int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float a = fmaf(x[j][0], y[j][0], x[j][2] * y[j][2]);
    float b = fmaf(x[j][1], y[j][1], x[j][3] * y[j][3]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (lane < 4) *reinterpret_cast<float2*>(out + 8 * j + 2 * lane) = make_float2(a, b);
  }
}

template <int N>
__device__ __forceinline__ void load_state(float (&s)[N / 8][4], const float* src, int lane) {
  const float* r0 = src + (lane >> 2) * N + 2 * (lane & 3);
#pragma unroll
  for (int j = 0; j < N / 8; ++j) {
    const float2 a = *reinterpret_cast<const float2*>(r0 + 8 * j);
    const float2 b = *reinterpret_cast<const float2*>(r0 + 8 * N + 8 * j);
    s[j][0] = a.x; s[j][1] = a.y; s[j][2] = b.x; s[j][3] = b.y;
  }
}
template <int N>
__device__ __forceinline__ void store_state(const float (&s)[N / 8][4], float* dst, int lane) {
  float* r0 = dst + (lane >> 2) * N + 2 * (lane & 3);
#pragma unroll
  for (int j = 0; j < N / 8; ++j) {
    *reinterpret_cast<float2*>(r0 + 8 * j) = make_float2(s[j][0], s[j][1]);
    *reinterpret_cast<float2*>(r0 + 8 * N + 8 * j) = make_float2(s[j][2], s[j][3]);
  }
}

__device__ __forceinline__ uint32_t max3u(uint32_t a, uint32_t b, uint32_t c) {
  return max(a, max(b, c));
}

// The producer warp: for step s = 0 .. nchunks-1 (chunk s, or nchunks-1-s in
// reverse) copies the chunk's tiles into stage s % stages.
template <int N>
__device__ __forceinline__ void produce(const DeltaChunkParams& p, const Layout& l,
                                        unsigned char* smem, uint64_t* full, uint64_t* empty,
                                        int b, int h, int p0, int active, bool reverse,
                                        const uint16_t* t0, const uint16_t* t1,
                                        const uint16_t* t2) {
  const int lane = threadIdx.x & 31;
  const DeltaParams& d = p.d;
  const int kh = h / (d.nheads / d.nkheads);
  const uint32_t row_bytes = (uint32_t)active * 32;
  const uint16_t* const tiles[3] = {t0, t1, t2};
  int issued = 0;
  bool ok = true;
  for (int s = 0; s < p.nchunks; ++s) {
    const int st = s % p.stages;
    if (s >= p.stages) {
      ok = mbar_wait_bounded(&empty[st], (uint32_t)((s / p.stages - 1) & 1), p.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
    }
    if (p.test_stall && s == 0 && blockIdx.x == 0 && blockIdx.y == 0) continue;  // never arrives
    const int c = reverse ? p.nchunks - 1 - s : s;
    const int64_t tk0 = (int64_t)c * kC;
    const int valid = (int)min((int64_t)kC, d.seqlen - tk0);
    const size_t bc = (size_t)b * p.nchunks + c;
    unsigned char* base = smem + (size_t)st * l.stage;
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[st], (uint32_t)(l.kq + l.head) +
                                           (uint32_t)(l.tiles * valid) * row_bytes);
      bulk_load(smem_u32(base), p.ws_kq + (bc * d.nkheads + kh) * (size_t)l.kq, l.kq, &full[st]);
      bulk_load(smem_u32(base + l.kq), p.ws_head + (bc * d.nheads + h) * (size_t)p.head_bytes,
                l.head, &full[st]);
    }
    __syncwarp();
    for (int t = 0; t < l.tiles; ++t)
      for (int row = lane; row < valid; row += 32)
        bulk_load(smem_u32(base + l.kq + l.head + t * l.rows + row * l.row_stride),
                  tiles[t] + (((size_t)b * d.seqlen + tk0 + row) * d.nheads + h) * d.headdim + p0,
                  row_bytes, &full[st]);
    issued = s + 1;
  }
  if (!ok && lane == 0) atomicExch(&g_delta_timeout, 1);
  // no copy of this CTA may be in flight when it ends
  const int first = issued > p.stages ? issued - p.stages : 0;
  for (int s = first; s < issued; ++s) {
    if (p.test_stall && s == 0 && blockIdx.x == 0 && blockIdx.y == 0) continue;
    mbar_wait_bounded(&full[s % p.stages], (uint32_t)((s / p.stages) & 1), p.wait_limit_ns);
  }
}

template <int N, bool BWD>
__global__ void __launch_bounds__(160, 1) delta_fwd_kernel(const __grid_constant__ DeltaChunkParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  const DeltaParams& d = p.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = (d.headdim / 16 + p.warps - 1) / p.warps;
  const int bh = blockIdx.x / slices, sl = blockIdx.x - bh * slices;
  const int b = bh / d.nheads, h = bh - b * d.nheads;
  const int w0 = sl * p.warps;                             // first 16-row block of this CTA
  const int active = min(p.warps, d.headdim / 16 - w0);
  const Layout l = layout(N, p.warps, BWD ? 2 : 1, BWD ? kDeltaHeadBwd : kDeltaHeadFwd);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], (uint32_t)active);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (warp == p.warps) {
    produce<N>(p, l, smem, full, empty, b, h, w0 * 16, active, false,
               static_cast<const uint16_t*>(d.v), p.dy, nullptr);
    return;
  }
  if (warp >= active) return;

  const LaneMap m = lane_map(lane);
  const int pw = (w0 + warp) * 16;  // the warp's first row of the state
  const size_t state_at = ((size_t)bh * d.headdim + pw) * N;
  const size_t vs = (size_t)d.nheads * d.headdim;
  float S[N / 8][4];
  if (d.h0) {
    load_state<N>(S, d.h0 + state_at, lane);
  } else {
#pragma unroll
    for (int j = 0; j < N / 8; ++j) S[j][0] = S[j][1] = S[j][2] = S[j][3] = 0.f;
  }

  bool ok = true;
  for (int c = 0; c < p.nchunks; ++c) {
    const int st = c % p.stages;
    if (BWD)
      store_state<N>(S, p.ws_state + (((size_t)b * (p.nchunks + 1) + c) * d.nheads + h) *
                                         ((size_t)d.headdim * N) + (size_t)pw * N, lane);
    ok = __all_sync(0xffffffffu,
                    mbar_wait_bounded(&full[st], (uint32_t)((c / p.stages) & 1), p.wait_limit_ns));
    if (!ok) break;
    const int64_t t0 = (int64_t)c * kC;
    const int valid = (int)min((int64_t)kC, d.seqlen - t0);
    unsigned char* base = smem + (size_t)st * l.stage;
    const uint32_t ks = smem_u32(base), qs = ks + l.kq / 2;
    const float* sc = reinterpret_cast<const float*>(base + l.kq);
    const uint32_t th = ks + l.kq + kDeltaScalBytes, tl = th + kDeltaTile, ph = tl + kDeltaTile,
                   pl = ph + kDeltaTile;
    const uint32_t vrow = ks + l.kq + l.head + warp * 32;

    // ---- S K^T and S Q^T
    float ms0, ms1;
    row_max(S, ms0, ms1);
    const uint32_t es0 = exponent_of(ms0), es1 = exponent_of(ms1);
    const RowScale a0 = row_scale(es0), a1 = row_scale(es1);
    float x[8][4], o[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) x[j][q] = o[j][q] = 0.f;
#pragma unroll
    for (int kt = 0; kt < N / 16; ++kt) {
      uint32_t hi[4], lo[4];
      split_a(S[2 * kt], S[2 * kt + 1], a0.s, a1.s, hi, lo);
#pragma unroll
      for (int jp = 0; jp < 4; ++jp) {
        uint32_t bb[4];
        ldsm4(bb, ks + swz<N * 2>(16 * jp + m.nt_row, 2 * kt + m.nt_unit));
        mma_pair<true>(x[2 * jp], x[2 * jp + 1], hi, lo, bb, false);
        ldsm4(bb, qs + swz<N * 2>(16 * jp + m.nt_row, 2 * kt + m.nt_unit));
        mma_pair<BWD>(o[2 * jp], o[2 * jp + 1], hi, lo, bb, false);
      }
    }
    scale_cols(o, sc + kScSq * kC, a0.inv, a1.inv, lane);

    // ---- R = V - ..., r = T R, u = beta r
    scale_cols(x, sc + kScSk * kC, a0.inv, a1.inv, lane);
    float u[8][4];
    load_rows(u, vrow, l.row_stride, valid, lane, m);
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
    tri_product<false, true, true>(u, x, r0.s, r1.s, th, tl, m);
    if (BWD) {
      scale_cols(u, sc + kScT * kC, r0.inv, r1.inv, lane);
      store_rows(u, vrow, l.row_stride, p.ws_r + ((size_t)b * d.seqlen + t0) * vs +
                                            (size_t)h * d.headdim + pw, vs, valid, lane, m);
      scale_cols(u, sc + kScBeta * kC, 1.f, 1.f, lane);
    } else {
      scale_cols(u, sc + kScU * kC, r0.inv, r1.inv, lane);
    }

    // ---- Y += P u
    float w[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        w[j][q] = u[j][q];
        x[j][q] = 0.f;
      }
    scale_cols(w, sc + kScK * kC, 1.f, 1.f, lane);
    row_max(w, m0, m1);
    r0 = row_scale(exponent_of(m0));
    r1 = row_scale(exponent_of(m1));
    tri_product<false, BWD, BWD>(x, w, r0.s, r1.s, ph, pl, m);
    scale_cols(x, sc + kScP * kC, r0.inv, r1.inv, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[j][q] += x[j][q];
    if (BWD) {
      load_rows(x, vrow + l.rows, l.row_stride, valid, lane, m);
      row_dots(x, o, p.ws_doto + ((((size_t)b * p.nchunks + c) * d.nheads + h) *
                                      (d.headdim / 16) + w0 + warp) * kC, lane);
    } else if (d.y) {
      store_rows(o, vrow, l.row_stride, static_cast<uint16_t*>(d.y) +
                                            ((size_t)b * d.seqlen + t0) * vs +
                                            (size_t)h * d.headdim + pw, vs, valid, lane, m);
    }

    // ---- S <- e^G_end S + u^T (e^(G_end - G) K), under one scale for both terms
    scale_cols(u, sc + kScKend * kC, 1.f, 1.f, lane);
    row_max(u, m0, m1);
    const RowScale c0 = row_scale(max(exponent_of(m0), es0)), c1 = row_scale(max(exponent_of(m1), es1));
    const float end = sc[kScEnd * kC];
    scale_state<N>(S, end * c0.s, end * c1.s);
    state_product<N>(S, u, c0.s, c1.s, ks, m);
    scale_state<N>(S, c0.inv, c1.inv);
    fence_async_smem();  // this warp's rows were overwritten by ordinary stores
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
  if (!ok) {
    if (lane == 0) atomicExch(&g_delta_timeout, 1);
    return;
  }
  if (BWD)
    store_state<N>(S, p.ws_state + (((size_t)b * (p.nchunks + 1) + p.nchunks) * d.nheads + h) *
                                       ((size_t)d.headdim * N) + (size_t)pw * N, lane);
  else if (d.h_last)
    store_state<N>(S, d.h_last + state_at, lane);
}

template <int N>
__global__ void __launch_bounds__(160, 1) delta_rev_kernel(const __grid_constant__ DeltaChunkParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  const DeltaParams& d = p.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = (d.headdim / 16 + p.warps - 1) / p.warps;
  const int bh = blockIdx.x / slices, sl = blockIdx.x - bh * slices;
  const int b = bh / d.nheads, h = bh - b * d.nheads;
  const int w0 = sl * p.warps;
  const int active = min(p.warps, d.headdim / 16 - w0);
  const Layout l = layout(N, p.warps, 3, kDeltaHeadBwd);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], (uint32_t)active);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (warp == p.warps) {
    produce<N>(p, l, smem, full, empty, b, h, w0 * 16, active, true,
               static_cast<const uint16_t*>(d.v), p.dy, p.ws_r);
    return;
  }
  if (warp >= active) return;

  const LaneMap m = lane_map(lane);
  const int pw = (w0 + warp) * 16;
  const size_t state_at = ((size_t)bh * d.headdim + pw) * N;
  const size_t vs = (size_t)d.nheads * d.headdim;
  float S[N / 8][4];  // the adjoint of the state
  if (p.dh_last) {
    load_state<N>(S, p.dh_last + state_at, lane);
  } else {
#pragma unroll
    for (int j = 0; j < N / 8; ++j) S[j][0] = S[j][1] = S[j][2] = S[j][3] = 0.f;
  }

  bool ok = true;
  for (int s = 0; s < p.nchunks; ++s) {
    const int st = s % p.stages, c = p.nchunks - 1 - s;
    const size_t bch = ((size_t)b * p.nchunks + c) * d.nheads + h;
    store_state<N>(S, p.ws_dstate + bch * ((size_t)d.headdim * N) + (size_t)pw * N, lane);
    ok = __all_sync(0xffffffffu,
                    mbar_wait_bounded(&full[st], (uint32_t)((s / p.stages) & 1), p.wait_limit_ns));
    if (!ok) break;
    const int64_t t0 = (int64_t)c * kC;
    const int valid = (int)min((int64_t)kC, d.seqlen - t0);
    unsigned char* base = smem + (size_t)st * l.stage;
    const uint32_t ks = smem_u32(base), qs = ks + l.kq / 2;
    const float* sc = reinterpret_cast<const float*>(base + l.kq);
    const uint32_t th = ks + l.kq + kDeltaScalBytes, tl = th + kDeltaTile, ph = tl + kDeltaTile,
                   pl = ph + kDeltaTile;
    const uint32_t vrow = ks + l.kq + l.head + warp * 32;
    const size_t dot_at = (bch * (d.headdim / 16) + w0 + warp) * kC;

    // ---- dU = P^T dY + e^(G_end - G) K dS^T
    float ms0, ms1;
    row_max(S, ms0, ms1);
    const uint32_t es0 = exponent_of(ms0), es1 = exponent_of(ms1);
    const RowScale a0 = row_scale(es0), a1 = row_scale(es1);
    float x[8][4], u[8][4], w[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) x[j][q] = u[j][q] = 0.f;
#pragma unroll
    for (int kt = 0; kt < N / 16; ++kt) {
      uint32_t hi[4], lo[4];
      split_a(S[2 * kt], S[2 * kt + 1], a0.s, a1.s, hi, lo);
#pragma unroll
      for (int jp = 0; jp < 4; ++jp) {
        uint32_t bb[4];
        ldsm4(bb, ks + swz<N * 2>(16 * jp + m.nt_row, 2 * kt + m.nt_unit));
        mma_pair<true>(x[2 * jp], x[2 * jp + 1], hi, lo, bb, false);
      }
    }
    scale_cols(x, sc + kScKend * kC, a0.inv, a1.inv, lane);
    load_rows(w, vrow + l.rows, l.row_stride, valid, lane, m);  // dY
    scale_cols(w, sc + kScP * kC, 1.f, 1.f, lane);
    float m0, m1;
    row_max(w, m0, m1);
    RowScale r0 = row_scale(exponent_of(m0)), r1 = row_scale(exponent_of(m1));
    tri_product<true, true, true>(u, w, r0.s, r1.s, ph, pl, m);
    scale_cols(u, sc + kScK * kC, r0.inv, r1.inv, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) u[j][q] += x[j][q];
    load_rows(w, vrow + 2 * l.rows, l.row_stride, valid, lane, m);  // r
    row_dots(u, w, p.ws_dotu + dot_at, lane);

    // ---- dR = T^T (beta dU) = dV
    scale_cols(u, sc + kScU * kC, 1.f, 1.f, lane);
    row_max(u, m0, m1);
    r0 = row_scale(exponent_of(m0));
    r1 = row_scale(exponent_of(m1));
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) x[j][q] = 0.f;
    tri_product<true, true, true>(x, u, r0.s, r1.s, th, tl, m);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j][0] *= r0.inv; x[j][1] *= r0.inv;
      x[j][2] *= r1.inv; x[j][3] *= r1.inv;
    }
    load_rows(w, vrow, l.row_stride, valid, lane, m);  // v
    row_dots(x, w, p.ws_dotv + dot_at, lane);
    __syncwarp();
    store_rows(x, vrow, l.row_stride,
               p.dv + ((size_t)b * d.seqlen + t0) * vs + (size_t)h * d.headdim + pw, vs, valid,
               lane, m);

    // ---- dS <- e^G_end dS + dY^T (e^G Q) - dR^T (e^G K), under one scale
    load_rows(w, vrow + l.rows, l.row_stride, valid, lane, m);
    scale_cols(w, sc + kScSq * kC, 1.f, 1.f, lane);
    scale_cols(x, sc + kScSk * kC, -1.f, -1.f, lane);
    float n0, n1;
    row_max(w, m0, m1);
    row_max(x, n0, n1);
    const RowScale c0 = row_scale(max3u(exponent_of(m0), exponent_of(n0), es0));
    const RowScale c1 = row_scale(max3u(exponent_of(m1), exponent_of(n1), es1));
    const float end = sc[kScEnd * kC];
    scale_state<N>(S, end * c0.s, end * c1.s);
    state_product<N>(S, w, c0.s, c1.s, qs, m);
    state_product<N>(S, x, c0.s, c1.s, ks, m);
    scale_state<N>(S, c0.inv, c1.inv);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
  if (!ok) {
    if (lane == 0) atomicExch(&g_delta_timeout, 1);
    return;
  }
  if (p.dh0) store_state<N>(S, p.dh0 + state_at, lane);
}

// Consumer warps per CTA and stages. One CTA fits an SM (its tiles take over
// half the shared memory), so few heads are spread over more CTAs of fewer
// warps until every SM has one.
template <typename K>
cudaError_t run(K* kern, DeltaChunkParams& p, int tiles, int head_load, int max_warps,
                cudaStream_t stream) {
  const int blocks16 = p.d.headdim / 16;
  const int64_t heads = (int64_t)p.d.batch * p.d.nheads;
  int warps = max_warps;
  while (warps > 1 && (warps / 2 >= blocks16 || heads * ((blocks16 + warps / 2 - 1) / (warps / 2)) <= 148))
    warps /= 2;
  p.warps = warps;
  const Layout l = layout(p.d.dstate, warps, tiles, head_load);
  int stages = (int)((225 * 1024) / l.stage);
  stages = stages > kMaxStages ? kMaxStages : stages;
  if (stages < 1) return cudaErrorInvalidValue;
  p.stages = stages;
  const int bytes = l.stage * stages;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(heads * ((blocks16 + warps - 1) / warps));
  kern<<<grid, (warps + 1) * 32, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

bool delta_chunk_supported(int dstate, int headdim) {
  return (dstate == 64 || dstate == 128) && headdim % 16 == 0 && headdim >= 16;
}

cudaError_t launch_delta_chunk_fwd(const DeltaChunkParams& pin, bool bwd, cudaStream_t stream) {
  DeltaChunkParams p = pin;
  if (bwd)
    return p.d.dstate == 64 ? run(delta_fwd_kernel<64, true>, p, 2, kDeltaHeadBwd, 4, stream)
                            : run(delta_fwd_kernel<128, true>, p, 2, kDeltaHeadBwd, 4, stream);
  return p.d.dstate == 64 ? run(delta_fwd_kernel<64, false>, p, 1, kDeltaHeadFwd, 4, stream)
                          : run(delta_fwd_kernel<128, false>, p, 1, kDeltaHeadFwd, 4, stream);
}

cudaError_t launch_delta_chunk_rev(const DeltaChunkParams& pin, cudaStream_t stream) {
  DeltaChunkParams p = pin;
  return p.d.dstate == 64 ? run(delta_rev_kernel<64>, p, 3, kDeltaHeadBwd, 4, stream)
                          : run(delta_rev_kernel<128>, p, 3, kDeltaHeadBwd, 4, stream);
}

cudaError_t delta_chunk_status(cudaStream_t stream, int* timed_out) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  const int zero = 0;
  e = cudaMemcpyFromSymbol(timed_out, g_delta_timeout, sizeof(int));
  if (e != cudaSuccess || !*timed_out) return e;
  return cudaMemcpyToSymbol(g_delta_timeout, &zero, sizeof(int));
}

}  // namespace ssm
