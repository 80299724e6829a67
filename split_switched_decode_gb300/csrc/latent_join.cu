// latent_join.cu -- joins the parts of latent_decode's rows that lie in several CTAs:
// out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i over a row's parts, in their order.
//
// Reads what the parts hold (fp32, in L2 since just before) and writes the row: latencies bound
// it, then instructions. A warp has a row, so that what is the same for its elements is done once:
// where the parts are, then maxima, sums and the first two parts together, then two at a time.
// While rows are few, 16 warps share the parts of 128 elements of a row. Sums are those of a
// sixteenth of the parts each, added in order, either way: the bits of a row depend on its
// parts alone. 12 us with its launch behind 64 ragged sequences of 64 heads (28 MB of parts), 6 for
// one row of 64 heads in parts of all SMs, 2.4 for one of 16 heads in a few.
#include "attn_kernel.cuh"
#include "latent.h"

namespace ssd {
namespace {

constexpr int LJ_SHARES = 16;

__device__ __forceinline__ float4 scaled(float f, float4 u) {
  return make_float4(__fmul_rn(f, u.x), __fmul_rn(f, u.y), __fmul_rn(f, u.z), __fmul_rn(f, u.w));
}
__device__ __forceinline__ float4 fused(float f, float4 u, float4 v) {
  return make_float4(__fmaf_rn(f, u.x, v.x), __fmaf_rn(f, u.y, v.y), __fmaf_rn(f, u.z, v.z),
                     __fmaf_rn(f, u.w, v.w));
}
__device__ __forceinline__ float4 plus(float4 u, float4 v) {
  return make_float4(__fadd_rn(u.x, v.x), __fadd_rn(u.y, v.y), __fadd_rn(u.z, v.z),
                     __fadd_rn(u.w, v.w));
}

// Rows of no sequence, before the first and behind the last, have no entry.
__device__ __forceinline__ int2 rows_in_use(const AttnParams &p) {
  if (!p.q_start) return make_int2(0, p.S * p.Hq);
  return make_int2(min(max(p.q_start[0], 0), p.T) * p.Hq,
                   min(max(p.q_start[p.S], 0), p.T) * p.Hq);
}

// The parts of a row.
template <int MQ>
struct RowParts {
  const float2 *ml_at;
  const float *partials;
  int workers, c0, n, r;
  __device__ __forceinline__ RowParts(const int2 *rows, int row, const float2 *ml,
                                      const float *parts, int most)
      : ml_at(ml), partials(parts), workers(most) {
    const int2 x = __ldcg(rows + row);  // kept in bounds, whatever stands there
    r = (x.x >> 16) & (MQ - 1);
    c0 = min(x.x & 0xffff, workers - 1);
    n = max(min(x.y, workers - c0), 0);
  }
  __device__ __forceinline__ float4 out(int i, int d) const {
    return __ldcg(reinterpret_cast<const float4 *>(
        partials + (static_cast<size_t>(part_slot(c0, i)) * MQ + r) * LATENT_MAX_R + d));
  }
  __device__ __forceinline__ float2 ml(int i) const {
    return __ldcg(ml_at + (2 * r + (i == 0 ? 1 : 0)) * workers + c0 + i);
  }
};

__device__ __forceinline__ void put_row(const AttnParams &p, int row, int d, float4 v, float m,
                                        float l) {
  const int t = row / p.Hq, h = row - t * p.Hq;
  const float inv = l == 0.0f ? 0.0f : (p.c.v_scale ? p.c.v_scale[0] : 1.0f) / l;
  uint2 u = make_uint2(0u, 0u);  // a row that saw nothing
  if (l != 0.0f) {
    u.x = pack2<false>(v.x * inv, v.y * inv);
    u.y = pack2<false>(v.z * inv, v.w * inv);
  }
  if (d < p.D)
    *reinterpret_cast<uint2 *>(p.out + t * p.out_stride + static_cast<long long>(h) * p.D + d) = u;
  if (d == 0 && p.lse) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2;
}

// Rows of up to 16 parts: a part a share.
template <int MQ>
__device__ __forceinline__ void join_row(const AttnParams &p, const RowParts<MQ> &x, int row,
                                         int lane) {
  constexpr int CUTS = LATENT_MAX_R / 128, AHEAD = 2;
  const int d = 4 * lane;
  float4 u[AHEAD][CUTS], v[CUTS];
  auto load = [&](int i0) {
#pragma unroll
    for (int e = 0; e < AHEAD; ++e)
#pragma unroll
      for (int c = 0; c < CUTS; ++c)
        if (i0 + e < x.n && d + 128 * c < p.D) u[e][c] = x.out(i0 + e, d + 128 * c);
  };
  load(0);
  const float2 one = lane < x.n ? x.ml(lane) : make_float2(-INFINITY, 0.0f);
  float m = one.x;
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, e));
  const float f = ex2(one.x - (m == -INFINITY ? 0.0f : m));
  float l = __fmul_rn(f, one.y);
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, e));
#pragma unroll
  for (int c = 0; c < CUTS; ++c) v[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i0 = 0;;) {
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) {
      const float g = __shfl_sync(0xffffffffu, f, (i0 + e) & 31);
#pragma unroll
      for (int c = 0; c < CUTS; ++c)
        if (i0 + e < x.n && d + 128 * c < p.D) v[c] = plus(v[c], scaled(g, u[e][c]));
    }
    i0 += AHEAD;
    if (i0 >= x.n) break;
    load(i0);
  }
  const int t = row / p.Hq, h = row - t * p.Hq;
  const float inv = l == 0.0f ? 0.0f : (p.c.v_scale ? p.c.v_scale[0] : 1.0f) / l;
  uint16_t *out = p.out + t * p.out_stride + static_cast<long long>(h) * p.D;
#pragma unroll
  for (int c = 0; c < CUTS; ++c)
    if (d + 128 * c < p.D) {
      uint2 y = make_uint2(0u, 0u);  // a row that saw nothing
      if (l != 0.0f) {
        y.x = pack2<false>(v[c].x * inv, v[c].y * inv);
        y.y = pack2<false>(v[c].z * inv, v[c].w * inv);
      }
      *reinterpret_cast<uint2 *>(out + d + 128 * c) = y;
    }
  if (lane == 0 && p.lse) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2;
}
// Rows of more parts.
template <int MQ>
__device__ __forceinline__ void join_long_row(const AttnParams &p, const RowParts<MQ> &x, int row,
                                           int d, int lane) {
  constexpr int AHEAD = 4;
  const bool in = d < p.D;
  float m = -INFINITY;
  for (int i = lane; i < x.n; i += 32) m = fmaxf(m, x.ml(i).x);
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, e));
  const float base = m == -INFINITY ? 0.0f : m;
  const int per = (x.n + LJ_SHARES - 1) / LJ_SHARES;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f), w = v;
  float l = 0.0f;
  int stop = per;
  for (int i0 = 0; i0 < x.n; i0 += 32) {
    float f = 0.0f;
    if (i0 + lane < x.n) {
      const float2 ml = x.ml(i0 + lane);
      f = ex2(ml.x - base);
      l = __fmaf_rn(f, ml.y, l);
    }
    const int to = min(x.n, i0 + 32);
    for (int i = i0; i < to; i += AHEAD) {
      float4 u[AHEAD];
#pragma unroll
      for (int e = 0; e < AHEAD; ++e)
        if (i + e < to && in) u[e] = x.out(i + e, d);
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        const float g = __shfl_sync(0xffffffffu, f, (i + e - i0) & 31);
        if (i + e < to && i + e == stop) {
          stop += per;
          v = plus(v, w);
          w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        if (i + e < to && in) w = fused(g, u[e], w);
      }
    }
  }
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, e));
  put_row(p, row, d, plus(v, w), m, l);
}

template <int MQ>
__global__ void __launch_bounds__(256, 3)
    latent_join_kernel(const __grid_constant__ AttnParams p, const int2 *rows, const float2 *ml,
                       const float *partials, int workers) {
  griddep_wait();
  griddep_launch_dependents();
  const int2 used = rows_in_use(p);
  const int lane = threadIdx.x & 31, all = p.T * p.Hq;
  for (int row = blockIdx.x * 8 + (threadIdx.x >> 5); row < all; row += gridDim.x * 8) {
    const RowParts<MQ> x(rows, row, ml, partials, workers);
    if (x.n < 2 || row < used.x || row >= used.y) continue;
    if (x.n <= LJ_SHARES) join_row<MQ>(p, x, row, lane);
    else
      for (int d = 0; d < p.D; d += 128) join_long_row<MQ>(p, x, row, d + 4 * lane, lane);
  }
}

// A CTA a row's 128 elements, a thread a part's maximum and sum (there are fewer SMs than threads).
template <int MQ>
__global__ void __launch_bounds__(32 * LJ_SHARES)
    latent_join_few_kernel(const __grid_constant__ AttnParams p, const int2 *rows,
                           const float2 *ml, const float *partials, int workers) {
  constexpr int AHEAD = 12;
  __shared__ float4 sums[LJ_SHARES][32];
  __shared__ float tops[LJ_SHARES], factor[32 * LJ_SHARES], part_l[32 * LJ_SHARES];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, d = blockIdx.y * 128 + 4 * lane;
  const bool in = d < p.D;
  const int2 used = rows_in_use(p);
  const RowParts<MQ> x(rows, blockIdx.x, ml, partials, workers);
  if (x.n < 2 || static_cast<int>(blockIdx.x) < used.x || static_cast<int>(blockIdx.x) >= used.y)
    return;
  const int per = (x.n + LJ_SHARES - 1) / LJ_SHARES, lo = min(warp * per, x.n);
  const int hi = min(lo + per, x.n);
  float4 u[AHEAD];
#pragma unroll
  for (int e = 0; e < AHEAD; ++e)
    if (lo + e < hi && in) u[e] = x.out(lo + e, d);
  const float2 one = tid < x.n ? x.ml(tid) : make_float2(-INFINITY, 0.0f);
  float m = one.x;
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, e));
  if (lane == 0) tops[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < LJ_SHARES; ++i) m = fmaxf(m, tops[i]);
  const float f = ex2(one.x - (m == -INFINITY ? 0.0f : m));
  factor[tid] = f;
  part_l[tid] = one.y;
  __syncthreads();
  float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i0 = lo;;) {
#pragma unroll
    for (int e = 0; e < AHEAD; ++e)
      if (i0 + e < hi && in) w = fused(factor[i0 + e], u[e], w);
    i0 += AHEAD;
    if (i0 >= hi) break;
#pragma unroll
    for (int e = 0; e < AHEAD; ++e)
      if (i0 + e < hi && in) u[e] = x.out(i0 + e, d);
  }
  sums[warp][lane] = w;
  __syncthreads();
  if (warp > 0) return;
  float l = 0.0f;
  for (int i = lane; i < x.n; i += 32) l = __fmaf_rn(factor[i], part_l[i], l);
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, e));
  float4 v = sums[0][lane];
#pragma unroll
  for (int i = 1; i < LJ_SHARES; ++i)
    if (i * per < x.n) v = plus(v, sums[i][lane]);
  put_row(p, blockIdx.x, d, v, m, l);
}

// The kernel for few rows while its CTAs fit two to an SM. us of latent_decode with it / with the other
// (CTAs; sequences of tokens each x heads):
//   64 CTAs,  1 x 777 x 16        9.2 / 13.2     256,  4 x 20000 x 16     27.5 /  55.3
//   256,      1 x 131072 x 64    43.2 / 145.6    512,  8 x 100 x 16       14.9 /   9.4
//   512,      8 x 777 x 16       15.7 / 16.2     512,  1 x 131072 x 128   62.9 / 115.7
//   1024,    16 x 100 x 16       20.6 /  9.6    1024, 16 x 20000 x 16     76.3 /  72.0
//   4096,    64 to 8192 x 16    102.0 / 63.2    1024,  one of 40000 and 15 of 100 x 16  21.9 / 91.8
// Beyond two an SM short sequences decide for the other kernel; a row of more than 16 parts then waits
// for one warp (all lengths are on the device).
template <int MQ>
cudaError_t launch_join(const AttnParams &p, const LatentLaunch &a, cudaStream_t s) {
  const int all = p.T * p.Hq, cuts = (p.D + 127) / 128, most = 3 * a.num_sms;
  const bool few = all * cuts <= 2 * a.num_sms && a.num_sms <= 32 * LJ_SHARES;
  const int ctas = (all + 7) / 8;
  return launch_pdl(few ? latent_join_few_kernel<MQ> : latent_join_kernel<MQ>,
                    few ? dim3(all, cuts) : dim3(ctas < most ? ctas : most),
                    dim3(few ? 32 * LJ_SHARES : 256), 0, s, p, static_cast<const int2 *>(a.rows),
                    static_cast<const float2 *>(a.ml), static_cast<const float *>(a.partials),
                    a.num_sms);
}

}  // namespace

cudaError_t launch_latent_join(const AttnParams &p, int rows, const LatentLaunch &a,
                               cudaStream_t s) {
  return rows == 16 ? launch_join<16>(p, a, s)
                    : (rows == 32 ? launch_join<32>(p, a, s) : launch_join<64>(p, a, s));
}

}  // namespace ssd
