// latent_join.cu -- joins the parts of latent_decode's rows that lie in several CTAs:
// out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i over a row's parts, in their order.
//
// Reads what the parts hold (fp32, in L2 since just before) and writes the row: latencies bound
// it. A warp has 128 elements of a row; of up to four parts everything is requested at once.
// While rows are few, 16 warps share a row's parts. Sums are those of a sixteenth of the parts
// each, added in order, either way: the bits of a row depend on its parts alone.
#include "attn_kernel.cuh"
#include "latent.h"

namespace ssd {
namespace {

constexpr int LJ_SHARES = 16, LJ_FEW = 4;

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

template <int MQ, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 512 : 256, WIDE ? 1 : 4) latent_join_kernel(
    const __grid_constant__ AttnParams p, const int2 *rows, const float2 *ml_at,
    const float *partials, const int workers) {
  constexpr int DP = LATENT_MAX_R, SLOT = MQ * DP, AHEAD = WIDE ? 8 : 4;
  constexpr int PER_CTA = WIDE ? 1 : 8;
  __shared__ float4 sums[WIDE ? LJ_SHARES : 1][32];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, H = p.Hq;
  const int cuts = (p.D + 127) >> 7;  // 128-element parts of a row
  const long long units = static_cast<long long>(p.T) * H * cuts;
  const float v_scale = p.c.v_scale ? p.c.v_scale[0] : 1.0f;
  for (long long base = static_cast<long long>(blockIdx.x) * PER_CTA; base < units;
       base += static_cast<long long>(gridDim.x) * PER_CTA) {
    const long long unit = WIDE ? base : base + warp;
    int row = 0, d = 0, c0 = 0, n = 0, r = 0;
    if (unit < units) {
      row = static_cast<int>(unit / cuts);
      d = static_cast<int>(unit - static_cast<long long>(row) * cuts) * 128 + 4 * lane;
      const int2 x = __ldcg(rows + row);  // kept in bounds, whatever stands there
      r = (x.x >> 16) & (MQ - 1);
      c0 = min(x.x & 0xffff, workers - 1);
      n = max(min(x.y, workers - c0), 0);
    }
    if (n < 2 && !WIDE) continue;
    auto part = [&](int i) {
      return reinterpret_cast<const float4 *>(
          partials + static_cast<size_t>(part_slot(c0, i)) * SLOT + r * DP + d);
    };
    auto ml_of = [&](int i) {
      return __ldcg(ml_at + (2 * r + (i == 0 ? 1 : 0)) * workers + c0 + i);
    };
    const bool in = d < p.D;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float m = -INFINITY, l = 0.0f;
    if (n <= LJ_FEW) {
      float2 ml[LJ_FEW];
      float4 u[LJ_FEW];
#pragma unroll
      for (int i = 0; i < LJ_FEW; ++i) {
        ml[i] = make_float2(-INFINITY, 0.0f);
        if (i < n) {
          ml[i] = ml_of(i);
          if (in) u[i] = __ldcg(part(i));
        }
        m = fmaxf(m, ml[i].x);
      }
      const float b = m == -INFINITY ? 0.0f : m;
      float x[LJ_FEW];
#pragma unroll
      for (int i = 0; i < LJ_FEW; ++i) {
        const float f = ex2(ml[i].x - b);
        x[i] = __fmul_rn(f, ml[i].y);
        if (i < n && in) v = plus(v, scaled(f, u[i]));
      }
      l = __fadd_rn(__fadd_rn(x[0], x[2]), __fadd_rn(x[1], x[3]));
    } else {
      for (int i = lane; i < n; i += 32) m = fmaxf(m, ml_of(i).x);
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, e));
      const float b = m == -INFINITY ? 0.0f : m;
      const int per = (n + LJ_SHARES - 1) / LJ_SHARES;
      const int lo = WIDE ? min(warp * per, n) : 0, hi = WIDE ? min(lo + per, n) : n;
      int stop = lo + per;  // the end of a share
      float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int i0 = 0; i0 < n; i0 += 32) {
        float f = 0.0f;
        if (i0 + lane < n) {
          const float2 ml = ml_of(i0 + lane);
          f = ex2(ml.x - b);
          l = __fmaf_rn(f, ml.y, l);
        }
        const int from = max(lo, i0), to = min(hi, i0 + 32);
        for (int i = from; i < to; i += AHEAD) {
          float4 u[AHEAD];
#pragma unroll
          for (int e = 0; e < AHEAD; ++e)
            if (i + e < to && in)
              u[e] = __ldcg(part(i + e));
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
      v = plus(v, w);
    }
    if (WIDE && n > LJ_FEW) {  // (the CTA has one row)
      sums[warp][lane] = v;
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int i = 1; i < LJ_SHARES; ++i)
          if (i * ((n + LJ_SHARES - 1) / LJ_SHARES) < n) v = plus(v, sums[i][lane]);
      }
      __syncthreads();
    }
    if (n > 1 && (!WIDE || warp == 0)) {
      const int t = row / H, h = row - t * H;
      const float inv = l == 0.0f ? 0.0f : v_scale / l;
      uint2 u = make_uint2(0u, 0u);  // a row that saw nothing
      if (l != 0.0f) {
        u.x = pack2<false>(v.x * inv, v.y * inv);
        u.y = pack2<false>(v.z * inv, v.w * inv);
      }
      if (in)
        *reinterpret_cast<uint2 *>(p.out + t * p.out_stride + static_cast<long long>(h) * p.D +
                                   d) = u;
      if (d == 0 && p.lse) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2;
    }
  }
}

template <int MQ>
cudaError_t launch_join(const AttnParams &p, const LatentLaunch &a, cudaStream_t s) {
  const long long units = static_cast<long long>(p.T) * p.Hq * ((p.D + 127) / 128);
  // few rows: a CTA of 16 warps each, two an SM
  const bool wide = units <= 2ll * a.num_sms;
  const long long ctas = wide ? units : (units + 7) / 8, most = 4ll * a.num_sms;
  return launch_pdl(wide ? latent_join_kernel<MQ, true> : latent_join_kernel<MQ, false>,
                    dim3(static_cast<unsigned>(ctas < most ? ctas : most)),
                    dim3(wide ? 512 : 256), 0, s, p, static_cast<const int2 *>(a.rows),
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
