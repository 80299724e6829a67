// latent_join.cu -- joins the parts of latent_decode's rows that lie in several CTAs:
// out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i over a row's parts, in their order.
//
// Reads what the parts hold (fp32, in L2 since just before) and writes the row: latencies bound
// it. A warp has a row of up to 8 parts, all of them requested at once; a CTA one of more parts,
// a quarter of them each four warps. Rows go around the CTAs so that an item's lie in many.
#include "latent.h"
#include "attn_kernel.cuh"

namespace ssd {
namespace {

constexpr int LJ_THREADS = 512, LJ_WARPS = LJ_THREADS / 32, LJ_FEW = 8;

template <int MQ>
__global__ void __launch_bounds__(LJ_THREADS, 1) latent_join_kernel(
    const __grid_constant__ AttnParams p, const int2 *rows, const float *partials,
    const int workers) {
  constexpr int DP = LATENT_MAX_R, SLOT = MQ * DP + 2 * MQ;
  __shared__ int2 many[LJ_WARPS];  // rows of more parts: row, first worker; parts beside
  __shared__ int many_parts[LJ_WARPS], n_many;
  __shared__ float factor[2048], red[2][LJ_WARPS];
  __shared__ float4 sums[3][128];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, H = p.Hq;
  const int all = p.T * H;
  const float v_scale = p.c.v_scale ? p.c.v_scale[0] : 1.0f;
  for (int base = blockIdx.x; base < all; base += gridDim.x * LJ_WARPS) {
    if (tid == 0) n_many = 0;
    __syncthreads();
    const int row = base + warp * gridDim.x;
    int c0 = 0, parts = 0, r = 0;
    if (row < all) {
      const int2 x = __ldcg(rows + row);  // kept in bounds, whatever stands there
      r = (x.x >> 16) & (MQ - 1);
      c0 = min(x.x & 0xffff, workers - 1);
      parts = min(x.y, workers - c0);
    }
    auto part = [&](int first, int i, int at) {
      return partials + static_cast<size_t>(part_slot(first, i)) * SLOT + at;
    };
    auto store = [&](int at, int d, float4 v, float inv) {
      const int t = at / H;
      uint2 u;
      u.x = pack2<false>(v.x * inv, v.y * inv);
      u.y = pack2<false>(v.z * inv, v.w * inv);
      if (inv == 0.0f) u = make_uint2(0u, 0u);
      *reinterpret_cast<uint2 *>(p.out + t * p.out_stride +
                                 static_cast<long long>(at - t * H) * p.D + d) = u;
    };
    auto put_lse = [&](int at, float m, float l) {
      if (p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2;
    };
    if (parts > LJ_FEW) {
      if (lane == 0) {
        const int i = atomicAdd(&n_many, 1);
        many[i] = make_int2(row, c0 | r << 16);
        many_parts[i] = parts;
      }
    } else if (parts > 1) {
      float f[LJ_FEW], m = -INFINITY, l = 0.0f;
      {
        float2 ml[LJ_FEW];
#pragma unroll
        for (int i = 0; i < LJ_FEW; ++i) {
          ml[i] = make_float2(-INFINITY, 0.0f);
          if (i < parts)
            ml[i] = __ldcg(reinterpret_cast<const float2 *>(part(c0, i, MQ * DP + 2 * r)));
        }
#pragma unroll
        for (int i = 0; i < LJ_FEW; ++i) m = fmaxf(m, ml[i].x);
        const float b = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < LJ_FEW; ++i) {
          f[i] = ex2(ml[i].x - b);
          l += f[i] * ml[i].y;
        }
      }
      const float inv = l == 0.0f ? 0.0f : v_scale / l;
#pragma unroll 2
      for (int d = 4 * lane; d < p.D; d += 128) {
        float4 u[LJ_FEW];
#pragma unroll
        for (int i = 0; i < LJ_FEW; ++i)
          if (i < parts) u[i] = __ldcg(reinterpret_cast<const float4 *>(part(c0, i, r * DP + d)));
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < LJ_FEW; ++i)
          if (i < parts) {
            v.x += f[i] * u[i].x;
            v.y += f[i] * u[i].y;
            v.z += f[i] * u[i].z;
            v.w += f[i] * u[i].w;
          }
        store(row, d, v, inv);
      }
      if (lane == 0) put_lse(row, m, l);
    }
    __syncthreads();
    for (int x = 0; x < n_many; ++x) {
      // the row by all threads: factors, then a quarter of the parts each 128 threads
      const int at = many[x].x, first = many[x].y & 0xffff, mr = many[x].y >> 16;
      const int n = many_parts[x];
      float m = -INFINITY, l = 0.0f;
      float2 mine[4];  // at most 2048 parts
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        mine[e] = make_float2(-INFINITY, 0.0f);
        if (tid + e * LJ_THREADS < n)
          mine[e] = __ldcg(reinterpret_cast<const float2 *>(
              part(first, tid + e * LJ_THREADS, MQ * DP + 2 * mr)));
        m = fmaxf(m, mine[e].x);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      if (lane == 0) red[0][warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < LJ_WARPS; ++w) m = fmaxf(m, red[0][w]);
      const float b = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (tid + e * LJ_THREADS < n) {
          const float f = ex2(mine[e].x - b);
          factor[tid + e * LJ_THREADS] = f;
          l += f * mine[e].y;
        }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      if (lane == 0) red[1][warp] = l;
      __syncthreads();
      l = 0.0f;
#pragma unroll
      for (int w = 0; w < LJ_WARPS; ++w) l += red[1][w];
      const int q = tid >> 7, d = 4 * (tid & 127), per = (n + 3) / 4;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (d < p.D) {
#pragma unroll 8
        for (int i = q * per; i < min(n, (q + 1) * per); ++i) {
          const float4 u = __ldcg(reinterpret_cast<const float4 *>(part(first, i, mr * DP + d)));
          const float f = factor[i];
          v.x += f * u.x;
          v.y += f * u.y;
          v.z += f * u.z;
          v.w += f * u.w;
        }
      }
      if (q > 0) sums[q - 1][tid & 127] = v;
      __syncthreads();
      if (q == 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const float4 u = sums[i][tid];
          v.x += u.x;
          v.y += u.y;
          v.z += u.z;
          v.w += u.w;
        }
        if (d < p.D) store(at, d, v, l == 0.0f ? 0.0f : v_scale / l);
        if (tid == 0) put_lse(at, m, l);
      }
      __syncthreads();
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_latent_join(const AttnParams &p, int rows, const LatentLaunch &a,
                               cudaStream_t s) {
  const long long all = static_cast<long long>(p.T) * p.Hq, most = 2ll * a.num_sms;
  const dim3 grid(static_cast<unsigned>(all < most ? all : most));
  auto kernel = rows == 16 ? latent_join_kernel<16>
                           : (rows == 32 ? latent_join_kernel<32> : latent_join_kernel<64>);
  return launch_pdl(kernel, grid, dim3(LJ_THREADS), 0, s, p, static_cast<const int2 *>(a.rows),
                    static_cast<const float *>(a.partials), a.num_sms);
}

}  // namespace ssd
