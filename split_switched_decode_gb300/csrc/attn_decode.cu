// attn_decode.cu -- attention of new tokens over a paged key-value cache.
#include <cuda_fp8.h>

#include "attn.h"
#include "common.cuh"

namespace ssd {
namespace {

// The simplest form: one warp per (row, head), a key at a time with the running maximum
// and sum, lane l holding elements l, l + 32, ... of q and of the output.
template <bool E4M3>
__global__ void __launch_bounds__(32) attn_simple_kernel(const AttnParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x;
  const int hk = hq / (p.Hq / p.Hkv);
  int s = t, first = t, rows = 1;
  if (p.q_start) {
    int lo = -1;
    for (s = 0; s < p.S; ++s)
      if (p.q_start[s] <= t && t < p.q_start[s + 1]) { lo = s; break; }
    if (lo < 0) return;
    first = max(p.q_start[s], 0);
    rows = min(p.q_start[s + 1], p.T) - first;
  }
  const long long cap = static_cast<long long>(p.max_pages) * p.c.page_size;
  const int len = static_cast<int>(min(static_cast<long long>(max(p.seq_len[s], 0)), cap));
  const int pos = len - rows + (t - first);
  const int begin = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  constexpr int PER = ATTN_MAX_D / 32;
  float q[PER], o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < p.D ? bf16_to_f32(p.q[t * p.q_stride + hq * p.D + d]) : 0.0f;
    o[i] = 0.0f;
  }
  const float ks = p.scale * (p.c.k_scale ? p.c.k_scale[hk] : 1.0f);
  const float vs = p.c.v_scale ? p.c.v_scale[hk] : 1.0f;
  auto load = [&](const void *base, long long i) {
    if (E4M3) {
      __nv_fp8_e4m3 x;
      x.__x = static_cast<const uint8_t *>(base)[i];
      return static_cast<float>(x);
    }
    return bf16_to_f32(static_cast<const uint16_t *>(base)[i]);
  };
  float m = -INFINITY, l = 0.0f;
  for (int j = begin; j <= pos; ++j) {
    const int page = p.block_table[static_cast<long long>(s) * p.max_pages + j / p.c.page_size];
    if (page < 0 || page >= p.c.num_pages) continue;
    const long long at = page * p.c.page_stride + hk * p.c.head_stride +
                         j % p.c.page_size * p.c.token_stride;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 32 * i < p.D) dot += q[i] * load(p.c.k, at + lane + 32 * i);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    const float x = dot * ks, mn = fmaxf(m, x);
    const float base = mn == -INFINITY ? 0.0f : mn;
    const float f = expf(m - base), w = expf(x - base);
    l = l * f + w;
    m = mn;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 32 * i < p.D) o[i] = o[i] * f + w * load(p.c.v, at + lane + 32 * i);
  }
  const bool none = m == -INFINITY && !(l != l);
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (lane + 32 * i < p.D)
      p.out[t * p.out_stride + hq * p.D + lane + 32 * i] =
          f32_to_bf16_rn(none ? 0.0f : o[i] / l * vs);
  if (p.lse && lane == 0)
    p.lse[static_cast<long long>(t) * p.Hq + hq] = none ? -INFINITY : m + logf(l);
}

}  // namespace

size_t attn_workspace_bytes(int, int, int, int, int, int) { return 16; }

cudaError_t launch_attn_decode(const AttnParams &p, bool e4m3, void *, int, cudaStream_t s) {
  return launch_pdl(e4m3 ? attn_simple_kernel<true> : attn_simple_kernel<false>,
                    dim3(p.T, p.Hq), dim3(32), 0, s, p);
}

}  // namespace ssd
