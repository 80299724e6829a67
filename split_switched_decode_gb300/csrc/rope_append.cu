// rope_append.cu -- rotary positions and the write of new keys and values into the paged
// cache.
#include <cuda_fp8.h>

#include "attn.h"
#include "common.cuh"

namespace ssd {
namespace {

constexpr int RA_THREADS = 256;
constexpr float E4M3_MAX = 448.0f;

__device__ __forceinline__ uint8_t to_e4m3(float x) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3));
}

// magnitude * (cos, sin) of position * frequency. The turn count is reduced in double
// precision (a fp32 product at position 131072 is off by up to 0.004 radians).
__device__ __forceinline__ float2 rope_angle(int pos, float freq, float magnitude) {
  const double turns = static_cast<double>(pos) * static_cast<double>(freq) *
                       0.15915494309189533576888376337251;  // 1 / (2 pi)
  const float r = static_cast<float>(turns - rint(turns));  // [-1/2, 1/2]
  float s, c;
  sincospif(2.0f * r, &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}

// One CTA per row: the row's angles once into shared memory, then a thread per element.
template <bool E4M3>
__global__ void __launch_bounds__(RA_THREADS) rope_append_kernel(const RopeParams p) {
  __shared__ float2 cs[ATTN_MAX_D / 2];
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x, D = p.D, half = p.rot / 2;
  const int pos = p.positions[t];
  for (int i = threadIdx.x; i < half; i += RA_THREADS)
    cs[i] = rope_angle(pos, p.inv_freq[i], p.magnitude);
  __syncthreads();
  const long long slot = p.slots[t];
  const bool stored = slot >= 0 && slot < static_cast<long long>(p.c.num_pages) * p.c.page_size;
  const long long at = stored ? slot / p.c.page_size * p.c.page_stride +
                                    slot % p.c.page_size * p.c.token_stride
                              : 0;
  auto put = [&](const void *base, const float *scale, int h, int d, float x) {
    const long long i = at + h * p.c.head_stride + d;
    if (E4M3) {
      if (scale) x /= scale[h];
      static_cast<uint8_t *>(const_cast<void *>(base))[i] = to_e4m3(x);
    } else {
      static_cast<uint16_t *>(const_cast<void *>(base))[i] = f32_to_bf16_rn(x);
    }
  };
  const int units = D / 2;  // a thread handles two elements: a pair, or two that stay
  for (int u = threadIdx.x; u < (p.Hq + 2 * p.Hkv) * units; u += RA_THREADS) {
    const int h = u / units, i = u - h * units;
    const bool pair = i < half;
    const int d0 = pair && !p.interleaved ? i : 2 * i;
    const int d1 = pair && !p.interleaved ? i + half : 2 * i + 1;
    const uint16_t *src = h < p.Hq ? p.q + t * p.q_stride + h * D
                          : h < p.Hq + p.Hkv
                              ? p.k + t * p.k_stride + (h - p.Hq) * D
                              : p.v + t * p.v_stride + (h - p.Hq - p.Hkv) * D;
    float x0 = bf16_to_f32(src[d0]), x1 = bf16_to_f32(src[d1]);
    if (pair && h < p.Hq + p.Hkv) {
      const float2 a = cs[i];
      const float y0 = x0 * a.x - x1 * a.y;
      x1 = x1 * a.x + x0 * a.y;
      x0 = y0;
    }
    if (h < p.Hq) {
      uint16_t *o = p.q_out + t * p.out_stride + h * D;
      o[d0] = f32_to_bf16_rn(x0);
      o[d1] = f32_to_bf16_rn(x1);
    } else if (stored) {
      const bool key = h < p.Hq + p.Hkv;
      const int hh = key ? h - p.Hq : h - p.Hq - p.Hkv;
      put(key ? p.c.k : p.c.v, key ? p.c.k_scale : p.c.v_scale, hh, d0, x0);
      put(key ? p.c.k : p.c.v, key ? p.c.k_scale : p.c.v_scale, hh, d1, x1);
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams &p, bool e4m3, cudaStream_t s) {
  return launch_pdl(e4m3 ? rope_append_kernel<true> : rope_append_kernel<false>, dim3(p.T),
                    dim3(RA_THREADS), 0, s, p);
}

}  // namespace ssd
