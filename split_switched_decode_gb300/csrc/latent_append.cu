// latent_append.cu -- norm, rotary positions and the write of new tokens' latent vectors into
// the paged latent cache.
#include "latent.h"
#include "rope.cuh"

namespace ssd {
namespace {

constexpr int LA_THREADS = 128;

// Elements 8i.. of a rotated part of `rot` elements; x: those, o: those half of the part away (half
// pairs); cs: the row's angles.
template <bool INTER>
__device__ __forceinline__ void turn8(uint4 x, uint4 o, int i, int rot, const float2 *cs,
                                      float (&y)[8]) {
  unpack8(x, y);
  if (8 * i >= rot) return;
  if (INTER) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 w = cs[4 * i + e];
      const float r = y[2 * e] * w.x - y[2 * e + 1] * w.y;
      y[2 * e + 1] = y[2 * e + 1] * w.x + y[2 * e] * w.y;
      y[2 * e] = r;
    }
  } else {
    const int half = rot / 2, d = 8 * i;
    const bool low = d < half;
    float z[8];
    unpack8(o, z);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 w = cs[low ? d + e : d - half + e];
      y[e] = low ? y[e] * w.x - z[e] * w.y : y[e] * w.x + z[e] * w.y;
    }
  }
}
__device__ __forceinline__ uint4 chunk(const uint16_t *x, int i) {
  return *reinterpret_cast<const uint4 *>(x + 8 * i);
}

// Eight elements of a token's row of the cache at element `at`.
template <bool E4M3>
__device__ __forceinline__ void put_cache8(const LatentAppendParams &p, long long at,
                                           const float (&x)[8]) {
  if (!E4M3) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.cache) + at) = pack8(x);
    return;
  }
  const float s = p.scale ? *p.scale : 1.0f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 y = make_float2(x[2 * k] / s, x[2 * k + 1] / s);
    w[k >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3))
                 << (16 * (k & 1));
  }
  *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.cache) + at) = make_uint2(w[0], w[1]);
}

// A CTA a token. Its latent row is one 16-byte chunk a thread (R + P is at most 576), read
// once: the squares are summed over the CTA while the angles are computed. Its query heads are
// units of a thread: a chunk (interleaved pairs, elements that stay) or two chunks half the
// rotary part apart, so that every thread owns what it overwrites and q_out may be q_rope.
// Read once and written once: the copy rate bounds it, the launch's latency when rows are few;
// then a row's heads are cut over gridDim.y, whose first CTA has the latent row. A thread requests
// AHEAD units at a time, the first before the CTA meets. With many rows (MANY) CTAs on an SM hide
// more than units ahead do: 14 or 12 of them with half of the units; with few, registers for units
// are better. us, MANY / not (64 heads, interleaved bf16, half pairs bf16, half pairs e4m3): 8192
// rows 29.3 / 31.8, 32.0 / 33.1, 32.8 / 36.2 (16 heads 15.6 / 18.3, 16.9 / 18.7, 18.5 / 22.6); 2048 rows
// 9.3 / 9.6, 10.8 / 10.3, 11.5 / 10.8; 512 rows 3.8 / 3.4, 4.0 / 3.7, 4.4 / 4.0. 8192 rows of 64 heads with
// rows kept are 163 MB: 5.5 TB/s.
template <bool E4M3, bool INTER, bool MANY>
__global__ void __launch_bounds__(LA_THREADS, MANY ? (INTER ? 14 : 12) : 0)
    latent_append_kernel(const LatentAppendParams p) {
  constexpr int AHEAD = (INTER ? 4 : 2) / (MANY ? 2 : 1);
  __shared__ float2 cs[LATENT_MAX_W / 2];
  __shared__ float sums[LA_THREADS / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x, tid = threadIdx.x, half = p.rot / 2;
  const bool row = blockIdx.y == 0, heads = p.H > 0 && (gridDim.y == 1 || blockIdx.y > 0);
  const int rc = p.R / 8, wc = (p.R + p.P) / 8;
  const int turning = INTER ? p.rot / 8 : p.rot / 16, per = turning + (p.P - p.rot) / 8;
  const int first = gridDim.y == 1 ? 0 : blockIdx.y - 1, every = gridDim.y == 1 ? 1 : gridDim.y - 1;
  const int units = heads ? p.H * per : 0, stride = every * LA_THREADS;
  // unit u: head, chunk, whether its partner half the rotary part on belongs to it
  auto place = [&](int u, int &h, int &c, bool &pair) {
    h = u / per;
    const int i = u - h * per;
    c = INTER || i < turning ? i : p.rot / 8 + i - turning;
    pair = !INTER && i < turning;
  };
  uint4 a[AHEAD], b[INTER ? 1 : AHEAD];
  auto load = [&](int u0) {
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) {
      const int u = u0 + e * stride;
      if (u >= units) break;
      int h, c;
      bool pair;
      place(u, h, c, pair);
      const uint16_t *x = p.q_rope + t * p.q_stride + h * p.q_head;
      a[e] = chunk(x, c);
      if (!INTER && pair) b[INTER ? 0 : e] = chunk(x, c + turning);
    }
  };
  // this row's part of the cache
  uint4 mine = make_uint4(0, 0, 0, 0), partner = mine;
  if (row && tid < rc) {
    mine = chunk(p.c + t * p.c_stride, tid);
  } else if (row && tid < wc) {
    const uint16_t *x = p.k_rope + t * p.k_stride;
    const int i = tid - rc;
    mine = chunk(x, i);
    if (!INTER && 8 * i < p.rot) partner = chunk(x, 8 * i < half ? i + turning : i - turning);
  }
  int u0 = heads ? first * LA_THREADS + tid : units;
  load(u0);
  // the threads after the latent row's have the angles
  const int pos = p.positions[t];
  for (int j = tid >= 64 ? tid - 64 : tid + 64; j < half; j += LA_THREADS)
    cs[j] = rope_angle(pos, p.inv_freq[j], p.magnitude);
  float y[8], sum = 0.0f;
  unpack8(mine, y);
  if (tid < rc) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += y[e] * y[e];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if ((tid & 31) == 0) sums[tid >> 5] = sum;
  __syncthreads();
  if (row && tid < wc) {
    if (tid < rc) {
      if (p.weight) {
        float w[8];
        unpack8(chunk(p.weight, tid), w);
        const float mean = ((sums[0] + sums[1]) + (sums[2] + sums[3])) / p.R;
        const float inv = rsqrtf(mean + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * w[e];
      }
    } else {
      turn8<INTER>(mine, partner, tid - rc, p.rot, cs, y);
    }
    if (p.rows) *reinterpret_cast<uint4 *>(p.rows + t * p.rows_stride + 8 * tid) = pack8(y);
    const int slot = p.slots[t];
    // num_pages * page_size fits an int (checked on the host)
    if (slot >= 0 && slot < p.num_pages * p.page_size) {
      const int page = slot / p.page_size;
      put_cache8<E4M3>(p, page * p.page_stride + (slot - page * p.page_size) * p.token_stride +
                              8 * tid, y);
    }
  }
  while (u0 < units) {
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) {
      const int u = u0 + e * stride;
      if (u >= units) break;
      int h, c;
      bool pair;
      place(u, h, c, pair);
      uint16_t *o = p.q_out + t * p.out_stride + h * p.out_head;
      const uint4 other = INTER ? a[e] : b[INTER ? 0 : e];
      turn8<INTER>(a[e], other, c, p.rot, cs, y);
      *reinterpret_cast<uint4 *>(o + 8 * c) = pack8(y);
      if (pair) {
        turn8<INTER>(other, a[e], c + turning, p.rot, cs, y);
        *reinterpret_cast<uint4 *>(o + 8 * (c + turning)) = pack8(y);
      }
    }
    u0 += AHEAD * stride;
    load(u0);
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendParams &p, bool e4m3, bool interleaved,
                                 int num_sms, cudaStream_t s) {
  // CTAs for one unit a thread while the row count alone does not give every SM two CTAs. us, with /
  // without (interleaved, bf16): 1 row of 64 heads 1.7 / 2.7, of 16 1.7 / 2.1; 64 rows 2.0 / 2.9,
  // 1.9 / 2.3; 256 rows 2.7 / 3.0, 2.0 / 2.4; 303 rows of 64 heads 3.4 / 3.1; 512 rows 4.5 / 3.3,
  // 2.6 / 2.5; 1024 rows of 64 heads 8.0 / 5.1
  const int turning = interleaved ? p.rot / 8 : p.rot / 16;
  const int units = p.H * (turning + (p.P - p.rot) / 8);
  const int cuts = p.T < 2 * num_sms && units > 0 ? 1 + (units + LA_THREADS - 1) / LA_THREADS : 1;
  const bool many = p.T >= 16 * num_sms;
  void (*kernel)(const LatentAppendParams);
  if (many && interleaved)
    kernel = e4m3 ? latent_append_kernel<true, true, true> : latent_append_kernel<false, true, true>;
  else if (many)
    kernel = e4m3 ? latent_append_kernel<true, false, true> : latent_append_kernel<false, false, true>;
  else if (interleaved)
    kernel = e4m3 ? latent_append_kernel<true, true, false> : latent_append_kernel<false, true, false>;
  else
    kernel = e4m3 ? latent_append_kernel<true, false, false> : latent_append_kernel<false, false, false>;
  return launch_pdl(kernel, dim3(p.T, cuts), dim3(LA_THREADS), 0, s, p);
}

}  // namespace ssd
