// rope_append.cu -- rotary positions and the write of new keys and values into the paged
// cache.
#include "attn.h"
#include "rope.cuh"

namespace ssd {
namespace {

constexpr int RA_THREADS = 128;

// Where a row's key and value go in the cache (elements), or not at all.
struct RowPlace {
  bool stored;
  long long at;
};
__device__ __forceinline__ RowPlace row_place(const RopeParams &p, int t) {
  const int slot = p.slots[t];
  RowPlace r;
  // num_pages * page_size fits an int (checked on the host)
  r.stored = slot >= 0 && slot < p.c.num_pages * p.c.page_size;
  const int page = slot / p.c.page_size;
  r.at = r.stored ? page * p.c.page_stride + (slot - page * p.c.page_size) * p.c.token_stride
                  : 0;
  return r;
}

// Eight elements of head h's row into the cache.
template <bool E4M3>
__device__ __forceinline__ void put8(const void *base, const float *scale, int h, long long at,
                                     const float (&x)[8]) {
  if (!E4M3) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(const_cast<void *>(base)) + at) = pack8(x);
    return;
  }
  const float s = scale ? scale[h] : 1.0f;
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 y = make_float2(x[4 * i + 2 * k] / s, x[4 * i + 2 * k + 1] / s);
      w[i] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3))
              << (16 * k);
    }
  }
  *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(const_cast<void *>(base)) + at) =
      make_uint2(w[0], w[1]);
}

// 16 bytes a thread. Read once and written once, 2 to 3 operations an element: the copy rate
// bounds it, the launch's latency when rows are few. A thread's unit is a chunk of 8
// elements with its partner half the rotary part away (half pairs), or alone (interleaved
// pairs, elements that stay), so every thread owns what it overwrites and q_out may
// be q. The row's angles are computed once per CTA into shared memory while the first unit's
// elements are on their way. Rows with many CTAs to spare are cut over gridDim.y so that a
// thread has one unit. Measured: 64 + 2 * 8 heads of 128, 8192 rows (335 MB read and written)
// in 54.8 us, 6.1 TB/s, where a plain copy reaches 6.76; the rest is the starts of 8192 CTAs:
// a second CTA a row costs 4 us more, 192 threads a row 6 (96: the same, but 1 us more for
// 1000 rows). 512 rows into an e4m3 cache take 3.9 us, one row 2.1.
template <bool E4M3, bool INTER>
__global__ void __launch_bounds__(RA_THREADS) rope_append_kernel(const RopeParams p) {
  __shared__ float2 cs[ATTN_MAX_D / 2];
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x, half = p.rot / 2;
  // units of a head: rotary pairs of chunks (half pairs) or chunks, then the rest; values are
  // cut like the other heads
  const int turning = INTER ? p.rot / 8 : p.rot / 16;
  const int per_head = turning + (p.D - p.rot) / 8, heads = p.Hq + 2 * p.Hkv;
  struct Unit {
    int h, d0, d1;  // head counted over q, k, v; first element, partner's (or -1)
    bool turns;
  };
  auto source = [&](int h) {
    return h < p.Hq ? p.q + t * p.q_stride + h * p.D
           : h < p.Hq + p.Hkv ? p.k + t * p.k_stride + (h - p.Hq) * p.D
                              : p.v + t * p.v_stride + (h - p.Hq - p.Hkv) * p.D;
  };
  // this thread's units, every `step`-th: head h, unit i of it (no division on the way)
  const int step = gridDim.y * RA_THREADS, u = blockIdx.y * RA_THREADS + threadIdx.x;
  const int step_h = step / per_head, step_i = step - step_h * per_head;
  int h = u / per_head, i = u - h * per_head;
  // a unit's elements are requested one unit before they are used
  Unit next = {};
  uint4 next_a = {}, next_b = {};
  auto load = [&]() {
    const bool paired = i < turning;
    next.h = h;
    next.d0 = paired || INTER ? 8 * i : p.rot + 8 * (i - turning);
    next.d1 = paired && !INTER ? half + 8 * i : -1;
    next.turns = paired && h < p.Hq + p.Hkv;
    const uint16_t *src = source(next.h);
    next_a = *reinterpret_cast<const uint4 *>(src + next.d0);
    if (next.d1 >= 0) next_b = *reinterpret_cast<const uint4 *>(src + next.d1);
    h += step_h;
    i += step_i;
    if (i >= per_head) {
      i -= per_head;
      ++h;
    }
  };
  bool more = h < heads;
  if (more) load();
  const RowPlace place = row_place(p, t);
  if (threadIdx.x < half) {
    const int pos = p.positions[t];
    for (int j = threadIdx.x; j < half; j += RA_THREADS)
      cs[j] = rope_angle(pos, p.inv_freq[j], p.magnitude);
  }
  __syncthreads();
  while (more) {
    const Unit x = next;
    float y0[8], y1[8];
    unpack8(next_a, y0);
    unpack8(next_b, y1);
    more = h < heads;
    if (more) load();
    if (x.turns && INTER) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 w = cs[x.d0 / 2 + e];
        const float r = y0[2 * e] * w.x - y0[2 * e + 1] * w.y;
        y0[2 * e + 1] = y0[2 * e + 1] * w.x + y0[2 * e] * w.y;
        y0[2 * e] = r;
      }
    } else if (x.turns) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 w = cs[x.d0 + e];
        const float r = y0[e] * w.x - y1[e] * w.y;
        y1[e] = y1[e] * w.x + y0[e] * w.y;
        y0[e] = r;
      }
    }
    if (x.h < p.Hq) {
      uint16_t *o = p.q_out + t * p.out_stride + x.h * p.D;
      *reinterpret_cast<uint4 *>(o + x.d0) = pack8(y0);
      if (x.d1 >= 0) *reinterpret_cast<uint4 *>(o + x.d1) = pack8(y1);
    } else if (place.stored) {
      const bool key = x.h < p.Hq + p.Hkv;
      const int to = key ? x.h - p.Hq : x.h - p.Hq - p.Hkv;
      const void *base = key ? p.c.k : p.c.v;
      const float *scale = key ? p.c.k_scale : p.c.v_scale;
      const long long at = place.at + to * p.c.head_stride;
      put8<E4M3>(base, scale, to, at + x.d0, y0);
      if (x.d1 >= 0) put8<E4M3>(base, scale, to, at + x.d1, y1);
    }
  }
}

// Rotary parts that chunks of 8 do not fit (rot % 16 with half pairs, rot % 8 interleaved): a
// thread per pair of elements, two bytes at a time. 8192 rows of 64 + 2 * 8 heads of 128 with
// 30 or 42 elements rotated take 139 us, where chunks take 55 to 60.
template <bool E4M3>
__global__ void __launch_bounds__(RA_THREADS) rope_append_pairs_kernel(const RopeParams p) {
  __shared__ float2 cs[ATTN_MAX_D / 2];
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x, half = p.rot / 2;
  const int pos = p.positions[t];
  for (int i = threadIdx.x; i < half; i += RA_THREADS)
    cs[i] = rope_angle(pos, p.inv_freq[i], p.magnitude);
  __syncthreads();
  const RowPlace place = row_place(p, t);
  auto put = [&](const void *base, const float *scale, int h, int d, float x) {
    const long long i = place.at + h * p.c.head_stride + d;
    if (E4M3) {
      if (scale) x /= scale[h];
      static_cast<uint8_t *>(const_cast<void *>(base))[i] = to_e4m3(x);
    } else {
      static_cast<uint16_t *>(const_cast<void *>(base))[i] = f32_to_bf16_rn(x);
    }
  };
  const int units = p.D / 2;  // two elements: a pair, or two that stay
  for (int u = blockIdx.y * RA_THREADS + threadIdx.x; u < (p.Hq + 2 * p.Hkv) * units;
       u += gridDim.y * RA_THREADS) {
    const int h = u / units, i = u - h * units;
    const bool pair = i < half;
    const int d0 = pair && !p.interleaved ? i : 2 * i;
    const int d1 = pair && !p.interleaved ? i + half : 2 * i + 1;
    const uint16_t *src = h < p.Hq ? p.q + t * p.q_stride + h * p.D
                          : h < p.Hq + p.Hkv
                              ? p.k + t * p.k_stride + (h - p.Hq) * p.D
                              : p.v + t * p.v_stride + (h - p.Hq - p.Hkv) * p.D;
    float x0 = bf16_to_f32(src[d0]), x1 = bf16_to_f32(src[d1]);
    if (pair && h < p.Hq + p.Hkv) {
      const float2 w = cs[i];
      const float y0 = x0 * w.x - x1 * w.y;
      x1 = x1 * w.x + x0 * w.y;
      x0 = y0;
    }
    if (h < p.Hq) {
      uint16_t *o = p.q_out + t * p.out_stride + h * p.D;
      o[d0] = f32_to_bf16_rn(x0);
      o[d1] = f32_to_bf16_rn(x1);
    } else if (place.stored) {
      const bool key = h < p.Hq + p.Hkv;
      const int hh = key ? h - p.Hq : h - p.Hq - p.Hkv;
      put(key ? p.c.k : p.c.v, key ? p.c.k_scale : p.c.v_scale, hh, d0, x0);
      put(key ? p.c.k : p.c.v, key ? p.c.k_scale : p.c.v_scale, hh, d1, x1);
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams &p, bool e4m3, int num_sms, cudaStream_t s) {
  const bool chunks = p.rot % (p.interleaved ? 8 : 16) == 0;
  const int heads = p.Hq + 2 * p.Hkv;
  // units of a row, and CTAs for one unit a thread while the row count alone does not give
  // every SM two CTAs
  const int turning = p.interleaved ? p.rot / 8 : p.rot / 16;
  const int units = heads * (chunks ? turning + (p.D - p.rot) / 8 : p.D / 2);
  const int cuts = (units + RA_THREADS - 1) / RA_THREADS;
  const dim3 grid(p.T, p.T < 2 * num_sms ? cuts : 1);
  void (*kernel)(const RopeParams);
  if (!chunks)
    kernel = e4m3 ? rope_append_pairs_kernel<true> : rope_append_pairs_kernel<false>;
  else if (p.interleaved)
    kernel = e4m3 ? rope_append_kernel<true, true> : rope_append_kernel<false, true>;
  else
    kernel = e4m3 ? rope_append_kernel<true, false> : rope_append_kernel<false, false>;
  return launch_pdl(kernel, grid, dim3(RA_THREADS), 0, s, p);
}

}  // namespace ssd
