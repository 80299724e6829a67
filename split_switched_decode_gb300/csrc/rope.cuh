// rope.cuh -- rotary angles and eight-element chunks, shared by rope_append.cu and
// latent_append.cu.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace ssd {
namespace {

__device__ __forceinline__ uint8_t to_e4m3(float x) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3));
}

// magnitude * (cos, sin) of position * frequency. The turns, position * frequency / (2 pi), are
// taken modulo one in integers of 2^-64 turns: exact but for position * 2^-64 turns and
// position * frequency * 2^-65, where a fp32 product at position 131072 is off by up to 0.004
// radians. (In double precision the rows of a prompt waited for its few units: 57.4 us for
// 8192 rows instead of 55.8.)
__device__ __forceinline__ float2 rope_angle(int pos, float freq, float magnitude) {
  constexpr uint64_t PER_RADIAN = 2935890503282001226ull;  // 2^64 / (2 pi)
  const uint32_t bits = __float_as_uint(freq), exponent = bits >> 23 & 255;
  const uint32_t mant = (bits & 0x7fffffu) | (exponent ? 0x800000u : 0u);
  // mant * PER_RADIAN, a point `shift` bits from the right: the turns of a step
  const uint64_t lo = mant * PER_RADIAN, hi = __umul64hi(mant, PER_RADIAN);
  const int shift = 150 - static_cast<int>(exponent ? exponent : 1u);
  uint64_t step;
  if (shift > 0 && shift < 64)
    step = lo >> shift | hi << (64 - shift);
  else if (shift >= 64)
    step = shift < 128 ? hi >> (shift - 64) : 0;
  else
    step = shift > -64 ? lo << -shift : 0;
  if (bits >> 31) step = 0 - step;
  const int64_t turns = static_cast<int64_t>(step * static_cast<uint64_t>(
                                                        static_cast<int64_t>(pos)));
  float r = static_cast<float>(turns) * 0x1p-63f;  // in half turns, [-1, 1]
  if (exponent == 255) r = freq - freq;            // not finite
  float s, c;
  sincospif(r, &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  x[0] = bf16lo(v.x), x[1] = bf16hi(v.x), x[2] = bf16lo(v.y), x[3] = bf16hi(v.y);
  x[4] = bf16lo(v.z), x[5] = bf16hi(v.z), x[6] = bf16lo(v.w), x[7] = bf16hi(v.w);
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]),
                    bf16x2(x[6], x[7]));
}

}  // namespace
}  // namespace ssd
