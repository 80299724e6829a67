// api_attn.cu -- host side of the attention entry points of
// include/split_switched_decode.h: kv_plan, rope_frequencies, rope_append, attn_decode.
#include <atomic>
#include <cmath>

#include "../../include/split_switched_decode.h"
#include "attn.h"
#include "common.cuh"

using namespace ssd;

namespace {

std::atomic<int> g_attn_hold{0};  // dec_debug_attn_timeout

bool off(const void *p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}
dec_status status_of(cudaError_t e) { return e == cudaSuccess ? DEC_OK : DEC_ERR_CUDA; }

// The cache arguments that rope_append and attn_decode share.
dec_status check_cache(const void *k, const void *v, int kv_type, const float *k_scale,
                       const float *v_scale, int num_pages, int page_size, int64_t page_stride,
                       int64_t head_stride, int64_t token_stride, int Hkv, int D) {
  if (!k || !v || num_pages < 1 || page_size < 1) return DEC_ERR_INVALID_ARG;
  if (kv_type != DEC_KV_BF16 && kv_type != DEC_KV_E4M3) return DEC_ERR_INVALID_ARG;
  if (D < 1 || Hkv < 1 || page_stride < 0 || head_stride < 0 || token_stride < 0)
    return DEC_ERR_INVALID_ARG;
  if (D % 16 != 0 || D > ATTN_MAX_D || Hkv > ATTN_MAX_HEADS) return DEC_ERR_UNSUPPORTED_SHAPE;
  // a slot is an int32, and an element offset stays inside 2^62
  if (static_cast<int64_t>(num_pages) * page_size > INT32_MAX) return DEC_ERR_UNSUPPORTED_SHAPE;
  const int64_t most = int64_t(1) << 40;
  if (page_stride > most || head_stride > most || token_stride > most)
    return DEC_ERR_UNSUPPORTED_SHAPE;
  const int64_t unit = kv_type == DEC_KV_E4M3 ? 16 : 8;  // elements in 16 bytes
  if (off(k, 16) || off(v, 16) || page_stride % unit || head_stride % unit ||
      token_stride % unit || off(k_scale, 4) || off(v_scale, 4))
    return DEC_ERR_MISALIGNED;
  return DEC_OK;
}

PagedCache cache_of(const void *k, const void *v, const float *k_scale, const float *v_scale,
                    int num_pages, int page_size, int64_t page_stride, int64_t head_stride,
                    int64_t token_stride) {
  PagedCache c;
  c.k = k;
  c.v = v;
  c.k_scale = k_scale;
  c.v_scale = v_scale;
  c.page_stride = page_stride;
  c.head_stride = head_stride;
  c.token_stride = token_stride;
  c.num_pages = num_pages;
  c.page_size = page_size;
  return c;
}

}  // namespace

namespace ssd {
bool host_attn_hold() { return g_attn_hold.load() != 0; }
}  // namespace ssd

extern "C" {

dec_status kv_plan(const int32_t *kv_len, const int32_t *new_len, int S, int page_size,
                   int32_t *block_table, int max_pages, const int32_t *free_pages, int num_free,
                   const int32_t *free_used, int32_t *seq_len, int32_t *q_start,
                   int32_t *positions, int32_t *slots, int max_tokens, int32_t *summary,
                   dec_stream_t s) {
  if (!kv_len || !block_table || !seq_len || !q_start || !positions || !slots || !summary)
    return DEC_ERR_INVALID_ARG;
  if (S < 1 || page_size < 1 || max_pages < 1 || num_free < 0 || max_tokens < 1)
    return DEC_ERR_INVALID_ARG;
  if (num_free > 0 && !free_pages) return DEC_ERR_INVALID_ARG;
  if (S > ATTN_MAX_SEQS || max_tokens > (1 << 28)) return DEC_ERR_UNSUPPORTED_SHAPE;
  if (off(kv_len, 4) || off(new_len, 4) || off(block_table, 4) || off(free_pages, 4) ||
      off(free_used, 4) || off(seq_len, 4) || off(q_start, 4) || off(positions, 4) ||
      off(slots, 4) || off(summary, 4))
    return DEC_ERR_MISALIGNED;
  cudaError_t ce;
  if (host_num_sms(&ce) <= 0) return DEC_ERR_CUDA;
  if (host_consume_fault()) return DEC_ERR_CUDA;
  KvPlanParams p;
  p.kv_len = kv_len;
  p.new_len = new_len;
  p.S = S;
  p.page_size = page_size;
  p.block_table = block_table;
  p.max_pages = max_pages;
  p.free_pages = free_pages;
  p.num_free = num_free;
  p.free_used = free_used;
  p.seq_len = seq_len;
  p.q_start = q_start;
  p.positions = positions;
  p.slots = slots;
  p.max_tokens = max_tokens;
  p.summary = summary;
  return status_of(launch_kv_plan(p, reinterpret_cast<cudaStream_t>(s)));
}

dec_status rope_frequencies(int rot, double base, int scaling, double factor, int orig_len,
                            double beta_fast, double beta_slow, float *inv_freq,
                            float *magnitude) {
  if (!inv_freq || !magnitude) return DEC_ERR_INVALID_ARG;
  if (rot < 2 || rot > ATTN_MAX_D || rot % 2 != 0) return DEC_ERR_INVALID_ARG;
  // written so that a NaN fails
  if (!(base > 1.0) || !(factor >= 1.0) || std::isinf(base) || std::isinf(factor))
    return DEC_ERR_INVALID_ARG;
  if (scaling < DEC_ROPE_PLAIN || scaling > DEC_ROPE_PARTS) return DEC_ERR_INVALID_ARG;
  if (scaling == DEC_ROPE_BASE) {
    if (rot < 4) return DEC_ERR_INVALID_ARG;
    base *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
  }
  double lo = 0.0, width = 1.0;
  if (scaling == DEC_ROPE_PARTS) {
    if (orig_len < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || std::isinf(beta_fast))
      return DEC_ERR_INVALID_ARG;
    // the pair that turns `turns` times within orig_len tokens
    const double two_pi = 6.283185307179586476925286766559;
    auto pair_of = [&](double turns) {
      return rot * std::log(orig_len / (turns * two_pi)) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
    const double hi = std::fmin(std::ceil(pair_of(beta_slow)), rot - 1.0);
    width = std::fmax(hi - lo, 1e-3);
  }
  *magnitude = 1.0f;
  if (scaling == DEC_ROPE_PARTS) *magnitude = static_cast<float>(0.1 * std::log(factor) + 1.0);
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == DEC_ROPE_LINEAR) f /= factor;
    if (scaling == DEC_ROPE_PARTS) {
      const double ramp = std::fmin(std::fmax((i - lo) / width, 0.0), 1.0);
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    inv_freq[i] = static_cast<float>(f);
  }
  return DEC_OK;
}

dec_status rope_append(const dec_bf16 *q, int64_t q_stride, const dec_bf16 *k, int64_t k_stride,
                       const dec_bf16 *v, int64_t v_stride, const int32_t *positions,
                       const int32_t *slots, const float *inv_freq, float magnitude, int T,
                       int Hq, int Hkv, int D, int rot, int interleaved, dec_bf16 *q_out,
                       int64_t q_out_stride, void *k_cache, void *v_cache, int kv_type,
                       const float *k_scale, const float *v_scale, int num_pages, int page_size,
                       int64_t page_stride, int64_t head_stride, int64_t token_stride,
                       dec_stream_t s) {
  if (!q || !k || !v || !positions || !slots || !q_out) return DEC_ERR_INVALID_ARG;
  if (T < 1 || Hq < 1 || rot < 0 || (interleaved != 0 && interleaved != 1))
    return DEC_ERR_INVALID_ARG;
  const dec_status st = check_cache(k_cache, v_cache, kv_type, k_scale, v_scale, num_pages,
                                    page_size, page_stride, head_stride, token_stride, Hkv, D);
  if (st != DEC_OK) return st;
  if (rot % 2 != 0 || rot > D || (rot > 0 && !inv_freq)) return DEC_ERR_INVALID_ARG;
  if (T > (1 << 20) || Hq > ATTN_MAX_HEADS) return DEC_ERR_UNSUPPORTED_SHAPE;
  const int64_t most = int64_t(1) << 40;
  if (q_stride > most || k_stride > most || v_stride > most || q_out_stride > most)
    return DEC_ERR_UNSUPPORTED_SHAPE;
  // rows that overlap: only a single row may have any stride
  const int64_t qn = static_cast<int64_t>(Hq) * D, kn = static_cast<int64_t>(Hkv) * D;
  if (T > 1 && (q_stride < qn || q_out_stride < qn || k_stride < kn || v_stride < kn))
    return DEC_ERR_INVALID_ARG;
  if (off(q, 16) || off(k, 16) || off(v, 16) || off(q_out, 16) || off(positions, 4) ||
      off(slots, 4) || off(inv_freq, 4))
    return DEC_ERR_MISALIGNED;
  if (T > 1 && (q_stride % 8 || k_stride % 8 || v_stride % 8 || q_out_stride % 8))
    return DEC_ERR_MISALIGNED;
  // in place means exactly in place
  const dec_bf16 *q_end = q + (T > 1 ? (T - 1) * q_stride : 0) + qn;
  const dec_bf16 *o_end = q_out + (T > 1 ? (T - 1) * q_out_stride : 0) + qn;
  if (q == q_out) {
    if (T > 1 && q_stride != q_out_stride) return DEC_ERR_INVALID_ARG;
  } else if (T == 1 && q < o_end && q_out < q_end) {
    return DEC_ERR_INVALID_ARG;
  }
  cudaError_t ce;
  const int sms = host_num_sms(&ce);
  if (sms <= 0) return DEC_ERR_CUDA;
  if (host_consume_fault()) return DEC_ERR_CUDA;
  RopeParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.out_stride = q_out_stride;
  p.positions = positions;
  p.slots = slots;
  p.inv_freq = inv_freq;
  p.magnitude = magnitude;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.rot = rot;
  p.interleaved = interleaved;
  p.q_out = q_out;
  p.c = cache_of(k_cache, v_cache, k_scale, v_scale, num_pages, page_size, page_stride,
                 head_stride, token_stride);
  return status_of(launch_rope_append(p, kv_type == DEC_KV_E4M3, sms,
                                      reinterpret_cast<cudaStream_t>(s)));
}

size_t attn_decode_workspace_bytes(int S, int T, int Hq, int Hkv, int D) {
  if (S < 1 || S > ATTN_MAX_SEQS || T < 1 || T > 65536 || Hq < 1 || Hq > ATTN_MAX_HEADS ||
      Hkv < 1 || Hq % Hkv != 0 || D < 16 || D > ATTN_MAX_D || D % 16 != 0)
    return 0;
  cudaError_t ce;
  const int sms = host_num_sms(&ce);
  return sms > 0 ? attn_workspace_bytes(S, T, Hq, Hkv, D, sms) : 0;
}

dec_status attn_decode(const dec_bf16 *q, int64_t q_stride, const void *k_cache,
                       const void *v_cache, int kv_type, const float *k_scale,
                       const float *v_scale, int num_pages, int page_size, int64_t page_stride,
                       int64_t head_stride, int64_t token_stride, const int32_t *block_table,
                       int max_pages, const int32_t *seq_len, const int32_t *q_start, int S,
                       int T, int Hq, int Hkv, int D, float scale, int window, dec_bf16 *out,
                       int64_t out_stride, float *lse_opt, void *ws, size_t ws_bytes,
                       dec_stream_t s) {
  if (!q || !block_table || !seq_len || !out || !ws) return DEC_ERR_INVALID_ARG;
  if (S < 1 || T < 1 || Hq < 1 || max_pages < 1 || window < 0) return DEC_ERR_INVALID_ARG;
  if (!q_start && T != S) return DEC_ERR_INVALID_ARG;
  const dec_status st = check_cache(k_cache, v_cache, kv_type, k_scale, v_scale, num_pages,
                                    page_size, page_stride, head_stride, token_stride, Hkv, D);
  if (st != DEC_OK) return st;
  if (Hq % Hkv != 0) return DEC_ERR_INVALID_ARG;
  if (S > ATTN_MAX_SEQS || T > 65536 || Hq > ATTN_MAX_HEADS) return DEC_ERR_UNSUPPORTED_SHAPE;
  const int64_t most = int64_t(1) << 40, qn = static_cast<int64_t>(Hq) * D;
  if (q_stride > most || out_stride > most) return DEC_ERR_UNSUPPORTED_SHAPE;
  if (T > 1 && (q_stride < 0 || out_stride < qn)) return DEC_ERR_INVALID_ARG;
  if (off(q, 16) || off(out, 16) || off(block_table, 4) || off(seq_len, 4) || off(q_start, 4) ||
      off(lse_opt, 4) || off(ws, 16))
    return DEC_ERR_MISALIGNED;
  if (T > 1 && (q_stride % 8 || out_stride % 8)) return DEC_ERR_MISALIGNED;
  if (q == out) return DEC_ERR_INVALID_ARG;
  cudaError_t ce;
  const int sms = host_num_sms(&ce);
  if (sms <= 0) return DEC_ERR_CUDA;
  if (ws_bytes < attn_workspace_bytes(S, T, Hq, Hkv, D, sms)) return DEC_ERR_WORKSPACE_TOO_SMALL;
  if (host_consume_fault()) return DEC_ERR_CUDA;
  AttnParams p;
  p.q = q;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.c = cache_of(k_cache, v_cache, k_scale, v_scale, num_pages, page_size, page_stride,
                 head_stride, token_stride);
  p.block_table = block_table;
  p.seq_len = seq_len;
  p.q_start = q_start;
  p.max_pages = max_pages;
  p.S = S;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.scale = scale;
  p.window = window;
  p.out = out;
  p.lse = lse_opt;
  uint64_t limit = 0;
  unsigned *status = host_wait_status(&limit);
  return status_of(launch_attn_decode(p, kv_type == DEC_KV_E4M3, ws, sms, status, limit,
                                      host_attn_hold(),
                                      reinterpret_cast<cudaStream_t>(s)));
}

dec_status dec_debug_attn_timeout(int on) {
  if (on != 0 && on != 1) return DEC_ERR_INVALID_ARG;
  g_attn_hold.store(on);
  return DEC_OK;
}

}  // extern "C"
