// api_latent.cu -- host side of the latent attention entry points of
// include/split_switched_decode.h: latent_append, latent_project, latent_decode, latent_prompt.
#include <cstring>

#include "../../include/split_switched_decode.h"
#include "common.cuh"
#include "latent.h"

using namespace ssd;

namespace {

constexpr int64_t MOST = int64_t(1) << 38;  // elements of a stride
constexpr int MAX_TOKENS = 1 << 20;

bool off(const void *p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}
dec_status status_of(cudaError_t e) { return e == cudaSuccess ? DEC_OK : DEC_ERR_CUDA; }

// Whether [count, heads, dim] with these strides can be read (written: no two elements in one
// place); strides of counts of one are not looked at.
dec_status check_rows(int count, int heads, int dim, int64_t stride, int64_t head, bool written) {
  if ((count > 1 && stride < 0) || (heads > 1 && head < 0)) return DEC_ERR_INVALID_ARG;
  if ((count > 1 && stride > MOST) || (heads > 1 && head > MOST)) return DEC_ERR_UNSUPPORTED_SHAPE;
  if ((count > 1 && stride < dim) || (heads > 1 && head < dim)) return DEC_ERR_INVALID_ARG;
  if ((count > 1 && stride % 8) || (heads > 1 && head % 8)) return DEC_ERR_MISALIGNED;
  if (written && count > 1 && heads > 1 && stride < (heads - 1) * head + dim &&
      head < (count - 1) * stride + dim)
    return DEC_ERR_INVALID_ARG;
  return DEC_OK;
}

// The cache arguments that latent_append and latent_decode share.
dec_status check_cache(const void *cache, int kv_type, const float *scale, int num_pages,
                       int page_size, int64_t page_stride, int64_t token_stride, int R, int P) {
  if (!cache || num_pages < 1 || page_size < 1 || R < 1 || P < 0) return DEC_ERR_INVALID_ARG;
  if (kv_type != DEC_KV_BF16 && kv_type != DEC_KV_E4M3) return DEC_ERR_INVALID_ARG;
  if (page_stride < 0 || token_stride < 0) return DEC_ERR_INVALID_ARG;
  if (R % 64 || P % 64 || R > LATENT_MAX_R || R + P > LATENT_MAX_W)
    return DEC_ERR_UNSUPPORTED_SHAPE;
  // a slot is an int32, and an element offset stays inside 2^62
  if (static_cast<int64_t>(num_pages) * page_size > INT32_MAX) return DEC_ERR_UNSUPPORTED_SHAPE;
  if (page_stride > MOST || token_stride > MOST) return DEC_ERR_UNSUPPORTED_SHAPE;
  const int64_t unit = kv_type == DEC_KV_E4M3 ? 16 : 8;  // elements in 16 bytes
  if (off(cache, 16) || page_stride % unit || token_stride % unit || off(scale, 4))
    return DEC_ERR_MISALIGNED;
  return DEC_OK;
}

}  // namespace

extern "C" {

dec_status latent_append(const dec_bf16 *c, int64_t c_stride, const dec_bf16 *weight, float eps,
                         const dec_bf16 *k_rope, int64_t k_stride, const dec_bf16 *q_rope,
                         int64_t q_stride, int64_t q_head, const int32_t *positions,
                         const int32_t *slots, const float *inv_freq, float magnitude, int T,
                         int H, int R, int P, int rot, int interleaved, dec_bf16 *q_out,
                         int64_t q_out_stride, int64_t q_out_head, dec_bf16 *rows_opt,
                         int64_t rows_stride, void *cache, int kv_type, const float *cache_scale,
                         int num_pages, int page_size, int64_t page_stride, int64_t token_stride,
                         dec_stream_t s) {
  if (!c || !positions || !slots || T < 1 || H < 0 || (interleaved != 0 && interleaved != 1))
    return DEC_ERR_INVALID_ARG;
  dec_status st = check_cache(cache, kv_type, cache_scale, num_pages, page_size, page_stride,
                              token_stride, R, P);
  if (st != DEC_OK) return st;
  if (rot < 0 || rot > P || rot % 2 || (rot > 0 && !inv_freq) || (P > 0 && !k_rope))
    return DEC_ERR_INVALID_ARG;
  if (page_size > 1 && token_stride < R + P) return DEC_ERR_INVALID_ARG;  // tokens that overlap
  if (P == 0) H = 0;
  if (H > 0 && (!q_rope || !q_out)) return DEC_ERR_INVALID_ARG;
  if (weight && !(eps >= 0.0f)) return DEC_ERR_INVALID_ARG;
  if (rot % 16 || T > MAX_TOKENS || H > ATTN_MAX_HEADS) return DEC_ERR_UNSUPPORTED_SHAPE;
  if ((st = check_rows(T, 1, R, c_stride, 0, false)) != DEC_OK) return st;
  if (P > 0 && (st = check_rows(T, 1, P, k_stride, 0, false)) != DEC_OK) return st;
  if (H > 0 && (st = check_rows(T, H, P, q_stride, q_head, false)) != DEC_OK) return st;
  if (H > 0 && (st = check_rows(T, H, P, q_out_stride, q_out_head, true)) != DEC_OK) return st;
  if (rows_opt && (st = check_rows(T, 1, R + P, rows_stride, 0, true)) != DEC_OK) return st;
  if (off(c, 16) || off(weight, 16) || (P > 0 && off(k_rope, 16)) ||
      (H > 0 && (off(q_rope, 16) || off(q_out, 16))) || off(rows_opt, 16) || off(positions, 4) ||
      off(slots, 4) || off(inv_freq, 4))
    return DEC_ERR_MISALIGNED;
  // in place means exactly in place
  if (H > 0 && q_rope == q_out &&
      ((T > 1 && q_stride != q_out_stride) || (H > 1 && q_head != q_out_head)))
    return DEC_ERR_INVALID_ARG;
  cudaError_t ce;
  const int sms = host_num_sms(&ce);
  if (sms <= 0) return DEC_ERR_CUDA;
  if (host_consume_fault()) return DEC_ERR_CUDA;
  LatentAppendParams p;
  p.c = c;
  p.k_rope = k_rope;
  p.q_rope = q_rope;
  p.weight = weight;
  p.c_stride = c_stride;
  p.k_stride = k_stride;
  p.q_stride = q_stride;
  p.q_head = q_head;
  p.out_stride = q_out_stride;
  p.out_head = q_out_head;
  p.rows_stride = rows_stride;
  p.eps = eps;
  p.magnitude = magnitude;
  p.positions = positions;
  p.slots = slots;
  p.inv_freq = inv_freq;
  p.T = T;
  p.H = H;
  p.R = R;
  p.P = P;
  p.rot = rot;
  p.q_out = q_out;
  p.rows = rows_opt;
  p.cache = cache;
  p.scale = cache_scale;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.num_pages = num_pages;
  p.page_size = page_size;
  return status_of(launch_latent_append(p, kv_type == DEC_KV_E4M3, interleaved != 0, sms,
                                        reinterpret_cast<cudaStream_t>(s)));
}

dec_status latent_project(const dec_bf16 *x, int64_t x_stride, int64_t x_head, const dec_bf16 *W,
                          dec_bf16 *y, int64_t y_stride, int64_t y_head, int T, int H, int K,
                          int N, dec_stream_t s) {
  if (!x || !W || !y || T < 1 || H < 1 || K < 1 || N < 1) return DEC_ERR_INVALID_ARG;
  if (K % 8 || N % 8 || K > 4096 || N > 4096 || T > MAX_TOKENS || H > ATTN_MAX_HEADS)
    return DEC_ERR_UNSUPPORTED_SHAPE;
  dec_status st = check_rows(T, H, K, x_stride, x_head, false);
  if (st != DEC_OK) return st;
  if ((st = check_rows(T, H, N, y_stride, y_head, true)) != DEC_OK) return st;
  if (off(x, 16) || off(W, 16) || off(y, 16)) return DEC_ERR_MISALIGNED;
  if (x == y || W == y) return DEC_ERR_INVALID_ARG;
  cudaError_t ce;
  const int sms = host_num_sms(&ce);
  if (sms <= 0) return DEC_ERR_CUDA;
  if (host_consume_fault()) return DEC_ERR_CUDA;
  uint64_t limit = 0;
  unsigned *status = host_wait_status(&limit);
  return status_of(launch_latent_project(x, x_stride, x_head, W, y, y_stride, y_head, T, H, K, N,
                                         sms, status, limit, host_attn_hold(),
                                         reinterpret_cast<cudaStream_t>(s)));
}

size_t latent_decode_workspace_bytes(int S, int T, int H, int R, int P) {
  if (S < 1 || S > ATTN_MAX_SEQS || T < 1 || T > 65536 || H < 1 || H > ATTN_MAX_HEADS || R < 1 ||
      P < 0 || R % 64 || P % 64 || R > LATENT_MAX_R || R + P > LATENT_MAX_W)
    return 0;
  cudaError_t ce;
  const int sms = host_num_sms(&ce);
  // the rows of an item grow with those of an average sequence: one sequence that has them all
  // takes the most, and what is enough for it is enough for every smaller call
  return sms > 0 ? latent_workspace_bytes(1, T, H, sms) : 0;
}

dec_status latent_decode(const dec_bf16 *q, int64_t q_stride, const void *cache, int kv_type,
                         const float *cache_scale, int num_pages, int page_size,
                         int64_t page_stride, int64_t token_stride, const int32_t *block_table,
                         int max_pages, const int32_t *seq_len, const int32_t *q_start, int S,
                         int T, int H, int R, int P, float scale, int window, dec_bf16 *out,
                         int64_t out_stride, float *lse_opt, void *ws, size_t ws_bytes,
                         dec_stream_t s) {
  if (!q || !block_table || !seq_len || !out || !ws) return DEC_ERR_INVALID_ARG;
  if (S < 1 || T < 1 || H < 1 || max_pages < 1 || window < 0) return DEC_ERR_INVALID_ARG;
  if (!q_start && T != S) return DEC_ERR_INVALID_ARG;
  const dec_status st = check_cache(cache, kv_type, cache_scale, num_pages, page_size,
                                    page_stride, token_stride, R, P);
  if (st != DEC_OK) return st;
  if (S > ATTN_MAX_SEQS || T > 65536 || H > ATTN_MAX_HEADS) return DEC_ERR_UNSUPPORTED_SHAPE;
  if (q_stride > MOST || out_stride > MOST) return DEC_ERR_UNSUPPORTED_SHAPE;
  if (T > 1 && (q_stride < 0 || out_stride < static_cast<int64_t>(H) * R))
    return DEC_ERR_INVALID_ARG;
  if (off(q, 16) || off(out, 16) || off(block_table, 4) || off(seq_len, 4) || off(q_start, 4) ||
      off(lse_opt, 4) || off(ws, 16))
    return DEC_ERR_MISALIGNED;
  if (T > 1 && (q_stride % 8 || out_stride % 8)) return DEC_ERR_MISALIGNED;
  if (q == out) return DEC_ERR_INVALID_ARG;
  cudaError_t ce;
  const int sms = host_num_sms(&ce);
  if (sms <= 0) return DEC_ERR_CUDA;
  if (ws_bytes < latent_workspace_bytes(S, T, H, sms)) return DEC_ERR_WORKSPACE_TOO_SMALL;
  if (host_consume_fault()) return DEC_ERR_CUDA;
  AttnParams p = {};
  p.q = q;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.c.k = p.c.v = cache;
  p.c.k_scale = p.c.v_scale = cache_scale;
  p.c.page_stride = page_stride;
  p.c.token_stride = token_stride;
  p.c.num_pages = num_pages;
  p.c.page_size = page_size;
  p.block_table = block_table;
  p.seq_len = seq_len;
  p.q_start = q_start;
  p.max_pages = max_pages;
  p.S = S;
  p.T = T;
  p.Hq = H;
  p.Hkv = 1;
  p.D = R;
  p.scale = scale;
  p.window = window;
  p.out = out;
  p.lse = lse_opt;
  uint64_t limit = 0;
  unsigned *status = host_wait_status(&limit);
  return status_of(launch_latent_decode(p, R + P, kv_type == DEC_KV_E4M3, ws, sms, status, limit,
                                        host_attn_hold(), reinterpret_cast<cudaStream_t>(s)));
}

dec_status latent_prompt(const dec_bf16 *q, int64_t q_stride, const dec_bf16 *k_nope,
                         int64_t k_stride, int64_t k_head, const dec_bf16 *k_rope,
                         int64_t r_stride, const dec_bf16 *v, int64_t v_stride, int64_t v_head,
                         const int32_t *q_start, const int32_t *k_start, int S, int T, int Tk,
                         int H, int N, int P, int V, float scale, dec_bf16 *out,
                         int64_t out_stride, float *lse_opt, dec_stream_t s) {
  if (!q || !k_nope || !v || !q_start || !out || S < 1 || T < 1 || Tk < 1 || H < 1 || N < 1 ||
      P < 0 || V < 1 || (P > 0 && !k_rope) || (!k_start && Tk != T))
    return DEC_ERR_INVALID_ARG;
  if ((N != 64 && N != 128) || (P != 0 && P != 64) || (V != 64 && V != 128) ||
      S > ATTN_MAX_SEQS || T > MAX_TOKENS || Tk > MAX_TOKENS || H > ATTN_MAX_HEADS)
    return DEC_ERR_UNSUPPORTED_SHAPE;
  dec_status st = check_rows(T, H, N + P, q_stride, N + P, true);
  if (st != DEC_OK) return st;
  if ((st = check_rows(Tk, H, N, k_stride, k_head, false)) != DEC_OK) return st;
  if (P > 0 && (st = check_rows(Tk, 1, P, r_stride, 0, false)) != DEC_OK) return st;
  if ((st = check_rows(Tk, H, V, v_stride, v_head, false)) != DEC_OK) return st;
  if ((st = check_rows(T, 1, H * V, out_stride, 0, true)) != DEC_OK) return st;
  if (off(q, 16) || off(k_nope, 16) || (P > 0 && off(k_rope, 16)) || off(v, 16) || off(out, 16) ||
      off(q_start, 4) || off(k_start, 4) || off(lse_opt, 4))
    return DEC_ERR_MISALIGNED;
  if (out == q || out == k_nope || out == v) return DEC_ERR_INVALID_ARG;
  cudaError_t ce;
  const int sms = host_num_sms(&ce);
  if (sms <= 0) return DEC_ERR_CUDA;
  if (host_consume_fault()) return DEC_ERR_CUDA;
  LatentPromptParams p = {};
  p.q_start = q_start;
  p.k_start = k_start ? k_start : q_start;
  p.S = S;
  p.T = T;
  p.Tk = Tk;
  p.H = H;
  p.N = N;
  p.P = P;
  p.V = V;
  p.scale = scale;
  p.out = out;
  p.out_stride = out_stride;
  p.lse = lse_opt;
  p.status = host_wait_status(&p.wait_limit_ns);
  p.hold = host_attn_hold();
  return status_of(launch_latent_prompt(p, q, q_stride, k_nope, k_stride, k_head, k_rope, r_stride,
                                        v, v_stride, v_head, sms,
                                        reinterpret_cast<cudaStream_t>(s)));
}

dec_status dec_latent_call(int which, const int64_t *a) {
  if (!a) return DEC_ERR_INVALID_ARG;
  auto f = [&](int i) {
    double d;
    static_assert(sizeof(d) == sizeof(*a), "a slot");
    memcpy(&d, a + i, sizeof(d));
    return static_cast<float>(d);
  };
  // beyond an int: its ends
  auto n = [&](int i) {
    return static_cast<int>(a[i] > INT32_MAX ? INT32_MAX : (a[i] < INT32_MIN ? INT32_MIN : a[i]));
  };
  auto at = [&](int i) { return reinterpret_cast<void *>(a[i]); };
  auto stream = [&](int i) { return reinterpret_cast<dec_stream_t>(a[i]); };
  auto rows = [&](int i) { return static_cast<dec_bf16 *>(at(i)); };
  auto ints = [&](int i) { return static_cast<const int32_t *>(at(i)); };
  auto floats = [&](int i) { return static_cast<float *>(at(i)); };
  switch (which) {
    case DEC_LATENT_APPEND:
      return latent_append(rows(0), a[1], rows(2), f(3), rows(4), a[5], rows(6), a[7], a[8], ints(9),
                           ints(10), floats(11), f(12), n(13), n(14), n(15), n(16), n(17), n(18),
                           rows(19), a[20], a[21], rows(22), a[23], at(24), n(25), floats(26), n(27),
                           n(28), a[29], a[30], stream(31));
    case DEC_LATENT_PROJECT:
      return latent_project(rows(0), a[1], a[2], rows(3), rows(4), a[5], a[6], n(7), n(8), n(9),
                            n(10), stream(11));
    case DEC_LATENT_DECODE:
      return latent_decode(rows(0), a[1], at(2), n(3), floats(4), n(5), n(6), a[7], a[8], ints(9),
                           n(10), ints(11), ints(12), n(13), n(14), n(15), n(16), n(17), f(18), n(19),
                           rows(20), a[21], floats(22), at(23), static_cast<size_t>(a[24]), stream(25));
    case DEC_LATENT_PROMPT:
      return latent_prompt(rows(0), a[1], rows(2), a[3], a[4], rows(5), a[6], rows(7), a[8], a[9],
                           ints(10), ints(11), n(12), n(13), n(14), n(15), n(16), n(17), n(18), f(19),
                           rows(20), a[21], floats(22), stream(23));
    default:
      return DEC_ERR_INVALID_ARG;
  }
}

}  // extern "C"
