// attn.h -- launches of the attention step over the paged cache (not installed):
// kv_plan.cu, rope_append.cu, attn_decode.cu; argument checks are in api_attn.cu.
#pragma once

#include "internal.h"

namespace ssd {

constexpr int ATTN_MAX_SEQS = 8192;
constexpr int ATTN_MAX_HEADS = 1024;
constexpr int ATTN_MAX_D = 256;

// Where the elements of a paged cache are (strides in elements, the same for K and V).
struct PagedCache {
  const void *k;
  const void *v;
  const float *k_scale;  // [Hkv] or nullptr
  const float *v_scale;
  long long page_stride, head_stride, token_stride;
  int num_pages, page_size;
};

// ---------------------------------------------------------------- kv_plan.cu --
struct KvPlanParams {
  const int32_t *kv_len, *new_len;  // new_len nullptr: one each
  int S, page_size;
  int32_t *block_table;
  int max_pages;
  const int32_t *free_pages;
  int num_free;
  const int32_t *free_used;  // nullptr: 0
  int32_t *seq_len, *q_start, *positions, *slots;
  int max_tokens;
  int32_t *summary;
};
cudaError_t launch_kv_plan(const KvPlanParams &p, cudaStream_t s);

// ------------------------------------------------------------ rope_append.cu --
struct RopeParams {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride, out_stride;
  const int32_t *positions, *slots;
  const float *inv_freq;
  float magnitude;
  int T, Hq, Hkv, D, rot, interleaved;
  uint16_t *q_out;
  PagedCache c;  // written
};
cudaError_t launch_rope_append(const RopeParams &p, bool e4m3, int num_sms, cudaStream_t s);

// ------------------------------------------------------------ attn_decode.cu --
struct AttnParams {
  const uint16_t *q;
  long long q_stride, out_stride;
  PagedCache c;
  const int32_t *block_table, *seq_len, *q_start;  // q_start nullptr: row s for sequence s
  int max_pages, S, T, Hq, Hkv, D;
  float scale;
  int window;
  uint16_t *out;
  float *lse;  // or nullptr
  int box;     // tokens of a TMA box of the caches (8..64), 0: 16-byte copies
};
// What a launch needs besides the parameters.
struct AttnLaunch {
  CUtensorMap kmap, vmap;  // of the caches where box > 0
  int num_sms;
  unsigned *status;
  uint64_t wait_limit_ns;
  bool hold;  // self-test: waits that run out
};
// Workers (CTAs) of a launch at most, and the workspace's counters: one per worker for items,
// two for groups of workers.
inline int attn_max_workers(int num_sms) { return 2 * num_sms; }
// Rows of an average sequence and kv head up to which the legacy products are taken, by the
// cache type and the padded head: up to 16 rows those keep up with the copies of a bf16 cache, and
// on an e4m3 one tcgen05 needs widened operands. Legacy / tcgen05 in us, 64 sequences (heads of
// 256: 24) of 512 to 8192 tokens, 8 kv heads, pages of 32:
//
//              bf16: 16 rows     32          64          e4m3: 16     32          64
//   heads of 64     98.7/100.9  165/103    292/112      91.7/198   156/200    289/198
//   128              170/170    229/173    406/179       140/211   245/213    452/227
//   256              137/137    237/142    408/152       127/231   219/233    405/235
constexpr int tc_min_rows(bool e4m3, int dp) {
  return !e4m3 || dp == 128 ? 16 : (dp == 64 ? 32 : 48);
}
inline size_t attn_counter_bytes(int num_sms) {
  return (static_cast<size_t>(3) * attn_max_workers(num_sms) * sizeof(int) + 255) / 256 * 256;
}
// One kernel per padded head size (attn_d64.cu, attn_d128.cu, attn_d256.cu); nr groups of 8
// rows a warp, wr warps sharing the rows.
cudaError_t launch_attn_d64(const AttnParams &p, bool e4m3, int nr, int wr, void *ws,
                            const AttnLaunch &a, cudaStream_t s);
cudaError_t launch_attn_d128(const AttnParams &p, bool e4m3, int nr, int wr, void *ws,
                             const AttnLaunch &a, cudaStream_t s);
cudaError_t launch_attn_d256(const AttnParams &p, bool e4m3, int nr, int wr, void *ws,
                             const AttnLaunch &a, cudaStream_t s);
// attn_tc.cu: bf16 caches in boxes, items of 32, 64 or 128 rows.
cudaError_t launch_attn_tc(const AttnParams &p, int padded, int rows, void *ws,
                           const AttnLaunch &a, cudaStream_t s);
cudaError_t launch_attn_tc_e4m3(const AttnParams &p, int padded, int rows, void *ws,
                           const AttnLaunch &a, cudaStream_t s);
// api.cu: a 4-D map (head element, token of the page, kv head, page) of a cache, boxes of
// 128 bytes (64 where a padded head has 64 bytes) x box tokens, swizzled accordingly.
bool host_cache_map(CUtensorMap *m, const PagedCache &c, const void *base, bool e4m3, int D,
                    int Hkv, int box, int padded);
size_t attn_workspace_bytes(int S, int T, int Hq, int Hkv, int D, int num_sms);
cudaError_t launch_attn_decode(const AttnParams &p, bool e4m3, void *ws, int num_sms,
                               unsigned *status, uint64_t wait_limit_ns, bool hold,
                               cudaStream_t s);

}  // namespace ssd
