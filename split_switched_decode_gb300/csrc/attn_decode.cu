// attn_decode.cu -- host side of the attention kernel (attn_kernel.cuh): the kernel's shape
// by head size and rows, the workspace, and the tensor maps of the caches.
#include "attn.h"

namespace ssd {
namespace {

int padded_dim(int D) { return D <= 64 ? 64 : (D <= 128 ? 128 : 256); }

struct AttnShape {
  int nr, wr;  // 8-row groups of a warp, warps sharing the rows
  int rows() const { return 8 * nr * wr; }
};

// Rows of an average sequence, which is what the host knows. More rows than an item holds
// read the keys once more per item (mostly from L2), and fewer compute on rows that are not
// there: a batch of very unequal rows is better split into a call for each kind (63 sequences
// of 4096 tokens with a row each beside one with a chunk of 512 rows: 464 us in one call, 165 and
// 73 in two).
int mean_rows(int S, int T, int Hq, int Hkv) {
  return static_cast<int>(static_cast<long long>((T + S - 1) / S) * (Hq / Hkv));
}

AttnShape attn_shape(int rows) {
  return rows <= 8 ? AttnShape{1, 1}
                   : (rows <= 16 ? AttnShape{2, 1}
                                 : (rows <= 32 ? AttnShape{2, 2} : AttnShape{2, 4}));
}

// Rows of an item on tcgen05 tensor cores, 0 for the legacy products, `dp` the padded head.
int tc_rows(bool e4m3, int dp, int rows) {
  if (rows <= tc_min_rows(e4m3, dp)) return 0;
  return rows <= 32 ? 32 : (rows <= 64 ? 64 : 128);
}

// Tokens of a TMA box: the largest power of two in the page size, up to what a copying warp
// brings of a stage; below 8 (a swizzle group) none.
int box_tokens(int page_size, int most) {
  int box = page_size & -page_size;
  if (box > most) box = most;
  return box >= 8 ? box : 0;
}

}  // namespace

size_t attn_workspace_bytes(int S, int T, int Hq, int Hkv, int D, int num_sms) {
  const int dp = padded_dim(D), grid = dp <= 128 ? attn_max_workers(num_sms) : num_sms;
  const int rows = mean_rows(S, T, Hq, Hkv);  // of whichever kernel and cache type has more
  const size_t tc = tc_rows(false, dp, rows);
  const size_t M = tc > 0 ? tc : attn_shape(rows).rows();
  return attn_counter_bytes(num_sms) + 2 * grid * (M * dp + 2 * M) * sizeof(float);
}

cudaError_t launch_attn_decode(const AttnParams &params, bool e4m3, void *ws, int num_sms,
                               unsigned *status, uint64_t wait_limit_ns, bool hold,
                               cudaStream_t s) {
  AttnParams p = params;
  AttnLaunch a = {};
  a.num_sms = num_sms;
  a.status = status;
  a.wait_limit_ns = wait_limit_ns;
  a.hold = hold;
  const int dp = padded_dim(p.D);
  const int rows = mean_rows(p.S, p.T, p.Hq, p.Hkv), tc = tc_rows(e4m3, dp, rows);
  p.box = box_tokens(p.c.page_size, e4m3 || tc > 0 ? 64 : 32);
  if (p.box > 0) {
    // strides of zero (a broadcast cache) or an encoder that refuses: plain copies
    const bool ok = p.c.page_stride > 0 && p.c.head_stride > 0 && p.c.token_stride > 0 &&
                    host_cache_map(&a.kmap, p.c, p.c.k, e4m3, p.D, p.Hkv, p.box, dp) &&
                    host_cache_map(&a.vmap, p.c, p.c.v, e4m3, p.D, p.Hkv, p.box, dp);
    if (!ok) p.box = 0;
  }
  if (tc > 0 && p.box > 0)
    return (e4m3 ? launch_attn_tc_e4m3 : launch_attn_tc)(p, dp, tc, ws, a, s);
  const AttnShape sh = attn_shape(rows);
  auto launch = dp == 64 ? launch_attn_d64 : (dp == 128 ? launch_attn_d128 : launch_attn_d256);
  return launch(p, e4m3, sh.nr, sh.wr, ws, a, s);
}

}  // namespace ssd
