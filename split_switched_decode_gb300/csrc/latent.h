// latent.h -- launches of latent attention (not installed): latent_append.cu,
// latent_project.cu, latent_decode.cuh, latent_prompt.cu; argument checks are in api_latent.cu.
#pragma once

#include "attn.h"

namespace ssd {

constexpr int LATENT_MAX_R = 512;  // latent elements of a token
constexpr int LATENT_MAX_W = 576;  // with the rotary ones

// ---------------------------------------------------------- latent_append.cu --
struct LatentAppendParams {
  const uint16_t *c, *k_rope, *q_rope;  // k_rope nullptr: P is 0; q_rope nullptr: no queries
  const uint16_t *weight;               // nullptr: c is written as it is
  long long c_stride, k_stride, q_stride, q_head, out_stride, out_head, rows_stride;
  float eps, magnitude;
  const int32_t *positions, *slots;
  const float *inv_freq;
  int T, H, R, P, rot;
  uint16_t *q_out, *rows;  // rows nullptr: not wanted
  void *cache;
  const float *scale;  // [1] or nullptr
  long long page_stride, token_stride;
  int num_pages, page_size;
};
cudaError_t launch_latent_append(const LatentAppendParams &p, bool e4m3, bool interleaved,
                                 int num_sms, cudaStream_t s);

// --------------------------------------------------------- latent_project.cu --
struct LatentProjectParams {
  int T, H, K, N;
  int kb, nb, tb;   // k-blocks of 64, column tiles, row tiles
  int stages;       // of the ring
  long long items;  // H * tb * nb
  unsigned *status;
  uint64_t wait_limit_ns;
  bool hold;  // self-test: waits that run out
};
cudaError_t launch_latent_project(const uint16_t *x, long long x_stride, long long x_head,
                                  const uint16_t *w, uint16_t *y, long long y_stride,
                                  long long y_head, int T, int H, int K, int N, int num_sms,
                                  unsigned *status, uint64_t wait_limit_ns, bool hold,
                                  cudaStream_t s);

// ---------------------------------------------------------- latent_decode.cu --
// AttnParams with one kv head of D = R elements, the first of a row of R + P in the cache.
struct LatentLaunch {
  CUtensorMap map, qmap;  // of the cache where AttnParams::box > 0; of q where q_boxes
  bool q_boxes;
  int num_sms;
  void *rows;       // workspace: a table entry a row of q and head,
  float2 *ml;       // two maxima and sums a worker and row of an item,
  float *partials;  // two parts a worker
  unsigned *status;
  uint64_t wait_limit_ns;
  bool hold;  // self-test: waits that run out
};
size_t latent_workspace_bytes(int S, int T, int H, int num_sms);  // of one call
cudaError_t launch_latent_decode(const AttnParams &p, int width, bool e4m3, void *ws, int num_sms,
                                 unsigned *status, uint64_t wait_limit_ns, bool hold,
                                 cudaStream_t s);
// latent_decode_e4m3.cu
cudaError_t launch_latent_e4m3(const AttnParams &p, int width, int rows, const LatentLaunch &a,
                               cudaStream_t s);
// latent_join.cu: parts of `rows` rows each.
cudaError_t launch_latent_join(const AttnParams &p, int rows, const LatentLaunch &a,
                               cudaStream_t s);

// ---------------------------------------------------------- latent_prompt.cu --
struct LatentPromptParams {
  const int32_t *q_start, *k_start;
  int S, T, Tk, H, N, P, V;
  float scale;
  uint16_t *out;
  long long out_stride;
  float *lse;  // or nullptr
  unsigned *status;
  uint64_t wait_limit_ns;
  bool hold;  // self-test: waits that run out
};
cudaError_t launch_latent_prompt(const LatentPromptParams &p, const uint16_t *q,
                                 long long q_stride, const uint16_t *k, long long k_stride,
                                 long long k_head, const uint16_t *k_rope, long long r_stride,
                                 const uint16_t *v, long long v_stride, long long v_head,
                                 int num_sms, cudaStream_t s);

// api.cu: a tensor map of bf16 elements in up to four dimensions (strides in elements, of dimensions
// 1 on) with boxes swizzled in 128 bytes; false where the encoder refuses.
bool host_map(CUtensorMap *m, const void *base, int rank, const long long *dims,
              const long long *strides, const int *box);

}  // namespace ssd
