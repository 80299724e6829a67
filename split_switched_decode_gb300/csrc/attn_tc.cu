// attn_tc.cu -- the tcgen05 attention kernel for bf16 caches.
#include "attn_tc.cuh"

namespace ssd {

cudaError_t launch_attn_tc(const AttnParams &p, int padded, int rows, void *ws,
                           const AttnLaunch &a, cudaStream_t s) {
  return launch_tc<false>(p, padded, rows, ws, a, s);
}

}  // namespace ssd
