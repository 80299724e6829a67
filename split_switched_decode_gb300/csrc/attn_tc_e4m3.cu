// attn_tc_e4m3.cu -- the tcgen05 attention kernel for e4m3 caches.
#include "attn_tc.cuh"

namespace ssd {

cudaError_t launch_attn_tc_e4m3(const AttnParams &p, int padded, int rows, void *ws,
                           const AttnLaunch &a, cudaStream_t s) {
  return launch_tc<true>(p, padded, rows, ws, a, s);
}

}  // namespace ssd
