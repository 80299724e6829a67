// attn_d256.cu -- the attention kernel for heads of 129 to 256 elements.
#include "attn_kernel.cuh"

namespace ssd {

cudaError_t launch_attn_d256(const AttnParams &p, bool e4m3, int nr, int wr, void *ws,
                           const AttnLaunch &a, cudaStream_t s) {
  return launch_dim<256>(p, e4m3, nr, wr, ws, a, s);
}

}  // namespace ssd
