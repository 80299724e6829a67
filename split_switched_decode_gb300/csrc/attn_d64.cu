// attn_d64.cu -- the attention kernel for heads of up to 64 elements.
#include "attn_kernel.cuh"

namespace ssd {

cudaError_t launch_attn_d64(const AttnParams &p, bool e4m3, int nr, int wr, void *ws,
                           const AttnLaunch &a, cudaStream_t s) {
  return launch_dim<64>(p, e4m3, nr, wr, ws, a, s);
}

}  // namespace ssd
