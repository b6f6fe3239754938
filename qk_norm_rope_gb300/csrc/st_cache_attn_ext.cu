// Cached attention with a window or a shared prefix, over 16-bit caches (st_cache_attn.cuh).
#include "st_cache_attn.cuh"

namespace st {

cudaError_t launch_cache_attn_ext(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream) {
  return launch_form<0, true>(p, nt, f16, stream);
}

}  // namespace st
