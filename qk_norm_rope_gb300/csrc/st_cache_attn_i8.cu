// Cached attention over caches of int8 (st_cache_attn.cuh).
#include "st_cache_attn.cuh"

namespace st {

cudaError_t launch_cache_attn_i8(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream) {
  return launch_form<kDtI8, false>(p, nt, f16, stream);
}

}  // namespace st
