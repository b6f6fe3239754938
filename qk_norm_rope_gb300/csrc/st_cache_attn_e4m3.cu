// Cached attention over caches of 8-bit floats (st_cache_attn.cuh).
#include "st_cache_attn.cuh"

namespace st {

cudaError_t launch_cache_attn_e4m3(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream) {
  return launch_form<kDtE4M3, false>(p, nt, f16, stream);
}

}  // namespace st
