// The same with a window or a shared prefix, apart for the instruction cache's sake.
#include "st_cache_attn.cuh"

namespace st {

cudaError_t launch_cache_attn_e4m3_ext(const TcAttnParams& p, int nt, bool f16, cudaStream_t stream) {
  return launch_form<kDtE4M3, true>(p, nt, f16, stream);
}

}  // namespace st
