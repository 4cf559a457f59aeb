// The tcgen05 kernel of the history cache for caches in bf16.
#include "cache_tc.cuh"

namespace gdpa {

gdpa_status launch_cache_tc_bf16(const AttnArgs& a, int grid, cudaStream_t st) {
    return cache_tc::launch_any<false>(a, grid, st);
}

}  // namespace gdpa
