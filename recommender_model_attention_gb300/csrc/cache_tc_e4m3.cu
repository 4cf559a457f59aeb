// The tcgen05 kernel of the history cache for caches in 8 bits.
#include "cache_tc.cuh"

namespace gdpa {

gdpa_status launch_cache_tc_e4m3(const AttnArgs& a, int grid, cudaStream_t st) {
    return cache_tc::launch_any<true>(a, grid, st);
}

}  // namespace gdpa
