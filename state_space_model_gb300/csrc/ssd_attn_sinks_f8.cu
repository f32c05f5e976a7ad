// Attention over the paged cache (ssd_attn.cuh): pools of 8-bit codes, with sinks.
#define SSD_ATTN_SINKS
#include "ssd_attn.cuh"

namespace ssd {

cudaError_t launch_paged_sinks_f8(const PagedArgs &a, cudaStream_t s) {
    return a.c.D == 64 ? launch_rows<64, kEight>(a, s) : launch_rows<128, kEight>(a, s);
}

}  // namespace ssd
