// Attention over the paged cache (ssd_attn.cuh): pools of bf16 and f32, with sinks.
#define SSD_ATTN_SINKS
#include "ssd_attn.cuh"

namespace ssd {

cudaError_t launch_paged_sinks(const PagedArgs &a, cudaStream_t s) {
    if (a.c.dt == DT_F32) return a.c.D == 64 ? launch_f32_rows<64>(a, s) : launch_f32_rows<128>(a, s);
    return a.c.D == 64 ? launch_rows<64, kBf16>(a, s) : launch_rows<128, kBf16>(a, s);
}

}  // namespace ssd
