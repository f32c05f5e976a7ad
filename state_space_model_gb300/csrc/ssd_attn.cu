// Attention over the paged cache (ssd_attn.cuh): the choice of a kernel, and pools of bf16 and
// f32 without sinks.
#include "ssd_attn.cuh"

namespace ssd {

size_t paged_workspace(const PagedArgs &a) {
    const Shape s = make_shape(a);
    return s.ncta * (sizeof(Cut) + 2 * part_floats(s.RB, a.c.D) * sizeof(float));
}

namespace {
cudaError_t launch_others(const PagedArgs &a, cudaStream_t s) {
    const bool sinks = a.sinks > 0;
    switch (a.c.dt) {
    case DT_F8E4M3: return sinks ? launch_paged_sinks_f8(a, s) : launch_paged_f8(a, s);
    case DT_F4E2M1X2: return sinks ? launch_paged_sinks_f4(a, s) : launch_paged_f4(a, s);
    case DT_F32:
        if (sinks) return launch_paged_sinks(a, s);
        return a.c.D == 64 ? launch_f32_rows<64>(a, s) : launch_f32_rows<128>(a, s);
    default:
        if (sinks) return launch_paged_sinks(a, s);
        return a.c.D == 64 ? launch_rows<64, kBf16>(a, s) : launch_rows<128, kBf16>(a, s);
    }
}
}  // namespace

cudaError_t launch_paged(const PagedArgs &in, cudaStream_t s) {
    PagedArgs a = in;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    Prompt many = prompt_fits(a);
    PromptMaps maps;
    if (many != Prompt::kNo && !make_prompt_maps(a, &maps)) many = Prompt::kNo;
    a.maps = &maps;
    if (many == Prompt::kYes) return launch_paged_prompt(a, s);
    if (many == Prompt::kAsk) ask_lengths(a);    // (k_paged_mma's launch brings the other)
    return launch_others(a, s);
}

}  // namespace ssd
