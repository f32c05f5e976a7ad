// Attention over the paged cache (ssd_attn.cuh): pools of bf16 and f32; those of codes are in
// ssd_attn_f8.cu and ssd_attn_f4.cu (translation units of their own, compiled side by side).
#include "ssd_attn.cuh"

namespace ssd {
namespace {

template <int D>
cudaError_t launch_f32_rows(const PagedArgs &a, cudaStream_t stream) {
    const Shape s = make_shape(a);
    if (s.RB == 1) return launch_f32<D, 1>(a, s, stream);
    if (s.RB == 2) return launch_f32<D, 2>(a, s, stream);
    return launch_f32<D, 4>(a, s, stream);
}

}  // namespace

size_t paged_workspace(const PagedArgs &a) {
    const Shape s = make_shape(a);
    return s.ncta * (sizeof(Cut) + 2 * part_floats(s.RB, a.c.D) * sizeof(float));
}

cudaError_t launch_paged(const PagedArgs &in, cudaStream_t s) {
    PagedArgs a = in;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    switch (a.c.dt) {
    case DT_F8E4M3: return launch_paged_f8(a, s);
    case DT_F4E2M1X2: return launch_paged_f4(a, s);
    case DT_F32: return a.c.D == 64 ? launch_f32_rows<64>(a, s) : launch_f32_rows<128>(a, s);
    default: return a.c.D == 64 ? launch_rows<64, kBf16>(a, s) : launch_rows<128, kBf16>(a, s);
    }
}

}  // namespace ssd
