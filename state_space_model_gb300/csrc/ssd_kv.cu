// The cache's write and read (ssd_kv.cuh) for pools of the layer's type or 8-bit codes, with
// positions of one axis; the rest is in ssd_kv_ex.cu.
#include "ssd_kv.cuh"

namespace ssd {

cudaError_t launch_kv_append(const KvAppendArgs &in, cudaStream_t s) {
    KvAppendArgs a = in;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    if (a.axes > 1 || a.c.dt == DT_F4E2M1X2) return launch_kv_append_ex(a, s);
    return a.c.dt == DT_F8E4M3 ? append_codes<kEight, false>(a, s) : append_codes<kPlain, false>(a, s);
}

cudaError_t launch_kv_read(const KvReadArgs &in, cudaStream_t s) {
    KvReadArgs a = in;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    if (a.c.dt == DT_F4E2M1X2) return launch_kv_read_ex(a, s);
    if (a.c.dt == DT_F8E4M3) return read_codes<uint8_t>(a, s);
    if (a.c.dt == DT_F32)
        return a.c.D == 64 ? read_t<float, float, 64>(a, s) : read_t<float, float, 128>(a, s);
    return a.c.D == 64 ? read_t<__nv_bfloat16, __nv_bfloat16, 64>(a, s)
                       : read_t<__nv_bfloat16, __nv_bfloat16, 128>(a, s);
}

}  // namespace ssd
