// The cache's write and read (ssd_kv.cuh) for pools of 4-bit codes, and the write with positions
// of several axes.  (A translation unit of its own, compiled beside ssd_kv.cu.)
#include "ssd_kv.cuh"

namespace ssd {

cudaError_t launch_kv_append_ex(const KvAppendArgs &a, cudaStream_t s) {
    if (a.c.dt == DT_F4E2M1X2)
        return a.axes > 1 ? append_codes<kFour, true>(a, s) : append_codes<kFour, false>(a, s);
    return a.c.dt == DT_F8E4M3 ? append_codes<kEight, true>(a, s) : append_codes<kPlain, true>(a, s);
}

cudaError_t launch_kv_read_ex(const KvReadArgs &a, cudaStream_t s) { return read_codes<Nibbles>(a, s); }

}  // namespace ssd
