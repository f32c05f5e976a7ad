// Which kernel takes the rows of a batch whose lengths only the device knows.
#pragma once
#include "ssd_attn.h"

#include <cuda_runtime.h>

namespace ssd {

// Whether k_paged_prompt takes the call (by a whole warp; the same answer in every warp of either
// kernel).  Its items do not share a sequence's positions, so that one long sequence among short ones
// is all that most SMs wait for; the kernels of ssd_attn.cuh spread any lengths evenly.  In
// units of 0.1 ns, for 128 positions: an item 1.55 us (D = 64: 1.36), one of less than half a round of
// items 1.23 (1.11); a block of 64 rows over all SMs 15.4 ns (10.6).  Beyond a round, items are dealt
// out in turn, and the longest may come on top of half a share.
__device__ __forceinline__ bool prompt_pays(const PagedArgs &a, int sms) {
    const int lane = threadIdx.x % 32, G = a.Hq / a.c.Hkv, rows = a.T * G;
    const bool wide = a.c.D == 128;
    const int64_t most = int64_t(a.M) * a.c.ps;
    int64_t sum = 0, longest = 0;
    for (int b = lane; b < a.B; b += 32) {
        int64_t n = a.lens[b];
        n = n < 0 ? 0 : n > most ? most : n;
        const int64_t seen = a.window + a.sinks + 256 / G;      // of an item's rows
        if (a.window > 0 && n > seen) n = seen;
        n = (n + 127) / 128;
        sum += n;
        longest = n > longest ? n : longest;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        const int64_t other = __shfl_xor_sync(~0u, longest, o);
        longest = other > longest ? other : longest;
    }
    const int64_t per = int64_t(a.c.Hkv) * ((rows + 255) / 256), items = a.B * per;
    const int64_t whole = wide ? 15500 : 13600, part = wide ? 12300 : 11100;
    const int64_t line = sum * a.c.Hkv * ((rows + 63) / 64) * (wide ? 154 : 106);
    const int64_t one = longest * (2 * items <= sms ? part : whole), share = sum * per * whole / sms;
    return (items <= sms ? one : one > share ? one + share / 2 : share + one / 2) <= line;
}

}  // namespace ssd
