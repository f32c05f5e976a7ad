// Which kernel takes the rows of a batch whose lengths only the device knows, and how kernels that start early
// follow one another.
#pragma once
#include "ssd_attn.h"

#include <cuda_runtime.h>

namespace ssd {

// Waits until the kernel before this one on the stream has finished (for a launch that may start early) / lets
// the next one start early.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Whether k_paged_prompt takes the call (by a whole warp; in whole numbers, so that every warp of
// either kernel finds the same).  Its items do not share a sequence's positions, so that one long
// sequence among short ones is all that most SMs wait for; the kernels of ssd_attn.cuh spread any lengths
// evenly.  With the costs of PagedArgs::Ask: the longest item, and where items are dealt out in turn
// (more than the SMs) half of the smaller of it and of an SM's share on top of the larger, against all
// blocks spread over the SMs.
__device__ __forceinline__ bool prompt_pays(const PagedArgs &a) {
    uint64_t sum = 0;
    int longest = 0;
    for (int b = threadIdx.x % 32; b < a.B; b += 32) {
        const int n = (min(max(a.lens[b], 0), a.ask.most) + 127) >> 7;
        sum += n;
        longest = max(longest, n);
    }
    longest = __reduce_max_sync(~0u, longest);
    sum = __reduce_add_sync(~0u, uint32_t(sum) & 0xffffffu) +
          (uint64_t(__reduce_add_sync(~0u, uint32_t(sum >> 24))) << 24);
    const uint64_t one = longest * a.ask.one, share = sum * a.ask.share;
    return 2 * max(one, share) + min(one, share) <= 2 * (sum * a.ask.line);
}

}  // namespace ssd
