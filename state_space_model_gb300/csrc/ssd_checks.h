// What the C ABI's entry points share: the error detail of the calling
// thread, and the checks of tensors, address ranges and device pointers that
// run before any launch.  Not part of the public ABI.
#pragma once

#include "ssd.h"

#include <cuda_runtime_api.h>

#include <initializer_list>
#include <string>

namespace ssd {
namespace checks {

// Text of the last failed check on this thread ("" after a successful call).
std::string &error_detail();

ssd_status fail(ssd_status st, const char *fmt, ...);   // records the text, returns st
ssd_status ok();                                        // clears the text

size_t elem_size(int dt);

// Address range [lo, hi) a tensor touches; empty when any extent is 0.
struct Range {
    uintptr_t lo = 0, hi = 0;
};
Range range_of(const ssd_tensor *t);
Range range_raw(const void *p, size_t bytes);
bool overlap(Range a, Range b);
// Two tensors that may share an element: their ranges meet, and no stride shows that they lie
// side by side (keys and values of a page next to one another in one allocation, say).
bool overlap(const ssd_tensor *a, const ssd_tensor *b);

// Checks one tensor's rank, dtype, shape, unit inner stride and alignment.
// dtype < 0 accepts f32 or bf16 (the others only where asked for by name).
// contiguous demands packed row-major strides.
ssd_status check_tensor(const ssd_tensor *t, const char *name, int ndim, const int64_t *shape,
                        int dtype, bool contiguous, bool align_strides16);

// An output's strides must keep its elements apart (a broadcast view, with a
// stride of 0, would be written by several threads at once).
ssd_status check_distinct(const ssd_tensor *t, const char *name);

// Every data pointer must be device (or managed) memory of the current
// device: a host pointer handed to a kernel would fault it.  Runs after all
// pure-host checks, so argument errors are reported without touching CUDA.
struct NamedPtr {
    const void *p;
    const char *name;
};
ssd_status check_device_ptrs(std::initializer_list<NamedPtr> ptrs);

ssd_status cuda_status(cudaError_t e, const char *what);

}  // namespace checks
}  // namespace ssd
