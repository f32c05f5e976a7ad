// The argument checks and error detail of the C ABI (see ssd_checks.h).
#include "ssd_checks.h"

#include "ssd_internal.h"

#include <cuda_runtime_api.h>

#include <cstdarg>
#include <cstdio>

namespace ssd {
namespace checks {

std::string &error_detail() {
    static thread_local std::string detail;
    return detail;
}

ssd_status fail(ssd_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    error_detail() = buf;
    return st;
}

ssd_status ok() {
    error_detail().clear();
    return SSD_OK;
}

size_t elem_size(int dt) { return dt == SSD_BF16 ? 2 : dt == SSD_F8E4M3 ? 1 : 4; }

Range range_of(const ssd_tensor *t) {
    Range r;
    if (!t || !t->data) return r;
    int64_t last = 0;
    for (int i = 0; i < t->ndim; ++i) {
        if (t->shape[i] == 0) return r;
        last += (t->shape[i] - 1) * t->stride[i];
    }
    r.lo = reinterpret_cast<uintptr_t>(t->data);
    r.hi = r.lo + size_t(last + 1) * elem_size(t->dtype);
    return r;
}
Range range_raw(const void *p, size_t bytes) {
    Range r;
    if (p && bytes) {
        r.lo = reinterpret_cast<uintptr_t>(p);
        r.hi = r.lo + bytes;
    }
    return r;
}
bool overlap(Range a, Range b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

// Modulo some stride m of either, every element of a tensor lies within the span of those of its
// dimensions whose strides are no multiples of m; spans that stay apart modulo m share nothing.
bool overlap(const ssd_tensor *a, const ssd_tensor *b) {
    const Range ra = range_of(a), rb = range_of(b);
    if (!overlap(ra, rb)) return false;
    auto span = [](const ssd_tensor *t, uint64_t m) {
        const uint64_t es = elem_size(t->dtype);
        uint64_t n = es;
        for (int i = 0; i < t->ndim; ++i)
            if (uint64_t(t->stride[i]) * es % m) n += uint64_t(t->shape[i] - 1) * t->stride[i] * es;
        return n;
    };
    for (const ssd_tensor *t : {a, b})
        for (int i = 0; i < t->ndim; ++i) {
            if (t->shape[i] <= 1 || t->stride[i] <= 0) continue;
            const uint64_t m = uint64_t(t->stride[i]) * elem_size(t->dtype);
            // where b begins modulo m, seen from a
            const uint64_t at = rb.lo >= ra.lo ? (rb.lo - ra.lo) % m : (m - (ra.lo - rb.lo) % m) % m;
            if (at >= span(a, m) && at + span(b, m) <= m) return false;
        }
    return true;
}

ssd_status check_tensor(const ssd_tensor *t, const char *name, int ndim,
                        const int64_t *shape, int dtype, bool contiguous,
                        bool align_strides16) {
    if (!t) return fail(SSD_ERR_INVALID_ARG, "%s: null tensor descriptor", name);
    if (t->ndim != ndim)
        return fail(SSD_ERR_INVALID_ARG, "%s: ndim %d, expected %d", name, t->ndim, ndim);
    auto dname = [](int d) {
        return d == SSD_F32 ? "f32" : d == SSD_BF16 ? "bf16" : d == SSD_I32 ? "i32" : "f8e4m3";
    };
    if (t->dtype < SSD_F32 || t->dtype > SSD_F8E4M3)
        return fail(SSD_ERR_INVALID_ARG, "%s: unknown dtype code %d", name, t->dtype);
    if ((dtype >= 0 && t->dtype != dtype) || (dtype < 0 && t->dtype != SSD_F32 && t->dtype != SSD_BF16))
        return fail(SSD_ERR_INVALID_ARG, "%s: dtype %s, expected %s", name, dname(t->dtype),
                    dtype >= 0 ? dname(dtype) : "f32 or bf16");
    int64_t numel = 1;
    for (int i = 0; i < ndim; ++i) {
        if (t->shape[i] != shape[i])
            return fail(SSD_ERR_INVALID_ARG, "%s: shape[%d] = %lld, expected %lld", name, i,
                        (long long)t->shape[i], (long long)shape[i]);
        numel *= shape[i];
    }
    if (numel > 0 && !t->data) return fail(SSD_ERR_INVALID_ARG, "%s: null data pointer", name);
    if (t->stride[ndim - 1] != 1 && shape[ndim - 1] > 1)
        return fail(SSD_ERR_INVALID_ARG, "%s: innermost stride %lld, must be 1", name,
                    (long long)t->stride[ndim - 1]);
    if (contiguous) {
        int64_t want = 1;
        for (int i = ndim - 1; i >= 0; --i) {
            if (shape[i] > 1 && t->stride[i] != want)
                return fail(SSD_ERR_INVALID_ARG, "%s: must be contiguous (stride[%d] = %lld, "
                            "expected %lld)", name, i, (long long)t->stride[i], (long long)want);
            want *= shape[i];
        }
    }
    for (int i = 0; i < ndim - 1; ++i)
        if (t->stride[i] < 0)
            return fail(SSD_ERR_INVALID_ARG, "%s: negative stride", name);
    const size_t es = elem_size(t->dtype);
    if (numel > 0 && (reinterpret_cast<uintptr_t>(t->data) % (align_strides16 ? 16 : es)))
        return fail(SSD_ERR_ALIGNMENT, "%s: base pointer %p not %zu-byte aligned", name, t->data,
                    align_strides16 ? size_t(16) : es);
    if (align_strides16)
        for (int i = 0; i < ndim - 1; ++i)
            if (shape[i] > 1 && (t->stride[i] * int64_t(es)) % 16)
                return fail(SSD_ERR_ALIGNMENT, "%s: stride[%d] = %lld elements is not a multiple "
                            "of 16 bytes", name, i, (long long)t->stride[i]);
    return SSD_OK;
}

ssd_status check_distinct(const ssd_tensor *t, const char *name) {
    // dimensions by stride, each at least as wide as all below it together
    int64_t reach = 1, below = -1;
    for (int k = 0; k < t->ndim; ++k) {
        int at = -1;
        for (int i = 0; i < t->ndim; ++i) {
            if (t->shape[i] <= 1) continue;
            const int64_t key = t->stride[i] * t->ndim + (t->ndim - 1 - i);
            if (key > below && (at < 0 || key < t->stride[at] * t->ndim + (t->ndim - 1 - at)))
                at = i;
        }
        if (at < 0) break;
        if (t->stride[at] < reach)
            return fail(SSD_ERR_INVALID_ARG, "%s: stride[%d] = %lld makes elements share memory",
                        name, at, (long long)t->stride[at]);
        reach = t->stride[at] * (t->shape[at] - 1) + reach;
        below = t->stride[at] * t->ndim + (t->ndim - 1 - at);
    }
    return SSD_OK;
}

ssd_status check_device_ptrs(std::initializer_list<NamedPtr> ptrs) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(SSD_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    for (const NamedPtr &np : ptrs) {
        if (!np.p) continue;
        cudaPointerAttributes at{};
        e = cudaPointerGetAttributes(&at, np.p);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return fail(SSD_ERR_INVALID_ARG, "%s: pointer %p is not CUDA memory (%s)", np.name,
                        np.p, cudaGetErrorString(e));
        }
        if (at.type == cudaMemoryTypeManaged) continue;
        if (at.type != cudaMemoryTypeDevice)
            return fail(SSD_ERR_INVALID_ARG, "%s: pointer %p is host memory; device memory is "
                        "required", np.name, np.p);
        if (at.device != dev)
            return fail(SSD_ERR_INVALID_ARG, "%s: pointer on device %d, current device is %d",
                        np.name, at.device, dev);
    }
    return SSD_OK;
}

ssd_status cuda_status(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return SSD_OK;
    return fail(SSD_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace checks

void set_error_detail(const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    checks::error_detail() = buf;
}
}  // namespace ssd

