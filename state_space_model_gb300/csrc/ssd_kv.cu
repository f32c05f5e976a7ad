// The key/value cache of attention layers: the normed, rotated and (for 8-bit
// pools) quantised write of new tokens, and the read back of cached ones.
#include "ssd_attn.h"
#include "ssd_debug.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#define SSD_DBG_FILE 7u   // kDbgKv

namespace ssd {
namespace {

constexpr float kCodeMax = 448.f;          // largest e4m3 value
constexpr float kAmaxFloor = 0x1p-96f;     // keeps the scale and its inverse normal numbers

// Eight consecutive elements of a row.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0];
    const float4 b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// Codes: v already divided by the row's scale (rounded to nearest even; above
// 448 saturated, which only the rounding of the division can reach).
__device__ __forceinline__ void store8_codes(uint8_t *p, const float (&v)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                     __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// grid (T, ceil(rows / rows per CTA)): the CTAs of token t take its Hq query,
// Hkv key and Hkv value rows, D/16 lanes to a row, two vectors of eight
// elements to a lane.  The two vectors of a lane hold partners of the
// rotation (i and i + R/2) where they lie in the first R places, so neither
// pairing needs another lane's values; the norm and the largest magnitude are
// sums and maxima over the D/16 lanes.  HBM-bound: every row is read once and
// written once, each lane's two 16-byte loads going out before the token's
// slot and position are known.
template <typename T, int D, bool kCodes>
__global__ void __launch_bounds__(512) k_kv_append(const KvAppendArgs a) {
    constexpr int LR = D / 16;
    const int t = blockIdx.x;
    const int rows = a.Hq + 2 * a.c.Hkv;
    const int j = (blockIdx.y * blockDim.x + threadIdx.x) / LR, l = threadIdx.x % LR;
    const int half = a.R / 16;
    const int v0 = l < half ? l : 2 * l, v1 = l < half ? l + half : 2 * l + 1;
    const bool is_q = j < a.Hq, is_v = j >= a.Hq + a.c.Hkv, live = j < rows;
    const int h = is_q ? j : (is_v ? j - a.Hq - a.c.Hkv : j - a.Hq);

    float x0[8] = {}, x1[8] = {};
    if (live) {
        const T *src = is_q   ? static_cast<const T *>(a.q) + t * a.q_st + h * a.q_sh
                       : is_v ? static_cast<const T *>(a.v) + t * a.v_st + h * a.v_sh
                              : static_cast<const T *>(a.k) + t * a.k_st + h * a.k_sh;
        load8(src + 8 * v0, x0);
        load8(src + 8 * v1, x1);
    }
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.c.pages * a.c.ps) return;      // padding (the whole CTA leaves)
    int pos = 0;
    if (a.cos) {
        pos = a.positions[t];
        if (pos < 0 || pos >= a.S) return;
    }

    const float *w = is_v ? nullptr : (is_q ? a.qw : a.kw);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], ss));
#pragma unroll
    for (int o = LR / 2; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
    if (w) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        float w0[8], w1[8];
        load8(w + 8 * v0, w0);
        load8(w + 8 * v1, w1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x0[i] *= r * w0[i];
            x1[i] *= r * w1[i];
        }
    }
    if (a.cos && !is_v && l < half) {
        const float *cs = a.cos + pos * a.cs_st, *sn = a.sin + pos * a.sn_st;
        if (a.interleaved) {   // pairs (2i, 2i + 1) inside each vector
            auto turn = [&](float (&x)[8], int v) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float c = cs[4 * v + i], s = sn[4 * v + i];
                    const float p = x[2 * i], q = x[2 * i + 1];
                    x[2 * i] = p * c - q * s;
                    x[2 * i + 1] = q * c + p * s;
                }
            };
            turn(x0, v0);
            turn(x1, v1);
        } else {               // x0 holds places i, x1 their partners i + R/2
            float c[8], s[8];
            load8(cs + 8 * l, c);
            load8(sn + 8 * l, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = x0[i], q = x1[i];
                x0[i] = p * c[i] - q * s[i];
                x1[i] = q * c[i] + p * s[i];
            }
        }
    }
    if (is_q) {
        T *o = static_cast<T *>(a.out) + t * a.o_st + h * a.o_sh;
        store8(o + 8 * v0, x0);
        store8(o + 8 * v1, x1);
    }
    const int page = slot / a.c.ps, at = slot - page * a.c.ps;
    const int64_t off = page * a.c.sp + h * a.c.sh + at * a.c.st;
    if constexpr (kCodes) {
        // the largest magnitude over the row's lanes; a NaN or an infinity
        // ends in a scale that makes the whole row NaN when it is read
        float amax = kAmaxFloor;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max_nan(amax, max_nan(fabsf(x0[i]), fabsf(x1[i])));
#pragma unroll
        for (int o = LR / 2; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(~0u, amax, o));
        if (!live || is_q) return;
        const float inv = kCodeMax / amax;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x0[i] *= inv;
            x1[i] *= inv;
        }
        if (SSD_IDX_OK(a.err, off + 8 * v1 + 7, a.c.n)) {
            uint8_t *o = static_cast<uint8_t *>(is_v ? a.c.v : a.c.k) + off;
            store8_codes(o + 8 * v0, x0);
            store8_codes(o + 8 * v1, x1);
        }
        const int64_t soff = page * a.c.ssp + h * a.c.ssh + at;
        if (l == 0 && SSD_IDX_OK(a.err, soff, a.c.ns))
            (is_v ? a.c.vs : a.c.ks)[soff] = amax * (1.f / kCodeMax);
    } else {
        if (!live || is_q) return;
        if (SSD_IDX_OK(a.err, off + 8 * v1 + 7, a.c.n)) {
            T *o = static_cast<T *>(is_v ? a.c.v : a.c.k) + off;
            store8(o + 8 * v0, x0);
            store8(o + 8 * v1, x1);
        }
    }
}

template <typename T, int D, bool kCodes>
cudaError_t append_t(const KvAppendArgs &a, cudaStream_t s) {
    constexpr int LR = D / 16;
    // a token's rows split evenly over the fewest CTAs of at most 512 threads
    const int lanes = (a.Hq + 2 * a.c.Hkv) * LR;
    const int ncta = (lanes + 511) / 512;
    const int threads = ((lanes + ncta - 1) / ncta + 31) / 32 * 32;
    k_kv_append<T, D, kCodes><<<dim3(unsigned(a.T), unsigned(ncta)), threads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t append_d(const KvAppendArgs &a, cudaStream_t s) {
    if (a.xdt == DT_F32)
        return a.c.dt == DT_F8E4M3 ? append_t<float, D, true>(a, s) : append_t<float, D, false>(a, s);
    return a.c.dt == DT_F8E4M3 ? append_t<__nv_bfloat16, D, true>(a, s)
                               : append_t<__nv_bfloat16, D, false>(a, s);
}

__device__ __forceinline__ void load8_codes(const uint8_t *p, float scale, float (&v)[8]) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = (i < 2 ? u.x : u.y) >> (16 * (i & 1));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w & 0xffffu), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        v[2 * i] = f.x * scale;
        v[2 * i + 1] = f.y * scale;
    }
}

// One thread to a vector of eight elements of a cached key and the same of
// its value, kReadUnroll tokens' worth of vectors apart, in the order of the
// output, so that stores are contiguous and loads are whole rows.  HBM-bound.
constexpr int kReadUnroll = 2;
template <typename T, typename P, int D>
__global__ void __launch_bounds__(256) k_kv_read(const KvReadArgs a) {
    constexpr int NV = D / 8;
    const int per = a.c.Hkv * NV;                              // vectors of a token
    const int64_t e0 = int64_t(blockIdx.x) * (256 * kReadUnroll);
    const int64_t i0 = e0 / per;
    const int r0 = int(e0 - i0 * per);
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
        const int r = r0 + u * 256 + threadIdx.x;
        const int64_t i = i0 + r / per;
        if (i >= a.T) break;
        const int hv = r % per, h = hv / NV, vec = hv % NV;
        // the sequence of row i: the last b with cu[b] <= i
        int lo = -1, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] <= i) lo = mid; else hi = mid;
        }
        float kx[8] = {}, vx[8] = {};
        if (lo >= 0 && i < a.cu[lo + 1]) {
            const int64_t pos = (a.starts ? a.starts[lo] : 0) + (i - a.cu[lo]);
            if (pos >= 0 && pos < int64_t(a.M) * a.c.ps) {
                const int pi = int(pos / a.c.ps), at = int(pos - int64_t(pi) * a.c.ps);
                const int page = a.table[lo * a.tb + pi];
                if (page >= 0 && page < a.c.pages) {
                    const int64_t off = page * a.c.sp + h * a.c.sh + at * a.c.st + 8 * vec;
                    if (SSD_IDX_OK(a.err, off + 7, a.c.n)) {
                        if constexpr (sizeof(P) == 1) {
                            const int64_t so = page * a.c.ssp + h * a.c.ssh + at;
                            load8_codes(static_cast<const uint8_t *>(a.c.k) + off, a.c.ks[so], kx);
                            load8_codes(static_cast<const uint8_t *>(a.c.v) + off, a.c.vs[so], vx);
                        } else {
                            load8(static_cast<const P *>(a.c.k) + off, kx);
                            load8(static_cast<const P *>(a.c.v) + off, vx);
                        }
                    }
                }
            }
        }
        store8(static_cast<T *>(a.k) + i * a.k_st + h * a.k_sh + 8 * vec, kx);
        store8(static_cast<T *>(a.v) + i * a.v_st + h * a.v_sh + 8 * vec, vx);
    }
}

template <typename T, typename P, int D>
cudaError_t read_t(const KvReadArgs &a, cudaStream_t s) {
    const int64_t items = a.T * a.c.Hkv * (D / 8);
    const int64_t blocks = (items + 256 * kReadUnroll - 1) / (256 * kReadUnroll);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    k_kv_read<T, P, D><<<unsigned(blocks), 256, 0, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t read_d(const KvReadArgs &a, cudaStream_t s) {
    if (a.c.dt == DT_F8E4M3)
        return a.odt == DT_F32 ? read_t<float, uint8_t, D>(a, s)
                               : read_t<__nv_bfloat16, uint8_t, D>(a, s);
    return a.c.dt == DT_F32 ? read_t<float, float, D>(a, s)
                            : read_t<__nv_bfloat16, __nv_bfloat16, D>(a, s);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &in, cudaStream_t s) {
    KvAppendArgs a = in;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    return a.c.D == 64 ? append_d<64>(a, s) : append_d<128>(a, s);
}

cudaError_t launch_kv_read(const KvReadArgs &in, cudaStream_t s) {
    KvReadArgs a = in;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    return a.c.D == 64 ? read_d<64>(a, s) : read_d<128>(a, s);
}

}  // namespace ssd
