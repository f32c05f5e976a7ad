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
constexpr int kFillRows = 152 * 16;        // warps that fill the GPU
constexpr float kAmaxFloor = 0x1p-96f;     // keeps the scale and its inverse normal numbers

// Eight consecutive elements of a row as they lie in memory (held like that while
// loads are under way: a kernel's registers decide how many can be), and in fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        u = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Raw8<uint8_t> {       // e4m3 codes
    uint2 u;
    __device__ __forceinline__ void load(const uint8_t *p) { u = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = (i < 2 ? u.x : u.y) >> (16 * (i & 1));
            const __half2_raw h =
                __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w & 0xffffu), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    Raw8<T> r;
    r.load(p);
    r.get(v);
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

// A token has Hq query, Hkv key and Hkv value rows; D/16 lanes take a row, two
// vectors of eight elements a lane, and a warp U times 512 / D rows of one token.
// The two vectors of a lane hold partners of the rotation (i and i + R/2) where
// they lie in the first R places, so neither pairing needs another lane's values;
// the norm and the largest magnitude are sums and maxima over the row's lanes.
// HBM-bound: every row is read once and written once, and all U loads of a warp go
// out before its token's slot, position and angles (which the rows share) are
// known.  8192 tokens of 32 + 2 x 8 heads of 128 with the four-byte angles of a token
// read again by each row took 53 us.
constexpr int kAppendWarps = 4;
template <typename T, int D, bool kCodes, int U>
__global__ void __launch_bounds__(32 * kAppendWarps) k_kv_append(const KvAppendArgs a, int warps) {
    constexpr int LR = D / 16, RPP = 32 / LR;
    const int64_t id = int64_t(blockIdx.x) * kAppendWarps + threadIdx.x / 32;
    const int t = int(id / warps);
    if (t >= a.T) return;
    const int lane = threadIdx.x % 32, l = lane % LR;
    const int j0 = int(id - int64_t(t) * warps) * (U * RPP) + lane / LR;    // this lane's first row
    const int rows = a.Hq + 2 * a.c.Hkv;
    const int half = a.R / 16;
    const int v0 = l < half ? l : 2 * l, v1 = l < half ? l + half : 2 * l + 1;

    const int slot = a.slots[t], pos = a.cos ? a.positions[t] : 0;
    Raw8<T> x[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int j = min(j0 + u * RPP, rows - 1);
        const T *src = j < a.Hq ? static_cast<const T *>(a.q) + t * a.q_st + j * a.q_sh
                       : j < a.Hq + a.c.Hkv
                           ? static_cast<const T *>(a.k) + t * a.k_st + (j - a.Hq) * a.k_sh
                           : static_cast<const T *>(a.v) + t * a.v_st + (j - a.Hq - a.c.Hkv) * a.v_sh;
        x[u][0].load(src + 8 * v0);
        x[u][1].load(src + 8 * v1);
    }
    // padding: the whole warp leaves
    if (slot < 0 || slot >= a.c.pages * a.c.ps || (a.cos && (pos < 0 || pos >= a.S))) return;
    const int page = slot / a.c.ps, at = slot - page * a.c.ps;

    float cs[8] = {}, sn[8] = {};       // interleaved: four for each vector
    if (a.cos && l < half) {
        const float *cp = a.cos + pos * a.cs_st, *sp = a.sin + pos * a.sn_st;
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 c = *reinterpret_cast<const float4 *>(cp + 4 * (i ? v1 : v0));
                const float4 s = *reinterpret_cast<const float4 *>(sp + 4 * (i ? v1 : v0));
                cs[4 * i] = c.x, cs[4 * i + 1] = c.y, cs[4 * i + 2] = c.z, cs[4 * i + 3] = c.w;
                sn[4 * i] = s.x, sn[4 * i + 1] = s.y, sn[4 * i + 2] = s.z, sn[4 * i + 3] = s.w;
            }
        } else {
            load8(cp + 8 * l, cs);
            load8(sp + 8 * l, sn);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int j = j0 + u * RPP;
        const bool is_q = j < a.Hq, is_v = j >= a.Hq + a.c.Hkv, live = j < rows;
        const int h = is_q ? j : (is_v ? j - a.Hq - a.c.Hkv : j - a.Hq);
        float x0[8], x1[8];
        x[u][0].get(x0);
        x[u][1].get(x1);
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
            if (a.interleaved) {   // pairs (2i, 2i + 1) inside each vector
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p0 = x0[2 * i], q0 = x0[2 * i + 1], p1 = x1[2 * i], q1 = x1[2 * i + 1];
                    x0[2 * i] = p0 * cs[i] - q0 * sn[i];
                    x0[2 * i + 1] = q0 * cs[i] + p0 * sn[i];
                    x1[2 * i] = p1 * cs[4 + i] - q1 * sn[4 + i];
                    x1[2 * i + 1] = q1 * cs[4 + i] + p1 * sn[4 + i];
                }
            } else {               // x0 holds places i, x1 their partners i + R/2
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = x0[i], q = x1[i];
                    x0[i] = p * cs[i] - q * sn[i];
                    x1[i] = q * cs[i] + p * sn[i];
                }
            }
        }
        float amax = kAmaxFloor;
        if constexpr (kCodes) {
            // the largest magnitude over the row's lanes; a NaN or an infinity
            // ends in a scale that makes the whole row NaN when it is read
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max_nan(amax, max_nan(fabsf(x0[i]), fabsf(x1[i])));
#pragma unroll
            for (int o = LR / 2; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(~0u, amax, o));
        }
        if (!live) continue;
        if (is_q) {
            T *o = static_cast<T *>(a.out) + t * a.o_st + h * a.o_sh;
            store8(o + 8 * v0, x0);
            store8(o + 8 * v1, x1);
            continue;
        }
        const int64_t off = page * a.c.sp + h * a.c.sh + at * a.c.st;
        if (!SSD_IDX_OK(a.err, off + 8 * v1 + 7, a.c.n)) continue;
        if constexpr (kCodes) {
            const float inv = kCodeMax / amax;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x0[i] *= inv;
                x1[i] *= inv;
            }
            uint8_t *o = static_cast<uint8_t *>(is_v ? a.c.v : a.c.k) + off;
            store8_codes(o + 8 * v0, x0);
            store8_codes(o + 8 * v1, x1);
            const int64_t soff = page * a.c.ssp + h * a.c.ssh + at;
            if (l == 0 && SSD_IDX_OK(a.err, soff, a.c.ns))
                (is_v ? a.c.vs : a.c.ks)[soff] = amax * (1.f / kCodeMax);
        } else {
            T *o = static_cast<T *>(is_v ? a.c.v : a.c.k) + off;
            store8(o + 8 * v0, x0);
            store8(o + 8 * v1, x1);
        }
    }
}

template <typename T, int D, bool kCodes, int U>
cudaError_t append_u(const KvAppendArgs &a, cudaStream_t s) {
    constexpr int per = U * 512 / D;          // rows of a warp
    const int warps = (a.Hq + 2 * a.c.Hkv + per - 1) / per;
    const int64_t blocks = (a.T * warps + kAppendWarps - 1) / kAppendWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    k_kv_append<T, D, kCodes, U><<<unsigned(blocks), 32 * kAppendWarps, 0, s>>>(a, warps);
    return cudaGetLastError();
}

// Four times 512 / D rows to a warp where that still fills the GPU with warps (one
// load of the angles for them, four rows' loads in flight); else one, so that a few
// tokens spread over as many SMs as they can.
template <typename T, int D, bool kCodes>
cudaError_t append_t(const KvAppendArgs &a, cudaStream_t s) {
    const int64_t rows = a.T * (a.Hq + 2 * a.c.Hkv);
    return rows * D >= int64_t(kFillRows) * 512 * 4 ? append_u<T, D, kCodes, 4>(a, s)
                                                    : append_u<T, D, kCodes, 1>(a, s);
}

template <int D>
cudaError_t append_d(const KvAppendArgs &a, cudaStream_t s) {
    if (a.xdt == DT_F32)
        return a.c.dt == DT_F8E4M3 ? append_t<float, D, true>(a, s) : append_t<float, D, false>(a, s);
    return a.c.dt == DT_F8E4M3 ? append_t<__nv_bfloat16, D, true>(a, s)
                               : append_t<__nv_bfloat16, D, false>(a, s);
}

// A CTA takes TB tokens: their places in the pools are looked up first (a thread
// a token: the sequence by bisection, then its page), then the threads copy vectors
// of eight elements of keys and values in the order of the output, kReadAhead of
// each in flight, so that stores are contiguous and loads are whole rows.
// HBM-bound.  With every vector looking up its own token (three dependent loads each),
// 32768 tokens of 8 heads of 128 in 8 bits took 47 us.
constexpr int kReadTokens = 32;      // most tokens of a CTA
template <typename T, typename P, int D>
__global__ void __launch_bounds__(256) k_kv_read(const KvReadArgs a, int TB) {
    constexpr int NV = D / 8;
    constexpr int kReadAhead = sizeof(P) == 4 ? 2 : 4;
    __shared__ int64_t off_of[kReadTokens], soff_of[kReadTokens];
    const int64_t i0 = int64_t(blockIdx.x) * TB;
    const int n = int(min(int64_t(TB), a.T - i0));
    if (threadIdx.x < n) {
        const int64_t i = i0 + threadIdx.x;
        // the sequence of row i: the last b with cu[b] <= i
        int lo = -1, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] <= i) lo = mid; else hi = mid;
        }
        int64_t off = -1, soff = 0;
        if (lo >= 0 && i < a.cu[lo + 1]) {
            const int64_t pos = (a.starts ? a.starts[lo] : 0) + (i - a.cu[lo]);
            if (pos >= 0 && pos < int64_t(a.M) * a.c.ps) {
                const int pi = int(pos) / a.c.ps, at = int(pos) - pi * a.c.ps;
                const int page = a.table[lo * a.tb + pi];
                if (page >= 0 && page < a.c.pages) {
                    off = page * a.c.sp + at * a.c.st;
                    soff = page * a.c.ssp + at;
                }
            }
        }
        off_of[threadIdx.x] = off;
        soff_of[threadIdx.x] = soff;
    }
    __syncthreads();
    const int per = a.c.Hkv * NV, all = n * per;      // vectors of a token, of the CTA
    for (int r0 = threadIdx.x; r0 < all; r0 += 256 * kReadAhead) {
        Raw8<P> kx[kReadAhead], vx[kReadAhead];
        float ks[kReadAhead], vs[kReadAhead];
        bool there[kReadAhead];
#pragma unroll
        for (int u = 0; u < kReadAhead; ++u) {
            const int r = min(r0 + 256 * u, all - 1), tok = r / per;
            const int h = (r - tok * per) / NV, vec = r % NV;     // per is a multiple of NV
            const int64_t off = off_of[tok] + h * a.c.sh + 8 * vec;
            there[u] = off_of[tok] >= 0 && SSD_IDX_OK(a.err, off + 7, a.c.n);
            if (there[u]) {
                kx[u].load(static_cast<const P *>(a.c.k) + off);
                vx[u].load(static_cast<const P *>(a.c.v) + off);
                if constexpr (sizeof(P) == 1) {
                    const int64_t so = soff_of[tok] + h * a.c.ssh;
                    ks[u] = a.c.ks[so];
                    vs[u] = a.c.vs[so];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kReadAhead; ++u) {
            const int r = r0 + 256 * u;
            if (r >= all) break;
            const int tok = r / per, h = (r - tok * per) / NV, vec = r % NV;
            float k[8] = {}, v[8] = {};
            if (there[u]) {
                kx[u].get(k);
                vx[u].get(v);
                if constexpr (sizeof(P) == 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        k[i] *= ks[u];
                        v[i] *= vs[u];
                    }
                }
            }
            store8(static_cast<T *>(a.k) + (i0 + tok) * a.k_st + h * a.k_sh + 8 * vec, k);
            store8(static_cast<T *>(a.v) + (i0 + tok) * a.v_st + h * a.v_sh + 8 * vec, v);
        }
    }
}

template <typename T, typename P, int D>
cudaError_t read_t(const KvReadArgs &a, cudaStream_t s) {
    // tokens of a CTA: 1024 vectors' worth, fewer where that leaves SMs without one
    int TB = 1024 / (a.c.Hkv * (D / 8));
    TB = TB < 1 ? 1 : TB > kReadTokens ? kReadTokens : TB;
    while (TB > 1 && (a.T + TB - 1) / TB < 152) TB /= 2;
    const int64_t blocks = (a.T + TB - 1) / TB;
    k_kv_read<T, P, D><<<unsigned(blocks), 256, 0, s>>>(a, TB);
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
