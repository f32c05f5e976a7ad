// The key/value cache of attention layers: the normed, rotated and (for 8-bit
// pools) quantised write of new tokens, and the read back of cached ones.
#include "ssd_attn.h"
#include "ssd_debug.cuh"
#include "ssd_f32x2.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#define SSD_DBG_FILE 7u   // kDbgKv

namespace ssd {
namespace {

constexpr float kCodeMax = 448.f;          // largest e4m3 value
constexpr int kSms = 152;                  // of a GB300, for the launches' rules
constexpr int kFillWarps = kSms * 16;      // warps that fill the GPU
constexpr float kAmaxFloor = 0x1p-96f;     // keeps the scale and its inverse normal numbers

// Eight consecutive elements of a row as they lie in memory (held like that while
// loads are under way: a kernel's registers decide how many can be), and in fp32.
// Everything is read and written once; bf16 loads and stores and code loads carry streaming
// hints (32768 cached tokens read back: 38.9 us without, 36.9 with).
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
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
        u = __ldcs(reinterpret_cast<const uint4 *>(p));
    }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { __stcs(reinterpret_cast<uint4 *>(p), u); }
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
    __device__ __forceinline__ void load(const uint8_t *p) { u = __ldcs(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ void zero() { u = make_uint2(0, 0); }
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
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
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

__device__ __forceinline__ void pairs(const float (&v)[8], F2 (&r)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = f2(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void unpair(const F2 (&r)[4], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = parts(r[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// v / scale for each element, given the rounded inverse: the rounded product is corrected by
// its remainder, which a fused multiply-add gives exactly (P. Markstein, 1990).  An exact
// quotient, such as a tie between two codes, comes out exact: bf16 rows hold many (0.1% of
// their codes differed with the product alone).  4999 tokens of 24 + 2 x 4 heads of 64: 12.45
// us, with the product alone 12.3, with the division operator 14.4.
__device__ __forceinline__ void quotients(float (&v)[8], float scale, float inv) {
    F2 x[4];
    pairs(v, x);
    const F2 s = f2(-scale, -scale), r = f2(inv, inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const F2 q = mul(x[i], r);
        x[i] = fma(fma(q, s, x[i]), r, q);
    }
    unpair(x, v);
}

// A token's query, key and value rows are taken in passes of 512 / D rows of one kind,
// D / 16 lanes to a row, two vectors of eight elements a lane; a warp takes U passes
// of one token.  The two vectors of a lane hold partners of the rotation (i and
// i + R/2) where they lie in the first R places, so neither pairing needs another
// lane's values; the norm and the largest magnitude are sums and maxima over the row's
// lanes.  HBM-bound: every row is read once and written once, and all U loads of a
// warp go out before its token's slot, position and angles (which the passes share)
// are known.  Measured: 8192 tokens of 32 + 2 x 8 heads of 128 in bf16 35.3 us, 86% of
// the copy rate (57 us with a row a thread group and its angles read again for each
// row); in fp8 38 us, 73%, where the instructions begin to count; in fp32 65 us, 93%.  Few key heads leave
// lanes of their passes idle (4 of 64: half): 4999 tokens of 24 + 2 x 4 take 12.3 us.
constexpr int kAppendWarps = 4;
// kWhole: every row is turned whole (R = D).  Elsewhere places that are not turned keep what
// they hold, by a choice of results: a factor of 0 would bring infinities and NaN over from
// their neighbours.  (The choice in every lane of the 8192 tokens: 36.2 us.)
template <typename T, int D, bool kCodes, bool kWhole, int U>
__global__ void __launch_bounds__(32 * kAppendWarps, 6)
k_kv_append(const __grid_constant__ KvAppendArgs a, int warps) {
    constexpr int LR = D / 16, RPP = 32 / LR;
    const int64_t id = int64_t(blockIdx.x) * kAppendWarps + threadIdx.x / 32;
    const int t = __shfl_sync(~0u, int(id / warps), 0);
    if (t >= a.T) return;
    const int lane = threadIdx.x % 32, l = lane % LR, row = lane / LR;
    const int p0 = __shfl_sync(~0u, int(id - int64_t(t) * warps) * U, 0);
    const int qp = (a.Hq + RPP - 1) / RPP, kp = (a.c.Hkv + RPP - 1) / RPP;   // passes of a kind
    const int half = a.R / 16;
    const int v0 = l < half ? l : 2 * l, v1 = l < half ? l + half : 2 * l + 1;

    const int slot = a.slots[t], pos = a.cos ? a.positions[t] : 0;
    // pass u: its kind (0 query, 1 key, 2 value), and this lane's head of it
    auto kind_of = [&](int p) { return p < qp ? 0 : p < qp + kp ? 1 : 2; };
    auto head_of = [&](int p) { return (p < qp ? p : p < qp + kp ? p - qp : p - qp - kp) * RPP + row; };
    Raw8<T> x[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = p0 + u, kind = kind_of(p), h = head_of(p);
        const int64_t off = kind == 0   ? t * a.q_st + h * a.q_sh
                            : kind == 1 ? t * a.k_st + h * a.k_sh
                                        : t * a.v_st + h * a.v_sh;
        if (h < (kind == 0 ? a.Hq : a.c.Hkv) &&
            SSD_IDX_OK(a.err, off + 8 * v1 + 7, kind == 0 ? a.q_n : kind == 1 ? a.k_n : a.v_n)) {
            const T *src = static_cast<const T *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + off;
            x[u][0].load(src + 8 * v0);
            x[u][1].load(src + 8 * v1);
        } else {
            x[u][0].zero();
            x[u][1].zero();
        }
    }
    // padding: the whole warp leaves
    if (slot < 0 || slot >= a.c.pages * a.c.ps || (a.cos && (pos < 0 || pos >= a.S))) return;
    const int page = slot / a.c.ps, at = slot - page * a.c.ps;

    float cs[8], sn[8];       // interleaved: four for each vector
    bool turn = a.cos && l < half;
    if (turn) {       // the last column read: R/2 - 1
        [[maybe_unused]] const int64_t last = a.interleaved ? 4 * v1 + 3 : 8 * l + 7;
        turn = SSD_IDX_OK(a.err, pos * a.cs_st + last, a.cs_n) && SSD_IDX_OK(a.err, pos * a.sn_st + last, a.sn_n);
    }
    if (turn) {
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
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
    }
    const int64_t place = page * a.c.sp + at * a.c.st;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = p0 + u, kind = kind_of(p), h = head_of(p);
        if (p >= qp + 2 * kp) break;
        const bool live = h < (kind == 0 ? a.Hq : a.c.Hkv);
        if (!kCodes && kind == 2) {              // values as they are
            const int64_t off = place + h * a.c.sh;
            if (live && SSD_IDX_OK(a.err, off + 8 * v1 + 7, a.c.n)) {
                x[u][0].store(static_cast<T *>(a.c.v) + off + 8 * v0);
                x[u][1].store(static_cast<T *>(a.c.v) + off + 8 * v1);
            }
            continue;
        }
        float y0[8], y1[8];
        x[u][0].get(y0);
        x[u][1].get(y1);
        if (kind < 2) {
            F2 x0[4], x1[4];
            pairs(y0, x0);
            pairs(y1, x1);
            const float *w = kind == 0 ? a.qw : a.kw;
            if (w) {
                F2 sq = f2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) sq = fma(x0[i], x0[i], fma(x1[i], x1[i], sq));
                float ss = parts(sq).x + parts(sq).y;
#pragma unroll
                for (int o = LR / 2; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
                const float r = rsqrtf(ss * (1.f / D) + a.eps);
                float w0[8], w1[8];
                F2 w0p[4], w1p[4];
                load8(w + 8 * v0, w0);
                load8(w + 8 * v1, w1);
                pairs(w0, w0p);
                pairs(w1, w1p);
                const F2 rr = f2(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x0[i] = mul(x0[i], mul(w0p[i], rr));
                    x1[i] = mul(x1[i], mul(w1p[i], rr));
                }
            }
            if (!a.interleaved) {    // x0 holds places i, x1 their partners i + R/2
                F2 c[4], n[4];
                pairs(cs, c);
                pairs(sn, n);
                const F2 minus = f2(-1.f, -1.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 p = x0[i], q = x1[i];
                    const F2 u = fma(p, c[i], mul(mul(q, n[i]), minus)), v = fma(q, c[i], mul(p, n[i]));
                    x0[i] = kWhole || turn ? u : p;
                    x1[i] = kWhole || turn ? v : q;
                }
                unpair(x0, y0);
                unpair(x1, y1);
            } else {                 // pairs (2i, 2i + 1) inside each vector
                unpair(x0, y0);
                unpair(x1, y1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p0 = y0[2 * i], q0 = y0[2 * i + 1], p1 = y1[2 * i], q1 = y1[2 * i + 1];
                    if (turn) {
                        y0[2 * i] = p0 * cs[i] - q0 * sn[i];
                        y0[2 * i + 1] = q0 * cs[i] + p0 * sn[i];
                        y1[2 * i] = p1 * cs[4 + i] - q1 * sn[4 + i];
                        y1[2 * i + 1] = q1 * cs[4 + i] + p1 * sn[4 + i];
                    }
                }
            }
        }
        if (kind == 0) {
            const int64_t off = t * a.o_st + h * a.o_sh;
            if (live && SSD_IDX_OK(a.err, off + 8 * v1 + 7, a.o_n)) {
                T *o = static_cast<T *>(a.out) + off;
                store8(o + 8 * v0, y0);
                store8(o + 8 * v1, y1);
            }
            continue;
        }
        const int64_t off = place + h * a.c.sh;
        const bool in = live && SSD_IDX_OK(a.err, off + 8 * v1 + 7, a.c.n);
        if constexpr (kCodes) {
            // the largest magnitude over the row's lanes; a NaN or an infinity
            // ends in a scale that makes the whole row NaN when it is read
            float amax = kAmaxFloor;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max_nan(amax, max_nan(fabsf(y0[i]), fabsf(y1[i])));
#pragma unroll
            for (int o = LR / 2; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(~0u, amax, o));
            const float scale = amax * (1.f / kCodeMax), inv = 1.f / scale;
            quotients(y0, scale, inv);
            quotients(y1, scale, inv);
            if (in) {
                uint8_t *o = static_cast<uint8_t *>(kind == 2 ? a.c.v : a.c.k) + off;
                store8_codes(o + 8 * v0, y0);
                store8_codes(o + 8 * v1, y1);
                const int64_t soff = page * a.c.ssp + h * a.c.ssh + at;
                if (l == 0 && SSD_IDX_OK(a.err, soff, a.c.ns))
                    (kind == 2 ? a.c.vs : a.c.ks)[soff] = scale;
            }
        } else if (in) {
            T *o = static_cast<T *>(a.c.k) + off;
            store8(o + 8 * v0, y0);
            store8(o + 8 * v1, y1);
        }
    }
}

template <typename T, int D, bool kCodes, int U>
cudaError_t append_u(const KvAppendArgs &a, cudaStream_t s) {
    constexpr int RPP = 512 / D;
    const int passes = (a.Hq + RPP - 1) / RPP + 2 * ((a.c.Hkv + RPP - 1) / RPP);
    const int warps = (passes + U - 1) / U;
    const int64_t blocks = (a.T * warps + kAppendWarps - 1) / kAppendWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    // (a warp a pass waits for its loads, whatever it computes)
    if (U > 1 && a.R == D)
        k_kv_append<T, D, kCodes, (U > 1), U><<<unsigned(blocks), 32 * kAppendWarps, 0, s>>>(a, warps);
    else
        k_kv_append<T, D, kCodes, false, U><<<unsigned(blocks), 32 * kAppendWarps, 0, s>>>(a, warps);
    return cudaGetLastError();
}

// As few warps a token as take at most four passes each (fp32: two, for their
// registers), the passes spread evenly over them, where that still fills the GPU with
// warps: one load of the angles for a warp's passes, all their loads in flight (4999
// tokens of 24 + 2 x 4 heads 12.3 us, with a warp a pass 14.4).  Else a warp a pass, so
// that a few tokens spread over as many SMs as they can (the kernel alone, 64 tokens of
// 64 + 2 x 8 heads in fp8 4.1 us, with four passes a warp 5.5; one token 3.7 and 5.8).
template <typename T, int D, bool kCodes>
cudaError_t append_t(const KvAppendArgs &a, cudaStream_t s) {
    constexpr int RPP = 512 / D, kMost = sizeof(T) == 4 ? 2 : 4;
    const int passes = (a.Hq + RPP - 1) / RPP + 2 * ((a.c.Hkv + RPP - 1) / RPP);
    const int warps = (passes + kMost - 1) / kMost;
    if (a.T * warps < kFillWarps) return append_u<T, D, kCodes, 1>(a, s);
    // three passes and more (a kind has at least one) spread as kMost or kMost - 1 to a warp
    if constexpr (kMost == 2) return append_u<T, D, kCodes, 2>(a, s);
    else if ((passes + warps - 1) / warps == 4) return append_u<T, D, kCodes, 4>(a, s);
    else return append_u<T, D, kCodes, 3>(a, s);
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
// HBM-bound.  Measured: 32768 tokens of 8 heads of 128 in 8 bits 34.9 us, 86% of the
// copy rate (47 us with every vector looking up its own token), 262144 of them 253 us,
// 95%.
constexpr int kReadTokens = 32;      // most tokens of a CTA
constexpr int kNearLens = 512;       // sequences whose cu_lens a CTA keeps near
template <typename T, typename P, int D>
__global__ void __launch_bounds__(256, 4) k_kv_read(const __grid_constant__ KvReadArgs a, int TB) {
    constexpr int NV = D / 8;
    constexpr int kReadAhead = sizeof(P) == 4 ? 2 : 4;
    __shared__ int64_t off_of[kReadTokens], soff_of[kReadTokens];
    __shared__ int32_t near_cu[kNearLens];
    const int64_t i0 = int64_t(blockIdx.x) * TB;
    const int n = int(min(int64_t(TB), a.T - i0));
    // the bisection's loads depend on one another: from shared memory where they fit (the
    // kernel alone, 300 sequences of up to 20: 5.7 us, from global memory 6.5)
    const int32_t *cu = a.cu;
    if (a.B < kNearLens) {
        for (int i = threadIdx.x; i <= a.B; i += 256) near_cu[i] = a.cu[i];
        __syncthreads();
        cu = near_cu;
    }
    if (threadIdx.x < n) {
        const int64_t i = i0 + threadIdx.x;
        // the sequence of row i: the last b with cu[b] <= i
        int lo = -1, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= i) lo = mid; else hi = mid;
        }
        int64_t off = -1, soff = 0;
        if (lo >= 0 && i < cu[lo + 1]) {
            const int64_t pos = (a.starts ? a.starts[lo] : 0) + (i - cu[lo]);
            if (pos >= 0 && pos < int64_t(a.M) * a.c.ps) {
                const int pi = int(pos) / a.c.ps, at = int(pos) - pi * a.c.ps;
                const int64_t entry = lo * a.tb + pi;
                const int page = SSD_IDX_OK(a.err, entry, a.t_n) ? a.table[entry] : -1;
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
    // A thread keeps its place in a token (head, vector) and takes every `apart`-th token;
    // where a token has more vectors than the CTA threads, one place after another.
    const int per = a.c.Hkv * NV, apart = per < 256 ? 256 / per : 1;
    const int tok0 = threadIdx.x / per;
    for (int place = threadIdx.x - tok0 * per; tok0 < apart && place < per; place += 256) {
        const int h = place / NV, vec = place % NV;
        const int64_t in = h * a.c.sh + 8 * vec, sin = h * a.c.ssh;
        T *ko = static_cast<T *>(a.k) + i0 * a.k_st + h * a.k_sh + 8 * vec;
        T *vo = static_cast<T *>(a.v) + i0 * a.v_st + h * a.v_sh + 8 * vec;
        for (int tok = tok0; tok < n; tok += apart * kReadAhead) {
            Raw8<P> kx[kReadAhead], vx[kReadAhead];
            float ks[kReadAhead], vs[kReadAhead];
#pragma unroll
            for (int u = 0; u < kReadAhead; ++u) {
                const int i = min(tok + u * apart, n - 1);
                const int64_t off = off_of[i] + in;
                ks[u] = vs[u] = 0.f;
                if (off_of[i] >= 0 && SSD_IDX_OK(a.err, off + 7, a.c.n)) {
                    kx[u].load(static_cast<const P *>(a.c.k) + off);
                    vx[u].load(static_cast<const P *>(a.c.v) + off);
                    if constexpr (sizeof(P) == 1) {
                        if (SSD_IDX_OK(a.err, soff_of[i] + sin, a.c.ns)) {
                            ks[u] = a.c.ks[soff_of[i] + sin];
                            vs[u] = a.c.vs[soff_of[i] + sin];
                        }
                    }
                } else {
                    kx[u].zero();
                    vx[u].zero();
                }
            }
#pragma unroll
            for (int u = 0; u < kReadAhead; ++u) {
                const int i = tok + u * apart;
                if (i >= n) break;
                if (!SSD_IDX_OK(a.err, (i0 + i) * a.k_st + h * a.k_sh + 8 * vec + 7, a.k_n) ||
                    !SSD_IDX_OK(a.err, (i0 + i) * a.v_st + h * a.v_sh + 8 * vec + 7, a.v_n))
                    continue;
                if constexpr (sizeof(P) == 1) {
                    float k[8], v[8];
                    kx[u].get(k);
                    vx[u].get(v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        k[j] *= ks[u];
                        v[j] *= vs[u];
                    }
                    store8(ko + i * a.k_st, k);
                    store8(vo + i * a.v_st, v);
                } else {
                    kx[u].store(ko + i * a.k_st);
                    vx[u].store(vo + i * a.v_st);
                }
            }
        }
    }
}

template <typename T, typename P, int D>
cudaError_t read_t(const KvReadArgs &a, cudaStream_t s) {
    // tokens of a CTA: 1024 vectors' worth, fewer where that leaves SMs without one (the
    // kernel alone, 300 tokens of 4 heads of 64: 4.4 us, with 32 a CTA 4.7)
    int TB = 1024 / (a.c.Hkv * (D / 8));
    TB = TB < 1 ? 1 : TB > kReadTokens ? kReadTokens : TB;
    while (TB > 1 && (a.T + TB - 1) / TB < kSms) TB /= 2;
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
