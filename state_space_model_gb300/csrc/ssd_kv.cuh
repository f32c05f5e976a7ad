// The key/value cache of attention layers: the normed, rotated and (for pools of codes)
// quantised write of new tokens, and the read back of cached ones.  The kernels and
// their launch rules; ssd_kv.cu and ssd_kv_ex.cu compile them for the pools' types and
// the positions' axes.
#pragma once
#include "ssd_attn.h"
#include "ssd_debug.cuh"
#include "ssd_f32x2.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <type_traits>

#define SSD_DBG_FILE 7u   // kDbgKv

namespace ssd {
namespace {

constexpr float kCodeMax = 448.f;          // largest e4m3 value
constexpr float kFourMax = 6.f;            // largest e2m1 value
// What the pools hold: the layer's type, or codes of 8 or 4 bits.
enum : int { kPlain = 0, kEight = 1, kFour = 2 };
struct Nibbles {};                         // the element type of a pool of 4-bit codes
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
// Four bytes of e2m1 codes -> eight values (exact), as pairs of fp16.
__device__ __forceinline__ void widen8(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}
template <>
struct Raw8<Nibbles> {
    uint32_t u;
    __device__ __forceinline__ void load(const uint8_t *p) { u = __ldcs(reinterpret_cast<const uint32_t *>(p)); }
    __device__ __forceinline__ void zero() { u = 0; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        uint32_t h[4];
        widen8(u, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};
__device__ __forceinline__ float from_e4m3(uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half *>(&h));
}
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

// 4-bit codes: v already divided by the group's step (rounded to nearest even, above 6
// saturated).
__device__ __forceinline__ uint32_t pack8_codes(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
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
// kAxes: positions of several axes; a warp collects the angles of its token's columns, each from its
// axis's row of the table, in shared memory (4999 tokens of 28 + 2 x 4 heads: 20.5 us; a lane that
// loads every axis's vectors and keeps what is its own, 0.7 more).
// CTAs of an SM, by the passes of a warp: a few spilled words (up to 96 bytes of loads) cost less than a CTA
// in flight.  8192 tokens, with these / with as many as nothing spills with: bf16, 32 + 2 x 8 heads of 128,
// four passes 33.6 / 35.6 us, to 4 bits 41.0 / 42.8; 28 + 2 x 4, three axes, three passes 31.9 / 36.4; fp32,
// 16 + 2 x 8, three axes, two passes to 8 bits 48.2 / 55.6.  Two passes in fp32 with one axis gain nothing from
// eight (to 8 bits 20.4 us with heads of 64, half turned 24.8; with seven, which spill nothing, 20.3 and 24.0;
// six 20.9 and 24.5).
template <typename T, bool kAxes, int U>
constexpr int append_ctas() {
    return U == 4 ? 6 : U == 3 || (U == 2 && sizeof(T) == 4 && !kAxes) ? 7 : 8;
}
template <typename T, int D, int kCodes, bool kWhole, bool kAxes, int U>
__global__ void __launch_bounds__(32 * kAppendWarps, (append_ctas<T, kAxes, U>()))
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
    int more[kMaxAxes - 1];                  // the other axes' positions
    bool on_table = !a.cos || (pos >= 0 && pos < a.S);
    if constexpr (kAxes) {
#pragma unroll
        for (int j = 1; j < kMaxAxes; ++j) more[j - 1] = j < a.axes ? a.positions[j * a.T + t] : pos;
#pragma unroll
        for (int j = 1; j < kMaxAxes; ++j) on_table = on_table && more[j - 1] >= 0 && more[j - 1] < a.S;
    }
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
    if (slot < 0 || slot >= a.c.pages * a.c.ps || !on_table) return;
    const int page = slot / a.c.ps, at = slot - page * a.c.ps;

    float cs[8], sn[8];       // interleaved: four for each vector
    bool turn = a.cos && l < half;
    if (turn) {       // the last column read: R/2 - 1
        [[maybe_unused]] const int64_t last = a.interleaved ? 4 * v1 + 3 : 8 * l + 7;
        turn = SSD_IDX_OK(a.err, pos * a.cs_st + last, a.cs_n) && SSD_IDX_OK(a.err, pos * a.sn_st + last, a.sn_n);
    }
    if constexpr (kAxes) {
        // column by column, each from its axis's row, for all rows of the warp
        __shared__ __align__(16) float angles[kAppendWarps][2][D / 2];
        float(&held)[2][D / 2] = angles[threadIdx.x / 32];
        for (int c = lane; c < a.R / 2; c += 32) {
            const int axis = a.axis_of[c / 16] >> (2 * (c % 16)) & 3;
            const int64_t p = axis == 0 ? pos : axis == 1 ? more[0] : axis == 2 ? more[1] : more[2];
            if (SSD_IDX_OK(a.err, p * a.cs_st + c, a.cs_n)) held[0][c] = a.cos[p * a.cs_st + c];
            if (SSD_IDX_OK(a.err, p * a.sn_st + c, a.sn_n)) held[1][c] = a.sin[p * a.sn_st + c];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c0 = a.interleaved ? 4 * (i ? v1 : v0) : 8 * l + 4 * i;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                cs[4 * i + k] = turn ? held[0][c0 + k] : 1.f;
                sn[4 * i + k] = turn ? held[1][c0 + k] : 0.f;
            }
        }
    } else if (turn) {
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
        if (kCodes == kPlain && kind == 2) {     // values as they are
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
        const bool in = live && SSD_IDX_OK(a.err, off + (kCodes == kFour ? 4 * v1 + 3 : 8 * v1 + 7), a.c.n);
        if constexpr (kCodes == kFour) {
            // a row's scale from its largest magnitude, a group's from that of its two vectors,
            // which two lanes hold or one; NaN as below
            float m[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[0] = max_nan(m[0], fabsf(y0[i]));
                m[1] = max_nan(m[1], fabsf(y1[i]));
            }
            float amax = max_nan(kAmaxFloor, max_nan(m[0], m[1]));
#pragma unroll
            for (int o = LR / 2; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(~0u, amax, o));
            const float scale = amax * (1.f / (kFourMax * kCodeMax)), six = kFourMax * scale;
            const int64_t goff = page * a.c.sgp + h * a.c.sgh + at * a.c.sgt;
            uint8_t *const rows = static_cast<uint8_t *>(kind == 2 ? a.c.v : a.c.k) + off;
            float own[2], step[2];
            uint8_t g[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int w = (i ? v1 : v0) ^ 1;          // the group's other vector: whose, which
                const bool low = w < half, mid = !low && w < 2 * half;
                const int from = row * LR + (low ? w : mid ? w - half : w >> 1);
                const float m0 = __shfl_sync(~0u, m[0], from), m1 = __shfl_sync(~0u, m[1], from);
                own[i] = max_nan(m[i], (low ? false : mid ? true : w & 1) ? m1 : m0);
                g[i] = __nv_cvt_float_to_fp8(own[i] / six, __NV_SATFINITE, __NV_E4M3);
                step[i] = from_e4m3(g[i]) * scale;
            }
            quotients(y0, step[0], step[0] == 0.f ? 0.f : 1.f / step[0]);
            quotients(y1, step[1], step[1] == 0.f ? 0.f : 1.f / step[1]);
            if (in) {
                *reinterpret_cast<uint32_t *>(rows + 4 * v0) = pack8_codes(y0);
                *reinterpret_cast<uint32_t *>(rows + 4 * v1) = pack8_codes(y1);
                uint8_t *const groups = (kind == 2 ? a.c.vg : a.c.kg) + goff;
                if (v0 % 2 == 0 && SSD_IDX_OK(a.err, goff + v0 / 2, a.c.ng)) groups[v0 / 2] = g[0];
                if (v1 % 2 == 0 && SSD_IDX_OK(a.err, goff + v1 / 2, a.c.ng)) groups[v1 / 2] = g[1];
                const int64_t soff = page * a.c.ssp + h * a.c.ssh + at;
                if (l == 0 && SSD_IDX_OK(a.err, soff, a.c.ns))
                    (kind == 2 ? a.c.vs : a.c.ks)[soff] = scale;
            }
        } else if constexpr (kCodes == kEight) {
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

template <typename T, int D, int kCodes, bool kAxes, int U>
cudaError_t append_u(const KvAppendArgs &a, cudaStream_t s) {
    constexpr int RPP = 512 / D;
    const int passes = (a.Hq + RPP - 1) / RPP + 2 * ((a.c.Hkv + RPP - 1) / RPP);
    const int warps = (passes + U - 1) / U;
    const int64_t blocks = (a.T * warps + kAppendWarps - 1) / kAppendWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    // (a warp a pass waits for its loads, whatever it computes)
    if (U > 1 && !kAxes && a.R == D)
        k_kv_append<T, D, kCodes, (U > 1 && !kAxes), kAxes, U>
            <<<unsigned(blocks), 32 * kAppendWarps, 0, s>>>(a, warps);
    else
        k_kv_append<T, D, kCodes, false, kAxes, U>
            <<<unsigned(blocks), 32 * kAppendWarps, 0, s>>>(a, warps);
    return cudaGetLastError();
}

// As few warps a token as take at most four passes each (fp32: two, for their
// registers; 4-bit heads of 64 too: 5000 tokens of 24 + 2 x 4 14.4 us, with up to four
// 16.4), the passes spread evenly over them, where that still fills the GPU with
// warps: one load of the angles for a warp's passes, all their loads in flight (4999
// tokens of 24 + 2 x 4 heads 12.3 us, with a warp a pass 14.4).  Else a warp a pass, so
// that a few tokens spread over as many SMs as they can (the kernel alone, 64 tokens of
// 64 + 2 x 8 heads in fp8 4.1 us, with four passes a warp 5.5; one token 3.7 and 5.8).
template <typename T, int D, int kCodes, bool kAxes>
cudaError_t append_t(const KvAppendArgs &a, cudaStream_t s) {
    constexpr int RPP = 512 / D, kMost = sizeof(T) == 4 || (kCodes == kFour && D == 64) ? 2 : 4;
    const int passes = (a.Hq + RPP - 1) / RPP + 2 * ((a.c.Hkv + RPP - 1) / RPP);
    const int warps = (passes + kMost - 1) / kMost;
    if (a.T * warps < kFillWarps) return append_u<T, D, kCodes, kAxes, 1>(a, s);
    // three passes and more (a kind has at least one) spread as kMost or kMost - 1 to a warp
    if constexpr (kMost == 2) return append_u<T, D, kCodes, kAxes, 2>(a, s);
    else if ((passes + warps - 1) / warps == 4) return append_u<T, D, kCodes, kAxes, 4>(a, s);
    else return append_u<T, D, kCodes, kAxes, 3>(a, s);
}

template <int kCodes, bool kAxes>
cudaError_t append_codes(const KvAppendArgs &a, cudaStream_t s) {
    if (a.xdt == DT_F32)
        return a.c.D == 64 ? append_t<float, 64, kCodes, kAxes>(a, s)
                           : append_t<float, 128, kCodes, kAxes>(a, s);
    return a.c.D == 64 ? append_t<__nv_bfloat16, 64, kCodes, kAxes>(a, s)
                       : append_t<__nv_bfloat16, 128, kCodes, kAxes>(a, s);
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
__global__ void __launch_bounds__(256, std::is_same_v<P, Nibbles> ? 5 : 4) k_kv_read(const __grid_constant__ KvReadArgs a, int TB) {
    constexpr int NV = D / 8;
    constexpr bool kFours = std::is_same_v<P, Nibbles>;
    constexpr bool kCodes = sizeof(P) == 1;
    using Byte = std::conditional_t<kFours, uint8_t, P>;
    constexpr int kReadAhead = sizeof(P) == 4 ? 2 : 4;
    constexpr int NB = kFours ? 4 : 8;       // elements of the pool (bytes, 4-bit codes) of a vector
    __shared__ int64_t off_of[kReadTokens], soff_of[kReadTokens], goff_of[kFours ? kReadTokens : 1];
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
        [[maybe_unused]] int64_t goff = 0;
        if (lo >= 0 && i < cu[lo + 1]) {
            const int64_t pos = (a.starts ? a.starts[lo] : 0) + (i - cu[lo]);
            if (pos >= 0 && pos < int64_t(a.M) * a.c.ps) {
                const int pi = int(pos) / a.c.ps, at = int(pos) - pi * a.c.ps;
                const int64_t entry = lo * a.tb + pi;
                const int page = SSD_IDX_OK(a.err, entry, a.t_n) ? a.table[entry] : -1;
                if (page >= 0 && page < a.c.pages) {
                    off = page * a.c.sp + at * a.c.st;
                    soff = page * a.c.ssp + at;
                    goff = page * a.c.sgp + at * a.c.sgt;
                }
            }
        }
        off_of[threadIdx.x] = off;
        soff_of[threadIdx.x] = soff;
        if constexpr (kFours) goff_of[threadIdx.x] = goff;
    }
    __syncthreads();
    // A thread keeps its place in a token (head, vector) and takes every `apart`-th token;
    // where a token has more vectors than the CTA threads, one place after another.
    const int per = a.c.Hkv * NV, apart = per < 256 ? 256 / per : 1;
    const int tok0 = threadIdx.x / per;
    for (int place = threadIdx.x - tok0 * per; tok0 < apart && place < per; place += 256) {
        const int h = place / NV, vec = place % NV;
        const int64_t in = h * a.c.sh + NB * vec, sin = h * a.c.ssh;
        [[maybe_unused]] const int64_t gin = h * a.c.sgh + vec / 2;
        T *ko = static_cast<T *>(a.k) + i0 * a.k_st + h * a.k_sh + 8 * vec;
        T *vo = static_cast<T *>(a.v) + i0 * a.v_st + h * a.v_sh + 8 * vec;
        for (int tok = tok0; tok < n; tok += apart * kReadAhead) {
            Raw8<P> kx[kReadAhead], vx[kReadAhead];
            float ks[kReadAhead], vs[kReadAhead];
            [[maybe_unused]] uint8_t kg[kReadAhead], vg[kReadAhead];
#pragma unroll
            for (int u = 0; u < kReadAhead; ++u) {
                const int i = min(tok + u * apart, n - 1);
                const int64_t off = off_of[i] + in;
                ks[u] = vs[u] = 0.f;
                if constexpr (kFours) kg[u] = vg[u] = 0;
                if (off_of[i] >= 0 && SSD_IDX_OK(a.err, off + NB - 1, a.c.n)) {
                    kx[u].load(static_cast<const Byte *>(a.c.k) + off);
                    vx[u].load(static_cast<const Byte *>(a.c.v) + off);
                    if constexpr (kFours) {
                        if (SSD_IDX_OK(a.err, goff_of[i] + gin, a.c.ng)) {
                            kg[u] = a.c.kg[goff_of[i] + gin];
                            vg[u] = a.c.vg[goff_of[i] + gin];
                        }
                    }
                    if constexpr (kCodes) {
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
                if constexpr (kCodes) {
                    float k[8], v[8];
                    kx[u].get(k);
                    vx[u].get(v);
                    if constexpr (kFours) {
                        const float kf = from_e4m3(kg[u]), vf = from_e4m3(vg[u]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            k[j] *= kf;
                            v[j] *= vf;
                        }
                    }
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
    // (4-bit codes, whose vectors are half the bytes: 2048, and five CTAs an SM; 32768 tokens of 8 heads of 128
    // 36.6 us with 1024 and four, 32.8 so, 78% of the copy rate; 262144 of them 258 and 225, 91%; rows of fp32,
    // where five CTAs spill 36 bytes: 75.8 and 509 us, with four 73.6 and 524)
    int TB = (std::is_same_v<P, Nibbles> ? 2048 : 1024) / (a.c.Hkv * (D / 8));
    TB = TB < 1 ? 1 : TB > kReadTokens ? kReadTokens : TB;
    while (TB > 1 && (a.T + TB - 1) / TB < kSms) TB /= 2;
    const int64_t blocks = (a.T + TB - 1) / TB;
    k_kv_read<T, P, D><<<unsigned(blocks), 256, 0, s>>>(a, TB);
    return cudaGetLastError();
}

template <typename P>
cudaError_t read_codes(const KvReadArgs &a, cudaStream_t s) {
    if (a.odt == DT_F32)
        return a.c.D == 64 ? read_t<float, P, 64>(a, s) : read_t<float, P, 128>(a, s);
    return a.c.D == 64 ? read_t<__nv_bfloat16, P, 64>(a, s) : read_t<__nv_bfloat16, P, 128>(a, s);
}

}  // namespace
}  // namespace ssd
