// Attention of new tokens over the paged key/value cache (ssd_paged_attention).
//
//   out = softmax(scale q K^T over the positions a row sees) V
//
// in one pass over the keys with a running maximum m and sum l: a new score s
// gives m' = max(m, s), and what was accumulated is scaled by 2^(m - m')
// (scores carry log2(e), so every exponential is one exp2).
#include "ssd_attn.h"
#include "ssd_debug.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#define SSD_DBG_FILE 8u   // kDbgAttn

namespace ssd {
namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__nv_fp8_e4m3 v) { return float(v); }

// grid (Hq, T, B): one row to a CTA of four warps, each warp every fourth
// position, each lane D/32 places of the head.
template <typename T, typename P, int D>
__global__ void __launch_bounds__(128) k_paged_rows(const PagedArgs a) {
    constexpr int E = D / 32;
    __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
    const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int hk = h / (a.Hq / a.c.Hkv);
    const T *q = static_cast<const T *>(a.q) + b * a.q_sb + t * a.q_st + h * a.q_sh + lane * E;
    float qv[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) qv[i] = to_f(q[i]) * (a.scale * 1.4426950408889634f);
    int64_t end = int64_t(a.lens[b]) - a.T + t + 1;
    const int64_t lo = a.window > 0 && end > a.window ? end - a.window : 0;
    if (end > int64_t(a.M) * a.c.ps) end = int64_t(a.M) * a.c.ps;
    for (int64_t j = lo + warp; j < end; j += 4) {
        const int pi = int(j / a.c.ps), at = int(j - int64_t(pi) * a.c.ps);
        const int page = a.table[b * a.tb + pi];
        if (page < 0 || page >= a.c.pages) continue;
        const int64_t off = page * a.c.sp + hk * a.c.sh + at * a.c.st + lane * E;
        if (!SSD_IDX_OK(a.err, off + E - 1, a.c.n)) continue;
        float ks = 1.f, vs = 1.f;
        if (a.c.ks) {
            ks = a.c.ks[page * a.c.ssp + hk * a.c.ssh + at];
            vs = a.c.vs[page * a.c.ssp + hk * a.c.ssh + at];
        }
        const P *k = static_cast<const P *>(a.c.k) + off, *v = static_cast<const P *>(a.c.v) + off;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(qv[i], to_f(k[i]), s);
#pragma unroll
        for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(~0u, s, w);
        s *= ks;
        const float m2 = fmaxf(m, s);
        const float base = m2 == -INFINITY ? 0.f : m2;
        const float c = exp2f(m - base), p = exp2f(s - base);
        m = m2;
        l = l * c + p;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = fmaf(o[i], c, p * vs * to_f(v[i]));
    }
    if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
    for (int i = 0; i < E; ++i) sm_o[warp][lane * E + i] = o[i];
    __syncthreads();
    if (warp) return;
    float mt = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3])), lt = 0.f, ot[E] = {};
    for (int w = 0; w < 4; ++w) {
        const float f = exp2f(sm_m[w] - (mt == -INFINITY ? 0.f : mt));
        lt = fmaf(sm_l[w], f, lt);
#pragma unroll
        for (int i = 0; i < E; ++i) ot[i] = fmaf(sm_o[w][lane * E + i], f, ot[i]);
    }
    T *out = static_cast<T *>(a.out) + b * a.o_sb + t * a.o_st + h * a.o_sh + lane * E;
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
    for (int i = 0; i < E; ++i) out[i] = T(ot[i] * inv);
    if (a.lse && lane == 0)
        a.lse[(int64_t(b) * a.T + t) * a.Hq + h] =
            lt == 0.f ? -INFINITY : (mt + log2f(lt)) * 0.6931471805599453f;
}

template <int D>
void launch_d(const PagedArgs &a, cudaStream_t s) {
    const dim3 grid(unsigned(a.Hq), unsigned(a.T), unsigned(a.B));
    if (a.c.dt == DT_F32)
        k_paged_rows<float, float, D><<<grid, 128, 0, s>>>(a);
    else if (a.c.dt == DT_BF16)
        k_paged_rows<__nv_bfloat16, __nv_bfloat16, D><<<grid, 128, 0, s>>>(a);
    else
        k_paged_rows<__nv_bfloat16, __nv_fp8_e4m3, D><<<grid, 128, 0, s>>>(a);
}

}  // namespace

size_t paged_workspace(const PagedArgs &) { return 0; }

cudaError_t launch_paged(const PagedArgs &in, cudaStream_t s) {
    PagedArgs a = in;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    if (a.c.D == 64) launch_d<64>(a, s); else launch_d<128>(a, s);
    return cudaGetLastError();
}

}  // namespace ssd
