// Attention of new tokens over the paged key/value cache (ssd_paged_attention).
//
//   out = softmax(scale q K^T over the positions a row sees) V
//
// in one pass over the keys with a running maximum m and sum l: scores s of a
// tile give m' = max(m, s), and what was accumulated is scaled by 2^(m - m')
// (scores carry log2(e), so every exponential is one exp2).  Parts of a
// sequence that different warps or CTAs took join by the same rule.
//
// What bounds it is the cache: each key and value is read once, 2 D elements
// for 4 D flops a query row, and the G = Hq / Hkv query heads of a key/value
// head (times the T new tokens) are the only rows that share them.  So the
// kernels are built to keep reads in flight, not for matrix rate: the two
// products run on mma.sync with 16 rows a warp.  (tcgen05 takes its operands
// from shared or tensor memory, 128 rows at least one way round; here the
// 8-bit keys are widened and the probabilities are made in registers, where
// mma.sync takes them, and at 16 rows it needs about a third of the time that
// the reads take.)
#include "ssd_attn.h"
#include "ssd_debug.cuh"
#include "ssd_tc.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#define SSD_DBG_FILE 8u   // kDbgAttn

namespace ssd {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;                 // of a CTA of the tensor-core kernel
constexpr int kCtasPerSm = 2;
constexpr int kStages = 3;

// ---- the schedule -----------------------------------------------------------------
//
// An item is a (sequence, key/value head, block of rows); its work is its
// tiles of KS positions.  All items' tiles, in that order, form one line that
// is cut into nc equal parts, one to a CTA, wherever the cuts fall: sequences
// of any lengths fill the GPU evenly, and lengths are needed on the device
// only.  An item that a cut falls into is finished by the join kernel from the
// parts that its CTAs leave in the workspace.  An item without positions has
// one (masked) tile, so that somebody writes its rows.

struct Shape {            // of the schedule: what both kernels derive alike
    int KS;               // positions of a tile
    int RB;               // rows of a row block (the rows of a sequence and head: T G)
    int nrb;              // row blocks
    int G;                // query heads to a key/value head
    int ncta;             // most parts of the line
};

struct Item {
    int b, hk, rb;
    int len;              // positions of the sequence, new ones included
    int lo, hi;           // what some row of the block sees (may be empty)
    int first;            // lo rounded down to a tile
    int ntiles;
};

__device__ __forceinline__ void item_range(const PagedArgs &a, const Shape &s, Item &it) {
    const int rows = a.T * s.G;
    const int r0 = it.rb * s.RB, r1 = min(r0 + s.RB, rows) - 1;
    const int e0 = it.len - a.T + r0 / s.G, e1 = it.len - a.T + r1 / s.G;   // rows' own places
    const int cap = a.M * a.c.ps;
    it.hi = min(e1 + 1, cap);
    it.lo = a.window > 0 ? min(max(0, e0 + 1 - int(a.window)), cap) : 0;
    it.first = it.lo / s.KS * s.KS;
    it.ntiles = max(1, (it.hi - it.first + s.KS - 1) / s.KS);
}

__device__ __forceinline__ int64_t seq_tiles(const PagedArgs &a, const Shape &s, int b) {
    Item it;
    it.len = max(a.lens[b], 0);
    int64_t n = 0;
    for (it.rb = 0; it.rb < s.nrb; ++it.rb) {
        item_range(a, s, it);
        n += it.ntiles;
    }
    return n * a.c.Hkv;
}

// Block-wide (128 threads): the inclusive prefix of w over the threads, and
// the block's sum.
__device__ __forceinline__ int64_t block_scan(int64_t w, int64_t *sums, int64_t &total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(~0u, w, o);
        if (lane >= o) w += v;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = w;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i < warp) before += sums[i];
        total += sums[i];
    }
    return w + before;
}

struct Line {
    int64_t total;
    int nc;
    __device__ __forceinline__ int64_t start(int c) const { return total * c / nc; }
};

// Where a position of the line lies; all 128 threads call it and get the same.
struct Finder {
    int64_t sums[4];
    int b;
    int64_t off;

    // The line's length (every sequence's tiles added up).
    __device__ int64_t total(const PagedArgs &a, const Shape &s) {
        int64_t w = 0, t;
        for (int i = threadIdx.x; i < a.B; i += 128) w += seq_tiles(a, s, i);
        block_scan(w, sums, t);
        return t;
    }
    // The item that holds tile `at` of the line, and the tile's number in it.
    __device__ int find(const PagedArgs &a, const Shape &s, int64_t at, Item &it) {
        int64_t run = 0;
        for (int base = 0; base < a.B && run <= at; base += 128) {
            const int i = base + threadIdx.x;
            const int64_t w = i < a.B ? seq_tiles(a, s, i) : 0;
            int64_t sum;
            const int64_t upto = run + block_scan(w, sums, sum);
            if (at < upto && at >= upto - w) {
                b = i;
                off = at - (upto - w);
            }
            run += sum;
        }
        __syncthreads();
        it.b = b;
        it.len = max(a.lens[it.b], 0);
        const int64_t per = seq_tiles(a, s, it.b) / a.c.Hkv;
        it.hk = int(off / per);
        int64_t left = off - it.hk * per;
        for (it.rb = 0;; ++it.rb) {
            item_range(a, s, it);
            if (left < it.ntiles) return int(left);
            left -= it.ntiles;
        }
    }
};

__device__ __forceinline__ Line make_line(int64_t total, int ncta) {
    return Line{total, int(total < ncta ? total : ncta)};
}

__device__ __forceinline__ void next_item(const PagedArgs &a, const Shape &s, Item &it) {
    if (++it.rb == s.nrb) {
        it.rb = 0;
        if (++it.hk == a.c.Hkv) {
            it.hk = 0;
            ++it.b;
            if (it.b < a.B) it.len = max(a.lens[it.b], 0);
        }
    }
    if (it.b < a.B) item_range(a, s, it);
}

// Partial results of the workspace: part 2 c is the first item of CTA c's
// stretch, part 2 c + 1 its last (if that is another).
__host__ __device__ __forceinline__ size_t part_floats(int RB, int D) {
    return size_t(RB) * (D + 2);
}

// ---- PTX ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 (or 4) bytes to shared memory, zeros if !ok (then src is not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(__cvta_generic_to_global(src)), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst),
                 "l"(__cvta_generic_to_global(src)), "r"(ok ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}
// d += a b, 16 x 8 x 16, fp32 accumulators
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_(float x) {   // 2 ulp, subnormal results flushed
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// two codes -> two fp16 values (exact)
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(codes & 0xffffu), __NV_E4M3);
    return uint32_t(h.x) | (uint32_t(h.y) << 16);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Waits until the kernel before this one on the stream has finished (for a
// launch that may start early) / lets the next one start early.
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---- the tensor-core kernel -----------------------------------------------------------
//
// Four warps, as WK groups of WR: the WR warps of a group take 16 query rows
// each and share the group's positions, the groups take different positions.
// Each warp copies KW positions of a tile itself (its lanes look the pages
// up), kStages - 1 tiles ahead, so with WR = 1 the warps run without waiting
// for one another until an item ends.
template <int D_, bool F8_, int WR_>
struct Cfg {
    static constexpr int D = D_, WR = WR_, WK = kWarps / WR_;
    static constexpr bool F8 = F8_;
    static constexpr int KW = (F8 || D == 64) ? 32 : 16;    // positions a warp copies a tile
    static constexpr int KS = KW * kWarps;                  // positions of a CTA tile
    static constexpr int ROW = D * (F8 ? 1 : 2);            // bytes of a cached row
    static constexpr int PART = KW * ROW;                   // bytes of a warp's keys (or values)
    static constexpr int STAGE = 2 * PART * kWarps;
    static constexpr int SCALES = F8 ? 2 * KW * 4 : 0;      // bytes of a warp's scales
    static constexpr int AUX = kWarps * (SCALES + 4);       // a stage's scales and mask words
    static constexpr int XCH = (WK > 1 ? 16 * D + 32 * WR : 0) * 4;   // exchange of the groups
    static constexpr int SMEM = kStages * (STAGE + AUX) + XCH;
};

// Byte offset of 16-byte chunk c of row r: chunks are exchanged so that the
// eight rows of a matrix fragment, and the rows and chunks that eight
// neighbouring lanes read, lie in different banks.
template <int ROW>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if constexpr (ROW == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return r * ROW + ((c ^ (r & 7)) << 4);
}

// With codes, which of a group of 16 positions stands in column n of score
// tile j (0 or 1).  Any order does, as long as keys and values follow the same
// one; this one keeps both kinds of reads free of bank conflicts.
template <int ROW>
__device__ __forceinline__ int code_pos(int j, int n) {
    const int c = n >> 1, odd = n & 1;
    if constexpr (ROW == 64) {
        const int even_at = (c & 1) | ((c & 2) << 1);           // 0 1 4 5
        return 8 * j + (odd ? (even_at ^ 3) : even_at);         // 3 2 7 6
    }
    return j + (odd ? 8 + ((2 * c) ^ 4) : 2 * c);
}

template <int D, bool F8, int WR>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
k_paged_mma(const PagedArgs a, const Shape s) {
    using C = Cfg<D, F8, WR>;
    constexpr int KW = C::KW, KS = C::KS, ROW = C::ROW, WK = C::WK;
    constexpr int NT = KW / 8;            // score tiles of a warp's positions
    constexpr int ND = D / 8;             // output tiles
    constexpr int LPR = ROW / 16;         // lanes that copy a row
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Finder finder;

    let_next_start();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int kg = warp / WR, wr = warp % WR;     // key group, row warp
    const int g = lane >> 2, c = lane & 3;        // fragment row and column pair

    const Line line = make_line(finder.total(a, s), s.ncta);
    if (int(blockIdx.x) >= line.nc) return;
    const int64_t beg = line.start(blockIdx.x), end = line.start(blockIdx.x + 1);
    const int cnt = int(end - beg);
    Item it;
    int tile = finder.find(a, s, beg, it);
    Item ld = it;                                 // runs ahead: the tile to be copied next
    int ld_tile = tile, issued = 0;

    unsigned char *aux = smem + kStages * C::STAGE;
    float *xch = reinterpret_cast<float *>(aux + kStages * C::AUX);
    auto stage_at = [&](int st, int w) { return smem_addr(smem) + st * C::STAGE + w * 2 * C::PART; };
    auto scale_at = [&](int st, int w) {
        return reinterpret_cast<float *>(aux + st * C::AUX + w * C::SCALES);
    };
    auto mask_at = [&](int st, int w) {
        return reinterpret_cast<uint32_t *>(aux + st * C::AUX + kWarps * C::SCALES) + w;
    };

    // the page of this lane's position of the tile at ld (looked up a tile early)
    int pos = 0, page = -1;
    auto look_up = [&]() {
        page = -1;
        if (issued >= cnt) return;
        pos = ld.first + ld_tile * KS + warp * KW + lane;
        if (lane < KW && pos >= ld.lo && pos < ld.hi) page = a.table[ld.b * a.tb + pos / a.c.ps];
    };
    auto issue = [&](int st) {
        if (issued < cnt) {
            const bool ok = page >= 0 && page < a.c.pages;
            const uint32_t mask = __ballot_sync(~0u, ok);
            const int at = pos % a.c.ps;
            const int64_t off = ok ? page * a.c.sp + ld.hk * a.c.sh + at * a.c.st : 0;
            const uint32_t kdst = stage_at(st, warp), vdst = kdst + C::PART;
            if constexpr (F8) {
                const int64_t so = ok ? page * a.c.ssp + ld.hk * a.c.ssh + at : 0;
                const uint32_t sd = smem_addr(scale_at(st, warp)) + lane * 4;
                copy4(sd, a.c.ks + so, ok);
                copy4(sd + KW * 4, a.c.vs + so, ok);
            }
#pragma unroll
            for (int i = 0; i < KW * LPR / 32; ++i) {
                const int r = i * (32 / LPR) + lane / LPR, ch = lane % LPR;
                const int64_t o = (__shfl_sync(~0u, off, r)) * (F8 ? 1 : 2) + ch * 16;
                const bool rok = (mask >> r) & 1 &&
                                 SSD_IDX_OK(a.err, o + 15, a.c.n * (F8 ? 1 : 2));
                copy16(kdst + chunk_at<ROW>(r, ch), static_cast<const char *>(a.c.k) + o, rok);
                copy16(vdst + chunk_at<ROW>(r, ch), static_cast<const char *>(a.c.v) + o, rok);
            }
            if (lane == 0) *mask_at(st, warp) = mask;
            ++issued;
            if (++ld_tile == ld.ntiles) {
                ld_tile = 0;
                next_item(a, s, ld);
            }
            look_up();
        }
        copy_commit();       // an empty group where nothing is left, so that the count goes on
    };
    auto group_sync = [&]() {
        if constexpr (WR == 1) __syncwarp();
        else if constexpr (WR == kWarps) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + kg), "n"(32 * WR) : "memory");
    };

    look_up();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // Per item: the query fragments, the running maximum and sum of the rows
    // g and g + 8 (the sum over this thread's columns), and the output.
    uint32_t qf[D / 16][4];
    float o[ND][4], m[2], l[2], qs[2];
    float xs = 0.f, xmax = 0.f;           // codes: the values' common factor (a power of two)
    int e[2];                             // the rows' own places
    bool fresh = true;
    const int tile_first = tile;          // of the first item; later ones begin at 0
    bool first_item = true;

    for (int n = 0, st = 0; n < cnt; ++n, st = st + 1 == kStages ? 0 : st + 1) {
        if (fresh) {
            fresh = false;
            const int rows = a.T * s.G;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = it.rb * s.RB + wr * 16 + g + 8 * i;
                const int t = min(r, rows - 1) / s.G;
                e[i] = it.len - a.T + t;
                m[i] = -INFINITY;
                l[i] = 0.f;
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) +
                                         it.b * a.q_sb + t * a.q_st +
                                         (it.hk * s.G + min(r, rows - 1) - t * s.G) * a.q_sh;
                if constexpr (!F8) {
                    qs[i] = a.scale * kLog2e;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        qf[k][i] = *reinterpret_cast<const uint32_t *>(q + 16 * k + 2 * c);
                        qf[k][i + 2] = *reinterpret_cast<const uint32_t *>(q + 16 * k + 8 + 2 * c);
                    }
                } else {
                    // fp16 for the product with widened codes: the row is scaled by a
                    // power of two that brings its largest value to [1, 2), so all but
                    // values 2^-14 times as large stay exact
                    float top = 0.f;
                    uint2 raw[D / 16];
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {   // places 64 h + 16 c + 4 (k % 4)
                        raw[k] = *reinterpret_cast<const uint2 *>(q + (k / 4) * 64 + 16 * c +
                                                                  4 * (k % 4));
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const uint32_t u = w ? raw[k].y : raw[k].x;
                            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u << 16)),
                                                   fabsf(__uint_as_float(u & 0xffff0000u))));
                        }
                    }
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    uint32_t ex = __float_as_uint(top) & 0x7f800000u;
                    ex = ex == 0 || ex > 0x7e800000u ? 0x3f800000u : ex;
                    const float down = __uint_as_float(0x7f000000u - ex);
                    qs[i] = a.scale * kLog2e * __uint_as_float(ex);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        qf[k][i] = pack_f16(__uint_as_float(raw[k].x << 16) * down,
                                            __uint_as_float(raw[k].x & 0xffff0000u) * down);
                        qf[k][i + 2] = pack_f16(__uint_as_float(raw[k].y << 16) * down,
                                                __uint_as_float(raw[k].y & 0xffff0000u) * down);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < ND; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
            if constexpr (F8) xs = xmax = 0.f;
        }
        copy_wait<kStages - 2>();
        group_sync();        // the group's copies are there, and its last tile is done with
        issue(st == 0 ? kStages - 1 : st - 1);

        const int kbase = it.first + tile * KS + kg * WR * KW;
        const int rows = a.T * s.G;
        const int emin = it.len - a.T + (it.rb * s.RB) / s.G;
        const int emax = it.len - a.T + (min(it.rb * s.RB + s.RB, rows) - 1) / s.G;
#pragma unroll 1
        for (int sub = 0; sub < WR; ++sub) {
            const int w = kg * WR + sub;
            const uint32_t mask = *mask_at(st, w);
            if (mask == 0) continue;
            const int k0 = kbase + sub * KW;
            const uint32_t ksm = stage_at(st, w), vsm = ksm + C::PART;
            const float *ksc = scale_at(st, w), *vsc = ksc + KW;

            // scores: 16 rows x KW positions
            float sc[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
            if constexpr (!F8) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int j = 0; j < NT; j += 2) {
                        uint32_t b[4];
                        ldsm4(b, ksm + chunk_at<ROW>(8 * j + (lane >> 4) * 8 + (lane & 7),
                                                     2 * k + ((lane >> 3) & 1)));
                        mma<false>(sc[j], qf[k], b[0], b[1]);
                        mma<false>(sc[j + 1], qf[k], b[2], b[3]);
                    }
            } else {
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const int r = (j / 2) * 16 + code_pos<ROW>(j & 1, g);
                        const uint4 u = lds16(ksm + chunk_at<ROW>(r, 4 * h + c));
                        const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma<true>(sc[j], qf[4 * h + k], widen2(v[k]), widen2(v[k] >> 16));
                    }
            }

            // scale, mask, running maximum.  vis[i]: bit 2 j + p, row i sees
            // position p of tile j's pair
            const bool partial = k0 + KW - 1 > emin || (a.window > 0 && k0 <= emax - int(a.window));
            float mn[2] = {m[0], m[1]};
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const int x = F8 ? (j / 2) * 16 + code_pos<ROW>(j & 1, 2 * c + p) : 8 * j + 2 * c + p;
                    const float f = F8 ? ksc[x] : 1.f;
                    const bool there = (mask >> x) & 1;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        bool see = there;
                        if (partial) {
                            see = see && k0 + x <= e[i];
                            if (a.window > 0) see = see && k0 + x > e[i] - int(a.window);
                        }
                        float &v = sc[j][2 * i + p];
                        v = see ? v * (F8 ? qs[i] * f : qs[i]) : -INFINITY;
                        mn[i] = fmaxf(mn[i], v);
                    }
                }
            float cor[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mn[i] = fmaxf(mn[i], __shfl_xor_sync(~0u, mn[i], 1));
                mn[i] = fmaxf(mn[i], __shfl_xor_sync(~0u, mn[i], 2));
            }
            bool moved = mn[0] != m[0] || mn[1] != m[1];
            float grow = 1.f;
            if constexpr (F8) {
                // the values' factor must cover this tile's largest finite scale
                const float vs = lane < KW && (mask >> lane) & 1 ? vsc[lane] : 0.f;
                const bool more = vs > xmax && vs < INFINITY;
                if (__any_sync(~0u, more)) {
                    float top = more ? vs : 0.f;
#pragma unroll
                    for (int q = 16; q; q >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, q));
                    // xmax: a power of two of at least top, at most 2^126
                    uint32_t ex = (__float_as_uint(top) + 0x7fffffu) & 0x7f800000u;
                    ex = min(max(ex, 0x01000000u), 0x7e800000u);
                    const float was = xmax;
                    xmax = __uint_as_float(ex);
                    // probability times scale goes to fp16 as p vs 2^14 / xmax <= 2^14
                    xs = __uint_as_float(0x7f000000u - ex);
                    grow = was * xs;      // 0 on the first tile, where o is 0
                    moved = true;
                }
            }
            float base[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                base[i] = mn[i] == -INFINITY ? 0.f : mn[i];
                cor[i] = exp2_(m[i] - base[i]);
                m[i] = mn[i];
            }
            if (__any_sync(~0u, moved)) {
                l[0] *= cor[0];
                l[1] *= cor[1];
                const float c0 = cor[0] * grow, c1 = cor[1] * grow;
#pragma unroll
                for (int j = 0; j < ND; ++j) {
                    o[j][0] *= c0;
                    o[j][1] *= c0;
                    o[j][2] *= c1;
                    o[j][3] *= c1;
                }
            }
            // probabilities (unnormalised, at most 1), summed in fp32 and rounded to
            // 16 bits as the left operand of the second product
            uint32_t pf[NT / 2][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float p0 = exp2_(sc[j][2 * i] - base[i]), p1 = exp2_(sc[j][2 * i + 1] - base[i]);
                    l[i] += p0 + p1;
                    if constexpr (F8) {
                        const int x0 = (j / 2) * 16 + code_pos<ROW>(j & 1, 2 * c);
                        const int x1 = (j / 2) * 16 + code_pos<ROW>(j & 1, 2 * c + 1);
                        // what the row does not see stays 0 whatever its scale is
                        p0 = p0 == 0.f ? 0.f : p0 * (vsc[x0] * xs * 16384.f);
                        p1 = p1 == 0.f ? 0.f : p1 * (vsc[x1] * xs * 16384.f);
                        pf[j / 2][(j & 1) * 2 + i] = pack_f16(p0, p1);
                    } else {
                        pf[j / 2][(j & 1) * 2 + i] = pack_bf16(p0, p1);
                    }
                }

            // Values.  pv(no, 0): all rows at once.  pv(yes, r): row r alone, with the
            // values that it does not see taken out.
            auto pv = [&](auto by_row, int row) {
                constexpr bool kByRow = decltype(by_row)::value;
                const int re = kByRow ? __shfl_sync(~0u, row < 8 ? e[0] : e[1], (row & 7) * 4) : 0;
                auto keep = [&](int x) {     // position x: all bits where the row sees it
                    const bool see = k0 + x <= re && (a.window == 0 || k0 + x > re - int(a.window));
                    return see ? 0xffffu : 0u;
                };
#pragma unroll
                for (int k = 0; k < NT / 2; ++k) {
                    uint32_t pr[4], keep0 = 0, keep1 = 0;
                    if constexpr (kByRow) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            pr[x] = g + 8 * (x & 1) == row ? pf[k][x] : 0u;
                        const int y = 16 * k;
                        auto at = [&](int j, int n) { return y + (F8 ? code_pos<ROW>(j, n) : 8 * j + n); };
                        keep0 = keep(at(0, 2 * c)) | keep(at(0, 2 * c + 1)) << 16;
                        keep1 = keep(at(1, 2 * c)) | keep(at(1, 2 * c + 1)) << 16;
                    }
                    auto add = [&](float (&d)[4], uint32_t b0, uint32_t b1) {
                        if constexpr (kByRow) {
                            float t[4] = {0.f, 0.f, 0.f, 0.f};
                            mma<F8>(t, pr, b0 & keep0, b1 & keep1);
                            if (g == (row & 7)) {
                                if (row < 8) d[0] += t[0], d[1] += t[1];
                                else d[2] += t[2], d[3] += t[3];
                            }
                        } else {
                            mma<F8>(d, pf[k], b0, b1);
                        }
                    };
                    if constexpr (!F8) {
#pragma unroll
                        for (int j = 0; j < ND; j += 2) {
                            uint32_t b[4];
                            ldsm4_trans(b, vsm + chunk_at<ROW>(16 * k + (lane & 15), j + (lane >> 4)));
                            add(o[j], b[0], b[1]);
                            add(o[j + 1], b[2], b[3]);
                        }
                    } else {
                        // four positions' codes for the D / 8 places from (D / 8) g on;
                        // place j of them is column g of output tile j
                        constexpr int NW = D / 32;     // words of a position
                        uint32_t v[4][NW];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int r = 16 * k + code_pos<ROW>(x >> 1, 2 * c + (x & 1));
                            if constexpr (D == 128) {
                                const uint4 u = lds16(vsm + chunk_at<ROW>(r, g));
                                v[x][0] = u.x, v[x][1] = u.y, v[x][2] = u.z, v[x][3] = u.w;
                            } else {
                                const uint2 u = lds8(vsm + chunk_at<ROW>(r, g >> 1) + (g & 1) * 8);
                                v[x][0] = u.x, v[x][1] = u.y;
                            }
                        }
#pragma unroll
                        for (int q = 0; q < NW; ++q) {
                            // bytes of two positions side by side, place by place
                            const uint32_t a0 = __byte_perm(v[0][q], v[1][q], 0x5140);
                            const uint32_t a1 = __byte_perm(v[0][q], v[1][q], 0x7362);
                            const uint32_t b0 = __byte_perm(v[2][q], v[3][q], 0x5140);
                            const uint32_t b1 = __byte_perm(v[2][q], v[3][q], 0x7362);
                            add(o[4 * q], widen2(a0), widen2(b0));
                            add(o[4 * q + 1], widen2(a0 >> 16), widen2(b0 >> 16));
                            add(o[4 * q + 2], widen2(a1), widen2(b1));
                            add(o[4 * q + 3], widen2(a1 >> 16), widen2(b1 >> 16));
                        }
                    }
                }
            };
            // Where rows of one warp see different positions, an infinity or NaN that one
            // row does not see must not meet its zero probability in the product: such a
            // tile (the values are looked through first) is taken row by row.
            bool foul = false;
            if (partial) {
#pragma unroll
                for (int x = 0; x < C::PART / 512; ++x) {
                    const uint4 u = lds16(vsm + (x * 32 + lane) * 16);
                    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        foul |= F8 ? (((v[y] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0
                                   : (v[y] & 0x7f80u) == 0x7f80u || (v[y] & 0x7f800000u) == 0x7f800000u;
                }
            }
            if (__any_sync(~0u, foul)) {
#pragma unroll 1
                for (int row = 0; row < 16; ++row) pv(std::true_type{}, row);
            } else {
                pv(std::false_type{}, 0);
            }
        }

        // the item's last tile, or the stretch's: join the groups, write
        if (tile + 1 == it.ntiles || n + 1 == cnt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[i] += __shfl_xor_sync(~0u, l[i], 1);
                l[i] += __shfl_xor_sync(~0u, l[i], 2);
            }
            if constexpr (F8) {
                const float back = xmax * (1.f / 16384.f);
#pragma unroll
                for (int j = 0; j < ND; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[j][i] *= back;
            }
            if constexpr (WK > 1) {
                // the groups' results one after another (in a fixed order), 16 D
                // floats at a time, a lane's values 32 floats apart
                float *ml = xch + 16 * D;
#pragma unroll
                for (int src = 1; src < WK; ++src) {
                    float f0[2], f1[2];
#pragma unroll
                    for (int part = 0; part < WR; ++part) {
                        constexpr int NP = ND / WR;
                        float *buf = xch + wr * (16 * D / WR);
                        __syncthreads();
                        if (kg == src) {
#pragma unroll
                            for (int j = 0; j < NP; ++j)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    buf[(j * 4 + i) * 32 + lane] = o[part * NP + j][i];
                            if (part == 0 && c == 0) {
                                ml[wr * 32 + g] = m[0];
                                ml[wr * 32 + g + 8] = m[1];
                                ml[wr * 32 + 16 + g] = l[0];
                                ml[wr * 32 + 24 + g] = l[1];
                            }
                        }
                        __syncthreads();
                        if (kg == 0) {
                            if (part == 0) {
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const float m1 = ml[wr * 32 + g + 8 * i];
                                    const float mt = fmaxf(m[i], m1);
                                    const float bs = mt == -INFINITY ? 0.f : mt;
                                    f0[i] = exp2_(m[i] - bs);
                                    f1[i] = exp2_(m1 - bs);
                                    m[i] = mt;
                                    l[i] = l[i] * f0[i] + ml[wr * 32 + 16 + g + 8 * i] * f1[i];
                                }
                            }
#pragma unroll
                            for (int j = 0; j < NP; ++j)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    float &v = o[part * NP + j][i];
                                    v = v * f0[i >> 1] + buf[(j * 4 + i) * 32 + lane] * f1[i >> 1];
                                }
                        }
                    }
                }
            }
            if (kg == 0) {
                const bool whole = tile + 1 == it.ntiles && (first_item ? tile_first == 0 : true);
                float *part = reinterpret_cast<float *>(a.ws) +
                              size_t(2 * blockIdx.x + (first_item ? 0 : 1)) * part_floats(s.RB, D);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int rr = wr * 16 + g + 8 * i, r = it.rb * s.RB + rr;
                    if (r >= rows) continue;
                    // this thread's places: pairs 8 j + 2 c, or with codes the D / 4
                    // places from (D / 4) c on
                    if (!whole) {
                        float *dst = part + rr * D;
                        if constexpr (!F8) {
#pragma unroll
                            for (int j = 0; j < ND; ++j)
                                *reinterpret_cast<float2 *>(dst + 8 * j + 2 * c) =
                                    make_float2(o[j][2 * i], o[j][2 * i + 1]);
                        } else {
#pragma unroll
                            for (int p = 0; p < 2; ++p)
#pragma unroll
                                for (int j = 0; j < ND; j += 4)
                                    *reinterpret_cast<float4 *>(dst + ND * (2 * c + p) + j) =
                                        make_float4(o[j][2 * i + p], o[j + 1][2 * i + p],
                                                    o[j + 2][2 * i + p], o[j + 3][2 * i + p]);
                        }
                        if (c == 0) {
                            part[s.RB * D + rr] = m[i];
                            part[s.RB * (D + 1) + rr] = l[i];
                        }
                        continue;
                    }
                    const int t = r / s.G, h = it.hk * s.G + r - t * s.G;
                    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + it.b * a.o_sb +
                                         t * a.o_st + h * a.o_sh;
                    if constexpr (!F8) {
#pragma unroll
                        for (int j = 0; j < ND; ++j)
                            *reinterpret_cast<uint32_t *>(dst + 8 * j + 2 * c) =
                                pack_bf16(o[j][2 * i] * inv, o[j][2 * i + 1] * inv);
                    } else {
#pragma unroll
                        for (int p = 0; p < 2; ++p)
#pragma unroll
                            for (int j = 0; j < ND; j += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    w[q] = pack_bf16(o[j + 2 * q][2 * i + p] * inv,
                                                     o[j + 2 * q + 1][2 * i + p] * inv);
                                *reinterpret_cast<uint4 *>(dst + ND * (2 * c + p) + j) =
                                    make_uint4(w[0], w[1], w[2], w[3]);
                            }
                    }
                    if (a.lse && c == 0)
                        a.lse[(int64_t(it.b) * a.T + t) * a.Hq + h] =
                            l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
                }
            }
        }
        if (++tile == it.ntiles) {
            tile = 0;
            first_item = false;
            fresh = true;
            next_item(a, s, it);
        }
    }
    copy_wait<0>();
}

// ---- the join -------------------------------------------------------------------------
//
// CTA (x, y): rows 4 y.. of the item that the cut between CTAs x and x + 1
// falls into, if it is that item's first cut; a warp a row.
template <typename T, int D>
__global__ void __launch_bounds__(128) k_paged_join(const PagedArgs a, const Shape s) {
    __shared__ Finder finder;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int x = blockIdx.x;
    const Line line = make_line(finder.total(a, s), s.ncta);
    if (x + 1 >= line.nc) return;
    const int64_t cut = line.start(x + 1);
    Item it;
    const int64_t t0 = cut - finder.find(a, s, cut, it), t1 = t0 + it.ntiles;
    if (t0 == cut || line.start(x) > t0) return;     // no item is cut here, or not first
    const int rr = blockIdx.y * 4 + warp, r = it.rb * s.RB + rr;
    if (rr >= s.RB || r >= a.T * s.G) return;

    constexpr int E = D / 32;
    wait_for_previous();
    const float *parts = reinterpret_cast<const float *>(a.ws);
    float m = -INFINITY, l = 0.f, o[E] = {};
    for (int c0 = x; c0 < line.nc && line.start(c0) < t1; c0 += 32) {
        // up to 32 parts: lane i weighs part c0 + i
        const int n = min(32, line.nc - c0), cc = c0 + lane;
        float pm = -INFINITY, pl = 0.f;
        const bool there = lane < n && line.start(cc) < t1;
        const float *part = parts + size_t(2 * cc + (line.start(cc) < t0 ? 1 : 0)) * part_floats(s.RB, D);
        if (there) {
            pm = part[s.RB * D + rr];
            pl = part[s.RB * (D + 1) + rr];
        }
        float mt = fmaxf(m, pm);
#pragma unroll
        for (int w = 16; w; w >>= 1) mt = fmaxf(mt, __shfl_xor_sync(~0u, mt, w));
        const float base = mt == -INFINITY ? 0.f : mt;
        const float f = exp2_(pm - base), old = exp2_(m - base);
        m = mt;
        float sum = pl * f;
#pragma unroll
        for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
        l = l * old + sum;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] *= old;
        const int k = __popc(__ballot_sync(~0u, there));
#pragma unroll 4
        for (int i = 0; i < k; ++i) {
            const float w = __shfl_sync(~0u, f, i);
            const float *src = parts + size_t(2 * (c0 + i) + (line.start(c0 + i) < t0 ? 1 : 0)) *
                                           part_floats(s.RB, D) + rr * D + lane * E;
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] = fmaf(src[j], w, o[j]);
        }
    }
    const int t = r / s.G, h = it.hk * s.G + r - t * s.G;
    T *dst = static_cast<T *>(a.out) + it.b * a.o_sb + t * a.o_st + h * a.o_sh + lane * E;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int j = 0; j < E; ++j) dst[j] = T(o[j] * inv);
    if (a.lse && lane == 0)
        a.lse[(int64_t(it.b) * a.T + t) * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---- fp32 -------------------------------------------------------------------------------
//
// grid (Hq, T, B): one row to a CTA of four warps, each warp every fourth
// position, each lane D / 32 places of the head.
template <int D>
__global__ void __launch_bounds__(128) k_paged_rows(const PagedArgs a) {
    constexpr int E = D / 32;
    __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
    const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int hk = h / (a.Hq / a.c.Hkv);
    const float *q = static_cast<const float *>(a.q) + b * a.q_sb + t * a.q_st + h * a.q_sh + lane * E;
    float qv[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) qv[i] = q[i] * (a.scale * kLog2e);
    int64_t end = int64_t(a.lens[b]) - a.T + t + 1;
    const int64_t lo = a.window > 0 && end > a.window ? end - a.window : 0;
    if (end > int64_t(a.M) * a.c.ps) end = int64_t(a.M) * a.c.ps;
    for (int64_t j = lo + warp; j < end; j += 4) {
        const int pi = int(j / a.c.ps), at = int(j - int64_t(pi) * a.c.ps);
        const int page = a.table[b * a.tb + pi];
        if (page < 0 || page >= a.c.pages) continue;
        const int64_t off = page * a.c.sp + hk * a.c.sh + at * a.c.st + lane * E;
        if (!SSD_IDX_OK(a.err, off + E - 1, a.c.n)) continue;
        const float *k = static_cast<const float *>(a.c.k) + off, *v = static_cast<const float *>(a.c.v) + off;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(qv[i], k[i], s);
#pragma unroll
        for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(~0u, s, w);
        const float m2 = fmaxf(m, s);
        const float base = m2 == -INFINITY ? 0.f : m2;
        const float f = exp2f(m - base), p = exp2f(s - base);
        m = m2;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = fmaf(o[i], f, p * v[i]);
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
    float *out = static_cast<float *>(a.out) + b * a.o_sb + t * a.o_st + h * a.o_sh + lane * E;
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
    for (int i = 0; i < E; ++i) out[i] = ot[i] * inv;
    if (a.lse && lane == 0)
        a.lse[(int64_t(b) * a.T + t) * a.Hq + h] =
            lt == 0.f ? -INFINITY : (mt + log2f(lt)) * kLn2;
}

// ---- launches -----------------------------------------------------------------------------

// More than 48 KB of dynamic shared memory needs the kernel's consent, once
// for each device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t> (&done)[4]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 256 && (done[dev / 64].load(std::memory_order_acquire) >> (dev % 64)) & 1)
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 256) done[dev / 64].fetch_or(uint64_t(1) << (dev % 64));
    return e;
}

template <int D, bool F8, int WR>
cudaError_t launch_mma(const PagedArgs &a, Shape s, cudaStream_t stream) {
    using C = Cfg<D, F8, WR>;
    static std::atomic<uint64_t> done[4];
    s.KS = C::KS;
    cudaError_t e = allow_smem(k_paged_mma<D, F8, WR>, C::SMEM, done);
    if (e != cudaSuccess) return e;
    k_paged_mma<D, F8, WR><<<s.ncta, kWarps * 32, C::SMEM, stream>>>(a, s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // The join may start while the last parts are being computed; it waits for
    // them before it reads any.
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(unsigned(s.ncta - 1), unsigned((min(s.RB, a.T * s.G) + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_paged_join<__nv_bfloat16, D>, a, s);
}

// Warps along the rows of a key/value head: 16 rows each, the rest of the
// four along the positions.  More rows than 64 are several row blocks, each of
// which reads the cache.
int row_warps(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

Shape make_shape(const PagedArgs &a) {
    Shape s{};
    s.G = a.Hq / a.c.Hkv;
    const int64_t rows = int64_t(a.T) * s.G;
    s.RB = 16 * row_warps(rows);
    s.nrb = int((rows + s.RB - 1) / s.RB);
    s.ncta = device_sm_count() * kCtasPerSm;
    return s;
}

template <int D, bool F8>
cudaError_t launch_rows(const PagedArgs &a, cudaStream_t stream) {
    const Shape s = make_shape(a);
    switch (s.RB) {
    case 16: return launch_mma<D, F8, 1>(a, s, stream);
    case 32: return launch_mma<D, F8, 2>(a, s, stream);
    default: return launch_mma<D, F8, 4>(a, s, stream);
    }
}

template <int D>
cudaError_t launch_d(const PagedArgs &a, cudaStream_t stream) {
    if (a.c.dt == DT_F32) {
        k_paged_rows<D><<<dim3(unsigned(a.Hq), unsigned(a.T), unsigned(a.B)), 128, 0, stream>>>(a);
        return cudaGetLastError();
    }
    return a.c.dt == DT_BF16 ? launch_rows<D, false>(a, stream) : launch_rows<D, true>(a, stream);
}

}  // namespace

size_t paged_workspace(const PagedArgs &a) {
    if (a.c.dt == DT_F32) return 0;
    const Shape s = make_shape(a);
    return size_t(2) * s.ncta * part_floats(s.RB, a.c.D) * sizeof(float);
}

cudaError_t launch_paged(const PagedArgs &in, cudaStream_t s) {
    PagedArgs a = in;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    return a.c.D == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace ssd
