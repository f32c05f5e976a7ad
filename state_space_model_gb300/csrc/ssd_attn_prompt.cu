// Attention of many new tokens over the paged cache (pieces of prompts, bf16 pools): the same
// sum as in ssd_attn.cuh, on the tensor cores' own path.
//
// Rows (the T G queries of a sequence and key/value head, in order of their tokens) stand in the
// 128 lanes of tensor memory, two blocks of 128 to a CTA, which share every tile of 128 cached
// positions:
//
//   S = Q K^T       tcgen05, both operands in shared memory, S in tensor memory (fp32)
//   P = 2^(..)      a thread a row: its scores to registers, the running maximum and sum, P (bf16)
//                   back over S
//   O += P V        tcgen05, P from tensor memory, O in tensor memory (fp32)
//
// What bounds it is the products, 4 D flops a row and position, and the way from one to the next: a
// block's scores, its exponentials and its outputs follow one another, 2900 cycles a tile, 1024 of
// them products.  So a warp issues nothing but products, in the order S0, S1, then for every tile O0,
// S0 (next), O1, S1 (next): while a block's exponentials run, the tensor core has the other's
// products. (All of that warp goes through the loop and one lane issues, so that descriptors stay
// uniform: a single thread's branch took 100 cycles a product instead of 25, 444 us instead of 418 for
// 8192 tokens of 32 over 8 heads; outputs and the next scores issued together, 407; a loop for each
// kind of item, its blocks' code once, so that it stays in the instruction cache, 399: 1376 TFLOP/s.)
// With 256 rows to a tile the reads from L2 are 64 KB for 2 x 4.2 Mflop of them each.  Two warps load
// (TMA), tiles ahead and across items, and the CTA goes from item to item (sequence, head, 256 rows)
// with the next one's queries and keys already there.  Where most SMs would have no item in the last
// round, an item is halved: 128 rows, for which the two blocks take half of every tile each and join
// their sums at the end (512 tokens over 8192: 64 items 104 us, 128 halves 70).
//
// The positions that some row of an item sees, sinks first and then the window's, are counted
// through as one run in boxes of 16 of a page (so pages are multiples of 16; others take the
// kernels of ssd_attn.cuh), so that a tile holds little that nobody needs wherever the window
// begins.  (Copies by three warps, 16 bytes a lane, took any page size and three times as
// long: 253 us for 4096 tokens under a window of 1024 where the loads take 75.)
#include "ptx_sm100.cuh"
#include "ssd_attn.h"
#include "ssd_attn_choice.cuh"
#include "ssd_block_math.cuh"
#include "ssd_debug.cuh"
#include "ssd_f32x2.cuh"
#include "ssd_tc.cuh"
#include "ssd_tmap.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#define SSD_DBG_FILE 9u   // kDbgPrompt

namespace ssd {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 128, kItemRows = 2 * kRows;   // rows of a block, of an item
constexpr int kTile = 128, kPart = kTile / 2;       // positions of a tile, of it for a block of a half item
constexpr int kBox = 16;                             // positions of a load
constexpr int kThreads = 2 * kRows + 32 * 4;         // and a warp that issues, two that load, one that checks
// Registers of a thread: 168 at the launch (65536 / 384), shared out as 208 for the rows'
// threads and 88 for the others: 256 x 208 + 128 x 88 = 384 x 168.
constexpr int kRowRegs = 208, kOtherRegs = 88;
// The maximum in use follows the true one when that is ahead by so much (log2 units): moving it
// means to go over the outputs in tensor memory.
constexpr float kSlack = 8.f;
// A row's reference is a whole number (RowThread::tile) below this (log2 units): rounded to fp32, the product
// that it is next to is off by 2^-5 at most.
constexpr float kFar = 1048576.f;

template <int D>
struct Cfg {
    static constexpr int HALF = kTile * 128;        // 128 rows of 64 places, 128-byte swizzle
    static constexpr int OPERAND = HALF * (D / 64);
    static constexpr int NK = D == 64 ? 3 : 2, NV = NK;
    static constexpr int Q = 0, K = 2 * OPERAND, V = K + NK * OPERAND, OUT = V + NV * OPERAND;
    static constexpr int SMEM = OUT + 8 * 32 * 128 + 1024; // 64 places of a warp's rows; alignment
    static constexpr int LPR = D / 8, RPI = 32 / LPR;      // 16-byte chunks of a row, rows a pass
    static constexpr int BOX = kBox * D * 2;               // bytes of a box
};
static_assert(Cfg<128>::SMEM + 2048 <= 227 * 1024, "a CTA fits an SM, with its barriers and notes");
// Tensor memory: scores of the two blocks (P over them), outputs.
constexpr uint32_t kS = 0, kO = 256;

// Division of 0 <= n < 2^31 by a number known at the launch (T. Granlund and P. Montgomery, 1994): an item's
// place takes several, one after another, where nothing else goes on.
struct Divisor {
    uint32_t d = 1, m = 0, shift = 0;
    __host__ Divisor(uint32_t n = 1) : d(n) {
        while ((uint64_t(1) << shift) < d) ++shift;
        m = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ int of(int n) const { return int((__umulhi(m, uint32_t(n)) + uint32_t(n)) >> shift); }
};

struct Shape {
    const int32_t *lens;
    int B, T, Hkv, cap, window, sinks, rows, nrb;
    int token, head, page;            // dimensions of the tensor maps
    int items, whole;                 // items with halves counted; those that are not halves
    Divisor heads, per_b, G, ps;      // by B Hkv, by Hkv, by the query heads of a key/value head, by the page
};

// Rows r0 on of sequence b and head hk.  Index v < total of the run of positions that some row
// sees: position v below ns, then lo + v - ns; ns and lo are multiples of a box.
struct Item {
    int b, hk, r0;
    bool half;
    int len, emin, emax;
    int lo, ns, total, ntiles;
};

// Item number x: the last rows come first, which see most where there is no window.  From s.whole
// on two numbers share an item, a block of rows each, of which the CTA's two blocks of threads see
// half of every tile each and join their sums at the end.  A CTA has one of those at most, its last
// item: they begin with a round of the SMs and are no more than these (launch_paged_prompt).
__device__ __forceinline__ Item item_of(const Shape &s, int x) {
    Item it;
    it.half = x >= s.whole;
    const int i = it.half ? s.whole + (x - s.whole) / 2 : x;
    const int y = s.heads.of(i), bh = i - y * int(s.heads.d);
    it.r0 = (s.nrb - 1 - y) * kItemRows + (it.half ? (x - s.whole) % 2 * kRows : 0);
    it.b = s.per_b.of(bh);
    it.hk = bh - it.b * s.Hkv;
    it.len = max(s.lens[it.b], 0);
    const int r1 = min(it.r0 + (it.half ? kRows : kItemRows), s.rows) - 1;
    it.emin = it.len - s.T + s.G.of(it.r0);
    it.emax = it.len - s.T + s.G.of(r1);
    const int hi = min(it.emax + 1, s.cap);
    it.lo = s.window > 0 ? min(max(0, it.emin + 1 - s.window), s.cap) / kBox * kBox : 0;
    it.ns = s.sinks < it.lo ? (s.sinks + kBox - 1) / kBox * kBox : it.lo;
    if (s.sinks == 0 || hi <= 0) it.ns = 0;
    it.total = it.r0 < s.rows ? it.ns + max(0, hi - it.lo) : 0;
    it.ntiles = (it.total + kTile - 1) / kTile;
    return it;
}
__device__ __forceinline__ int pos_of(const Item &it, int v) { return v < it.ns ? v : it.lo + (v - it.ns); }

// Waits for a phase of bar: false after two seconds, and at once where some thread of the CTA
// has given up.
__device__ __forceinline__ bool wait_one(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
#pragma unroll 1
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (*gave_up) return false;
        if (ptx::globaltimer_ns() - t0 > 2000000000ull) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    return __all_sync(~0u, wait_one(bar, parity, gave_up));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(__cvta_generic_to_global(src)), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at));
    return v;
}
__device__ __forceinline__ void sts16(uint32_t at, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
    ptx::tmem_ld_wait();
    return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v))
                 : "memory");
    ptx::tmem_st_wait();
}

// Chunk c (16 bytes) of row r of an operand: 64 places to a row of 128 bytes, chunks exchanged
// by the 128-byte swizzle, the second 64 places behind all rows' first.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return (c / 8) * Cfg<D>::HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *m, uint64_t *bar, int c0, int c1,
                                         int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(ptx::smem_u32(bar))
        : "memory");
}

struct Barriers {
    uint64_t k_land[3], v_land[3];
    uint64_t ready[3];                // a tile's values, looked through, and the next tile's keys
    uint64_t q_full[2], s_full[2][3], p_full[2], o_full[2];
    uint64_t parted;                  // a half item's second sums are written
    uint64_t done;
};
// What is known of the last four tiles (a tile's loads begin when the products of scores of the
// tile NK before it are done, so the rows' threads are at most three tiles behind).
struct Notes {
    uint32_t there[4];                // bit i: box i's page exists
    int foul[4];                      // of the last four items: the item's number + 1 if a value that was
                                      // looked at is infinite or NaN
    float3 sums[kRows];               // a half item's second maxima, references (RowThread::tile) and sums
};

// The rows of an item: from where on some do not see all that is there (v >= least), and below
// where some don't any more (v < most, sinks apart).
__device__ __forceinline__ bool all_see(const Shape &s, const Item &it, int v0) {
    const int least = it.ns + it.emin - it.lo + 1;
    const int most = s.window > 0 ? it.ns + max(it.emax - s.window + 1 - it.lo, 0) : 0;
    return v0 + kTile <= least && (most <= v0 || v0 + kTile <= s.sinks);
}

// ---- the loading warps, one for keys and one for values ---------------------------------------
template <int D>
__device__ __forceinline__ void load_tiles(const PagedArgs &a, const Shape &s, const CUtensorMap *map,
                                           Barriers &bar, Notes &notes, volatile int *gave_up, uint32_t base,
                                           bool values) {
    using C = Cfg<D>;
    constexpr int N = C::NK;
    static_assert(C::NK == C::NV, "");
    uint64_t *const landed = values ? bar.v_land : bar.k_land;
    const uint32_t slots = base + (values ? C::V : C::K);
    const int lane = threadIdx.x % 32;
    int jt = 0;                       // tile of the CTA
    // Where a wait ran out: what is under way lands before the CTA leaves.
    auto settle = [&]() {
        for (int i = max(0, jt - N); i < jt; ++i) ptx::mbar_wait(&landed[i % N], (i / N) & 1);
    };
#pragma unroll 1
    for (int x = blockIdx.x; x < s.items; x += gridDim.x) {
        const Item it = item_of(s, x);
#pragma unroll 1
        for (int t = 0; t < it.ntiles; ++t, ++jt) {
            const int st = jt % N;
            const int v = t * kTile + lane * kBox, pos = pos_of(it, v);
            const int p = s.ps.of(pos), at = pos - p * a.c.ps;
            const int boxes = min(kTile / kBox, (it.total - t * kTile + kBox - 1) / kBox);
            int page = -1;
            if (lane < boxes && SSD_IDX_OK(a.err, it.b * a.tb + p, a.t_n)) page = a.table[it.b * a.tb + p];
            const bool ok = page >= 0 && page < a.c.pages;
            const uint32_t there = __ballot_sync(~0u, ok);
            if (!ok) page = a.c.pages;        // outside: zeros
            auto place = [&](int dim) { return dim == s.token ? at : dim == s.head ? it.hk : page; };
            const int c1 = place(1), c2 = place(2), c3 = place(3);
            // Block 1's scores of tile j are made: the keys of tile j have been read, and (its products are
            // made in order) the values of tile j - 1.
            const int j = jt - N + (values ? 1 : 0);
            if (jt >= N && !wait_warp(&bar.s_full[1][j % N], (j / N) & 1, gave_up)) return settle();
            if (lane == 0) {
                if (!values) notes.there[jt & 3] = there;
                ptx::mbar_arrive_expect_tx(&landed[st], boxes * C::BOX);
            }
            __syncwarp();
            if (lane < boxes) {
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    load_box(slots + st * C::OPERAND + h * C::HALF + lane * kBox * 128, map, &landed[st], 64 * h,
                             c1, c2, c3);
            }
        }
    }
    if (*gave_up) settle();
}

// ---- the checking warp ------------------------------------------------------------------
//
// A probability of 0 would make NaN of an infinity or NaN that a row does not see: where some row
// of the item does not see all of a tile, those of its values become zeros here, and at the item's
// end the rows' threads add them to the rows that see them.  Other tiles pass as they are.
template <int D>
__device__ __forceinline__ void check_values(const Shape &s, Barriers &bar, Notes &notes,
                                             volatile int *gave_up, uint32_t base) {
    using C = Cfg<D>;
    const int lane = threadIdx.x % 32;
    int jt = 0, nitem = 0;
#pragma unroll 1
    for (int x = blockIdx.x; x < s.items; x += gridDim.x) {
        const Item it = item_of(s, x);
        if (it.ntiles == 0) continue;
        bool more = false;            // another item with tiles follows
        for (int y = x + gridDim.x; y < s.items && !more; y += gridDim.x) more = item_of(s, y).ntiles > 0;
#pragma unroll 1
        for (int t = 0; t < it.ntiles; ++t, ++jt) {
            const int vs = jt % C::NV;
            if (!wait_warp(&bar.v_land[vs], (jt / C::NV) & 1, gave_up)) return;
            if (!all_see(s, it, t * kTile)) {
                const int rows = min(kTile, (it.total - t * kTile + kBox - 1) / kBox * kBox);
                const uint32_t slot = base + C::V + vs * C::OPERAND;
                // the largest magnitude of each lane's values, as 16-bit integers
                uint32_t most = 0;
#pragma unroll 8
                for (int r0 = 0; r0 < rows; r0 += C::RPI) {
                    const uint4 u = lds16(slot + chunk_at<D>(r0 + lane / C::LPR, lane % C::LPR));
                    most = __vmaxu2(__vmaxu2(most, u.x & 0x7fff7fffu), u.y & 0x7fff7fffu);
                    most = __vmaxu2(__vmaxu2(most, u.z & 0x7fff7fffu), u.w & 0x7fff7fffu);
                }
                if (__any_sync(~0u, __vcmpgeu2(most, 0x7f807f80u) != 0)) {
#pragma unroll 1
                    for (int r0 = 0; r0 < rows; r0 += C::RPI) {
                        const uint32_t at = slot + chunk_at<D>(r0 + lane / C::LPR, lane % C::LPR);
                        const uint4 u = lds16(at);
                        uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] &= ~__vcmpgeu2(w[i] & 0x7fff7fffu, 0x7f807f80u);
                        sts16(at, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                    if (lane == 0) notes.foul[nitem & 3] = nitem + 1;
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
            }
            // the next tile's keys too, so that the issuing thread waits once
            if ((t + 1 < it.ntiles || more) && !wait_warp(&bar.k_land[(jt + 1) % C::NK], ((jt + 1) / C::NK) & 1, gave_up))
                return;
            if (lane == 0) ptx::mbar_arrive(&bar.ready[vs]);
        }
        ++nitem;
    }
}

// ---- the issuing thread -----------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void issue(const Shape &s, Barriers &bar, volatile int *gave_up, uint32_t base,
                                      uint32_t tmem) {
    using C = Cfg<D>;
    constexpr uint32_t kIdS = ptx::idesc_bf16_f32(kRows, 0, false, false);
    constexpr uint32_t kIdO = ptx::idesc_bf16_f32(kRows, D, false, true);
    int x = blockIdx.x, t = 0, jt = 0, nitem = 0;
    // this item's positions and tiles, and the next one's (found while rows are worked on: what
    // this thread waits for, the tensor core waits for)
    int total = 0, ntiles = 0, next_total = 0, next_tiles = 0;
    bool half = false, next_half = false;
    auto find_next = [&]() {
        next_tiles = 0;
        for (; x < s.items && next_tiles == 0; x += gridDim.x) {
            const Item it = item_of(s, x);
            next_total = __shfl_sync(~0u, it.total, 0);
            next_tiles = __shfl_sync(~0u, it.ntiles, 0);
            next_half = it.half;
        }
    };
    auto take_next = [&]() {
        total = next_total;
        ntiles = next_tiles;
        half = next_half;
    };
    // a block's scores of tile t of the item, tile jt of the CTA (one lane's); halved: of a half item
    auto scores = [&](int blk, auto halved) {
        const int ks = jt % C::NK, left = total - t * kTile;
        auto multiply = [&](int n, uint32_t q_at, uint32_t k_at) {
            const uint32_t id = kIdS | uint32_t((n + 31) & ~31) >> 3 << 17;
            const uint64_t q = ptx::sdesc(q_at, 16, 1024), k = ptx::sdesc(k_at, 16, 1024);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const uint64_t o = uint64_t((i / 4) * C::HALF + (i % 4) * 32) >> 4;
                ptx::mma_bf16_ss(tmem + kS + 128 * blk, q + o, k + o, id, i != 0);
            }
        };
        if constexpr (!decltype(halved)::value)
            multiply(min(kTile, left), base + C::Q + blk * C::OPERAND, base + C::K + ks * C::OPERAND);
        else if (left > blk * kPart)  // a part of the tile each, for the same queries
            multiply(min(kPart, left - blk * kPart), base + C::Q, base + C::K + ks * C::OPERAND + blk * kPart * 128);
        ptx::mma_commit(&bar.s_full[blk][ks]);
    };
    // the first ones of an item
    auto first_scores = [&](int blk) {
        if (jt == 0 && !wait_warp(&bar.k_land[0], 0, gave_up)) return false;
        if (!wait_warp(&bar.q_full[blk], nitem & 1, gave_up)) return false;
        if (ptx::elect_one()) {
            ptx::tc_fence_after();
            if (half)
                scores(blk, std::true_type());
            else
                scores(blk, std::false_type());
        }
        __syncwarp();
        return true;
    };
    // The items of a kind (a loop for each keeps its instructions together): false where the CTA has no more.
    auto items = [&](auto halved) {
        constexpr bool kHalf = decltype(halved)::value;
        constexpr int kSteps = (kHalf ? kPart : kTile) / 16;
        for (;;) {
            const int vs = jt % C::NV, at = jt, left = total - t * kTile;
            const bool first = t == 0, last = t + 1 == ntiles;
            bool more = true;
            if (!kHalf && first) find_next();
            if (last) {
                t = 0;
                ++nitem;
                if (!kHalf) take_next();
                more = !kHalf && ntiles > 0;
            } else {
                ++t;
            }
            ++jt;
            const uint64_t v = ptx::sdesc(base + C::V + vs * C::OPERAND, C::HALF, 1024);
#pragma unroll(kHalf ? 2 : 1)
            for (int blk = 0; blk < 2; ++blk) {
                if (blk == 0 && !wait_warp(&bar.ready[vs], (at / C::NV) & 1, gave_up)) return false;
                if (!wait_warp(&bar.p_full[blk], at & 1, gave_up)) return false;
                if (ptx::elect_one()) {
                    ptx::tc_fence_after();
                    const int behind = kHalf ? blk * kPart : 0, steps = (left - behind + 15) / 16;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i)
                        if (i < steps)
                            ptx::mma_bf16_ts(tmem + kO + 128 * blk, tmem + kS + 128 * blk + 8 * i,
                                             v + uint64_t((behind / 16 + i) * 128), kIdO, !first || i > 0);
                    if (last)
                        ptx::mma_commit(&bar.o_full[blk]);
                    else
                        scores(blk, halved);
                }
                __syncwarp();
                if (!kHalf && last && more && !first_scores(blk)) return false;
            }
            if (!more) return false;
            if (half != kHalf) return true;
        }
    };
    find_next();
    take_next();
    if (ntiles == 0 || !first_scores(0) || !first_scores(1)) return;
    if (!half && !items(std::false_type())) return;
    items(std::true_type());
}

// ---- the rows' threads ----------------------------------------------------------------------
template <int D>
struct RowThread {
    using C = Cfg<D>;
    const PagedArgs &a;
    const Shape &s;
    Barriers &bar;
    Notes &notes;
    volatile int *gave_up;
    uint32_t base, ts, to;            // shared memory; this warp's lanes of S and O
    int blk, lane, warp;              // warp: 0 to 3 of its block

    // Infinities and NaN of an item's values, added to the rows that see them where zeros stand in
    // their place (a probability makes no difference to them).
    __device__ __forceinline__ void add_foul(const Item &it, int own) {
#pragma unroll 1
        for (int v = 0; v < it.total; ++v) {
            if (all_see(s, it, v / kTile * kTile)) continue;
            const int pos = pos_of(it, v), p = s.ps.of(pos);
            const int page = SSD_IDX_OK(a.err, it.b * a.tb + p, a.t_n) ? a.table[it.b * a.tb + p] : -1;
            if (page < 0 || page >= a.c.pages) continue;
            const int64_t off = page * a.c.sp + it.hk * a.c.sh + (pos - p * a.c.ps) * a.c.st;
            const bool see = pos <= own && (s.window == 0 || pos > own - s.window || pos < s.sinks);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                const float x = SSD_IDX_OK(a.err, off + c + lane, a.c.n)
                                    ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.c.v)[off + c + lane])
                                    : 0.f;
                for (uint32_t bad = __ballot_sync(~0u, !isfinite(x)); bad; bad &= bad - 1) {
                    const int d = __ffs(bad) - 1;
                    const float add = __shfl_sync(~0u, x, d), was = tmem_ld1(to + c + d);
                    tmem_st1(to + c + d, see ? was + add : was);
                }
            }
        }
    }

    __device__ __forceinline__ int row_of(const Item &it) const {
        return it.r0 + (it.half ? 0 : blk * kRows) + warp * 32 + lane;
    }
    // This warp's 32 rows of an item's queries to shared memory (the products that read the ones
    // before them are done); and their arrival.
    __device__ __forceinline__ int64_t query_of(const Item &it) const {     // the lane's row of them
        const int r = min(row_of(it), s.rows - 1), t = s.G.of(r), G = int(s.G.d);
        return it.b * a.q_sb + t * a.q_st + (it.hk * G + r - t * G) * a.q_sh;
    }
    __device__ __forceinline__ void load_queries(int64_t off) {
        const uint32_t dst = base + C::Q + blk * C::OPERAND;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += C::RPI) {
            const int row = r0 + lane / C::LPR;
            const int64_t o = __shfl_sync(~0u, off, row) + (lane % C::LPR) * 8;
            const bool ok = SSD_IDX_OK(a.err, o + 7, a.q_n);
            copy16(dst + chunk_at<D>(warp * 32 + row, lane % C::LPR),
                   static_cast<const __nv_bfloat16 *>(a.q) + (ok ? o : 0), ok);
        }
    }
    __device__ __forceinline__ void queries_loaded() {
        asm volatile("cp.async.wait_all;" ::: "memory");
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&bar.q_full[blk]);
    }

    // Tile t of an item for this thread's row, which sees [va, vb) of its run, and below vb what lies
    // below `sinks` too: scores to weights 2^(qs s - r), with the row's sum l.  r = -minus follows qs m, m
    // the largest score when it was set, as the nearest whole number: qs s - r is one operation, rounded
    // once, all weights of a row stand to one another as their scores do, and a change of r is a power of
    // two.  large: for scores from 2^20 on the nearest number may be far off, and the warp's weights are
    // 2^(qs (s - m)).  (r = qs m rounded took as long, and moved by up to 2^-14 from tile to tile.)
    // kAll: all rows of the warp see all positions.  W: 128, or 64 of a half item, from v0 on.
    template <bool kAll, int W>
    __device__ __forceinline__ void tile(int t, int v0, int va, int vb, uint32_t there, float qs, float &m,
                                         float &l, float &minus, bool &large) {
        uint32_t raw[W / 32][32];
        // (of a narrower tile too: what its products have not written is not seen)
#pragma unroll
        for (int c = 0; c < W / 32; ++c) ptx::tmem_ld32(ts + 32 * c, raw[c]);
        float mx = -INFINITY;
        auto look = [&](int c) {
            if constexpr (!kAll) {
                const int b = v0 + 32 * c;
                auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
                uint32_t vis = (there >> (2 * c) & 1 ? 0xffffu : 0u) | (there >> (2 * c + 1) & 1 ? 0xffff0000u : 0u);
                vis &= below(vb - b) & (~below(va - b) | below(s.sinks - b));
#pragma unroll
                for (int i = 0; i < 32; ++i) raw[c][i] = vis & (1u << i) ? raw[c][i] : 0xff800000u;
            }
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; i += 4)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    top[k] = max3(top[k], __uint_as_float(raw[c][i + 2 * k]), __uint_as_float(raw[c][i + 2 * k + 1]));
            mx = max3(mx, top[0], top[1]);
        };
        ptx::tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < W / 32; ++c) look(c);
        if (__any_sync(~0u, (mx - m) * qs > kSlack || (m == -INFINITY && mx != m)) || large) {
            const float to_m = fmaxf(m, mx), whole = rintf(to_m * qs);
            const bool none = to_m == -INFINITY, far = __any_sync(~0u, !none && !(fabsf(whole) < kFar));
            const float next = none || far ? 0.f : -whole;
            const float f = m == -INFINITY ? 1.f
                                           : ex2(large && far ? (m - to_m) * qs
                                                 : large      ? fmaf(m, qs, next)
                                                 : far        ? fmaf(-to_m, qs, -minus)
                                                              : next - minus);
            m = to_m;
            minus = next;
            large = far;
            l *= f;
            if (t > 0) {              // (the outputs so far are complete: the scores came after them)
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    ptx::tmem_ld16(to + c, o);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    ptx::tmem_st16(to + c, o);
                }
                ptx::tmem_st_wait();
            }
            if (large) {
                const float ref = none ? 0.f : m;
#pragma unroll
                for (int i = 0; i < W; ++i)
                    raw[i / 32][i % 32] = __float_as_uint(__uint_as_float(raw[i / 32][i % 32]) - ref);
            }
        }
        const F2 mm = f2(minus, minus), qq = f2(qs, qs);
        F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
        auto weights = [&](int c) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 e = parts(fma(f2(__uint_as_float(raw[c][2 * i]), __uint_as_float(raw[c][2 * i + 1])),
                                           qq, mm));
                const float x0 = ex2(e.x), x1 = ex2(e.y);
                sum[i & 1] = add(sum[i & 1], f2(x0, x1));
                p[i] = pack_bf16(x0, x1);
            }
            ptx::tmem_st16(ts + 16 * c, p);
        };
#pragma unroll
        for (int c = 0; c < W / 32; ++c) weights(c);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bar.p_full[blk]);
        const float2 s0 = parts(add(sum[0], sum[1]));
        l += s0.x + s0.y;
    }

    // An item's tiles.  loaded: the next one's queries are on their way.
    template <bool kHalf>
    __device__ __forceinline__ bool tiles(const Item &it, int x, int va, int vb, float qs, int &jt, bool &loaded,
                                          float &m, float &l, float &minus, bool &large) {
        constexpr int W = kHalf ? kPart : kTile;
        // the next item's queries, loaded when the last scores of this one are made
        [[maybe_unused]] int64_t next = -1;     // where the lane's row of them is
        [[maybe_unused]] bool follow = false;
#pragma unroll 1
        for (int t = 0; t < it.ntiles; ++t, ++jt) {
            if (!wait_warp(&bar.s_full[blk][jt % C::NK], (jt / C::NK) & 1, gave_up)) return false;
            ptx::tc_fence_after();
            if constexpr (!kHalf) {
                if (t == it.ntiles / 2 && x + gridDim.x < s.items) {
                    const Item after = item_of(s, x + gridDim.x);
                    follow = after.ntiles > 0;
                    if (follow && (blk == 0 || !after.half)) next = query_of(after);
                }
                if (t + 1 == it.ntiles && follow) {
                    if (next >= 0) load_queries(next);
                    loaded = true;
                }
            }
            const int v0 = t * kTile + (kHalf ? blk * W : 0);
            constexpr uint32_t kAll = (1u << W / kBox) - 1;
            const uint32_t there = notes.there[jt & 3] >> (kHalf ? blk * (W / kBox) : 0) & kAll;
            if (__all_sync(~0u, v0 + W <= vb && (va <= v0 || v0 + W <= s.sinks) && there == kAll))
                tile<true, W>(t, v0, va, vb, there, qs, m, l, minus, large);
            else
                tile<false, W>(t, v0, va, vb, there, qs, m, l, minus, large);
        }
        return true;
    }

    __device__ __forceinline__ bool run() {
        const float qs = a.scale * kLog2e;
        int jt = 0, nitem = 0;
        bool loaded = false;          // this item's queries
#pragma unroll 1
        for (int x = blockIdx.x; x < s.items; x += gridDim.x) {
            const Item it = item_of(s, x);
            const bool mine = blk == 0 || !it.half;    // (of a half item the first block's threads write)
            const int r = row_of(it), rr = min(r, s.rows - 1);
            const int tk = s.G.of(rr), own = it.len - s.T + tk;
            // what it sees of the item's run: [va, vb), and below vb what lies below `sinks` too (where
            // ns < sinks it is lo, and the run has no gap)
            const int vb = own < it.lo ? min(own + 1, it.ns) : it.ns + own - it.lo + 1;
            const int va = s.window > 0 ? it.ns + max(own - s.window + 1 - it.lo, 0) : 0;
            float m = -INFINITY, l = 0.f, minus = 0.f;
            bool large = false;
            if (it.ntiles) {
                if (!loaded) {
                    if (mine) load_queries(query_of(it));
                    queries_loaded();
                }
                loaded = false;
            }
            if (!(it.half ? tiles<true>(it, x, va, vb, qs, jt, loaded, m, l, minus, large)
                          : tiles<false>(it, x, va, vb, qs, jt, loaded, m, l, minus, large)))
                return false;
            if (loaded) queries_loaded();
            float f0 = 1.f, f1 = 0.f;             // the two sums' factors
            bool two = false;                     // there is something in the second
            if (it.ntiles) {
                if (!wait_warp(&bar.o_full[blk], nitem & 1, gave_up)) return false;
                if (it.half) {
                    if (blk == 1) {
                        notes.sums[warp * 32 + lane] = make_float3(m, large ? NAN : minus, l);
                        ptx::mbar_arrive(&bar.parted);
                    } else {
                        if (!wait_warp(&bar.o_full[1], nitem & 1, gave_up) ||
                            !wait_warp(&bar.parted, 0, gave_up))
                            return false;
                        const float3 other = notes.sums[warp * 32 + lane];
                        const float to_m = fmaxf(m, other.x);
                        const bool one = m != -INFINITY;
                        two = other.x != -INFINITY;
                        const bool far = isnan(other.y);
                        if (large || far) {   // the weights' own references in terms of the maxima
                            f0 = one ? ex2((m - to_m) * qs - (large ? 0.f : fmaf(m, qs, minus))) : 0.f;
                            f1 = two ? ex2((other.x - to_m) * qs - (far ? 0.f : fmaf(other.x, qs, other.y))) : 0.f;
                            large = true;
                        } else {
                            const float both = fminf(one ? minus : INFINITY, two ? other.y : INFINITY);
                            f0 = one ? ex2(both - minus) : 0.f;
                            f1 = two ? ex2(both - other.y) : 0.f;
                            minus = both;
                        }
                        l = l * f0 + other.z * f1;
                        m = to_m;
                    }
                }
                ptx::tc_fence_after();
            }
            const bool joins = it.half && it.ntiles && blk == 0, foul = it.ntiles && notes.foul[nitem & 3] == nitem + 1;
            nitem += it.ntiles > 0;
            if (!mine) continue;
            if (joins) {              // O = f0 O + f1 O of the other block, back where it was
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16], p[16];
                    ptx::tmem_ld16(to + c, o);
                    ptx::tmem_ld16(to + kRows + c, p);
                    ptx::tmem_ld_wait();
                    // (what was never written may be anything)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = __float_as_uint(__uint_as_float(o[i]) * f0 + (two ? __uint_as_float(p[i]) * f1 : 0.f));
                    ptx::tmem_st16(to + c, o);
                }
                ptx::tmem_st_wait();
            }
            if (foul) add_foul(it, own);
            // Rows of 64 places go through shared memory, so that stores are whole lines (a row a
            // thread, 16 bytes at a time, took 3800 cycles an item).
            const int h = it.hk * int(s.G.d) + rr - tk * int(s.G.d);
            const int64_t off = r < s.rows ? it.b * a.o_sb + tk * a.o_st + h * a.o_sh : -1;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const uint32_t stage = base + C::OUT + (blk * 4 + warp) * 32 * 128;
            uint32_t out[D / 32][32];
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                if (it.ntiles) {
                    ptx::tmem_ld32(to + 32 * k, out[k]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) out[k][i] = 0;
                }
            }
            ptx::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < D; c += 64) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t *const o = &out[c / 32 + k / 4][8 * (k % 4)];
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = pack_bf16(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                    sts16(stage + lane * 128 + ((k ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = 4 * k + lane / 8, chunk = lane % 8;
                    const int64_t at = __shfl_sync(~0u, off, row);
                    const uint4 u = lds16(stage + row * 128 + ((chunk ^ (row & 7)) << 4));
                    if (at >= 0 && SSD_IDX_OK(a.err, at + c + chunk * 8 + 7, a.o_n))
                        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at + c + chunk * 8) = u;
                }
                __syncwarp();
            }
            const int64_t at = (int64_t(it.b) * s.T + tk) * a.Hq + h;
            if (a.lse && r < s.rows && SSD_IDX_OK(a.err, at, int64_t(s.B) * s.T * a.Hq))
                a.lse[at] = l == 0.f ? -INFINITY : ((large ? m * qs : -minus) + log2f(l)) * kLn2;
        }
        return true;
    }
};

// kAsk: the lengths tell whether this kernel works or k_paged_mma, which is launched before it.  It may start
// while that one's CTAs leave: it reads nothing that they write, and is not done before they are.
template <int D, bool kAsk>
__global__ void __launch_bounds__(kThreads, 1)
k_paged_prompt(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
               const __grid_constant__ PagedArgs a, const __grid_constant__ Shape s) {
    using C = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Barriers bar;
    __shared__ Notes notes;
    __shared__ int gave_up;
    __shared__ uint32_t tmem_at;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t base = (ptx::smem_u32(smem_raw) + 1023) & ~1023u;
    if constexpr (kAsk) {
        let_next_start();
        if (!prompt_pays(a)) return wait_for_previous();
    }
    if (threadIdx.x == 0) {
        gave_up = 0;
        notes.foul[0] = notes.foul[1] = notes.foul[2] = notes.foul[3] = 0;
        for (int i = 0; i < 3; ++i) {
            ptx::mbar_init(&bar.k_land[i], 1);
            ptx::mbar_init(&bar.v_land[i], 1);
            ptx::mbar_init(&bar.ready[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bar.q_full[i], kRows);
            ptx::mbar_init(&bar.p_full[i], kRows);
            ptx::mbar_init(&bar.o_full[i], 1);
            for (int k = 0; k < 3; ++k) ptx::mbar_init(&bar.s_full[i][k], 1);
        }
        ptx::mbar_init(&bar.parted, kRows);
        ptx::mbar_init(&bar.done, 1);
        ptx::fence_mbar_init();
    }
    if (warp == 8) {
        ptx::tmem_alloc(&tmem_at, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, tmem_at, 0);
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        const int blk = warp / 4;
        const uint32_t lanes = uint32_t(warp % 4 * 32) << 16;
        RowThread<D> rows{a, s, bar, notes, &gave_up, base, tmem + lanes + kS + 128 * blk,
                          tmem + lanes + kO + 128 * blk, blk, lane, warp % 4};
        if (!rows.run()) asm volatile("cp.async.wait_all;" ::: "memory");    // (given up: queries under way)
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) {
            issue<D>(s, bar, &gave_up, base, tmem);
            // nothing is under way when tensor memory is given back
            if (ptx::elect_one()) {
                ptx::mma_commit(&bar.done);
                ptx::mbar_wait(&bar.done, 0);
            }
            __syncwarp();
        } else if (warp < 11) {
            load_tiles<D>(a, s, warp == 9 ? &kmap : &vmap, bar, notes, &gave_up, base, warp == 10);
        } else {
            check_values<D>(s, bar, notes, &gave_up, base);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && gave_up) atomicOr(a.err, kErrTimeout);
    if (warp == 8) ptx::tmem_dealloc(tmem, 512);
    if constexpr (kAsk) wait_for_previous();
}

template <int D, bool kAsk>
cudaError_t launch_d(const PagedArgs &a, const Shape &s, cudaStream_t stream) {
    static std::atomic<uint64_t> done[4];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 256 || !((done[dev / 64].load(std::memory_order_acquire) >> (dev % 64)) & 1)) {
        e = cudaFuncSetAttribute(k_paged_prompt<D, kAsk>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 256) done[dev / 64].fetch_or(uint64_t(1) << (dev % 64));
    }
    const int grid = s.items < device_sm_count() ? s.items : device_sm_count();
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::SMEM;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = kAsk ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_paged_prompt<D, kAsk>, a.maps->k, a.maps->v, a, s);
}

int64_t items_of(const PagedArgs &a, int block) {       // row blocks of a size
    const int64_t rows = int64_t(a.T) * (a.Hq / a.c.Hkv);
    return int64_t(a.B) * a.c.Hkv * ((rows + block - 1) / block);
}

}  // namespace

// An item's time goes by its positions alone, 1.55 us for 128 of them (D = 64: 1.36), a half item's 1.10
// (0.93), with all of its rows there or not; the kernels of ssd_attn.cuh split a sequence's positions
// over the SMs and take 0.0154 us (0.0106) for 128 positions and a block of 64 rows.  So this kernel is
// the faster one from 72 (88) such blocks on, and taken from 84 (107).  Measured, here / there: 88 blocks
// (176 tokens of 32 over 8 heads over 8192) 70 / 102 us; 112 blocks, D = 64, 59 / 91; 256 blocks (512
// tokens over 8192) 70 / 261 us, D = 64 60 / 184; 8192 tokens 399 / 2167, 344 / 1500.  (A scale below 0
// would have to turn the scores' signs, which no model asks for.  Fewer rows than a block of a sequence
// and head take the others too: 96 sequences, 4 rows, a window of 1024: 93 us here, 47 there.)
// Where a single sequence has so many blocks (what whole items need: 106, D = 64 137) no lengths make
// this the slower one, and as little where no row can see more than 1536 positions (one of so many among
// 13 of 33: 27 / 31 us, D = 64 23 / 25); where it takes all of a batch's blocks, the lengths tell
// (prompt_pays).
Prompt prompt_fits(const PagedArgs &a) {
    const int64_t blocks = items_of(a, 64), sms = device_sm_count();
    const bool wide = a.c.D == 128;
    if (a.c.dt != DT_BF16 || a.T * (a.Hq / a.c.Hkv) < kRows || !(a.scale > 0.f) || a.c.ps % kBox ||
        a.c.pages <= 0 || 20 * blocks < (wide ? 11 : 14) * sms || items_of(a, kItemRows) >= (1 << 30))
        return Prompt::kNo;
    int64_t most = int64_t(a.M) * a.c.ps;
    if (a.window > 0) most = std::min(most, a.window + a.sinks + kItemRows / (a.Hq / a.c.Hkv));
    const bool any = a.B == 1 || most <= 1536 || 20 * blocks >= int64_t(a.B) * (wide ? 14 : 18) * sms;
    return any ? Prompt::kYes : Prompt::kAsk;
}

// A map's strides grow, each a multiple of the one before and below 2^40 bytes: so the tokens, heads and pages
// of the pools are its dimensions in the order of their strides, and pools with others (a stride of 0 that heads
// share, heads apart by some places more than their tokens take) have none.  A dimension of one comes last, with
// any stride.
bool make_prompt_maps(const PagedArgs &a, PromptMaps *m) {
    struct Dim {
        uint64_t n, stride;
        int *at;
    } d[3] = {{uint64_t(a.c.ps), uint64_t(a.c.st) * 2, &m->token},
              {uint64_t(a.c.Hkv), uint64_t(a.c.sh) * 2, &m->head},
              {uint64_t(a.c.pages), uint64_t(a.c.sp) * 2, &m->page}};
    std::stable_sort(d, d + 3, [](const Dim &x, const Dim &y) {
        return x.n > 1 && (y.n <= 1 || x.stride < y.stride);
    });
    uint64_t dims[4] = {uint64_t(a.c.D)}, strides[3], below = uint64_t(a.c.D) * 2;
    uint32_t box[4] = {64, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        *d[i].at = i + 1;
        dims[i + 1] = d[i].n;
        strides[i] = d[i].n > 1 ? d[i].stride : below;
        if (strides[i] < below || strides[i] >= uint64_t(1) << 40 || (i && strides[i] % below)) return false;
        below = strides[i];
    }
    box[m->token] = kBox;
    return make_tmap_bf16(&m->k, a.c.k, 4, dims, strides, box) == cudaSuccess &&
           make_tmap_bf16(&m->v, a.c.v, 4, dims, strides, box) == cudaSuccess;
}

// The costs that prompt_fits' comment gives; of less than half a round of items all are halved.
void ask_lengths(PagedArgs &a) {
    const bool wide = a.c.D == 128;
    const int G = a.Hq / a.c.Hkv;
    const uint64_t sms = device_sm_count(), items = items_of(a, kItemRows), per = items / a.B;
    int64_t most = int64_t(a.M) * a.c.ps;
    if (a.window > 0) most = std::min(most, a.window + a.sinks + kItemRows / G);
    const uint64_t whole = wide ? 15500 : 13600, part = wide ? 11000 : 9300;
    a.ask.on = 1;
    a.ask.most = int(most);
    a.ask.one = (2 * items <= sms ? part : whole) * sms;
    a.ask.share = items <= sms ? 0 : per * whole;
    a.ask.line = items_of(a, 64) / a.B * (wide ? 154 : 106) * sms;
}

cudaError_t launch_paged_prompt(const PagedArgs &a, cudaStream_t stream) {
    Shape s{};
    s.lens = a.lens;
    s.B = a.B;
    s.T = a.T;
    s.Hkv = a.c.Hkv;
    s.cap = a.M * a.c.ps;
    s.window = int(a.window);
    s.sinks = int(a.sinks);
    s.heads = Divisor(uint32_t(a.B * a.c.Hkv));
    s.per_b = Divisor(uint32_t(a.c.Hkv));
    s.G = Divisor(uint32_t(a.Hq / a.c.Hkv));
    s.ps = Divisor(uint32_t(a.c.ps));
    s.rows = a.T * (a.Hq / a.c.Hkv);
    s.nrb = (s.rows + kItemRows - 1) / kItemRows;
    // Where the items do not go up in whole rounds of the SMs, and half of them are free in the last one,
    // that round's items are halved.
    const int n = int(items_of(a, kItemRows)), sms = device_sm_count(), over = n % sms;
    s.whole = 2 * over <= sms ? n - over : n;
    s.items = 2 * n - s.whole;
    s.token = a.maps->token;
    s.head = a.maps->head;
    s.page = a.maps->page;
    if (a.ask.on) return a.c.D == 64 ? launch_d<64, true>(a, s, stream) : launch_d<128, true>(a, s, stream);
    return a.c.D == 64 ? launch_d<64, false>(a, s, stream) : launch_d<128, false>(a, s, stream);
}

}  // namespace ssd
