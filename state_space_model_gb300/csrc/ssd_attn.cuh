// Attention of new tokens over the paged key/value cache (ssd_paged_attention): the kernels and
// their launch rules.  ssd_attn.cu, ssd_attn_f8.cu and ssd_attn_f4.cu compile them for the
// pools' types, ssd_attn_sinks*.cu the same with sinks beside the window (SSD_ATTN_SINKS; as a
// choice at run time they cost the calls without 4% at 16 sequences of four tokens under a
// window, and 1.5% in fp32).
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
// kernels are built to keep reads in flight, not for matrix rate.  The two
// products are turned round, S^T = K Q^T and O^T = V^T P^T, with positions and
// places as the 16 rows of mma.sync and eight queries as its columns: the
// usual 4 or 8 query heads fill a tile, which with queries as rows would be
// half empty, and scores, probabilities and output take half the registers
// and instructions.  (tcgen05 would take 128 positions as rows with as few
// columns, but its operands come from shared and tensor memory: 8-bit codes
// would have to be widened there and back, and probabilities stored.  At 8 to
// 16 queries mma.sync needs a fifth to a third of the time of the reads.)
#pragma once

#include "ptx_sm100.cuh"
#include "ssd_attn.h"
#include "ssd_attn_choice.cuh"
#include "ssd_block_math.cuh"
#include "ssd_debug.cuh"
#include "ssd_f32x2.cuh"
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

#ifdef SSD_ATTN_SINKS
constexpr bool kSinks = true;
#else
constexpr bool kSinks = false;
#endif
constexpr float kLn2 = 0.6931471805599453f;
// 8-bit values: a row's largest weight is 2^kLift to 2^(kLift + kAhead) in fp16 (so weights
// keep their 11 bits down to 2^-22 of it), with log2 of a value's scale taken as [kLeastLog,
// kMostLog].  At the lower end the fp32 sum of 2^22 probabilities of 2^(kLift + kAhead - kLeastLog) is
// finite, and scales down to 2^(kLeastLog - 22) still have weights of 11 bits; at the upper end
// a probability of 2^-kMostLog is a normal number, and the largest finite scales stay below
// fp16's end.
constexpr float kLift = 8.f, kAhead = 5.f, kLeastLog = -92.f, kMostLog = 119.f;
constexpr int kWarps = 4;                 // of a CTA that compute
constexpr int kCopyWarps = 4;             // and that copy
constexpr int kThreads = 32 * (kWarps + kCopyWarps);
constexpr int kCtasPerSm = 2;
constexpr int kF32Warps = 6;              // of a CTA of the fp32 kernel
// What the tensor-core kernel's pools hold: bf16, or codes of 8 or 4 bits.
enum : int { kBf16 = 0, kEight = 1, kFour = 2 };
// CTAs of the tensor-core kernel on an SM, by the rows of a block.
constexpr int ctas_of(int format, int rows) { return format == kFour && rows == 8 ? 3 : kCtasPerSm; }

// ---- the schedule -----------------------------------------------------------------
//
// An item is a (sequence, key/value head, block of rows).  Its cost is its
// tiles of KS positions, and kItemCost more for what an item takes whatever
// its length (its queries, the join of the warps, the write).  All items, in
// that order, form one line of cost units that is cut into nc equal parts, one
// to a CTA, wherever the cuts fall: sequences of any lengths fill the GPU
// evenly, and lengths are needed on the device only.  (Without the constant, a
// CTA whose part is 40 one-tile items takes as long as 120 tiles of one item: 96
// sequences of 17 to 16384 positions in 8 bits took 160 us where they took 94
// with it.  2 is 2% better there now, and 14% worse for a few short ones.)  An
// item that a cut falls into is finished by the join kernel from the parts that
// its CTAs leave in the workspace.  An item without positions has one (masked)
// tile, so that somebody writes its rows.
constexpr int kItemCost = 3;

// What both kernels derive the schedule from.
struct Shape {
    const int32_t *lens;
    int B, T, Hkv;
    int cap;              // positions that the page table has room for
    int window;
    int back;             // how far back a row sees: the window, or further than there are positions
    int sinks;            // positions below this are seen beside the window; 0 without one
    int RB;               // rows of a row block (the rows of a sequence and head: T G)
    int nrb;              // row blocks
    int G;                // query heads to a key/value head
    int ncta;             // most parts of the line
};

struct Item {
    int b, hk, rb;
    int len;              // positions of the sequence, new ones included
    int emin, emax;       // the places of the block's first and last row
    int lo, hi;           // what some row of the block sees (may be empty), sinks apart
    int first;            // lo rounded down to a tile
    int nsink;            // tiles of sinks that end before `first`
    int ntiles;           // those, then the ones from `first` on
};

// (What runs once for an item or a CTA is kept small, so that the loop over tiles stays
// near: when a kernel was 120 KB of code, a fifth of the loop's time was spent waiting
// for instructions.  2% more of it on the way of a short call cost that 2 to 7%: 16 sequences of four
// tokens under a window 20.2 -> 21.2 us, eight of 32 tokens over fp8 18.5 -> 19.9.  Calls out of line are
// no way, they fix the registers of both kinds of warps.)
template <int KS>
__device__ __forceinline__ void item_range(const Shape &s, Item &it) {
    it.emin = it.len - s.T;
    it.emax = it.len - 1;
    if (s.nrb > 1) {
        const int r0 = it.rb * s.RB, r1 = min(r0 + s.RB, s.T * s.G) - 1;
        it.emin = it.len - s.T + r0 / s.G;
        it.emax = it.len - s.T + r1 / s.G;
    }
    it.hi = min(it.emax + 1, s.cap);
    it.lo = s.window > 0 ? min(max(0, it.emin + 1 - s.window), s.cap) : 0;
    it.first = it.lo / KS * KS;
    if constexpr (kSinks) {
        it.nsink = s.sinks > 0 ? min((s.sinks - 1) / KS + 1, it.first / KS) : 0;
        it.ntiles = max(1, it.nsink + max(0, it.hi - it.first + KS - 1) / KS);
    } else {
        it.ntiles = max(1, (it.hi - it.first + KS - 1) / KS);
    }
}

// The first position of tile t of an item.
template <int KS>
__device__ __forceinline__ int tile_at(const Item &it, int t) {
    if constexpr (!kSinks) return it.first + t * KS;
    return t < it.nsink ? t * KS : it.first + (t - it.nsink) * KS;
}
// Whether some row of the item's block may see position pos.
__device__ __forceinline__ bool in_range(const Shape &s, const Item &it, int pos) {
    return pos < it.hi && (pos >= it.lo || (kSinks && pos < s.sinks));
}
// Whether the row at place `own` sees position pos.
__device__ __forceinline__ bool sees(const Shape &s, int own, int pos) {
    return pos <= own && (pos > own - s.back || (kSinks && pos < s.sinks));
}

// The cost of one key/value head of a sequence.
template <int KS>
__device__ __forceinline__ int64_t head_cost(const Shape &s, int len) {
    Item it;
    it.len = len;
    int64_t n = 0;
#pragma unroll 1
    for (it.rb = 0; it.rb < s.nrb; ++it.rb) {
        item_range<KS>(s, it);
        n += it.ntiles + kItemCost;
    }
    return n;
}

// The token of row r of a sequence and head.
__device__ __forceinline__ int token_of(const Shape &s, int r) { return s.T == 1 ? 0 : r / s.G; }

// The inclusive prefix of w over the lanes of a warp.
__device__ __forceinline__ int64_t warp_scan(int64_t w) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(~0u, w, o);
        if (int(threadIdx.x % 32) >= o) w += v;
    }
    return w;
}
// The same over the threads of a CTA of NW warps, and the sum of all.
template <int NW>
__device__ __forceinline__ int64_t block_scan(int64_t w, int64_t *sums, int64_t &total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    w = warp_scan(w);
    __syncthreads();
    if (lane == 31) sums[warp] = w;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        if (i < warp) before += sums[i];
        total += sums[i];
    }
    return w + before;
}

__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {   // both >= 0; mostly short
    return ((x | y) >> 32) == 0 ? int64_t(uint32_t(x) / uint32_t(y)) : x / y;
}

// A stretch of the line: CTA c takes units [c part, (c + 1) part) of the total.
struct Stretch {
    Item it;              // the item that holds its first unit
    int unit;             // that unit's number in the item
    int64_t beg, left;    // the first unit, how many
    int64_t part;
};

// The place in a sequence's items of the unit `rest` from its first.
template <int KS>
__device__ __forceinline__ void place(const Shape &s, int64_t rest, int64_t per, Stretch &f) {
    f.it.hk = s.Hkv > 1 ? int(divide(rest, per)) : 0;
    rest -= f.it.hk * per;
#pragma unroll 1
    for (f.it.rb = 0;; ++f.it.rb) {
        item_range<KS>(s, f.it);
        if (rest < f.it.ntiles + kItemCost) break;
        rest -= f.it.ntiles + kItemCost;
    }
    f.unit = int(rest);
}

struct FinderRoom {
    int64_t sums[32], rest, per;
    int b, len;
};

// Stretch number cta; left <= 0: there is none.  All threads of a CTA call it and get
// the same.  Up to 32 sequences each warp finds for itself, a lane a sequence (with
// barriers between the warps, more divisions and parameters read through memory this
// took half of a short call: 2.6 us); more go a thread a sequence, twice over.
template <int KS>
__device__ __forceinline__ Stretch find_few(const Shape &s, int cta) {
    Stretch f;
    const int lane = threadIdx.x % 32;
    const int len = lane < s.B ? max(s.lens[lane], 0) : 0;
    const int64_t per = head_cost<KS>(s, len), w = lane < s.B ? per * s.Hkv : 0;
    const int64_t upto = warp_scan(w), total = __shfl_sync(~0u, upto, 31);
    f.part = divide(total + s.ncta - 1, s.ncta);
    f.beg = cta * f.part;
    f.left = min(f.part, total - f.beg);
    if (f.left <= 0) return f;
    const int who = __ffs(__ballot_sync(~0u, f.beg < upto && f.beg >= upto - w)) - 1;
    f.it.b = who;
    f.it.len = __shfl_sync(~0u, len, who);
    place<KS>(s, f.beg - __shfl_sync(~0u, upto - w, who), __shfl_sync(~0u, per, who), f);
    return f;
}
template <int KS, int NW>
__device__ __forceinline__ Stretch find_many(const Shape s, int cta, FinderRoom *room) {
    Stretch f;
    int64_t total = 0;
#pragma unroll 1
    for (int base = 0; base < s.B; base += 32 * NW) {
        const int i = base + threadIdx.x;
        int64_t sum;
        block_scan<NW>(i < s.B ? head_cost<KS>(s, max(s.lens[i], 0)) * s.Hkv : 0, room->sums, sum);
        total += sum;
    }
    f.part = divide(total + s.ncta - 1, s.ncta);
    f.beg = cta * f.part;
    f.left = min(f.part, total - f.beg);
    if (f.left <= 0) return f;
    int64_t run = 0;
#pragma unroll 1
    for (int base = 0; base < s.B && run <= f.beg; base += 32 * NW) {
        const int i = base + threadIdx.x;
        const int len = i < s.B ? max(s.lens[i], 0) : 0;
        const int64_t per = head_cost<KS>(s, len), w = i < s.B ? per * s.Hkv : 0;
        int64_t sum;
        const int64_t upto = run + block_scan<NW>(w, room->sums, sum);
        run += sum;
        if (f.beg < upto && f.beg >= upto - w) {
            room->b = i;
            room->len = len;
            room->per = per;
            room->rest = f.beg - (upto - w);
        }
    }
    __syncthreads();
    f.it.b = room->b;
    f.it.len = room->len;
    place<KS>(s, room->rest, room->per, f);
    return f;
}
template <int KS, int NW>
__device__ __forceinline__ Stretch find(const Shape &s, int cta, FinderRoom *room) {
    return s.B <= 32 ? find_few<KS>(s, cta) : find_many<KS, NW>(s, cta, room);
}

// len: the length of the next sequence
template <int KS>
__device__ __forceinline__ Item next_item(const Shape s, Item it, int len) {
    if (++it.rb == s.nrb) {
        it.rb = 0;
        if (++it.hk == s.Hkv) {
            it.hk = 0;
            ++it.b;
            it.len = max(len, 0);
        }
    }
    item_range<KS>(s, it);
    return it;
}

// The workspace: a Cut for each CTA, then the partial results, output rows and
// their maxima (in log2 units) and sums.  Part 2 c is the first item of CTA
// c's stretch, part 2 c + 1 its last (if that is another).  The CTA that has an
// item's first tiles, but not all, says in its Cut who has the others.
struct __align__(16) Cut {
    int parts;            // CTAs that share the item, from this one on; 0: none
    int first;            // this one's part, 0 or 1 (the others' is 0)
    int b, hk, rb;
    int pad[3];
};
__host__ __device__ __forceinline__ size_t part_floats(int RB, int D) {
    return size_t(RB) * (D + 2);
}
__device__ __forceinline__ float *part_at(const PagedArgs &a, const Shape &s, int i) {
    return reinterpret_cast<float *>(a.ws + s.ncta * sizeof(Cut)) +
           size_t(i) * part_floats(s.RB, a.c.D);
}

// The debug build's look at a record, and at the last place of row rr of part i.
__device__ __forceinline__ bool cut_ok(const PagedArgs &a, const Shape &s, int i) {
    return SSD_IDX_OK(a.err, i, s.ncta) && SSD_IDX_OK(a.err, (i + 1) * int64_t(sizeof(Cut)) - 1, a.ws_n);
}
__device__ __forceinline__ bool part_ok(const PagedArgs &a, const Shape &s, int i, int rr) {
    return SSD_IDX_OK(a.err, rr, s.RB) &&
           SSD_IDX_OK(a.err,
                      int64_t(s.ncta * sizeof(Cut) + (i + 1) * part_floats(s.RB, a.c.D) * sizeof(float)) - 1,
                      a.ws_n);
}
__device__ __forceinline__ bool lse_ok(const PagedArgs &a, int64_t i) {
    return SSD_IDX_OK(a.err, i, int64_t(a.B) * a.T * a.Hq);
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
template <int N>
__device__ __forceinline__ void copy_few(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst),
                 "l"(__cvta_generic_to_global(src)), "r"(ok ? N : 0), "n"(N)
                 : "memory");
}
// n bytes (of 16) in one piece, counted at bar.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t n, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(__cvta_generic_to_global(src)), "r"(n), "r"(smem_addr(bar))
                 : "memory");
}
// An arrival at bar once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// All of this thread's copies have landed.
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// The computing warps of a CTA wait for one another.
__device__ __forceinline__ void warps_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
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
__device__ __forceinline__ uint32_t lds1(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
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
// four codes -> two pairs of fp16 values (exact)
__device__ __forceinline__ void widen4(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}
// eight 4-bit codes -> four pairs of fp16 values (exact)
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
// two e4m3 scales -> a pair of fp16 (exact)
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 a;\n\t"
        "cvt.u16.u32 a, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
        : "=r"(r)
        : "r"(codes));
    return r;
}
// products of pairs of fp16; exact for a 4-bit code (2 significant bits, 0.5 to 6) and its
// group's scale (4 bits, 2^-9 to 448)
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// The 8 x 8 matrix of 16-bit values that the warp holds (two to a lane), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// ---- the tensor-core kernel -----------------------------------------------------------
//
// Four warps compute, as WK groups of WR: the WR warps of a group take 8 NQ
// query rows each and share the group's positions, the groups take different
// positions.  Four more warps copy, up to kStages tiles ahead, across items:
// looking up pages and making addresses took a third of the computing warps'
// instructions when each copied its own, and one warp cannot keep up; they also give
// the computing warps most of their registers.  Two CTAs fill an SM, so 128 KB of
// copies are under way while two tiles are worked on.
//
// Measured (GB300, of the rate of a large copy, 6765 GB/s): 64 sequences of 4096, 64
// query heads over 8 of 128, bf16: 167 us, 95%; the same in fp8 95 us, 86%; in 4 bits
// 80 us, 59%; one sequence of 131072, 32 over 8: 86 us, 92%; 96 of 17 to 16384 over fp8:
// 77 us, 82%.
// Query rows cost little up to 32 a key/value head in bf16 (177 us) and 16 in fp8
// (105 us); at 64 in bf16 (265 us) and 32 in fp8 (168 us) the products take longer than
// the reads.  In 4 bits they do from 8 rows on (16 rows 104 us, 32 179): a conversion and a
// product with the group's scale for every four codes share the issue slots, the latter
// the tensor cores' pipe too.  Pieces of prompts are blocks of 64 rows (8192 tokens of 32 over
// 8 heads: 2.4 ms in fp8); over bf16 pools ssd_attn_prompt.cu takes them.
template <int D_, int FMT_, int NQ_, int WR_>
struct Cfg {
    static constexpr int D = D_, FMT = FMT_, NQ = NQ_, WR = WR_, WK = kWarps / WR_;
    static constexpr bool F8 = FMT != kBf16;                // codes, of 8 or 4 bits
    static constexpr bool F4 = FMT == kFour;
    static constexpr int RB = 8 * NQ * WR;                  // rows of a row block
    static constexpr int KW = (F8 || D == 64) ? 32 : 16;    // positions of a warp's part of a tile
    static constexpr int KS = KW * kWarps;                  // positions of a tile
    static constexpr int ROW = F4 ? D / 2 : D * (F8 ? 1 : 2);   // bytes of a cached row
    static constexpr int GROUPS = F4 ? D / kGroup : 0;      // and of its groups' scales
    static constexpr int STAGE = 2 * KS * ROW;              // keys, then values
    // key and value scales, those of the groups, mask words
    static constexpr int AUX = (F8 ? 2 * KS * 4 : 0) + 2 * KS * GROUPS + 16;
    // at an item's end the warps' outputs (f32) meet in the stage of its last tile, or, where
    // they don't fit, in room of their own
    static constexpr int OUTS = kWarps * 8 * NQ * D * 4;
    static constexpr bool APART = OUTS > STAGE;
    // tiles that a CTA has room for
    static constexpr int CTAS = ctas_of(FMT, RB);           // of an SM
    static constexpr int STAGES = !F4 ? 3 : CTAS == 3 ? (D == 64 ? 6 : 3) : D == 64 ? 8 : 4;
    // registers of a thread: as many as the SM has at the launch, shared out again
    static constexpr int REGS = 65536 / (CTAS * kThreads) / 8 * 8;
    static constexpr int COPY_REGS = 48, COMPUTE_REGS = 2 * REGS - COPY_REGS;
    static constexpr int SMEM = STAGES * (STAGE + AUX) + (APART ? OUTS : 0);
    static_assert(F4 || !APART, "the outputs fit a stage");
    static_assert(CTAS * (SMEM + 2048) <= 228 * 1024, "CTAs fit an SM");
};

// Byte offset of 16-byte chunk c of row r: chunks are exchanged so that the
// eight rows of a matrix fragment, and the rows and chunks that eight
// neighbouring lanes read, lie in different banks.
// (Rows of 4-bit codes lie as in a page, so that whole runs are copied at once: the values' reads meet in
// pairs, which costs less than the instructions of copying row by row.)
template <int ROW, bool LINEAR>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if constexpr (LINEAR) return r * ROW + (c << 4);
    if constexpr (ROW == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return r * ROW + ((c ^ (r & 7)) << 4);
}

// With codes, which of a group of 16 positions stands in row 8 j + n of a
// score tile.  Any order does, as long as keys and values follow the same
// one; this one keeps both kinds of reads free of bank conflicts.
template <int ROW>
__device__ __forceinline__ int code_pos(int j, int n) {
    const int c = n >> 1, odd = n & 1;
    if constexpr (ROW == 32) return 8 * j + (odd ? 4 + (c ^ 2) : c);
    if constexpr (ROW == 64) {
        const int even_at = (c & 1) | ((c & 2) << 1);           // 0 1 4 5
        return 8 * j + (odd ? (even_at ^ 3) : even_at);         // 3 2 7 6
    }
    return j + (odd ? 8 + ((2 * c) ^ 4) : 2 * c);
}

// Position r of a tile: its row of the keys (or values), see chunk_at.
template <typename C>
struct Room {
    unsigned char *smem;
    __device__ __forceinline__ uint32_t keys(int st) const { return smem_addr(smem) + st * C::STAGE; }
    __device__ __forceinline__ uint32_t values(int st) const { return keys(st) + C::KS * C::ROW; }
    __device__ __forceinline__ unsigned char *aux(int st) const {
        return smem + C::STAGES * C::STAGE + st * C::AUX;
    }
    // the key scales of a tile, then its value scales
    __device__ __forceinline__ float *scales(int st) const { return reinterpret_cast<float *>(aux(st)); }
    // the scales of the groups of a tile's keys, then of its values
    __device__ __forceinline__ uint32_t groups(int st) const {
        return smem_addr(aux(st)) + 2 * C::KS * 4;
    }
    // where the warps' outputs meet
    __device__ __forceinline__ float *outs(int st) const {
        return reinterpret_cast<float *>(smem + (C::APART ? C::STAGES * (C::STAGE + C::AUX)
                                                          : st * C::STAGE));
    }
    // bit r % KW of word r / KW: position r is there
    __device__ __forceinline__ uint32_t *masks(int st) const {
        return reinterpret_cast<uint32_t *>(aux(st) + C::AUX - 16);
    }
};

// The left operand of the second product from the values at vsm (their groups' scales at
// vgr): output tile by output tile for the 16 positions of score tile j, use(tile, fragment).
template <typename C, typename Use>
__device__ __forceinline__ void value_tiles(uint32_t vsm, uint32_t vgr, int j, Use &&use) {
    constexpr int ROW = C::ROW, D = C::D;
    const int lane = threadIdx.x % 32, g = lane >> 2, c = lane & 3;
    if constexpr (!C::F8) {
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            uint32_t f[4];
            ldsm4_trans(f, vsm + chunk_at<ROW, C::F4>(16 * j + (lane & 7) + ((lane >> 4) << 3),
                                               2 * mt + ((lane >> 3) & 1)));
            use(mt, f);
        }
    } else if constexpr (C::F4) {
        // as below with D / 16 bytes a position: the codes of a place of two positions are put
        // into one byte, its low and its high bits
        constexpr int NW = D / 64;     // words of a position
        uint32_t v[4][NW], s[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int r = 16 * j + code_pos<ROW>(x >> 1, 2 * c + (x & 1));
            if constexpr (D == 128) {
                const uint2 u = lds8(vsm + chunk_at<ROW, C::F4>(r, g >> 1) + (g & 1) * 8);
                v[x][0] = u.x, v[x][1] = u.y;
                s[x] = lds1(vgr + r * C::GROUPS + g);
            } else {
                v[x][0] = lds4(vsm + chunk_at<ROW, C::F4>(r, g >> 2) + (g & 3) * 4);
                s[x] = lds1(vgr + r * C::GROUPS + (g >> 1));
            }
        }
        const uint32_t s01 = widen2(s[0] | s[1] << 8), s23 = widen2(s[2] | s[3] << 8);
#pragma unroll
        for (int q = 0; q < NW; ++q) {
            const uint32_t lo = 0x0f0f0f0fu, hi = 0xf0f0f0f0u;
            uint32_t even01[4], odd01[4], even23[4], odd23[4];
            widen8((v[0][q] & lo) | (v[1][q] << 4 & hi), even01);
            widen8((v[0][q] >> 4 & lo) | (v[1][q] & hi), odd01);
            widen8((v[2][q] & lo) | (v[3][q] << 4 & hi), even23);
            widen8((v[2][q] >> 4 & lo) | (v[3][q] & hi), odd23);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                uint32_t f[4] = {mul_f16(even01[z], s01), mul_f16(odd01[z], s01),
                                 mul_f16(even23[z], s23), mul_f16(odd23[z], s23)};
                use(4 * q + z, f);
            }
        }
    } else {
        // four positions' codes for the D / 8 places from (D / 8) g on;
        // places 2 t and 2 t + 1 of them are rows g and g + 8 of output tile t
        constexpr int NW = D / 32;     // words of a position
        uint32_t v[4][NW];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int r = 16 * j + code_pos<ROW>(x >> 1, 2 * c + (x & 1));
            if constexpr (D == 128) {
                const uint4 u = lds16(vsm + chunk_at<ROW, C::F4>(r, g));
                v[x][0] = u.x, v[x][1] = u.y, v[x][2] = u.z, v[x][3] = u.w;
            } else {
                const uint2 u = lds8(vsm + chunk_at<ROW, C::F4>(r, g >> 1) + (g & 1) * 8);
                v[x][0] = u.x, v[x][1] = u.y;
            }
        }
#pragma unroll
        for (int q = 0; q < NW; ++q)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                // bytes of two positions side by side, place by place
                const uint32_t sel = z ? 0x7362 : 0x5140;
                uint32_t f[4];
                widen4(__byte_perm(v[0][q], v[1][q], sel), f[0], f[1]);
                widen4(__byte_perm(v[2][q], v[3][q], sel), f[2], f[3]);
                use(2 * q + z, f);
            }
    }
}

__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// ln(2^m l).  Codes: the sum's exponent is added to m before anything is rounded, as they may be
// far apart and nearly cancel.
template <bool F8>
__device__ __forceinline__ float log_sum(float m, float l) {
    if (l == 0.f) return -INFINITY;
    if constexpr (!F8) return (m + log2f(l)) * kLn2;
    const uint32_t u = __float_as_uint(l), e = u >> 23;
    if (e == 0 || e >= 255) return (m + log2f(l)) * kLn2;     // subnormal, infinite, NaN (or negative)
    return ((m + (float(e) - 127.f)) + log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u))) * kLn2;
}

// The factor 2^x, x <= 0, of a part's sum and outputs.  Codes: by halves, as a sum may be large
// where its factor is below 2^-126 (in every join: 0.2 us of a short call's 4.5).
template <bool F8>
struct Factor {
    float f;
    __device__ __forceinline__ explicit Factor(float x) : f(ex2(F8 ? 0.5f * x : x)) {}
    __device__ __forceinline__ float sum(float l) const { return F8 ? l * f * f : l * f; }
    __device__ __forceinline__ float out() const { return F8 ? f * f : f; }
};

// Infinities and NaN of a pair of 16-bit values, replaced by 0.
template <bool F16>
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
    const uint32_t top = F16 ? 0x7c00u : 0x7f80u;
    if ((v & top) == top) v &= 0xffff0000u;
    if ((v & (top << 16)) == top << 16) v &= 0xffffu;
    return v;
}

// Waits for a phase of bar; false after two seconds, and at once where some warp of the CTA
// has given up.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    bool done = ptx::mbar_try_wait(bar, parity);
    if (!__all_sync(~0u, done)) {
        const uint64_t t0 = ptx::globaltimer_ns();
#pragma unroll 1
        while (!done && !*gave_up && ptx::globaltimer_ns() - t0 < 2000000000ull)
            done = ptx::mbar_try_wait(bar, parity);
        if (!__all_sync(~0u, done)) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}

// A copying warp: fills KW positions of each stage, from the first-th on, with the
// stretch's tiles, one after another.  full[st] is arrived at by each lane's copies as
// they land and by lane 0 for the mask, empty[st] by each computing warp.
template <typename C>
__device__ __forceinline__ bool copy_tiles(const PagedArgs &a, const Shape &s, const Room<C> room,
                                           uint64_t *full, uint64_t *empty, volatile int *gave_up,
                                           Item it, int tile, int64_t left, int first) {
    constexpr int KS = C::KS, KW = C::KW, ROW = C::ROW, ES = C::F8 ? 1 : 2, STAGES = C::STAGES;
    constexpr int GROUPS = C::GROUPS;
    constexpr int LPR = ROW / 16, RPI = 32 / LPR;           // lanes a row, rows a copy
    constexpr int RUN = 16;
    constexpr uint32_t kAll = 0xffffffffu >> (32 - KW);
    const int lane = threadIdx.x % 32;
    const int lrow = lane / LPR, lch = lane % LPR;
    const int shift = (a.c.ps & (a.c.ps - 1)) ? -1 : __ffs(a.c.ps) - 1;
    // RUN positions of one page after another in memory: no addresses from other lanes
    // (96 ragged sequences over fp8 77.0 us, without this way 79.0; bf16 alike)
    const bool runs = a.c.ps % RUN == 0 && a.c.st == ROW / ES;
    const char *const kpool = static_cast<const char *>(a.c.k);
    const char *const vpool = static_cast<const char *>(a.c.v);

    // Where this lane's position of the next tile lies, looked up a tile early, and the
    // length of the next sequence.
    int page, at;
    int len = a.lens[min(it.b + 1, a.B - 1)];
    auto look_up = [&]() {
        page = -1;
        const int pos = tile_at<KS>(it, tile) + first + lane;
        const int p = shift >= 0 ? pos >> shift : pos / a.c.ps;
        at = pos - p * a.c.ps;
        if (left > 0 && lane < KW && in_range(s, it, pos) &&
            SSD_IDX_OK(a.err, it.b * a.tb + p, a.t_n))
            page = a.table[it.b * a.tb + p];
    };
    look_up();
    for (int n = 0, st = 0; left > 0; ++n, st = st + 1 == STAGES ? 0 : st + 1) {
        if (n >= STAGES && !wait_for(&empty[st], (n / STAGES - 1) & 1, gave_up)) return false;
        const bool ok = page >= 0 && page < a.c.pages;
        const uint32_t mask = __ballot_sync(~0u, ok);
        const int64_t off = ok ? page * a.c.sp + it.hk * a.c.sh + at * a.c.st : 0;
        const uint32_t kdst = room.keys(st) + first * ROW, vdst = room.values(st) + first * ROW;
        if (__all_sync(~0u, runs && mask == kAll)) {
#pragma unroll
            for (int h = 0; h < KW / RUN; ++h) {
                const int64_t mine = __shfl_sync(~0u, off, h * RUN) * ES + lrow * ROW + lch * 16;
#pragma unroll
                for (int j = 0; j < RUN / RPI; ++j) {
                    const uint32_t d = chunk_at<ROW, C::F4>(h * RUN + j * RPI + lrow, lch);
                    const bool in = SSD_IDX_OK(a.err, mine + j * RPI * ROW + 15, a.c.n * ES);
                    copy16(kdst + d, kpool + mine + j * RPI * ROW, in);
                    copy16(vdst + d, vpool + mine + j * RPI * ROW, in);
                }
            }
        } else {
            // zeros where there is no position (a pass may take another warp's along)
#pragma unroll 1
            for (int r0 = 0; r0 < KW; r0 += RPI) {
                const int r = r0 + lrow;
                const int64_t o = __shfl_sync(~0u, off, r) * ES + lch * 16;
                const bool in = (mask >> r) & 1 && SSD_IDX_OK(a.err, o + 15, a.c.n * ES);
                copy16(kdst + chunk_at<ROW, C::F4>(r, lch), kpool + o, in);
                copy16(vdst + chunk_at<ROW, C::F4>(r, lch), vpool + o, in);
            }
        }
        if constexpr (C::F8) {
            const int64_t so = ok ? page * a.c.ssp + it.hk * a.c.ssh + at : 0;
            const uint32_t d = smem_addr(room.scales(st)) + (first + lane) * 4;
            const bool in = ok && SSD_IDX_OK(a.err, so, a.c.ns);
            copy_few<4>(d, a.c.ks + so, in);
            copy_few<4>(d + KS * 4, a.c.vs + so, in);
        }
        if constexpr (C::F4) {
            const int64_t go = ok ? page * a.c.sgp + it.hk * a.c.sgh + at * a.c.sgt : 0;
            const uint32_t d = room.groups(st) + (first + lane) * GROUPS;
            const bool in = ok && SSD_IDX_OK(a.err, go + GROUPS - 1, a.c.ng);
            copy_few<C::F4 ? GROUPS : 4>(d, a.c.kg + go, in);
            copy_few<C::F4 ? GROUPS : 4>(d + KS * GROUPS, a.c.vg + go, in);
        }
        copies_arrive(&full[st]);
        if (lane == 0) {
            room.masks(st)[first / KW] = mask;
            ptx::mbar_arrive(&full[st]);
        }
        --left;
        if (++tile == it.ntiles) {
            tile = 0;
            left -= kItemCost;
            it = next_item<KS>(s, it, len);
            len = a.lens[min(it.b + 1, a.B - 1)];
        }
        look_up();
    }
    return true;
}

// The same for 4-bit codes whose runs of 16 or 32 positions of a page lie in one piece, their scales
// too: a lane copies a run of one kind (codes, groups' scales or scales, of keys or values).  Tiles
// are half the bytes of 8-bit ones while a tile's instructions stay, and copying and computing warps
// share the SM's: a run found and copied takes a third of those of 16 bytes a lane.  Where some
// position is not there, the part is filled a position a lane, with zeros.
template <typename C>
__device__ __forceinline__ bool copy_runs(const PagedArgs &a, const Shape &s, const Room<C> room,
                                          uint64_t *full, uint64_t *empty, volatile int *gave_up,
                                          Item it, int tile, int64_t left, int first) {
    constexpr int KS = C::KS, KW = C::KW, ROW = C::ROW, GROUPS = C::GROUPS, STAGES = C::STAGES;
    constexpr int LPR = ROW / 16, RPI = 32 / LPR;
    static_assert(KW == 32, "");
    const int lane = threadIdx.x % 32;
    const int shift = (a.c.ps & (a.c.ps - 1)) ? -1 : __ffs(a.c.ps) - 1;
    const int run = a.c.ps % 32 == 0 ? 32 : 16, kind = lane % 6, part = lane / 6 * run;
    const bool value = kind & 1, mine = part < KW;
    // in bytes: a kind's page, head and token strides, and its place in a stage
    const char *const base = kind < 2   ? static_cast<const char *>(value ? a.c.v : a.c.k)
                             : kind < 4 ? reinterpret_cast<const char *>(value ? a.c.vg : a.c.kg)
                                        : reinterpret_cast<const char *>(value ? a.c.vs : a.c.ks);
    const int64_t per_page = kind < 2 ? a.c.sp : kind < 4 ? a.c.sgp : a.c.ssp * 4;
    const int64_t per_head = kind < 2 ? a.c.sh : kind < 4 ? a.c.sgh : a.c.ssh * 4;
    const int each = kind < 2 ? ROW : kind < 4 ? GROUPS : 4;
    [[maybe_unused]] const int64_t extent = kind < 2 ? a.c.n : kind < 4 ? a.c.ng : a.c.ns * 4;
    const uint32_t place = (kind < 2 ? room.keys(0) : kind < 4 ? room.groups(0) : smem_addr(room.scales(0))) +
                           (value ? KS * each : 0) + (first + part) * each;
    const uint32_t per_stage = kind < 2 ? C::STAGE : C::AUX;

    int page, at;
    int len = a.lens[min(it.b + 1, a.B - 1)];
    auto page_of = [&](int pos) { return shift >= 0 ? pos >> shift : pos / a.c.ps; };
    auto look_up = [&]() {            // this lane's run of the next tile
        page = -1;
        const int pos = tile_at<KS>(it, tile) + first + part, p = page_of(pos);
        at = pos - p * a.c.ps;
        if (left > 0 && mine && pos + run <= it.hi && (pos >= it.lo || (kSinks && pos + run <= s.sinks)) &&
            SSD_IDX_OK(a.err, it.b * a.tb + p, a.t_n))
            page = a.table[it.b * a.tb + p];
    };
    look_up();
    bool mixed = false;
    uint32_t phase = 1;
#pragma unroll 1
    for (int n = 0, st = 0; left > 0; ++n) {
        if (n >= STAGES && !wait_for(&empty[st], phase, gave_up)) return false;
        const bool ok = page >= 0 && page < a.c.pages;
        if (__all_sync(~0u, ok || !mine)) {
            const int64_t off = page * per_page + it.hk * per_head + at * each;
            const bool in = mine && SSD_IDX_OK(a.err, off + run * each - 1, extent);
            if (lane == 0) {
                room.masks(st)[first / KW] = 0xffffffffu;
                ptx::mbar_arrive_expect_tx(&full[st], 2 * KW * (ROW + GROUPS + 4));
            }
            __syncwarp();
            if (mixed) ptx::fence_proxy_async_smem();    // after copies of the other kind
            if (in) bulk_load(place + st * per_stage, base + off, run * each, &full[st]);
        } else {
            mixed = true;
            const int pos = tile_at<KS>(it, tile) + first + lane, p = page_of(pos), from = pos - p * a.c.ps;
            int pg = -1;
            if (in_range(s, it, pos) && SSD_IDX_OK(a.err, it.b * a.tb + p, a.t_n)) pg = a.table[it.b * a.tb + p];
            const bool there = pg >= 0 && pg < a.c.pages;
            const uint32_t mask = __ballot_sync(~0u, there);
            const int64_t off = there ? pg * a.c.sp + it.hk * a.c.sh + from * a.c.st : 0;
            const uint32_t kdst = room.keys(st) + first * ROW, vdst = room.values(st) + first * ROW;
#pragma unroll 1
            for (int r0 = 0; r0 < KW; r0 += RPI) {
                const int r = r0 + lane / LPR;
                const int64_t o = __shfl_sync(~0u, off, r) + lane % LPR * 16;
                const bool in = (mask >> r) & 1 && SSD_IDX_OK(a.err, o + 15, a.c.n);
                copy16(kdst + chunk_at<ROW, true>(r, lane % LPR), static_cast<const char *>(a.c.k) + o, in);
                copy16(vdst + chunk_at<ROW, true>(r, lane % LPR), static_cast<const char *>(a.c.v) + o, in);
            }
            const int64_t so = there ? pg * a.c.ssp + it.hk * a.c.ssh + from : 0;
            const uint32_t d = smem_addr(room.scales(st)) + (first + lane) * 4;
            bool in = there && SSD_IDX_OK(a.err, so, a.c.ns);
            copy_few<4>(d, a.c.ks + so, in);
            copy_few<4>(d + KS * 4, a.c.vs + so, in);
            const int64_t go = there ? pg * a.c.sgp + it.hk * a.c.sgh + from * a.c.sgt : 0;
            const uint32_t e = room.groups(st) + (first + lane) * GROUPS;
            in = there && SSD_IDX_OK(a.err, go + GROUPS - 1, a.c.ng);
            copy_few<GROUPS>(e, a.c.kg + go, in);
            copy_few<GROUPS>(e + KS * GROUPS, a.c.vg + go, in);
            if (lane == 0) {
                room.masks(st)[first / KW] = mask;
                ptx::mbar_arrive(&full[st]);
            }
        }
        copies_arrive(&full[st]);
        --left;
        if (++tile == it.ntiles) {
            tile = 0;
            left -= kItemCost;
            it = next_item<KS>(s, it, len);
            len = a.lens[min(it.b + 1, a.B - 1)];
        }
        look_up();
        if (++st == STAGES) {
            st = 0;
            phase ^= 1;
        }
    }
    return true;
}

// ASK: the lengths tell whether this kernel works or k_paged_prompt, which is launched between this and the
// join (compiled apart: as a choice at run time it cost the calls that are not asked 4 to 7%).  Where this one
// works (a batch of one of 32768 positions among seven of 100; 12 of 17 to 16384): 95.4 and 67.9 us, with the
// other launched first 96.4 and 68.8, behind the join 96.5 and 68.8, not launched at all 92.9 and 65.6.
template <int D, int FMT, int NQ, int WR, bool ASK>
__global__ void __launch_bounds__(kThreads, (Cfg<D, FMT, NQ, WR>::CTAS))
k_paged_mma(const __grid_constant__ PagedArgs a, const __grid_constant__ Shape s) {
    using C = Cfg<D, FMT, NQ, WR>;
    constexpr bool F8 = C::F8, F4 = C::F4;
    constexpr int STAGES = C::STAGES;
    constexpr int KW = C::KW, KS = C::KS, ROW = C::ROW, WK = C::WK, RB = C::RB;
    constexpr int KP = KW * WR < 32 ? KW * WR : 32;     // positions of a pass over a group's part
    constexpr int KT = KP / 16;           // its score tiles
    constexpr int MT = D / 16;            // output tiles
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ FinderRoom finder;
    __shared__ uint64_t full[STAGES], empty[STAGES];
    __shared__ int gave_up;
    __shared__ float top_of[kWarps][8 * NQ], sum_of[kWarps][8 * NQ];

    let_next_start();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (threadIdx.x == 0) gave_up = 0;
    if (threadIdx.x < STAGES) {
        ptx::mbar_init(&full[threadIdx.x], kCopyWarps * (32 + 1));
        ptx::mbar_init(&empty[threadIdx.x], kWarps);
    }
    __syncthreads();
    if (ASK && prompt_pays(a)) {
        if (threadIdx.x == 0 && cut_ok(a, s, blockIdx.x)) reinterpret_cast<Cut *>(a.ws)[blockIdx.x].parts = 0;
        return;
    }
    const Stretch span = find<KS, kThreads / 32>(s, blockIdx.x, &finder);
    if (threadIdx.x == 0 && cut_ok(a, s, blockIdx.x)) reinterpret_cast<Cut *>(a.ws)[blockIdx.x].parts = 0;
    // A cursor: an item, a tile of it, and the units left; the tiles of an item come
    // after its constant.
    Item it = span.it;
    int tile = max(0, span.unit - kItemCost);
    int64_t left = span.left - max(0, kItemCost - span.unit);
    if (span.left <= 0 || left <= 0) return;
    const Room<C> room{smem};
    static_assert(kCopyWarps == kWarps, "two warpgroups");
    if (warp >= kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::COPY_REGS));
        bool done;
        if constexpr (F4)
            done = a.c.whole ? copy_runs<C>(a, s, room, full, empty, &gave_up, it, tile, left, (warp - kWarps) * KW)
                             : copy_tiles<C>(a, s, room, full, empty, &gave_up, it, tile, left, (warp - kWarps) * KW);
        else
            done = copy_tiles<C>(a, s, room, full, empty, &gave_up, it, tile, left, (warp - kWarps) * KW);
        if (!done) {
            copies_wait();
            if constexpr (F4) {       // pieces under way land in microseconds
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 1000000ull) {}
            }
            if (lane == 0) atomicOr(a.err, kErrTimeout);
        }
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::COMPUTE_REGS));
    const int kg = warp / WR, wr = warp % WR;     // key group, row warp
    const int g = lane >> 2, c = lane & 3;        // fragment row and column pair

    // Per item: the query fragments (row 8 n + g of the warp's), and for the queries
    // 8 n + 2 c + p, which this thread's columns hold, the running maximum, the sum
    // over this thread's positions, and the output.  Scores stay as the product leaves
    // them (times the key's scale): a row's factor qs >= 0 (scale log2(e), the sign of
    // the scale being in the queries) enters with the exponential, p = 2^(qs (s - m)).
    // (The difference first: qs m rounded would be off by any power of two for large scores.)
    // Codes: a weight p vs (vs: the value's scale) goes to fp16, so p = 2^(qs (s - m) - k), where m
    // is some score that the row has seen and k the largest qs (s - m) + log2 vs (less kLift) over
    // the positions that it sees: the largest weight is about 2^kLift, whatever the scales are, and
    // positions that it does not see have no part in it.  m and k follow, together, when
    // a weight may be ahead by kAhead, since moving them means to go over the outputs.
    // p, summed in fp32, may be as large as 2^(kLift + kAhead - kLeastLog) and as small as 2^-kMostLog.
    uint32_t qf[NQ][D / 16][2];
    float o[MT][NQ][4], m[NQ][2], l[NQ][2], qs[NQ][2], k[NQ][2];
    int e[NQ][2];                         // the rows' own places
    const float qscale = fabsf(a.scale) * kLog2e;
    const uint32_t qsign = a.scale < 0.f ? 0x80008000u : 0u;
    const int rows = a.T * s.G;
    auto load_queries = [&]() {           // of the item at `it`, used once `fresh` is seen
#pragma unroll
        for (int b = 0; b < NQ; ++b) {
            const int r = min(it.rb * RB + wr * 8 * NQ + 8 * b + g, rows - 1), t = token_of(s, r);
            const int64_t off = it.b * a.q_sb + t * a.q_st + (it.hk * s.G + r - t * s.G) * a.q_sh;
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) +
                                     (SSD_IDX_OK(a.err, off + D - 1, a.q_n) ? off : 0);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                if constexpr (F8) {       // places 64 h + 16 c + 4 (k % 4), or D / 4 c + 4 k
                    const uint2 u = *reinterpret_cast<const uint2 *>(
                        q + (F4 ? D / 4 * c + 4 * k : (k / 4) * 64 + 16 * c + 4 * (k % 4)));
                    qf[b][k][0] = u.x;
                    qf[b][k][1] = u.y;
                } else {
                    qf[b][k][0] = *reinterpret_cast<const uint32_t *>(q + 16 * k + 2 * c);
                    qf[b][k][1] = *reinterpret_cast<const uint32_t *>(q + 16 * k + 8 + 2 * c);
                }
            }
        }
    };
    load_queries();
    bool fresh = true;
    const int tile_first = tile;          // of the first item; later ones begin at 0
    bool first_item = true;

    uint32_t phase = 0;
    auto next_stage = [&](int &st) {
        if (++st == STAGES) {
            st = 0;
            phase ^= 1;
        }
    };
    for (int st = 0; left > 0; next_stage(st)) {
        if (fresh) {
            fresh = false;
#pragma unroll
            for (int b = 0; b < NQ; ++b) {
                float factor = qscale;
                if constexpr (!F8) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i) qf[b][k][i] ^= qsign;
                } else {
                    // fp16 for the product with widened codes: the row is scaled by a
                    // power of two that brings its largest value to [1, 2) (to [2, 4) from
                    // 2^127 on, the inverse being a normal number), so all but values 2^-14
                    // times as large stay exact
                    float top = 0.f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[b][k][i] << 16)),
                                                   fabsf(__uint_as_float(qf[b][k][i] & 0xffff0000u))));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    uint32_t ex = __float_as_uint(top) & 0x7f800000u;
                    ex = ex == 0 ? 0x3f800000u : min(ex, 0x7e800000u);
                    const float down = __uint_as_float(0x7f000000u - ex);
                    factor *= __uint_as_float(ex);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            qf[b][k][i] = pack_f16(__uint_as_float(qf[b][k][i] << 16) * down,
                                                   __uint_as_float(qf[b][k][i] & 0xffff0000u) * down) ^
                                          qsign;
                }
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const int row = it.rb * RB + wr * 8 * NQ + 8 * b + 2 * c + p;
                    qs[b][p] = F8 ? __shfl_sync(~0u, factor, (2 * c + p) * 4) : qscale;
                    e[b][p] = it.len - a.T + token_of(s, min(row, rows - 1));
                    m[b][p] = F8 ? 0.f : -INFINITY;
                    k[b][p] = -INFINITY;
                    l[b][p] = 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int b = 0; b < NQ; ++b) o[j][b][0] = o[j][b][1] = o[j][b][2] = o[j][b][3] = 0.f;
        }
        // A warp whose wait ran out goes on without waiting, over whatever the stages hold:
        // others may have seen the same copies land, and would wait for it at the barriers
        // below for ever.
        if (!wait_for(&full[st], phase, &gave_up) && lane == 0) atomicOr(a.err, kErrTimeout);
        const int kbase = tile_at<KS>(it, tile) + kg * WR * KW;
#pragma unroll 1
        for (int sub = 0; sub < KW * WR / KP; ++sub) {
            const int x0 = kg * WR * KW + sub * KP, k0 = kbase + sub * KP;   // the pass's first position
            uint32_t mask = room.masks(st)[x0 / KW];
            if constexpr (KP > KW) mask |= room.masks(st)[x0 / KW + 1] << KW;
            // (votes, so that the compiler knows these for the same in all lanes)
            if (!__any_sync(~0u, mask != 0)) continue;
            // partial: rows of the block see different positions of the pass
            const bool partial = __any_sync(~0u, it.emin != it.emax &&
                                                     (k0 + KP - 1 > it.emin ||
                                                      (s.window > 0 && k0 <= it.emax - s.window &&
                                                       (!kSinks || k0 + KP > s.sinks))));
            const bool all = __all_sync(~0u, !partial && mask == 0xffffffffu >> (32 - KP));
            const uint32_t ksm = room.keys(st) + x0 * ROW, vsm = room.values(st) + x0 * ROW;
            const float *ksc = room.scales(st) + x0, *vsc = ksc + KS;
            [[maybe_unused]] const uint32_t kgr = room.groups(st) + x0 * C::GROUPS, vgr = kgr + KS * C::GROUPS;
            // row g + 8 i of score tile j is position pos_of(j, i) of the pass
            auto pos_of = [&](int j, int i) {
                return 16 * j + (F8 ? code_pos<ROW>(i, g) : g + 8 * i);
            };

            // scores: KP positions x 8 NQ queries
            float sc[KT][NQ][4];
#pragma unroll
            for (int j = 0; j < KT; ++j)
#pragma unroll
                for (int b = 0; b < NQ; ++b)
                    sc[j][b][0] = sc[j][b][1] = sc[j][b][2] = sc[j][b][3] = 0.f;
            if constexpr (!F8) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int j = 0; j < KT; ++j) {
                        uint32_t f[4];
                        ldsm4(f, ksm + chunk_at<ROW, C::F4>(16 * j + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
                        for (int b = 0; b < NQ; ++b)
                            mma<false>(sc[j][b], f, qf[b][k][0], qf[b][k][1]);
                    }
            } else if constexpr (F4) {
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    // D / 4 places of two positions: all steps of the product, a group each
                    // four of them
                    constexpr int NW = D / 32;
                    uint32_t u[2][NW], gs[2][2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = pos_of(j, i);
                        if constexpr (D == 128) {
                            const uint4 v = lds16(ksm + chunk_at<ROW, C::F4>(r, c));
                            u[i][0] = v.x, u[i][1] = v.y, u[i][2] = v.z, u[i][3] = v.w;
                            const uint32_t w = widen2(lds2(kgr + r * C::GROUPS + 2 * c));
                            gs[i][0] = __byte_perm(w, w, 0x1010);
                            gs[i][1] = __byte_perm(w, w, 0x3232);
                        } else {
                            const uint2 v = lds8(ksm + chunk_at<ROW, C::F4>(r, c >> 1) + (c & 1) * 8);
                            u[i][0] = v.x, u[i][1] = v.y;
                            const uint32_t w = widen2(lds1(kgr + r * C::GROUPS + c));
                            gs[i][0] = gs[i][1] = __byte_perm(w, w, 0x1010);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < NW; ++k) {
                        uint32_t h[2][4];
                        widen8(u[0][k], h[0]);
                        widen8(u[1][k], h[1]);
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t s0 = gs[0][k / 2], s1 = gs[1][k / 2];
                            uint32_t f[4] = {mul_f16(h[0][2 * z], s0), mul_f16(h[1][2 * z], s1),
                                             mul_f16(h[0][2 * z + 1], s0), mul_f16(h[1][2 * z + 1], s1)};
#pragma unroll
                            for (int b = 0; b < NQ; ++b)
                                mma<true>(sc[j][b], f, qf[b][2 * k + z][0], qf[b][2 * k + z][1]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
#pragma unroll
                    for (int j = 0; j < KT; ++j) {
                        // 16 places of two positions: four steps of the product
                        const uint4 u = lds16(ksm + chunk_at<ROW, C::F4>(pos_of(j, 0), 4 * h + c));
                        const uint4 v = lds16(ksm + chunk_at<ROW, C::F4>(pos_of(j, 1), 4 * h + c));
                        const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t f[4];
                            widen4(uu[k], f[0], f[2]);
                            widen4(vv[k], f[1], f[3]);
#pragma unroll
                            for (int b = 0; b < NQ; ++b)
                                mma<true>(sc[j][b], f, qf[b][4 * h + k][0], qf[b][4 * h + k][1]);
                        }
                    }
            }
            if constexpr (F8) {
#pragma unroll
                for (int j = 0; j < KT; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float f = ksc[pos_of(j, i)];
#pragma unroll
                        for (int b = 0; b < NQ; ++b) {
                            sc[j][b][2 * i] *= f;
                            sc[j][b][2 * i + 1] *= f;
                        }
                    }
            }
            // Masks, where some position is missing or not every row sees every one: a bit
            // of vis for each of this thread's scores, in their order.
            uint32_t vis = 0;
            if (!all) {
#pragma unroll
                for (int j = 0; j < KT; ++j)
#pragma unroll
                    for (int b = 0; b < NQ; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int x = pos_of(j, i >> 1);
                            const bool see = (mask >> x) & 1 && sees(s, e[b][i & 1], k0 + x);
                            vis |= uint32_t(see) << ((j * NQ + b) * 4 + i);
                            if (!see) sc[j][b][i] = -INFINITY;
                        }
            }
            float mn[NQ][2];                 // this thread's largest scores
#pragma unroll
            for (int b = 0; b < NQ; ++b)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    float v = F8 ? -INFINITY : m[b][p];
#pragma unroll
                    for (int j = 0; j < KT; ++j) v = fmaxf(v, fmaxf(sc[j][b][p], sc[j][b][2 + p]));
                    mn[b][p] = v;
                }
            auto row_max = [](float v) {     // over the lanes that hold the row
                v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
                v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
                return fmaxf(v, __shfl_xor_sync(~0u, v, 16));
            };
            bool moved = false;
            float vs[KT][2], f[NQ][2];       // codes: value scales; what the outputs are multiplied by
            if constexpr (F8) {
                float lv[KT][2], most = -INFINITY;
                auto log_scale = [](float v) { return fminf(fmaxf(lg2(fabsf(v)), kLeastLog), kMostLog) - kLift; };
#pragma unroll
                for (int j = 0; j < KT; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        vs[j][i] = vsc[pos_of(j, i)];
                        if constexpr (F4) {           // the largest first, its log then
                            most = fmaxf(most, fabsf(vs[j][i]));
                        } else {
                            lv[j][i] = log_scale(vs[j][i]);
                            most = fmaxf(most, lv[j][i]);
                        }
                    }
                if constexpr (F4) most = log_scale(most);
                // the largest score with the largest scale: mostly no weight is ahead of that bound
#pragma unroll
                for (int b = 0; b < NQ; ++b)
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        moved = moved || fmaf(mn[b][p] - m[b][p], qs[b][p], most) > k[b][p] + kAhead;
                moved = __any_sync(~0u, moved);
                if (moved) {
                    if constexpr (F4) {
#pragma unroll
                        for (int j = 0; j < KT; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i) lv[j][i] = log_scale(vs[j][i]);
                    }
#pragma unroll
                    for (int b = 0; b < NQ; ++b)
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const float top = row_max(mn[b][p]);
                            const bool none = k[b][p] == -INFINITY;      // nothing seen before
                            const float to = top == -INFINITY ? m[b][p] : none ? top : fmaxf(m[b][p], top);
                            const float was = none ? k[b][p] : fmaf(m[b][p] - to, qs[b][p], k[b][p]);
                            float v = was;
#pragma unroll
                            for (int j = 0; j < KT; ++j)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    v = fmaxf(v, fmaf(sc[j][b][2 * i + p] - to, qs[b][p], lv[j][i]));
                            v = row_max(v);
                            const Factor<true> old(was == -INFINITY ? was : was - v);
                            f[b][p] = old.out();
                            l[b][p] = old.sum(l[b][p]);
                            m[b][p] = to;
                            k[b][p] = v;
                        }
                }
            } else {
#pragma unroll
                for (int b = 0; b < NQ; ++b)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        mn[b][p] = row_max(mn[b][p]);
                        moved = moved || mn[b][p] != m[b][p];
                    }
                moved = __any_sync(~0u, moved);
                if (moved) {
#pragma unroll
                    for (int b = 0; b < NQ; ++b)
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            f[b][p] = m[b][p] == -INFINITY ? 0.f : ex2((m[b][p] - mn[b][p]) * qs[b][p]);
                            m[b][p] = mn[b][p];
                            l[b][p] *= f[b][p];
                        }
                }
            }
            if (moved) {
#pragma unroll
                for (int b = 0; b < NQ; ++b)
#pragma unroll
                    for (int j = 0; j < MT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[j][b][i] *= f[b][i & 1];
            }
            // probabilities (unnormalised; at most 1, with codes after their values' scales at most
            // 2^(kLift + kAhead)), summed in fp32 and rounded to 16 bits as the right operand of the
            // second product: its type is that of the values (bf16, or fp16 for codes).  (A second
            // bf16 product with what the rounding leaves costs nothing at 8 and 16 rows of 64 x
            // 4096, but 175 -> 189 us at 32, 265 -> 329 at 64 and 23.0 -> 24.7 for 128 short
            // sequences; the output, bf16 too, is off by 2.1e-3 as it is, 1.7e-3 by its own rounding.)
#pragma unroll
            for (int b = 0; b < NQ; ++b) {
                auto less = [](const float (&x)[2]) {     // two rows' references, to be added
                    return f2(x[0] == -INFINITY ? 0.f : -x[0], x[1] == -INFINITY ? 0.f : -x[1]);
                };
                const F2 q = f2(qs[b][0], qs[b][1]), z = less(m[b]);
                F2 zk;
                if constexpr (F8) zk = less(k[b]);
#pragma unroll
                for (int j = 0; j < KT; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const F2 d = add(f2(sc[j][b][2 * i], sc[j][b][2 * i + 1]), z);
                        float2 x;
                        if constexpr (F8) x = parts(fma(d, q, zk));
                        else x = parts(mul(d, q));
                        sc[j][b][2 * i] = ex2(x.x);
                        sc[j][b][2 * i + 1] = ex2(x.y);
                    }
            }
            auto blank = [&]() {      // what a row does not see
#pragma unroll
                for (int j = 0; j < KT; ++j)
#pragma unroll
                    for (int b = 0; b < NQ; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!((vis >> ((j * NQ + b) * 4 + i)) & 1)) sc[j][b][i] = 0.f;
            };
            if (!all) blank();
#pragma unroll
            for (int j = 0; j < KT; ++j)
#pragma unroll
                for (int b = 0; b < NQ; ++b) {
                    l[b][0] += sc[j][b][0] + sc[j][b][2];
                    l[b][1] += sc[j][b][1] + sc[j][b][3];
                }
            if constexpr (F8) {
#pragma unroll
                for (int j = 0; j < KT; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int b = 0; b < NQ; ++b) {
                            sc[j][b][2 * i] *= vs[j][i];
                            sc[j][b][2 * i + 1] *= vs[j][i];
                        }
                if (!all) blank();    // (whatever its scale is)
            }
            uint32_t pf[KT][NQ][2];   // transposed: query g, positions 2 c and 2 c + 1
#pragma unroll
            for (int j = 0; j < KT; ++j)
#pragma unroll
                for (int b = 0; b < NQ; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        pf[j][b][i] = transpose8(F8 ? pack_f16(sc[j][b][2 * i], sc[j][b][2 * i + 1])
                                                    : pack_bf16(sc[j][b][2 * i], sc[j][b][2 * i + 1]));

            // Where rows of one warp see different positions, an infinity or NaN that one
            // row does not see must not meet its zero probability in the product.  A tile
            // that holds one (the values are looked through first) goes into the product
            // with zeros in their place, after they were added to the rows that see them
            // (a probability makes no difference to an infinity or NaN).
            bool foul = false;
            if (partial) {
                // (4-bit codes are finite, their groups' scales may be NaN)
                constexpr int SPAN = KP * (F4 ? C::GROUPS : ROW) / 16;
#pragma unroll 1
                for (int x = 0; x < (SPAN + 31) / 32; ++x) {
                    if (SPAN % 32 && x * 32 + lane >= SPAN) continue;
                    const uint4 u = lds16((F4 ? vgr : vsm) + (x * 32 + lane) * 16);
                    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        foul |= F8 ? (((v[y] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0
                                   : (v[y] & 0x7f80u) == 0x7f80u || (v[y] & 0x7f800000u) == 0x7f800000u;
                }
                foul = __any_sync(~0u, foul);
            }
            if (!foul) {
#pragma unroll
                for (int j = 0; j < KT; ++j)
                    value_tiles<C>(vsm, vgr, j, [&](int mt, uint32_t (&f)[4]) {
#pragma unroll
                        for (int b = 0; b < NQ; ++b) mma<F8>(o[mt][b], f, pf[j][b][0], pf[j][b][1]);
                    });
            } else {
#pragma unroll 1
                for (int y = 0; y < KP * (D / 32); ++y) {
                    const int x = y / (D / 32), mine = 32 * (y % (D / 32)) + lane;   // position, place
                    const uint32_t at = F4 ? vgr + x * C::GROUPS + mine / kGroup
                                           : vsm + chunk_at<ROW, C::F4>(x, mine * (F8 ? 1 : 2) / 16) +
                                                 mine * (F8 ? 1 : 2) % 16;
                    float v;
                    if constexpr (F8) v = (lds1(at) & 0x7f) == 0x7f ? NAN : 0.f;
                    else v = __uint_as_float(lds2(at) << 16);
                    for (uint32_t bad = __ballot_sync(~0u, !isfinite(v)); bad; bad &= bad - 1) {
                        const int from = __ffs(bad) - 1, d = 32 * (y % (D / 32)) + from;
                        const float add = __shfl_sync(~0u, v, from);
                        // place d is row dr of output tile dt, in the lanes of group dg
                        const int dg = F8 ? d / (D / 8) : d % 8;
                        const int half = F8 ? d % 2 : d / 8 % 2, dt = F8 ? d % (D / 8) / 2 : d / 16;
                        bool see[NQ][2];
#pragma unroll
                        for (int b = 0; b < NQ; ++b)
#pragma unroll
                            for (int p = 0; p < 2; ++p) see[b][p] = g == dg && sees(s, e[b][p], k0 + x);
#pragma unroll
                        for (int j = 0; j < MT; ++j)
#pragma unroll
                            for (int b = 0; b < NQ; ++b)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (j == dt && i >> 1 == half && see[b][i & 1]) o[j][b][i] += add;
                    }
                }
#pragma unroll
                for (int j = 0; j < KT; ++j)
                    value_tiles<C>(vsm, vgr, j, [&](int mt, uint32_t (&f)[4]) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[i] = finite2<F8>(f[i]);
#pragma unroll
                        for (int b = 0; b < NQ; ++b) mma<F8>(o[mt][b], f, pf[j][b][0], pf[j][b][1]);
                    });
            }
        }
        --left;
        const bool item_end = ++tile == it.ntiles;
        if (!item_end && left > 0) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&empty[st]);
            continue;
        }

        // The item's last tile, or the stretch's.  The next item's queries are loaded
        // while this one is joined: each warp puts its output, maxima (in log2 units) and
        // sums into this tile's stage, and takes every fourth row from there.
        const Item done = it;
        const int tiles_left = it.ntiles - tile;
        if (item_end) {
            tile = 0;
            left -= kItemCost;
            fresh = true;
            it = next_item<KS>(s, it, a.lens[min(it.b + 1, a.B - 1)]);
            if (left > 0) load_queries();
        }
        warps_sync();
        // place d of row r: turned by 4 r places, so that neither side meets in one bank
        float *const outs = room.outs(st);
        auto spot = [&](int w, int r, int d) { return (w * 8 * NQ + r) * D + ((d + 4 * r) & (D - 1)); };
#pragma unroll
        for (int b = 0; b < NQ; ++b)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int r = 8 * b + 2 * c + p;
#pragma unroll
                for (int q = 4; q < 32; q <<= 1) l[b][p] += __shfl_xor_sync(~0u, l[b][p], q);
                if (g == 0) {
                    top_of[warp][r] = (F8 ? k[b][p] : m[b][p]) == -INFINITY ? -INFINITY
                                      : F8 ? fmaf(m[b][p], qs[b][p], k[b][p])
                                           : m[b][p] * qs[b][p];
                    sum_of[warp][r] = l[b][p];
                }
                if constexpr (F8) {      // places (D / 8) g + 2 j + i
#pragma unroll
                    for (int j = 0; j < MT; j += 2)
                        if (SSD_IDX_OK(a.err, spot(warp, r, (D / 8) * g + 2 * j) + 3, C::OUTS / 4))
                            *reinterpret_cast<float4 *>(outs + spot(warp, r, (D / 8) * g + 2 * j)) =
                            make_float4(o[j][b][p], o[j][b][2 + p], o[j + 1][b][p], o[j + 1][b][2 + p]);
                } else {                 // places 16 j + 8 i + g
#pragma unroll
                    for (int j = 0; j < MT; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (SSD_IDX_OK(a.err, spot(warp, r, 16 * j + 8 * i + g), C::OUTS / 4))
                                outs[spot(warp, r, 16 * j + 8 * i + g)] = o[j][b][2 * i + p];
                }
            }
        warps_sync();
        const bool whole = item_end && (first_item ? tile_first == 0 : true);
        float *const part = part_at(a, s, 2 * blockIdx.x + (first_item ? 0 : 1));
        if (threadIdx.x == 0 && !whole && !(first_item && tile_first > 0)) {
            // this CTA has the item's first tiles, others the last
            const int64_t t1 = span.beg + span.left + tiles_left;
            Cut cut;
            cut.parts = int(divide(t1 + span.part - 1, span.part)) - int(blockIdx.x);
            cut.first = first_item ? 0 : 1;
            cut.b = done.b;
            cut.hk = done.hk;
            cut.rb = done.rb;
            if (cut_ok(a, s, blockIdx.x)) reinterpret_cast<Cut *>(a.ws)[blockIdx.x] = cut;
        }
#pragma unroll 1
        for (int rr = warp; rr < min(RB, rows - done.rb * RB); rr += kWarps) {
            constexpr int E = D / 32;                           // places of a lane: one vector
            using Vec = std::conditional_t<E == 4, float4, float2>;
            union Places {
                Vec x;
                float f[E];
            };
            const int w0 = rr / (8 * NQ), r = rr % (8 * NQ);    // the row's warp of the first group
            float mt = -INFINITY, lt = 0.f;
            Places v;
#pragma unroll
            for (int k = 0; k < WK; ++k) mt = fmaxf(mt, top_of[k * WR + w0][r]);
            const float base = mt == -INFINITY ? 0.f : mt;
#pragma unroll
            for (int i = 0; i < E; ++i) v.f[i] = 0.f;
#pragma unroll
            for (int k = 0; k < WK; ++k) {
                const Factor<F8> f(top_of[k * WR + w0][r] - base);
                Places src;
                src.x = *reinterpret_cast<const Vec *>(outs + spot(k * WR + w0, r, E * lane));
                lt += f.sum(sum_of[k * WR + w0][r]);
#pragma unroll
                for (int i = 0; i < E; ++i) v.f[i] = fmaf(src.f[i], f.out(), v.f[i]);
            }
            if (whole) {
                const int row = done.rb * RB + rr, t = token_of(s, row), h = done.hk * s.G + row - t * s.G;
                const float inv = lt == 0.f ? 0.f : 1.f / lt;
                const int64_t off = done.b * a.o_sb + t * a.o_st + h * a.o_sh + E * lane;
                if (!SSD_IDX_OK(a.err, off + E - 1, a.o_n)) continue;
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + off;
                if constexpr (E == 4)
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(v.f[0] * inv, v.f[1] * inv),
                                                                 pack_bf16(v.f[2] * inv, v.f[3] * inv));
                else
                    *reinterpret_cast<uint32_t *>(dst) = pack_bf16(v.f[0] * inv, v.f[1] * inv);
                const int64_t at = (int64_t(done.b) * a.T + t) * a.Hq + h;
                if (a.lse && lane == 0 && lse_ok(a, at)) a.lse[at] = log_sum<F8>(mt, lt);
            } else if (part_ok(a, s, 2 * blockIdx.x + (first_item ? 0 : 1), rr)) {
                *reinterpret_cast<Vec *>(part + rr * D + E * lane) = v.x;
                if (lane == 0) {
                    part[RB * D + rr] = mt;
                    part[RB * (D + 1) + rr] = lt;
                }
            }
        }
        if constexpr (F4 && !C::APART) ptx::fence_proxy_async_smem();    // outputs, then copies in pieces
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&empty[st]);
        if (item_end) first_item = false;
    }
}

// ---- the join -------------------------------------------------------------------------
//
// CTA (x, y): rows of the item whose first part CTA x left, `per` of the CTA's four
// warps to a row (each every per-th part), 4 / per rows at a time, gridDim.y of
// them apart.  A CTA for every row of a wide block would mostly be CTAs that find
// nothing to do (32 rows: 9 us in place of 4).
constexpr int kJoinAhead = 8;     // parts that a warp loads at once
template <typename T, int D, bool F8>
__global__ void __launch_bounds__(128)
k_paged_join(const __grid_constant__ PagedArgs a, const __grid_constant__ Shape s, int per) {
    constexpr int E = D / 32;
    __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, x = blockIdx.x;
    wait_for_previous();
    if (!cut_ok(a, s, x)) return;
    const Cut it = reinterpret_cast<const Cut *>(a.ws)[x];
    if (it.parts == 0) return;
    const int rows = min(s.RB, a.T * s.G - it.rb * s.RB);
    for (int r0 = blockIdx.y * (4 / per); r0 < rows; r0 += gridDim.y * (4 / per)) {
        const int rr = min(r0 + warp / per, rows - 1);
        float m = -INFINITY, l = 0.f, o[E] = {};
#pragma unroll 1
        for (int c0 = warp % per; c0 < it.parts; c0 += per * kJoinAhead) {
            float v[kJoinAhead][E], pm[kJoinAhead], pl[kJoinAhead];
#pragma unroll
            for (int u = 0; u < kJoinAhead; ++u) {
                const int c = c0 + per * u;
                pm[u] = -INFINITY;
                pl[u] = 0.f;
                if (c < it.parts && part_ok(a, s, 2 * (x + c) + (c == 0 ? it.first : 0), rr)) {
                    const float *part = part_at(a, s, 2 * (x + c) + (c == 0 ? it.first : 0));
                    pm[u] = part[s.RB * D + rr];
                    pl[u] = part[s.RB * (D + 1) + rr];
#pragma unroll
                    for (int j = 0; j < E; ++j) v[u][j] = part[rr * D + lane * E + j];
                } else {
#pragma unroll
                    for (int j = 0; j < E; ++j) v[u][j] = 0.f;
                }
            }
            float mt = m;
#pragma unroll
            for (int u = 0; u < kJoinAhead; ++u) mt = fmaxf(mt, pm[u]);
            const float base = mt == -INFINITY ? 0.f : mt;
            const Factor<F8> old(m - base);
            m = mt;
            l = old.sum(l);
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] *= old.out();
#pragma unroll
            for (int u = 0; u < kJoinAhead; ++u) {
                const Factor<F8> f(pm[u] - base);
                l += f.sum(pl[u]);
#pragma unroll
                for (int j = 0; j < E; ++j) o[j] = fmaf(v[u][j], f.out(), o[j]);
            }
        }
        __syncthreads();          // the rows before have been read
        if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
        for (int j = 0; j < E; ++j) sm_o[warp][lane * E + j] = o[j];
        __syncthreads();
        if (warp % per || r0 + warp / per >= rows) continue;
        float mt = m;
        for (int w = 1; w < per; ++w) mt = fmaxf(mt, sm_m[warp + w]);
        const float base = mt == -INFINITY ? 0.f : mt;
        l = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = 0.f;
        for (int w = 0; w < per; ++w) {
            const Factor<F8> f(sm_m[warp + w] - base);
            l += f.sum(sm_l[warp + w]);
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] = fmaf(sm_o[warp + w][lane * E + j], f.out(), o[j]);
        }
        const int r = it.rb * s.RB + rr, t = token_of(s, r), h = it.hk * s.G + r - t * s.G;
        const int64_t off = it.b * a.o_sb + t * a.o_st + h * a.o_sh + lane * E;
        if (!SSD_IDX_OK(a.err, off + E - 1, a.o_n)) continue;
        T *dst = static_cast<T *>(a.out) + off;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int j = 0; j < E; ++j) dst[j] = T(o[j] * inv);
        const int64_t at = (int64_t(it.b) * a.T + t) * a.Hq + h;
        if (a.lse && lane == 0 && lse_ok(a, at)) a.lse[at] = log_sum<F8>(mt, l);
    }
}

// ---- fp32 -------------------------------------------------------------------------------
//
// The same line, cuts and join, with products on the CUDA cores (tensor cores would
// round the operands).  D / 16 lanes take a position, six warps of a CTA 512 / D
// positions of a tile each: a lane holds 16 places of its position's key and value,
// loaded straight into registers a tile ahead, and of the outputs of NR rows.  The
// lanes of a position keep maxima and sums of their own, so nothing but parts of
// scores crosses lanes until an item ends.  (More places a lane leave room for fewer
// rows, and rows of another block read the cache again.)
//
// The maximum in use follows the true one when that is ahead by kSlack (log2 units:
// probabilities reach 2^kSlack until then), not at every new one, since moving it means
// to go over the outputs.
constexpr float kSlack = 8.f;
template <int D, int NR>
__global__ void __launch_bounds__(32 * kF32Warps, kCtasPerSm)
k_paged_f32(const __grid_constant__ PagedArgs a, const __grid_constant__ Shape s) {
    constexpr int LP = D / 16, PW = 32 / LP;     // lanes of a position, positions of a warp
    constexpr int V = 4;                         // float4 of a lane
    constexpr int KS = PW * kF32Warps;
    __shared__ FinderRoom finder;
    __shared__ __align__(16) float qsm[NR][D];   // queries times scale log2(e)
    __shared__ __align__(16) float outs[kF32Warps][NR][D];
    __shared__ float top_of[kF32Warps][NR], sum_of[kF32Warps][NR];
    let_next_start();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int at_pos = lane / LP, at_place = 4 * (lane % LP);   // places at_place + 4 LP i ..
    const Stretch span = find<KS, kF32Warps>(s, blockIdx.x, &finder);
    if (threadIdx.x == 0 && cut_ok(a, s, blockIdx.x)) reinterpret_cast<Cut *>(a.ws)[blockIdx.x].parts = 0;
    Item it = span.it;
    int tile = max(0, span.unit - kItemCost);
    int64_t left = span.left - max(0, kItemCost - span.unit);
    if (span.left <= 0 || left <= 0) return;
    const int rows = a.T * s.G;

    // the second cursor: the tile whose page is looked up, then loaded
    Item ld = it;
    int ld_tile = tile, page = -1, at = 0;
    int64_t ld_left = left;
    auto look_up = [&]() {
        page = -1;
        const int pos = tile_at<KS>(ld, ld_tile) + warp * PW + at_pos;
        const int p = pos / a.c.ps;
        at = pos - p * a.c.ps;
        if (ld_left > 0 && in_range(s, ld, pos) && SSD_IDX_OK(a.err, ld.b * a.tb + p, a.t_n))
            page = a.table[ld.b * a.tb + p];
    };
    float4 nk[V], nv[V];
    bool nthere = false;
    auto load = [&]() {
        const int64_t off = page * a.c.sp + ld.hk * a.c.sh + at * a.c.st;
        nthere = page >= 0 && page < a.c.pages && SSD_IDX_OK(a.err, off + D - 1, a.c.n);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            nk[i] = nv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (nthere) {
                const int64_t o = off + 4 * LP * i + at_place;
                nk[i] = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(a.c.k) + o));
                nv[i] = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(a.c.v) + o));
            }
        }
        --ld_left;
        if (++ld_tile == ld.ntiles) {
            ld_tile = 0;
            ld_left -= kItemCost;
            ld = next_item<KS>(s, ld, a.lens[min(ld.b + 1, a.B - 1)]);
        }
        look_up();
    };
    look_up();
    load();

    F2 o[NR][V][2];
    float m[NR], l[NR];
    int e[NR];
    bool fresh = true, first_item = true;
    const int tile_first = tile;
    while (left > 0) {
        if (fresh) {
            fresh = false;
            __syncthreads();
            for (int i = threadIdx.x; i < NR * D; i += 32 * kF32Warps) {
                const int r = min(it.rb * NR + i / D, rows - 1), t = token_of(s, r);
                const int64_t off = it.b * a.q_sb + t * a.q_st + (it.hk * s.G + r - t * s.G) * a.q_sh + i % D;
                const float q = SSD_IDX_OK(a.err, off, a.q_n) ? static_cast<const float *>(a.q)[off] : 0.f;
                qsm[i / D][i % D] = q * (a.scale * kLog2e);
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                e[r] = it.len - a.T + token_of(s, min(it.rb * NR + r, rows - 1));
                m[r] = -INFINITY;
                l[r] = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) o[r][i][0] = o[r][i][1] = f2(0.f, 0.f);
            }
        }
        F2 k[V][2], v[V][2];
        const bool there = nthere;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            k[i][0] = f2(nk[i].x, nk[i].y), k[i][1] = f2(nk[i].z, nk[i].w);
            v[i][0] = f2(nv[i].x, nv[i].y), v[i][1] = f2(nv[i].z, nv[i].w);
        }
        const int pos = tile_at<KS>(it, tile) + warp * PW + at_pos;
        if (left > 1) load();
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            F2 sum = f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 q = *reinterpret_cast<const float4 *>(&qsm[r][4 * LP * i + at_place]);
                sum = fma(f2(q.x, q.y), k[i][0], fma(f2(q.z, q.w), k[i][1], sum));
            }
            float sc = parts(sum).x + parts(sum).y;
#pragma unroll
            for (int w = 1; w < LP; w <<= 1) sc += __shfl_xor_sync(~0u, sc, w);
            if (there && sees(s, e[r], pos)) {
                if (sc - m[r] > kSlack || (m[r] == -INFINITY && sc != m[r])) {
                    const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - sc);
                    const F2 ff = f2(f, f);
                    m[r] = sc;
                    l[r] *= f;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        o[r][i][0] = mul(o[r][i][0], ff);
                        o[r][i][1] = mul(o[r][i][1], ff);
                    }
                }
                const float p = ex2(sc - (m[r] == -INFINITY ? 0.f : m[r]));
                const F2 pp = f2(p, p);
                l[r] += p;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    o[r][i][0] = fma(pp, v[i][0], o[r][i][0]);
                    o[r][i][1] = fma(pp, v[i][1], o[r][i][1]);
                }
            }
        }
        --left;
        const bool item_end = ++tile == it.ntiles;
        if (!item_end && left > 0) continue;

        // join the positions of each warp, then the warps
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float mt = m[r];
#pragma unroll
            for (int w = LP; w < 32; w <<= 1) mt = fmaxf(mt, __shfl_xor_sync(~0u, mt, w));
            const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - mt);
            l[r] *= f;
#pragma unroll
            for (int w = LP; w < 32; w <<= 1) l[r] += __shfl_xor_sync(~0u, l[r], w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 lo = parts(o[r][i][0]), hi = parts(o[r][i][1]);
                float x[4] = {lo.x * f, lo.y * f, hi.x * f, hi.y * f};
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int w = LP; w < 32; w <<= 1) x[j] += __shfl_xor_sync(~0u, x[j], w);
                if (at_pos == 0)
                    *reinterpret_cast<float4 *>(&outs[warp][r][4 * LP * i + at_place]) =
                        make_float4(x[0], x[1], x[2], x[3]);
            }
            if (lane == 0) top_of[warp][r] = mt, sum_of[warp][r] = l[r];
        }
        __syncthreads();
        const bool whole = item_end && (first_item ? tile_first == 0 : true);
        float *const part = part_at(a, s, 2 * blockIdx.x + (first_item ? 0 : 1));
        if (threadIdx.x == 0 && !whole && !(first_item && tile_first > 0)) {
            const int64_t t1 = span.beg + span.left + it.ntiles - tile;
            Cut cut;
            cut.parts = int(divide(t1 + span.part - 1, span.part)) - int(blockIdx.x);
            cut.first = first_item ? 0 : 1;
            cut.b = it.b;
            cut.hk = it.hk;
            cut.rb = it.rb;
            if (cut_ok(a, s, blockIdx.x)) reinterpret_cast<Cut *>(a.ws)[blockIdx.x] = cut;
        }
        for (int i = threadIdx.x; i < NR * D; i += 32 * kF32Warps) {
            const int rr = i / D, d = i % D, row = it.rb * NR + rr;
            if (row >= rows) break;
            float mt = -INFINITY, lt = 0.f, x = 0.f;
#pragma unroll
            for (int w = 0; w < kF32Warps; ++w) mt = fmaxf(mt, top_of[w][rr]);
            const float base = mt == -INFINITY ? 0.f : mt;
#pragma unroll
            for (int w = 0; w < kF32Warps; ++w) {
                const float f = ex2(top_of[w][rr] - base);
                lt = fmaf(sum_of[w][rr], f, lt);
                x = fmaf(outs[w][rr][d], f, x);
            }
            if (whole) {
                const int t = token_of(s, row), h = it.hk * s.G + row - t * s.G;
                const int64_t off = it.b * a.o_sb + t * a.o_st + h * a.o_sh + d;
                if (SSD_IDX_OK(a.err, off, a.o_n)) static_cast<float *>(a.out)[off] = lt == 0.f ? 0.f : x / lt;
                const int64_t at = (int64_t(it.b) * a.T + t) * a.Hq + h;
                if (a.lse && d == 0 && lse_ok(a, at)) a.lse[at] = log_sum<false>(mt, lt);
            } else if (part_ok(a, s, 2 * blockIdx.x + (first_item ? 0 : 1), rr)) {
                part[rr * D + d] = x;
                if (d == 0) {
                    part[NR * D + rr] = mt;
                    part[NR * (D + 1) + rr] = lt;
                }
            }
        }
        if (item_end) {
            tile = 0;
            left -= kItemCost;
            fresh = true;
            first_item = false;
            it = next_item<KS>(s, it, a.lens[min(it.b + 1, a.B - 1)]);
        }
    }
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

// The join may start while the last parts are being computed; it waits for them before
// it reads any.
template <typename T, int D, bool F8>
cudaError_t launch_join(const PagedArgs &a, const Shape &s, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    // Items of few parts, which a warp loads at once: a warp a row.  Else about 8 CTAs for an item, one
    // wave of them all.
    const int64_t items = int64_t(s.B) * s.Hkv * s.nrb;
    const bool few = s.ncta <= items * (kJoinAhead - 1);
    const int per = few || s.RB > 16 ? 1 : s.RB <= 8 ? 4 : 2, at_once = 4 / per;
    cfg.gridDim = dim3(unsigned(s.ncta), unsigned(min(8, (min(s.RB, a.T * s.G) + at_once - 1) / at_once)));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_paged_join<T, D, F8>, a, s, per);
}

template <int D, int FMT, int NQ, int WR, bool ASK = false>
cudaError_t launch_mma(const PagedArgs &a, const Shape &s, cudaStream_t stream) {
    using C = Cfg<D, FMT, NQ, WR>;
    static std::atomic<uint64_t> done[4];
    cudaError_t e = allow_smem(k_paged_mma<D, FMT, NQ, WR, ASK>, C::SMEM, done);
    if (e != cudaSuccess) return e;
    k_paged_mma<D, FMT, NQ, WR, ASK><<<s.ncta, kThreads, C::SMEM, stream>>>(a, s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if constexpr (ASK) {
        if ((e = launch_paged_prompt(a, stream)) != cudaSuccess) return e;
    }
    return launch_join<__nv_bfloat16, D, C::F8>(a, s, stream);
}

template <int D, int NR>
cudaError_t launch_f32(const PagedArgs &a, const Shape &s, cudaStream_t stream) {
    k_paged_f32<D, NR><<<s.ncta, 32 * kF32Warps, 0, stream>>>(a, s);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join<float, D, false>(a, s, stream);
}

// Rows of a block: 8 or 16 to a warp, then up to four warps along the rows (and
// the rest of the four along the positions).  More rows than 64 are several row
// blocks, each of which reads the cache.  64 sequences of 4096 over 8 key/value heads of
// 128, microseconds for bf16 / fp8 with blocks of half the rows, this rule's, twice:
//   8 rows              -  167 /  95  170 /  99
//   16 rows     327 / 176  174 / 105  171 / 163
//   32 rows     334 / 191  177 / 168  252 / 290
inline Shape make_shape(const PagedArgs &a) {
    Shape s{};
    s.lens = a.lens;
    s.B = a.B;
    s.T = a.T;
    s.Hkv = a.c.Hkv;
    s.cap = a.M * a.c.ps;
    s.window = int(a.window);
    s.back = a.window > 0 ? s.window : 0x7fff0000;    // (rows' places are -65535 and more: no overflow)
    s.sinks = int(a.sinks);
    s.G = a.Hq / a.c.Hkv;
    const int64_t rows = int64_t(a.T) * s.G;
    if (a.c.dt == DT_F32)      // (the outputs of NR rows are 16 NR registers)
        s.RB = rows == 1 ? 1 : rows == 2 ? 2 : 4;
    else
        s.RB = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    s.nrb = int((rows + s.RB - 1) / s.RB);
    s.ncta = device_sm_count() * (a.c.dt == DT_F4E2M1X2 ? ctas_of(kFour, s.RB) : kCtasPerSm);
    return s;
}

template <int D>
cudaError_t launch_f32_rows(const PagedArgs &a, cudaStream_t stream) {
    const Shape s = make_shape(a);
    if (s.RB == 1) return launch_f32<D, 1>(a, s, stream);
    if (s.RB == 2) return launch_f32<D, 2>(a, s, stream);
    return launch_f32<D, 4>(a, s, stream);
}

template <int D, int FMT>
cudaError_t launch_rows(const PagedArgs &a, cudaStream_t stream) {
    const Shape s = make_shape(a);
    if constexpr (FMT == kBf16)       // (blocks of 64 rows)
        if (a.ask.on) return launch_mma<D, FMT, 2, 4, true>(a, s, stream);
    switch (s.RB) {
    case 8: return launch_mma<D, FMT, 1, 1>(a, s, stream);
    case 16: return launch_mma<D, FMT, 2, 1>(a, s, stream);
    case 32: return launch_mma<D, FMT, 2, 2>(a, s, stream);
    default: return launch_mma<D, FMT, 2, 4>(a, s, stream);
    }
}

}  // namespace
}  // namespace ssd
