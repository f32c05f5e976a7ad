// Arguments of the launchers for the attention layers' key/value cache
// (ssd_kv_append, ssd_kv_read, ssd_paged_attention).  Not part of the public
// ABI.
#pragma once

#include "ssd_common.h"
#include "ssd_tmap.h"

#include <stddef.h>

namespace ssd {

// The codes' dtypes of the public header (DT_F32, DT_BF16 beside them).
enum : int { DT_F8E4M3 = 3, DT_F4E2M1X2 = 4 };
constexpr int kGroup = 16;                    // places of a row that share a scale (4-bit codes)
constexpr int kMaxAxes = 4;                   // of positions

// Key and value pools [pages, Hkv, ps, D] (strides in elements, the same for
// both pools; 4-bit codes: [pages, Hkv, ps, D/2] bytes), their scales [pages, Hkv, ps] for
// codes, and the groups' [pages, Hkv, ps, D/16] for 4-bit codes.
struct KvPools {
    void *k = nullptr, *v = nullptr;
    float *ks = nullptr, *vs = nullptr;       // null unless the pools hold codes
    uint8_t *kg = nullptr, *vg = nullptr;     // null unless the codes have 4 bits
    int dt = DT_BF16;
    int Hkv = 1, D = 128;
    int ps = 64, pages = 0;
    int64_t sp = 0, sh = 0, st = 0;           // page, head, token stride of the pools
    int64_t ssp = 0, ssh = 0;                 // page, head stride of the scales
    int64_t sgp = 0, sgh = 0, sgt = 0;        // page, head, token stride of the group scales
    int whole = 0;                            // 4-bit: 16 tokens of a page and head, with their scales, can
                                              // be copied in pieces of 16 bytes
    int64_t n = 0, ns = 0, ng = 0;            // extents (largest index + 1), debug build
};

struct KvAppendArgs {
    KvPools c;
    int xdt = DT_BF16;                        // dtype of q, k, v, q_out
    int64_t T = 0;
    int Hq = 1, R = 0, interleaved = 0;
    float eps = 0.f;
    const void *q = nullptr; int64_t q_st = 0, q_sh = 0;
    const void *k = nullptr; int64_t k_st = 0, k_sh = 0;
    const void *v = nullptr; int64_t v_st = 0, v_sh = 0;
    void *out = nullptr;     int64_t o_st = 0, o_sh = 0;
    const int32_t *slots = nullptr, *positions = nullptr;
    const float *cos = nullptr, *sin = nullptr;   // [S, R/2], null = no rotation
    int64_t S = 0, cs_st = 0, sn_st = 0;
    int axes = 1;                                 // positions [axes, T]
    uint32_t axis_of[kMaxAxes] = {};              // axes > 1: column i's, bits 2 i .. 2 i + 1
    const float *qw = nullptr, *kw = nullptr;     // [D], null = no norm
    int64_t q_n = 0, k_n = 0, v_n = 0, o_n = 0, cs_n = 0, sn_n = 0;   // extents, debug build
    unsigned int *err = nullptr;
};
cudaError_t launch_kv_append(const KvAppendArgs &a, cudaStream_t s);
cudaError_t launch_kv_append_ex(const KvAppendArgs &a, cudaStream_t s);   // its 4-bit pools, its axes

struct KvReadArgs {
    KvPools c;
    int odt = DT_BF16;
    int64_t T = 0;
    int B = 0, M = 0;
    const int32_t *table = nullptr; int64_t tb = 0;   // [B, M], row stride tb
    const int32_t *cu = nullptr, *starts = nullptr;
    void *k = nullptr; int64_t k_st = 0, k_sh = 0;
    void *v = nullptr; int64_t v_st = 0, v_sh = 0;
    int64_t t_n = 0, k_n = 0, v_n = 0;                // extents, debug build
    unsigned int *err = nullptr;
};
cudaError_t launch_kv_read(const KvReadArgs &a, cudaStream_t s);
cudaError_t launch_kv_read_ex(const KvReadArgs &a, cudaStream_t s);       // its 4-bit pools

// The pools' tensor maps for k_paged_prompt: 64 places, then tokens, heads and pages, by their strides.
struct PromptMaps {
    CUtensorMap k, v;
    int token = 1, head = 2, page = 3;        // the maps' dimensions
};

struct PagedArgs {
    KvPools c;
    int B = 0, T = 1, Hq = 1, M = 0;
    float scale = 1.f;                        // of the scores, natural exponent
    int64_t window = 0;                       // 0 = none
    int64_t sinks = 0;                        // positions that stay visible beside a window
    const void *q = nullptr; int64_t q_sb = 0, q_st = 0, q_sh = 0;
    void *out = nullptr;     int64_t o_sb = 0, o_st = 0, o_sh = 0;
    float *lse = nullptr;                     // [B, T, Hq], may be null
    const int32_t *table = nullptr; int64_t tb = 0;
    const int32_t *lens = nullptr;
    char *ws = nullptr;
    int64_t q_n = 0, o_n = 0, t_n = 0, ws_n = 0;      // extents (ws_n: bytes), debug build
    unsigned int *err = nullptr;
    // Where two kernels are launched and the lengths tell which works: costs for each 128 positions
    // (units of 0.1 ns times the SMs) of the longest sequence, of all where items are dealt out in turn, and of
    // all for the other kernel; no row sees more positions than `most`.
    struct Ask {
        int on = 0, most = 0;
        uint64_t one = 0, share = 0, line = 0;
    } ask;
    const PromptMaps *maps = nullptr;         // host memory, for the launch
};
// Workspace for this problem (c.dt, c.Hkv, c.D, B, T, Hq set).
size_t paged_workspace(const PagedArgs &a);
cudaError_t launch_paged(const PagedArgs &a, cudaStream_t s);
// its parts: many rows, pools of codes, calls with sinks
enum class Prompt { kNo, kYes, kAsk };   // kAsk: by the lengths, which the kernels look at
Prompt prompt_fits(const PagedArgs &a);
bool make_prompt_maps(const PagedArgs &a, PromptMaps *m);     // false: there are none for these pools
void ask_lengths(PagedArgs &a);          // kAsk: sets a.ask
cudaError_t launch_paged_prompt(const PagedArgs &a, cudaStream_t s);
cudaError_t launch_paged_f8(const PagedArgs &a, cudaStream_t s);
cudaError_t launch_paged_f4(const PagedArgs &a, cudaStream_t s);
cudaError_t launch_paged_sinks(const PagedArgs &a, cudaStream_t s);
cudaError_t launch_paged_sinks_f8(const PagedArgs &a, cudaStream_t s);
cudaError_t launch_paged_sinks_f4(const PagedArgs &a, cudaStream_t s);

}  // namespace ssd
