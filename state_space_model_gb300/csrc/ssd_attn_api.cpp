// Host side of the attention layers' entry points declared in include/ssd.h:
// argument checks, then one launcher call on the caller's stream.  Nothing
// here allocates, frees or synchronises.
#include "ssd.h"
#include "ssd_attn.h"
#include "ssd_checks.h"

#include <cmath>

namespace {

using namespace ssd::checks;

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
// Positions leave room below 2^31 for a tile and for the new tokens, so that
// the kernels count them in 32 bits.
constexpr int64_t kMaxPos = kMaxInt - (1 << 17);
constexpr int64_t kMaxRows = 1 << 24;   // of a sequence and key/value head

int64_t extent(const ssd_tensor *t) {
    int64_t last = 0;
    for (int i = 0; i < t->ndim; ++i) {
        if (t->shape[i] == 0) return 0;
        last += (t->shape[i] - 1) * t->stride[i];
    }
    return last + 1;
}

bool same_strides(const ssd_tensor *a, const ssd_tensor *b) {
    for (int i = 0; i < a->ndim; ++i)
        if (a->shape[i] > 1 && a->stride[i] != b->stride[i]) return false;
    return true;
}

// The pools and their scales; fills p.  out: they are written.
ssd_status check_pools(const ssd_tensor *k, const ssd_tensor *v, const ssd_tensor *ks,
                       const ssd_tensor *vs, bool out, ssd::KvPools *p) {
    if (!k || !v) return fail(SSD_ERR_INVALID_ARG, "k_cache / v_cache: null tensor descriptor");
    if (k->ndim != 4) return fail(SSD_ERR_INVALID_ARG, "k_cache: ndim %d, expected 4", k->ndim);
    const int64_t pages = k->shape[0], Hkv = k->shape[1], ps = k->shape[2], D = k->shape[3];
    if (pages < 0 || Hkv <= 0 || ps <= 0)
        return fail(SSD_ERR_INVALID_ARG, "k_cache: %lld pages of %lld tokens, %lld heads",
                    (long long)pages, (long long)ps, (long long)Hkv);
    if (D != 64 && D != 128)
        return fail(SSD_ERR_UNSUPPORTED, "headdim %lld unsupported (64 or 128)", (long long)D);
    if (Hkv > 65535)
        return fail(SSD_ERR_UNSUPPORTED, "%lld key/value heads above 65535", (long long)Hkv);
    if (pages > kMaxInt || ps > kMaxInt || pages * ps > kMaxInt)
        return fail(SSD_ERR_UNSUPPORTED, "%lld pages of %lld tokens: more than 2^31 - 1 slots",
                    (long long)pages, (long long)ps);
    const int dt = k->dtype;
    if (dt == SSD_I32) return fail(SSD_ERR_INVALID_ARG, "k_cache: dtype i32");
    const int64_t shape[4] = {pages, Hkv, ps, D}, sscale[3] = {pages, Hkv, ps};
    ssd_status st;
    if ((st = check_tensor(k, "k_cache", 4, shape, dt, false, true))) return st;
    if ((st = check_tensor(v, "v_cache", 4, shape, dt, false, true))) return st;
    if (!same_strides(k, v))
        return fail(SSD_ERR_INVALID_ARG, "k_cache and v_cache must have the same strides");
    if (dt == SSD_F8E4M3) {
        if (!ks || !vs)
            return fail(SSD_ERR_INVALID_ARG, "f8e4m3 pools need k_scale and v_scale");
        if ((st = check_tensor(ks, "k_scale", 3, sscale, SSD_F32, false, false))) return st;
        if ((st = check_tensor(vs, "v_scale", 3, sscale, SSD_F32, false, false))) return st;
        if (!same_strides(ks, vs))
            return fail(SSD_ERR_INVALID_ARG, "k_scale and v_scale must have the same strides");
    } else if (ks || vs) {
        return fail(SSD_ERR_INVALID_ARG, "k_scale / v_scale: only with f8e4m3 pools");
    }
    if (out) {
        if ((st = check_distinct(k, "k_cache")) || (st = check_distinct(v, "v_cache"))) return st;
        if (ks && ((st = check_distinct(ks, "k_scale")) || (st = check_distinct(vs, "v_scale"))))
            return st;
    }
    p->k = k->data;
    p->v = v->data;
    p->ks = ks ? static_cast<float *>(ks->data) : nullptr;
    p->vs = vs ? static_cast<float *>(vs->data) : nullptr;
    p->dt = dt;
    p->Hkv = int(Hkv);
    p->D = int(D);
    p->ps = int(ps);
    p->pages = int(pages);
    p->sp = k->stride[0];
    p->sh = k->stride[1];
    p->st = k->stride[2];
    p->n = extent(k);
    if (ks) {
        p->ssp = ks->stride[0];
        p->ssh = ks->stride[1];
        p->ns = extent(ks);
    }
    return SSD_OK;
}

// A page table [B, M]: innermost stride 1.
ssd_status check_table(const ssd_tensor *t, int64_t B, int64_t ps) {
    if (!t) return fail(SSD_ERR_INVALID_ARG, "page_table: null tensor descriptor");
    if (t->ndim != 2) return fail(SSD_ERR_INVALID_ARG, "page_table: ndim %d, expected 2", t->ndim);
    const int64_t shape[2] = {B, t->shape[1]};
    ssd_status st;
    if ((st = check_tensor(t, "page_table", 2, shape, SSD_I32, false, false))) return st;
    if (t->shape[1] < 0 || t->shape[1] > kMaxInt || t->shape[1] * ps > kMaxPos)
        return fail(SSD_ERR_UNSUPPORTED, "page_table: %lld pages of %lld tokens, more than "
                    "2^31 - 2^17 positions", (long long)t->shape[1], (long long)ps);
    return SSD_OK;
}

struct Named {
    const ssd_tensor *t;
    const char *name;
};
// No output may share an element with an input or another output.
ssd_status check_aliasing(std::initializer_list<Named> outs, std::initializer_list<Named> ins) {
    const Named *all[16];
    Range at[16];
    int n = 0;
    for (const Named &o : outs) all[n++] = &o;
    for (const Named &i : ins) all[n++] = &i;
    for (int i = 0; i < n; ++i) at[i] = range_of(all[i]->t);
    const int nouts = int(outs.size());
    for (int o = 0; o < nouts; ++o)
        for (int i = o + 1; i < n; ++i)
            if (overlap(at[o], at[i]) && overlap(all[o]->t, all[i]->t))   // (ranges seldom meet)
                return fail(SSD_ERR_INVALID_ARG, "%s overlaps %s", all[o]->name, all[i]->name);
    return SSD_OK;
}

const void *dp(const ssd_tensor *t) { return t ? t->data : nullptr; }

}  // namespace

extern "C" {

ssd_status ssd_kv_append(const ssd_tensor *q, const ssd_tensor *k, const ssd_tensor *v,
                         const ssd_tensor *slots, const ssd_tensor *positions,
                         const ssd_tensor *cos, const ssd_tensor *sin,
                         const ssd_tensor *q_weight, const ssd_tensor *k_weight, float eps,
                         int32_t interleaved, ssd_tensor *k_cache, ssd_tensor *v_cache,
                         ssd_tensor *k_scale, ssd_tensor *v_scale, ssd_tensor *q_out,
                         void *stream) {
    ssd::KvAppendArgs a;
    ssd_status st;
    if ((st = check_pools(k_cache, v_cache, k_scale, v_scale, true, &a.c))) return st;
    if (!q) return fail(SSD_ERR_INVALID_ARG, "q: null tensor descriptor");
    if (q->ndim != 3) return fail(SSD_ERR_INVALID_ARG, "q: ndim %d, expected 3", q->ndim);
    const int64_t T = q->shape[0], Hq = q->shape[1], Hkv = a.c.Hkv, D = a.c.D;
    if (T < 0 || Hq <= 0)
        return fail(SSD_ERR_INVALID_ARG, "q: %lld tokens of %lld heads", (long long)T,
                    (long long)Hq);
    if (Hq % Hkv)
        return fail(SSD_ERR_INVALID_ARG, "%lld query heads are not a multiple of %lld key/value "
                    "heads", (long long)Hq, (long long)Hkv);
    if (T > kMaxInt || Hq > 65535)
        return fail(SSD_ERR_UNSUPPORTED, "%lld tokens above 2^31 - 1 or %lld query heads above "
                    "65535", (long long)T, (long long)Hq);
    const int64_t sq[3] = {T, Hq, D}, skv[3] = {T, Hkv, D}, st1[1] = {T}, sd[1] = {D};
    if ((st = check_tensor(q, "q", 3, sq, -1, false, true))) return st;
    const int xdt = q->dtype;
    if ((st = check_tensor(k, "k", 3, skv, xdt, false, true))) return st;
    if ((st = check_tensor(v, "v", 3, skv, xdt, false, true))) return st;
    if (a.c.dt != SSD_F8E4M3 && a.c.dt != xdt)
        return fail(SSD_ERR_INVALID_ARG, "k_cache: the pools hold the dtype of q or f8e4m3 codes");
    if ((st = check_tensor(slots, "slots", 1, st1, SSD_I32, true, false))) return st;
    if (!cos != !sin || !cos != !positions)
        return fail(SSD_ERR_INVALID_ARG, "positions, cos and sin come together");
    if (cos) {
        if (cos->ndim != 2) return fail(SSD_ERR_INVALID_ARG, "cos: ndim %d, expected 2", cos->ndim);
        const int64_t S = cos->shape[0], R = 2 * cos->shape[1], scs[2] = {S, R / 2};
        if (R <= 0 || R % 16 || R > D)
            return fail(SSD_ERR_UNSUPPORTED, "cos: %lld columns rotate %lld places; a multiple of "
                        "16 up to headdim %lld is supported", (long long)cos->shape[1],
                        (long long)R, (long long)D);
        if ((st = check_tensor(cos, "cos", 2, scs, SSD_F32, false, true))) return st;
        if ((st = check_tensor(sin, "sin", 2, scs, SSD_F32, false, true))) return st;
        if ((st = check_tensor(positions, "positions", 1, st1, SSD_I32, true, false))) return st;
        a.R = int(R);
        a.S = S;
        a.cos = static_cast<const float *>(cos->data);
        a.sin = static_cast<const float *>(sin->data);
        a.cs_st = cos->stride[0];
        a.sn_st = sin->stride[0];
        a.cs_n = extent(cos);
        a.sn_n = extent(sin);
        a.positions = static_cast<const int32_t *>(positions->data);
    }
    if (q_weight && (st = check_tensor(q_weight, "q_weight", 1, sd, SSD_F32, true, true)))
        return st;
    if (k_weight && (st = check_tensor(k_weight, "k_weight", 1, sd, SSD_F32, true, true)))
        return st;
    if (!(eps >= 0.f) || std::isinf(eps))
        return fail(SSD_ERR_INVALID_ARG, "eps %g must be finite and not negative", double(eps));
    if ((st = check_tensor(q_out, "q_out", 3, sq, xdt, false, true))) return st;
    if ((st = check_distinct(q_out, "q_out"))) return st;
    if ((st = check_aliasing({{k_cache, "k_cache"}, {v_cache, "v_cache"}, {k_scale, "k_scale"},
                              {v_scale, "v_scale"}, {q_out, "q_out"}},
                             {{q, "q"}, {k, "k"}, {v, "v"}, {slots, "slots"},
                              {positions, "positions"}, {cos, "cos"}, {sin, "sin"},
                              {q_weight, "q_weight"}, {k_weight, "k_weight"}})))
        return st;
    // no table row or no slot: every token is padding
    if (T == 0 || a.c.pages == 0 || (cos && a.S == 0)) return ok();
    if ((st = check_device_ptrs({{dp(q), "q"}, {dp(k), "k"}, {dp(v), "v"}, {dp(slots), "slots"},
                                 {dp(positions), "positions"}, {dp(cos), "cos"}, {dp(sin), "sin"},
                                 {dp(q_weight), "q_weight"}, {dp(k_weight), "k_weight"},
                                 {dp(k_cache), "k_cache"}, {dp(v_cache), "v_cache"},
                                 {dp(k_scale), "k_scale"}, {dp(v_scale), "v_scale"},
                                 {dp(q_out), "q_out"}})))
        return st;
    a.xdt = xdt;
    a.T = T;
    a.Hq = int(Hq);
    a.interleaved = interleaved ? 1 : 0;
    a.eps = eps;
    a.q = q->data;
    a.q_st = q->stride[0];
    a.q_sh = q->stride[1];
    a.k = k->data;
    a.k_st = k->stride[0];
    a.k_sh = k->stride[1];
    a.v = v->data;
    a.v_st = v->stride[0];
    a.v_sh = v->stride[1];
    a.out = q_out->data;
    a.o_st = q_out->stride[0];
    a.o_sh = q_out->stride[1];
    a.q_n = extent(q);
    a.k_n = extent(k);
    a.v_n = extent(v);
    a.o_n = extent(q_out);
    a.slots = static_cast<const int32_t *>(slots->data);
    a.qw = q_weight ? static_cast<const float *>(q_weight->data) : nullptr;
    a.kw = k_weight ? static_cast<const float *>(k_weight->data) : nullptr;
    if ((st = cuda_status(ssd::launch_kv_append(a, static_cast<cudaStream_t>(stream)),
                          "kv append")))
        return st;
    return ok();
}

ssd_status ssd_kv_read(const ssd_tensor *k_cache, const ssd_tensor *v_cache,
                       const ssd_tensor *k_scale, const ssd_tensor *v_scale,
                       const ssd_tensor *page_table, const ssd_tensor *cu_lens,
                       const ssd_tensor *starts, ssd_tensor *k, ssd_tensor *v, void *stream) {
    ssd::KvReadArgs a;
    ssd_status st;
    if ((st = check_pools(k_cache, v_cache, k_scale, v_scale, false, &a.c))) return st;
    if (!page_table || !k) return fail(SSD_ERR_INVALID_ARG, "page_table / k: null tensor descriptor");
    const int64_t B = page_table->ndim > 0 ? page_table->shape[0] : 0;
    if ((st = check_table(page_table, B, a.c.ps))) return st;
    if (B > kMaxInt - 1) return fail(SSD_ERR_UNSUPPORTED, "batch %lld too large", (long long)B);
    if (k->ndim != 3) return fail(SSD_ERR_INVALID_ARG, "k: ndim %d, expected 3", k->ndim);
    const int64_t T = k->shape[0], skv[3] = {T, a.c.Hkv, a.c.D}, scu[1] = {B + 1}, sb[1] = {B};
    if (T < 0) return fail(SSD_ERR_INVALID_ARG, "k: %lld tokens", (long long)T);
    if (T > kMaxInt) return fail(SSD_ERR_UNSUPPORTED, "%lld tokens above 2^31 - 1", (long long)T);
    if ((st = check_tensor(cu_lens, "cu_lens", 1, scu, SSD_I32, true, false))) return st;
    if (starts && (st = check_tensor(starts, "starts", 1, sb, SSD_I32, true, false))) return st;
    if ((st = check_tensor(k, "k", 3, skv, a.c.dt == SSD_F8E4M3 ? -1 : a.c.dt, false, true)))
        return st;
    if ((st = check_tensor(v, "v", 3, skv, k->dtype, false, true))) return st;
    if ((st = check_distinct(k, "k")) || (st = check_distinct(v, "v"))) return st;
    if ((st = check_aliasing({{k, "k"}, {v, "v"}},
                             {{k_cache, "k_cache"}, {v_cache, "v_cache"}, {k_scale, "k_scale"},
                              {v_scale, "v_scale"}, {page_table, "page_table"},
                              {cu_lens, "cu_lens"}, {starts, "starts"}})))
        return st;
    if (T == 0) return ok();
    if ((st = check_device_ptrs({{dp(k_cache), "k_cache"}, {dp(v_cache), "v_cache"},
                                 {dp(k_scale), "k_scale"}, {dp(v_scale), "v_scale"},
                                 {dp(page_table), "page_table"}, {dp(cu_lens), "cu_lens"},
                                 {dp(starts), "starts"}, {dp(k), "k"}, {dp(v), "v"}})))
        return st;
    a.odt = k->dtype;
    a.T = T;
    a.B = int(B);
    a.M = int(page_table->shape[1]);
    a.table = static_cast<const int32_t *>(page_table->data);
    a.tb = page_table->stride[0];
    a.cu = static_cast<const int32_t *>(cu_lens->data);
    a.starts = starts ? static_cast<const int32_t *>(starts->data) : nullptr;
    a.k = k->data;
    a.k_st = k->stride[0];
    a.k_sh = k->stride[1];
    a.v = v->data;
    a.v_st = v->stride[0];
    a.v_sh = v->stride[1];
    a.t_n = extent(page_table);
    a.k_n = extent(k);
    a.v_n = extent(v);
    if ((st = cuda_status(ssd::launch_kv_read(a, static_cast<cudaStream_t>(stream)), "kv read")))
        return st;
    return ok();
}

// The geometry both paged-attention calls accept.
static ssd_status check_paged(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int32_t dt) {
    if (B < 0 || T < 0 || Hq <= 0 || Hkv <= 0)
        return fail(SSD_ERR_INVALID_ARG, "batch %lld, %lld tokens, %lld query and %lld key/value "
                    "heads", (long long)B, (long long)T, (long long)Hq, (long long)Hkv);
    if (Hq % Hkv)
        return fail(SSD_ERR_INVALID_ARG, "%lld query heads are not a multiple of %lld key/value "
                    "heads", (long long)Hq, (long long)Hkv);
    if (D != 64 && D != 128)
        return fail(SSD_ERR_UNSUPPORTED, "headdim %lld unsupported (64 or 128)", (long long)D);
    if (dt != SSD_F32 && dt != SSD_BF16 && dt != SSD_F8E4M3)
        return fail(SSD_ERR_INVALID_ARG, "cache dtype code %d: f32, bf16 or f8e4m3 expected", dt);
    if (B > 65535 || Hq > 65535 || T > 65535)
        return fail(SSD_ERR_UNSUPPORTED, "batch %lld, %lld tokens or %lld query heads above 65535",
                    (long long)B, (long long)T, (long long)Hq);
    if (T * (Hq / Hkv) > kMaxRows)
        return fail(SSD_ERR_UNSUPPORTED, "%lld tokens of %lld query heads a key/value head: more "
                    "than 2^24 rows", (long long)T, (long long)(Hq / Hkv));
    return SSD_OK;
}

ssd_status ssd_paged_attention_workspace_size(int64_t batch, int64_t tokens, int64_t q_heads,
                                              int64_t kv_heads, int64_t headdim,
                                              int32_t cache_dtype, size_t *bytes) {
    if (!bytes) return fail(SSD_ERR_INVALID_ARG, "bytes: null pointer");
    *bytes = 0;
    ssd_status st;
    if ((st = check_paged(batch, tokens, q_heads, kv_heads, headdim, cache_dtype))) return st;
    ssd::PagedArgs a;
    a.B = int(batch);
    a.T = int(tokens);
    a.Hq = int(q_heads);
    a.c.Hkv = int(kv_heads);
    a.c.D = int(headdim);
    a.c.dt = cache_dtype;
    *bytes = batch && tokens ? ssd::paged_workspace(a) : 0;
    return ok();
}

ssd_status ssd_paged_attention(const ssd_tensor *q, const ssd_tensor *k_cache,
                               const ssd_tensor *v_cache, const ssd_tensor *k_scale,
                               const ssd_tensor *v_scale, const ssd_tensor *page_table,
                               const ssd_tensor *lens, float scale, int64_t window,
                               ssd_tensor *out, ssd_tensor *lse, void *workspace,
                               size_t workspace_bytes, void *stream) {
    ssd::PagedArgs a;
    ssd_status st;
    if ((st = check_pools(k_cache, v_cache, k_scale, v_scale, false, &a.c))) return st;
    if (!q) return fail(SSD_ERR_INVALID_ARG, "q: null tensor descriptor");
    if (q->ndim != 4) return fail(SSD_ERR_INVALID_ARG, "q: ndim %d, expected 4", q->ndim);
    const int64_t B = q->shape[0], T = q->shape[1], Hq = q->shape[2], D = a.c.D;
    if ((st = check_paged(B, T, Hq, a.c.Hkv, D, a.c.dt))) return st;
    const int64_t sq[4] = {B, T, Hq, D}, sb[1] = {B}, slse[3] = {B, T, Hq};
    const int xdt = a.c.dt == SSD_F32 ? SSD_F32 : SSD_BF16;
    if ((st = check_tensor(q, "q", 4, sq, xdt, false, true))) return st;
    if ((st = check_table(page_table, B, a.c.ps))) return st;
    if ((st = check_tensor(lens, "lens", 1, sb, SSD_I32, true, false))) return st;
    if (!std::isfinite(scale)) return fail(SSD_ERR_INVALID_ARG, "scale %g is not finite", double(scale));
    if (window < 0) return fail(SSD_ERR_INVALID_ARG, "window %lld is negative", (long long)window);
    if ((st = check_tensor(out, "out", 4, sq, xdt, false, true))) return st;
    if ((st = check_distinct(out, "out"))) return st;
    if (lse && (st = check_tensor(lse, "lse", 3, slse, SSD_F32, true, false))) return st;
    if ((st = check_aliasing({{out, "out"}, {lse, "lse"}},
                             {{q, "q"}, {k_cache, "k_cache"}, {v_cache, "v_cache"},
                              {k_scale, "k_scale"}, {v_scale, "v_scale"},
                              {page_table, "page_table"}, {lens, "lens"}})))
        return st;
    a.B = int(B);
    a.T = int(T);
    a.Hq = int(Hq);
    if (B == 0 || T == 0) return ok();
    const size_t need = ssd::paged_workspace(a);
    if (need) {
        if (!workspace || workspace_bytes < need)
            return fail(SSD_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes,
                        need);
        if (reinterpret_cast<uintptr_t>(workspace) % 256)
            return fail(SSD_ERR_ALIGNMENT, "workspace %p is not 256-byte aligned", workspace);
        const Range rw = range_raw(workspace, need);
        const Named others[] = {{q, "q"}, {k_cache, "k_cache"}, {v_cache, "v_cache"},
                                {k_scale, "k_scale"}, {v_scale, "v_scale"},
                                {page_table, "page_table"}, {lens, "lens"}, {out, "out"},
                                {lse, "lse"}};
        for (const Named &o : others)
            if (overlap(rw, range_of(o.t)))
                return fail(SSD_ERR_INVALID_ARG, "workspace overlaps %s", o.name);
    }
    if ((st = check_device_ptrs({{dp(q), "q"}, {dp(k_cache), "k_cache"}, {dp(v_cache), "v_cache"},
                                 {dp(k_scale), "k_scale"}, {dp(v_scale), "v_scale"},
                                 {dp(page_table), "page_table"}, {dp(lens), "lens"},
                                 {dp(out), "out"}, {dp(lse), "lse"},
                                 {need ? workspace : nullptr, "workspace"}})))
        return st;
    a.scale = scale;
    a.window = window > kMaxPos ? 0 : window;   // such a window hides nothing
    a.q = q->data;
    a.q_sb = q->stride[0];
    a.q_st = q->stride[1];
    a.q_sh = q->stride[2];
    a.out = out->data;
    a.o_sb = out->stride[0];
    a.o_st = out->stride[1];
    a.o_sh = out->stride[2];
    a.lse = lse ? static_cast<float *>(lse->data) : nullptr;
    a.M = int(page_table->shape[1]);
    a.table = static_cast<const int32_t *>(page_table->data);
    a.tb = page_table->stride[0];
    a.lens = static_cast<const int32_t *>(lens->data);
    a.ws = static_cast<char *>(workspace);
    a.q_n = extent(q);
    a.o_n = extent(out);
    a.t_n = extent(page_table);
    a.ws_n = int64_t(need);
    if ((st = cuda_status(ssd::launch_paged(a, static_cast<cudaStream_t>(stream)),
                          "paged attention")))
        return st;
    return ok();
}

}  // extern "C"
