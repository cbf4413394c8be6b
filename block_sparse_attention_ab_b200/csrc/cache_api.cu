// cache_api.cu -- the key/value cache calls of include/ab_attn.h: host-side argument checks
// and launches on the caller's stream. No device memory is allocated and no state is kept.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "ab_kernels.h"
#include "cache_kernels.h"

namespace {

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// row starts must be 16-byte aligned; strides are below the 2^40 bytes that a tensor map holds.
// (Products with an index are made in 64 bits, which is enough for any tensor in memory.)
bool stride_ok(int64_t s) { return s % 8 == 0 && s >= 0 && s < (1ll << 38); }

ab_status check_cache(const ab_cache &c, bool pages = true)
{
    if (!c.table || !c.length || (pages && (!c.k || !c.v))) return AB_ERR_NULL;
    if (c.B <= 0 || c.Hk <= 0 || c.n_pages <= 0 || c.max_pages <= 0) return AB_ERR_SHAPE;
    if (c.dtype != AB_BF16 && c.dtype != AB_F16) return AB_ERR_DTYPE;
    if (c.d != 64 && c.d != 128) return AB_ERR_UNSUPPORTED;
    if (c.page != 16 && c.page != 32 && c.page != 64 && c.page != 128) return AB_ERR_UNSUPPORTED;
    // slots, grid indices and the per-call item counts stay in int
    if (c.B > 65535 || c.Hk > 65535 || (long long)c.B * c.Hk > 1 << 20) return AB_ERR_RANGE;
    if ((long long)c.max_pages * c.page > 1 << 30) return AB_ERR_RANGE;
    if (!aligned(c.table, 4) || !aligned(c.length, 4) || !aligned(c.ksum, 16) || !aligned(c.mass, 4) ||
        !aligned(c.pos, 4))
        return AB_ERR_ALIGN;
    if (pages && (!aligned(c.k, 16) || !aligned(c.v, 16) || !stride_ok(c.k_page) ||
                  !stride_ok(c.k_head) || !stride_ok(c.k_row) || !stride_ok(c.v_page) ||
                  !stride_ok(c.v_head) || !stride_ok(c.v_row)))
        return AB_ERR_ALIGN;
    return AB_OK;
}

// pages that are written must not lie over one another (an expanded dimension)
ab_status check_written(const ab_cache &c)
{
    using ab::stride_maps;
    return stride_maps(c.k_row, c.page) && stride_maps(c.k_head, c.Hk) && stride_maps(c.k_page, c.n_pages) &&
                   stride_maps(c.v_row, c.page) && stride_maps(c.v_head, c.Hk) && stride_maps(c.v_page, c.n_pages)
               ? AB_OK
               : AB_ERR_UNSUPPORTED;
}

// An array that a call writes while its other CTAs read `in` must not share memory with it.
bool overlap(const int32_t *out, size_t n_out, const int32_t *in, size_t n_in)
{
    const uintptr_t o = reinterpret_cast<uintptr_t>(out), i = reinterpret_cast<uintptr_t>(in);
    return out && in && o < i + 4 * n_in && i < o + 4 * n_out;
}

ab_status check_tokens(const ab_tokens &t)
{
    if (!t.p) return AB_ERR_NULL;
    if (!aligned(t.p, 16) || !stride_ok(t.sb) || !stride_ok(t.sh) || !stride_ok(t.st)) return AB_ERR_ALIGN;
    return AB_OK;
}

ab_status check_heads(const ab_cache &c, int Hq, int T)
{
    if (Hq <= 0 || Hq % c.Hk != 0 || T <= 0) return AB_ERR_SHAPE;
    if (T > AB_MAX_TREE || Hq / c.Hk > 1024) return AB_ERR_RANGE;
    if ((long long)c.B * Hq * T > 1ll << 30) return AB_ERR_RANGE;
    return AB_OK;
}

ab_status check_plan(const int32_t *idx, const int32_t *cnt, const float *w)
{
    if (!idx != !cnt || (w && !idx)) return AB_ERR_NULL;
    if (!aligned(idx, 4) || !aligned(cnt, 4) || !aligned(w, 4)) return AB_ERR_ALIGN;
    return AB_OK;
}

int log2_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

float softmax_scale_log2(int d) { return 1.4426950408889634f / std::sqrt((float)d); }

}  // namespace

#define AB_TRY(x)                     \
    do {                              \
        const ab_status st_ = (x);    \
        if (st_ != AB_OK) return st_; \
    } while (0)

extern "C" {

ab_status ab_cache_append(ab_cache c, ab_tokens k, ab_tokens v, int T, const int32_t *n_new,
                          const int32_t *sel, const int32_t *start, const int32_t *pos0,
                          int *dev_flag, void *stream)
{
    NvtxRange nvtx("ab_cache_append");
    AB_TRY(check_cache(c));
    AB_TRY(check_written(c));
    if (T <= 0) return AB_ERR_SHAPE;
    if (T > 1 << 20) return AB_ERR_RANGE;
    AB_TRY(check_tokens(k));
    AB_TRY(check_tokens(v));
    if (!aligned(n_new, 4) || !aligned(sel, 4) || !aligned(start, 4) || !aligned(pos0, 4)) return AB_ERR_ALIGN;
    // with start, one CTA writes a sequence's length while the others read these; without it a
    // kernel behind the first one adds n_new to length, sequence by sequence
    if (start && (overlap(c.length, c.B, start, c.B) || overlap(c.length, c.B, n_new, c.B) ||
                  overlap(c.length, c.B, pos0, c.B) || overlap(c.length, c.B, sel, (size_t)c.B * T)))
        return AB_ERR_UNSUPPORTED;
    if (!start && n_new != c.length && overlap(c.length, c.B, n_new, c.B)) return AB_ERR_UNSUPPORTED;
    return ab::status_of(ab::launch_cache_append(c, k, v, T, n_new, sel, start, pos0, dev_flag,
                                                 (cudaStream_t)stream));
}

ab_status ab_cache_score(ab_cache c, ab_tokens q, int Hq, int T, const int32_t *n_tok, int per_token,
                         int first, int recent, float *scores, int *dev_flag, void *stream)
{
    NvtxRange nvtx("ab_cache_score");
    AB_TRY(check_cache(c, false));
    if (!c.ksum || !scores) return AB_ERR_NULL;
    AB_TRY(check_heads(c, Hq, T));
    AB_TRY(check_tokens(q));
    if (c.max_pages > AB_MAX_UNITS || first < 0 || recent < 0) return AB_ERR_RANGE;
    if (!aligned(n_tok, 4) || !aligned(scores, 4)) return AB_ERR_ALIGN;
    if ((long long)c.B * c.Hk * (per_token ? T : 1) > 1 << 26) return AB_ERR_RANGE;
    return ab::status_of(ab::launch_cache_score(c, q, Hq / c.Hk, T, n_tok, per_token != 0, first, recent,
                                                scores, dev_flag, (cudaStream_t)stream));
}

ab_status ab_cache_attn_workspace_size(ab_cache c, int Hq, int T, int per_token, size_t *bytes)
{
    if (!bytes) return AB_ERR_NULL;
    *bytes = 0;
    AB_TRY(check_cache(c));
    AB_TRY(check_heads(c, Hq, T));
    *bytes = ab::cache_attn_plan(c, Hq / c.Hk, T, per_token != 0).bytes;
    return AB_OK;
}

ab_status ab_cache_attn(ab_cache c, ab_tokens q, ab_tokens k, ab_tokens v, int Hq, int T,
                        const int32_t *n_tok, const uint8_t *tree, const int32_t *idx,
                        const int32_t *cnt, const float *w, int per_token, void *out,
                        ab_dtype out_dtype, float *lse, void *workspace, size_t workspace_bytes,
                        int *dev_flag, void *stream)
{
    NvtxRange nvtx("ab_cache_attn");
    AB_TRY(check_cache(c));
    AB_TRY(check_heads(c, Hq, T));
    if (!out || !k.p != !v.p) return AB_ERR_NULL;
    AB_TRY(check_tokens(q));
    if (k.p) {
        AB_TRY(check_tokens(k));
        AB_TRY(check_tokens(v));
    }
    AB_TRY(check_plan(idx, cnt, w));
    if (per_token && !idx) return AB_ERR_NULL;
    if ((int)out_dtype != c.dtype && out_dtype != AB_F32) return AB_ERR_DTYPE;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(n_tok, 4) || !aligned(workspace, 16)) return AB_ERR_ALIGN;
    const ab::CacheAttnPlan plan = ab::cache_attn_plan(c, Hq / c.Hk, T, per_token != 0);
    if (!workspace || workspace_bytes < plan.bytes) return AB_ERR_WORKSPACE;
    ab::CacheAttn a = {};
    a.c = c;
    a.q = q;
    a.k = k;
    a.v = v;
    a.n_tok = n_tok;
    a.tree = tree;
    a.idx = idx;
    a.cnt = cnt;
    a.w = w;
    a.G = Hq / c.Hk;
    a.T = T;
    a.per_token = per_token != 0;
    a.Tp = a.per_token ? T : 1;
    a.page_shift = log2_of(c.page);
    a.out_f32 = out_dtype == AB_F32;
    a.groups = idx ? c.B * c.Hk * a.Tp : c.B;
    a.scale_log2 = softmax_scale_log2(c.d);
    a.out = out;
    a.lse = lse;
    a.flag = dev_flag;
    return ab::status_of(ab::launch_cache_attn(a, plan, workspace, (cudaStream_t)stream));
}

ab_status ab_cache_mass(ab_cache c, ab_tokens q, int Hq, int T, const int32_t *n_tok,
                        const int32_t *sel, const float *lse, const int32_t *idx,
                        const int32_t *cnt, const float *w, int per_token, float *mass_out,
                        int *dev_flag, void *stream)
{
    NvtxRange nvtx("ab_cache_mass");
    AB_TRY(check_cache(c));
    if (!c.mass || !lse) return AB_ERR_NULL;
    AB_TRY(check_heads(c, Hq, T));
    AB_TRY(check_tokens(q));
    AB_TRY(check_plan(idx, cnt, w));
    if (per_token && !idx) return AB_ERR_NULL;
    if (!aligned(n_tok, 4) || !aligned(sel, 4) || !aligned(lse, 4) || !aligned(mass_out, 4)) return AB_ERR_ALIGN;
    ab::CacheMass a = {};
    a.c = c;
    a.q = q;
    a.n_tok = n_tok;
    a.sel = sel;
    a.lse = lse;
    a.idx = idx;
    a.cnt = cnt;
    a.w = w;
    a.G = Hq / c.Hk;
    a.T = T;
    a.per_token = per_token != 0;
    a.Tp = a.per_token ? T : 1;
    a.page_shift = log2_of(c.page);
    a.scale_log2 = softmax_scale_log2(c.d);
    a.out = mass_out ? mass_out : c.mass;
    a.flag = dev_flag;
    return ab::status_of(ab::launch_cache_mass(a, (cudaStream_t)stream));
}

ab_status ab_cache_keep_workspace_size(ab_cache c, int budget, size_t *bytes)
{
    if (!bytes) return AB_ERR_NULL;
    *bytes = 0;
    AB_TRY(check_cache(c, false));
    if (budget < 1 || budget > 1 << 30) return AB_ERR_RANGE;
    *bytes = (size_t)c.B * c.Hk * budget * sizeof(int32_t);
    return AB_OK;
}

ab_status ab_cache_keep(ab_cache c, int budget, int recent, const int32_t *next_pos,
                        const float *score, const int32_t *pos, const int32_t *length,
                        int32_t *src, int32_t *n_keep, void *workspace, size_t workspace_bytes,
                        int *dev_flag, void *stream)
{
    NvtxRange nvtx("ab_cache_keep");
    size_t need = 0;
    AB_TRY(check_cache(c, false));
    AB_TRY(ab_cache_keep_workspace_size(c, budget, &need));
    if (recent < 0) return AB_ERR_RANGE;
    if (!score) score = c.mass;
    if (!pos) pos = c.pos;
    if (!score || !src || !n_keep || (recent > 0 && (!pos || !next_pos))) return AB_ERR_NULL;
    if (!aligned(score, 4) || !aligned(pos, 4) || !aligned(length, 4) || !aligned(next_pos, 4) ||
        !aligned(src, 4) || !aligned(n_keep, 4) || !aligned(workspace, 4))
        return AB_ERR_ALIGN;
    if (!workspace || workspace_bytes < need) return AB_ERR_WORKSPACE;
    if (!length) length = c.length;
    const size_t n_src = (size_t)c.B * c.Hk * budget;
    if (overlap(n_keep, c.B, length, c.B) || overlap(src, n_src, length, c.B) ||
        (recent > 0 && (overlap(n_keep, c.B, next_pos, c.B) || overlap(src, n_src, next_pos, c.B))))
        return AB_ERR_UNSUPPORTED;  // written by one head's CTA while the others read them
    ab::CacheKeep a = {};
    a.c = c;
    a.budget = budget;
    a.recent = recent;
    a.next_pos = next_pos;
    a.score = score;
    a.pos = pos;
    a.length = length;
    a.src = src;
    a.n_keep = n_keep;
    a.movers = static_cast<int32_t *>(workspace);
    a.flag = dev_flag;
    return ab::status_of(ab::launch_cache_keep(a, (cudaStream_t)stream));
}

ab_status ab_cache_compact(ab_cache c, int budget, const int32_t *src, const int32_t *n_keep,
                           int *dev_flag, void *stream)
{
    NvtxRange nvtx("ab_cache_compact");
    AB_TRY(check_cache(c));
    AB_TRY(check_written(c));
    if (!src || !n_keep) return AB_ERR_NULL;
    if (budget < 1 || budget > 1 << 30) return AB_ERR_RANGE;
    if (!aligned(src, 4) || !aligned(n_keep, 4)) return AB_ERR_ALIGN;
    // read by some CTAs while one writes length
    if (overlap(c.length, c.B, n_keep, c.B) || overlap(c.length, c.B, src, (size_t)c.B * c.Hk * budget))
        return AB_ERR_UNSUPPORTED;
    return ab::status_of(ab::launch_cache_compact(c, budget, src, n_keep, dev_flag, (cudaStream_t)stream));
}

}  // extern "C"
