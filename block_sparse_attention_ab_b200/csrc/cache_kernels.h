// cache_kernels.h -- internal launchers of the key/value cache kernels (not part of the C
// ABI). The host checks of cache_api.cu have passed when one of these is called.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ab_attn.h"

namespace ab {

struct CacheAttn {
    ab_cache c;
    ab_tokens q, k, v;
    const int32_t *n_tok;
    const uint8_t *tree;
    const int32_t *idx, *cnt;
    const float *w;
    int G, T, Tp, page_shift;
    bool per_token, out_f32;
    int groups;  // sequences, or (sequence, key head, plan row)s
    float scale_log2;
    void *out;
    float *lse;
    int *flag;
    // set by the launcher
    float *part;
    float2 *part_ml;
    int2 *info;  // per (item, row tile): the CTAs with its first and its last unit
    int row_tiles;
    bool whole_groups;
};

// How a call is cut: a function of the shapes alone, so the workspace can be sized first.
struct CacheAttnPlan {
    int tile_rows, row_tiles, ctas;
    size_t items, off_ml, off_info, bytes;
};

CacheAttnPlan cache_attn_plan(const ab_cache &c, int G, int T, bool per_token);
cudaError_t launch_cache_attn(CacheAttn a, const CacheAttnPlan &p, void *workspace, cudaStream_t st);

// many query rows per key head: the tile kernel (cache_tiles.cu), without the join
cudaError_t launch_cache_tiles(const CacheAttn &a, const CacheAttnPlan &p, cudaStream_t st);

cudaError_t launch_cache_append(const ab_cache &c, const ab_tokens &k, const ab_tokens &v, int T,
                                const int32_t *n_new, const int32_t *sel, const int32_t *start,
                                const int32_t *pos0, int *flag, cudaStream_t st);

cudaError_t launch_cache_score(const ab_cache &c, const ab_tokens &q, int G, int T,
                               const int32_t *n_tok, bool per_token, int first, int recent,
                               float *scores, int *flag, cudaStream_t st);

struct CacheMass {
    ab_cache c;
    ab_tokens q;
    const int32_t *n_tok, *sel;
    const float *lse;
    const int32_t *idx, *cnt;
    const float *w;
    int G, T, Tp, page_shift;
    bool per_token;
    float scale_log2;
    float *out;
    int *flag;
};
cudaError_t launch_cache_mass(const CacheMass &a, cudaStream_t st);
// many query rows per key head, no plan (cache_mass_tiles.cu)
cudaError_t launch_cache_mass_tiles(const CacheMass &a, cudaStream_t st);

// A stride of 0 over more than one element (an expanded tensor) has no tensor map.
inline bool stride_maps(int64_t stride, int n) { return stride != 0 || n == 1; }

struct CacheKeep {
    ab_cache c;
    int budget, recent;
    const int32_t *next_pos;
    const float *score;
    const int32_t *pos, *length;
    int32_t *src, *n_keep;
    int32_t *movers;  // workspace, [B, Hk, budget]
    int *flag;
};
cudaError_t launch_cache_keep(const CacheKeep &a, cudaStream_t st);
cudaError_t launch_cache_compact(const ab_cache &c, int budget, const int32_t *src,
                                 const int32_t *n_keep, int *flag, cudaStream_t st);

}  // namespace ab
