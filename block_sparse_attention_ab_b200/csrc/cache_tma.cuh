// cache_tma.cuh -- tensor-memory-accelerator access to the pages of a key/value cache: a map
// over (d, row, head, page) for any strides, and its loads; and the instruction descriptor of
// the tensor core for either 16-bit type.
#pragma once

#include "cache_common.cuh"
#include "cache_kernels.h"
#include "tmap_host.h"

namespace ab {

constexpr int kBoxRows = 64;  // most rows of a page in one copy

__device__ __forceinline__ void tma_load_4d(void *smem_dst, const void *tmap, uint64_t *bar, int x,
                                            int y, int z, int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

template <typename E>
constexpr uint32_t idesc(int M, int N, int a_mn, int b_mn)
{
    return sizeof(E) && E::kBias == 0.f ? idesc_bf16_f32(M, N, a_mn, b_mn) : idesc_f16_f32(M, N, a_mn, b_mn);
}

// Map of 16-bit values over (d, rows, heads, batches), strides in elements; one box is 64 of d
// by box_rows rows, written with the 128-byte swizzle; rows behind the last read as zero. A
// dimension of one element gets a stride that is never used; a stride of 0 has no map.
inline bool rows_map(CUtensorMap *tm, const void *base, int d, int rows, int heads, int batches, int64_t row,
                     int64_t head, int64_t batch, int box_rows)
{
    EncodeTiledFn enc = tmap_encode_fn();
    if (!enc || !stride_maps(row, rows) || !stride_maps(head, heads) || !stride_maps(batch, batches)) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)heads, (cuuint64_t)batches};
    const cuuint64_t strides[3] = {2 * (cuuint64_t)(row ? row : d), 2 * (cuuint64_t)(head ? head : d),
                                   2 * (cuuint64_t)(batch ? batch : d)};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The pages' (d, row, head, page); a box is the rows of a page, 64 at most.
inline bool page_map(CUtensorMap *tm, const ab_cache &c, const void *base, int64_t row, int64_t head, int64_t pg)
{
    return rows_map(tm, base, c.d, c.page, c.Hk, c.n_pages, row, head, pg, c.page < kBoxRows ? c.page : kBoxRows);
}

// New tokens [B, Hk, T, d].
inline bool token_map(CUtensorMap *tm, const ab_cache &c, const ab_tokens &t, int T)
{
    return rows_map(tm, t.p, c.d, T, c.Hk, c.B, t.st, t.sh, t.sb, kBoxRows);
}

}  // namespace ab
