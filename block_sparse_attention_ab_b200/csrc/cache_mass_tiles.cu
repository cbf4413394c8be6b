// cache_mass_tiles.cu -- ab_cache_mass for many query rows per key head (a prompt's last
// tokens, a long accepted path): the 5th-generation tensor core.
//
// S^T = K Q^T with 128 keys as the rows of the product and up to 256 query rows as its
// columns, so a thread owns a key and adds its weights over the query rows in registers: no
// exchange between threads. One CTA per SM: a warp copies key tiles (TMA through the page map;
// what lies in rows that are no key's goes to sums that nobody writes), a warp issues the
// products into two tensor memory buffers of 256 columns, and eight warps per buffer (each
// thread every other 32 of its key's columns; the two sums meet in shared memory) compute
// p = 2^(s scale - lse), summed in fp32. Bound by the exponentials once there
// are more than about 160 rows (16 a cycle and SM), by reading K below that; a warp-level
// product with shared query fragments (cache_mass.cu) took 361 us against 129 us for 192 rows
// over 2 x 60000..118800 slots of 8 heads (eight summing warps: 147 us).
#include <cstdint>

#include "cache_common.cuh"
#include "cache_kernels.h"
#include "cache_tma.cuh"

namespace ab {
namespace {

constexpr int kSums = 512;     // threads that add: two buffers, two halves of the columns, four warps
constexpr int kThreads = kSums + 64;
constexpr int kWarpK = 16, kWarpS = 17;
constexpr int kKeys = 128;     // keys per unit
constexpr int kRows = 256;     // query rows per pass
constexpr int kEnt = 8;        // page slots of a unit, at most (16-token pages)
constexpr int kInfos = 16;

struct TileInfo {
    int page[kEnt];  // pool pages, -1: nothing there
};

template <int D>
struct MassSmem {
    static constexpr int kSlots = D == 128 ? 4 : 8;
    static constexpr int kQBox = kRows * 128;  // 64 of d of every query row
    static constexpr int kQ = kQBox * (D / 64);
    static constexpr int kTileBox = kKeys * 128, kTile = kTileBox * (D / 64);
    static constexpr int kRing = kQ;
    static constexpr int kLse = kRing + kSlots * kTile;  // -log-sum in base 2 [kRows]
    static constexpr int kBound = kLse + kRows * 4;      // the row sees slots below this
    static constexpr int kPart = kBound + kRows * 4;     // the second half's sums [2][2][kKeys]
    static constexpr int kInfo = kPart + 4 * kKeys * 4;
    static constexpr int kBars = kInfo + kInfos * (int)sizeof(TileInfo);
    // k_full, k_empty [kSlots], s_full, s_free [2], q_full, drain
    static constexpr int kNumBars = 2 * kSlots + 6;
    static constexpr int kMisc = kBars + kNumBars * 8;  // tensor memory address, abort flag, run
    static constexpr int kVoid = kMisc + 16 + 18 * 8 + 16;  // some row of these 32 adds nothing [kRows / 32]
    static constexpr int kBytes = kVoid + kRows / 32 * 4;
    static constexpr int kAlloc = kBytes + 1024;
    // info slot i is rewritten for unit i + kInfos, whose tile waits for the product of unit i +
    // kInfos - kSlots, which waits until the sets have read buffers (and info) of two units before
    static_assert(kSlots + 2 < kInfos && kAlloc <= 227 * 1024, "ring");
};

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1)
    cache_mass_tile_kernel(const CacheMass a, const __grid_constant__ CUtensorMap tmK)
{
    using L = MassSmem<D>;
    constexpr int NS = L::kSlots;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    float *nlse = reinterpret_cast<float *>(smem + L::kLse);
    int *bound = reinterpret_cast<int *>(smem + L::kBound);
    int *voids = reinterpret_cast<int *>(smem + L::kVoid);
    float *part = reinterpret_cast<float *>(smem + L::kPart);
    TileInfo *info = reinterpret_cast<TileInfo *>(smem + L::kInfo);
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::kBars), *k_empty = k_full + NS;
    uint64_t *s_full = k_empty + NS, *s_free = s_full + 2, *q_full = s_free + 2, *drain = q_full + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + L::kMisc + 8);
    long long *scan = reinterpret_cast<long long *>(smem + L::kMisc + 16);
    int *found = reinterpret_cast<int *>(smem + L::kMisc + 16 + 18 * 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int page = a.c.page, shift = a.page_shift;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_free[s], 8);
        }
        mbar_init(q_full, kSums);
        mbar_init(drain, 1);
        *abort = 0;
        fence_barrier_init();
    }
    if (warp == kWarpS) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    cudaGridDependencySynchronize();
    // ---- this CTA's run of units, in order of sequences and key heads
    int *flag0 = blockIdx.x == 0 ? a.flag : nullptr;  // one CTA reports the bad lengths and counts
    auto units_of = [&](int b, int *flag) {
        return (cache_len(a.c, a.c.length, b, flag) + kKeys - 1) / kKeys;
    };
    const int per = (a.c.B + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int b = tid * per; b < min((tid + 1) * per, a.c.B); ++b) {
        mine += (long long)units_of(b, flag0) * a.c.Hk;
        if (flag0) tok_count(a.n_tok, b, a.T, flag0);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) incl += scan[w];
        total += scan[w];
    }
    const long long lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
    if (lo < hi && lo >= incl - mine && lo < incl) {
        long long at = incl - mine;
        int b = tid * per;
        for (;; ++b) {
            const long long u = (long long)units_of(b, nullptr) * a.c.Hk;
            if (lo < at + u) break;
            at += u;
        }
        found[0] = b;
        *reinterpret_cast<long long *>(found + 2) = lo - at;
    }
    __syncthreads();

    // The run's pieces: units [u0, u1) of one key head of one sequence.
    struct Piece {
        int b, hk, u0, u1, len, n;
    };
    int run_b = lo < hi ? found[0] : 0;
    long long in_group = lo < hi ? *reinterpret_cast<long long *>(found + 2) : 0, left = hi - lo;
    auto next_piece = [&](Piece &p) -> bool {
        while (left > 0) {
            p.len = cache_len(a.c, a.c.length, run_b, nullptr);
            const int units = (p.len + kKeys - 1) / kKeys;
            if (in_group >= (long long)units * a.c.Hk) {
                in_group = 0;
                ++run_b;
                continue;
            }
            p.b = run_b;
            p.hk = (int)(in_group / units);
            p.u0 = (int)(in_group % units);
            p.u1 = (int)min((long long)units, p.u0 + left);
            p.n = min(tok_count(a.n_tok, p.b, a.T, nullptr), p.len);
            left -= p.u1 - p.u0;
            in_group += p.u1 - p.u0;
            return true;
        }
        return false;
    };
    auto wait = [&](uint64_t *bar, uint32_t phase) -> bool {
        return __all_sync(~0u, mbar_wait(bar, phase & 1, abort, a.flag));
    };
    Piece pc;

    if (warp == kWarpK) {
        if (elect_one()) prefetch_tmap(&tmK);
        __syncwarp();
        const int nent = max(1, kKeys >> shift), box_rows = min(page, kBoxRows), boxes = kKeys / box_rows;
        int it = 0, s = 0;
        uint32_t par_e = 1, phase = 0, loaded = 0;
        bool ok = true;
        while (ok && next_piece(pc)) {
            const int slots = (pc.len + page - 1) >> shift, rows = pc.n * a.G;
            for (int r0 = 0; ok && r0 < rows; r0 += kRows) {
                const int batch = 32 / nent;  // units whose pages are looked up together
                int pages = -1, behind = batch;
                for (int u = pc.u0; ok && u < pc.u1; ++u, ++it, ++behind) {
                    if (behind == batch) {
                        behind = 0;
                        const int uu = u + lane / nent, slot = ((uu * kKeys) >> shift) + lane % nent;
                        pages = uu < pc.u1 && slot < slots ? cache_page(a.c, pc.b, slot, a.flag) : -1;
                    }
                    const int pg = __shfl_sync(~0u, pages, (behind * nent + lane) & 31);
                    if (it >= NS) ok = wait(&k_empty[s], par_e);
                    if (!ok) break;
                    if (lane < nent) info[it % kInfos].page[lane] = pg;
                    __syncwarp();  // the info is written before the barrier is armed
                    uint8_t *tile = smem + L::kRing + s * L::kTile;
                    // lane: a box of rows; pages above 64 tokens take two
                    const int bp = __shfl_sync(~0u, pg, page > kBoxRows ? 0 : lane);
                    const bool has = lane < boxes && bp >= 0;
                    const uint32_t bytes = __popc(__ballot_sync(~0u, has)) * box_rows * (D * 2);
                    if (lane == 0) {
                        if (bytes)
                            mbar_arrive_expect_tx(&k_full[s], bytes);
                        else
                            mbar_arrive(&k_full[s]);
                    }
                    __syncwarp();
                    loaded = bytes ? loaded | 1u << s : loaded & ~(1u << s);
                    if (has) {
                        const int row = page > kBoxRows ? lane * kBoxRows : 0;
#pragma unroll
                        for (int y = 0; y < D / 64; ++y)
                            tma_load_4d(tile + y * L::kTileBox + lane * box_rows * 128, &tmK, &k_full[s], y * 64, row,
                                        pc.hk, bp);
                    }
                    phase ^= 1u << s;
                    __syncwarp();
                    if (++s == NS) {
                        s = 0;
                        par_e ^= 1;
                    }
                }
            }
        }
        if (!ok) {  // copies that may still be in flight land before the CTA ends
            for (int x = 0; x < NS; ++x)
                if (loaded >> x & 1) drain_wait(&k_full[x], (phase >> x & 1) ^ 1);
        }
    } else if (warp == kWarpS) {
        const uint64_t qd = smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + L::kRing), 16, 1024);
        int it = 0, s = 0;
        uint32_t tiles = 0, q = 0;
        bool ok = true;
        while (ok && next_piece(pc)) {
            const int rows = pc.n * a.G;
            for (int r0 = 0; ok && r0 < rows; r0 += kRows) {
                const uint32_t id = idesc<E>(kKeys, (min(kRows, rows - r0) + 31) & ~31, 0, 0);
                ok = wait(q_full, q++);
                for (int u = pc.u0; ok && u < pc.u1; ++u, ++it) {
                    ok = wait(&k_full[s], tiles >> s);
                    tiles ^= 1u << s;
                    if (ok && it >= 2) ok = wait(&s_free[it & 1], (it >> 1) - 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t kd = kd0 + (uint64_t)s * (L::kTile >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss(tmem + (it & 1) * kRows, kd + ((kk >> 2) * L::kTileBox + (kk & 3) * 32 >> 4),
                                   qd + ((kk >> 2) * L::kQBox + (kk & 3) * 32 >> 4), id, kk > 0);
                        mma_commit(&s_full[it & 1]);
                        mma_commit(&k_empty[s]);
                    }
                    __syncwarp();
                    if (++s == NS) s = 0;
                }
            }
        }
        if (!ok) {
            if (elect_one()) {
                mma_commit(drain);
                drain_wait(drain, 0);
            }
            __syncwarp();
        }
    } else {
        // ---- the sums. After a failed wait these warps run out their loops (they meet at named
        // barriers) and write nothing.
        const int set = warp >> 2 & 1, half = warp >> 3, th = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        bool ok = true;
        int it = 0;
        while (next_piece(pc)) {
            const int rows = pc.n * a.G, old_len = pc.len - pc.n;
            if (rows == 0) {  // nothing to add: the masses as they are
                if (a.out != a.c.mass)
                    for (int key = pc.u0 * kKeys + tid; key < min(pc.len, pc.u1 * kKeys); key += kSums) {
                        const int pg = cache_page(a.c, pc.b, key >> shift, a.flag);
                        if (pg < 0) continue;
                        const int64_t at = ((int64_t)pg * a.c.Hk + pc.hk) * page + (key & (page - 1));
                        a.out[at] = a.c.mass[at];
                    }
                continue;
            }
            for (int r0 = 0; r0 < rows; r0 += kRows) {
                const int nr = min(kRows, rows - r0), np = (nr + 31) & ~31;
                // the products that read the last rows are done when everybody is here
                asm volatile("bar.sync 1, %0;" ::"n"(kSums) : "memory");
                auto row_of = [&](int r) -> int {  // row of q and lse, or -1
                    if (r >= rows) return -1;
                    const int k = r / a.G, t = a.sel ? a.sel[(size_t)pc.b * a.T + k] : k;
                    return (unsigned)t < (unsigned)a.T ? t : -1;
                };
                static_assert(kRows <= kSums, "a thread per row");
                if (tid < np) {  // whole warps: np is a multiple of 32
                    const int r = r0 + tid, t = row_of(r);
                    float nl = -INFINITY;
                    if (t >= 0) {
                        const int h = pc.hk * a.G + r % a.G;
                        const float l = a.lse[((size_t)pc.b * a.c.Hk * a.G + h) * a.T + t];
                        if (l != -INFINITY) nl = -l * 1.4426950408889634f;
                    } else if (r < rows) {
                        raise_flag(a.flag, AB_FLAG_BAD_INDEX);
                    }
                    // a row that does not exist or saw nothing adds nothing, whatever its logit
                    const bool none = nl == -INFINITY;
                    nlse[tid] = nl;
                    bound[tid] = none ? 0 : old_len + r / a.G + 1;
                    const bool some = __any_sync(~0u, none);
                    if (lane == 0) voids[warp] = some;
                }
                constexpr int kChunks = D / 8;
#pragma unroll 4
                for (int i = tid; i < np * kChunks; i += kSums) {
                    const int r = i / kChunks, c = i % kChunks, t = row_of(r0 + r);
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (t >= 0) {
                        const int h = pc.hk * a.G + (r0 + r) % a.G;
                        x = *reinterpret_cast<const uint4 *>(static_cast<const char *>(a.q.p) +
                                                             2 * (pc.b * a.q.sb + h * a.q.sh + t * a.q.st) + c * 16);
                    }
                    *reinterpret_cast<uint4 *>(smem + (c >> 3) * L::kQBox + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
                }
                fence_proxy_async_smem();
                mbar_arrive(q_full);
                asm volatile("bar.sync 1, %0;" ::"n"(kSums) : "memory");
                for (int u = pc.u0; u < pc.u1; ++u, ++it) {
                    if ((it & 1) != set) continue;
                    if (ok) ok = wait(&s_full[set], it >> 1);
                    tc_fence_after();
                    const int key = u * kKeys + th;
                    int64_t at = -1;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f}, old = 0.f;
                    if (half == 0 && ok && key < pc.len) {
                        const int pg = info[it % kInfos].page[page >= kKeys ? 0 : th >> shift];
                        if (pg >= 0) {
                            at = ((int64_t)pg * a.c.Hk + pc.hk) * page + (key & (page - 1));
                            old = (r0 ? a.out : a.c.mass)[at];
                        }
                    }
                    __syncwarp();
                    const bool edge = (u + 1) * kKeys > old_len;
                    for (int c0 = 32 * half; c0 < np; c0 += 64) {
                        const bool masked = edge || voids[c0 >> 5];
                        uint32_t x[32];
                        tmem_ld32(tmem + lanes + set * kRows + c0, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 nl = *reinterpret_cast<const float4 *>(nlse + c0 + j);
                            float y[4] = {fmaf(__uint_as_float(x[j]), a.scale_log2, nl.x),
                                          fmaf(__uint_as_float(x[j + 1]), a.scale_log2, nl.y),
                                          fmaf(__uint_as_float(x[j + 2]), a.scale_log2, nl.z),
                                          fmaf(__uint_as_float(x[j + 3]), a.scale_log2, nl.w)};
                            if (masked) {
                                const int4 bd = *reinterpret_cast<const int4 *>(bound + c0 + j);
                                if (key >= bd.x) y[0] = -INFINITY;
                                if (key >= bd.y) y[1] = -INFINITY;
                                if (key >= bd.z) y[2] = -INFINITY;
                                if (key >= bd.w) y[3] = -INFINITY;
                            }
#pragma unroll
                            for (int z = 0; z < 4; ++z) sum[z] += fast_exp2(y[z]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_free[set]);
                    // the halves meet; a buffer's next sums go to the other place
                    const float mine = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    float *other = part + (2 * set + (it >> 1 & 1)) * kKeys + th;
                    if (half == 1) *other = mine;
                    asm volatile("bar.sync %0, 256;" ::"r"(2 + set) : "memory");
                    if (at >= 0) a.out[at] = old + (mine + *other);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpS) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <typename E, int D>
cudaError_t launch_one(const CacheMass &a, const CUtensorMap &tk, cudaStream_t st)
{
    return launch_kernel(cache_mass_tile_kernel<E, D>, dim3(kCacheSms), kThreads, MassSmem<D>::kAlloc,
                         MassSmem<D>::kAlloc, 1, st, a, tk);
}

}  // namespace

cudaError_t launch_cache_mass_tiles(const CacheMass &a, cudaStream_t st)
{
    CUtensorMap tk;
    const ab_cache &c = a.c;
    if (!page_map(&tk, c, c.k, c.k_row, c.k_head, c.k_page)) return cudaErrorInvalidValue;
    if (c.dtype == AB_F16) return c.d == 64 ? launch_one<Fp16, 64>(a, tk, st) : launch_one<Fp16, 128>(a, tk, st);
    return c.d == 64 ? launch_one<Bf16, 64>(a, tk, st) : launch_one<Bf16, 128>(a, tk, st);
}

}  // namespace ab
