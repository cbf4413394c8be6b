// cache_tiles.cu -- ab_cache_attn for many query rows per key head (a tree of drafted tokens
// times the heads that share a key head): the 5th-generation tensor core.
//
// One CTA holds one to three halves of 128 query rows and walks units of 64 keys
// (cache_sched.cuh); for each half in turn
//   S = Q K^T (128 x 64) -> softmax in registers, a thread per row, four warps per half ->
//   P over S's own tensor memory -> O += P V (128 x d, fp32 in tensor memory).
// S has several buffers, so the products of the next halves run while a half's threads work
// on theirs. With one half two CTAs share an SM; with two or three, every tile of keys is
// read once for all of them (320 rows: 3 halves fill tensor memory, 384 columns of O and two
// S buffers, against three CTAs that read it three times). Units whose 64 keys all
// exist come by TMA through a map over (d, row, head, page): the page's number is a coordinate,
// so any strides and page sizes do, and pages of 16 and 32 tokens are 4 and 2 boxes of one
// tile. The others (a sequence's last keys, the new tokens, a tile with an absent page) are
// written by the softmax threads themselves, with zeros where no key is, in the same swizzle;
// a run is walked from its end, so that this happens while the first copies are on their way.
// CTAs of the row tiles of one key head take the same runs and share K and V in L2.
#include <cstdint>

#include "cache_common.cuh"
#include "cache_kernels.h"
#include "cache_sched.cuh"
#include "tmap_host.h"

namespace ab {
namespace {

constexpr int kRows = 128;                 // query rows of a half: lanes of tensor memory
constexpr int kEnt = 4;                    // page slots of a unit, at most (16-token pages)

struct TileInfo {
    Staged ent[kEnt];
    int manual;  // the softmax threads write this unit's tile
};

// NH halves; tensor memory: kSBufs S buffers of 64 columns, then NH accumulators of D.
template <int D, int NH>
struct TileSmem {
    static constexpr int kThreads = NH * 128 + 64;  // four softmax warps per half, TMA, MMA
    static constexpr int kWarpTma = NH * 4, kWarpMma = NH * 4 + 1;
    static constexpr int kSBufs = NH == 1 ? 2 : NH == 2 ? 4 : D == 128 ? 2 : 4;
    static constexpr int kColO = kSBufs * kUnit;
    static constexpr int kTmemCols = NH == 1 ? 256 : 512;
    static_assert(kColO + NH * D <= kTmemCols, "tensor memory");
    static constexpr int kStages = (D == 128 ? (NH == 1 ? 2 : 7 - NH) : (NH == 1 ? 4 : 8));
    static constexpr int kBoxes = D / 64;
    static constexpr int kQHalf = kRows * D * 2;
    static constexpr int kQBytes = NH * kQHalf;
    static constexpr int kTile = kUnit * D * 2;  // one K or V tile
    static constexpr int kKv = kQBytes;          // [stage][K, V]
    static constexpr int kInfo = kKv + kStages * 2 * kTile;
    static constexpr int kBars = (kInfo + kStages * (int)sizeof(TileInfo) + 7) / 8 * 8;
    // info_full, kv_full, filled, kv_empty [stages], s_full [NH][2], p_full [kSBufs], q_full,
    // pv_done [NH], drain. A parity wait is exact for a waiter that sees every phase: s_full
    // belongs to a half (its even and odd units), p_full to the MMA warp, which waits for
    // every job in turn.
    static constexpr int kNumBars = 4 * kStages + 2 * NH + kSBufs + 2 * NH + 1;
    static constexpr int kMisc = kBars + kNumBars * 8;  // tensor memory address, abort flag
    static constexpr int kRun = kMisc + 16;
    static constexpr int kBytes = kRun + (int)sizeof(RunSmem);
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= (NH == 1 ? 113 : 227) * 1024, "shared memory");
};

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

template <typename E, int D, int NH>
__global__ void __launch_bounds__(TileSmem<D, NH>::kThreads, NH == 1 ? 2 : 1)
    cache_tile_kernel(const CacheAttn a, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV)
{
    using L = TileSmem<D, NH>;
    constexpr int NS = L::kStages, SB = L::kSBufs, kColO = L::kColO;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    TileInfo *info = reinterpret_cast<TileInfo *>(smem + L::kInfo);
    uint64_t *info_full = reinterpret_cast<uint64_t *>(smem + L::kBars);
    uint64_t *kv_full = info_full + NS;  // by TMA
    uint64_t *filled = kv_full + NS;     // by the softmax threads
    uint64_t *kv_empty = filled + NS;
    uint64_t *s_full = kv_empty + NS, *p_full = s_full + 2 * NH;
    uint64_t *q_full = p_full + SB, *pv_done = q_full + NH, *drain = pv_done + NH;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + L::kMisc + 8);
    RunSmem &run_sm = *reinterpret_cast<RunSmem *>(smem + L::kRun);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, nct = gridDim.x, rt = blockIdx.y, row0 = rt * NH * kRows;
    const int page = a.c.page, shift = a.page_shift;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&info_full[s], 1);
            mbar_init(&kv_full[s], 1);
            mbar_init(&filled[s], 128);
            mbar_init(&kv_empty[s], 1);
        }
        for (int s = 0; s < SB; ++s) mbar_init(&p_full[s], 128);
        for (int h = 0; h < NH; ++h) {
            mbar_init(&s_full[2 * h], 1);
            mbar_init(&s_full[2 * h + 1], 1);
            mbar_init(&q_full[h], 128);
            mbar_init(&pv_done[h], 1);
        }
        mbar_init(drain, 1);
        *abort = 0;
        fence_barrier_init();
    }
    if (warp == L::kWarpMma) {
        tmem_alloc(tmem_slot, L::kTmemCols);
        tmem_relinquish();
    }
    int *flag0 = rt == 0 ? a.flag : nullptr;  // one report per bad length or count
    Run run = find_run<L::kThreads>(a, run_sm, cta, nct, flag0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Piece pc;

    auto wait = [&](uint64_t *bar, int n) -> bool {  // phase n of bar
        return __all_sync(~0u, mbar_wait(bar, n & 1, abort, a.flag));
    };

    if (warp == L::kWarpTma) {
        if (elect_one()) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
        }
        __syncwarp();
        const int nent = max(1, kUnit >> shift), box_rows = min(page, kUnit);
        int it = 0;
        uint32_t phase = 0, loaded = 0;  // bit s: parity of stage s's next copy; its last unit came by TMA
        bool ok = true;
        while (ok && next_piece(a, run, nct, pc, nullptr)) {
            if (row0 >= group_rows(a, pc.g)) continue;
            const int cap = cache_len(a.c, a.c.length, pc.g.b, flag0);
            const int slots = (pc.g.ctx + page - 1) >> shift;
            for (int u = pc.u1 - 1; ok && u >= pc.u0; --u, ++it) {
                const int s = it % NS;
                Staged e = {-1, 0, 0.f};
                const int slot = ((u * kUnit) >> shift) + lane;
                const bool ctx = u < pc.g.ctx_units;
                if (ctx && lane < nent && slot < slots) e = stage_entry(a, pc, slot, cap);
                const int r0 = page > kUnit ? (u * kUnit) & (page - 1) : 0;
                const bool clean = lane >= nent || (e.page >= 0 && e.valid >= r0 + box_rows);
                const bool manual = !__all_sync(~0u, clean);
                if (it >= NS) ok = wait(&kv_empty[s], it / NS - 1);
                if (!ok) break;
                if (lane < nent) info[s].ent[lane] = e;
                if (lane == 0) info[s].manual = manual;
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&info_full[s]);
                    if (!manual) mbar_arrive_expect_tx(&kv_full[s], 2 * L::kTile);
                }
                __syncwarp();
                loaded = manual ? loaded & ~(1u << s) : loaded | 1u << s;
                if (!manual) phase ^= 1u << s;
                if (!manual && lane < nent) {
                    uint8_t *k = smem + L::kKv + s * 2 * L::kTile + lane * box_rows * 128;
#pragma unroll
                    for (int x = 0; x < L::kBoxes; ++x)
                        tma_load_4d(k + x * (kUnit * 128), &tmK, &kv_full[s], x * 64, r0, pc.hk, e.page);
#pragma unroll
                    for (int x = 0; x < L::kBoxes; ++x)
                        tma_load_4d(k + L::kTile + x * (kUnit * 128), &tmV, &kv_full[s], x * 64, r0, pc.hk,
                                    e.page);
                }
                __syncwarp();
            }
        }
        if (!ok) {  // copies that may still be in flight land before the CTA ends
            for (int s = 0; s < NS; ++s)
                if (loaded >> s & 1) drain_wait(&kv_full[s], (phase >> s & 1) ^ 1);
        }
    } else if (warp == L::kWarpMma) {
        constexpr uint32_t idesc_s = idesc<E>(kRows, kUnit, 0, 0), idesc_o = idesc<E>(kRows, D, 0, 1);
        const uint64_t qd = smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + L::kKv), 16, 1024);
        const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + L::kKv + L::kTile), kUnit * 128, 1024);
        int it = 0, job = 0;  // units and (unit, half) jobs before this piece
        uint32_t copied = 0, written = 0;  // bit s: parity of stage s's next copy / next written tile
        uint32_t qphase = 0;               // bit h: parity of half h's next Q
        uint32_t odd = 0;                  // bit h: half h's next unit is an odd one of its own
        bool ok = true;
        int na = 1;  // halves with rows in this piece
        // job j of the piece: unit j / na, half j % na
        auto issue_s = [&](int j) {
            const int i = it + j / na, h = j % na, s = i % NS, buf = (job + j) % SB;
            if (h == 0) {
                if (!wait(&info_full[s], i / NS)) return false;
                const bool manual = info[s].manual;
                if (!(manual ? wait(&filled[s], written >> s) : wait(&kv_full[s], copied >> s))) return false;
                if (manual)
                    written ^= 1u << s;
                else
                    copied ^= 1u << s;
                tc_fence_after();
            }
            const uint64_t kd = kd0 + (uint64_t)s * (2 * L::kTile >> 4);
            const uint64_t qh = qd + (uint64_t)h * (L::kQHalf >> 4);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + buf * kUnit, qh + ((kk >> 2) * (kRows * 128) + (kk & 3) * 32 >> 4),
                           kd + ((kk >> 2) * (kUnit * 128) + (kk & 3) * 32 >> 4), idesc_s, kk > 0);
                mma_commit(&s_full[2 * h + (odd >> h & 1)]);
            }
            odd ^= 1u << h;
            __syncwarp();
            return true;
        };
        while (ok && next_piece(a, run, nct, pc, nullptr)) {
            const int rows = group_rows(a, pc.g) - row0;
            if (rows <= 0) continue;
            na = min(NH, (rows + kRows - 1) / kRows);
            const int n = (pc.u1 - pc.u0) * na;
            for (int h = 0; ok && h < na; ++h) {
                ok = wait(&q_full[h], qphase >> h);
                qphase ^= 1u << h;
            }
            tc_fence_after();
            // S products ahead of the softmax: as many as there are buffers, two per half
            const int ahead = min(SB, 2 * na);
            for (int j = 0; ok && j < min(ahead, n); ++j) ok = issue_s(j);
            for (int j = 0; ok && j < n; ++j) {
                const int buf = (job + j) % SB, h = j % na, s = (it + j / na) % NS;
                ok = wait(&p_full[buf], (job + j) / SB);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vd = vd0 + (uint64_t)s * (2 * L::kTile >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kUnit / 16; ++kk)
                        mma_ts(tmem + kColO + h * D, tmem + buf * kUnit + kk * 8, vd + (kk * 2048 >> 4), idesc_o,
                               j >= na || kk > 0);
                    mma_commit(&pv_done[h]);
                    if (h == na - 1) mma_commit(&kv_empty[s]);
                }
                __syncwarp();
                if (j + ahead < n) ok = issue_s(j + ahead);
            }
            it += pc.u1 - pc.u0;
            job += n;
        }
        if (!ok) {
            if (elect_one()) {
                mma_commit(drain);
                drain_wait(drain, 0);
            }
            __syncwarp();
        }
    } else {
        // ---- softmax: thread = query row. After a failed wait a warp runs out its loops
        // without waiting, and reads no page.
        bool ok = true;
        auto wait_on = [&](uint64_t *bar, int n) {
            if (ok) ok = wait(bar, n);
        };
        const int half = warp >> 2, th = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t acc = tmem + lanes + kColO + half * D;
        int it = 0, job = 0;  // units and jobs before this piece
        int pv = 0;           // products of this half so far
        while (next_piece(a, run, nct, pc, half == 0 ? flag0 : nullptr)) {
            const int rows = group_rows(a, pc.g);
            if (row0 >= rows) continue;
            const int na = min(NH, (rows - row0 + kRows - 1) / kRows);
            if (half >= na) {
                it += pc.u1 - pc.u0;
                job += (pc.u1 - pc.u0) * na;
                continue;
            }
            const int hrow0 = row0 + half * kRows, row = hrow0 + th, b = pc.g.b;
            const bool live = row < rows, warp_live = hrow0 + (warp & 3) * 32 < rows;
            const int t = a.per_token ? pc.g.tp : row / a.G;
            const int h = pc.hk * a.G + (a.per_token ? row : row % a.G);
            // Q rows into the swizzled operand tile: the previous piece's products are done
            {
                constexpr int kChunks = D / 8;
                const int left = min(kRows, rows - hrow0);
#pragma unroll 8
                for (int i = th; i < kRows * kChunks; i += 128) {
                    const int r = i / kChunks, c = i % kChunks;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (r < left) {
                        const int rr = hrow0 + r, tt = a.per_token ? pc.g.tp : rr / a.G;
                        const int hh = pc.hk * a.G + (a.per_token ? rr : rr % a.G);
                        x = *reinterpret_cast<const uint4 *>(
                            static_cast<const char *>(a.q.p) +
                            2 * (b * a.q.sb + hh * a.q.sh + tt * a.q.st) + c * 16);
                    }
                    *reinterpret_cast<uint4 *>(smem + half * L::kQHalf + (c >> 3) * (kRows * 128) + r * 128 +
                                               (((c & 7) ^ (r & 7)) << 4)) = x;
                }
                fence_proxy_async_smem();
                mbar_arrive(&q_full[half]);
            }
            float m = -INFINITY, l = 0.f;
            job += half;
            for (int u = pc.u1 - 1; u >= pc.u0; --u, ++it, job += na, ++pv) {
                const int s = it % NS, buf = job % SB;
                const bool ctx = u < pc.g.ctx_units;
                wait_on(&info_full[s], it / NS);
                const TileInfo &ti = info[s];
                const bool manual = ok && ti.manual;
                const int j0 = ctx ? 0 : (u - pc.g.ctx_units) * kUnit;  // first new token
                uint64_t sees = ~0ull;  // this row's keys of the unit
                if (manual && half == 0) {
                    constexpr int kChunks = D / 8;
                    uint8_t *kt = smem + L::kKv + s * 2 * L::kTile;
                    const char *kn = static_cast<const char *>(a.k.p) + 2 * (b * a.k.sb + pc.hk * a.k.sh);
                    const char *vn = static_cast<const char *>(a.v.p) + 2 * (b * a.v.sb + pc.hk * a.v.sh);
#pragma unroll 4
                    for (int i = th; i < kUnit * kChunks; i += 128) {
                        const int j = i / kChunks, c = i % kChunks;
                        uint4 x = make_uint4(0, 0, 0, 0), y = x;
                        if (!ctx) {
                            if (j0 + j < pc.g.n) {
                                x = ldg_stream(kn + 2 * (j0 + j) * a.k.st + c * 16);
                                y = ldg_stream(vn + 2 * (j0 + j) * a.v.st + c * 16);
                            }
                        } else {
                            const Staged e = ti.ent[page >= kUnit ? 0 : j >> shift];
                            const int64_t r = (u * kUnit + j) & (page - 1);
                            if (e.page >= 0 && r < e.valid) {
                                x = ldg_stream(static_cast<const char *>(a.c.k) +
                                               2 * (e.page * a.c.k_page + pc.hk * a.c.k_head + r * a.c.k_row) +
                                               c * 16);
                                y = ldg_stream(static_cast<const char *>(a.c.v) +
                                               2 * (e.page * a.c.v_page + pc.hk * a.c.v_head + r * a.c.v_row) +
                                               c * 16);
                            }
                        }
                        uint8_t *d = kt + (c >> 3) * (kUnit * 128) + j * 128 + (((c & 7) ^ (j & 7)) << 4);
                        *reinterpret_cast<uint4 *>(d) = x;
                        *reinterpret_cast<uint4 *>(d + L::kTile) = y;
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&filled[s]);
                }
                if (manual) {
                    sees = 0;
                    if (ctx) {
#pragma unroll
                        for (int e = 0; e < kEnt; ++e) {
                            // keys e * 16 .. e * 16 + 15 lie in one page
                            const Staged x = ti.ent[page >= kUnit ? 0 : (e * 16) >> shift];
                            const int r = (u * kUnit + e * 16) & (page - 1);
                            const int nv = x.page >= 0 ? min(16, max(0, x.valid - r)) : 0;
                            sees |= (uint64_t)((1u << nv) - 1) << (16 * e);
                        }
                    } else if (live) {
                        const int nv = min(kUnit, pc.g.n - j0);
                        if (a.tree) {
                            const uint8_t *tr = a.tree + ((size_t)b * a.T + t) * a.T + j0;
#pragma unroll 8
                            for (int j = 0; j < nv; ++j) sees |= (uint64_t)(tr[j] != 0) << j;
                        } else {
                            const int nk = min(nv, max(0, t - j0 + 1));
                            sees = nk >= 64 ? ~0ull : (1ull << nk) - 1;
                        }
                    }
                }
                float sh[kEnt];
#pragma unroll
                for (int e = 0; e < kEnt; ++e)
                    sh[e] = a.w && ctx ? ti.ent[page >= kUnit ? 0 : (e * 16) >> shift].shift : 0.f;
                wait_on(&s_full[2 * half + (pv & 1)], pv >> 1);
                tc_fence_after();
                const uint32_t st = tmem + lanes + buf * kUnit;
                if (warp_live) {
                    uint32_t x0[32], x1[32];
                    tmem_ld32(st, x0);
                    tmem_ld32(st + 32, x1);
                    tmem_wait_ld();
                    auto at = [&](int j) -> uint32_t & { return j < 32 ? x0[j] : x1[j - 32]; };
                    // in units of the scaled base-2 logit
                    if (manual || a.w) {
#pragma unroll
                        for (int j = 0; j < kUnit; ++j) {
                            const float v = fmaf(__uint_as_float(at(j)), a.scale_log2, sh[j >> 4]);
                            at(j) = __float_as_uint(sees >> j & 1 ? v : -INFINITY);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < kUnit; ++j)
                            at(j) = __float_as_uint(__uint_as_float(at(j)) * a.scale_log2);
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < kUnit; j += 8)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            mx[y] = fmax3(mx[y], __uint_as_float(at(j + 2 * y)), __uint_as_float(at(j + 2 * y + 1)));
                    const float mt = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                    if (__any_sync(~0u, mt > m + kLazy)) {
                        const float mn = fmaxf(m, mt);
                        const float f = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
                        m = mn;
                        l *= f;
                        if (u != pc.u1 - 1) {  // the accumulator holds this piece's earlier units
                            wait_on(&pv_done[half], pv - 1);
                            tc_fence_after();
#pragma unroll 1
                            for (int ch = 0; ch < D / 32; ++ch) {
                                uint32_t o[32];
                                tmem_ld32(acc + ch * 32, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st32(acc + ch * 32, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float mb = m == -INFINITY ? 0.f : m - E::kBias;
                    float ls[4] = {0.f, 0.f, 0.f, 0.f};
                    uint32_t p[32];
#pragma unroll
                    for (int j = 0; j < kUnit; j += 2) {
                        const float p0 = fast_exp2(__uint_as_float(at(j)) - mb);
                        const float p1 = fast_exp2(__uint_as_float(at(j + 1)) - mb);
                        ls[(j >> 1) & 3] += p0 + p1;
                        p[j >> 1] = E::pack(p0, p1);  // rounded for the second product, the sum is not
                    }
                    l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                    tmem_st32(st, p);
                    tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(&p_full[buf]);
            }
            // ---- the piece's end: rows out, or into the workspace
            job -= half;
            wait_on(&pv_done[half], pv - 1);
            tc_fence_after();
            const bool whole = pc.u0 == 0 && pc.u1 == pc.g.units;
            const int item = ((b * a.c.Hk + pc.hk) * a.Tp + pc.g.tp) * a.row_tiles + rt;
            if (tid == 0) {  // half 0 has rows whenever another half has
                if (pc.u0 == 0) a.info[item].x = cta;
                if (pc.u1 == pc.g.units) a.info[item].y = cta;
            }
            const size_t slot = ((size_t)rt * nct + cta) * 2 + (pc.u0 == 0 ? 1 : 0);
            const size_t orow = ((size_t)b * a.c.Hk * a.G + h) * a.T + t;
            const float inv = !whole ? 1.f : l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
            if (live) {
                if (!whole)
                    a.part_ml[slot * (NH * kRows) + tid] = make_float2(m, l);
                else if (a.lse)
                    a.lse[orow] = l == 0.f ? -INFINITY : (m - E::kBias + log2f(l)) * kLn2;
            }
            if (warp_live) {
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t o[32];
                    tmem_ld32(acc + ch * 32, o);
                    tmem_wait_ld();
                    if (live) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] = __float_as_uint(l == 0.f ? 0.f : __uint_as_float(o[j]) * inv);
                        if (!whole || a.out_f32) {
                            float *d = whole ? static_cast<float *>(a.out) + orow * D
                                             : a.part + (slot * (NH * kRows) + tid) * D;
                            uint4 *v = reinterpret_cast<uint4 *>(d + ch * 32);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                v[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                        } else {
                            uint4 *v = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + orow * D + ch * 32);
                            auto f = [&](int j) { return E::pack(__uint_as_float(o[j]), __uint_as_float(o[j + 1])); };
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                v[j] = make_uint4(f(8 * j), f(8 * j + 2), f(8 * j + 4), f(8 * j + 6));
                        }
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == L::kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Map over the pages' (d, row, head, page); one box is 64 of d by the rows of a page (64 at
// most), written with the 128-byte swizzle. A dimension of one element gets a stride that
// is never used.
bool page_map(CUtensorMap *tm, const ab_cache &c, const void *base, int64_t row, int64_t head, int64_t pg)
{
    EncodeTiledFn enc = tmap_encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.page, (cuuint64_t)c.Hk, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {2 * (cuuint64_t)(row ? row : c.d), 2 * (cuuint64_t)(head ? head : c.d),
                                   2 * (cuuint64_t)(pg ? pg : c.d)};
    const cuuint32_t box[4] = {64, (cuuint32_t)(c.page < kUnit ? c.page : kUnit), 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename E, int D, int NH>
cudaError_t launch_one(const CacheAttn &a, int nct, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t st)
{
    using L = TileSmem<D, NH>;
    auto kern = cache_tile_kernel<E, D, NH>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
    if (e != cudaSuccess) return e;
    kern<<<dim3(nct, a.row_tiles), L::kThreads, L::kAlloc, st>>>(a, tk, tv);
    return cudaGetLastError();
}

template <typename E, int D>
cudaError_t launch_halves(const CacheAttn &a, const CacheAttnPlan &p, const CUtensorMap &tk, const CUtensorMap &tv,
                          cudaStream_t st)
{
    switch (p.tile_rows / kRows) {
    case 1: return launch_one<E, D, 1>(a, p.ctas, tk, tv, st);
    case 2: return launch_one<E, D, 2>(a, p.ctas, tk, tv, st);
    default: return launch_one<E, D, 3>(a, p.ctas, tk, tv, st);
    }
}

}  // namespace

cudaError_t launch_cache_tiles(const CacheAttn &a, const CacheAttnPlan &p, cudaStream_t st)
{
    CUtensorMap tk, tv;
    const ab_cache &c = a.c;
    if (!page_map(&tk, c, c.k, c.k_row, c.k_head, c.k_page) || !page_map(&tv, c, c.v, c.v_row, c.v_head, c.v_page))
        return cudaErrorInvalidValue;
    if (c.dtype == AB_F16)
        return c.d == 64 ? launch_halves<Fp16, 64>(a, p, tk, tv, st) : launch_halves<Fp16, 128>(a, p, tk, tv, st);
    return c.d == 64 ? launch_halves<Bf16, 64>(a, p, tk, tv, st) : launch_halves<Bf16, 128>(a, p, tk, tv, st);
}

}  // namespace ab
