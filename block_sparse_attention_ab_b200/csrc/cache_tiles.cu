// cache_tiles.cu -- ab_cache_attn for many query rows per key head (a tree of drafted tokens
// times the heads that share a key head): the 5th-generation tensor core.
//
// One CTA per SM holds one to three halves of 128 query rows and walks units of 64 keys
// (cache_sched.cuh), so a key tile is read once for up to 384 rows. For each half in turn
//   S = Q K^T (128 x 64, in one of a few tensor memory buffers) -> softmax in registers, four
//   warps per half, a thread per row -> P (shared memory) -> O += P V (tensor memory, fp32).
// S leaves its buffer as soon as a half's threads have loaded it, so two buffers serve three
// halves (their accumulators fill the other 384 of 512 columns) and every half's threads find
// their next S waiting. A 64-token tree over 8 x 16001..32760 slots, 40 / 8 heads (320 rows; floor
// 125 us) takes 365 us where the keys change from call to call, 562 TFLOP/s. What each step was
// worth, on unchanged keys: P over S's buffer, held until the second product, and one warp for
// all copies and products 490 us; P in shared memory and four independent warps 387 us; partial
// units by the copying warps, so that the softmax waits for S alone, 350 us; those by TMA 326 us.
// Halves of a second CTA that read K and V again took 537 us. What bounds it now: the chain from
// S to P of each half (a unit takes about 4100 cycles under ncu, of which the tensor core is busy
// 43%) and shared memory bandwidth, of which the products' operands use 47% and the threads 12%.
// Fetching units into L2 ahead, spinning or one-lane waits, a later wait for the second product
// and cheaper exponentials changed nothing; one thread instead of a converged warp issuing the
// products took 394 us.
// Units whose 64 keys all exist come by TMA through a map over (d, row, head, page): the page's
// number is a coordinate, so any strides and page sizes do, and pages of 16 and 32 tokens are 4
// and 2 boxes of one tile. The others (a sequence's last keys, the new tokens, a tile with an
// absent page) come the same way, the new tokens through a map of their own; a key that does
// not exist is masked out of S whatever its row holds, and its row of V is set to zero once the
// copy is there (0 * NaN is NaN). New tokens with a stride of 0 are written by the copying
// warps' lanes.
#include <cstdint>

#include "cache_common.cuh"
#include "cache_kernels.h"
#include "cache_sched.cuh"
#include "cache_tma.cuh"

namespace ab {
namespace {

constexpr int kRows = 128;                 // query rows of a half: lanes of tensor memory
static_assert(kUnit == kBoxRows, "a unit is one copy of a page of 64 tokens or more");
constexpr int kEnt = 4;                    // page slots of a unit, at most (16-token pages)

struct TileInfo {
    Staged ent[kEnt];
    int partial;  // some of the unit's keys do not exist
};

// NH halves. Tensor memory: kSBufs S buffers of 64 columns, then NH accumulators of D.
// Shared memory: Q and P of every half, a ring of K tiles and one of V tiles. Four warps
// beside the softmax: one copies K, one V, one issues S = Q K^T, one O += P V. Each waits for
// its own needs only, so neither a late copy nor a late P holds back anything else, and each
// warp's loop is short enough to keep ahead of the tensor core (all four roles in one polling
// warp: 510 us for the case above).
template <int D, int NH>
struct TileSmem {
    static constexpr int kThreads = NH * 128 + 128;  // four softmax warps per half
    static constexpr int kWarpK = NH * 4, kWarpV = kWarpK + 1, kWarpS = kWarpK + 2, kWarpO = kWarpK + 3;
    static constexpr int kSBufs = NH == 3 && D == 128 ? 2 : 4;
    static constexpr int kColO = kSBufs * kUnit;
    static constexpr int kTmemCols = 512;
    static_assert(kColO + NH * D <= kTmemCols, "tensor memory");
    static constexpr int kBoxes = D / 64;
    static constexpr int kQHalf = kRows * D * 2;
    static constexpr int kPHalf = kRows * kUnit * 2;
    static constexpr int kTile = kUnit * D * 2;  // one K or V tile
    static constexpr int kP = NH * kQHalf;
    static constexpr int kKv = kP + NH * kPHalf;
    static constexpr int kFit = (224 * 1024 - kKv) / kTile, kSlots = kFit > 10 ? 10 : kFit;
    static constexpr int kK = kSlots / 2, kV = kSlots - kK;  // V is held longer
    static constexpr int kVAt = kKv + kK * kTile;
    // A unit's info is read until its second product is issued. K of unit i is loaded when S of
    // unit i - kK is done; S runs at most 4 units (the S buffers) ahead of the loads from its
    // buffers, and those 2 units ahead of the second products
    static constexpr int kInfos = 16;
    static_assert(kK >= 2 && kK + 4 + 2 <= kInfos, "ring");
    static constexpr int kInfo = kKv + kSlots * kTile;
    static constexpr int kBars = (kInfo + kInfos * (int)sizeof(TileInfo) + 7) / 8 * 8;
    // k_full, v_full, k_empty, v_empty [kSlots], s_free [kSBufs], s_full [NH][4], p_full,
    // q_full, pv_done [NH], drain [2], edge. A parity wait is exact for a waiter that sees every phase:
    // s_full (its units in turn) and pv_done belong to a half, the others to one of the
    // four warps, which waits for every use in turn.
    static constexpr int kNumBars = 2 * kSlots + kSBufs + 7 * NH + 3;
    static constexpr int kMisc = kBars + kNumBars * 8;  // tensor memory address, abort flag
    static constexpr int kRun = kMisc + 16;
    static constexpr int kBytes = kRun + (int)sizeof(RunSmem);
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= 227 * 1024, "shared memory");
};

// kSplit (NH = 2): the two halves are the same 128 rows, and take every other unit; each has its
// own running maximum, sum and accumulator, which meet at a piece's end. One half's chain from S
// to P is then hidden behind the other's (24 rows per key head: 175 -> 153 us over
// 8 x 16001..32760 slots, 128 rows 225 -> 169 us).
template <typename E, int D, int NH, bool kSplit>
__global__ void __launch_bounds__(TileSmem<D, NH>::kThreads, 1)
    cache_tile_kernel(const CacheAttn a, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKn,
                      const __grid_constant__ CUtensorMap tmVn, bool fresh_map)
{
    using L = TileSmem<D, NH>;
    constexpr int NK = L::kK, NV = L::kV, NI = L::kInfos, SB = L::kSBufs;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw);
    TileInfo *info = reinterpret_cast<TileInfo *>(smem + L::kInfo);
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::kBars), *v_full = k_full + NK;
    uint64_t *k_empty = v_full + NV, *v_empty = k_empty + NK, *s_free = v_empty + NV, *s_full = s_free + SB;
    uint64_t *p_full = s_full + 4 * NH, *q_full = p_full + NH, *pv_done = q_full + NH;
    uint64_t *drain = pv_done + NH, *edge_bar = drain + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + L::kMisc + 8);
    RunSmem &run_sm = *reinterpret_cast<RunSmem *>(smem + L::kRun);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, nct = gridDim.x, rt = blockIdx.y;
    constexpr int kTileRows = kSplit ? kRows : NH * kRows;
    const int row0 = rt * kTileRows;
    const int page = a.c.page, shift = a.page_shift;

    if (tid == 0) {
        for (int s = 0; s < L::kSlots; ++s) {
            mbar_init(&k_full[s], 1);   // and v_full behind it
            mbar_init(&k_empty[s], 1);  // and v_empty
        }
        for (int s = 0; s < SB; ++s) mbar_init(&s_free[s], 4);
        for (int h = 0; h < NH; ++h) {
            for (int i = 0; i < 4; ++i) mbar_init(&s_full[4 * h + i], 1);
            mbar_init(&p_full[h], 4);
            mbar_init(&q_full[h], kSplit ? 256 : 128);
            mbar_init(&pv_done[h], 1);
        }
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        mbar_init(edge_bar, 1);
        *abort = 0;
        fence_barrier_init();
    }
    if (warp == L::kWarpS) {
        tmem_alloc(tmem_slot, L::kTmemCols);
        tmem_relinquish();
    }
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();  // the join may come up, read the call's inputs and wait
    int *flag0 = rt == 0 ? a.flag : nullptr;  // one report per bad length or count
    Run run = find_run<L::kThreads>(a, run_sm, cta, nct, flag0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Piece pc;

    auto wait = [&](uint64_t *bar, uint32_t phase) -> bool {
        return __all_sync(~0u, mbar_wait(bar, phase & 1, abort, a.flag));
    };
    if (warp == L::kWarpK || warp == L::kWarpV) {
        const bool is_k = warp == L::kWarpK;
        const CUtensorMap *tm = is_k ? &tmK : &tmV, *tmn = is_k ? &tmKn : &tmVn;
        uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
        uint8_t *ring = smem + (is_k ? L::kKv : L::kVAt);
        const int ns = is_k ? NK : NV;
        if (elect_one()) prefetch_tmap(tm);
        __syncwarp();
        const int nent = max(1, kUnit >> shift), box_rows = min(page, kUnit);
        // the lanes look up 32 / nent units together, so that a table (and a plan) is waited
        // for once in so many units
        const int batch = 32 / nent;
        int it = 0, s = 0;                  // units so far, their ring slot
        uint32_t par_e = 1;                 // parity of the slots' last release
        uint32_t phase = 0, loaded = 0;     // bit s: parity of slot s's next tile; its last one was copied
        uint32_t edges = 0;                 // V copies that were waited for here
        bool ok = true;
        while (ok && next_piece(a, run, nct, pc, nullptr)) {
            if (row0 >= group_rows(a, pc.g)) continue;
            const int cap = cache_len(a.c, a.c.length, pc.g.b, is_k ? flag0 : nullptr);
            const int slots = (pc.g.ctx + page - 1) >> shift;
            Staged eb = {-1, 0, 0.f};
            int behind = batch;  // units of the batch that are done
            for (int u = pc.u1 - 1; ok && u >= pc.u0; --u, ++it, ++behind) {
                if (behind == batch) {
                    behind = 0;
                    eb = {-1, 0, 0.f};
                    const int uu = u - lane / nent, slot = ((uu * kUnit) >> shift) + lane % nent;
                    if (uu >= pc.u0 && uu < pc.g.ctx_units && slot < slots)
                        eb = stage_entry(a, pc, slot, cap, is_k ? a.flag : nullptr);
                }
                const int from = (behind * nent + lane) & 31;
                Staged e;
                e.page = __shfl_sync(~0u, eb.page, from);
                e.valid = __shfl_sync(~0u, eb.valid, from);
                e.shift = __shfl_sync(~0u, eb.shift, from);
                const int r0 = page > kUnit ? (u * kUnit) & (page - 1) : 0;
                const bool clean = lane >= nent || (e.page >= 0 && e.valid >= r0 + box_rows);
                const bool ctx = u < pc.g.ctx_units, whole = __all_sync(~0u, clean);
                if (it >= ns) ok = wait(&empty[s], par_e);
                if (!ok) break;
                if (is_k) {
                    TileInfo &ti = info[it % NI];
                    if (lane < nent) ti.ent[lane] = e;
                    if (lane == 0) ti.partial = !whole;
                }
                uint8_t *tile = ring + s * L::kTile;
                const int j0 = (u - pc.g.ctx_units) * kUnit;  // first new token of the unit
                // rows of V that are no key's have to be zero
                const bool mend = !is_k && (ctx ? !whole : j0 + kUnit > pc.g.n && pc.g.n < a.T);
                loaded &= ~(1u << s);
                if (ctx || fresh_map) {
                    const unsigned has = ctx ? __ballot_sync(~0u, lane < nent && e.page >= 0) : 1u;
                    const uint32_t bytes = ctx ? __popc(has) * box_rows * (D * 2) : L::kTile;
                    uint64_t *bar = mend ? edge_bar : &full[s];
                    __syncwarp();  // the info is written before the barrier is armed
                    if (lane == 0) {
                        if (bytes)
                            mbar_arrive_expect_tx(bar, bytes);
                        else if (!mend)
                            mbar_arrive(bar);
                    }
                    __syncwarp();
                    if (bytes && !mend) loaded |= 1u << s;
                    if (has >> lane & 1) {
#pragma unroll
                        for (int y = 0; y < L::kBoxes; ++y) {
                            uint8_t *d = tile + lane * box_rows * 128 + y * (kUnit * 128);
                            if (ctx)
                                tma_load_4d(d, tm, bar, y * 64, r0, pc.hk, e.page);
                            else
                                tma_load_4d(d, tmn, bar, y * 64, j0, pc.hk, pc.g.b);
                        }
                    }
                    __syncwarp();
                    if (mend) {
                        if (bytes) {
                            ok = wait(edge_bar, edges);
                            if (!ok) {
                                drain_wait(edge_bar, edges & 1);
                                break;
                            }
                            ++edges;
                        }
                        for (int j = 0; j < kUnit; ++j) {
                            const int en = page >= kUnit ? 0 : j >> shift, r = (u * kUnit + j) & (page - 1);
                            const int pg = __shfl_sync(~0u, e.page, en), valid = __shfl_sync(~0u, e.valid, en);
                            if (ctx ? pg >= 0 && r < valid : j0 + j < pc.g.n) continue;
                            if (lane < L::kBoxes * 8)
                                *reinterpret_cast<uint4 *>(tile + (lane >> 3) * (kUnit * 128) + j * 128 +
                                                           (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                } else {
                    constexpr int kChunks = D / 8;
                    const ab_tokens &nt = is_k ? a.k : a.v;
                    const char *rows = static_cast<const char *>(nt.p) + 2 * (pc.g.b * nt.sb + pc.hk * nt.sh);
#pragma unroll 8
                    for (int i = lane; i < kUnit * kChunks; i += 32) {
                        const int j = i / kChunks, c = i % kChunks;
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (j0 + j < pc.g.n) x = ldg_stream(rows + 2 * (j0 + j) * nt.st + c * 16);
                        *reinterpret_cast<uint4 *>(tile + (c >> 3) * (kUnit * 128) + j * 128 +
                                                   (((c & 7) ^ (j & 7)) << 4)) = x;
                    }
                }
                if (mend || !(ctx || fresh_map)) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[s]);
                }
                phase ^= 1u << s;
                __syncwarp();
                if (++s == ns) {
                    s = 0;
                    par_e ^= 1;
                }
            }
        }
        if (!ok) {  // copies that may still be in flight land before the CTA ends
            for (int x = 0; x < ns; ++x)
                if (loaded >> x & 1) drain_wait(&full[x], (phase >> x & 1) ^ 1);
        }
    } else if (warp == L::kWarpS) {
        constexpr uint32_t idesc_s = idesc<E>(kRows, kUnit, 0, 0);
        const uint64_t qd = smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + L::kKv), 16, 1024);
        int s = 0, it = 0;                // ring slot of the next unit, units so far
        int buf = 0;                      // S buffer of the next job
        uint32_t tiles = 0;               // bit s: parity of slot s's next tile
        uint32_t turn = 0, phase_q = 0;   // two bits per half: its next S's barrier; bit h: its next Q
        uint32_t par_b = 1;               // parity of the S buffers' last release
        bool ok = true, used = false;     // used: every S buffer has had a job
        while (ok && next_piece(a, run, nct, pc, nullptr)) {
            const int rows = group_rows(a, pc.g) - row0;
            if (rows <= 0) continue;
            // halves with rows in this piece (kSplit: one Q)
            const int na = kSplit ? 1 : min(NH, (rows + kRows - 1) / kRows);
            for (int h = 0; ok && h < na; ++h) {
                ok = wait(&q_full[h], phase_q >> h);
                phase_q ^= 1u << h;
            }
            for (int n = pc.u1 - pc.u0; ok && n > 0; --n, ++it) {
                ok = wait(&k_full[s], tiles >> s);
                tiles ^= 1u << s;
                const uint64_t kd = kd0 + (uint64_t)s * (L::kTile >> 4);
                for (int x = 0; ok && x < na; ++x) {
                    const int h = kSplit ? it & 1 : x;
                    if (used) ok = wait(&s_free[buf], par_b);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t qh = qd + (uint64_t)x * (L::kQHalf >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss(tmem + buf * kUnit, qh + ((kk >> 2) * (kRows * 128) + (kk & 3) * 32 >> 4),
                                   kd + ((kk >> 2) * (kUnit * 128) + (kk & 3) * 32 >> 4), idesc_s, kk > 0);
                        mma_commit(&s_full[4 * h + (turn >> 2 * h & 3)]);
                        if (x == na - 1) mma_commit(&k_empty[s]);
                    }
                    __syncwarp();
                    turn = (turn & ~(3u << 2 * h)) | ((turn + (1u << 2 * h)) & (3u << 2 * h));
                    if (++buf == SB) {
                        buf = 0;
                        used = true;
                        par_b ^= 1;
                    }
                }
                if (++s == NK) s = 0;
            }
        }
        if (!ok) {
            if (elect_one()) {
                mma_commit(&drain[0]);
                drain_wait(&drain[0], 0);
            }
            __syncwarp();
        }
    } else if (warp == L::kWarpO) {
        constexpr uint32_t idesc_o = idesc<E>(kRows, D, 0, 1);
        const uint64_t pd = smem_desc_sw128(smem_u32(smem + L::kP), 16, 1024);
        const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + L::kVAt), kUnit * 128, 1024);
        int s = 0, it = 0;
        uint32_t tiles = 0, phase_p = 0;  // bit s: slot s's next tile; bit h: half h's next P
        bool ok = true;
        while (ok && next_piece(a, run, nct, pc, nullptr)) {
            const int rows = group_rows(a, pc.g) - row0;
            if (rows <= 0) continue;
            const int na = kSplit ? 1 : min(NH, (rows + kRows - 1) / kRows);
            for (int n = 0; ok && n < pc.u1 - pc.u0; ++n, ++it) {
                ok = wait(&v_full[s], tiles >> s);
                tiles ^= 1u << s;
                const uint64_t vd = vd0 + (uint64_t)s * (L::kTile >> 4);
                for (int x = 0; ok && x < na; ++x) {
                    const int h = kSplit ? it & 1 : x;
                    ok = wait(&p_full[h], phase_p >> h);
                    if (!ok) break;
                    phase_p ^= 1u << h;
                    tc_fence_after();
                    const uint64_t ph = pd + (uint64_t)h * (L::kPHalf >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kUnit / 16; ++kk)
                            mma_ss(tmem + L::kColO + h * D, ph + (kk * 32 >> 4), vd + (kk * 2048 >> 4), idesc_o,
                                   n > (kSplit ? 1 : 0) || kk > 0);
                        mma_commit(&pv_done[h]);
                        if (x == na - 1) mma_commit(&v_empty[s]);
                    }
                    __syncwarp();
                }
                if (++s == NV) s = 0;
            }
        }
        if (!ok) {
            if (elect_one()) {
                mma_commit(&drain[1]);
                drain_wait(&drain[1], 0);
            }
            __syncwarp();
        }
    } else {
        // ---- softmax: thread = query row. After a failed wait a warp runs out its loops
        // without waiting, and reads no page.
        bool ok = true;
        auto wait_on = [&](uint64_t *bar, uint32_t phase) {
            if (ok) ok = wait(bar, phase);
        };
        const int half = warp >> 2, th = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t acc = tmem + lanes + L::kColO + half * D;
        uint8_t *prow = smem + L::kP + half * L::kPHalf + th * 128;
        const float inv_scale = 1.f / a.scale_log2;
        int it = 0, job = 0;  // units and jobs before this piece
        int pv = 0;           // units of this half so far
        while (next_piece(a, run, nct, pc, half == 0 ? flag0 : nullptr)) {
            const int rows = group_rows(a, pc.g);
            if (row0 >= rows) continue;
            const int na = kSplit ? 1 : min(NH, (rows - row0 + kRows - 1) / kRows), units = pc.u1 - pc.u0;
            if (!kSplit && half >= na) {
                it += units;
                job += units * na;
                continue;
            }
            const int hrow0 = row0 + (kSplit ? 0 : half * kRows), row = hrow0 + th, b = pc.g.b;
            const bool live = row < rows, warp_live = hrow0 + (warp & 3) * 32 < rows;
            const int t = a.per_token ? pc.g.tp : row / a.G;
            const int h = pc.hk * a.G + (a.per_token ? row : row % a.G);
            // Q rows into the swizzled operand tile: the previous piece's products are done
            {
                constexpr int kChunks = D / 8;
                const int left = min(kRows, rows - hrow0);
                // kSplit: both halves are done with the last piece's rows and with what they left
                if (kSplit) asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll 8
                for (int i = kSplit ? tid : th; i < kRows * kChunks; i += kSplit ? 256 : 128) {
                    const int r = i / kChunks, c = i % kChunks;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (r < left) {
                        const int rr = hrow0 + r, tt = a.per_token ? pc.g.tp : rr / a.G;
                        const int hh = pc.hk * a.G + (a.per_token ? rr : rr % a.G);
                        x = *reinterpret_cast<const uint4 *>(
                            static_cast<const char *>(a.q.p) +
                            2 * (b * a.q.sb + hh * a.q.sh + tt * a.q.st) + c * 16);
                    }
                    *reinterpret_cast<uint4 *>(smem + (kSplit ? 0 : half * L::kQHalf) + (c >> 3) * (kRows * 128) + r * 128 +
                                               (((c & 7) ^ (r & 7)) << 4)) = x;
                }
                fence_proxy_async_smem();
                mbar_arrive(&q_full[kSplit ? 0 : half]);
            }
            float m = -INFINITY, l = 0.f;
            bool first = true;  // the accumulator holds nothing of this piece yet
            if (!kSplit) job += half;
            for (int u = pc.u1 - 1; u >= pc.u0; --u, ++it, job += na) {
                if (kSplit && (it & 1) != half) continue;
                const bool ctx = u < pc.g.ctx_units;
                uint64_t sees = ~0ull;  // this row's keys of the unit
                bool masked = false;
                if (!ctx) {
                    masked = true;
                    sees = 0;
                    const int j0 = (u - pc.g.ctx_units) * kUnit, nv = min(kUnit, pc.g.n - j0);
                    if (live && !a.tree) {
                        const int nk = min(nv, max(0, t - j0 + 1));
                        sees = nk >= 64 ? ~0ull : (1ull << nk) - 1;
                    } else if (live) {
                        const uint8_t *tr = a.tree + ((size_t)b * a.T + t) * a.T + j0;
                        int j = 0;
                        if ((reinterpret_cast<uintptr_t>(tr) & 3) == 0) {  // four bytes at a time
                            uint32_t w[kUnit / 4];
#pragma unroll
                            for (int i = 0; i < kUnit / 4; ++i)
                                w[i] = 4 * i + 4 <= nv ? *reinterpret_cast<const uint32_t *>(tr + 4 * i) : 0;
#pragma unroll
                            for (int i = 0; i < kUnit / 4; ++i) {
                                const uint32_t x = __vcmpne4(w[i], 0);
                                sees |= (uint64_t)((x & 1) | (x >> 7 & 2) | (x >> 14 & 4) | (x >> 21 & 8)) << (4 * i);
                            }
                            j = nv & ~3;
                        }
#pragma unroll 4
                        for (; j < nv; ++j) sees |= (uint64_t)(tr[j] != 0) << j;
                    }
                    __syncwarp();
                }
                wait_on(&s_full[4 * half + (pv & 3)], pv >> 2);
                tc_fence_after();
                // the unit's info was written before its keys were announced to the S warp
                const TileInfo &ti = info[it % NI];
                float sh[kEnt] = {0.f, 0.f, 0.f, 0.f};
                if (ctx && (ti.partial || a.w)) {
                    masked = true;
                    sees = 0;
#pragma unroll
                    for (int e = 0; e < kEnt; ++e) {
                        // keys e * 16 .. e * 16 + 15 lie in one page
                        const Staged x = ti.ent[page >= kUnit ? 0 : (e * 16) >> shift];
                        const int r = (u * kUnit + e * 16) & (page - 1);
                        const int nv = x.page >= 0 ? min(16, max(0, x.valid - r)) : 0;
                        sees |= (uint64_t)((1u << nv) - 1) << (16 * e);
                        sh[e] = x.shift;
                    }
                }
                const uint32_t st = tmem + lanes + (job % SB) * kUnit;
                if (warp_live) {
                    uint32_t x0[32], x1[32];
                    tmem_ld32(st, x0);
                    tmem_ld32(st + 32, x1);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_free[job % SB]);
                    auto at = [&](int j) -> uint32_t & { return j < 32 ? x0[j] : x1[j - 32]; };
                    if (masked) {  // weights as a shift of the raw logit; -inf where not seen
#pragma unroll
                        for (int j = 0; j < kUnit; ++j) {
                            const float v = fmaf(sh[j >> 4], inv_scale, __uint_as_float(at(j)));
                            at(j) = __float_as_uint(sees >> j & 1 ? v : -INFINITY);
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < kUnit; j += 8)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            mx[y] = fmax3(mx[y], __uint_as_float(at(j + 2 * y)), __uint_as_float(at(j + 2 * y + 1)));
                    const float mt = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * a.scale_log2;
                    // this half's earlier products are done: P is free, and O may be scaled
                    if (pv > 0) wait_on(&pv_done[half], pv - 1);
                    if (__any_sync(~0u, mt > m + kLazy)) {
                        const float mn = fmaxf(m, mt);
                        const float f = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
                        m = mn;
                        l *= f;
                        if (!first) {
                            tc_fence_after();
#pragma unroll 1
                            for (int ch = 0; ch < D / 16; ++ch) {
                                uint32_t o[16];
                                tmem_ld16(acc + ch * 16, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st16(acc + ch * 16, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float mb = m == -INFINITY ? 0.f : E::kBias - m;
                    float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 8; ++c) {  // eight keys: one 16-byte chunk of the row
                        uint32_t p[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float p0 = fast_exp2(fmaf(__uint_as_float(at(8 * c + 2 * j)), a.scale_log2, mb));
                            const float p1 = fast_exp2(fmaf(__uint_as_float(at(8 * c + 2 * j + 1)), a.scale_log2, mb));
                            ls[j] += p0 + p1;
                            p[j] = E::pack(p0, p1);  // rounded for the second product, the sum is not
                        }
                        *reinterpret_cast<uint4 *>(prow + ((c ^ (th & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                    l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                    fence_proxy_async_smem();
                } else {
                    if (lane == 0) mbar_arrive(&s_free[job % SB]);
                    if (pv > 0) wait_on(&pv_done[half], pv - 1);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[half]);
                first = false;
                ++pv;
            }
            // ---- the piece's end: rows out, or into the workspace
            if (!kSplit) job -= half;
            if (pv > 0) wait_on(&pv_done[half], pv - 1);
            tc_fence_after();
            float f0 = 1.f, f1 = 0.f;  // kSplit: weights of the halves' accumulators
            float *half1 = reinterpret_cast<float *>(smem);  // [D][128] over Q, which is done with
            if constexpr (kSplit) {
                float2 *ml1 = reinterpret_cast<float2 *>(smem + L::kP) + th;  // over P
                static_assert(NH == 2 && D * kRows * 4 <= L::kP, "room for an accumulator");
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (half == 1) {
                    *ml1 = make_float2(m, l);
                    if (warp_live && !first) {
#pragma unroll 1
                        for (int ch = 0; ch < D / 32; ++ch) {
                            uint32_t o[32];
                            tmem_ld32(acc + ch * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) half1[(ch * 32 + j) * kRows + th] = __uint_as_float(o[j]);
                        }
                    }
                    tc_fence_before();
                }
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (half == 1) continue;
                const float2 o = *ml1;
                const float mt = fmaxf(m, o.x);
                f0 = m == -INFINITY ? 0.f : fast_exp2(m - mt);
                f1 = o.x == -INFINITY ? 0.f : fast_exp2(o.x - mt);
                // beside a maximum of -inf the sum is 0, or NaN where every logit was
                l = (m == -INFINITY ? l : l * f0) + (o.x == -INFINITY ? o.y : o.y * f1);
                m = mt;
            }
            const bool whole = pc.u0 == 0 && pc.u1 == pc.g.units;
            const int item = ((b * a.c.Hk + pc.hk) * a.Tp + pc.g.tp) * a.row_tiles + rt;
            if (tid == 0) {  // half 0 has rows whenever another half has
                if (pc.u0 == 0) a.info[item].x = cta;
                if (pc.u1 == pc.g.units) a.info[item].y = cta;
            }
            const size_t slot = ((size_t)rt * nct + cta) * 2 + (pc.u0 == 0 ? 1 : 0);
            const size_t prt = slot * kTileRows + (kSplit ? 0 : half * kRows) + th;  // row of the workspace
            const size_t orow = ((size_t)b * a.c.Hk * a.G + h) * a.T + t;
            const float inv = !whole ? 1.f : l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
            if (live) {
                if (!whole)
                    a.part_ml[prt] = make_float2(m, l);
                else if (a.lse)
                    a.lse[orow] = l == 0.f ? -INFINITY : (m - E::kBias + log2f(l)) * kLn2;
            }
            __syncwarp();
            if (warp_live) {
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t o[32];
                    tmem_ld32(acc + ch * 32, o);
                    tmem_wait_ld();
                    if (live) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            float x = __uint_as_float(o[j]);
                            if (kSplit)
                                x = (f0 != 0.f ? x * f0 : 0.f) +
                                    (f1 != 0.f ? half1[(ch * 32 + j) * kRows + th] * f1 : 0.f);
                            o[j] = __float_as_uint(l == 0.f ? 0.f : x * inv);
                        }
                        if (!whole || a.out_f32) {
                            float *d = whole ? static_cast<float *>(a.out) + orow * D : a.part + prt * D;
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
    if (warp == L::kWarpS) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

struct Maps {
    CUtensorMap k, v, kn, vn;
    bool fresh;  // kn and vn are there
};

template <typename E, int D, int NH, bool kSplit>
cudaError_t launch_one(const CacheAttn &a, int nct, const Maps &m, cudaStream_t st)
{
    using L = TileSmem<D, NH>;
    return launch_kernel(cache_tile_kernel<E, D, NH, kSplit>, dim3(nct, a.row_tiles), L::kThreads, L::kAlloc, L::kAlloc, 1,
                         st, a, m.k, m.v, m.kn, m.vn, m.fresh);
}

template <typename E, int D>
cudaError_t launch_halves(const CacheAttn &a, const CacheAttnPlan &p, const Maps &m, cudaStream_t st)
{
    switch (p.tile_rows / kRows) {
    case 1: return launch_one<E, D, 2, true>(a, p.ctas, m, st);
    case 2: return launch_one<E, D, 2, false>(a, p.ctas, m, st);
    default: return launch_one<E, D, 3, false>(a, p.ctas, m, st);
    }
}

}  // namespace

cudaError_t launch_cache_tiles(const CacheAttn &a, const CacheAttnPlan &p, cudaStream_t st)
{
    Maps m;
    const ab_cache &c = a.c;
    if (!page_map(&m.k, c, c.k, c.k_row, c.k_head, c.k_page) || !page_map(&m.v, c, c.v, c.v_row, c.v_head, c.v_page))
        return cudaErrorInvalidValue;
    m.kn = m.k;
    m.vn = m.v;
    m.fresh = a.k.p && token_map(&m.kn, c, a.k, a.T) && token_map(&m.vn, c, a.v, a.T);
    if (c.dtype == AB_F16) return c.d == 64 ? launch_halves<Fp16, 64>(a, p, m, st) : launch_halves<Fp16, 128>(a, p, m, st);
    return c.d == 64 ? launch_halves<Bf16, 64>(a, p, m, st) : launch_halves<Bf16, 128>(a, p, m, st);
}

}  // namespace ab
