// cache_attn.cu -- attention of new tokens over a paged key/value cache (ab_cache_attn):
// softmax over the cache's slots (all, or the pages of a plan with weights) and over the new
// tokens that a tree's mask lets each row see. This file holds the kernel for few query rows
// per key head and the kernel that joins the parts of a split row.
//
// Few rows: bound by reading K and V once. Each warp computes S^T = K Q^T for 16 keys and 8
// query rows at a time, then O^T += V^T P^T, with keys and values as the A operand of the
// warp-level m16n8k16 product, loaded from global memory straight into the fragments (16
// bytes per lane and load; the order of d inside a product is free, so no shuffle is needed;
// V's pairs of keys are zipped with two byte permutes per register). No shared memory, no
// barrier and no copy queue stand between the loads and the products: the loads in flight
// are the registers of 12 warps per SM, 8 KB each. 16 sequences of 1023..32760 slots, 40 / 8
// heads, d = 128: 182 us, 6.1 TB/s of K and V, 0.93 of the copy rate.
//
// Work is cut into units of 64 keys of one (sequence, key head[, plan row]); the CTAs take
// equal runs of units in order, whatever the lengths, and a run that covers part of a row
// leaves its running maximum, sum and unnormalised output in the workspace for the second
// kernel. Which CTA takes which units depends on lengths and counts alone, so equal calls add
// in the same order.
#include <cstdint>

#include "cache_common.cuh"
#include "cache_kernels.h"
#include "cache_sched.cuh"

namespace ab {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStage = 128;  // page slots staged at a time
static_assert(kUnit == 16 * kWarps, "a warp takes 16 keys of a unit");

template <typename E, int D, int NT>
struct Smem {
    Staged stage[kStage];
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    float merge[2][8 * NT][D];
    RunSmem run;
};

template <typename E, int D, int NT, int OCC>
__global__ void __launch_bounds__(kThreads, OCC) cache_attn_kernel(const CacheAttn a)
{
    constexpr int DI = D / 32, DJ = D / 64;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<E, D, NT> &sm = *reinterpret_cast<Smem<E, D, NT> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int cta = blockIdx.x, nct = gridDim.x, rt = blockIdx.y;
    const int page = a.c.page, page_shift = a.page_shift;

    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();  // the join may come up, read the call's inputs and wait
    Run run = find_run<kThreads>(a, sm.run, cta, nct, rt == 0 ? a.flag : nullptr);
    Piece pc;
    while (next_piece(a, run, nct, pc, rt == 0 ? a.flag : nullptr)) {
        const Group &gr = pc.g;
        const int rows = group_rows(a, gr), hk = pc.hk, u0 = pc.u0, u1 = pc.u1;
        const int row0 = rt * 8 * NT;
        if (row0 < rows) {
            // ---- query fragments: row n = g of each tile of 8 (head fastest, then token)
            uint4 qf[NT][DI];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = row0 + nt * 8 + g;
                if (r < rows) {
                    const int t = a.per_token ? gr.tp : r / a.G, h = hk * a.G + (a.per_token ? r : r % a.G);
                    const char *p = static_cast<const char *>(a.q.p) +
                                    2 * (gr.b * a.q.sb + h * a.q.sh + t * a.q.st) + c * 16;
#pragma unroll
                    for (int i = 0; i < DI; ++i) qf[nt][i] = *reinterpret_cast<const uint4 *>(p + 64 * i);
                } else {
#pragma unroll
                    for (int i = 0; i < DI; ++i) qf[nt][i] = make_uint4(0, 0, 0, 0);
                }
            }
            float o[NT][4 * DJ][4], m[NT][2], l[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int x = 0; x < 4 * DJ; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[nt][x][y] = 0.f;
                m[nt][0] = m[nt][1] = -INFINITY;
                l[nt][0] = l[nt][1] = 0.f;
            }
            const char *kbase = static_cast<const char *>(a.c.k) + 2 * hk * a.c.k_head;
            const char *vbase = static_cast<const char *>(a.c.v) + 2 * hk * a.c.v_head;
            const char *knew = static_cast<const char *>(a.k.p) + 2 * (gr.b * a.k.sb + hk * a.k.sh);
            const char *vnew = static_cast<const char *>(a.v.p) + 2 * (gr.b * a.v.sb + hk * a.v.sh);
            const int cap = a.idx ? cache_len(a.c, a.c.length, gr.b, rt == 0 ? a.flag : nullptr) : gr.ctx;
            const int slots = (gr.ctx + page - 1) >> page_shift;  // page slots of the context
            int staged0 = -1;  // first staged page slot

            // 16 keys of unit u as this warp sees them
            struct Keys {
                const char *kp, *vp;
                int64_t krow, vrow;
                int nv;
                float shift;
            };
            auto keys_of = [&](int u) {
                Keys x;
                if (u < gr.ctx_units) {
                    const int key = u * kUnit + warp * 16;
                    x.krow = 2 * a.c.k_row;
                    x.vrow = 2 * a.c.v_row;
                    x.nv = 0;
                    x.shift = 0.f;
                    x.kp = kbase;
                    x.vp = vbase;
                    if (key < gr.ctx) {
                        const Staged s = sm.stage[(key >> page_shift) - staged0];
                        const int r = key & (page - 1);
                        if (s.page >= 0) {
                            x.nv = min(16, s.valid - r);
                            x.kp = kbase + 2 * (s.page * a.c.k_page + r * a.c.k_row);
                            x.vp = vbase + 2 * (s.page * a.c.v_page + r * a.c.v_row);
                            x.shift = s.shift;
                        }
                    }
                } else {
                    const int j = (u - gr.ctx_units) * kUnit + warp * 16;
                    x.krow = 2 * a.k.st;
                    x.vrow = 2 * a.v.st;
                    x.nv = min(16, gr.n - j);
                    x.shift = 0.f;
                    x.kp = knew + j * x.krow;
                    x.vp = vnew + j * x.vrow;
                }
                return x;
            };
            // stage the page slots of unit u and what follows
            auto stage_from = [&](int u) {
                __syncthreads();
                staged0 = (u * kUnit) >> page_shift;
                for (int i = tid; i < kStage && staged0 + i < slots; i += kThreads) {
                    sm.stage[i] = stage_entry(a, pc, staged0 + i, cap, a.flag);
                }
                __syncthreads();
            };
            // units whose page slots are staged end here
            auto staged_end = [&]() {
                return min(gr.ctx_units, (int)(((long long)(staged0 + kStage) << page_shift) / kUnit));
            };

            uint4 kr[2][DI], vr[4][DJ];
            int u = u0;
            int seg_end = u1;  // end of the units that can be walked without staging
            if (u < gr.ctx_units) {
                stage_from(u);
                seg_end = min(u1, staged_end());
            }
            Keys cur = keys_of(u);
            load_k_frag<DI>(kr, cur.kp, cur.krow, cur.nv, g, c);
            load_v_frag<DJ>(vr, cur.vp, cur.vrow, cur.nv, g, c);
            while (true) {
                float s[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
                    qk_product<E, DI>(s[nt], kr, qf[nt]);
                }
                const bool more = u + 1 < u1;
                if (more && u + 1 >= seg_end) {
                    if (u + 1 < gr.ctx_units) {
                        stage_from(u + 1);
                        seg_end = min(u1, staged_end());
                    } else {
                        seg_end = u1;
                    }
                }
                Keys nxt = cur;
                if (more) {
                    nxt = keys_of(u + 1);
                    load_k_frag<DI>(kr, nxt.kp, nxt.krow, nxt.nv, g, c);
                }
                // ---- softmax: rows n = 2c, 2c + 1 of each tile, keys g and g + 8
                uint32_t pb[NT][2];
                const bool k0 = g < cur.nv, k1 = g + 8 < cur.nv;
                const bool fresh = u >= gr.ctx_units;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float x[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        bool sees = y < 2 ? k0 : k1;
                        if (fresh && sees) {
                            const int r = row0 + nt * 8 + 2 * c + (y & 1);
                            const int t = a.per_token ? gr.tp : r / a.G;
                            const int j = (u - gr.ctx_units) * kUnit + warp * 16 + g + (y < 2 ? 0 : 8);
                            if (r < rows)
                                sees = a.tree ? a.tree[((size_t)gr.b * a.T + t) * a.T + j] != 0 : j <= t;
                        }
                        x[y] = sees ? fmaf(s[nt][y], a.scale_log2, cur.shift) : -INFINITY;
                    }
                    const float m0 = fmaxf(x[0], x[2]), m1 = fmaxf(x[1], x[3]);
                    const bool up = m0 > m[nt][0] + kLazy || m1 > m[nt][1] + kLazy;
                    if (__any_sync(~0u, up)) {
                        float n0 = m0, n1 = m1;
#pragma unroll
                        for (int sft = 4; sft < 32; sft <<= 1) {
                            n0 = fmaxf(n0, __shfl_xor_sync(~0u, n0, sft));
                            n1 = fmaxf(n1, __shfl_xor_sync(~0u, n1, sft));
                        }
                        n0 = fmaxf(n0, m[nt][0]);
                        n1 = fmaxf(n1, m[nt][1]);
                        const float f0 = n0 == -INFINITY ? 1.f : fast_exp2(m[nt][0] - n0);
                        const float f1 = n1 == -INFINITY ? 1.f : fast_exp2(m[nt][1] - n1);
                        m[nt][0] = n0;
                        m[nt][1] = n1;
                        l[nt][0] *= f0;
                        l[nt][1] *= f1;
#pragma unroll
                        for (int z = 0; z < 4 * DJ; ++z) {
                            o[nt][z][0] *= f0;
                            o[nt][z][1] *= f1;
                            o[nt][z][2] *= f0;
                            o[nt][z][3] *= f1;
                        }
                    }
                    const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - E::kBias;
                    const float b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - E::kBias;
                    const float p0 = fast_exp2(x[0] - b0), p1 = fast_exp2(x[1] - b1);
                    const float p2 = fast_exp2(x[2] - b0), p3 = fast_exp2(x[3] - b1);
                    l[nt][0] += p0 + p2;
                    l[nt][1] += p1 + p3;
                    // the probabilities of the second product are rounded to the values'
                    // type (the sum above is not): half an ulp of each, independent over keys
                    pb[nt][0] = movmatrix_trans(E::pack(p0, p1));
                    pb[nt][1] = movmatrix_trans(E::pack(p2, p3));
                }
#pragma unroll
                for (int j = 0; j < DJ; ++j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t w0 = (&vr[0][j].x)[e], w1 = (&vr[1][j].x)[e];
                        const uint32_t w2 = (&vr[2][j].x)[e], w3 = (&vr[3][j].x)[e];
                        const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
                        const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<E>(o[nt][j * 4 + e], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    }
                }
                if (!more) break;
                load_v_frag<DJ>(vr, nxt.vp, nxt.vrow, nxt.nv, g, c);
                cur = nxt;
                ++u;
            }

            // ---- join the four warps: common maximum, then sums in warp order
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float ls = l[nt][y];
#pragma unroll
                    for (int sft = 4; sft < 32; sft <<= 1) ls += __shfl_xor_sync(~0u, ls, sft);
                    l[nt][y] = ls;
                    if (g == 0) {
                        // a warp whose logits were all NaN has a maximum of -inf, but takes part
                        sm.m[warp][nt * 8 + 2 * c + y] = ls != ls ? 0.f : m[nt][y];
                        sm.l[warp][nt * 8 + 2 * c + y] = ls;
                    }
                }
            __syncthreads();
            float mt[NT][2], lt[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int n = nt * 8 + 2 * c + y;
                    float mm = sm.m[0][n];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, sm.m[w][n]);
                    float ll = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        if (sm.m[w][n] != -INFINITY) ll += sm.l[w][n] * fast_exp2(sm.m[w][n] - mm);
                    mt[nt][y] = mm;
                    lt[nt][y] = ll;
                    const float f = m[nt][y] == -INFINITY ? 0.f : fast_exp2(m[nt][y] - mm);
#pragma unroll
                    for (int z = 0; z < 4 * DJ; ++z) {
                        o[nt][z][y] *= f;
                        o[nt][z][y + 2] *= f;
                    }
                }
            auto merge_io = [&](int slot, bool add) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int z = 0; z < 4 * DJ; ++z) {
                            float2 *p = reinterpret_cast<float2 *>(
                                &sm.merge[slot][nt * 8 + 2 * c + y][8 * (g + 8 * (z >> 2)) + 2 * (z & 3)]);
                            if (add) {
                                const float2 v = *p;
                                o[nt][z][y] += v.x;
                                o[nt][z][y + 2] += v.y;
                            } else {
                                *p = make_float2(o[nt][z][y], o[nt][z][y + 2]);
                            }
                        }
            };
            if (warp >= 2) merge_io(warp - 2, false);
            __syncthreads();
            if (warp < 2) merge_io(warp, true);
            __syncthreads();
            if (warp == 1) merge_io(0, false);
            __syncthreads();
            if (warp == 0) {
                merge_io(0, true);
                const bool whole = u0 == 0 && u1 == gr.units;
                const int item = ((gr.b * a.c.Hk + hk) * a.Tp + gr.tp) * a.row_tiles + rt;
                const size_t slot = ((size_t)rt * nct + cta) * 2 + (u0 == 0 ? 1 : 0);
                if (lane == 0) {
                    if (u0 == 0) a.info[item].x = cta;
                    if (u1 == gr.units) a.info[item].y = cta;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int n = nt * 8 + 2 * c + y, r = row0 + n;
                        if (r >= rows) continue;
                        if (!whole) {
                            float *po = a.part + slot * (size_t)(8 * NT) * D + (size_t)n * D;
                            float2 *pml = a.part_ml + slot * (8 * NT) + n;
                            if (g == 0) *pml = make_float2(mt[nt][y], lt[nt][y]);
#pragma unroll
                            for (int j = 0; j < DJ; ++j) {
                                float4 *p = reinterpret_cast<float4 *>(po + 8 * (g + 8 * j));
                                p[0] = make_float4(o[nt][4 * j][y], o[nt][4 * j][y + 2],
                                                   o[nt][4 * j + 1][y], o[nt][4 * j + 1][y + 2]);
                                p[1] = make_float4(o[nt][4 * j + 2][y], o[nt][4 * j + 2][y + 2],
                                                   o[nt][4 * j + 3][y], o[nt][4 * j + 3][y + 2]);
                            }
                            continue;
                        }
                        const int t = a.per_token ? gr.tp : r / a.G, h = hk * a.G + (a.per_token ? r : r % a.G);
                        const size_t orow = ((size_t)gr.b * a.c.Hk * a.G + h) * a.T + t;
                        const float ll = lt[nt][y], inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
                        if (a.lse && g == 0)
                            a.lse[orow] = ll == 0.f ? -INFINITY
                                                    : (mt[nt][y] - E::kBias + log2f(ll)) * kLn2;
#pragma unroll
                        for (int j = 0; j < DJ; ++j) {
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                v[2 * e] = o[nt][4 * j + e][y] * inv;
                                v[2 * e + 1] = o[nt][4 * j + e][y + 2] * inv;
                            }
                            const size_t at = orow * D + 8 * (g + 8 * j);
                            if (a.out_f32) {
                                float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at);
                                p[0] = make_float4(v[0], v[1], v[2], v[3]);
                                p[1] = make_float4(v[4], v[5], v[6], v[7]);
                            } else {
                                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at) =
                                    make_uint4(E::pack(v[0], v[1]), E::pack(v[2], v[3]),
                                               E::pack(v[4], v[5]), E::pack(v[6], v[7]));
                            }
                        }
                    }
            }
            __syncthreads();  // the merge buffers and the staged pages are free again
        }
    }
}

// Joins the parts of rows that several CTAs computed, and writes the rows nobody computed
// (behind n_tok, or with nothing to see). kRowWarps warps share a row and take its parts in
// turn: one where a row has few (29 -> 17 us for 20480 rows of 2 or 3 parts), four, or sixteen
// where a long row is cut into very many. The order of the sums depends on the parts alone.
constexpr int join_threads(int row_warps) { return row_warps > 4 ? 32 * row_warps : 128; }

template <typename E, int D, int kRowWarps>
__global__ void __launch_bounds__(join_threads(kRowWarps)) cache_join_kernel(const CacheAttn a, int tile_rows, int nct, int rows)
{
    constexpr int kPer = join_threads(kRowWarps) / 32 / kRowWarps;  // rows of a CTA
    constexpr int V = D / 32;                                      // values per lane
    __shared__ float sm_m[kRowWarps], sm_l[kRowWarps], sm_o[kRowWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % kRowWarps;
    const int row = blockIdx.x * kPer + warp / kRowWarps;
    const bool exists = row < rows;
    const int rr = exists ? row : rows - 1;
    const int t = rr % a.T, h = (rr / a.T) % (a.c.Hk * a.G), b = rr / a.T / (a.c.Hk * a.G), hk = h / a.G;
    const int tp = a.per_token ? t : 0;
    const int gi = a.idx ? (b * a.c.Hk + hk) * a.Tp + tp : b;
    const Group gr = load_group(a, gi, nullptr);  // inputs of the call: there before its first kernel went on
    float o[V], mt = -INFINITY, lt = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.f;
    const bool dead = t >= gr.n;
    bool write = exists;
    cudaGridDependencySynchronize();
    if (exists && !dead && gr.units > 0) {
        const int r = a.per_token ? h % a.G : t * a.G + h % a.G;
        const int rt = r / tile_rows, n = r % tile_rows;
        int2 who = a.info[((b * a.c.Hk + hk) * a.Tp + tp) * a.row_tiles + rt];
        // inside the workspace even where a kernel gave up waiting before it wrote them
        who.x = min(max(who.x, 0), nct - 1);
        who.y = min(max(who.y, who.x), nct - 1);
        write = who.x != who.y;  // else one CTA had it all and wrote it
        const int parts = write ? who.y - who.x + 1 : 0;
        // 32 parts at a time: their maxima and weights by lane, then their rows, whose loads do
        // not wait for one another (one part after the other: 72 us against 32 us for a
        // call on one sequence of 100000 slots with one key head, whose rows have 444 parts;
        // sixteen warps a row instead of four then 22 us)
        const size_t slot0 = ((size_t)rt * nct + who.x) * 2;
        for (int base = 0; sub + kRowWarps * base < parts; base += 32) {
            auto row_at = [&](int k) {  // row n of part sub + kRowWarps k
                const int p = sub + kRowWarps * k;
                return (slot0 + 2 * p + (p == 0 ? 1 : 0)) * tile_rows + n;
            };
            const bool there = sub + kRowWarps * (base + lane) < parts;
            const float2 ml = there ? a.part_ml[row_at(base + lane)] : make_float2(-INFINITY, 0.f);
            float mn = ml.x;
#pragma unroll
            for (int sft = 16; sft; sft >>= 1) mn = fmaxf(mn, __shfl_xor_sync(~0u, mn, sft));
            mn = fmaxf(mn, mt);
            const float f0 = mt == -INFINITY ? 0.f : fast_exp2(mt - mn);
            const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - mn);
            float lw = ml.x == -INFINITY ? ml.y : ml.y * w;  // beside -inf: 0, or NaN where every logit was
#pragma unroll
            for (int sft = 16; sft; sft >>= 1) lw += __shfl_xor_sync(~0u, lw, sft);
            lt = (mt == -INFINITY ? lt : lt * f0) + lw;
            if (mn == -INFINITY) continue;
            mt = mn;
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] *= f0;
            const int count = min(32, (parts - sub + kRowWarps - 1) / kRowWarps - base);
#pragma unroll 8
            for (int k = 0; k < count; ++k) {
                const float wk = __shfl_sync(~0u, w, k);
                const float *po = a.part + row_at(base + k) * D + lane * V;
                float x[V];
                if constexpr (V == 4)
                    *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(po);
                else
                    *reinterpret_cast<float2 *>(x) = *reinterpret_cast<const float2 *>(po);
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = wk == 0.f ? o[v] : fmaf(x[v], wk, o[v]);
            }
        }
    }
    if constexpr (kRowWarps > 1) {
        if (lane == 0) {
            sm_m[warp] = mt;
            sm_l[warp] = lt;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) sm_o[warp][lane * V + v] = o[v];
        __syncthreads();
        if (warp != 0) return;
        mt = sm_m[0];
#pragma unroll
        for (int w = 1; w < kRowWarps; ++w) mt = fmaxf(mt, sm_m[w]);
        lt = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            if (sm_m[w] == -INFINITY) {
                lt += sm_l[w];
                continue;
            }
            const float f = fast_exp2(sm_m[w] - mt);
            lt += sm_l[w] * f;
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] += sm_o[w][lane * V + v] * f;
        }
    }
    if (!write) return;
    const float inv = lt > 0.f ? 1.f / lt : (lt == 0.f ? 0.f : lt);
    if (a.lse && lane == 0)
        a.lse[rr] = dead ? 0.f : (lt == 0.f ? -INFINITY : (mt - E::kBias + log2f(lt)) * kLn2);
    const size_t at = (size_t)rr * D + lane * V;
    if (a.out_f32) {
#pragma unroll
        for (int v = 0; v < V; ++v) static_cast<float *>(a.out)[at + v] = o[v] * inv;
    } else {
#pragma unroll
        for (int v = 0; v < V; v += 2)
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at + v) =
                E::pack(o[v] * inv, o[v + 1] * inv);
    }
}

template <typename E, int D, int NT, int OCC>
cudaError_t launch_rows(const CacheAttn &a, int nct, cudaStream_t st)
{
    return launch_kernel(cache_attn_kernel<E, D, NT, OCC>, dim3(nct, a.row_tiles), kThreads, sizeof(Smem<E, D, NT>),
                         sizeof(Smem<E, D, NT>), 1, st, a);
}

template <typename E>
cudaError_t launch_few(const CacheAttn &a, const CacheAttnPlan &p, cudaStream_t st)
{
    static_assert(sizeof(Smem<E, 128, 2>) <= 48 * 1024, "static limit");
    if (a.c.d == 64)
        return p.tile_rows == 8 ? launch_rows<E, 64, 1, 4>(a, p.ctas, st)
                                : launch_rows<E, 64, 2, 3>(a, p.ctas, st);
    return p.tile_rows == 8 ? launch_rows<E, 128, 1, 3>(a, p.ctas, st)
                            : launch_rows<E, 128, 2, 2>(a, p.ctas, st);
}

template <typename E, int D>
cudaError_t launch_join(const CacheAttn &a, const CacheAttnPlan &p, cudaStream_t st)
{
    const int rows = a.c.B * a.c.Hk * a.G * a.T;
    // a row's parts, about: the CTAs of its row tile over the rows of work they share
    const int parts = p.ctas / (a.c.B * a.c.Hk * a.Tp);
    if (parts > 64)
        return launch_kernel(cache_join_kernel<E, D, 16>, dim3(rows), join_threads(16), 0, 0, 1, st, a, p.tile_rows,
                             p.ctas, rows);
    const bool few = parts <= 8;
    return launch_kernel(few ? cache_join_kernel<E, D, 1> : cache_join_kernel<E, D, 4>,
                         dim3(few ? (rows + 3) / 4 : rows), 128, 0, 0, 1, st, a, p.tile_rows, p.ctas, rows);
}

bool strides_map(const ab_cache &c)
{
    return stride_maps(c.k_row, c.page) && stride_maps(c.k_head, c.Hk) && stride_maps(c.k_page, c.n_pages) &&
           stride_maps(c.v_row, c.page) && stride_maps(c.v_head, c.Hk) && stride_maps(c.v_page, c.n_pages);
}

}  // namespace

CacheAttnPlan cache_attn_plan(const ab_cache &c, int G, int T, bool per_token)
{
    CacheAttnPlan p;
    const int rows = per_token ? G : G * T;
    int occ = 2;
    // Over 8 x 16001..32760 slots of 8 heads, d = 128: 24 rows take 281 us in two tiles of 16
    // rows here, which read K and V twice, and 188 us in the tile kernel; 16 rows take 159 us
    // here and 206 us there.
    if (rows > 16 && strides_map(c)) {
        // up to three halves of 128 rows in one CTA (one CTA per SM), as evenly as they come
        const int halves = (rows + 127) / 128, tiles = (halves + 2) / 3;
        p.tile_rows = 128 * ((halves + tiles - 1) / tiles);
        occ = 1;
    } else if (rows <= 8) {
        p.tile_rows = 8;
        occ = c.d == 64 ? 4 : 3;
    } else {
        p.tile_rows = 16;
        occ = c.d == 64 ? 3 : 2;
    }
    p.row_tiles = (rows + p.tile_rows - 1) / p.tile_rows;
    p.ctas = kCacheSms * occ / p.row_tiles;
    if (p.ctas < 1) p.ctas = 1;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t slots = (size_t)2 * p.ctas * p.row_tiles * p.tile_rows;
    p.items = (size_t)c.B * c.Hk * (per_token ? T : 1) * p.row_tiles;
    p.off_ml = up(slots * c.d * sizeof(float));
    p.off_info = p.off_ml + up(slots * sizeof(float2));
    p.bytes = p.off_info + up(p.items * sizeof(int2));
    return p;
}

cudaError_t launch_cache_attn(CacheAttn a, const CacheAttnPlan &p, void *workspace, cudaStream_t st)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.part = reinterpret_cast<float *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(ws + p.off_ml);
    a.info = reinterpret_cast<int2 *>(ws + p.off_info);
    a.row_tiles = p.row_tiles;
    // Every CTA scans the groups to find its run of units, which evens out plans and counts that
    // differ. With very many groups the scan costs more than that can give back: then the CTAs
    // take whole groups in turn. On equal plans (a tenth of 3000..7000 slots, 4 rows, d = 128) whole
    // groups take 647 us and runs 854 us at 16384 groups, 1354 and 1786 at 32768, 330 and 425 at
    // 8192, 48 and 54 at 1024, 15 and 16.5 at 128.
    a.whole_groups = a.idx && a.groups > 8192;
    const bool h = a.c.dtype == AB_F16;
    cudaError_t e = p.tile_rows >= 128 ? launch_cache_tiles(a, p, st)
                    : h                ? launch_few<Fp16>(a, p, st)
                                       : launch_few<Bf16>(a, p, st);
    if (e != cudaSuccess) return e;
    if (a.c.d == 64) return h ? launch_join<Fp16, 64>(a, p, st) : launch_join<Bf16, 64>(a, p, st);
    return h ? launch_join<Fp16, 128>(a, p, st) : launch_join<Bf16, 128>(a, p, st);
}

}  // namespace ab
