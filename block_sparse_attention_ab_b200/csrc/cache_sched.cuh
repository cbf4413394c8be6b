// cache_sched.cuh -- how the attention kernels over a key/value cache share out their work:
// units of 64 keys of one (sequence, key head[, plan row]), which the CTAs take in equal runs.
#pragma once

#include "cache_common.cuh"
#include "cache_kernels.h"

namespace ab {

constexpr int kUnit = 64;    // keys per unit
constexpr float kLazy = 8.f; // the running maximum may lag by 2^8
constexpr float kLn2 = 0.69314718055994531f;

struct Staged {
    int page;     // pool page, -1: takes no part
    int valid;    // its valid rows
    float shift;  // log2 of its weight
};

// Units and multiplicity of group `gi`: a sequence (without a plan) or a (b, hk, plan row).
struct Group {
    int b, hk, tp;      // hk -1: all key heads
    int n;              // new tokens
    int ctx;            // virtual keys of the cache: slots, or plan entries times page
    int ctx_units, units, mult;
};

__device__ __forceinline__ Group load_group(const CacheAttn &a, int gi, int *flag)
{
    Group g;
    g.tp = 0;
    g.hk = -1;
    g.mult = a.c.Hk;
    if (a.idx) {
        g.tp = gi % a.Tp;
        const int bh = gi / a.Tp;
        g.hk = bh % a.c.Hk;
        g.b = bh / a.c.Hk;
        g.mult = 1;
    } else {
        g.b = gi;
    }
    g.n = tok_count(a.n_tok, g.b, a.T, flag);
    g.units = 0;
    g.ctx = 0;
    g.ctx_units = 0;
    if (g.n == 0 || (a.per_token && g.tp >= g.n)) return g;
    if (a.idx)
        g.ctx = clamp_flag(a.cnt[gi], 0, a.c.max_pages, flag) * a.c.page;
    else
        g.ctx = cache_len(a.c, a.c.length, g.b, flag);
    g.ctx_units = (g.ctx + kUnit - 1) / kUnit;
    g.units = g.ctx_units + (a.k.p ? (g.n + kUnit - 1) / kUnit : 0);
    return g;
}

__device__ __forceinline__ int group_rows(const CacheAttn &a, const Group &g)
{
    return a.per_token ? a.G : g.n * a.G;
}

// A CTA's place in the run of all units: group, units of it already behind, units to do.
struct Run {
    int group;
    long long in_group, left;
};

struct RunSmem {  // up to 16 warps
    long long scan[16];
    int group;
    long long in_group;
};

// The run of CTA `cta` of `nct` (all kThreads threads call this); left = 0: nothing to do.
// With a.whole_groups the CTA starts at group `cta` and steps by nct itself.
template <int kThreads>
__device__ __forceinline__ Run find_run(const CacheAttn &a, RunSmem &sm, int cta, int nct, int *flag)
{
    static_assert(kThreads / 32 <= 16, "RunSmem");
    Run run = {a.groups, 0, 0};
    if (a.whole_groups) {
        run.group = cta;
        run.left = 1;
        return run;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.groups + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int i = tid * per; i < min((tid + 1) * per, a.groups); ++i) {
        const Group gr = load_group(a, i, flag);
        mine += (long long)gr.units * gr.mult;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) incl += sm.scan[w];
        total += sm.scan[w];
    }
    // at least one unit for every CTA that takes part: a row's parts lie in CTAs without a
    // gap between them
    const long long parts = min((long long)nct, total);
    if (cta >= parts) return run;
    const long long lo = total * cta / parts, hi = total * (cta + 1) / parts;
    if (lo >= incl - mine && lo < incl) {
        long long at = incl - mine;
        for (int i = tid * per;; ++i) {
            const Group gr = load_group(a, i, nullptr);
            const long long u = (long long)gr.units * gr.mult;
            if (lo < at + u) {
                sm.group = i;
                sm.in_group = lo - at;
                break;
            }
            at += u;
        }
    }
    __syncthreads();
    run.group = sm.group;
    run.in_group = sm.in_group;
    run.left = hi - lo;
    return run;
}

// One piece of a run: units [u0, u1) of key head hk of the group.
struct Piece {
    Group g;
    int hk, u0, u1, gi;
};

// The run's next piece; false when it has ended. The run moves on past it.
__device__ __forceinline__ bool next_piece(const CacheAttn &a, Run &run, int nct, Piece &p, int *flag)
{
    while (run.group < a.groups && run.left > 0) {
        p.gi = run.group;
        p.g = load_group(a, run.group, a.whole_groups ? flag : nullptr);
        p.hk = p.g.hk;
        if (a.whole_groups) {
            run.group += nct;
            if (p.g.units == 0) continue;
            p.u0 = 0;
            p.u1 = p.g.units;
            return true;
        }
        if (run.in_group >= (long long)p.g.units * p.g.mult) {
            run.in_group = 0;
            ++run.group;
            continue;
        }
        if (p.hk < 0) p.hk = (int)(run.in_group / p.g.units);
        p.u0 = (int)(run.in_group % p.g.units);
        p.u1 = (int)min((long long)p.g.units, p.u0 + run.left);
        run.in_group += p.u1 - p.u0;
        run.left -= p.u1 - p.u0;
        return true;
    }
    return false;
}

// Page slot `slot` of the piece's context as the kernels use it. cap: the sequence's length.
__device__ __forceinline__ Staged stage_entry(const CacheAttn &a, const Piece &p, int slot, int cap, int *flag)
{
    Staged s = {-1, 0, 0.f};
    int lp = slot;
    if (a.idx) {
        const size_t at = (size_t)p.gi * a.c.max_pages + slot;
        lp = a.idx[at];
        if ((unsigned)lp >= (unsigned)a.c.max_pages) {
            raise_flag(flag, AB_FLAG_BAD_INDEX);
            return s;
        }
        if (a.w) {
            const float w = a.w[at];
            if (!(w > 0.f && w < INFINITY)) {
                raise_flag(flag, AB_FLAG_BAD_WEIGHT);
                return s;
            }
            s.shift = log2f(w);
        }
    }
    if (lp * a.c.page < cap) {
        s.page = cache_page(a.c, p.g.b, lp, flag);
        s.valid = min(a.c.page, cap - lp * a.c.page);
    }
    return s;
}

}  // namespace ab
