// cache_ops.cu -- keeping a paged key/value cache: writing new tokens (ab_cache_append),
// scoring its pages for a query (ab_cache_score), choosing the slots a bounded cache keeps
// (ab_cache_keep) and moving them together (ab_cache_compact).
#include <cooperative_groups.h>
#include <cstdint>

#include "cache_common.cuh"
#include "cache_kernels.h"

namespace cg = cooperative_groups;

namespace ab {
namespace {

// ---------------------------------------------------------------------------------
// A page's key sum, the same bits whoever computes it: 128 threads, D / 8 lanes per row;
// row group r0 adds rows r0, r0 + RG, r0 + 2 RG, ... in that order, and the groups' sums
// are added in group order, all in fp32.
// ---------------------------------------------------------------------------------
constexpr int kPageThreads = 128;

template <int D>
struct PageSum {
    static constexpr int kLanes = D / 8, kGroups = kPageThreads / kLanes;
    float acc[8];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    }
    template <typename E>
    __device__ __forceinline__ void add(const uint4 &x)
    {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[2 * i] += E::lo(w[i]);
            acc[2 * i + 1] += E::hi(w[i]);
        }
    }
    // all threads; sm: kGroups * D floats
    __device__ __forceinline__ void finish(float *sm, float *out)
    {
        const int tid = threadIdx.x;
        float4 *p = reinterpret_cast<float4 *>(sm + (tid / kLanes) * D + (tid % kLanes) * 8);
        p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        __syncthreads();
        for (int d = tid; d < D; d += kPageThreads) {
            float s = sm[d];
#pragma unroll
            for (int r = 1; r < kGroups; ++r) s += sm[r * D + d];
            out[d] = s;
        }
    }
};

// ---------------------------------------------------------------------------------
// ab_cache_append: one CTA per (page that receives a token, key head, sequence). The page's
// older keys are read once more for its sum; every new row is read and written once. A sequence
// that is cut inside a page and receives nothing has that page's sum made anew too. Bound by
// that for a prompt (49140 tokens of 12 heads: 108 us, 5.7 TB/s), by the launch for a token.
// ---------------------------------------------------------------------------------
struct AppendArgs {
    ab_cache c;
    ab_tokens k, v;
    int T;
    const int32_t *n_new, *sel, *start, *pos0;
    int *flag;
};

template <typename E, int D>
__global__ void __launch_bounds__(kPageThreads) cache_append_kernel(const AppendArgs a)
{
    using Sum = PageSum<D>;
    __shared__ __align__(16) float sm[Sum::kGroups * D];
    cudaGridDependencySynchronize();
    const int b = blockIdx.z, hk = blockIdx.y, tid = threadIdx.x;
    const bool first = blockIdx.x == 0 && hk == 0;
    int *flag = first && tid == 0 ? a.flag : nullptr;
    const int page = a.c.page, cap = a.c.max_pages * page;
    const int n_ask = tok_count(a.n_new, b, a.T, flag);
    const int s0 = a.start ? a.start[b] : a.c.length[b];
    if (s0 < 0 || s0 > cap) {
        raise_flag(flag, AB_FLAG_BAD_INDEX);
        return;
    }
    const int n = min(n_ask, cap - s0), len = s0 + n;
    if (n < n_ask) raise_flag(flag, AB_FLAG_CACHE_FULL);
    if (first && tid == 0 && a.start) a.c.length[b] = len;
    const int lp = s0 / page + blockIdx.x;
    if (lp * page >= len || (n == 0 && !(a.start && a.c.ksum))) return;
    const int pg = cache_page(a.c, b, lp, a.flag);
    if (pg < 0) return;
    const int rows = min(page, len - lp * page), lane = tid % Sum::kLanes;
    char *kp = static_cast<char *>(a.c.k) + 2 * (pg * a.c.k_page + hk * a.c.k_head) + lane * 16;
    char *vp = static_cast<char *>(a.c.v) + 2 * (pg * a.c.v_page + hk * a.c.v_head) + lane * 16;
    const char *kn = static_cast<const char *>(a.k.p) + 2 * (b * a.k.sb + hk * a.k.sh) + lane * 16;
    const char *vn = static_cast<const char *>(a.v.p) + 2 * (b * a.v.sb + hk * a.v.sh) + lane * 16;
    Sum sum;
    sum.clear();
#pragma unroll 4
    for (int r = tid / Sum::kLanes; r < rows; r += Sum::kGroups) {
        const int i = lp * page + r - s0;  // new token, or an older row
        uint4 x;
        if (i < 0) {
            x = *reinterpret_cast<const uint4 *>(kp + 2 * r * a.c.k_row);
        } else {
            const int t = a.sel ? a.sel[(size_t)b * a.T + i] : i;
            uint4 y;
            if ((unsigned)t < (unsigned)a.T) {
                x = ldg_stream(kn + 2 * t * a.k.st);
                y = ldg_stream(vn + 2 * t * a.v.st);
            } else {
                raise_flag(a.flag, AB_FLAG_BAD_INDEX);
                x = y = make_uint4(0, 0, 0, 0);
            }
            *reinterpret_cast<uint4 *>(kp + 2 * r * a.c.k_row) = x;
            *reinterpret_cast<uint4 *>(vp + 2 * r * a.c.v_row) = y;
        }
        sum.template add<E>(x);
    }
    const size_t head = (size_t)pg * a.c.Hk + hk;
    for (int r = tid; r < rows; r += kPageThreads) {
        const int i = lp * page + r - s0;
        if (i < 0) continue;
        if (a.c.mass) a.c.mass[head * page + r] = 0.f;
        if (a.c.pos) a.c.pos[head * page + r] = (a.pos0 ? a.pos0[b] : s0) + i;
    }
    if (a.c.ksum) sum.finish(sm, a.c.ksum + head * D);
}

// length += n_new where the append started at length: in a kernel behind it, because every
// CTA of the append reads the old length.
__global__ void cache_length_kernel(const AppendArgs a)
{
    cudaGridDependencySynchronize();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= a.c.B) return;
    const int cap = a.c.max_pages * a.c.page, s0 = a.c.length[b];
    if (s0 < 0 || s0 > cap) return;
    a.c.length[b] = s0 + min(tok_count(a.n_new, b, a.T, nullptr), cap - s0);
}

// ---------------------------------------------------------------------------------
// ab_cache_score: bound by one read of the pages' key sums. A cluster of CTAs takes one
// (sequence, key head[, token]); each CTA keeps its pages' logits in shared memory, the
// clusters exchange row maxima and sums through distributed shared memory, so one launch
// reads every sum once and writes every score once. Eight lanes share a page; a warp has
// 8 pages (4 KB at d = 128) in flight. 32 sequences of 4097..32760 slots in pages of 16, 40 / 8
// heads: 42 us, 3.6 TB/s: the longest clusters' chain of phases. Clusters twice as large took 53
// us, one CTA each 66, half the pages in flight 67, twice as many 43.
// ---------------------------------------------------------------------------------
constexpr int kScoreThreads = 256;
constexpr int kScoreLanes = 8;

struct ScoreArgs {
    ab_cache c;
    ab_tokens q;
    const int32_t *n_tok;
    int G, T, Tp, first, recent;
    bool per_token;
    float scale_log2;
    float *scores;
    int *flag;
    int chunk;   // query rows at a time
    int slice;   // most pages of one CTA
};

template <typename E, int D>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const ScoreArgs a)
{
    constexpr int V = D / 32;  // float4s per lane
    extern __shared__ __align__(16) float sm[];
    cudaGridDependencySynchronize();
    cg::cluster_group cl = cg::this_cluster();
    const int cs = cl.num_blocks(), rank = cl.block_rank();
    const int item = blockIdx.x / cs;
    const int tp = item % a.Tp, hk = item / a.Tp % a.c.Hk, b = item / a.Tp / a.c.Hk;
    float *sm_q = sm;                               // [chunk][D]
    float2 *sm_st = reinterpret_cast<float2 *>(sm_q + a.chunk * D);  // [chunk] this CTA's max, sum
    float2 *sm_tot = sm_st + a.chunk;               // [chunk] the cluster's max, 1 / sum
    float *sm_acc = reinterpret_cast<float *>(sm_tot + a.chunk);     // [slice]
    int *sm_page = reinterpret_cast<int *>(sm_acc + a.slice);        // [slice]
    float *sm_x = reinterpret_cast<float *>(sm_page + a.slice);      // [chunk][slice]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = tok_count(a.n_tok, b, a.T, tid == 0 ? a.flag : nullptr);
    const int len = cache_len(a.c, a.c.length, b, tid == 0 ? a.flag : nullptr);
    const int page = a.c.page, pages = (len + page - 1) / page;
    const int t0 = a.per_token ? tp : 0, t1 = a.per_token ? tp + 1 : n;
    const int rows = t0 < n ? (t1 - t0) * a.G : 0;
    const int sl = (pages + cs - 1) / cs, p0 = min(pages, rank * sl), np = min(pages, p0 + sl) - p0;
    float *out = a.scores + (size_t)item * a.c.max_pages;

    for (int i = tid; i < np; i += kScoreThreads) {
        sm_page[i] = rows ? cache_page(a.c, b, p0 + i, a.flag) : -1;
        sm_acc[i] = 0.f;
    }
    for (int r0 = 0; r0 < rows; r0 += a.chunk) {
        const int nr = min(a.chunk, rows - r0);
        for (int i = tid; i < nr * (D / 8); i += kScoreThreads) {
            const int r = r0 + i / (D / 8), e = i % (D / 8);
            const int t = t0 + r / a.G, h = hk * a.G + r % a.G;
            const uint4 x = *reinterpret_cast<const uint4 *>(
                static_cast<const char *>(a.q.p) + 2 * (b * a.q.sb + h * a.q.sh + t * a.q.st) + e * 16);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            float *d = sm_q + (i / (D / 8)) * D + e * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[2 * j] = E::lo(w[j]);
                d[2 * j + 1] = E::hi(w[j]);
            }
        }
        __syncthreads();
        // ---- logits, in the base-2 exponent's scale
        constexpr int kPer = 32 / kScoreLanes, kUnroll = 2;
        const int sub = lane / kScoreLanes, l8 = lane % kScoreLanes;
        for (int i0 = warp * kPer * kUnroll; i0 < np; i0 += (kScoreThreads / 32) * kPer * kUnroll) {
            float4 x[kUnroll][V];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = i0 + u * kPer + sub;
                const int pg = i < np ? sm_page[i] : -1;
                const float *p = a.c.ksum + ((size_t)max(pg, 0) * a.c.Hk + hk) * D + l8 * 4;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    x[u][v] = pg >= 0 ? *reinterpret_cast<const float4 *>(p + v * 32)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            for (int r = 0; r < nr; ++r) {
                float4 q[V];
#pragma unroll
                for (int v = 0; v < V; ++v)
                    q[v] = *reinterpret_cast<const float4 *>(sm_q + r * D + l8 * 4 + v * 32);
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float s = 0.f;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        s = fmaf(x[u][v].x, q[v].x, s);
                        s = fmaf(x[u][v].y, q[v].y, s);
                        s = fmaf(x[u][v].z, q[v].z, s);
                        s = fmaf(x[u][v].w, q[v].w, s);
                    }
#pragma unroll
                    for (int o = 1; o < kScoreLanes; o <<= 1) s += __shfl_xor_sync(~0u, s, o);
                    const int i = i0 + u * kPer + sub;
                    if (l8 == 0 && i < np) {
                        const int size = min(page, len - (p0 + i) * page);
                        sm_x[r * a.slice + i] = sm_page[i] >= 0 ? s * (a.scale_log2 / size) : -INFINITY;
                    }
                }
            }
        }
        __syncthreads();
        // ---- each row's maximum and sum over this CTA's pages, one warp per row
        for (int r = warp; r < nr; r += kScoreThreads / 32) {
            float m = -INFINITY;
            for (int i = lane; i < np; i += 32) m = fmaxf(m, sm_x[r * a.slice + i]);
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            // nothing but bad pages: a sum of 0; nothing but NaN: NaN
            const float base = m == -INFINITY ? 0.f : m;
            float s = 0.f;
            for (int i = lane; i < np; i += 32) s += exp2f(sm_x[r * a.slice + i] - base);
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
            if (lane == 0) sm_st[r] = make_float2(m, s);
        }
        cl.sync();
        for (int r = tid; r < nr; r += kScoreThreads) {
            float m = -INFINITY, s = 0.f;
            for (int k = 0; k < cs; ++k) m = fmaxf(m, cl.map_shared_rank(sm_st, k)[r].x);
            for (int k = 0; k < cs; ++k) {
                const float2 st = cl.map_shared_rank(sm_st, k)[r];
                s += st.x == -INFINITY ? st.y : st.y * exp2f(st.x - m);
            }
            sm_tot[r] = make_float2(m == -INFINITY ? 0.f : m, s > 0.f ? 1.f / s : (s == 0.f ? 0.f : s));
        }
        __syncthreads();
        for (int i = tid; i < np; i += kScoreThreads) {
            float acc = sm_acc[i];
            for (int r = 0; r < nr; ++r) {
                const float2 t = sm_tot[r];
                acc += exp2f(sm_x[r * a.slice + i] - t.x) * t.y;
            }
            sm_acc[i] = acc;
        }
        cl.sync();  // nobody reads this chunk's maxima any more
    }
    __syncthreads();
    const float inv = rows ? 1.f / rows : 0.f;
    for (int i = tid; i < np; i += kScoreThreads) {
        const int p = p0 + i;
        const bool kept = rows && (p < a.first || p >= pages - a.recent);
        out[p] = kept ? 2.f : sm_acc[i] * inv;
    }
    for (int p = pages + rank * kScoreThreads + tid; p < a.c.max_pages; p += cs * kScoreThreads) out[p] = 0.f;
}

// ---------------------------------------------------------------------------------
// ab_cache_keep: a radix selection of the budget-th largest score (three digits of the
// fp32 bits, which order as the values do for values >= 0), then one ordered pass that
// ranks holes and movers. Bound by one read of scores and positions (8 bytes per slot); its
// CTAs hold the keys of their slots in shared memory, so that happens once. One CTA takes a
// (sequence, key head); long ones take a cluster of CTAs that add their histograms through
// distributed shared memory (launch_cache_keep has the rule and its figures). 256 heads of 4160
// slots: 19 us in one CTA each, 50 in clusters of two.
// ---------------------------------------------------------------------------------
constexpr int kKeepBins = 2048;
constexpr int kKeepSmem = 45 * 1024;  // keys of one CTA held in shared memory (180 KB)
static_assert((kKeepBins + 64) * sizeof(int) <= kMostStatic, "the histogram and the scans' words");

// The key of a slot at index `at` of score and pos: order of the score, +inf when recent.
__device__ __forceinline__ uint32_t keep_key(float x, int pos, int recent, int limit, int *flag)
{
    if (recent > 0 && pos >= limit) return 0x7f800000u;
    if (!(x >= 0.f)) {
        raise_flag(flag, AB_FLAG_BAD_SCORE);
        return 0;
    }
    return __float_as_uint(x) & 0x7fffffffu;  // -0 counts as 0
}

// Sum of x over the threads before this one, and over all.
template <int kThreads>
__device__ __forceinline__ int block_scan(int x, int *sm_warp, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) sm_warp[warp] = incl;
    __syncthreads();
    // every warp scans the warps' sums
    const int mine = lane < kThreads / 32 ? sm_warp[lane] : 0;
    int w = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(~0u, w, 31);
    return __shfl_sync(~0u, w - mine, warp) + incl - x;
}

// kFar: a CTA has more slots than it holds keys; those are read again in every pass.
template <bool kCluster, bool kFar, int kThreads>
__global__ void __launch_bounds__(kThreads, kFar ? 1 : 2) cache_keep_kernel(const CacheKeep a, int held, int page_shift)
{
    extern __shared__ __align__(16) uint32_t keys[];  // [held]: keys, later the slots' sources
    __shared__ int hist[kKeepBins];
    __shared__ int sm_warp[32];
    __shared__ int sm_digit, sm_above;
    __shared__ int3 sm_cnt;  // this CTA's keys equal to the threshold, holes, movers
    cudaGridDependencySynchronize();
    cg::cluster_group cl = cg::this_cluster();
    const int cs = kCluster ? cl.num_blocks() : 1, rank = kCluster ? cl.block_rank() : 0, tid = threadIdx.x;
    auto sync = [&]() {
        if (kCluster)
            cl.sync();
        else
            __syncthreads();
    };
    const int item = blockIdx.x / cs, hk = item % a.c.Hk, b = item / a.c.Hk;
    const int page = a.c.page;
    const int len = cache_len(a.c, a.length, b, tid == 0 ? a.flag : nullptr);
    const int m = min(len, a.budget);
    int32_t *src = a.src + (size_t)item * a.budget;
    if (hk == 0 && rank == 0 && tid == 0) a.n_keep[b] = m;
    for (int j = m + rank * kThreads + tid; j < a.budget; j += cs * kThreads) src[j] = -1;
    if (len <= a.budget) {
        for (int j = rank * kThreads + tid; j < m; j += cs * kThreads) src[j] = j;
        return;
    }
    const int limit = a.recent > 0 ? (int)max((long long)a.next_pos[b] - a.recent, (long long)INT32_MIN) : 0;
    const int sl = (len + cs - 1) / cs, s0 = min(len, rank * sl), ns = min(len, s0 + sl) - s0;
    auto index_of = [&](int i) -> int64_t {  // of slot s0 + i in score and pos, or -1
        const int slot = s0 + i, pg = cache_page(a.c, b, slot >> page_shift, a.flag);
        return pg < 0 ? -1 : ((int64_t)pg * a.c.Hk + hk) * page + (slot & (page - 1));
    };
    auto key_far = [&](int i) -> uint32_t {  // a key that is not held
        const int64_t at = index_of(i);
        return at < 0 ? 0 : keep_key(a.score[at], a.recent > 0 ? a.pos[at] : 0, a.recent, limit, a.flag);
    };
    auto key_of = [&](int i) { return !kFar || i < held ? keys[i] : key_far(i); };
    for (int i = tid; i < kKeepBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    // four slots per thread in flight; the first digit is counted on the way
    const int nh = min(ns, held);
    for (int i0 = tid; i0 < nh; i0 += 4 * kThreads) {
        int64_t at[4];
        float x[4];
        int p[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) at[q] = i0 + q * kThreads < nh ? index_of(i0 + q * kThreads) : -1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[q] = at[q] >= 0 ? a.score[at[q]] : 0.f;
            p[q] = at[q] >= 0 && a.recent > 0 ? a.pos[at[q]] : INT32_MIN;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (i0 + q * kThreads >= nh) break;
            const uint32_t k = at[q] < 0 ? 0 : keep_key(x[q], p[q], a.recent, limit, a.flag);
            keys[i0 + q * kThreads] = k;
            atomicAdd(&hist[k >> 20], 1);
        }
    }

    // ---- threshold: `need` keys are kept among those that share the digits found so far
    uint32_t prefix = 0, mask = 0;
    int need = m;
    constexpr int kPer = kKeepBins / kThreads;
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 20 : d == 1 ? 9 : 0, bits = d == 2 ? 9 : 11;
        if (d > 0) {
            for (int i = tid; i < kKeepBins; i += kThreads) hist[i] = 0;
            __syncthreads();
        }
        for (int i = (d == 0 ? nh : 0) + tid; i < ns; i += kThreads) {  // none at first unless kFar
            const uint32_t k = key_of(i);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
        }
        sync();
        // bins from the highest down, kPer per thread
        int h[kPer], sum = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int bin = kKeepBins - 1 - (kPer * tid + j);
            h[j] = 0;
            if (kCluster)
                for (int k = 0; k < cs; ++k) h[j] += cl.map_shared_rank(hist, k)[bin];
            else
                h[j] = hist[bin];
            sum += h[j];
        }
        int total;
        int above = block_scan<kThreads>(sum, sm_warp, &total);
        if (above < need && above + sum >= need) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (above < need && above + h[j] >= need) {
                    sm_digit = kKeepBins - 1 - (kPer * tid + j);
                    sm_above = above;
                    break;
                }
                above += h[j];
            }
        }
        sync();  // the histograms are read; the digit is visible
        prefix |= (uint32_t)sm_digit << shift;
        mask |= ((1u << bits) - 1) << shift;
        need -= sm_above;
        __syncthreads();
    }

    // ---- one ordered pass: thread t takes the slots [t per, (t + 1) per) of the CTA (an odd
    // number, so that the threads' shared memory reads fall into different banks)
    const int per = ((ns + kThreads - 1) / kThreads) | 1;
    const int i0 = min(ns, tid * per), i1 = min(ns, i0 + per);
    int eq = 0;
    for (int i = i0; i < i1; ++i) eq += key_of(i) == prefix;
    int total;
    int eq_rank = block_scan<kThreads>(eq, sm_warp, &total);
    if (kCluster) {
        if (tid == 0) sm_cnt.x = total;
        cl.sync();
        for (int k = 0; k < rank; ++k) eq_rank += cl.map_shared_rank(&sm_cnt, k)->x;
    }
    int holes = 0, movers = 0, e = eq_rank;
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = key_of(i);
        const bool kept = k > prefix || (k == prefix && e < need);
        e += k == prefix;
        if (s0 + i < m)
            holes += !kept;
        else
            movers += kept;
    }
    int hole_rank = block_scan<kThreads>(holes, sm_warp, &total);
    if (kCluster && tid == 0) sm_cnt.y = total;
    int mover_rank = block_scan<kThreads>(movers, sm_warp, &total);
    if (kCluster) {
        if (tid == 0) sm_cnt.z = total;
        cl.sync();
        for (int k = 0; k < rank; ++k) {
            const int3 *o = cl.map_shared_rank(&sm_cnt, k);
            hole_rank += o->y;
            mover_rank += o->z;
        }
    }
    // the movers' slots by rank; a held slot below m keeps its own number, or its rank among
    // the holes, in place of its key
    int32_t *mv = a.movers + (size_t)item * a.budget;
    e = eq_rank;
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = key_of(i);
        const bool kept = k > prefix || (k == prefix && e < need);
        e += k == prefix;
        const int s = s0 + i;
        if (s >= m) {
            if (kept) mv[mover_rank++] = s;
        } else if (!kFar || i < held) {
            keys[i] = kept ? (uint32_t)s : 0x80000000u | hole_rank;
            hole_rank += !kept;
        } else {
            src[s] = kept ? s : -1 - hole_rank;
            hole_rank += !kept;
        }
    }
    __threadfence();
    sync();
    for (int i = tid; i < ns && s0 + i < m; i += kThreads) {
        const int s = s0 + i;
        if (!kFar || i < held) {
            const uint32_t k = keys[i];
            src[s] = k & 0x80000000u ? __ldcg(mv + (k & 0x7fffffffu)) : (int)k;
        } else {
            const int k = __ldcg(src + s);
            if (k < 0) src[s] = __ldcg(mv + (-1 - k));
        }
    }
}

// ---------------------------------------------------------------------------------
// ab_cache_compact: one CTA per (page below the budget, key head, sequence). Rows move from
// slots >= n_keep to slots < n_keep only, so no CTA writes what another one reads. A page
// that changed is read whole for its sum. Bound by the moved rows (read and written once) and
// those sums; the first threads look the rows' sources up, so that every row's loads are
// independent. 256 heads with 64 of 4096 slots to fill: 38 us for 170 MB of changed pages; 32
// heads, 0.33 GB of moves: 73 us.
// ---------------------------------------------------------------------------------
template <typename E, int D>
__global__ void __launch_bounds__(kPageThreads, 8)
    cache_compact_kernel(const ab_cache c, int budget, int page_shift, const int32_t *src_all,
                         const int32_t *n_keep, int *flag)
{
    using Sum = PageSum<D>;
    __shared__ __align__(16) float sm[Sum::kGroups * D];
    __shared__ int sm_page[128], sm_row[128];  // pool page and row of each row's source
    cudaGridDependencySynchronize();
    const int lp = blockIdx.x, hk = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int page = c.page, cap = c.max_pages << page_shift;
    const bool first = lp == 0 && hk == 0 && tid == 0;
    const int n = clamp_flag(n_keep[b], 0, min(budget, cap), first ? flag : nullptr);
    if (first) c.length[b] = n;
    if (lp << page_shift >= n) return;
    const int rows = min(page, n - (lp << page_shift));
    bool moves = false;
    int s = 0;
    const int j = (lp << page_shift) + tid;
    if (tid < rows) {
        s = src_all[((size_t)b * c.Hk + hk) * budget + j];
        if (s != j && (s < n || s >= cap)) {
            raise_flag(flag, AB_FLAG_BAD_INDEX);
            s = j;
        }
        moves = s != j;
    }
    const bool changed = __syncthreads_or(moves);
    if (!changed && rows == page) return;
    const int pg = cache_page(c, b, lp, flag);
    if (pg < 0) return;
    const size_t head = (size_t)pg * c.Hk + hk;
    if (tid < rows) {
        int from = moves ? cache_page(c, b, s >> page_shift, flag) : -1;
        sm_page[tid] = from;
        sm_row[tid] = s & (page - 1);
        if (from >= 0) {
            const size_t f = ((size_t)from * c.Hk + hk) * page + (s & (page - 1)), t = head * page + tid;
            if (c.mass) c.mass[t] = c.mass[f];
            if (c.pos) c.pos[t] = c.pos[f];
        }
    }
    __syncthreads();
    const int lane = tid % Sum::kLanes;
    char *kc = static_cast<char *>(c.k) + 2 * hk * c.k_head + lane * 16;
    char *vc = static_cast<char *>(c.v) + 2 * hk * c.v_head + lane * 16;
    char *kp = kc + 2 * pg * c.k_page, *vp = vc + 2 * pg * c.v_page;
    Sum sum;
    sum.clear();
    constexpr int kBatch = 4;
    for (int r0 = tid / Sum::kLanes; r0 < rows; r0 += kBatch * Sum::kGroups) {
        uint4 x[kBatch], y[kBatch];
        int from[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int r = r0 + q * Sum::kGroups;
            from[q] = r < rows ? sm_page[r] : -1;
            const int64_t fr = from[q] >= 0 ? sm_row[r] : r;
            if (r < rows && (from[q] >= 0 || c.ksum))
                x[q] = ldg_stream(from[q] >= 0 ? kc + 2 * (from[q] * c.k_page + fr * c.k_row) : kp + 2 * fr * c.k_row);
            if (from[q] >= 0) y[q] = ldg_stream(vc + 2 * (from[q] * c.v_page + fr * c.v_row));
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int64_t r = r0 + q * Sum::kGroups;
            if (from[q] >= 0) {
                *reinterpret_cast<uint4 *>(kp + 2 * r * c.k_row) = x[q];
                *reinterpret_cast<uint4 *>(vp + 2 * r * c.v_row) = y[q];
            }
            if (r < rows) sum.template add<E>(x[q]);
        }
    }
    if (c.ksum) sum.finish(sm, c.ksum + head * D);
}

int shift_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

}  // namespace

cudaError_t launch_cache_append(const ab_cache &c, const ab_tokens &k, const ab_tokens &v, int T,
                                const int32_t *n_new, const int32_t *sel, const int32_t *start,
                                const int32_t *pos0, int *flag, cudaStream_t st)
{
    const AppendArgs a = {c, k, v, T, n_new, sel, start, pos0, flag};
    // T tokens touch at most this many pages, wherever they start
    const dim3 grid((T - 1) / c.page + 2, c.Hk, c.B);
    const bool h = c.dtype == AB_F16;
    auto kern = c.d == 64 ? (h ? cache_append_kernel<Fp16, 64> : cache_append_kernel<Bf16, 64>)
                          : (h ? cache_append_kernel<Fp16, 128> : cache_append_kernel<Bf16, 128>);
    const cudaError_t e = launch_kernel(kern, grid, kPageThreads, 0, 0, 1, st, a);
    if (e != cudaSuccess || start) return e;
    return launch_kernel(cache_length_kernel, dim3((c.B + 127) / 128), 128, 0, 0, 1, st, a);
}

cudaError_t launch_cache_score(const ab_cache &c, const ab_tokens &q, int G, int T,
                               const int32_t *n_tok, bool per_token, int first, int recent,
                               float *scores, int *flag, cudaStream_t st)
{
    ScoreArgs a;
    a.c = c;
    a.q = q;
    a.n_tok = n_tok;
    a.G = G;
    a.T = T;
    a.Tp = per_token ? T : 1;
    a.first = first;
    a.recent = recent;
    a.per_token = per_token;
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)c.d);
    a.scores = scores;
    a.flag = flag;
    const int items = c.B * c.Hk * a.Tp;
    // enough CTAs for every SM, at least 32 pages each; more than 8 pages' logits per thread
    // of a CTA always split
    int cs = 1;
    while (cs < 16 && ((items * cs < 2 * kCacheSms && c.max_pages >= 64 * cs) || c.max_pages > 2048 * cs)) cs *= 2;
    a.slice = (c.max_pages + cs - 1) / cs;
    const int rows = per_token ? G : G * T;
    const size_t most = 160 * 1024, room = most - (size_t)a.slice * 8;
    a.chunk = (int)(room / ((size_t)a.slice * 4 + c.d * 4 + 16));
    if (a.chunk > 32) a.chunk = 32;
    if (a.chunk > rows) a.chunk = rows;
    const size_t smem = (size_t)a.chunk * (c.d * 4 + 16 + a.slice * 4) + (size_t)a.slice * 8;
    const bool h = c.dtype == AB_F16;
    auto kern = c.d == 64 ? (h ? page_score_kernel<Fp16, 64> : page_score_kernel<Bf16, 64>)
                          : (h ? page_score_kernel<Fp16, 128> : page_score_kernel<Bf16, 128>);
    return launch_kernel(kern, dim3(items * cs), kScoreThreads, smem, most, cs, st, a);
}

cudaError_t launch_cache_keep(const CacheKeep &a, cudaStream_t st)
{
    const int cap = a.c.max_pages * a.c.page, items = a.c.B * a.c.Hk;
    const int shift = shift_of(a.c.page);
    // As few CTAs as hold a head's keys (36864 each), because a cluster's barriers and remote
    // histograms cost more than they share out; up to four where the GPU would stand empty. 128
    // heads of 32760 slots: 34 us in one CTA each, 41 in two, 71 in four; 32 heads of 118800: 43
    // in four, 69 in eight; 32 heads of 60000: 29 in four, 38 in two.
    int cs = 1;
    while (cs < 8 && cap > 36864 * cs) cs *= 2;
    while (cs < 4 && cap > 8192 * cs && items * cs * 2 <= kCacheSms) cs *= 2;
    if (cs == 1)
        return launch_kernel(cache_keep_kernel<false, false, 1024>, dim3(items), 1024, (size_t)cap * 4, kKeepSmem * 4,
                             1, st, a, cap, shift);
    int held = (cap + cs - 1) / cs;
    if (held > kKeepSmem) held = kKeepSmem;
    auto kern = held * cs < cap ? cache_keep_kernel<true, true, 1024> : cache_keep_kernel<true, false, 1024>;
    return launch_kernel(kern, dim3(items * cs), 1024, (size_t)held * 4, kKeepSmem * 4, cs, st, a, held, shift);
}

cudaError_t launch_cache_compact(const ab_cache &c, int budget, const int32_t *src,
                                 const int32_t *n_keep, int *flag, cudaStream_t st)
{
    const int most = budget < c.max_pages * c.page ? budget : c.max_pages * c.page;
    const dim3 grid((most + c.page - 1) / c.page, c.Hk, c.B);
    const bool h = c.dtype == AB_F16;
    auto kern = c.d == 64 ? (h ? cache_compact_kernel<Fp16, 64> : cache_compact_kernel<Bf16, 64>)
                          : (h ? cache_compact_kernel<Fp16, 128> : cache_compact_kernel<Bf16, 128>);
    return launch_kernel(kern, grid, kPageThreads, 0, 0, 1, st, c, budget, shift_of(c.page), src, n_keep, flag);
}

}  // namespace ab
