// cache_mass.cu -- ab_cache_mass: the attention weight that every slot of a paged cache
// received from the newest tokens, added to the slot's mass.
//
// With the rows' log-sums at hand a slot's weight needs its key alone: one read of K, a
// product with all query rows, sum over rows of exp2. As in cache_attn.cu a warp holds 16
// keys as the A operand of m16n8k16, loaded from global memory straight into the fragment;
// the query rows' fragments (up to 256 rows) and log-sums lie in shared memory, in the
// fragment's own order, so a step is one 16-byte shared load per lane for two products. A
// key's sum over rows stays in one warp: no atomics, and the same bits for equal calls. The
// CTAs take equal runs of 64-key units of the sequences' heads in order. Bound by reading K: 16
// sequences of 1023..32760 slots, 40 / 8 heads, d = 128: 105 us, 5.4 TB/s, where the keys change
// from call to call. CTAs per SM, on unchanged keys: three 110 us, four 99, five 120 (they spill);
// d = 64: four 77 us, five 69, six 74, seven 86. More than 8 rows without a plan go to
// cache_mass_tiles.cu.
#include <cstdint>

#include "cache_common.cuh"
#include "cache_kernels.h"

namespace ab {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 16 * kWarps;
constexpr int kStage = 128;       // page slots staged at a time
constexpr int kRows = 256;        // query rows per pass over the keys
constexpr int kUnitPages = kUnit / 16;

struct Staged {
    int page;     // pool page; -1: nothing to do
    int seen;     // some row may see slots of this page
    float shift;  // one plan row for all: log2 of the page's weight, -inf outside the plan
};

template <int D>
struct Smem {
    Staged stage[kStage];
    float row_shift[kUnitPages][AB_MAX_TREE];  // a plan row per token: log2 weight or -inf
    float lse2[kRows];                         // log-sum in base 2; +inf: the row adds nothing
    int bound[kRows];                          // the row sees slots below this
    int tok[kRows];
    long long scan[kWarps];
    int found_group;
    long long found_left;
    uint4 q[1];  // [rows / 8][D / 32][32 lanes]
};

// log2 weight of logical page lp in plan row `at` (ascending), or -inf outside it
__device__ __forceinline__ float plan_shift(const CacheMass &a, size_t row, int lp, int *flag)
{
    const int32_t *idx = a.idx + row * a.c.max_pages;
    int lo = 0, hi = clamp_flag(a.cnt[row], 0, a.c.max_pages, flag);
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (idx[mid] < lp)
            lo = mid + 1;
        else
            hi = mid;
    }
    if (lo >= min(max(a.cnt[row], 0), a.c.max_pages) || idx[lo] != lp) return -INFINITY;
    if (!a.w) return 0.f;
    const float w = a.w[row * a.c.max_pages + lo];
    if (!(w > 0.f && w < INFINITY)) {
        raise_flag(flag, AB_FLAG_BAD_WEIGHT);
        return -INFINITY;
    }
    return log2f(w);
}

template <typename E, int D, int OCC>
__global__ void __launch_bounds__(kThreads, OCC) cache_mass_kernel(const CacheMass a)
{
    constexpr int DI = D / 32;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int page = a.c.page, page_shift = a.page_shift;

    cudaGridDependencySynchronize();
    // ---- this CTA's run of units
    const int per = (a.c.B + kThreads - 1) / kThreads;
    auto units_of = [&](int b, int *flag) {
        const int len = cache_len(a.c, a.c.length, b, flag);
        return (long long)((len + kUnit - 1) / kUnit) * a.c.Hk;
    };
    int *flag0 = blockIdx.x ? nullptr : a.flag;  // one CTA reports the bad lengths and counts, of every sequence
    long long mine = 0;
    for (int b = tid * per; b < min((tid + 1) * per, a.c.B); ++b) {
        mine += units_of(b, flag0);
        if (flag0) tok_count(a.n_tok, b, a.T, flag0);
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
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) incl += sm.scan[w];
        total += sm.scan[w];
    }
    const long long lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
    if (lo >= hi) return;
    if (lo >= incl - mine && lo < incl) {
        long long at = incl - mine;
        for (int b = tid * per;; ++b) {
            const long long u = units_of(b, nullptr);
            if (lo < at + u) {
                sm.found_group = b;
                sm.found_left = lo - at;
                break;
            }
            at += u;
        }
    }
    __syncthreads();
    int b = sm.found_group;
    long long in_group = sm.found_left, left = hi - lo;

    while (left > 0) {
        const int len = cache_len(a.c, a.c.length, b, nullptr);
        const int units = (len + kUnit - 1) / kUnit;
        if (in_group >= (long long)units * a.c.Hk) {
            in_group = 0;
            ++b;
            continue;
        }
        const int hk = (int)(in_group / units), u0 = (int)(in_group % units);
        const int u1 = (int)min((long long)units, u0 + left);
        const int n = min(tok_count(a.n_tok, b, a.T, nullptr), len);
        const int old_len = len - n, rows = n * a.G;
        const char *kbase = static_cast<const char *>(a.c.k) + 2 * hk * a.c.k_head;
        const bool per_row = a.idx && a.per_token;
        int r0 = 0;
        do {  // passes of kRows query rows; one when there are none
            const int nr = min(kRows, rows - r0), tiles = (nr + 7) / 8;
            __syncthreads();
            for (int i = tid; i < tiles * 8; i += kThreads) {
                const int r = r0 + i;
                float l2 = INFINITY;
                int bound = 0, t = 0;
                if (r < rows) {
                    const int k = r / a.G, h = hk * a.G + r % a.G;
                    t = a.sel ? a.sel[(size_t)b * a.T + k] : k;
                    if ((unsigned)t < (unsigned)a.T) {
                        const float l = a.lse[((size_t)b * a.c.Hk * a.G + h) * a.T + t];
                        if (l != -INFINITY) l2 = l * 1.4426950408889634f;
                        bound = old_len + k + 1;
                    } else {
                        raise_flag(a.flag, AB_FLAG_BAD_INDEX);
                        t = 0;
                    }
                }
                sm.lse2[i] = l2;
                sm.bound[i] = bound;
                sm.tok[i] = t;
            }
            for (int i = tid; i < tiles * DI * 32; i += kThreads) {
                const int ln = i & 31, x = (i >> 5) % DI, r = r0 + i / (32 * DI) * 8 + (ln >> 2);
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    const int k = r / a.G, h = hk * a.G + r % a.G;
                    const int t = a.sel ? a.sel[(size_t)b * a.T + k] : k;
                    if ((unsigned)t < (unsigned)a.T)
                        v = *reinterpret_cast<const uint4 *>(static_cast<const char *>(a.q.p) +
                                                             2 * (b * a.q.sb + h * a.q.sh + t * a.q.st) +
                                                             (ln & 3) * 16 + 64 * x);
                }
                sm.q[i] = v;
            }
            __syncthreads();

            const int window = per_row ? kUnitPages : kStage;  // page slots staged together
            int staged0 = -1, seg_end = u0;
            auto stage_from = [&](int u) {
                __syncthreads();
                staged0 = (u * kUnit) >> page_shift;
                const int slots = (len + page - 1) >> page_shift;
                if (per_row) {
                    const int in_unit = max(1, kUnit >> page_shift);
                    for (int i = tid; i < in_unit * n; i += kThreads) {
                        const int s = i / n, k = i % n;
                        const int t = a.sel ? a.sel[(size_t)b * a.T + k] : k;
                        sm.row_shift[s][k] = -INFINITY;
                        if (staged0 + s < slots && (unsigned)t < (unsigned)a.T)
                            sm.row_shift[s][k] = plan_shift(
                                a, ((size_t)b * a.c.Hk + hk) * a.Tp + t, staged0 + s, a.flag);
                    }
                }
                for (int i = tid; i < window && staged0 + i < slots; i += kThreads) {
                    const int lp = staged0 + i;
                    Staged s;
                    s.page = cache_page(a.c, b, lp, a.flag);
                    s.shift = a.idx && !per_row
                                  ? plan_shift(a, ((size_t)b * a.c.Hk + hk) * a.Tp, lp, a.flag)
                                  : 0.f;
                    s.seen = rows > 0 && (s.shift != -INFINITY || (lp + 1) * page > old_len);
                    sm.stage[i] = s;
                }
                __syncthreads();
                seg_end = min(u1, (int)(((long long)(staged0 + window) << page_shift) / kUnit));
                if (per_row) seg_end = u + 1;
            };
            struct Keys {
                int64_t mass;  // index of the first key's mass; -1: nothing to write
                const char *kp;
                int nv, nload;
                float shift;
            };
            auto keys_of = [&](int u) {
                Keys x = {-1, kbase, 0, 0, 0.f};
                const int key = u * kUnit + warp * 16;
                if (key < len) {
                    const Staged s = sm.stage[(key >> page_shift) - staged0];
                    const int r = key & (page - 1);
                    if (s.page >= 0) {
                        x.nv = min(16, len - key);
                        x.nload = s.seen ? x.nv : 0;
                        x.mass = ((int64_t)s.page * a.c.Hk + hk) * page + r;
                        x.kp = kbase + 2 * (s.page * a.c.k_page + r * a.c.k_row);
                        x.shift = s.shift;
                    }
                }
                return x;
            };
            uint4 kr[2][2][DI];
            stage_from(u0);
            Keys cur = keys_of(u0);
            load_k_frag<DI>(kr[0], cur.kp, 2 * a.c.k_row, cur.nload, g, c);
            auto step = [&](int u, uint4 (&kc)[2][DI], uint4 (&kn)[2][DI]) {
                const bool more = u + 1 < u1;
                const float *rsh = sm.row_shift[page >= kUnit ? 0 : (warp * 16) >> page_shift];
                Keys nxt = cur;
                const bool restage = more && u + 1 >= seg_end;
                if (more && !restage) {
                    nxt = keys_of(u + 1);
                    load_k_frag<DI>(kn, nxt.kp, 2 * a.c.k_row, nxt.nload, g, c);
                }
                if (cur.nv > 0) {
                    float old0 = 0.f, old1 = 0.f;
                    const float *in = r0 ? a.out : a.c.mass;
                    const int key = u * kUnit + warp * 16 + g;
                    const bool w0 = c == 0 && g < cur.nv, w1 = c == 1 && g + 8 < cur.nv;
                    if (w0) old0 = in[cur.mass + g];
                    if (w1) old1 = in[cur.mass + g + 8];
                    float s0 = 0.f, s1 = 0.f;
                    if (cur.nload > 0) {
                        const bool edge = u * kUnit + warp * 16 + 16 > old_len;
                        const float sh0 = key < old_len ? cur.shift : 0.f;
                        const float sh1 = key + 8 < old_len ? cur.shift : 0.f;
                        for (int nt = 0; nt < tiles; ++nt) {
                            float s[4] = {0.f, 0.f, 0.f, 0.f};
                            uint4 qf[DI];
#pragma unroll
                            for (int i = 0; i < DI; ++i) qf[i] = sm.q[(nt * DI + i) * 32 + lane];
                            qk_product<E, DI>(s, kc, qf);
                            const float2 l2 = *reinterpret_cast<const float2 *>(&sm.lse2[nt * 8 + 2 * c]);
                            float a0 = sh0 - l2.x, a1 = sh0 - l2.y, a2 = sh1 - l2.x, a3 = sh1 - l2.y;
                            if (per_row) {
                                const int k0 = min(n - 1, (r0 + nt * 8 + 2 * c) / a.G);
                                const int k1 = min(n - 1, (r0 + nt * 8 + 2 * c + 1) / a.G);
                                const float h0 = rsh[k0], h1 = rsh[k1];
                                if (key < old_len) a0 += h0, a1 += h1;
                                if (key + 8 < old_len) a2 += h0, a3 += h1;
                            }
                            // -inf: the row does not exist, saw nothing, or its plan has no such
                            // page; then nothing comes of a logit that is infinite or NaN either
                            float x0 = a0 == -INFINITY ? a0 : fmaf(s[0], a.scale_log2, a0);
                            float x1 = a1 == -INFINITY ? a1 : fmaf(s[1], a.scale_log2, a1);
                            float x2 = a2 == -INFINITY ? a2 : fmaf(s[2], a.scale_log2, a2);
                            float x3 = a3 == -INFINITY ? a3 : fmaf(s[3], a.scale_log2, a3);
                            if (edge) {
                                const int2 bd = *reinterpret_cast<const int2 *>(&sm.bound[nt * 8 + 2 * c]);
                                if (key >= bd.x) x0 = -INFINITY;
                                if (key >= bd.y) x1 = -INFINITY;
                                if (key + 8 >= bd.x) x2 = -INFINITY;
                                if (key + 8 >= bd.y) x3 = -INFINITY;
                            }
                            s0 += fast_exp2(x0) + fast_exp2(x1);
                            s1 += fast_exp2(x2) + fast_exp2(x3);
                        }
#pragma unroll
                        for (int o = 1; o < 4; o <<= 1) {
                            s0 += __shfl_xor_sync(~0u, s0, o);
                            s1 += __shfl_xor_sync(~0u, s1, o);
                        }
                    }
                    if (w0) a.out[cur.mass + g] = old0 + s0;
                    if (w1) a.out[cur.mass + g + 8] = old1 + s1;
                }
                if (restage) {
                    stage_from(u + 1);
                    nxt = keys_of(u + 1);
                    load_k_frag<DI>(kn, nxt.kp, 2 * a.c.k_row, nxt.nload, g, c);
                }
                cur = nxt;
            };
            for (int u = u0; u < u1; u += 2) {
                step(u, kr[0], kr[1]);
                if (u + 1 < u1) step(u + 1, kr[1], kr[0]);
            }
            r0 += kRows;
        } while (r0 < rows);
        left -= u1 - u0;
        in_group += u1 - u0;
    }
}

template <typename E, int D, int OCC>
cudaError_t launch_one(const CacheMass &a, cudaStream_t st)
{
    auto kern = cache_mass_kernel<E, D, OCC>;
    int rows = a.G * a.T;
    if (rows > kRows) rows = kRows;
    auto bytes = [](int tiles) { return (int)(sizeof(Smem<D>) + (size_t)tiles * (D / 32) * 32 * 16); };
    const int smem = bytes((rows + 7) / 8);
    int occ = 220 * 1024 / (smem + 1024);  // CTAs per SM that the shared memory leaves room for
    if (occ > OCC) occ = OCC;
    return launch_kernel(kern, dim3(kCacheSms * occ), kThreads, smem, bytes(kRows / 8), 1, st, a);
}

template <typename E>
cudaError_t launch_d(const CacheMass &a, cudaStream_t st)
{
    return a.c.d == 64 ? launch_one<E, 64, 5>(a, st) : launch_one<E, 128, 4>(a, st);
}

}  // namespace

cudaError_t launch_cache_mass(const CacheMass &a, cudaStream_t st)
{
    const ab_cache &c = a.c;
    // Over 8 x 16380..32760 slots of 8 heads: 8 rows 71 us here and 72 us in the tile kernel, 16
    // rows 76 and 72, 32 rows 96 and 72, 64 rows 139 and 75, 128 rows 225 and 103. The tile
    // kernel takes no plan: of a shared plan's tiles most pages would be outside it, and for plans
    // per token, whose union may be nearly every page, it has no mask of rows by page.
    if (!a.idx && a.G * a.T > 8 && stride_maps(c.k_row, c.page) && stride_maps(c.k_head, c.Hk) &&
        stride_maps(c.k_page, c.n_pages))
        return launch_cache_mass_tiles(a, st);
    return c.dtype == AB_F16 ? launch_d<Fp16>(a, st) : launch_d<Bf16>(a, st);
}

}  // namespace ab
