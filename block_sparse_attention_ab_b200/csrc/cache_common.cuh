// cache_common.cuh -- what the key/value cache kernels share: the cache as the kernels see
// it, guarded reads of lengths, counts and table entries, 16-bit loads into matrix
// fragments, and the warp-level matrix products of the kernels that are bound by memory.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ab_device.cuh"
#include "ab_kernels.h"

namespace ab {

constexpr int kCacheSms = 148;  // B200: the grids below are sized for its SMs

// Logical page i of sequence b as a pool page, or -1 (with the flag) when the entry is no
// page: nothing is read or written through a bad entry.
__device__ __forceinline__ int cache_page(const ab_cache &c, int b, int i, int *flag)
{
    const int p = c.table[(size_t)b * c.max_pages + i];
    if ((unsigned)p >= (unsigned)c.n_pages) {
        raise_flag(flag, AB_FLAG_BAD_INDEX);
        return -1;
    }
    return p;
}

__device__ __forceinline__ int clamp_flag(int x, int lo, int hi, int *flag)
{
    if (x < lo || x > hi) {
        raise_flag(flag, AB_FLAG_BAD_INDEX);
        x = x < lo ? lo : hi;
    }
    return x;
}

__device__ __forceinline__ int cache_len(const ab_cache &c, const int32_t *len, int b, int *flag)
{
    return clamp_flag(len[b], 0, c.max_pages * c.page, flag);
}

__device__ __forceinline__ int tok_count(const int32_t *n, int b, int T, int *flag)
{
    return n ? clamp_flag(n[b], 0, T, flag) : T;
}

// 16 bytes read once: kept out of L1.
__device__ __forceinline__ uint4 ldg_stream(const void *p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

struct Bf16 {
    using Elem = __nv_bfloat16;
    static constexpr float kBias = 0.f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
    static __device__ __forceinline__ float lo(uint32_t x) { return __uint_as_float(x << 16); }
    static __device__ __forceinline__ float hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
};

struct Fp16 {
    using Elem = __half;
    // fp16 holds nothing below 2^-24: probabilities are kept times 2^7, so that with the
    // running maximum at most 2^8 behind they use 2^15 down to 2^-24 of the type's range
    static constexpr float kBias = 7.f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ float lo(uint32_t x)
    {
        return __half2float(__ushort_as_half((unsigned short)(x & 0xffffu)));
    }
    static __device__ __forceinline__ float hi(uint32_t x)
    {
        return __half2float(__ushort_as_half((unsigned short)(x >> 16)));
    }
};

// d (16 x 8, fp32) += a (16 x 16) b (16 x 8).
template <typename E>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<Bf16>(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<Fp16>(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose an 8 x 8 matrix of 16-bit values held one row of two per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Matrix fragments straight from global memory. A warp takes 16 keys; lane = 4 g + c.
// Keys as the A operand of S^T = K Q^T (16 keys x 16 of d): lane (g, c) loads 16 bytes of
// keys g and g + 8 at d = 32 i + 8 c: two k-steps, whose d order is permuted alike in Q's
// fragment (q_frag), which leaves the dot products as they are. `nv`: keys that exist; the
// others read as 0.
template <int DI>
__device__ __forceinline__ void load_k_frag(uint4 (&kr)[2][DI], const char *kp, int64_t row_bytes,
                                            int nv, int g, int c)
{
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int key = g + 8 * r;
        if (key < nv) {
            const char *p = kp + key * row_bytes + c * 16;
#pragma unroll
            for (int i = 0; i < DI; ++i) kr[r][i] = ldg_stream(p + 64 * i);
        } else {
#pragma unroll
            for (int i = 0; i < DI; ++i) kr[r][i] = make_uint4(0, 0, 0, 0);
        }
    }
}

// Values for O^T = V^T P^T: lane (g, c) loads keys 2c, 2c+1, 2c+8, 2c+9 at d = 8 (g + 8 j).
template <int DJ>
__device__ __forceinline__ void load_v_frag(uint4 (&vr)[4][DJ], const char *vp, int64_t row_bytes,
                                            int nv, int g, int c)
{
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int key = 2 * c + (r & 1) + 8 * (r >> 1);
        if (key < nv) {
            const char *p = vp + key * row_bytes + g * 16;
#pragma unroll
            for (int j = 0; j < DJ; ++j) vr[r][j] = ldg_stream(p + 128 * j);
        } else {
#pragma unroll
            for (int j = 0; j < DJ; ++j) vr[r][j] = make_uint4(0, 0, 0, 0);
        }
    }
}

// s (16 keys x 8 query rows): c0, c1 = (key g, rows 2c, 2c+1), c2, c3 = (key g + 8, ...).
template <typename E, int DI>
__device__ __forceinline__ void qk_product(float (&s)[4], const uint4 (&kr)[2][DI],
                                           const uint4 (&qf)[DI])
{
#pragma unroll
    for (int i = 0; i < DI; ++i) {
        mma16816<E>(s, kr[0][i].x, kr[1][i].x, kr[0][i].y, kr[1][i].y, qf[i].x, qf[i].y);
        mma16816<E>(s, kr[0][i].z, kr[1][i].z, kr[0][i].w, kr[1][i].w, qf[i].z, qf[i].w);
    }
}

// Launch `kern`, as clusters of `cluster` CTAs where that is above 1. Programmatic stream
// serialization: its CTAs may come up while the kernel before it ends, so every kernel launched
// here waits (cudaGridDependencySynchronize) before it reads or writes global memory. That takes
// 1 to 2 us off each of a step's short kernels.
// `smem_most`: the most dynamic shared memory that this kernel is ever launched with. A kernel's
// limit is state of the process that all its calls share, so every call that sets it sets this
// same value: two threads' calls cannot lower it under one another, nor a later call under a
// captured one. The default limit of 48 KB holds for static and dynamic memory together; the
// kernels here have kMostStatic bytes of static memory at most.
constexpr size_t kMostStatic = 12 * 1024;
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kern)(P...), dim3 grid, int threads, size_t smem, size_t smem_most, int cluster,
                          cudaStream_t st, A... args)
{
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024 - kMostStatic)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_most);
    if (e == cudaSuccess && cluster > 8)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace ab
