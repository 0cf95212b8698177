// norm_common.cuh -- what both directions of the residual norm (norm.cu) share: the layout of a row
// over threads, loads and stores of bf16 and fp32 in fp32 pairs, the ring of rows on their way,
// and the sums over a row.
#pragma once
#include <atomic>
#include <type_traits>
#include <cuda_bf16.h>

#include "sb_internal.h"
#include "sb_ptx.cuh"

namespace sb {

constexpr int kMaxNormD = 16384;
constexpr int kMaxDepth = 4;
constexpr int kMaxGroups = 12;                 // of a block; each has a barrier of its own
constexpr size_t kNormRingBytes = 200 * 1024;  // of an SM's shared memory

// How a row is laid out: a group of row_threads threads, EPT values to a thread in steps of VEC
// consecutive ones, step i at (i * row_threads + thread) * VEC.
struct NormShape {
    int vec, ept, max_threads;
};

struct NormParams {
    int M, d;
    int row_threads;  // threads of a row's group, a multiple of 32
    int groups;       // of a block
    int depth;        // rows of a group's ring; 0: no ring
    int w32;          // weights in fp32 (otherwise bf16)
    float scale, eps, inv_d;
    const void *h, *y, *pre, *post;
    const void *gate;           // one vector (null: none)
    const void *gate_rows;      // one per row (null: none)
    void *h_out, *x;            // forward
    const void *dx, *dh;        // backward
    void *dh_out, *dy, *dgate_rows;
    float *part;                // [blocks][sums][d]: dx·h'·rh, and t·(gate of the row)·y·ry
    int sums;
};

cudaError_t launch_norm_forward(const NormParams &p, NormShape s, bool h32, int blocks, size_t smem,
                                cudaStream_t st);
cudaError_t launch_norm_backward(const NormParams &p, NormShape s, bool h32, int blocks, size_t smem,
                                 cudaStream_t st);

__device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 v) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ float2 both(float f) { return make_float2(f, f); }

// N values (8 or 4) as pairs; the address is aligned to them (to 16 bytes where that is more).
template <int N>
__device__ __forceinline__ void load_pairs(const float *p, float2 *v) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float4 x = reinterpret_cast<const float4 *>(p)[i];
        v[2 * i] = make_float2(x.x, x.y);
        v[2 * i + 1] = make_float2(x.z, x.w);
    }
}
template <int N>
__device__ __forceinline__ void load_pairs(const __nv_bfloat16 *p, float2 *v) {
    if constexpr (N == 8) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        v[0] = unpack2(x.x), v[1] = unpack2(x.y), v[2] = unpack2(x.z), v[3] = unpack2(x.w);
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        v[0] = unpack2(x.x), v[1] = unpack2(x.y);
    }
}
template <int N>
__device__ __forceinline__ void store_pairs(float *p, const float2 *v) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        reinterpret_cast<float4 *>(p)[i] =
            make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
}
template <int N>
__device__ __forceinline__ void store_pairs(__nv_bfloat16 *p, const float2 *v) {
    if constexpr (N == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3]));
    else
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(v[0]), pack2(v[1]));
}
__device__ __forceinline__ float one(const float *p) { return *p; }
__device__ __forceinline__ float one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put_one(float *p, float v) { *p = v; }
__device__ __forceinline__ void put_one(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// This thread's values of a row in memory, zeros past its end.
template <int VEC, int EPT, typename T>
__device__ __forceinline__ void get(const T *row, int rt, int t, int d, float2 (&v)[EPT / 2]) {
#pragma unroll
    for (int i = 0; i < EPT / VEC; ++i) {
        const int e = (i * rt + t) * VEC;
        if constexpr (VEC == 1) {
            const float f = e < d ? one(row + e) : 0.f;
            if (i & 1)
                v[i / 2].y = f;
            else
                v[i / 2].x = f;
        } else if (e < d) {
            load_pairs<VEC>(row + e, v + i * (VEC / 2));
        } else {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) v[i * (VEC / 2) + j] = both(0.f);
        }
    }
}
template <int VEC, int EPT, typename T>
__device__ __forceinline__ void put(T *row, int rt, int t, int d, const float2 (&v)[EPT / 2]) {
#pragma unroll
    for (int i = 0; i < EPT / VEC; ++i) {
        const int e = (i * rt + t) * VEC;
        if (e < d) {
            if constexpr (VEC == 1)
                put_one(row + e, (i & 1) ? v[i / 2].y : v[i / 2].x);
            else
                store_pairs<VEC>(row + e, v + i * (VEC / 2));
        }
    }
}
// A weight vector (w32 is the same for all threads); ones where there is none.
template <int VEC, int EPT>
__device__ __forceinline__ void get_weight(const void *w, int w32, int rt, int t, int d,
                                           float2 (&v)[EPT / 2]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < EPT / 2; ++i) v[i] = both(1.f);
    } else if (w32) {
        get<VEC, EPT>(static_cast<const float *>(w), rt, t, d, v);
    } else {
        get<VEC, EPT>(static_cast<const __nv_bfloat16 *>(w), rt, t, d, v);
    }
}

// ------------------------------------------------------------------ the ring of rows ahead
// One array of a row in shared memory: a thread's VEC values of a step lie in pieces of 16 (or
// 8) bytes, piece by piece over the group's threads, so that neighbours touch neighbours.
template <int VEC, int EPT, typename T>
struct RingArray {
    static constexpr int kBytes = VEC * static_cast<int>(sizeof(T));
    static constexpr int kCount = kBytes > 16 ? kBytes / 16 : 1;
    static constexpr int kPiece = kBytes / kCount;
    static constexpr int kPerThread = EPT * static_cast<int>(sizeof(T));

    static __device__ __forceinline__ void copy(uint8_t *at, const T *row, int rt, int t, int d) {
#pragma unroll
        for (int i = 0; i < EPT / VEC; ++i) {
            const int e = (i * rt + t) * VEC;
            if (e < d) {
#pragma unroll
                for (int c = 0; c < kCount; ++c) {
                    const uint32_t dst = smem_u32(at) + ((i * kCount + c) * rt + t) * kPiece;
                    const T *from = row + e + c * (VEC / kCount);
                    if constexpr (kPiece == 16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(from)
                                     : "memory");
                    else
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(from)
                                     : "memory");
                }
            }
        }
    }
    // Zeros where `copy` never writes, past the row's end: `get` then reads without asking.
    static __device__ __forceinline__ void clear(uint8_t *at, int rt, int t, int d) {
#pragma unroll
        for (int i = 0; i < EPT / VEC; ++i)
            if ((i * rt + t) * VEC >= d)
                for (int c = 0; c < kCount * kPiece / 4; ++c)
                    *reinterpret_cast<uint32_t *>(
                        at + ((i * kCount + c / (kPiece / 4)) * rt + t) * kPiece +
                        c % (kPiece / 4) * 4) = 0u;
    }
    static __device__ __forceinline__ void get(const uint8_t *at, int rt, int t,
                                               float2 (&v)[EPT / 2]) {
        constexpr int N = VEC / kCount;
#pragma unroll
        for (int i = 0; i < EPT / VEC; ++i)
#pragma unroll
            for (int c = 0; c < kCount; ++c)
                load_pairs<N>(
                    reinterpret_cast<const T *>(at + ((i * kCount + c) * rt + t) * kPiece),
                    v + i * (VEC / 2) + c * (N / 2));
    }
};
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the last `pending` rows of this thread's have arrived.
__device__ __forceinline__ void ring_wait(int pending) {
    switch (pending) {
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
}
static_assert(kMaxDepth <= 4, "ring_wait");

// ------------------------------------------------------------------ sums over a row
// Barrier of one group (several groups of a block wait independently).
__device__ __forceinline__ void group_sync(int group, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// Words of shared memory that a group of at most WARPS warps needs for one value's sum, and
// how far apart the groups' words are.
__host__ __device__ constexpr int sum_words(int warps) { return (warps + 3) / 4 * 4; }

// Sum of one value over the group; every thread gets it.  red: the group's own sum_words(warps)
// words, 16-byte aligned, zero past the last warp's, not to be written again before another
// group_sync.  Every thread adds up the warps' sums itself: fewer dependent steps than a second
// round of shuffles.
template <int MAXT>
__device__ __forceinline__ float row_sum(float v, int group, int threads, float *red) {
    const int warps = threads >> 5;
    const int warp = (threadIdx.x - group * threads) >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (warps > 1) {
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        group_sync(group, threads);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < MAXT / 32; w += 4)
            if (w < warps) {
                const float4 x = *reinterpret_cast<const float4 *>(red + w);
                a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
            }
        v = (a.x + a.y) + (a.z + a.w);
    }
    return v;
}

// Sums of N <= 8 values.  In the warp, eight values take nine shuffles: three halving steps
// leave each lane one value's sum over eight lanes.  red: the group's own 8 * warps words, not
// to be written again before another group_sync.
template <int MAXT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int group, int threads, float *red) {
    const int lane = threadIdx.x & 31, warps = threads >> 5;
    const int warp = (threadIdx.x - group * threads) >> 5;
    float x[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = n < N ? v[n] : 0.f;
#pragma unroll
    for (int half = 4; half > 0; half >>= 1) {
        const bool up = lane & (half * 4);  // bits 4, 3, 2 of the lane
#pragma unroll
        for (int n = 0; n < half; ++n) {
            const float keep = up ? x[n + half] : x[n], give = up ? x[n] : x[n + half];
            x[n] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, half * 4);
        }
    }
    float a = x[0];
    a += __shfl_xor_sync(0xFFFFFFFFu, a, 1);
    a += __shfl_xor_sync(0xFFFFFFFFu, a, 2);
    // lanes 4k .. 4k + 3 hold value k's sum over the warp
    if (warps > 1) {
        if ((lane & 3) == 0) red[warp * 8 + (lane >> 2)] = a;
        group_sync(group, threads);
        a = 0.f;
#pragma unroll
        for (int w = 0; w < MAXT / 32; w += 4)
            if (w + (lane & 3) < warps) a += red[(w + (lane & 3)) * 8 + (lane >> 2)];
        a += __shfl_xor_sync(0xFFFFFFFFu, a, 1);
        a += __shfl_xor_sync(0xFFFFFFFFu, a, 2);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = __shfl_sync(0xFFFFFFFFu, a, 4 * n);
}

// ------------------------------------------------------------------ launch
template <typename P, typename K>
cudaError_t launch_dependent(K kern, dim3 grid, int threads, size_t smem, const P &p,
                             cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// `kern` with the shared-memory opt-in, which is per device (remembered in `opted_in`).
inline cudaError_t launch_norm_kernel(void (*kern)(const NormParams), std::atomic<uint64_t> &opted_in,
                                      const NormParams &p, int blocks, size_t smem,
                                      cudaStream_t st) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (!bit || !(opted_in.load() & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kNormRingBytes));
        if (e != cudaSuccess) return e;
        opted_in.fetch_or(bit);
    }
    return launch_dependent(kern, dim3(blocks), p.groups * p.row_threads, smem, p, st);
}

// Calls f.template operator()<T, VEC, EPT, MAXT, ROWS>() for the call's types and shape.
template <typename F>
cudaError_t for_norm_shape(NormShape s, bool h32, bool rows, F f) {
    auto typed = [&](auto h) {
        using T = decltype(h);
        auto shaped = [&](auto with_rows) {
            constexpr bool R = decltype(with_rows)::value;
            if (s.vec == 8) {
                if (s.max_threads == 384) return f.template operator()<T, 8, 16, 384, R>();
                if (s.max_threads == 512) return f.template operator()<T, 8, 16, 512, R>();
                return f.template operator()<T, 8, 16, 1024, R>();
            }
            if (s.vec == 4) {
                if (s.max_threads == 384) return f.template operator()<T, 4, 16, 384, R>();
                return f.template operator()<T, 4, 16, 1024, R>();
            }
            if (s.max_threads == 384) return f.template operator()<T, 1, 16, 384, R>();
            return f.template operator()<T, 1, 16, 1024, R>();
        };
        return rows ? shaped(std::true_type{}) : shaped(std::false_type{});
    };
    return h32 ? typed(float{}) : typed(__nv_bfloat16{});
}

}  // namespace sb
