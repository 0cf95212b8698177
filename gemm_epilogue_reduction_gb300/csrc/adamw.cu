// adamw.cu -- one AdamW step over many tensors, with both moments in 32 bits or in 8 bits.
//
// Per value (formulas and formats in sb.h): read gradient, weight and moments, write weight and
// moments; nothing is read twice, so memory bounds it (28 bytes a value for a bf16 parameter with
// its 32-bit copy and 32-bit moments, 16 with 8-bit moments).  Measured: 622 M values with 32-bit
// moments 2.46 to 2.47 ms (7.1 TB/s), 778 M with 8-bit moments 1.96 to 1.98 ms (6.3 TB/s; the IEEE
// roots keep the SMs busy for half of the time); 128 small tensors 3.1 us back to back in a graph
// (4.4 in 8 bits), of which the search and the 28 KB of kernel parameters are most.
//
// The tensors' descriptors travel in the kernel's parameters, so a call allocates and copies
// nothing; a block finds its tensor by a binary search over the running count of chunks.  A chunk
// is kChunk values of one tensor, and every warp works on one group of 256 values, eight
// consecutive ones to a lane: in 8 bits a group is one block of the format, and its largest
// magnitude is one warp reduction.
//
// What the states keep is rounded operation by operation (no contraction into FMAs; IEEE square
// roots in 8 bits), so that an 8-bit code or scale never differs from the one that the formulas
// give: one differing code changes the next step's update by its spacing.  What meets the weight
// only (the reciprocal, and the root in 32 bits) is the hardware's approximation, with relative
// errors below 2^-22: below the rounding of the weight unless the update is larger than the
// weight.  (With IEEE division as well, the 8-bit kernel was bound by instructions instead of
// memory: 2.98 ms.  Approximate roots with IEEE ones only where a code was in doubt took 2.14 ms.)
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "sb.h"
#include "sb_internal.h"

namespace sb {
namespace {

constexpr int kThreadsAdam = 128;                  // small blocks: more of them fit an SM (2 % over 256)
constexpr int kGroup = 256;                        // values of a block of the 8-bit format
constexpr int kChunk = kGroup * kThreadsAdam / 32; // a group per warp
constexpr int kMaxTensors = 384;                   // of one launch
constexpr float kTop = 448.f;                      // largest E4M3 value
constexpr float kLeast = 0.001953125f;             // smallest one above zero, 2^-9

struct AdamTensor {
    void *p;
    const void *g;
    float *w;  // the 32-bit weight: master, or a 32-bit param
    void *m, *v;
    float *sm, *sv;
    long long n;
    float decay;  // 1 - lr * weight_decay
    int flags;
};
enum : int { kParamF32 = 1, kGradF32 = 2, kWide = 4 };

struct AdamScalars {
    float b1, c1, b2, c2, root, eps, rate;
};

template <int CAP>
struct AdamParams {
    AdamTensor t[CAP];
    unsigned first[CAP + 1];  // running count of chunks
    int count;
    AdamScalars s;
    const float *grad_scale;
};

__device__ __forceinline__ float2 both(float f) { return make_float2(f, f); }
template <bool EXACT>
__device__ __forceinline__ float root_of(float v) {
    if (EXACT) return __fsqrt_rn(v);
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float inverse(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// a·x + b·y with every operation rounded by itself.  (Pair instructions would not do: a product
// and a sum of them may still become one FMA.)
__device__ __forceinline__ float mixed(float x, float a, float y, float b) {
    return __fadd_rn(__fmul_rn(x, a), __fmul_rn(y, b));
}

// One step of two values: m, v and w are replaced; returns the roots of the new v.  EXACT: the
// roots are kept (as 8-bit codes).
template <bool EXACT>
__device__ __forceinline__ float2 advance(const AdamScalars &s, float decay, float2 g, float2 &m,
                                          float2 &v, float2 &w) {
    m = make_float2(mixed(m.x, s.b1, g.x, s.c1), mixed(m.y, s.b1, g.y, s.c1));
    v = make_float2(mixed(v.x, s.b2, __fmul_rn(g.x, g.x), s.c2),
                    mixed(v.y, s.b2, __fmul_rn(g.y, g.y), s.c2));
    const float2 root = make_float2(root_of<EXACT>(v.x), root_of<EXACT>(v.y));
    const float2 den = __ffma2_rn(root, both(s.root), both(s.eps));
    const float2 step = __fmul2_rn(m, make_float2(inverse(den.x), inverse(den.y)));
    w = __ffma2_rn(step, both(-s.rate), __fmul2_rn(w, both(decay)));
    return root;
}

__device__ __forceinline__ float bf16_f(uint16_t b) {
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
}
__device__ __forceinline__ uint16_t f_bf16(float f) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// Eight consecutive values from (to) p, of which the first n count; wide: n == 8 and the address
// is aligned.
__device__ __forceinline__ void load_f32(const float *p, bool wide, int n, float2 (&v)[4]) {
    if (wide) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0];
        const float4 b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w);
        v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = make_float2(2 * j < n ? p[2 * j] : 0.f, 2 * j + 1 < n ? p[2 * j + 1] : 0.f);
    }
}
__device__ __forceinline__ void store_f32(float *p, bool wide, int n, const float2 (&v)[4]) {
    if (wide) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (2 * j < n) p[2 * j] = v[j].x;
            if (2 * j + 1 < n) p[2 * j + 1] = v[j].y;
        }
    }
}
__device__ __forceinline__ void load_bf16(const uint16_t *p, bool wide, int n, float2 (&v)[4]) {
    if (wide) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = make_float2(2 * j < n ? bf16_f(p[2 * j]) : 0.f,
                               2 * j + 1 < n ? bf16_f(p[2 * j + 1]) : 0.f);
    }
}
__device__ __forceinline__ void store_bf16(uint16_t *p, bool wide, int n, const float2 (&v)[4]) {
    if (wide) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[j].x, v[j].y);
            w[j] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (2 * j < n) p[2 * j] = f_bf16(v[j].x);
            if (2 * j + 1 < n) p[2 * j + 1] = f_bf16(v[j].y);
        }
    }
}

// E4M3: two codes in 16 bits, the lower value first.
__device__ __forceinline__ float2 codes_f(uint32_t two) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ void load_codes(const uint8_t *p, float scale, bool wide, int n,
                                           float2 (&v)[4]) {
    uint2 c;
    if (wide) {
        c = *reinterpret_cast<const uint2 *>(p);
    } else {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) w[j / 4] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
        c = make_uint2(w[0], w[1]);
    }
    v[0] = __fmul2_rn(codes_f(c.x & 0xFFFFu), both(scale));
    v[1] = __fmul2_rn(codes_f(c.x >> 16), both(scale));
    v[2] = __fmul2_rn(codes_f(c.y & 0xFFFFu), both(scale));
    v[3] = __fmul2_rn(codes_f(c.y >> 16), both(scale));
}
// The largest magnitude of the warp's 256 values.
__device__ __forceinline__ float warp_top(const float2 (&v)[4]) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(v[j].x), fabsf(v[j].y)));
    // magnitudes order like their bits
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));
}
// What the values are multiplied by to become codes; lane 0 leaves the block's scale.
__device__ __forceinline__ float scale_of(float top, float *scale, int lane) {
    const bool small = top < 7.888609052210118e-31f;  // 2^-100
    if (lane == 0) *scale = small ? 0.f : __fmul_rn(top, static_cast<float>(1.0 / 448.0));
    return small ? 0.f : __fmul_rn(__frcp_rn(top), kTop);
}
// The codes of the warp's 256 values and their scale.  ROOT: values >= 0 whose codes are zero
// only where the value is.
template <bool ROOT>
__device__ __forceinline__ void store_codes(uint8_t *p, float *scale, bool wide, int n, int lane,
                                            const float2 (&v)[4]) {
    const float2 mul = both(scale_of(warp_top(v), scale, lane));
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float2 q = __fmul2_rn(v[j], mul);
        if (ROOT) {
            if (q.x > 0.f) q.x = fmaxf(q.x, kLeast);
            if (q.y > 0.f) q.y = fmaxf(q.y, kLeast);
        }
        c[j] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    }
    const uint2 all = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    if (wide) {
        *reinterpret_cast<uint2 *>(p) = all;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = static_cast<uint8_t>((j < 4 ? all.x : all.y) >> (8 * (j & 3)));
    }
}

template <bool BITS8, int CAP>
__global__ void __launch_bounds__(kThreadsAdam)
    adamw_kernel(const __grid_constant__ AdamParams<CAP> p) {
    int lo = 0, hi = p.count;  // the tensor with first[lo] <= blockIdx.x < first[lo + 1]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.first[mid] <= blockIdx.x)
            lo = mid;
        else
            hi = mid;
    }
    const AdamTensor &t = p.t[lo];
    const int lane = threadIdx.x & 31;
    const long long group =
        static_cast<long long>(blockIdx.x - p.first[lo]) * (kChunk / kGroup) + (threadIdx.x >> 5);
    const long long g0 = group * kGroup;
    if (g0 >= t.n) return;  // the whole warp
    const long long i = g0 + 8 * lane;
    const int n = t.n - i >= 8 ? 8 : (t.n - i > 0 ? static_cast<int>(t.n - i) : 0);
    const bool wide = n == 8 && (t.flags & kWide);
    float2 g[4], w[4], m[4], v[4];
    if (t.flags & kGradF32)
        load_f32(static_cast<const float *>(t.g) + i, wide, n, g);
    else
        load_bf16(static_cast<const uint16_t *>(t.g) + i, wide, n, g);
    if (t.w)
        load_f32(t.w + i, wide, n, w);
    else
        load_bf16(static_cast<const uint16_t *>(t.p) + i, wide, n, w);
    if (BITS8) {
        load_codes(static_cast<const uint8_t *>(t.m) + i, t.sm[group], wide, n, m);
        load_codes(static_cast<const uint8_t *>(t.v) + i, t.sv[group], wide, n, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(v[j], v[j]);
    } else {
        load_f32(static_cast<const float *>(t.m) + i, wide, n, m);
        load_f32(static_cast<const float *>(t.v) + i, wide, n, v);
    }
    const float gs = p.grad_scale ? *p.grad_scale : 1.f;
    float2 root[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        root[j] = advance<BITS8>(p.s, t.decay, __fmul2_rn(g[j], both(gs)), m[j], v[j], w[j]);
    if (t.w) store_f32(t.w + i, wide, n, w);
    if (!(t.flags & kParamF32)) store_bf16(static_cast<uint16_t *>(t.p) + i, wide, n, w);
    if (BITS8) {
        // lanes past the tensor's end hold zeros (their gradients and codes were read as zeros),
        // which change no block's largest magnitude
        store_codes<false>(static_cast<uint8_t *>(t.m) + i, t.sm + group, wide, n, lane, m);
        store_codes<true>(static_cast<uint8_t *>(t.v) + i, t.sv + group, wide, n, lane, root);
    } else {
        store_f32(static_cast<float *>(t.m) + i, wide, n, m);
        store_f32(static_cast<float *>(t.v) + i, wide, n, v);
    }
}

bool on(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Launches tensors[from ..] that are not empty, up to CAP of them and a grid's worth of chunks;
// returns where the next launch starts, or -1 on a launch error.
template <bool BITS8, int CAP>
int64_t launch_some(const sb_adamw_tensor *tensors, int64_t from, int64_t count, double lr,
                    const AdamScalars &s, const float *grad_scale, cudaStream_t stream) {
    AdamParams<CAP> p;
    p.count = 0;
    p.s = s;
    p.grad_scale = grad_scale;
    int64_t chunks = 0, k = from;
    for (; k < count && p.count < CAP; ++k) {
        const sb_adamw_tensor &x = tensors[k];
        if (x.n == 0) continue;
        const int64_t c = (x.n + kChunk - 1) / kChunk;
        if (p.count && chunks + c >= (int64_t(1) << 31)) break;
        AdamTensor &t = p.t[p.count];
        t.p = x.param;
        t.g = x.grad;
        t.w = x.param_type == SB_F32 ? static_cast<float *>(x.param) : x.master;
        t.m = x.exp_avg;
        t.v = x.exp_avg_sq;
        t.sm = x.scale;
        t.sv = x.scale_sq;
        t.n = x.n;
        t.decay = static_cast<float>(1.0 - lr * x.weight_decay);
        const bool wide = on(x.param, 16) && on(x.grad, 16) && on(x.master, 16) &&
                          on(x.exp_avg, 16) && on(x.exp_avg_sq, 16);
        t.flags = (x.param_type == SB_F32 ? kParamF32 : 0) |
                  (x.grad_type == SB_F32 ? kGradF32 : 0) | (wide ? kWide : 0);
        p.first[p.count++] = static_cast<unsigned>(chunks);
        chunks += c;
    }
    if (p.count == 0) return k;
    p.first[p.count] = static_cast<unsigned>(chunks);
    adamw_kernel<BITS8, CAP><<<static_cast<unsigned>(chunks), kThreadsAdam, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? k : -1;
}

template <bool BITS8>
int32_t launch_all(const sb_adamw_tensor *tensors, int64_t count, double lr, const AdamScalars &s,
                   const float *grad_scale, cudaStream_t stream) {
    // the parameters of a launch are copied whole: a short list takes a short structure
    for (int64_t k = 0; k < count;) {
        k = count - k <= 16
                ? launch_some<BITS8, 16>(tensors, k, count, lr, s, grad_scale, stream)
                : launch_some<BITS8, kMaxTensors>(tensors, k, count, lr, s, grad_scale, stream);
        if (k < 0) return SB_ERR_CUDA;
    }
    return SB_OK;
}

}  // namespace
}  // namespace sb

using namespace sb;

extern "C" int32_t sb_adamw_step(const sb_adamw_tensor *tensors, int64_t count, double lr,
                                 double beta1, double beta2, double eps, int64_t step,
                                 int32_t state_bits, const float *grad_scale, void *stream) {
    if (count < 0 || (count > 0 && !tensors) || !(lr >= 0 && std::isfinite(lr)) ||
        !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) ||
        !(eps >= 0 && std::isfinite(eps)) || step < 1 || (state_bits != 8 && state_bits != 32))
        return SB_ERR_INVALID_ARG;
    if (!on(grad_scale, 4)) return SB_ERR_ALIGNMENT;
    for (int64_t k = 0; k < count; ++k) {
        const sb_adamw_tensor &x = tensors[k];
        if (x.n < 0 || x.n > (int64_t(1) << 40) || x.param_type < SB_BF16 ||
            x.param_type > SB_F32 || x.grad_type < SB_BF16 || x.grad_type > SB_F32 ||
            !(x.weight_decay >= 0 && std::isfinite(x.weight_decay)))
            return SB_ERR_INVALID_ARG;
        if (x.n == 0) continue;
        if (!x.param || !x.grad || !x.exp_avg || !x.exp_avg_sq ||
            (x.master && x.param_type == SB_F32) || (state_bits == 8 && (!x.scale || !x.scale_sq)))
            return SB_ERR_INVALID_ARG;
        const uintptr_t sa = state_bits == 8 ? 1 : 4;
        if (!on(x.param, x.param_type == SB_F32 ? 4 : 2) ||
            !on(x.grad, x.grad_type == SB_F32 ? 4 : 2) || !on(x.master, 4) || !on(x.exp_avg, sa) ||
            !on(x.exp_avg_sq, sa) || !on(x.scale, 4) || !on(x.scale_sq, 4))
            return SB_ERR_ALIGNMENT;
    }
    if (int32_t e = device_sms_cc(nullptr, nullptr)) return e;
    AdamScalars s{};
    s.b1 = static_cast<float>(beta1);
    s.c1 = static_cast<float>(1.0 - beta1);
    s.b2 = static_cast<float>(beta2);
    s.c2 = static_cast<float>(1.0 - beta2);
    s.root = static_cast<float>(
        1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
    s.eps = static_cast<float>(eps);
    s.rate = static_cast<float>(lr / (1.0 - std::pow(beta1, static_cast<double>(step))));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return state_bits == 8 ? launch_all<true>(tensors, count, lr, s, grad_scale, st)
                           : launch_all<false>(tensors, count, lr, s, grad_scale, st);
}
