// dropout.cu -- dropout from a counter-based generator, with or without the sum into a residual
// stream: out_i = residual_i + keep_i x_i / (1 - p)  (which elements are kept: sb_dropout.cuh).
// The call is its own gradient: the gradient of x is dropout of the gradient of out.
//
// Bound by memory: x (and the residual) in once, out once.  Eight values to a thread and step, four
// steps of loads in flight; blocks end with their 8192 values (8192 x 6144 bf16 with residual: 43.5 us,
// 6.9 TB/s).  Some ten instructions an element, half of them the draw, hide behind that.
#include "norm_common.cuh"
#include "sb.h"
#include "sb_dropout.cuh"

namespace sb {
namespace {

constexpr int kDropThreads = 256;
constexpr int kDropSteps = 4;

struct DropoutParams {
    const void *x, *residual;
    void *out;
    long long n;
    Dropout drop;
};

// VEC 8: arrays on 16-byte boundaries; VEC 4: any, value by value.  (Four is what a draw serves.)
template <typename X, typename O, int VEC, bool RES>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const DropoutParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // no early launch_dependents: what follows may read `out` as a weight, ahead of this kernel's end
    const X *x = static_cast<const X *>(p.x);
    const O *res = static_cast<const O *>(p.residual);
    O *out = static_cast<O *>(p.out);
    const unsigned long long seed = dropout_seed(p.drop);
    const long long first =
        (static_cast<long long>(blockIdx.x) * (kDropThreads * kDropSteps) + threadIdx.x) * VEC;
    float2 v[kDropSteps][VEC / 2], r[kDropSteps][VEC / 2];
#pragma unroll
    for (int s = 0; s < kDropSteps; ++s) {
        const long long i = first + static_cast<long long>(s) * kDropThreads * VEC;
        if (VEC == 8 && i + VEC <= p.n) {
            load_pairs<VEC>(x + i, v[s]);
            if (RES) load_pairs<VEC>(res + i, r[s]);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float a = i + k < p.n ? one(x + i + k) : 0.f;
                const float b = RES && i + k < p.n ? one(res + i + k) : 0.f;
                (k & 1 ? v[s][k / 2].y : v[s][k / 2].x) = a;
                (k & 1 ? r[s][k / 2].y : r[s][k / 2].x) = b;
            }
        }
    }
#pragma unroll
    for (int s = 0; s < kDropSteps; ++s) {
        const long long i = first + static_cast<long long>(s) * kDropThreads * VEC;
        if (i >= p.n) break;
#pragma unroll
        for (int h = 0; h < VEC / 4; ++h) {
            DropoutFields f{~0u, ~0u};
            uint32_t below = 0;
            if (p.drop.on) {
                f = dropout_fields(seed, static_cast<unsigned long long>(i) / 4 + h);
                below = p.drop.below;
            }
            if (!RES) r[s][2 * h] = r[s][2 * h + 1] = both(0.f);
            dropout_add4(r[s] + 2 * h, v[s] + 2 * h, f, below, p.drop.scale);
        }
        if (VEC == 8 && i + VEC <= p.n) {
            store_pairs<VEC>(out + i, v[s]);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (i + k < p.n) put_one(out + i + k, k & 1 ? v[s][k / 2].y : v[s][k / 2].x);
        }
    }
}

template <typename X, typename O>
cudaError_t launch_dropout(const DropoutParams &p, bool wide, cudaStream_t st) {
    const long long per = static_cast<long long>(kDropThreads) * kDropSteps * (wide ? 8 : 4);
    const dim3 grid(static_cast<unsigned>((p.n + per - 1) / per));
    if (wide)
        return p.residual
                   ? launch_dependent(dropout_kernel<X, O, 8, true>, grid, kDropThreads, 0, p, st)
                   : launch_dependent(dropout_kernel<X, O, 8, false>, grid, kDropThreads, 0, p, st);
    return p.residual
               ? launch_dependent(dropout_kernel<X, O, 4, true>, grid, kDropThreads, 0, p, st)
               : launch_dependent(dropout_kernel<X, O, 4, false>, grid, kDropThreads, 0, p, st);
}

}  // namespace
}  // namespace sb

using namespace sb;

extern "C" int32_t sb_dropout(const void *x, const void *residual, int64_t n, int32_t x_type,
                              int32_t out_type, float p, uint64_t seed,
                              const uint64_t *seed_offset, void *out, void *stream) {
    if (n < 0 || n > (int64_t(1) << 42) || (n > 0 && (!x || !out)) || x_type < SB_BF16 ||
        x_type > SB_F32 || out_type < SB_BF16 || out_type > SB_F32 || !(p >= 0.f && p <= 1.f))
        return SB_ERR_INVALID_ARG;
    const uintptr_t xa = x_type == SB_F32 ? 4 : 2, oa = out_type == SB_F32 ? 4 : 2;
    if (!on(x, xa) || !on(residual, oa) || !on(out, oa) || !on(seed_offset, 8))
        return SB_ERR_ALIGNMENT;
    const size_t ob = n * oa;
    if ((x_type == out_type ? overlap_partly(out, ob, x, n * xa) : overlap(out, ob, x, n * xa)) ||
        overlap_partly(out, ob, residual, ob) || overlap(out, ob, seed_offset, 8))
        return SB_ERR_INVALID_ARG;
    if (int32_t e = device_sms_cc(nullptr, nullptr)) return e;
    if (n == 0) return SB_OK;
    DropoutParams d{};
    d.x = x;
    d.residual = residual;
    d.out = out;
    d.n = n;
    d.drop = make_dropout(p, seed, seed_offset);
    const bool wide = on(x, 16) && on(residual, 16) && on(out, 16);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    using B = __nv_bfloat16;
    cudaError_t e;
    if (x_type == SB_BF16)
        e = out_type == SB_BF16 ? launch_dropout<B, B>(d, wide, st) : launch_dropout<B, float>(d, wide, st);
    else
        e = out_type == SB_BF16 ? launch_dropout<float, B>(d, wide, st)
                                : launch_dropout<float, float>(d, wide, st);
    return e == cudaSuccess ? SB_OK : SB_ERR_CUDA;
}
