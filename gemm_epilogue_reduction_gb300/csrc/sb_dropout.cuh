// sb_dropout.cuh -- which elements dropout keeps, and what it does to them (dropout.cu and the
// layer norm's branch).
//
// Element i takes the 16-bit field i mod 4 of draw i / 4 (sb_counter.cuh), counted from the lowest
// bits, and is dropped where the field is below t = round(65536 p): one draw serves four elements,
// some 7 integer instructions each, which hides behind the memory traffic of bf16 (one draw for
// each element would not: 25 instructions for 4 bytes).  What is kept is multiplied by 65536 /
// (65536 - t), the inverse of the probability that is really met, so the expectation is exact
// whatever the rounding of p.  The mask is a function of seed and index alone: the backward pass
// forms it again, and no pass stores it.
#pragma once
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "sb_counter.cuh"

namespace sb {

struct Dropout {
    unsigned long long seed;
    const unsigned long long *offset;  // added to the seed (null: 0), read when the kernel runs
    uint32_t below;                    // (t << 16) - 1 for t of 1 .. 65536
    int on;                            // t > 0
    float scale;
};

inline Dropout make_dropout(float p, uint64_t seed, const void *offset) {
    const uint32_t t = static_cast<uint32_t>(std::nearbyint(static_cast<double>(p) * 65536.0));
    Dropout d{};
    d.seed = seed;
    d.offset = static_cast<const unsigned long long *>(offset);
    d.below = (t << 16) - 1u;
    d.on = t > 0;
    d.scale = t < 65536u ? static_cast<float>(65536.0 / (65536.0 - t)) : 0.f;
    return d;
}

__device__ __forceinline__ unsigned long long dropout_seed(const Dropout &d) {
    return d.seed + (d.offset ? *d.offset : 0ull);
}

// The draws of four consecutive elements that start at a multiple of 4: element k of them is kept
// where field(k) > below, with the field in the upper half of a word.
struct DropoutFields {
    uint32_t lo, hi;
    __device__ __forceinline__ uint32_t field(int k) const {
        const uint32_t w = k & 2 ? hi : lo;
        return k & 1 ? w : w << 16;  // what lies below the field cannot change the comparison
    }
};
__device__ __forceinline__ DropoutFields dropout_fields_at(unsigned long long state) {
    const unsigned long long x = bits64_from_state(state);
    return DropoutFields{static_cast<uint32_t>(x), static_cast<uint32_t>(x >> 32)};
}
__device__ __forceinline__ DropoutFields dropout_fields(unsigned long long seed,
                                                        unsigned long long group) {
    return dropout_fields_at(splitmix_state(seed, group));
}
// x, or zero where it is dropped: no trace of it, not even of a NaN or an infinity.
__device__ __forceinline__ float dropout_keep(float x, uint32_t field, uint32_t below) {
    return field > below ? x : 0.f;
}
// v = base + dropout(v) for the four elements of a draw, in two pairs.
__device__ __forceinline__ void dropout_add4(const float2 *base, float2 *v, const DropoutFields &f,
                                             uint32_t below, float scale) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        v[k].x = f.field(2 * k) > below ? fmaf(v[k].x, scale, base[k].x) : base[k].x;
        v[k].y = f.field(2 * k + 1) > below ? fmaf(v[k].y, scale, base[k].y) : base[k].y;
    }
}

}  // namespace sb
