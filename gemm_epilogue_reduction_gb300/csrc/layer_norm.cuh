// layer_norm.cuh -- what the layer norm's kernels and their host side (layer_norm.cu) share.
#pragma once
#include "norm_common.cuh"
#include "sb_dropout.cuh"

namespace sb {

struct LayerNormParams {
    int M, d;
    int row_threads;  // threads of a row's group, a multiple of 32
    int groups;       // of a block
    int depth;        // rows of a group's ring; 0: no ring
    int w32;          // weights in fp32 (otherwise bf16)
    float eps, inv_d;
    const void *h, *y, *weight, *bias;
    void *h_out, *x;          // forward
    const void *dx, *dh;      // backward
    void *dh_out, *dy;
    float *part;              // [blocks][sums][d]: dx·(h - mean)·r, and dx
    int sums;
    Dropout drop;
};

cudaError_t launch_layer_norm_forward(const LayerNormParams &p, NormShape s, bool h32, int blocks,
                                      size_t smem, cudaStream_t st);
cudaError_t launch_layer_norm_backward(const LayerNormParams &p, NormShape s, bool h32, int blocks,
                                       size_t smem, cudaStream_t st);

// v less the row's mean; zeros stay past the row's end, where they add nothing to the sums.
template <int VEC, int EPT>
__device__ __forceinline__ void centre(float mean, int rt, int t, int d, float2 (&v)[EPT / 2]) {
#pragma unroll
    for (int i = 0; i < EPT / VEC; ++i) {
        const float m = (i * rt + t) * VEC < d ? mean : 0.f;
        if constexpr (VEC == 1) {
            (i & 1 ? v[i / 2].y : v[i / 2].x) -= m;
        } else {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) v[i * (VEC / 2) + j] = __fadd2_rn(v[i * (VEC / 2) + j], both(-m));
        }
    }
}

// base + dropout(v) for this thread's values of the row that starts at element `row`.
template <int VEC, int EPT>
__device__ __forceinline__ void add_dropped(const Dropout &drop, unsigned long long seed,
                                            unsigned long long row, int rt, int t, int d,
                                            const float2 (&base)[EPT / 2], float2 (&v)[EPT / 2]) {
    if (!drop.on) {
#pragma unroll
        for (int i = 0; i < EPT / 2; ++i) v[i] = __fadd2_rn(base[i], v[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < EPT / VEC; ++i) {
        const unsigned long long at = row + static_cast<unsigned>((i * rt + t) * VEC);
        if constexpr (VEC == 1) {
            // past the row's end the draw is another row's; the zeros there stay zeros
            const DropoutFields f = dropout_fields(seed, at / 4);
            const int k = static_cast<int>(at & 3);
            const uint32_t w = k & 2 ? f.hi : f.lo, field = k & 1 ? w : w << 16;
            float &x = i & 1 ? v[i / 2].y : v[i / 2].x;
            x = dropout_add(i & 1 ? base[i / 2].y : base[i / 2].x, x, field, drop.below, drop.scale);
        } else {
#pragma unroll
            for (int h = 0; h < VEC / 4; ++h) {
                const DropoutFields f = dropout_fields(seed, at / 4 + h);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int j = i * (VEC / 2) + 2 * h + k;
                    v[j].x = dropout_add(base[j].x, v[j].x, f.field(2 * k), drop.below, drop.scale);
                    v[j].y = dropout_add(base[j].y, v[j].y, f.field(2 * k + 1), drop.below, drop.scale);
                }
            }
        }
    }
}

}  // namespace sb
