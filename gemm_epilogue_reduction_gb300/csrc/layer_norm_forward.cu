// layer_norm_forward.cu -- the forward kernel of the layer norm (formulas and design in layer_norm.cu).
#include "layer_norm.cuh"

namespace sb {
namespace {

// BRANCH: h' = h + dropout(y).  The groups of all blocks take rows in turn.
template <typename T, int VEC, int EPT, int MAXT, bool BRANCH>
__global__ void __launch_bounds__(MAXT, 1) forward_kernel(const LayerNormParams p) {
    constexpr int P = EPT / 2;
    using B = __nv_bfloat16;
    using RH = RingArray<VEC, EPT, T>;
    using RB = RingArray<VEC, EPT, B>;
    constexpr int kRow = RH::kPerThread + (BRANCH ? RB::kPerThread : 0);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[2][MAXT / 32 + 4 * kMaxGroups];
    const int rt = p.row_threads, d = p.d;
    const int group = threadIdx.x / rt, t = threadIdx.x - group * rt;
    float *red1 = red[0] + group * sum_words(rt / 32), *red2 = red[1] + group * sum_words(rt / 32);
    uint8_t *ring = smem + group * p.depth * kRow * rt;
    const int first = blockIdx.x * p.groups + group, stride = gridDim.x * p.groups;
    const T *h = static_cast<const T *>(p.h);
    const B *y = static_cast<const B *>(p.y);

    auto copy = [&](int slot, long long row) {
        if constexpr (VEC > 1) {
            if (row < p.M) {
                uint8_t *at = ring + slot * kRow * rt;
                const size_t o = static_cast<size_t>(row) * d;
                RH::copy(at, h + o, rt, t, d);
                if (BRANCH) RB::copy(at + RH::kPerThread * rt, y + o, rt, t, d);
            }
            ring_commit();  // also without a row, so that the count of groups stays in step
        }
    };
    if (t < sum_words(rt / 32)) red1[t] = red2[t] = 0.f;
    if constexpr (VEC > 1)
        for (int s = 0; s < p.depth; ++s) {
            uint8_t *at = ring + s * kRow * rt;
            RH::clear(at, rt, t, d);
            if (BRANCH) RB::clear(at + RH::kPerThread * rt, rt, t, d);
        }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int s = 0; s + 1 < p.depth; ++s) copy(s, first + static_cast<long long>(s) * stride);
    const unsigned long long seed = BRANCH ? dropout_seed(p.drop) : 0ull;
    float2 w[P], b[P];
    get_weight<VEC, EPT>(p.weight, p.w32, rt, t, d, w);
    if (p.bias) {
        get_weight<VEC, EPT>(p.bias, p.w32, rt, t, d, b);
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) b[i] = both(0.f);
    }
    int slot = 0;
    for (long long row = first; row < p.M; row += stride) {
        const size_t base = static_cast<size_t>(row) * d;
        float2 a[P];
        if (VEC > 1 && p.depth) {
            int ahead = slot + p.depth - 1;
            if (ahead >= p.depth) ahead -= p.depth;
            copy(ahead, row + static_cast<long long>(p.depth - 1) * stride);
            ring_wait(p.depth - 1);
            if constexpr (VEC > 1) RH::get(ring + slot * kRow * rt, rt, t, a);
        } else {
            get<VEC, EPT>(h + base, rt, t, d, a);
        }
        if constexpr (BRANCH) {
            float2 v[P];
            if (VEC > 1 && p.depth) {
                if constexpr (VEC > 1) RB::get(ring + (slot * kRow + RH::kPerThread) * rt, rt, t, v);
            } else {
                get<VEC, EPT>(y + base, rt, t, d, v);
            }
            add_dropped<VEC, EPT>(p.drop, seed, base, rt, t, d, a, v);
#pragma unroll
            for (int i = 0; i < P; ++i) a[i] = v[i];
            put<VEC, EPT>(static_cast<T *>(p.h_out) + base, rt, t, d, a);
        }
        float2 acc = both(0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) acc = __fadd2_rn(acc, a[i]);
        const float mean = row_sum<MAXT>(acc.x + acc.y, group, rt, red1) * p.inv_d;
        centre<VEC, EPT>(mean, rt, t, d, a);
        acc = both(0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) acc = __ffma2_rn(a[i], a[i], acc);
        const float r = rsqrtf(row_sum<MAXT>(acc.x + acc.y, group, rt, red2) * p.inv_d + p.eps);
#pragma unroll
        for (int i = 0; i < P; ++i) a[i] = __ffma2_rn(__fmul2_rn(a[i], both(r)), w[i], b[i]);
        put<VEC, EPT>(static_cast<B *>(p.x) + base, rt, t, d, a);
        if (++slot >= p.depth) slot = 0;
    }
}

}  // namespace

cudaError_t launch_layer_norm_forward(const LayerNormParams &p, NormShape s, bool h32, int blocks,
                                      size_t smem, cudaStream_t st) {
    return for_norm_shape(s, h32, p.y != nullptr,
                          [&]<typename T, int VEC, int EPT, int MAXT, bool BRANCH>() {
                              static std::atomic<uint64_t> opted_in{0};
                              return launch_norm_kernel(forward_kernel<T, VEC, EPT, MAXT, BRANCH>,
                                                        opted_in, p, blocks, smem, st);
                          });
}

}  // namespace sb
