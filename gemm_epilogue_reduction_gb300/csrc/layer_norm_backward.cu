// layer_norm_backward.cu -- the backward kernel of the layer norm (formulas and design in layer_norm.cu).
#include "layer_norm.cuh"

namespace sb {
namespace {

// BRANCH: the gradient of the branch in front of its dropout is written too.
template <typename T, int VEC, int EPT, int MAXT, bool BRANCH>
__global__ void __launch_bounds__(MAXT, 1) backward_kernel(const LayerNormParams p) {
    constexpr int P = EPT / 2;
    using B = __nv_bfloat16;
    using RH = RingArray<VEC, EPT, T>;
    using RB = RingArray<VEC, EPT, B>;
    // a row of the ring: h, dh, dx
    constexpr int kDh = RH::kPerThread, kDx = 2 * RH::kPerThread, kRow = kDx + RB::kPerThread;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red1_all[MAXT / 32 + 4 * kMaxGroups];
    __shared__ float red2_all[MAXT / 32 * 8];
    const int rt = p.row_threads, d = p.d;
    const int group = threadIdx.x / rt, t = threadIdx.x - group * rt;
    float *red1 = red1_all + group * sum_words(rt / 32), *red2 = red2_all + group * (rt / 32) * 8;
    uint8_t *ring = smem + group * p.depth * kRow * rt;
    const int first = blockIdx.x * p.groups + group, stride = gridDim.x * p.groups;
    const T *h = static_cast<const T *>(p.h), *dh = static_cast<const T *>(p.dh);
    const B *dx = static_cast<const B *>(p.dx);

    auto copy = [&](int slot, long long row) {
        if constexpr (VEC > 1) {
            if (row < p.M) {
                uint8_t *at = ring + slot * kRow * rt;
                const size_t o = static_cast<size_t>(row) * d;
                RH::copy(at, h + o, rt, t, d);
                if (dh) RH::copy(at + kDh * rt, dh + o, rt, t, d);
                RB::copy(at + kDx * rt, dx + o, rt, t, d);
            }
            ring_commit();  // also without a row, so that the count of groups stays in step
        }
    };
    if (t < sum_words(rt / 32)) red1[t] = 0.f;
    if constexpr (VEC > 1)
        for (int s = 0; s < p.depth; ++s) {
            uint8_t *at = ring + s * kRow * rt;
            RH::clear(at, rt, t, d);
            RH::clear(at + kDh * rt, rt, t, d);
            RB::clear(at + kDx * rt, rt, t, d);
        }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int s = 0; s + 1 < p.depth; ++s) copy(s, first + static_cast<long long>(s) * stride);
    const unsigned long long seed = BRANCH ? dropout_seed(p.drop) : 0ull;
    float2 w[P], s_w[P], s_b[P], zero[P];
    get_weight<VEC, EPT>(p.weight, p.w32, rt, t, d, w);
#pragma unroll
    for (int i = 0; i < P; ++i) s_w[i] = s_b[i] = zero[i] = both(0.f);
    int slot = 0;
    for (long long row = first; row < p.M; row += stride) {
        const size_t base = static_cast<size_t>(row) * d;
        float2 vh[P], vdh[P], vdx[P];
#pragma unroll
        for (int i = 0; i < P; ++i) vdh[i] = both(0.f);
        if (VEC > 1 && p.depth) {
            int ahead = slot + p.depth - 1;
            if (ahead >= p.depth) ahead -= p.depth;
            copy(ahead, row + static_cast<long long>(p.depth - 1) * stride);
            ring_wait(p.depth - 1);
            const uint8_t *at = ring + slot * kRow * rt;
            if constexpr (VEC > 1) {
                RH::get(at, rt, t, vh);
                if (dh) RH::get(at + kDh * rt, rt, t, vdh);
                RB::get(at + kDx * rt, rt, t, vdx);
            }
        } else {
            get<VEC, EPT>(h + base, rt, t, d, vh);
            if (dh) get<VEC, EPT>(dh + base, rt, t, d, vdh);
            get<VEC, EPT>(dx + base, rt, t, d, vdx);
        }
        float2 acc = both(0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) acc = __fadd2_rn(acc, vh[i]);
        const float mean = row_sum<MAXT>(acc.x + acc.y, group, rt, red1) * p.inv_d;
        centre<VEC, EPT>(mean, rt, t, d, vh);
        // sums of c², a and a·c with c = h - mean
        float2 s0 = both(0.f), s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 a = __fmul2_rn(vdx[i], w[i]);
            s0 = __ffma2_rn(vh[i], vh[i], s0);
            s1 = __fadd2_rn(s1, a);
            s2 = __ffma2_rn(a, vh[i], s2);
        }
        float sum[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
        row_sum<MAXT>(sum, group, rt, red2);
        const float r = rsqrtf(sum[0] * p.inv_d + p.eps);
        const float ma = -r * (sum[1] * p.inv_d), c2 = -r * r * r * (sum[2] * p.inv_d);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 xr = __fmul2_rn(vdx[i], both(r));
            s_w[i] = __ffma2_rn(xr, vh[i], s_w[i]);
            s_b[i] = __fadd2_rn(s_b[i], vdx[i]);
            vdh[i] = __ffma2_rn(both(c2), vh[i], __ffma2_rn(xr, w[i], __fadd2_rn(vdh[i], both(ma))));
        }
        put<VEC, EPT>(static_cast<T *>(p.dh_out) + base, rt, t, d, vdh);
        if constexpr (BRANCH) {
            add_dropped<VEC, EPT>(p.drop, seed, base, rt, t, d, zero, vdh);
            put<VEC, EPT>(static_cast<B *>(p.dy) + base, rt, t, d, vdh);
        }
        if (++slot >= p.depth) slot = 0;
    }
    // the groups' column sums in ascending order, through shared memory (the ring's rows have
    // all been read), then this block's partial vectors
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    float *all = reinterpret_cast<float *>(smem);
    float *part = p.part + static_cast<size_t>(blockIdx.x) * p.sums * d;
    for (int g = 0; g < p.groups; ++g) {
        if (p.groups > 1) __syncthreads();
        if (group != g) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k >= p.sums) break;
            float2 v[P];
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = k == 0 ? s_w[i] : s_b[i];
            if (g > 0) {
                float2 x[P];
                get<VEC, EPT>(all + k * d, rt, t, d, x);
#pragma unroll
                for (int i = 0; i < P; ++i) v[i] = __fadd2_rn(v[i], x[i]);
            }
            put<VEC, EPT>((g + 1 < p.groups ? all : part) + k * d, rt, t, d, v);
        }
    }
}

}  // namespace

cudaError_t launch_layer_norm_backward(const LayerNormParams &p, NormShape s, bool h32, int blocks,
                                       size_t smem, cudaStream_t st) {
    return for_norm_shape(s, h32, p.dy != nullptr,
                          [&]<typename T, int VEC, int EPT, int MAXT, bool BRANCH>() {
                              static std::atomic<uint64_t> opted_in{0};
                              return launch_norm_kernel(backward_kernel<T, VEC, EPT, MAXT, BRANCH>,
                                                        opted_in, p, blocks, smem, st);
                          });
}

}  // namespace sb
