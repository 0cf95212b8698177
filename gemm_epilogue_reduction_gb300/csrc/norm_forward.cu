// norm_forward.cu -- the forward kernel of the residual norm (formulas and design in norm.cu).
#include "norm_common.cuh"

namespace sb {
namespace {

// ROWS: a gate for each row.  The groups of all blocks take rows in turn.
template <typename T, int VEC, int EPT, int MAXT, bool ROWS>
__global__ void __launch_bounds__(MAXT, 1) forward_kernel(const NormParams p) {
    constexpr int P = EPT / 2;
    using B = __nv_bfloat16;
    using RH = RingArray<VEC, EPT, T>;
    using RB = RingArray<VEC, EPT, B>;
    constexpr int kRow = RH::kPerThread + RB::kPerThread * (ROWS ? 2 : 1);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[2][MAXT / 32 + 4 * kMaxGroups];
    const int rt = p.row_threads, d = p.d;
    const int group = threadIdx.x / rt, t = threadIdx.x - group * rt;
    float *red1 = red[0] + group * sum_words(rt / 32), *red2 = red[1] + group * sum_words(rt / 32);
    uint8_t *ring = smem + group * p.depth * kRow * rt;
    const int first = blockIdx.x * p.groups + group, stride = gridDim.x * p.groups;
    const T *h = static_cast<const T *>(p.h);
    const B *y = static_cast<const B *>(p.y), *gr = static_cast<const B *>(p.gate_rows);

    auto copy = [&](int slot, long long row) {
        if constexpr (VEC > 1) {
            if (row < p.M) {
                uint8_t *at = ring + slot * kRow * rt;
                const size_t o = static_cast<size_t>(row) * d;
                RH::copy(at, h + o, rt, t, d);
                RB::copy(at + RH::kPerThread * rt, y + o, rt, t, d);
                if (ROWS) RB::copy(at + (RH::kPerThread + RB::kPerThread) * rt, gr + o, rt, t, d);
            }
            ring_commit();  // also without a row, so that the count of groups stays in step
        }
    };
    if (t < sum_words(rt / 32)) red1[t] = red2[t] = 0.f;
    if constexpr (VEC > 1)
        for (int s = 0; s < p.depth; ++s) {
            uint8_t *at = ring + s * kRow * rt;
            RH::clear(at, rt, t, d);
            RB::clear(at + RH::kPerThread * rt, rt, t, d);
            if (ROWS) RB::clear(at + (RH::kPerThread + RB::kPerThread) * rt, rt, t, d);
        }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int s = 0; s + 1 < p.depth; ++s) copy(s, first + static_cast<long long>(s) * stride);
    float2 pre[P], post[P];  // post: times the gate where that is one vector
    get_weight<VEC, EPT>(p.pre, p.w32, rt, t, d, pre);
    get_weight<VEC, EPT>(p.post, p.w32, rt, t, d, post);
    if (!ROWS) {
        float2 g[P];
        get_weight<VEC, EPT>(p.gate, p.w32, rt, t, d, g);
#pragma unroll
        for (int i = 0; i < P; ++i) post[i] = __fmul2_rn(post[i], g[i]);
    }
    const float2 scale = both(p.scale);
    int slot = 0;
    for (long long row = first; row < p.M; row += stride) {
        const size_t base = static_cast<size_t>(row) * d;
        float2 a[P], b[P];
        if (VEC > 1 && p.depth) {
            int ahead = slot + p.depth - 1;
            if (ahead >= p.depth) ahead -= p.depth;
            copy(ahead, row + static_cast<long long>(p.depth - 1) * stride);
            ring_wait(p.depth - 1);
            const uint8_t *at = ring + slot * kRow * rt;
            if constexpr (VEC > 1) {
                RH::get(at, rt, t, a);
                RB::get(at + RH::kPerThread * rt, rt, t, b);
            }
        } else {
            get<VEC, EPT>(h + base, rt, t, d, a);
            get<VEC, EPT>(y + base, rt, t, d, b);
        }
        float2 acc = both(0.f);
        float ry = 1.f;
        if (p.post) {
#pragma unroll
            for (int i = 0; i < P; ++i) acc = __ffma2_rn(b[i], b[i], acc);
            ry = rsqrtf(row_sum<MAXT>(acc.x + acc.y, group, rt, red1) * p.inv_d + p.eps);
        }
        if (ROWS) {
            float2 g[P];
            if (VEC > 1 && p.depth) {
                if constexpr (VEC > 1)
                    RB::get(ring + (slot * kRow + RH::kPerThread + RB::kPerThread) * rt, rt, t, g);
            } else {
                get<VEC, EPT>(gr + base, rt, t, d, g);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) b[i] = __fmul2_rn(b[i], g[i]);
        }
        acc = both(0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            a[i] = __ffma2_rn(__fmul2_rn(b[i], post[i]), both(ry), __fmul2_rn(a[i], scale));
            acc = __ffma2_rn(a[i], a[i], acc);
        }
        put<VEC, EPT>(static_cast<T *>(p.h_out) + base, rt, t, d, a);
        const float rh = rsqrtf(row_sum<MAXT>(acc.x + acc.y, group, rt, red2) * p.inv_d + p.eps);
#pragma unroll
        for (int i = 0; i < P; ++i) a[i] = __fmul2_rn(__fmul2_rn(a[i], both(rh)), pre[i]);
        put<VEC, EPT>(static_cast<B *>(p.x) + base, rt, t, d, a);
        // without post there is one barrier per row, and red2 would be written again before
        // every thread has read it
        if (!p.post && rt > 32) group_sync(group, rt);
        if (++slot >= p.depth) slot = 0;
    }
}

}  // namespace

cudaError_t launch_norm_forward(const NormParams &p, NormShape s, bool h32, int blocks, size_t smem,
                                cudaStream_t st) {
    return for_norm_shape(s, h32, p.gate_rows != nullptr,
                          [&]<typename T, int VEC, int EPT, int MAXT, bool ROWS>() {
                              static std::atomic<uint64_t> opted_in{0};
                              return launch_norm_kernel(forward_kernel<T, VEC, EPT, MAXT, ROWS>,
                                                        opted_in, p, blocks, smem, st);
                          });
}

}  // namespace sb
