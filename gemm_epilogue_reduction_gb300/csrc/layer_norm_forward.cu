// layer_norm_forward.cu -- the forward kernel of the layer norm (formulas and design in layer_norm.cu).
#include "layer_norm.cuh"

namespace sb {
namespace {

// BRANCH: h' = h + dropout(y).  The groups of all blocks take rows in turn; in kShifted all rows of a
// group have the same shift (the host sees to that), so that a thread's columns stay the same.
template <typename T, int MODE, bool BRANCH, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) forward_kernel(const LayerNormParams p) {
    constexpr int NV = kNormVectors;
    using B = __nv_bfloat16;
    using ST = Slots<T>;
    using SB = Slots<B>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[2][MAXT / 32 + 4 * kMaxGroups];
    const int rt = p.row_threads, d = p.d;
    const int group = threadIdx.x / rt, t = threadIdx.x - group * rt;
    float *red1 = red[0] + group * sum_words(rt / 32), *red2 = red[1] + group * sum_words(rt / 32);
    const uint32_t pitch = rt * 16, kY = ST::kThread * rt, kRow = kY + (BRANCH ? SB::kThread * rt : 0);
    const uint32_t kRing = p.steps * kRow, kBias = 32 * NV * rt, kWeights = 2 * kBias;
    // weight and bias in fp32 (one copy, or one for each group's shift), then the groups' rings;
    // addresses of this thread's pieces
    const uint32_t copies = !p.shared_weights ? 0 : MODE == kShifted ? p.groups : 1;
    const uint32_t weights = smem_u32(smem) + (MODE == kShifted ? group * kWeights : 0) + t * 16;
    const uint32_t ring = smem_u32(smem) + copies * kWeights + group * kRing + t * 16;
    const int first = blockIdx.x * p.groups + group, stride = gridDim.x * p.groups;
    const long long base = static_cast<long long>(first) * d, advance = static_cast<long long>(stride) * d;
    const int shift = MODE == kShifted ? static_cast<int>(base & 7) : 0;
    const int e0 = t * 8 - shift, per = rt * 8;  // this thread's first vector, and from one to the next
    const bool last_has = MODE != kAligned && (static_cast<long long>(p.M) * d & 7) != 0;

    // the row whose copy comes next, and where this thread's first vector of it is
    long long next = first;
    const T *h_next = static_cast<const T *>(p.h) + base + e0;
    const B *y_next = static_cast<const B *>(p.y) + base + e0;
    auto copy = [&](uint32_t at) {
        if constexpr (MODE != kSingle) {
            if (next < p.M) {
                // the array's last row may end inside a vector
                const bool inner = !last_has || next + 1 < p.M;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int e = e0 + i * per;
                    const bool whole = inner || e + 8 <= d;
                    ST::template copy<MODE>(at, pitch, i, h_next + i * per, e, d, whole);
                    if (BRANCH) SB::template copy<MODE>(at + kY, pitch, i, y_next + i * per, e, d, whole);
                }
            }
            next += stride;
            h_next += advance;
            if (BRANCH) y_next += advance;
            ring_commit();  // also without a row, so that the count of groups stays in step
        }
    };
    if (t < sum_words(rt / 32)) red1[t] = red2[t] = 0.f;
    if constexpr (MODE != kSingle)
        for (int s = 0; s < p.steps; ++s)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                ST::clear(ring + s * kRow, pitch, i, e0 + i * per, d);
                if (BRANCH) SB::clear(ring + s * kRow + kY, pitch, i, e0 + i * per, d);
            }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int s = 0; s + 1 < p.steps; ++s) copy(ring + s * kRow);
    auto read_bias = [&](int e, float2 (&v)[4]) {
        if (p.bias) {
            load_weight8<MODE>(p.bias, p, e, v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = both(0.f);
        }
    };
    if (p.shared_weights && (MODE == kShifted || group == 0)) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float2 v[4];
            load_weight8<MODE>(p.weight, p, e0 + i * per, v);
            Slots<float>::put(weights, pitch, i, v);
            read_bias(e0 + i * per, v);
            Slots<float>::put(weights + kBias, pitch, i, v);
        }
    }
    __syncthreads();
    // the draws' state goes from row to row by an addition: stride·d is a multiple of four (or there
    // is no second row)
    unsigned long long seed = 0, state = 0, state_row = 0, state_vector = 0;
    if (BRANCH) {
        seed = dropout_seed(p.drop);
        state = splitmix_state(seed, static_cast<unsigned long long>(base + e0) / 4);
        state_row = static_cast<unsigned long long>(advance / 4) * kGolden;
        state_vector = static_cast<unsigned long long>(rt * 2) * kGolden;
    }
    T *h_out = static_cast<T *>(p.h_out) + base + e0;
    B *x_out = static_cast<B *>(p.x) + base + e0;
    uint32_t slot = 0, ahead = (p.steps - 1) * kRow;  // of the ring, in bytes
    long long at_row = base;  // (kSingle)
    for (long long row = first; row < p.M; row += stride) {
        if constexpr (MODE != kSingle) {
            copy(ring + ahead);
            ahead = ahead + kRow == kRing ? 0 : ahead + kRow;
            ring_wait(p.steps - 1);
        }
        const uint32_t at = ring + slot;
        float2 a[NV][4];
        float2 acc = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = e0 + i * per;
            if constexpr (MODE == kSingle)
                load_singles(static_cast<const T *>(p.h) + at_row, e, d, a[i]);
            else
                ST::get(at, pitch, i, a[i]);
            mask8<MODE>(e, d, a[i]);
            if constexpr (BRANCH) {
                float2 v[4];
                if constexpr (MODE == kSingle)
                    load_singles(static_cast<const B *>(p.y) + at_row, e, d, v);
                else
                    SB::get(at + kY, pitch, i, v);
                mask8<MODE>(e, d, v);
                add_dropped<MODE>(p.drop, seed, state + i * state_vector,
                                  static_cast<unsigned long long>(at_row + e), a[i], v);
#pragma unroll
                for (int j = 0; j < 4; ++j) a[i][j] = v[j];
                store8<MODE>(h_out + i * per, e, d, a[i]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) acc = __fadd2_rn(acc, a[i][j]);
        }
        const float mean = row_sum<MAXT>(acc.x + acc.y, group, rt, red1) * p.inv_d;
        acc = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            centre8<MODE>(mean, e0 + i * per, d, a[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc = __ffma2_rn(a[i][j], a[i][j], acc);
        }
        const float r = rsqrtf(row_sum<MAXT>(acc.x + acc.y, group, rt, red2) * p.inv_d + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float2 w[4], b[4];
            if (p.shared_weights) {
                Slots<float>::get(weights, pitch, i, w);
                Slots<float>::get(weights + kBias, pitch, i, b);
            } else {
                load_weight8<MODE>(p.weight, p, e0 + i * per, w);
                read_bias(e0 + i * per, b);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) a[i][j] = __ffma2_rn(__fmul2_rn(a[i][j], both(r)), w[j], b[j]);
            store8<MODE>(x_out + i * per, e0 + i * per, d, a[i]);
        }
        if (BRANCH) h_out += advance, state += state_row;
        x_out += advance;
        if (MODE == kSingle) at_row += advance;
        slot = slot + kRow == kRing ? 0 : slot + kRow;
    }
}

}  // namespace

cudaError_t launch_layer_norm_forward(const LayerNormParams &p, LayerNormShape s, unsigned blocks,
                                      size_t smem, cudaStream_t st) {
    return for_layer_norm(s, p.y != nullptr, [&]<typename T, int MODE, bool BRANCH>() {
        static std::atomic<uint64_t> small{0}, large{0};
        if (s.threads <= kForwardThreads)
            return launch_norm_kernel(forward_kernel<T, MODE, BRANCH, kForwardThreads>, small, p,
                                      static_cast<int>(blocks), smem, st);
        return launch_norm_kernel(forward_kernel<T, MODE, BRANCH, 1024>, large, p,
                                  static_cast<int>(blocks), smem, st);
    });
}

}  // namespace sb
