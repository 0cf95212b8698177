// layer_norm_forward.cu -- the forward kernel of the layer norm (formulas and design in layer_norm.cu).
#include "layer_norm.cuh"

namespace sb {
namespace {

// BRANCH: h' = h + dropout(y).  The groups of all blocks take ROWS rows in turn; in kShifted all rows of
// a group have the same shift (the host sees to that), so that a thread's columns stay the same.  KEPT:
// weight and bias stay in registers; else in shared memory, or are read again for each row.
template <typename T, int MODE, bool BRANCH, int MAXT, int ROWS, bool KEPT>
__global__ void __launch_bounds__(MAXT, 1) forward_kernel(const LayerNormParams p) {
    static_assert(MODE != kSingle || ROWS == 1, "a row behind the last is in the ring only");
    constexpr int NV = kNormVectors;
    using B = __nv_bfloat16;
    using ST = Slots<T>;
    using SB = Slots<B>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[2][MAXT / 32 * 8];
    const int rt = p.row_threads, d = p.d;
    const int group = threadIdx.x / rt, t = threadIdx.x - group * rt;
    float *red1 = red[0] + group * (rt / 32) * 8, *red2 = red[1] + group * (rt / 32) * 8;
    const uint32_t pitch = rt * 16, kY = ST::kThread * rt, kRow = kY + (BRANCH ? SB::kThread * rt : 0);
    const uint32_t kStep = ROWS * kRow, kRing = p.steps * kStep, kBias = 32 * NV * rt, kWeights = 2 * kBias;
    // weight and bias in fp32 (the block is one group then), then the groups' rings; addresses of this
    // thread's pieces
    const uint32_t weights = smem_u32(smem) + t * 16;
    const uint32_t ring = weights + (p.shared_weights ? kWeights : 0) + group * kRing;
    const int first = blockIdx.x * p.groups + group, stride = gridDim.x * p.groups;
    const long long base = static_cast<long long>(first) * d, advance = static_cast<long long>(stride) * d;
    const int shift = MODE == kShifted ? static_cast<int>(base & 7) : 0;
    const int e0 = t * 8 - shift, per = rt * 8;  // this thread's first vector, and from one to the next
    uint32_t in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) in[i] = inside8<MODE>(e0 + i * per, d);
    const bool last_has = MODE != kAligned && (static_cast<long long>(p.M) * d & 7) != 0;

    // the row whose copy comes next, and where this thread's first vector of it is
    long long next = first;
    const T *h_next = static_cast<const T *>(p.h) + base + e0;
    const B *y_next = static_cast<const B *>(p.y) + base + e0;
    auto copy = [&](uint32_t at) {
        if constexpr (MODE != kSingle) {
#pragma unroll
            for (int k = 0; k < ROWS; ++k, next += stride, h_next += advance, y_next += advance, at += kRow)
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
            ring_commit();  // also without a row, so that the count of groups stays in step
        }
    };
    // the sums of a row each over the group
    auto sums = [&](float (&v)[ROWS], float *words) {
        if constexpr (ROWS == 1)
            v[0] = row_sum<MAXT>(v[0], group, rt, words);
        else
            row_sum<MAXT>(v, group, rt, words);
    };
    if (ROWS == 1 && t < sum_words(rt / 32)) red1[t] = red2[t] = 0.f;
    if constexpr (MODE != kSingle)
        for (int s = 0; s < p.steps * ROWS; ++s)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                ST::clear(ring + s * kRow, pitch, i, e0 + i * per, d);
                if (BRANCH) SB::clear(ring + s * kRow + kY, pitch, i, e0 + i * per, d);
            }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int s = 0; s + 1 < p.steps; ++s) copy(ring + s * kStep);
    auto read_bias = [&](int e, float2 (&v)[4]) {
        if (p.bias) {
            load_weight8<MODE>(p.bias, p, e, v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = both(0.f);
        }
    };
    float2 w_kept[KEPT ? NV : 1][4], b_kept[KEPT ? NV : 1][4];
    if constexpr (KEPT) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            load_weight8<MODE>(p.weight, p, e0 + i * per, w_kept[i]);
            read_bias(e0 + i * per, b_kept[i]);
        }
    } else if (p.shared_weights) {
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
    uint32_t slot = 0, ahead = (p.steps - 1) * kStep;  // of the ring, in bytes
    long long at_row = base;                           // (kSingle)
    for (long long row0 = first; row0 < p.M; row0 += ROWS * stride) {
        if constexpr (MODE != kSingle) {
            copy(ring + ahead);
            ahead = ahead + kStep == kRing ? 0 : ahead + kStep;
            ring_wait(p.steps - 1);
        }
        const uint32_t at = ring + slot;
        float2 a[ROWS][NV][4];
        float sum[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            float2 acc = both(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = e0 + i * per;
                if constexpr (MODE == kSingle)
                    load_singles(static_cast<const T *>(p.h) + at_row, e, d, a[k][i]);
                else
                    ST::get(at + k * kRow, pitch, i, a[k][i]);  // (a row behind the last: an old one)
                mask8<MODE>(in[i], a[k][i]);
                if constexpr (BRANCH) {
                    float2 v[4];
                    if constexpr (MODE == kSingle)
                        load_singles(static_cast<const B *>(p.y) + at_row, e, d, v);
                    else
                        SB::get(at + k * kRow + kY, pitch, i, v);
                    mask8<MODE>(in[i], v);
                    add_dropped<MODE>(p.drop, seed, state + i * state_vector,
                                      static_cast<unsigned long long>(at_row + e), a[k][i], v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[k][i][j] = v[j];
                    if (k == 0 || row0 + k * stride < p.M) store8<MODE>(h_out + i * per, in[i], a[k][i]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) acc = __fadd2_rn(acc, a[k][i][j]);
            }
            sum[k] = acc.x + acc.y;
            if (BRANCH) h_out += advance, state += state_row;
        }
        sums(sum, red1);
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const float mean = sum[k] * p.inv_d;
            float2 acc = both(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                centre8<MODE>(mean, in[i], a[k][i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc = __ffma2_rn(a[k][i][j], a[k][i][j], acc);
            }
            sum[k] = acc.x + acc.y;
        }
        sums(sum, red2);
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const float r = rsqrtf(sum[k] * p.inv_d + p.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 w[4], b[4];
                if constexpr (KEPT) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = w_kept[i][j], b[j] = b_kept[i][j];
                } else if (p.shared_weights) {
                    Slots<float>::get(weights, pitch, i, w);
                    Slots<float>::get(weights + kBias, pitch, i, b);
                } else {
                    load_weight8<MODE>(p.weight, p, e0 + i * per, w);
                    read_bias(e0 + i * per, b);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    a[k][i][j] = __ffma2_rn(__fmul2_rn(a[k][i][j], both(r)), w[j], b[j]);
                if (k == 0 || row0 + k * stride < p.M) store8<MODE>(x_out + i * per, in[i], a[k][i]);
            }
            x_out += advance;
        }
        if (MODE == kSingle) at_row += advance;
        slot = slot + kStep == kRing ? 0 : slot + kStep;
    }
}

}  // namespace

cudaError_t launch_layer_norm_forward(const LayerNormParams &p, LayerNormShape s, unsigned blocks,
                                      size_t smem, cudaStream_t st) {
    return for_layer_norm(s, p.y != nullptr, [&]<typename T, int MODE, bool BRANCH>() {
        static std::atomic<uint64_t> two{0}, small{0}, wide_two{0}, wide{0}, large{0};
        const int n = static_cast<int>(blocks);
        if (s.threads <= kNormThreads) {
            if constexpr (MODE != kSingle)
                if (s.rows == 2)
                    return launch_norm_kernel(forward_kernel<T, MODE, BRANCH, kNormThreads, 2, true>, two, p,
                                              n, smem, st);
            return launch_norm_kernel(forward_kernel<T, MODE, BRANCH, kNormThreads, 1, true>, small, p, n,
                                      smem, st);
        }
        if (s.threads <= kWideThreads) {
            if constexpr (MODE != kSingle)
                if (s.rows == 2)
                    return launch_norm_kernel(forward_kernel<T, MODE, BRANCH, kWideThreads, 2, true>,
                                              wide_two, p, n, smem, st);
            return launch_norm_kernel(forward_kernel<T, MODE, BRANCH, kWideThreads, 1, true>, wide, p, n,
                                      smem, st);
        }
        return launch_norm_kernel(forward_kernel<T, MODE, BRANCH, 1024, 1, false>, large, p, n, smem, st);
    });
}

}  // namespace sb
