// layer_norm_backward.cu -- the backward kernel of the layer norm (formulas and design in layer_norm.cu).
#include "layer_norm.cuh"

namespace sb {
namespace {

// BRANCH: the gradient of the branch in front of its dropout is written too.  The groups of all
// blocks take ROWS rows in turn; in kShifted all rows of a group have the same shift (the host sees to
// that), so that a thread's columns stay the same.
template <typename T, int MODE, bool BRANCH, int MAXT, int ROWS>
__global__ void __launch_bounds__(MAXT, 1) backward_kernel(const LayerNormParams p) {
    static_assert(MODE != kSingle || ROWS == 1, "a row behind the last is in the ring only");
    constexpr int NV = kNormVectors;
    using B = __nv_bfloat16;
    using ST = Slots<T>;
    using SB = Slots<B>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red1_all[MAXT / 32 * 8], red2_all[MAXT / 32 * 8];
    const int rt = p.row_threads, d = p.d;
    const int group = threadIdx.x / rt, t = threadIdx.x - group * rt;
    float *red1 = red1_all + group * (rt / 32) * 8, *red2 = red2_all + group * (rt / 32) * 8;
    // a row of the ring: h, dh, dx
    const uint32_t pitch = rt * 16, kDh = ST::kThread * rt, kDx = 2 * kDh, kRow = kDx + SB::kThread * rt;
    const uint32_t kRing = p.steps * ROWS * kRow;
    const uint32_t ring = smem_u32(smem) + group * kRing + t * 16;  // this thread's pieces of it
    const int first = blockIdx.x * p.groups + group, stride = gridDim.x * p.groups;
    const long long base = static_cast<long long>(first) * d, advance = static_cast<long long>(stride) * d;
    const int shift = MODE == kShifted ? static_cast<int>(base & 7) : 0;
    const int e0 = t * 8 - shift, per = rt * 8;  // this thread's first vector, and from one to the next
    uint32_t in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) in[i] = inside8<MODE>(e0 + i * per, d);
    const bool last_has = MODE != kAligned && (static_cast<long long>(p.M) * d & 7) != 0;

    // the row whose copy comes next, and where this thread's first vector of it is
    long long next = first, from = base + e0;
    const T *h = static_cast<const T *>(p.h), *dh = static_cast<const T *>(p.dh);
    const B *dx = static_cast<const B *>(p.dx);
    auto copy = [&](uint32_t at) {
        if constexpr (MODE != kSingle) {
#pragma unroll
            for (int k = 0; k < ROWS; ++k, next += stride, from += advance, at += kRow)
                if (next < p.M) {
                    // the array's last row may end inside a vector
                    const bool inner = !last_has || next + 1 < p.M;
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int e = e0 + i * per;
                        const bool whole = inner || e + 8 <= d;
                        ST::template copy<MODE>(at, pitch, i, h + from + i * per, e, d, whole);
                        if (dh) ST::template copy<MODE>(at + kDh, pitch, i, dh + from + i * per, e, d, whole);
                        SB::template copy<MODE>(at + kDx, pitch, i, dx + from + i * per, e, d, whole);
                    }
                }
            ring_commit();  // also without a row, so that the count of groups stays in step
        }
    };
    long long at_row = base;  // of the row in hand
    auto get_dx = [&](uint32_t at, int i, float2 (&v)[4]) {
        if constexpr (MODE == kSingle)
            load_singles(dx + at_row, e0 + i * per, d, v);
        else
            SB::get(at + kDx, pitch, i, v);
        mask8<MODE>(in[i], v);
    };
    if constexpr (MODE != kSingle)
        for (int s = 0; s < p.steps * ROWS; ++s)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                ST::clear(ring + s * kRow, pitch, i, e0 + i * per, d);
                SB::clear(ring + s * kRow + kDx, pitch, i, e0 + i * per, d);
            }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int s = 0; s + 1 < p.steps; ++s) copy(ring + s * ROWS * kRow);
    float2 w[NV][4], s_w[NV][4], s_b[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_weight8<MODE>(p.weight, p, e0 + i * per, w[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) s_w[i][j] = s_b[i][j] = both(0.f);
    }
    // the draws' state goes from row to row by an addition: stride·d is a multiple of four (or there
    // is no second row)
    unsigned long long seed = 0, state = 0, state_row = 0, state_vector = 0;
    if (BRANCH) {
        seed = dropout_seed(p.drop);
        state = splitmix_state(seed, static_cast<unsigned long long>(base + e0) / 4);
        state_row = static_cast<unsigned long long>(advance / 4) * kGolden;
        state_vector = static_cast<unsigned long long>(rt * 2) * kGolden;
    }
    uint32_t slot = 0, ahead = (p.steps - 1) * ROWS * kRow;  // of the ring, in bytes
    for (long long row0 = first; row0 < p.M; row0 += ROWS * stride) {
        if constexpr (MODE != kSingle) {
            copy(ring + ahead);
            ahead = ahead + ROWS * kRow == kRing ? 0 : ahead + ROWS * kRow;
            ring_wait(p.steps - 1);
        }
        const uint32_t at = ring + slot;
        float2 c[ROWS][NV][4];
        float sum1[ROWS], sum2[3 * ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            float2 acc = both(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = e0 + i * per;
                if constexpr (MODE == kSingle)
                    load_singles(h + at_row, e, d, c[k][i]);
                else
                    ST::get(at + k * kRow, pitch, i, c[k][i]);  // (a row behind the last: an old one)
                mask8<MODE>(in[i], c[k][i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc = __fadd2_rn(acc, c[k][i][j]);
            }
            sum1[k] = acc.x + acc.y;
        }
        row_sum<MAXT>(sum1, group, rt, red1);
        // sums of c², a and a·c with c = h - mean
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const float mean = sum1[k] * p.inv_d;
            float2 s0 = both(0.f), s1 = both(0.f), s2 = both(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 x[4];
                get_dx(at + k * kRow, i, x);
                centre8<MODE>(mean, in[i], c[k][i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = __fmul2_rn(x[j], w[i][j]);
                    s0 = __ffma2_rn(c[k][i][j], c[k][i][j], s0);
                    s1 = __fadd2_rn(s1, a);
                    s2 = __ffma2_rn(a, c[k][i][j], s2);
                }
            }
            sum2[3 * k] = s0.x + s0.y, sum2[3 * k + 1] = s1.x + s1.y, sum2[3 * k + 2] = s2.x + s2.y;
        }
        row_sum<MAXT>(sum2, group, rt, red2);
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            if (k > 0 && row0 + k * stride >= p.M) break;
            const float r = rsqrtf(sum2[3 * k] * p.inv_d + p.eps);
            // t = dh + r·(a - mean(a) - r·(r·mean(a·c))·c): no r³, which leaves fp32's range for deviations
            // whose squares are far from doing so
            const float ma = -(sum2[3 * k + 1] * p.inv_d), mac = -r * (r * (sum2[3 * k + 2] * p.inv_d));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = e0 + i * per;
                float2 x[4], v[4];
                get_dx(at + k * kRow, i, x);
                if (!dh) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = both(0.f);
                } else if constexpr (MODE == kSingle) {
                    load_singles(dh + at_row, e, d, v);
                } else {
                    ST::get(at + k * kRow + kDh, pitch, i, v);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s_w[i][j] = __ffma2_rn(__fmul2_rn(x[j], both(r)), c[k][i][j], s_w[i][j]);
                    s_b[i][j] = __fadd2_rn(s_b[i][j], x[j]);
                    const float2 a = __ffma2_rn(x[j], w[i][j], both(ma));
                    v[j] = __ffma2_rn(both(r), __ffma2_rn(both(mac), c[k][i][j], a), v[j]);
                }
                store8<MODE>(static_cast<T *>(p.dh_out) + at_row + e, in[i], v);
                if constexpr (BRANCH) {
                    const float2 zero[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
                    add_dropped<MODE>(p.drop, seed, state + i * state_vector,
                                      static_cast<unsigned long long>(at_row + e), zero, v);
                    store8<MODE>(static_cast<B *>(p.dy) + at_row + e, in[i], v);
                }
            }
            at_row += advance;
            state += state_row;
        }
        slot = slot + ROWS * kRow == kRing ? 0 : slot + ROWS * kRow;
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
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = e0 + i * per;
                float2 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = k == 0 ? s_w[i][j] : s_b[i][j];
                if (g > 0) {
                    float2 x[4];
                    if (MODE == kAligned && e < d)
                        load_pairs<8>(all + k * d + e, x);
                    else
                        load_singles(all + k * d, e, d, x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = __fadd2_rn(v[j], x[j]);
                }
                float *to = (g + 1 < p.groups ? all : part) + k * d;
                if (MODE == kAligned && e < d)
                    store_pairs<8>(to + e, v);
                else
                    store_singles(to, e, d, v);
            }
        }
    }
}

}  // namespace

cudaError_t launch_layer_norm_backward(const LayerNormParams &p, LayerNormShape s, unsigned blocks,
                                       size_t smem, cudaStream_t st) {
    return for_layer_norm(s, p.dy != nullptr, [&]<typename T, int MODE, bool BRANCH>() {
        static std::atomic<uint64_t> pairs{0}, small{0}, wide{0}, medium{0}, large{0};
        const int n = static_cast<int>(blocks);
        if (s.threads <= kNormThreads) {
            if constexpr (MODE != kSingle)
                if (s.rows == 2)
                    return launch_norm_kernel(backward_kernel<T, MODE, BRANCH, kNormThreads, 2>, pairs, p,
                                              n, smem, st);
            return launch_norm_kernel(backward_kernel<T, MODE, BRANCH, kNormThreads, 1>, small, p, n,
                                      smem, st);
        }
        // (two rows at a time do not fit into 128 registers)
        if (s.threads <= kWideThreads)
            return launch_norm_kernel(backward_kernel<T, MODE, BRANCH, kWideThreads, 1>, wide, p, n, smem,
                                      st);
        if (s.threads <= 640)
            return launch_norm_kernel(backward_kernel<T, MODE, BRANCH, 640, 1>, medium, p, n, smem, st);
        return launch_norm_kernel(backward_kernel<T, MODE, BRANCH, 1024, 1>, large, p, n, smem, st);
    });
}

}  // namespace sb
