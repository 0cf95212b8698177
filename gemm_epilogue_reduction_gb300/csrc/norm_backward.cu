// norm_backward.cu -- the backward kernel of the residual norm (formulas and design in norm.cu).
#include "norm_common.cuh"

namespace sb {
namespace {

// ROWS: a gate for each row.  The groups of all blocks take rows in turn.
template <typename T, int VEC, int EPT, int MAXT, bool ROWS>
__global__ void __launch_bounds__(MAXT, 1) backward_kernel(const NormParams p) {
    constexpr int P = EPT / 2;
    using B = __nv_bfloat16;
    using RH = RingArray<VEC, EPT, T>;
    using RB = RingArray<VEC, EPT, B>;
    // a row of the ring: h, dh, dx, y and the row's gate
    constexpr int kDh = RH::kPerThread, kDx = 2 * RH::kPerThread, kY = kDx + RB::kPerThread,
                  kG = kY + RB::kPerThread, kRow = kG + (ROWS ? RB::kPerThread : 0);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][MAXT / 32 * 8];
    const int rt = p.row_threads, d = p.d;
    const int group = threadIdx.x / rt, t = threadIdx.x - group * rt;
    uint8_t *ring = smem + group * p.depth * kRow * rt;
    const int first = blockIdx.x * p.groups + group, stride = gridDim.x * p.groups;
    const T *h = static_cast<const T *>(p.h), *dh = static_cast<const T *>(p.dh);
    const B *y = static_cast<const B *>(p.y), *dx = static_cast<const B *>(p.dx),
            *gr = static_cast<const B *>(p.gate_rows);

    auto copy = [&](int slot, long long row) {
        if constexpr (VEC > 1) {
            if (row < p.M) {
                uint8_t *at = ring + slot * kRow * rt;
                const size_t o = static_cast<size_t>(row) * d;
                RH::copy(at, h + o, rt, t, d);
                if (dh) RH::copy(at + kDh * rt, dh + o, rt, t, d);
                RB::copy(at + kDx * rt, dx + o, rt, t, d);
                RB::copy(at + kY * rt, y + o, rt, t, d);
                if (ROWS) RB::copy(at + kG * rt, gr + o, rt, t, d);
            }
            ring_commit();  // also without a row, so that the count of groups stays in step
        }
    };
    if constexpr (VEC > 1)
        for (int s = 0; s < p.depth; ++s) {
            uint8_t *at = ring + s * kRow * rt;
            RH::clear(at, rt, t, d);
            RH::clear(at + kDh * rt, rt, t, d);
            RB::clear(at + kDx * rt, rt, t, d);
            RB::clear(at + kY * rt, rt, t, d);
            if (ROWS) RB::clear(at + kG * rt, rt, t, d);
        }
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
    float2 s_pre[P], s_y[P];
#pragma unroll
    for (int i = 0; i < P; ++i) s_pre[i] = s_y[i] = both(0.f);
    const float2 scale = both(p.scale);
    int slot = 0, turn = 0;
    for (long long row = first; row < p.M; row += stride, turn ^= 1) {
        const size_t base = static_cast<size_t>(row) * d;
        float2 vh[P], vdh[P], vdx[P], vy[P], vg[ROWS ? P : 1];
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
                RB::get(at + kY * rt, rt, t, vy);
                if constexpr (ROWS) RB::get(at + kG * rt, rt, t, vg);
            }
        } else {
            get<VEC, EPT>(h + base, rt, t, d, vh);
            if (dh) get<VEC, EPT>(dh + base, rt, t, d, vdh);
            get<VEC, EPT>(dx + base, rt, t, d, vdx);
            get<VEC, EPT>(y + base, rt, t, d, vy);
            if constexpr (ROWS) get<VEC, EPT>(gr + base, rt, t, d, vg);
        }
        // sums of h², a·h, y², b·dh, b·a, b·h
        float2 acc[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) acc[k] = both(0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 a = __fmul2_rn(vdx[i], pre[i]);
            float2 b = __fmul2_rn(vy[i], post[i]);
            if constexpr (ROWS) b = __fmul2_rn(b, vg[i]);
            acc[0] = __ffma2_rn(vh[i], vh[i], acc[0]);
            acc[1] = __ffma2_rn(a, vh[i], acc[1]);
            acc[2] = __ffma2_rn(vy[i], vy[i], acc[2]);
            acc[3] = __ffma2_rn(b, vdh[i], acc[3]);
            acc[4] = __ffma2_rn(b, a, acc[4]);
            acc[5] = __ffma2_rn(b, vh[i], acc[5]);
        }
        float sum[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) sum[k] = acc[k].x + acc[k].y;
        row_sum<MAXT>(sum, group, rt, red[turn] + group * (rt / 32) * 8);
        const float rh = rsqrtf(sum[0] * p.inv_d + p.eps);
        const float c = rh * rh * rh * (sum[1] * p.inv_d);
        float ry = 1.f, c2 = 0.f;
        if (p.post) {
            ry = rsqrtf(sum[2] * p.inv_d + p.eps);
            c2 = ry * ry * ry * ((sum[3] + rh * sum[4] - c * sum[5]) * p.inv_d);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 xr = __fmul2_rn(vdx[i], both(rh));
            s_pre[i] = __ffma2_rn(xr, vh[i], s_pre[i]);
            vdh[i] = __ffma2_rn(both(-c), vh[i], __ffma2_rn(xr, pre[i], vdh[i]));  // t
            vh[i] = __fmul2_rn(scale, vdh[i]);
            float2 tr = __fmul2_rn(vdh[i], both(ry));
            if constexpr (ROWS) {
                vdx[i] = __fmul2_rn(__fmul2_rn(tr, vy[i]), post[i]);  // the gate's gradient
                tr = __fmul2_rn(tr, vg[i]);
            }
            s_y[i] = __ffma2_rn(tr, vy[i], s_y[i]);
            vy[i] = __ffma2_rn(tr, post[i], __fmul2_rn(both(-c2), vy[i]));
        }
        put<VEC, EPT>(static_cast<T *>(p.dh_out) + base, rt, t, d, vh);
        if (ROWS) put<VEC, EPT>(static_cast<B *>(p.dgate_rows) + base, rt, t, d, vdx);
        put<VEC, EPT>(static_cast<B *>(p.dy) + base, rt, t, d, vy);
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
            for (int i = 0; i < P; ++i) v[i] = k == 0 ? s_pre[i] : s_y[i];
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

cudaError_t launch_norm_backward(const NormParams &p, NormShape s, bool h32, int blocks, size_t smem,
                                 cudaStream_t st) {
    return for_norm_shape(s, h32, p.gate_rows != nullptr,
                          [&]<typename T, int VEC, int EPT, int MAXT, bool ROWS>() {
                              static std::atomic<uint64_t> opted_in{0};
                              return launch_norm_kernel(backward_kernel<T, VEC, EPT, MAXT, ROWS>,
                                                        opted_in, p, blocks, smem, st);
                          });
}

}  // namespace sb
