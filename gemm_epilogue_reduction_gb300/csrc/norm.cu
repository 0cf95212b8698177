// norm.cu -- the end of a transformer block in one pass: the norm after the block, its gate, the
// scaled residual sum and the norm before the next block (or the output head), with the
// gradients.  With n(x; w) = w·x / sqrt(mean(x²) + eps) over a row of d values:
//   forward    h' = scale·h + gate·n(y; post),   x = n(h'; pre)
//   backward   given h' and y and the gradients dx of x and dh of h':
//     rh = 1 / sqrt(mean(h'²) + eps),  t = dh + rh·(dx·pre - h'·rh²·mean(dx·pre·h'))
//     dpre = sum over rows of dx·h'·rh,   gradient of h = scale·t
//     u = n(y; post),  dgate = t·u (summed over the rows when the gate is one vector)
//     f = t·gate·post,  dpost = sum over rows of t·gate·y·ry,
//     dy = ry·(f - y·ry²·mean(f·y))
// (post and gate are optional: u = y without the one, factor 1 without the other).
//
// Both kernels are bound by memory: forward reads h and y and writes h' and x, backward reads
// dx, dh, h' and y and writes two gradients, each once.  A row belongs to one group of threads
// that keeps its values in registers between the row reductions; the second reduction needs the
// first one's result, so a row costs two barriers.  All sums are fp32; x comes from the
// unrounded h' (one rounding per output), backward differentiates at the h' that was stored.
// Backward's column sums: every block adds up its rows in registers and leaves one partial
// vector each, and columns_kernel adds the partials in ascending order, so equal calls give
// equal bits.
#include <cmath>
#include <cuda_bf16.h>

#include "sb.h"
#include "sb_internal.h"

namespace sb {
namespace {

constexpr int kMaxRowThreads = 1024;
constexpr int kMaxWarpsN = kMaxRowThreads / 32;
constexpr int kMaxNormD = 16384;

struct NormParams {
    int M, d;
    int row_threads;  // threads of a row's group, a multiple of 32
    int gate_kind;    // 0: none, 1: one vector, 2: one per row
    float scale, eps, inv_d;
    const void *h, *y, *pre, *post, *gate;
    void *h_out, *x;            // forward
    const void *dx, *dh;        // backward
    void *dh_out, *dy, *dgate;  // dgate: of a gate per row
    float *part;                // [blocks][sums][d]
    int sums;                   // vectors of column sums: dpre, dpost, dgate (those there are)
};

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }

// VEC consecutive values; the address is VEC * sizeof(T) aligned (up to 16 bytes).
template <int VEC, typename T>
__device__ __forceinline__ void load(const T *p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = to_f(*p);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 x = reinterpret_cast<const float4 *>(p)[i];
            v[4 * i] = x.x;
            v[4 * i + 1] = x.y;
            v[4 * i + 2] = x.z;
            v[4 * i + 3] = x.w;
        }
    } else {
        uint32_t w[VEC / 2];
        if constexpr (VEC == 8) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(p);
            w[0] = x.x, w[1] = x.y;
        }
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

template <int VEC, typename T>
__device__ __forceinline__ void store(T *p, const float (&v)[VEC]) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (VEC == 1) {
            *p = v[0];
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i)
                reinterpret_cast<float4 *>(p)[i] =
                    make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
    } else if constexpr (VEC == 1) {
        *p = __float2bfloat16_rn(v[0]);
    } else {
        uint32_t w[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        if constexpr (VEC == 8)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// Sums of N values over the row's group; every thread gets them.  `red` is the group's own
// space of kMaxWarpsN * N words (not reused before another barrier has passed).  All groups of
// the block call it together.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int warps, int warp, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xFFFFFFFFu, v[n], o);
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int n = 0; n < N; ++n) red[warp * N + n] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = 0.f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += red[w * N + n];
}

// A thread's values: EPT = VEC * steps, step i at (i * row_threads + thread) * VEC.
template <typename HT, typename WT, int VEC, int EPT>
__global__ void __launch_bounds__(kMaxRowThreads) forward_kernel(const NormParams p) {
    constexpr int S = EPT / VEC;
    __shared__ float red[2][kMaxWarpsN];
    const int group = threadIdx.x / p.row_threads, t = threadIdx.x - group * p.row_threads;
    const int warps = p.row_threads / 32, warp = t >> 5;
    const int row = blockIdx.x * (blockDim.x / p.row_threads) + group;
    const bool rv = row < p.M;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const size_t base = static_cast<size_t>(rv ? row : 0) * p.d;
    const HT *h = static_cast<const HT *>(p.h) + base;
    const __nv_bfloat16 *y = static_cast<const __nv_bfloat16 *>(p.y) + base;
    const WT *pre = static_cast<const WT *>(p.pre), *post = static_cast<const WT *>(p.post);
    float a[S][VEC], b[S][VEC];
    float yy[1] = {0.f};
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int e = (i * p.row_threads + t) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[i][j] = b[i][j] = 0.f;
        if (rv && e < p.d) {
            load<VEC>(h + e, a[i]);
            load<VEC>(y + e, b[i]);
        }
    }
    if (post) {
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) yy[0] = fmaf(b[i][j], b[i][j], yy[0]);
        row_sum<1>(yy, warps, warp, red[0] + group * warps);
    }
    const float ry = post ? rsqrtf(yy[0] * p.inv_d + p.eps) : 1.f;
    float hh[1] = {0.f};
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int e = (i * p.row_threads + t) * VEC;
        if (e >= p.d) continue;
        if (post) {
            float w[VEC];
            load<VEC>(post + e, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) b[i][j] = b[i][j] * ry * w[j];
        }
        if (p.gate_kind == 1) {
            float g[VEC];
            load<VEC>(static_cast<const WT *>(p.gate) + e, g);
#pragma unroll
            for (int j = 0; j < VEC; ++j) b[i][j] *= g[j];
        } else if (p.gate_kind == 2 && rv) {
            float g[VEC];
            load<VEC>(static_cast<const __nv_bfloat16 *>(p.gate) + base + e, g);
#pragma unroll
            for (int j = 0; j < VEC; ++j) b[i][j] *= g[j];
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            a[i][j] = fmaf(a[i][j], p.scale, b[i][j]);
            hh[0] = fmaf(a[i][j], a[i][j], hh[0]);
        }
        if (rv) store<VEC>(static_cast<HT *>(p.h_out) + base + e, a[i]);
    }
    row_sum<1>(hh, warps, warp, red[1] + group * warps);
    if (!rv) return;
    const float rh = rsqrtf(hh[0] * p.inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int e = (i * p.row_threads + t) * VEC;
        if (e >= p.d) continue;
        float w[VEC];
        load<VEC>(pre + e, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] *= a[i][j] * rh;
        store<VEC>(static_cast<__nv_bfloat16 *>(p.x) + base + e, w);
    }
}

// One row at a time per block, rows dealt out in turn.
template <typename HT, typename WT, int VEC, int EPT>
__global__ void __launch_bounds__(kMaxRowThreads) backward_kernel(const NormParams p) {
    constexpr int S = EPT / VEC;
    __shared__ float red1[2][kMaxWarpsN * 3], red2[2][kMaxWarpsN];
    const int t = threadIdx.x;
    const int warps = p.row_threads / 32, warp = t >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const WT *pre = static_cast<const WT *>(p.pre), *post = static_cast<const WT *>(p.post);
    float s_pre[S][VEC], s_post[S][VEC], s_gate[S][VEC];
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) s_pre[i][j] = s_post[i][j] = s_gate[i][j] = 0.f;
    int turn = 0;
    for (int row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
        const size_t base = static_cast<size_t>(row) * p.d;
        float dx[S][VEC], tt[S][VEC], h[S][VEC], y[S][VEC];
        float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int e = (i * p.row_threads + t) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) dx[i][j] = tt[i][j] = h[i][j] = y[i][j] = 0.f;
            if (e < p.d) {
                load<VEC>(static_cast<const __nv_bfloat16 *>(p.dx) + base + e, dx[i]);
                if (p.dh) load<VEC>(static_cast<const HT *>(p.dh) + base + e, tt[i]);
                load<VEC>(static_cast<const HT *>(p.h) + base + e, h[i]);
                load<VEC>(static_cast<const __nv_bfloat16 *>(p.y) + base + e, y[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int e = (i * p.row_threads + t) * VEC;
            if (e >= p.d) continue;
            float w[VEC];
            load<VEC>(pre + e, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                sum[0] = fmaf(h[i][j], h[i][j], sum[0]);
                sum[1] = fmaf(dx[i][j] * w[j], h[i][j], sum[1]);
                sum[2] = fmaf(y[i][j], y[i][j], sum[2]);
            }
        }
        row_sum<3>(sum, warps, warp, red1[turn]);
        const float rh = rsqrtf(sum[0] * p.inv_d + p.eps);
        const float c = rh * rh * (sum[1] * p.inv_d);
        const float ry = post ? rsqrtf(sum[2] * p.inv_d + p.eps) : 1.f;
        float fy[1] = {0.f};
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int e = (i * p.row_threads + t) * VEC;
            if (e >= p.d) continue;
            float w[VEC], g[VEC], o[VEC];
            load<VEC>(pre + e, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                s_pre[i][j] = fmaf(dx[i][j], h[i][j] * rh, s_pre[i][j]);
                tt[i][j] += rh * (dx[i][j] * w[j] - h[i][j] * c);
                o[j] = p.scale * tt[i][j];
            }
            store<VEC>(static_cast<HT *>(p.dh_out) + base + e, o);
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[j] = 1.f;
            if (post) load<VEC>(post + e, w);
            if (p.gate_kind) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) o[j] = tt[i][j] * (y[i][j] * ry * w[j]);
                if (p.gate_kind == 1) {
                    load<VEC>(static_cast<const WT *>(p.gate) + e, g);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) s_gate[i][j] += o[j];
                } else {
                    load<VEC>(static_cast<const __nv_bfloat16 *>(p.gate) + base + e, g);
                    store<VEC>(static_cast<__nv_bfloat16 *>(p.dgate) + base + e, o);
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) tt[i][j] *= g[j];
            }
            if (post) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    s_post[i][j] = fmaf(tt[i][j], y[i][j] * ry, s_post[i][j]);
                    tt[i][j] *= w[j];
                    fy[0] = fmaf(tt[i][j], y[i][j], fy[0]);
                }
            }
        }
        if (post) row_sum<1>(fy, warps, warp, red2[turn]);
        const float c2 = post ? ry * ry * (fy[0] * p.inv_d) : 0.f;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int e = (i * p.row_threads + t) * VEC;
            if (e >= p.d) continue;
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] = ry * (tt[i][j] - y[i][j] * c2);
            store<VEC>(static_cast<__nv_bfloat16 *>(p.dy) + base + e, o);
        }
    }
    float *part = p.part + static_cast<size_t>(blockIdx.x) * p.sums * p.d;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int e = (i * p.row_threads + t) * VEC;
        if (e >= p.d) continue;
        float *to = part + e;
        store<VEC>(to, s_pre[i]);
        if (post) store<VEC>(to += p.d, s_post[i]);
        if (p.gate_kind == 1) store<VEC>(to + p.d, s_gate[i]);
    }
}

// Column sums of the blocks' partial vectors, in ascending order: 32 columns x 8 slices of the
// partials per block; out[k]: where vector k of p.sums goes.
struct ColumnParams {
    const float *part;
    int blocks, sums, d;
    void *out[3];
    int f32;
};
constexpr int kSlices = 8;
__global__ void __launch_bounds__(32 * kSlices) columns_kernel(const ColumnParams p) {
    __shared__ float sh[kSlices][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane, k = blockIdx.y;
    float a = 0.f;
    if (col < p.d) {
        const float *src = p.part + static_cast<size_t>(k) * p.d + col;
        const size_t step = static_cast<size_t>(p.sums) * p.d;
        const int b0 = p.blocks * slice / kSlices, b1 = p.blocks * (slice + 1) / kSlices;
#pragma unroll 8
        for (int b = b0; b < b1; ++b) a += src[b * step];
    }
    sh[slice][lane] = a;
    __syncthreads();
    if (slice != 0 || col >= p.d) return;
#pragma unroll
    for (int s = 1; s < kSlices; ++s) a += sh[s][lane];
    if (p.f32)
        static_cast<float *>(p.out[k])[col] = a;
    else
        static_cast<__nv_bfloat16 *>(p.out[k])[col] = __float2bfloat16_rn(a);
}

template <typename P, typename K>
cudaError_t launch_pdl(K kern, dim3 grid, int threads, const P &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool BACK, typename HT, typename WT>
cudaError_t launch_types(const NormParams &p, int vec, int ept, dim3 grid, int threads,
                         cudaStream_t st) {
    if (vec == 8 && ept == 8)
        return launch_pdl(BACK ? backward_kernel<HT, WT, 8, 8> : forward_kernel<HT, WT, 8, 8>, grid,
                          threads, p, st);
    if (vec == 8)
        return launch_pdl(BACK ? backward_kernel<HT, WT, 8, 16> : forward_kernel<HT, WT, 8, 16>,
                          grid, threads, p, st);
    if (vec == 4)
        return launch_pdl(BACK ? backward_kernel<HT, WT, 4, 16> : forward_kernel<HT, WT, 4, 16>,
                          grid, threads, p, st);
    return launch_pdl(BACK ? backward_kernel<HT, WT, 1, 16> : forward_kernel<HT, WT, 1, 16>, grid,
                      threads, p, st);
}

template <bool BACK>
cudaError_t launch_norm(const NormParams &p, bool h32, bool w32, int vec, int ept, dim3 grid,
                        int threads, cudaStream_t st) {
    if (h32)
        return w32 ? launch_types<BACK, float, float>(p, vec, ept, grid, threads, st)
                   : launch_types<BACK, float, __nv_bfloat16>(p, vec, ept, grid, threads, st);
    return w32 ? launch_types<BACK, __nv_bfloat16, float>(p, vec, ept, grid, threads, st)
               : launch_types<BACK, __nv_bfloat16, __nv_bfloat16>(p, vec, ept, grid, threads, st);
}

bool on(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int32_t check_norm(const void *h, const void *y, const void *pre, const void *post,
                   const void *gate, int32_t gate_kind, int64_t M, int64_t d, int32_t stream_type,
                   int32_t weight_type, float scale, float eps) {
    if (M < 0 || M >= (int64_t(1) << 31) - 65536 || d < 1 || d > kMaxNormD || !pre ||
        (M > 0 && (!h || !y)) || gate_kind < SB_GATE_NONE || gate_kind > SB_GATE_TOKEN ||
        (gate_kind == SB_GATE_CHANNEL && !gate) || (gate_kind == SB_GATE_TOKEN && M > 0 && !gate) ||
        stream_type < SB_BF16 || stream_type > SB_F32 || weight_type < SB_BF16 ||
        weight_type > SB_F32 || !std::isfinite(scale) || !(std::isfinite(eps) && eps >= 0.f))
        return SB_ERR_INVALID_ARG;
    const uintptr_t ha = stream_type == SB_F32 ? 4 : 2, wa = weight_type == SB_F32 ? 4 : 2;
    if (!on(h, ha) || !on(y, 2) || !on(pre, wa) || !on(post, wa) ||
        !on(gate, gate_kind == SB_GATE_TOKEN ? 2 : wa))
        return SB_ERR_ALIGNMENT;
    return SB_OK;
}

// The widest vector that d and every address allow: 8, 4 or 1 values.
template <typename... Ptr>
int vector_width(int64_t d, Ptr... ptrs) {
    uintptr_t bits = 0;
    ((bits |= reinterpret_cast<uintptr_t>(ptrs)), ...);
    if ((bits & 15u) == 0) {
        if (d % 8 == 0) return 8;
        if (d % 4 == 0) return 4;
    }
    return 1;
}

int round32(int64_t n) { return static_cast<int>((n + 31) / 32 * 32); }

// Blocks of the backward kernel: what is resident on the device at once, at most one row each.
int backward_blocks(int64_t M, int sms) {
    const int64_t b = 2 * static_cast<int64_t>(sms);
    return static_cast<int>(M < b ? M : b);
}

}  // namespace
}  // namespace sb

using namespace sb;

extern "C" {

int32_t sb_residual_norm_forward(const void *h, const void *y, const void *pre, const void *post,
                                 const void *gate, int32_t gate_kind, int64_t M, int64_t d,
                                 int32_t stream_type, int32_t weight_type, float scale, float eps,
                                 void *h_out, void *x, void *stream) {
    if (int32_t e = check_norm(h, y, pre, post, gate, gate_kind, M, d, stream_type, weight_type,
                               scale, eps))
        return e;
    if (M > 0 && (!h_out || !x)) return SB_ERR_INVALID_ARG;
    if (!on(h_out, stream_type == SB_F32 ? 4 : 2) || !on(x, 2)) return SB_ERR_ALIGNMENT;
    int sms = 0;
    if (int32_t e = device_sms_cc(&sms, nullptr)) return e;
    if (M == 0) return SB_OK;
    NormParams p{};
    p.M = static_cast<int>(M);
    p.d = static_cast<int>(d);
    p.gate_kind = gate_kind;
    p.scale = scale;
    p.eps = eps;
    p.inv_d = 1.f / static_cast<float>(d);
    p.h = h;
    p.y = y;
    p.pre = pre;
    p.post = post;
    p.gate = gate_kind ? gate : nullptr;
    p.h_out = h_out;
    p.x = x;
    const int vec = vector_width(d, h, y, pre, post, p.gate, h_out, x);
    const int ept = vec == 8 && d <= 8 * kMaxRowThreads && M <= 2 * sms ? 8 : 16;
    p.row_threads = round32((d + ept - 1) / ept);
    const int groups = p.row_threads >= 128 ? 1 : 128 / p.row_threads;
    const dim3 grid(static_cast<unsigned>((M + groups - 1) / groups));
    return launch_norm<false>(p, stream_type == SB_F32, weight_type == SB_F32, vec, ept, grid,
                              groups * p.row_threads,
                              static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SB_OK
               : SB_ERR_CUDA;
}

size_t sb_residual_norm_workspace_bytes(int64_t M, int64_t d) {
    if (M < 0 || M >= (int64_t(1) << 31) - 65536 || d < 1 || d > kMaxNormD) return 0;
    int sms = 0;
    if (device_sms_cc(&sms, nullptr) != SB_OK) return 0;
    const size_t n = up256(static_cast<size_t>(backward_blocks(M, sms)) * 3 * d * 4);
    return n ? n : 256;
}

int32_t sb_residual_norm_backward(const void *dx, const void *dh, const void *h, const void *y,
                                  const void *pre, const void *post, const void *gate,
                                  int32_t gate_kind, int64_t M, int64_t d, int32_t stream_type,
                                  int32_t weight_type, float scale, float eps, void *dh_out,
                                  void *dy, void *dpre, void *dpost, void *dgate, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    if (int32_t e = check_norm(h, y, pre, post, gate, gate_kind, M, d, stream_type, weight_type,
                               scale, eps))
        return e;
    if ((M > 0 && (!dx || !dh_out || !dy)) || !dpre || (post && !dpost) ||
        (gate_kind == SB_GATE_CHANNEL && !dgate) || (gate_kind == SB_GATE_TOKEN && M > 0 && !dgate) ||
        !workspace)
        return SB_ERR_INVALID_ARG;
    const uintptr_t ha = stream_type == SB_F32 ? 4 : 2, wa = weight_type == SB_F32 ? 4 : 2;
    if (!on(dx, 2) || !on(dh, ha) || !on(dh_out, ha) || !on(dy, 2) || !on(dpre, wa) ||
        !on(dpost, wa) || !on(dgate, gate_kind == SB_GATE_TOKEN ? 2 : wa) || !on(workspace, 16))
        return SB_ERR_ALIGNMENT;
    int sms = 0;
    if (int32_t e = device_sms_cc(&sms, nullptr)) return e;
    if (workspace_bytes < sb_residual_norm_workspace_bytes(M, d)) return SB_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    ColumnParams c{};
    c.d = static_cast<int>(d);
    c.f32 = weight_type == SB_F32;
    c.out[c.sums++] = dpre;
    if (post) c.out[c.sums++] = dpost;
    if (gate_kind == SB_GATE_CHANNEL) c.out[c.sums++] = dgate;
    if (M == 0) {  // the empty sums
        for (int k = 0; k < c.sums; ++k)
            if (cudaMemsetAsync(c.out[k], 0, static_cast<size_t>(d) * wa, st) != cudaSuccess)
                return SB_ERR_CUDA;
        return SB_OK;
    }
    NormParams p{};
    p.M = static_cast<int>(M);
    p.d = static_cast<int>(d);
    p.gate_kind = gate_kind;
    p.scale = scale;
    p.eps = eps;
    p.inv_d = 1.f / static_cast<float>(d);
    p.h = h;
    p.y = y;
    p.pre = pre;
    p.post = post;
    p.gate = gate_kind ? gate : nullptr;
    p.dx = dx;
    p.dh = dh;
    p.dh_out = dh_out;
    p.dy = dy;
    p.dgate = gate_kind == SB_GATE_TOKEN ? dgate : nullptr;
    p.part = static_cast<float *>(workspace);
    p.sums = c.sums;
    const int vec =
        vector_width(d, dx, dh, h, y, pre, post, p.gate, dh_out, dy, p.dgate, workspace);
    const int ept = vec == 8 && d <= 8 * kMaxRowThreads ? 8 : 16;
    p.row_threads = round32((d + ept - 1) / ept);
    const int blocks = backward_blocks(M, sms);
    c.part = p.part;
    c.blocks = blocks;
    if (launch_norm<true>(p, stream_type == SB_F32, weight_type == SB_F32, vec, ept, dim3(blocks),
                          p.row_threads, st) != cudaSuccess ||
        launch_pdl(columns_kernel, dim3(static_cast<unsigned>((d + 31) / 32), c.sums), 32 * kSlices,
                   c, st) != cudaSuccess)
        return SB_ERR_CUDA;
    return SB_OK;
}

}  // extern "C"
