// norm.cu -- the end of a transformer block in one pass: the norm after the block, its gate, the
// scaled residual sum and the norm before the next block (or the output head), with the
// gradients.  With n(x; w) = w·x / sqrt(mean(x²) + eps) over a row of d values:
//   forward    h' = scale·h + gate·n(y; post),   x = n(h'; pre)
//   backward   given h' and y and the gradients dx of x and dh of h':
//     a = dx·pre,  rh = 1 / sqrt(mean(h'²) + eps),  t = dh + rh·(a - h'·rh²·mean(a·h'))
//     dpre = sum over rows of dx·h'·rh,   gradient of h = scale·t
//     u = n(y; post),  dgate = t·u (summed over the rows when the gate is one vector)
//     f = t·gate·post,  dpost = sum over rows of t·gate·y·ry,
//     dy = ry·(f - y·ry²·mean(f·y))
// (post and gate are optional: u = y without the one, factor 1 without the other).
//
// Both kernels are bound by memory: forward reads h and y and writes h' and x, backward reads
// dx, dh, h' and y and writes two gradients, each once (8192 x 6144 in bf16: 62.6 and 99.6 us,
// 6.4 and 6.1 TB/s).  A row belongs to a group of threads, sixteen values to a thread, and its
// values stay in registers, as do the weights over all rows of the group; sums are formed in
// pairs of fp32.  Row reductions would stall the loads behind them, so the next rows are on their
// way meanwhile: every thread copies its own values of the rows ahead to shared memory with
// cp.async, and as it alone reads them no barrier is needed (a ring of up to kMaxDepth rows per
// group; without it forward took 107 us and backward 232).  Arrays that are not 16-byte aligned,
// or have d not a multiple of 4, or rows too long for two of them to fit, are read directly.
//
// All sums are fp32.  Forward needs two row reductions in turn, and x comes from the unrounded
// h' (one rounding per output).  Backward differentiates at the h' that was stored and needs
// one: with b = gate·post·y, sum(f·y) = sum(b·dh) + rh·(sum(b·a) - rh²·mean(a·h')·sum(b·h')),
// so all six sums are known at once, with the rounding of t's own terms.  Its column sums stay
// in registers over all rows of a group; the groups of a block add up in shared memory, every
// block leaves one partial vector each, and columns_kernel adds the partials in ascending
// order: equal calls give equal bits.  Its vector 1, the sum of t·(gate of the row)·y·ry, serves
// dpost and the gate vector's gradient.
#include <cmath>

#include "norm_common.cuh"
#include "sb.h"

namespace sb {
namespace {

__device__ __forceinline__ float weight_at(const void *w, int f32, int i) {
    if (!w) return 1.f;
    return f32 ? one(static_cast<const float *>(w) + i)
               : one(static_cast<const __nv_bfloat16 *>(w) + i);
}
__device__ __forceinline__ void put_at(void *w, int f32, int i, float v) {
    if (f32)
        put_one(static_cast<float *>(w) + i, v);
    else
        put_one(static_cast<__nv_bfloat16 *>(w) + i, v);
}
template <int SLICES>
__global__ void __launch_bounds__(32 * SLICES) columns_kernel(const ColumnParams p) {
    __shared__ float sh[SLICES][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane, k = blockIdx.y;
    float a = 0.f;
    if (col < p.d) {
        const float *src = p.part + static_cast<size_t>(k) * p.d + col;
        const size_t step = static_cast<size_t>(p.sums) * p.d;
        const int b0 = p.blocks * slice / SLICES, b1 = p.blocks * (slice + 1) / SLICES;
#pragma unroll 8
        for (int b = b0; b < b1; ++b) a += src[b * step];
    }
    sh[slice][lane] = a;
    __syncthreads();
    if (slice != 0 || col >= p.d) return;
#pragma unroll
    for (int s = 1; s < SLICES; ++s) a += sh[s][lane];
    if (k == 0) {
        put_at(p.dpre, p.f32, col, a);
    } else {
        if (p.dpost) put_at(p.dpost, p.f32, col, a * weight_at(p.gate, p.f32, col));
        if (p.dgate) put_at(p.dgate, p.f32, col, a * weight_at(p.post, p.f32, col));
    }
}

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
        (gate_kind != SB_GATE_NONE && !on(gate, gate_kind == SB_GATE_TOKEN ? 2 : wa)))
        return SB_ERR_ALIGNMENT;
    return SB_OK;
}

}  // namespace

cudaError_t launch_norm_columns(const ColumnParams &p, bool many, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((p.d + 31) / 32), p.sums);
    return many ? launch_dependent(columns_kernel<16>, grid, 32 * 16, 0, p, st)
                : launch_dependent(columns_kernel<8>, grid, 32 * 8, 0, p, st);
}

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
    p.scale = scale;
    p.eps = eps;
    p.inv_d = 1.f / static_cast<float>(d);
    p.h = h;
    p.y = y;
    p.pre = pre;
    p.post = post;
    p.gate = gate_kind == SB_GATE_CHANNEL ? gate : nullptr;
    p.gate_rows = gate_kind == SB_GATE_TOKEN ? gate : nullptr;
    p.w32 = weight_type == SB_F32;
    p.h_out = h_out;
    p.x = x;
    const bool h32 = stream_type == SB_F32;
    const int vec = vector_width(d, h, y, pre, post, gate_kind ? gate : nullptr, h_out, x);
    const int value_bytes = (h32 ? 4 : 2) + 2 + (p.gate_rows ? 2 : 0);
    const NormLayout l = layout_of(M, d, vec, value_bytes, 0, sms);
    p.row_threads = l.row_threads;
    p.groups = l.groups;
    p.depth = l.depth;
    return launch_norm_forward(p, l.shape, h32, l.blocks, l.smem,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SB_OK
               : SB_ERR_CUDA;
}

size_t sb_residual_norm_workspace_bytes(int64_t M, int64_t d) {
    if (M < 0 || M >= (int64_t(1) << 31) - 65536 || d < 1 || d > kMaxNormD) return 0;
    int sms = 0;
    if (device_sms_cc(&sms, nullptr) != SB_OK) return 0;
    const int64_t blocks = M < sms ? (M < 1 ? 1 : M) : sms;
    return up256(static_cast<size_t>(blocks) * 2 * d * 4);
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
        (post && !on(dpost, wa)) ||
        (gate_kind != SB_GATE_NONE && !on(dgate, gate_kind == SB_GATE_TOKEN ? 2 : wa)) ||
        !on(workspace, 16))
        return SB_ERR_ALIGNMENT;
    int sms = 0;
    if (int32_t e = device_sms_cc(&sms, nullptr)) return e;
    if (workspace_bytes < sb_residual_norm_workspace_bytes(M, d)) return SB_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    ColumnParams c{};
    c.d = static_cast<int>(d);
    c.f32 = weight_type == SB_F32;
    c.dpre = dpre;
    c.dpost = post ? dpost : nullptr;
    c.dgate = gate_kind == SB_GATE_CHANNEL ? dgate : nullptr;
    c.sums = c.dpost || c.dgate ? 2 : 1;
    if (M == 0) {  // the empty sums
        for (void *v : {c.dpre, c.dpost, c.dgate})
            if (v && cudaMemsetAsync(v, 0, static_cast<size_t>(d) * wa, st) != cudaSuccess)
                return SB_ERR_CUDA;
        return SB_OK;
    }
    NormParams p{};
    p.M = static_cast<int>(M);
    p.d = static_cast<int>(d);
    p.scale = scale;
    p.eps = eps;
    p.inv_d = 1.f / static_cast<float>(d);
    p.h = h;
    p.y = y;
    p.pre = pre;
    p.post = post;
    p.gate = gate_kind == SB_GATE_CHANNEL ? gate : nullptr;
    p.gate_rows = gate_kind == SB_GATE_TOKEN ? gate : nullptr;
    p.w32 = weight_type == SB_F32;
    p.dx = dx;
    p.dh = dh;
    p.dh_out = dh_out;
    p.dy = dy;
    p.dgate_rows = gate_kind == SB_GATE_TOKEN ? dgate : nullptr;
    p.part = static_cast<float *>(workspace);
    p.sums = c.sums;
    const bool h32 = stream_type == SB_F32;
    const int vec = vector_width(d, dx, dh, h, y, pre, post, gate_kind ? gate : nullptr, dh_out, dy,
                                 p.dgate_rows, workspace);
    const int value_bytes = (h32 ? 8 : 4) + 4 + (p.gate_rows ? 2 : 0);
    const NormLayout l =
        layout_of(M, d, vec, value_bytes, static_cast<size_t>(c.sums) * d * 4, sms);
    p.row_threads = l.row_threads;
    p.groups = l.groups;
    p.depth = l.depth;
    c.part = p.part;
    c.blocks = l.blocks;
    c.post = p.post;
    c.gate = p.gate;
    if (launch_norm_backward(p, l.shape, h32, l.blocks, l.smem, st) != cudaSuccess ||
        launch_norm_columns(c, false, st) != cudaSuccess)
        return SB_ERR_CUDA;
    return SB_OK;
}

}  // extern "C"
