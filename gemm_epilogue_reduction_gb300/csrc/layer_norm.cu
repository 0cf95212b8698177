// layer_norm.cu -- a branch's dropout, its sum with the residual stream and the layer norm behind it
// in one pass, with the gradients.  Over a row of d values:
//   forward    h' = h + dropout(y)  (without y: h' = h, not written),
//              x = (h' - mean)·r·weight + bias,   r = 1 / sqrt(mean((h' - mean)²) + eps)
//   backward   given h' and the gradients dx of x and dh of h', with c = h' - mean, a = dx·weight:
//     t = dh + r·(a - mean(a) - c·r²·mean(a·c)),  gradient of h = t,  dy = dropout(t),
//     dweight = sum over rows of dx·c·r,  dbias = sum over rows of dx.
//
// The layout is that of the residual norm (norm.cu): sixteen values to a thread, a row to a group
// of threads, weights and column sums in registers, the next rows on their way in a cp.async ring.
// The variance is summed over the centred values, in a second reduction over the registers: a
// stream's level may be far from zero, and E(h²) - E(h)² would cancel.  Backward forms the same two
// from the stored h' instead of reading them; its other two sums go with the variance's.
#include <cmath>

#include "layer_norm.cuh"
#include "sb.h"

namespace sb {
namespace {

int32_t check_layer_norm(const void *h, const void *weight, const void *bias, int64_t M, int64_t d,
                         int32_t stream_type, int32_t weight_type, float p, const void *seed_offset,
                         float eps) {
    if (M < 0 || M >= (int64_t(1) << 31) - 65536 || d < 1 || d > kMaxNormD || !weight ||
        (M > 0 && !h) || stream_type < SB_BF16 || stream_type > SB_F32 || weight_type < SB_BF16 ||
        weight_type > SB_F32 || !(p >= 0.f && p <= 1.f) || !(std::isfinite(eps) && eps >= 0.f))
        return SB_ERR_INVALID_ARG;
    const uintptr_t ha = stream_type == SB_F32 ? 4 : 2, wa = weight_type == SB_F32 ? 4 : 2;
    if (!on(h, ha) || !on(weight, wa) || !on(bias, wa) || !on(seed_offset, 8))
        return SB_ERR_ALIGNMENT;
    return SB_OK;
}

LayerNormParams params_of(const void *h, const void *weight, const void *bias, int64_t M, int64_t d,
                          int32_t weight_type, float p, uint64_t seed, const void *seed_offset,
                          float eps) {
    LayerNormParams q{};
    q.M = static_cast<int>(M);
    q.d = static_cast<int>(d);
    q.w32 = weight_type == SB_F32;
    q.eps = eps;
    q.inv_d = 1.f / static_cast<float>(d);
    q.h = h;
    q.weight = weight;
    q.bias = bias;
    q.drop = make_dropout(p, seed, seed_offset);
    return q;
}

}  // namespace
}  // namespace sb

using namespace sb;

extern "C" {

int32_t sb_layer_norm_forward(const void *h, const void *y, const void *weight, const void *bias,
                              int64_t M, int64_t d, int32_t stream_type, int32_t weight_type,
                              float p, uint64_t seed, const uint64_t *seed_offset, float eps,
                              void *h_out, void *x, void *stream) {
    if (int32_t e = check_layer_norm(h, weight, bias, M, d, stream_type, weight_type, p,
                                     seed_offset, eps))
        return e;
    if (M > 0 && (!x || (y && !h_out))) return SB_ERR_INVALID_ARG;
    if (!on(y, 2) || (y && !on(h_out, stream_type == SB_F32 ? 4 : 2)) || !on(x, 2))
        return SB_ERR_ALIGNMENT;
    int sms = 0;
    if (int32_t e = device_sms_cc(&sms, nullptr)) return e;
    if (M == 0) return SB_OK;
    LayerNormParams q =
        params_of(h, weight, bias, M, d, weight_type, p, seed, seed_offset, eps);
    q.y = y;
    q.h_out = h_out;
    q.x = x;
    const bool h32 = stream_type == SB_F32;
    const int vec = vector_width(d, h, y, weight, bias, y ? h_out : nullptr, x);
    const NormLayout l = layout_of(M, d, vec, (h32 ? 4 : 2) + (y ? 2 : 0), 0, sms);
    q.row_threads = l.row_threads;
    q.groups = l.groups;
    q.depth = l.depth;
    return launch_layer_norm_forward(q, l.shape, h32, l.blocks, l.smem,
                                     static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SB_OK
               : SB_ERR_CUDA;
}

size_t sb_layer_norm_workspace_bytes(int64_t M, int64_t d) {
    if (M < 0 || M >= (int64_t(1) << 31) - 65536 || d < 1 || d > kMaxNormD) return 0;
    int sms = 0;
    if (device_sms_cc(&sms, nullptr) != SB_OK) return 0;
    const int64_t blocks = M < sms ? (M < 1 ? 1 : M) : sms;
    return up256(static_cast<size_t>(blocks) * 2 * d * 4);
}

int32_t sb_layer_norm_backward(const void *dx, const void *dh, const void *h, const void *weight,
                               int64_t M, int64_t d, int32_t stream_type, int32_t weight_type,
                               float p, uint64_t seed, const uint64_t *seed_offset, float eps,
                               void *dh_out, void *dy, void *dweight, void *dbias, void *workspace,
                               size_t workspace_bytes, void *stream) {
    if (int32_t e = check_layer_norm(h, weight, nullptr, M, d, stream_type, weight_type, p,
                                     seed_offset, eps))
        return e;
    if ((M > 0 && (!dx || !dh_out)) || !dweight || !workspace) return SB_ERR_INVALID_ARG;
    const uintptr_t ha = stream_type == SB_F32 ? 4 : 2, wa = weight_type == SB_F32 ? 4 : 2;
    if (!on(dx, 2) || !on(dh, ha) || !on(dh_out, ha) || !on(dy, 2) || !on(dweight, wa) ||
        !on(dbias, wa) || !on(workspace, 16))
        return SB_ERR_ALIGNMENT;
    int sms = 0;
    if (int32_t e = device_sms_cc(&sms, nullptr)) return e;
    if (workspace_bytes < sb_layer_norm_workspace_bytes(M, d)) return SB_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (M == 0) {  // the empty sums
        for (void *v : {dweight, dbias})
            if (v && cudaMemsetAsync(v, 0, static_cast<size_t>(d) * wa, st) != cudaSuccess)
                return SB_ERR_CUDA;
        return SB_OK;
    }
    LayerNormParams q =
        params_of(h, weight, nullptr, M, d, weight_type, p, seed, seed_offset, eps);
    q.dx = dx;
    q.dh = dh;
    q.dh_out = dh_out;
    q.dy = dy;
    q.part = static_cast<float *>(workspace);
    q.sums = dbias ? 2 : 1;
    const bool h32 = stream_type == SB_F32;
    const int vec = vector_width(d, dx, dh, h, weight, dh_out, dy, workspace);
    const NormLayout l = layout_of(M, d, vec, (h32 ? 8 : 4) + 2,
                                   static_cast<size_t>(q.sums) * d * 4, sms);
    q.row_threads = l.row_threads;
    q.groups = l.groups;
    q.depth = l.depth;
    ColumnParams c{};
    c.part = q.part;
    c.blocks = l.blocks;
    c.sums = q.sums;
    c.d = static_cast<int>(d);
    c.f32 = weight_type == SB_F32;
    c.dpre = dweight;
    c.dpost = dbias;
    if (launch_layer_norm_backward(q, l.shape, h32, l.blocks, l.smem, st) != cudaSuccess ||
        launch_norm_columns(c, st) != cudaSuccess)
        return SB_ERR_CUDA;
    return SB_OK;
}

}  // extern "C"
