// layer_norm.cu -- a branch's dropout, its sum with the residual stream and the layer norm behind it
// in one pass, with the gradients.  Over a row of d values:
//   forward    h' = h + dropout(y)  (without y: h' = h, not written),
//              x = (h' - mean)·r·weight + bias,   r = 1 / sqrt(mean((h' - mean)²) + eps)
//   backward   given h' and the gradients dx of x and dh of h', with c = h' - mean, a = dx·weight:
//     t = dh + r·(a - mean(a) - c·r²·mean(a·c)),  gradient of h = t,  dy = dropout(t),
//     dweight = sum over rows of dx·c·r,  dbias = sum over rows of dx.
//
// The variance is summed over the centred values, in a second reduction over registers: a stream's
// level may be far from zero, and E(h²) - E(h)² would cancel.  Backward forms mean and deviation from
// the stored h' instead of reading them; its other two sums go with the variance's.
//
// Both are bound by memory, and what keeps them from it is the time that a row's threads wait for
// each other in the two reductions.  As in the residual norm (norm.cu) a row belongs to a group of
// threads, sixteen values to a thread, and the next rows are on their way in a cp.async ring.
// A thread works on two rows side by side: their sums go through the same two reductions, and one's
// arithmetic fills the other's waits.  8192 x 6144 bf16 with branch and dropout: forward 64 us, 6.3
// TB/s, backward 82, 6.1 TB/s; one row at a time: 74 and 94; four rows in forward, whose ring then has
// no third step: 71; two groups of 384 threads with the weights in shared memory: 70; a block to a
// row, which ends with it: 108 (its fixed work and its loads of weights weigh more than the waits).
// Weights and column sums are in registers; backward reads dx and dh again from the ring.  A draw's
// state goes from row to row by one addition.
//
// A block has 384 threads, with up to 168 registers each, where a row or several fill it (up to 6144
// values), and 512 with 128 registers for rows of up to 8192 and for two groups of 193 to 256 threads.
// Two rows at a time still fit into those in forward, in backward they would spill: it takes one.
// Measured with branch and dropout, bf16, against 384 threads for short rows and 640 to 1024 for long:
// 8192 x 4096 forward 50 -> 46 us, backward 69 -> 61; 4096 x 8192 58 -> 45 and 118 -> 64 (91 with two rows
// at a time).  Two groups need a ring of three steps: with two, 8192 x 4096 fp32 forward takes 83 us
// against 73, backward 120 against 114.  Longer rows have up to 1024 threads of 64 registers, which
// spill: 2048 x 16384 without branch forward 33 us, backward 130.
//
// A row length that is no multiple of eight shifts each row against the vectors' boundaries
// (layer_norm.cuh); a group's rows are a multiple of eight apart, so that their shift, and with it a
// thread's columns, stay the same.  8192 x 6135: forward 82 us, backward 119; 8192
// x 6143: 95 and 145 (with a shift of up to seven values such a row is one vector more than 384 threads
// hold, and the wider block takes one row at a time in backward).
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
    q.wide_weights = on(weight, 16) && on(bias, 16);
    q.drop = make_dropout(p, seed, seed_offset);
    return q;
}

template <typename... Ptr>
LoadMode mode_of(int64_t d, Ptr... ptrs) {
    uintptr_t bits = 0;
    ((bits |= reinterpret_cast<uintptr_t>(ptrs)), ...);
    if (bits & 15u) return kSingle;
    return d % 8 == 0 ? kAligned : d > 8 ? kShifted : kSingle;
}
// A row's threads, the groups of a block, the rows that a group works on at a time and the steps of its
// ring.  row_bytes: of a thread for a row of the ring; weight_bytes: of a thread, for the weights of rows
// too long to keep them in registers; wide_rows: rows at a time in a block of more than 384 threads.
struct Layout {
    LoadMode mode;
    int row_threads, groups, steps, rows;
    bool weights;  // kept in shared memory
    int64_t blocks;
    size_t smem;
};
Layout lay_out(int64_t M, int64_t d, LoadMode mode, size_t row_bytes, size_t weight_bytes, int wide_rows,
               int sms) {
    Layout l{};
    auto threads_of = [d](int shift) {
        return round32(((d + shift + 7) / 8 + kNormVectors - 1) / kNormVectors);
    };
    if (mode == kShifted && threads_of(7) > 1024) mode = kSingle;
    l.mode = mode;
    l.row_threads = threads_of(mode == kShifted ? 7 : 0);
    const int64_t share = (M + sms - 1) / sms;  // rows of an SM
    const size_t step = l.row_threads * row_bytes;
    // longer rows have a block of 512 threads, and so have two groups where one leaves much of 384 idle,
    // if their ring still has three steps
    l.groups = kNormThreads / l.row_threads;
    if (l.groups == 0 ||
        (l.groups == 1 && 2 * l.row_threads <= kWideThreads && 3 * 2 * wide_rows * step <= kNormRingBytes))
        l.groups = kWideThreads / l.row_threads;
    l.rows = mode == kSingle || l.groups < 1 ? 1 : l.groups * l.row_threads > kNormThreads ? wide_rows : 2;
    if (l.groups > kMaxGroups) l.groups = kMaxGroups;
    if (l.groups > share) l.groups = static_cast<int>(share);
    // rows of up to 8192 have their weights in registers; rows too long for weights and two steps in
    // shared memory read the weights from memory again for each row
    if (l.groups >= 1 || 2 * step + weight_bytes * l.row_threads > kNormRingBytes) weight_bytes = 0;
    if (l.groups < 1) l.groups = 1;
    l.weights = weight_bytes > 0;
    const size_t weights = weight_bytes * l.row_threads;  // (one group then)
    // a ring of two steps at least: one is on its way while another one is worked on; two rows at a
    // time where the SM's share fills that twice, and one row, then fewer groups, where they do not fit
    auto fit = [&] { return (kNormRingBytes - weights) / (l.rows * l.groups * step); };
    if (share < 2 * l.rows * l.groups || fit() < 2) l.rows = 1;
    while (mode != kSingle && fit() < 2 && l.groups > 1) --l.groups;
    // (a row of backward beyond 10240 in fp32 has the ring to itself: nothing is ahead)
    l.steps = mode == kSingle ? 1 : static_cast<int>(fit());
    if (l.steps < 1) l.mode = kSingle, l.steps = 1;  // (no row is that long)
    if (l.steps > kMaxDepth) l.steps = kMaxDepth;
    l.smem = weights + (l.mode == kSingle ? 0 : l.steps * l.rows * l.groups * step);
    l.blocks = (M + l.groups - 1) / l.groups;
    // (a multiple of eight: the rows of a group then have the same shift)
    if (l.blocks > sms) l.blocks = mode == kShifted && sms > 8 ? sms & ~7 : sms;
    return l;
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
    // outputs over an input's memory: only the ones that the same thread has read by then (which then
    // stand here once)
    const size_t hb = M * d * (stream_type == SB_F32 ? 4 : 2), bb = M * d * 2;
    const size_t wb = d * (weight_type == SB_F32 ? 4 : 2);
    const Span arrays[] = {{x, bb}, {y ? h_out : nullptr, hb}, {x == y ? nullptr : y, bb},
                           {y && h_out == h ? nullptr : h, hb}, {weight, wb}, {bias, wb}, {seed_offset, 8}};
    if (any_overlap(arrays, 2)) return SB_ERR_INVALID_ARG;
    int sms = 0;
    if (int32_t e = device_sms_cc(&sms, nullptr)) return e;
    if (M == 0) return SB_OK;
    LayerNormParams q =
        params_of(h, weight, bias, M, d, weight_type, p, seed, seed_offset, eps);
    q.y = y;
    q.h_out = h_out;
    q.x = x;
    const bool h32 = stream_type == SB_F32;
    const Layout l = lay_out(M, d, mode_of(d, h, y, y ? h_out : nullptr, x),
                             kNormVectors * 8 * ((h32 ? 4 : 2) + (y ? 2 : 0)), kNormVectors * 64, 2, sms);
    q.row_threads = l.row_threads;
    q.groups = l.groups;
    q.steps = l.steps;
    q.shared_weights = l.weights;
    const LayerNormShape shape{l.mode, h32, l.groups * l.row_threads, l.rows};
    return launch_layer_norm_forward(q, shape, static_cast<unsigned>(l.blocks), l.smem,
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
    const size_t hb = M * d * ha, bb = M * d * 2, wb = d * wa;
    Span arrays[] = {{workspace, 0}, {dweight, wb}, {dbias, wb}, {dh_out, hb}, {dy, bb},
                     {dy == dx ? nullptr : dx, bb}, {dh_out == dh ? nullptr : dh, hb}, {h, hb}, {weight, wb},
                     {seed_offset, 8}};
    if (any_overlap(arrays, 5)) return SB_ERR_INVALID_ARG;
    int sms = 0;
    if (int32_t e = device_sms_cc(&sms, nullptr)) return e;
    const size_t need = sb_layer_norm_workspace_bytes(M, d);
    arrays[0].bytes = need;  // (which the device decides)
    if (any_overlap(arrays, 1)) return SB_ERR_INVALID_ARG;
    if (workspace_bytes < need) return SB_ERR_WORKSPACE_TOO_SMALL;
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
    const Layout l = lay_out(M, d, mode_of(d, dx, dh, h, dh_out, dy),
                             kNormVectors * 8 * ((h32 ? 8 : 4) + 2), 0, 1, sms);
    q.row_threads = l.row_threads;
    q.groups = l.groups;
    q.steps = l.steps;
    const LayerNormShape shape{l.mode, h32, l.groups * l.row_threads, l.rows};
    size_t smem = l.smem;
    const size_t sum_bytes = static_cast<size_t>(q.sums) * d * 4;
    if (q.groups > 1 && smem < sum_bytes) smem = sum_bytes;
    ColumnParams c{};
    c.part = q.part;
    c.blocks = static_cast<int>(l.blocks);
    c.sums = q.sums;
    c.d = static_cast<int>(d);
    c.f32 = weight_type == SB_F32;
    c.dpre = dweight;
    c.dpost = dbias;
    if (launch_layer_norm_backward(q, shape, static_cast<unsigned>(l.blocks), smem, st) != cudaSuccess ||
        launch_norm_columns(c, true, st) != cudaSuccess)
        return SB_ERR_CUDA;
    return SB_OK;
}

}  // extern "C"
