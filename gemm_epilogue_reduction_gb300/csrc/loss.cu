// loss.cu -- the cross entropy of the output head: the rows' losses from the projection
// records, and the host side of both directions.
//
// Forward is the record GEMM of lmhead.cu (with the targets' logits) followed by one kernel:
//   lse_r  = m + log sum_t s_rt·exp(m_rt - m),  m = max_t m_rt   (records t of 128 columns)
//   loss_r = lse_r - z_r,target + z_loss·lse_r²,  0 where the target is the ignored index,
// one block per row.  The tensor cores truncate as they accumulate, which leaves a logit of d =
// 5120 products some 1e-5 short; the target's logit stands alone in the loss (every other one is
// averaged in lse), so its block forms it again in fp32 FMAs (loss_common.cuh):
//   lse - z = log(1 + R·e^(z_tc - z)),   R = sum over the others of e^(z_j - z_tc),
// where R is summed without the target's term if that leads its record (below), so that a small R
// keeps its own precision.  lse is z plus that: backward, which gets lse, forms the same z and
// p - 1 from the two.  The last block to finish adds the rows' losses up (SUM, MEAN) in a fixed
// order, so the bits do not depend on which block that is.
//
// The rows kernel reads 8 bytes for each 128 columns of a row, H's row and the target's row of W:
// next to the GEMM it is small (M = 4096, d = 6144, V = 200,064: 150 MB, 35 us against 5.1 ms),
// and for few rows its chain of dependent loads costs some 4 us.  The GEMM is bound by reading W
// up to some 256 rows (16 x 5120 x 151,936: 233 to 239 us in all, 96 to 98 % of the measured memory rate) and
// by the tensor cores beyond.  Backward is loss_grad.cu; its host side here cuts the vocabulary
// into pieces and chooses the split of the dH reduction.
#include <cmath>

#include "loss_common.cuh"
#include "sb.h"
#include "sb_internal.h"
#include "sb_ptx.cuh"

namespace sb {
namespace {

constexpr int kRowThreads = kDotParts;
constexpr float kLog2e = 1.4426950408889634f;

struct MaxSum {
    float m, s;
};
// Sums of exp relative to the larger maximum; -inf maxima (nothing seen) carry s = 0.
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return MaxSum{m, 0.f};
    return MaxSum{m, a.s * ex2_approx((a.m - m) * kLog2e) + b.s * ex2_approx((b.m - m) * kLog2e)};
}

__global__ void __launch_bounds__(kRowThreads) rows_kernel(const LossParams p) {
    __shared__ float sm[kRowThreads / 32], ss[kRowThreads / 32], sz[kRowThreads / 32];
    __shared__ int is_last;
    const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // all the records' writes first, then let the next kernel set up
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = p.targets[row];
    const bool inside = t >= 0 && t < p.V && t != p.ignore_index;
    // the target's logit
    float dot = 0.f;
    if (inside) {
        float part[1];
        dot_parts(p.H + static_cast<size_t>(row) * p.d, p.W + static_cast<size_t>(t) * p.d, p.d,
                  threadIdx.x, part);
        dot = part[0];
    }
    const float *rm = p.ws.m + static_cast<size_t>(row) * p.T;
    const float *rs = p.ws.s + static_cast<size_t>(row) * p.T;
    // The target's record, where the target is its largest column: its exponential was then the one
    // below, bit for bit, and no rounded sum of it and other terms >= 0 is smaller.
    int lead = -1;
    float tz = 0.f, own = 0.f;
    if (inside) {
        tz = p.ws.tz[row];
        if (rm[t / kTileA] == tz && tz > -INFINITY) lead = t / kTileA;
        own = ex2_approx(fmaf(tz, kLog2e, -(tz * kLog2e)));
    }
    MaxSum a{-INFINITY, 0.f};
    for (int k = threadIdx.x; k < p.T; k += 4 * kRowThreads) {
        MaxSum x[4];  // four records in flight
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = k + u * kRowThreads;
            x[u] = i < p.T ? MaxSum{rm[i], rs[i]} : MaxSum{-INFINITY, 0.f};
            if (i == lead) x[u].s -= own;
        }
        a = join(a, join(join(x[0], x[1]), join(x[2], x[3])));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a = join(a, MaxSum{__shfl_xor_sync(0xFFFFFFFFu, a.m, o),
                           __shfl_xor_sync(0xFFFFFFFFu, a.s, o)});
        dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
    }
    if (lane == 0) {
        sm[warp] = a.m;
        ss[warp] = a.s;
        sz[warp] = dot;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kRowThreads / 32; ++w) {
            a = join(a, MaxSum{sm[w], ss[w]});
            dot += sz[w];
        }
        float lse = a.m + logf(a.s);
        float loss = 0.f;
        if (inside) {
            const float more = tz - dot;  // what the tensor cores' number has in excess
            float n = (a.m - tz) + logf(a.s);
            if (dot == -INFINITY) {
                n = INFINITY;  // no share of the sum, which is the others' lse
            } else {
                // from n = 16 on the target's share is below fp32's half unit
                if (n >= 16.f || n != n)
                    n += more;
                else
                    n = log1pf(lead >= 0 ? expf(n + more) : expm1f(n) * expf(more));
                lse = dot + n;
            }
            loss = n + p.z_loss * lse * lse;
        } else if (t != p.ignore_index) {
            // a target outside the vocabulary has no logit: the status word reports it
            loss = __uint_as_float(0x7FC00000u);
        }
        p.lse[row] = lse;
        p.rows[row] = loss;
        is_last = 0;
        if (p.reduction != SB_REDUCE_NONE) {
            __threadfence();  // this row's loss before its count
            is_last = atomicAdd(p.ws.epoch + 1, 1u) == static_cast<uint32_t>(p.M) - 1u;
        }
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    // 64-bit partial sums: M terms of one size
    double sum = 0.0;
    int count = 0;
    for (int r = threadIdx.x; r < p.M; r += kRowThreads)
        if (p.targets[r] != p.ignore_index) {
            sum += static_cast<double>(__ldcg(p.rows + r));
            ++count;
        }
    __shared__ double sd[kRowThreads];
    __shared__ int sc[kRowThreads];
    sd[threadIdx.x] = sum;
    sc[threadIdx.x] = count;
    __syncthreads();
    for (int w = kRowThreads / 2; w > 0; w >>= 1) {
        if (threadIdx.x < w) {
            sd[threadIdx.x] += sd[threadIdx.x + w];
            sc[threadIdx.x] += sc[threadIdx.x + w];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0)
        *p.loss = static_cast<float>(
            p.reduction == SB_REDUCE_MEAN ? sd[0] / (sc[0] > 0 ? sc[0] : 1) : sd[0]);
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool on(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// min(floor(2^32 / n), 2^32 - 1)
uint32_t inverse(int n) {
    return n == 1 ? 0xFFFFFFFFu : static_cast<uint32_t>((uint64_t(1) << 32) / n);
}

// M = 0 (a batch without tokens) is a valid problem of its own.
bool loss_shape_ok(int64_t M, int64_t d, int64_t V) {
    return M >= 0 && M <= (int64_t(1) << 30) && V >= 1 && V < (int64_t(1) << 31) - 512 && d >= 8 &&
           d <= (int64_t(1) << 24);
}

int32_t check_loss(const void *H, const void *W, const int32_t *targets, int64_t M, int64_t d,
                   int64_t V, int32_t reduction, float z_loss) {
    if (!W || (M > 0 && (!H || !targets)) || !loss_shape_ok(M, d, V) ||
        reduction < SB_REDUCE_NONE || reduction > SB_REDUCE_MEAN || !std::isfinite(z_loss))
        return SB_ERR_INVALID_ARG;
    if (d % 8 != 0 || !on(H, 16) || !on(W, 16) || !on(targets, 4)) return SB_ERR_ALIGNMENT;
    return SB_OK;
}

// Rows of G: up to kTwoPartRows rows are held in two bf16 parts (loss_grad.cu), the second ones
// from row `lo` on, which is the next multiple of an output box's 32 rows.  Up to 32 rows they
// cost nothing (both parts are one 64-wide reduction block of dW); at 64 rows they cost 7 % (4096 x
// 151,936, a step: 993 against 932 us when that was measured), and the roundings of that many
// targets average out.
constexpr int64_t kTwoPartRows = 32;
int64_t lo_row(int64_t M) { return M <= kTwoPartRows ? (M + 31) / 32 * 32 : 0; }
int64_t g_rows(int64_t M) { return M <= kTwoPartRows ? 2 * lo_row(M) : M; }

// How a backward call runs: the piece of the vocabulary, the split of the dH reduction, and the
// workspace.
struct Plan {
    int64_t piece, ldg;
    int splits;
    size_t g_off, h_off, part_off, total;
};

constexpr int64_t kPieceBytes = int64_t(256) << 20;  // of G, where the caller leaves the choice

// A block of work is one 256 x 256 tile over ATOMS * 64 of the reduction (0.34 us per 64 on one
// CTA pair); a dW tile costs at least its 128 KB of output, about six 64-blocks' time.
struct Work {
    int64_t kb, long_blocks, short_blocks, longs, shorts;
};
Work work_of(int64_t M, int64_t d, int64_t cols, bool with_dH, bool with_dW) {
    Work w;
    const int64_t rt = (M + 255) / 256, dt = (d + 255) / 256, ct = (cols + 255) / 256;
    const int atoms = loss_box_rows(static_cast<int>(rt)) / 64;
    w.kb = 64 * atoms;
    w.long_blocks = (cols + w.kb - 1) / w.kb;
    w.short_blocks = (g_rows(M) + w.kb - 1) / w.kb;
    if (w.short_blocks < 6 / atoms) w.short_blocks = 6 / atoms;
    w.longs = with_dH ? rt * dt : 0;
    w.shorts = with_dW ? ct * dt : 0;
    return w;
}

// Splits of the dH reduction: the smallest estimated time over both products.  Unsplit, few
// dH tiles of a long reduction leave most CTA pairs idle (16 rows, d = 5120: 20 tiles of 2374
// blocks for 76 pairs); every split adds its fp32 partial sums' traffic.  Of several row tiles
// the pairs without a dH unit can make it up with dW tiles, as both are bound by the tensor
// cores; of one row tile dH is bound by reading W, which wants all SMs, so its rounds count in
// full (64 rows, d = 4096, V = 151,936, both products: two splits on 32 pairs took 541 us when 19
// on all of them took 505).
int choose_splits(int64_t M, int64_t d, int64_t piece, bool with_dH, bool with_dW, int pairs) {
    if (!with_dH) return 1;
    const Work w = work_of(M, d, piece, with_dH, with_dW);
    int best = 1;
    double best_t = 0;
    for (int s = 1; s <= 64 && s <= w.long_blocks; ++s) {
        const int64_t blocks = (w.long_blocks + s - 1) / s;
        const int64_t rounds = (w.longs * s + pairs - 1) / pairs;
        const double dh = static_cast<double>(rounds * blocks);
        const double dw = static_cast<double>(w.shorts) * w.short_blocks / pairs;
        const double even = static_cast<double>(w.longs) * s * blocks / pairs + dw;
        double t = w.kb == 64 ? dh + dw : (dh > even ? dh : even);
        t *= 0.34 * static_cast<double>(w.kb) / 64;                     // us
        // the partial sums are written and read again, by a kernel of its own
        if (s > 1) t += 3 + 0.05 * s + static_cast<double>(s) * g_rows(M) * d * 8 / 6.8e6;
        if (s == 1 || t < best_t) {
            best = s;
            best_t = t;
        }
    }
    return best;
}

Plan plan_of(int64_t M, int64_t d, int64_t V, int64_t piece, bool with_dH, bool with_dW,
             int pairs) {
    Plan pl{};
    if (piece == 0) {
        const int64_t n = (2 * g_rows(M) * V + kPieceBytes - 1) / kPieceBytes;
        piece = (V + n - 1) / n;
    }
    pl.piece = piece < V ? (piece + 255) / 256 * 256 : V;
    if (pl.piece > V) pl.piece = V;
    pl.ldg = (pl.piece + 63) / 64 * 64;
    pl.splits = choose_splits(M, d, pl.piece, with_dH, with_dW, pairs);
    pl.g_off = 256;
    const size_t rows = static_cast<size_t>(g_rows(M));
    pl.h_off = pl.g_off + up256(rows * pl.ldg * 2);
    pl.part_off = pl.h_off + (with_dW ? up256(rows * d * 2) : 0);
    pl.total = pl.part_off;
    if (with_dH && (pl.splits > 1 || pl.piece < V || lo_row(M)))
        pl.total += up256(pl.splits * rows * d * 4);
    return pl;
}

}  // namespace

cudaError_t launch_loss_rows(const LossParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.M);
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rows_kernel, p);
}

}  // namespace sb

using namespace sb;

extern "C" {

size_t sb_cross_entropy_workspace_bytes(int64_t M, int64_t d, int64_t V) {
    if (!loss_shape_ok(M, d, V) || d % 8 != 0) return 0;
    if (M == 0) return 256;
    const size_t records = sb_workspace_bytes(M, V, 1, SB_TOKEN);
    return records ? records + up256(static_cast<size_t>(M) * 4) : 0;
}

int32_t sb_cross_entropy_forward(const void *H, const void *W, const int32_t *targets, int64_t M,
                                 int64_t d, int64_t V, int32_t ignore_index, int32_t reduction,
                                 float z_loss, float *loss, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    if (int32_t e = check_loss(H, W, targets, M, d, V, reduction, z_loss)) return e;
    const bool scalar = reduction != SB_REDUCE_NONE;
    if (((M > 0 || scalar) && !loss) || (M > 0 && !lse) || !workspace) return SB_ERR_INVALID_ARG;
    if (!on(loss, 4) || !on(lse, 4) || !on(workspace, 256)) return SB_ERR_ALIGNMENT;
    if (workspace_bytes < sb_cross_entropy_workspace_bytes(M, d, V))
        return SB_ERR_WORKSPACE_TOO_SMALL;
    if (int32_t e = device_sms_cc(nullptr, nullptr)) return e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (M == 0) {  // no rows: the sum (and the mean) of nothing is 0
        if (cudaMemsetAsync(workspace, 0, 256, st) != cudaSuccess ||
            (scalar && cudaMemsetAsync(loss, 0, 4, st) != cudaSuccess))
            return SB_ERR_CUDA;
        return SB_OK;
    }
    const size_t records = sb_workspace_bytes(M, V, 1, SB_TOKEN);
    LossParams p{};
    if (int32_t e = enqueue_target_records(H, W, targets, M, d, V, ignore_index, workspace,
                                           records, &p.ws, st))
        return e;
    p.M = static_cast<int>(M);
    p.V = static_cast<int>(V);
    p.T = sb_tiles_per_shard(M, V, 1);
    p.reduction = reduction;
    p.ignore_index = ignore_index;
    p.z_loss = z_loss;
    p.H = static_cast<const uint16_t *>(H);
    p.W = static_cast<const uint16_t *>(W);
    p.d = static_cast<int>(d);
    p.targets = targets;
    p.lse = lse;
    p.loss = loss;
    p.rows = scalar ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + records)
                    : loss;
    return launch_loss_rows(p, st) == cudaSuccess ? SB_OK : SB_ERR_CUDA;
}

size_t sb_cross_entropy_backward_workspace_bytes(int64_t M, int64_t d, int64_t V, int64_t piece,
                                                 int32_t with_dH, int32_t with_dW) {
    if (!loss_shape_ok(M, d, V) || d % 8 != 0 || piece < 0 || !(with_dH || with_dW)) return 0;
    if (M == 0) return 256;
    int sms = 0;
    if (device_sms_cc(&sms, nullptr) != SB_OK) return 0;
    return plan_of(M, d, V, piece, with_dH != 0, with_dW != 0, sms / 2).total;
}

int32_t sb_cross_entropy_backward(const void *H, const void *W, const int32_t *targets,
                                  const float *lse, const float *grad, int64_t M, int64_t d,
                                  int64_t V, int32_t ignore_index, int32_t reduction,
                                  float z_loss, int64_t piece, void *dH, void *dW,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    if (int32_t e = check_loss(H, W, targets, M, d, V, reduction, z_loss)) return e;
    if ((!dH && !dW) || (M > 0 && !lse) || !workspace || piece < 0) return SB_ERR_INVALID_ARG;
    if (!on(lse, 4) || !on(grad, 4) || !on(dH, 16) || !on(dW, 16) || !on(workspace, 256))
        return SB_ERR_ALIGNMENT;
    int sms = 0;
    if (int32_t e = device_sms_cc(&sms, nullptr)) return e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (M == 0) {  // no rows: dW is the empty sum
        if (workspace_bytes < 256) return SB_ERR_WORKSPACE_TOO_SMALL;
        if (cudaMemsetAsync(workspace, 0, 256, st) != cudaSuccess ||
            (dW && cudaMemsetAsync(dW, 0, static_cast<size_t>(V) * d * 2, st) != cudaSuccess))
            return SB_ERR_CUDA;
        return SB_OK;
    }
    const int pairs = sms / 2;
    const Plan pl = plan_of(M, d, V, piece, dH != nullptr, dW != nullptr, pairs);
    if (workspace_bytes < pl.total) return SB_ERR_WORKSPACE_TOO_SMALL;

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    LossGradParams p{};
    p.M = static_cast<int>(M);
    p.d = static_cast<int>(d);
    p.V = static_cast<int>(V);
    p.ldg = static_cast<int>(pl.ldg);
    p.lo = static_cast<int>(lo_row(M));
    p.g_rows = static_cast<int>(g_rows(M));
    p.row_tiles = static_cast<int>((M + 255) / 256);
    p.d_tiles = static_cast<int>((d + 255) / 256);
    p.row_tiles_inv = inverse(p.row_tiles);
    p.d_tiles_inv = inverse(p.d_tiles);
    p.splits = pl.splits;
    p.reduction = reduction;
    p.ignore_index = ignore_index;
    p.z_loss = z_loss;
    p.targets = targets;
    p.lse = lse;
    p.grad = grad;
    p.G = reinterpret_cast<uint16_t *>(ws + pl.g_off);
    p.H = static_cast<const uint16_t *>(H);
    p.W = static_cast<const uint16_t *>(W);
    p.part = reinterpret_cast<float *>(ws + pl.part_off);
    p.scale = reinterpret_cast<float *>(ws + 16);
    p.dH = static_cast<uint16_t *>(dH);
    p.dW = static_cast<uint16_t *>(dW);
    p.epoch_word = reinterpret_cast<uint32_t *>(ws);
    p.status = reinterpret_cast<unsigned long long *>(ws + 8);
    p.epoch = next_epoch();
    p.timeout_ns = wait_limit_ns();
    p.debug_stall = debug_stall();
    const int64_t most = (pl.piece + 255) / 256 * p.d_tiles +
                         static_cast<int64_t>(p.row_tiles) * p.d_tiles * p.splits;
    if (most >= (int64_t(1) << 31) ||
        (pl.piece + 255) / 256 * p.row_tiles >= (int64_t(1) << 31))
        return SB_ERR_INVALID_ARG;

    uint16_t *copy = dW ? reinterpret_cast<uint16_t *>(ws + pl.h_off) : nullptr;
    const int rows = loss_box_rows(p.row_tiles);
    // fewer rows of H than a box has: a box of as many (a multiple of the swizzle's eight)
    const int h_rows = M < rows ? static_cast<int>((M + 7) / 8 * 8) : rows;
    p.h_box_bytes = static_cast<uint32_t>(h_rows) * 128;
    LossGradMaps logits{}, operands{};  // maps of gradients not asked for are not used
    if (!encode_bf16_map(&logits.x, H, M, d, h_rows) || !encode_bf16_map(&logits.y, W, V, d, rows) ||
        !encode_bf16_map(&operands.z, copy ? copy : H, copy ? p.g_rows : M, d, rows) ||
        !encode_bf16_map(&operands.dw, dW ? dW : W, V, d, 32) ||
        !encode_bf16_map(&operands.dh, dH ? dH : H, M, d, 32))
        return SB_ERR_CUDA;
    operands.y = logits.y;
    int64_t mapped = 0;
    for (int64_t c0 = 0; c0 < V; c0 += pl.piece) {
        const int64_t cols = V - c0 < pl.piece ? V - c0 : pl.piece;
        // the map ends at the piece's last column: what lies past it reads as zero
        if (mapped != cols && (!encode_bf16_map(&operands.x, p.G, p.g_rows, cols, rows, pl.ldg) ||
                               !encode_bf16_map(&logits.g, p.G, p.g_rows, cols, 32, pl.ldg)))
            return SB_ERR_CUDA;
        mapped = cols;
        p.c0 = static_cast<int>(c0);
        p.cols = static_cast<int>(cols);
        p.first = c0 == 0;
        p.Hc = p.first ? copy : nullptr;
        p.last = c0 + cols == V;
        p.col_tiles = static_cast<int>((cols + 255) / 256);
        const Work w = work_of(M, d, cols, dH != nullptr, dW != nullptr);
        p.dh_units = static_cast<int>(w.longs * pl.splits);
        p.dw_units = static_cast<int>(w.shorts);
        p.fill = static_cast<int>(((w.long_blocks + pl.splits - 1) / pl.splits) / w.short_blocks);
        if (launch_loss_logits(logits, p, sms, st) != cudaSuccess ||
            launch_loss_operands(operands, p, sms, st) != cudaSuccess)
            return SB_ERR_CUDA;
    }
    if (dH && (pl.splits > 1 || p.lo) && launch_loss_sum(p, st) != cudaSuccess) return SB_ERR_CUDA;
    return SB_OK;
}

}  // extern "C"
