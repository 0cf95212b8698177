// verify.cu -- which of a small model's drafted tokens the head's distribution keeps.
//
// Row r of a request has the target's distribution p = softmax(z_r / T) and, but for the request's
// last row, a drafted token x and the distribution q that it was drawn from (or none: then q is 1
// at x).  With the given uniform u_r the draft stays if u_r < p(x) / q(x).  The first one that does
// not is replaced by a sample of max(p - q, 0) (p without x where there is no q), and where all
// stay the last row adds a sample of its p; either way the tokens are distributed as the target's
// own (Leviathan, Kalman and Matias, ICML 2023).  The sample is the column with the largest w / E,
// E = -log2 u_rj with the 24-bit uniform at index r*V + j of the seed's stream: the Gumbel-max
// choice of sb_lmhead_project's SB_GUMBEL_TOKEN with the logarithms taken away, which differences
// of probabilities would not survive.
//
// lse_kernel: per (row, piece of the vocabulary) the maximum and the sum of exponentials; bound by
// reading the logits.  Skipped where the caller has the logsumexp (the head's projection returns
// it).  verify_kernel: a cluster of blocks per request.  Every block joins the rows' pieces and
// decides for itself, then scans its share of the one row that a sample is drawn from, with q's
// beside it; the blocks exchange their best through distributed shared memory.  Most columns of
// the scan cannot win and do not compute a logarithm: -ln u >= 1 - u, so w·ln 2 / (1 - u), which
// takes one product each way, bounds the score from above.
#include <cmath>

#include "norm_common.cuh"
#include "sb.h"
#include "sb_counter.cuh"
#include "sb_gumbel.cuh"
#include "sb_pipe.cuh"

namespace sb {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kLseThreads = 256;
constexpr int kLseAhead = 4;         // 16-byte vectors in flight
constexpr int kLsePiece = 4096;      // fewest columns of a piece
constexpr int kVerifyThreads = 512;
constexpr int kVerifyCluster = 8;

struct VerifyParams {
    const void *z, *q;
    const int32_t *drafts, *starts;
    const float *u, *lse, *qlse;
    int R, B, V, Rd;
    int with_q;         // drafts have distributions of their own
    int zrows, qrows;   // of them, how many lse_kernel reduces
    int splits;
    float inv_t;
    unsigned long long seed;
    int32_t *token, *accepted;
    float *logprob;
    float2 *part;       // [zrows + qrows][splits] (max, sum of exponentials relative to it)
    uint32_t *epoch_word;
    unsigned long long *status;
    uint32_t epoch;
};

struct MaxSum {
    float m, s;
};
// c: 1/T times log2(e).  -inf maxima (nothing seen) carry s = 0.
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return MaxSum{m, a.s + b.s};
    return MaxSum{m, a.s * ex2_approx((a.m - m) * c) + b.s * ex2_approx((b.m - m) * c)};
}
__device__ __forceinline__ MaxSum warp_join(MaxSum a, float c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a = join(a, MaxSum{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o)}, c);
    return a;
}

__device__ __forceinline__ void unpack(uint4 x, float (&v)[8], __nv_bfloat16) {
    const float2 a = unpack2(x.x), b = unpack2(x.y), c = unpack2(x.z), d = unpack2(x.w);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
}
__device__ __forceinline__ void unpack(uint4 x, float (&v)[4], float) {
    v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y);
    v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
}

template <typename T>
__global__ void __launch_bounds__(kLseThreads) lse_kernel(const VerifyParams p) {
    constexpr int E = 16 / sizeof(T);
    __shared__ float sm[kLseThreads / 32], ss[kLseThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int row = blockIdx.x / p.splits, split = blockIdx.x - row * p.splits;
    const bool draft = row >= p.zrows;
    const int at = draft ? row - p.zrows : row;
    if (at >= p.starts[p.B]) return;  // behind the last request
    const T *from = static_cast<const T *>(draft ? p.q : p.z) + static_cast<size_t>(at) * p.V;
    const float c = p.inv_t * kLog2e;
    // whole 16-byte vectors, and the values before and behind them
    const int head = min(p.V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(from) & 15)) & 15) /
                                  static_cast<int>(sizeof(T)));
    const int nv = (p.V - head) / E;
    const int v0 = static_cast<int>(static_cast<long long>(nv) * split / p.splits);
    const int v1 = static_cast<int>(static_cast<long long>(nv) * (split + 1) / p.splits);
    const uint4 *vec = reinterpret_cast<const uint4 *>(from + head);
    MaxSum a{-INFINITY, 0.f};
    if (split == 0) {
        const int tail = p.V - head - nv * E, i = threadIdx.x;
        if (i < head) a = MaxSum{one(from + i), 1.f};
        if (i >= 32 && i - 32 < tail) a = MaxSum{one(from + head + nv * E + i - 32), 1.f};
        if (a.m == -INFINITY) a.s = 0.f;
    }
    for (int i0 = v0 + static_cast<int>(threadIdx.x); i0 < v1; i0 += kLseThreads * kLseAhead) {
        uint4 x[kLseAhead];
#pragma unroll
        for (int k = 0; k < kLseAhead; ++k) {
            const int i = i0 + k * kLseThreads;
            x[k] = i < v1 ? vec[i] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kLseAhead; ++k) {
            if (i0 + k * kLseThreads >= v1) break;
            float v[E];
            unpack(x[k], v, T{});
            float m = a.m;
#pragma unroll
            for (int j = 0; j < E; ++j) m = fmaxf(m, v[j]);
            if (m > a.m) {  // (not at all while every value is -inf)
                a.s *= ex2_approx((a.m - m) * c);
                a.m = m;
            }
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int j = 0; j < E; ++j) a.s += ex2_approx((v[j] - ref) * c);
        }
    }
    a = warp_join(a, c);
    if ((threadIdx.x & 31) == 0) {
        sm[threadIdx.x >> 5] = a.m;
        ss[threadIdx.x >> 5] = a.s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kLseThreads / 32; ++w) a = join(a, MaxSum{sm[w], ss[w]}, c);
        p.part[blockIdx.x] = make_float2(a.m, a.s);
    }
}

// The logsumexp of row `at` of the target (or the draft), by a warp.
__device__ double row_lse(const VerifyParams &p, bool draft, int at, int lane) {
    const float *given = draft ? p.qlse : p.lse;
    if (given) return given[at];
    const float c = p.inv_t * kLog2e;
    const float2 *part = p.part + (static_cast<size_t>(draft ? p.zrows : 0) + at) * p.splits;
    MaxSum a{-INFINITY, 0.f};
    for (int s = lane; s < p.splits; s += 32) a = join(a, MaxSum{part[s].x, part[s].y}, c);
    a = warp_join(a, c);
    if (a.m == -INFINITY && a.s == 0.f) return -INFINITY;
    return static_cast<double>(a.m) * p.inv_t + log(static_cast<double>(a.s));
}

__device__ __forceinline__ uint32_t cluster_blocks() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}

// Score (as bits: it is not negative) over the inverted column, so that the larger word is the
// larger score, and of equal ones the lower column; 0: no column.
__device__ __forceinline__ unsigned long long pack(float score, int column) {
    return score > 0.f ? (static_cast<unsigned long long>(__float_as_uint(score)) << 32) |
                             static_cast<uint32_t>(~column)
                       : 0ull;
}

enum : int { kTarget = 0, kDifference = 1, kWithout = 2 };  // what a sample is drawn from

// This thread's best of columns [c0, c1).
template <typename T, int FROM>
__device__ __forceinline__ unsigned long long scan(const VerifyParams &p, const T *z, const T *q,
                                                   float lse, float qlse, int x,
                                                   unsigned long long first, int c0, int c1) {
    constexpr int U = 4;
    float best = 0.f;
    int column = 0;
    for (int j0 = c0 + static_cast<int>(threadIdx.x); j0 < c1; j0 += U * kVerifyThreads) {
        float a[U], b[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int j = j0 + k * kVerifyThreads;
            a[k] = j < c1 ? one(z + j) : -INFINITY;
            b[k] = FROM == kDifference && j < c1 ? one(q + j) : -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int j = j0 + k * kVerifyThreads;
            float w = ex2_approx(fmaf(a[k], p.inv_t, -lse) * kLog2e);
            if (FROM == kDifference) w -= ex2_approx(fmaf(b[k], p.inv_t, -qlse) * kLog2e);
            if (FROM == kWithout && j == x) w = 0.f;
            const uint32_t bits = bits24_from_state(splitmix_state(p.seed, first + j));
            // an upper bound of the score: -ln u >= 1 - u
            const float left = static_cast<float>(16777216u - bits) * 5.9604644775390625e-8f;
            if (w * 0.69314790f > best * left && j < c1 && bits != 0) {  // ln 2 and its rounding
                const float score = w / -log2_uniform(bits);
                if (score > best) {
                    best = score;
                    column = j;
                }
            }
        }
    }
    return pack(best, column);
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p) {
    __shared__ int end, busy;
    __shared__ double end_lse, end_qlse;
    __shared__ unsigned long long bests[2][16], warps[kVerifyThreads / 32];
    const int blocks = static_cast<int>(cluster_blocks()), rank = static_cast<int>(cluster_ctarank());
    const int b = static_cast<int>(blockIdx.x) / blocks;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    // the peers run before anything is written into their shared memory
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int total = p.B ? p.starts[p.B] : 0;
    if (blockIdx.x == 0 && tid == 0) *p.epoch_word = p.epoch;
    if (b == (p.B ? p.B - 1 : 0) && total >= 0)  // the rows behind the last request
        for (long long r = total + static_cast<long long>(rank) * kVerifyThreads + tid; r < p.R;
             r += static_cast<long long>(blocks) * kVerifyThreads) {
            p.token[r] = -1;
            if (p.logprob) p.logprob[r] = 0.f;
        }
    const int s0 = p.B ? p.starts[b] : 0, s1 = p.B ? p.starts[b + 1] : 0;
    // draft rows are those of the requests before this one that have any rows
    if (tid == 0) busy = 0;
    __syncthreads();
    int mine = 0;
    for (int i = tid; i < b; i += kVerifyThreads) mine += p.starts[i + 1] > p.starts[i];
    if (mine) atomicAdd(&busy, mine);
    const int n = static_cast<int>(static_cast<unsigned>(s1) - static_cast<unsigned>(s0) - 1u);
    if (tid == 0) end = n;
    __syncthreads();
    const int q0 = s0 - busy;  // the draft's row of row s0
    const bool sane = s0 >= 0 && s1 >= s0 && s1 <= total && total <= p.R &&
                      (!p.with_q || n <= 0 || (q0 >= 0 && q0 + n <= p.Rd));
    if (!sane && tid == 0 && rank == 0) record_status(p.status, p.epoch, 1u);  // SB_ERR_INVALID_ARG
    if (!sane || n < 0) {  // the same for all blocks of the cluster
        if (p.B && tid == 0 && rank == 0) p.accepted[b] = sane ? 0 : -1;
        __syncwarp();
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        return;
    }
    const T *z = static_cast<const T *>(p.z) + static_cast<size_t>(s0) * p.V;
    const T *q = p.with_q && n > 0 ? static_cast<const T *>(p.q) + static_cast<size_t>(q0) * p.V : nullptr;
    // which drafts stay
    for (int i = warp; i < n; i += kVerifyThreads / 32) {
        const int r = s0 + i, x = p.drafts[r];
        const double lse = row_lse(p, false, r, lane), qlse = q ? row_lse(p, true, q0 + i, lane) : 0.0;
        if (lane == 0) {
            bool stays = false;
            float lp = 0.f;
            if (x >= 0 && x < p.V) {
                const double l = static_cast<double>(one(z + static_cast<size_t>(i) * p.V + x) * p.inv_t) - lse;
                const double m = q ? static_cast<double>(one(q + static_cast<size_t>(i) * p.V + x) * p.inv_t) - qlse : 0.0;
                lp = static_cast<float>(l);
                stays = exp(l - m) > static_cast<double>(p.u[r]);
            } else if (rank == 0) {
                record_status(p.status, p.epoch, 1u);
            }
            if (!stays) atomicMin(&end, i);
            if (rank == 0) {  // (of a row behind the end it is taken back below)
                p.token[r] = x;
                if (p.logprob) p.logprob[r] = lp;
            }
        }
    }
    __syncthreads();
    const int e = end, r = s0 + e;
    if (warp == 0) {
        const double l = row_lse(p, false, r, lane);
        const double m = q && e < n ? row_lse(p, true, q0 + e, lane) : 0.0;
        if (lane == 0) end_lse = l, end_qlse = m;
    }
    __syncthreads();
    z += static_cast<size_t>(e) * p.V;
    const int x = e < n ? p.drafts[r] : -1;
    const bool known = x >= 0 && x < p.V;  // otherwise nothing is taken off p
    const int c0 = static_cast<int>(static_cast<long long>(p.V) * rank / blocks);
    const int c1 = static_cast<int>(static_cast<long long>(p.V) * (rank + 1) / blocks);
    const unsigned long long first = static_cast<unsigned long long>(r) * static_cast<unsigned>(p.V);
    const float lse = static_cast<float>(end_lse), qlse = static_cast<float>(end_qlse);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    unsigned long long best = 0;
    for (int turn = 0; turn < 2 && !best; ++turn) {
        // a difference that is nowhere positive (p and q equal but for roundings): p itself
        if (turn == 0 && known && q)
            best = scan<T, kDifference>(p, z, q + static_cast<size_t>(e) * p.V, lse, qlse, x, first, c0, c1);
        else if (turn == 0 && known)
            best = scan<T, kWithout>(p, z, nullptr, lse, 0.f, x, first, c0, c1);
        else
            best = scan<T, kTarget>(p, z, nullptr, lse, 0.f, x, first, c0, c1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long other = __shfl_xor_sync(0xFFFFFFFFu, best, o);
            best = other > best ? other : best;
        }
        if (lane == 0) warps[warp] = best;
        __syncthreads();
        if (tid < blocks) {
            for (int w = 0; w < kVerifyThreads / 32; ++w) best = warps[w] > best ? warps[w] : best;
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_rank(&bests[turn][rank], tid)),
                         "l"(best)
                         : "memory");
        }
        __syncwarp();
        cluster_sync();
        best = 0;
        for (int k = 0; k < blocks; ++k) best = bests[turn][k] > best ? bests[turn][k] : best;
    }
    if (rank != 0) return;
    for (int i = e + tid; i <= n; i += kVerifyThreads) {
        int token = -1;
        float lp = 0.f;
        if (i == e) {
            lp = __uint_as_float(0x7FC00000u);  // no column of the row has any probability
            if (best) {
                token = ~static_cast<int>(static_cast<uint32_t>(best));
                lp = static_cast<float>(static_cast<double>(one(z + token) * p.inv_t) - end_lse);
            }
        }
        p.token[s0 + i] = token;
        if (p.logprob) p.logprob[s0 + i] = lp;
    }
    if (tid == 0) p.accepted[b] = e;
}

// The same where the target's own choice of each row is known: a draft stays while it is that.
struct GreedyParams {
    const int32_t *target, *drafts, *starts;
    int R, B;
    int32_t *token, *accepted;
};
__global__ void __launch_bounds__(128) greedy_kernel(const GreedyParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, b = blockIdx.x * 4 + threadIdx.x / 32;
    const int total = p.B ? p.starts[p.B] : 0;
    if (b == (p.B ? p.B - 1 : 0) && total >= 0)
        for (long long r = static_cast<long long>(total) + lane; r < p.R; r += 32) p.token[r] = -1;
    if (b >= p.B) return;
    const int s0 = p.starts[b], s1 = p.starts[b + 1];
    if (s0 < 0 || s1 < s0 || s1 > total || total > p.R) {
        if (lane == 0) p.accepted[b] = -1;
        return;
    }
    const int n = s1 - s0;  // rows
    int e = n;
    for (int i0 = 0; i0 < n && e == n; i0 += 32) {
        const int i = i0 + lane;
        const bool stops = i < n && (i == n - 1 || p.drafts[s0 + i] != p.target[s0 + i]);
        const uint32_t where = __ballot_sync(0xFFFFFFFFu, stops);
        if (where) e = i0 + __ffs(where) - 1;
    }
    for (int i = lane; i < n; i += 32) p.token[s0 + i] = i <= e ? p.target[s0 + i] : -1;
    if (lane == 0) p.accepted[b] = n ? e : 0;
}

template <typename T>
cudaError_t launch_verify(const VerifyParams &p, cudaStream_t st) {
    const long long rows = static_cast<long long>(p.zrows) + p.qrows;
    if (rows > 0 && p.B > 0) {
        const cudaError_t e = launch_dependent(lse_kernel<T>, dim3(static_cast<unsigned>(rows * p.splits)),
                                               kLseThreads, 0, p, st);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B > 0 ? p.B : 1) * kVerifyCluster);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kVerifyCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p);
}

// Pieces of a row: enough blocks for the GPU to be full several times over, but no piece that a
// block has hardly begun with before it ends.
int splits_of(int64_t rows, int64_t V) {
    if (rows < 1) return 1;
    int64_t s = (152 * 8 + rows - 1) / rows;
    const int64_t most = (V + kLsePiece - 1) / kLsePiece;
    if (s > most) s = most;
    return static_cast<int>(s < 1 ? 1 : s);
}

bool verify_sizes(int64_t R, int64_t draft_rows, int64_t V) {
    return R >= 0 && R < (int64_t(1) << 24) && draft_rows >= -1 && draft_rows < (int64_t(1) << 24) &&
           V >= 1 && V < (int64_t(1) << 31) - 65536;
}

}  // namespace
}  // namespace sb

using namespace sb;

extern "C" {

size_t sb_verify_workspace_bytes(int64_t R, int64_t draft_rows, int64_t V) {
    if (!verify_sizes(R, draft_rows, V)) return 0;
    // the number of pieces falls with the rows that are reduced: the largest product of the two
    const int64_t rows = R + (draft_rows > 0 ? draft_rows : 0), most = (V + kLsePiece - 1) / kLsePiece;
    int64_t parts = rows * most;
    if (parts > rows + 152 * 8) parts = rows + 152 * 8;
    return 256 + up256(static_cast<size_t>(parts) * 8);
}

int32_t sb_verify_drafts(const void *logits, const void *draft_logits, const int32_t *drafts,
                         const int32_t *starts, const float *uniforms, const float *lse,
                         const float *draft_lse, int64_t R, int64_t draft_rows, int64_t B,
                         int64_t V, int32_t logits_type, float temperature, uint64_t seed,
                         int32_t *token, int32_t *accepted, float *token_logprob, void *workspace,
                         size_t workspace_bytes, void *stream) {
    if (!verify_sizes(R, draft_rows, V) || B < 0 || B > (int64_t(1) << 24) ||
        logits_type < SB_BF16 || logits_type > SB_F32 ||
        !(std::isfinite(temperature) && temperature > 0.f) ||
        !std::isfinite(1.f / temperature) || (R > 0 && (!logits || !drafts || !uniforms || !token)) ||
        (B > 0 && (!starts || !accepted)) || (draft_rows > 0 && !draft_logits) || !workspace)
        return SB_ERR_INVALID_ARG;
    const uintptr_t za = logits_type == SB_F32 ? 4 : 2;
    if (!on(logits, za) || !on(draft_logits, za) || !on(drafts, 4) || !on(starts, 4) ||
        !on(uniforms, 4) || !on(lse, 4) || !on(draft_lse, 4) || !on(token, 4) || !on(accepted, 4) ||
        !on(token_logprob, 4) || !on(workspace, 256))
        return SB_ERR_ALIGNMENT;
    if (int32_t e = device_sms_cc(nullptr, nullptr)) return e;
    if (workspace_bytes < sb_verify_workspace_bytes(R, draft_rows, V)) return SB_ERR_WORKSPACE_TOO_SMALL;
    if (R == 0 && B == 0) return SB_OK;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    VerifyParams p{};
    p.z = logits;
    p.q = draft_logits;
    p.with_q = draft_rows >= 0;
    p.drafts = drafts;
    p.starts = starts;
    p.u = uniforms;
    p.lse = lse;
    p.qlse = draft_lse;
    p.R = static_cast<int>(R);
    p.B = static_cast<int>(B);
    p.V = static_cast<int>(V);
    p.Rd = draft_rows > 0 ? static_cast<int>(draft_rows) : 0;
    p.zrows = lse ? 0 : p.R;
    p.qrows = draft_lse ? 0 : p.Rd;
    p.splits = splits_of(static_cast<int64_t>(p.zrows) + p.qrows, V);
    p.inv_t = 1.0f / temperature;
    p.seed = seed;
    p.token = token;
    p.accepted = accepted;
    p.logprob = token_logprob;
    p.part = reinterpret_cast<float2 *>(ws + 256);
    p.epoch_word = reinterpret_cast<uint32_t *>(ws);
    p.status = reinterpret_cast<unsigned long long *>(ws + 8);
    p.epoch = next_epoch();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (logits_type == SB_BF16 ? launch_verify<__nv_bfloat16>(p, st) : launch_verify<float>(p, st)) ==
                   cudaSuccess
               ? SB_OK
               : SB_ERR_CUDA;
}

int32_t sb_verify_greedy(const int32_t *target, const int32_t *drafts, const int32_t *starts,
                         int64_t R, int64_t B, int32_t *token, int32_t *accepted, void *stream) {
    if (R < 0 || R >= (int64_t(1) << 31) - 65536 || B < 0 || B > (int64_t(1) << 24) ||
        (R > 0 && (!target || !drafts || !token)) || (B > 0 && (!starts || !accepted)))
        return SB_ERR_INVALID_ARG;
    if (!on(target, 4) || !on(drafts, 4) || !on(starts, 4) || !on(token, 4) || !on(accepted, 4))
        return SB_ERR_ALIGNMENT;
    if (int32_t e = device_sms_cc(nullptr, nullptr)) return e;
    if (R == 0 && B == 0) return SB_OK;
    const GreedyParams p{target, drafts, starts, static_cast<int>(R), static_cast<int>(B), token, accepted};
    return launch_dependent(greedy_kernel, dim3(static_cast<unsigned>((B > 0 ? B : 1) + 3) / 4), 128, 0, p,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SB_OK
               : SB_ERR_CUDA;
}

}  // extern "C"
