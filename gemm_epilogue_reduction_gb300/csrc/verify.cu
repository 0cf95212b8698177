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
// beside it; the blocks exchange their best through distributed shared memory.  Few columns of the
// scan can win: bounds of every score from both sides, without a logarithm, leave one or two columns
// of a warp's vectors whose score is formed.
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
constexpr int kLseBlocks = 152 * 16;  // that many pieces at least, where the rows are long enough
constexpr int kVerifyThreads = 512;
constexpr int kVerifyCluster = 8;      // blocks of a request
constexpr int kWideCluster = 16;       // the same for few requests, where the device allows it
constexpr int kWideRequests = 9;       // 9 x 16 blocks: one to an SM

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

__device__ __forceinline__ void unpack(uint4 x, float2 (&v)[4], __nv_bfloat16) {
    v[0] = unpack2(x.x), v[1] = unpack2(x.y), v[2] = unpack2(x.z), v[3] = unpack2(x.w);
}
__device__ __forceinline__ void unpack(uint4 x, float2 (&v)[2], float) {
    v[0] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
    v[1] = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
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
    const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf: adds nothing
    uint4 x[kLseAhead];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kLseAhead; ++k) {
            const int i = i0 + k * kLseThreads;
            x[k] = i < v1 ? vec[i] : make_uint4(none, none, none, none);
        }
    };
    int i0 = v0 + static_cast<int>(threadIdx.x);
    load(i0);
    while (i0 < v1) {
        float2 v[kLseAhead][E / 2];
        float top[kLseAhead];
#pragma unroll
        for (int k = 0; k < kLseAhead; ++k) {
            unpack(x[k], v[k], T{});
            top[k] = fmaxf(v[k][0].x, v[k][0].y);
#pragma unroll
            for (int j = 1; j < E / 2; ++j) top[k] = fmaxf(top[k], fmaxf(v[k][j].x, v[k][j].y));
        }
        i0 += kLseThreads * kLseAhead;
        load(i0);  // the next ones are on their way meanwhile
        float m = a.m;
#pragma unroll
        for (int k = 0; k < kLseAhead; ++k) m = fmaxf(m, top[k]);
        const float ref = m == -INFINITY ? 0.f : m;
        float2 sum[2] = {make_float2(a.s * ex2_approx((a.m - ref) * c), 0.f), both(0.f)};
#pragma unroll
        for (int k = 0; k < kLseAhead; ++k)
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const float2 y = __fmul2_rn(__fadd2_rn(v[k][j], both(-ref)), both(c));
                sum[j & 1] = __fadd2_rn(sum[j & 1], make_float2(ex2_approx(y.x), ex2_approx(y.y)));
            }
        a.m = m;
        a.s = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
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
    // log s = e ln 2 + log f with s = f·2^e, f in [1, 2): in fp32 log s would be off by its own ulp
    const uint32_t bits = __float_as_uint(a.s);
    const int e = static_cast<int>((bits >> 23) & 255) - 127;  // s is 1 at least, but for roundings
    const float f = __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u);
    if (!(a.s > 0.f && a.s < INFINITY)) return static_cast<double>(a.m) * p.inv_t + a.s;  // not finite
    return static_cast<double>(a.m) * p.inv_t + (e * 0.69314718055994531 + logf(f));
}

// Whether e^x > u, for x whose rounding to fp32 would count.
__device__ __forceinline__ bool exp_above(double x, float u) {
    const float hi = static_cast<float>(x), e = expf(hi);
    if (!(e > 0.f && e < INFINITY)) return e > u;
    return fmaf(e, static_cast<float>(x - hi), e) > u;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// One row's scan: what a sample is drawn from, this thread's best so far, and what a column has to reach
// (a lower bound of the best score that the warp has seen).
template <typename T, int FROM>
struct Scan {
    const VerifyParams &p;
    const T *z, *q;
    float lse, qlse;
    int x;
    unsigned long long first;  // index of the row's first draw
    float best, bar;
    int column;

    __device__ __forceinline__ float weight(float a, float b, int j) const {
        float w = ex2_approx(fmaf(a, p.inv_t, -lse) * kLog2e);
        if (FROM == kDifference) w -= ex2_approx(fmaf(b, p.inv_t, -qlse) * kLog2e);
        if (FROM == kWithout && j == x) w = 0.f;
        return w;
    }
    __device__ __forceinline__ void exact(int j) {
        const uint32_t bits = bits24_from_state(splitmix_state(p.seed, first + j));
        const float score =
            bits ? weight(one(z + j), FROM == kDifference ? one(q + j) : 0.f, j) / -log2_uniform(bits) : 0.f;
        // columns come in any order: of equal scores the lowest stays
        if (score > best || (score == best && j < column)) best = score, column = j;
    }
    // N columns of each thread of the warp, with their logits: j, j + STEP, ...; `have` of them count.
    template <int N, int STEP>
    __device__ __forceinline__ void columns(const float (&a)[N], const float (&b)[N], int j, int have) {
        float bound[N], low = 0.f;
        const unsigned long long state = splitmix_state(p.seed, first + j);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float w = weight(a[k], b[k], j + k * STEP);
            const uint32_t bits = bits24_from_state(state + static_cast<unsigned long long>(k * STEP) * kGolden);
            // With l = 1 - u:  l <= -ln u <= l / (1 - l), so the score w / -log2 u lies between
            // w·ln 2 / l and that times 1 - l.  The constants leave room for the roundings of both and
            // of the score itself (2e-6 and 4e-6 against some 1e-6).
            const float l = static_cast<float>(16777216u - bits) * 5.9604644775390625e-8f;
            const float top = k < have ? w * 0.69314860f * rcp_approx(l) : 0.f;
            bound[k] = top;
            low = fmaxf(low, top * fmaf(l, -0.999994f, 0.999994f));
        }
        const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(low));  // (low >= 0)
        bar = fmaxf(bar, __uint_as_float(most));
        uint32_t promising = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) promising |= static_cast<uint32_t>(bound[k] > bar) << k;
        for (; promising; promising &= promising - 1) exact(j + (__ffs(promising) - 1) * STEP);
    }
};

// This thread's best of the share of block `rank` of `blocks`.
template <typename T, int FROM>
__device__ __forceinline__ unsigned long long scan(const VerifyParams &p, const T *z, const T *q,
                                                   float lse, float qlse, int x,
                                                   unsigned long long first, int rank, int blocks) {
    constexpr int E = 16 / sizeof(T);
    const int tid = threadIdx.x;
    Scan<T, FROM> s{p, z, q, lse, qlse, x, first, 0.f, 0.f, 0};
    const uintptr_t off = reinterpret_cast<uintptr_t>(z) & 15;
    if (FROM != kDifference || off == (reinterpret_cast<uintptr_t>(q) & 15)) {
        const int head = min(p.V, static_cast<int>((16 - off) & 15) / static_cast<int>(sizeof(T)));
        const int nv = (p.V - head) / E, tail = head + nv * E;
        const int v0 = static_cast<int>(static_cast<long long>(nv) * rank / blocks);
        const int v1 = static_cast<int>(static_cast<long long>(nv) * (rank + 1) / blocks);
        const uint4 *za = reinterpret_cast<const uint4 *>(z + head);
        const uint4 *qa = reinterpret_cast<const uint4 *>(q + head);
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (v0 + tid < v1) {
            a = za[v0 + tid];
            if (FROM == kDifference) b = qa[v0 + tid];
        }
        for (int i0 = v0; i0 < v1; i0 += kVerifyThreads) {  // (the same turns for all threads)
            const int i = i0 + tid, next = i + kVerifyThreads;
            float2 pa[E / 2], pb[E / 2];
            unpack(a, pa, T{});
            unpack(b, pb, T{});
            if (next < v1) {
                a = za[next];
                if (FROM == kDifference) b = qa[next];
            }
            float va[E], vb[E];
#pragma unroll
            for (int j = 0; j < E / 2; ++j)
                va[2 * j] = pa[j].x, va[2 * j + 1] = pa[j].y, vb[2 * j] = pb[j].x, vb[2 * j + 1] = pb[j].y;
            s.template columns<E, 1>(va, vb, head + i * E, i < v1 ? E : 0);
        }
        if (rank == 0 && tid < head) s.exact(tid);
        if (rank == blocks - 1 && tid < p.V - tail) s.exact(tail + tid);
    } else {
        // rows of an odd vocabulary: z's and q's vectors never lie side by side
        constexpr int W = 8;
        const int c0 = static_cast<int>(static_cast<long long>(p.V) * rank / blocks);
        const int c1 = static_cast<int>(static_cast<long long>(p.V) * (rank + 1) / blocks);
        for (int j0 = c0; j0 < c1; j0 += W * kVerifyThreads) {
            const int j = j0 + tid;
            float a[W], b[W];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const int i = min(j + k * kVerifyThreads, c1 - 1);
                a[k] = one(z + i);
                b[k] = one(q + i);
            }
            s.template columns<W, kVerifyThreads>(a, b, j,
                                                  max(0, (c1 - j + kVerifyThreads - 1) / kVerifyThreads));
        }
    }
    return pack(s.best, s.column);
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
                stays = exp_above(l - m, p.u[r]);
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
    const unsigned long long first = static_cast<unsigned long long>(r) * static_cast<unsigned>(p.V);
    const float lse = static_cast<float>(end_lse), qlse = static_cast<float>(end_qlse);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    unsigned long long best = 0;
    for (int turn = 0; turn < 2 && !best; ++turn) {
        // a difference that is nowhere positive (p and q equal but for roundings): p itself
        if (turn == 0 && known && q)
            best = scan<T, kDifference>(p, z, q + static_cast<size_t>(e) * p.V, lse, qlse, x, first, rank, blocks);
        else if (turn == 0 && known)
            best = scan<T, kWithout>(p, z, nullptr, lse, 0.f, x, first, rank, blocks);
        else
            best = scan<T, kTarget>(p, z, nullptr, lse, 0.f, x, first, rank, blocks);
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
    auto config = [&](int blocks, cudaLaunchAttribute (&attr)[2]) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(static_cast<unsigned>(p.B > 0 ? p.B : 1) * blocks);
        cfg.blockDim = dim3(kVerifyThreads);
        cfg.stream = st;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = blocks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cfg;
    };
    cudaLaunchAttribute attr[2];
    int blocks = kVerifyCluster;
    if (p.B <= kWideRequests) {
        // more than eight blocks to a cluster are no part of the portable model: asked once a device
        static std::atomic<uint64_t> asked{0}, allowed{0};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
        if (bit && !(asked.load() & bit)) {
            int clusters = 0;
            cudaLaunchConfig_t cfg = config(kWideCluster, attr);
            cfg.numAttrs = 1;
            e = cudaFuncSetAttribute(verify_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, verify_kernel<T>, &cfg);
            if (e == cudaSuccess && clusters > 0) allowed.fetch_or(bit);
            cudaGetLastError();  // a refusal is an answer here
            asked.fetch_or(bit);
        }
        if (allowed.load() & bit) blocks = kWideCluster;
    }
    const cudaLaunchConfig_t cfg = config(blocks, attr);
    return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p);
}

// Pieces of a row: enough blocks for the GPU to be full several times over, but no piece that a
// block has hardly begun with before it ends.
int splits_of(int64_t rows, int64_t V) {
    if (rows < 1) return 1;
    int64_t s = (kLseBlocks + rows - 1) / rows;
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
    if (parts > rows + kLseBlocks) parts = rows + kLseBlocks;
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
