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
// lse_kernel: the maxima and sums of exponentials of the rows, where the caller has not got their
// logsumexps (the head's projection returns them); bound by reading the logits.  All rows' vectors
// are one sequence, cut into equal pieces for kLseBlocks blocks, whatever the number of rows and their
// length (a block per row, or per part of one, took 36 us for 576 rows of 151,936 in waves that did
// not fill the GPU).  verify_kernel: a cluster of blocks per request.  Every block joins the rows'
// pieces and decides for itself which drafts stay, then scans its share of the one row that a sample
// is drawn from, with q's beside it; the blocks exchange their best through distributed shared
// memory.  Few columns of the scan can win: bounds of every score from both sides, without a
// logarithm, leave one or two columns of a warp's vectors whose score is formed.  (One kernel for
// both, each cluster with its own request's rows, took 108 us for 64 requests of 1 to 9 rows: the
// long ones come last.)
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
constexpr int kLseBlocks = 152 * 4;    // as many as fit 152 SMs at a time (the workspace's size goes by it)
constexpr int kAhead = 4;               // 16-byte vectors of a thread in flight
constexpr int kVerifyThreads = 512;
// Blocks of a request's cluster: as many as leave all blocks on the GPU at a time, two to an SM (64
// requests, when that was measured: 4 blocks 62 us, 8 in two turns 71, 8 of 256 threads 64); 16 where
// they have an SM each and the device allows such clusters.
constexpr int kWideBlocks = 16, kMostBlocks = 8, kLeastBlocks = 2;
// Which draft row is a request's first depends on how many requests in front of it have rows.  A cluster
// counts them itself; of more than this many it counts its own share's, and count_kernel has counted the
// shares in front (4096 requests: 78 us either way; 8192: 131 -> 127; 16,384: 258 -> 217, shares of 8192 240;
// 262,144: 18.4 ms -> 3).
constexpr int kCountRequests = 2048, kCountThreads = 512;
constexpr int64_t kMostRequests = int64_t(1) << 24;

struct VerifyParams {
    const void *z, *q;
    const int32_t *drafts, *starts;
    const float *u, *lse, *qlse;
    int R, B, V, Rd;
    int zrows, qrows;   // of them, how many lse_kernel reduces (those behind the last request aside)
    int with_q;         // drafts have distributions of their own
    float t, inv_t;
    unsigned long long seed;
    const unsigned long long *seed_offset;  // added to it (null: 0), read when the kernel runs
    int32_t *token, *accepted;
    float *logprob;
    float2 *part;       // MaxSum, see Pieces
    int *counts;        // of kCountRequests requests each, how many have rows (null: not counted)
    uint32_t *epoch_word;
    unsigned long long *status;
    uint32_t epoch;
};

// The largest logit m and the sum s of 2^((v - m)·c) with c = 1/T·log2(e), so that the largest one's term is
// exactly 1.  m = -inf where nothing has been seen (s is then 0, or no number).
struct MaxSum {
    float m, s;
};
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
    const float m = fmaxf(a.m, b.m), ref = m == -INFINITY ? 0.f : m;
    return MaxSum{m, a.s * ex2_approx((a.m - ref) * c) + b.s * ex2_approx((b.m - ref) * c)};
}
__device__ __forceinline__ MaxSum warp_join(MaxSum a, float c) {
    // (a maximum that is no number is none: its sum says so)
    const float m = ordered_to_float(
        __reduce_max_sync(0xFFFFFFFFu, float_to_ordered(a.m == a.m ? a.m : -INFINITY)));
    a.s *= ex2_approx((a.m - (m == -INFINITY ? 0.f : m)) * c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a.s += __shfl_xor_sync(0xFFFFFFFFu, a.s, o);
    return MaxSum{m, a.s};
}

__device__ __forceinline__ void unpack(uint4 x, float2 (&v)[4], __nv_bfloat16) {
    v[0] = unpack2(x.x), v[1] = unpack2(x.y), v[2] = unpack2(x.z), v[3] = unpack2(x.w);
}
__device__ __forceinline__ float largest(uint4 x) {
    const auto pair = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
    const __nv_bfloat162 m = __hmax2(__hmax2(pair(x.x), pair(x.y)), __hmax2(pair(x.z), pair(x.w)));
    return __bfloat162float(__hmax(m.x, m.y));
}
__device__ __forceinline__ void unpack(uint4 x, float2 (&v)[2], float) {
    v[0] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
    v[1] = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
}

// Where a row's 16-byte vectors are, and a block's share of them; head and tail: the values before and
// behind the vectors, which the first and the last block have.
template <typename T>
struct Share {
    static constexpr int E = 16 / sizeof(T);
    const uint4 *vec;
    int head, tail, v0, v1;
    __device__ __forceinline__ Share(const T *row, int V, int rank, int blocks) {
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
        head = min(V, ((16 - off) & 15) / static_cast<int>(sizeof(T)));
        const int nv = (V - head) / E;
        tail = head + nv * E;
        vec = reinterpret_cast<const uint4 *>(row + head);
        v0 = static_cast<int>(static_cast<long long>(nv) * rank / blocks);
        v1 = static_cast<int>(static_cast<long long>(nv) * (rank + 1) / blocks);
    }
};

// How the rows' vectors are dealt out to lse_kernel's blocks.  Row k of `rows` (the target's, then the
// drafts') has the places k·nv .. (k + 1)·nv - 1 of one sequence; block i takes i·per .. (i + 1)·per - 1,
// and leaves what it has of row k in part[i + k] (walking along the sequence, block or row goes up by
// one at a time, so every pair that occurs has a number of its own).  Rows start anywhere, so a row
// may have one vector less than nv = V / E: its last place is then empty.
struct Pieces {
    int zrows, rows, nv;
    long long per;
};
template <typename T>
__device__ __forceinline__ Pieces pieces_of(const VerifyParams &p) {
    const int total = max(0, min(p.starts[p.B], p.R));
    Pieces c;
    c.zrows = min(p.zrows, total);
    c.rows = c.zrows + min(p.qrows, total);
    c.nv = max(1, p.V / Share<T>::E);
    c.per = max(1LL, (static_cast<long long>(c.rows) * c.nv + kLseBlocks - 1) / kLseBlocks);
    return c;
}

__global__ void __launch_bounds__(kCountThreads) count_kernel(const VerifyParams p) {
    __shared__ int count;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    const int first = blockIdx.x * kCountRequests, end = min(p.B, first + kCountRequests);
    int mine = 0;
#pragma unroll 4
    for (int i = first + threadIdx.x; i < end; i += kCountThreads) mine += p.starts[i + 1] > p.starts[i];
    if (mine) atomicAdd(&count, mine);
    __syncthreads();
    if (threadIdx.x == 0) p.counts[blockIdx.x] = count;
}

template <typename T>
__global__ void __launch_bounds__(kLseThreads, 4) lse_kernel(const VerifyParams p) {
    constexpr int E = Share<T>::E, WARPS = kLseThreads / 32;
    __shared__ float sm[2][WARPS], ss[2][WARPS];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Pieces pieces = pieces_of<T>(p);
    const int tid = threadIdx.x;
    const float c = p.inv_t * kLog2e;
    const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf: adds nothing
    const long long all = static_cast<long long>(pieces.rows) * pieces.nv;
    long long from = blockIdx.x * pieces.per;
    const long long to = min(all, from + pieces.per);
    if (from >= to) return;
    int row = static_cast<int>(from / pieces.nv), turn = 0;
    // the part of `row` that is this block's: vectors i .. end - 1 of it
    const T *at;
    const uint4 *vec;
    int i, end, head, tail;
    auto open = [&] {
        const bool draft = row >= pieces.zrows;
        at = static_cast<const T *>(draft ? p.q : p.z) +
             static_cast<size_t>(draft ? row - pieces.zrows : row) * p.V;
        const Share<T> s(at, p.V, 0, 1);
        vec = s.vec, head = s.head, tail = s.tail;
        const long long begin = static_cast<long long>(row) * pieces.nv;
        i = static_cast<int>(from - begin);
        end = static_cast<int>(min(to - begin, static_cast<long long>(pieces.nv)));
        // the values in front of the vectors go with the first place, those behind with the last one
        if (i > 0) head = 0;
        if (end < pieces.nv) tail = p.V;
        end = min(end, s.v1);
    };
    uint4 x[kAhead];
    auto load = [&] {
        if (i + kLseThreads * kAhead <= end) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) x[u] = vec[i + tid + u * kLseThreads];
        } else {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int k = i + u * kLseThreads + tid;
                x[u] = k < end ? vec[k] : make_uint4(none, none, none, none);
            }
        }
        i += kLseThreads * kAhead;
    };
    open();
    load();
    MaxSum a{-INFINITY, 0.f};
    while (true) {
        float2 v[kAhead][E / 2];
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            unpack(x[u], v[u], T{});
            if constexpr (sizeof(T) == 2)
                top = fmaxf(top, largest(x[u]));
            else
                top = fmaxf(fmaxf(top, fmaxf(v[u][0].x, v[u][0].y)), fmaxf(v[u][1].x, v[u][1].y));
        }
        // the next vectors, of this row or the next one, are on their way meanwhile
        const bool ends = i >= end;
        const T *ended = at;
        const int last_head = head, last_tail = tail, ended_row = row;
        if (ends) {
            from = static_cast<long long>(++row) * pieces.nv;
            if (from < to) open();
        }
        if (from < to) load();
        const float m = fmaxf(a.m, top), ref = m == -INFINITY ? 0.f : m;
        float2 sum[2] = {make_float2(a.s * ex2_approx((a.m - ref) * c), 0.f), both(0.f)};
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const float2 y = __fmul2_rn(__fadd2_rn(v[u][j], both(-ref)), both(c));
                sum[j & 1] = __fadd2_rn(sum[j & 1], make_float2(ex2_approx(y.x), ex2_approx(y.y)));
            }
        a = MaxSum{m, (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)};
        if (!ends) continue;
        if (tid < last_head) a = join(a, MaxSum{one(ended + tid), 1.f}, c);
        if (tid < p.V - last_tail) a = join(a, MaxSum{one(ended + last_tail + tid), 1.f}, c);
        a = warp_join(a, c);
        if ((tid & 31) == 0) sm[turn][tid / 32] = a.m, ss[turn][tid / 32] = a.s;
        __syncthreads();  // (two turns' arrays: the next row's are written before these have been read)
        if (tid < 32) {
            a = warp_join(tid < WARPS ? MaxSum{sm[turn][tid], ss[turn][tid]} : MaxSum{-INFINITY, 0.f}, c);
            if (tid == 0) p.part[blockIdx.x + ended_row] = make_float2(a.m, a.s);
        }
        a = MaxSum{-INFINITY, 0.f};
        turn ^= 1;
        if (from >= to) return;
    }
}

// The rounded difference and what it is off by (Knuth's sum of two numbers).
__device__ __forceinline__ float2 difference(float a, float b) {
    const float d = a - b, t = d - a, off = (a - (d - t)) + (-b - t);
    return make_float2(d, fabsf(d) < INFINITY ? off : 0.f);
}

// A row's distribution: log p = (z - m) / T - (l + rest).  Formed here m is the largest logit and l the
// logarithm of the sum of exponentials, so that no number of the size of z / T is ever rounded, whatever T
// is; given m is 0 and l the logsumexp.  Two fp32 parts where one is not enough: a row's chain in 64 bits took
// 13.0 us instead of 10.4 (32 requests, logsumexps given), the fp64 pipe being as narrow as it is.
struct Norm {
    float m, l, rest;
};
__device__ __forceinline__ Norm norm_of(MaxSum a) {
    if (!(a.s > 0.f && a.s < INFINITY)) return Norm{a.m, a.s == 0.f ? -INFINITY : a.s, 0.f};  // no finite logit
    // log s = e ln 2 + log f with s = f·2^e, f in [1, 2), and ln 2 as 2839/4096 and the rest
    const uint32_t bits = __float_as_uint(a.s);
    const float e = static_cast<float>(static_cast<int>(bits >> 23) - 127);  // (s is no subnormal: its largest term is 1)
    const float2 l = difference(e * 0.693115234375f, -logf(__uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u)));
    return Norm{a.m, l.x, fmaf(e, 3.194618494530942e-05f, l.y)};
}
// The same for the scan: log2 p = (z - ref)·c + rest.  ref is m, or where the logsumexp is given the logit whose
// p is 1 (inside fp32's range), so that columns near the largest keep their precision.
__device__ __forceinline__ float2 ref_of(Norm a, bool given, const VerifyParams &p) {
    if (!given) return make_float2(a.m, fmaf(-a.l, kLog2e, -a.rest * kLog2e));
    const float ref = fabsf(a.l) < INFINITY ? fminf(fmaxf(a.l * p.t, -3.4e38f), 3.4e38f) : a.l * 0.f;
    return make_float2(ref, fmaf(ref, p.inv_t, -a.l) * kLog2e);
}
// log p of a column of logit z.
__device__ __forceinline__ float log_p(float z, Norm a, float inv_t) {
    const float2 gap = difference(z, a.m);
    return fmaf(gap.x, inv_t, -a.l) + fmaf(gap.y, inv_t, -a.rest);
}
// Whether p / q > u, for p of logit z and q of logit x (1 where there is no q).  The two logits' differences
// come first: of the size of z / T they may cancel.
__device__ __forceinline__ bool stays(float z, Norm a, float x, Norm b, bool with_q, float inv_t, float u) {
    float2 d = difference(z, a.m);
    if (with_q) {
        const float2 g = d, h = difference(x, b.m);
        d = difference(g.x, h.x);
        d.y += g.y - h.y;
    }
    float2 l = difference(a.l, b.l);
    l.y += a.rest - b.rest;
    const float y = d.x * inv_t;
    if (!(fabsf(y) < INFINITY)) return y - l.x > 0.f;
    const float2 sum = difference(y, l.x);
    const float e = expf(sum.x);
    if (!(e > 0.f && e < INFINITY)) return e > u;
    return fmaf(e, sum.y + (fmaf(d.x, inv_t, -y) + fmaf(d.y, inv_t, -l.y)), e) > u;
}

// The distribution of row `at` of the target (or the draft), by a warp.
template <typename T>
__device__ __forceinline__ Norm row_norm(const VerifyParams &p, const Pieces &c, bool draft, int at,
                                         int lane) {
    const float *given = draft ? p.qlse : p.lse;
    if (given) return Norm{0.f, given[at], 0.f};
    const int row = draft ? c.zrows + at : at;
    const long long begin = static_cast<long long>(row) * c.nv;
    const int first = static_cast<int>(begin / c.per), last = static_cast<int>((begin + c.nv - 1) / c.per);
    MaxSum a{-INFINITY, 0.f};
    for (int i = first + lane; i <= last; i += 32)
        a = join(a, MaxSum{p.part[i + row].x, p.part[i + row].y}, p.inv_t * kLog2e);
    return norm_of(warp_join(a, p.inv_t * kLog2e));
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
    float c, ref, rest, qref, qrest;  // see ref_of
    int x;
    unsigned long long seed, first;  // of the stream; index of the row's first draw in it
    float best, bar;
    int column;
    static constexpr float kUpper = 0.69314860f * 16777216.f;
    static constexpr float kLeastScore = 1.40129846e-45f;  // fp32's smallest number

    __device__ __forceinline__ Scan(const VerifyParams &p_, const T *z_, const T *q_, float4 refs, int x_,
                                    unsigned long long seed_, unsigned long long first_)
        : p(p_), z(z_), q(q_), c(p_.inv_t * kLog2e), ref(refs.x), rest(refs.y), qref(refs.z),
          qrest(refs.w), x(x_), seed(seed_), first(first_), best(0.f), bar(0.f), column(0) {}
    // Of two columns, j and j + step; v, u: their logits, the target's and the draft's.
    __device__ __forceinline__ float2 weights(float2 v, float2 u, int j, int step) const {
        const float2 y = __ffma2_rn(__fadd2_rn(v, both(-ref)), both(c), both(rest));
        float2 w = make_float2(ex2_approx(y.x), ex2_approx(y.y));
        if (FROM == kDifference) {
            const float2 n = __ffma2_rn(__fadd2_rn(u, both(-qref)), both(c), both(qrest));
            w = make_float2(w.x - ex2_approx(n.x), w.y - ex2_approx(n.y));
        }
        if (FROM == kWithout) {
            if (j == x) w.x = 0.f;
            if (j + step == x) w.y = 0.f;
        }
        return w;
    }
    __device__ __forceinline__ void exact(int j) {
        const uint32_t bits = bits24_from_state(splitmix_state(seed, first + j));
        const float2 w = weights(both(one(z + j)), both(FROM == kDifference ? one(q + j) : 0.f), j, 1);
        // A uniform of 0, or a weight too small for the quotient, scores less than any other column but more
        // than none: a row with a weight has a sample.
        const float score = w.x > 0.f ? fmaxf(w.x / -log2_uniform(bits), kLeastScore) : 0.f;
        // columns come in any order: of equal scores the lowest stays
        if (score > best || (score == best && j < column)) best = score, column = j;
    }
    // N columns of each thread of the warp, with their logits: j, j + STEP, ...; `have` of them count.
    template <int N, int STEP>
    __device__ __forceinline__ void columns(const float2 (&a)[N / 2], const float2 (&b)[N / 2], int j,
                                            int have) {
        float bound[N], low = 0.f;
        const float all = have >= N ? kUpper : 0.f;  // (`have` is N or 0 but where columns are STEP apart)
        const unsigned long long state = splitmix_state(seed, first + j);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 pair = weights(a[i / 2], b[i / 2], j + i * STEP, STEP);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t bits =
                    bits24_from_state(state + static_cast<unsigned long long>((i + h) * STEP) * kGolden);
                // With l = 1 - u:  l <= -ln u <= l / (1 - l), so the score w / -log2 u lies between
                // w·ln 2 / l and that times 1 - l.  The constants leave room for the roundings of both and
                // of the score itself (2e-6 and 4e-6 against some 1e-6); l is counted in 2^-24.
                const float l = static_cast<float>(16777216u - bits), w = h ? pair.y : pair.x;
                bound[i + h] = w * (STEP == 1 ? all : i + h < have ? kUpper : 0.f) * rcp_approx(l);
                low = fmaxf(low, bound[i + h] * fmaf(l, -0.999994f * 5.9604644775390625e-8f, 0.999994f));
            }
        }
        const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(low));  // (low >= 0)
        bar = fmaxf(bar, __uint_as_float(most));
        uint32_t promising = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) promising |= static_cast<uint32_t>(bound[i] > bar) << i;
        for (; promising; promising &= promising - 1) exact(j + (__ffs(promising) - 1) * STEP);
    }
};

// This thread's best of the share of block `rank` of `blocks`.
template <typename T, int FROM>
__device__ __forceinline__ unsigned long long scan(const VerifyParams &p, const T *z, const T *q,
                                                   float4 refs, int x, unsigned long long seed,
                                                   unsigned long long first, int rank, int blocks) {
    constexpr int E = Share<T>::E;
    const int tid = threadIdx.x;
    Scan<T, FROM> s(p, z, q, refs, x, seed, first);
    if (FROM != kDifference || ((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0) {
        const Share<T> za(z, p.V, rank, blocks);
        const uint4 *qa = FROM == kDifference ? reinterpret_cast<const uint4 *>(q + za.head) : nullptr;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (za.v0 + tid < za.v1) {
            a = za.vec[za.v0 + tid];
            if (FROM == kDifference) b = qa[za.v0 + tid];
        }
        for (int i0 = za.v0; i0 < za.v1; i0 += kVerifyThreads) {  // (the same turns for all threads)
            const int i = i0 + tid, next = i + kVerifyThreads;
            float2 pa[E / 2], pb[E / 2];
            unpack(a, pa, T{});
            unpack(b, pb, T{});
            if (next < za.v1) {
                a = za.vec[next];
                if (FROM == kDifference) b = qa[next];
            }
            s.template columns<E, 1>(pa, pb, za.head + i * E, i < za.v1 ? E : 0);
        }
        if (rank == 0 && tid < za.head) s.exact(tid);
        if (rank == blocks - 1 && tid < p.V - za.tail) s.exact(za.tail + tid);
    } else {
        // rows of an odd vocabulary: z's and q's vectors never lie side by side
        constexpr int W = 8;
        const int c0 = static_cast<int>(static_cast<long long>(p.V) * rank / blocks);
        const int c1 = static_cast<int>(static_cast<long long>(p.V) * (rank + 1) / blocks);
        for (int j0 = c0; j0 < c1; j0 += W * kVerifyThreads) {
            const int j = j0 + tid;
            float2 a[W / 2], b[W / 2];
#pragma unroll
            for (int k = 0; k < W; k += 2) {
                const int i = min(j + k * kVerifyThreads, c1 - 1), n = min(i + kVerifyThreads, c1 - 1);
                a[k / 2] = make_float2(one(z + i), one(z + n));
                b[k / 2] = make_float2(one(q + i), one(q + n));
            }
            s.template columns<W, kVerifyThreads>(a, b, j, max(0, (c1 - j + kVerifyThreads - 1) / kVerifyThreads));
        }
    }
    return pack(s.best, s.column);
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const VerifyParams p) {
    constexpr int THREADS = kVerifyThreads, WARPS = THREADS / 32;
    __shared__ int end, busy;
    __shared__ Norm norms[WARPS];
    __shared__ float4 refs[WARPS];  // see ref_of: the target's and the draft's
    __shared__ unsigned long long bests[2][kWideBlocks], warps[WARPS];
    const int blocks = static_cast<int>(cluster_blocks()), rank = static_cast<int>(cluster_ctarank());
    const int b = static_cast<int>(blockIdx.x) / blocks;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    // the peers run before anything is written into their shared memory
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int total = p.B ? p.starts[p.B] : 0;
    const int s0 = p.B ? p.starts[b] : 0, s1 = p.B ? p.starts[b + 1] : 0, front = p.B ? p.starts[0] : 0;
    const unsigned long long seed = p.seed + (p.seed_offset ? *p.seed_offset : 0ull);
    if (blockIdx.x == 0 && tid == 0) *p.epoch_word = p.epoch;
    auto clear = [&](int from, int to) {
        for (long long r = from + static_cast<long long>(rank) * THREADS + tid; r < to;
             r += static_cast<long long>(blocks) * THREADS) {
            p.token[r] = -1;
            if (p.logprob) p.logprob[r] = 0.f;
        }
    };
    // the rows in front of the first request and behind the last one, where no request has its own
    if (b == 0) clear(0, min(front, p.R));
    if (b == (p.B ? p.B - 1 : 0) && total >= 0) clear(total, p.R);
    // draft rows are those of the requests before this one that have any rows
    const int n = static_cast<int>(static_cast<unsigned>(s1) - static_cast<unsigned>(s0) - 1u);
    if (tid == 0) busy = 0, end = n;
    __syncthreads();
    int mine = 0;
    if (p.Rd > 0) {
        const int shares = p.counts ? b / kCountRequests : 0;
        for (int i = tid; i < shares; i += THREADS) mine += p.counts[i];
        for (int i = shares * kCountRequests + tid; i < b; i += THREADS) mine += p.starts[i + 1] > p.starts[i];
    }
    if (mine) atomicAdd(&busy, mine);
    __syncthreads();
    const int q0 = s0 - max(front, 0) - busy;  // the draft's row of row s0
    const bool sane = s0 >= 0 && s0 >= front && s1 >= s0 && s1 <= total && total <= p.R &&
                      (!p.with_q || n <= 0 || (q0 >= 0 && q0 + n <= p.Rd));
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (!sane || n < 0) {  // the same for all blocks of the cluster
        if (!sane && tid == 0 && rank == 0) record_status(p.status, p.epoch, 1u);  // SB_ERR_INVALID_ARG
        if (p.B && tid == 0 && rank == 0) p.accepted[b] = sane ? 0 : -1;
        return;
    }
    const T *z = static_cast<const T *>(p.z) + static_cast<size_t>(s0) * p.V;
    const T *q = p.with_q && n > 0 ? static_cast<const T *>(p.q) + static_cast<size_t>(q0) * p.V : nullptr;
    const Pieces pieces = pieces_of<T>(p);
    // which drafts stay, one to a warp at a time; the last row has none, and ends the request
    int g = 0;
    for (;; g += WARPS) {
        const int i = g + warp, r = s0 + i;
        if (i <= n) {
            const bool has = i < n;
            const int x = has ? p.drafts[r] : -1;
            const bool known = x >= 0 && x < p.V;
            const size_t at = static_cast<size_t>(i) * p.V + (known ? x : 0);
            const float zx = known ? one(z + at) : 0.f, qx = known && q ? one(q + at) : 0.f;
            const float u = has ? p.u[r] : 0.f;
            const Norm norm = row_norm<T>(p, pieces, false, r, lane);
            const Norm qnorm = has && q ? row_norm<T>(p, pieces, true, q0 + i, lane) : Norm{};
            if (lane == 0) {
                const float2 a = ref_of(norm, p.lse, p), b = ref_of(qnorm, p.qlse, p);
                norms[warp] = norm;
                refs[warp] = make_float4(a.x, a.y, b.x, b.y);
                if (has) {
                    if (!known && rank == 0) record_status(p.status, p.epoch, 1u);
                    if (!known || !stays(zx, norm, qx, qnorm, q, p.inv_t, u)) atomicMin(&end, i);
                    if (rank == 0) {  // (of a row behind the end it is taken back below)
                        p.token[r] = x;
                        if (p.logprob) p.logprob[r] = log_p(zx, norm, p.inv_t);
                    }
                }
            }
        }
        __syncthreads();
        if (end < g + WARPS) break;  // (end is n at most, the last row's)
        __syncthreads();             // before the next rows' are written
    }
    const int e = end, r = s0 + e;
    const Norm norm = norms[e - g];
    const float4 ref = refs[e - g];
    z += static_cast<size_t>(e) * p.V;
    const int x = e < n ? p.drafts[r] : -1;
    const bool known = x >= 0 && x < p.V;  // otherwise nothing is taken off p
    const unsigned long long first = static_cast<unsigned long long>(r) * static_cast<unsigned>(p.V);
    unsigned long long best = 0;
    for (int turn = 0; turn < 2 && !best; ++turn) {
        // a difference that is nowhere positive (p and q equal but for roundings): p itself
        if (turn == 0 && known && q)
            best = scan<T, kDifference>(p, z, q + static_cast<size_t>(e) * p.V, ref, x, seed, first, rank, blocks);
        else if (turn == 0 && known)
            best = scan<T, kWithout>(p, z, nullptr, ref, x, seed, first, rank, blocks);
        else
            best = scan<T, kTarget>(p, z, nullptr, ref, x, seed, first, rank, blocks);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long other = __shfl_xor_sync(0xFFFFFFFFu, best, o);
            best = other > best ? other : best;
        }
        if (lane == 0) warps[warp] = best;
        __syncthreads();
        if (tid < blocks) {
            for (int w = 0; w < WARPS; ++w) best = warps[w] > best ? warps[w] : best;
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
    for (int i = e + tid; i <= n; i += THREADS) {
        int token = -1;
        float lp = 0.f;
        if (i == e) {
            lp = __uint_as_float(0x7FC00000u);  // no column of the row has any probability
            if (best) {
                token = ~static_cast<int>(static_cast<uint32_t>(best));
                lp = log_p(one(z + token), norm, p.inv_t);
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
    const int total = p.B ? p.starts[p.B] : 0, front = p.B ? p.starts[0] : 0;
    if (b == 0)
        for (int r = lane; r < min(front, p.R); r += 32) p.token[r] = -1;
    if (b == (p.B ? p.B - 1 : 0) && total >= 0)
        for (long long r = static_cast<long long>(total) + lane; r < p.R; r += 32) p.token[r] = -1;
    if (b >= p.B) return;
    const int s0 = p.starts[b], s1 = p.starts[b + 1];
    if (s0 < 0 || s0 < front || s1 < s0 || s1 > total || total > p.R) {
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
cudaError_t launch_verify(const VerifyParams &p, int sms, cudaStream_t st) {
    if (p.counts) {
        const unsigned shares = static_cast<unsigned>((p.B + kCountRequests - 1) / kCountRequests);
        const cudaError_t e = launch_dependent(count_kernel, dim3(shares), kCountThreads, 0, p, st);
        if (e != cudaSuccess) return e;
    }
    if (p.zrows + p.qrows > 0 && p.B > 0) {
        const cudaError_t e = launch_dependent(lse_kernel<T>, dim3(kLseBlocks), kLseThreads, 0, p, st);
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
    int blocks = kMostBlocks;
    while (blocks > kLeastBlocks && static_cast<int64_t>(p.B) * blocks > 2 * sms) blocks /= 2;
    if (p.B * kWideBlocks <= sms) {
        // more than eight blocks to a cluster are no part of the portable model: asked once a device
        static std::atomic<uint64_t> asked{0}, allowed{0};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
        if (bit && !(asked.load() & bit)) {
            int clusters = 0;
            cudaLaunchConfig_t cfg = config(kWideBlocks, attr);
            cfg.numAttrs = 1;
            e = cudaFuncSetAttribute(verify_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, verify_kernel<T>, &cfg);
            if (e == cudaSuccess && clusters > 0) allowed.fetch_or(bit);
            if (e != cudaSuccess) cudaGetLastError();  // a refusal is an answer here
            asked.fetch_or(bit);
        }
        if (allowed.load() & bit) blocks = kWideBlocks;
    }
    const cudaLaunchConfig_t cfg = config(blocks, attr);
    return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p);
}

bool verify_sizes(int64_t R, int64_t draft_rows, int64_t V) {
    return R >= 0 && R < (int64_t(1) << 24) && draft_rows >= -1 && draft_rows < (int64_t(1) << 24) &&
           V >= 1 && V < (int64_t(1) << 31) - 65536;
}

size_t verify_part_bytes(int64_t R, int64_t draft_rows) {
    return up256(static_cast<size_t>(R + (draft_rows > 0 ? draft_rows : 0) + kLseBlocks) * 8);
}

}  // namespace
}  // namespace sb

using namespace sb;

extern "C" {

size_t sb_verify_workspace_bytes(int64_t R, int64_t draft_rows, int64_t V) {
    if (!verify_sizes(R, draft_rows, V)) return 0;
    // the header, lse_kernel's parts and count_kernel's counts
    return 256 + verify_part_bytes(R, draft_rows) + (draft_rows > 0 ? kMostRequests / kCountRequests * 4 : 0);
}

int32_t sb_verify_drafts(const void *logits, const void *draft_logits, const int32_t *drafts,
                         const int32_t *starts, const float *uniforms, const float *lse,
                         const float *draft_lse, int64_t R, int64_t draft_rows, int64_t B,
                         int64_t V, int32_t logits_type, float temperature, uint64_t seed,
                         int32_t *token, int32_t *accepted, float *token_logprob, void *workspace,
                         size_t workspace_bytes, void *stream) {
    return sb_verify_drafts_at(logits, draft_logits, drafts, starts, uniforms, lse, draft_lse, R,
                               draft_rows, B, V, logits_type, temperature, seed, nullptr, token,
                               accepted, token_logprob, workspace, workspace_bytes, stream);
}

int32_t sb_verify_drafts_at(const void *logits, const void *draft_logits, const int32_t *drafts,
                            const int32_t *starts, const float *uniforms, const float *lse,
                            const float *draft_lse, int64_t R, int64_t draft_rows, int64_t B,
                            int64_t V, int32_t logits_type, float temperature, uint64_t seed,
                            const uint64_t *seed_offset, int32_t *token, int32_t *accepted,
                            float *token_logprob, void *workspace, size_t workspace_bytes,
                            void *stream) {
    if (!verify_sizes(R, draft_rows, V) || B < 0 || B > kMostRequests ||
        logits_type < SB_BF16 || logits_type > SB_F32 ||
        !(std::isfinite(temperature) && temperature > 0.f) ||
        temperature < 1e-30f || (R > 0 && (!logits || !drafts || !uniforms || !token)) ||
        (B > 0 && (!starts || !accepted)) || (draft_rows > 0 && !draft_logits) || !workspace)
        return SB_ERR_INVALID_ARG;
    const uintptr_t za = logits_type == SB_F32 ? 4 : 2;
    if (!on(logits, za) || !on(draft_logits, za) || !on(drafts, 4) || !on(starts, 4) ||
        !on(uniforms, 4) || !on(lse, 4) || !on(draft_lse, 4) || !on(token, 4) || !on(accepted, 4) ||
        !on(token_logprob, 4) || !on(workspace, 256) || !on(seed_offset, 8))
        return SB_ERR_ALIGNMENT;
    // every block of a request reads its drafts, uniforms and sums for itself, while one of them writes
    const size_t need = sb_verify_workspace_bytes(R, draft_rows, V), rows = R * 4;
    const size_t q_rows = draft_rows > 0 ? draft_rows : 0;
    const Span arrays[] = {{token, rows}, {accepted, static_cast<size_t>(B) * 4}, {token_logprob, rows},
                           {workspace, need}, {logits, R * V * za}, {draft_logits, q_rows * V * za},
                           // (a draft's place takes the draft itself until all blocks have read it)
                           {token == drafts ? nullptr : drafts, rows}, {starts, B > 0 ? (B + 1) * size_t(4) : 0},
                           {uniforms, rows}, {lse, rows}, {draft_lse, q_rows * 4}, {seed_offset, 8}};
    if (any_overlap(arrays, 4)) return SB_ERR_INVALID_ARG;
    int sms = 0;
    if (int32_t e = device_sms_cc(&sms, nullptr)) return e;
    if (workspace_bytes < need) return SB_ERR_WORKSPACE_TOO_SMALL;
    // (without rows or requests too: the header's status is this call's)
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    VerifyParams p{};
    p.z = logits;
    p.q = draft_logits;
    p.with_q = draft_rows >= 0;
    if (draft_rows > 0 && B > kCountRequests)
        p.counts = reinterpret_cast<int *>(ws + 256 + verify_part_bytes(R, draft_rows));
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
    p.part = reinterpret_cast<float2 *>(ws + 256);
    p.t = temperature;
    p.inv_t = 1.0f / temperature;
    p.seed = seed;
    p.seed_offset = reinterpret_cast<const unsigned long long *>(seed_offset);
    p.token = token;
    p.accepted = accepted;
    p.logprob = token_logprob;
    p.epoch_word = reinterpret_cast<uint32_t *>(ws);
    p.status = reinterpret_cast<unsigned long long *>(ws + 8);
    p.epoch = next_epoch();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (logits_type == SB_BF16 ? launch_verify<__nv_bfloat16>(p, sms, st) : launch_verify<float>(p, sms, st)) ==
                   cudaSuccess
               ? SB_OK
               : SB_ERR_CUDA;
}

int32_t sb_verify_greedy(const int32_t *target, const int32_t *drafts, const int32_t *starts,
                         int64_t R, int64_t B, int32_t *token, int32_t *accepted, void *stream) {
    if (R < 0 || R >= (int64_t(1) << 31) - 65536 || B < 0 || B > kMostRequests ||
        (R > 0 && (!target || !drafts || !token)) || (B > 0 && (!starts || !accepted)))
        return SB_ERR_INVALID_ARG;
    if (!on(target, 4) || !on(drafts, 4) || !on(starts, 4) || !on(token, 4) || !on(accepted, 4))
        return SB_ERR_ALIGNMENT;
    // (a request's warp has read its drafts when it writes, and a row's target in the same thread)
    const size_t rows = R * 4;
    const Span arrays[] = {{token, rows}, {accepted, static_cast<size_t>(B) * 4},
                           {token == drafts ? nullptr : drafts, rows}, {token == target ? nullptr : target, rows},
                           {starts, B > 0 ? (B + 1) * size_t(4) : 0}};
    if (any_overlap(arrays, 2)) return SB_ERR_INVALID_ARG;
    if (int32_t e = device_sms_cc(nullptr, nullptr)) return e;
    if (R == 0 && B == 0) return SB_OK;
    const GreedyParams p{target, drafts, starts, static_cast<int>(R), static_cast<int>(B), token, accepted};
    return launch_dependent(greedy_kernel, dim3(static_cast<unsigned>((B > 0 ? B : 1) + 3) / 4), 128, 0, p,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SB_OK
               : SB_ERR_CUDA;
}

}  // extern "C"
