// embedding.cu -- the tokens' rows of the vocabulary matrix, and the gradient of that lookup.
//   forward    out_t = scale·W[id_t]            (zeros for the ignored index, NaN for other ids
//                                                outside the vocabulary)
//   backward   dW_v = [dW_v +] scale·sum over t with id_t = v of dout_t
//
// Forward is bound by memory: the rows in, the rows out.  A row is a run of consecutive vectors of
// eight values; threads of a block take them side by side, several rows to a block where rows are
// short, up to four vectors (64 bytes) of loads in flight each.
//
// Backward sums rows in a fixed order, so that equal calls give equal bits; atomics on fp32 values
// would not.  Three kernels:
//   sort_kernel    every token's rank among the tokens by (id, position): the count of smaller
//                  keys, and of equal ones at earlier positions.  All pairs are compared, 32 tokens
//                  to a block, a lane each, the keys broadcast from shared memory: M²/32·2.25 warp
//                  instructions, 5 us of this GPU for 8192 tokens, in one launch without a pass
//                  that waits for another.  Beyond kChunk tokens each chunk is sorted by itself and
//                  merge_kernel adds the ranks in the other chunks, by binary search.
//                  When the whole gradient is asked for, further blocks of the same launch write its
//                  zeros meanwhile (that is most of its bytes: V rows against at most M that are
//                  not zero).
//   reduce_kernel  a block takes a piece of consecutive sorted tokens and a slice of columns, and
//                  adds the rows of each run of equal ids in registers; a run inside the piece is
//                  scaled, added and rounded here.  What a piece holds of a run that crosses its
//                  ends goes to the workspace in fp32.  So a token that takes most of the batch costs
//                  no more than others.
//   join_kernel    adds the pieces' parts of such runs, in ascending order.
#include <cmath>

#include "norm_common.cuh"
#include "sb.h"

namespace sb {
namespace {

constexpr int kNoToken = 0x7FFFFFFF;  // the key of a token without a row: sorts behind all others

// ------------------------------------------------------------------ forward
struct LookupParams {
    const int32_t *ids;
    const void *W;
    void *out;
    int M, V, ignore;
    int rows;         // of a block
    long long d;
    float scale;
};
constexpr int kLookupThreads = 256;

template <typename W, typename O, int VEC>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(const LookupParams p) {
    constexpr int U = VEC == 1 ? 8 : 4;  // vectors in flight
    const int tx = kLookupThreads / p.rows;
    const int x = threadIdx.x % tx;
    const long long row = static_cast<long long>(blockIdx.x) * p.rows + threadIdx.x / tx;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // no early launch_dependents: what follows may read `out` as a weight, ahead of this kernel's end
    if (row >= p.M) return;
    const int id = p.ids[row];
    const bool has = id >= 0 && id < p.V && id != p.ignore;
    const W *from = static_cast<const W *>(p.W) + (has ? static_cast<size_t>(id) * p.d : 0);
    O *to = static_cast<O *>(p.out) + static_cast<size_t>(row) * p.d;
    const float none = id == p.ignore ? 0.f : __uint_as_float(0x7FC00000u);
    for (long long e0 = static_cast<long long>(x) * VEC; e0 < p.d;
         e0 += static_cast<long long>(U) * tx * VEC) {
        float2 v[U][(VEC + 1) / 2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long e = e0 + static_cast<long long>(u) * tx * VEC;
            if (has && e < p.d) {
                if constexpr (VEC == 1)
                    v[u][0].x = one(from + e);
                else
                    load_pairs<VEC>(from + e, v[u]);
            } else {
#pragma unroll
                for (int j = 0; j < (VEC + 1) / 2; ++j) v[u][j] = both(none);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long e = e0 + static_cast<long long>(u) * tx * VEC;
            if (e < p.d) {
#pragma unroll
                for (int j = 0; j < (VEC + 1) / 2; ++j) v[u][j] = __fmul2_rn(v[u][j], both(has ? p.scale : 1.f));
                if constexpr (VEC == 1)
                    put_one(to + e, v[u][0].x);
                else
                    store_pairs<VEC>(to + e, v[u]);
            }
        }
    }
}

template <typename W, typename O>
cudaError_t launch_lookup(LookupParams p, int vec, cudaStream_t st) {
    const long long steps = (p.d + vec - 1) / vec;
    const int per = vec == 1 ? 8 : 4;
    int tx = 8;
    while (tx < kLookupThreads && static_cast<long long>(tx) * per < steps) tx *= 2;
    p.rows = kLookupThreads / tx;
    const dim3 grid(static_cast<unsigned>((p.M + p.rows - 1) / p.rows));
    if (vec == 8) return launch_dependent(lookup_kernel<W, O, 8>, grid, kLookupThreads, 0, p, st);
    if (vec == 4) return launch_dependent(lookup_kernel<W, O, 4>, grid, kLookupThreads, 0, p, st);
    return launch_dependent(lookup_kernel<W, O, 1>, grid, kLookupThreads, 0, p, st);
}

// ------------------------------------------------------------------ backward: order
constexpr int kChunk = 8192;       // tokens sorted by all pairs
constexpr int kSortThreads = 256;  // of a block, which ranks 32 tokens
constexpr int kZeroBlocks = 152 * 4;

struct SortParams {
    const int32_t *ids;
    int M, V, ignore;
    int sort_blocks;
    int2 *sorted;      // (key, position), sorted within each chunk
    uint8_t *zero;     // bytes to clear (null: none)
    size_t zero_bytes;
};

__device__ void clear_bytes(uint8_t *p, size_t n, size_t thread, size_t threads) {
    // values are 2 or 4 bytes wide: so are what lies before and behind the 32-byte units
    size_t head = (32 - (reinterpret_cast<uintptr_t>(p) & 31)) & 31;
    if (head > n) head = n;
    const size_t units = (n - head) / 32, tail = head + units * 32;
    for (size_t i = thread; i < units; i += threads)
        st_global_v8(p + head + i * 32, 0, 0, 0, 0, 0, 0, 0, 0);
    if (thread < head / 2) *reinterpret_cast<uint16_t *>(p + thread * 2) = 0;
    if (thread < (n - tail) / 2) *reinterpret_cast<uint16_t *>(p + tail + thread * 2) = 0;
}

__global__ void __launch_bounds__(kSortThreads) sort_kernel(const SortParams p) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ int counts[kSortThreads / 32][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (static_cast<int>(blockIdx.x) >= p.sort_blocks) {
        const size_t blocks = gridDim.x - p.sort_blocks, block = blockIdx.x - p.sort_blocks;
        clear_bytes(p.zero, p.zero_bytes, block * kSortThreads + threadIdx.x, blocks * kSortThreads);
        return;
    }
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int chunk = blockIdx.x / (kChunk / 32), base = chunk * kChunk;
    const int n = min(kChunk, p.M - base), groups = (n + 31) / 32;
    const int mine = static_cast<int>(blockIdx.x) - chunk * (kChunk / 32);  // my group of 32
    for (int j = threadIdx.x; j < groups * 32; j += kSortThreads) {
        uint32_t key = 0xFFFFFFFFu;  // behind the last token: never counted
        if (j < n) {
            const int id = p.ids[base + j];
            key = id >= 0 && id < p.V && id != p.ignore ? id : kNoToken;
        }
        keys[j] = key;
    }
    __syncthreads();
    const uint32_t key = keys[mine * 32 + lane];
    int count = 0;
    for (int g = warp; g < groups; g += kSortThreads / 32) {
        const uint4 *k4 = reinterpret_cast<const uint4 *>(keys + g * 32);
        if (g != mine) {
            const uint32_t limit = key + (g < mine);  // equal keys count where they come before
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4 k = k4[j];
                count += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4 k = k4[j];
                count += (k.x < key + (4 * j < lane)) + (k.y < key + (4 * j + 1 < lane)) +
                         (k.z < key + (4 * j + 2 < lane)) + (k.w < key + (4 * j + 3 < lane));
            }
        }
    }
    counts[warp][lane] = count;
    __syncthreads();
    if (warp == 0 && mine * 32 + lane < n) {
        int rank = 0;
#pragma unroll
        for (int w = 0; w < kSortThreads / 32; ++w) rank += counts[w][lane];
        p.sorted[base + rank] = make_int2(static_cast<int>(key), base + mine * 32 + lane);
    }
}

// The chunks' orders become one: a token's place is its rank in its own chunk and the counts of
// smaller keys (of keys not larger, in earlier chunks) in the others.
struct MergeParams {
    const int2 *from;
    int2 *to;
    int M;
};
__global__ void __launch_bounds__(256) merge_kernel(const MergeParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.M) return;
    const int2 token = p.from[i];
    const int chunks = (p.M + kChunk - 1) / kChunk, own = static_cast<int>(i / kChunk);
    int place = static_cast<int>(i - static_cast<long long>(own) * kChunk);
#pragma unroll 4
    for (int c = 0; c < chunks; ++c) {
        const int2 *k = p.from + static_cast<size_t>(c) * kChunk;
        const uint32_t limit = static_cast<uint32_t>(token.x) + (c < own);
        int lo = 0, hi = min(kChunk, p.M - c * kChunk);
        if (c == own) hi = 0;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (static_cast<uint32_t>(k[mid].x) < limit)
                lo = mid + 1;
            else
                hi = mid;
        }
        place += lo;
    }
    p.to[place] = token;
}

// ------------------------------------------------------------------ backward: sums
constexpr int kPiece = 32;           // sorted tokens of a block
constexpr int kReduceThreads = 128;
constexpr int kAhead = 8;            // rows in flight

struct ReduceParams {
    const int2 *sorted;
    const void *dout;
    void *dW;
    float *part;  // [pieces][2][d]: of the run that comes in from the piece before, and of the one
                  // that starts here and goes on behind
    int M, pieces;
    long long d;
    float scale;
    int add;
};

template <typename G, typename W, int VEC>
__global__ void __launch_bounds__(kReduceThreads) reduce_kernel(const ReduceParams p) {
    constexpr int N = (VEC + 1) / 2;
    __shared__ int2 token[kPiece + 2];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // no early launch_dependents: nothing that follows may read dW ahead of this kernel's end
    const int first = blockIdx.x * kPiece;
    if (threadIdx.x < kPiece + 2) {
        const int i = first + static_cast<int>(threadIdx.x) - 1;
        token[threadIdx.x] = i >= 0 && i < p.M ? p.sorted[i] : make_int2(-1, 0);
    }
    __syncthreads();
    const long long e = (static_cast<long long>(blockIdx.y) * kReduceThreads + threadIdx.x) * VEC;
    if (e >= p.d) return;
    const G *dout = static_cast<const G *>(p.dout) + e;
    W *dW = static_cast<W *>(p.dW) + e;
    float2 acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = both(0.f);
    bool came = token[0].x == token[1].x;  // the run is one of the piece before
    for (int k0 = 1; k0 <= kPiece; k0 += kAhead) {
        const int key0 = token[k0].x;
        if (key0 < 0 || key0 == kNoToken) break;
        float2 v[kAhead][N], old[kAhead][N];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int2 t = token[k0 + u];
            const bool there = t.x >= 0 && t.x != kNoToken;
            const bool ends = there && t.x != token[k0 + u + 1].x;
#pragma unroll
            for (int j = 0; j < N; ++j) v[u][j] = old[u][j] = both(0.f);
            if (there) {
                const G *from = dout + static_cast<size_t>(t.y) * p.d;
                if constexpr (VEC == 1)
                    v[u][0].x = one(from);
                else
                    load_pairs<VEC>(from, v[u]);
            }
            if (p.add && ends) {
                const W *from = dW + static_cast<size_t>(t.x) * p.d;
                if constexpr (VEC == 1)
                    old[u][0].x = one(from);
                else
                    load_pairs<VEC>(from, old[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int2 t = token[k0 + u];
            if (t.x < 0 || t.x == kNoToken) break;
            const bool ends = t.x != token[k0 + u + 1].x;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = __fadd2_rn(acc[j], v[u][j]);
            if (!ends && k0 + u < kPiece) continue;
            if (ends && !came) {
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = __ffma2_rn(acc[j], both(p.scale), old[u][j]);
                W *to = dW + static_cast<size_t>(t.x) * p.d;
                if constexpr (VEC == 1)
                    put_one(to, acc[0].x);
                else
                    store_pairs<VEC>(to, acc);
            } else {
                float *to = p.part + (static_cast<size_t>(blockIdx.x) * 2 + !came) * p.d + e;
                if constexpr (VEC == 1)
                    *to = acc[0].x;
                else
                    store_pairs<VEC>(to, acc);
            }
            came = false;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = both(0.f);
        }
    }
}

// The run that starts in a piece and ends in a later one: its parts in ascending order, eight
// slices of them side by side, and then the slices.
constexpr int kJoinSlices = 8;
template <typename W, int VEC>
__global__ void __launch_bounds__(32 * kJoinSlices) join_kernel(const ReduceParams p) {
    constexpr int N = (VEC + 1) / 2;
    __shared__ float2 sums[kJoinSlices][32][N];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int piece = blockIdx.x;
    const long long behind = static_cast<long long>(piece + 1) * kPiece;
    if (behind >= p.M) return;
    const int key = p.sorted[behind - 1].x;
    if (key == kNoToken || key != p.sorted[behind].x) return;
    if (piece > 0 && p.sorted[behind - kPiece - 1].x == key) return;  // it started in an earlier one
    // the last piece with a part of it
    long long lo = behind, hi = p.M;
    while (lo < hi) {
        const long long mid = (lo + hi) / 2;
        if (p.sorted[mid].x <= key)
            lo = mid + 1;
        else
            hi = mid;
    }
    const int parts = static_cast<int>((lo - 1) / kPiece) - piece + 1;
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int q0 = static_cast<int>(static_cast<long long>(parts) * slice / kJoinSlices);
    const int q1 = static_cast<int>(static_cast<long long>(parts) * (slice + 1) / kJoinSlices);
    for (long long e0 = static_cast<long long>(blockIdx.y) * 32 * VEC; e0 < p.d;
         e0 += static_cast<long long>(gridDim.y) * 32 * VEC) {
        const long long e = e0 + lane * VEC;
        float2 acc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = both(0.f);
        if (e < p.d)
#pragma unroll 4
            for (int q = q0; q < q1; ++q) {
                const float *from = p.part + (static_cast<size_t>(piece + q) * 2 + (q == 0)) * p.d + e;
                float2 v[N];
                if constexpr (VEC == 1)
                    v[0] = make_float2(*from, 0.f);
                else
                    load_pairs<VEC>(from, v);
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = __fadd2_rn(acc[j], v[j]);
            }
#pragma unroll
        for (int j = 0; j < N; ++j) sums[slice][lane][j] = acc[j];
        __syncthreads();
        if (slice == 0 && e < p.d) {
            W *to = static_cast<W *>(p.dW) + static_cast<size_t>(key) * p.d + e;
            float2 old[N];
#pragma unroll
            for (int j = 0; j < N; ++j) old[j] = both(0.f);
            if (p.add) {
                if constexpr (VEC == 1)
                    old[0].x = one(to);
                else
                    load_pairs<VEC>(to, old);
            }
#pragma unroll
            for (int s = 1; s < kJoinSlices; ++s)
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = __fadd2_rn(acc[j], sums[s][lane][j]);
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = __ffma2_rn(acc[j], both(p.scale), old[j]);
            if constexpr (VEC == 1)
                put_one(to, acc[0].x);
            else
                store_pairs<VEC>(to, acc);
        }
        __syncthreads();
    }
}

template <typename G, typename W, int VEC>
cudaError_t launch_sums(const ReduceParams &p, cudaStream_t st) {
    const long long slices = (p.d + kReduceThreads * VEC - 1) / (kReduceThreads * VEC);
    cudaError_t e = launch_dependent(reduce_kernel<G, W, VEC>,
                                     dim3(p.pieces, static_cast<unsigned>(slices)), kReduceThreads,
                                     0, p, st);
    if (e != cudaSuccess || p.pieces == 1) return e;
    constexpr int J = VEC == 1 ? 1 : 4;  // four values to a lane, of fp32 parts
    long long cols = (p.d + 32 * J - 1) / (32 * J);
    if (cols > 8) cols = 8;
    return launch_dependent(join_kernel<W, J>, dim3(p.pieces, static_cast<unsigned>(cols)),
                            32 * kJoinSlices, 0, p, st);
}
template <typename G, typename W>
cudaError_t launch_sums(const ReduceParams &p, int vec, cudaStream_t st) {
    if constexpr (sizeof(G) == 2 && sizeof(W) == 2)
        if (vec == 8) return launch_sums<G, W, 8>(p, st);
    if (vec >= 4) return launch_sums<G, W, 4>(p, st);  // fp32: four values are 16 bytes
    return launch_sums<G, W, 1>(p, st);
}

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 65536;
constexpr int64_t kMaxWidth = int64_t(1) << 22;  // columns of a row

int64_t pieces_of(int64_t M) { return (M + kPiece - 1) / kPiece; }

int32_t check_embedding(const int32_t *ids, int64_t M, int64_t d, int64_t V, float scale,
                        int32_t row_type, int32_t weight_type) {
    if (M < 0 || M > kMaxTokens || d < 1 || d > kMaxWidth || V < 1 ||
        V >= (int64_t(1) << 31) - 1 || (M > 0 && !ids) || !std::isfinite(scale) ||
        row_type < SB_BF16 || row_type > SB_F32 || weight_type < SB_BF16 || weight_type > SB_F32)
        return SB_ERR_INVALID_ARG;
    return on(ids, 4) ? SB_OK : SB_ERR_ALIGNMENT;
}

}  // namespace
}  // namespace sb

using namespace sb;

extern "C" {

int32_t sb_embedding_forward(const int32_t *ids, const void *W, int64_t M, int64_t d, int64_t V,
                             int32_t ignore_index, float scale, int32_t weight_type,
                             int32_t out_type, void *out, void *stream) {
    if (int32_t e = check_embedding(ids, M, d, V, scale, out_type, weight_type)) return e;
    if (!W || (M > 0 && !out)) return SB_ERR_INVALID_ARG;
    if (!on(W, weight_type == SB_F32 ? 4 : 2) || !on(out, out_type == SB_F32 ? 4 : 2))
        return SB_ERR_ALIGNMENT;
    if (int32_t e = device_sms_cc(nullptr, nullptr)) return e;
    if (M == 0) return SB_OK;
    LookupParams p{};
    p.ids = ids;
    p.W = W;
    p.out = out;
    p.M = static_cast<int>(M);
    p.V = static_cast<int>(V);
    p.ignore = ignore_index;
    p.d = d;
    p.scale = scale;
    const int vec = vector_width(d, W, out);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    using B = __nv_bfloat16;
    cudaError_t e;
    if (weight_type == SB_BF16)
        e = out_type == SB_BF16 ? launch_lookup<B, B>(p, vec, st) : launch_lookup<B, float>(p, vec, st);
    else
        e = out_type == SB_BF16 ? launch_lookup<float, B>(p, vec, st)
                                : launch_lookup<float, float>(p, vec, st);
    return e == cudaSuccess ? SB_OK : SB_ERR_CUDA;
}

// [chunk-sorted tokens (only beyond one chunk)] [sorted tokens] [parts]
size_t sb_embedding_backward_workspace_bytes(int64_t M, int64_t d) {
    if (M < 0 || M > kMaxTokens || d < 1 || d > kMaxWidth) return 0;
    const size_t tokens = up256(static_cast<size_t>(M) * 8) * (M > kChunk ? 2 : 1);
    const size_t parts = M > kPiece ? up256(static_cast<size_t>(pieces_of(M)) * 2 * d * 4) : 0;
    return 256 + tokens + parts;
}

int32_t sb_embedding_backward(const int32_t *ids, const void *dout, int64_t M, int64_t d, int64_t V,
                              int32_t ignore_index, float scale, int32_t grad_type,
                              int32_t weight_type, int32_t add, void *dW, void *workspace,
                              size_t workspace_bytes, void *stream) {
    if (int32_t e = check_embedding(ids, M, d, V, scale, grad_type, weight_type)) return e;
    if ((M > 0 && !dout) || !dW || !workspace || add < 0 || add > 1) return SB_ERR_INVALID_ARG;
    if (!on(dout, grad_type == SB_F32 ? 4 : 2) || !on(dW, weight_type == SB_F32 ? 4 : 2) ||
        !on(workspace, 256))
        return SB_ERR_ALIGNMENT;
    if (int32_t e = device_sms_cc(nullptr, nullptr)) return e;
    if (workspace_bytes < sb_embedding_backward_workspace_bytes(M, d)) return SB_ERR_WORKSPACE_TOO_SMALL;
    if (M == 0 && add) return SB_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const size_t tokens = up256(static_cast<size_t>(M) * 8);
    int2 *sorted = reinterpret_cast<int2 *>(ws), *merged = sorted;
    ws += tokens;
    if (M > kChunk) {
        merged = reinterpret_cast<int2 *>(ws);
        ws += tokens;
    }
    SortParams s{};
    s.ids = ids;
    s.M = static_cast<int>(M);
    s.V = static_cast<int>(V);
    s.ignore = ignore_index;
    s.sort_blocks = static_cast<int>((M + 31) / 32);
    s.sorted = sorted;
    if (!add) {
        s.zero = static_cast<uint8_t *>(dW);
        s.zero_bytes = static_cast<size_t>(V) * d * (weight_type == SB_F32 ? 4 : 2);
    }
    const size_t keys = static_cast<size_t>(M < kChunk ? (M + 31) / 32 * 32 : kChunk) * 4;
    if (launch_dependent(sort_kernel, dim3(s.sort_blocks + (add ? 0 : kZeroBlocks)), kSortThreads,
                         keys, s, st) != cudaSuccess)
        return SB_ERR_CUDA;
    if (M == 0) return SB_OK;
    if (M > kChunk) {
        const MergeParams m{sorted, merged, static_cast<int>(M)};
        if (launch_dependent(merge_kernel, dim3(static_cast<unsigned>((M + 255) / 256)), 256, 0, m,
                             st) != cudaSuccess)
            return SB_ERR_CUDA;
    }
    ReduceParams r{};
    r.sorted = merged;
    r.dout = dout;
    r.dW = dW;
    r.part = reinterpret_cast<float *>(ws);
    r.M = static_cast<int>(M);
    r.pieces = static_cast<int>(pieces_of(M));
    r.d = d;
    r.scale = scale;
    r.add = add;
    const int vec = vector_width(d, dout, dW);
    using B = __nv_bfloat16;
    cudaError_t e;
    if (grad_type == SB_BF16)
        e = weight_type == SB_BF16 ? launch_sums<B, B>(r, vec, st) : launch_sums<B, float>(r, vec, st);
    else
        e = weight_type == SB_BF16 ? launch_sums<float, B>(r, vec, st)
                                   : launch_sums<float, float>(r, vec, st);
    return e == cudaSuccess ? SB_OK : SB_ERR_CUDA;
}

}  // extern "C"
