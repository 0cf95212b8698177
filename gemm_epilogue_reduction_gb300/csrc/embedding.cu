// embedding.cu -- the tokens' rows of the vocabulary matrix, and the gradient of that lookup.
//   forward    out_t = scale·W[id_t]            (zeros for the ignored index, NaN for other ids
//                                                outside the vocabulary)
//   backward   dW_v = [dW_v +] scale·sum over t with id_t = v of dout_t
//
// Forward moves the rows in and the rows out.  A row is a run of consecutive vectors of eight values;
// threads of a block take them side by side, several rows to a block where rows are short, up to four
// vectors (64 bytes) of loads in flight each.  8192 x 6144 bf16: 29.5 us, 73 % of the copy's rate: a block
// has one chain of id, row and store, and nothing of a next row on its way.  Rows of odd lengths are
// shifted into whole vectors: 8192 x 6143 34 us, against 71 value by value.
//
// Backward sums rows in a fixed order, so that equal calls give equal bits; atomics on fp32 values
// would not.  Its kernels:
//   sort_kernel    tokens by (id, position), in chunks of 8192: a token's place is the count of smaller
//                  keys, and of equal ones at earlier positions.  All pairs are compared, two
//                  tokens to a lane, the keys broadcast from shared memory, in one pass that waits
//                  for no other block.  Ids below 2^24 are compared as fp32: the saturated
//                  difference of two whole numbers is 1 or 0, an addition at full rate, where integer
//                  compares run at half of it (8192 tokens: 9 us against 17; sorted runs merged by
//                  binary search in a second kernel took 15).  When the whole gradient is asked for,
//                  further blocks of the same launch write its zeros meanwhile (that is most of its
//                  bytes: V rows against at most M that are not zero).
//   merge_kernel   eight chunks, or merged ones, to one: the counts of smaller keys in the others by
//                  binary search.
//   reduce_kernel  a block takes a piece of consecutive sorted tokens (of up to 64 in all: sorts them
//                  too) and a slice of columns, and adds the rows of each run of equal ids in
//                  registers; a run inside the piece is scaled, added and rounded here.  What a
//                  piece holds of a run that crosses its ends goes to the workspace in fp32.
//   join_kernel    adds the pieces' parts of such runs, in ascending order.  A run over many pieces
//                  has few blocks there: one id for all of 8192 x 6144 takes 68 us, where ids spread as
//                  in text take 43 and move more bytes.
// 8192 x 6144 bf16 into a matrix of 200,064 rows: 44 us, 9 of them the sort, 30 the rows (183 MB, 6.1
// TB/s: memory), 5 the join.  The whole gradient of 4096 x 4096, V = 151,936: 174 us, 7.3 TB/s.
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

// Rows of an odd length: a row of W and its row of the output start at different places of a vector's
// eight values.  A thread stores whole vectors of the output; what belongs into one lies in two vectors
// of W, and a shift through their registers, by the same number of values along the row, brings it into
// place.  (The second vector is the neighbour's first: it comes from L1.)
//
// Values from .. from + 8 of an array of n values, as 32-bit words; from: a multiple of eight.
template <typename T>
__device__ __forceinline__ void load_words(const T *base, long long from, long long n, uint32_t *w) {
    constexpr int WORDS = 2 * static_cast<int>(sizeof(T));
    if (from >= 0 && from + 8 <= n) {
#pragma unroll
        for (int c = 0; c < WORDS / 4; ++c) {
            const uint4 x = *reinterpret_cast<const uint4 *>(base + from + c * 4 * (4 / sizeof(T)));
            w[4 * c] = x.x, w[4 * c + 1] = x.y, w[4 * c + 2] = x.z, w[4 * c + 3] = x.w;
        }
        return;
    }
    // the array's end, or in front of it
#pragma unroll
    for (int j = 0; j < WORDS; ++j) {
        w[j] = 0;
        if constexpr (sizeof(T) == 4) {
            if (from + j >= 0 && from + j < n) w[j] = reinterpret_cast<const uint32_t *>(base)[from + j];
        } else {
            const uint16_t *b = reinterpret_cast<const uint16_t *>(base) + from + 2 * j;
            if (from + 2 * j >= 0 && from + 2 * j < n) w[j] = b[0];
            if (from + 2 * j + 1 >= 0 && from + 2 * j + 1 < n) w[j] |= static_cast<uint32_t>(b[1]) << 16;
        }
    }
}
// The eight values that begin r values behind the first of sixteen.
template <typename T>
__device__ __forceinline__ void shift_words(uint32_t (&w)[4 * sizeof(T)], int r, float2 (&v)[4]) {
    constexpr int WORDS = 4 * static_cast<int>(sizeof(T));
    const int words = sizeof(T) == 4 ? r : r >> 1;
#pragma unroll
    for (int by = WORDS / 4; by > 0; by >>= 1)
#pragma unroll
        for (int j = 0; j + by < WORDS; ++j) w[j] = words & by ? w[j + by] : w[j];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = unpack2(__funnelshift_r(w[j], w[j + 1], r & 1 ? 16 : 0));
    }
}

template <typename W, typename O>
__global__ void __launch_bounds__(kLookupThreads) lookup_shifted_kernel(const LookupParams p) {
    constexpr int U = 4 / sizeof(W);  // vectors in flight, two loads each and two of 16 bytes in fp32
    const int tx = kLookupThreads / p.rows;
    const int x = threadIdx.x % tx;
    const long long row = static_cast<long long>(blockIdx.x) * p.rows + threadIdx.x / tx;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // no early launch_dependents: as above
    if (row >= p.M) return;
    const int id = p.ids[row];
    const bool has = id >= 0 && id < p.V && id != p.ignore;
    const float none = id == p.ignore ? 0.f : __uint_as_float(0x7FC00000u);
    const W *all = static_cast<const W *>(p.W);
    const long long n = p.V * p.d, at = has ? id * p.d : 0;
    O *to = static_cast<O *>(p.out) + row * p.d;
    const int shift = static_cast<int>(row * p.d & 7), r = static_cast<int>((at - shift) & 7);
    for (long long e0 = x * 8 - shift; e0 < p.d; e0 += U * tx * 8) {
        uint32_t w[U][4 * sizeof(W)];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long e = e0 + u * tx * 8;
            if (has && e < p.d) {
                load_words(all, at + e - r, n, w[u]);
                load_words(all, at + e - r + 8, n, w[u] + 2 * sizeof(W));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long e = e0 + u * tx * 8;
            if (e >= p.d) break;
            float2 v[4] = {both(none), both(none), both(none), both(none)};
            if (has) {
                shift_words<W>(w[u], r, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(v[j], both(p.scale));
            }
            if (e >= 0 && e + 8 <= p.d) {
                store_pairs<8>(to + e, v);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (e + j >= 0 && e + j < p.d) put_one(to + e + j, j & 1 ? v[j / 2].y : v[j / 2].x);
            }
        }
    }
}

template <typename W, typename O>
cudaError_t launch_lookup(LookupParams p, int vec, cudaStream_t st) {
    if (vec == 1 && p.d > 8 && on(p.W, 16) && on(p.out, 16)) {
        int tx = 8;
        while (tx < kLookupThreads && tx * (4 / static_cast<long long>(sizeof(W))) * 8 < p.d + 7) tx *= 2;
        p.rows = kLookupThreads / tx;
        const dim3 grid(static_cast<unsigned>((p.M + p.rows - 1) / p.rows));
        return launch_dependent(lookup_shifted_kernel<W, O>, grid, kLookupThreads, 0, p, st);
    }
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
constexpr int kSortThreads = 1024;
constexpr int kSortTokens = 64;      // of a block, two to a lane
constexpr int kChunk = 8192;         // tokens whose keys a block holds in shared memory
static_assert(kSortTokens == 2 * 32 && kChunk % kSortTokens == 0, "two tokens to a lane");

struct SortParams {
    const int32_t *ids;
    int M, V, ignore;
    int sort_blocks;
    int last;          // no kernel of this call follows
    uint32_t *key;     // sorted within each chunk
    int *at;           // their positions
    uint8_t *zero;     // bytes to clear (null: none)
    size_t zero_bytes;
};

// A block's share of the zeros; values are 2 or 4 bytes wide, and so is what lies before and behind
// the 32-byte units.  A store to a thread and 32 KB to a block: 1.24 GB in 163 us, against 192 where
// blocks of a grid that just fills the GPU (or bulk stores) go over the matrix in turn.
__device__ __forceinline__ void clear_share(uint8_t *p, size_t n, size_t block) {
    size_t head = (32 - (reinterpret_cast<uintptr_t>(p) & 31)) & 31;
    if (head > n) head = n;
    const size_t o = head + (block * kSortThreads + threadIdx.x) * 32;
    if (o + 32 <= n) {
        st_global_v8(p + o, 0, 0, 0, 0, 0, 0, 0, 0);
    } else {
        for (size_t i = o; i < n; i += 2) *reinterpret_cast<uint16_t *>(p + i) = 0;
    }
    if (block == 0 && threadIdx.x < head / 2) reinterpret_cast<uint16_t *>(p)[threadIdx.x] = 0;
}

// How many of four keys are below each lane's limit.  AS_FLOAT: whole numbers up to 2^25 as fp32, in
// pairs of counts.
struct Count {
    float2 f;
    int i;
};
template <bool AS_FLOAT>
__device__ __forceinline__ void count_below(Count &c, uint4 k, uint32_t limit) {
    if constexpr (AS_FLOAT) {
        const float l = __uint_as_float(limit);
        c.f = __fadd2_rn(c.f, make_float2(__saturatef(l - __uint_as_float(k.x)),
                                          __saturatef(l - __uint_as_float(k.y))));
        c.f = __fadd2_rn(c.f, make_float2(__saturatef(l - __uint_as_float(k.z)),
                                          __saturatef(l - __uint_as_float(k.w))));
    } else {
        c.i += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
    }
}

template <bool AS_FLOAT>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const SortParams p) {
    constexpr int WARPS = kSortThreads / 32;
    __shared__ __align__(16) uint32_t keys[kChunk];
    __shared__ int counts[WARPS][kSortTokens];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!p.last) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (static_cast<int>(blockIdx.x) >= p.sort_blocks) {
        clear_share(p.zero, p.zero_bytes, blockIdx.x - p.sort_blocks);
        return;
    }
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int base = blockIdx.x / (kChunk / kSortTokens) * kChunk;
    const int n = min(kChunk, p.M - base), groups = (n + 31) / 32;
    const int mine = blockIdx.x % (kChunk / kSortTokens) * (kSortTokens / 32);  // my first group of 32
    // what is compared: the number, or its fp32; a limit is the next number
    auto coded = [](uint32_t v) { return AS_FLOAT ? __float_as_uint(static_cast<float>(v)) : v; };
    // (fp32 has every whole number up to 2^24, the limit of kNone's equals)
    constexpr uint32_t kNone = AS_FLOAT ? (1u << 24) - 1 : kNoToken, kBehind = AS_FLOAT ? 1u << 25 : ~0u;
    auto key_of = [&](int j) {
        if (j >= n) return kBehind;  // behind the last token: never counted
        const int id = p.ids[base + j];
        return id >= 0 && id < p.V && id != p.ignore ? static_cast<uint32_t>(id) : kNone;
    };
#pragma unroll 8
    for (int j = tid; j < groups * 32; j += kSortThreads) keys[j] = coded(key_of(j));
    uint32_t key[2], below[2], up_to[2];
    Count c[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        key[k] = key_of((mine + k) * 32 + lane);
        below[k] = coded(key[k]);
        up_to[k] = coded(key[k] + 1);  // equal keys count where they come before
        c[k] = Count{both(0.f), 0};
    }
    __syncthreads();
    for (int g = warp; g < groups; g += WARPS) {
        const uint4 *k4 = reinterpret_cast<const uint4 *>(keys) + g * 8;
        if (g < mine || g > mine + 1) {
            const uint32_t l0 = g < mine ? up_to[0] : below[0], l1 = g < mine ? up_to[1] : below[1];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4 k = k4[j];
                count_below<AS_FLOAT>(c[0], k, l0);
                count_below<AS_FLOAT>(c[1], k, l1);
            }
        } else {
            // a group of my own tokens: equal keys of it count below their lane
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {
                const uint32_t k = keys[g * 32 + j];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const bool before = g < mine + t || (g == mine + t && j < lane);
                    const uint32_t l = before ? up_to[t] : below[t];
                    c[t].i += AS_FLOAT ? __uint_as_float(k) < __uint_as_float(l) : k < l;
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)  // (counts up to 8192 are exact)
        counts[warp][t * 32 + lane] = c[t].i + static_cast<int>(c[t].f.x + c[t].f.y);
    __syncthreads();
    if (warp < 2 && (mine + warp) * 32 + lane < n) {
        int rank = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) rank += counts[w][warp * 32 + lane];
        const uint32_t k = warp ? key[1] : key[0];
        p.key[base + rank] = k == kNone ? kNoToken : k;
        p.at[base + rank] = base + (mine + warp) * 32 + lane;
    }
}

// Sorted runs become runs of kFan times their length: a token's place is its place in its own run and the
// counts of smaller keys (of keys not larger, in earlier runs) in the others.
struct MergeParams {
    const uint32_t *key;
    const int *at;
    uint32_t *to_key;
    int *to_at;
    int M;
    long long run;
};
constexpr int kMergeThreads = 256;
constexpr int kFan = 8;

__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const MergeParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long i = static_cast<long long>(blockIdx.x) * kMergeThreads + threadIdx.x;
    if (i >= p.M) return;
    const uint32_t key = p.key[i];
    const long long base = i / (kFan * p.run) * (kFan * p.run);
    const int own = static_cast<int>((i - base) / p.run);
    long long place = i - own * p.run;
#pragma unroll
    for (int c = 0; c < kFan; ++c) {
        const long long from = base + c * p.run;
        const uint32_t *k = p.key + from;
        const uint32_t limit = key + (c < own);
        long long lo = 0, hi = c == own ? 0 : max(0LL, min(p.run, p.M - from));
        while (lo < hi) {
            const long long mid = (lo + hi) / 2;
            if (k[mid] < limit)
                lo = mid + 1;
            else
                hi = mid;
        }
        place += lo;
    }
    p.to_key[place] = key;
    p.to_at[place] = p.at[i];
}

// ------------------------------------------------------------------ backward: sums
constexpr int kPiece = 32;           // sorted tokens of a block, or twice as many:
constexpr int kLongPiece = 64;
constexpr int kReduceThreads = 128;
constexpr int kAhead = 8;            // rows in flight
static_assert(kPiece % kAhead == 0 && kLongPiece % kAhead == 0 && kLongPiece + 2 <= kReduceThreads);

struct ReduceParams {
    const int32_t *ids;  // of one piece at most: every block sorts them itself (null: key and at are given)
    int V, ignore;
    const uint32_t *key;
    const int *at;
    const void *dout;
    void *dW;
    float *part;  // [pieces][2][d]: of the run that comes in from the piece before, and of the one
                  // that starts here and goes on behind
    int M, piece, pieces;
    long long d;
    float scale;
    int add;
};

// VEC values as they lie in memory: what is on its way takes no more registers than bytes.
template <typename T, int VEC>
using Raw = std::conditional_t<VEC == 1, T, std::conditional_t<VEC * sizeof(T) == 16, uint4, uint2>>;
template <int VEC, typename T>
__device__ __forceinline__ void widen(const Raw<T, VEC> &x, float2 (&v)[(VEC + 1) / 2], T) {
    if constexpr (VEC == 1)
        v[0] = make_float2(one(&x), 0.f);
    else if constexpr (sizeof(T) == 4)
        v[0] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y)),
        v[1] = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
    else if constexpr (VEC == 8)
        v[0] = unpack2(x.x), v[1] = unpack2(x.y), v[2] = unpack2(x.z), v[3] = unpack2(x.w);
    else
        v[0] = unpack2(x.x), v[1] = unpack2(x.y);
}

template <typename G, typename W, int VEC, bool ADD>
__global__ void __launch_bounds__(kReduceThreads) reduce_kernel(const ReduceParams p) {
    constexpr int N = (VEC + 1) / 2;
    using RG = Raw<G, VEC>;
    using RW = Raw<W, VEC>;
    __shared__ int2 token[kLongPiece + 2];  // (key, position); key -1: none
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Where join_kernel follows it may get ready (it waits for this kernel's end); else no early
    // launch_dependents: nothing that follows may read dW ahead of that.
    if (p.pieces > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int first = blockIdx.x * p.piece, tid = threadIdx.x;
    if (p.ids) {
        __shared__ int keys[kLongPiece];
        if (tid < kLongPiece + 2) token[tid] = make_int2(-1, 0);
        if (tid < kLongPiece) {
            const int id = tid < p.M ? p.ids[tid] : -1;
            keys[tid] = id >= 0 && id < p.V && id != p.ignore ? id : kNoToken;
        }
        __syncthreads();
        if (tid < kLongPiece && keys[tid] != kNoToken) {
            int rank = 0;
#pragma unroll 16
            for (int j = 0; j < kLongPiece; ++j) rank += keys[j] < keys[tid] + (j < tid);
            token[1 + rank] = make_int2(keys[tid], tid);
        }
    } else if (tid < p.piece + 2) {
        const int i = first + tid - 1;
        int2 t = make_int2(-1, 0);
        if (i >= 0 && i < p.M) {
            t = make_int2(static_cast<int>(p.key[i]), p.at[i]);
            if (t.x == kNoToken) t.x = -1;
        }
        token[tid] = t;
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
    for (int k0 = 1; k0 <= p.piece; k0 += kAhead) {
        if (token[k0].x < 0) break;
        RG v[kAhead];
        RW old[ADD ? kAhead : 1];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int2 t = token[k0 + u];
            if (t.x >= 0) v[u] = *reinterpret_cast<const RG *>(dout + static_cast<size_t>(t.y) * p.d);
            if constexpr (ADD)
                if (t.x >= 0 && t.x != token[k0 + u + 1].x)
                    old[u] = *reinterpret_cast<const RW *>(dW + static_cast<size_t>(t.x) * p.d);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int2 t = token[k0 + u];
            if (t.x < 0) break;
            const bool ends = t.x != token[k0 + u + 1].x;
            float2 x[N];
            widen<VEC>(v[u], x, G{});
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = __fadd2_rn(acc[j], x[j]);
            if (!ends && k0 + u < p.piece) continue;
            if (ends && !came) {
                if constexpr (ADD)
                    widen<VEC>(old[u], x, W{});
                else
#pragma unroll
                    for (int j = 0; j < N; ++j) x[j] = both(0.f);
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = __ffma2_rn(acc[j], both(p.scale), x[j]);
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

// The run that starts in a piece and ends in a later one: its parts in ascending order, or, where
// they are many, sixteen slices of them side by side and then the slices.
constexpr int kJoinSlices = 16;
template <typename W, int VEC>
__global__ void __launch_bounds__(32 * kJoinSlices) join_kernel(const ReduceParams p) {
    constexpr int N = (VEC + 1) / 2;
    __shared__ float2 sums[kJoinSlices][32][N];
    // What it reads before it waits for reduce_kernel's end: the order, which was complete before any
    // block of reduce_kernel let this kernel start, and rows of dW, where none are reduce_kernel's.
    const int piece = blockIdx.x, lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int behind = (piece + 1) * p.piece;  // (of a piece that is not the last one)
    const uint32_t key = p.key[behind - 1];
    const uint32_t before = piece > 0 ? p.key[behind - p.piece - 1] : kNoToken;
    // the pieces behind that begin with the run's key: 32 at a time, the first of them beside the
    // loads above
    int parts = 1;
    for (int q = piece + 1;; q += 32) {
        const bool more = q + lane < p.pieces && p.key[(q + lane) * p.piece] == key;
        const uint32_t with = __ballot_sync(0xFFFFFFFFu, more);
        parts += __popc(with);
        if (with != 0xFFFFFFFFu) break;
    }
    if (key == kNoToken || parts == 1 || before == key) {  // (before: it started earlier)
        // every block waits: what follows on the stream waits for this kernel alone
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    // few parts: every warp has columns of its own; many: the warps share the parts
    const bool share = parts > 2 * kJoinSlices;
    const int q0 = share ? static_cast<int>(static_cast<long long>(parts) * slice / kJoinSlices) : 0;
    const int q1 = share ? static_cast<int>(static_cast<long long>(parts) * (slice + 1) / kJoinSlices) : parts;
    const int width = (share ? 32 : 32 * kJoinSlices) * VEC;
    for (long long e0 = static_cast<long long>(blockIdx.y) * width; e0 < p.d;
         e0 += static_cast<long long>(gridDim.y) * width) {
        const long long e = e0 + (share ? lane : static_cast<int>(threadIdx.x)) * VEC;
        W *to = static_cast<W *>(p.dW) + static_cast<size_t>(key) * p.d + e;
        float2 acc[N], old[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = old[j] = both(0.f);
        if (p.add && (!share || slice == 0) && e < p.d) {
            if constexpr (VEC == 1)
                old[0].x = one(to);
            else
                load_pairs<VEC>(to, old);
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
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
        if (share) {
#pragma unroll
            for (int j = 0; j < N; ++j) sums[slice][lane][j] = acc[j];
            __syncthreads();
#pragma unroll
            for (int s = 1; s < kJoinSlices; ++s)
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = __fadd2_rn(acc[j], sums[s][lane][j]);
        }
        if ((!share || slice == 0) && e < p.d) {
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = __ffma2_rn(acc[j], both(p.scale), old[j]);
            if constexpr (VEC == 1)
                put_one(to, acc[0].x);
            else
                store_pairs<VEC>(to, acc);
        }
        if (share) __syncthreads();
    }
}

template <typename G, typename W, int VEC>
cudaError_t launch_sums(const ReduceParams &p, cudaStream_t st) {
    const long long slices = (p.d + kReduceThreads * VEC - 1) / (kReduceThreads * VEC);
    const dim3 grid(p.pieces, static_cast<unsigned>(slices));
    cudaError_t e =
        p.add ? launch_dependent(reduce_kernel<G, W, VEC, true>, grid, kReduceThreads, 0, p, st)
              : launch_dependent(reduce_kernel<G, W, VEC, false>, grid, kReduceThreads, 0, p, st);
    if (e != cudaSuccess || p.pieces == 1) return e;
    constexpr int J = VEC == 1 ? 1 : 4;  // four values to a lane, of fp32 parts
    const long long cols = (p.d + 32 * kJoinSlices * J - 1) / (32 * kJoinSlices * J);
    return launch_dependent(join_kernel<W, J>, dim3(p.pieces - 1, static_cast<unsigned>(cols)),
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

int64_t pieces_of(int64_t M, int piece) { return (M + piece - 1) / piece; }

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
    const size_t ws = weight_type == SB_F32 ? 4 : 2, os = out_type == SB_F32 ? 4 : 2;
    if (overlap(out, M * d * os, W, V * d * ws) || overlap(out, M * d * os, ids, M * 4))
        return SB_ERR_INVALID_ARG;
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

// [keys, positions] [the same, of the chunks merged (beyond one chunk)] [parts]
size_t sb_embedding_backward_workspace_bytes(int64_t M, int64_t d) {
    if (M < 0 || M > kMaxTokens || d < 1 || d > kMaxWidth) return 0;
    const size_t tokens = up256(static_cast<size_t>(M) * 4) * (M > kChunk ? 4 : 2);
    const size_t parts = M > kPiece ? up256(static_cast<size_t>(pieces_of(M, kPiece)) * 2 * d * 4) : 0;
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
    const size_t dw_bytes = V * d * (weight_type == SB_F32 ? 4 : 2);
    const size_t dout_bytes = M * d * (grad_type == SB_F32 ? 4 : 2);
    const size_t need = sb_embedding_backward_workspace_bytes(M, d);
    const Span arrays[] = {{workspace, need}, {dW, dw_bytes}, {dout, dout_bytes}, {ids, static_cast<size_t>(M) * 4}};
    if (any_overlap(arrays, 2)) return SB_ERR_INVALID_ARG;
    int sms = 0;
    if (int32_t e = device_sms_cc(&sms, nullptr)) return e;
    if (workspace_bytes < need) return SB_ERR_WORKSPACE_TOO_SMALL;
    if (M == 0 && add) return SB_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const size_t array = up256(static_cast<size_t>(M) * 4);
    uint32_t *key[2];
    int *at[2];
    for (int k = 0; k < (M > kChunk ? 2 : 1); ++k, ws += 2 * array) {
        key[k] = reinterpret_cast<uint32_t *>(ws);
        at[k] = reinterpret_cast<int *>(ws + array);
    }
    int now = 0;  // where the tokens are
    SortParams s{};
    s.ids = ids;
    s.M = static_cast<int>(M);
    s.V = static_cast<int>(V);
    s.ignore = ignore_index;
    const bool few = M <= kLongPiece;  // reduce_kernel sorts them itself
    s.sort_blocks = few ? 0 : static_cast<int>((M + kSortTokens - 1) / kSortTokens);
    s.last = M == 0;
    s.key = key[0];
    s.at = at[0];
    if (!add) {
        s.zero = static_cast<uint8_t *>(dW);
        s.zero_bytes = static_cast<size_t>(V) * d * (weight_type == SB_F32 ? 4 : 2);
    }
    // (rounded up, and one more for what an unaligned head shifts to the end)
    const size_t zero_blocks = add ? 0 : s.zero_bytes / (kSortThreads * 32) + 1;
    if (zero_blocks > (size_t(1) << 30)) return SB_ERR_INVALID_ARG;
    const dim3 grid(s.sort_blocks + static_cast<unsigned>(zero_blocks));
    if (grid.x > 0 &&
        (V < 1 << 24 ? launch_dependent(sort_kernel<true>, grid, kSortThreads, 0, s, st)
                      : launch_dependent(sort_kernel<false>, grid, kSortThreads, 0, s, st)) != cudaSuccess)
        return SB_ERR_CUDA;
    if (M == 0) return SB_OK;
    for (int64_t run = kChunk; run < M; run *= kFan, now = 1 - now) {
        const MergeParams m{key[now], at[now], key[1 - now], at[1 - now], static_cast<int>(M), run};
        if (launch_dependent(merge_kernel, dim3(static_cast<unsigned>((M + kMergeThreads - 1) / kMergeThreads)),
                             kMergeThreads, 0, m, st) != cudaSuccess)
            return SB_ERR_CUDA;
    }
    ReduceParams r{};
    r.ids = few ? ids : nullptr;
    r.V = static_cast<int>(V);
    r.ignore = ignore_index;
    r.key = key[now];
    r.at = at[now];
    r.dout = dout;
    r.dW = dW;
    r.part = reinterpret_cast<float *>(ws);
    r.M = static_cast<int>(M);
    r.d = d;
    r.scale = scale;
    r.add = add;
    const int vec = vector_width(d, dout, dW);
    // Long pieces where they fill the GPU four times over, and where one is all there is, so that there
    // is nothing to join; else twice the blocks are worth more.  Long against short, in us (bf16, 50,257
    // rows): 8192 x 6144 41.0 and 43.0, 8192 x 5120 35.7 and 37.6, 65,536 x 768 121.7 and 124.6; below the
    // limit 1000 x 4096 15.3 and 10.9, 4096 x 6144 23.2 and 19.3.
    const int64_t slices = (d + kReduceThreads * vec - 1) / (kReduceThreads * vec);
    const bool long_pieces = M <= kLongPiece || pieces_of(M, kLongPiece) * slices >= 4 * sms;
    r.piece = long_pieces ? kLongPiece : kPiece;
    r.pieces = static_cast<int>(pieces_of(M, r.piece));
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
