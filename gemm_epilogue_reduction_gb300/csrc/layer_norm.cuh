// layer_norm.cuh -- what the layer norm's kernels and their host side (layer_norm.cu) share: vectors
// of a row wherever it starts, and the branch's dropout.
#pragma once
#include "norm_common.cuh"
#include "sb_dropout.cuh"

namespace sb {

// How the arrays of rows are read, always as vectors of eight values of a thread:
//   kAligned   every row starts on a vector: 16-byte aligned arrays, d a multiple of 8;
//   kShifted   16-byte aligned arrays of any other d above 8: a row that starts s = row·d mod 8 values behind a
//              vector's boundary is read from there on, and what belongs to its neighbours is
//              masked (so vectors, and the four elements of a draw, lie as they do in kAligned);
//   kSingle    the rest: value by value.
enum LoadMode : int { kAligned = 0, kShifted = 1, kSingle = 2 };

constexpr int kNormVectors = 2;         // of a thread: sixteen values
constexpr int kNormThreads = 384;       // of a block, or, where a row's groups then fill it better,
constexpr int kWideThreads = 512;       // this many, with fewer registers; longer rows have up to 1024

struct LayerNormParams {
    int M, d;
    int row_threads;  // threads of a row's group, a multiple of 32
    int groups;       // of a block
    int steps;        // of a group's ring
    int w32;          // weights in fp32 (otherwise bf16)
    int wide_weights; // weight and bias on 16 bytes
    int shared_weights;  // forward, rows too long for the registers: kept in shared memory
    float eps, inv_d;
    const void *h, *y, *weight, *bias;
    void *h_out, *x;          // forward
    const void *dx, *dh;      // backward
    void *dh_out, *dy;
    float *part;              // [blocks][sums][d]: dx·(h - mean)·r, and dx
    int sums;
    Dropout drop;
};

struct LayerNormShape {
    LoadMode mode;
    bool h32;
    int threads;  // of a block
    int rows;     // that a group works on at a time
};

cudaError_t launch_layer_norm_forward(const LayerNormParams &p, LayerNormShape s, unsigned blocks,
                                      size_t smem, cudaStream_t st);
cudaError_t launch_layer_norm_backward(const LayerNormParams &p, LayerNormShape s, unsigned blocks,
                                       size_t smem, cudaStream_t st);

// Which values of a vector at e are the row's, a bit for each.  They are the same for all rows of a
// thread, and a test of a bit is all that the vectors at a row's ends cost more than the others.
template <int MODE>
__device__ __forceinline__ uint32_t inside8(int e, int d) {
    if (MODE == kAligned) return e < d ? 0xFFu : 0u;
    const uint32_t from = e < 0 ? 0xFFu << min(-e, 8) : 0xFFu;
    const uint32_t to = e + 8 > d ? 0xFFu >> min(e + 8 - d, 8) : 0xFFu;
    return from & to & 0xFFu;
}
// Zeros in the places of a vector that are not the row's (in kAligned no vector has both, and the
// ones past the row's end are zeros already).
template <int MODE>
__device__ __forceinline__ void mask8(uint32_t in, float2 (&v)[4]) {
    if constexpr (MODE != kAligned) {
        if (in == 0xFFu) return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!(in >> (2 * j) & 1)) v[j].x = 0.f;
            if (!(in >> (2 * j + 1) & 1)) v[j].y = 0.f;
        }
    }
}
// v less the row's mean; zeros stay past the row's ends, where they add nothing to the sums.
template <int MODE>
__device__ __forceinline__ void centre8(float mean, uint32_t in, float2 (&v)[4]) {
    const float m = MODE != kAligned || in ? -mean : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __fadd2_rn(v[j], both(m));
    mask8<MODE>(in, v);
}

template <typename T>
__device__ __forceinline__ void load_singles(const T *row, int e, int d, float2 (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = e + 2 * j;
        v[j].x = i >= 0 && i < d ? one(row + i) : 0.f;
        v[j].y = i + 1 >= 0 && i + 1 < d ? one(row + i + 1) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store_singles(T *row, int e, int d, const float2 (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = e + 2 * j;
        if (i >= 0 && i < d) put_one(row + i, v[j].x);
        if (i + 1 >= 0 && i + 1 < d) put_one(row + i + 1, v[j].y);
    }
}
// The row's values of the vector that is at `to`.
template <int MODE, typename T>
__device__ __forceinline__ void store8(T *to, uint32_t in, const float2 (&v)[4]) {
    if (MODE != kSingle && in == 0xFFu) {
        store_pairs<8>(to, v);
    } else if (MODE != kAligned) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (in >> (2 * j) & 1) put_one(to + 2 * j, v[j].x);
            if (in >> (2 * j + 1) & 1) put_one(to + 2 * j + 1, v[j].y);
        }
    }
}
template <int MODE>
__device__ __forceinline__ void load_weight8(const void *w, const LayerNormParams &p, int e,
                                             float2 (&v)[4]) {
    if (MODE == kAligned && p.wide_weights && e < p.d) {
        if (p.w32)
            load_pairs<8>(static_cast<const float *>(w) + e, v);
        else
            load_pairs<8>(static_cast<const __nv_bfloat16 *>(w) + e, v);
    } else if (p.w32) {
        load_singles(static_cast<const float *>(w), e, p.d, v);
    } else {
        load_singles(static_cast<const __nv_bfloat16 *>(w), e, p.d, v);
    }
}

// base + dropout(v) for the vector whose first value is element `at`.  state: of the draw of that
// element, which in kAligned and kShifted is the first of its draw's four.
template <int MODE>
__device__ __forceinline__ void add_dropped(const Dropout &drop, unsigned long long seed,
                                            unsigned long long state, unsigned long long at,
                                            const float2 (&base)[4], float2 (&v)[4]) {
    if (!drop.on) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __fadd2_rn(base[j], v[j]);
        return;
    }
    // what is masked is a zero, dropped or not
    if constexpr (MODE != kSingle) {
        dropout_add4(base, v, dropout_fields_at(state), drop.below, drop.scale);
        dropout_add4(base + 2, v + 2, dropout_fields_at(state + kGolden), drop.below, drop.scale);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const DropoutFields f = dropout_fields(seed, (at + j) / 4);
            const int k = static_cast<int>((at + j) & 3);
            const uint32_t w = k & 2 ? f.hi : f.lo, field = k & 1 ? w : w << 16;
            float &x = j & 1 ? v[j / 2].y : v[j / 2].x;
            x = fmaf(dropout_keep(x, field, drop.below), drop.scale,
                     j & 1 ? base[j / 2].y : base[j / 2].x);
        }
    }
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "r"(at)
                 : "memory");
    return x;
}
__device__ __forceinline__ void st_shared16(uint32_t at, uint4 x) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                 : "memory");
}

// One array of a row in a ring: a thread's vectors in pieces of 16 bytes, piece by piece over the
// group's threads, so that neighbours touch neighbours.  A thread copies its own vectors and reads
// them back: no barrier in between.  `at`: shared address of the thread's first piece; pitch: bytes
// from piece to piece.
template <typename T>
struct Slots {
    static constexpr int kPieces = static_cast<int>(sizeof(T)) / 2;  // of a vector of eight
    static constexpr int kThread = 16 * kPieces * kNormVectors;      // bytes of a thread
    // Vector i, which is at `from` in memory and at e in its row; whole: the array does not end in it.
    template <int MODE>
    static __device__ __forceinline__ void copy(uint32_t at, uint32_t pitch, int i, const T *from, int e,
                                                int d, bool whole) {
        if (e >= d) return;
        at += i * kPieces * pitch;
        if (MODE == kShifted && !whole) {
            float2 v[4];
            load_singles(from - e, e, d, v);
            put(at, pitch, 0, v);
            return;
        }
#pragma unroll
        for (int c = 0; c < kPieces; ++c)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + c * pitch),
                         "l"(from + c * (8 / kPieces))
                         : "memory");
    }
    // Zeros where `copy` never writes, past the row's end.
    static __device__ __forceinline__ void clear(uint32_t at, uint32_t pitch, int i, int e, int d) {
        if (e < d) return;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) st_shared16(at + (i * kPieces + c) * pitch, make_uint4(0, 0, 0, 0));
    }
    static __device__ __forceinline__ void put(uint32_t at, uint32_t pitch, int i, const float2 (&v)[4]) {
        if constexpr (kPieces == 1) {
            st_shared16(at + i * pitch, make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3])));
        } else {
#pragma unroll
            for (int c = 0; c < 2; ++c)
                st_shared16(at + (i * 2 + c) * pitch,
                            make_uint4(__float_as_uint(v[2 * c].x), __float_as_uint(v[2 * c].y),
                                       __float_as_uint(v[2 * c + 1].x), __float_as_uint(v[2 * c + 1].y)));
        }
    }
    static __device__ __forceinline__ void get(uint32_t at, uint32_t pitch, int i, float2 (&v)[4]) {
        if constexpr (kPieces == 1) {
            const uint4 x = ld_shared16(at + i * pitch);
            v[0] = unpack2(x.x), v[1] = unpack2(x.y), v[2] = unpack2(x.z), v[3] = unpack2(x.w);
        } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 x = ld_shared16(at + (i * 2 + c) * pitch);
                v[2 * c] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
                v[2 * c + 1] = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
            }
        }
    }
};

// Calls f.template operator()<T, MODE, BRANCH>() for the call's types and addresses.
template <typename F>
cudaError_t for_layer_norm(LayerNormShape s, bool branch, F f) {
    auto branched = [&]<typename T, int MODE>() {
        return branch ? f.template operator()<T, MODE, true>() : f.template operator()<T, MODE, false>();
    };
    auto typed = [&]<typename T>() {
        if (s.mode == kAligned) return branched.template operator()<T, kAligned>();
        if (s.mode == kShifted) return branched.template operator()<T, kShifted>();
        return branched.template operator()<T, kSingle>();
    };
    return s.h32 ? typed.template operator()<float>() : typed.template operator()<__nv_bfloat16>();
}

}  // namespace sb
