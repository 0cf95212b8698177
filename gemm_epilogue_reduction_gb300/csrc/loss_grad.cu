// loss_grad.cu -- the gradient of the output head's cross entropy, in pieces of the
// vocabulary, without keeping logits.
//
// With z = H·Wᵀ, lse_r = log sum_j exp(z_rj), t_r the target of row r, g_r the gradient of the
// loss in row r's loss and l = z_loss weight, row r's loss is lse_r - z_rt + l·lse_r², so
//   G_rj = dL/dz_rj = g_r·((1 + 2·l·lse_r)·exp(z_rj - lse_r) - [j = t_r]),
//   dH = G·W,   dW = Gᵀ·H,
// three products of 2·M·d·V operations (the logits are formed again from H and W).  Rows whose
// target is the ignored index have G = 0.  For each piece of `cols` vocabulary columns:
//   logits_kernel    z tile by tile as in the forward pass, and G in bf16 through shared memory
//                    into the piece buffer [M][cols]; with the first piece also a copy of H whose
//                    ignored rows are zero, so that what those rows hold (an infinity, a NaN)
//                    does not meet the zeros of G in dW;
//   operands_kernel  one launch for both products that read G: the dH tiles (reduction over
//                    the piece's columns) and the dW tiles (reduction over the rows);
// and, when the dH reduction was split, sum_kernel adds the splits in ascending order.
//
// G is held in bf16, the type of the tensor cores' operands here: a relative error of 2^-8 at
// most per entry (rms 2^-9), independent from entry to entry, so that a sum over many of them
// loses less than the rounding of dH and dW to bf16 does.  For that the scale that all rows share
// (the incoming gradient, 1/count, or the largest |g|) stays out of G and is applied in fp32 in
// the epilogue: rounding it into G would shift every entry the same way.  A few rows have few
// large entries (their targets'), whose roundings do not average out, so up to 32 rows G is held as
// two bf16 numbers, the value and what its rounding left (2^-16 together): the second ones are
// further rows of G, which fill the row tile and the 64-wide reduction block that few rows leave
// empty.  Accumulation is fp32 in TMEM and, over the pieces, fp32 in memory.
//
// Bounds.  From some 2000 rows on the tensor cores (and under a long load the power limit): 4096 x
// 6144 x 200,064 takes 23.4 to 24.3 ms forward and backward, 1.66 to 1.72 PFLOP/s over its four
// products of 2·M·d·V (the logits are formed twice), 97 to 100 % of a library product's rate under
// the same load; the kernels have 90 to 92 % of the tensor pipe's cycles there.  Around 500 rows what L2 delivers to
// an SM (some 54 bytes a cycle; a 256 x 256 tile wants 64 per CTA for the full tensor rate, and a
// dW tile of so few rows stores 64 KB besides).  For few rows the memory: W is read three times
// (forward, logits, dH) and dW written once: 64 x 4096 x 151,936 takes 787 to 817 us (at 797:
// forward 189, logits 195, dH 204, dW 209).
//
// Both kernels: persistent CTA pairs, one cta_group::2 MMA of 256 x 256 per 16-wide K step
// (tcgen05, bf16 x bf16 -> fp32), joint TMA stages, two TMEM accumulators, eight epilogue
// warps; bounded waits as in sb_pipe.cuh.  Operands whose reduction index is the outer one in
// memory (W in dH = G·W; G and H in dW = Gᵀ·H) are staged in boxes of 64 contiguous elements x
// 64 reduction rows and read by the MMA "MN-major", so that nothing is transposed.
#include <atomic>
#include <cuda_bf16.h>
#include <type_traits>

#include "loss_common.cuh"
#include "sb_internal.h"
#include "sb_pipe.cuh"
#include "sb_ptx.cuh"

namespace sb {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 256;                       // rows and columns of a pair's tile
constexpr uint32_t kAtomBytes = kTileA * 128;    // one operand, one CTA, 64 of the reduction
constexpr uint32_t kOutBytes = 32 * 128;         // an output box: 32 rows x 64 bf16

// ATOMS 64-wide slices of the reduction per stage: 2 halves the waits and commits per operation;
// 1, for few rows, gives more stages and a second output box per epilogue warp (of few rows a dW
// tile is written nearly as fast as it is computed).  Every operand box is 64 elements (128
// bytes) wide and 64 * ATOMS rows high, two boxes to an operand.
template <int ATOMS>
struct Ring {
    static constexpr int kBoxRows = 64 * ATOMS;
    static constexpr uint32_t kBoxBytes = kBoxRows * 128;
    static constexpr uint32_t kOperand = ATOMS * kAtomBytes;
    static_assert(kOperand == 2 * kBoxBytes);
    static constexpr uint32_t kStage = 2 * kOperand;  // A, then B
    static constexpr int kStages = ATOMS == 1 ? 5 : 3;
    static constexpr int kOutBoxes = ATOMS == 1 ? 2 : 1;
    // shared memory: stages, output boxes, barriers and scalars
    static constexpr uint32_t kOutAt = kStages * kStage;
    static constexpr uint32_t kBarAt = kOutAt + kEpiWarps * kOutBoxes * kOutBytes;
    static constexpr uint32_t kSmem = kBarAt + 1024 + 1024 /* align */;
    static_assert(kSmem <= kSmemLimit);
};

// Shared-memory matrix descriptor of an MN-major bf16 operand: two blocks of 64 contiguous M (or
// N) elements (128 bytes, 128-byte swizzle) x the stage's reduction rows, as a TMA box leaves
// them.  Leading byte offset: from one block of 64 elements to the next; stride byte offset:
// from 8 reduction rows to the next 8 (1024 bytes).  A 16-wide K step adds 2048 bytes.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(block_bytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// This CTA's 128 rows (columns of the output, for B) of an operand from `mn`, reduction indexes
// from `k`, `boxes` (0 to 2) of its boxes.  MN: the map's x is the operand's row and y the
// reduction index; else the other way round.  What is not loaded keeps whatever shared memory
// held: those rows of the operand meet only rows (columns) of the output that nothing stores.
template <bool MN, int ATOMS>
__device__ __forceinline__ void load_operand(uint8_t *dst, const CUtensorMap *tm, uint32_t bar,
                                             int mn, int k, uint64_t pol, int boxes) {
    using R = Ring<ATOMS>;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (b >= boxes) break;
        uint8_t *to = dst + b * R::kBoxBytes;
        if (MN)
            tma_load_2d_pair(to, tm, bar, mn + 64 * b, k, pol);
        else if (ATOMS == 2)
            tma_load_2d_pair(to, tm, bar, k + 64 * b, mn, pol);
        else
            tma_load_2d_pair(to, tm, bar, k, mn + 64 * b, pol);
    }
}
// The boxes of a K-major operand's rows from mn that hold any of `rows` rows.
template <int ATOMS>
__device__ __forceinline__ int boxes_of(int rows, int mn) {
    if (ATOMS == 2) return rows > mn ? 2 : 0;  // both 64-wide slices of the same 128 rows
    return min(max((rows - mn + 63) >> 6, 0), 2);
}
constexpr uint32_t kIdescAMajorMN = 1u << 15, kIdescBMajorMN = 1u << 16;

// One 256 x 256 tile of work.
struct Unit {
    bool dw;             // operands_kernel: a tile of dW (otherwise of dH)
    int row0, col0;      // of the output, this CTA's rows
    int split;
    int k0, kblocks;     // first reduction index and blocks of ATOMS * 64
    int slices;          // 64-wide slices of the last block that hold anything
    int n;               // columns of the tile that the MMA forms: 256, less (a multiple of 32) in
                         // the last tile of dH and dW
};

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }
// t / d and t % d with inv = min(floor(2^32 / d), 2^32 - 1): the product is one too low at most.
// (Every role walks through the units; with integer divisions that took longer than the MMAs of
// a dW tile of 64 tokens.)
__device__ __forceinline__ void div_mod(int t, int d, uint32_t inv, int &q, int &r) {
    q = static_cast<int>(__umulhi(static_cast<uint32_t>(t), inv));
    r = t - q * d;
    if (r >= d) {
        ++q;
        r -= d;
    }
}

// The units of one pair, in order.  Logits: the tiles dealt out in turn, neighbouring pairs on
// the same tile of W.  Operands: the dH units, which are long (the piece's columns), are dealt
// out in turn; the short dW tiles then even out the pairs: those that are one dH unit behind
// the others take `fill` dW tiles each before the rest is dealt out in turn.
//
// (With few rows dH reads W and dW writes its gradient.  Letting half of the pairs start with dW,
// so that reads and writes overlap, was slower: 747 against 681 us for the backward call at 64 x
// 4096 x 151,936, when that was measured.)
template <bool LOGITS, int ATOMS>
struct Walk {
    static constexpr int KB = ATOMS * kBlockK;
    const LossGradParams &p;
    int pair, pairs, rank, own, rem, n;

    __device__ __forceinline__ Walk(const LossGradParams &p, int pair, int pairs, int rank)
        : p(p), pair(pair), pairs(pairs), rank(rank), own(0), rem(0) {
        if (LOGITS) {
            n = div_up(max(p.row_tiles * p.col_tiles - pair, 0), pairs);
            return;
        }
        rem = p.dh_units % pairs;
        own = p.dh_units / pairs + (pair < rem ? 1 : 0);
        const int late = pairs - rem;  // pairs that are behind (all of them if rem == 0)
        n = own;
        int taken = 0, turn = pair;    // dW tiles of the first dealing; this pair's place after it
        if (rem != 0) {
            taken = min(late * p.fill, p.dw_units);
            turn = pair >= rem ? pair - rem : late + pair;
            if (pair >= rem) n += div_up(max(taken - turn, 0), late);
        }
        n += div_up(max(p.dw_units - taken - turn, 0), pairs);
    }

    // the blocks of `len` reduction indexes
    static __device__ __forceinline__ void reduce_over(Unit &u, int len) {
        u.kblocks = div_up(len, KB);
        u.slices = ATOMS - (u.kblocks * KB - len) / kBlockK;
    }
    // the columns of a tile of dH or dW
    __device__ __forceinline__ void columns(Unit &u, int tile) const {
        u.col0 = tile * kTile;
        u.n = min(kTile, (p.d - u.col0 + 31) & ~31);
    }

    __device__ __forceinline__ Unit at(int i) const {
        Unit u;
        u.split = 0;
        u.k0 = 0;
        u.dw = false;
        int q, r;
        if (LOGITS) {
            div_mod(pair + i * pairs, p.row_tiles, p.row_tiles_inv, q, r);
            u.col0 = q * kTile;
            u.row0 = r * kTile + rank * kTileA;
            u.n = kTile;
            reduce_over(u, p.d);
            return u;
        }
        if (i < own) {
            div_mod(pair + i * pairs, p.d_tiles, p.d_tiles_inv, q, r);
            u.split = q / p.row_tiles;
            u.row0 = (q - u.split * p.row_tiles) * kTile + rank * kTileA;
            columns(u, r);
            const int blocks = div_up(p.cols, KB);
            const long long blocks64 = blocks;
            const int b0 = static_cast<int>(blocks64 * u.split / p.splits);
            const int b1 = static_cast<int>(blocks64 * (u.split + 1) / p.splits);
            u.k0 = b0 * KB;
            reduce_over(u, min(b1 * KB, p.cols) - u.k0);
            return u;
        }
        int j = i - own, t;
        if (rem == 0) {
            t = j * pairs + pair;
        } else {
            const int late = pairs - rem, first = min(late * p.fill, p.dw_units);
            if (pair >= rem) {
                const int mine = div_up(max(first - (pair - rem), 0), late);
                t = j < mine ? j * late + (pair - rem) : first + (j - mine) * pairs + (pair - rem);
            } else {
                t = first + j * pairs + late + pair;
            }
        }
        div_mod(t, p.d_tiles, p.d_tiles_inv, q, r);
        u.dw = true;
        u.row0 = q * kTile + rank * kTileA;
        columns(u, r);
        reduce_over(u, p.g_rows);
        return u;
    }
};

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Everything that the kernel before may have written is read with __ldcg: that kernel can still be
// running when this one starts, which the read-only path of __ldg does not allow for.
// The incoming gradient where it is one number (SUM, MEAN), else 1.
__device__ __forceinline__ float incoming(const LossGradParams &p) {
    return (p.reduction != 0 && p.grad) ? __ldcg(p.grad) : 1.f;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// The scale that all rows share, by all 256 epilogue threads (e = 0..255); red: 16 words of
// shared memory.  SUM: the incoming gradient; MEAN: that over the count of rows that are not
// ignored (at least 1); NONE: the largest |g_r| of those rows.  It multiplies every row, so it is
// always finite and (NONE) above zero: infinities and NaN stay with the rows' own weights.
__device__ __forceinline__ float shared_scale(const LossGradParams &p, int e, float *red) {
    const float all = incoming(p), up = finite(all) ? all : 1.f;
    if (p.reduction == 1 || (p.reduction == 0 && !p.grad)) return up;
    float best = 0.f;
    int count = 0;
    for (int r = e; r < p.M; r += 256)
        if (__ldcg(p.targets + r) != p.ignore_index) {
            ++count;
            if (p.reduction == 0) {
                const float g = fabsf(__ldcg(p.grad + r));
                if (finite(g)) best = fmaxf(best, g);
            }
        }
    count = __reduce_add_sync(0xFFFFFFFFu, count);
    // |g| >= 0: its bits order like the values
    best = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(best)));
    if ((e & 31) == 0) {
        red[e >> 5] = best;
        reinterpret_cast<int *>(red)[8 + (e >> 5)] = count;
    }
    epi_sync();
    count = 0;
    best = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        best = fmaxf(best, red[w]);
        count += reinterpret_cast<int *>(red)[8 + w];
    }
    if (p.reduction == 2) return up / static_cast<float>(count > 0 ? count : 1);
    return best > 0.f ? best : 1.f;
}

// ------------------------------------------------------------------ epilogues
// Warp (quadrant q, half h) owns 32 rows of the tile (thread: one row) and 128 of its 256
// columns, in two parts of 64.  bf16 output leaves through shared memory: the warp's 32 x 64 box
// in the 128-byte swizzle, then one TMA store (32 rows of whole 128-byte lines; from the threads,
// row by row, the dW tiles of few rows took 40 % longer, and read back from shared memory in
// whole lines 4 %).
struct Out {
    uint8_t *box;        // this warp's boxes, 1024-byte aligned
    int next;            // the box that is written next
    uint64_t *tempty;    // the accumulator's release: local, or
    uint32_t tempty_remote;  // the pair leader's, if not 0
    int q, h, lane;
};

// This warp is done with the accumulator: its loads from TMEM have completed (each one waits), so
// the arrival has no memory writes to publish, and is a relaxed one.  With release semantics it
// waited some 1000 cycles for the stores of the part before, which nothing behind the barrier
// reads: a third of the time of a dW tile of few rows.
__device__ __forceinline__ void release(const Out &o) {
    tc_fence_before();
    __syncwarp();
    if (o.lane == 0) {
        if (o.tempty_remote)
            mbar_arrive_remote_relaxed(o.tempty_remote);
        else
            mbar_arrive_relaxed(o.tempty);
    }
}

// f(column in the tile, values): what becomes of 64 columns of the thread's row; `parts` of them
// (of two) hold anything to store.
template <typename F>
__device__ __forceinline__ void for_parts(uint32_t taddr, int parts, const Out &o, F f) {
    if (parts <= 0) return release(o);
#pragma unroll 1
    for (int part = 0; part < parts; ++part) {
        uint32_t raw[64];
        tmem_ld32x32b_x64(taddr + 128 * o.h + 64 * part, raw);
        if (part + 1 == parts) release(o);
        float v[64];
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] = __uint_as_float(raw[j]);
        f(128 * o.h + 64 * part, v);
    }
}

// The warp's 32 x 64 box to column x, row y of the map.
template <int ATOMS>
__device__ __forceinline__ void store_box(const CUtensorMap *tm, Out &o, const float (&v)[64],
                                          int x, int y, uint64_t pol) {
    constexpr int N = Ring<ATOMS>::kOutBoxes;
    if (o.lane == 0) bulk_wait_read<N - 1>();  // what this box held before has been read
    __syncwarp();
    uint8_t *box = o.box + o.next * kOutBytes;
    o.next = o.next + 1 == N ? 0 : o.next + 1;
    const uint32_t row = smem_u32(box) + o.lane * 128;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const float *x = v + 8 * c;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         row + ((c ^ (o.lane & 7)) << 4)),
                     "r"(pack_bf16(x[0], x[1])), "r"(pack_bf16(x[2], x[3])),
                     "r"(pack_bf16(x[4], x[5])), "r"(pack_bf16(x[6], x[7]))
                     : "memory");
    }
    fence_async_smem();
    __syncwarp();
    if (o.lane == 0) {
        tma_store_2d(tm, box, x, y, pol);
        bulk_commit();
    }
}

// What G's row needs of its loss: G_rj = a·exp(z_rj - lse_r), and `at` in the target's column.
struct RowTerms {
    int row0 = -1;       // of the warp's rows; the thread's is row0 + lane
    int target = -1;     // inside the vocabulary, else -1
    float a = 0.f, b = 0.f, lse = 0.f;  // b: the weight, a: times 1 + 2·z_loss·lse
    float at = 0.f;
    __device__ __forceinline__ bool dead() const { return a == 0.f && b == 0.f; }
};
__device__ __forceinline__ RowTerms row_terms(const LossGradParams &p, int row0, int lane,
                                              float scale) {
    RowTerms r;
    r.row0 = row0;
    const int row = row0 + lane;
    if (row >= p.M) return r;
    const int t = __ldcg(p.targets + row);
    if (t == p.ignore_index) return r;
    r.lse = __ldcg(p.lse + row);
    // the row's own weight relative to the shared scale
    const float up = incoming(p);
    r.b = (p.reduction == 0 && p.grad) ? __ldcg(p.grad + row) / scale : (finite(up) ? 1.f : up);
    r.a = r.b * (1.f + 2.f * p.z_loss * r.lse);
    if (t >= 0 && t < p.V) r.target = t;
    return r;
}

// The entries of those of the warp's rows whose target is among this warp's 128 columns of the
// tile: b·(p - 1 + 2·z_loss·lse·p).  lse holds the target's fp32 logit, which the accumulator misses by
// what the tensor cores truncate: with that one p - 1 would be wrong by as much, and where p is near
// 1 by more than its size (z = 25, 1 - p = 1e-3, d = 5120: 15 %).  So the warp forms the fp32 logit
// again, row by row (a row has one target: M sums of d products in all, each while its tile is still
// being formed), and p - 1 = expm1(z - lse) comes without a difference of two numbers near 1.
// Random targets cost nothing measurable (64 x 4096 x 151,936: 597 and 600 us without and with;
// 2048 x 4096 x 2000: 94 and 89), one target for all rows 15 us at most.  (A kernel of its own for
// the M sums took 1 to 7 us of every call.)
__device__ __forceinline__ void target_terms(const LossGradParams &p, int col0, int lane,
                                             RowTerms &r) {
    const int col = r.target - p.c0 - col0;
    unsigned rows = __ballot_sync(0xFFFFFFFFu,
                                  r.target >= 0 && col >= 0 && col < 128 && !r.dead());
    while (rows) {
        const int l = __ffs(rows) - 1;
        rows &= rows - 1;
        const int t = __shfl_sync(0xFFFFFFFFu, r.target, l);
        const float z = warp_dot(p.H + static_cast<size_t>(r.row0 + l) * p.d,
                                 p.W + static_cast<size_t>(t) * p.d, p.d, lane);
        if (lane == l) {
            const float less = expm1f(z - r.lse);
            r.at = r.b * (less + 2.f * p.z_loss * r.lse * (1.f + less));
        }
    }
}

template <int ATOMS>
__device__ __forceinline__ void epilogue_logits(const LossGradParams &p, const CUtensorMap *tmG,
                                                const Unit &u, uint32_t taddr, Out &o,
                                                const RowTerms &r, uint64_t pol) {
    // the target's column in this tile
    const int tgt = r.target >= 0 ? r.target - p.c0 - u.col0 : -1;
    const bool dead = r.dead();  // an ignored row, whatever its logits are
    const float l2 = r.lse * kLog2e;
    const int parts = r.row0 < p.M ? min(div_up(p.cols - u.col0 - 128 * o.h, 64), 2) : 0;
    for_parts(taddr, parts, o, [&](int c, float (&v)[64]) {
#pragma unroll
        for (int j = 0; j < 64; ++j) {
            const float e = r.a * ex2_approx(fmaf(v[j], kLog2e, -l2));
            v[j] = dead ? 0.f : (c + j == tgt ? r.at : e);
        }
        store_box<ATOMS>(tmG, o, v, u.col0 + c, r.row0, pol);
        if (p.lo) {  // (rows past M, up to the next 32, are zero in both)
#pragma unroll
            for (int j = 0; j < 64; ++j) {
                const float hi = __bfloat162float(__float2bfloat16_rn(v[j]));
                v[j] = finite(hi) ? v[j] - hi : 0.f;
            }
            store_box<ATOMS>(tmG, o, v, u.col0 + c, p.lo + r.row0, pol);
        }
    });
}

template <int ATOMS>
__device__ __forceinline__ void epilogue_operands(const LossGradParams &p, const CUtensorMap *tmDW,
                                                  const CUtensorMap *tmDH, const Unit &u,
                                                  uint32_t taddr, Out &o, float scale,
                                                  uint64_t pol) {
    const int row0 = u.row0 + 32 * o.q, row = row0 + o.lane;
    const int rows = u.dw ? p.cols : p.g_rows;
    // dH: fp32 partial sums in memory unless this piece is the only one, not split and G one number
    const bool sums = p.splits > 1 || p.lo;
    const bool through = !u.dw && (sums || !(p.first && p.last));
    const bool out = u.dw || (!sums && p.last);
    float *part = p.part + (static_cast<size_t>(u.split) * p.g_rows + row) * p.d;
    const int parts = row0 < rows ? min(div_up(p.d - u.col0 - 128 * o.h, 64), 2) : 0;
    for_parts(taddr, parts, o, [&](int c, float (&v)[64]) {
        const int col = u.col0 + c;
        const int n = min(64, p.d - col);
        if (u.kblocks == 0) {
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j] = 0.f;
        }
        if (through && !p.first && row < rows) {
            const float4 *src = reinterpret_cast<const float4 *>(part + col);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (4 * j < n) {
                    const float4 x = src[j];
                    v[4 * j] += x.x;
                    v[4 * j + 1] += x.y;
                    v[4 * j + 2] += x.z;
                    v[4 * j + 3] += x.w;
                }
        }
        if (out) {
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j] *= scale;
            store_box<ATOMS>(u.dw ? tmDW : tmDH, o, v, col, (u.dw ? p.c0 : 0) + row0, pol);
        } else if (row < rows) {
            float4 *to = reinterpret_cast<float4 *>(part + col);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (4 * j < n)
                    to[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
    });
}

// ------------------------------------------------------------------ the kernel
// LOGITS: m.x = H, m.y = W (both K-major: x is the reduction index), output m.g.  Otherwise m.x =
// the piece of G, m.y = W, m.z = the copy of H, outputs m.dw and m.dh.
template <bool LOGITS, int ATOMS>
__global__ void __launch_bounds__(kThreads, 1)
    grad_kernel(const __grid_constant__ LossGradMaps m, const LossGradParams p) {
    using R = Ring<ATOMS>;
    constexpr int KB = ATOMS * kBlockK;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + R::kBarAt);
    uint64_t *empty = full + R::kStages;
    uint64_t *tfull = empty + R::kStages;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint64_t *stall = drain + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + R::kBarAt + 512);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + R::kBarAt + 516);
    float *red = reinterpret_cast<float *>(smem + R::kBarAt + 528);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const Walk<LOGITS, ATOMS> walk(p, blockIdx.x / 2, gridDim.x / 2, rank);
    const WaitCtx wc{p.status, p.epoch, p.timeout_ns, abort_flag};

    if (threadIdx.x == 0) {
        for (int i = 0; i < R::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * kEpiWarps);  // the epilogue warps of both CTAs
        }
        mbar_init(drain, 1);
        mbar_init(stall, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&m.x);
        tma_prefetch_desc(&m.y);
        if (!LOGITS) tma_prefetch_desc(&m.z);
    }
    if (warp == 1) {
        tmem_alloc2(tmem_slot, 512);
        tmem_relinquish2();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers are initialised before any copy lands
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // Everything read from here on may have been written by the kernel before (G, the partial
    // sums, and W by an optimizer step), so all of it waits; the next kernel may then set up.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (LOGITS && blockIdx.x == 0 && threadIdx.x == 0) *p.epoch_word = p.epoch;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer.  The leader's full
        // barrier counts every copy of the pair; its one commit per stage frees the stage in
        // both CTAs.
        if (lane == 0) {
            // H and G are read by many pairs and again soon: kept in L2.  W is too where several
            // row tiles read it; few read it once, and it then leaves room for the others.
            const uint64_t pol = policy_evict_last();
            const uint64_t pol_w = p.row_tiles <= kWEvictFirstGroups ? policy_evict_first() : pol;
            int st = 0;
            uint32_t ph = 0, issued = 0;
            bool ok = true;
            // One thread issues all copies, and its own instructions per stage bound how fast
            // they go out: the layouts are compile-time constants of the loop (with a branch at
            // every copy and boxes of 64 rows the operands kernel had 71 % of the tensor
            // pipe's cycles).
            auto tile = [&](const Unit &u, auto a_mn, auto b_mn, const CUtensorMap *ta,
                            const CUtensorMap *tb, int b_row, int b_k, uint64_t pol_b) {
                // 64 or 128 of the B operand's rows per CTA, and those of A that there are
                const int boxes = decltype(b_mn)::value && u.n <= 128 ? 1 : 2;
                int a_boxes = 2, a_all = 4;
                if (!decltype(a_mn)::value) {
                    const int rows = LOGITS ? p.M : p.g_rows, r0 = u.row0 - rank * kTileA;
                    a_boxes = boxes_of<ATOMS>(rows, u.row0);
                    a_all = boxes_of<ATOMS>(rows, r0) + boxes_of<ATOMS>(rows, r0 + kTileA);
                }
                const uint32_t bytes = a_all * (LOGITS ? p.h_box_bytes : R::kBoxBytes) +
                                       2 * boxes * R::kBoxBytes;
                for (int kb = 0; kb < u.kblocks; ++kb) {
                    if (!bwait_cluster(&empty[st], ph ^ 1u, wc)) return false;
                    if (rank == 0) mbar_arrive_expect_tx(&full[st], bytes);
                    uint8_t *sa = smem + st * R::kStage;
                    // the leader's barrier at its cluster address, for both CTAs
                    const uint32_t bar = mapa_rank(&full[st], 0);
                    const int k = u.k0 + kb * KB;  // past the end: zeros
                    load_operand<decltype(a_mn)::value, ATOMS>(sa, ta, bar, u.row0, k, pol,
                                                               a_boxes);
                    load_operand<decltype(b_mn)::value, ATOMS>(sa + R::kOperand, tb, bar, b_row,
                                                               b_k + k, pol_b, boxes);
                    ++issued;
                    if (++st == R::kStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                return true;
            };
            for (int i = 0; ok && i < walk.n; ++i) {
                const Unit u = walk.at(i);
                const int bn = u.col0 + rank * (u.n / 2);  // this CTA's half of the B operand
                const std::true_type mn;
                const std::false_type km;
                if (LOGITS)
                    ok = tile(u, km, km, &m.x, &m.y, p.c0 + bn, 0, pol_w);
                else if (u.dw)
                    ok = tile(u, mn, mn, &m.x, &m.z, bn, 0, pol);
                else
                    ok = tile(u, km, mn, &m.x, &m.y, bn, p.c0, pol_w);
            }
            if (rank == 0) {
                // every copy that the barriers count has landed before this CTA exits
                const uint32_t n = issued < R::kStages ? issued : R::kStages;
                for (uint32_t i = issued - n; i < issued; ++i)
                    if (!bwait_drain(&full[i % R::kStages], (i / R::kStages) & 1u, wc)) break;
            } else if (!ok) {
                // the peer's copies complete on the leader's barriers: after an abort it gives
                // the last ones (issued at least one wait limit ago) a bounded time to land
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 50000u) {
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (the pair's leader)
        if (rank == 0 && lane == 0) {
            constexpr uint16_t kBoth = 3;
            const uint32_t s0 = smem_u32(smem);
            const uint64_t k_desc = sw128_kmajor_desc(s0);
            const uint64_t mn_desc = sw128_mnmajor_desc(s0, R::kBoxBytes);
            int st = 0;
            uint32_t ph = 0;
            bool ok = true, any = false;
            for (int i = 0; ok && i < walk.n; ++i) {
                const Unit u = walk.at(i);
                const int b = i & 1;
                const uint32_t tph = (i >> 1) & 1;
                if (!bwait_cluster(&tempty[b], tph ^ 1u, wc)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * kTile);
                const bool a_mn = !LOGITS && u.dw, b_mn = !LOGITS;
                const uint32_t idesc = idesc_bf16_f32(2 * kTileA, u.n) |
                                       (a_mn ? kIdescAMajorMN : 0u) | (b_mn ? kIdescBMajorMN : 0u);
                const uint64_t ad0 = a_mn ? mn_desc : k_desc;
                const uint64_t bd0 = (b_mn ? mn_desc : k_desc) + (R::kOperand >> 4);
                // a 16-wide K step: 32 bytes along a K-major row (the next 64-wide slice is the
                // next atom), 16 rows of an MN-major one
                const uint32_t a_step = a_mn ? 2048u >> 4 : 32u >> 4;
                const uint32_t b_step = b_mn ? 2048u >> 4 : 32u >> 4;
                const uint32_t a_atom = a_mn ? 4 * (2048u >> 4) : kAtomBytes >> 4;
                const uint32_t b_atom = b_mn ? 4 * (2048u >> 4) : kAtomBytes >> 4;
                for (int kb = 0; kb < u.kblocks; ++kb) {
                    if (!bwait_cluster(&full[st], ph, wc)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t so = (static_cast<uint32_t>(st) * R::kStage) >> 4;
                    const int slices = kb + 1 < u.kblocks ? ATOMS : u.slices;
#pragma unroll
                    for (int at = 0; at < ATOMS; ++at) {
                        if (at >= slices) break;  // nothing but zeros
#pragma unroll
                        for (int ks = 0; ks < kBlockK / 16; ++ks)
                            umma_bf16_pair(d_tmem, ad0 + so + at * a_atom + ks * a_step,
                                           bd0 + so + at * b_atom + ks * b_step, idesc,
                                           (kb | at | ks) != 0 ? 1u : 0u);
                    }
                    umma_commit_pair(&empty[st], kBoth);
                    any = true;
                    if (++st == R::kStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) umma_commit_pair(&tfull[b], kBoth);
                any = true;
            }
            if (any) {  // until every MMA this thread issued has completed
                umma_commit_pair(drain, 1);
                bwait_drain(drain, 0, wc);
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------ the copy of H for dW (first piece)
        if (LOGITS && p.Hc) {
            const int n16 = p.d / 8;
            for (int r = blockIdx.x; r < p.g_rows; r += gridDim.x) {
                const int from = p.lo && r >= p.lo ? r - p.lo : r;  // once for each part of G
                const bool keep = from < p.M && __ldcg(p.targets + from) != p.ignore_index;
                const uint4 *src =
                    reinterpret_cast<const uint4 *>(p.H + static_cast<size_t>(keep ? from : 0) *
                                                              p.d);
                uint4 *dst = reinterpret_cast<uint4 *>(p.Hc + static_cast<size_t>(r) * p.d);
                constexpr int kAtOnce = 8;  // loads before the first store
                for (int i = lane; i < n16; i += 32 * kAtOnce) {
                    uint4 x[kAtOnce];
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u)
                        x[u] = keep && i + 32 * u < n16 ? __ldcg(src + i + 32 * u)
                                                        : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u)
                        if (i + 32 * u < n16) dst[i + 32 * u] = x[u];
                }
            }
        }
    } else {
        // ------------------------------------------------ epilogue warps
        Out o;
        o.q = warp & 3;                     // TMEM lane quadrant this warp may read
        o.h = (warp - kFirstEpiWarp) >> 2;  // which half of the columns
        o.lane = lane;
        o.box = smem + R::kOutAt + (warp - kFirstEpiWarp) * R::kOutBoxes * kOutBytes;
        o.next = 0;
        // G is read next (by the operands kernel); dW and dH are not read here again
        const uint64_t pol = LOGITS ? policy_evict_normal() : policy_evict_first();
        float scale;
        if (LOGITS) {
            scale = shared_scale(p, threadIdx.x - 32 * kFirstEpiWarp, red);
            if (blockIdx.x == 0 && threadIdx.x == 32 * kFirstEpiWarp) *p.scale = scale;
        } else {
            scale = *p.scale;
        }
        // the leader's release barriers
        const uint32_t remote0 = rank == 1 ? mapa_rank(&tempty[0], 0) : 0u;
        const uint32_t remote1 = rank == 1 ? mapa_rank(&tempty[1], 0) : 0u;
        RowTerms terms;
        for (int i = 0; i < walk.n; ++i) {
            const Unit u = walk.at(i);
            const int b = i & 1;
            const uint32_t tph = (i >> 1) & 1;
            // the rows' terms while the tile is formed (few rows: once)
            const int row0 = u.row0 + 32 * o.q;
            if (LOGITS) {
                if (row0 != terms.row0) terms = row_terms(p, row0, lane, scale);
                target_terms(p, u.col0 + 128 * o.h, lane, terms);
            }
            const bool ok = p.debug_stall ? bwait(stall, 0, wc) : bwait_cluster(&tfull[b], tph, wc);
            if (__any_sync(0xFFFFFFFFu, !ok)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * o.q) << 16) +
                                   static_cast<uint32_t>(b * kTile);
            o.tempty = &tempty[b];
            o.tempty_remote = b ? remote1 : remote0;
            if (LOGITS)
                epilogue_logits<ATOMS>(p, &m.g, u, taddr, o, terms, pol);
            else
                epilogue_operands<ATOMS>(p, &m.dw, &m.dh, u, taddr, o, scale, pol);
        }
        if (lane == 0) bulk_wait();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // nothing of the peer's lands here after this CTA has left
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc2(tmem_base, 512);
    }
}

// dH = scale * (split 0 + split 1 + ...), of both parts of G: n4 groups of four values, stride4
// from split to split, the second part's rows lo4 after the first's (0: one part).  A block sums
// 32 groups: eight warps take an eighth of the splits each, in ascending order, and their sums
// add up in ascending order.
constexpr int kSumSlices = 8;
__global__ void __launch_bounds__(32 * kSumSlices) sum_kernel(const float4 *part, uint2 *dH,
                                                              size_t n4, size_t stride4,
                                                              size_t lo4, int splits,
                                                              const float *scale) {
    __shared__ float4 sh[kSumSlices][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const size_t i = static_cast<size_t>(blockIdx.x) * 32 + lane;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4 x) {
        a.x += x.x;
        a.y += x.y;
        a.z += x.z;
        a.w += x.w;
    };
    if (i < n4) {
        const int s1 = splits * (slice + 1) / kSumSlices;
#pragma unroll 4
        for (int s = splits * slice / kSumSlices; s < s1; ++s) {
            add(part[s * stride4 + i]);
            if (lo4) add(part[s * stride4 + lo4 + i]);
        }
    }
    sh[slice][lane] = a;
    __syncthreads();
    if (slice != 0 || i >= n4) return;
    const float f = *scale;
#pragma unroll
    for (int s = 1; s < kSumSlices; ++s) add(sh[s][lane]);
    dH[i] = make_uint2(pack_bf16(f * a.x, f * a.y), pack_bf16(f * a.z, f * a.w));
}

template <bool LOGITS, int ATOMS>
cudaError_t launch_grad(const LossGradMaps &m, const LossGradParams &p, int units, int num_sms,
                        cudaStream_t stream) {
    auto kern = grad_kernel<LOGITS, ATOMS>;
    static std::atomic<uint64_t> opted_in{0};
    static std::atomic<int> pairs_by_dev[64];  // co-resident pairs (GPCs may not pair every SM)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
    if (!bit || !(opted_in.load() & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Ring<ATOMS>::kSmem);
        if (e != cudaSuccess) return e;
        opted_in.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<ATOMS>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    int pairs = dev < 64 ? pairs_by_dev[dev].load() : 0;
    if (pairs <= 0) {
        cfg.gridDim = dim3(num_sms / 2 * 2);
        if (cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg) != cudaSuccess || pairs <= 0 ||
            pairs > num_sms / 2)
            pairs = num_sms / 2;
        if (dev < 64) pairs_by_dev[dev].store(pairs);
    }
    if (pairs > units) pairs = units;
    if (pairs < 1) pairs = 1;
    cfg.gridDim = dim3(2 * pairs);
    return cudaLaunchKernelEx(&cfg, kern, m, p);
}

}  // namespace

// One 64-wide slice per stage when a single pair of row tiles reads each W tile (the W stream
// sets the pace and wants more stages), two otherwise.
int loss_box_rows(int row_tiles) { return row_tiles < 2 ? Ring<1>::kBoxRows : Ring<2>::kBoxRows; }

cudaError_t launch_loss_logits(const LossGradMaps &m, const LossGradParams &p, int num_sms,
                               cudaStream_t stream) {
    const int units = p.row_tiles * p.col_tiles;
    return loss_box_rows(p.row_tiles) == Ring<1>::kBoxRows
               ? launch_grad<true, 1>(m, p, units, num_sms, stream)
               : launch_grad<true, 2>(m, p, units, num_sms, stream);
}

cudaError_t launch_loss_operands(const LossGradMaps &m, const LossGradParams &p, int num_sms,
                                 cudaStream_t stream) {
    const int units = p.dh_units + p.dw_units;
    return loss_box_rows(p.row_tiles) == Ring<1>::kBoxRows
               ? launch_grad<false, 1>(m, p, units, num_sms, stream)
               : launch_grad<false, 2>(m, p, units, num_sms, stream);
}

cudaError_t launch_loss_sum(const LossGradParams &p, cudaStream_t stream) {
    const size_t n4 = static_cast<size_t>(p.M) * p.d / 4;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((n4 + 31) / 32));
    cfg.blockDim = dim3(32 * kSumSlices);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sum_kernel, reinterpret_cast<const float4 *>(p.part),
                              reinterpret_cast<uint2 *>(p.dH), n4,
                              static_cast<size_t>(p.g_rows) * p.d / 4,
                              static_cast<size_t>(p.lo) * p.d / 4, p.splits, p.scale);
}

}  // namespace sb
