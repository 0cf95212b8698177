// loss_common.cuh -- the target's logit in fp32, as both directions of the cross entropy form it.
//
// Forward returns lse with the logit in it and backward subtracts the logit again, so the two sums
// have the same order and the same bits: kDotParts partial sums, part i over the 16-byte chunks i, i +
// kDotParts, ... (even and odd elements apart), the parts of 32 consecutive indexes added by a
// shuffle butterfly, and these four in ascending order.
#pragma once
#include <cstdint>

namespace sb {

constexpr int kDotParts = 128;

// The parts first, first + 32, ... (N of them) of h·w over d bf16 values, d a multiple of 8.
template <int N>
__device__ __forceinline__ void dot_parts(const uint16_t *h, const uint16_t *w, int d, int first,
                                          float (&part)[N]) {
    const uint4 *h8 = reinterpret_cast<const uint4 *>(h), *w8 = reinterpret_cast<const uint4 *>(w);
    float even[N], odd[N];
#pragma unroll
    for (int n = 0; n < N; ++n) even[n] = odd[n] = 0.f;
    // a single warp has the loads of kAtOnce rounds in flight before the first sum (with two rounds a
    // row took 1.9 us of its tile's time, and one target for all of 64 rows 65 us)
    constexpr int kAtOnce = N == 1 ? 1 : 4;
#pragma unroll(N == 1 ? 2 : 1)
    for (int k = first; k < d / 8; k += kAtOnce * kDotParts) {
        uint4 x[kAtOnce][N], y[kAtOnce][N];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int i = k + u * kDotParts + 32 * n;
                const bool in = (u == 0 && n == 0) || i < d / 8;  // else products that are zero
                x[u][n] = in ? h8[i] : make_uint4(0, 0, 0, 0);
                y[u][n] = in ? w8[i] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint32_t xs[4] = {x[u][n].x, x[u][n].y, x[u][n].z, x[u][n].w};
                const uint32_t ys[4] = {y[u][n].x, y[u][n].y, y[u][n].z, y[u][n].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    even[n] = fmaf(__uint_as_float(xs[j] << 16), __uint_as_float(ys[j] << 16),
                                   even[n]);
                    odd[n] = fmaf(__uint_as_float(xs[j] & 0xFFFF0000u),
                                  __uint_as_float(ys[j] & 0xFFFF0000u), odd[n]);
                }
            }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) part[n] = even[n] + odd[n];
}

// The whole sum by one warp; every lane gets it.
__device__ __forceinline__ float warp_dot(const uint16_t *h, const uint16_t *w, int d, int lane) {
    float part[kDotParts / 32];
    dot_parts(h, w, d, lane, part);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < kDotParts / 32; ++n)
            part[n] += __shfl_xor_sync(0xFFFFFFFFu, part[n], o);
    float sum = part[0];
#pragma unroll
    for (int n = 1; n < kDotParts / 32; ++n) sum += part[n];
    return sum;
}

}  // namespace sb
