// sb_counter.cuh -- the counter-based generator of the sampling and dropout kernels.
//
// SplitMix64 (Steele, Lea and Flood, OOPSLA 2014) at stream index n of the stream seeded with
// `seed`: the state is seed + (n + 1) * golden-ratio increment, then the finaliser.
#pragma once
#include <cstdint>

namespace sb {

constexpr unsigned long long kGolden = 0x9E3779B97F4A7C15ull;
__device__ __forceinline__ unsigned long long splitmix_state(unsigned long long seed,
                                                             unsigned long long n) {
    return seed + (n + 1ull) * kGolden;
}
// The finaliser ends with x ^= x >> 31; its top 24 bits are those of x itself (x >> 31
// contributes nothing above bit 32), so that last step is left out.  They give u = b * 2^-24 in
// [0, 1).
__device__ __forceinline__ uint32_t bits24_from_state(unsigned long long x) {
    x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
    x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
    return static_cast<uint32_t>(x >> 40);
}
// All 64 bits.
__device__ __forceinline__ unsigned long long bits64_from_state(unsigned long long x) {
    x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
    x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
    return x ^ (x >> 31);
}

}  // namespace sb
