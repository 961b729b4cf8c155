// random.cuh -- the counter-based generator of the dropout entry points.
//
// Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64-bit
// products, the key advanced by two constants each round.  Element i of an
// array uses word i % 4 of the block with counter (i / 4, offset) and key
// seed, and is kept where that word is at least round(p 2^32), or 2^32 - 1 where
// that rounds to 2^32.  The mask is a function of (seed, offset, i) alone: the
// backward pass recomputes it, no mask is stored, and any kernel that knows an
// element's index draws the same bit whatever its schedule.
#pragma once

#include <math.h>
#include <stdint.h>

namespace ag {

struct Drop {
    uint32_t key[20];     // the seed's round keys, two a round: a constant operand each in the kernels
    uint32_t o0, o1;      // offset: the counter's upper half
    uint32_t threshold;   // keep an element where its word is >= threshold
    float scale;          // 1 / (1 - p)
    int on;               // p > 0
};

// p in [0, 1) (checked by the entry points).
inline Drop make_drop(double p, uint64_t seed, uint64_t offset) {
    Drop d;
    for (int r = 0; r < 10; ++r) {
        d.key[2 * r] = uint32_t(seed) + uint32_t(r) * 0x9E3779B9u;
        d.key[2 * r + 1] = uint32_t(seed >> 32) + uint32_t(r) * 0xBB67AE85u;
    }
    d.o0 = uint32_t(offset);
    d.o1 = uint32_t(offset >> 32);
    const double t = rint(p * 4294967296.0);
    d.threshold = t >= 4294967295.0 ? 0xffffffffu : uint32_t(t);
    d.scale = float(1.0 / (1.0 - p));
    d.on = p > 0.0;
    return d;
}

#ifdef __CUDACC__
namespace {

// The rounds take their keys as constant operands (dropout of [2^20, 128] bf16
// 121 us against 127 with keys in registers), or, IN_LOOP, derive them from
// the first: one kernel that draws once in many steps runs 4 % faster so
// (attention on R-MAT-18 1.17 against 1.21 ms).  The first key is made opaque
// there, or the compiler would keep all twenty in registers across the loop.
template <bool IN_LOOP = false>
__device__ __forceinline__ uint4 philox(uint64_t block, const Drop &d) {
    uint32_t k0 = d.key[0], k1 = d.key[1];
    if (IN_LOOP) asm volatile("" : "+r"(k0), "+r"(k1));
    uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32), c2 = d.o0, c3 = d.o1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t m0 = uint64_t(c0) * 0xD2511F53u, m1 = uint64_t(c2) * 0xCD9E8D57u;
        c0 = uint32_t(m1 >> 32) ^ c1 ^ (IN_LOOP ? k0 + uint32_t(r) * 0x9E3779B9u : d.key[2 * r]);
        c2 = uint32_t(m0 >> 32) ^ c3 ^ (IN_LOOP ? k1 + uint32_t(r) * 0xBB67AE85u : d.key[2 * r + 1]);
        c1 = uint32_t(m1);
        c3 = uint32_t(m0);
    }
    return make_uint4(c0, c1, c2, c3);
}

// Bit j: whether element 4 block + j is kept.
template <bool IN_LOOP = false>
__device__ __forceinline__ uint32_t keep4(uint64_t block, const Drop &d) {
    const uint4 w = philox<IN_LOOP>(block, d);
    return uint32_t(w.x >= d.threshold) | uint32_t(w.y >= d.threshold) << 1 | uint32_t(w.z >= d.threshold) << 2 |
           uint32_t(w.w >= d.threshold) << 3;
}

// Bit j: whether element i + j is kept, j < count <= 28.
template <bool IN_LOOP = false>
__device__ __forceinline__ uint32_t keep_bits(uint64_t i, int count, const Drop &d) {
    uint32_t bits = 0;
    const uint64_t last = (i + uint64_t(count) - 1) >> 2;
    int at = -int(i & 3);
    for (uint64_t b = i >> 2; b <= last; ++b, at += 4) {
        const uint32_t k = keep4<IN_LOOP>(b, d);
        bits |= at >= 0 ? k << at : k >> -at;
    }
    return bits;
}

}  // namespace
#endif

}  // namespace ag
