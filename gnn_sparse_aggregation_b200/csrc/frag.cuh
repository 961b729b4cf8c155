// frag.cuh -- VEC consecutive features as one register fragment: loads and
// stores of 16, 8, 4 or 2 bytes, the conversion to fp32 and exact products.
#pragma once

#include "device_common.cuh"

namespace ag {
namespace {

template <int BYTES> struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };

template <typename T, int VEC> struct Frag {
    static constexpr int kBytes = VEC * int(sizeof(T));
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    using raw = typename RawOf<kBytes>::type;
    union Bits {
        raw r;
        uint32_t w[kWords];
        __device__ __forceinline__ Bits() {}
    };

    static __device__ __forceinline__ raw zero() {
        Bits b;
#pragma unroll
        for (int i = 0; i < kWords; ++i) b.w[i] = 0u;
        return b.r;
    }
    static __device__ __forceinline__ raw load(const T *p) { return __ldg(reinterpret_cast<const raw *>(p)); }
    // read once: does not displace what is read again
    static __device__ __forceinline__ raw load_stream(const T *p) { return __ldcs(reinterpret_cast<const raw *>(p)); }
    static __device__ __forceinline__ void unpack(raw r, float (&v)[VEC]) {
        Bits b;
        if (kBytes < 4) b.w[0] = 0u;
        b.r = r;
        if (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = __uint_as_float(b.w[i]);
        } else if (VEC == 1) {
            v[0] = __uint_as_float(b.w[0] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                v[2 * i] = bf16_lo(b.w[i]);
                v[2 * i + 1] = bf16_hi(b.w[i]);
            }
        }
    }
    static __device__ __forceinline__ raw pack(const float (&v)[VEC]) {
        Bits b;
        if (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) b.w[i] = __float_as_uint(v[i]);
        } else if (VEC == 1) {
            b.w[0] = bf16_bits(v[0]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) b.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        }
        return b.r;
    }
    static __device__ __forceinline__ void store(T *p, const float (&v)[VEC]) {
        __stcs(reinterpret_cast<raw *>(p), pack(v));
    }
    // c + the products of the fragments' elements, in order (bf16 products
    // are exact in fp32, so each term is rounded once)
    static __device__ __forceinline__ float dot(raw x, raw y, float c) {
        if (sizeof(T) == 2 && VEC > 1) {
            Bits a, b;
            a.r = x;
            b.r = y;
#pragma unroll
            for (int i = 0; i < kWords; ++i) c = dot2_bf16(a.w[i], b.w[i], c);
        } else {
            float u[VEC], v[VEC];
            unpack(x, u);
            unpack(y, v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) c = fmaf(u[i], v[i], c);
        }
        return c;
    }
};

}  // namespace
}  // namespace ag
