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
    // written by an earlier launch of the same call
    static __device__ __forceinline__ raw load_written(const T *p) { return *reinterpret_cast<const raw *>(p); }
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
    // the features where `keep`, else zeros whatever they hold (bf16: the
    // shift and the mask that unpack take the factor and the mask 0 instead)
    static __device__ __forceinline__ void unpack_if(raw r, bool keep, float (&v)[VEC]) {
        Bits b;
        if (kBytes < 4) b.w[0] = 0u;
        b.r = r;
        if (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = keep ? __uint_as_float(b.w[i]) : 0.f;
        } else {
            const uint32_t up = keep ? 65536u : 0u, high = keep ? 0xffff0000u : 0u;
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = __uint_as_float(i & 1 ? b.w[i / 2] & high : b.w[i / 2] * up);
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
            for (int i = 0; i < VEC / 2; ++i)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b.w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        }
        return b.r;
    }
    static __device__ __forceinline__ void store_raw(T *p, raw r) { __stcs(reinterpret_cast<raw *>(p), r); }
    static __device__ __forceinline__ void store(T *p, const float (&v)[VEC]) { store_raw(p, pack(v)); }
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

// VEC fp32 sums, in pairs where there are pairs: one fma.rn.f32x2 adds to two.
template <int VEC> struct Sums {
    static constexpr int kPairs = VEC / 2;
    uint64_t s[kPairs];

    static __device__ __forceinline__ uint64_t pair(float a, float b) {
        uint64_t r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
        return r;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) s[i] = 0ull;
    }
    __device__ __forceinline__ void add(uint64_t ff, const float (&v)[VEC]) {  // s += f v, ff = pair(f, f)
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(s[i]) : "l"(ff), "l"(pair(v[2 * i], v[2 * i + 1])));
    }
    __device__ __forceinline__ void get(float (&v)[VEC]) const {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) asm("mov.b64 {%0, %1}, %2;" : "=f"(v[2 * i]), "=f"(v[2 * i + 1]) : "l"(s[i]));
    }
    __device__ __forceinline__ void set(const float (&v)[VEC]) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) s[i] = pair(v[2 * i], v[2 * i + 1]);
    }
};
template <> struct Sums<1> {
    float s;
    static __device__ __forceinline__ uint64_t pair(float a, float b) { return Sums<2>::pair(a, b); }
    __device__ __forceinline__ void zero() { s = 0.f; }
    __device__ __forceinline__ void add(uint64_t ff, const float (&v)[1]) { s = fmaf(__uint_as_float(uint32_t(ff)), v[0], s); }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = s; }
    __device__ __forceinline__ void set(const float (&v)[1]) { s = v[0]; }
};

// x = x * f + c element by element, two at a time where there are two
template <int VEC>
__device__ __forceinline__ void fma_all(float (&x)[VEC], const float (&f)[VEC], const float (&c)[VEC]) {
    if constexpr (VEC == 1) {
        x[0] = fmaf(x[0], f[0], c[0]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            uint64_t v = Sums<2>::pair(x[i], x[i + 1]);
            asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(Sums<2>::pair(f[i], f[i + 1])), "l"(Sums<2>::pair(c[i], c[i + 1])));
            asm("mov.b64 {%0, %1}, %2;" : "=f"(x[i]), "=f"(x[i + 1]) : "l"(v));
        }
    }
}
template <int VEC>
__device__ __forceinline__ void mul_all(float (&x)[VEC], float f) {
    if constexpr (VEC == 1) {
        x[0] *= f;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            uint64_t v = Sums<2>::pair(x[i], x[i + 1]);
            asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(Sums<2>::pair(f, f)));
            asm("mov.b64 {%0, %1}, %2;" : "=f"(x[i]), "=f"(x[i + 1]) : "l"(v));
        }
    }
}
template <int VEC>
__device__ __forceinline__ void add_all(float (&x)[VEC], const float (&y)[VEC]) {
    if constexpr (VEC == 1) {
        x[0] += y[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            uint64_t v = Sums<2>::pair(x[i], x[i + 1]);
            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(Sums<2>::pair(y[i], y[i + 1])));
            asm("mov.b64 {%0, %1}, %2;" : "=f"(x[i]), "=f"(x[i + 1]) : "l"(v));
        }
    }
}
// sums of the elements and of their squares
template <int VEC>
__device__ __forceinline__ float sum_all(const float (&x)[VEC]) {
    if constexpr (VEC == 1) return x[0];
    uint64_t v = Sums<2>::pair(x[0], x[VEC > 1 ? 1 : 0]);
#pragma unroll
    for (int i = 2; i + 1 < VEC; i += 2) asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(Sums<2>::pair(x[i], x[i + 1])));
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    return a + b;
}
template <int VEC>
__device__ __forceinline__ float squares_all(const float (&x)[VEC]) {
    if constexpr (VEC == 1) return x[0] * x[0];
    uint64_t v = 0ull;
#pragma unroll
    for (int i = 0; i + 1 < VEC; i += 2) {
        const uint64_t p = Sums<2>::pair(x[i], x[i + 1]);
        asm("fma.rn.f32x2 %0, %1, %1, %0;" : "+l"(v) : "l"(p));
    }
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    return a + b;
}

}  // namespace
}  // namespace ag
