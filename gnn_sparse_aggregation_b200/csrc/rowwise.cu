// Row-wise operators around an attention layer: dropout, rotary positions and
// the norm / gate / residual block with its gradients.  Each makes one pass
// over its matrices and is bound by HBM; none needs a graph.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "aggraph.h"
#include "frag.cuh"
#include "internal.h"
#include "launch.cuh"
#include "operands.h"
#include "random.cuh"

namespace ag {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSMs = 148;

// ---------------------------------------------------------------------------- dropout

// y_i = keep_i x_i / (1 - p).  A thread takes VEC (a multiple of 4) elements at
// a time: VEC / 4 Philox blocks.  [2^20, 128] bf16: 119-124 us, 66-69 % of the
// measured copy rate.  Bound by the integer pipes: with 92 % of the warps active
// the most frequent stall is on a busy pipe (the exclusive-ors, compares and
// moves hold theirs 66 % busy, the twenty wide products a block theirs 39 %, where
// such a product takes more than one slot).  Two vectors per thread at a time
// measured 127-131 us.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) k_dropout(const T *__restrict__ x, T *__restrict__ y, int64_t n, const Drop drop) {
    using F = Frag<T, VEC>;
    const int64_t vecs = n / VEC;
    const int64_t stride = int64_t(gridDim.x) * blockDim.x;
    const int64_t i0 = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    for (int64_t i = i0; i < vecs; i += stride) {
        const typename F::raw r = F::load_stream(x + i * VEC);
        uint32_t k[VEC / 4];
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q) k[q] = keep4(uint64_t(i) * (VEC / 4) + q, drop);
        float v[VEC];
        F::unpack(r, v);
        mul_all<VEC>(v, drop.scale);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = k[j / 4] >> (j & 3) & 1u ? v[j] : 0.f;
        F::store(y + i * VEC, v);
    }
    // the last n % VEC elements
    const int64_t i = vecs * VEC + i0;
    if (i < n) {
        float v[1];
        Frag<T, 1>::unpack(Frag<T, 1>::load_stream(x + i), v);
        v[0] = keep4(uint64_t(i) >> 2, drop) >> (i & 3) & 1u ? v[0] * drop.scale : 0.f;
        Frag<T, 1>::store(y + i, v);
    }
}
// Addresses without a vector: four elements per block one by one.
template <typename T>
__global__ void __launch_bounds__(256) k_dropout_scalar(const T *__restrict__ x, T *__restrict__ y, int64_t n,
                                                        const Drop drop) {
    const int64_t stride = int64_t(gridDim.x) * blockDim.x;
    for (int64_t b = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; b * 4 < n; b += stride) {
        const uint32_t k = keep4(uint64_t(b), drop);
        for (int j = 0; j < 4 && b * 4 + j < n; ++j) {
            float v[1];
            Frag<T, 1>::unpack(Frag<T, 1>::load_stream(x + b * 4 + j), v);
            v[0] = k >> j & 1u ? v[0] * drop.scale : 0.f;
            Frag<T, 1>::store(y + b * 4 + j, v);
        }
    }
}

unsigned grid_of(int64_t work, int64_t per_block, int64_t most) {
    const int64_t b = (work + per_block - 1) / per_block;
    return unsigned(b < 1 ? 1 : (b > most ? most : b));
}

template <typename T, int VEC>
void launch_dropout(const void *X, void *Y, int64_t n, const Drop &drop, cudaStream_t st) {
    const T *x = static_cast<const T *>(X);
    T *y = static_cast<T *>(Y);
    if ((uintptr_t(X) | uintptr_t(Y)) % (VEC * sizeof(T)) == 0)
        k_dropout<T, VEC><<<grid_of(n / VEC + 1, 256, kSMs * 64), 256, 0, st>>>(x, y, n, drop);
    else
        k_dropout_scalar<T><<<grid_of((n + 3) / 4, 256, kSMs * 64), 256, 0, st>>>(x, y, n, drop);
}

// ---------------------------------------------------------------------------- rotary positions

// Pair i of a head (i < rot / 2) is rotated by the angle pos[n] inv_freq[i]
// and scaled by `factor`; the columns from rot on are copied.  The angle is
// reduced in turns in fp64 (an fp32 angle at position 2^20 is off by 0.03),
// then one fp32 sincospi.  A block takes `rows` rows: it computes their
// rot / 2 angles once into shared memory, for all heads of both matrices.
// Bound by HBM: [2^20, 128] bf16, two matrices, 184-189 us, 88-90 % of the
// measured copy rate (232 us with one row's loads at a time and a branch
// between rotated and copied vectors, 251 us with an index division a vector).
struct RotaryParams {
    const void *in[2];
    void *out[2];
    const int64_t *pos;
    const double *inv_freq;
    int64_t N;
    int mats, H, D, rot, heads, rows;
    float factor, sign;
};

constexpr int kMaxRot = 4096;

template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(256) k_rotary(const RotaryParams P) {
    extern __shared__ float2 turn[];  // [rows][rot / 2]: factor * (cos, sin)
    using F = Frag<T, VEC>;
    const int64_t n0 = int64_t(blockIdx.x) * P.rows;
    const int rows = int(P.N - n0 < P.rows ? P.N - n0 : P.rows);
    const int pairs = P.rot / 2;
    for (int i = threadIdx.x; i < rows * pairs; i += blockDim.x) {
        const int r = i / pairs;
        const double u = double(P.pos[n0 + r]) * (P.inv_freq[i - r * pairs] * 0.15915494309189535);  // turns
        float s, c;
        sincospif(float(2.0 * (u - rint(u))), &s, &c);
        turn[i] = make_float2(P.factor * c, P.sign * P.factor * s);
    }
    __syncthreads();
    // units of a head: rotated (two vectors, or one with both halves of its
    // pairs), then copied vectors.  A thread keeps its units and walks the rows.
    constexpr bool kPairInVec = !HALF && VEC > 1;
    const int rot_units = kPairInVec ? P.rot / VEC : pairs / VEC;
    const int head_units = rot_units + (P.D - P.rot) / VEC;
    const int row_units = head_units * P.heads;
    const int lanes = row_units < int(blockDim.x) ? row_units : int(blockDim.x);  // threads of one row
    const int row_step = int(blockDim.x) / lanes;
    const int r0 = threadIdx.x / lanes;
    if (r0 >= row_step) return;
    for (int q = threadIdx.x % lanes; q < row_units; q += lanes) {
        const int head = q / head_units;
        const int u = q - head * head_units;
        const bool copied = u >= rot_units;
        const int at = head * P.D + (copied ? P.rot + (u - rot_units) * VEC : (kPairInVec || HALF ? u * VEC : 2 * u));
        const int other = HALF ? pairs : 1;     // from a pair's first to its second
        const int pair0 = kPairInVec ? u * VEC / 2 : u * VEC;
        // two rows of both matrices at a time: all their loads first
        for (int r = r0; r < rows; r += 2 * row_step) {
            typename F::raw ra[2][2], rb[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t base = (n0 + r + i * row_step) * P.H + at;
                const bool in = r + i * row_step < rows;
#pragma unroll
                for (int mat = 0; mat < 2; ++mat) {
                    const T *x = static_cast<const T *>(P.in[mat]) + base;
                    const bool have = in && mat < P.mats;
                    ra[i][mat] = have ? F::load_stream(x) : F::zero();
                    if (!kPairInVec) rb[i][mat] = have && !copied ? F::load_stream(x + other) : F::zero();
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ri = r + i * row_step;
                if (ri >= rows) break;
                const float2 *cs = turn + ri * pairs + (copied ? 0 : pair0);
                float t[VEC][2];
#pragma unroll
                for (int v = 0; v < (kPairInVec ? VEC / 2 : VEC); ++v) {
                    const float2 f = copied ? make_float2(1.f, 0.f) : cs[v];
                    t[v][0] = f.x, t[v][1] = f.y;
                }
                const int64_t base = (n0 + ri) * P.H + at;
#pragma unroll
                for (int mat = 0; mat < 2; ++mat) {
                    if (mat == P.mats) break;
                    T *y = static_cast<T *>(P.out[mat]) + base;
                    float a[VEC], b[VEC];
                    F::unpack(ra[i][mat], a);
                    if constexpr (kPairInVec) {
#pragma unroll
                        for (int v = 0; v + 1 < VEC; v += 2) {
                            b[v] = a[v] * t[v / 2][0] - a[v + 1] * t[v / 2][1];
                            b[v + 1] = a[v + 1] * t[v / 2][0] + a[v] * t[v / 2][1];
                        }
                        F::store_raw(y, copied ? ra[i][mat] : F::pack(b));
                    } else {
                        F::unpack(rb[i][mat], b);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) {
                            const float p = a[v];
                            a[v] = p * t[v][0] - b[v] * t[v][1];
                            b[v] = b[v] * t[v][0] + p * t[v][1];
                        }
                        F::store_raw(y, copied ? ra[i][mat] : F::pack(a));
                        if (!copied) F::store(y + other, b);
                    }
                }
            }
        }
    }
}

template <typename T, int VEC, bool HALF>
void launch_rotary(RotaryParams &P, cudaStream_t st) {
    // about 1024 vectors per block, fewer rows where that leaves SMs idle
    int64_t rows = 1024 / (int64_t(P.mats) * P.H / VEC) + 1;
    const int64_t spread = (P.N + 2 * kSMs - 1) / (2 * kSMs);
    const int64_t fit = kMaxRot / P.rot;
    if (rows > spread) rows = spread;
    if (rows > fit) rows = fit;
    if (rows < 1) rows = 1;
    P.rows = int(rows);
    const size_t smem = size_t(rows) * (P.rot / 2) * sizeof(float2);
    k_rotary<T, VEC, HALF><<<unsigned((P.N + rows - 1) / rows), 256, smem, st>>>(P);
}
template <typename T, int VEC>
void launch_rotary(RotaryParams &P, bool half, cudaStream_t st) {
    if (half) launch_rotary<T, VEC, true>(P, st);
    else launch_rotary<T, VEC, false>(P, st);
}
template <typename T>
void dispatch_rotary(RotaryParams &P, bool half, uintptr_t addresses, cudaStream_t st) {
    // the widest vector that divides the pairs' run, the head, what is copied, and the addresses
    const int run = half ? P.rot / 2 : P.rot;
    auto fits = [&](int vec) {
        return run % vec == 0 && P.D % vec == 0 && P.rot % vec == 0 && addresses % (vec * sizeof(T)) == 0;
    };
    if (sizeof(T) == 2 && fits(8)) launch_rotary<T, sizeof(T) == 2 ? 8 : 4>(P, half, st);
    else if (fits(4)) launch_rotary<T, 4>(P, half, st);
    else if (fits(2)) launch_rotary<T, 2>(P, half, st);
    else launch_rotary<T, 1>(P, half, st);
}

// ---------------------------------------------------------------------------- norm, gate and residual

// forward:  X = R + scale * drop(act(G) * (norm(B) * gamma1 + beta1)),  Z = norm(X) * gamma2 + beta2
// norm: x / sqrt(mean(x^2) + eps), or with the mean subtracted first.  One pass;
// a row stays in registers, its statistics are sums over the lanes that hold it.
// Forward [2^20, 128] bf16, LAYER, SiLU: 258 us, with p = 0.1 275-296 us, 69-75 %
// of the measured copy rate at 47 instructions an element (556 us with vectors
// loaded value by value): no pipe is full (issue slots 63 %, DRAM 56 % of nominal),
// but 96 registers, 32 of them the four vectors and 12 the next row, leave 28 % of
// the warps.  Backward [156323, 256] fp32, p = 0.1: 232-248 us, 79-84 %, HBM (352
// us with 64 threads and eight barriers a row in place of a warp).  Backward in
// bf16 takes four features a thread and fp32 arithmetic value by value, and is
// bound by instructions: [2^20, 128], p = 0.1: 863 us against 328 for the bytes.
// Rows of more than 64 vectors of four span several warps and wait at block
// barriers: 2^26 elements in rows of 512 to 8192, p = 0.1, run at 33 to 92 % of the
// copy rate forward and 42 to 70 % backward in fp32, 26 to 63 % and 23 to 43 % in
// bf16 (the least from 4096 on).
struct NormParams {
    const void *R, *B, *G, *X, *dX, *dZ;      // inputs (absent: null)
    void *oX, *oZ, *dR, *dB, *dG;             // outputs (absent: null)
    const float *gamma1, *beta1, *scale, *gamma2, *beta2;
    float *partial;                           // [blocks][5][H] (backward)
    int64_t N;
    int H, layer, silu;
    float eps, inv_h;
    Drop drop;
};

// Sums of up to two values over the TPR threads of a row (all get them).
template <int TPR>
__device__ __forceinline__ float2 row_sum(float2 v, float2 *red) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(kAll, v.x, o);
        v.y += __shfl_xor_sync(kAll, v.y, o);
    }
    if (TPR > 32) {
        constexpr int warps = TPR / 32;
        const int group = threadIdx.x / TPR * warps, w = threadIdx.x / 32;
        __syncthreads();  // the previous sums have been read
        if ((threadIdx.x & 31) == 0) red[w] = v;
        __syncthreads();
        v = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < warps; ++k) {
            v.x += red[group + k].x;
            v.y += red[group + k].y;
        }
    }
    return v;
}

// 1 / (1 + 2^y), and of y = -x log2(e) the logistic function.  The constant and
// the product round once each, which moves the exponential by 2 |x| 2^-24,
// relative; the exponential and the division are off by 2 steps (2^-22) each, the
// sum by half a step: (2 |x| + 9) 2^-24 down to x = -87.3.  Below, where it is
// less than 2^-126, the result is 0.
__device__ __forceinline__ float logistic2(float y) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    return __fdividef(1.f, 1.f + e);
}
__device__ __forceinline__ float sigmoid(float x) { return logistic2(x * -1.4426950408889634f); }

// VEC values of a vector from column c on, or `none` where there is no vector
template <int VEC>
__device__ __forceinline__ void load_param(const float *p, int c, float none, float (&v)[VEC]) {
    if (p) {
#pragma unroll
        for (int i = 0; i < VEC; i += VEC < 4 ? 1 : 4) {
            if constexpr (VEC < 4) {
                v[i] = __ldg(p + c + i);
            } else {
                const float4 q = __ldg(reinterpret_cast<const float4 *>(p + c + i));
                v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = none;
    }
}

// Keep bits of VEC elements from i on (a multiple of VEC where VEC >= 4).
template <int VEC>
__device__ __forceinline__ uint32_t keep_vec(uint64_t i, const Drop &d) {
    if constexpr (VEC == 1) return keep4(i >> 2, d) >> (i & 3) & 1u;
    uint32_t k = 0;
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) k |= keep4((i >> 2) + q, d) << (4 * q);
    return k;
}

constexpr int norm_threads(int tpr) { return tpr < 128 ? 128 : tpr; }

// x - mean(x) (layer), then 1 / sqrt(mean(x^2) + eps).  whole: every lane of
// the row holds VEC * NV of its columns (else the others' stay 0).
template <int VEC, int NV, int TPR>
__device__ __forceinline__ float normalise(float (&x)[NV][VEC], const bool (&ok)[NV], bool whole, const NormParams &P,
                                           float2 *red) {
    float2 s = make_float2(0.f, 0.f);
    if (P.layer) {
#pragma unroll
        for (int k = 0; k < NV; ++k) s.x += sum_all<VEC>(x[k]);
        const float mean = row_sum<TPR>(s, red).x * P.inv_h;
        float minus[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) minus[v] = -mean;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            add_all<VEC>(x[k], minus);
            if (!whole && !ok[k]) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) x[k][v] = 0.f;
            }
        }
    }
    s.x = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) s.x += squares_all<VEC>(x[k]);
    return rsqrtf(fmaf(row_sum<TPR>(s, red).x, P.inv_h, P.eps));
}

template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(norm_threads(TPR)) k_resnorm_fwd(const NormParams P) {
    constexpr int THREADS = norm_threads(TPR);
    constexpr int RPB = THREADS / TPR;
    constexpr bool AHEAD = NV * VEC <= 8 && TPR <= 256;  // the next row's loads, and the vectors, in registers
    using F = Frag<T, VEC>;
    using raw = typename F::raw;
    __shared__ float2 red[THREADS / 32];
    const int l = threadIdx.x % TPR;
    bool ok[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) ok[k] = (l + k * TPR) * VEC < P.H;
    const bool whole = P.H == TPR * NV * VEC;
    // scale / (1 - p) times gamma1 and beta1; gamma2, beta2
    float g1[NV][VEC], b1[NV][VEC], g2[NV][VEC], b2[NV][VEC];
    auto load_params = [&](int k) {
        const int c = ok[k] ? (l + k * TPR) * VEC : 0;
        float s[VEC];
        load_param<VEC>(P.scale, c, 1.f, s);
        load_param<VEC>(P.gamma1, c, 1.f, g1[k]);
        load_param<VEC>(P.beta1, c, 0.f, b1[k]);
        load_param<VEC>(P.gamma2, c, 1.f, g2[k]);
        load_param<VEC>(P.beta2, c, 0.f, b2[k]);
#pragma unroll
        for (int v = 0; v < VEC; ++v) s[v] *= P.drop.scale, g1[k][v] *= s[v], b1[k][v] *= s[v];
    };
    raw nR[NV], nB[NV], nG[NV];
    auto load_row = [&](int64_t n) {
        const int64_t at = n * P.H;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (l + k * TPR) * VEC;
            const bool in = n < P.N && ok[k];
            nR[k] = in && P.R ? F::load_stream(static_cast<const T *>(P.R) + at + c) : F::zero();
            nB[k] = in && P.B ? F::load_stream(static_cast<const T *>(P.B) + at + c) : F::zero();
            nG[k] = in && P.G ? F::load_stream(static_cast<const T *>(P.G) + at + c) : F::zero();
        }
    };
    const int64_t step = int64_t(gridDim.x) * RPB;
    const int64_t first = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR;
    if (AHEAD) {
#pragma unroll
        for (int k = 0; k < NV; ++k) load_params(k);
        load_row(first);
    }
    for (int64_t n0 = int64_t(blockIdx.x) * RPB; n0 < P.N; n0 += step) {
        const int64_t n = n0 + threadIdx.x / TPR;
        const bool row = n < P.N;
        const int64_t at = n * P.H;
        if (!AHEAD) load_row(n);
        float x[NV][VEC], b[NV][VEC], g[NV][VEC];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            F::unpack(nR[k], x[k]);
            F::unpack(nB[k], b[k]);
            F::unpack(nG[k], g[k]);
        }
        if (AHEAD) load_row(n + step);
        if (P.B) {
            const float r = normalise<VEC, NV, TPR>(b, ok, whole, P, red);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (l + k * TPR) * VEC;
                if (!AHEAD) load_params(k);
                mul_all<VEC>(b[k], r);
                fma_all<VEC>(b[k], g1[k], b1[k]);
                if (P.G) {
                    float s[VEC], none[VEC];
#pragma unroll
                    for (int v = 0; v < VEC; ++v) s[v] = g[k][v], none[v] = -0.f;
                    mul_all<VEC>(s, -1.4426950408889634f);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) s[v] = logistic2(s[v]);
                    if (P.silu) fma_all<VEC>(s, g[k], none);
                    fma_all<VEC>(b[k], s, none);
                }
                if (P.drop.on) {
                    const uint32_t kept = keep_vec<VEC>(uint64_t(at + c), P.drop);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) b[k][v] = kept >> v & 1u ? b[k][v] : 0.f;
                }
                if (!whole && !ok[k]) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) b[k][v] = 0.f;
                }
                add_all<VEC>(x[k], b[k]);
                if (row && ok[k]) F::store(static_cast<T *>(P.oX) + at + c, x[k]);
            }
        }
        if (P.oZ) {
            const float r = normalise<VEC, NV, TPR>(x, ok, whole, P, red);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (!AHEAD) load_params(k);
                mul_all<VEC>(x[k], r);
                fma_all<VEC>(x[k], g2[k], b2[k]);
                if (row && ok[k]) F::store(static_cast<T *>(P.oZ) + at + (l + k * TPR) * VEC, x[k]);
            }
        }
    }
}

// backward, from the stored X and B (the norms' statistics are recomputed
// from the row, which is in registers):
//   n2 = norm(X): dR = dX + norm'(dZ gamma2), dgamma2 += dZ n2, dbeta2 += dZ
//   n1 = norm(B), u = n1 gamma1 + beta1, k = keep / (1 - p):
//   dscale += dR k act u, dG = dR scale k act' u, du = dR scale k act,
//   dgamma1 += du n1, dbeta1 += du, dB = norm'(du gamma1)
// with norm'(y) = r (y - n mean(y n) [- mean(y)]).  A thread keeps the column
// sums of the rows it visits in registers; a block adds its threads' sums in
// shared memory and writes one partial row, and k_resnorm_join adds the
// blocks' in order.
template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(norm_threads(TPR)) k_resnorm_bwd(const NormParams P) {
    constexpr int THREADS = norm_threads(TPR);
    constexpr int RPB = THREADS / TPR;
    using F = Frag<T, VEC>;
    __shared__ float2 red[THREADS / 32];
    __shared__ float cols[RPB > 1 ? THREADS * VEC * NV : 1];
    follow_on();
    const int l = threadIdx.x % TPR;
    bool ok[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) ok[k] = (l + k * TPR) * VEC < P.H;
    float sum[5][NV][VEC];  // dgamma1, dbeta1, dscale, dgamma2, dbeta2
#pragma unroll
    for (int a = 0; a < 5; ++a)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) sum[a][k][v] = 0.f;
    for (int64_t n0 = int64_t(blockIdx.x) * RPB; n0 < P.N; n0 += int64_t(gridDim.x) * RPB) {
        const int64_t n = n0 + threadIdx.x / TPR;
        const bool row = n < P.N;
        const int64_t at = n * P.H;
        float x[NV][VEC], b[NV][VEC], dr[NV][VEC];
        typename F::raw rz[NV], rg[NV];
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (l + k * TPR) * VEC;
            const bool in = row && ok[k];
            F::unpack(in && P.X && P.dZ ? F::load_stream(static_cast<const T *>(P.X) + at + c) : F::zero(), x[k]);
            F::unpack(in && P.B ? F::load_stream(static_cast<const T *>(P.B) + at + c) : F::zero(), b[k]);
            F::unpack(in && P.dX ? F::load_stream(static_cast<const T *>(P.dX) + at + c) : F::zero(), dr[k]);
            rz[k] = in && P.dZ ? F::load_stream(static_cast<const T *>(P.dZ) + at + c) : F::zero();
            rg[k] = in && P.G ? F::load_stream(static_cast<const T *>(P.G) + at + c) : F::zero();
        }
        if (P.layer) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) s.x += x[k][v], s.y += b[k][v];
            s = row_sum<TPR>(s, red);
            const float mx = s.x * P.inv_h, mb = s.y * P.inv_h;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) x[k][v] = ok[k] ? x[k][v] - mx : 0.f, b[k][v] = ok[k] ? b[k][v] - mb : 0.f;
            s = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) s.x = fmaf(x[k][v], x[k][v], s.x), s.y = fmaf(b[k][v], b[k][v], s.y);
        s = row_sum<TPR>(s, red);
        // (a row behind the last one adds nothing: its zeros times 0, not times 1 / sqrt(eps = 0))
        const float rx = row ? rsqrtf(fmaf(s.x, P.inv_h, P.eps)) : 0.f;
        const float rb = row ? rsqrtf(fmaf(s.y, P.inv_h, P.eps)) : 0.f;
        if (P.dZ) {
            float2 q = make_float2(0.f, 0.f);
            float y[NV][VEC];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float gamma[VEC];
                load_param<VEC>(P.gamma2, ok[k] ? (l + k * TPR) * VEC : 0, 1.f, gamma);
                F::unpack(rz[k], y[k]);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    x[k][v] *= rx;
                    sum[3][k][v] = fmaf(y[k][v], x[k][v], sum[3][k][v]);
                    sum[4][k][v] += y[k][v];
                    y[k][v] *= gamma[v];
                    q.x = fmaf(y[k][v], x[k][v], q.x);
                    q.y += y[k][v];
                }
            }
            q = row_sum<TPR>(q, red);
            const float c1 = q.x * P.inv_h, c0 = P.layer ? q.y * P.inv_h : 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) dr[k][v] = fmaf(rx, fmaf(-x[k][v], c1, y[k][v] - c0), dr[k][v]);
        }
        if (P.dR) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (row && ok[k]) F::store(static_cast<T *>(P.dR) + at + (l + k * TPR) * VEC, dr[k]);
        }
        if (P.B) {
            float2 q = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = ok[k] ? (l + k * TPR) * VEC : 0;
                float gamma[VEC], beta[VEC], sc[VEC], g[VEC];
                load_param<VEC>(P.gamma1, c, 1.f, gamma);
                load_param<VEC>(P.beta1, c, 0.f, beta);
                load_param<VEC>(P.scale, c, 1.f, sc);
                F::unpack(rg[k], g);
                // (rows and columns outside hold dr = 0 or are not stored)
                if (P.drop.on) {
                    const uint32_t kept = keep_vec<VEC>(uint64_t(at + c), P.drop);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        dr[k][v] = kept >> v & 1u ? dr[k][v] * P.drop.scale : 0.f;
                        g[v] = kept >> v & 1u ? g[v] : 0.f;  // (0 times an infinite gate is no 0)
                    }
                }
                if (!ok[k]) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) dr[k][v] = 0.f;
                }
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float nb = b[k][v] * rb;
                    b[k][v] = nb;
                    const float u = fmaf(nb, gamma[v], beta[v]);
                    float act = 1.f, slope = 0.f;
                    if (P.G) {
                        const float sg = sigmoid(g[v]);
                        act = sg;
                        slope = fmaf(-sg, sg, sg);
                        if (P.silu) slope = fmaf(g[v], slope, sg), act = g[v] * sg;
                    }
                    const float d = dr[k][v], ds = d * sc[v];
                    sum[2][k][v] = fmaf(d, act * u, sum[2][k][v]);
                    g[v] = ds * u * slope;
                    float du = ds * act;
                    sum[0][k][v] = fmaf(du, nb, sum[0][k][v]);
                    sum[1][k][v] += du;
                    du *= gamma[v];
                    dr[k][v] = du;
                    q.x = fmaf(du, nb, q.x);
                    q.y += du;
                }
                if (row && ok[k] && P.dG) F::store(static_cast<T *>(P.dG) + at + c, g);
            }
            q = row_sum<TPR>(q, red);
            const float c1 = q.x * P.inv_h, c0 = P.layer ? q.y * P.inv_h : 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) dr[k][v] = rb * fmaf(-b[k][v], c1, dr[k][v] - c0);
                if (row && ok[k]) F::store(static_cast<T *>(P.dB) + at + (l + k * TPR) * VEC, dr[k]);
            }
        }
    }
    if (!P.partial) return;
#pragma unroll
    for (int a = 0; a < 5; ++a) {
        float *out = P.partial + (int64_t(blockIdx.x) * 5 + a) * P.H;
        if (RPB > 1) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) cols[(threadIdx.x / TPR * TPR * NV + k * TPR + l) * VEC + v] = sum[a][k][v];
            __syncthreads();
            for (int c = threadIdx.x; c < P.H; c += THREADS) {
                float s = 0.f;
                for (int q = 0; q < RPB; ++q) s += cols[q * TPR * NV * VEC + c];
                out[c] = s;
            }
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    if (ok[k]) out[(l + k * TPR) * VEC + v] = sum[a][k][v];
        }
    }
}

struct JoinParams {
    const float *partial;
    float *out[5];
    int blocks, H;
};
// Column sums of the blocks' partial rows: a block takes 32 columns of one
// vector, its 32 warps each add every 32nd row, then the 32 in order.
__global__ void __launch_bounds__(1024) k_resnorm_join(const JoinParams P) {
    __shared__ float red[32][33];
    follow_on();
    float *out = P.out[blockIdx.y];
    if (!out) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < P.H) {
#pragma unroll 8
        for (int b = w; b < P.blocks; b += 32) s += P.partial[(int64_t(b) * 5 + blockIdx.y) * P.H + c];
    }
    red[w][lane] = s;
    __syncthreads();
    // warp w adds the 32 partial sums of column w by a fixed tree
    s = red[lane][w];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if (lane == 0 && blockIdx.x * 32 + w < P.H) out[blockIdx.x * 32 + w] = s;
}

constexpr int kMaxNormWidth = 8192;
// Blocks of the backward pass: a bound of its partial rows that depends on
// the sizes alone.
int64_t norm_blocks(int64_t N, int64_t H) {
    int64_t per_sm = 8192 / H;
    per_sm = per_sm < 2 ? 2 : (per_sm > 8 ? 8 : per_sm);
    return N < kSMs * per_sm ? N : kSMs * per_sm;
}

template <typename T, int VEC, int NV, int TPR, bool BACK>
void launch_norm(const NormParams &P, int *blocks, cudaStream_t st) {
    constexpr int THREADS = norm_threads(TPR);
    constexpr int RPB = THREADS / TPR;
    if constexpr (BACK) {
        *blocks = int(grid_of(P.N, RPB, norm_blocks(P.N, P.H)));
        launch(k_resnorm_bwd<T, VEC, NV, TPR>, dim3(unsigned(*blocks)), THREADS, false, P, st);
    } else {
        k_resnorm_fwd<T, VEC, NV, TPR><<<grid_of(P.N, RPB, kSMs * 16), THREADS, 0, st>>>(P);
    }
}
// Threads per row: the power of two that covers the row's n vectors.  Up to
// 64 vectors of four a row stays in a warp (two vectors a thread: no block
// barrier in the row sums; [156323, 256] fp32 backward 352 -> 234 us).  Wider rows
// in a warp, with more vectors a thread, are not measured.
template <typename T, int VEC, bool BACK>
void dispatch_norm(const NormParams &P, int *blocks, cudaStream_t st) {
    const int n = (P.H + VEC - 1) / VEC;
    if constexpr (VEC == 1) {
        if (n <= 32) launch_norm<T, VEC, 1, 32, BACK>(P, blocks, st);
        else if (n <= 256) launch_norm<T, VEC, 8, 32, BACK>(P, blocks, st);
        else if (n <= 2048) launch_norm<T, VEC, 8, 256, BACK>(P, blocks, st);
        else launch_norm<T, VEC, 8, 1024, BACK>(P, blocks, st);
    } else {
        if (n <= 4) launch_norm<T, VEC, 1, 4, BACK>(P, blocks, st);
        else if (n <= 8) launch_norm<T, VEC, 1, 8, BACK>(P, blocks, st);
        else if (n <= 16) launch_norm<T, VEC, 1, 16, BACK>(P, blocks, st);
        else if (n <= 32) launch_norm<T, VEC, 1, 32, BACK>(P, blocks, st);
        else if (n <= 64) launch_norm<T, VEC, VEC == 4 ? 2 : 1, VEC == 4 ? 32 : 64, BACK>(P, blocks, st);
        else if (n <= 128) launch_norm<T, VEC, 1, 128, BACK>(P, blocks, st);
        else if (n <= 256) launch_norm<T, VEC, 1, 256, BACK>(P, blocks, st);
        else if (n <= 512) launch_norm<T, VEC, 1, 512, BACK>(P, blocks, st);
        else if (n <= 1024) launch_norm<T, VEC, 1, 1024, BACK>(P, blocks, st);
        else if constexpr (VEC == 4) launch_norm<T, VEC, 2, 1024, BACK>(P, blocks, st);
    }
}
// The widest vector that divides the rows and every address.  Backward, four
// features at most: the five column sums of eight take 40 registers.
template <typename T, bool BACK>
void dispatch_norm(const NormParams &P, uintptr_t addresses, uintptr_t vectors, int *blocks, cudaStream_t st) {
    auto fits = [&](int vec) { return P.H % vec == 0 && addresses % (vec * sizeof(T)) == 0 && vectors % 16 == 0; };
    if constexpr (sizeof(T) == 2 && !BACK) {
        if (fits(8)) return dispatch_norm<T, 8, BACK>(P, blocks, st);
    }
    if (fits(4)) dispatch_norm<T, 4, BACK>(P, blocks, st);
    else dispatch_norm<T, 1, BACK>(P, blocks, st);
}

// ---------------------------------------------------------------------------- checks

int check_dtype(int dtype, const char *fn) {
    return dtype == AG_F32 || dtype == AG_BF16 ? int(AG_OK) : fail(AG_ERR_DTYPE, "%s: unknown dtype %d", fn, dtype);
}
int check_drop(double p, const char *fn) {
    return p >= 0.0 && p < 1.0 ? int(AG_OK) : fail(AG_ERR_INVALID_ARG, "%s: p = %g outside [0, 1)", fn, p);
}
int element_size(int dtype) { return dtype == AG_F32 ? 4 : 2; }

int check_resnorm(const ag_resnorm *op, int64_t N, int64_t H, int dtype, const char *fn) {
    if (!op) return fail(AG_ERR_INVALID_ARG, "%s: null parameters", fn);
    if (N < 0 || N >= (int64_t(1) << 31) || H < 1 || H > kMaxNormWidth)
        return fail(AG_ERR_SHAPE, "%s: N = %lld outside [0, 2^31) or H = %lld outside [1, %d]", fn, (long long)N,
                    (long long)H, kMaxNormWidth);
    if (int rc = check_dtype(dtype, fn)) return rc;
    if (op->norm != AG_NORM_RMS && op->norm != AG_NORM_LAYER) return fail(AG_ERR_INVALID_ARG, "%s: unknown norm %d", fn, op->norm);
    if (op->act != AG_ACT_SIGMOID && op->act != AG_ACT_SILU) return fail(AG_ERR_INVALID_ARG, "%s: unknown gate %d", fn, op->act);
    if (!(op->eps >= 0.f) || !isfinite(op->eps)) return fail(AG_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
    return check_drop(op->p, fn);
}

NormParams norm_params(const ag_resnorm *op, int64_t N, int64_t H) {
    NormParams P = {};
    P.gamma1 = op->gamma1;
    P.beta1 = op->beta1;
    P.scale = op->scale;
    P.gamma2 = op->gamma2;
    P.beta2 = op->beta2;
    P.N = N;
    P.H = int(H);
    P.layer = op->norm == AG_NORM_LAYER;
    P.silu = op->act == AG_ACT_SILU;
    P.eps = op->eps;
    P.inv_h = 1.f / float(H);
    P.drop = make_drop(op->p, op->seed, op->offset);
    return P;
}

uintptr_t vector_addresses(const NormParams &P) {
    return uintptr_t(P.gamma1) | uintptr_t(P.beta1) | uintptr_t(P.scale) | uintptr_t(P.gamma2) | uintptr_t(P.beta2);
}

}  // namespace
}  // namespace ag

using namespace ag;

extern "C" {

int ag_dropout(const void *X, void *Y, int64_t n, double p, uint64_t seed, uint64_t offset, int dtype, void *stream) {
    const char *fn = "ag_dropout";
    clear_error();
    if (n < 0 || n >= (int64_t(1) << 40)) return fail(AG_ERR_SHAPE, "%s: n = %lld outside [0, 2^40)", fn, (long long)n);
    int rc;
    if ((rc = check_dtype(dtype, fn)) != AG_OK) return rc;
    if ((rc = check_drop(p, fn)) != AG_OK) return rc;
    if (n == 0) return AG_OK;
    const int b = element_size(dtype);
    const Operand ops[] = {{X, "X", size_t(n) * size_t(b), b, kIn}, {Y, "Y", size_t(n) * size_t(b), b, kOut}};
    if ((rc = check_operands(ops, kCurrent, true, fn)) != AG_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Drop drop = make_drop(p, seed, offset);
    if (dtype == AG_F32) launch_dropout<float, 4>(X, Y, n, drop, st);
    else launch_dropout<bf16_t, 8>(X, Y, n, drop, st);
    cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? AG_OK : cuda_fail(err, fn);
}

int ag_rotary_freqs(int64_t rot, double base, int scaling, double factor, double original, double beta_fast,
                    double beta_slow, double *inv_freq_host, double *factor_host) {
    const char *fn = "ag_rotary_freqs";
    clear_error();
    if (rot < 2 || rot > kMaxRot || rot % 2) return fail(AG_ERR_SHAPE, "%s: rot = %lld is not even in [2, %d]", fn, (long long)rot, kMaxRot);
    if (!inv_freq_host) return fail(AG_ERR_INVALID_ARG, "%s: null inv_freq", fn);
    if (!(base > 0.0) || !isfinite(base)) return fail(AG_ERR_INVALID_ARG, "%s: base must be positive", fn);
    if (scaling < AG_ROPE_NONE || scaling > AG_ROPE_YARN) return fail(AG_ERR_INVALID_ARG, "%s: unknown scaling %d", fn, scaling);
    if (scaling != AG_ROPE_NONE && (!(factor >= 1.0) || !isfinite(factor)))
        return fail(AG_ERR_INVALID_ARG, "%s: factor must be at least 1", fn);
    const double pi2 = 6.283185307179586;
    if (scaling == AG_ROPE_YARN && !(original > 0.0 && isfinite(original) && beta_fast > beta_slow && beta_slow > 0.0 && base != 1.0))
        return fail(AG_ERR_INVALID_ARG, "%s: needs original > 0, beta_fast > beta_slow > 0 and base != 1", fn);
    if (scaling == AG_ROPE_NTK && rot > 2) base *= pow(factor, double(rot) / double(rot - 2));
    double lo = 0.0, hi = 0.0;
    if (scaling == AG_ROPE_YARN) {
        // the pair that makes `turns` turns within the original range
        auto at = [&](double turns) { return double(rot) * log(original / (turns * pi2)) / (2.0 * log(base)); };
        lo = fmax(0.0, floor(at(beta_fast)));
        hi = fmin(double(rot - 1), ceil(at(beta_slow)));
    }
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = pow(base, -2.0 * double(i) / double(rot));
        if (scaling == AG_ROPE_LINEAR) f /= factor;
        if (scaling == AG_ROPE_YARN) {
            const double r = fmin(1.0, fmax(0.0, (double(i) - lo) / fmax(hi - lo, 0.001)));
            f = f / factor * r + f * (1.0 - r);
        }
        inv_freq_host[i] = f;
    }
    if (factor_host) *factor_host = scaling == AG_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
    return AG_OK;
}

int ag_rotary(const void *Q, const void *K, const int64_t *pos, const double *inv_freq, void *Qo, void *Ko, int64_t N,
              int64_t H, int64_t heads, int64_t rot, int interleaved, float factor, int inverse, int dtype,
              void *stream) {
    const char *fn = "ag_rotary";
    clear_error();
    if (N < 0 || N >= (int64_t(1) << 31) || H < 1 || H > (int64_t(1) << 20))
        return fail(AG_ERR_SHAPE, "%s: N = %lld outside [0, 2^31) or H = %lld outside [1, 2^20]", fn, (long long)N, (long long)H);
    if (heads < 1 || heads > H || H % heads) return fail(AG_ERR_SHAPE, "%s: H = %lld is not heads = %lld equal heads", fn, (long long)H, (long long)heads);
    if (rot < 2 || rot % 2 || rot > H / heads || rot > kMaxRot)
        return fail(AG_ERR_SHAPE, "%s: rot = %lld is not even in [2, min(H / heads, %d)]", fn, (long long)rot, kMaxRot);
    int rc;
    if ((rc = check_dtype(dtype, fn)) != AG_OK) return rc;
    if (!isfinite(factor)) return fail(AG_ERR_INVALID_ARG, "%s: factor must be finite", fn);
    if (N == 0) return AG_OK;
    const int b = element_size(dtype);
    const size_t f = size_t(N) * size_t(H) * size_t(b);
    const Operand ops[] = {{Q, "Q", f, b, kIn}, {K, "K", f, b, kMaybeIn}, {pos, "pos", size_t(N) * 8, 8, kParam},
                           {inv_freq, "inv_freq", size_t(rot) * 4, 8, kParam}, {Qo, "Q's output", f, b, kOut},
                           {K ? Ko : nullptr, "K's output", f, b, K ? kOut : kMaybeOut}};
    if ((rc = check_operands(ops, kCurrent, true, fn)) != AG_OK) return rc;
    RotaryParams P = {};
    P.in[0] = Q;
    P.in[1] = K;
    P.out[0] = Qo;
    P.out[1] = Ko;
    P.pos = pos;
    P.inv_freq = inv_freq;
    P.N = N;
    P.mats = K ? 2 : 1;
    P.H = int(H);
    P.heads = int(heads);
    P.D = int(H / heads);
    P.rot = int(rot);
    P.factor = factor;
    P.sign = inverse ? -1.f : 1.f;
    uintptr_t at = uintptr_t(Q) | uintptr_t(Qo);
    if (K) at |= uintptr_t(K) | uintptr_t(Ko);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == AG_F32) dispatch_rotary<float>(P, !interleaved, at, st);
    else dispatch_rotary<bf16_t>(P, !interleaved, at, st);
    cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? AG_OK : cuda_fail(err, fn);
}

int ag_resnorm_fwd(const ag_resnorm *op, const void *R, const void *B, const void *G, void *X, void *Z, int64_t N,
                   int64_t H, int dtype, void *stream) {
    const char *fn = "ag_resnorm_fwd";
    clear_error();
    int rc = check_resnorm(op, N, H, dtype, fn);
    if (rc != AG_OK) return rc;
    if (N == 0) return AG_OK;
    if (!B && G) return fail(AG_ERR_INVALID_ARG, "%s: a gate without a block output", fn);
    if (!B && X) return fail(AG_ERR_INVALID_ARG, "%s: X without a block output (the sum is R)", fn);
    if (!B && !R) return fail(AG_ERR_INVALID_ARG, "%s: neither R nor B", fn);
    if (!X && !Z) return fail(AG_ERR_INVALID_ARG, "%s: neither X nor Z", fn);
    const int b = element_size(dtype);
    const size_t f = size_t(N) * size_t(H) * size_t(b), h = size_t(H) * 4;
    const Operand ops[] = {{R, "R", f, b, kMaybeIn}, {B, "B", f, b, kMaybeIn}, {G, "G", f, b, kMaybeIn},
                           {X, "X", f, b, B ? kOut : kMaybeOut}, {Z, "Z", f, b, kMaybeOut},
                           {op->gamma1, "gamma1", h, 4, kMaybeParam}, {op->beta1, "beta1", h, 4, kMaybeParam},
                           {op->scale, "scale", h, 4, kMaybeParam}, {op->gamma2, "gamma2", h, 4, kMaybeParam},
                           {op->beta2, "beta2", h, 4, kMaybeParam}};
    if ((rc = check_operands(ops, kCurrent, true, fn)) != AG_OK) return rc;
    NormParams P = norm_params(op, N, H);
    P.R = R;
    P.B = B;
    P.G = G;
    P.oX = X;
    P.oZ = Z;
    const uintptr_t at = uintptr_t(R) | uintptr_t(B) | uintptr_t(G) | uintptr_t(X) | uintptr_t(Z);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == AG_F32) dispatch_norm<float, false>(P, at, vector_addresses(P), nullptr, st);
    else dispatch_norm<bf16_t, false>(P, at, vector_addresses(P), nullptr, st);
    cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? AG_OK : cuda_fail(err, fn);
}

size_t ag_resnorm_scratch_bytes(int64_t N, int64_t H) {
    if (N < 0 || N >= (int64_t(1) << 31) || H < 1 || H > kMaxNormWidth) return 0;
    return align_up(size_t(norm_blocks(N, H)) * 5 * size_t(H) * 4);
}

int ag_resnorm_backward(const ag_resnorm *op, const void *X, const void *B, const void *G, const void *dX,
                        const void *dZ, void *dR, void *dB, void *dG, float *dgamma1, float *dbeta1, float *dscale,
                        float *dgamma2, float *dbeta2, int64_t N, int64_t H, int dtype, void *scratch,
                        size_t scratch_bytes, void *stream) {
    const char *fn = "ag_resnorm_backward";
    clear_error();
    int rc = check_resnorm(op, N, H, dtype, fn);
    if (rc != AG_OK) return rc;
    if (N > 0) {  // matrices without rows have no addresses
        if (!B && (G || dB || dG || dgamma1 || dbeta1 || dscale))
            return fail(AG_ERR_INVALID_ARG, "%s: a gate or a gradient of the block without its output B", fn);
        if (!dZ && (dgamma2 || dbeta2)) return fail(AG_ERR_INVALID_ARG, "%s: dgamma2 or dbeta2 without dZ", fn);
        if (!G && dG) return fail(AG_ERR_INVALID_ARG, "%s: dG without a gate", fn);
        if (!dX && !dZ) return fail(AG_ERR_INVALID_ARG, "%s: neither dX nor dZ", fn);
    }
    float *const sums[5] = {dgamma1, dbeta1, dscale, dgamma2, dbeta2};
    bool any = false;
    for (float *s : sums) any = any || s;
    const size_t need = any ? ag_resnorm_scratch_bytes(N, H) : 0;
    if (need && (!scratch || scratch_bytes < need))
        return fail(AG_ERR_WORKSPACE, "%s: scratch of %zu bytes, need %zu", fn, scratch_bytes, need);
    if (reinterpret_cast<uintptr_t>(scratch) % kAlign != 0)
        return fail(AG_ERR_WORKSPACE, "%s: scratch must be 256-byte aligned", fn);
    const int b = element_size(dtype);
    const size_t f = size_t(N) * size_t(H) * size_t(b), h = size_t(H) * 4;
    const Operand ops[] = {{X, "X", f, b, N > 0 && dZ ? kIn : kMaybeIn}, {B, "B", f, b, kMaybeIn}, {G, "G", f, b, kMaybeIn},
                           {dX, "dX", f, b, kMaybeIn}, {dZ, "dZ", f, b, kMaybeIn}, {dR, "dR", f, b, kMaybeOut},
                           {dB, "dB", f, b, N > 0 && B ? kOut : kMaybeOut}, {dG, "dG", f, b, kMaybeOut},
                           {op->gamma1, "gamma1", h, 4, kMaybeParam}, {op->beta1, "beta1", h, 4, kMaybeParam},
                           {op->scale, "scale", h, 4, kMaybeParam}, {op->gamma2, "gamma2", h, 4, kMaybeParam},
                           {op->beta2, "beta2", h, 4, kMaybeParam}, {dgamma1, "dgamma1", h, 4, kMaybeLast},
                           {dbeta1, "dbeta1", h, 4, kMaybeLast}, {dscale, "dscale", h, 4, kMaybeLast},
                           {dgamma2, "dgamma2", h, 4, kMaybeLast}, {dbeta2, "dbeta2", h, 4, kMaybeLast},
                           {need ? scratch : nullptr, "scratch", need, 1, kMaybeScratch}};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((rc = check_operands(ops, kCurrent, true, fn)) != AG_OK) return rc;
    int blocks = 0;
    if (N > 0) {
        NormParams P = norm_params(op, N, H);
        P.X = X;
        P.B = B;
        P.G = G;
        P.dX = dX;
        P.dZ = dZ;
        P.dR = dR;
        P.dB = dB;
        P.dG = dG;
        P.partial = any ? static_cast<float *>(scratch) : nullptr;
        uintptr_t at = uintptr_t(X) | uintptr_t(B) | uintptr_t(G) | uintptr_t(dX) | uintptr_t(dZ);
        at |= uintptr_t(dR) | uintptr_t(dB) | uintptr_t(dG);
        if (dtype == AG_F32) dispatch_norm<float, true>(P, at, vector_addresses(P), &blocks, st);
        else dispatch_norm<bf16_t, true>(P, at, vector_addresses(P), &blocks, st);
    }
    if (any) {
        JoinParams J;
        J.partial = static_cast<const float *>(scratch);
        for (int k = 0; k < 5; ++k) J.out[k] = sums[k];
        J.blocks = blocks;
        J.H = int(H);
        launch(k_resnorm_join, dim3(unsigned((H + 31) / 32), 5), 1024, N > 0, J, st);
    }
    cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? AG_OK : cuda_fail(err, fn);
}

}  // extern "C"
