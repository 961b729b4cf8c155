// Differential edge-softmax attention over the forward adjacency: every head
// holds two softmax maps over a destination row's edges, and the second map,
// times a learned factor, is subtracted from the first.  With d = H / (2
// heads), q_m / k_m the d columns of map m of one head and v its 2d columns:
//
//   s_m,e   = scale * dot(q_m[dst_e], k_m[src_e])               m = 1, 2
//   alpha_m = softmax of s_m over the edges into each row
//   Y[r]    = sum over edges e into r of u_e (alpha_1,e - lambda alpha_2,e) v[src_e]
//
// u_e is 1, or with dropout keep_e / (1 - p).  Gradients, with da_e = u_e
// dot(dY[dst_e], v[src_e]) and D_m[r] = sum over r's edges of alpha_m da:
//
//   ds_1 = scale alpha_1 (da - D_1)     ds_2 = -lambda scale alpha_2 (da - D_2)
//   dq_m[r] = sum over edges into r of ds_m k_m[src_e]
//   dk_m[s] = sum over edges out of s of ds_m q_m[dst_e]
//   dv[s]   = sum over edges out of s of u (alpha_1 - lambda alpha_2) dY[dst_e]
//   dlambda = -sum over rows of D_2
//
// Three walks of the library's CSR tiles, each gathering two feature rows per
// edge once and keeping everything per edge in registers:
//   forward (kFwd)   destination rows; running maximum and sum per map, both
//                    maps' weighted sums of v (their factors are known only
//                    at the row's end), log-sum-exp written for the backward;
//   kDQ              destination rows; alpha from the log-sum-exp; D is not
//                    known before the row's end, so the walk sums
//                    A = sum alpha (da - c) k, B = sum alpha k and
//                    D' = sum alpha (da - c) for a reference c (the row's
//                    first da): dq = scale (A - D' B), D = c + D'.  The shift
//                    by c keeps A and D' B from cancelling;
//   kDKV             source rows of the transpose CSR; D known.
// No per-edge array is written or read besides the CSR itself.
//
// A warp walks one tile of T consecutive CSR positions (the tile schedule of
// the other aggregations).  2 DL lanes hold one head of one gathered row (DL
// lanes per map, NV vectors of VEC features per lane), head slots fill the
// warp up, and the remaining factor splits a row's edges over lane groups
// ("subs") that are summed at the row's end.  A lane's columns of K belong to
// its own map; its columns of V take the weights of both maps, the other
// one's by a shuffle.  Rows cut by tile boundaries leave fp32 partials that a
// fix-up kernel adds in tile order, so results are bitwise reproducible.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "aggraph.h"
#include "frag.cuh"
#include "internal.h"
#include "random.cuh"

namespace ag {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 4;            // warps (tiles) per block
constexpr int kZeroPerWarp = 32;     // rows without edges per warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxHeadDim = 256;     // per map
constexpr int kMaxHeads = 256;

enum Mode { kFwd = 0, kDQ = 1, kDKV = 2 };

struct DiffParams {
    const int32_t *col, *order, *tile_nz, *nz_rows, *nz_rowptr, *zero_rows;
    const void *own_a, *own_b;   // rows of the walk's owners: Q, dY (kFwd, kDQ) or K, V (kDKV)
    const void *nbr_a, *nbr_b;   // gathered rows: K, V or Q, dY
    const float *lam;            // [heads]
    const float *lse;            // [N, heads, 2] (kDQ)
    float *lse_out;              // [N, heads, 2] (kFwd)
    float2 *stat;                // [N, heads, 2] (log-sum-exp in base 2, D): written by kDQ, read by kDKV
    void *out_a, *out_b;         // Y | dQ | dK, dV
    float *partial;              // [2 * n_tiles] slots of `slot` floats
    int64_t slot;
    int64_t n_nz, n_zero, n_tiles;
    int64_t E;
    unsigned tile_blocks;
    int T, H, heads, d, hb_log2;
    float c2;                    // scale * log2(e)
    float scale;
    Drop drop;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Sum over the W lanes of an aligned group (a fixed butterfly).
template <int W>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Edges of a row in flight per sub.
constexpr int edges_in_flight(int nv) { return nv == 1 ? 4 : (nv == 2 ? 2 : 1); }

template <typename T, int VEC, int DL, int NV, int MODE>
__global__ void __launch_bounds__(kWarps * 32) k_diff_walk(const DiffParams P) {
    using F = Frag<T, VEC>;
    using raw = typename F::raw;
    constexpr int U = edges_in_flight(NV);
    constexpr int HL = 2 * DL;
    const int lane = threadIdx.x & 31;
    const int head_slots = 1 << P.hb_log2;
    const int sub_lanes = HL << P.hb_log2;       // lanes of one sub
    const int nsub = 32 / sub_lanes;
    const int sub = lane / sub_lanes;
    const int hs = (lane / HL) & (head_slots - 1);
    const int map = (lane / DL) & 1;
    const int l = lane & (DL - 1);
    const int h0 = int(blockIdx.y) << P.hb_log2;
    const int head = h0 + hs;
    const bool live = head < P.heads;
    // columns of this lane: col0 + k * DL * VEC
    const int col0 = (live ? head * 2 + map : 0) * P.d + l * VEC;
    bool ok[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) ok[k] = live && (l + k * DL) * VEC < P.d;

    auto load_row = [&](const void *base, int64_t row, bool valid, raw (&r)[NV]) {
        const T *p = static_cast<const T *>(base) + row * P.H + col0;
#pragma unroll
        for (int k = 0; k < NV; ++k) r[k] = valid && ok[k] ? F::load(p + k * DL * VEC) : F::zero();
    };
    auto store_row = [&](void *base, int64_t row, const float (&v)[NV][VEC]) {
        T *p = static_cast<T *>(base) + row * P.H + col0;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (ok[k]) F::store(p + k * DL * VEC, v[k]);
    };
    const int64_t stat_col = int64_t(live ? head : 0) * 2 + map;   // of [N, heads, 2]

    if (blockIdx.x >= P.tile_blocks) {  // rows without edges
        const int64_t z0 = (int64_t(blockIdx.x - P.tile_blocks) * kWarps + (threadIdx.x >> 5)) * kZeroPerWarp;
        float z[NV][VEC];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) z[k][v] = 0.f;
        for (int i = sub; i < kZeroPerWarp && z0 + i < P.n_zero; i += nsub) {
            const int64_t row = P.zero_rows[z0 + i];
            store_row(P.out_a, row, z);
            if (MODE == kDKV) store_row(P.out_b, row, z);
            if (live && l == 0) {
                if (MODE == kFwd) P.lse_out[row * P.heads * 2 + stat_col] = -INFINITY;
                if (MODE == kDQ) P.stat[row * P.heads * 2 + stat_col] = make_float2(0.f, 0.f);
            }
        }
        return;
    }
    const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= P.n_tiles) return;  // whole warps
    const int64_t p0 = t * P.T;
    const int len = int(P.E - p0 < P.T ? P.E - p0 : P.T);
    const int32_t *col = P.col + p0;

    const float lam = live ? P.lam[head] : 0.f;
    const float sign = map ? -lam : 1.f;

    // the open row, and the next one's id, end and owner rows ahead of use
    int64_t r = P.tile_nz[t];
    bool before = P.nz_rowptr[r] < p0;
    int row = 0, row_end = 0;
    int next_row = P.nz_rows[r];
    int next_end = int(P.nz_rowptr[r + 1] - p0);
    raw own_a[NV], own_b[NV], pre_a[NV], pre_b[NV];
    float own_lse = 0.f, pre_lse = 0.f;
    auto prefetch_owner = [&]() {
        load_row(P.own_a, next_row, true, pre_a);
        if (MODE != kFwd) load_row(P.own_b, next_row, true, pre_b);
        if (MODE == kDQ) pre_lse = P.lse[int64_t(next_row) * P.heads * 2 + stat_col];
    };
    prefetch_owner();

    // kFwd: sums of alpha v for the own and the other map; kDQ: A, B; kDKV: dk, dv
    float acc[2][NV][VEC];
    float m = 0.f, sum = 0.f, ref = 0.f;  // kFwd: maximum, sum; kDQ: sum of alpha, D', c
    float dsum = 0.f;
    bool open = false, first = false;

    // adds the subs' acc and sums (kFwd: first to one maximum)
    auto join_stats = [&]() {
        if (MODE == kFwd) {
            float M = m;
            for (int o = sub_lanes; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
            const float f = ex2(m - (M == -INFINITY ? 0.f : M));
            const float g = __shfl_xor_sync(kAll, f, DL);
            sum *= f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[0][k][v] *= f, acc[1][k][v] *= g;
            m = M;
        }
        for (int o = sub_lanes; o < 32; o <<= 1) {
            sum += __shfl_xor_sync(kAll, sum, o);
            if (MODE == kDQ) dsum += __shfl_xor_sync(kAll, dsum, o);
        }
    };
    auto join = [&](float (&a)[NV][VEC]) {
        for (int o = sub_lanes; o < 32; o <<= 1)
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) a[k][v] += __shfl_xor_sync(kAll, a[k][v], o);
    };
    // the open row's partial of this tile
    auto write_slot = [&](int64_t s) {
        join_stats();
        join(acc[0]);
        join(acc[1]);
        if (sub != 0 || !live) return;
        float *base = P.partial + s * P.slot;
        const int which = MODE == kFwd ? map : 0;  // kFwd: maps in order, whichever is the lane's own
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            float *p = base + int64_t(a ^ which) * P.H + col0;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    if (ok[k]) p[k * DL * VEC + v] = acc[a][k][v];
        }
        if (MODE != kDKV && l == 0) {
            float *q = base + 2 * int64_t(P.H) + stat_col;
            q[0] = m;
            q[2 * P.heads] = sum;
            if (MODE == kDQ) q[4 * P.heads] = dsum;
        }
    };
    auto finish_row = [&]() {
        if (before) {  // continued from the previous tile
            write_slot(2 * t);
            before = false;
            return;
        }
        join_stats();
        if (MODE == kFwd) {
            const float inv = P.drop.scale / sum;
            const float own_w = sign * inv;
            const float other_w = __shfl_xor_sync(kAll, own_w, DL);
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[0][k][v] = fmaf(acc[0][k][v], own_w, acc[1][k][v] * other_w);
            join(acc[0]);
            if (sub == 0) {
                store_row(P.out_a, row, acc[0]);
                if (live && l == 0) P.lse_out[int64_t(row) * P.heads * 2 + stat_col] = (m + log2f(sum)) * kLn2;
            }
        } else if (MODE == kDQ) {
            const float w = sign * P.scale;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[0][k][v] = w * fmaf(-dsum, acc[1][k][v], acc[0][k][v]);
            join(acc[0]);
            if (sub == 0) {
                store_row(P.out_a, row, acc[0]);
                if (live && l == 0) P.stat[int64_t(row) * P.heads * 2 + stat_col] = make_float2(own_lse, ref + dsum);
            }
        } else {
            join(acc[0]);
            join(acc[1]);
            if (sub == 0) {
                store_row(P.out_a, row, acc[0]);
                store_row(P.out_b, row, acc[1]);
            }
        }
    };

    int cid_next = lane < len ? __ldg(col + lane) : 0;
    for (int b0 = 0; b0 < len; b0 += 32) {
        const int cid = cid_next;
        cid_next = b0 + 32 + lane < len ? __ldg(col + b0 + 32 + lane) : 0;
        uint32_t bits = 0xffffffffu;
        if (P.drop.on && b0 + lane < len) {
            const int64_t e = P.order[p0 + b0 + lane];
            const int count = P.heads - h0 < head_slots ? P.heads - h0 : head_slots;
            bits = keep_bits(uint64_t(e) * P.heads + h0, count, P.drop);
        }
        const int b1 = b0 + 32 < len ? b0 + 32 : len;
        int pos = b0;
        while (pos < b1) {
            if (!open) {
                row = next_row;
                row_end = next_end;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    own_a[k] = pre_a[k];
                    if (MODE != kFwd) own_b[k] = pre_b[k];
#pragma unroll
                    for (int v = 0; v < VEC; ++v) acc[0][k][v] = acc[1][k][v] = 0.f;
                }
                if (MODE == kDQ) own_lse = pre_lse * kLog2e;
                m = MODE == kFwd ? -INFINITY : 0.f;
                sum = dsum = 0.f;
                open = first = true;
                if (r + 1 < P.n_nz) {
                    next_row = P.nz_rows[r + 1];
                    next_end = int(P.nz_rowptr[r + 2] - p0);
                    prefetch_owner();
                }
            }
            const int seg_end = row_end < b1 ? row_end : b1;
            for (int i = pos; i < seg_end; i += nsub * U) {
                raw na[U][NV], nb[U][NV];
                float2 st[U];
                bool valid[U];
                uint32_t kept[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int j = i + u * nsub + sub;
                    valid[u] = j < seg_end;
                    const int64_t c = __shfl_sync(kAll, cid, j & 31);
                    kept[u] = P.drop.on ? __shfl_sync(kAll, bits, j & 31) >> hs & 1u : 1u;
                    load_row(P.nbr_a, c, valid[u], na[u]);
                    load_row(P.nbr_b, c, valid[u], nb[u]);
                    if (MODE == kDKV) st[u] = valid[u] ? __ldg(P.stat + c * P.heads * 2 + stat_col) : make_float2(0.f, 0.f);
                }
                float x[U], da[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    x[u] = da[u] = 0.f;
#pragma unroll
                    for (int k = 0; k < NV; ++k) x[u] = F::dot(own_a[k], na[u][k], x[u]);
                    x[u] = group_sum<DL>(x[u]);
                    if (MODE != kFwd) {
#pragma unroll
                        for (int k = 0; k < NV; ++k) da[u] = F::dot(own_b[k], nb[u][k], da[u]);
                        da[u] = group_sum<HL>(da[u]);
                        da[u] = kept[u] ? da[u] * P.drop.scale : 0.f;
                    }
                }
                if (MODE == kFwd) {
                    float top = m;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        x[u] = valid[u] ? x[u] * P.c2 : -INFINITY;
                        top = fmaxf(top, x[u]);
                    }
                    const float base = top == -INFINITY ? 0.f : top;
                    if (__any_sync(kAll, top > m)) {
                        const float f = ex2(m - base);
                        const float g = __shfl_xor_sync(kAll, f, DL);
                        sum *= f;
#pragma unroll
                        for (int k = 0; k < NV; ++k)
#pragma unroll
                            for (int v = 0; v < VEC; ++v) acc[0][k][v] *= f, acc[1][k][v] *= g;
                        m = top;
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float p = ex2(x[u] - base);
                        sum += p;
                        p = kept[u] ? p : 0.f;
                        const float q = __shfl_xor_sync(kAll, p, DL);
#pragma unroll
                        for (int k = 0; k < NV; ++k) {
                            float vv[VEC];
                            F::unpack(nb[u][k], vv);
#pragma unroll
                            for (int v = 0; v < VEC; ++v) {
                                acc[0][k][v] = fmaf(p, vv[v], acc[0][k][v]);
                                acc[1][k][v] = fmaf(q, vv[v], acc[1][k][v]);
                            }
                        }
                    }
                } else if (MODE == kDQ) {
                    if (first) {  // the row's first edge in this tile: edge 0 of sub 0
                        ref = __shfl_sync(kAll, da[0], lane & (sub_lanes - 1));
                        m = ref;
                        first = false;
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float p = valid[u] ? ex2(fmaf(x[u], P.c2, -own_lse)) : 0.f;
                        const float q = valid[u] ? p * (da[u] - ref) : 0.f;
                        sum += p;
                        dsum += q;
#pragma unroll
                        for (int k = 0; k < NV; ++k) {
                            float vv[VEC];
                            F::unpack(na[u][k], vv);
#pragma unroll
                            for (int v = 0; v < VEC; ++v) {
                                acc[0][k][v] = fmaf(q, vv[v], acc[0][k][v]);
                                acc[1][k][v] = fmaf(p, vv[v], acc[1][k][v]);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float p = valid[u] ? sign * ex2(fmaf(x[u], P.c2, -st[u].x)) : 0.f;
                        const float both = p + __shfl_xor_sync(kAll, p, DL);
                        const float ds = valid[u] ? P.scale * p * (da[u] - st[u].y) : 0.f;
                        const float w = kept[u] ? both * P.drop.scale : 0.f;
#pragma unroll
                        for (int k = 0; k < NV; ++k) {
                            float va[VEC], vb[VEC];
                            F::unpack(na[u][k], va);
                            F::unpack(nb[u][k], vb);
#pragma unroll
                            for (int v = 0; v < VEC; ++v) {
                                acc[0][k][v] = fmaf(ds, va[v], acc[0][k][v]);
                                acc[1][k][v] = fmaf(w, vb[v], acc[1][k][v]);
                            }
                        }
                    }
                }
            }
            pos = seg_end;
            if (seg_end == row_end) {
                finish_row();
                open = false;
                ++r;
            }
        }
    }
    if (open) write_slot(before ? 2 * t : 2 * t + 1);
}

// Rows cut by tile boundaries: the partials of slot 2 first + 1 and of the
// slots 2t of tiles first + 1 .. last, added in tile order.  One block per
// row for the rows cut into many tiles (listed first; its threads split into
// stripes of columns, each taking every stripes-th slot, then the stripes are
// added in order), one warp for every other row.
constexpr int kFixThreads = 256;

struct FixParams {
    const int4 *spans;
    int64_t n_long, n_span;
    const float *partial;
    int64_t slot;
    const float *lam, *lse;
    float *lse_out;
    float2 *stat;
    void *out_a, *out_b;
    int H, heads, d;
    float scale, drop_scale;
};

// The sums over slots first, first + step, ... of one column: kFwd weights
// the maps' sums by exp2(m - M), kDQ shifts A by (c - C) B.
template <int MODE>
__device__ __forceinline__ float2 fix_column(const FixParams &P, int64_t s0, int64_t t0, int n, int first, int step,
                                             int c, float M1, float M2) {
    const int head = c / (2 * P.d), map = c / P.d & 1;
    float2 a = make_float2(0.f, 0.f);
    for (int i = first; i < n; i += step) {
        const float *b = P.partial + (i == 0 ? s0 : 2 * (t0 + i)) * P.slot;
        const float u = b[c], v = b[P.H + c];
        const float *q = b + 2 * int64_t(P.H) + 2 * head;
        if (MODE == kFwd) {
            a.x = fmaf(u, ex2(q[0] - M1), a.x);
            a.y = fmaf(v, ex2(q[1] - M2), a.y);
        } else if (MODE == kDQ) {
            a.x += fmaf(q[map] - M1, v, u);  // M1: the row's c
            a.y += v;
        } else {
            a.x += u;
            a.y += v;
        }
    }
    return a;
}

// Statistics of (head, map) index j over slots first, first + step, ...:
// kFwd (M, L); kDQ (C, D' rebased to C).
template <int MODE>
__device__ __forceinline__ float2 fix_stats(const FixParams &P, int64_t s0, int64_t t0, int n, int j) {
    const float *q0 = P.partial + 2 * int64_t(P.H) + j;
    auto at = [&](int i) { return q0 + (i == 0 ? s0 : 2 * (t0 + i)) * P.slot; };
    float2 a;
    if (MODE == kFwd) {
        float M = -INFINITY;
        for (int i = 0; i < n; ++i) M = fmaxf(M, at(i)[0]);
        if (M == -INFINITY) M = 0.f;
        float L = 0.f;
        for (int i = 0; i < n; ++i) L = fmaf(at(i)[2 * P.heads], ex2(at(i)[0] - M), L);
        a = make_float2(M, L);
    } else {
        const float C = at(0)[0];
        float D = 0.f;
        for (int i = 0; i < n; ++i) D += fmaf(at(i)[0] - C, at(i)[2 * P.heads], at(i)[4 * P.heads]);
        a = make_float2(C, D);
    }
    return a;
}

template <typename T, int MODE>
__device__ __forceinline__ void fix_store(const FixParams &P, int64_t row, int c, float2 a, float2 s1, float2 s2) {
    const int head = c / (2 * P.d), map = c / P.d & 1;
    const float lam = P.lam[head];
    float y[1];
    if (MODE == kFwd) {
        y[0] = P.drop_scale * (a.x / s1.y - lam * (a.y / s2.y));
    } else if (MODE == kDQ) {
        y[0] = (map ? -lam : 1.f) * P.scale * fmaf(-s1.y, a.y, a.x);  // s1: this map's (C, D')
    } else {
        y[0] = a.x;
    }
    Frag<T, 1>::store(static_cast<T *>(P.out_a) + row * P.H + c, y);
    if (MODE == kDKV) {
        y[0] = a.y;
        Frag<T, 1>::store(static_cast<T *>(P.out_b) + row * P.H + c, y);
    }
}
template <int MODE>
__device__ __forceinline__ void fix_store_stats(const FixParams &P, int64_t row, int j, float2 s) {
    const int64_t k = row * P.heads * 2 + j;
    if (MODE == kFwd) P.lse_out[k] = (s.x + log2f(s.y)) * kLn2;
    if (MODE == kDQ) P.stat[k] = make_float2(P.lse[k] * kLog2e, s.x + s.y);
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kFixThreads) k_diff_fixup(const FixParams P) {
    __shared__ float2 stats[2 * kMaxHeads];  // long rows: per (head, map)
    __shared__ float2 red[kFixThreads];
    if (blockIdx.x < P.n_long) {
        const int4 sp = P.spans[blockIdx.x];
        const int n = sp.z - sp.y + 1;
        const int64_t s0 = 2 * int64_t(sp.y) + 1, t0 = sp.y;
        if (MODE != kDKV) {
            for (int j = threadIdx.x; j < 2 * P.heads; j += kFixThreads) {
                stats[j] = fix_stats<MODE>(P, s0, t0, n, j);
                fix_store_stats<MODE>(P, sp.x, j, stats[j]);
            }
            __syncthreads();
        }
        int cols = 32;
        while (cols < P.H && cols < kFixThreads) cols <<= 1;
        const int stripes = kFixThreads / cols;
        const int stripe = threadIdx.x / cols;
        for (int c0 = 0; c0 < P.H; c0 += cols) {
            const int c = c0 + threadIdx.x % cols;
            float2 s1 = make_float2(0.f, 1.f), s2 = s1, a = make_float2(0.f, 0.f);
            if (c < P.H) {
                if (MODE == kFwd) s1 = stats[c / (2 * P.d) * 2], s2 = stats[c / (2 * P.d) * 2 + 1];
                if (MODE == kDQ) s1 = stats[c / P.d];
                a = fix_column<MODE>(P, s0, t0, n, stripe, stripes, c, s1.x, s2.x);
            }
            red[threadIdx.x] = a;
            __syncthreads();
            if (stripe == 0 && c < P.H) {
                for (int k = 1; k < stripes; ++k) {
                    const float2 b = red[k * cols + threadIdx.x];
                    a.x += b.x;
                    a.y += b.y;
                }
                fix_store<T, MODE>(P, sp.x, c, a, s1, s2);
            }
            __syncthreads();
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t s = P.n_long + (int64_t(blockIdx.x) - P.n_long) * (kFixThreads / 32) + (threadIdx.x >> 5);
    if (s >= P.n_span) return;
    const int4 sp = P.spans[s];
    const int n = sp.z - sp.y + 1;
    const int64_t s0 = 2 * int64_t(sp.y) + 1, t0 = sp.y;
    for (int c = lane; c < P.H; c += 32) {
        const int head = c / (2 * P.d);
        float2 s1 = make_float2(0.f, 1.f), s2 = s1;
        if (MODE == kFwd) s1 = fix_stats<MODE>(P, s0, t0, n, 2 * head), s2 = fix_stats<MODE>(P, s0, t0, n, 2 * head + 1);
        if (MODE == kDQ) s1 = fix_stats<MODE>(P, s0, t0, n, c / P.d);
        fix_store<T, MODE>(P, sp.x, c, fix_column<MODE>(P, s0, t0, n, 0, 1, c, s1.x, s2.x), s1, s2);
    }
    if (MODE != kDKV)
        for (int j = lane; j < 2 * P.heads; j += 32) fix_store_stats<MODE>(P, sp.x, j, fix_stats<MODE>(P, s0, t0, n, j));
}

// dlambda[h] = -sum over rows of D_2: block b sums rows b, b + blocks, ...
// in fp64 (a row's threads fixed), then one block adds the blocks in order.
constexpr int kLamBlocks = 148;

__global__ void __launch_bounds__(256) k_diff_dlam(const float2 *__restrict__ stat, int64_t N, int heads,
                                                   double *__restrict__ partial) {
    __shared__ double red[256];
    for (int h = 0; h < heads; ++h) {
        double s = 0.0;
        for (int64_t r = int64_t(blockIdx.x) * 256 + threadIdx.x; r < N; r += int64_t(gridDim.x) * 256)
            s += double(stat[(r * heads + h) * 2 + 1].y);
        red[threadIdx.x] = s;
        __syncthreads();
        for (int o = 128; o > 0; o >>= 1) {
            if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
            __syncthreads();
        }
        if (threadIdx.x == 0) partial[int64_t(blockIdx.x) * heads + h] = red[0];
        __syncthreads();
    }
}
__global__ void k_diff_dlam_join(const double *__restrict__ partial, int blocks, int heads, float *__restrict__ dlam) {
    for (int h = threadIdx.x; h < heads; h += blockDim.x) {
        double s = 0.0;
        for (int b = 0; b < blocks; ++b) s += partial[int64_t(b) * heads + h];
        dlam[h] = float(-s);
    }
}

// ---------------------------------------------------------------------------- host side

// scratch: slots of cut rows | stat [N, heads, 2] | dlambda partials
struct DiffLayout {
    size_t partial, stat, dlam, total;
    int64_t slot;
};
DiffLayout diff_layout(const ag_graph *g, int64_t H, int64_t heads) {
    DiffLayout L;
    L.slot = (2 * H + 6 * heads + 3) / 4 * 4;
    const bool spans = g->dir[0].n_span > 0 || g->dir[1].n_span > 0;
    L.partial = 0;
    L.stat = align_up(spans ? size_t(2) * size_t(g->n_tiles) * size_t(L.slot) * 4 : 0);
    L.dlam = L.stat + align_up(size_t(g->N) * size_t(heads) * 2 * sizeof(float2));
    L.total = L.dlam + align_up(size_t(kLamBlocks) * size_t(heads) * 8);
    return L;
}

bool heads_fit(int64_t H, int64_t heads) {
    return heads >= 1 && heads <= kMaxHeads && H >= 2 && H % (2 * heads) == 0 && H / (2 * heads) <= kMaxHeadDim;
}

template <typename T, int VEC, int DL, int NV, int MODE>
void launch_walk(DiffParams &P, cudaStream_t st) {
    int hb = 0;  // head slots: fill the warp, not beyond the heads
    while ((4 * DL << hb) <= 32 && (1 << hb) < P.heads) ++hb;
    P.hb_log2 = hb;
    P.tile_blocks = unsigned((P.n_tiles + kWarps - 1) / kWarps);
    const int64_t zero = (P.n_zero + kWarps * kZeroPerWarp - 1) / (kWarps * kZeroPerWarp);
    const unsigned y = unsigned((P.heads + (1 << hb) - 1) >> hb);
    const dim3 grid(unsigned(P.tile_blocks + zero), y);
    if (grid.x > 0) k_diff_walk<T, VEC, DL, NV, MODE><<<grid, kWarps * 32, 0, st>>>(P);
}

// Vectors per map n = d / VEC: the next power of two of lanes up to 16, then
// more vectors per lane.
template <typename T, int VEC, int MODE>
void launch_vec(DiffParams &P, cudaStream_t st) {
    const int n = P.d / VEC;
    if constexpr (VEC == 1) {  // one feature at a time: sizes and addresses without a wider vector
        if (n <= 4) launch_walk<T, VEC, 4, 1, MODE>(P, st);
        else if (n <= 16) launch_walk<T, VEC, 16, 1, MODE>(P, st);
        else if (n <= 64) launch_walk<T, VEC, 16, 4, MODE>(P, st);
        else launch_walk<T, VEC, 16, 16, MODE>(P, st);
    } else {
        constexpr int kWide = VEC * int(sizeof(T)) == 16 && sizeof(T) == 2 ? 2 : 4;  // kMaxHeadDim / (16 VEC)
        if (n <= 1) launch_walk<T, VEC, 1, 1, MODE>(P, st);
        else if (n <= 2) launch_walk<T, VEC, 2, 1, MODE>(P, st);
        else if (n <= 4) launch_walk<T, VEC, 4, 1, MODE>(P, st);
        else if (n <= 8) launch_walk<T, VEC, 8, 1, MODE>(P, st);
        else if (n <= 16) launch_walk<T, VEC, 16, 1, MODE>(P, st);
        else if (n <= 32) launch_walk<T, VEC, 16, 2, MODE>(P, st);
        else launch_walk<T, VEC, 16, kWide, MODE>(P, st);
    }
}

// The widest vector that divides the head size and every address.
template <int MODE>
void launch_mode(DiffParams &P, int dtype, uintptr_t addresses, cudaStream_t st) {
    const int b = dtype == AG_F32 ? 4 : 2;
    auto fits = [&](int vec) { return P.d % vec == 0 && addresses % uintptr_t(vec * b) == 0; };
    if (dtype == AG_F32) {
        if (fits(4)) launch_vec<float, 4, MODE>(P, st);
        else launch_vec<float, 1, MODE>(P, st);
    } else {
        if (fits(8)) launch_vec<bf16_t, 8, MODE>(P, st);
        else if (fits(4)) launch_vec<bf16_t, 4, MODE>(P, st);
        else launch_vec<bf16_t, 1, MODE>(P, st);
    }
}

template <int MODE>
void launch_fixup(const Direction &D, const DiffParams &P, int dtype, cudaStream_t st) {
    if (D.n_span == 0) return;
    FixParams F;
    F.spans = D.spans;
    F.n_long = D.n_span_long;
    F.n_span = D.n_span;
    F.partial = P.partial;
    F.slot = P.slot;
    F.lam = P.lam;
    F.lse = P.lse;
    F.lse_out = P.lse_out;
    F.stat = P.stat;
    F.out_a = P.out_a;
    F.out_b = P.out_b;
    F.H = P.H;
    F.heads = P.heads;
    F.d = P.d;
    F.scale = P.scale;
    F.drop_scale = P.drop.scale;
    const unsigned grid = unsigned(F.n_long + (F.n_span - F.n_long + kFixThreads / 32 - 1) / (kFixThreads / 32));
    if (dtype == AG_F32) k_diff_fixup<float, MODE><<<grid, kFixThreads, 0, st>>>(F);
    else k_diff_fixup<bf16_t, MODE><<<grid, kFixThreads, 0, st>>>(F);
}

void set_direction(DiffParams &P, const ag_graph *g, int dir) {
    const Direction &D = g->dir[dir];
    P.col = D.col;
    P.order = D.order;
    P.tile_nz = D.tile_nz;
    P.nz_rows = D.nz_rows;
    P.nz_rowptr = D.nz_rowptr;
    P.zero_rows = D.zero_rows;
    P.n_nz = D.n_nz;
    P.n_zero = g->N - D.n_nz;
    P.n_tiles = g->n_tiles;
    P.E = g->E;
    P.T = g->tile_edges;
}

int check_diff(const ag_graph *g, int64_t H, int64_t heads, int dtype, float scale, double p, const void *scratch,
               size_t scratch_bytes, const char *fn, DiffLayout *L) {
    if (!g) return fail(AG_ERR_INVALID_ARG, "%s: null graph", fn);
    if (!heads_fit(H, heads))
        return fail(AG_ERR_SHAPE, "%s: H = %lld is not 2 * heads * d with heads = %lld in [1, %d] and d in [1, %d]", fn,
                    (long long)H, (long long)heads, kMaxHeads, kMaxHeadDim);
    if (g->N * H >= (int64_t(1) << 40)) return fail(AG_ERR_SHAPE, "%s: N * H too large", fn);
    if (dtype != AG_F32 && dtype != AG_BF16) return fail(AG_ERR_DTYPE, "%s: unknown dtype %d", fn, dtype);
    if (!isfinite(scale)) return fail(AG_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    if (!(p >= 0.0 && p < 1.0)) return fail(AG_ERR_INVALID_ARG, "%s: p = %g outside [0, 1)", fn, p);
    if (int rc = check_current_device(g, fn)) return rc;
    *L = diff_layout(g, H, heads);
    if (!scratch || scratch_bytes < L->total)
        return fail(AG_ERR_WORKSPACE, "%s: scratch of %zu bytes, need %zu", fn, scratch_bytes, L->total);
    if (reinterpret_cast<uintptr_t>(scratch) % kAlign != 0)
        return fail(AG_ERR_WORKSPACE, "%s: scratch must be 256-byte aligned", fn);
    return check_device_ptr(scratch, g->device, "scratch");
}

struct Named {
    const void *p;
    const char *name;
};
template <int K>
int check_pointers(const Named (&a)[K], const ag_graph *g, int align, const char *fn) {
    for (const Named &x : a) {
        if (!x.p) return fail(AG_ERR_INVALID_ARG, "%s: null %s", fn, x.name);
        if (reinterpret_cast<uintptr_t>(x.p) % uintptr_t(align) != 0)
            return fail(AG_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", fn, x.name);
        if (int rc = check_device_ptr(x.p, g->device, x.name)) return rc;
    }
    return AG_OK;
}

DiffParams base_diff(const ag_graph *g, int64_t H, int64_t heads, const float *lam, float scale, const Drop &drop,
                     char *scr, const DiffLayout &L) {
    DiffParams P = {};
    P.lam = lam;
    P.partial = reinterpret_cast<float *>(scr + L.partial);
    P.slot = L.slot;
    P.stat = reinterpret_cast<float2 *>(scr + L.stat);
    P.H = int(H);
    P.heads = int(heads);
    P.d = int(H / (2 * heads));
    P.scale = scale;
    P.c2 = scale * kLog2e;
    P.drop = drop;
    return P;
}

}  // namespace
}  // namespace ag

using namespace ag;

extern "C" {

size_t ag_diff_attn_scratch_bytes(const ag_graph *g, int64_t H, int64_t heads) {
    if (!g || !heads_fit(H, heads)) return 0;
    return diff_layout(g, H, heads).total;
}

int ag_diff_attn_fwd(const ag_graph *g, const void *Q, const void *K, const void *V, const float *lam, float scale,
                     double p, uint64_t seed, uint64_t offset, void *Y, float *lse, int64_t H, int64_t heads, int dtype,
                     void *scratch, size_t scratch_bytes, void *stream) {
    const char *fn = "ag_diff_attn_fwd";
    clear_error();
    DiffLayout L;
    int rc = check_diff(g, H, heads, dtype, scale, p, scratch, scratch_bytes, fn, &L);
    if (rc != AG_OK) return rc;
    const int b = dtype == AG_F32 ? 4 : 2;
    const Named feats[] = {{Q, "Q"}, {K, "K"}, {V, "V"}, {Y, "Y"}}, floats[] = {{lam, "lambda"}, {lse, "lse"}};
    if ((rc = check_pointers(feats, g, b, fn)) != AG_OK) return rc;
    if ((rc = check_pointers(floats, g, 4, fn)) != AG_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DiffParams P = base_diff(g, H, heads, lam, scale, make_drop(p, seed, offset), static_cast<char *>(scratch), L);
    set_direction(P, g, 0);
    P.own_a = Q;
    P.nbr_a = K;
    P.nbr_b = V;
    P.out_a = Y;
    P.lse_out = lse;
    const uintptr_t at = uintptr_t(Q) | uintptr_t(K) | uintptr_t(V) | uintptr_t(Y);
    launch_mode<kFwd>(P, dtype, at, st);
    launch_fixup<kFwd>(g->dir[0], P, dtype, st);
    cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? AG_OK : cuda_fail(err, fn);
}

int ag_diff_attn_backward(const ag_graph *g, const void *Q, const void *K, const void *V, const float *lam, float scale,
                          double p, uint64_t seed, uint64_t offset, const float *lse, const void *dY, void *dQ, void *dK,
                          void *dV, float *dlam, int64_t H, int64_t heads, int dtype, void *scratch,
                          size_t scratch_bytes, void *stream) {
    const char *fn = "ag_diff_attn_backward";
    clear_error();
    DiffLayout L;
    int rc = check_diff(g, H, heads, dtype, scale, p, scratch, scratch_bytes, fn, &L);
    if (rc != AG_OK) return rc;
    const int b = dtype == AG_F32 ? 4 : 2;
    const Named feats[] = {{Q, "Q"}, {K, "K"}, {V, "V"}, {dY, "dY"}, {dQ, "dQ"}, {dK, "dK"}, {dV, "dV"}};
    const Named floats[] = {{lam, "lambda"}, {lse, "lse"}, {dlam, "dlambda"}};
    if ((rc = check_pointers(feats, g, b, fn)) != AG_OK) return rc;
    if ((rc = check_pointers(floats, g, 4, fn)) != AG_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    char *scr = static_cast<char *>(scratch);
    DiffParams P = base_diff(g, H, heads, lam, scale, make_drop(p, seed, offset), scr, L);
    // dQ and D over the destination rows
    set_direction(P, g, 0);
    P.own_a = Q;
    P.own_b = dY;
    P.nbr_a = K;
    P.nbr_b = V;
    P.lse = lse;
    P.out_a = dQ;
    const uintptr_t in = uintptr_t(Q) | uintptr_t(K) | uintptr_t(V) | uintptr_t(dY);
    launch_mode<kDQ>(P, dtype, in | uintptr_t(dQ), st);
    launch_fixup<kDQ>(g->dir[0], P, dtype, st);
    // dlambda from the rows' D
    double *part = reinterpret_cast<double *>(scr + L.dlam);
    const int64_t rows = (g->N + 255) / 256;
    const int blocks = int(rows < kLamBlocks ? rows : kLamBlocks);
    k_diff_dlam<<<blocks, 256, 0, st>>>(P.stat, g->N, int(heads), part);
    k_diff_dlam_join<<<1, 256, 0, st>>>(part, blocks, int(heads), dlam);
    // dK and dV over the source rows
    set_direction(P, g, 1);
    P.own_a = K;
    P.own_b = V;
    P.nbr_a = Q;
    P.nbr_b = dY;
    P.out_a = dK;
    P.out_b = dV;
    launch_mode<kDKV>(P, dtype, in | uintptr_t(dK) | uintptr_t(dV), st);
    launch_fixup<kDKV>(g->dir[1], P, dtype, st);
    cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? AG_OK : cuda_fail(err, fn);
}

}  // extern "C"
