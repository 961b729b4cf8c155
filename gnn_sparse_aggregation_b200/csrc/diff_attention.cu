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
//                    A = sum alpha da k, B = sum alpha k and D = sum alpha da:
//                    dq = scale (A - D B).  What A and D B have in common is of
//                    the size of sum alpha |da|, whose rounding D has in any form,
//                    so the difference costs no digits that ds = alpha (da - D)
//                    would keep.  (Sums about a reference c in place of 0 would,
//                    where c is the da of an edge of little weight.)  A row of one
//                    edge has dq = 0.  The alphas are divided by their own sum:
//                    the log-sum-exp is rounded, by up to 2.4e-7 between 4 and 8,
//                    one factor for the whole row;
//   kDKV             source rows of the transpose CSR; D known.
// No per-edge array is written or read besides the CSR itself.
//
// 2 DL lanes hold one head of one gathered row (DL lanes per map, NV vectors
// of VEC features per lane), and as many heads as fit share a lane group of a
// warp; each group walks a tile of T consecutive CSR positions of its own (the
// tile schedule of the other aggregations, joined where there are tiles to
// spare); heads beyond a warp's lanes take further blocks.  A lane's columns of
// K belong to its own map; its columns of V take the weights of both maps, the
// other one's by a shuffle.  A group takes several positions at a time while
// no group's row ends among them, and one position otherwise.  Gathered rows
// come through a ring in shared memory by cp.async, each lane reading only what
// it copied, so there is no barrier.  Rows cut by tile boundaries leave fp32
// partials that a fix-up kernel adds in tile order: results are bitwise
// reproducible.
//
// What bounds it where rows are even: warp instructions, then the L2's rate for
// gathered rows (15.1 TB/s for random 256-byte rows).  Every node of 64 edges,
// H = 128 bf16, 4 heads, 4.2 M edges (two rows, so 512 bytes, per edge):
// forward 185-194 us = 11 TB/s at 63 warp instructions per two edges, 248-256
// us with dropout (Philox, 23 more), dQ 218 us, dK and dV 274-282 us.  On
// R-MAT-18 (the same sizes, dropout) 364 / 394 / 430 us, and neither bound is
// reached: issue slots are busy 57 to 62 %, with 21 % of the warps active of
// the 25 % that 128 registers allow, so the warps wait on their own last
// results and on gathered rows; 15 % of the time the last tiles run alone, and
// a row's end costs about 120 instructions, the other lane groups of its warp
// masked.  Measured and not taken: a row split over the lane groups of a warp
// with sums across them at its end (660 us forward); tiles cut finer than the
// schedule's (a warp's first loads and its partials cost about 4 us: 1.41 ms in
// place of 1.19 for the step); 32 lanes of 8 bytes per row in place of 16 of 16
// (1.54 ms); four tiles per warp (2.2 ms); 96 registers and 20 warps per SM in
// place of 128 and 16 (1.24 ms).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <type_traits>

#include "aggraph.h"
#include "frag.cuh"
#include "internal.h"
#include "launch.cuh"
#include "operands.h"
#include "random.cuh"

namespace ag {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 2;            // warps per block
constexpr int kMinBlocks = 8;        // per SM: at most 128 registers a thread
constexpr int kResidentWarps = 148 * kMinBlocks * kWarps;
// Tiles of the schedule are joined while that leaves kMergeWarps warps (1.75
// times the resident ones: uneven tiles still fill in for one another).  564 K
// edges, 8 heads of 2 x 32, bf16: forward 238 -> 145 us, backward 522 -> 364;
// with one wave of warps in place of 1.75 R-MAT-18 takes 1.55 ms against 1.19.
constexpr int kMergeWarps = 4144, kMaxWalkTile = 1024;
// Owner rows per lane of a group that go to L2 ahead (16.8 M rows of one edge,
// H = 128 bf16: forward 4.86 ms, with all of a tile's 5.28).
constexpr int kRowsAhead = 2;
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
    int64_t n_zero, n_tiles;
    int64_t E;
    int n_nz;
    unsigned tile_blocks, zero_blocks;
    double *lam_partial;         // kDKV: sums of D_2 by block, [lam_blocks, heads]
    int lam_blocks;
    int64_t N;
    int T, H, heads, d, hb_log2;
    int groups;                  // lane groups of a warp that walk a tile
    int shift;                   // 2^shift tiles of the graph's schedule to one of the walk's
    int64_t graph_tiles;
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

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16) {
        cp_async16(dst, src);
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
    }
}

// dlambda[h] = -sum over rows of D_2, in fp64.  Blocks of the kDKV walk's
// launch add rows (a thread rows of one head, at a fixed stride, then the
// block its threads in a fixed tree), the last block of the kDKV fix-up's
// launch adds their sums: no launch of its own, and under the walk's work.
constexpr int kLamBlocks = 592;
constexpr int kLamRows = 16;      // per thread at least, before another block takes part

template <typename LOAD>
__device__ __forceinline__ double lam_sum(double *red, int threads, int heads, int64_t n, int64_t block, int64_t blocks,
                                          LOAD load) {
    // threads beyond a multiple of the heads idle; more heads than threads go round (the caller loops)
    const int per = threads / heads, g = threadIdx.x / heads, h = threadIdx.x % heads;
    double s = 0.0;
    if (g < per) {
#pragma unroll 4
        for (int64_t r = block * per + g; r < n; r += blocks * per) s += load(r, h);
    }
    red[threadIdx.x] = s;
    __syncthreads();
    for (int k = per; k > 1;) {
        const int half = (k + 1) / 2;
        if (g < k - half) red[threadIdx.x] += red[threadIdx.x + half * heads];
        k = half;
        __syncthreads();
    }
    s = threadIdx.x < heads ? red[threadIdx.x] : 0.0;
    __syncthreads();
    return s;
}

// A running maximum is replaced only by a score beyond it by this much (in
// powers of two), so that a row of scores of one size rescales its sums hardly
// ever.  The sums hold up to 2^kSlack times the values: V times the row's edges
// has to stay 2^8 below the largest number, and sums of exp2(x - m) stay below
// 2^(8 + 31).  A slack of 40, which costs 32 more powers of two of V, measured
// the same (training steps on 20 blocks and two-hop within 0.1 %, on R-MAT-18
// within their spread of 1.5 %).
constexpr float kSlack = 8.f;

// Positions that a lane group takes at a time while no row ends among them.
// Two such units are in flight: 8 KB of shared memory a warp.
constexpr int unit_positions(int nv) { return nv == 1 ? 4 : (nv == 2 ? 2 : 1); }

template <typename T, int VEC, int DL, int NV, int MODE, bool DROP>
__global__ void __launch_bounds__(kWarps * 32, NV <= 2 ? kMinBlocks : 1) k_diff_walk(const DiffParams P) {
    using F = Frag<T, VEC>;
    using raw = typename F::raw;
    constexpr int PIECE = F::kBytes;
    constexpr bool RING = PIECE >= 4;            // cp.async moves 4 bytes at least: else loads where they are used
    constexpr int U = unit_positions(NV);
    constexpr int HL = 2 * DL;
    constexpr int kRowBytes = NV * 32 * PIECE;   // a warp's pieces of one gathered row each
    constexpr int kPosBytes = 2 * kRowBytes;
    constexpr int kRing = RING ? 2 * U * kPosBytes : 16;
    constexpr int kStatRing = RING && MODE == kDKV ? 2 * U * 32 * 8 : 0;
    __shared__ __align__(16) unsigned char ring_mem[kWarps][kRing + kStatRing];
    follow_on();
    const int lane = threadIdx.x & 31;
    const int head_slots = 1 << P.hb_log2;
    const int group_lanes = HL << P.hb_log2;     // lanes that walk one tile
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

    auto load_row = [&](const void *base, int64_t row, raw (&r)[NV]) {
        const T *p = static_cast<const T *>(base) + row * P.H + col0;
#pragma unroll
        for (int k = 0; k < NV; ++k) r[k] = ok[k] ? F::load(p + k * DL * VEC) : F::zero();
    };
    const int stat_col = (live ? head : 0) * 2 + map;   // of [N, heads, 2]

    if (MODE == kDKV && blockIdx.x >= P.tile_blocks + P.zero_blocks) {
        if (blockIdx.y != 0) return;
        __shared__ double sums[kWarps * 32];
        const int block = int(blockIdx.x - P.tile_blocks - P.zero_blocks);
        for (int h0 = 0; h0 < P.heads; h0 += kWarps * 32) {  // as many heads as threads at a time
            const int heads = P.heads - h0 < kWarps * 32 ? P.heads - h0 : kWarps * 32;
            const double s = lam_sum(sums, kWarps * 32, heads, P.N, block, P.lam_blocks, [&](int64_t r, int h) {
                return double(P.stat[(r * P.heads + h0 + h) * 2 + 1].y);
            });
            if (threadIdx.x < heads) P.lam_partial[int64_t(block) * P.heads + h0 + threadIdx.x] = s;
        }
        return;
    }
    if (blockIdx.x >= P.tile_blocks) {  // rows without edges
        const int64_t z0 = (int64_t(blockIdx.x - P.tile_blocks) * kWarps + (threadIdx.x >> 5)) * kZeroPerWarp;
        for (int i = lane / group_lanes; i < kZeroPerWarp && z0 + i < P.n_zero; i += 32 / group_lanes) {
            const int64_t row = P.zero_rows[z0 + i];
            float z[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) z[v] = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (ok[k]) {
                    const int64_t at = row * P.H + col0 + k * DL * VEC;
                    F::store(static_cast<T *>(P.out_a) + at, z);
                    if (MODE == kDKV) F::store(static_cast<T *>(P.out_b) + at, z);
                }
            if (live && l == 0) {
                if (MODE == kFwd) P.lse_out[row * P.heads * 2 + stat_col] = -INFINITY;
                if (MODE == kDQ) P.stat[row * P.heads * 2 + stat_col] = make_float2(0.f, 0.f);
            }
        }
        return;
    }
    // a tile per lane group; groups behind the last tile walk none (len 0)
    // (the last tiles first: nodes of few edges, whose tiles hold many rows and
    // take longest, tend to have the high ids)
    const int64_t t0 = (int64_t(P.tile_blocks - 1 - blockIdx.x) * kWarps + (threadIdx.x >> 5)) * P.groups;
    if (t0 >= P.n_tiles) return;  // whole warps
    const int64_t t = t0 + lane / group_lanes;
    const bool tile = t < P.n_tiles && lane / group_lanes < P.groups;
#pragma unroll
    for (int k = 0; k < NV; ++k) ok[k] = ok[k] && tile;
    const int64_t p0 = tile ? t * P.T : 0;
    const int len = tile ? int(P.E - p0 < P.T ? P.E - p0 : P.T) : 0;
    const int steps = int(P.E - t0 * P.T < P.T ? P.E - t0 * P.T : P.T);  // the first group's: the longest

    // Loads that wait on one another go out in three rounds: ids, first row and
    // masks' edges; gathered rows and rows' ends; owner rows.
    int r = tile ? P.tile_nz[t << P.shift] : 0;
    const int r_last = tile ? (t + 1 < P.n_tiles ? P.tile_nz[(t + 1) << P.shift] : P.n_nz - 1) : 0;  // the row at the tile's end
    const float lam = live ? P.lam[head] : 0.f;
    const float sign = map ? -lam : 1.f;
    const int gl = lane & (group_lanes - 1);
    const int group0 = lane & ~(group_lanes - 1);
    int edge = DROP && gl < len ? __ldg(P.order + p0 + gl) : 0;

    // ------------------------------------------------------------ the ring of gathered rows
    unsigned char *const ring = ring_mem[threadIdx.x >> 5];
    if (RING) {  // pieces that no copy fills stay 0
#pragma unroll
        for (int s = 0; s < 4 * U; ++s)
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (!ok[k]) *reinterpret_cast<raw *>(ring + (s * NV + k) * 32 * PIECE + lane * PIECE) = F::zero();
    }
    const int32_t *const col = P.col + p0;
    const int last_unit = len > 0 ? (len - 1) & ~(U - 1) : 0;
    // every group's tile is whole, with three units of positions behind it (groups
    // without a tile read the first one's ids and fetch nothing)
    const bool inner = __all_sync(kAll, p0 + P.T + 3 * U <= P.E);
    struct Ids {
        int id[U];
    };
    auto load_ids = [&](int p) {  // the gathered rows of positions p .. p + U - 1 (p a multiple of U)
        Ids q;
        const int32_t *at = col + (inner || p < last_unit ? p : last_unit);
        if constexpr (U == 4) {
            const int4 v = __ldg(reinterpret_cast<const int4 *>(at));
            q.id[0] = v.x, q.id[1] = v.y, q.id[2] = v.z, q.id[3] = v.w;
        } else if constexpr (U == 2) {
            const int2 v = __ldg(reinterpret_cast<const int2 *>(at));
            q.id[0] = v.x, q.id[1] = v.y;
        } else {
            q.id[0] = __ldg(at);
        }
        if (!inner) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (p + i >= len) q.id[i] = 0;
        }
        return q;
    };
    const char *const nbr_a = static_cast<const char *>(P.nbr_a) + size_t(col0) * sizeof(T);
    const char *const nbr_b = static_cast<const char *>(P.nbr_b) + size_t(col0) * sizeof(T);
    const float2 *const nbr_st = P.stat + stat_col;
    const uint32_t row_bytes = uint32_t(P.H) * uint32_t(sizeof(T));
    const uint32_t stat_row = 2 * uint32_t(P.heads);
    auto fetch = [&](uint32_t at, int id, int s) {  // into position s of the unit at `at`
        const char *a = nbr_a + uint64_t(uint32_t(id)) * row_bytes;
        const char *b = nbr_b + uint64_t(uint32_t(id)) * row_bytes;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (ok[k]) {
                copy_async<PIECE>(at + s * kPosBytes + k * 32 * PIECE, a + k * DL * PIECE);
                copy_async<PIECE>(at + s * kPosBytes + kRowBytes + k * 32 * PIECE, b + k * DL * PIECE);
            }
    };
    const uint32_t ring_at = smem_addr(ring) + lane * PIECE;
    const uint32_t stat_at = smem_addr(ring) + kRing + lane * 8;
    auto fetch_unit = [&](int parity, const Ids &q) {
#pragma unroll
        for (int s = 0; s < U; ++s) {
            fetch(ring_at + parity * U * kPosBytes, q.id[s], s);
            if (MODE == kDKV)
                copy_async<8>(stat_at + (parity * U + s) * 32 * 8, nbr_st + uint64_t(uint32_t(q.id[s])) * stat_row);
        }
        cp_async_commit();
    };
    auto read = [&](int parity, int s, const Ids &q, raw (&a)[NV], raw (&b)[NV], float2 &st) {
        if constexpr (RING) {
            const unsigned char *at = ring + lane * PIECE + (parity * U + s) * kPosBytes;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                a[k] = *reinterpret_cast<const raw *>(at + k * 32 * PIECE);
                b[k] = *reinterpret_cast<const raw *>(at + kRowBytes + k * 32 * PIECE);
            }
            if (MODE == kDKV) st = *reinterpret_cast<const float2 *>(ring + kRing + ((parity * U + s) * 32 + lane) * 8);
        } else {
            int id = q.id[0];
#pragma unroll
            for (int i = 1; i < U; ++i) id = s == i ? q.id[i] : id;
            const T *pa = reinterpret_cast<const T *>(nbr_a + uint64_t(uint32_t(id)) * row_bytes);
            const T *pb = reinterpret_cast<const T *>(nbr_b + uint64_t(uint32_t(id)) * row_bytes);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                a[k] = ok[k] ? F::load(pa + k * DL * VEC) : F::zero();
                b[k] = ok[k] ? F::load(pb + k * DL * VEC) : F::zero();
            }
            if (MODE == kDKV) st = nbr_st[uint64_t(uint32_t(id)) * stat_row];  // (an earlier launch's: no __ldg)
        }
    };

    Ids ids = load_ids(0);
    if (RING) {
        const Ids second = load_ids(U), third = load_ids(2 * U);
        fetch_unit(0, ids);
        fetch_unit(1, second);
        ids = third;
    }

    // the open row, the next one with its owner rows, and the id and end of the one after
    bool before = tile && P.nz_rowptr[r] < p0;
    int row = 0, row_end, row_begin = 0;
    int next_row = 0, next_end = 0x7fffffff, far_row = 0, far_end = 0x7fffffff;
    raw own_a[NV], own_b[NV], pre_a[NV], pre_b[NV];
    float own_lse = 0.f, pre_lse = 0.f;
    auto load_owner = [&](int id, raw (&a)[NV], raw (&b)[NV], float &lse) {
        load_row(P.own_a, id, a);
        if (MODE != kFwd) load_row(P.own_b, id, b);
        if (MODE == kDQ) lse = P.lse[int64_t(id) * P.heads * 2 + stat_col] * kLog2e;
    };
    auto meta = [&](int i, int &id, int &end) {  // row i of the rows with edges, if there is one
        if (i < P.n_nz) {
            id = __ldg(P.nz_rows + i);
            end = int(__ldg(P.nz_rowptr + i + 1) - p0);
        }
    };
    meta(r, row, row_end);
    if (!tile) row_end = 0x7fffffff;
    meta(r + 1, next_row, next_end);
    meta(r + 2, far_row, far_end);
    load_owner(row, own_a, own_b, own_lse);
    load_owner(next_row, pre_a, pre_b, pre_lse);
    if (tile) {
        // the owner rows of the tile's next rows into L2: where rows are short,
        // one opens every few positions
        const int n = r_last - r < kRowsAhead * group_lanes ? r_last - r : kRowsAhead * group_lanes;
        const int bytes = (P.heads - h0 < head_slots ? P.heads - h0 : head_slots) * 2 * P.d * int(sizeof(T));
        for (int i = 2 + gl; i <= n; i += group_lanes) {
            const int64_t at = (int64_t(P.nz_rows[r + i]) * P.H + int64_t(h0) * 2 * P.d) * int64_t(sizeof(T));
            for (int o = 0; o < bytes; o += 128) {
                prefetch_l2(static_cast<const char *>(P.own_a) + at + o);
                if (MODE != kFwd) prefetch_l2(static_cast<const char *>(P.own_b) + at + o);
            }
        }
    }

    // kFwd: sums of p v for the own and the other map; kDQ: A, B; kDKV: dk, dv
    Sums<VEC> acc[2][NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) acc[0][k].zero(), acc[1][k].zero();
    float m = 0.f;            // kFwd: the reference of exp2(x - m)
    float sum = 0.f;          // of exp2(x - m), or of alpha
    float dsum = 0.f;         // kDQ: sum of alpha da
    bool first = true;        // the next position opens a row

    // the open row's partial of this tile
    auto write_slot = [&](int64_t s) {
        if (!live) return;
        float *base = P.partial + s * P.slot;
        const int which = MODE == kFwd ? map : 0;  // kFwd: maps in order, whichever is the lane's own
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            float *p = base + (a ^ which) * P.H + col0;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (ok[k]) {
                    float v[VEC];
                    acc[a][k].get(v);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) p[k * DL * VEC + i] = v[i];
                }
        }
        if (MODE != kDKV && l == 0) {
            float *q = base + 2 * P.H + stat_col;
            q[0] = MODE == kFwd ? m : dsum;
            q[2 * P.heads] = sum;
        }
    };
    // writes the rows that end before position pos and opens the next ones (all lanes call it)
    auto end_rows = [&](bool ends, int pos) {
        float own_w = 0.f, other_w = 0.f;
        if (MODE == kFwd) {
            own_w = sign * __fdividef(P.drop.scale, sum);  // (sum below 2^39)
            other_w = __shfl_xor_sync(kAll, own_w, DL);
        }
        if (MODE == kDQ) other_w = __fdividef(1.f, sum);   // near 1: what the rounded log-sum-exp left
        if (!ends) return;
        if (before) {  // continued from the previous tile
            write_slot(2 * t);
            before = false;
        } else {
            const bool lone = pos - row_begin == 1;
            const float w = lone ? 0.f : sign * P.scale * other_w, D = dsum * other_w;  // kDQ
            const int64_t at = int64_t(row) * P.H + col0;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float u[VEC], v[VEC];
                acc[0][k].get(u);
                acc[1][k].get(v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    if (MODE == kFwd) u[i] = fmaf(u[i], own_w, v[i] * other_w);
                    if (MODE == kDQ) u[i] = w * fmaf(-D, v[i], u[i]);
                }
                if (ok[k]) {
                    F::store(static_cast<T *>(P.out_a) + at + k * DL * VEC, u);
                    if (MODE == kDKV) F::store(static_cast<T *>(P.out_b) + at + k * DL * VEC, v);
                }
            }
            if (live && l == 0) {
                const int64_t c = int64_t(row) * P.heads * 2 + stat_col;
                if (MODE == kFwd) P.lse_out[c] = (m + log2f(sum)) * kLn2;
                if (MODE == kDQ) P.stat[c] = make_float2(fmaf(sum - 1.f, kLog2e, own_lse), D);
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            own_a[k] = pre_a[k];
            if (MODE != kFwd) own_b[k] = pre_b[k];
            acc[0][k].zero();
            acc[1][k].zero();
        }
        own_lse = pre_lse;
        sum = dsum = 0.f;
        first = true;
        row = next_row;
        row_end = next_end;
        row_begin = pos;
        next_row = far_row;
        next_end = far_end;
        ++r;
        load_owner(next_row, pre_a, pre_b, pre_lse);
        meta(r + 2, far_row, far_end);
    };
    // n positions of the unit, from s on, none of which opens a row but the
    // first; in the group's range where valid (kFwd: scores of -inf outside, else factors of 0)
    auto take = [&](auto count, int parity, int s0, const Ids &q, uint32_t kept, bool valid) {
        constexpr int n = decltype(count)::value;
        raw a[n][NV], b[n][NV];
        float2 st[n];
        float x[n], da[n];
#pragma unroll
        for (int s = 0; s < n; ++s) {
            read(parity, s0 + s, q, a[s], b[s], st[s]);
            x[s] = da[s] = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) x[s] = F::dot(own_a[k], a[s][k], x[s]);
            x[s] = group_sum<DL>(x[s]);
            if (MODE != kFwd) {
#pragma unroll
                for (int k = 0; k < NV; ++k) da[s] = F::dot(own_b[k], b[s][k], da[s]);
                da[s] = group_sum<HL>(da[s]);
                if (DROP) da[s] = kept >> s & 1u ? da[s] * P.drop.scale : 0.f;
            }
        }
        if (MODE == kFwd) {
            float top = -INFINITY;
#pragma unroll
            for (int s = 0; s < n; ++s) {
                x[s] = valid ? x[s] * P.c2 : -INFINITY;
                top = fmaxf(top, x[s]);
            }
            if (first) m = fmaxf(x[0], -3.402823466e38f);  // never -inf: exp2(-inf - m) is 0
            const bool beyond = top > m + kSlack;
            if (__any_sync(kAll, beyond)) {
                top = beyond ? top : m;  // (the warp's other rows keep their bits)
                const float f = ex2(m - top);
                const float g = __shfl_xor_sync(kAll, f, DL);
                sum *= f;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    float u[VEC], v[VEC];
                    acc[0][k].get(u);
                    acc[1][k].get(v);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) u[i] *= f, v[i] *= g;
                    acc[0][k].set(u);
                    acc[1][k].set(v);
                }
                m = top;
            }
        }
        first = false;
#pragma unroll
        for (int s = 0; s < n; ++s) {
            float f0, f1;  // the factors of acc[0] and acc[1]
            if (MODE == kFwd) {
                f0 = ex2(x[s] - m);
                sum += f0;
                f1 = __shfl_xor_sync(kAll, f0, DL);
            } else if (MODE == kDQ) {
                f1 = ex2(fmaf(x[s], P.c2, -own_lse));
                f0 = f1 * da[s];
                if (!valid) f0 = f1 = 0.f;
                sum += f1;
                dsum += f0;
            } else {
                const float p = sign * ex2(fmaf(x[s], P.c2, -st[s].x));
                f1 = p + __shfl_xor_sync(kAll, p, DL);
                f0 = P.scale * p * (da[s] - st[s].y);
                if (!valid) f0 = f1 = 0.f;
                if (DROP) f1 = kept >> s & 1u ? f1 * P.drop.scale : 0.f;
            }
            const uint64_t ff0 = Sums<VEC>::pair(f0, f0), ff1 = Sums<VEC>::pair(f1, f1);
            // what is outside may hold infinities, and the V (kFwd) or dY (kDKV) of what is dropped
            const bool use = valid && (!DROP || (kept >> s & 1u));
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float va[VEC], vb[VEC];
                if (MODE != kFwd) F::unpack_if(a[s][k], valid, va);
                if (MODE != kDQ) F::unpack_if(b[s][k], use, vb);
                if (MODE == kFwd) acc[0][k].add(ff0, vb), acc[1][k].add(ff1, vb);
                if (MODE == kDQ) acc[0][k].add(ff0, va), acc[1][k].add(ff1, va);
                if (MODE == kDKV) acc[0][k].add(ff0, va), acc[1][k].add(ff1, vb);
            }
        }
    };

    // keep bits of this lane's head: of `batch` positions from mask_at on
    const int batch = group_lanes > U ? group_lanes : U;
    uint32_t bits = 0xffffffffu;
    int stop = row_end < len || !tile ? row_end : len;  // the end of what is taken without a look
    for (int pos = 0; pos < steps; pos += U) {
        const int parity = pos / U & 1;
        if (DROP && (pos & (batch - 1)) == 0) {  // a position per lane, then a word per head
            const int count = P.heads - h0 < head_slots ? P.heads - h0 : head_slots;
            bits = 0;
            for (int o = 0; o < batch; o += group_lanes) {
                const uint32_t k = keep_bits<true>(uint64_t(uint32_t(edge)) * uint32_t(P.heads) + uint32_t(h0), count, P.drop);
                for (int h = 0; h < head_slots; ++h) {
                    const uint32_t w = __ballot_sync(kAll, k >> h & 1u) >> group0;
                    if (h == hs) bits |= (group_lanes == 32 ? w : w & ((1u << group_lanes) - 1u)) << o;
                }
                const int ahead = pos + o + group_lanes + gl;
                edge = ahead < len ? __ldg(P.order + p0 + ahead) : 0;
            }
        }
        if (RING) cp_async_wait<1>();
        // the whole unit at once where no group's row ends inside it
        const bool whole = __all_sync(kAll, stop >= pos + U);
        if (whole) take(std::integral_constant<int, U>(), parity, 0, ids, bits, true);
        for (int s = whole ? U - 1 : 0; s < U; ++s) {
            if (!whole) take(std::integral_constant<int, 1>(), parity, s, ids, bits >> s, pos + s < len);
            const bool ends = pos + s + 1 == row_end;
            if (__any_sync(kAll, ends)) {
                end_rows(ends, pos + s + 1);
                stop = row_end < len || !tile ? row_end : len;
            }
        }
        if (DROP) bits >>= U;
        if (RING) {
            fetch_unit(parity, ids);
            ids = load_ids(pos + 3 * U);
        } else {
            ids = load_ids(pos + U);
        }
    }
    if (RING) cp_async_wait<0>();
    if (tile && row_begin < len) write_slot(before ? 2 * t : 2 * t + 1);  // the row open at the tile's end
}

// Rows cut by tile boundaries: the partials of slot 2 first + 1 and of the
// slots 2t of tiles first + 1 .. last, in one pass (statistics and columns
// together, as a softmax that runs over the slots).  Where the walk's tiles are
// the schedule's, the schedule lists the cut rows, those of many tiles first;
// where they are several of them, a row's lanes look at one tile boundary and
// take the row that it is the first to cut.  A row of many slots takes a whole
// block (one of the list's, or after the block's other rows): stripes of
// threads take every stripes-th slot, then the stripes are joined in order.
// Every other row takes the lanes of its columns, which take the slots in
// order.  All orders are fixed by the graph and the sizes.
constexpr int kFixThreads = 512;
constexpr int kLongCut = 10;

struct FixParams {
    const int4 *spans;           // the cut rows, or null: by boundary
    int64_t n_long, n_span;
    const int32_t *tile_nz, *nz_rows, *nz_rowptr;
    int64_t n_tiles;
    int T, shift;
    const float *partial;
    int64_t slot;
    const float *lam, *lse;
    float *lse_out;
    float2 *stat;
    void *out_a, *out_b;
    int H, heads, d, lanes_log2;
    float scale, drop_scale;
    const double *lam_partial;   // kDKV: the last block adds up dlambda
    float *dlam;
    int lam_blocks;
};

struct Span {  // one cut row's slots, 0 .. n - 1
    const float *first, *rest;
    int64_t step;
    int n;
    int row;
    // span k of the list, or the row that boundary k (the first position of
    // tile k) is the first to cut; n = 0 where there is none
    __device__ __forceinline__ Span(const FixParams &P, int64_t k) : first(nullptr), rest(nullptr), step(2 * P.slot), n(0), row(0) {
        int64_t from;
        if (P.spans) {
            if (k >= P.n_span) return;
            const int4 sp = P.spans[k];
            from = sp.y;
            n = sp.z - sp.y + 1;
            row = sp.x;
        } else {
            if (k < 1 || k >= P.n_tiles) return;
            const int r = P.tile_nz[k << P.shift];
            const int64_t start = P.nz_rowptr[r], end = P.nz_rowptr[r + 1];
            if (start >= k * P.T || start < (k - 1) * P.T) return;
            from = k - 1;
            n = int((end - 1) / P.T - from) + 1;
            row = P.nz_rows[r];
        }
        first = P.partial + (2 * from + 1) * P.slot;
        rest = P.partial + 2 * from * P.slot;
    }
    __device__ __forceinline__ const float *operator[](int i) const { return i == 0 ? first : rest + i * step; }
};

// A thread's sums over slots: CV columns of one map.  kFwd: s1, s2 the maps'
// (maximum, sum), a, b their weighted sums; kDQ: s1 = the sums of (alpha da,
// alpha), a = A, b = B; kDKV: a, b.
template <int MODE, int CV>
struct FixSums {
    float2 s1, s2;
    float a[CV], b[CV];

    __device__ __forceinline__ void start() {
        s1 = s2 = make_float2(MODE == kDQ ? 0.f : -3.402823466e38f, 0.f);
#pragma unroll
        for (int v = 0; v < CV; ++v) a[v] = b[v] = 0.f;
    }
    // the terms (t1, t2, u, w) of a slot or of another thread's sums
    __device__ __forceinline__ void add(float2 t1, float2 t2, const float (&u)[CV], const float (&w)[CV]) {
        if (MODE == kFwd) {
            const float m1 = fmaxf(s1.x, t1.x), m2 = fmaxf(s2.x, t2.x);
            const float f1 = ex2(s1.x - m1), g1 = ex2(t1.x - m1), f2 = ex2(s2.x - m2), g2 = ex2(t2.x - m2);
            s1 = make_float2(m1, fmaf(s1.y, f1, g1 * t1.y));
            s2 = make_float2(m2, fmaf(s2.y, f2, g2 * t2.y));
#pragma unroll
            for (int v = 0; v < CV; ++v) a[v] = fmaf(a[v], f1, g1 * u[v]), b[v] = fmaf(b[v], f2, g2 * w[v]);
        } else {
            if (MODE == kDQ) s1.x += t1.x, s1.y += t1.y;
#pragma unroll
            for (int v = 0; v < CV; ++v) a[v] += u[v], b[v] += w[v];
        }
    }
    // slots i0, i0 + step, ...; q: where the head's statistics lie in a slot
    __device__ __forceinline__ void add_slots(const FixParams &P, const Span &S, int i0, int step, int c, int q, int map) {
        const int h2 = 2 * P.heads;
#pragma unroll 4
        for (int i = i0; i < S.n; i += step) {
            const float *p = S[i];
            float u[CV], w[CV];
            using F = Frag<float, CV>;
            F::unpack(F::load_written(p + c), u);
            F::unpack(F::load_written(p + c + P.H), w);
            if (MODE == kFwd) add(make_float2(p[q], p[q + h2]), make_float2(p[q + 1], p[q + 1 + h2]), u, w);
            else if (MODE == kDQ) add(make_float2(p[q + map], p[q + map + h2]), s2, u, w);
            else add(s1, s2, u, w);
        }
    }
};

template <typename T, int MODE, int CV>
__device__ __forceinline__ void fix_store(const FixParams &P, int64_t row, int c, int head, int map,
                                          FixSums<MODE, CV> &s) {
    const float lam = P.lam[head];
    float f = 1.f, g = 0.f;
    if (MODE == kFwd) f = __fdividef(P.drop_scale, s.s1.y), g = -lam * __fdividef(P.drop_scale, s.s2.y);
    const float inv = MODE == kDQ ? __fdividef(1.f, s.s1.y) : 0.f;
    if (MODE == kDQ) f = (map ? -lam : 1.f) * P.scale * inv, g = -s.s1.x * inv * f;
    T *out = static_cast<T *>(P.out_a) + row * P.H + c;
    if (MODE != kDKV) {
#pragma unroll
        for (int v = 0; v < CV; ++v) s.a[v] = fmaf(f, s.a[v], g * s.b[v]);
    }
    Frag<T, CV>::store(out, s.a);
    if (MODE == kDKV) Frag<T, CV>::store(static_cast<T *>(P.out_b) + row * P.H + c, s.b);
    if (MODE != kDKV && c % P.d == 0) {  // the map's statistics, once
        const int64_t k = (row * P.heads + head) * 2 + map;
        const float2 m = MODE == kFwd && map ? s.s2 : s.s1;
        if (MODE == kFwd) P.lse_out[k] = (m.x + log2f(m.y)) * kLn2;
        if (MODE == kDQ) P.stat[k] = make_float2(fmaf(s.s1.y - 1.f, kLog2e, P.lse[k] * kLog2e), s.s1.x * inv);
    }
}

template <typename T, int MODE, int CV>
__global__ void __launch_bounds__(kFixThreads, 1024 / kFixThreads) k_diff_fixup(const FixParams P) {
    constexpr int kWords = 2 * CV + (MODE == kFwd ? 4 : (MODE == kDQ ? 2 : 0));
    __shared__ float red[kWords][kFixThreads];
    follow_on();
    if (MODE == kDKV && P.lam_blocks > 0 && blockIdx.x == gridDim.x - 1) {
        __shared__ double sums[kFixThreads];
        const double s = lam_sum(sums, kFixThreads, P.heads, P.lam_blocks, 0, 1,
                                 [&](int64_t b, int h) { return P.lam_partial[b * P.heads + h]; });
        if (threadIdx.x < P.heads) P.dlam[threadIdx.x] = float(-s);
        return;
    }
    __shared__ int64_t later[kFixThreads];
    __shared__ int n_later;
    const bool listed = P.spans != nullptr, whole = listed && blockIdx.x < P.n_long;
    if (threadIdx.x == 0) {
        n_later = whole ? 1 : 0;
        later[0] = blockIdx.x;
    }
    __syncthreads();
    const int q_at = 2 * P.H;  // a slot's statistics
    FixSums<MODE, CV> sum;
    if (!whole) {
        const int lanes = 1 << P.lanes_log2, tc = threadIdx.x & (lanes - 1);
        const int64_t block = listed ? blockIdx.x - P.n_long : blockIdx.x;
        const int64_t k = (listed ? P.n_long : 1) + ((block * kFixThreads + threadIdx.x) >> P.lanes_log2);
        const Span S(P, k);
        if (!listed && S.n > kLongCut) {
            if (tc == 0) later[atomicAdd(&n_later, 1)] = k;  // (in any order: each row by itself)
        } else if (S.n > 0) {
            for (int c = tc * CV; c < P.H; c += lanes * CV) {
                const int head = c / (2 * P.d), map = c / P.d & 1, q = q_at + 2 * head;
                sum.start();
                sum.add_slots(P, S, 0, 1, c, q, map);
                fix_store<T, MODE, CV>(P, S.row, c, head, map, sum);
            }
        }
    }
    __syncthreads();
    int cols = 1;
    while (cols * CV < P.H && cols < kFixThreads) cols <<= 1;
    const int stripes = kFixThreads / cols, stripe = threadIdx.x / cols, tc = threadIdx.x % cols;
    for (int j = 0; j < n_later; ++j) {
        const Span S(P, later[j]);
        for (int c0 = 0; c0 < P.H; c0 += cols * CV) {
            const int c = c0 + tc * CV;
            const int head = c / (2 * P.d), map = c / P.d & 1, q = q_at + 2 * head;
            if (c < P.H) {
                sum.start();
                sum.add_slots(P, S, stripe, stripes, c, q, map);
#pragma unroll
                for (int v = 0; v < CV; ++v) red[v][threadIdx.x] = sum.a[v], red[CV + v][threadIdx.x] = sum.b[v];
                if constexpr (MODE != kDKV) red[2 * CV][threadIdx.x] = sum.s1.x, red[2 * CV + 1][threadIdx.x] = sum.s1.y;
                if constexpr (MODE == kFwd) red[2 * CV + 2][threadIdx.x] = sum.s2.x, red[2 * CV + 3][threadIdx.x] = sum.s2.y;
            }
            __syncthreads();
            if (stripe == 0 && c < P.H) {
                for (int k = 1; k < stripes; ++k) {
                    const int i = k * cols + tc;
                    float u[CV], w[CV];
#pragma unroll
                    for (int v = 0; v < CV; ++v) u[v] = red[v][i], w[v] = red[CV + v][i];
                    float2 t1 = sum.s1, t2 = sum.s2;
                    if constexpr (MODE != kDKV) t1 = make_float2(red[2 * CV][i], red[2 * CV + 1][i]);
                    if constexpr (MODE == kFwd) t2 = make_float2(red[2 * CV + 2][i], red[2 * CV + 3][i]);
                    sum.add(t1, t2, u, w);
                }
                fix_store<T, MODE, CV>(P, S.row, c, head, map, sum);
            }
            __syncthreads();
        }
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
    L.slot = (2 * H + 4 * heads + 3) / 4 * 4;
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
    // as many tiles per warp as there are groups, but fewer while that leaves
    // warps idle: a warp takes its groups' row ends one after another
    P.groups = 32 / (2 * DL << hb);
    P.shift = 0;
    while ((P.T << P.shift) < kMaxWalkTile && (P.graph_tiles >> (P.shift + 1)) / P.groups >= kMergeWarps) ++P.shift;
    P.T <<= P.shift;
    P.n_tiles = (P.graph_tiles + (int64_t(1) << P.shift) - 1) >> P.shift;
    while (P.groups > 1 && (P.n_tiles + P.groups - 1) / P.groups < kResidentWarps) P.groups >>= 1;
    const int tiles = kWarps * P.groups;  // per block
    P.tile_blocks = unsigned((P.n_tiles + tiles - 1) / tiles);
    const int64_t zero = (P.n_zero + kWarps * kZeroPerWarp - 1) / (kWarps * kZeroPerWarp);
    const unsigned y = unsigned((P.heads + (1 << hb) - 1) >> hb);
    P.zero_blocks = unsigned(zero);
    const dim3 grid(P.tile_blocks + P.zero_blocks + (MODE == kDKV ? P.lam_blocks : 0), y);
    if (grid.x == 0) return;
    if (P.drop.on) launch(k_diff_walk<T, VEC, DL, NV, MODE, true>, grid, kWarps * 32, MODE == kDKV, P, st);
    else launch(k_diff_walk<T, VEC, DL, NV, MODE, false>, grid, kWarps * 32, MODE == kDKV, P, st);
}

// Lanes and vectors per lane of a map's n = d / VEC vectors.  From eight
// vectors of four features (sixteen of eight) on, two vectors a lane halve the
// lanes of a score's sum: 564 K edges, fp32, 4 heads of 2 x 64: backward 992
// -> 624 us, of 2 x 32: 419 -> 345 us.  Below, they only put more tiles, and
// their row ends, into a warp: R-MAT-18, bf16, 4 heads of 2 x 16: forward 0.37
// -> 0.75 ms, so one vector stays there.  Four vectors a lane (2 x 64, fp32)
// measured 690 us against 624.
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
        else if (n <= 8) launch_walk<T, VEC, VEC == 4 ? 4 : 8, VEC == 4 ? 2 : 1, MODE>(P, st);
        else if (n <= 16) launch_walk<T, VEC, 8, 2, MODE>(P, st);
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
void launch_fixup(const Direction &D, const DiffParams &P, int dtype, float *dlam, cudaStream_t st) {
    const bool cuts = P.n_tiles > 1 && D.n_span > 0;
    if (!cuts && MODE != kDKV) return;
    FixParams F = {};
    F.spans = P.shift == 0 ? D.spans : nullptr;
    F.n_long = D.n_span_long;
    F.n_span = D.n_span;
    F.tile_nz = D.tile_nz;
    F.nz_rows = D.nz_rows;
    F.nz_rowptr = D.nz_rowptr;
    F.n_tiles = P.n_tiles;
    F.T = P.T;
    F.shift = P.shift;
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
    F.lam_partial = P.lam_partial;
    F.lam_blocks = MODE == kDKV ? P.lam_blocks : 0;
    F.dlam = dlam;
    // four columns a thread where maps and rows divide so (slots are 16-byte aligned) and the outputs' addresses do
    const bool four = P.d % 4 == 0 && (uintptr_t(P.out_a) | uintptr_t(P.out_b)) % (dtype == AG_F32 ? 16 : 8) == 0;
    F.lanes_log2 = 0;
    while (F.lanes_log2 < 5 && (four ? 4 : 1) << F.lanes_log2 < F.H) ++F.lanes_log2;
    const int rows = kFixThreads >> F.lanes_log2;
    const int64_t shorts = P.shift == 0 ? F.n_span - F.n_long : F.n_tiles - 1;
    const unsigned grid = unsigned(cuts ? (P.shift == 0 ? F.n_long : 0) + (shorts + rows - 1) / rows : 0) + (MODE == kDKV ? 1 : 0);
    if (dtype == AG_F32) {
        if (four) launch(k_diff_fixup<float, MODE, 4>, dim3(grid), kFixThreads, true, F, st);
        else launch(k_diff_fixup<float, MODE, 1>, dim3(grid), kFixThreads, true, F, st);
    } else {
        if (four) launch(k_diff_fixup<bf16_t, MODE, 4>, dim3(grid), kFixThreads, true, F, st);
        else launch(k_diff_fixup<bf16_t, MODE, 1>, dim3(grid), kFixThreads, true, F, st);
    }
}

void set_direction(DiffParams &P, const ag_graph *g, int dir) {
    const Direction &D = g->dir[dir];
    P.col = D.col;
    P.order = D.order;
    P.tile_nz = D.tile_nz;
    P.nz_rows = D.nz_rows;
    P.nz_rowptr = D.nz_rowptr;
    P.zero_rows = D.zero_rows;
    P.n_nz = int(D.n_nz);
    P.n_zero = g->N - D.n_nz;
    P.n_tiles = P.graph_tiles = g->n_tiles;
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
    const size_t f = size_t(g->N) * size_t(H) * size_t(b), h = size_t(heads) * 4, s = size_t(g->N) * h * 2;
    const Operand ops[] = {{Q, "Q", f, b, kIn}, {K, "K", f, b, kIn}, {V, "V", f, b, kIn}, {lam, "lambda", h, 4, kIn},
                           {Y, "Y", f, b, kOut}, {lse, "lse", s, 4, kOut}, {scratch, "scratch", L.total, 1, kOut}};
    if ((rc = check_operands(ops, g->device, false, fn)) != AG_OK) return rc;
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
    launch_fixup<kFwd>(g->dir[0], P, dtype, nullptr, st);
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
    const size_t f = size_t(g->N) * size_t(H) * size_t(b), h = size_t(heads) * 4, s = size_t(g->N) * h * 2;
    const Operand ops[] = {{Q, "Q", f, b, kIn}, {K, "K", f, b, kIn}, {V, "V", f, b, kIn}, {dY, "dY", f, b, kIn},
                           {lam, "lambda", h, 4, kIn}, {lse, "lse", s, 4, kIn}, {dQ, "dQ", f, b, kOut},
                           {dK, "dK", f, b, kOut}, {dV, "dV", f, b, kOut}, {dlam, "dlambda", h, 4, kOut},
                           {scratch, "scratch", L.total, 1, kOut}};
    if ((rc = check_operands(ops, g->device, false, fn)) != AG_OK) return rc;
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
    launch_fixup<kDQ>(g->dir[0], P, dtype, nullptr, st);
    // dK and dV over the source rows, and dlambda from the rows' D
    P.N = g->N;
    P.lam_partial = reinterpret_cast<double *>(scr + L.dlam);
    const int64_t per = kLamRows * (heads < kWarps * 32 ? kWarps * 32 / heads : 1);
    const int64_t want = (g->N + per - 1) / per;
    P.lam_blocks = int(want < kLamBlocks ? want : kLamBlocks);
    set_direction(P, g, 1);
    P.own_a = K;
    P.own_b = V;
    P.nbr_a = Q;
    P.nbr_b = dY;
    P.out_a = dK;
    P.out_b = dV;
    launch_mode<kDKV>(P, dtype, in | uintptr_t(dK) | uintptr_t(dV), st);
    launch_fixup<kDKV>(g->dir[1], P, dtype, dlam, st);
    cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? AG_OK : cuda_fail(err, fn);
}

}  // extern "C"
