// mm_kernel.cuh -- the matrix products over packed rows (8-bit block-scaled,
// grouped by expert, and the Gram factor per expert) on the 5th-generation
// tensor cores (tcgen05, sm_100a): one persistent kernel template, specialised
// by a policy P.
//
// Every product is a set of output tiles D = A B^T, D of BM = 128 rows (TMEM
// lanes) by BN columns, each accumulated over a contraction range:
//   kTokensB  D[i, t] = sum_k W_e[i, k] X[t, k]: the weight's rows are the lanes
//             and the packed rows the columns, so a ragged group costs MMA time
//             for its own length (the instruction's N is the group tile's length
//             rounded up to 16), not for whole tiles;
//   kTokensA  D[t, j] = sum_k X[t, k] W_e[j, k]: packed rows are the lanes, so a
//             row's 8-bit step is one register of the thread that owns the lane;
//   kContract D_e[i, j] = sum_{t in group e} P[t, i] Q[t, j]: the packed rows are
//             the contraction and both operands are read column-major (the
//             instruction's transpose bits), straight from the packed rows.
// Tiles are numbered group by group; every CTA derives the numbering from the
// group offsets in device memory (no host round trip) and takes tiles
// blockIdx.x, blockIdx.x + gridDim.x, ...
//
// Warp roles: warp 0 lane 0 issues TMA into a ring of kStages stages; warp 1
// owns TMEM and issues the MMAs; the other warps read finished accumulator
// chunks (kChunk stages each, double buffered in TMEM) and add them in FP32
// registers, scaled by the 8-bit operands' steps where there are any.  The
// tensor cores' accumulator truncates, so sums are kept to kChunk stages there.
// Every mbarrier wait is bounded; on expiry the CTA records
// BAKRON_ERR_DEVICE_TIMEOUT, drains what it issued, frees its tensor memory and
// exits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "mm.cuh"
#include "tcgen05.cuh"

namespace bakron {
namespace mm {

using namespace tc;

constexpr int kBM = 128;
constexpr int kReserve = 9 * 1024;  // barriers, tile numbering, alignment, staged steps

template <class P>
struct Shape {
    // one operand row of a stage is 128 bytes (the swizzle width)
    static constexpr int kElems = P::kEight ? 128 : 64;             // operand elements in 128 bytes
    static constexpr int kKB = P::kRagged == kContract ? P::kKRows : kElems;  // contraction per stage
    static constexpr int kABytes = P::kRagged == kContract ? kBM / 64 * kKB * 128 : kBM * 128;
    static constexpr int kBBytes = P::kRagged == kContract ? P::kBN / 64 * kKB * 128 : P::kBN * 128;
    static constexpr int kStageBytes = P::kPlanes * (kABytes + kBBytes);
    static constexpr int kStages = (227 * 1024 - kReserve) / kStageBytes < 8 ? (227 * 1024 - kReserve) / kStageBytes : 8;
    static constexpr int kAcc = P::kPlanes > 1 ? 2 : 1;             // accumulators per buffer
    static constexpr int kTmemCols = 2 * kAcc * P::kBN;
    static constexpr int kEpiWarps = 8;
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    static constexpr int kCols = P::kBN / (kEpiWarps / 4);          // columns per epilogue thread
    static constexpr size_t kSmem = (size_t)kStages * kStageBytes + kReserve;
};

// One output tile: group e, D rows a0.. (na valid), D columns b0.. (nb valid),
// contraction over [k0, k1).
struct Tile {
    int e, a0, na, b0, nb, k0, k1, count;
};

// Group e's packed rows [lo, hi), empty if the offsets are not a valid range.
__device__ __forceinline__ bool group_range(const Args &g, int e, int &lo, int &hi)
{
    if (!g.offsets) {
        lo = 0;
        hi = g.rows;
        return true;
    }
    lo = __ldg(g.offsets + e);
    hi = __ldg(g.offsets + e + 1);
    if (lo >= 0 && lo <= hi && hi <= g.rows) return true;
    lo = hi = 0;
    return false;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Lower-triangle tiles of a square of `rows` 128-row tiles by BN columns.
template <int BN>
__host__ __device__ __forceinline__ int lower_tiles_of_row(int i)
{
    return (i * kBM + kBM - 1) / BN + 1;
}

template <class P>
__device__ __forceinline__ int tiles_of_group(const Args &g, int len)
{
    if (P::kRagged == kTokensB) return ceil_div(g.a_total, kBM) * ceil_div(len, P::kBN);
    if (P::kRagged == kTokensA) return ceil_div(len, kBM) * ceil_div(g.b_total, P::kBN);
    if (P::kLower) {
        int n = 0;
        for (int i = 0; i < ceil_div(g.a_total, kBM); ++i) n += lower_tiles_of_row<P::kBN>(i);
        return n;
    }
    return ceil_div(g.a_total, kBM) * ceil_div(g.b_total, P::kBN);
}

template <class P>
__device__ __forceinline__ Tile find_tile(const Args &g, const int *first, int t)
{
    int a = 0, b = g.experts;  // the last group whose first tile is <= t
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (first[m] <= t) a = m;
        else b = m;
    }
    Tile x;
    x.e = a;
    int lo, hi;
    group_range(g, a, lo, hi);
    int i = t - first[a];
    x.count = hi - lo;
    if (P::kRagged == kTokensB) {
        const int mt = ceil_div(g.a_total, kBM);
        x.a0 = (i % mt) * kBM;
        x.b0 = lo + (i / mt) * P::kBN;
        x.na = min(kBM, g.a_total - x.a0);
        x.nb = min(P::kBN, hi - x.b0);
        x.k0 = 0;
        x.k1 = g.k_total;
    } else if (P::kRagged == kTokensA) {
        const int mt = ceil_div(hi - lo, kBM);
        x.a0 = lo + (i % mt) * kBM;
        x.b0 = (i / mt) * P::kBN;
        x.na = min(kBM, hi - x.a0);
        x.nb = min(P::kBN, g.b_total - x.b0);
        x.k0 = 0;
        x.k1 = g.k_total;
    } else {
        int r, c;
        if (P::kLower) {
            for (r = 0; i >= lower_tiles_of_row<P::kBN>(r); ++r) i -= lower_tiles_of_row<P::kBN>(r);
            c = i;
        } else {
            const int nt = ceil_div(g.b_total, P::kBN);
            r = i / nt;
            c = i % nt;
        }
        x.a0 = r * kBM;
        x.b0 = c * P::kBN;
        x.na = min(kBM, g.a_total - x.a0);
        x.nb = min(P::kBN, g.b_total - x.b0);
        x.k0 = lo;
        x.k1 = hi;
    }
    return x;
}

template <typename T>
__device__ __forceinline__ T round_to(float v);
template <>
__device__ __forceinline__ float round_to<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half round_to<__half>(float v) { return __float2half_rn(v); }

// Store this thread's accumulators: D row `lane_row` of the tile, columns
// [col0, col0 + C).
template <class P, typename T, int C>
__device__ __forceinline__ void store_tile(const Args &g, const Tile &x, int lane_row, int col0, const float (&acc)[C])
{
    T *out = (T *)g.out;
    if (P::kRagged == kTokensB) {
        // D row = output column: the 32 lanes of a warp write consecutive
        // elements of one packed row
        if (lane_row >= x.na) return;
        T *p = out + (int64_t)(x.b0 + col0) * g.ldo + x.a0 + lane_row;
        float s = 1.f;
        if (P::kEight && g.w_step_rows == 1) s = __ldg(g.w_steps + (int64_t)x.e * g.a_total + x.a0 + lane_row);
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (col0 + c < x.nb) p[(int64_t)c * g.ldo] = round_to<T>(P::kEight ? acc[c] * s : acc[c]);
    } else {
        if (lane_row >= x.na) return;
        T *p = out + (P::kRagged == kContract ? (int64_t)x.e * g.out_expert_stride : 0) +
               (int64_t)(x.a0 + lane_row) * g.ldo + x.b0 + col0;
        const int n = min(C, x.nb - col0);
        const bool per_row = P::kEight && g.w_step_rows == 1;
        const float *s = per_row ? g.w_steps + (int64_t)x.e * g.b_total + x.b0 + col0 : nullptr;
        constexpr int kVec = 16 / sizeof(T);
        if (n == C && ((uintptr_t)p & 15) == 0) {
#pragma unroll
            for (int c = 0; c < C; c += kVec) {
                __align__(16) T v[kVec];
#pragma unroll
                for (int u = 0; u < kVec; ++u) v[u] = round_to<T>(per_row ? acc[c + u] * __ldg(s + c + u) : acc[c + u]);
                *(uint4 *)(p + c) = *(const uint4 *)v;
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (c < n) p[c] = round_to<T>(per_row ? acc[c] * __ldg(s + c) : acc[c]);
        }
    }
}

// Gram tile: entries on and below the diagonal, divided by the group's count,
// and their mirror images.
template <int C>
__device__ __forceinline__ void store_gram(const Args &g, const Tile &x, int lane_row, int col0, const float (&acc)[C])
{
    if (lane_row >= x.na) return;
    const int64_t d = g.ldo;
    float *out = (float *)g.out + (int64_t)x.e * g.out_expert_stride;
    const int i = x.a0 + lane_row;
    const float count = (float)max(x.count, 1);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int j = x.b0 + col0 + c;
        if (col0 + c < x.nb && j <= i) {
            const float v = __fdiv_rn(acc[c], count);
            out[i * d + j] = v;
            out[j * d + i] = v;
        }
    }
}

template <class P>
__global__ void __launch_bounds__(Shape<P>::kThreads, 1)
mm_kernel(const __grid_constant__ Maps maps, const Args g)
{
    using S = Shape<P>;
    constexpr int BN = P::kBN;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t *bars = (uint64_t *)(smem + S::kStages * S::kStageBytes);
    int *first = (int *)(bars + 32);                        // tile numbering: kMaxExperts + 1
    float *steps_sh = (float *)(first + kMaxExperts + 4);   // staged row steps (kTokensB, 8-bit)
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S::kStages + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (2 * S::kStages + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (2 * S::kStages + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * S::kStages + 4);

    if (threadIdx.x == 0) {
        prefetch_map(&maps.a);
        prefetch_map(&maps.b);
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 1);
            mbar_init(acce_bar(b), S::kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        abort_sh = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_base_sh)),
                     "r"(S::kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (warp == 2) {
        // tile numbering: exclusive prefix sum of the groups' tile counts
        int base = 0;
        const int fixed = P::kRagged == kContract ? tiles_of_group<P>(g, 0) : 0;
        for (int e0 = 0; e0 < g.experts; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            if (e < g.experts) {
                int lo, hi;
                if (!group_range(g, e, lo, hi) && blockIdx.x == 0) record_error(g.st, BAKRON_ERR_INVALID_ARG, e);
                n = P::kRagged == kContract ? fixed : tiles_of_group<P>(g, hi - lo);
            }
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (e < g.experts) first[e] = base + inc - n;
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) first[g.experts] = base;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_sh;
    const int total = first[g.experts];
    volatile int *abort_flag = &abort_sh;

    // Bounded wait: false once it has run for the time limit or another role
    // has given up.
    auto wait = [&](uint32_t bar, uint32_t parity, int where) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = now_ns();
        for (;;) {
            for (int i = 0; i < 16; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) return false;
            if (now_ns() - t0 > g.timeout_ns) {
                record_error(g.st, BAKRON_ERR_DEVICE_TIMEOUT, where);
                atomicExch(&abort_sh, 1);
                return false;
            }
        }
    };

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer
            int it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const Tile x = find_tile<P>(g, first, t);
                const int nkb = ceil_div(x.k1 - x.k0, S::kKB);
                const int boxes = P::kRagged == kTokensB ? ceil_div(x.nb, P::kBoxRows) : 1;
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const int s = it % S::kStages;
                    if (it >= S::kStages && !wait(empty_bar(s), (it / S::kStages - 1) & 1, 1000)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a = smem_u32(smem + s * S::kStageBytes), b = a + P::kPlanes * S::kABytes;
                    const int k = x.k0 + kb * S::kKB;
                    if (P::kRagged == kTokensB) {
                        mbar_expect_tx(full_bar(s), S::kABytes + boxes * P::kBoxRows * 128);
                        if (P::kAColumns) {
                            tma_load_3d(a, &maps.a, x.a0, k, x.e, full_bar(s));
                            tma_load_3d(a + S::kABytes / 2, &maps.a, x.a0 + 64, k, x.e, full_bar(s));
                        } else {
                            tma_load_3d(a, &maps.a, k, x.a0, x.e, full_bar(s));
                        }
                        for (int r = 0; r < boxes; ++r)
                            tma_load_2d(b + r * P::kBoxRows * 128, &maps.b, k, x.b0 + r * P::kBoxRows, full_bar(s));
                    } else if (P::kRagged == kTokensA) {
                        mbar_expect_tx(full_bar(s), S::kStageBytes);
                        tma_load_2d(a, &maps.a, k, x.a0, full_bar(s));
                        tma_load_3d(b, &maps.b, k, x.b0, x.e, full_bar(s));
                    } else {
                        mbar_expect_tx(full_bar(s), S::kStageBytes);
#pragma unroll
                        for (int p = 0; p < P::kPlanes; ++p) {
#pragma unroll
                            for (int c = 0; c < kBM / 64; ++c)
                                tma_load_3d(a + p * S::kABytes + c * S::kKB * 128, &maps.a, x.a0 + 64 * c, k, p,
                                            full_bar(s));
#pragma unroll
                            for (int c = 0; c < BN / 64; ++c)
                                tma_load_3d(b + p * S::kBBytes + c * S::kKB * 128, &maps.b, x.b0 + 64 * c, k, p,
                                            full_bar(s));
                        }
                    }
                }
            }
            // every issued copy has to land before the CTA may exit
            for (int i = max(0, it - S::kStages); i < it; ++i) {
                const uint64_t t0 = now_ns();
                while (!mbar_try_wait(full_bar(i % S::kStages), (i / S::kStages) & 1) &&
                       now_ns() - t0 < g.timeout_ns + 50000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer (the whole warp walks the loop; lane 0 issues)
        int it = 0, chunk = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Tile x = find_tile<P>(g, first, t);
            const int nkb = ceil_div(x.k1 - x.k0, S::kKB);
            const int n_mma = P::kRagged == kTokensB ? (x.nb + 15) & ~15 : BN;
            const uint32_t idesc = g.idesc | ((uint32_t)(n_mma >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
            for (int kb = 0; kb < nkb; ++kb, ++it) {
                const int buf = chunk & 1, in_chunk = kb % P::kChunk;
                if (in_chunk == 0 && chunk >= 2) ok = wait(acce_bar(buf), ((chunk >> 1) - 1) & 1, 2000);
                const int s = it % S::kStages;
                ok = ok && wait(full_bar(s), (it / S::kStages) & 1, 2001);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint8_t *stage = smem + s * S::kStageBytes;
                const uint32_t a = smem_u32(stage), b = a + P::kPlanes * S::kABytes;
                constexpr int kSteps = S::kKB / (P::kEight ? 32 : 16);
                int steps = kSteps;
                if (P::kRagged == kContract) {
                    // The group may end inside this stage: its last step's
                    // missing rows (the next group's, or whatever lies behind
                    // the last one) are zeroed in both operands, NaN and all.
                    const int valid = min(S::kKB, x.k1 - (x.k0 + kb * S::kKB));
                    steps = (valid + 15) >> 4;
                    if (valid & 15) {
                        constexpr int kAtoms = P::kPlanes * (kBM + BN) / 64;
                        const int rows = 16 * steps - valid;
                        for (int i = lane; i < kAtoms * rows * 8; i += 32) {
                            const int atom = i / (rows * 8), w = i % (rows * 8);
                            *(uint4 *)(stage + atom * S::kKB * 128 + (valid + (w >> 3)) * 128 + (w & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t d = tmem_base + (uint32_t)(buf * S::kAcc * BN);
                    for (int ks = 0; ks < steps; ++ks) {
                        const uint32_t fresh = (in_chunk | ks) != 0;
                        if (P::kPlanes > 1) {
                            // x = h + m + l in three bf16 parts: hh into one
                            // accumulator, the five smaller products into another
                            const uint32_t off = ks * 2048;
                            uint64_t ad[3], bd[3];
#pragma unroll
                            for (int p = 0; p < 3; ++p) {
                                ad[p] = umma_desc_mn(a + p * S::kABytes + off, S::kKB * 128);
                                bd[p] = umma_desc_mn(b + p * S::kBBytes + off, S::kKB * 128);
                            }
                            umma_f16(d, ad[0], bd[0], idesc, fresh);
                            umma_f16(d + BN, ad[0], bd[2], idesc, fresh);
                            umma_f16(d + BN, ad[2], bd[0], idesc, 1);
                            umma_f16(d + BN, ad[1], bd[1], idesc, 1);
                            umma_f16(d + BN, ad[0], bd[1], idesc, 1);
                            umma_f16(d + BN, ad[1], bd[0], idesc, 1);
                        } else if (P::kRagged == kContract) {
                            umma_f16(d, umma_desc_mn(a + ks * 2048, S::kKB * 128),
                                     umma_desc_mn(b + ks * 2048, S::kKB * 128), idesc, fresh);
                        } else if (P::kEight) {
                            umma_f8(d, umma_desc(a + ks * 32), umma_desc(b + ks * 32), idesc, fresh);
                        } else {
                            umma_f16(d, P::kAColumns ? umma_desc_mn(a + ks * 2048, S::kKB * 128)
                                                     : umma_desc(a + ks * 32),
                                     umma_desc(b + ks * 32), idesc, fresh);
                        }
                    }
                    umma_commit(empty_bar(s));
                    if (in_chunk == P::kChunk - 1 || kb == nkb - 1) umma_commit(accf_bar(buf));
                }
                __syncwarp();
                if (in_chunk == P::kChunk - 1 || kb == nkb - 1) ++chunk;
            }
        }
        if (!ok) {
            // let issued MMAs finish before TMEM is released
            if (lane == 0) {
                umma_commit(drain_bar);
                const uint64_t t0 = now_ns();
                while (!mbar_try_wait(drain_bar, 0) && now_ns() - t0 < g.timeout_ns + 50000000ull) {
                }
            }
            __syncwarp();
        }
    } else {
        // ---------------- epilogue: chunks TMEM -> FP32 registers, then store
        const int quad = warp & 3;                   // TMEM lanes [32 quad, 32 quad + 32)
        const int half = (warp - 2) >> 2;            // columns [half kCols, half kCols + kCols)
        const int lane_row = quad * 32 + lane, col0 = half * S::kCols;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        float *steps_w = steps_sh + (warp - 2) * 2 * S::kCols;
        int chunk = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Tile x = find_tile<P>(g, first, t);
            const int nkb = ceil_div(x.k1 - x.k0, S::kKB);
            const int nchunk = ceil_div(nkb, P::kChunk);
            float acc[S::kCols];
#pragma unroll
            for (int i = 0; i < S::kCols; ++i) acc[i] = 0.f;
            // 8-bit operands: the steps of this thread's share of the tile
            const float *xs = nullptr, *ws = nullptr;
            bool own_row = false;
            if (P::kEight) {
                if (P::kRagged == kTokensA) {
                    own_row = lane_row < x.na;
                    xs = g.x_steps + (int64_t)(x.a0 + (own_row ? lane_row : 0)) * nkb;
                    if (g.w_step_rows != 1)
                        ws = g.w_steps + ((int64_t)x.e * ceil_div(g.b_total, 128) +
                                          min((x.b0 + col0) / 128, ceil_div(g.b_total, 128) - 1)) * nkb;
                } else if (g.w_step_rows != 1) {
                    ws = g.w_steps + ((int64_t)x.e * ceil_div(g.a_total, 128) + x.a0 / 128) * nkb;
                }
            }
            for (int c = 0; c < nchunk; ++c, ++chunk) {
                const int buf = chunk & 1;
                float row_step = 1.f;
                if (P::kEight && P::kRagged == kTokensA)
                    row_step = (own_row ? __ldg(xs + c) : 0.f) * (ws ? __ldg(ws + c) : 1.f);
                float *steps = steps_w + (c & 1) * S::kCols;
                if (P::kEight && P::kRagged == kTokensB) {
                    const float s = ws ? __ldg(ws + c) : 1.f;
                    for (int j = lane; j < S::kCols; j += 32)
                        steps[j] = col0 + j < x.nb ? __ldg(g.x_steps + (int64_t)(x.b0 + col0 + j) * nkb + c) * s : 0.f;
                    __syncwarp();
                }
                ok = __all_sync(0xffffffffu, wait(accf_bar(buf), (chunk >> 1) & 1, 3000));
                if (!ok) break;
                tc_fence_after();
                const uint32_t src = tmem_base + lane_off + (uint32_t)(buf * S::kAcc * BN + col0);
#pragma unroll
                for (int c0 = 0; c0 < S::kCols; c0 += 32) {
                    if (col0 + c0 < x.nb) {
                        float v[32];
                        tmem_ld32(src + c0, v);
                        if (P::kEight && P::kRagged == kTokensA) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) acc[c0 + i] = fmaf(v[i], row_step, acc[c0 + i]);
                        } else if (P::kEight) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) acc[c0 + i] = fmaf(v[i], steps[c0 + i], acc[c0 + i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) acc[c0 + i] += v[i];
                        }
                        if (P::kPlanes > 1) {
                            tmem_ld32(src + BN + c0, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) acc[c0 + i] += v[i];
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce_bar(buf));
            }
            if (!ok) break;
            if (P::kLower) store_gram<S::kCols>(g, x, lane_row, col0, acc);
            else if (g.out_type == BAKRON_BF16) store_tile<P, __nv_bfloat16, S::kCols>(g, x, lane_row, col0, acc);
            else if (g.out_type == BAKRON_F16) store_tile<P, __half, S::kCols>(g, x, lane_row, col0, acc);
            else store_tile<P, float, S::kCols>(g, x, lane_row, col0, acc);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(S::kTmemCols));
    }
}

template <class P>
cudaError_t configure()
{
    return cudaFuncSetAttribute(mm_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<P>::kSmem);
}

template <class P>
cudaError_t launch(const Maps &maps, const Args &g, int blocks, cudaStream_t stream)
{
    mm_kernel<P><<<blocks, Shape<P>::kThreads, Shape<P>::kSmem, stream>>>(maps, g);
    return cudaGetLastError();
}

}  // namespace mm
}  // namespace bakron
