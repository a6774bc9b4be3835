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
// With kPair two CTAs of a cluster share one MMA of 256 rows: each holds half
// of A's, B's and D's rows, so an operand byte brought into shared memory feeds
// twice the multiply-adds; the pair's first CTA issues the MMAs, and both CTAs'
// loads complete on its barriers.
//
// Warp roles: warp 0 lane 0 issues TMA into a ring of kStages stages; warp 1
// owns TMEM and issues the MMAs; warps 4..11 read finished accumulator chunks
// (a few stages each, double buffered in TMEM) and add them in FP32 registers,
// scaled by the 8-bit operands' steps where there are any.  With kJoin the CTAs of
// a cluster may share one tile's contraction (Args::split).  The tensor cores'
// accumulator truncates, so an FP32 result's sums are kept short there.  Where the
// packed rows are the contraction, warp 3 zeroes what a group's last stage
// holds beyond the group.
// Every mbarrier wait is bounded; on expiry the CTA records
// BAKRON_ERR_DEVICE_TIMEOUT, drains what it issued, frees its tensor memory and
// exits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "mm.cuh"
#include "mm_groups.h"
#include "tcgen05.cuh"

namespace bakron {
namespace mm {

using namespace tc;

constexpr int kBM = 128;
constexpr int kMaxSorted = 128;  // groups up to which they are sorted by length
constexpr uint16_t kNoRows = 0x8000;  // beside a group's number: it counts as empty, whatever its bounds
constexpr int kReserve = 10 * 1024;  // barriers, tile numbering, alignment, staged steps

// Self-test of the ways out (bakron_selftest_rows_abort), by Args::gives_up: 1, one
// epilogue warp's last wait of its first tile counts as run out, its neighbours' do
// not; 2, the epilogue gives up before the last chunk once all MMAs are issued, and
// the status block's `where` says 1 if they had finished when tensor memory was
// released.
template <class P>
constexpr bool kGivesUp = false;

template <class P>
struct Shape {
    static constexpr int kCtas = P::kPair ? 2 : 1;
    static constexpr int kM = kBM * kCtas;                          // D rows of a tile
    static constexpr int kBRows = P::kBN / kCtas;                   // B rows in one CTA
    // one operand row of a stage is 128 bytes (the swizzle width)
    static constexpr int kElems = P::kEight ? 128 : 64;             // operand elements in 128 bytes
    static constexpr int kKB = P::kRagged == kContract ? P::kKRows : kElems;  // contraction per stage
    static constexpr int kABytes = P::kRagged == kContract ? kBM / 64 * kKB * 128 : kBM * 128;
    static constexpr int kBBytes = P::kRagged == kContract ? kBRows / 64 * kKB * 128 : kBRows * 128;
    static constexpr int kStageBytes = P::kPlanes * (kABytes + kBBytes);
    // shared memory in which results are turned (store_turned, store_staged)
    static constexpr bool kTurn = P::kRagged == kTokensB && P::kBN == 256;  // (16-bit operands only)
    static constexpr int kTurnSpace = kTurn ? 2 * 32 * kBM * 2 : P::kRagged == kTokensB ? 0 : 8 * 32 * 17 * 4;
    static constexpr int kEpiWarps = 8;
    static constexpr int kCols = P::kBN / (kEpiWarps / 4);          // columns per epilogue thread
    // a warp's staged steps: two chunks of its columns' (kTokensB), or one of them
    static constexpr int kStepFloats = P::kRagged == kTokensB ? 2 * kCols : kCols;
    // tiles whose contraction a cluster may split (few tiles, one per cluster)
    static constexpr bool kSplit = P::kJoin;
    static constexpr int kRing = 227 * 1024 - kReserve - kTurnSpace;
    static constexpr int kStages = kRing / kStageBytes < 8 ? kRing / kStageBytes : 8;
    static constexpr int kAcc = P::kPlanes > 1 ? 2 : 1;             // accumulators per buffer
    // accumulator buffers: two, or as many as tensor memory holds where a chunk
    // is one stage, so that the round trip MMA - epilogue - MMA (about 2000
    // clocks, whatever the tile) is shared by several chunks
    static constexpr int kBufs = P::kEight ? (P::kBN == 256 ? 2 : 4) : 2;
    static constexpr int kTmemCols = kBufs * kAcc * P::kBN;
    static constexpr int kThreads = 128 + 32 * kEpiWarps;
    // registers: the epilogue's accumulators and two loads in flight need more
    // than a 12-warp CTA's even share (168), the other warps far less
    static constexpr bool kRowSteps = P::kEight && P::kRagged == kTokensA;  // a step per lane and chunk
    static constexpr bool kSplitRegs = kCols > 64 || (kSplit && kCols == 64);
    static constexpr int kRegsOthers = 56, kRegsEpilogue = 224;
    // a warpgroup can only take registers that the block was launched with
    static constexpr int kRegsNeeded = 128 * kRegsOthers + 32 * kEpiWarps * kRegsEpilogue;
    static constexpr size_t kSmem = (size_t)kStages * kStageBytes + kTurnSpace + kReserve;
};

// One output tile: group e, D rows a0.. (na valid), D columns b0.. (nb valid),
// contraction over [k0, k1).
struct Tile {
    int e, a0, na, b0, nb, k0, k1, count;
};

// Group e's packed rows [lo, hi), empty if its bounds are no range.
__device__ __forceinline__ bool group_range(const Args &g, int e, int &lo, int &hi)
{
    if (!g.offsets) {
        lo = 0;
        hi = g.rows;
        return true;
    }
    lo = __ldg(g.offsets + e);
    hi = __ldg(g.offsets + e + 1);
    if (is_range(lo, hi, g.rows)) return true;
    lo = hi = 0;
    return false;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Tiles of tile row i that reach on or below the diagonal of a square result.
template <class P>
__device__ __forceinline__ int lower_tiles_of_row(const Args &g, int i)
{
    return min((i * Shape<P>::kM + Shape<P>::kM - 1) / P::kBN + 1, ceil_div(g.b_total, P::kBN));
}

template <class P>
__device__ __forceinline__ int tiles_of_group(const Args &g, int len)
{
    constexpr int kM = Shape<P>::kM;
    if (P::kRagged == kTokensB) return ceil_div(g.a_total, kM) * ceil_div(len, P::kBN);
    if (P::kRagged == kTokensA) return ceil_div(len, kM) * ceil_div(g.b_total, P::kBN);
    if (P::kLower) {
        int n = 0;
        for (int i = 0; i < ceil_div(g.a_total, kM); ++i) n += lower_tiles_of_row<P>(g, i);
        return n;
    }
    return ceil_div(g.a_total, kM) * ceil_div(g.b_total, P::kBN);
}

// Tile i of rows x cols ones, in bands of eight rows, down each band's columns:
// the tiles of one round over the SMs then form a block about as high as it is
// wide, which reads the fewest operand bytes.
__device__ __forceinline__ void raster(int i, int rows, int cols, int &row, int &col)
{
    const int band = i / (8 * cols), high = min(8, rows - 8 * band), in_band = i - band * 8 * cols;
    row = 8 * band + in_band % high;
    col = in_band / high;
}

template <class P>
__device__ __forceinline__ Tile find_tile(const Args &g, const int *first, const uint16_t *order, int t)
{
    constexpr int kM = Shape<P>::kM;
    int a = 0, b = g.experts;  // the last group whose first tile is <= t
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (first[m] <= t) a = m;
        else b = m;
    }
    Tile x;
    x.e = P::kRagged == kContract ? order[a] & ~kNoRows : a;
    int lo, hi;
    group_range(g, x.e, lo, hi);
    if (P::kRagged == kContract && (order[a] & kNoRows)) lo = hi = 0;
    int i = t - first[a];
    x.count = hi - lo;
    if (P::kRagged == kTokensB) {
        int row, col;
        raster(i, ceil_div(g.a_total, kM), ceil_div(hi - lo, P::kBN), row, col);
        x.a0 = row * kM;
        x.b0 = lo + col * P::kBN;
        x.na = min(kM, g.a_total - x.a0);
        x.nb = min(P::kBN, hi - x.b0);
        x.k0 = 0;
        x.k1 = g.k_total;
    } else if (P::kRagged == kTokensA) {
        int row, col;
        raster(i, ceil_div(hi - lo, kM), ceil_div(g.b_total, P::kBN), row, col);
        x.a0 = lo + row * kM;
        x.b0 = col * P::kBN;
        x.na = min(kM, hi - x.a0);
        x.nb = min(P::kBN, g.b_total - x.b0);
        x.k0 = 0;
        x.k1 = g.k_total;
    } else {
        int r, c;
        if (P::kLower) {
            for (r = 0; i >= lower_tiles_of_row<P>(g, r); ++r) i -= lower_tiles_of_row<P>(g, r);
            c = i;
        } else {
            const int nt = ceil_div(g.b_total, P::kBN);
            r = i / nt;
            c = i % nt;
        }
        x.a0 = r * kM;
        x.b0 = c * P::kBN;
        x.na = min(kM, g.a_total - x.a0);
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

__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
template <typename T>
__device__ __forceinline__ uint32_t word_of(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t word_of<__nv_bfloat16>(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t *)&v;
}
template <>
__device__ __forceinline__ uint32_t word_of<__half>(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *(const uint32_t *)&v;
}

// Columns [0, cols) of a warp's 32 rows (the lanes'; `rows` of them valid, the
// first at `first`), N columns of each in its lane's registers, through the
// warp's own shared memory, so that stores run along the rows: for results whose
// rows are not 32-byte aligned.  (Written from the lanes' own rows, every store
// touches 32 sectors: it took ten times as long.)
constexpr int kStageWords = 32 * 17;
template <typename T, int N, class Value, class Keep>
__device__ __forceinline__ void store_staged(T *first, int64_t ld, int rows, int cols, int lane, uint32_t *buf,
                                             Value value, Keep keep)
{
    constexpr int kWide = 64 / sizeof(T);  // columns a round: 16 words per row
#pragma unroll
    for (int c0 = 0; c0 < N; c0 += kWide) {
        if (c0 >= cols) break;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            if constexpr (sizeof(T) == 4) buf[lane * 17 + w] = __float_as_uint(value(c0 + w));
            else buf[lane * 17 + w] = word_of<T>(value(c0 + 2 * w), value(c0 + 2 * w + 1));
        }
        __syncwarp();
        constexpr int kRows = 32 / kWide;  // rows a store covers
        const int c = lane % kWide;
        if (c0 + c < cols) {
#pragma unroll 4
            for (int r = lane / kWide; r < rows; r += kRows)
                if (keep(r, c0 + c)) first[r * ld + c0 + c] = ((const T *)(buf + r * 17))[c];
        }
        __syncwarp();
    }
}

// Store this thread's accumulators: D row `lane_row` of the tile, columns
// [col0, col0 + N).  All lanes of the warp take part.
template <class P, typename T, int N>
__device__ __forceinline__ void store_tile(const Args &g, const Tile &x, int lane_row, int col0,
                                           const float (&acc)[N], uint32_t *buf)
{
    T *out = (T *)g.out;
    const int cols = min(N, x.nb - col0);
    if (P::kRagged == kTokensB) {
        // D row = output column: the 32 lanes of a warp write consecutive
        // elements of one packed row
        if (lane_row >= x.na) return;
        T *p = out + (int64_t)(x.b0 + col0) * g.ldo + x.a0 + lane_row;
        float s = 1.f;
        if (P::kEight && g.w_step_rows == 1) s = __ldg(g.w_steps + (int64_t)x.e * g.a_total + x.a0 + lane_row);
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (c < cols) p[(int64_t)c * g.ldo] = round_to<T>(P::kEight ? acc[c] * s : acc[c]);
    } else {
        T *tile = out + (P::kRagged == kContract ? (int64_t)x.e * g.out_expert_stride : 0) + (int64_t)x.a0 * g.ldo +
                  x.b0 + col0;
        const uintptr_t align = (uintptr_t)tile | (uintptr_t)(g.ldo * (int64_t)sizeof(T));  // of every row
        if (align & 31) {
            const int lane = threadIdx.x & 31;
            store_staged<T, N>(tile + (int64_t)(lane_row - lane) * g.ldo, g.ldo, min(32, x.na - (lane_row - lane)), cols,
                               lane, buf, [&](int c) { return acc[c]; }, [](int, int) { return true; });
            return;
        }
        if (lane_row >= x.na) return;
        T *p = tile + (int64_t)lane_row * g.ldo;
        constexpr int kVec = 32 / sizeof(T);
#pragma unroll
        for (int c = 0; c < N; c += kVec) {
            if (c + kVec <= cols) {
                uint32_t v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if constexpr (sizeof(T) == 4) v[u] = __float_as_uint(acc[c + u]);
                    else v[u] = word_of<T>(acc[c + 2 * u], acc[c + 2 * u + 1]);
                }
                store32(p + c, v);  // one whole 32-byte sector
            } else {
#pragma unroll
                for (int u = 0; u < kVec; ++u)
                    if (c + u < cols) p[c + u] = round_to<T>(acc[c + u]);
            }
        }
    }
}

// kTokensB, 16-bit results whose rows keep 16-byte alignment: the four warps of
// a column half turn 32 packed rows at a time in shared memory and write whole
// 256-byte row pieces.  (Written from the accumulators' own lanes, a warp's
// store is 64 bytes: 128 of them per thread held the next tile's MMAs up.)
// All four warps come here or none: half_agrees() decides for them, and its
// barrier stands before the first use of the buffer.
constexpr int kTurnRows = 32;
constexpr int kTurnBytes = kTurnRows * kBM * 2;
// Whether `ok` holds in all four warps of a column half, which meet here.  A wait
// that has run out, or that another role's giving up has ended, may have failed in
// one of them and not in its neighbours.
__device__ __forceinline__ bool half_agrees(int half, bool ok)
{
    uint32_t all;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)ok), "r"(1 + half)
        : "memory");
    return all != 0;
}
template <class P, typename T, int N>
__device__ __forceinline__ void store_turned(const Args &g, const Tile &x, int rank, int thread, int half,
                                             const float (&acc)[N], T *buf)
{
    const int row0 = rank * kBM;                 // this CTA's first D row
    const int col0 = half * N;
    const int piece = (thread & 15) * 8;         // D rows this thread writes: 8 of the CTA's 128
    const int valid = x.na - row0 - piece;
    T *out = (T *)g.out + (int64_t)(x.b0 + col0) * g.ldo + x.a0 + row0 + piece;
#pragma unroll
    for (int c0 = 0; c0 < N; c0 += kTurnRows) {
        if (col0 + c0 >= x.nb) break;
        if (c0) asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
#pragma unroll
        for (int c = 0; c < kTurnRows; ++c) buf[c * kBM + thread] = round_to<T>(acc[c0 + c]);
        asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
#pragma unroll
        for (int r = 0; r < kTurnRows; r += 8) {
            const int t = r + (thread >> 4);
            if (col0 + c0 + t < x.nb) {
                const uint4 v = *(const uint4 *)(buf + t * kBM + piece);
                T *p = out + (int64_t)(c0 + t) * g.ldo;
                if (valid >= 8) {
                    *(uint4 *)p = v;
                } else {
                    const T *e = (const T *)&v;
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (u < valid) p[u] = e[u];
                }
            }
        }
    }
}

// Gram tile: entries on and below the diagonal, divided by the group's count,
// and their mirror images.  All lanes of the warp take part.
template <int N>
__device__ __forceinline__ void store_gram(const Args &g, const Tile &x, int lane_row, int col0,
                                           const float (&acc)[N], uint32_t *buf)
{
    const int64_t d = g.ldo;
    float *out = (float *)g.out + (int64_t)x.e * g.out_expert_stride;
    const int lane = threadIdx.x & 31, i = x.a0 + lane_row, j0 = x.b0 + col0;
    const float count = (float)max(x.count, 1), rcount = __frcp_rn(count);
    auto value = [&](int c) { return div_rn_recip(acc[c], count, rcount); };
    // columns of this row up to the diagonal
    const int cols = lane_row < x.na ? min(x.nb - col0, i + 1 - j0) : 0;
    float *col = out + j0 * d + i;
    const uintptr_t align = (uintptr_t)(out + j0) | (uintptr_t)(d * 4);
    if (align & 31) {
        // the mirror image runs along the lanes as it is
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (c < cols) col[(int64_t)c * d] = value(c);
        const int row0 = lane_row - lane;  // the warp's first row
        store_staged<float, N>(out + (int64_t)(x.a0 + row0) * d + j0, d, min(32, x.na - row0), min(N, x.nb - col0), lane,
                               buf, value, [&](int r, int c) { return j0 + c <= x.a0 + row0 + r; });
        return;
    }
    float *row = out + i * d + j0;
    // Eight columns at a time: along the row where all eight are below the
    // diagonal, and a warp's 32 rows next to each other in the mirror image.
#pragma unroll
    for (int c = 0; c < N; c += 8) {
        if (c + 8 <= cols) {
            uint32_t v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                v[u] = __float_as_uint(value(c + u));
                col[(int64_t)(c + u) * d] = __uint_as_float(v[u]);
            }
            store32(row + c, v);  // one whole 32-byte sector
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (c + u < cols) {
                    const float v = value(c + u);
                    row[c + u] = v;
                    col[(int64_t)(c + u) * d] = v;
                }
        }
    }
}

// The last stage of a group that ends inside it: rows [valid, 16 steps) of both
// operands (the next group's, or whatever lies behind the last one) are zeroed
// in this CTA's shared memory by one warp, NaN and all.
template <class P>
__device__ __forceinline__ void zero_tail(uint8_t *stage, int valid, int steps, int lane)
{
    using S = Shape<P>;
    constexpr int kAtoms = S::kStageBytes / (S::kKB * 128);
    const int rows = 16 * steps - valid;
    for (int i = lane; i < kAtoms * rows * 8; i += 32) {
        const int atom = i / (rows * 8), w = i % (rows * 8);
        *(uint4 *)(stage + atom * S::kKB * 128 + (valid + (w >> 3)) * 128 + (w & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// Every CTA reports in a byte of its own, so that no call needs the status
// block cleared first: the first CTA clears the recorded code and the bytes
// that no CTA of this grid owns.
__device__ __forceinline__ void report(DeviceStatus *st, int error)
{
    if (blockIdx.x == 0) {
        st->code = 0;
        st->where = 0;
        for (int i = gridDim.x; i < kStatusSlots; ++i) st->slots[i] = 0;
    }
    st->slots[blockIdx.x] = (uint8_t)error;
}

template <class P>
__global__ void __launch_bounds__(Shape<P>::kThreads, 1)
mm_kernel(const __grid_constant__ Maps maps, const Args g)
{
    using S = Shape<P>;
    constexpr int BN = P::kBN;
    constexpr bool kPair = P::kPair;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *turn_sh = smem + S::kStages * S::kStageBytes;
    uint64_t *bars = (uint64_t *)(turn_sh + S::kTurnSpace);
    int *first = (int *)(bars + 48);                        // tile numbering: kMaxExperts + 1
    uint16_t *order = (uint16_t *)(first + kMaxExperts + 4);  // groups, longest first (kContract)
    float *steps_sh = (float *)(first + kMaxExperts + 4);     // staged row steps (8-bit)
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh, error_sh;
    [[maybe_unused]] __shared__ volatile int issued_sh;  // (self-test)

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = kPair ? (int)cluster_rank() : 0;
    // Split contraction: the CTAs of a cluster share one tile, each taking a
    // part of its stages; one tile per cluster.
    const int split = S::kSplit ? g.split : 1, part = S::kSplit && split > 1 ? (int)cluster_rank() : 0;
    const uint32_t bar0 = smem_u32(bars);
    // Barriers.  In a pair, full, accumulator-empty and tail-done barriers are
    // the first CTA's; the others each CTA has for itself.
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S::kStages + s); };
    auto tail_full_bar = [&](int s) { return bar0 + 8u * (2 * S::kStages + s); };  // a tail stage has landed in this CTA
    auto tail_done_bar = [&](int s) { return bar0 + 8u * (3 * S::kStages + s); };  // the CTAs have zeroed their tails
    auto accf_bar = [&](int b) { return bar0 + 8u * (4 * S::kStages + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (4 * S::kStages + S::kBufs + b); };
    const uint32_t drain_bar = bar0 + 8u * (4 * S::kStages + 2 * S::kBufs);
    static_assert(4 * S::kStages + 2 * S::kBufs + 1 <= 48, "barriers");
    static_assert(48 * 8 + (kMaxExperts + 4) * 4 + 1024 +
                          (P::kEight ? S::kEpiWarps * S::kStepFloats * 4 : kMaxExperts * 2) <= kReserve,
                  "what lies behind the ring");
    static_assert(!S::kSplit || S::kStages * S::kStageBytes >= kBM * BN * 4, "a part's sums take its ring");
    // accumulator chunk number c: its buffer and the parity of its buffer's use
    auto buf_of = [](int c) { return c % S::kBufs; };
    auto use_of = [](int c) { return c / S::kBufs & 1; };

    if (threadIdx.x == 0) {
        prefetch_map(&maps.a);
        prefetch_map(&maps.b);
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
            mbar_init(tail_full_bar(s), 1);
            mbar_init(tail_done_bar(s), S::kCtas);
        }
        for (int b = 0; b < S::kBufs; ++b) {
            mbar_init(accf_bar(b), 1);
            mbar_init(acce_bar(b), S::kEpiWarps * S::kCtas);
        }
        mbar_init(drain_bar, 1);
        abort_sh = 0;
        if constexpr (kGivesUp<P>) issued_sh = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&tmem_base_sh)),
                         "r"(S::kTmemCols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&tmem_base_sh)),
                         "r"(S::kTmemCols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    pdl_wait();  // everything below may touch what earlier kernels wrote
    if (warp == 2) {
        // tile numbering: exclusive prefix sum of the groups' tile counts, those
        // of groups whose rows no earlier group has; where a tile's cost is its
        // group's length, longest groups first
        int base = 0, reach = 0;
        if (lane == 0) error_sh = BAKRON_OK;
        __syncwarp();
        const int fixed = P::kRagged == kContract ? tiles_of_group<P>(g, 0) : 0;
        for (int e0 = 0; e0 < g.experts; e0 += 32) {
            const int e = e0 + lane;
            int lo = 0, hi = 0;
            const bool range = e < g.experts && group_range(g, e, lo, hi);
            int most = hi;  // the largest end up to this group
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, most, o);
                if (lane >= o) most = max(most, v);
            }
            const int before = __shfl_up_sync(0xffffffffu, most, 1);
            const bool rows = range && has_rows(lo, hi, g.rows, lane ? max(reach, before) : reach);
            reach = max(reach, __shfl_sync(0xffffffffu, most, 31));
            int n = 0;
            if (e < g.experts) {
                if (!rows) error_sh = BAKRON_ERR_INVALID_ARG;
                n = P::kRagged == kContract ? fixed : rows ? tiles_of_group<P>(g, hi - lo) : 0;
                if (P::kRagged == kContract) {
                    int place = e;
                    if (g.experts <= kMaxSorted) {
                        place = 0;
                        for (int o = 0; o < g.experts; ++o) {
                            int a, b;
                            group_range(g, o, a, b);
                            place += b - a > hi - lo || (b - a == hi - lo && o < e);
                        }
                    }
                    order[place] = (uint16_t)e | (rows ? 0 : kNoRows);
                }
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
    if (kPair) cluster_sync();  // the other CTA's barriers exist before anything signals them
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_sh;
    const int chunk_stages = P::kEight ? 1 : g.chunk;
    const int tile0 = blockIdx.x / (S::kCtas * split), tile_step = gridDim.x / (S::kCtas * split);
    // The host launches a cluster per tile where a contraction is split.  A second
    // tile would need the join's barriers again, which have no time limit, so none
    // is taken even if the bounds change while the kernels of a call read them.
    int total = first[g.experts];
    if (S::kSplit && split > 1 && total > tile_step) {
        total = tile_step;
        if (threadIdx.x == 0) error_sh = BAKRON_ERR_INVALID_ARG;
    }
    // The tile after t.  Where a tile's cost is its group's length, every other
    // round runs backwards, so that who had a long tile gets a short one.
    auto next_tile = [&](int t) {
        if (P::kRagged != kContract) return t + tile_step;
        const int round = t / tile_step;
        return round & 1 ? (round + 1) * tile_step + tile0 : (round + 2) * tile_step - 1 - tile0;
    };
    // this CTA's stages of a tile with n of them
    auto stage_begin = [&](int n) { return S::kSplit ? n * part / split : 0; };
    auto stage_end = [&](int n) { return S::kSplit ? n * (part + 1) / split : n; };
    volatile int *abort_flag = &abort_sh;
    bool joined = false;

    // Bounded wait: false once it has run for the time limit of a pipeline step,
    // or of `steps` of them, or another role has given up.
    auto wait = [&](uint32_t bar, uint32_t parity, int steps = 1) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = now_ns(), limit = g.timeout_ns * (uint64_t)min(steps, 1 << 24);  // (600 s at most a step)
        for (;;) {
            for (int i = 0; i < 16; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) return false;
            if (now_ns() - t0 > limit) {
                error_sh = BAKRON_ERR_DEVICE_TIMEOUT;
                atomicExch(&abort_sh, 1);
                return false;
            }
        }
    };

    if (warp < 4) {
        if constexpr (S::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsOthers));
        if (warp == 0 && elect_one()) {
            // ---------------- TMA producer
            const uint32_t first_cta = kPair ? map_rank(bar0, 0) : bar0;  // the pair's first CTA's barriers
            int it = 0;
            uint32_t tail_last = 0, tail_count = 0;  // per stage: last use was a tail; parity of its tails
            bool ok = true;
            for (int t = tile0; t < total && ok; t = next_tile(t)) {
                const Tile x = find_tile<P>(g, first, order, t);
                const int nkb = ceil_div(x.k1 - x.k0, S::kKB);
                const int a0 = x.a0 + rank * kBM;
                // rows of B this CTA loads: its share of the instruction's N
                const int share = P::kRagged == kTokensB ? ((x.nb + 15) & ~15) / S::kCtas : S::kBRows;
                const int b0 = x.b0 + rank * share;
                const int boxes = P::kRagged == kTokensB ? ceil_div(share, P::kBoxRows) : 1;
                const uint32_t bytes = P::kRagged == kTokensB ? S::kABytes + boxes * P::kBoxRows * 128 : S::kStageBytes;
                for (int kb = stage_begin(nkb); kb < stage_end(nkb); ++kb, ++it) {
                    const int s = it % S::kStages;
                    if (it >= S::kStages && !wait(empty_bar(s), (it / S::kStages - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a = smem_u32(smem + s * S::kStageBytes), b = a + P::kPlanes * S::kABytes;
                    const int k = x.k0 + kb * S::kKB;
                    // In a pair both CTAs' loads complete on the first one's
                    // barrier.  A tail stage completes on a barrier of its own
                    // CTA's, whose warp 3 zeroes what lies beyond the group.
                    const bool tail = P::kRagged == kContract && ((x.k1 - k) & 15) && x.k1 - k < S::kKB;
                    uint32_t bar = full_bar(s);
                    tail_last = tail ? tail_last | 1u << s : tail_last & ~(1u << s);
                    if (tail) {
                        tail_count ^= 1u << s;
                        if (!rank) mbar_arrive(bar);  // the stage's phases go on
                        bar = tail_full_bar(s);
                        mbar_expect_tx(bar, bytes);
                        if (kPair) bar = map_rank(bar, rank);
                    } else if (!kPair) {
                        mbar_expect_tx(bar, bytes);
                    } else {
                        if (!rank) mbar_expect_tx(bar, 2 * bytes);
                        bar = first_cta + 8u * s;
                    }
                    auto load2 = [&](uint32_t dst, const CUtensorMap *m, int cx, int cy) {
                        if (kPair) tma_load_2d_pair(dst, m, cx, cy, bar);
                        else tma_load_2d(dst, m, cx, cy, bar);
                    };
                    auto load3 = [&](uint32_t dst, const CUtensorMap *m, int cx, int cy, int cz) {
                        if (kPair) tma_load_3d_pair(dst, m, cx, cy, cz, bar);
                        else tma_load_3d(dst, m, cx, cy, cz, bar);
                    };
                    if (P::kRagged == kTokensB) {
                        if (P::kAColumns) {
                            load3(a, &maps.a, a0, k, x.e);
                            load3(a + S::kABytes / 2, &maps.a, a0 + 64, k, x.e);
                        } else {
                            load3(a, &maps.a, k, a0, x.e);
                        }
                        if (boxes == 2) {
                            load2(b, &maps.b2, k, b0);
                        } else {
                            for (int r = 0; r < boxes; ++r)
                                load2(b + r * P::kBoxRows * 128, &maps.b, k, b0 + r * P::kBoxRows);
                        }
                    } else if (P::kRagged == kTokensA) {
                        load2(a, &maps.a, k, a0);
                        load3(b, &maps.b, k, b0, x.e);
                    } else {
#pragma unroll
                        for (int p = 0; p < P::kPlanes; ++p) {
#pragma unroll
                            for (int c = 0; c < kBM / 64; ++c)
                                load3(a + p * S::kABytes + c * S::kKB * 128, &maps.a, a0 + 64 * c, k, p);
#pragma unroll
                            for (int c = 0; c < S::kBRows / 64; ++c)
                                load3(b + p * S::kBBytes + c * S::kKB * 128, &maps.b, b0 + 64 * c, k, p);
                        }
                    }
                }
            }
            // every issued copy has to land before the CTA may exit (in a pair
            // the first CTA's full barriers count both CTAs' copies)
            for (int i = max(0, it - S::kStages); i < it; ++i) {
                const int s = i % S::kStages;
                const bool tail = (tail_last >> s) & 1;
                if (rank && !tail) continue;
                const uint32_t bar = tail ? tail_full_bar(s) : full_bar(s);
                const uint32_t parity = tail ? ((tail_count >> s) & 1) ^ 1 : (i / S::kStages) & 1;
                const uint64_t t0 = now_ns();
                while (!mbar_try_wait(bar, parity) && now_ns() - t0 < g.timeout_ns + 50000000ull) {
                }
            }
        } else if (warp == 1 && rank == 0 && elect_one()) {
            // ---------------- MMA issuer
            int it = 0, chunk = 0;
            uint32_t tail_parity = 0;  // one bit per stage
            bool ok = true;
            // descriptors of stage 0; another address only changes the low bits
            constexpr bool kACols = P::kRagged == kContract || P::kAColumns, kBCols = P::kRagged == kContract;
            const uint32_t base = smem_u32(smem), base_b = base + P::kPlanes * S::kABytes;
            const uint64_t a_desc = kACols ? umma_desc_mn(base, S::kKB * 128) : umma_desc(base);
            const uint64_t b_desc = kBCols ? umma_desc_mn(base_b, S::kKB * 128) : umma_desc(base_b);
            constexpr int kSteps = S::kKB / (P::kEight ? 32 : 16);
            constexpr int kAStep = (kACols ? 2048 : 32) >> 4, kBStep = (kBCols ? 2048 : 32) >> 4;
            auto mma = [&](uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t add) {
                if (P::kEight) {
                    if (kPair) umma_f8_pair(d, ad, bd, idesc, add);
                    else umma_f8(d, ad, bd, idesc, add);
                } else {
                    if (kPair) umma_f16_pair(d, ad, bd, idesc, add);
                    else umma_f16(d, ad, bd, idesc, add);
                }
            };
            auto commit = [&](uint32_t bar) {
                if (kPair) umma_commit_pair(bar);
                else umma_commit(bar);
            };
            for (int t = tile0; t < total && ok; t = next_tile(t)) {
                const Tile x = find_tile<P>(g, first, order, t);
                const int nkb = ceil_div(x.k1 - x.k0, S::kKB);
                const int n_mma = P::kRagged == kTokensB ? (x.nb + 15) & ~15 : BN;
                const uint32_t idesc = g.idesc | ((uint32_t)(n_mma >> 3) << 17) | ((uint32_t)(S::kM >> 4) << 24);
                const int kb0 = stage_begin(nkb), kb1 = stage_end(nkb);
                for (int kb = kb0, in_chunk = 0; kb < kb1; ++kb, ++it) {
                    const int buf = buf_of(chunk);
                    const int s = it % S::kStages;
                    if (in_chunk == 0 && chunk >= S::kBufs) ok = wait(acce_bar(buf), use_of(chunk) ^ 1);
                    ok = ok && wait(full_bar(s), (it / S::kStages) & 1);
                    int steps = kSteps;
                    if (P::kRagged == kContract) {
                        const int valid = min(S::kKB, x.k1 - (x.k0 + kb * S::kKB));
                        steps = (valid + 15) >> 4;
                        if (valid & 15) {
                            // (the zeroes written there are ordered by an
                            // acquire at cluster scope once they are complete)
                            ok = ok && wait(tail_done_bar(s), (tail_parity >> s) & 1) &&
                                 mbar_try_wait_cluster(tail_done_bar(s), (tail_parity >> s) & 1);
                            tail_parity ^= 1u << s;
                        }
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem_base + (uint32_t)(buf * S::kAcc * BN);
                    const uint64_t ad = a_desc + (uint32_t)(s * (S::kStageBytes >> 4));
                    const uint64_t bd = b_desc + (uint32_t)(s * (S::kStageBytes >> 4));
#pragma unroll
                    for (int ks = 0; ks < kSteps; ++ks) {
                        if (P::kRagged == kContract && ks >= steps) break;
                        const uint32_t add = (in_chunk | ks) != 0;
                        const uint64_t ak = ad + ks * kAStep, bk = bd + ks * kBStep;
                        if (P::kPlanes > 1) {
                            // x = h + m + l in three bf16 parts: hh into one
                            // accumulator, the five smaller products into another
                            constexpr uint32_t kAm = S::kABytes >> 4, kBm = S::kBBytes >> 4;
                            mma(d, ak, bk, idesc, add);
                            mma(d + BN, ak, bk + 2 * kBm, idesc, add);
                            mma(d + BN, ak + 2 * kAm, bk, idesc, 1);
                            mma(d + BN, ak + kAm, bk + kBm, idesc, 1);
                            mma(d + BN, ak, bk + kBm, idesc, 1);
                            mma(d + BN, ak + kAm, bk, idesc, 1);
                        } else {
                            mma(d, ak, bk, idesc, add);
                        }
                    }
                    commit(empty_bar(s));
                    if (++in_chunk == chunk_stages || kb == kb1 - 1) {
                        commit(accf_bar(buf));
                        in_chunk = 0;
                        ++chunk;
                    }
                }
            }
            if constexpr (kGivesUp<P>) issued_sh = ok;
            // Issued MMAs finish before tensor memory is released, also where the
            // epilogue gives up while the last of them run: the last chunk's commit
            // says so, or one more where the loop was left inside a chunk.
            const uint32_t done_bar = ok ? accf_bar(buf_of(chunk - 1)) : drain_bar;
            const uint32_t done_parity = ok ? use_of(chunk - 1) : 0;
            if (!ok) commit(drain_bar);
            if (!ok || chunk) {
                const uint64_t t0 = now_ns();
                while (!mbar_try_wait(done_bar, done_parity) && now_ns() - t0 < g.timeout_ns + 50000000ull) {
                }
            }
        } else if (warp == 3 && P::kRagged == kContract) {
            // ---------------- zero the tails of this CTA's operands
            // (a tail may be many stages away: its wait has the limit of them all)
            int it = 0, last = 0;
            uint32_t tail_parity = 0;
            for (int t = tile0; t < total; t = next_tile(t)) {
                const Tile x = find_tile<P>(g, first, order, t);
                const int nkb = ceil_div(x.k1 - x.k0, S::kKB);
                it += stage_end(nkb) - stage_begin(nkb);
                const int valid = (x.k1 - x.k0) % S::kKB;
                if (!(valid & 15) || (S::kSplit && part != split - 1)) continue;  // (the last part has the last stage)
                const int s = (it - 1) % S::kStages;
                if (!__all_sync(0xffffffffu, wait(tail_full_bar(s), (tail_parity >> s) & 1, it - last + 1))) break;
                last = it;
                tail_parity ^= 1u << s;
                zero_tail<P>(smem + s * S::kStageBytes, valid, (valid + 15) >> 4, lane);
                if (lane == 0) {
                    if (kPair) mbar_arrive_cluster(map_rank(tail_done_bar(s), 0));
                    else mbar_arrive(tail_done_bar(s));
                }
                __syncwarp();
            }
        }
        __syncwarp();
    } else {
        // ---------------- epilogue: chunks TMEM -> FP32 registers, then store
        if constexpr (S::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegsEpilogue));
        const int quad = warp & 3;                   // TMEM lanes [32 quad, 32 quad + 32)
        const int half = (warp - 4) >> 2;            // columns [half kCols, half kCols + kCols)
        const int lane_row = rank * kBM + quad * 32 + lane;
        int col0 = half * S::kCols;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        float *steps_w = steps_sh + (warp - 4) * S::kStepFloats;
        uint32_t *stage_buf = (uint32_t *)turn_sh + (warp - 4) * kStageWords;  // (not with kTokensB)
        const uint32_t first_cta_acce = kPair ? map_rank(acce_bar(0), 0) : acce_bar(0);
        int chunk = 0;
        bool ok = true;
        for (int t = tile0; t < total && ok; t = next_tile(t)) {
            Tile x = find_tile<P>(g, first, order, t);
            const int nkb = ceil_div(x.k1 - x.k0, S::kKB);
            const int kb0 = stage_begin(nkb);
            const int nchunk = ceil_div(stage_end(nkb) - kb0, chunk_stages);
            // 16-column loads of each chunk: the tile's valid columns only
            const int loads = min(max(ceil_div(x.nb - col0, 16), 0), S::kCols / 16) * S::kAcc;
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
                    ws = g.w_steps + ((int64_t)x.e * ceil_div(g.a_total, 128) +
                                      min((x.a0 + rank * kBM) / 128, ceil_div(g.a_total, 128) - 1)) * nkb;
                }
            }
            // One chunk: wait for it, add it, give its buffer back.
            auto take = [&](float row_step, const float *steps) {
                const int buf = buf_of(chunk);
                ok = wait(accf_bar(buf), use_of(chunk)) && ok;
                __syncwarp();
                tc_fence_after();
                const uint32_t src = tmem_base + lane_off + (uint32_t)(buf * S::kAcc * BN + col0);
                auto addr = [&](int l) { return src + (uint32_t)((l / S::kAcc) * 16 + (l % S::kAcc) * BN); };
                auto add = [&](const uint32_t (&r)[16], int l) {
                    const int c0 = (l / S::kAcc) * 16;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float v = __uint_as_float(r[i]);
                        if (S::kRowSteps) acc[c0 + i] = fmaf(v, row_step, acc[c0 + i]);
                        else if (P::kEight) acc[c0 + i] = fmaf(v, steps[c0 + i], acc[c0 + i]);
                        else acc[c0 + i] += v;
                    }
                };
                constexpr int kLoads = S::kCols / 16 * S::kAcc;
                // the buffer is free once its last load has arrived
                auto release = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        const uint32_t bar = first_cta_acce + 8u * buf;
                        if (kPair) mbar_arrive_remote(bar);
                        else mbar_arrive(bar);
                    }
                };
                if (loads == kLoads) {
                    // one load in flight while the one before it is added
                    // (straight-line code: the loads' registers then feed the
                    // additions without copies)
                    uint32_t r[kLoads][16];
                    tmem_ld16_start(addr(0), r[0]);
#pragma unroll
                    for (int l = 0; l < kLoads; ++l) {
                        tmem_ld16_wait(r[l]);
                        if (l + 1 < kLoads) tmem_ld16_start(addr(l + 1), r[l + 1]);
                        else release();
                        add(r[l], l);
                    }
                } else {
#pragma unroll
                    for (int l = 0; l + 1 < kLoads; ++l)
                        if (l < loads) {
                            uint32_t r[16];
                            tmem_ld16_start(addr(l), r);
                            tmem_ld16_wait(r);
                            add(r, l);
                        }
                    release();
                }
                ++chunk;
            };
            if constexpr (S::kRowSteps) {
                // the row's and the weight's steps four chunks at a time, fetched
                // four chunks ahead
                const bool vec = ((nkb | kb0) & 3) == 0;  // both start on 16-byte boundaries
                auto four = [&](const float *p, int c) {
                    if (vec) return __ldg((const float4 *)(p + c));
                    return make_float4(__ldg(p + c), c + 1 < nkb ? __ldg(p + c + 1) : 0.f,
                                       c + 2 < nkb ? __ldg(p + c + 2) : 0.f, c + 3 < nkb ? __ldg(p + c + 3) : 0.f);
                };
                float4 xn = make_float4(0, 0, 0, 0), wn = make_float4(1, 1, 1, 1);
                if (own_row) xn = four(xs, kb0);
                if (ws) wn = four(ws, kb0);
                for (int c = 0; c < nchunk && ok; c += 4) {
                    const float s[4] = {xn.x * wn.x, xn.y * wn.y, xn.z * wn.z, xn.w * wn.w};
                    if (c + 4 < nchunk) {
                        if (own_row) xn = four(xs, kb0 + c + 4);
                        if (ws) wn = four(ws, kb0 + c + 4);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + i < nchunk) take(s[i], nullptr);
                    ok = __all_sync(0xffffffffu, ok);
                }
            } else {
                for (int c = 0; c < nchunk && ok; ++c) {
                    float *steps = steps_w + (c & 1) * S::kCols;
                    if (P::kEight) {
                        const float s = ws ? __ldg(ws + kb0 + c) : 1.f;
                        for (int j = lane; j < S::kCols; j += 32)
                            steps[j] =
                                col0 + j < x.nb ? __ldg(g.x_steps + (int64_t)(x.b0 + col0 + j) * nkb + kb0 + c) * s : 0.f;
                        __syncwarp();
                    }
                    if constexpr (kGivesUp<P>) {
                        if (g.gives_up == 2 && rank == 0 && c == nchunk - 1) {
                            const uint64_t t0 = now_ns();
                            while (!issued_sh && now_ns() - t0 < g.timeout_ns) {
                            }
                            error_sh = BAKRON_ERR_DEVICE_TIMEOUT;
                            atomicExch(&abort_sh, 1);
                            ok = false;
                            break;
                        }
                    }
                    take(0.f, steps);
                    ok = __all_sync(0xffffffffu, ok);
                }
            }
            if constexpr (S::kSplit) {
                if (split > 1) {
                    // This part's MMAs have read all its stages, so its ring can
                    // take its sums.  Each part then adds up, in the parts'
                    // order, its share of the columns, and stores those (one
                    // CTA adding all of them took 20 us for eight parts of 128
                    // columns); nobody leaves before everybody has read.
                    float *mine = (float *)smem + (int64_t)col0 * kBM + quad * 32 + lane;
#pragma unroll
                    for (int c = 0; c < S::kCols; ++c)
                        if (c < 16 * loads) mine[c * kBM] = acc[c];
                    cluster_sync();
                    const int share = S::kCols / split;  // a power of two, at least four
                    col0 = half * S::kCols + part * share;
                    x.nb = min(x.nb, col0 + share);
                    const uint32_t from = smem_u32(mine + part * share * kBM);
#pragma unroll
                    for (int c = 0; c < S::kCols; ++c) acc[c] = 0.f;
#pragma unroll
                    for (int c = 0; c < S::kCols / 2; c += 4) {
                        if (c >= share) break;
                        float v[8][4];  // up to 32 loads in flight
#pragma unroll
                        for (int p = 0; p < 8; ++p)
                            if (p < split) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) v[p][i] = load_cluster(map_rank(from, p) + (c + i) * (kBM * 4));
                            }
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[c + i] = v[0][i];
#pragma unroll
                        for (int p = 1; p < 8; ++p)
                            if (p < split) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) acc[c + i] += v[p][i];
                            }
                    }
                    cluster_arrive();
                    joined = true;
                }
            }
            if constexpr (kGivesUp<P>) {
                if (g.gives_up == 1 && warp == 4 && rank == 0 && t == tile0) {
                    error_sh = BAKRON_ERR_DEVICE_TIMEOUT;
                    atomicExch(&abort_sh, 1);
                    ok = false;
                }
            }
            if constexpr (S::kTurn) {
                if (g.turn) ok = half_agrees(half, ok);
            }
            if (!ok) break;
            if (P::kEight && P::kRagged == kTokensA && g.w_step_rows == 1) {
                // one step per column, through shared memory (a warp's own)
                const float *s = g.w_steps + (int64_t)x.e * g.b_total + x.b0 + col0;
                __syncwarp();
                for (int j = lane; j < S::kCols; j += 32) steps_w[j] = col0 + j < x.nb ? __ldg(s + j) : 0.f;
                __syncwarp();
#pragma unroll
                for (int c = 0; c < S::kCols; ++c) acc[c] *= steps_w[c];
            }
            if constexpr (P::kLower) {
                store_gram(g, x, lane_row, col0, acc, stage_buf);
                continue;
            }
            if constexpr (S::kTurn) {
                if (g.turn) {
                    const int thread = quad * 32 + lane;
                    if (g.out_type == BAKRON_BF16)
                        store_turned<P>(g, x, rank, thread, half, acc, (__nv_bfloat16 *)(turn_sh + half * kTurnBytes));
                    else
                        store_turned<P>(g, x, rank, thread, half, acc, (__half *)(turn_sh + half * kTurnBytes));
                    continue;
                }
            }
            if (g.out_type == BAKRON_BF16) store_tile<P, __nv_bfloat16>(g, x, lane_row, col0, acc, stage_buf);
            else if (g.out_type == BAKRON_F16) store_tile<P, __half>(g, x, lane_row, col0, acc, stage_buf);
            else store_tile<P, float>(g, x, lane_row, col0, acc, stage_buf);
        }
    }
    if constexpr (S::kSplit) {
        // warps that have not taken part in the join arrive at its barriers
        __syncwarp();
        if (split > 1) {
            if (!joined) {
                cluster_sync();
                cluster_arrive();
            }
            cluster_wait();
        }
    }
    pdl_trigger();  // the next kernel's CTAs may start their own set-up
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) report(g.st, error_sh);
    if (kPair) cluster_sync();  // neither CTA leaves while the other can still reach its memory
    if constexpr (kGivesUp<P>) {  // (its two chunks: each buffer's first use)
        if (g.gives_up == 2 && rank == 0 && threadIdx.x == 0) g.st->where = mbar_try_wait(accf_bar(1), 0) ? 1 : 2;
    }
    if (warp == 1) {
        tc_fence_after();
        if (kPair)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(S::kTmemCols));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(S::kTmemCols));
    }
}

template <class P>
cudaError_t configure()
{
    using S = Shape<P>;
    if (S::kSplitRegs) {
        // refuse a build whose launch does not bring the registers the
        // warpgroups will ask for: they would wait for them for ever
        cudaFuncAttributes a;
        const cudaError_t e = cudaFuncGetAttributes(&a, mm_kernel<P>);
        if (e != cudaSuccess) return e;
        if (a.numRegs * S::kThreads < S::kRegsNeeded) return cudaErrorLaunchOutOfResources;
    }
    return cudaFuncSetAttribute(mm_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
}

// As many CTAs as the device has SMs (`sms`), fewer if there are fewer tiles
// (`tiles`, an upper bound).
template <class P>
cudaError_t launch(const Maps &maps, const Args &g, int64_t tiles, int sms, cudaStream_t stream)
{
    using S = Shape<P>;
    const int64_t groups = min64(tiles, min64(sms, kStatusSlots) / S::kCtas);  // (a split call has fewer tiles)
    const int cluster = S::kSplit ? g.split : S::kCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(groups * cluster));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, mm_kernel<P>, maps, g);
}

}  // namespace mm
}  // namespace bakron
