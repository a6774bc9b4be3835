// mm_api.cu -- the C ABI of the products over packed rows and of the 8-bit
// block quantiser (include/bakron.h): argument checks, tensor maps and the
// choice of kernel variant.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "common.cuh"
#include "kernels.cuh"
#include "mm.cuh"
#include "mm_groups.h"

using namespace bakron;

using namespace bakron::mm;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
int64_t ceil64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Largest extent of a dimension, tensor-map strides and tile counts.
constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 39;  // bytes; tensor maps take strides below 2^40
constexpr int64_t kMaxTiles = (int64_t)1 << 30;

// Stages (64 operand columns, or packed rows where those are the contraction; 32
// from three bf16 parts) that one accumulator sums before it is added to FP32
// registers.  The tensor cores truncate, so the sums of an FP32 result are kept
// to 512 products: 4e-7 of the result for 4096 random products, against 2e-7 at
// 256 and 2e-6 at 2048.  A 16-bit result rounds a thousand times more.
constexpr int kChunkF32 = 8, kChunk16 = 16;

std::mutex g_mu;
// What a configured device holds at once: SMs, and clusters of p CTAs (one CTA an
// SM).  Clusters stay within a part of the chip, so that 15 of 8 and 33 of 4 CTAs
// run on 148 SMs; one more waits for a whole round.
struct Device {
    int sms;
    int clusters[9];
};
Device g_devices[64] = {};

// Kernel attributes once per device; the device's limits.
cudaError_t configure_device(Device &device)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_devices[dev].sms) {
        Device d = {};
        if ((e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if ((e = configure_rows()) != cudaSuccess) return e;
        if ((e = configure_eight()) != cudaSuccess) return e;
        if ((e = configure_outer()) != cudaSuccess) return e;
        for (int p = 1; p <= 8; p *= 2)
            if ((e = clusters_that_fit(p, d.clusters[p])) != cudaSuccess) return e;
        g_devices[dev] = d;
    }
    device = g_devices[dev];
    return cudaSuccess;
}

// Workspace and time limit.  The status block is cleared here unless the call's
// first kernel writes all of it.
bakron_status_t begin(void *ws, size_t ws_bytes, size_t need, bool clear, cudaStream_t stream, Args &g)
{
    if (!ws || ws_bytes < need) return BAKRON_ERR_WORKSPACE;
    if (!aligned16(ws)) return BAKRON_ERR_ALIGNMENT;
    int ms = 0;
    if (!default_timeout_ms(ms)) return BAKRON_ERR_INVALID_ARG;
    g.timeout_ns = (uint64_t)ms * 1000000ull;
    g.st = (DeviceStatus *)ws;
    g.split = 1;
    if (clear && cudaMemsetAsync(ws, 0, kStatusBytes, stream) != cudaSuccess) return BAKRON_ERR_CUDA;
    return BAKRON_OK;
}

bool type16(int32_t t) { return t == BAKRON_BF16 || t == BAKRON_F16; }
int64_t type_size(int32_t t) { return t == BAKRON_F32 ? 4 : 2; }
bool dim_ok(int64_t x) { return x >= 1 && x <= kMaxDim; }

// A row-major operand read by TMA: rows of `cols` elements, `stride` elements apart.
bakron_status_t check_operand(const void *p, int64_t cols, int64_t stride, int64_t size)
{
    if (!p || stride < cols) return BAKRON_ERR_INVALID_ARG;
    if (!aligned16(p) || (stride * size) % 16) return BAKRON_ERR_ALIGNMENT;
    return stride * size > kMaxStride ? BAKRON_ERR_INVALID_ARG : BAKRON_OK;
}

// Instruction descriptor without M and N: FP32 accumulator, operand types, transposes.
uint32_t idesc16(int32_t type, bool a_columns, bool b_columns)
{
    const uint32_t t = type == BAKRON_BF16 ? 1u : 0u;
    return (1u << 4) | (t << 7) | (t << 10) | ((uint32_t)a_columns << 15) | ((uint32_t)b_columns << 16);
}
constexpr uint32_t kIdescE4m3 = 1u << 4;

CUtensorMapDataType map_type(int32_t type)
{
    return type == BAKRON_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// Packed rows (rows x cols) / expert matrices (experts x rows x cols).
bool map2(CUtensorMap *m, CUtensorMapDataType t, int64_t size, const void *p, int64_t cols, int64_t rows,
          int64_t stride, uint32_t box_cols, uint32_t box_rows)
{
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)(stride * size)};
    const uint32_t box[2] = {box_cols, box_rows};
    return encode_tensor_map(m, t, 2, p, dims, strides, box);
}
bool map3(CUtensorMap *m, CUtensorMapDataType t, int64_t size, const void *p, int64_t cols, int64_t rows,
          int64_t stride, int64_t planes, int64_t plane_stride, uint32_t box_cols, uint32_t box_rows)
{
    const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)planes};
    const uint64_t strides[2] = {(uint64_t)(stride * size), (uint64_t)(plane_stride * size)};
    const uint32_t box[3] = {box_cols, box_rows, 1};
    return encode_tensor_map(m, t, 3, p, dims, strides, box);
}

// CTAs per tile of a call with short groups: while the tiles would leave half
// the SMs idle the contraction is split, down to two stages a CTA (eight CTAs
// are the most a cluster holds on every device).
int split_of(int64_t tiles, int64_t stages, const Device &device)
{
    int s = 1;
    while (s < 8 && tiles <= device.clusters[2 * s] && stages >= 4 * s) s *= 2;
    return s;
}

// Tile of an 8-bit product with the packed rows on D's rows, and the CTAs that
// share a tile's contraction: whichever needs the least time in whole rounds of
// tiles over the SMs, at the clocks measured per 128-long step of the
// contraction (8192 x 14336 x 4096) and for a join of parts.  Half of a group's
// last tile is empty on average.  A tile's first steps and its stores are not
// counted: for 4100 rows of 16 experts, 4096 x 2048, the estimate is 47 us and 68
// to 77 are measured.
Variant eight_variant(int64_t rows, int64_t n, int64_t k, int64_t experts, const Device &device, int &split)
{
    const int sms = device.sms;
    struct Shape { Variant v; int64_t m, w, ctas; double clocks; };
    const Shape shapes[] = {{kEightPair256, 256, 256, 2, 1000}, {kEightPair128, 256, 128, 2, 600},
                            {kEightOne128, 128, 128, 1, 630}};
    const double join = 1800;
    const int64_t steps = ceil64(k, 128);
    Variant best = kEightPair256;
    double least = 1e300;
    split = 1;
    for (const Shape &s : shapes) {
        const double row_tiles_mean = experts == 1 ? (double)ceil64(rows, s.m) : (double)rows / s.m + 0.5 * experts;
        const double mean = row_tiles_mean * ceil64(n, s.w);
        const int64_t most = row_tiles(rows, experts, s.m) * ceil64(n, s.w);
        for (int p = 1; p <= (s.ctas == 1 ? 8 : 1); p *= 2) {
            if (p > 1 && (most > device.clusters[p] || steps < 2 * p)) break;
            const double cost = ceil(mean * s.ctas * p / sms) * ceil64(steps, p) * s.clocks + (p > 1 ? join : 0);
            if (cost < least) {
                least = cost;
                best = s.v;
                split = p;
            }
        }
    }
    return best;
}

// Products over the packed rows of a group: tiles of CTA pairs (256 x 256, from
// three parts 256 x 128), or of one CTA (128 x 128), whose contraction up to eight
// may share; whichever needs the least time, as above, at the clocks measured per
// `step` rows of the contraction (pair 570, one 510 per 64 rows of 16 bits; 1050
// and 1250 per 32 rows of three parts), for a tile's stores and for a join.
// Measured, pairs and one CTA a tile: dw 2048 x 2048, 2 experts, 8192 rows 59 and
// 88 us; 76 x 3788, 23 experts, 1191 rows 43 and 25 us; Gram factors at d = 1024
// of 4 experts from 4096 fp32 rows 56 and 39 us, d = 1612 of one expert from 5844
// rows 114 and 133 us; shared by eight: dw 256 x 256 from 16384 rows 82 and 17 us.
// `tiles` and `split` are set for the tile taken.
bool outer_pair(int64_t rows, int64_t experts, int64_t pair_tiles, int64_t one_tiles, int64_t step, double pair_clocks,
                double one_clocks, const Device &device, int64_t &tiles, int &split)
{
    const int sms = device.sms;
    const double store = 2500, join = 1800;
    const int64_t steps = ceil64(ceil64(rows, experts), step);
    double least = ceil64(2 * pair_tiles, sms) * (steps * pair_clocks + 2 * store);
    bool pair = true;
    tiles = pair_tiles;
    split = 1;
    for (int p = 1; p <= 8; p *= 2) {
        if (p > 1 && (one_tiles > device.clusters[p] || steps < 2 * p)) break;
        const double cost = ceil64(one_tiles * p, sms) * (ceil64(steps, p) * one_clocks + store / p) + (p > 1 ? join : 0);
        if (cost < least) {
            least = cost;
            pair = false;
            tiles = one_tiles;
            split = p;
        }
    }
    return pair;
}

// y[t, :] = x[t, :] w_e^T (columns = false: contraction over w's columns) or
// x[t, :] w_e (columns = true: over w's rows).
bakron_status_t grouped_rows(bool columns, const void *x, int32_t type, int64_t ldx, const void *w, int64_t ldw,
                             int64_t w_stride, const int32_t *offsets, int64_t experts, void *y, int32_t y_type,
                             int64_t ldy, int64_t rows, int64_t n, int64_t k, void *ws, size_t ws_bytes,
                             bakron_stream_t stream)
{
    const int64_t in = columns ? n : k, out = columns ? k : n;  // widths of x and y
    if (rows < 0 || rows > kMaxDim || !dim_ok(n) || !dim_ok(k) || experts < 1 || experts > kMaxExperts)
        return BAKRON_ERR_INVALID_ARG;
    if (!type16(type) || (y_type != type && y_type != BAKRON_F32) || !offsets) return BAKRON_ERR_INVALID_ARG;
    if (((uintptr_t)offsets & 3u) || w_stride < n * ldw) return BAKRON_ERR_INVALID_ARG;
    bakron_status_t s = check_operand(w, k, ldw, 2);
    if (s == BAKRON_OK && w_stride * 2 > kMaxStride) s = BAKRON_ERR_INVALID_ARG;
    if (s == BAKRON_OK && (w_stride * 2) % 16) s = BAKRON_ERR_ALIGNMENT;
    if (s == BAKRON_OK && rows) s = check_operand(x, in, ldx, 2);
    if (s != BAKRON_OK) return s;
    if (rows && (!y || ldy < out)) return BAKRON_ERR_INVALID_ARG;
    if (rows && !aligned16(y)) return BAKRON_ERR_ALIGNMENT;
    // Tiles of 64 packed rows when the groups are short on average: the same
    // weight tile then takes half the stage bytes, so twice the weights are in
    // flight.  Beyond that tiles of CTA pairs, which nothing splits: one matrix of
    // 4096 x 4096 takes 10.9 us with 48 rows and 20.2 with 49, 30 with 1000.
    const bool small = rows <= 48 * experts;
    const int64_t bn = small ? 64 : 256;
    const int64_t tiles = row_tiles(rows, experts, bn) * ceil64(out, 128);
    if (tiles > kMaxTiles) return BAKRON_ERR_INVALID_ARG;
    Device device;
    if (configure_device(device) != cudaSuccess) return BAKRON_ERR_CUDA;
    Args g{};
    if ((s = begin(ws, ws_bytes, kStatusBytes, !rows, (cudaStream_t)stream, g)) != BAKRON_OK) return s;
    if (!rows) return BAKRON_OK;
    g.offsets = offsets;
    g.experts = (int)experts;
    g.rows = (int)rows;
    g.a_total = (int)out;
    g.k_total = (int)in;
    g.out = y;
    g.ldo = ldy;
    g.out_type = y_type;
    g.turn = y_type != BAKRON_F32 && ldy % 8 == 0;
    if (small) g.split = split_of(tiles, ceil64(in, 64), device);
    g.idesc = idesc16(type, columns, false);
    g.chunk = y_type == BAKRON_F32 ? kChunkF32 : kChunk16;
    Maps m;
    const CUtensorMapDataType t = map_type(type);
    if (!map3(&m.a, t, 2, w, k, n, ldw, experts, w_stride, 64, columns ? 64 : 128) ||
        !map2(&m.b, t, 2, x, in, rows, ldx, 64, small ? 32 : 64) ||
        !map2(&m.b2, t, 2, x, in, rows, ldx, 64, small ? 64 : 128))
        return BAKRON_ERR_CUDA;
    const Variant v = columns ? (small ? kRowsDx64 : kRowsDx256) : (small ? kRows64 : kRows256);
    if (launch_rows(v, m, g, tiles, device.sms, (cudaStream_t)stream) != cudaSuccess) return BAKRON_ERR_CUDA;
    return BAKRON_OK;
}

// The self-test's problem: one or two tiles of 256 x 256 for one CTA pair, each of
// two accumulator chunks, behind the status block.
struct AbortLayout {
    static constexpr int64_t rows = 256, n = 512, k = 2 * 64 * kChunk16;
    static constexpr size_t y = kAlign, x = y + rows * n * 2, w = x + rows * k * 2, total = w + n * k * 2;
};

struct GramGroupedLayout {
    int64_t ld;
    size_t status, planes, total;
    void compute(int32_t type, int64_t rows, int64_t d)
    {
        ld = ceil64(d, 8) * 8;
        status = 0;
        planes = kAlign;
        total = align_up(planes + (type == BAKRON_F32 ? (size_t)3 * rows * ld * 2 : 0));
    }
};

}  // namespace

extern "C" {

bakron_status_t bakron_quantize_blocks(const void *x_dev, int32_t x_type, int64_t batch, int64_t rows, int64_t cols,
                                       int64_t x_batch_stride, int64_t x_row_stride, int32_t block_rows,
                                       uint8_t *q_dev, int64_t q_row_stride, float *scales_dev, void *ws_dev,
                                       size_t ws_bytes, bakron_stream_t stream)
{
    if (batch < 0 || rows < 0 || batch > kMaxDim || rows > kMaxDim || !dim_ok(cols)) return BAKRON_ERR_INVALID_ARG;
    if (x_type != BAKRON_F32 && !type16(x_type)) return BAKRON_ERR_INVALID_ARG;
    if (block_rows != 1 && block_rows != 128) return BAKRON_ERR_INVALID_ARG;
    if (x_row_stride < cols || q_row_stride < cols || x_batch_stride < 0) return BAKRON_ERR_INVALID_ARG;
    if (batch * ceil64(rows, block_rows) > kMaxDim) return BAKRON_ERR_INVALID_ARG;
    const int64_t blocks = batch * ceil64(rows, block_rows) * ceil64(cols, 128);
    if (block_rows == 128 && blocks > kMaxTiles) return BAKRON_ERR_INVALID_ARG;
    if (blocks && (!x_dev || !q_dev || !scales_dev)) return BAKRON_ERR_INVALID_ARG;
    if (!aligned16(x_dev) || !aligned16(q_dev) || !aligned16(scales_dev) || q_row_stride % 16)
        return BAKRON_ERR_ALIGNMENT;
    Args g{};
    const bakron_status_t s = begin(ws_dev, ws_bytes, kStatusBytes, true, (cudaStream_t)stream, g);
    if (s != BAKRON_OK || !blocks) return s;
    const QuantArgs a{x_dev, x_type, batch, rows, cols, x_batch_stride, x_row_stride, block_rows,
                      q_dev, q_row_stride, scales_dev, g.st};
    return launch_quantize(a, (cudaStream_t)stream) == cudaSuccess ? BAKRON_OK : BAKRON_ERR_CUDA;
}

bakron_status_t bakron_matmul_blocks(const uint8_t *x_dev, int64_t x_row_stride, const float *x_scales_dev,
                                     const uint8_t *w_dev, int64_t w_row_stride, int64_t w_expert_stride,
                                     const float *w_scales_dev, int32_t w_scale_rows, const int32_t *offsets_dev,
                                     int64_t experts, void *y_dev, int32_t y_type, int64_t y_row_stride, int64_t rows,
                                     int64_t n, int64_t k, void *ws_dev, size_t ws_bytes, bakron_stream_t stream)
{
    if (rows < 0 || rows > kMaxDim || !dim_ok(n) || !dim_ok(k) || experts < 1 || experts > kMaxExperts)
        return BAKRON_ERR_INVALID_ARG;
    if (!offsets_dev && experts != 1) return BAKRON_ERR_INVALID_ARG;
    if (y_type != BAKRON_F32 && !type16(y_type)) return BAKRON_ERR_INVALID_ARG;
    if (w_scale_rows != 1 && w_scale_rows != 128) return BAKRON_ERR_INVALID_ARG;
    if (!w_scales_dev || ((uintptr_t)offsets_dev & 3u) || w_expert_stride < n * w_row_stride)
        return BAKRON_ERR_INVALID_ARG;
    bakron_status_t s = check_operand(w_dev, k, w_row_stride, 1);
    if (s == BAKRON_OK && w_expert_stride > kMaxStride) s = BAKRON_ERR_INVALID_ARG;
    if (s == BAKRON_OK && w_expert_stride % 16) s = BAKRON_ERR_ALIGNMENT;
    if (s == BAKRON_OK && rows) s = check_operand(x_dev, k, x_row_stride, 1);
    if (s != BAKRON_OK) return s;
    if (rows && (!x_scales_dev || !y_dev || y_row_stride < n)) return BAKRON_ERR_INVALID_ARG;
    if (!aligned16(w_scales_dev) || (rows && (!aligned16(y_dev) || !aligned16(x_scales_dev))))
        return BAKRON_ERR_ALIGNMENT;
    // Packed rows on the tile's columns (64 at a time) while the groups are
    // short, on its 128 rows beyond that.
    const bool small = rows <= 32 * experts;
    if ((small ? row_tiles(rows, experts, 64) : row_tiles(rows, experts, 128)) * ceil64(n, 128) > kMaxTiles)
        return BAKRON_ERR_INVALID_ARG;
    Device device;
    if (configure_device(device) != cudaSuccess) return BAKRON_ERR_CUDA;
    int split = 1;
    const Variant v = small ? kEightB64 : eight_variant(rows, n, k, experts, device, split);
    const int64_t m = small ? 64 : v == kEightOne128 ? 128 : 256, bn = v == kEightPair256 ? 256 : 128;
    const int64_t tiles = row_tiles(rows, experts, m) * ceil64(n, bn);
    Args g{};
    if ((s = begin(ws_dev, ws_bytes, kStatusBytes, !rows, (cudaStream_t)stream, g)) != BAKRON_OK) return s;
    if (!rows) return BAKRON_OK;
    g.offsets = offsets_dev;
    g.experts = (int)experts;
    g.rows = (int)rows;
    g.a_total = (int)n;
    g.b_total = (int)n;
    g.k_total = (int)k;
    g.out = y_dev;
    g.ldo = y_row_stride;
    g.out_type = y_type;
    g.idesc = kIdescE4m3;
    g.x_steps = x_scales_dev;
    g.w_steps = w_scales_dev;
    g.w_step_rows = w_scale_rows;
    g.split = small ? split_of(tiles, ceil64(k, 128), device) : split;
    Maps maps;
    const CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    CUtensorMap *xm = small ? &maps.b : &maps.a, *wm = small ? &maps.a : &maps.b;
    if (!map2(xm, t, 1, x_dev, k, rows, x_row_stride, 128, small ? 32 : 128) ||
        (small && !map2(&maps.b2, t, 1, x_dev, k, rows, x_row_stride, 128, 64)) ||
        !map3(wm, t, 1, w_dev, k, n, w_row_stride, experts, w_expert_stride, 128,
              small ? 128 : (uint32_t)(bn * 128 / m)))
        return BAKRON_ERR_CUDA;
    if (launch_eight(v, maps, g, tiles, device.sms, (cudaStream_t)stream) !=
        cudaSuccess)
        return BAKRON_ERR_CUDA;
    return BAKRON_OK;
}

bakron_status_t bakron_matmul_grouped(const void *x_dev, int32_t type, int64_t x_row_stride, const void *w_dev,
                                      int64_t w_row_stride, int64_t w_expert_stride, const int32_t *offsets_dev,
                                      int64_t experts, void *y_dev, int32_t y_type, int64_t y_row_stride, int64_t rows,
                                      int64_t n, int64_t k, void *ws_dev, size_t ws_bytes, bakron_stream_t stream)
{
    return grouped_rows(false, x_dev, type, x_row_stride, w_dev, w_row_stride, w_expert_stride, offsets_dev, experts,
                        y_dev, y_type, y_row_stride, rows, n, k, ws_dev, ws_bytes, stream);
}

bakron_status_t bakron_matmul_grouped_dx(const void *dy_dev, int32_t type, int64_t dy_row_stride, const void *w_dev,
                                         int64_t w_row_stride, int64_t w_expert_stride, const int32_t *offsets_dev,
                                         int64_t experts, void *dx_dev, int32_t dx_type, int64_t dx_row_stride,
                                         int64_t rows, int64_t n, int64_t k, void *ws_dev, size_t ws_bytes,
                                         bakron_stream_t stream)
{
    return grouped_rows(true, dy_dev, type, dy_row_stride, w_dev, w_row_stride, w_expert_stride, offsets_dev, experts,
                        dx_dev, dx_type, dx_row_stride, rows, n, k, ws_dev, ws_bytes, stream);
}

bakron_status_t bakron_matmul_grouped_dw(const void *dy_dev, int32_t type, int64_t dy_row_stride, const void *x_dev,
                                         int64_t x_row_stride, const int32_t *offsets_dev, int64_t experts,
                                         void *dw_dev, int32_t dw_type, int64_t rows, int64_t n, int64_t k,
                                         void *ws_dev, size_t ws_bytes, bakron_stream_t stream)
{
    if (rows < 0 || rows > kMaxDim || !dim_ok(n) || !dim_ok(k) || experts < 1 || experts > kMaxExperts)
        return BAKRON_ERR_INVALID_ARG;
    if (!type16(type) || (dw_type != type && dw_type != BAKRON_F32) || !offsets_dev || !dw_dev)
        return BAKRON_ERR_INVALID_ARG;
    if ((uintptr_t)offsets_dev & 3u) return BAKRON_ERR_INVALID_ARG;
    bakron_status_t s = BAKRON_OK;
    if (rows) s = check_operand(dy_dev, n, dy_row_stride, 2);
    if (s == BAKRON_OK && rows) s = check_operand(x_dev, k, x_row_stride, 2);
    if (s != BAKRON_OK) return s;
    if (!aligned16(dw_dev)) return BAKRON_ERR_ALIGNMENT;
    const int64_t one_tiles = experts * ceil64(n, 128) * ceil64(k, 128);
    if (one_tiles > kMaxTiles) return BAKRON_ERR_INVALID_ARG;
    Device device;
    if (configure_device(device) != cudaSuccess) return BAKRON_ERR_CUDA;
    Args g{};
    if ((s = begin(ws_dev, ws_bytes, kStatusBytes, !rows, (cudaStream_t)stream, g)) != BAKRON_OK) return s;
    if (!rows) {
        const size_t bytes = (size_t)experts * n * k * type_size(dw_type);
        return cudaMemsetAsync(dw_dev, 0, bytes, (cudaStream_t)stream) == cudaSuccess ? BAKRON_OK : BAKRON_ERR_CUDA;
    }
    g.offsets = offsets_dev;
    g.experts = (int)experts;
    g.rows = (int)rows;
    g.a_total = (int)n;
    g.b_total = (int)k;
    g.out = dw_dev;
    g.ldo = k;
    g.out_expert_stride = n * k;
    g.out_type = dw_type;
    g.idesc = idesc16(type, true, true);
    g.chunk = dw_type == BAKRON_F32 ? kChunkF32 : kChunk16;
    Maps m;
    const CUtensorMapDataType t = map_type(type);
    if (!map3(&m.a, t, 2, dy_dev, n, rows, dy_row_stride, 1, rows * dy_row_stride, 64, 64) ||
        !map3(&m.b, t, 2, x_dev, k, rows, x_row_stride, 1, rows * x_row_stride, 64, 64))
        return BAKRON_ERR_CUDA;
    int64_t tiles = 0;
    const bool pair = outer_pair(rows, experts, experts * ceil64(n, 256) * ceil64(k, 256), one_tiles, 64, 570, 510, device,
                                 tiles, g.split);
    if (launch_outer(pair ? kOuterPair : kOuterOne, m, g, tiles, device.sms, (cudaStream_t)stream) != cudaSuccess)
        return BAKRON_ERR_CUDA;
    return BAKRON_OK;
}

size_t bakron_gram_grouped_workspace_size(int32_t type, int64_t rows, int64_t d)
{
    if ((type != BAKRON_F32 && !type16(type)) || rows < 0 || rows > kMaxDim || !dim_ok(d)) return 0;
    GramGroupedLayout L;
    L.compute(type, rows, d);
    return L.total;
}

bakron_status_t bakron_gram_grouped(const void *X_dev, int32_t type, int64_t x_row_stride, const int32_t *offsets_dev,
                                    int64_t experts, float damping, float *A_dev, int64_t rows, int64_t d,
                                    void *ws_dev, size_t ws_bytes, bakron_stream_t stream)
{
    if (rows < 0 || rows > kMaxDim || !dim_ok(d) || experts < 1 || experts > kMaxExperts)
        return BAKRON_ERR_INVALID_ARG;
    if ((type != BAKRON_F32 && !type16(type)) || !offsets_dev || !A_dev || ((uintptr_t)offsets_dev & 3u))
        return BAKRON_ERR_INVALID_ARG;
    if (!(damping >= 0.f) || !isfinite(damping)) return BAKRON_ERR_INVALID_ARG;
    bakron_status_t s = BAKRON_OK;
    if (rows && type == BAKRON_F32) {
        // read by plain loads: any row stride
        if (!X_dev || x_row_stride < d) return BAKRON_ERR_INVALID_ARG;
        if (!aligned16(X_dev)) return BAKRON_ERR_ALIGNMENT;
    } else if (rows) {
        s = check_operand(X_dev, d, x_row_stride, 2);
    }
    if (s != BAKRON_OK) return s;
    if (!aligned16(A_dev)) return BAKRON_ERR_ALIGNMENT;
    const int64_t mt = ceil64(d, 128), one_tiles = experts * (mt * (mt + 1) / 2);
    if (mt > 16384 || one_tiles > kMaxTiles) return BAKRON_ERR_INVALID_ARG;
    GramGroupedLayout L;
    L.compute(type, rows, d);
    Device device;
    if (configure_device(device) != cudaSuccess) return BAKRON_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    Args g{};
    if ((s = begin(ws_dev, ws_bytes, L.total, !rows, st, g)) != BAKRON_OK) return s;
    if (!rows)
        return cudaMemsetAsync(A_dev, 0, (size_t)experts * d * d * 4, st) == cudaSuccess ? BAKRON_OK : BAKRON_ERR_CUDA;
    g.offsets = offsets_dev;
    g.experts = (int)experts;
    g.rows = (int)rows;
    g.a_total = (int)d;
    g.b_total = (int)d;
    g.out = A_dev;
    g.ldo = d;
    g.out_expert_stride = d * d;
    g.out_type = BAKRON_F32;
    g.chunk = kChunkF32;
    Maps m;
    if (type == BAKRON_F32) {
        uint16_t *planes = (uint16_t *)((char *)ws_dev + L.planes);
        if (launch_split_three((const float *)X_dev, rows, d, x_row_stride, planes, L.ld, st) != cudaSuccess)
            return BAKRON_ERR_CUDA;
        g.idesc = idesc16(BAKRON_BF16, true, true);
        if (!map3(&m.a, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, planes, d, rows, L.ld, 3, rows * L.ld, 64, 32))
            return BAKRON_ERR_CUDA;
    } else {
        g.idesc = idesc16(type, true, true);
        if (!map3(&m.a, map_type(type), 2, X_dev, d, rows, x_row_stride, 1, rows * x_row_stride, 64, 64))
            return BAKRON_ERR_CUDA;
    }
    m.b = m.a;
    m.b2 = m.a;
    // pairs' tiles of a lower triangle: 256 rows, 256 (from three parts 128) columns
    const int64_t mp = ceil64(d, 256), triangle = mp * (mp + 1) / 2;
    int64_t tiles = 0;
    Variant v;
    if (type == BAKRON_F32)
        v = outer_pair(rows, experts, experts * (2 * triangle - (mt & 1)), one_tiles, 32, 1050, 1250, device, tiles, g.split)
                ? kGramThreePair : kGramThreeOne;
    else
        v = outer_pair(rows, experts, experts * triangle, one_tiles, 64, 570, 510, device, tiles, g.split)
                ? kGramPair : kGramOne;
    if (launch_outer(v, m, g, tiles, device.sms, st) != cudaSuccess)
        return BAKRON_ERR_CUDA;
    return launch_gram_damp(A_dev, d, (int)experts, damping, g.st, st) == cudaSuccess ? BAKRON_OK : BAKRON_ERR_CUDA;
}

size_t bakron_selftest_rows_abort_workspace_size(void) { return AbortLayout::total; }

bakron_status_t bakron_selftest_rows_abort(int32_t timeout_ms, int32_t way, void *ws_dev, size_t ws_bytes,
                                           bakron_stream_t stream)
{
    using L = AbortLayout;
    if (timeout_ms < 1 || timeout_ms > 10000 || way < 1 || way > 2) return BAKRON_ERR_INVALID_ARG;
    Args g{};
    Device device;
    Maps m;
    cudaStream_t st = (cudaStream_t)stream;
    const bakron_status_t s = begin(ws_dev, ws_bytes, L::total, false, st, g);
    if (s != BAKRON_OK) return s;
    if (configure_device(device) != cudaSuccess) return BAKRON_ERR_CUDA;
    char *ws = (char *)ws_dev;
    if (cudaMemsetAsync(ws + L::y, 0xff, L::x - L::y, st) != cudaSuccess ||
        cudaMemsetAsync(ws + L::x, 0, L::total - L::x, st) != cudaSuccess)
        return BAKRON_ERR_CUDA;
    g.timeout_ns = (uint64_t)timeout_ms * 1000000ull;
    g.experts = 1;
    g.rows = (int)L::rows;
    g.a_total = (int)(way == 1 ? L::n : L::n / 2);
    g.k_total = (int)L::k;
    g.out = ws + L::y;
    g.ldo = L::n;
    g.out_type = BAKRON_BF16;
    g.turn = 1;
    g.idesc = idesc16(BAKRON_BF16, false, false);
    g.chunk = kChunk16;
    g.gives_up = way;
    const CUtensorMapDataType t = map_type(BAKRON_BF16);
    if (!map3(&m.a, t, 2, ws + L::w, L::k, L::n, L::k, 1, L::n * L::k, 64, 128) ||
        !map2(&m.b, t, 2, ws + L::x, L::k, L::rows, L::k, 64, 64) ||
        !map2(&m.b2, t, 2, ws + L::x, L::k, L::rows, L::k, 64, 128))
        return BAKRON_ERR_CUDA;
    return launch_rows(kRowsAbort, m, g, 1, device.sms, st) == cudaSuccess ? BAKRON_OK : BAKRON_ERR_CUDA;
}

}  // extern "C"
