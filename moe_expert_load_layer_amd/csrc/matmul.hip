// Grouped matrix product in 8-bit floating point (e4m3) with a power-of-two
// scale for each block of 128:
//   y[m][n] = sum over blocks b of 128:  2^(ca[m][b] + cw[g][n / 128][b] - 254) * sum_k x[m][k] w_g[n][k]
// for the rows m of group g.
//
// The 32x32x64 matrix instruction takes a scale byte for each 32 values of
// either operand, so a block's scale costs no arithmetic: the bytes go to the
// instruction as they are.  It sums its 64 products with about 16 bits (1.5e-5
// relative to the result, measured against 64 bits, at any K) and adds to an
// fp32 accumulator; the bf16 output rounds 100 times coarser.
//
// Weights are the instruction's rows and x its columns, so that a lane ends
// with 4 consecutive n of one row m.  A K step is one block: tiles of BM rows of
// x and BN rows of w, 128 bytes each, go from memory into LDS without passing
// registers (1 KiB an instruction, 8 rows of 128 bytes), two stages deep: the
// next step's loads are in flight while this one's products run, one barrier a
// step.  The 16-byte chunks of an LDS row are exchanged by the row's low 3 bits
// (the loads fetch them in that order), so that 8 lanes reading one chunk of 8
// rows meet 8 different bank groups.
#include "groups.h"

namespace ep {
namespace {

#ifndef EP_BIG
#define EP_BIG 256, 256, 64, 128, 2
#define EP_S2 2
#define EP_S3 3
#endif
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct MatmulArgs {
    const uint8_t *x;
    const uint8_t *xs;
    const int32_t *rows;  // row of x for each output row, times rows_div; null: the row itself
    int32_t rows_div;
    int32_t x_rows;  // rows of x
    const uint8_t *w, *ws, *slot_w, *slot_ws;
    int64_t w_stride, ws_stride, slot_w_stride, slot_ws_stride;
    Groups groups;
    GroupRows where;
    int32_t N, kb, sb;  // columns of y, K blocks, bytes of a row of x scales
    uint16_t *y;
};

// A K step is a block of 128 values; LDS rows are its 128 bytes, their 16-byte
// chunks exchanged by the row's bits 1 to 3: 16 lanes reading one chunk of 16
// rows (256 bytes, a cycle's worth) meet every bank once.
constexpr int kStep = 128;
__device__ __forceinline__ int exchange(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// 32 bytes of LDS row r from chunk c on (c even)
__device__ __forceinline__ i32x8 read_frag(const uint8_t *tile, int r, int c) {
    const u32x4 a = *reinterpret_cast<const u32x4 *>(tile + r * kStep + (exchange(r, c) << 4));
    const u32x4 b = *reinterpret_cast<const u32x4 *>(tile + r * kStep + (exchange(r, c + 1) << 4));
    i32x8 f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        f[i] = (int)a[i];
        f[4 + i] = (int)b[i];
    }
    return f;
}

constexpr int kScaleBlocks = 32;             // blocks whose scales are in LDS at a time
constexpr int kScaleRow = kScaleBlocks + 4;  // rows 9 banks apart

// One K step of a wave: starts the loads of a later stage and multiplies this
// one.  ahead: how far the sources move (0 at the end: the last step is fetched
// again, so that every step has the same count of loads).  xs: scale bytes of
// the block, one a row of x (kScaleRow bytes apart), ws: the scale byte of the
// wave's weights.
template <int BM, int FM, int FN, int kLoads, int kWaves>
__device__ __forceinline__ void matmul_step(const uint8_t *cur, uint8_t *next, const uint8_t *(&src)[kLoads],
                                            int ahead, int wave, int xrow, int wrow, const uint8_t *xs,
                                            const uint8_t *ws, f32x16 (&acc)[FN][FM]) {
    const int l = lane_id(), r = l & 31, h = l >> 5;
    const uint8_t *tx = cur + xrow * kStep, *tw = cur + (BM + wrow) * kStep;
    int sx[FM];
#pragma unroll
    for (int j = 0; j < FM; j++) sx[j] = xs[(xrow + j * 32 + r) * kScaleRow];
    const int sw = ws[0];
#pragma unroll
    for (int s = 0; s < 2; s++) {
        i32x8 fx[FM], fw[FN];
#pragma unroll
        for (int j = 0; j < FM; j++) fx[j] = read_frag(tx, j * 32 + r, s * 4 + h * 2);
#pragma unroll
        for (int i = 0; i < FN; i++) fw[i] = read_frag(tw, i * 32 + r, s * 4 + h * 2);
#pragma unroll
        for (int i = 0; i < FN; i++) {
#pragma unroll
            for (int j = 0; j < FM; j++)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[i], fx[j], acc[i][j], 0, 0, 0, sw, 0,
                                                                            sx[j]);
            // the loads go out between the products: at the step's start they
            // would all wait for the address unit, and the products for them
#pragma unroll
            for (int p = (s * FN + i) * kLoads / (2 * FN); p < (s * FN + i + 1) * kLoads / (2 * FN); p++) {
                load_lds_1k(src[p], next + (wave + p * kWaves) * 1024);
                src[p] += ahead;
            }
        }
    }
}

template <int BM, int BN, int WM, int WN, int kStages>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * kWave, 2) void matmul_kernel(const MatmulArgs A) {
    constexpr int kWavesM = BM / WM, kWaves = kWavesM * (BN / WN), kThreads = kWaves * kWave;
    constexpr int FM = WM / 32, FN = WN / 32;
    constexpr int kLoads = (BM + BN) / 8 / kWaves;  // 1 KiB loads of a wave in a step
    constexpr int kStage = (BM + BN) * kStep;
    constexpr int kWScales = (BN + kScaleBlock - 1) / kScaleBlock;
    static_assert((BM + BN) % (8 * kWaves) == 0 && BM % 8 == 0, "whole loads");
    static_assert(kScaleBlock % WN == 0, "a wave's columns share a scale");
    constexpr int kOut = BM * BN * 2, kRing = kStages * kStage;
    __shared__ __align__(16) uint8_t stages[kRing > kOut ? kRing : kOut];
    __shared__ __align__(16) uint8_t scales[(BM + kWScales) * kScaleRow];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), l = lane_id();
    const int nt = (A.N + BN - 1) / BN;
    const int mt = total_tiles(A.groups, BM);
    // the workgroups of one XCD (consecutive ones go round the 8 XCDs) take
    // consecutive tiles: 4 row tiles by all column tiles, columns last, so that
    // the tiles in flight on an XCD share rows of x and of w in its L2
    const int64_t all = (int64_t)mt * nt;
    const int64_t per = (all + 7) / 8;
    const int64_t at = (int64_t)(blockIdx.x % 8) * per + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per || at >= all) return;
    constexpr int kBand = 4;
    const int band = (int)(at / ((int64_t)kBand * nt));
    const int in = (int)(at - (int64_t)band * kBand * nt), high = min(kBand, mt - band * kBand);
    const int tn = in / high, tile = band * kBand + in % high;
    int g, first;
    if (!find_tile(A.groups, BM, tile, &g, &first)) return;
    const bool tail = g == A.groups.G;  // rows past the last group: zeros
    const int m0 = A.groups.start(g) + (tile - first) * BM;
    const int m1 = tail ? A.groups.M : A.groups.end(g);
    const int n0 = tn * BN;

    const int wm = wave % kWavesM, wn = wave / kWavesM;
    f32x16 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; i++)
#pragma unroll
        for (int j = 0; j < FM; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;

    // x row of output row m, -1: none
    auto source = [&](int m) {
        if (!A.rows) return m;
        const int p = A.rows[m];
        const int r = p < 0 ? -1 : p / A.rows_div;
        return r < A.x_rows ? r : -1;
    };

    if (!tail) {
        int row;
        const bool spare = A.where.spare(g, &row);
        const uint8_t *w = spare ? A.slot_w + row * A.slot_w_stride : A.w + row * A.w_stride;
        const uint8_t *ws = spare ? A.slot_ws + row * A.slot_ws_stride : A.ws + row * A.ws_stride;
        const int64_t row_bytes = (int64_t)A.kb * 128;

        // the 16 bytes that this lane fetches in each of the wave's loads
        const uint8_t *src[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
            const int r = (wave + i * kWaves) * 8 + l / 8, c = exchange(r, l % 8);
            if (r < BM) {
                const int s = source(min(m0 + r, m1 - 1));  // rows past the end repeat the last
                src[i] = A.x + max(s, 0) * row_bytes + c * 16;
            } else {
                src[i] = w + (int64_t)min(n0 + r - BM, A.N - 1) * row_bytes + c * 16;
            }
        }
        // scale bytes of blocks b0 .. b0 + 63: 4 blocks of a row a thread
        auto scale_bytes = [&](int b0) {
            const int nb = min(kScaleBlocks, A.kb - b0);
            for (int i = threadIdx.x; i < BM * (kScaleBlocks / 4); i += kThreads) {
                const int r = i / (kScaleBlocks / 4), b = i % (kScaleBlocks / 4) * 4;
                if (b < nb) {
                    const int s = source(min(m0 + r, m1 - 1));
                    *reinterpret_cast<uint32_t *>(scales + r * kScaleRow + b) =
                        *reinterpret_cast<const uint32_t *>(A.xs + (int64_t)max(s, 0) * A.sb + b0 + b);
                }
            }
            for (int i = threadIdx.x; i < kWScales * kScaleBlocks; i += kThreads) {
                const int j = i / kScaleBlocks, b = i % kScaleBlocks;
                if (b < nb)
                    scales[(BM + j) * kScaleRow + b] =
                        ws[(int64_t)min(n0 / kScaleBlock + j, (A.N - 1) / kScaleBlock) * A.kb + b0 + b];
            }
        };
        // steps go round the ring; kStages - 1 of them are in flight or being read
        const int steps = A.kb;
#pragma unroll
        for (int p = 0; p < kStages - 1; p++)
#pragma unroll
            for (int i = 0; i < kLoads; i++) {
                load_lds_1k(src[i], stages + p * kStage + (wave + i * kWaves) * 1024);
                src[i] += p + 1 < steps ? kStep : 0;
            }
        int slot = 0;
        for (int b0 = 0; b0 < A.kb; b0 += kScaleBlocks) {
            if (b0 > 0) __syncthreads();  // the scales before have been read
            scale_bytes(b0);
            const int s1 = min(b0 + kScaleBlocks, A.kb);
            for (int s = b0; s < s1; s++) {
                // this step's stage is complete once every wave's loads are, and
                // the stage before has been read
                wait_loads_but<(kStages - 2) * kLoads>();
                __syncthreads();
                const uint8_t *xs = scales + (s - b0);
                matmul_step<BM, FM, FN, kLoads, kWaves>(
                    stages + slot * kStage, stages + (slot == 0 ? kStages - 1 : slot - 1) * kStage, src,
                    s + kStages < steps ? kStep : 0, wave, wm * WM, wn * WN, xs,
                    xs + (BM + wn * WN / kScaleBlock) * kScaleRow, acc);
                slot = slot == kStages - 1 ? 0 : slot + 1;
            }
        }
        wait_loads();  // the load that nobody reads
        __syncthreads();
    }

    // The tile goes through LDS as bf16 and out in whole rows, 16 bytes a lane.
    // Chunks of 16 bytes are exchanged by the row, so that 32 rows written at one
    // column meet different banks.
    constexpr int kChunks = BN / 8;
    uint16_t *out = reinterpret_cast<uint16_t *>(stages);
#pragma unroll
    for (int j = 0; j < FM; j++) {
        const int r = wm * WM + j * 32 + (l & 31);
#pragma unroll
        for (int i = 0; i < FN; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int n = wn * WN + i * 32 + e * 8 + (l >> 5) * 4;
                *reinterpret_cast<u32x2 *>(out + r * BN + (((n / 8) ^ (r % kChunks)) * 8 + n % 8)) =
                    u32x2{pack_bf16(acc[i][j][4 * e], acc[i][j][4 * e + 1]),
                          pack_bf16(acc[i][j][4 * e + 2], acc[i][j][4 * e + 3])};
            }
    }
    __syncthreads();
    const bool vec = A.N % 8 == 0 && ((uintptr_t)A.y & 15) == 0;
    for (int i = threadIdx.x; i < BM * kChunks; i += kThreads) {
        const int r = i / kChunks, c = i % kChunks, m = m0 + r, n = n0 + c * 8;
        if (m >= m1 || n >= A.N) continue;
        u32x4 v = *reinterpret_cast<const u32x4 *>(out + r * BN + ((c ^ (r % kChunks)) * 8));
        if (tail || source(m) < 0) v = u32x4{0, 0, 0, 0};
        uint16_t *y = A.y + (int64_t)m * A.N + n;
        if (vec) {
            *reinterpret_cast<u32x4 *>(y) = v;
        } else {
            for (int q = 0; q < 8 && n + q < A.N; q++) y[q] = (uint16_t)(v[q / 2] >> (16 * (q % 2)));
        }
    }
}

template <int BM, int BN, int WM, int WN, int kStages>
hipError_t launch(const MatmulArgs &A, hipStream_t s) {
    constexpr int kThreads = (BM / WM) * (BN / WN) * kWave;
    // every group may end in a part tile, and so may the rows past the last
    const int64_t mt = A.groups.M / BM + A.groups.G + 1;
    const int64_t blocks = ceil_div(mt * ceil_div(A.N, BN), 8) * 8;
    if (blocks > 0xffffffffll / kThreads) return hipErrorInvalidConfiguration;
    matmul_kernel<BM, BN, WM, WN, kStages><<<(uint32_t)blocks, kThreads, 0, s>>>(A);
    return hipGetLastError();
}

}  // namespace

}  // namespace ep

using namespace ep;

extern "C" int ep_grouped_matmul(const ep_grouped_matmul_t *p, ep_stream_t stream) {
    if (!p || p->m < 0 || p->m > kMaxRows || p->n < 1 || p->n > (1 << 24) || p->k < 1 || p->k > (1 << 24) ||
        p->groups < 1 || p->groups > EP_MAX_EXPERTS * 65)
        return EP_ERR_INVALID_ARG;
    if (!p->offsets && p->groups != 1) return EP_ERR_INVALID_ARG;
    if (p->m == 0) return EP_OK;
    const int64_t kb = ceil_div(p->k, kScaleBlock), bytes = p->n * kb * 128, sbytes = ceil_div(p->n, kScaleBlock) * kb;
    MatmulArgs A;
    const bool slots = p->slot_w.data && p->slot_w.scale;
    if (!layout_groups(p->layout, p->groups, slots, &A.where)) return EP_ERR_INVALID_ARG;
    if (!p->x || !p->x_scale || !p->w.data || !p->w.scale || !p->y) return EP_ERR_INVALID_ARG;
    if (!is_aligned(p->x, 16) || !is_aligned(p->x_scale, 4) || !is_aligned(p->w.data, 16) || p->w.stride % 16 != 0 ||
        !is_aligned(p->y, 2) || !is_aligned(p->offsets, 4) || !is_aligned(p->rows, 4))
        return EP_ERR_INVALID_ARG;
    if (p->groups > 1 && (p->w.stride < bytes || p->w.scale_stride < sbytes)) return EP_ERR_INVALID_ARG;
    if (slots && (!is_aligned(p->slot_w.data, 16) || p->slot_w.stride % 16 != 0 ||
                  (p->layout && p->layout->num_spare > 1 &&
                   (p->slot_w.stride < bytes || p->slot_w.scale_stride < sbytes))))
        return EP_ERR_INVALID_ARG;
    if (p->rows ? (p->rows_div < 1 || p->x_rows < 1) : p->x_rows < p->m) return EP_ERR_INVALID_ARG;
    if (p->x_rows > kMaxRows) return EP_ERR_INVALID_ARG;
    A.x = static_cast<const uint8_t *>(p->x);
    A.xs = p->x_scale;
    A.rows = p->rows;
    A.rows_div = p->rows_div;
    A.x_rows = (int32_t)p->x_rows;
    A.w = static_cast<const uint8_t *>(p->w.data);
    A.ws = p->w.scale;
    A.w_stride = p->w.stride;
    A.ws_stride = p->w.scale_stride;
    A.slot_w = static_cast<const uint8_t *>(p->slot_w.data);
    A.slot_ws = p->slot_w.scale;
    A.slot_w_stride = p->slot_w.stride;
    A.slot_ws_stride = p->slot_w.scale_stride;
    A.groups = Groups{p->offsets, p->groups, (int32_t)p->m};
    A.N = (int32_t)p->n;
    A.kb = (int32_t)kb;
    A.sb = (int32_t)ep_scale_stride(p->k);
    A.y = static_cast<uint16_t *>(p->y);
    const hipStream_t s = to_stream(stream);
    const int64_t rows = p->m / p->groups;  // of a group, on average
    if (rows >= 384) return rc_of(launch<EP_BIG>(A, s));
    if (rows >= 64) return rc_of(launch<128, 128, 64, 64, EP_S2>(A, s));
    return rc_of(launch<32, 128, 32, 32, EP_S3>(A, s));
}
