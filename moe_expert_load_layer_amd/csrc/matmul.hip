// Grouped matrix product in 8-bit floating point (e4m3) with a power-of-two
// scale for each block of 128:
//   y[m][n] = sum over blocks b of 128:  2^(ca[m][b] + cw[g][n / 128][b] - 254) * sum_k x[m][k] w_g[n][k]
// for the rows m of group g.
//
// The 32x32x64 matrix instruction takes a scale byte for each 32 values of
// either operand, so a block's scale costs no arithmetic: the bytes go to the
// instruction as they are.  It aligns every 8 products to their largest, drops
// what lies below 2^-13 of it (1.5e-5 of a result as a rule, measured against 64
// bits, at any K) and adds to an fp32 accumulator; the bf16 output rounds 100
// times coarser.
//
// Weights are the instruction's rows and x its columns, so that a lane ends
// with 4 consecutive n of one row m, and two lanes exchange them into 16-byte
// stores.  Tiles of BM rows of x and BN rows of w go from memory into a ring of
// LDS stages without passing registers, 64 values of K at a time (1 KiB an
// instruction, 16 rows of 64 bytes).
//
// What bounds such a loop is waiting in step: past one barrier all waves first
// read LDS, then all multiply.  So a step's operands are read into registers
// during the step before, each right after the products that free its
// registers, and the loads into LDS go out between the products too (issued
// together they wait for the address unit: 8 % slower).  At 65536 x 4096 x 4096
// the matrix pipes are busy 57 % of the cycles, at 1.8 GHz (the card lowers its
// clock from 2.4 under this load): 2.0 PFLOP/s alone, 1.9 in a row.
#include "groups.h"

namespace ep {
namespace {

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

// A K step is 64 values, half a block; LDS rows are its 64 bytes, their 16-byte
// chunks exchanged by the row's bits 2 and 3: 16 lanes reading one chunk of 16
// rows (256 bytes, a cycle's worth) meet every bank once.
constexpr int kStep = 64;
constexpr int kParts = kScaleBlock / kStep;
constexpr int kScaleBlocks = 32;             // blocks of a chunk of scales; two chunks are in LDS
constexpr int kScaleRow = kScaleBlocks + 4;  // rows 9 banks apart

__device__ __forceinline__ int exchange(int row, int chunk) { return chunk ^ ((row >> 2) & 3); }

// this lane's 32 bytes of LDS row r (lanes 0 .. 31 the first half of its 64)
__device__ __forceinline__ i32x8 read_frag(const uint8_t *tile, int r) {
    const int c = lane_id() >> 5 << 1;
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

// One K step of a wave: multiplies the operands fx, fw with the scales sx, sw
// while the next step's are read from `next` (nx, ns; fw right after the
// products that use it) and a later step's loads go into `fill`.  The empty asm
// statements hold the products in this order: together at the front, they would
// leave nothing to wait behind.
template <int BM, int FM, int FN, int kLoads, int kWaves>
__device__ __forceinline__ void matmul_step(const uint8_t *next, uint8_t *fill, const uint8_t *(&src)[kLoads],
                                            int ahead, int wave, int xrow, int wrow, const uint8_t *xs,
                                            const uint8_t *ws, const i32x8 (&fx)[FM], i32x8 (&nx)[FM],
                                            i32x8 (&fw)[FN], const int (&sx)[FM], int (&ns)[FM], int &sw,
                                            f32x16 (&acc)[FN][FM]) {
    const int r = lane_id() & 31;
    const int nsw = ws[0];
#pragma unroll
    for (int i = 0; i < FN; i++) {
        asm volatile("" : "+v"(fw[i]));
#pragma unroll
        for (int j = 0; j < FM; j++)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[i], fx[j], acc[i][j], 0, 0, 0, sw, 0, sx[j]);
        if (i == 0) {
#pragma unroll
            for (int j = 0; j < FM; j++) {
                nx[j] = read_frag(next, xrow + j * 32 + r);
                ns[j] = xs[(xrow + j * 32 + r) * kScaleRow];
            }
        }
        fw[i] = read_frag(next, BM + wrow + i * 32 + r);
#pragma unroll
        for (int p = i * kLoads / FN; p < (i + 1) * kLoads / FN; p++) {
            load_lds_1k(src[p], fill + (wave + p * kWaves) * 1024);
            src[p] += ahead;
        }
    }
    sw = nsw;
}

// kStages: the next step's stage, the one being filled, and those in flight
template <int BM, int BN, int WM, int WN, int kStages>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * kWave, 2) void matmul_kernel(const MatmulArgs A) {
    constexpr int kWavesM = BM / WM, kWaves = kWavesM * (BN / WN), kThreads = kWaves * kWave;
    constexpr int FM = WM / 32, FN = WN / 32;
    constexpr int kLoadRows = 1024 / kStep;
    constexpr int kLoads = (BM + BN) / kLoadRows / kWaves;  // 1 KiB loads of a wave in a step
    constexpr int kStage = (BM + BN) * kStep;
    constexpr int kWScales = (BN + kScaleBlock - 1) / kScaleBlock, kChunk = (BM + kWScales) * kScaleRow;
    static_assert((BM + BN) % (kLoadRows * kWaves) == 0 && BM % kLoadRows == 0, "whole loads");
    static_assert(kScaleBlock % WN == 0, "a wave's columns share a scale");
    __shared__ __align__(16) uint8_t stages[kStages * kStage];
    __shared__ __align__(16) uint8_t scales[2 * kChunk];

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
            const int r = (wave + i * kWaves) * kLoadRows + l / (kStep / 16), c = exchange(r, l % (kStep / 16));
            if (r < BM) {
                const int s = source(min(m0 + r, m1 - 1));  // rows past the end repeat the last
                src[i] = A.x + max(s, 0) * row_bytes + c * 16;
            } else {
                src[i] = w + (int64_t)min(n0 + r - BM, A.N - 1) * row_bytes + c * 16;
            }
        }
        // scale bytes of blocks b0 .. b0 + 31: 4 blocks of a row a thread
        auto scale_bytes = [&](int b0) {
            uint8_t *to = scales + (b0 / kScaleBlocks & 1) * kChunk;
            const int nb = min(kScaleBlocks, A.kb - b0);
            for (int i = threadIdx.x; i < BM * (kScaleBlocks / 4); i += kThreads) {
                const int r = i / (kScaleBlocks / 4), b = i % (kScaleBlocks / 4) * 4;
                if (b < nb) {
                    const int s = source(min(m0 + r, m1 - 1));
                    *reinterpret_cast<uint32_t *>(to + r * kScaleRow + b) =
                        *reinterpret_cast<const uint32_t *>(A.xs + (int64_t)max(s, 0) * A.sb + b0 + b);
                }
            }
            for (int i = threadIdx.x; i < kWScales * kScaleBlocks; i += kThreads) {
                const int j = i / kScaleBlocks, b = i % kScaleBlocks;
                if (b < nb)
                    to[(BM + j) * kScaleRow + b] =
                        ws[(int64_t)min(n0 / kScaleBlock + j, (A.N - 1) / kScaleBlock) * A.kb + b0 + b];
            }
        };
        const int steps = A.kb * kParts;  // even
#pragma unroll
        for (int p = 0; p < kStages - 1; p++)
#pragma unroll
            for (int i = 0; i < kLoads; i++) {
                load_lds_1k(src[i], stages + p * kStage + (wave + i * kWaves) * 1024);
                src[i] += p + 1 < steps ? kStep : 0;
            }
        scale_bytes(0);
        if (A.kb > kScaleBlocks) scale_bytes(kScaleBlocks);
        wait_loads_but<(kStages - 2) * kLoads>();
        __syncthreads();
        i32x8 fx[FM], fx2[FM], fw[FN];
        int sx[FM], sx2[FM], sw = scales[(BM + wn * WN / kScaleBlock) * kScaleRow];
#pragma unroll
        for (int j = 0; j < FM; j++) {
            fx[j] = read_frag(stages, wm * WM + j * 32 + (l & 31));
            sx[j] = scales[(wm * WM + j * 32 + (l & 31)) * kScaleRow];
        }
#pragma unroll
        for (int i = 0; i < FN; i++) fw[i] = read_frag(stages, BM + wn * WN + i * 32 + (l & 31));
        int slot = 0;
        // step s: its operands are in `fx`, `sx` and fw, the next one's go to `nx`, `ns`
        auto step = [&](int s, const i32x8 (&x)[FM], i32x8 (&nx)[FM], const int (&c)[FM], int (&nc)[FM]) {
            // the next step's stage is complete once every wave's loads are, and
            // the stage to fill has been read
            wait_loads_but<(kStages - 3) * kLoads>();
            __syncthreads();
            const int after = (slot + 1) % kStages, b = (s + 1) / kParts;
            const uint8_t *xs = scales + (b / kScaleBlocks & 1) * kChunk + b % kScaleBlocks;
            matmul_step<BM, FM, FN, kLoads, kWaves>(stages + after * kStage, stages + (slot + kStages - 1) % kStages * kStage,
                                                    src, s + kStages < steps ? kStep : 0, wave, wm * WM, wn * WN, xs,
                                                    xs + (BM + wn * WN / kScaleBlock) * kScaleRow, x, nx, fw, c, nc, sw,
                                                    acc);
            slot = after;
        };
        for (int b0 = 0; b0 < A.kb; b0 += kScaleBlocks) {
            const int s1 = kParts * min(b0 + kScaleBlocks, A.kb);
            for (int s = kParts * b0; s < s1; s += 2) {
                step(s, fx, fx2, sx, sx2);
                step(s + 1, fx2, fx, sx2, sx);
            }
            if (b0 + 2 * kScaleBlocks < A.kb) {
                __syncthreads();  // this chunk's scales have been read
                scale_bytes(b0 + 2 * kScaleBlocks);
            }
        }
        wait_loads();  // those that nobody reads
    }

    // Two lanes exchange halves of their rows of 4 values, for 16-byte stores.
    const bool vec = A.N % 8 == 0 && ((uintptr_t)A.y & 15) == 0;
#pragma unroll
    for (int j = 0; j < FM; j++) {
        const int m = m0 + wm * WM + j * 32 + (l & 31);
        const bool in = m < m1, real = in && !tail && source(m) >= 0;
        uint16_t *y = A.y + (int64_t)m * A.N;
#pragma unroll
        for (int i = 0; i < FN; i++)
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
                const f32x16 &c = acc[i][j];
                const auto a = __builtin_amdgcn_permlane32_swap(pack_bf16(c[e], c[e + 1]), pack_bf16(c[e + 4], c[e + 5]),
                                                                false, false);
                const auto b = __builtin_amdgcn_permlane32_swap(pack_bf16(c[e + 2], c[e + 3]),
                                                                pack_bf16(c[e + 6], c[e + 7]), false, false);
                u32x4 v{a[0], b[0], a[1], b[1]};  // n .. n + 7
                if (!real) v = u32x4{0, 0, 0, 0};
                const int n = n0 + wn * WN + i * 32 + e * 2 + (l >> 5) * 8;
                if (vec) {
                    if (in && n < A.N) *reinterpret_cast<u32x4 *>(y + n) = v;
                } else if (in) {
#pragma unroll
                    for (int q = 0; q < 8; q++)
                        if (n + q < A.N) y[n + q] = (uint16_t)(v[q / 2] >> (16 * (q % 2)));
                }
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
    // The largest tile whose groups mostly fill it and whose count fills the card
    // (about 200 tiles).  Measured, us for 8 groups of N = K = 4096 with tiles of
    // 256 x 256, 128 x 128, 64 x 64: 400 rows a group 64, 91, 139; 200 rows 56, 54,
    // 79; 50 rows 44, 29, 38; 20 rows 44, 28, 25.  One group of 2048 x 2048 x 2048:
    // 30, 20, 29; of 1024 x 1024 x 4096: 43, 22, 17.
    const int64_t rows = p->m / p->groups;
    auto enough = [&](int64_t tile) { return ceil_div(p->m, tile) * ceil_div(p->n, tile) >= 192; };
    if (rows >= 256 && enough(256)) return rc_of(launch<256, 256, 64, 128, 4>(A, s));
    if (rows >= 32 && enough(128)) return rc_of(launch<128, 128, 64, 64, 4>(A, s));
    return rc_of(launch<64, 64, 32, 32, 6>(A, s));
}
