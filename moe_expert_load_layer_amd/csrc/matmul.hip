// Grouped matrix product in 8-bit floating point (e4m3) with a power-of-two
// scale for each block of 128:
//   y[m][n] = sum over blocks b of 128:  2^(ca[m][b] + cw[g][n / 128][b] - 254) * sum_k x[m][k] w_g[n][k]
// for the rows m of group g.
//
// The 32x32x64 matrix instruction takes a scale byte for each 32 values of
// either operand, so a block's scale costs no arithmetic: the bytes go to the
// instruction as they are.  It aligns every 8 products to their largest, drops
// what lies below 2^-13 of it and adds to an fp32 accumulator.  Against 64 bits that
// is 1.5e-5 of a result for normal values at any K, and by that rule 6e-5 where one
// channel in a hundred is 20 times larger: one bf16 output in fifty then rounds the
// other way (measured), where each is off by up to 2^-9 of itself anyway.
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
// together they wait for the address unit: 8 % slower).  At 65536 x 4096 x 4096:
// 969 us, 2.27 PFLOP/s, against 2.93 of a large library product in 8 bits without
// scales; at 32749 x 7168 x 2048 2.02, at 16381 x 2048 x 4096 1.76.  Zeros instead of
// random values take a fifth less, as the card lowers its clock (2.4 GHz to 1.8)
// under this load.
#include "groups.h"
#include "walk.h"

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
constexpr int kScaleBlocks = 32;  // blocks of a chunk of scales; three chunks are in LDS
constexpr int kWScaleBytes = 256;  // of a chunk: 32 scales of each 128 rows of w (two at most), 4 bytes each

__device__ __forceinline__ int exchange(int row, int chunk) { return chunk ^ ((row >> 2) & 3); }

// A chunk of x scales is 32 bytes a row, their dwords exchanged by the row's bits
// 3 and 4: 32 rows' scales of one block lie in 32 banks.
__device__ __forceinline__ int scale_exchange(int row) { return (row >> 3 & 3) << 2; }
__device__ __forceinline__ int scale_at(int row, int block) {
    return (row * kScaleBlocks | scale_exchange(row)) ^ block;
}

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
__device__ __forceinline__ void matmul_step(const uint8_t *next, uint32_t fill, const uint8_t *(&src)[kLoads],
                                            int ahead, int xrow, int wrow, const uint8_t *xs, const uint8_t *ws,
                                            int block, const i32x8 (&fx)[FM], i32x8 (&nx)[FM], i32x8 (&fw)[FN],
                                            const int (&sx)[FM], int (&ns)[FM], int &sw, f32x16 (&acc)[FN][FM]) {
    const int r = lane_id() & 31;
    const int nsw = ws[block * 4];
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
                ns[j] = xs[scale_at(xrow + r, block) + j * 32 * kScaleBlocks];
            }
        }
        fw[i] = read_frag(next, BM + wrow + i * 32 + r);
#pragma unroll
        for (int p = i * kLoads / FN; p < (i + 1) * kLoads / FN; p++) {
            load_lds_1k(src[p], fill + p * kWaves * 1024);
            src[p] += ahead;
            asm volatile("" : "+v"(src[p]));  // one pointer a load, not one for each of two steps
        }
    }
    sw = nsw;
}

// A workgroup takes one tile after the other, and the ring never empties: a
// tile's last steps fetch the first ones of the next.  Finding a tile, its rows'
// places, the first loads and the wait for them, and the stores of the tile
// before cost 12 us a tile where each of them had a workgroup of its own.
// kChained false: the steps are too few for that (walk.h), a workgroup has one
// tile, or begins again where groups overlap and there are more.
//
// kStages: the next step's stage, those in flight, and this step's, whose
// operands are in registers and which is filled again.
template <int BM, int BN, int WM, int WN, int kStages, bool kChained>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * kWave, 2) void matmul_kernel(const MatmulArgs A) {
    constexpr int kWavesM = BM / WM, kWaves = kWavesM * (BN / WN), kThreads = kWaves * kWave;
    constexpr int FM = WM / 32, FN = WN / 32;
    constexpr int kLoadRows = 1024 / kStep;
    constexpr int kLoads = (BM + BN) / kLoadRows / kWaves;  // 1 KiB loads of a wave in a step
    constexpr int kStage = (BM + BN) * kStep;
    constexpr int kChunk = BM * kScaleBlocks + kWScaleBytes;  // bytes of a chunk of scales: of x, then of w
    constexpr int kScaleLoads = BM * (kScaleBlocks / 4) / kThreads;
    static_assert((BM + BN) % (kLoadRows * kWaves) == 0 && BM % kLoadRows == 0, "whole loads");
    static_assert(BM * (kScaleBlocks / 4) % kThreads == 0 && BM <= kThreads, "whole loads of scales");
    static_assert(kScaleBlock % WN == 0 && BN <= 2 * kScaleBlock, "a wave's columns share a scale");
    static_assert(kStages % 2 == 0 && (kStages - 2) * kLoads < 64, "steps go in pairs; a wait's largest count");
    __shared__ __align__(16) uint8_t stages[kStages * kStage];
    __shared__ __align__(16) uint8_t scales[3 * kChunk];
    // This tile and the next one, in LDS rather than in registers: a tile's rows and
    // columns, its matrix, and the row of x of each of its rows (-1: none)
    struct Tile {
        int m0, m1, n0;
        const uint8_t *w, *ws;
    };
    __shared__ Tile tiles[2];
    __shared__ int32_t places[2][BM];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave % kWavesM, wn = wave / kWavesM;
    const int nt = (A.N + BN - 1) / BN;
    const int mt = __builtin_amdgcn_readfirstlane(total_tiles(A.groups, BM));  // kept in a scalar register
    // an XCD's consecutive tiles: 4 row tiles by all column tiles, columns last, so
    // that the tiles in flight there share rows of x and of w in its L2
    const TileWalk walk = tile_walk((int64_t)mt * nt, blockIdx.x, gridDim.x);
    const int64_t row_bytes = (int64_t)A.kb * 128;
    const int steps = A.kb * kParts;  // even

    // What is computed once a tile from the lane's number starts from this copy, or
    // its values would be kept in registers throughout.
    auto lane_now = [] {
        int v = lane_id();
        asm volatile("" : "+v"(v));
        return v;
    };
    // finds the at-th tile and puts it into tiles[buf] and places[buf]
    auto locate = [&](int64_t at, int buf) {
        const int thread = wave * kWave + lane_now();
        constexpr int kBand = 4;
        const int band = (int)(at / ((int64_t)kBand * nt));
        const int in = (int)(at - (int64_t)band * kBand * nt), high = min(kBand, mt - band * kBand);
        const int tn = in / high, tile = band * kBand + in % high;
        int g = 0, first = 0;
        find_tile(A.groups, BM, tile, &g, &first);
        Tile t;
        // inside the group also where groups that overlap have more tiles than an int counts
        const int start = A.groups.start(g);
        t.m1 = A.groups.end(g);
        t.m0 = start + min(max(tile - first, 0), max(t.m1 - start - 1, 0) / BM) * BM;
        t.n0 = tn * BN;
        int row;
        const bool spare = A.where.spare(g, &row);
        t.w = spare ? A.slot_w + row * A.slot_w_stride : A.w + row * A.w_stride;
        t.ws = spare ? A.slot_ws + row * A.slot_ws_stride : A.ws + row * A.ws_stride;
        if (thread == 0) tiles[buf] = t;
        if (thread < BM) {
            int r = max(min(t.m0 + thread, t.m1 - 1), 0);  // rows past the end repeat the last
            if (A.rows) {
                const int p = A.rows[r];
                r = p < 0 ? -1 : p / A.rows_div;
                r = r < A.x_rows ? r : -1;
            }
            places[buf][thread] = r;
        }
        __syncthreads();
    };
    // the 16 bytes that this lane fetches in each of the wave's loads of step 0
    const uint8_t *src[kLoads];
    auto sources = [&](int buf) {
        const Tile &t = tiles[buf];
        const int l = lane_now();
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
            const int r = (wave + i * kWaves) * kLoadRows + l / (kStep / 16), c = exchange(r, l % (kStep / 16));
            if (r < BM) src[i] = A.x + max(places[buf][r], 0) * row_bytes + c * 16;
            else src[i] = t.w + (int64_t)min(t.n0 + r - BM, A.N - 1) * row_bytes + c * 16;
        }
    };
    // starts the loads of scale chunk `chunk` of a tile
    auto scale_loads = [&](int buf, int chunk, int slot) {
        const Tile &t = tiles[buf];
        const uint32_t to = lds_address(scales) + slot * kChunk;
        const int l = lane_now();
        const int b0 = chunk * kScaleBlocks;
#pragma unroll
        for (int i = 0; i < kScaleLoads; i++) {
            const int r = (wave + i * kWaves) * 8 + l / 8;
            // dwords past the row's end repeat its last one and are not used
            const int at = min(b0 + (l % 8 * 4 ^ scale_exchange(r)), A.sb - 4);
            load_lds_dwords(A.xs + (int64_t)max(places[buf][r], 0) * A.sb + at, to + (wave + i * kWaves) * 256);
        }
        const int nb = min(t.n0 / kScaleBlock + l / kScaleBlocks, (A.N - 1) / kScaleBlock);
        // every wave the same bytes to the same place
        load_lds_bytes(t.ws + (int64_t)nb * A.kb + min(b0 + l % kScaleBlocks, A.kb - 1), to + BM * kScaleBlocks);
    };

    int64_t at = walk.at;
    if (at < walk.to) {
        const uint32_t ring = lds_address(stages) + wave * 1024;
        int buf = 0, slot = 0, chunk0 = 0;  // chunk0: where the tile's first chunk of scales lies
        f32x16 acc[FN][FM];
        i32x8 fx[FM], fx2[FM], fw[FN];
        int sx[FM], sx2[FM], sw;
        // a tile from nothing: fills the ring and reads the first step's operands
        auto begin = [&] {
            const int l = lane_now();
            locate(at, buf);
            sources(buf);
            scale_loads(buf, 0, chunk0);
#pragma unroll
            for (int p = 0; p < kStages; p++)
#pragma unroll
                for (int i = 0; i < kLoads; i++) {
                    load_lds_1k(src[i], stages + p * kStage + (wave + i * kWaves) * 1024);
                    src[i] += p + 1 < steps ? kStep : 0;
                }
            wait_loads_but<(kStages - 1) * kLoads>();
            __syncthreads();
            sw = scales[BM * kScaleBlocks + wn * WN / kScaleBlock * kScaleBlocks * 4];
#pragma unroll
            for (int j = 0; j < FM; j++) {
                fx[j] = read_frag(stages, wm * WM + j * 32 + (l & 31));
                sx[j] = scales[scale_at(wm * WM + (l & 31), 0) + j * 32 * kScaleBlocks];
            }
#pragma unroll
            for (int i = 0; i < FN; i++) fw[i] = read_frag(stages, BM + wn * WN + i * 32 + (l & 31));
        };
        begin();
        for (;;) {
#pragma unroll
            for (int i = 0; i < FN; i++)
#pragma unroll
                for (int j = 0; j < FM; j++)
#pragma unroll
                    for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
            const bool more = at + walk.stride < walk.to;
            const int chunks = (A.kb + kScaleBlocks - 1) / kScaleBlocks;
            int ahead = kStep;
            // A step: its operands are in x, c and fw, the next one's (block `block` of
            // the chunk at `chunk`) go to nx, nc and fw.
            auto step = [&](int chunk, int block, const i32x8 (&x)[FM], i32x8 (&nx)[FM], const int (&c)[FM],
                            int (&nc)[FM]) {
                // the next step's stage is complete once every wave's loads are, and
                // this step's has been read by all
                wait_loads_but<(kStages - 2) * kLoads>();
                __syncthreads();
                const int after = slot == kStages - 1 ? 0 : slot + 1;
                const uint8_t *xs = scales + chunk;
                matmul_step<BM, FM, FN, kLoads, kWaves>(
                    stages + after * kStage, ring + slot * kStage, src, ahead, wm * WM, wn * WN, xs,
                    xs + BM * kScaleBlocks + wn * WN / kScaleBlock * kScaleBlocks * 4, block, x, nx, fw, c, nc, sw, acc);
                slot = after;
            };
            // Between the steps at which something happens besides, the loop is bare.
            for (int s = 0; s < steps;) {
                if (s % (kParts * kScaleBlocks) == 0) {
                    const int ch = s / (kParts * kScaleBlocks) + 1;
                    if (ch < chunks) scale_loads(buf, ch, (chunk0 + ch) % 3);
                }
                if (kChained && more && s == find_step(steps, kStages)) {
                    locate(at + walk.stride, buf ^ 1);
                    scale_loads(buf ^ 1, 0, (chunk0 + chunks) % 3);
                }
                if (s == max(steps - kStages, 0)) {  // from here on steps of the next tile are fetched
                    if (kChained && more) {
                        sources(buf ^ 1);
                    } else {  // or bytes that nobody reads, so that the count of loads stays
                        ahead = 0;
#pragma unroll
                        for (int i = 0; i < kLoads; i++) src[i] = tiles[buf].w;
                    }
                }
                // the chunk's last step, and with it the next chunk's place
                const int ch = s / (kParts * kScaleBlocks), end = min(steps, (ch + 1) * (kParts * kScaleBlocks));
                const int here = (chunk0 + ch) % 3 * kChunk, there = (chunk0 + ch + 1) % 3 * kChunk;
                int stop = end;
                if (s < steps - kStages) stop = min(stop, steps - kStages);
                if (kChained && more && s < find_step(steps, kStages)) stop = min(stop, find_step(steps, kStages));
                for (int b = s / kParts % kScaleBlocks; s < stop; s += 2, b++) {
                    step(here, b, fx, fx2, sx, sx2);  // the second half of this block
                    const bool last = s + 2 == end;
                    step(last ? there : here, last ? 0 : b + 1, fx2, fx, sx2, sx);
                }
            }

            // Two lanes exchange halves of their rows of 4 values, for 16-byte stores.
            const int l = lane_now();
            const Tile &tile = tiles[buf];
            const bool full =
                __builtin_amdgcn_readfirstlane(tile.m0 + BM <= tile.m1 && tile.n0 + BN <= A.N);
            auto eight = [&](const f32x16 &c, int e, bool real) {
                const auto a = __builtin_amdgcn_permlane32_swap(pack_bf16(c[e], c[e + 1]), pack_bf16(c[e + 4], c[e + 5]),
                                                                false, false);
                const auto b = __builtin_amdgcn_permlane32_swap(pack_bf16(c[e + 2], c[e + 3]),
                                                                pack_bf16(c[e + 6], c[e + 7]), false, false);
                return real ? u32x4{a[0], b[0], a[1], b[1]} : u32x4{0, 0, 0, 0};  // n .. n + 7
            };
#pragma unroll
            for (int j = 0; j < FM; j++) {
                const int r = wm * WM + j * 32 + (l & 31), m = tile.m0 + r, n0 = tile.n0 + wn * WN + (l >> 5) * 8;
                const bool real = places[buf][r] >= 0;
                uint16_t *y = A.y + (int64_t)m * A.N + n0;
                if (full) {
#pragma unroll
                    for (int i = 0; i < FN; i++)
#pragma unroll
                        for (int e = 0; e < 16; e += 8)
                            *reinterpret_cast<u32x4_at2 *>(y + i * 32 + e * 2) = eight(acc[i][j], e, real);
                } else {
                    const int end = m < tile.m1 ? A.N - n0 : 0;
#pragma unroll
                    for (int i = 0; i < FN; i++)
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            const u32x4 v = eight(acc[i][j], e, real);
                            const int n = i * 32 + e * 2;
                            if (n + 8 <= end) {
                                *reinterpret_cast<u32x4_at2 *>(y + n) = v;
                            } else {
#pragma unroll
                                for (int q = 0; q < 8; q++)
                                    if (n + q < end) y[n + q] = (uint16_t)(v[q / 2] >> (16 * (q % 2)));
                            }
                        }
                }
            }
            if (!more) break;
            at += walk.stride;
            buf ^= 1;
            chunk0 = (chunk0 + chunks) % 3;
            if constexpr (!kChained) {
                slot = chunk0 = 0;
                wait_loads();
                __syncthreads();  // every wave's, before the ring is filled again
                begin();
            }
        }
        wait_loads();  // those that nobody reads
    }

    // rows past the last group: zeros
    if (!A.groups.offsets) return;
    const int64_t z0 = (int64_t)A.groups.start(A.groups.G) * A.N, z1 = (int64_t)A.groups.M * A.N;
    const int64_t threads = (int64_t)gridDim.x * kThreads, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    for (int64_t i = z0 + id * 8; i < z1; i += threads * 8) {
        if (i + 8 <= z1) *reinterpret_cast<u32x4_at2 *>(A.y + i) = u32x4{0, 0, 0, 0};
        else
            for (int64_t j = i; j < z1; j++) A.y[j] = 0;
    }
}

template <int BM, int BN, int WM, int WN, int kStages>
hipError_t launch(const MatmulArgs &A, hipStream_t s) {
    constexpr int kThreads = (BM / WM) * (BN / WN) * kWave;
    int64_t blocks = tile_blocks(A.groups.M, A.groups.G, A.N, BM, BN);
    // As many workgroups as the card holds; where a tile's steps are too few to be
    // chained, as many as there are tiles.
    const auto kernel = tiles_chained(A.kb * kParts, kStages) ? matmul_kernel<BM, BN, WM, WN, kStages, true>
                                                              : matmul_kernel<BM, BN, WM, WN, kStages, false>;
    if (tiles_chained(A.kb * kParts, kStages)) {
        const int64_t resident = resident_blocks((const void *)kernel, kThreads, 0) / 8 * 8;
        if (resident > 0 && resident < blocks) blocks = resident;
    }
    if (blocks > 0xffffffffll / kThreads) return hipErrorInvalidConfiguration;
    kernel<<<(uint32_t)blocks, kThreads, 0, s>>>(A);
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
    // 256 x 256, 128 x 128, 64 x 64: 400 rows a group 61, 79, 117; 200 rows 45, 42,
    // 61; 50 rows 42, 25, 24; 20 rows 42, 25, 23.  One group of 2048 x 2048 x 2048:
    // 26, 15, 22; of 1024 x 1024 x 4096: 40, 19, 14; of 4096 x 4096 x 2048: 36, 44, 74.
    const int64_t rows = p->m / p->groups;
    auto enough = [&](int64_t tile) { return ceil_div(p->m, tile) * ceil_div(p->n, tile) >= 192; };
    if (rows >= 256 && enough(256)) return rc_of(launch<256, 256, 64, 128, 4>(A, s));
    if (rows >= 32 && enough(128)) return rc_of(launch<128, 128, 64, 64, 4>(A, s));
    return rc_of(launch<64, 64, 32, 32, 6>(A, s));
}
