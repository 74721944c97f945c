// Weight gradient of the grouped product: dW_g[n][k] = sum over the rows m of
// group g of dy[m][n] x[m][k], bf16 in, fp32 out.
//
// bf16 and not 8 bits: the 8-bit instruction's inner sums keep about 16 bits
// (1.5e-5 relative), which an fp32 gradient would show; the bf16 instruction
// stays within 2e-7 over 16384 rows (measured against 64 bits).
//
// The sum runs over the rows of both operands, so both tiles are needed
// transposed: rows go into LDS as they lie in memory (without passing
// registers, a ring of three stages of 32 rows, one barrier a step), and
// ds_read_b64_tr hands each lane 4 consecutive rows of one column.  It reads 4
// rows of 32 bytes for 16 lanes; the 16-byte chunks of an LDS row are exchanged
// by the row's bits 0 and 1, so that the rows read together meet different banks.
//
// Bound: the matrix pipes.  16381 rows in 3 groups, N = 2048, K = 4096: 272 us,
// 1010 TFLOP/s, against 1190 of a large library product in bf16.  Tiles of
// 256 x 128 by 4 waves of 128 x 64 leave LDS for two workgroups a CU: while one
// waits at its barrier or stores its tile, the other multiplies.  One workgroup
// of 256 x 256 a CU took 13 us more.
//
// x is the instruction's row operand: a lane ends with 4 consecutive k of one n
// and stores 16 bytes.  Rows past the group's end and columns past the matrix
// are fetched from a block of zeros, so that neighbours' values (which may be
// infinite) never enter.
#include "groups.h"

namespace ep {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __align__(16) const uint32_t kZeros[4] = {0, 0, 0, 0};

struct WgradArgs {
    const uint16_t *dy, *x;
    int64_t dy_stride, x_stride;  // elements between rows
    Groups groups;
    GroupRows where;
    int32_t N, K;
    float *out, *slot_out;
    int64_t out_stride, slot_out_stride;  // elements between groups
    bool vec;                             // rows of whole 16-byte chunks
    int32_t band;                         // tiles of x side by side, see the kernel
};

constexpr int kRows = 32;              // rows of a step
constexpr int kTileK = 256, kTileN = 128;  // columns of x and of dy
constexpr int kWaveK = 128, kWaveN = 64;
constexpr int kWavesK = kTileK / kWaveK, kWaves = kWavesK * (kTileN / kWaveN), kThreads = kWaves * kWave;
constexpr int kStages = 3;

// the 16-byte chunk of an LDS row that holds chunk c of the matrix row
__device__ __forceinline__ int swizzle(int row, int c) { return c ^ ((row & 3) << 2); }

// rows t .. t + 7 (this lane's half of 16) of column c0 + l % 32, as 8 bf16
template <int kCols>
__device__ __forceinline__ bf16x8 read_columns(const uint16_t *tile, int t0, int c0) {
    const int l = lane_id(), i = l & 15, c = c0 + ((l >> 4) & 1) * 16 + (i & 3) * 4;
    union {
        s16x4 h[2];
        bf16x8 v;
    } u;
#pragma unroll
    for (int p = 0; p < 2; p++) {
        const int t = t0 + (l >> 5) * 8 + p * 4 + (i >> 2);
        const uint16_t *a = tile + t * kCols + swizzle(t, c / 8) * 8 + c % 8;
        u.h[p] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)a);
    }
    return u.v;
}

// The loads of one operand: a wave's 1 KiB loads hold whole LDS rows of kCols.
template <int kCols, bool kVec>
struct Operand {
    static constexpr int kLoadRows = 512 / kCols;
    static constexpr int kLoads = kRows / kLoadRows / kWaves;
    const uint16_t *p[kLoads];  // this lane's 8 values of the next step
    int64_t step;               // elements to the next step
    int cols, col;  // the matrix's columns, and this lane's first: its rows are alike by 4
    int back;       // columns of this lane's 8 that the matrix does not have, if it has others
    u32x4 held[kVec ? 1 : kLoads];

    __device__ __forceinline__ static int row(int wave, int i) {
        return (wave + i * kWaves) * kLoadRows + lane_id() / (kCols / 8);
    }
    __device__ __forceinline__ void set(const uint16_t *x, int64_t stride, int m, int c0, int width, int wave) {
        static_assert(kLoadRows * kWaves % 4 == 0, "one column for all of a lane's rows");
        step = stride * kRows;
        cols = width;
        col = c0 + swizzle(row(wave, 0), lane_id() % (kCols / 8)) * 8;
        back = !kVec && col < cols ? max(col + 8 - cols, 0) : 0;
#pragma unroll
        for (int i = 0; i < kLoads; i++) p[i] = x + (int64_t)(m + row(wave, i)) * stride + col;
    }
    // load i into `tile`, or into `held`; rows: of the step that the group has
    __device__ __forceinline__ void fetch(uint16_t *tile, int i, int rows, int wave) {
        const bool in = row(wave, i) < rows && col < cols;
        if constexpr (kVec) {
            load_lds_1k(in ? static_cast<const void *>(p[i]) : static_cast<const void *>(kZeros),
                        tile + (wave + i * kWaves) * 512);
        } else if (cols >= 8) {  // the row's last 8 where some are past its end; put() moves them
            const void *q = in ? static_cast<const void *>(p[i] - back) : static_cast<const void *>(kZeros);
            held[i] = *static_cast<const u32x4_at2 *>(q);
        } else {
            held[i] = u32x4{0, 0, 0, 0};
            if (in)
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (j < cols) held[i][j / 2] |= (uint32_t)p[i][j] << (16 * (j % 2));
        }
        p[i] += step;
    }
    // without kVec: what fetch brought, into its tile
    __device__ __forceinline__ void put(uint16_t *tile, int i, int wave) const {
        if constexpr (!kVec) {
            u32x4 v = held[i];
            if (cols >= 8 && __any(back != 0)) {  // 128 bits shifted down by 16 for each column
                const uint32_t zero = 0;
                u32x4 w;
#pragma unroll
                for (int j = 0; j < 4; j++) w[j] = __builtin_amdgcn_alignbit(j < 3 ? v[j + 1] : zero, v[j], back % 2 * 16);
                if (back & 2) w = u32x4{w[1], w[2], w[3], 0};
                if (back & 4) w = u32x4{w[2], w[3], 0, 0};
                v = w;
            }
            *reinterpret_cast<u32x4 *>(tile + (wave + i * kWaves) * 512 + lane_id() * 8) = v;
        }
    }
};

template <bool kVec>
__global__ __launch_bounds__(kThreads, 2) void wgrad_kernel(const WgradArgs A) {
    constexpr int FK = kWaveK / 32, FN = kWaveN / 32;
    constexpr int kStage = kRows * (kTileK + kTileN);  // rows of x, then rows of dy
    typedef Operand<kTileK, kVec> X;
    typedef Operand<kTileN, kVec> D;
    constexpr int kLoads = X::kLoads + D::kLoads;
    __shared__ __align__(16) uint16_t stages[kStages * kStage];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), l = lane_id();
    const int tn = (A.N + kTileN - 1) / kTileN, tk = (A.K + kTileK - 1) / kTileK, tiles = (tn * tk + 7) / 8 * 8;
    // Groups one after the other, so that a CU's two workgroups tend to come
    // from different ones.  In a group an XCD takes consecutive tiles, counted along
    // bands of x, so that its L2 serves about as many columns of x as of dy (0.54 GB
    // from memory for 16381 rows, 2048 x 4096; with all of x in one band 1.14 GB).
    const int g = blockIdx.x / tiles, at = blockIdx.x - g * tiles, in = at % 8 * (tiles / 8) + at / 8;
    if (in >= tn * tk) return;
    const int bar = in / (A.band * tn), rest = in - bar * A.band * tn, wide = min(A.band, tk - bar * A.band);
    const int n0 = rest / wide * kTileN, k0 = (bar * A.band + rest % wide) * kTileK;
    const int m0 = A.groups.start(g), m1 = A.groups.end(g);
    const int wk = wave % kWavesK, wn = wave / kWavesK;

    f32x16 acc[FK][FN];
#pragma unroll
    for (int i = 0; i < FK; i++)
#pragma unroll
        for (int j = 0; j < FN; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;

    X x;
    D d;
    x.set(A.x, A.x_stride, m0, k0, A.K, wave);
    d.set(A.dy, A.dy_stride, m0, n0, A.N, wave);
    const int steps = (m1 - m0 + kRows - 1) / kRows;
    // past the last step: zeros that nobody reads, so that the count of loads stays
    auto fetch = [&](uint16_t *stage, int s, int i) {
        const int rows = m1 - m0 - s * kRows;
        if (i < X::kLoads) x.fetch(stage, i, rows, wave);
        else d.fetch(stage + kRows * kTileK, i - X::kLoads, rows, wave);
    };
    auto put = [&](uint16_t *stage) {
#pragma unroll
        for (int i = 0; i < X::kLoads; i++) x.put(stage, i, wave);
#pragma unroll
        for (int i = 0; i < D::kLoads; i++) d.put(stage + kRows * kTileK, i, wave);
    };
    if (steps > 0) {
#pragma unroll
        for (int s = 0; s < kStages - 1; s++) {
#pragma unroll
            for (int i = 0; i < kLoads; i++) fetch(stages + s * kStage, s, i);
            put(stages + s * kStage);
        }
    }
    int slot = 0;
    for (int s = 0; s < steps; s++) {
        // this step's stage is complete once every wave's loads are, and the
        // stage before has been read
        wait_loads_but<kVec ? (kStages - 2) * kLoads : 0>();
        __syncthreads();
        const uint16_t *tx = stages + slot * kStage, *td = tx + kRows * kTileK;
        uint16_t *next = stages + (slot == 0 ? kStages - 1 : slot - 1) * kStage;
        if constexpr (!kVec) {  // through registers: fetched before the products, put after them
#pragma unroll
            for (int p = 0; p < kLoads; p++) fetch(next, s + kStages - 1, p);
        }
#pragma unroll
        for (int t = 0; t < kRows; t += 16) {
            bf16x8 fx[FK], fd[FN];
#pragma unroll
            for (int i = 0; i < FK; i++) fx[i] = read_columns<kTileK>(tx, t, wk * kWaveK + i * 32);
#pragma unroll
            for (int j = 0; j < FN; j++) fd[j] = read_columns<kTileN>(td, t, wn * kWaveN + j * 32);
#pragma unroll
            for (int i = 0; i < FK; i++) {
#pragma unroll
                for (int j = 0; j < FN; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fx[i], fd[j], acc[i][j], 0, 0, 0);
                // the loads go out between the products, not all at the step's start
                constexpr int kSlots = kRows / 16 * FK;
                if constexpr (kVec) {
#pragma unroll
                    for (int p = (t / 16 * FK + i) * kLoads / kSlots; p < (t / 16 * FK + i + 1) * kLoads / kSlots; p++)
                        fetch(next, s + kStages - 1, p);
                }
            }
        }
        put(next);
        slot = slot == kStages - 1 ? 0 : slot + 1;
    }
    wait_loads();  // those that nobody reads

    int row;
    const bool spare = A.where.spare(g, &row);
    float *out = spare ? A.slot_out + row * A.slot_out_stride : A.out + row * A.out_stride;
#pragma unroll
    for (int j = 0; j < FN; j++) {
        const int n = n0 + wn * kWaveN + j * 32 + (l & 31);
        if (n >= A.N) continue;
#pragma unroll
        for (int i = 0; i < FK; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int k = k0 + wk * kWaveK + i * 32 + e * 8 + (l >> 5) * 4;
                float *o = out + (int64_t)n * A.K + k;
                if (k + 4 <= A.K) {
                    *reinterpret_cast<f32x4_at4 *>(o) = f32x4{acc[i][j][4 * e], acc[i][j][4 * e + 1],
                                                          acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
                } else {
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        if (k + q < A.K) o[q] = acc[i][j][4 * e + q];
                }
            }
    }
}

hipError_t launch(WgradArgs &A, hipStream_t s) {
    const int64_t tiles = ceil_div(ceil_div(A.N, kTileN) * ceil_div(A.K, kTileK), 8) * 8;
    // an XCD's eighth of the tiles, as a rectangle of about as many columns of x as of dy
    A.band = 1;
    while ((int64_t)(A.band + 1) * (A.band + 1) * (kTileK / kTileN) <= tiles / 8) A.band++;
    const int64_t blocks = A.groups.G * tiles;
    if (blocks > 0xffffffffll / kThreads) return hipErrorInvalidConfiguration;
    if (A.vec) wgrad_kernel<true><<<(uint32_t)blocks, kThreads, 0, s>>>(A);
    else wgrad_kernel<false><<<(uint32_t)blocks, kThreads, 0, s>>>(A);
    return hipGetLastError();
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_grouped_wgrad(const ep_grouped_wgrad_t *p, ep_stream_t stream) {
    if (!p || p->m < 0 || p->m > kMaxRows || p->n < 1 || p->n > (1 << 24) || p->k < 1 || p->k > (1 << 24) ||
        p->groups < 1 || p->groups > EP_MAX_EXPERTS * 65)
        return EP_ERR_INVALID_ARG;
    if (!p->offsets && p->groups != 1) return EP_ERR_INVALID_ARG;
    WgradArgs A;
    if (!layout_groups(p->layout, p->groups, p->slot_out != nullptr, &A.where)) return EP_ERR_INVALID_ARG;
    if (!p->out || !is_aligned(p->out, 4) || !is_aligned(p->slot_out, 4) || !is_aligned(p->offsets, 4))
        return EP_ERR_INVALID_ARG;
    if (p->m > 0 && (!p->dy || !p->x || !is_aligned(p->dy, 2) || !is_aligned(p->x, 2) || p->dy_stride < p->n ||
                     p->x_stride < p->k))
        return EP_ERR_INVALID_ARG;
    if ((p->groups > 1 && p->out_stride < p->n * p->k) ||
        (p->slot_out && p->layout && p->layout->num_spare > 1 && p->slot_out_stride < p->n * p->k))
        return EP_ERR_INVALID_ARG;
    A.dy = static_cast<const uint16_t *>(p->dy);
    A.x = static_cast<const uint16_t *>(p->x);
    A.dy_stride = p->dy_stride;
    A.x_stride = p->x_stride;
    A.groups = Groups{p->offsets, p->groups, (int32_t)p->m};
    A.N = (int32_t)p->n;
    A.K = (int32_t)p->k;
    A.out = p->out;
    A.slot_out = p->slot_out;
    A.out_stride = p->out_stride;
    A.slot_out_stride = p->slot_out_stride;
    // Straight into LDS where whole chunks of 8 columns are inside or outside and every
    // row starts on 16 bytes; else through registers, with one step's loads in flight
    // instead of two: 12001 rows in 5 groups, 2047 x 3001 330 us, 450 TFLOP/s, less than
    // half of the other form's rate.
    A.vec = p->n % 8 == 0 && p->k % 8 == 0 && is_aligned(p->dy, 16) && is_aligned(p->x, 16) && p->dy_stride % 8 == 0 &&
            p->x_stride % 8 == 0;
    return rc_of(launch(A, to_stream(stream)));
}
