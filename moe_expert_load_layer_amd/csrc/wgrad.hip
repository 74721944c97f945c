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
//
// Rows that are held in 8 bits (ep_grouped_wgrad_mixed) are widened to bf16 in the
// workspace first, which holds them exactly, by a kernel of its own: 65536 rows in 8
// groups, N = 4096, K = 4096 take 2100 us so, the bf16 form with plain rows 1945.  Opened
// inside the loop, where every tile of N opens its rows of x again and they pass
// registers on their way into LDS, 2440.  A list of rows (either operand, or both) is
// read 128 places ahead into LDS and costs 8 % of the loop.
#include "columns.h"

namespace ep {
namespace {

struct WgradArgs {
    const uint16_t *dy, *x;
    int64_t dy_stride, x_stride;  // elements between rows
    Groups groups;
    GroupRows where;
    int32_t N, K;
    float *out, *slot_out;
    int64_t out_stride, slot_out_stride;  // elements between groups
    bool vec, vec_x;                      // rows of whole 16-byte chunks: of both operands, of x
    int32_t band;                         // tiles of x side by side, see the kernel
    int32_t x_cols;                       // columns that x may be read to
    // rows of a list: row i of a gathered operand is list[i] / list_div, if that is in [0, listed)
    const int32_t *list;
    int32_t list_div, listed;
    bool gather_dy, gather_x;
};

constexpr int kRows = 32;              // rows of a step
constexpr int kTileK = 256, kTileN = 128;  // columns of x and of dy
constexpr int kWaveK = 128, kWaveN = 64;
constexpr int kWavesK = kTileK / kWaveK, kWaves = kWavesK * (kTileN / kWaveN), kThreads = kWaves * kWave;
constexpr int kStages = 3;
constexpr int kChunkRows = 128, kChunkSteps = kChunkRows / kRows;  // of a list's places

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
    const uint16_t *base;  // with a list: this lane's columns of row 0,
    uint32_t bytes;        // a row's bytes,
    int places[kLoads];    // the rows of the step that is fetched next (-1: none),
    int coming[kLoads];    // and of the one after it

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
    __device__ __forceinline__ void set_list(const uint16_t *x, int64_t stride) {
        base = x + col;
        bytes = (uint32_t)(stride * 2);
    }
    __device__ __forceinline__ void look(const int32_t *from, int wave) {
#pragma unroll
        for (int i = 0; i < kLoads; i++) coming[i] = from[row(wave, i)];
    }
    __device__ __forceinline__ void arrive() {
#pragma unroll
        for (int i = 0; i < kLoads; i++) places[i] = coming[i];
    }
    // load i of a step whose rows are `places`, this operand's or the other's
    template <bool kListed>
    __device__ __forceinline__ void fetch_listed(uint16_t *tile, int i, int wave) {
        const bool in = places[i] >= 0 && col < cols;
        if constexpr (kListed) {  // one multiplication that adds, of 32 bits by 32
            const char *there = reinterpret_cast<const char *>(base) + (uint64_t)(uint32_t)places[i] * bytes;
            fetch_from(reinterpret_cast<const uint16_t *>(there), in, tile, i, wave);
        } else {
            fetch_from(p[i], in, tile, i, wave);
            p[i] += step;
        }
    }
    // load i into `tile`, or into `held`; rows: of the step that the group has
    __device__ __forceinline__ void fetch(uint16_t *tile, int i, int rows, int wave) {
        fetch_from(p[i], row(wave, i) < rows && col < cols, tile, i, wave);
        p[i] += step;
    }
    __device__ __forceinline__ void fetch_from(const uint16_t *from, bool in, uint16_t *tile, int i, int wave) {
        if constexpr (kVec) {
            load_lds_1k(in ? static_cast<const void *>(from) : static_cast<const void *>(kZeros),
                        tile + (wave + i * kWaves) * 512);
        } else if (cols >= 8) {  // the row's last 8 where some are past its end; put() moves them
            const void *q = in ? static_cast<const void *>(from - back) : static_cast<const void *>(kZeros);
            held[i] = *static_cast<const u32x4_at2 *>(q);
        } else {
            held[i] = u32x4{0, 0, 0, 0};
            if (in)
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (j < cols) held[i][j / 2] |= (uint32_t)from[j] << (16 * (j % 2));
        }
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

// kVecX, kVecD: rows of x, of dy, straight into LDS.
//
// kGather: which operand's rows come from a list (1: x, 2: dy, 3: both).  The rows'
// places, -1 past the group's end, come in chunks of 128 in LDS:
// the list's entries straight into LDS two chunks ahead, the places found from them by
// two waves three steps later, and looked up by every lane a step before it fetches.
template <bool kVecX, bool kVecD, int kGather>
__global__ __launch_bounds__(kThreads, 2) void wgrad_kernel(const WgradArgs A) {
    constexpr int FK = kWaveK / 32, FN = kWaveN / 32;
    constexpr int kStage = kRows * (kTileK + kTileN);  // rows of x, then rows of dy
    typedef Operand<kTileK, kVecX> X;
    typedef Operand<kTileN, kVecD> D;
    constexpr int kLoads = X::kLoads + D::kLoads;
    constexpr int kDirect = (kVecX ? X::kLoads : 0) + (kVecD ? D::kLoads : 0);  // straight into LDS
    __shared__ int32_t entries[kGather ? kChunkRows : 1], places[2][kGather ? kChunkRows : 1];
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
    x.set(A.x, A.x_stride, m0, k0, A.x_cols, wave);
    d.set(A.dy, A.dy_stride, m0, n0, A.N, wave);
    if constexpr (kGather) {
        x.set_list(A.x, A.x_stride);
        d.set_list(A.dy, A.dy_stride);
    }
    auto ask = [&](int c) {  // chunk c's entries, by the waves that turn them into places
        if (wave < kChunkRows / kWave) {
            const int i = min(m0 + c * kChunkRows + wave * kWave + l, A.groups.M - 1);
            load_lds_dwords(A.list + i, lds_address(entries) + wave * 256);
        }
    };
    auto place = [&](int c) {
        if (wave < kChunkRows / kWave) {
            const int t = wave * kWave + l, p = entries[t];
            int r = (int64_t)m0 + c * kChunkRows + t < m1 && p >= 0 ? p / A.list_div : -1;
            places[c & 1][t] = r < A.listed ? r : -1;
        }
    };
    auto look = [&](int s) {  // step s's places
        const int32_t *from = places[s / kChunkSteps & 1] + s % kChunkSteps * kRows;
        x.look(from, wave);
        d.look(from, wave);
    };
    auto arrive = [&] {
        x.arrive();
        d.arrive();
    };
    const int steps = (m1 - m0 + kRows - 1) / kRows;
    // past the last step: zeros that nobody reads, so that the count of loads stays
    auto fetch = [&](uint16_t *stage, int s, int i) {
        const int rows = m1 - m0 - s * kRows;
        if constexpr (kGather) {
            if (i < X::kLoads) x.template fetch_listed<(kGather & 1) != 0>(stage, i, wave);
            else d.template fetch_listed<(kGather & 2) != 0>(stage + kRows * kTileK, i - X::kLoads, wave);
        } else {
            if (i < X::kLoads) x.fetch(stage, i, rows, wave);
            else d.fetch(stage + kRows * kTileK, i - X::kLoads, rows, wave);
        }
    };
    auto put = [&](uint16_t *stage) {
#pragma unroll
        for (int i = 0; i < X::kLoads; i++) x.put(stage, i, wave);
#pragma unroll
        for (int i = 0; i < D::kLoads; i++) d.put(stage + kRows * kTileK, i, wave);
    };
    if (steps > 0) {
        if constexpr (kGather)
            for (int c = 0; c < 2; c++) {
                ask(c);
                wait_loads();
                place(c);
                __syncthreads();
            }
#pragma unroll
        for (int s = 0; s < kStages - 1; s++) {
            if constexpr (kGather) {
                look(s);
                arrive();
            }
#pragma unroll
            for (int i = 0; i < kLoads; i++) fetch(stages + s * kStage, s, i);
            put(stages + s * kStage);
        }
        if constexpr (kGather) {
            look(kStages - 1);
            arrive();
        }
    }
    int slot = 0;
    for (int s = 0; s < steps; s++) {
        // this step's stage is complete once every wave's loads are, and the
        // stage before has been read
        wait_loads_but<(kStages - 2) * kDirect>();
        __syncthreads();
        if constexpr (kGather) {
            // chunk c (steps 4 c .. 4 c + 3): entries at step 4 c - 8, places at 4 c - 5, two
            // barriers before step 4 c's are looked up, at 4 c - 3
            if (s % kChunkSteps == 0) ask(s / kChunkSteps + 2);
            if (s % kChunkSteps == 3) place(s / kChunkSteps + 2);
            look(s + kStages);
        }
        const uint16_t *tx = stages + slot * kStage, *td = tx + kRows * kTileK;
        uint16_t *next = stages + (slot == 0 ? kStages - 1 : slot - 1) * kStage;
        // through registers: fetched before the products, put after them
#pragma unroll
        for (int p = 0; p < kLoads; p++)
            if (p < X::kLoads ? !kVecX : !kVecD) fetch(next, s + kStages - 1, p);
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
#pragma unroll
                for (int p = (t / 16 * FK + i) * kLoads / kSlots; p < (t / 16 * FK + i + 1) * kLoads / kSlots; p++)
                    if (p < X::kLoads ? kVecX : kVecD) fetch(next, s + kStages - 1, p);
            }
        }
        put(next);
        if constexpr (kGather) arrive();
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
    const uint32_t grid = (uint32_t)blocks;
    const int gather = A.list ? (A.gather_x ? 1 : 0) + (A.gather_dy ? 2 : 0) : 0;
    auto run = [&](auto kernel) { kernel<<<grid, kThreads, 0, s>>>(A); };
    if (gather == 1) {
        A.vec ? run(wgrad_kernel<true, true, 1>) : run(wgrad_kernel<true, false, 1>);
    } else if (gather == 2) {
        A.vec ? run(wgrad_kernel<true, true, 2>) : run(wgrad_kernel<true, false, 2>);
    } else if (gather == 3) {
        A.vec ? run(wgrad_kernel<true, true, 3>) : run(wgrad_kernel<true, false, 3>);
    } else if (A.vec) {
        run(wgrad_kernel<true, true, 0>);
    } else if (A.vec_x) {
        run(wgrad_kernel<true, false, 0>);
    } else {
        run(wgrad_kernel<false, false, 0>);
    }
    return hipGetLastError();
}

// Rows in 8 bits as bf16, which holds e4m3 times a power of two exactly for scale bytes
// from 3 to 246 (product.h).  A unit is one row's block: 8 lanes of 16 values.
constexpr int kWidenThreads = 256;
__device__ __forceinline__ u32x4 widen(uint32_t lo, uint32_t hi, float scale) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                 __builtin_bit_cast(uint32_t, d)};
}
__global__ __launch_bounds__(kWidenThreads) void widen_kernel(const uint8_t *__restrict__ q,
                                                              const uint8_t *__restrict__ scale, int64_t units, int kb,
                                                              int sb, uint16_t *__restrict__ y) {
    const int64_t u = (int64_t)blockIdx.x * (kWidenThreads / 8) + threadIdx.x / 8;
    if (u >= units) return;
    const int64_t m = u / kb;
    const float s = __builtin_bit_cast(float, (uint32_t)scale[m * sb + (u - m * kb)] << 23);
    const int64_t at = u * kScaleBlock + threadIdx.x % 8 * 16;
    const u32x4 v = *reinterpret_cast<const u32x4 *>(q + at);
    u32x4 *o = reinterpret_cast<u32x4 *>(y + at);
    o[0] = widen(v[0], v[1], s);
    o[1] = widen(v[2], v[3], s);
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
    A.vec_x = false;
    A.x_cols = A.K;
    A.list = nullptr;
    return rc_of(launch(A, to_stream(stream)));
}

extern "C" size_t ep_wgrad_mixed_workspace_bytes(int64_t x_rows, int64_t k) {
    if (x_rows < 1 || x_rows > kMaxRows || k < 1 || k > (1 << 24)) return 0;
    return (size_t)x_rows * (size_t)ceil_div(k, kScaleBlock) * kScaleBlock * sizeof(uint16_t);
}

extern "C" int ep_grouped_wgrad_mixed(const ep_grouped_wgrad_mixed_t *p, ep_stream_t stream) {
    if (!p || p->m < 0 || p->m > kMaxRows || p->n < 1 || p->n > (1 << 24) || p->k < 1 || p->k > (1 << 24) ||
        p->groups < 1 || p->groups > EP_MAX_EXPERTS * 65)
        return EP_ERR_INVALID_ARG;
    if (!p->offsets && p->groups != 1) return EP_ERR_INVALID_ARG;
    WgradArgs A;
    if (!layout_groups(p->layout, p->groups, p->slot_out != nullptr, &A.where)) return EP_ERR_INVALID_ARG;
    if (!p->out || !is_aligned(p->out, 4) || !is_aligned(p->slot_out, 4) || !is_aligned(p->offsets, 4) ||
        !is_aligned(p->dy_places, 4) || !is_aligned(p->x_places, 4))
        return EP_ERR_INVALID_ARG;
    if (p->dy_rows < 0 || p->x_rows < 0 || p->dy_rows > kMaxRows || p->x_rows > kMaxRows) return EP_ERR_INVALID_ARG;
    if (p->dy_places && p->x_places && (p->dy_places != p->x_places || p->dy_rows != p->x_rows))
        return EP_ERR_INVALID_ARG;
    const bool gathered = p->dy_places || p->x_places;
    if (gathered && p->rows_div < 1) return EP_ERR_INVALID_ARG;
    if ((!p->dy_places && p->dy_rows < p->m) || (!p->x_places && p->x_rows < p->m)) return EP_ERR_INVALID_ARG;
    if (p->m > 0 && (!p->dy || !p->x || !p->x_scale || !is_aligned(p->dy, 2) || !is_aligned(p->x, 16) ||
                     !is_aligned(p->x_scale, 4) || p->dy_stride < p->n || p->dy_stride >= (int64_t)1 << 31))
        return EP_ERR_INVALID_ARG;
    if ((p->groups > 1 && p->out_stride < p->n * p->k) ||
        (p->slot_out && p->layout && p->layout->num_spare > 1 && p->slot_out_stride < p->n * p->k))
        return EP_ERR_INVALID_ARG;
    if (p->m > 0 && (!p->ws || !is_aligned(p->ws, 16) ||
                     p->ws_bytes < ep_wgrad_mixed_workspace_bytes(p->x_rows, p->k)))
        return EP_ERR_INVALID_ARG;
    const int64_t kb = ceil_div(p->k, kScaleBlock);
    const hipStream_t s = to_stream(stream);
    if (p->m > 0) {
        const int64_t units = p->x_rows * kb, grid = ceil_div(units, kWidenThreads / 8);
        if (grid > kMaxBlocks) return EP_ERR_INVALID_ARG;
        if (grid > 0)
            widen_kernel<<<(uint32_t)grid, kWidenThreads, 0, s>>>(static_cast<const uint8_t *>(p->x), p->x_scale, units,
                                                                 (int32_t)kb, (int32_t)ep_scale_stride(p->k),
                                                                 static_cast<uint16_t *>(p->ws));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return EP_ERR_HIP;
    }
    A.dy = static_cast<const uint16_t *>(p->dy);
    A.x = static_cast<const uint16_t *>(p->ws);
    A.dy_stride = p->dy_stride;
    A.x_stride = A.x_cols = (int32_t)(kb * kScaleBlock);
    A.groups = Groups{p->offsets, p->groups, (int32_t)p->m};
    A.N = (int32_t)p->n;
    A.K = (int32_t)p->k;
    A.out = p->out;
    A.slot_out = p->slot_out;
    A.out_stride = p->out_stride;
    A.slot_out_stride = p->slot_out_stride;
    A.list = p->dy_places ? p->dy_places : p->x_places;
    A.list_div = p->rows_div;
    A.listed = (int32_t)(p->dy_places ? p->dy_rows : p->x_rows);
    A.gather_dy = p->dy_places != nullptr;
    A.gather_x = p->x_places != nullptr;
    A.vec_x = true;
    A.vec = p->n % 8 == 0 && is_aligned(p->dy, 16) && p->dy_stride % 8 == 0;
    return rc_of(launch(A, s));
}
