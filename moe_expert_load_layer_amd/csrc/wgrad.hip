// Weight gradient of the grouped product: dW_g[n][k] = sum over the rows m of
// group g of dy[m][n] x[m][k], bf16 in, fp32 out.
//
// bf16 and not 8 bits: the 8-bit instruction's inner sums keep about 16 bits
// (1.5e-5 relative), which an fp32 gradient would show; the bf16 instruction
// stays within 2e-7 over 16384 rows (measured against 64 bits).
//
// The sum runs over the rows of both operands, so both tiles are needed
// transposed: rows go into LDS as they lie in memory (without passing
// registers, two stages deep, one barrier a step), and ds_read_b64_tr hands
// each lane 4 consecutive rows of one column.  It reads 4 rows of 32 bytes for
// 16 lanes; the 16-byte chunks of an LDS row are exchanged by the row's bits
// 0, 1 and 3, so that the rows read together meet different banks.
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
    bool vec;                             // 16-byte rows and stores
};

constexpr int kRows = 64;  // rows of a step

// the chunk of an LDS row that holds chunk c of the matrix row
__device__ __forceinline__ int swizzle(int row, int c) { return c ^ (((row & 3) << 1) | (row & 8)); }

// rows t .. t + 7 (this lane's half of 16) of column c0 + l % 32, as 8 bf16
template <int BC>
__device__ __forceinline__ bf16x8 read_columns(const uint16_t *tile, int t0, int c0) {
    const int l = lane_id(), i = l & 15, c = c0 + ((l >> 4) & 1) * 16 + (i & 3) * 4;
    union {
        s16x4 h[2];
        bf16x8 v;
    } u;
#pragma unroll
    for (int p = 0; p < 2; p++) {
        const int t = t0 + (l >> 5) * 8 + p * 4 + (i >> 2);
        const uint16_t *a = tile + t * BC + swizzle(t, c / 8) * 8 + c % 8;
        u.h[p] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)a);
    }
    return u.v;
}

// BC x BC tiles of dW, 128 x 64 of them a wave (BC = 256) or 64 x 64
template <int BC, int WK, int WN, bool kVec>
__global__ __launch_bounds__((BC / WK) * (BC / WN) * kWave) void wgrad_kernel(const WgradArgs A) {
    constexpr int kWavesK = BC / WK, kWaves = kWavesK * (BC / WN);
    constexpr int FK = WK / 32, FN = WN / 32;
    constexpr int kLoadRows = 512 / BC;                       // rows of a 1 KiB load
    constexpr int kLoads = 2 * kRows / kLoadRows / kWaves;    // loads of a wave in a step
    static_assert(2 * kRows % (kLoadRows * kWaves) == 0, "whole loads");
    constexpr int kStage = 2 * kRows * BC;  // rows of x, then rows of dy
    __shared__ __align__(16) uint16_t stages[2 * kStage];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), l = lane_id();
    const int tn = (A.N + BC - 1) / BC, tk = (A.K + BC - 1) / BC;
    // an XCD takes consecutive tiles of one group
    const int64_t all = (int64_t)A.groups.G * tn * tk, per = (all + 7) / 8;
    const int64_t at = (int64_t)(blockIdx.x % 8) * per + blockIdx.x / 8;
    if (at >= all || blockIdx.x / 8 >= per) return;
    const int g = (int)(at / ((int64_t)tn * tk)), in = (int)(at - (int64_t)g * tn * tk);
    const int n0 = in / tk * BC, k0 = in % tk * BC;
    const int m0 = A.groups.start(g), m1 = A.groups.end(g);
    const int wk = wave % kWavesK, wn = wave / kWavesK;

    f32x16 acc[FK][FN];
#pragma unroll
    for (int i = 0; i < FK; i++)
#pragma unroll
        for (int j = 0; j < FN; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;

    // this lane's chunk of each of the wave's loads: its row in the step and its
    // columns; the first kRows rows of a stage are x, the others dy
    auto fetch = [&](uint16_t *stage, int m) {
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
            const int r0 = (wave + i * kWaves) * kLoadRows;
            const bool isx = r0 < kRows;
            const int r = (r0 % kRows) + l / (BC / 8);
            const int c = swizzle(r, l % (BC / 8)) * 8 + (isx ? k0 : n0), cols = isx ? A.K : A.N;
            const uint16_t *p = isx ? A.x + (int64_t)(m + r) * A.x_stride : A.dy + (int64_t)(m + r) * A.dy_stride;
            uint16_t *to = stage + r0 * BC;
            if constexpr (kVec) {
                const bool ok = m + r < m1 && c < cols;
                load_lds_1k(ok ? static_cast<const void *>(p + c) : static_cast<const void *>(kZeros), to);
            } else {
                u32x4 v;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint32_t a = m + r < m1 && c + 2 * j < cols ? p[c + 2 * j] : 0;
                    const uint32_t b = m + r < m1 && c + 2 * j + 1 < cols ? p[c + 2 * j + 1] : 0;
                    v[j] = a | (b << 16);
                }
                *reinterpret_cast<u32x4 *>(to + l * 8) = v;
            }
        }
    };
    auto step = [&](const uint16_t *stage) {
        const uint16_t *tx = stage, *td = stage + kRows * BC;
#pragma unroll
        for (int t = 0; t < kRows; t += 16) {
            bf16x8 fx[FK], fd[FN];
#pragma unroll
            for (int i = 0; i < FK; i++) fx[i] = read_columns<BC>(tx, t, wk * WK + i * 32);
#pragma unroll
            for (int j = 0; j < FN; j++) fd[j] = read_columns<BC>(td, t, wn * WN + j * 32);
#pragma unroll
            for (int i = 0; i < FK; i++)
#pragma unroll
                for (int j = 0; j < FN; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fx[i], fd[j], acc[i][j], 0, 0, 0);
        }
    };
    if (m0 < m1) fetch(stages, m0);
    for (int m = m0, b = 0; m < m1; m += kRows, b ^= 1) {
        // this step's stage is complete once every wave's loads are, and the
        // other stage has been read
        wait_loads();
        __syncthreads();
        fetch(stages + (b ^ 1) * kStage, m + kRows);  // past the end: zeros that nobody reads
        step(stages + b * kStage);
    }
    wait_loads();

    int row;
    const bool spare = A.where.spare(g, &row);
    float *out = spare ? A.slot_out + row * A.slot_out_stride : A.out + row * A.out_stride;
#pragma unroll
    for (int j = 0; j < FN; j++) {
        const int n = n0 + wn * WN + j * 32 + (l & 31);
        if (n >= A.N) continue;
#pragma unroll
        for (int i = 0; i < FK; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int k = k0 + wk * WK + i * 32 + e * 8 + (l >> 5) * 4;
                float *o = out + (int64_t)n * A.K + k;
                if (kVec && k + 4 <= A.K) {
                    *reinterpret_cast<f32x4 *>(o) = f32x4{acc[i][j][4 * e], acc[i][j][4 * e + 1],
                                                          acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
                } else {
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        if (k + q < A.K) o[q] = acc[i][j][4 * e + q];
                }
            }
    }
}

template <int BC, int WK, int WN>
hipError_t launch(const WgradArgs &A, hipStream_t s) {
    constexpr int kThreads = (BC / WK) * (BC / WN) * kWave;
    const int64_t blocks = ceil_div((int64_t)A.groups.G * ceil_div(A.N, BC) * ceil_div(A.K, BC), 8) * 8;
    if (blocks > 0xffffffffll / kThreads) return hipErrorInvalidConfiguration;
    if (A.vec) wgrad_kernel<BC, WK, WN, true><<<(uint32_t)blocks, kThreads, 0, s>>>(A);
    else wgrad_kernel<BC, WK, WN, false><<<(uint32_t)blocks, kThreads, 0, s>>>(A);
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
    // whole chunks of 8 columns are inside or outside, and every row starts on 16 bytes
    A.vec = p->n % 8 == 0 && p->k % 8 == 0 && is_aligned(p->dy, 16) && is_aligned(p->x, 16) &&
            p->dy_stride % 8 == 0 && p->x_stride % 8 == 0 && is_aligned(p->out, 16) && p->out_stride % 4 == 0 &&
            is_aligned(p->slot_out, 16) && p->slot_out_stride % 4 == 0;
    return rc_of(launch<256, 128, 64>(A, to_stream(stream)));
}
