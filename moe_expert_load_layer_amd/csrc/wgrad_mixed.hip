// Weight gradient of the grouped product from rows that are held in 8 bits:
//   dW_g[n][k] = sum over the rows i of group g of dy[r(i)][n] x[q(i)][k]
// dy in bf16, x in e4m3 with a power-of-two scale for each 128 columns of a row,
// either one gathered by pair; fp32 out.  It is what a layer's backward pass needs of
// activations that were kept as the 8-bit products took them.
//
// A scale belongs to a row, which the sum runs over, so it cannot wait for the
// end; e4m3 times a power of two is exact in bf16, and the bf16 instruction then
// keeps the sums within 2e-7 of 64 bits, where the 8-bit one would show 1.5e-5.
//
// Rows go into LDS as they lie in memory, without passing registers.  dy's are
// read transposed from there.  x's are widened first: a lane reads back the 16
// bytes that it fetched, which lie in one row and under one scale, and writes 32
// bytes into a second place.  The tile is 256 columns of dy by 128 of x, so that
// each x is widened for as many columns of dy as LDS has room for.
//
// The rows' places (gathered, or past the group's end) and their scales come in
// chunks of 128 rows, fetched two chunks ahead the same way.
#include "columns.h"

namespace ep {
namespace {

struct MixedArgs {
    const uint16_t *dy;
    const uint8_t *x, *x_scale;
    int64_t dy_stride;        // elements
    int32_t kb, sb;           // blocks of x's columns, bytes of a row of its scales
    const int32_t *rows;      // or null: no row is gathered
    int32_t rows_div;
    int32_t gathered;         // rows that a gathered operand has
    bool gather_dy, gather_x;
    Groups groups;
    GroupRows where;
    int32_t N, K;
    float *out, *slot_out;
    int64_t out_stride, slot_out_stride;  // elements between groups
    int32_t band;                         // tiles of x side by side, see the kernel
};

constexpr int kRows = 32;  // rows of a step
constexpr int kTileK = 128, kTileN = 256;
constexpr int kWaveN = 64;
constexpr int kWaves = kTileN / kWaveN, kThreads = kWaves * kWave;
constexpr int kStages = 3;
constexpr int kChunkRows = 128, kChunkSteps = kChunkRows / kRows;
constexpr int kDyLoads = kRows * kTileN / 512 / kWaves;  // 1 KiB loads of a wave in a step
static_assert(kTileK == kScaleBlock && kRows * kTileK == 1024 * kWaves, "a wave fetches 1 KiB of x in a step");
static_assert(kChunkRows == 2 * kWave, "two waves find a chunk's places");

// e4m3 bytes times a power of two, as bf16
__device__ __forceinline__ u32x4 widen(uint32_t lo, uint32_t hi, float scale) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                 __builtin_bit_cast(uint32_t, d)};
}

// kVec: rows of dy of whole 16-byte chunks
template <bool kVec>
__global__ __launch_bounds__(kThreads, 2) void wgrad_mixed_kernel(const MixedArgs A) {
    constexpr int FK = kTileK / 32, FN = kWaveN / 32;
    constexpr int kLoads = kVec ? kDyLoads + 1 : 0;  // of a step, that may be in flight past a wait
    __shared__ __align__(16) uint16_t dys[kStages][kRows * kTileN];
    __shared__ __align__(16) uint8_t raws[3][kRows * kTileK];
    __shared__ __align__(16) uint16_t xs[2][kRows * kTileK];
    __shared__ int32_t indices[kChunkRows];
    __shared__ int32_t places[2][kChunkRows];  // row of the gathered operand, or of both; -1: none
    __shared__ uint32_t codes[2][kChunkRows];  // scale bytes

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), l = lane_id();
    const int tn = (A.N + kTileN - 1) / kTileN, tk = (A.K + kTileK - 1) / kTileK, tiles = (tn * tk + 7) / 8 * 8;
    // Groups one after the other; in a group an XCD takes consecutive tiles, counted
    // along bands of x, so that its L2 serves about as many columns of x as of dy.
    const int g = blockIdx.x / tiles, at = blockIdx.x - g * tiles, in = at % 8 * (tiles / 8) + at / 8;
    if (in >= tn * tk) return;
    const int bar = in / (A.band * tn), rest = in - bar * A.band * tn, wide = min(A.band, tk - bar * A.band);
    const int n0 = rest / wide * kTileN, kt = bar * A.band + rest % wide;
    const int m0 = A.groups.start(g), m1 = A.groups.end(g);
    const int steps = (m1 - m0 + kRows - 1) / kRows;

    f32x16 acc[FK][FN];
#pragma unroll
    for (int i = 0; i < FK; i++)
#pragma unroll
        for (int j = 0; j < FN; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;

    // ---- places and scales of a chunk ----
    auto ask = [&](int c) {  // its indices, by the waves that turn them into places
        if (A.rows && wave < 2) {
            const int i = min(m0 + c * kChunkRows + (int)wave * kWave + l, A.groups.M - 1);
            load_lds_dwords(A.rows + i, lds_address(indices) + wave * 256);
        }
    };
    auto place = [&](int c) {
        if (wave < 2) {
            const int t = wave * kWave + l;
            const int64_t m = (int64_t)m0 + c * kChunkRows + t;
            int r = m < m1 ? (int)m : -1;
            if (A.rows && r >= 0) {
                const int p = indices[t];
                r = p < 0 ? -1 : p / A.rows_div;
                r = r < A.gathered ? r : -1;
            }
            places[c & 1][t] = r;
            const int64_t row = A.gather_x || !A.rows ? r : m;
            const void *code = r >= 0 ? static_cast<const void *>(A.x_scale + row * A.sb + kt)
                                      : static_cast<const void *>(kZeros);
            load_lds_bytes(code, lds_address(codes[c & 1]) + wave * 256);
        }
    };
    // ---- a step's rows ----
    const int dcol = n0 + swizzle(wave * 2 + l / 32, l % 32) * 8;  // alike for all of a lane's rows
    const int back = !kVec && dcol < A.N ? max(dcol + 8 - A.N, 0) : 0;
    auto place_of = [&](int s, int row) { return places[s / kChunkSteps & 1][s % kChunkSteps * kRows + row]; };
    u32x4 held[kVec ? 1 : kDyLoads];
    auto fetch_dy = [&](int s, int slot, int i) {
        const int row = (wave + i * kWaves) * 2 + l / 32, r = place_of(s, row);
        const bool has = r >= 0 && dcol < A.N;
        const int64_t from = A.gather_dy || !A.rows ? r : (int64_t)m0 + s * kRows + row;
        const uint16_t *p = A.dy + from * A.dy_stride + dcol;
        if constexpr (kVec) {
            load_lds_1k(has ? static_cast<const void *>(p) : static_cast<const void *>(kZeros),
                        dys[slot] + (wave + i * kWaves) * 512);
        } else if (A.N >= 8) {  // the row's last 8 where some are past its end
            const void *q = has ? static_cast<const void *>(p - back) : static_cast<const void *>(kZeros);
            held[i] = *static_cast<const u32x4_at2 *>(q);
        } else {
            held[i] = u32x4{0, 0, 0, 0};
            if (has)
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (j < A.N) held[i][j / 2] |= (uint32_t)p[j] << (16 * (j % 2));
        }
    };
    auto put_dy = [&](int slot) {  // without kVec: what was fetched, into its tile
        if constexpr (!kVec) {
#pragma unroll
            for (int i = 0; i < kDyLoads; i++) {
                u32x4 v = held[i];
                if (A.N >= 8 && __any(back != 0)) {  // 128 bits shifted down by 16 for each column
                    const uint32_t zero = 0;
                    u32x4 w;
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        w[j] = __builtin_amdgcn_alignbit(j < 3 ? v[j + 1] : zero, v[j], back % 2 * 16);
                    if (back & 2) w = u32x4{w[1], w[2], w[3], 0};
                    if (back & 4) w = u32x4{w[2], w[3], 0, 0};
                    v = w;
                }
                *reinterpret_cast<u32x4 *>(dys[slot] + (wave + i * kWaves) * 512 + l * 8) = v;
            }
        }
    };
    auto fetch_x = [&](int s, int slot) {
        const int row = wave * 8 + l / 8, r = place_of(s, row);
        const int64_t from = A.gather_x || !A.rows ? r : (int64_t)m0 + s * kRows + row;
        const void *p = r >= 0 ? static_cast<const void *>(A.x + (from * A.kb + kt) * kTileK + l % 8 * 16)
                               : static_cast<const void *>(kZeros);
        load_lds_1k(p, raws[slot] + wave * 1024);
    };
    auto widen_x = [&](int s, int slot) {  // the bytes that this lane fetched
        const int row = wave * 8 + l / 8;
        const u32x4 v = *reinterpret_cast<const u32x4 *>(raws[slot] + wave * 1024 + l * 16);
        const float scale = __builtin_bit_cast(float, codes[s / kChunkSteps & 1][s % kChunkSteps * kRows + row] << 23);
        uint16_t *to = xs[s & 1] + row * kTileK;
        *reinterpret_cast<u32x4 *>(to + swizzle(row, l % 8 * 2) * 8) = widen(v[0], v[1], scale);
        *reinterpret_cast<u32x4 *>(to + swizzle(row, l % 8 * 2 + 1) * 8) = widen(v[2], v[3], scale);
    };

    if (steps > 0) {
        // places of chunks 0 and 1, then the first steps' rows
        for (int c = 0; c < 2; c++) {
            ask(c);
            wait_loads();
            place(c);
            wait_loads();
            __syncthreads();
        }
        for (int s = 0; s < 3; s++) fetch_x(s, s);
        for (int s = 0; s < 2; s++) {
#pragma unroll
            for (int i = 0; i < kDyLoads; i++) fetch_dy(s, s, i);
            put_dy(s);
        }
        wait_loads();
        widen_x(0, 0);
    }
    // Step s: multiplies dy(s) and x(s), widens x(s + 1), fetches dy(s + 2) and
    // x(s + 3), which takes the place of x(s).  Past its wait only what step s - 1
    // fetched is in flight.  Chunk c (steps 4 c .. 4 c + 3) has its indices fetched at
    // step 4 c - 8 and its places found at 4 c - 5, two barriers before x(4 c) is
    // fetched; its scales are there two barriers before x(4 c) is widened.
    int slot = 0;  // s mod 3
    for (int s = 0; s < steps; s++) {
        wait_loads_but<kLoads>();
        __syncthreads();
        const int after = slot == 2 ? 0 : slot + 1, two = slot == 0 ? 2 : slot - 1;
        if (s % kChunkSteps == 0) ask(s / kChunkSteps + 2);
        if (s % kChunkSteps == 3) place(s / kChunkSteps + 2);
        widen_x(s + 1, after);
        if constexpr (!kVec) {
#pragma unroll
            for (int i = 0; i < kDyLoads; i++) fetch_dy(s + 2, two, i);
        }
        const uint16_t *td = dys[slot], *tx = xs[s & 1];
#pragma unroll
        for (int t = 0; t < kRows; t += 16) {
            bf16x8 fx[FK], fd[FN];
#pragma unroll
            for (int i = 0; i < FK; i++) fx[i] = read_columns<kTileK>(tx, t, i * 32);
#pragma unroll
            for (int j = 0; j < FN; j++) fd[j] = read_columns<kTileN>(td, t, wave * kWaveN + j * 32);
#pragma unroll
            for (int i = 0; i < FK; i++) {
#pragma unroll
                for (int j = 0; j < FN; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fx[i], fd[j], acc[i][j], 0, 0, 0);
                // the loads go out between the products
                if constexpr (kVec)
                    if (i % 2 == 1) fetch_dy(s + 2, two, t / 16 * 2 + i / 2);
            }
        }
        fetch_x(s + 3, slot);
        put_dy(two);
        slot = after;
    }
    wait_loads();  // those that nobody reads

    int row;
    const bool spare = A.where.spare(g, &row);
    float *out = spare ? A.slot_out + row * A.slot_out_stride : A.out + row * A.out_stride;
#pragma unroll
    for (int j = 0; j < FN; j++) {
        const int n = n0 + wave * kWaveN + j * 32 + (l & 31);
        if (n >= A.N) continue;
#pragma unroll
        for (int i = 0; i < FK; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int k = kt * kTileK + i * 32 + e * 8 + (l >> 5) * 4;
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

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_grouped_wgrad_mixed(const ep_grouped_wgrad_mixed_t *p, ep_stream_t stream) {
    if (!p || p->m < 0 || p->m > kMaxRows || p->n < 1 || p->n > (1 << 24) || p->k < 1 || p->k > (1 << 24) ||
        p->groups < 1 || p->groups > EP_MAX_EXPERTS * 65)
        return EP_ERR_INVALID_ARG;
    if (!p->offsets && p->groups != 1) return EP_ERR_INVALID_ARG;
    MixedArgs A;
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
                     !is_aligned(p->x_scale, 4) || p->dy_stride < p->n))
        return EP_ERR_INVALID_ARG;
    if ((p->groups > 1 && p->out_stride < p->n * p->k) ||
        (p->slot_out && p->layout && p->layout->num_spare > 1 && p->slot_out_stride < p->n * p->k))
        return EP_ERR_INVALID_ARG;
    A.dy = static_cast<const uint16_t *>(p->dy);
    A.x = static_cast<const uint8_t *>(p->x);
    A.x_scale = p->x_scale;
    A.dy_stride = p->dy_stride;
    A.kb = (int32_t)ceil_div(p->k, kScaleBlock);
    A.sb = (int32_t)ep_scale_stride(p->k);
    A.rows = p->dy_places ? p->dy_places : p->x_places;
    A.rows_div = p->rows_div;
    A.gathered = (int32_t)(p->dy_places ? p->dy_rows : p->x_rows);
    A.gather_dy = p->dy_places != nullptr;
    A.gather_x = p->x_places != nullptr;
    A.groups = Groups{p->offsets, p->groups, (int32_t)p->m};
    A.N = (int32_t)p->n;
    A.K = (int32_t)p->k;
    A.out = p->out;
    A.slot_out = p->slot_out;
    A.out_stride = p->out_stride;
    A.slot_out_stride = p->slot_out_stride;
    const int64_t tiles = ceil_div(ceil_div(A.N, kTileN) * ceil_div(A.K, kTileK), 8) * 8;
    // an XCD's eighth of the tiles, as a rectangle of about as many columns of x as of dy
    A.band = 1;
    while ((int64_t)(A.band + 1) * (A.band + 1) * kTileK <= tiles / 8 * kTileN) A.band++;
    const int64_t blocks = A.groups.G * tiles;
    if (blocks > 0xffffffffll / kThreads) return EP_ERR_INVALID_ARG;
    const bool vec = p->n % 8 == 0 && is_aligned(p->dy, 16) && p->dy_stride % 8 == 0;
    const hipStream_t s = to_stream(stream);
    if (vec) wgrad_mixed_kernel<true><<<(uint32_t)blocks, kThreads, 0, s>>>(A);
    else wgrad_mixed_kernel<false><<<(uint32_t)blocks, kThreads, 0, s>>>(A);
    return rc_of(hipGetLastError());
}
