// Grouped matrix product in 8-bit floating point (product.h): y[m][n] in bf16.
//
// At 65536 x 4096 x 4096: 969 us, 2.27 PFLOP/s, against 2.93 of a large library
// product in 8 bits without scales; at 32749 x 7168 x 2048 2.02, at 16381 x 2048 x
// 4096 1.76.  Zeros instead of random values take a fifth less, as the card lowers
// its clock (2.4 GHz to 1.8) under this load.
#include "product.h"

namespace ep {
namespace {

struct WholeTile {
    static constexpr int kMatrices = 1;
    static constexpr bool kLong = false;
    struct Args {
        uint16_t *y;
    };
    template <int BM, int kWavesN>
    struct Shared {};

    template <class S>
    __device__ __forceinline__ static void locate(const ProductArgs &, const Args &, S &, int, int, int, int) {}

    // Two lanes exchange halves of their rows of 4 values, for 16-byte stores.
    template <int BM, int BN, int WM, int WN, int FM, int FN, class S>
    __device__ __forceinline__ static void store(const ProductArgs &A, const Args &B, const ProductTile<1> &tile,
                                                 const int32_t *places, S &, int, int wm, int wn, int l,
                                                 f32x16 (&acc)[FN][FM]) {
        const bool full = __builtin_amdgcn_readfirstlane(tile.m0 + BM <= tile.m1 && tile.n0 + BN <= A.N);
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
            const bool real = places[r] >= 0;
            uint16_t *y = B.y + (int64_t)m * A.N + n0;
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
    }

    // zeros
    __device__ __forceinline__ static void tail(const ProductArgs &A, const Args &B, int64_t id, int64_t threads) {
        const int64_t z0 = (int64_t)A.groups.start(A.groups.G) * A.N, z1 = (int64_t)A.groups.M * A.N;
        for (int64_t i = z0 + id * 8; i < z1; i += threads * 8) {
            if (i + 8 <= z1) *reinterpret_cast<u32x4_at2 *>(B.y + i) = u32x4{0, 0, 0, 0};
            else
                for (int64_t j = i; j < z1; j++) B.y[j] = 0;
        }
    }
};

template <int BM, int BN, int WM, int WN, int kStages>
hipError_t launch(const ProductArgs &A, const WholeTile::Args &B, hipStream_t s) {
    return launch_product<WholeTile, BM, BN, WM, WN, kStages>(A, B, s);
}

}  // namespace

bool product_args(const ProductShape &p, const ep_layout_t *layout, bool slots, ProductArgs *A) {
    if (!layout_groups(layout, p.groups, slots, &A->where)) return false;
    if (!p.x || !p.x_scale || !is_aligned(p.x, 16) || !is_aligned(p.x_scale, 4) || !is_aligned(p.offsets, 4) ||
        !is_aligned(p.rows, 4))
        return false;
    if (p.rows ? (p.rows_div < 1 || p.x_rows < 1) : p.x_rows < p.m) return false;
    if (p.x_rows > kMaxRows) return false;
    if (p.weights && (!is_aligned(p.weights, 4) || p.pairs < (p.rows ? 0 : p.m))) return false;
    A->x = static_cast<const uint8_t *>(p.x);
    A->xs = p.x_scale;
    A->rows = p.rows;
    A->rows_div = p.rows_div;
    int64_t pairs = p.rows ? p.x_rows * p.rows_div : 0;  // both below 2^31
    if (p.weights && p.pairs < pairs) pairs = p.pairs;
    A->pairs = (int32_t)(pairs < 0x7fffffff ? pairs : 0x7fffffff);
    A->groups = Groups{p.offsets, p.groups, (int32_t)p.m};
    A->N = (int32_t)p.n;
    A->kb = (int32_t)ceil_div(p.k, kScaleBlock);
    A->sb = (int32_t)ep_scale_stride(p.k);
    return true;
}

bool product_matrix_ok(const ep_matrix_t &w, const ep_matrix_t &slot_w, const ep_layout_t *layout, int32_t groups,
                       int64_t n, int64_t k) {
    const int64_t kb = ceil_div(k, kScaleBlock), bytes = n * kb * 128, sbytes = ceil_div(n, kScaleBlock) * kb;
    if (!w.data || !w.scale || !is_aligned(w.data, 16) || w.stride % 16 != 0) return false;
    if (groups > 1 && (w.stride < bytes || w.scale_stride < sbytes)) return false;
    if (!slot_w.data || !slot_w.scale) return true;  // whether they are needed is the layout's matter
    if (!is_aligned(slot_w.data, 16) || slot_w.stride % 16 != 0) return false;
    return !(layout && layout->num_spare > 1 && (slot_w.stride < bytes || slot_w.scale_stride < sbytes));
}

}  // namespace ep

using namespace ep;

extern "C" int ep_grouped_matmul(const ep_grouped_matmul_t *p, ep_stream_t stream) {
    if (!p) return EP_ERR_INVALID_ARG;
    const ProductShape shape{p->x, p->x_scale, p->x_rows, p->rows, p->rows_div, p->groups, p->offsets, p->m, p->n, p->k,
                             nullptr, 0};
    if (!product_sizes_ok(shape)) return EP_ERR_INVALID_ARG;
    if (p->m == 0) return EP_OK;
    ProductArgs A;
    if (!product_args(shape, p->layout, p->slot_w.data && p->slot_w.scale, &A) ||
        !product_matrix_ok(p->w, p->slot_w, p->layout, p->groups, p->n, p->k) || !p->y || !is_aligned(p->y, 2))
        return EP_ERR_INVALID_ARG;
    A.w = static_cast<const uint8_t *>(p->w.data);
    A.ws = p->w.scale;
    A.w_stride = p->w.stride;
    A.ws_stride = p->w.scale_stride;
    A.slot_w = static_cast<const uint8_t *>(p->slot_w.data);
    A.slot_ws = p->slot_w.scale;
    A.slot_w_stride = p->slot_w.stride;
    A.slot_ws_stride = p->slot_w.scale_stride;
    const WholeTile::Args B{static_cast<uint16_t *>(p->y)};
    const hipStream_t s = to_stream(stream);
    // The largest tile whose groups mostly fill it and whose count fills the card
    // (about 200 tiles).  Measured, us for 8 groups of N = K = 4096 with tiles of
    // 256 x 256, 128 x 128, 64 x 64: 400 rows a group 61, 79, 117; 200 rows 45, 42,
    // 61; 50 rows 42, 25, 24; 20 rows 42, 25, 23.  One group of 2048 x 2048 x 2048:
    // 26, 15, 22; of 1024 x 1024 x 4096: 40, 19, 14; of 4096 x 4096 x 2048: 36, 44, 74.
    const int64_t rows = p->m / p->groups;
    auto enough = [&](int64_t tile) { return ceil_div(p->m, tile) * ceil_div(p->n, tile) >= 192; };
    if (rows >= 256 && enough(256)) return rc_of(launch<256, 256, 64, 128, 4>(A, B, s));
    if (rows >= 32 && enough(128)) return rc_of(launch<128, 128, 64, 64, 4>(A, B, s));
    return rc_of(launch<64, 64, 32, 32, 6>(A, B, s));
}
