// The gated feed-forward block over groups of rows, forward and backward, on the
// loop of the 8-bit grouped products (product.h).  For row i of group e, which
// serves pair p of token t:
//   forward   g = gate_e x_t,  u = up_e x_t,  h = w_p silu(g) u   in 8 bits
//             and, for a backward pass, g and u kept in 8 bits or bf16
//   backward  d = down_e^T dout_t,  s = sigmoid(g):
//             dw_p = sum_n d g s u,  dg = w_p d u s (1 + g (1 - s)),  du = w_p d g s
//             as bf16 (for the weight gradient) and in 8 bits (for the input gradient)
// Both are one product whose tile becomes the outputs before it leaves the
// registers: neither [g u] nor d is ever written in 16 bits and read again.
//
// What they measured, 8 groups, 65536 rows, hidden 4096, inter 2048, us: forward 1720 (2.2
// TFLOP at 1.28 PFLOP/s by the 16-bit instruction, which bounds it; with g and u kept in 8
// bits 1770), with the 8-bit sums 943 (two plain products of these sizes 1013; 2.33 PFLOP/s,
// bound as they are, by waiting in step; 1016), backward 1214 and 820 (one plain product
// 500).  With 8-bit sums the backward kernel needs 576 for d and the arithmetic, and 805 MB
// more of HBM traffic than the product (bf16 and 8-bit gradients out, g and u in), which
// comes in bursts at a tile's end while no wave multiplies: one workgroup a CU has all
// registers.  Two of 128 x 128, which take turns, load their operands twice as often and
// need 952; starting workgroups apart and stores that pass the caches by gained nothing.
#include <utility>

#include "product.h"

namespace ep {
namespace {

enum Keep { kNone, kSixteen, kEight };

// ---- a lane's 16 values of a 32 x 32 fragment ----
// Value e belongs to column 8 (e / 4) + 4 (lane / 32) + e % 4 of the fragment's
// row lane % 32.  Memory takes rows in pieces of 64 bytes best, 16 from each of 4
// lanes (in pieces of 32 the backward kernel's bf16 stores cost 145 us over the 580 of
// the kernel without them, at 65536 x 2048 and K = 4096; so they cost 118), and two
// swaps bring them together:
//   between the halves of the wave, after which a lane has 16 bytes in a row;
//   between rows of 16 lanes, of two such vectors that lie side by side in memory: one
//   then has both of rows 0 .. 15 of the fragment, the other both of rows 16 .. 31.
// Each swap undoes itself, so that the same way leads back.

struct Two {
    uint32_t a, b;
};
__device__ __forceinline__ Two swap_halves(uint32_t a, uint32_t b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    return Two{r[0], r[1]};
}
struct Pair {
    u32x4 lo, hi;  // 16 bytes and the 16 or 32 that follow; or rows 0 .. 15 and 16 .. 31
};
__device__ __forceinline__ Pair swap_rows(const Pair &p) {
    Pair r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const auto t = __builtin_amdgcn_permlane16_swap(p.lo[i], p.hi[i], false, false);
        r.lo[i] = t[0], r.hi[i] = t[1];
    }
    return r;
}

// four bytes for every 4 values, to and from 16 consecutive bytes
__device__ __forceinline__ u32x4 bytes_to_memory(const u32x4 &v) {
    const Two p = swap_halves(v[0], v[2]), q = swap_halves(v[1], v[3]);
    return u32x4{p.a, p.b, q.a, q.b};
}
__device__ __forceinline__ u32x4 bytes_from_memory(const u32x4 &v) {
    const Two p = swap_halves(v[0], v[1]), q = swap_halves(v[2], v[3]);
    return u32x4{p.a, q.a, p.b, q.b};
}
// 16-bit values, two a word: 8 columns and the 8 that lie 16 further on
__device__ __forceinline__ Pair words_to_memory(const uint32_t (&v)[8]) {
    const Two a = swap_halves(v[0], v[2]), b = swap_halves(v[1], v[3]), c = swap_halves(v[4], v[6]),
              d = swap_halves(v[5], v[7]);
    return Pair{u32x4{a.a, b.a, a.b, b.b}, u32x4{c.a, d.a, c.b, d.b}};
}
__device__ __forceinline__ void words_from_memory(const Pair &w, uint32_t (&v)[8]) {
    const Two a = swap_halves(w.lo[0], w.lo[2]), b = swap_halves(w.lo[1], w.lo[3]), c = swap_halves(w.hi[0], w.hi[2]),
              d = swap_halves(w.hi[1], w.hi[3]);
    v[0] = a.a, v[2] = a.b, v[1] = b.a, v[3] = b.b, v[4] = c.a, v[6] = c.b, v[5] = d.a, v[7] = d.b;
}
// Where a lane's 16 bytes lie once rows are swapped: its row of a Pair's first half (the
// second's is 16 further), its byte of two fragments' 64 in 8 bits, its column of a
// fragment's 32 in 16
__device__ __forceinline__ int piece_row(int l) { return l & 15; }
__device__ __forceinline__ int piece_byte(int l) { return (l >> 4 & 1) * 32 + (l >> 5) * 16; }
__device__ __forceinline__ int piece_column(int l) { return (l >> 4 & 1) * 16 + (l >> 5) * 8; }

__device__ __forceinline__ float other_half_max(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const Two t = swap_halves(b, b);
    return fmaxf(__builtin_bit_cast(float, t.a), __builtin_bit_cast(float, t.b));
}
__device__ __forceinline__ float other_half_sum(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const Two t = swap_halves(b, b);
    return __builtin_bit_cast(float, t.a) + __builtin_bit_cast(float, t.b);
}

// The largest finite magnitude, for a block's scale: infinity times 0 is NaN, which a
// maximum passes over.  (One instruction a value; a second look at the values of rows that
// hold infinities needs the registers that their sums leave: 12 % of the backward kernel.)
__device__ __forceinline__ float finite(float v) { return fmaf(v, 0.0f, fabsf(v)); }
__device__ __forceinline__ float largest(float m, float a, float b) { return fmaxf(fmaxf(m, finite(a)), finite(b)); }

// The upper halves of two floats with the lowest bit set: rounding these 8 bits of
// mantissa to the 4 of 8-bit floating point then gives what rounding the floats
// themselves does, but for ties, which go away from zero.  (A bit set only where
// something was below it would take three more instructions a value, a sixth of the
// backward kernel's, for cases that the sums' own error decides.)
__device__ __forceinline__ uint32_t odd_pair(float a, float b) {
    uint32_t v = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u) |
                 0x00010001u;
    asm volatile("" : "+v"(v));  // one register, not the two that it could be made of again
    return v;
}

// 8-bit values of floats, or of odd pairs, over a block's scale: the hardware's
// conversion divides by a power of two, rounds to nearest with ties to even and makes
// infinities NaN.
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// Where a block's scale is next to the least (of blocks of zeros, it is), the set bits
// would not vanish below its steps: they are taken away again.
template <int kCount>
__device__ __forceinline__ void settle(uint32_t (&v)[kCount][8], int code) {
    if (!__any(code <= 8)) return;
    const uint32_t kept = code <= 8 ? 0xfffefffeu : 0xffffffffu;
#pragma unroll
    for (int i = 0; i < kCount; i++)
#pragma unroll
        for (int e = 0; e < 8; e++) v[i][e] &= kept;
}

__device__ __forceinline__ uint32_t four_bytes(float a, float b, float c, float d, float scale) {
    const s16x2 v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(s16x2{0, 0}, a, b, scale, false);
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, c, d, scale, true));
}
__device__ __forceinline__ uint32_t four_bytes(uint32_t a, uint32_t b, float scale) {
    const s16x2 v = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(s16x2{0, 0}, __builtin_bit_cast(bf16x2, a), scale, false);
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(v, __builtin_bit_cast(bf16x2, b),
                                                                                 scale, true));
}
// of a fragment held in odd pairs, in its memory order
__device__ __forceinline__ u32x4 odd_to_memory(const uint32_t (&v)[8], float scale) {
    u32x4 q;
#pragma unroll
    for (int e = 0; e < 4; e++) q[e] = four_bytes(v[2 * e], v[2 * e + 1], scale);
    return bytes_to_memory(q);
}

// The sigmoid takes the hardware's exponential and reciprocal: 2^-16 of a value at
// most, against the 2^-4 (8 bits) or 2^-9 (bf16) of the roundings that follow.
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// Columns n .. n + 7 of a bf16 row of N
__device__ __forceinline__ void store_words(bool whole, uint16_t *row, int n, int N, const u32x4 &w) {
    if (whole || n + 8 <= N) {
        *reinterpret_cast<u32x4_at2 *>(row + n) = w;
    } else {
#pragma unroll
        for (int q = 0; q < 8; q++)
            if (n + q < N) row[n + q] = (uint16_t)(w[q / 2] >> (16 * (q % 2)));
    }
}
__device__ __forceinline__ u32x4 load_words(bool whole, const uint16_t *row, int n, int N) {
    u32x4 w{0, 0, 0, 0};
    if (whole || n + 8 <= N) {
        w = *reinterpret_cast<const u32x4_at2 *>(row + n);
    } else {
#pragma unroll
        for (int q = 0; q < 8; q++)
            if (n + q < N) w[q / 2] |= (uint32_t)row[n + q] << (16 * (q % 2));
    }
    return w;
}

// Sets what a fragment has past column `end`, counted from its first, to 0, whatever it
// was (rows without an input: end = 0), so that the steps after it need not mind.
__device__ __forceinline__ void mask(f32x16 &v, int end, int l) {
#pragma unroll
    for (int e = 0; e < 16; e++) v[e] = e / 4 * 8 + e % 4 + (l >> 5) * 4 < end ? v[e] : 0.0f;
}
// f(0), f(1) .. f(N - 1) with constants, however long f is: a loop that the compiler
// leaves rolled would index registers, and so keep the tile's sums in memory.
template <class F, int... I>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f) {
    each(std::make_integer_sequence<int, N>{}, f);
}

// Keeps what comes before and after apart, so that the registers of one fragment's
// steps are free before the next one's.  `now`: computed here and not where it is
// needed, or all that goes into it is kept until then (hundreds of registers).
__device__ __forceinline__ void next_fragment() { __builtin_amdgcn_sched_barrier(0); }
__device__ __forceinline__ void now(float &v) { asm volatile("" : "+v"(v)); }

// A row of scale bytes past its blocks, as ep_quant_rows writes it
__device__ __forceinline__ void pad_scales(uint8_t *row, int blocks, int stride) {
    for (int b = blocks; b < stride; b++) row[b] = 127;
}

// rows [m0, m1) of bytes in 8 bits and their scales, as rows of zeros have them
__device__ __forceinline__ void zero_rows(uint8_t *q, uint8_t *scale, int blocks, int stride, int64_t m0, int64_t m1,
                                          int64_t id, int64_t threads) {
    for (int64_t i = m0 * blocks * 8 + id; i < m1 * blocks * 8; i += threads)
        reinterpret_cast<u32x4 *>(q)[i] = u32x4{0, 0, 0, 0};
    for (int64_t i = m0 * stride + id; i < m1 * stride; i += threads) scale[i] = i % stride < blocks ? 1 : 127;
}
__device__ __forceinline__ void zero_words(uint16_t *y, int64_t from, int64_t to, int64_t id, int64_t threads) {
    for (int64_t i = from + id; i < to; i += threads) y[i] = 0;
}

// Whether a tile has all its rows and columns, and every row an input
template <int BM, class Tile, class S>
__device__ __forceinline__ bool whole_tile(const Tile &tile, int columns, int N, const S &shared, int buf) {
    bool whole = tile.m0 + BM <= tile.m1 && tile.n0 + columns <= N;
#pragma unroll
    for (int i = 0; i < BM / kWave; i++) whole = whole && shared.full[buf][i];
    return __builtin_amdgcn_readfirstlane(whole);
}

// the weight of a tile's row, 1 without weights
__device__ __forceinline__ float row_weight(const ProductArgs &A, const float *weights, int row, int place) {
    return !weights ? 1.0f : place < 0 ? 0.0f : weights[A.rows ? A.rows[row] : row];
}

// ------------------------------------------------------------------ forward

// A tile is 128 columns of gate and the same ones of up; a wave has the same half
// (or quarter) of both, so that silu(g) u needs no exchange.  A block's scale does:
// every wave puts the scale bytes of its part into LDS, and the largest counts.
template <Keep kKeep>
struct GatedTile {
    static constexpr int kMatrices = 2;
    static constexpr bool kLong = true;
    struct Args {
        SecondArgs up;
        const float *weights;
        uint8_t *h, *h_scale;
        void *kept;
        uint8_t *kept_scale;
        int32_t ib, hs, ks;  // blocks of inter, bytes of a row of scales of h and of what is kept
    };
    template <int BM, int kWavesN>
    struct Shared {
        float weight[2][BM];
        bool full[2][BM / kWave];  // whether every row of 64 has an input
        uint32_t codes[kWavesN][BM];
    };

    __device__ __forceinline__ static const SecondArgs &second(const Args &B) { return B.up; }

    template <class S>
    __device__ __forceinline__ static void locate(const ProductArgs &A, const Args &B, S &shared, int buf, int thread,
                                                  int row, int place) {
        shared.weight[buf][thread] = row_weight(A, B.weights, row, place);
        shared.full[buf][thread / kWave] = __all(place >= 0);
    }

    // h of the wave's columns of a row, and the scale bytes that they need by themselves:
    // of h, and of g and u where those are kept in 8 bits
    template <int F>
    __device__ __forceinline__ static uint32_t activate(const f32x16 *const (&g)[F], const f32x16 *const (&u)[F],
                                                        float weight, uint32_t (&h)[F][8]) {
        float th = 0, tg = 0, tu = 0;
#pragma unroll
        for (int i = 0; i < F; i++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                next_fragment();
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float a = (*g[i])[4 * q + e];
                    v[e] = a * sigmoid(a) * (*u[i])[4 * q + e] * weight;
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    if constexpr (kKeep == kEight) {
                        tg = largest(tg, (*g[i])[4 * q + e], (*g[i])[4 * q + e + 1]);
                        tu = largest(tu, (*u[i])[4 * q + e], (*u[i])[4 * q + e + 1]);
                    }
                    th = largest(th, v[e], v[e + 1]);
                    h[i][2 * q + e / 2] = odd_pair(v[e], v[e + 1]);
                }
                now(th);
                if constexpr (kKeep == kEight) {
                    now(tg);
                    now(tu);
                }
            }
        uint32_t code = fp8_scale_code(other_half_max(th));
        if constexpr (kKeep == kEight) {
            code |= fp8_scale_code(other_half_max(tg)) << 8 | fp8_scale_code(other_half_max(tu)) << 16;
        }
        return code;
    }

    template <int BM, int BN, int WM, int WN, int FM, int FN, class S>
    __device__ __forceinline__ static void store(const ProductArgs &A, const Args &B, const ProductTile<2> &tile,
                                                 const int32_t *places, S &shared, int buf, int wm, int wn, int l,
                                                 f32x16 (&acc)[FN][FM]) {
        constexpr int F = FN / 2, kWavesN = BN / WN;
        const int b = tile.n0 / kScaleBlock, c0 = tile.n0 + wn * (WN / 2);
        const bool whole = whole_tile<BM>(tile, kScaleBlock, A.N, shared, buf);
        if (!whole)
            each<FM>([&](auto J) {
                constexpr int j = J;
                const int end = places[wm * WM + j * 32 + (l & 31)] >= 0 ? A.N - c0 : 0;
#pragma unroll
                for (int i = 0; i < F; i++) {
                    mask(acc[i][j], end - i * 32, l);
                    mask(acc[F + i][j], end - i * 32, l);
                }
            });
        uint32_t held[FM][F][8];  // h in odd pairs
        each<FM>([&](auto J) {
            constexpr int j = J;
            const int r = wm * WM + j * 32 + (l & 31);
            const float weight = shared.weight[buf][r];
            const f32x16 *g[F], *u[F];
#pragma unroll
            for (int i = 0; i < F; i++) g[i] = &acc[i][j], u[i] = &acc[F + i][j];
            const uint32_t code = activate(g, u, weight, held[j]);
            if (l < 32) shared.codes[wn][r] = code;
        });
        __syncthreads();
        each<FM>([&](auto J) {
            constexpr int j = J;
            const int r = wm * WM + j * 32 + (l & 31), m = tile.m0 + r;
            const bool in = m < tile.m1;
            int ch = 0, cg = 0, cu = 0;
#pragma unroll
            for (int i = 0; i < kWavesN; i++) {
                const uint32_t code = shared.codes[i][r];
                ch = max(ch, (int)(code & 255));
                cg = max(cg, (int)(code >> 8 & 255));
                cu = max(cu, (int)(code >> 16));
            }
            settle(held[j], ch);
            // rows of 16 lanes' pieces, and whether they are the group's
            const int m0 = tile.m0 + wm * WM + j * 32 + piece_row(l);
            const bool in0 = m0 < tile.m1, in1 = m0 + 16 < tile.m1;
            const int wide = B.ib * kScaleBlock;
            constexpr int kSide = F % 2 == 0 ? 2 : 1;  // fragments side by side in 8 bits
            // 8-bit rows `stride` bytes apart, two fragments or one
            auto put = [&](uint8_t *to, int stride, const u32x4 (&v)[kSide], int i) {
                if constexpr (kSide == 2) {
                    const Pair p = swap_rows(Pair{v[0], v[1]});
                    uint8_t *o = to + (int64_t)m0 * stride + c0 + i * 32 + piece_byte(l);
                    if (in0) *reinterpret_cast<u32x4 *>(o) = p.lo;
                    if (in1) *reinterpret_cast<u32x4 *>(o + (int64_t)16 * stride) = p.hi;
                } else {
                    if (in) *reinterpret_cast<u32x4 *>(to + (int64_t)m * stride + c0 + i * 32 + (l >> 5) * 16) = v[0];
                }
            };
#pragma unroll
            for (int i = 0; i < F; i += kSide) {
                next_fragment();
                u32x4 v[kSide];
#pragma unroll
                for (int k = 0; k < kSide; k++) v[k] = odd_to_memory(held[j][i + k], pow2_of(ch));
                put(B.h, wide, v, i);
                if constexpr (kKeep == kEight) {
                    uint8_t *kept = static_cast<uint8_t *>(B.kept);
#pragma unroll
                    for (int k = 0; k < kSide; k++) v[k] = bytes_of(acc[i + k][j], pow2_of(cg));
                    put(kept, 2 * wide, v, i);
#pragma unroll
                    for (int k = 0; k < kSide; k++) v[k] = bytes_of(acc[F + i + k][j], pow2_of(cu));
                    put(kept + wide, 2 * wide, v, i);
                }
                if constexpr (kKeep == kSixteen)
#pragma unroll
                    for (int k = 0; k < kSide; k++) {
                        uint16_t *kept = static_cast<uint16_t *>(B.kept) + (int64_t)m0 * 2 * A.N;
                        const int64_t down = (int64_t)16 * 2 * A.N;
                        const int n = c0 + (i + k) * 32 + piece_column(l);
                        const Pair g = swap_rows(words_of(acc[i + k][j])), u = swap_rows(words_of(acc[F + i + k][j]));
                        if (in0) {
                            store_words(whole, kept, n, A.N, g.lo);
                            store_words(whole, kept + A.N, n, A.N, u.lo);
                        }
                        if (in1) {
                            store_words(whole, kept + down, n, A.N, g.hi);
                            store_words(whole, kept + down + A.N, n, A.N, u.hi);
                        }
                    }
            }
            if (in && wn == 0 && l < 32) {
                uint8_t *hs = B.h_scale + (int64_t)m * B.hs;
                hs[b] = (uint8_t)ch;
                if (b == B.ib - 1) pad_scales(hs, B.ib, B.hs);
                if constexpr (kKeep == kEight) {
                    uint8_t *ks = B.kept_scale + (int64_t)m * B.ks;
                    ks[b] = (uint8_t)cg;
                    ks[B.ib + b] = (uint8_t)cu;
                    if (b == B.ib - 1) pad_scales(ks, 2 * B.ib, B.ks);
                }
            }
        });
    }

    __device__ __forceinline__ static u32x4 bytes_of(const f32x16 &v, float scale) {
        u32x4 q;
#pragma unroll
        for (int e = 0; e < 4; e++) q[e] = four_bytes(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3], scale);
        return bytes_to_memory(q);
    }
    __device__ __forceinline__ static Pair words_of(const f32x16 &v) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; e++) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
        return words_to_memory(w);
    }

    // rows of zeros
    __device__ __forceinline__ static void tail(const ProductArgs &A, const Args &B, int64_t id, int64_t threads) {
        const int64_t m0 = A.groups.start(A.groups.G), m1 = A.groups.M;
        zero_rows(B.h, B.h_scale, B.ib, B.hs, m0, m1, id, threads);
        if constexpr (kKeep == kEight)
            zero_rows(static_cast<uint8_t *>(B.kept), B.kept_scale, 2 * B.ib, B.ks, m0, m1, id, threads);
        if constexpr (kKeep == kSixteen)
            zero_words(static_cast<uint16_t *>(B.kept), m0 * 2 * A.N, m1 * 2 * A.N, id, threads);
    }
};

// ----------------------------------------------------------------- backward

// A wave's 128 columns are a block of dg and one of du, so its scales need no
// exchange, and its share of dw is one number a row, added up by the second
// kernel in the blocks' order.
template <Keep kKeep>
struct GatedBackTile {
    static constexpr int kMatrices = 1;
    static constexpr bool kLong = true;
    struct Args {
        const float *weights;
        const void *kept;
        const uint8_t *kept_scale;
        uint16_t *dgu;           // or null
        uint8_t *q, *q_scale;    // or null
        float *dots;             // [rows][blocks], or null
        int32_t ib, qs;          // blocks of inter, bytes of a row of scales
    };
    template <int BM, int kWavesN>
    struct Shared {
        float weight[2][BM];
        bool full[2][BM / kWave];
    };

    template <class S>
    __device__ __forceinline__ static void locate(const ProductArgs &A, const Args &B, S &shared, int buf, int thread,
                                                  int row, int place) {
        shared.weight[buf][thread] = row_weight(A, B.weights, row, place);
        shared.full[buf][thread / kWave] = __all(place >= 0);
    }

    // What was kept of two fragments' rows (8 bits) or of one's (bf16), as it lies in
    // memory.  Rows without an input are rows of zeros there.
    static constexpr int kSide = kKeep == kEight ? 2 : 1;
    struct Kept {
        Pair g, u;
    };
    // A wave's 32 rows: the place of a lane's pieces
    struct Rows {
        int64_t row;    // of the first piece; the second's is 16 further
        bool in0, in1;  // whether they are the group's
        bool whole;     // and all columns are there
    };
    __device__ __forceinline__ static Kept load_kept(const Args &B, const Rows &R, int n, int N, int l) {
        Kept k{};
        if constexpr (kKeep == kEight) {
            const int64_t wide = (int64_t)B.ib * kScaleBlock;
            const uint8_t *p = static_cast<const uint8_t *>(B.kept) + R.row * 2 * wide + n + piece_byte(l);
            if (R.in0) {
                k.g.lo = *reinterpret_cast<const u32x4 *>(p);
                k.u.lo = *reinterpret_cast<const u32x4 *>(p + wide);
            }
            if (R.in1) {
                k.g.hi = *reinterpret_cast<const u32x4 *>(p + 32 * wide);
                k.u.hi = *reinterpret_cast<const u32x4 *>(p + 33 * wide);
            }
        } else {
            const uint16_t *p = static_cast<const uint16_t *>(B.kept) + R.row * 2 * N;
            const int64_t down = (int64_t)32 * N;
            n += piece_column(l);
            k.g.lo = load_words(R.whole, p, n, R.in0 ? N : 0);
            k.u.lo = load_words(R.whole, p + N, n, R.in0 ? N : 0);
            k.g.hi = load_words(R.whole, p + down, n, R.in1 ? N : 0);
            k.u.hi = load_words(R.whole, p + down + N, n, R.in1 ? N : 0);
        }
        k.g = swap_rows(k.g);
        k.u = swap_rows(k.u);
        return k;
    }
    __device__ __forceinline__ static void open_bytes(uint32_t w, float scale, float (&v)[4]) {
        const auto x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false);
        const auto y = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
        v[0] = x[0], v[1] = x[1], v[2] = y[0], v[3] = y[1];
    }

    // A lane's row of the wave's block: what its steps share, and what they leave
    struct Row {
        float weight, gs, us;  // the scales of what was kept
        float tg, tu, dot;     // the largest of dg and du, the sum for dw
    };
    template <int FN>
    __device__ __forceinline__ static void differentiate(const Args &B, const Rows &W, Row &R,
                                                         const f32x16 *const (&acc)[FN], int c0, int N, int l,
                                                         uint32_t (&vg)[FN][8], uint32_t (&vu)[FN][8]) {
        R.tg = R.tu = R.dot = 0.0f;
        // a fragment's are on their way while the one before is computed
        Kept now_kept{}, next = load_kept(B, W, c0, N, l);
#pragma unroll
        for (int i = 0; i < FN; i++) {
            next_fragment();
            if (i % kSide == 0) {
                now_kept = next;
                if (i + kSide < FN) next = load_kept(B, W, c0 + (i + kSide) * 32, N, l);
            }
            u32x4 bg{}, bu{};
            uint32_t pg[8], pu[8], wg[8], wu[8];
            if constexpr (kKeep == kEight) {
                bg = bytes_from_memory(i % 2 ? now_kept.g.hi : now_kept.g.lo);
                bu = bytes_from_memory(i % 2 ? now_kept.u.hi : now_kept.u.lo);
            } else {
                words_from_memory(now_kept.g, pg);
                words_from_memory(now_kept.u, pu);
            }
            // 4 values at a time, which is all that the registers of a wave beside its sums are for
#pragma unroll
            for (int q = 0; q < 4; q++) {
                next_fragment();
                float g[4], u[4];
                if constexpr (kKeep == kEight) {
                    open_bytes(bg[q], R.gs, g);
                    open_bytes(bu[q], R.us, u);
                } else {
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        g[2 * e] = bf16_lo(pg[2 * q + e]), g[2 * e + 1] = bf16_hi(pg[2 * q + e]);
                        u[2 * e] = bf16_lo(pu[2 * q + e]), u[2 * e + 1] = bf16_hi(pu[2 * q + e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float d = (*acc[i])[4 * q + e];
                    const float s = sigmoid(g[e]), act = g[e] * s, both = d * u[e];
                    R.dot = fmaf(act, both, R.dot);
                    g[e] = both * fmaf(act, 1.0f - s, s) * R.weight;
                    u[e] = d * act * R.weight;
                }
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    R.tg = largest(R.tg, g[2 * e], g[2 * e + 1]);
                    R.tu = largest(R.tu, u[2 * e], u[2 * e + 1]);
                    vg[i][2 * q + e] = odd_pair(g[2 * e], g[2 * e + 1]);
                    vu[i][2 * q + e] = odd_pair(u[2 * e], u[2 * e + 1]);
                    wg[2 * q + e] = pack_bf16(g[2 * e], g[2 * e + 1]);
                    wu[2 * q + e] = pack_bf16(u[2 * e], u[2 * e + 1]);
                }
                now(R.tg);
                now(R.tu);
                now(R.dot);
            }
            if (B.dgu) {
                const Pair g = swap_rows(words_to_memory(wg)), u = swap_rows(words_to_memory(wu));
                uint16_t *o = B.dgu + W.row * 2 * N;
                const int64_t down = (int64_t)32 * N;
                const int n = c0 + i * 32 + piece_column(l);
                if (W.in0) {
                    store_words(W.whole, o, n, N, g.lo);
                    store_words(W.whole, o + N, n, N, u.lo);
                }
                if (W.in1) {
                    store_words(W.whole, o + down, n, N, g.hi);
                    store_words(W.whole, o + down + N, n, N, u.hi);
                }
            }
        }
    }

    template <int BM, int BN, int WM, int WN, int FM, int FN, class S>
    __device__ __forceinline__ static void store(const ProductArgs &A, const Args &B, const ProductTile<1> &tile,
                                                 const int32_t *places, S &shared, int buf, int wm, int wn, int l,
                                                 f32x16 (&acc)[FN][FM]) {
        static_assert(WN == kScaleBlock, "a wave's columns are one block");
        const int c0 = __builtin_amdgcn_readfirstlane(tile.n0) + wn * WN, b = c0 / kScaleBlock;
        if (b >= B.ib) return;
        const int64_t wide = (int64_t)B.ib * kScaleBlock;
        const bool whole = whole_tile<BM>(tile, BN, A.N, shared, buf);
        if (!whole)
            each<FM>([&](auto J) {
                constexpr int j = J;
                const int end = places[wm * WM + j * 32 + (l & 31)] >= 0 ? A.N - c0 : 0;
#pragma unroll
                for (int i = 0; i < FN; i++) mask(acc[i][j], end - i * 32, l);
            });
        each<FM>([&](auto J) {
            constexpr int j = J;
            const int r = wm * WM + j * 32 + (l & 31), m = tile.m0 + r;
            const int m0 = tile.m0 + wm * WM + j * 32 + piece_row(l);
            const Rows W{m0, m0 < tile.m1, m0 + 16 < tile.m1, whole};
            const bool in = m < tile.m1;
            const int64_t row = in ? m : tile.m0;
            Row R;
            R.weight = shared.weight[buf][r];
            R.gs = R.us = 1.0f;
            if constexpr (kKeep == kEight) {
                R.gs = pow2_of(B.kept_scale[row * B.qs + b]);
                R.us = pow2_of(B.kept_scale[row * B.qs + B.ib + b]);
            }
            const f32x16 *d[FN];
#pragma unroll
            for (int i = 0; i < FN; i++) d[i] = &acc[i][j];
            uint32_t vg[FN][8], vu[FN][8];
            differentiate(B, W, R, d, c0, A.N, l, vg, vu);
            if (B.q) {
                const int cg = fp8_scale_code(other_half_max(R.tg)), cu = fp8_scale_code(other_half_max(R.tu));
                settle(vg, cg);
                settle(vu, cu);
                uint8_t *q = B.q + W.row * 2 * wide + c0 + piece_byte(l);
#pragma unroll
                for (int i = 0; i < FN; i += 2) {
                    next_fragment();
                    const Pair g = swap_rows(Pair{odd_to_memory(vg[i], pow2_of(cg)), odd_to_memory(vg[i + 1], pow2_of(cg))});
                    const Pair u = swap_rows(Pair{odd_to_memory(vu[i], pow2_of(cu)), odd_to_memory(vu[i + 1], pow2_of(cu))});
                    if (W.in0) {
                        *reinterpret_cast<u32x4 *>(q + i * 32) = g.lo;
                        *reinterpret_cast<u32x4 *>(q + wide + i * 32) = u.lo;
                    }
                    if (W.in1) {
                        *reinterpret_cast<u32x4 *>(q + 32 * wide + i * 32) = g.hi;
                        *reinterpret_cast<u32x4 *>(q + 33 * wide + i * 32) = u.hi;
                    }
                }
                if (in && l < 32) {
                    uint8_t *s = B.q_scale + row * B.qs;
                    s[b] = (uint8_t)cg;
                    s[B.ib + b] = (uint8_t)cu;
                    if (b == B.ib - 1) pad_scales(s, 2 * B.ib, B.qs);
                }
            }
            if (B.dots) {
                const float sum = other_half_sum(R.dot);
                if (in && l < 32) B.dots[row * B.ib + b] = sum;
            }
        });
    }

    // rows of zeros
    __device__ __forceinline__ static void tail(const ProductArgs &A, const Args &B, int64_t id, int64_t threads) {
        const int64_t m0 = A.groups.start(A.groups.G), m1 = A.groups.M;
        if (B.dgu) zero_words(B.dgu, m0 * 2 * A.N, m1 * 2 * A.N, id, threads);
        if (B.q) zero_rows(B.q, B.q_scale, 2 * B.ib, B.qs, m0, m1, id, threads);
        if (B.dots)
            for (int64_t i = m0 * B.ib + id; i < m1 * B.ib; i += threads) B.dots[i] = 0.0f;
    }
};

// dw of each pair: its position's blocks in order, in fp32; 0 without a position
constexpr int kDotThreads = 256;
template <bool kBf16>
__global__ __launch_bounds__(kDotThreads) void pair_dots_kernel(const float *__restrict__ dots, int ib, int64_t m,
                                                                const int32_t *__restrict__ pos, int64_t pairs,
                                                                void *__restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * kDotThreads + threadIdx.x;
    if (i >= pairs) return;
    const int64_t p = pos ? pos[i] : i;
    float s = 0.0f;
    if (p >= 0 && p < m)
        for (int b = 0; b < ib; b++) s += dots[p * ib + b];
    if constexpr (kBf16) static_cast<uint16_t *>(out)[i] = to_bf16(s);
    else static_cast<float *>(out)[i] = s;
}

// The sums decide which way values are rounded to 8 bits, steps of a sixteenth: one that
// is off by the 8-bit instruction's 2^-14 sends one value in 300 the other way, and where
// a few rows or values carry an output's norm, one is seen there.  So the forward kernel
// opens its operands (product.h) and adds in fp32 whatever the sizes, and a row's outputs
// do not depend on how many others there are.  The 8-bit sums are the caller's choice.
//
// Error of the block's output y against 64 bits, exact and 8-bit sums: 65536 rows, 4096 x
// 2048 1.66e-3 (what its rounding to bf16 gives) and 2.5e-3, 3001 rows, 1000 x 777 1.66e-3
// and 2.0 to 3.0e-3 over four seeds (up to 9e-3 seen).  us for 8 groups of hidden 4096,
// inter 2048, exact and 8-bit: 8192 rows a group 1720 and 940 to 990 (1.28 PFLOP/s; a library
// product in bf16 has 1.19 under load, 1.54 in a short run), 1000 rows 283 and 155, 400 rows
// 110 and 62, 100 rows 39 and 32, one row 35 and 28.
//
// The backward kernel the same, since its gradients are rounded to 8 bits again and dw adds
// up terms that cancel.  Error of the input gradient formed from q, with the same g and u:
// 1.66e-3 and 1.9e-3.  us, exact and 8-bit: 8192 rows a group 1214 and 820, 1000 rows 167 and
// 130, 400 rows 78 and 59, 100 rows 46 and 32.
template <Keep kKeep, bool kExact>
hipError_t forward(const ProductArgs &A, const typename GatedTile<kNone>::Args &B, hipStream_t s) {
    typedef GatedTile<kKeep> Tile;
    const typename Tile::Args C{B.up, B.weights, B.h, B.h_scale, B.kept, B.kept_scale, B.ib, B.hs, B.ks};
    // 256 rows where tiles of 128 would take the 256 CUs more than one round, and groups
    // mostly fill them.  Measured, us for 8 groups, hidden 4096, inter 2048 with tiles of
    // 256, 128, 64 rows: 1000 rows a group 283, 285, 307; 400 rows 110, 126, 142; 200 rows
    // 91, 63, 74; 100 rows 86, 54, 39.  5003 rows in 3 groups of 1999 x 1003 (160 tiles of
    // 256): 50, 61, 58; 3001 rows in 5 of 1000 x 777 (84): 32, 22, 29.  With 8-bit sums:
    // 158, 175, 243; 62, 74, 109; 52, 41, 59; 48, 34, 32; 32, 39, 46; 21, 15, 21.  A row or
    // two a group of hidden 4096, inter 2048 (128 tiles, 134 MB of weights from HBM) take 42
    // us; tiles of 32 rows with 6 or 8 stages 40 to 45, and 8-bit sums 40.  A kernel that
    // only loads these tiles takes 34 (27 in pieces of 1 KiB a row, which the loop has no use
    // for), and no less with more in flight.
    const int64_t rows = A.groups.M / A.groups.G;
    if (rows >= 256 && ceil_div(A.groups.M, 256) * ceil_div(A.N, kScaleBlock) > 128)
        return launch_product<Tile, 256, 256, 64, 128, 4, kExact>(A, C, s);
    if (rows >= 128) return launch_product<Tile, 128, 256, 32, 128, 4, kExact>(A, C, s);
    return launch_product<Tile, 64, 256, 32, 128, 6, kExact>(A, C, s);
}
template <Keep kKeep>
hipError_t forward(bool sums8, const ProductArgs &A, const typename GatedTile<kNone>::Args &B, hipStream_t s) {
    return sums8 ? forward<kKeep, false>(A, B, s) : forward<kKeep, true>(A, B, s);
}

template <Keep kKeep, bool kExact>
hipError_t backward(const ProductArgs &A, const typename GatedBackTile<kEight>::Args &B, hipStream_t s) {
    typedef GatedBackTile<kKeep> Tile;
    const typename Tile::Args C{B.weights, B.kept, B.kept_scale, B.dgu, B.q, B.q_scale, B.dots, B.ib, B.qs};
    // Two workgroups a CU; with 8-bit sums the largest tiles where every CU has two.
    // Measured, us for 8 groups, hidden 4096, inter 2048 with tiles of 256 x 256, 128 x 128,
    // 64 x 128: 8192 rows a group 1135, 1214, 1425; 4000 rows 612, 602, 696; 1000 rows 222,
    // 167, 208; 400 rows 110, 78, 88; 200 rows 106, 49, 52; 100 rows 103, 46, 46.  65536 rows in
    // 16 groups of 512 x 1024: 246, 222, 314.  With 8-bit sums, 8192 rows a group: 815, 952,
    // 1218; 1000 rows (256 of the largest) 148, 130, 168; 400 rows 75, 59, 77; 200 rows 71, 37,
    // 46; 100 rows 66, 34, 32.
    const int64_t rows = A.groups.M / A.groups.G;
    if constexpr (!kExact)
        if (rows >= 256 && ceil_div(A.groups.M, 256) * ceil_div(A.N, 256) >= 512)
            return launch_product<Tile, 256, 256, 64, 128, 4>(A, C, s);
    if (rows >= 128) return launch_product<Tile, 128, 128, 32, 128, 4, kExact>(A, C, s);
    return launch_product<Tile, 64, 128, 32, 128, 6, kExact>(A, C, s);
}
template <Keep kKeep>
hipError_t backward(bool sums8, const ProductArgs &A, const typename GatedBackTile<kEight>::Args &B, hipStream_t s) {
    return sums8 ? backward<kKeep, false>(A, B, s) : backward<kKeep, true>(A, B, s);
}

// what a matrix argument becomes
struct Matrix {
    const uint8_t *w, *ws, *slot_w, *slot_ws;
    int64_t w_stride, ws_stride, slot_w_stride, slot_ws_stride;
    Matrix(const ep_matrix_t &m, const ep_matrix_t &slot)
        : w(static_cast<const uint8_t *>(m.data)), ws(m.scale), slot_w(static_cast<const uint8_t *>(slot.data)),
          slot_ws(slot.scale), w_stride(m.stride), ws_stride(m.scale_stride), slot_w_stride(slot.stride),
          slot_ws_stride(slot.scale_stride) {}
};

void set_matrix(ProductArgs *A, const Matrix &m) {
    A->w = m.w, A->ws = m.ws, A->slot_w = m.slot_w, A->slot_ws = m.slot_ws;
    A->w_stride = m.w_stride, A->ws_stride = m.ws_stride;
    A->slot_w_stride = m.slot_w_stride, A->slot_ws_stride = m.slot_ws_stride;
}

bool keep_dtype(int32_t d) { return d == EP_DTYPE_BF16 || d == EP_DTYPE_FP8; }

// what is kept, or was: bf16 [m][2 inter], or bytes with their scales
bool kept_ok(int32_t dtype, const void *kept, const uint8_t *scale) {
    return dtype == EP_DTYPE_BF16 ? kept && is_aligned(kept, 2)
                                  : kept && scale && is_aligned(kept, 16) && is_aligned(scale, 4);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_grouped_swiglu(const ep_grouped_swiglu_t *p, ep_stream_t stream) {
    if (!p) return EP_ERR_INVALID_ARG;
    const ProductShape shape{p->x, p->x_scale, p->x_rows, p->rows, p->rows_div, p->groups, p->offsets, p->m, p->inter,
                             p->k, p->weights, p->weights_count};
    if (!product_sizes_ok(shape) || (p->keep && !keep_dtype(p->keep_dtype)) || (p->sums8 != 0 && p->sums8 != 1))
        return EP_ERR_INVALID_ARG;
    if (p->m == 0) return EP_OK;
    const bool slots = p->slot_gate.data && p->slot_gate.scale && p->slot_up.data && p->slot_up.scale;
    ProductArgs A;
    if (!product_args(shape, p->layout, slots, &A) ||
        !product_matrix_ok(p->gate, p->slot_gate, p->layout, p->groups, p->inter, p->k) ||
        !product_matrix_ok(p->up, p->slot_up, p->layout, p->groups, p->inter, p->k))
        return EP_ERR_INVALID_ARG;
    if (!p->h || !p->h_scale || !is_aligned(p->h, 16) || !is_aligned(p->h_scale, 4) ||
        (p->keep && !kept_ok(p->keep_dtype, p->keep, p->keep_scale)))
        return EP_ERR_INVALID_ARG;
    set_matrix(&A, Matrix(p->gate, p->slot_gate));
    const Matrix up(p->up, p->slot_up);
    const int ib = (int)ceil_div(p->inter, kScaleBlock);
    const GatedTile<kNone>::Args B{
        SecondArgs{up.w, up.ws, up.slot_w, up.slot_ws, up.w_stride, up.ws_stride, up.slot_w_stride, up.slot_ws_stride},
        p->weights, p->h, p->h_scale, p->keep, p->keep_scale, ib, (int32_t)ep_scale_stride(p->inter),
        (int32_t)ep_scale_stride((int64_t)2 * ib * kScaleBlock)};
    const hipStream_t s = to_stream(stream);
    const bool sums8 = p->sums8 != 0;
    if (!p->keep) return rc_of(forward<kNone>(sums8, A, B, s));
    return rc_of(p->keep_dtype == EP_DTYPE_BF16 ? forward<kSixteen>(sums8, A, B, s) : forward<kEight>(sums8, A, B, s));
}

extern "C" size_t ep_swiglu_backward_workspace_bytes(int64_t m, int64_t inter) {
    if (m < 1 || m > kMaxRows || inter < 1 || inter > (1 << 24)) return 0;
    return (size_t)m * (size_t)ceil_div(inter, kScaleBlock) * sizeof(float);
}

extern "C" int ep_grouped_swiglu_backward(const ep_grouped_swiglu_backward_t *p, ep_stream_t stream) {
    if (!p) return EP_ERR_INVALID_ARG;
    const ProductShape shape{p->dy, p->dy_scale, p->dy_rows, p->rows, p->rows_div, p->groups, p->offsets, p->m,
                             p->inter, p->k, p->weights, p->weights_count};
    if (!product_sizes_ok(shape) || !keep_dtype(p->keep_dtype) || (p->sums8 != 0 && p->sums8 != 1))
        return EP_ERR_INVALID_ARG;
    if (p->grad_weights && (!float_dtype(p->grad_weights_dtype) || p->pairs < 0 || p->pairs > kMaxBlocks * kDotThreads ||
                            !is_aligned(p->grad_weights, p->grad_weights_dtype == EP_DTYPE_BF16 ? 2 : 4) ||
                            !is_aligned(p->pos, 4) || (!p->pos && p->pairs != p->m)))
        return EP_ERR_INVALID_ARG;
    if (p->m > 0) {
        ProductArgs A;
        if (!product_args(shape, p->layout, p->slot_down.data && p->slot_down.scale, &A) ||
            !product_matrix_ok(p->down, p->slot_down, p->layout, p->groups, p->inter, p->k))
            return EP_ERR_INVALID_ARG;
        if (!kept_ok(p->keep_dtype, p->keep, p->keep_scale) || !is_aligned(p->grad, 2) ||
            (!p->q != !p->q_scale) || !is_aligned(p->q, 16) || !is_aligned(p->q_scale, 4) ||
            (!p->grad && !p->q && !p->grad_weights))
            return EP_ERR_INVALID_ARG;
        if (p->grad_weights && (!p->ws || !is_aligned(p->ws, 16) ||
                                p->ws_bytes < ep_swiglu_backward_workspace_bytes(p->m, p->inter)))
            return EP_ERR_INVALID_ARG;
        set_matrix(&A, Matrix(p->down, p->slot_down));
        const int ib = (int)ceil_div(p->inter, kScaleBlock);
        const GatedBackTile<kEight>::Args B{p->weights, p->keep, p->keep_scale, static_cast<uint16_t *>(p->grad), p->q,
                                            p->q_scale, p->grad_weights ? static_cast<float *>(p->ws) : nullptr, ib,
                                            (int32_t)ep_scale_stride((int64_t)2 * ib * kScaleBlock)};
        const hipStream_t s = to_stream(stream);
        const bool sums8 = p->sums8 != 0;
        const hipError_t e = p->keep_dtype == EP_DTYPE_BF16 ? backward<kSixteen>(sums8, A, B, s)
                                                            : backward<kEight>(sums8, A, B, s);
        if (e != hipSuccess) return EP_ERR_HIP;
    }
    if (p->grad_weights && p->pairs > 0) {
        const int64_t blocks = ceil_div(p->pairs, kDotThreads);
        const int ib = (int)ceil_div(p->inter, kScaleBlock);
        auto run = [&](auto kernel) {
            kernel<<<(uint32_t)blocks, kDotThreads, 0, to_stream(stream)>>>(static_cast<const float *>(p->ws), ib, p->m,
                                                                            p->pos, p->pairs, p->grad_weights);
        };
        p->grad_weights_dtype == EP_DTYPE_BF16 ? run(pair_dots_kernel<true>) : run(pair_dots_kernel<false>);
        return rc_of(hipGetLastError());
    }
    return EP_OK;
}
