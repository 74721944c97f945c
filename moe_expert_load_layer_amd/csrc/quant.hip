// Rounding to 8-bit floating point (e4m3) with a power-of-two scale for each
// block of 128, and the two elementwise steps between the experts' products.
//
// A block's scale is 2^(c - 127) with the byte c the smallest for which its
// largest finite magnitude is at most 448 scales.  Scaling by a power of two is
// exact, so a value is rounded once, to nearest with ties to even.  NaN and
// infinities become NaN, and leave their block's scale alone.  All four kernels are one pass over the data, bound by HBM.
// Measured, bytes read and written once (a 2 GiB copy reaches 4.95 TB/s):
//   rows of bf16      65536 x 4096      139 us  5.8 TB/s   (8192 x 4096: 22 us, 4.6)
//   rows of fp32      32768 x 4096      115 us  5.8 TB/s
//   silu(g) u         65536 x 2 x 2048  113 us  6.0 TB/s
//   blocks of bf16    16 x 8192 x 4096  288 us  5.6 TB/s, transposed or not
//   combine           8192 x 8 x 4096   126 us  4.8 TB/s
//
// A unit is one row's block: 16 lanes (a DPP row) of 8 values, so that loads
// are 16 (bf16) or 32 bytes a lane and the block's maximum takes 4 DPP steps.
#include "layer.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kUnitLanes = kScaleBlock / 8;
constexpr int kUnits = kThreads / kUnitLanes;  // blocks of a workgroup

__device__ __forceinline__ int fp8_scale_code(float amax) {
    const uint32_t b = __builtin_bit_cast(uint32_t, amax);
    const int c = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u);
    return min(max(c, 1), 254);
}

// x / 2^(c - 127) as 8 bytes.  The conversion turns infinities into NaN.
__device__ __forceinline__ u32x2 to_fp8(const float (&x)[8], int c) {
    const float inv = pow2_of(254 - c);
    u32x2 q;
#pragma unroll
    for (int j = 0; j < 2; j++) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * j] * inv, x[4 * j + 1] * inv, 0, false);
        q[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * j + 2] * inv, x[4 * j + 3] * inv, w, true);
    }
    return q;
}

// 8 values of a row from column k on, zeros past its K columns
template <bool kBf16>
__device__ __forceinline__ void load_row8(const void *x, int64_t at, int64_t k, int64_t K, float (&v)[8]) {
    if constexpr (kBf16) {
        const uint16_t *p = static_cast<const uint16_t *>(x) + at + k;
        if (k + 8 <= K) {
            const u32x4 w = *reinterpret_cast<const u32x4_at2 *>(p);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                v[2 * j] = bf16_lo(w[j]);
                v[2 * j + 1] = bf16_hi(w[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = k + j < K ? __builtin_bit_cast(float, (uint32_t)p[j] << 16) : 0.0f;
        }
    } else {
        const float *p = static_cast<const float *>(x) + at + k;
        if (k + 8 <= K) {
            const f32x4 a = reinterpret_cast<const f32x4_at4 *>(p)[0], b = reinterpret_cast<const f32x4_at4 *>(p)[1];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                v[j] = a[j];
                v[4 + j] = b[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = k + j < K ? p[j] : 0.0f;
        }
    }
}

// The largest finite magnitude: infinity * 0 is NaN, and fmaxf passes over NaN
__device__ __forceinline__ float amax8(const float (&v)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) m = fmaxf(m, fmaf(v[j], 0.0f, fabsf(v[j])));
    return m;
}

// q [M][128 kb], scale [M][sb]; sb is kb rounded up to 4, the bytes past kb are 127
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(const void *__restrict__ x, int64_t stride, int64_t M,
                                                              int64_t K, int kb, int sb, uint8_t *__restrict__ q,
                                                              uint8_t *__restrict__ scale) {
    const int64_t u = (int64_t)blockIdx.x * kUnits + threadIdx.x / kUnitLanes;
    const int lane = threadIdx.x % kUnitLanes;
    const int64_t m = u / sb;
    const int b = (int)(u - m * sb);
    if (m >= M) return;  // whole DPP rows leave
    if (b >= kb) {
        if (lane == 0) scale[m * sb + b] = 127;
        return;
    }
    float v[8];
    load_row8<kBf16>(x, m * stride, (int64_t)b * kScaleBlock + lane * 8, K, v);
    const int c = fp8_scale_code(row_max_f32(amax8(v)));
    *reinterpret_cast<u32x2 *>(q + (m * kb + b) * kScaleBlock + lane * 8) = to_fp8(v, c);
    if (lane == 0) scale[m * sb + b] = (uint8_t)c;
}

// The same for silu(gate) * up, gate and up the halves of a bf16 row of 2 I
// values.  The sigmoid takes the hardware's exponential and reciprocal (2^-16 of
// a value at most, against the 2^-4 of the rounding that follows): with exact
// division and exponential, arithmetic bounds the pass, 199 us for 65536 x 2048.
__global__ __launch_bounds__(kThreads) void swiglu_quant_kernel(const uint16_t *__restrict__ x, int64_t M, int64_t I,
                                                                int kb, int sb, uint8_t *__restrict__ q,
                                                                uint8_t *__restrict__ scale) {
    const int64_t u = (int64_t)blockIdx.x * kUnits + threadIdx.x / kUnitLanes;
    const int lane = threadIdx.x % kUnitLanes;
    const int64_t m = u / sb;
    const int b = (int)(u - m * sb);
    if (m >= M) return;
    if (b >= kb) {
        if (lane == 0) scale[m * sb + b] = 127;
        return;
    }
    float g[8], v[8];
    load_row8<true>(x, m * 2 * I, (int64_t)b * kScaleBlock + lane * 8, I, g);
    load_row8<true>(x, m * 2 * I + I, (int64_t)b * kScaleBlock + lane * 8, I, v);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] *= g[j] * __builtin_amdgcn_rcpf(1.0f + __expf(-g[j]));
    const int c = fp8_scale_code(row_max_f32(amax8(v)));
    *reinterpret_cast<u32x2 *>(q + (m * kb + b) * kScaleBlock + lane * 8) = to_fp8(v, c);
    if (lane == 0) scale[m * sb + b] = (uint8_t)c;
}

// One 128 x 128 block of a weight matrix [N][K] a workgroup; kTrans writes the
// transposed matrix [K][N up to 128] and its transposed scales.
template <bool kBf16, bool kTrans>
__global__ __launch_bounds__(kThreads) void quant_blocks_kernel(const void *__restrict__ w, int64_t group_stride,
                                                                int64_t N, int64_t K, int nb, int kb,
                                                                uint8_t *__restrict__ q,
                                                                uint8_t *__restrict__ scale) {
    __shared__ float top[kThreads / kWave];
    // rows of 128 bytes and 8 more: the transposing byte writes spread over the banks
    __shared__ __align__(8) uint8_t tile[kTrans ? 128 * 136 : 8];
    const int64_t g = blockIdx.z;
    const int bn = blockIdx.y, bk = blockIdx.x, c0 = (threadIdx.x % 16) * 8, r0 = threadIdx.x / 16;
    float v[8][8], m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t n = (int64_t)bn * 128 + r0 + 16 * i;
        if (n < N) {
            load_row8<kBf16>(w, g * group_stride + n * K, (int64_t)bk * 128 + c0, K, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] = 0.0f;
        }
        m = fmaxf(m, amax8(v[i]));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    if (threadIdx.x % kWave == 0) top[threadIdx.x / kWave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const int c = fp8_scale_code(m);
    if (threadIdx.x == 0) scale[(g * nb + (kTrans ? 0 : bn)) * kb + (kTrans ? (int64_t)bk * nb + bn : bk)] = (uint8_t)c;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const u32x2 b = to_fp8(v[i], c);
        const int64_t n = (int64_t)bn * 128 + r0 + 16 * i;
        if constexpr (kTrans) {
#pragma unroll
            for (int j = 0; j < 8; j++) tile[(c0 + j) * 136 + r0 + 16 * i] = (uint8_t)(b[j / 4] >> (8 * (j % 4)));
        } else if (n < N) {
            *reinterpret_cast<u32x2 *>(q + ((g * N + n) * kb + bk) * 128 + c0) = b;
        }
    }
    if constexpr (kTrans) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int64_t k = (int64_t)bk * 128 + r0 + 16 * i;
            if (k < K)
                *reinterpret_cast<u32x2 *>(q + ((g * K + k) * nb + bn) * 128 + c0) =
                    *reinterpret_cast<const u32x2 *>(tile + (r0 + 16 * i) * 136 + c0);
        }
    }
}

// out_t = sum_j w_tj y[pos_tj] in fp32, j ascending; positions outside [0, rows) give nothing
__global__ __launch_bounds__(kThreads) void combine_kernel(const uint16_t *__restrict__ y, int64_t rows,
                                                           const int32_t *__restrict__ pos,
                                                           const float *__restrict__ weights, int64_t T, int k,
                                                           int64_t H, int64_t chunks,
                                                           uint16_t *__restrict__ out) {
    const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t t = u / chunks, h = (u - t * chunks) * 8;
    if (t >= T) return;
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j = 0; j < k; j++) {
        const int32_t p = pos[t * k + j];
        if (p < 0 || p >= rows) continue;
        const float w = weights[t * k + j];
        float v[8];
        load_row8<true>(y, (int64_t)p * H, h, H, v);
#pragma unroll
        for (int i = 0; i < 8; i++) s[i] += w * v[i];
    }
    uint16_t *o = out + t * H + h;
    if (h + 8 <= H) {
        *reinterpret_cast<u32x4_at2 *>(o) =
            u32x4{pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]), pack_bf16(s[6], s[7])};
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (h + i < H) o[i] = to_bf16(s[i]);
    }
}

constexpr int64_t kMaxDim = 1 << 24;  // columns; block counts fit 32 bits

bool fits_grid(int64_t units, int64_t per) { return ceil_div(units, per) <= kMaxBlocks; }

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int64_t ep_scale_stride(int64_t cols) {
    return cols < 1 ? 0 : ceil_div(ceil_div(cols, kScaleBlock), 4) * 4;
}

extern "C" int ep_quant_rows(const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride, uint8_t *q,
                             uint8_t *scale, ep_stream_t stream) {
    if (!float_dtype(dtype) || rows < 0 || cols < 1 || cols > kMaxDim || stride < cols) return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    const bool bf16 = dtype == EP_DTYPE_BF16;
    const int width = bf16 ? 2 : 4;
    if (!x || !q || !scale || !is_aligned(x, width) || !is_aligned(q, 16) || !is_aligned(scale, 4))
        return EP_ERR_INVALID_ARG;
    const int kb = (int)ceil_div(cols, kScaleBlock), sb = (int)ep_scale_stride(cols);
    if (rows > (int64_t)1 << 40 || !fits_grid(rows * sb, kUnits)) return EP_ERR_INVALID_ARG;
    const uint32_t grid = (uint32_t)ceil_div(rows * sb, kUnits);
    const hipStream_t s = to_stream(stream);
    if (bf16) quant_rows_kernel<true><<<grid, kThreads, 0, s>>>(x, stride, rows, cols, kb, sb, q, scale);
    else quant_rows_kernel<false><<<grid, kThreads, 0, s>>>(x, stride, rows, cols, kb, sb, q, scale);
    return rc_of(hipGetLastError());
}

extern "C" int ep_swiglu_quant(const void *gate_up, int64_t rows, int64_t inter, uint8_t *q, uint8_t *scale,
                               ep_stream_t stream) {
    if (rows < 0 || inter < 1 || inter > kMaxDim) return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    if (!gate_up || !q || !scale || !is_aligned(gate_up, 2) || !is_aligned(q, 16) || !is_aligned(scale, 4))
        return EP_ERR_INVALID_ARG;
    const int kb = (int)ceil_div(inter, kScaleBlock), sb = (int)ep_scale_stride(inter);
    if (rows > (int64_t)1 << 40 || !fits_grid(rows * sb, kUnits)) return EP_ERR_INVALID_ARG;
    swiglu_quant_kernel<<<(uint32_t)ceil_div(rows * sb, kUnits), kThreads, 0, to_stream(stream)>>>(
        static_cast<const uint16_t *>(gate_up), rows, inter, kb, sb, q, scale);
    return rc_of(hipGetLastError());
}

extern "C" int ep_quant_blocks(const void *w, int32_t dtype, int32_t groups, int64_t group_stride, int64_t rows,
                               int64_t cols, int32_t transpose, uint8_t *q, uint8_t *scale, ep_stream_t stream) {
    if (!float_dtype(dtype) || groups < 0 || rows < 1 || cols < 1 || rows > kMaxDim || cols > kMaxDim)
        return EP_ERR_INVALID_ARG;
    if (groups == 0) return EP_OK;
    const int64_t nb = ceil_div(rows, kScaleBlock), kb = ceil_div(cols, kScaleBlock);
    if (groups > 65535 || nb > 65535 || (groups > 1 && group_stride < rows * cols)) return EP_ERR_INVALID_ARG;
    const bool bf16 = dtype == EP_DTYPE_BF16;
    const int width = bf16 ? 2 : 4;
    if (!w || !q || !scale || !is_aligned(w, width) || !is_aligned(q, 16)) return EP_ERR_INVALID_ARG;
    const dim3 grid((uint32_t)kb, (uint32_t)nb, (uint32_t)groups);
    const hipStream_t s = to_stream(stream);
    auto run = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, s>>>(w, group_stride, rows, cols, (int)nb, (int)kb, q, scale);
    };
    if (bf16) transpose ? run(quant_blocks_kernel<true, true>) : run(quant_blocks_kernel<true, false>);
    else transpose ? run(quant_blocks_kernel<false, true>) : run(quant_blocks_kernel<false, false>);
    return rc_of(hipGetLastError());
}

extern "C" int ep_moe_combine(const void *y, int64_t rows, const int32_t *pos, const float *weights,
                              int64_t num_tokens, int32_t top_k, int64_t hidden, void *out, ep_stream_t stream) {
    if (rows < 0 || num_tokens < 0 || top_k < 1 || hidden < 1 || hidden > kMaxDim) return EP_ERR_INVALID_ARG;
    if (num_tokens == 0) return EP_OK;
    if ((rows > 0 && !y) || !pos || !weights || !out || !is_aligned(y, 2) || !is_aligned(out, 2) ||
        !is_aligned(pos, 4) || !is_aligned(weights, 4))
        return EP_ERR_INVALID_ARG;
    const int64_t chunks = ceil_div(hidden, 8);
    if (num_tokens > (int64_t)1 << 38 || !fits_grid(num_tokens * chunks, kThreads)) return EP_ERR_INVALID_ARG;
    combine_kernel<<<(uint32_t)ceil_div(num_tokens * chunks, kThreads), kThreads, 0, to_stream(stream)>>>(
        static_cast<const uint16_t *>(y), rows, pos, weights, num_tokens, top_k, hidden, chunks,
        static_cast<uint16_t *>(out));
    return rc_of(hipGetLastError());
}
