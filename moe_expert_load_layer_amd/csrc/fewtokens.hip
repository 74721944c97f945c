// A whole mixture-of-experts layer for a few tokens (at most 64), in two kernels:
//   up    gate (gate.h), then h_p = silu(Wg_e x_t) * (Wu_e x_t) for every pair p = (t, j), e = id_tj
//   down  out_t = sum_j w_tj Wd_e h_p
//
// Bound: HBM.  Every distinct expert's three matrices are read once, which is
// all but a fraction of a percent of the bytes.  The tokens of one expert are
// the 16 columns of a matrix instruction (2 or 4 column tiles for experts
// with more), the weights its 16 rows, loaded straight into registers: no
// weight is used twice by a workgroup, so LDS would only add a hop.
//
// up: one work item is 8 rows of the gate and the same 8 rows of the up matrix
// (one 16-row tile) of one expert; its 8 waves take every eighth 128-byte
// window of the rows and meet in LDS, in wave order.  A fixed grid of two
// workgroups per CU walks the items, so that each workgroup chooses experts and
// groups pairs once.  h is kept as the sum of two bf16 (16 bits of mantissa):
// one bf16 would add as much error as the output's own rounding.
// down: one workgroup owns 16 rows of the output over all experts, its waves
// equal shares of the (expert, window) sequence; partial sums stay per wave in
// LDS and are added in wave order.  No atomics on sums: results do not depend
// on scheduling.
//
// 8-bit weights: a window is 128 values with one scale byte; v_cvt_scalef32
// gives bf16 exactly (3 bits of mantissa, power-of-two scale), so products and
// sums are those of the bf16 path.
#include "gate.h"

namespace ep {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kMaxTokens = EP_MAX_FEW_TOKENS;
constexpr int kMaxPairs = kMaxTokens * kGateMaxK;
constexpr int kUnroll = 4;         // windows whose loads are in flight together
constexpr int kWindowBytes = 128;  // of one weight row

struct Matrix {
    const uint8_t *data;
    const uint8_t *scale;
    int64_t stride, scale_stride;  // bytes between experts
};

struct FewArgs {
    GateArgs gate;
    const uint16_t *x;
    int64_t x_stride, out_stride;  // elements
    Matrix wg, wu, wd;
    int32_t T, H, I, k;
    int32_t *ids;
    float *weights;
    uint16_t *out;
    uint16_t *hhi, *hlo;  // [T * k][I]
};

// The pairs of each chosen expert, in LDS.
struct Lists {
    int32_t ids[kMaxPairs];
    uint16_t pair[kMaxPairs];             // pairs ordered by expert
    uint16_t expert[kGateMaxExperts];     // the chosen experts, ascending
    uint16_t start[kGateMaxExperts + 1];  // their first entry in `pair`
    int32_t count[kGateMaxExperts];       // pairs of each expert, then fill cursors
    int32_t active;
};

// L->ids holds T * k IDs.  The order of an expert's pairs does not matter to
// any result: a pair is a column of its own.
__device__ void build_lists(Lists *L, int pairs, int E) {
    for (int e = threadIdx.x; e < E; e += kThreads) L->count[e] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kThreads)
        if (L->ids[p] >= 0) atomicAdd(&L->count[L->ids[p]], 1);
    __syncthreads();
    if (threadIdx.x < kWave) {
        int act = 0, first = 0;
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int e = e0 + (int)threadIdx.x;
            const int c = e < E ? L->count[e] : 0;
            const uint64_t on = __ballot(c > 0);
            const int incl = wave_incl_scan_i32(c);
            if (c > 0) {
                const int a = act + __popcll(on & lanemask_lt());
                L->expert[a] = (uint16_t)e;
                L->start[a] = (uint16_t)(first + incl - c);
            }
            if (e < E) L->count[e] = first + incl - c;
            act += __popcll(on);
            first += __builtin_amdgcn_readlane(incl, kWave - 1);
        }
        if (threadIdx.x == 0) {
            L->active = act;
            L->start[act] = (uint16_t)first;
        }
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kThreads)
        if (L->ids[p] >= 0) L->pair[atomicAdd(&L->count[L->ids[p]], 1)] = (uint16_t)p;
    __syncthreads();
}

// The 128-byte window `win` of a weight row, as this lane's part: bf16 two
// times 8 values at k = 64 win + 8 q and + 32, 8 bits two times 16 values at
// k = 128 win + 32 q and + 16.
template <bool kFp8>
__device__ __forceinline__ void load_window(const uint8_t *row, int win, int q, int K, u32x4 (&w)[2]) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
        int off = win * kWindowBytes + (kFp8 ? q * 32 + j * 16 : q * 16 + j * 64);
        if (!kFp8 && off >= K * 2) off = 0;  // past the row's end: not used (8-bit rows are whole windows)
        w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(row + off));
    }
}

template <bool kFp8>
constexpr int kSteps = kFp8 ? 4 : 2;  // matrix instructions of a window

// first value of step s of window win in this lane
template <bool kFp8>
__device__ __forceinline__ int step_k(int win, int q, int s) {
    return kFp8 ? win * 128 + q * 32 + s * 8 : win * 64 + q * 8 + s * 32;
}

// the weights of step s as 8 bf16
template <bool kFp8>
__device__ __forceinline__ bf16x8 step_weights(const u32x4 (&w)[2], int s, float scale) {
    if constexpr (kFp8) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        union {
            bf16x2 h[4];
            bf16x8 v;
        } u;
        const uint32_t a = w[s / 2][2 * (s % 2)], b = w[s / 2][2 * (s % 2) + 1];
        u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false);
        u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true);
        u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false);
        u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true);
        return u.v;
    } else {
        return __builtin_bit_cast(bf16x8, w[s]);
    }
}

// acc[n] += rows x columns over the windows first, first + stride, ... below
// last.  col[n][c]: this lane's column of tile n, kParts arrays summed.
template <bool kFp8, int NT, int kParts>
__device__ __forceinline__ void stream_rows(const uint8_t *row, const uint8_t *scale, int K, int first, int last,
                                            int stride, int q, const uint16_t *const (&col)[kParts][NT],
                                            f32x4 (&acc)[NT]) {
    for (int w0 = first; w0 < last; w0 += kUnroll * stride) {
        u32x4 w[kUnroll][2];
        float sc[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int win = min(w0 + u * stride, last - 1);  // past the end: loaded, not used
            load_window<kFp8>(row, win, q, K, w[u]);
            sc[u] = kFp8 ? pow2_of(scale[win]) : 1.0f;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int win = w0 + u * stride;
            if (win >= last) break;
#pragma unroll
            for (int s = 0; s < kSteps<kFp8>; s++) {
                const int k = step_k<kFp8>(win, q, s);
                const bool in = k < K;  // K is a multiple of 8
                const u32x4 zero{0, 0, 0, 0};
                bf16x8 a = step_weights<kFp8>(w[u], s, sc[u]);
                if (!in) a = __builtin_bit_cast(bf16x8, zero);
#pragma unroll
                for (int c = 0; c < kParts; c++)
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        const u32x4 b = in ? *reinterpret_cast<const u32x4 *>(col[c][n] + k) : zero;
                        acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, b), acc[n], 0,
                                                                         0, 0);
                    }
            }
        }
    }
}

template <bool kFp8>
__device__ __forceinline__ int windows_of(int K) {
    return kFp8 ? (K + 127) / 128 : (K + 63) / 64;
}

template <bool kFp8>
__device__ __forceinline__ int64_t row_bytes(int K) {
    return kFp8 ? (int64_t)((K + 127) / 128) * 128 : (int64_t)K * 2;
}

// One item: rows i0 .. i0 + 7 of gate and up of one expert, columns = its pairs.
template <bool kFp8, int NT>
__device__ __forceinline__ void up_item(const FewArgs &A, const Lists *L, int a, int i0, float *red) {
    const int wave = threadIdx.x / kWave, l = lane_id(), r = l & 15, q = l >> 4;
    const int e = L->expert[a], first = L->start[a], n = L->start[a + 1] - first;
    const int i = min(i0 + (r & 7), A.I - 1);
    const Matrix &M = r < 8 ? A.wg : A.wu;
    const uint8_t *row = M.data + e * M.stride + i * row_bytes<kFp8>(A.H);
    const int nw = windows_of<kFp8>(A.H);
    const uint8_t *scale = kFp8 ? M.scale + e * M.scale_stride + (int64_t)(i / kScaleBlock) * nw : nullptr;
    const uint16_t *col[1][NT];
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int c = min(t * 16 + r, n - 1);  // columns past the end repeat the last
        col[0][t] = A.x + (int64_t)(L->pair[first + c] / A.k) * A.x_stride;
        acc[t] = f32x4{0, 0, 0, 0};
    }
    stream_rows<kFp8, NT, 1>(row, scale, A.H, wave, nw, kWaves, q, col, acc);
    // red [wave][column][16 rows]: a lane's 4 rows are one 16-byte store
#pragma unroll
    for (int t = 0; t < NT; t++)
        *reinterpret_cast<f32x4 *>(red + ((wave * NT + t) * 16 + r) * 16 + 4 * q) = acc[t];
    __syncthreads();
    for (int o = threadIdx.x; o < NT * 16 * 8; o += kThreads) {
        const int c = o / 8, j = o % 8;
        if (c >= n || i0 + j >= A.I) continue;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; w++) {
            g += red[(w * NT * 16 + c) * 16 + j];
            u += red[(w * NT * 16 + c) * 16 + 8 + j];
        }
        const float h = g / (1.0f + expf(-g)) * u;
        const int64_t at = (int64_t)L->pair[first + c] * A.I + i0 + j;
        const uint16_t hi = to_bf16(h);
        const float rest = h - __builtin_bit_cast(float, (uint32_t)hi << 16);
        A.hhi[at] = hi;
        // an h that is infinite as bf16, or NaN, has no rest
        A.hlo[at] = to_bf16(fabsf(rest) < INFINITY ? rest : 0.0f);
    }
    __syncthreads();
}

template <bool kFp8, int V>
__global__ __launch_bounds__(kThreads, 4) void up_kernel(const FewArgs A) {
    __shared__ Lists L;
    __shared__ union {
        GateSlot slot[kThreads / kGateLanes];
        float red[kWaves * 4 * 256];
    } S;
    // every workgroup chooses for itself; the first one writes the choice
    constexpr int kPass = kThreads / kGateLanes;
    for (int t0 = 0; t0 < A.T; t0 += kPass) {
        const int s = threadIdx.x / kGateLanes, j = threadIdx.x % kGateLanes, t = t0 + s;
        int id;
        float w;
        gate_token<V>(A.gate, min(t, A.T - 1), &S.slot[s], id, w);
        if (t < A.T && j < A.k) {
            L.ids[t * A.k + j] = id;
            if (blockIdx.x == 0) {
                A.ids[t * A.k + j] = id;
                A.weights[t * A.k + j] = w;
            }
        }
    }
    __syncthreads();
    build_lists(&L, A.T * A.k, A.gate.E);
    const int tiles = (A.I + 7) / 8, items = L.active * tiles;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int a = it / tiles, i0 = (it - a * tiles) * 8;
        const int n = L.start[a + 1] - L.start[a];
        if (n <= 16) up_item<kFp8, 1>(A, &L, a, i0, S.red);
        else if (n <= 32) up_item<kFp8, 2>(A, &L, a, i0, S.red);
        else up_item<kFp8, 4>(A, &L, a, i0, S.red);
    }
}

// windows [w0, w1) of expert a for output rows o0 .. o0 + 15, into `part`
template <bool kFp8, int NT>
__device__ __forceinline__ void down_run(const FewArgs &A, const Lists *L, int a, int o0, int w0, int w1,
                                         float *part) {
    const int l = lane_id(), r = l & 15, q = l >> 4;
    const int e = L->expert[a], first = L->start[a], n = L->start[a + 1] - first;
    const int o = min(o0 + r, A.H - 1);
    const uint8_t *row = A.wd.data + e * A.wd.stride + o * row_bytes<kFp8>(A.I);
    const uint8_t *scale =
        kFp8 ? A.wd.scale + e * A.wd.scale_stride + (int64_t)(o / kScaleBlock) * windows_of<kFp8>(A.I) : nullptr;
    const uint16_t *col[2][NT];
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int64_t at = (int64_t)L->pair[first + min(t * 16 + r, n - 1)] * A.I;
        col[0][t] = A.hhi + at;
        col[1][t] = A.hlo + at;
        acc[t] = f32x4{0, 0, 0, 0};
    }
    stream_rows<kFp8, NT, 2>(row, scale, A.I, w0, w1, 1, q, col, acc);
    // the wave's own sums: an expert has a token once, so lanes do not meet
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int c = t * 16 + r;
        if (c < n) {
            const int p = L->pair[first + c];
            f32x4 *d = reinterpret_cast<f32x4 *>(part + (p / A.k) * 16 + 4 * q);
            const float w = A.weights[p];
            f32x4 v = *d;
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] += w * acc[t][i];
            *d = v;
        }
    }
}

template <bool kFp8>
__global__ __launch_bounds__(kThreads, 4) void down_kernel(const FewArgs A) {
    __shared__ Lists L;
    extern __shared__ float part[];  // [kWaves][T][16]
    for (int p = threadIdx.x; p < A.T * A.k; p += kThreads) L.ids[p] = A.ids[p];
    for (int i = threadIdx.x; i < kWaves * A.T * 16; i += kThreads) part[i] = 0.0f;
    __syncthreads();
    build_lists(&L, A.T * A.k, A.gate.E);
    const int wave = threadIdx.x / kWave, o0 = blockIdx.x * 16;
    const int nw = windows_of<kFp8>(A.I), units = L.active * nw;
    const int u1 = (int)((int64_t)units * (wave + 1) / kWaves);
    float *mine = part + wave * A.T * 16;
    for (int u = (int)((int64_t)units * wave / kWaves); u < u1;) {
        const int a = u / nw, w0 = u - a * nw, w1 = min(nw, w0 + (u1 - u));
        const int n = L.start[a + 1] - L.start[a];
        if (n <= 16) down_run<kFp8, 1>(A, &L, a, o0, w0, w1, mine);
        else if (n <= 32) down_run<kFp8, 2>(A, &L, a, o0, w0, w1, mine);
        else down_run<kFp8, 4>(A, &L, a, o0, w0, w1, mine);
        u += w1 - w0;
        wave_lds_fence();  // the next expert adds to sums that other lanes wrote
    }
    __syncthreads();
    for (int i = threadIdx.x; i < A.T * 16; i += kThreads) {
        const int t = i / 16, o = o0 + i % 16;
        if (o >= A.H) continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; w++) s += part[w * A.T * 16 + i];
        A.out[t * A.out_stride + o] = to_bf16(s);
    }
}

template <bool kFp8>
hipError_t launch(const FewArgs &A, hipStream_t s) {
    const int64_t most = (int64_t)(A.gate.E < A.T * A.k ? A.gate.E : A.T * A.k) * ((A.I + 7) / 8);
    const int per = (A.gate.E + kGateLanes - 1) / kGateLanes;
    const void *fn = per <= 8    ? (const void *)up_kernel<kFp8, 8>
                     : per <= 16 ? (const void *)up_kernel<kFp8, 16>
                     : per <= 24 ? (const void *)up_kernel<kFp8, 24>
                     : per <= 32 ? (const void *)up_kernel<kFp8, 32>
                                 : (const void *)up_kernel<kFp8, 64>;
    const int64_t resident = resident_blocks(fn, kThreads, 0);
    const int64_t blocks = resident > 0 && resident < most ? resident : most;
    void *args[] = {const_cast<FewArgs *>(&A)};
    hipError_t e = hipLaunchKernel(fn, dim3((uint32_t)blocks), dim3(kThreads), args, 0, s);
    if (e != hipSuccess) return e;
    down_kernel<kFp8><<<(uint32_t)ceil_div(A.H, 16), kThreads, (size_t)kWaves * A.T * 16 * sizeof(float), s>>>(A);
    return hipGetLastError();
}

// one expert matrix [rows][K]: pointers, alignment and strides that hold it
bool matrix_ok(const ep_matrix_t &m, bool fp8, int64_t rows, int64_t K, int32_t E) {
    const int64_t bytes = rows * (fp8 ? ceil_div(K, 128) * 128 : K * 2);
    if (!m.data || !is_aligned(m.data, 16) || m.stride % 16 != 0 || (E > 1 && m.stride < bytes)) return false;
    return !fp8 || (m.scale && (E == 1 || m.scale_stride >= ceil_div(rows, kScaleBlock) * ceil_div(K, kScaleBlock)));
}

Matrix matrix_of(const ep_matrix_t &m) {
    return Matrix{static_cast<const uint8_t *>(m.data), m.scale, m.stride, m.scale_stride};
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_few_tokens_workspace_bytes(int32_t num_tokens, int32_t top_k, int32_t inter) {
    if (num_tokens < 0 || num_tokens > kMaxTokens || top_k < 1 || top_k > kGateMaxK || inter < 1) return 0;
    return (size_t)num_tokens * top_k * inter * 2 * sizeof(uint16_t);
}

extern "C" int ep_moe_few_tokens(const void *x, int64_t x_stride, int32_t num_tokens, const void *logits,
                                 int64_t logits_stride, const ep_gate_t *gate, const ep_experts_t *experts, void *out,
                                 int64_t out_stride, int32_t *ids, float *weights, void *ws, size_t ws_bytes,
                                 ep_stream_t stream) {
    if (!gate_ok(gate) || !experts || num_tokens < 0 || num_tokens > kMaxTokens) return EP_ERR_INVALID_ARG;
    const int32_t H = experts->hidden, I = experts->inter, E = gate->num_experts;
    if (H < 8 || I < 8 || H % 8 != 0 || I % 8 != 0 || H > (1 << 20) || I > (1 << 20)) return EP_ERR_INVALID_ARG;
    if (experts->dtype != EP_DTYPE_BF16 && experts->dtype != EP_DTYPE_FP8) return EP_ERR_INVALID_ARG;
    const bool fp8 = experts->dtype == EP_DTYPE_FP8;
    if (!matrix_ok(experts->gate, fp8, I, H, E) || !matrix_ok(experts->up, fp8, I, H, E) ||
        !matrix_ok(experts->down, fp8, H, I, E))
        return EP_ERR_INVALID_ARG;
    if (logits_stride < E || x_stride < H || x_stride % 8 != 0 || out_stride < H) return EP_ERR_INVALID_ARG;
    if (num_tokens == 0) return EP_OK;
    const size_t width = gate->logits_dtype == EP_DTYPE_BF16 ? 2 : 4;
    if (!x || !logits || !out || !ids || !weights || !is_aligned(x, 16) || !is_aligned(logits, width) ||
        !is_aligned(out, 2) || !is_aligned(ids, 4) || !is_aligned(weights, 4))
        return EP_ERR_INVALID_ARG;
    if (!ws || !is_aligned(ws, 16) || ws_bytes < ep_few_tokens_workspace_bytes(num_tokens, gate->top_k, I))
        return EP_ERR_INVALID_ARG;
    FewArgs A;
    A.gate = gate_args(logits, logits_stride, gate);
    A.x = static_cast<const uint16_t *>(x);
    A.x_stride = x_stride;
    A.out_stride = out_stride;
    A.wg = matrix_of(experts->gate);
    A.wu = matrix_of(experts->up);
    A.wd = matrix_of(experts->down);
    A.T = num_tokens;
    A.H = H;
    A.I = I;
    A.k = gate->top_k;
    A.ids = ids;
    A.weights = weights;
    A.out = static_cast<uint16_t *>(out);
    A.hhi = static_cast<uint16_t *>(ws);
    A.hlo = A.hhi + (size_t)num_tokens * gate->top_k * I;
    return rc_of(fp8 ? launch<true>(A, to_stream(stream)) : launch<false>(A, to_stream(stream)));
}
