// AdamW over many tensors in one launch, with first and second moments in
// fp32 or in 8 bits.
//
// Per element, in fp32 and rounded after every operation (contraction is off,
// so that the moments, and with them the 8-bit codes, have one value that any
// IEEE implementation reproduces):
//   g = grad * grad_scale
//   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g g
//   p = p (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// 8-bit moments: blocks of 128 elements of the flattened tensor share a scale
// byte c (scale 2^(c - 127), the largest magnitude at most 1.875 scale).  m is
// sign, 4 bits of exponent, 3 of mantissa; v, never negative, 5 bits of
// exponent and 3 of mantissa.  Both codes are bits 20.. of the scaled fp32
// pattern, so encoding is an integer add and a shift.  Rounding is stochastic:
// 20 bits hashed from (seed, step, tensor, element) are added below the code.
// To nearest, v would stand still as soon as one step changes it by less than
// half a code (6 %), long before 1 / (1 - beta2) steps; the random rounding
// keeps its mean.  v > 0 is never stored as 0: m / eps would follow.
//
// Bound: HBM.  28 bytes an element with fp32 moments and gradients, 16 with
// 8-bit moments.  A lane takes 8 consecutive elements (32-byte accesses, 16
// lanes = one scale block = one DPP row, whose maximum takes 4 DPP steps).
// Measured: 8-bit moments 341 us for 113 million elements (5.3 TB/s), their
// values 231 us (4.9); fp32 moments, bf16 gradients and a bf16 copy 507 us for 94
// million (5.2).  12 tensors of 5003 elements take one launch of 4.9 us.
#include <math.h>

#include "layer.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 8;                                   // elements of a lane
constexpr int kChunk = kThreads * kUnit;                   // elements of a workgroup
constexpr int kMaxTensors = 48;                            // descriptors in one launch's arguments
constexpr int kMLow = 896, kVLow = 768;                    // pattern >> 20 of code 0

struct Args {
    ep_adamw_tensor_t t[kMaxTensors];
    uint32_t first[kMaxTensors + 1];  // first workgroup of each tensor
    int32_t n;
};

struct Hyper {
    float beta1, rest1, beta2, rest2, rate, root, eps, decay, gscale;
    uint32_t word, tensor0;  // hash word of the step, index of the launch's first tensor
};

__device__ __forceinline__ uint32_t mix(uint32_t h) {
    h *= 0x9E3779B9u;
    h ^= h >> 15;
    h *= 0x6A09E667u;
    h ^= h >> 13;
    h *= 0xBB67AE85u;
    return h ^ (h >> 16);
}

__device__ __forceinline__ int scale_code(float amax) {
    const uint32_t b = __builtin_bit_cast(uint32_t, amax);
    const int c = (int)(b >> 23) + ((b & 0x7fffffu) > 0x700000u);
    return min(max(c, 1), 253);
}

__device__ __forceinline__ float decode_m(uint32_t q, float s) {
    const uint32_t mag = q & 127u;
    const float x = mag ? __builtin_bit_cast(float, (mag + kMLow) << 20) * s : 0.0f;
    return q & 128u ? -x : x;
}

__device__ __forceinline__ float decode_v(uint32_t q, float s) {
    return q ? __builtin_bit_cast(float, (q + kVLow) << 20) * s : 0.0f;
}

__device__ __forceinline__ uint32_t encode_m(float x, float inv, uint32_t r20) {
    const int c = (int)((__builtin_bit_cast(uint32_t, fabsf(x) * inv) + r20) >> 20) - kMLow;
    return (uint32_t)min(max(c, 0), 127) | (x < 0.0f ? 128u : 0u);
}

__device__ __forceinline__ uint32_t encode_v(float x, float inv, uint32_t r20) {
    const int c = (int)((__builtin_bit_cast(uint32_t, x * inv) + r20) >> 20) - kVLow;
    return x > 0.0f ? (uint32_t)min(max(c, 1), 255) : 0u;
}

// the workgroup's tensor: the last one whose first workgroup is not past b
__device__ __forceinline__ int find_tensor(const Args &A, uint32_t b) {
    int lo = 0, hi = A.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (A.first[mid] <= b) lo = mid; else hi = mid;
    }
    return lo;
}

// 8 values from `base + i`; past the end zeros
template <typename T, bool kBf16>
__device__ __forceinline__ void load8(const void *base, int64_t i, int left, float (&x)[kUnit]) {
    const T *p = static_cast<const T *>(base) + i;
    if (left >= kUnit) {
        if constexpr (kBf16) {
            const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_at2 *>(p));
#pragma unroll
            for (int k = 0; k < 4; k++) {
                x[2 * k] = bf16_lo(w[k]);
                x[2 * k + 1] = bf16_hi(w[k]);
            }
        } else {
            const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4_at4 *>(p));
            const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4_at4 *>(p) + 1);
#pragma unroll
            for (int k = 0; k < 4; k++) {
                x[k] = a[k];
                x[4 + k] = b[k];
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < kUnit; k++) {
            if constexpr (kBf16)
                x[k] = k < left ? __builtin_bit_cast(float, (uint32_t)p[k] << 16) : 0.0f;
            else
                x[k] = k < left ? p[k] : 0.0f;
        }
    }
}

__device__ __forceinline__ void store8(float *base, int64_t i, int left, const float (&x)[kUnit]) {
    float *p = base + i;
    if (left >= kUnit) {
        __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4_at4 *>(p));
        __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, reinterpret_cast<f32x4_at4 *>(p) + 1);
    } else {
#pragma unroll
        for (int k = 0; k < kUnit; k++)
            if (k < left) p[k] = x[k];
    }
}

__device__ __forceinline__ void load_codes(const void *base, int64_t i, int left, uint32_t (&q)[kUnit]) {
    const uint8_t *p = static_cast<const uint8_t *>(base) + i;
    if (left >= kUnit) {
        const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2_at1 *>(p));
#pragma unroll
        for (int k = 0; k < kUnit; k++) q[k] = (w[k / 4] >> (8 * (k % 4))) & 255u;
    } else {
#pragma unroll
        for (int k = 0; k < kUnit; k++) q[k] = k < left ? p[k] : 0u;
    }
}

__device__ __forceinline__ void store_codes(void *base, int64_t i, int left, const uint32_t (&q)[kUnit]) {
    uint8_t *p = static_cast<uint8_t *>(base) + i;
    if (left >= kUnit) {
        u32x2 w;
        w[0] = q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
        w[1] = q[4] | (q[5] << 8) | (q[6] << 16) | (q[7] << 24);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2_at1 *>(p));
    } else {
#pragma unroll
        for (int k = 0; k < kUnit; k++)
            if (k < left) p[k] = (uint8_t)q[k];
    }
}

template <bool kEight, bool kGradBf16>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Args A, const Hyper H) {
#pragma clang fp contract(off)
    const int ti = find_tensor(A, blockIdx.x);
    const ep_adamw_tensor_t &t = A.t[ti];
    const int64_t i = (int64_t)(blockIdx.x - A.first[ti]) * kChunk + (int64_t)threadIdx.x * kUnit;
    const int left = (int)min((int64_t)kUnit, t.numel - i);  // may be negative: the lane stores nothing
    float p[kUnit], g[kUnit], m[kUnit], v[kUnit];
    load8<float, false>(t.param, i, left, p);
    if constexpr (kGradBf16)
        load8<uint16_t, true>(t.grad, i, left, g);
    else
        load8<float, false>(t.grad, i, left, g);
    const int64_t block = i / kScaleBlock;
    if constexpr (kEight) {
        uint32_t qm[kUnit], qv[kUnit];
        load_codes(t.exp_avg, i, left, qm);
        load_codes(t.exp_avg_sq, i, left, qv);
        const float sm = pow2_of(left > 0 ? t.exp_avg_scale[block] : 1);
        const float sv = pow2_of(left > 0 ? t.exp_avg_sq_scale[block] : 1);
#pragma unroll
        for (int k = 0; k < kUnit; k++) {
            m[k] = decode_m(qm[k], sm);
            v[k] = decode_v(qv[k], sv);
        }
    } else {
        load8<float, false>(t.exp_avg, i, left, m);
        load8<float, false>(t.exp_avg_sq, i, left, v);
    }
#pragma unroll
    for (int k = 0; k < kUnit; k++) {
        const float x = g[k] * H.gscale;
        m[k] = m[k] * H.beta1 + x * H.rest1;
        v[k] = v[k] * H.beta2 + (x * x) * H.rest2;
        p[k] = p[k] * H.decay - H.rate * (m[k] / (sqrtf(v[k]) * H.root + H.eps));
    }
    store8(t.param, i, left, p);
    if (t.copy) {
        uint16_t *c = static_cast<uint16_t *>(t.copy) + i;
        if (left >= kUnit) {
            u32x4 w;
#pragma unroll
            for (int k = 0; k < 4; k++) w[k] = pack_bf16(p[2 * k], p[2 * k + 1]);
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4_at2 *>(c));
        } else {
#pragma unroll
            for (int k = 0; k < kUnit; k++)
                if (k < left) c[k] = to_bf16(p[k]);
        }
    }
    if constexpr (kEight) {
        float am = 0.0f, av = 0.0f;
#pragma unroll
        for (int k = 0; k < kUnit; k++) {
            // an infinite or NaN gradient: the parameter is lost, and its moments must
            // not set the scale of the block's others
            if (!(fabsf(m[k]) < INFINITY)) m[k] = v[k] = 0.0f;
            am = fmaxf(am, fabsf(m[k]));
            av = fmaxf(av, v[k]);
        }
        const int cm = scale_code(row_max_f32(am)), cv = scale_code(row_max_f32(av));
        const float im = pow2_of(254 - cm), iv = pow2_of(254 - cv);
        const uint32_t word = H.word + (H.tensor0 + (uint32_t)ti) * 0x6A09E667u + (uint32_t)i;
        uint32_t qm[kUnit], qv[kUnit];
#pragma unroll
        for (int k = 0; k < kUnit; k++) {
            const uint32_t h = mix(word + k);
            qv[k] = encode_v(v[k], iv, h & 0xfffffu);
            qm[k] = encode_m(m[k], im, (h * 0x9E3779B9u) >> 12);
        }
        store_codes(t.exp_avg, i, left, qm);
        store_codes(t.exp_avg_sq, i, left, qv);
        if (threadIdx.x % (kScaleBlock / kUnit) == 0 && left > 0) {
            t.exp_avg_scale[block] = (uint8_t)cm;
            t.exp_avg_sq_scale[block] = (uint8_t)cv;
        }
    } else {
        store8(static_cast<float *>(t.exp_avg), i, left, m);
        store8(static_cast<float *>(t.exp_avg_sq), i, left, v);
    }
}

// The fp32 values of 8-bit moments; the descriptor's param and copy hold the
// two outputs here.
__global__ __launch_bounds__(kThreads) void adamw_values_kernel(const Args A) {
    const int ti = find_tensor(A, blockIdx.x);
    const ep_adamw_tensor_t &t = A.t[ti];
    const int64_t i = (int64_t)(blockIdx.x - A.first[ti]) * kChunk + (int64_t)threadIdx.x * kUnit;
    const int left = (int)min((int64_t)kUnit, t.numel - i);
    if (left <= 0) return;
    uint32_t qm[kUnit], qv[kUnit];
    load_codes(t.exp_avg, i, left, qm);
    load_codes(t.exp_avg_sq, i, left, qv);
    const float sm = pow2_of(t.exp_avg_scale[i / kScaleBlock]), sv = pow2_of(t.exp_avg_sq_scale[i / kScaleBlock]);
    float m[kUnit], v[kUnit];
#pragma unroll
    for (int k = 0; k < kUnit; k++) {
        m[k] = decode_m(qm[k], sm);
        v[k] = decode_v(qv[k], sv);
    }
    store8(t.param, i, left, m);
    store8(static_cast<float *>(t.copy), i, left, v);
}

// Calls launch(args, workgroups, index of the first tensor) for as many
// descriptors at a time as one launch's arguments hold.
template <typename F>
int for_batches(const ep_adamw_tensor_t *tensors, int32_t n, F launch) {
    for (int32_t i = 0; i < n;) {
        Args A;
        A.n = 0;
        uint64_t blocks = 0;
        const int32_t first = i;
        for (; i < n && A.n < kMaxTensors; i++) {
            const uint64_t b = (uint64_t)ceil_div(tensors[i].numel, kChunk);
            if (blocks + b > (uint64_t)kMaxBlocks) break;
            const ep_adamw_tensor_t &t = tensors[i];
            A.t[A.n] = t;
            A.first[A.n] = (uint32_t)blocks;
            A.n++;
            blocks += b;
        }
        A.first[A.n] = (uint32_t)blocks;
        if (blocks == 0) continue;
        const hipError_t e = launch(A, (uint32_t)blocks, first);
        if (e != hipSuccess) return EP_ERR_HIP;
    }
    return EP_OK;
}

bool tensors_ok(const ep_adamw_tensor_t *tensors, int32_t n, bool eight, bool grads, size_t grad_align) {
    if (n < 0 || (n > 0 && !tensors)) return false;
    for (int32_t i = 0; i < n; i++) {
        const ep_adamw_tensor_t &t = tensors[i];
        // one tensor's workgroups have to fit one launch
        if (t.numel < 0 || ceil_div(t.numel, kChunk) > kMaxBlocks) return false;
        if (t.numel == 0) continue;
        if (!t.param || !t.exp_avg || !t.exp_avg_sq || !is_aligned(t.param, 4)) return false;
        if (grads && (!t.grad || !is_aligned(t.grad, grad_align) || !is_aligned(t.copy, 2))) return false;
        if (eight && (!t.exp_avg_scale || !t.exp_avg_sq_scale)) return false;
        if (!eight && !(is_aligned(t.exp_avg, 4) && is_aligned(t.exp_avg_sq, 4))) return false;
    }
    return true;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_adamw_step(const ep_adamw_tensor_t *tensors, int32_t num_tensors, const ep_adamw_t *hp,
                             ep_stream_t stream) {
    if (!hp || hp->step < 1 || (hp->state_bits != 32 && hp->state_bits != 8) || !float_dtype(hp->grad_dtype))
        return EP_ERR_INVALID_ARG;
    // written so that NaN fails too
    if (!(hp->beta1 >= 0 && hp->beta1 < 1 && hp->beta2 >= 0 && hp->beta2 < 1 && hp->eps >= 0)) return EP_ERR_INVALID_ARG;
    if (!(fabs(hp->lr) <= 1e30 && fabs(hp->weight_decay) <= 1e30 && fabs(hp->grad_scale) <= 1e30))
        return EP_ERR_INVALID_ARG;
    const bool eight = hp->state_bits == 8, gbf16 = hp->grad_dtype == EP_DTYPE_BF16;
    if (!tensors_ok(tensors, num_tensors, eight, true, gbf16 ? 2 : 4)) return EP_ERR_INVALID_ARG;
    Hyper H;
    H.beta1 = (float)hp->beta1;
    H.rest1 = (float)(1 - hp->beta1);
    H.beta2 = (float)hp->beta2;
    H.rest2 = (float)(1 - hp->beta2);
    H.rate = (float)(hp->lr / (1 - pow(hp->beta1, (double)hp->step)));
    H.root = (float)(1 / sqrt(1 - pow(hp->beta2, (double)hp->step)));
    H.eps = (float)hp->eps;
    H.decay = (float)(1 - hp->lr * hp->weight_decay);
    H.gscale = (float)hp->grad_scale;
    H.word = hp->seed + (uint32_t)hp->step * 0x9E3779B9u;
    const hipStream_t s = to_stream(stream);
    return for_batches(tensors, num_tensors, [&](const Args &A, uint32_t blocks, int32_t first) {
        H.tensor0 = (uint32_t)first;
        if (eight)
            gbf16 ? adamw_kernel<true, true><<<blocks, kThreads, 0, s>>>(A, H)
                  : adamw_kernel<true, false><<<blocks, kThreads, 0, s>>>(A, H);
        else
            gbf16 ? adamw_kernel<false, true><<<blocks, kThreads, 0, s>>>(A, H)
                  : adamw_kernel<false, false><<<blocks, kThreads, 0, s>>>(A, H);
        return hipGetLastError();
    });
}

extern "C" int ep_adamw_values(const ep_adamw_tensor_t *tensors, int32_t num_tensors, float *const *exp_avg,
                               float *const *exp_avg_sq, ep_stream_t stream) {
    if (num_tensors < 0 || (num_tensors > 0 && (!tensors || !exp_avg || !exp_avg_sq))) return EP_ERR_INVALID_ARG;
    for (int32_t i = 0; i < num_tensors; i++)
        if (tensors[i].numel != 0 && (!exp_avg[i] || !exp_avg_sq[i] || !is_aligned(exp_avg[i], 4) ||
                                      !is_aligned(exp_avg_sq[i], 4)))
            return EP_ERR_INVALID_ARG;
    if (!tensors_ok(tensors, num_tensors, true, false, 1)) return EP_ERR_INVALID_ARG;
    const hipStream_t s = to_stream(stream);
    // the two outputs take the place of param and copy in a copy of each descriptor
    for (int32_t i = 0; i < num_tensors; i += kMaxTensors) {
        ep_adamw_tensor_t t[kMaxTensors];
        const int32_t n = num_tensors - i < kMaxTensors ? num_tensors - i : kMaxTensors;
        for (int32_t j = 0; j < n; j++) {
            t[j] = tensors[i + j];
            t[j].param = exp_avg[i + j];
            t[j].copy = exp_avg_sq[i + j];
            t[j].grad = nullptr;
        }
        const int rc = for_batches(t, n, [&](const Args &A, uint32_t blocks, int32_t) {
            adamw_values_kernel<<<blocks, kThreads, 0, s>>>(A);
            return hipGetLastError();
        });
        if (rc != EP_OK) return rc;
    }
    return EP_OK;
}
