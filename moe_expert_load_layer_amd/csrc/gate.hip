// The gate: top-k expert IDs and weights from router logits, and its gradient.
//
// 16 lanes take a token (gate.h), a wave four, a workgroup 16.  Forward reads
// the logits once and is bound by the instructions of the selection; backward
// writes the dense gradient rows, assembled in LDS, and is bound by HBM.
// Measured for 131071 tokens x 384 experts in bf16, k = 8: forward 36 us (3.0
// TB/s; 28 where the logits are in the last-level cache, and k rounds of a maximum
// over the row take 66), backward 18 us (6.3 TB/s); 64 tokens x 256 experts in fp32
// 7 us, most of it a launch and the loads' latency.
#include "gate.h"

namespace ep {

bool gate_ok(const ep_gate_t *g) {
    if (!g || g->num_experts < 1 || g->num_experts > kGateMaxExperts || !float_dtype(g->logits_dtype)) return false;
    if (g->num_groups < 1 || g->num_groups > kGateMaxGroups || g->num_experts % g->num_groups != 0) return false;
    if (g->topk_groups < 1 || g->topk_groups > g->num_groups) return false;
    if (g->top_k < 1 || g->top_k > kGateMaxK || g->top_k > g->num_experts) return false;
    return is_aligned(g->bias, 4) && g->scale - g->scale == 0;  // finite
}

GateArgs gate_args(const void *logits, int64_t stride, const ep_gate_t *g) {
    GateArgs A;
    A.logits = logits;
    A.stride = stride;
    A.bias = g->bias;
    A.E = g->num_experts;
    A.k = g->top_k;
    A.G = g->topk_groups == g->num_groups ? 1 : g->num_groups;  // all groups stay: no limit
    A.TG = g->topk_groups;
    A.scale = g->scale;
    A.bf16 = g->logits_dtype == EP_DTYPE_BF16;
    return A;
}

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / kGateLanes;  // tokens of a workgroup

template <int V>
__global__ __launch_bounds__(kThreads) void gate_kernel(const GateArgs A, int64_t T, int32_t *__restrict__ ids,
                                                        float *__restrict__ weights) {
    __shared__ GateSlot slots[kTokens];
    const int s = threadIdx.x / kGateLanes, lane = threadIdx.x % kGateLanes;
    const int64_t t = (int64_t)blockIdx.x * kTokens + s;
    int id;
    float w;
    gate_token<V>(A, t < T ? t : T - 1, &slots[s], id, w);  // rows past the end repeat the last token
    if (t < T && lane < A.k) {
        ids[t * A.k + lane] = id;
        weights[t * A.k + lane] = w;
    }
}

// dl_j = w_j (g_j - sum_i w_i g_i / scale) at the chosen experts, 0 elsewhere.
// A wave forms its 4 tokens' rows in LDS, in the output's type, and stores them
// as one run of memory.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void gate_backward_kernel(const int32_t *__restrict__ ids,
                                                                 const float *__restrict__ weights,
                                                                 const float *__restrict__ grad, int64_t T, int E,
                                                                 int k, float scale, void *__restrict__ out) {
    constexpr int kTok = kWave / kGateLanes, kWidth = kBf16 ? 2 : 4, kPer = 16 / kWidth;
    extern __shared__ u32x4 lds[];  // [waves][4 rows of E, up to 16 bytes]
    const int l = lane_id(), wave = threadIdx.x / kWave, lane = l % kGateLanes;
    const int words = (kTok * E + kPer - 1) / kPer;  // of 16 bytes, a wave
    u32x4 *mine = lds + wave * words;
    const int64_t t0 = ((int64_t)blockIdx.x * (kThreads / kWave) + wave) * kTok, t = t0 + l / kGateLanes;
    const bool on = t < T && lane < k;
    const int id = on ? ids[t * k + lane] : -1;
    const bool use = id >= 0 && id < E;
    const float w = use ? weights[t * k + lane] : 0.0f;
    const float g = use ? grad[t * k + lane] : 0.0f;
    for (int i = l; i < words; i += kWave) mine[i] = u32x4{0, 0, 0, 0};
    const float sum = row_sum_f32(w * g);
    // divided, since the smallest scales have no finite inverse
    const float mean = scale != 0.0f ? sum / scale : 0.0f;
    wave_lds_fence();
    if (use) {
        const float d = w * (g - mean);
        const int at = l / kGateLanes * E + id;
        if constexpr (kBf16) reinterpret_cast<uint16_t *>(mine)[at] = to_bf16(d);
        else reinterpret_cast<float *>(mine)[at] = d;
    }
    wave_lds_fence();
    if (t0 >= T) return;
    const int64_t n = min((int64_t)kTok, T - t0) * E, o = t0 * E, whole = n / kPer;
    u32x4_at2 *to = reinterpret_cast<u32x4_at2 *>(static_cast<uint8_t *>(out) + o * kWidth);
    for (int64_t i = l; i < whole; i += kWave) to[i] = mine[i];
    for (int64_t i = whole * kPer + l; i < n; i += kWave) {
        if constexpr (kBf16)
            static_cast<uint16_t *>(out)[o + i] = reinterpret_cast<const uint16_t *>(mine)[i];
        else
            static_cast<float *>(out)[o + i] = reinterpret_cast<const float *>(mine)[i];
    }
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_gate_topk(const void *logits, int64_t stride, int64_t num_tokens, const ep_gate_t *gate,
                            int32_t *ids, float *weights, ep_stream_t stream) {
    if (!gate_ok(gate) || num_tokens < 0 || num_tokens > kMaxBlocks * kTokens || stride < gate->num_experts)
        return EP_ERR_INVALID_ARG;
    if (num_tokens == 0) return EP_OK;
    const size_t width = gate->logits_dtype == EP_DTYPE_BF16 ? 2 : 4;
    if (!logits || !ids || !weights || !is_aligned(logits, width) || !is_aligned(ids, 4) || !is_aligned(weights, 4))
        return EP_ERR_INVALID_ARG;
    const GateArgs A = gate_args(logits, stride, gate);
    const dim3 grid((uint32_t)ceil_div(num_tokens, kTokens));
    const hipStream_t s = to_stream(stream);
    const int per = (A.E + kGateLanes - 1) / kGateLanes;
    if (per <= 8) gate_kernel<8><<<grid, kThreads, 0, s>>>(A, num_tokens, ids, weights);
    else if (per <= 16) gate_kernel<16><<<grid, kThreads, 0, s>>>(A, num_tokens, ids, weights);
    else if (per <= 24) gate_kernel<24><<<grid, kThreads, 0, s>>>(A, num_tokens, ids, weights);
    else if (per <= 32) gate_kernel<32><<<grid, kThreads, 0, s>>>(A, num_tokens, ids, weights);
    else gate_kernel<64><<<grid, kThreads, 0, s>>>(A, num_tokens, ids, weights);
    return rc_of(hipGetLastError());
}

extern "C" int ep_gate_topk_backward(const int32_t *ids, const float *weights, const float *grad_weights,
                                     int64_t num_tokens, const ep_gate_t *gate, void *grad_logits,
                                     ep_stream_t stream) {
    if (!gate_ok(gate) || num_tokens < 0 || num_tokens > kMaxBlocks * kTokens) return EP_ERR_INVALID_ARG;
    if (num_tokens == 0) return EP_OK;
    const bool bf16 = gate->logits_dtype == EP_DTYPE_BF16;
    if (!ids || !weights || !grad_weights || !grad_logits || !is_aligned(ids, 4) || !is_aligned(weights, 4) ||
        !is_aligned(grad_weights, 4) || !is_aligned(grad_logits, bf16 ? 2 : 4))
        return EP_ERR_INVALID_ARG;
    const dim3 grid((uint32_t)ceil_div(num_tokens, kTokens));
    const size_t lds = (size_t)(kThreads / kWave) * ceil_div(4 * (int64_t)gate->num_experts * (bf16 ? 2 : 4), 16) * 16;
    const hipStream_t s = to_stream(stream);
    if (bf16)
        gate_backward_kernel<true><<<grid, kThreads, lds, s>>>(ids, weights, grad_weights, num_tokens,
                                                               gate->num_experts, gate->top_k, gate->scale, grad_logits);
    else
        gate_backward_kernel<false><<<grid, kThreads, lds, s>>>(ids, weights, grad_weights, num_tokens,
                                                                gate->num_experts, gate->top_k, gate->scale, grad_logits);
    return rc_of(hipGetLastError());
}
