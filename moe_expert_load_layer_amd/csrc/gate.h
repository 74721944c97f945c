// Top-k selection and weights of one token by the 16 lanes of a DPP row, used
// by the gate's own kernel and by the layer for a few tokens.
//
//   score  s_e = l_e + b_e in fp32 (NaN counts as -inf; -inf is never chosen)
//   groups a group's score is its best s; the topk_groups best groups stay
//   chosen the k largest s, equal ones by lowest expert
//   weight w_j = scale * exp(l_j - max l) / sum_i exp(l_i - max l) over the chosen
//
// Lane i holds the V consecutive experts from i * V on, so that among equal
// scores the lowest lane, and in it the lowest register, is the lowest expert.
// k rounds: the lanes' maxima meet in 4 DPP steps, a ballot names the lowest
// lane that has it, and that lane drops the value.
#pragma once

#include "layer.h"

namespace ep {

constexpr int kGateLanes = 16;      // lanes of one token
constexpr int kGateMaxK = 16;       // one lane of the row per chosen expert
constexpr int kGateMaxGroups = 16;  // one lane of the row per group
constexpr int kGateMaxExperts = 1024;

struct GateArgs {
    const void *logits;
    int64_t stride;  // elements between two tokens
    const float *bias;
    int32_t E, k, G, TG;
    float scale;
    int32_t bf16;  // the logits' type
    int32_t vec;   // rows start on 16 bytes
};

// LDS of one token
struct GateSlot {
    int32_t chosen[kGateMaxK];
    uint32_t group[kGateMaxGroups];
};

// unsigned order of floats
__device__ __forceinline__ uint32_t float_order(float f) {
    const uint32_t u = __builtin_bit_cast(uint32_t, f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float gate_logit(const GateArgs &A, int64_t t, int e) {
    if (A.bf16)
        return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t *>(A.logits)[t * A.stride + e] << 16);
    return static_cast<const float *>(A.logits)[t * A.stride + e];
}

template <int V>
__device__ __forceinline__ void gate_scores(const GateArgs &A, int64_t t, int lane, float (&v)[V]) {
    const int e0 = lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 8) {
        const int e = e0 + i;
        if (A.vec && e + 8 <= A.E) {
            if (A.bf16) {
                const u32x4 w = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(A.logits) +
                                                                 t * A.stride + e);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    v[i + 2 * j] = bf16_lo(w[j]);
                    v[i + 2 * j + 1] = bf16_hi(w[j]);
                }
            } else {
                const f32x4 *p = reinterpret_cast<const f32x4 *>(static_cast<const float *>(A.logits) + t * A.stride + e);
                const f32x4 a = p[0], b = p[1];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    v[i + j] = a[j];
                    v[i + 4 + j] = b[j];
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[i + j] = e + j < A.E ? gate_logit(A, t, e + j) : -INFINITY;
        }
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
        float s = v[i];
        if (A.bias && e0 + i < A.E) s += A.bias[e0 + i];
        s += 0.0f;  // -0 and 0 are equal scores
        v[i] = s == s ? s : -INFINITY;
    }
}

// Drops the scores outside the best groups.
template <int V>
__device__ __forceinline__ void gate_groups(const GateArgs &A, int lane, GateSlot *slot, float (&v)[V]) {
    const int gs = A.E / A.G, e0 = lane * V;
    slot->group[lane] = 0;
    wave_lds_fence();
    {
        int g = e0 / gs, next = (g + 1) * gs;
        float best = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; i++) {
            if (e0 + i == next) {
                if (g < A.G) atomicMax(&slot->group[g], float_order(best));
                best = -INFINITY;
                g++;
                next += gs;
            }
            best = fmaxf(best, v[i]);
        }
        if (g < A.G) atomicMax(&slot->group[g], float_order(best));
    }
    wave_lds_fence();
    const uint32_t mine = slot->group[lane];
    int rank = 0;
    for (int g = 0; g < A.G; g++) {
        const uint32_t o = slot->group[g];
        rank += o > mine || (o == mine && g < lane);
    }
    const uint64_t all = __ballot(lane < A.G && rank < A.TG);
    const uint32_t keep = (uint32_t)(all >> (lane_id() & ~(kGateLanes - 1))) & 0xffffu;
    int g = e0 / gs, next = (g + 1) * gs;
#pragma unroll
    for (int i = 0; i < V; i++) {
        if (e0 + i == next) {
            g++;
            next += gs;
        }
        if (!((keep >> (g & 31)) & 1u)) v[i] = -INFINITY;
    }
}

// Token t: lane j of the row gets the j-th chosen expert (-1: none) and its
// weight.  Every lane of the wave takes part.
template <int V>
__device__ __forceinline__ void gate_token(const GateArgs &A, int64_t t, GateSlot *slot, int &id, float &w) {
    const int lane = lane_id() & (kGateLanes - 1);
    float v[V];
    gate_scores<V>(A, t, lane, v);
    if (A.G > 1) gate_groups<V>(A, lane, slot, v);
    for (int j = 0; j < A.k; j++) {
        float best = v[0];
#pragma unroll
        for (int i = 1; i < V; i++) best = fmaxf(best, v[i]);
        const float top = row_max_f32(best);
        const bool has = best == top && top > -INFINITY;
        const uint64_t all = __ballot(has);
        const uint32_t row = (uint32_t)(all >> (lane_id() & ~(kGateLanes - 1))) & 0xffffu;
        const bool win = has && (row & ((1u << lane) - 1)) == 0;
        int at = -1;
#pragma unroll
        for (int i = V - 1; i >= 0; i--) at = v[i] == top ? i : at;
        if (win) slot->chosen[j] = lane * V + at;
        if (row == 0) slot->chosen[j] = -1;  // every lane of the row writes the same
        at = win ? at : -1;
#pragma unroll
        for (int i = 0; i < V; i++) v[i] = i == at ? -INFINITY : v[i];
    }
    wave_lds_fence();
    id = lane < A.k ? slot->chosen[lane] : -1;
    const float l = id >= 0 ? gate_logit(A, t, id) : -INFINITY;
    const float top = row_max_f32(l);
    // l == top also where both are infinite
    const float e = id < 0 ? 0.0f : (l == top ? 1.0f : expf(l - top));
    const float sum = row_sum_f32(e);
    w = sum > 0.0f ? A.scale * (e / sum) : 0.0f;
    wave_lds_fence();
}

bool gate_ok(const ep_gate_t *g);
GateArgs gate_args(const void *logits, int64_t stride, const ep_gate_t *g);

}  // namespace ep
