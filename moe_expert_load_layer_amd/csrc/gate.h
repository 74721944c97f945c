// Top-k selection and weights of one token by the 16 lanes of a DPP row, used
// by the gate's own kernel and by the layer for a few tokens.
//
//   score  s_e = l_e + b_e in fp32 (NaN counts as -inf; -inf is never chosen)
//   groups a group's score is its best s; the topk_groups best groups stay
//   chosen the k largest s, equal ones by lowest expert
//   weight w_j = scale * exp(l_j - max l) / sum_i exp(l_i - max l) over the chosen
//
// Lane i holds the experts of the chunks of 8 with numbers i, i + 16, ...  The
// lanes' maxima are ranked by rotating them round the row; the k-th of them, tau,
// is a lower bound of the k-th largest score, so only scores from tau on (11 or
// so of 384 for k = 8) are candidates.  They go to LDS, and each counts those
// before it.  Where masks or ties leave more than 32 candidates, k rounds of a
// maximum over the row choose instead.  The choice is the same either way.
#pragma once

#include <float.h>

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
};

constexpr int kGateCandidates = 2 * kGateLanes;

// LDS of one token
struct alignas(16) GateSlot {
    uint64_t key[kGateCandidates];  // of a candidate: its score's order, then ~expert; 0: none
    float logit[kGateCandidates];
    int32_t chosen[kGateMaxK];
    float chosen_logit[kGateMaxK];
    uint32_t group[kGateMaxGroups];
};

// expert of register i of a lane
__device__ __forceinline__ int gate_expert(int lane, int i) { return ((i / 8) * kGateLanes + lane) * 8 + i % 8; }

// unsigned order of floats, -0 and 0 alike
__device__ __forceinline__ uint32_t float_order(float f) {
    const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float gate_logit(const GateArgs &A, int64_t t, int e) {
    if (A.bf16)
        return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t *>(A.logits)[t * A.stride + e] << 16);
    return static_cast<const float *>(A.logits)[t * A.stride + e];
}

template <int V>
__device__ __forceinline__ void gate_scores(const GateArgs &A, int64_t t, int lane, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 8) {
        const int e = gate_expert(lane, i);
        if (e + 8 <= A.E) {
            if (A.bf16) {
                const u32x4 w = *reinterpret_cast<const u32x4_at2 *>(static_cast<const uint16_t *>(A.logits) +
                                                                     t * A.stride + e);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    v[i + 2 * j] = bf16_lo(w[j]);
                    v[i + 2 * j + 1] = bf16_hi(w[j]);
                }
            } else {
                const f32x4_at4 *p =
                    reinterpret_cast<const f32x4_at4 *>(static_cast<const float *>(A.logits) + t * A.stride + e);
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
    if (A.bias) {
#pragma unroll
        for (int i = 0; i < V; i += 8) {
            const int e = gate_expert(lane, i);
            if (e + 8 <= A.E) {
                const f32x4_at4 *p = reinterpret_cast<const f32x4_at4 *>(A.bias + e);
                const f32x4 a = p[0], b = p[1];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    v[i + j] += a[j];
                    v[i + 4 + j] += b[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++) v[i + j] += e + j < A.E ? A.bias[e + j] : 0.0f;
            }
        }
    }
}

// Drops the scores outside the best groups.
template <int V>
__device__ __forceinline__ void gate_groups(const GateArgs &A, int lane, GateSlot *slot, float (&v)[V]) {
    const int gs = A.E / A.G;
    slot->group[lane] = 0;
    wave_lds_fence();
    // a chunk's 8 experts are consecutive: their maxima go out group by group
#pragma unroll
    for (int i = 0; i < V; i += 8) {
        const int e0 = gate_expert(lane, i);
        int g = e0 / gs, next = (g + 1) * gs;
        float best = -INFINITY;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (e0 + j == next) {
                if (g < A.G) atomicMax(&slot->group[g], float_order(best));
                best = -INFINITY;
                g++;
                next += gs;
            }
            best = fmaxf(best, v[i + j]);
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
#pragma unroll
    for (int i = 0; i < V; i += 8) {
        const int e0 = gate_expert(lane, i);
        int g = e0 / gs, next = (g + 1) * gs;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (e0 + j == next) {
                g++;
                next += gs;
            }
            if (!((keep >> (g & 31)) & 1u)) v[i + j] = -INFINITY;
        }
    }
}

// lanes of the row whose value is greater, by rotating the row's values
template <int kStep>
__device__ __forceinline__ int row_greater(float v) {
    if constexpr (kStep == kGateLanes) return 0;
    else return (dpp_f32<0x120 + kStep>(v) > v ? 1 : 0) + row_greater<kStep + 1>(v);
}

__device__ __forceinline__ int row_min_i32(int v) {
    v = min(v, __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true));
    v = min(v, __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true));
    v = min(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true));
    return min(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true));
}

// inclusive prefix sum over the row of 16 (row_shr fills zeros from the left)
__device__ __forceinline__ int row_scan_i32(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    return v + __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
}

// k rounds of the row's maximum, the lowest expert among equal ones; v is used up
template <int V>
__device__ __forceinline__ void gate_rounds(const GateArgs &A, int lane, GateSlot *slot, float (&v)[V]) {
    for (int j = 0; j < A.k; j++) {
        float best = v[0];
#pragma unroll
        for (int i = 1; i < V; i++) best = fmaxf(best, v[i]);
        const float top = row_max_f32(best);
        int e = INT32_MAX;
#pragma unroll
        for (int i = V - 1; i >= 0; i--) e = v[i] == top ? gate_expert(lane, i) : e;  // ascending in i
        const int first = row_min_i32(e);
        slot->chosen[j] = top > -INFINITY ? first : -1;  // every lane of the row writes the same
#pragma unroll
        for (int i = 0; i < V; i++) v[i] = gate_expert(lane, i) == first ? -INFINITY : v[i];
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
    float best = -INFINITY;  // fmaxf takes the other operand where one is NaN
#pragma unroll
    for (int i = 0; i < V; i++) best = fmaxf(best, v[i]);
    // at least k lanes have fewer than k greater maxima, so k scores at least
    // are not below the least of those maxima; -inf is no candidate
    const float tau = fmaxf(-row_max_f32(row_greater<1>(best) < A.k ? -best : -INFINITY), -FLT_MAX);
    constexpr int kWords = (V + 31) / 32;
    uint32_t mine[kWords];  // a bit for each candidate register
    int count = 0;
#pragma unroll
    for (int h = 0; h < kWords; h++) {
        mine[h] = 0;
#pragma unroll
        for (int i = min(V, 32 * h + 32) - 1; i >= 32 * h; i--) mine[h] += mine[h] + (v[i] >= tau ? 1u : 0u);
        count += __popc(mine[h]);
    }
    const int upto = row_scan_i32(count);
    const int n = __shfl(upto, lane_id() | (kGateLanes - 1));
    float l;
    if (__any(n > kGateCandidates)) {
        gate_rounds<V>(A, lane, slot, v);
        wave_lds_fence();
        id = lane < A.k ? slot->chosen[lane] : -1;
        l = id >= 0 ? gate_logit(A, t, id) : -INFINITY;
    } else {
        slot->chosen[lane] = -1;
        slot->key[lane] = slot->key[lane + kGateLanes] = 0;
        wave_lds_fence();
        // a lane has few: the scores are formed again rather than picked out of
        // the registers one by one
        int at = upto - count;
#pragma unroll
        for (int h = 0; h < kWords; h++)
            for (; __any(mine[h] != 0); at++) {
                if (mine[h] == 0) {
                    at--;
                } else {
                    const int e = gate_expert(lane, 32 * h + __builtin_ctz(mine[h]));
                    const float raw = gate_logit(A, t, e);
                    slot->key[at] = (uint64_t)float_order(raw + (A.bias ? A.bias[e] : 0.0f)) << 32 | (uint32_t)~e;
                    slot->logit[at] = raw;
                    mine[h] &= mine[h] - 1;
                }
            }
        wave_lds_fence();
        const bool two = __any(n > kGateLanes);
        const uint64_t k0 = slot->key[lane], k1 = slot->key[lane + kGateLanes];
        const float l0 = slot->logit[lane], l1 = slot->logit[lane + kGateLanes];  // past the n-th: not used
        int before0 = 0, before1 = 0;
        for (int o = 0; o < n; o += 4) {
            uint64_t key[4];
#pragma unroll
            for (int i = 0; i < 4; i++) key[i] = slot->key[o + i];
#pragma unroll
            for (int i = 0; i < 4; i++) before0 += key[i] > k0;
            if (two) {
#pragma unroll
                for (int i = 0; i < 4; i++) before1 += key[i] > k1;
            }
        }
        if (lane < n && before0 < A.k) {
            slot->chosen[before0] = (int32_t)~(uint32_t)k0;
            slot->chosen_logit[before0] = l0;
        }
        if (lane + kGateLanes < n && before1 < A.k) {
            slot->chosen[before1] = (int32_t)~(uint32_t)k1;
            slot->chosen_logit[before1] = l1;
        }
        wave_lds_fence();
        id = lane < A.k ? slot->chosen[lane] : -1;
        l = id >= 0 ? slot->chosen_logit[lane] : -INFINITY;
    }
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
