// A whole mixture-of-experts layer for a few tokens (at most 64), in two kernels:
//   up    gate (gate.h), then h_p = silu(Wg_e x_t) * (Wu_e x_t) for every pair p = (t, j), e = id_tj
//   down  out_t = sum_j w_tj Wd_e h_p
//
// With more than 32 tokens the gate is a launch of its own before them.
//
// Bound: HBM.  With up to 8 tokens every distinct expert's three matrices are read
// once, which is all but a fraction of a percent of the bytes.  With more, gate
// and up are read once for every 32 tokens of an expert and down once for every
// 16 (more columns would leave LDS for fewer workgroups): 10 % more bytes of down
// at 61 tokens on 160 experts, four times its bytes where all 64 tokens agree.
// Measured, up and down: 1 token, 8 of 128 experts, 4096 x 1536 in bf16 43 + 22 us
// (302 MB, 4.6 TB/s); 7 tokens, 7168 x 2048 in 8 bits 175 + 91 us (1.40 GB, 5.3);
// 61 tokens, 160 experts, 5120 x 1536 in bf16 5 + 508 + 282 us (4.34 GB, 5.5).
//
// Both kernels stream: a workgroup takes 64 weight rows of an expert and walks
// them in windows of 128 bytes a row, together with the same window of the
// expert's columns (tokens, or pairs' h).  Windows go from memory into a ring of
// LDS stages without passing registers; all but one stage of the ring are in
// flight, across the borders between experts too, and one barrier a window
// hands a stage over.  Each of the 4 waves multiplies its own 16 rows, so no
// sum crosses waves, and a column is fetched once for 64 rows.
//
// up: 64 rows are 32 of gate and the same 32 of up, 8 and 8 in each wave, whose
// halves exchange them for silu.  h is kept as the sum of two bf16 (16 bits of
// mantissa): one bf16 would add as much error as the output's own rounding.
// down: the high and low parts of 8 pairs' h are the 16 columns of one matrix
// instruction.  The (expert, window) sequence of 64 output rows is cut into
// shares so that about 512 workgroups run; the last share to arrive adds all of
// them in order.  No atomics on sums: results do not depend on scheduling.
//
// 8-bit weights: a window is 128 values with one scale byte; v_cvt_scalef32
// gives bf16 exactly (3 bits of mantissa, power-of-two scale), so products and
// sums are those of the bf16 path.
#include <math.h>

#include "gate.h"
#include "groups.h"

namespace ep {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kMaxTokens = EP_MAX_FEW_TOKENS;
constexpr int kMaxPairs = kMaxTokens * kGateMaxK;
constexpr int kMaxWidth = 65536;  // hidden and inter
constexpr int kRows = kWaves * 16;     // weight rows of a workgroup
constexpr int kUpRows = kRows / 2;     // of gate and of up
constexpr int kWindowBytes = 128;      // of one row
constexpr int kScaleUnits = 512;       // windows whose scale bytes are in LDS at a time
// pairs of one expert that are multiplied together: 8 where no expert can have more
constexpr int kFew = 8, kUpMany = 32, kDownMany = 16;
constexpr int kGateAlone = 32;  // tokens up to which the first kernel chooses for itself
constexpr int kMaxEntries = kGateMaxExperts + kMaxPairs / kDownMany;

__device__ __align__(16) const uint32_t kNothing[4] = {0, 0, 0, 0};

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
    bool chosen;  // ids and weights are there already
    int32_t *ids;
    float *weights;
    uint16_t *out;
    uint16_t *hhi, *hlo;  // [T * k][I]
    int32_t *arrivals;    // of each block of output rows, zeroed by the first kernel
    float *sums;          // [shares][T][H]
};

// The pairs of each chosen expert, in LDS.  An entry is an expert with up to
// kCols of its pairs.
struct Lists {
    uint16_t pair[kMaxPairs];     // pairs ordered by expert
    uint16_t expert[kMaxEntries];
    uint16_t start[kMaxEntries];  // the entry's first place in `pair`
    uint8_t count[kMaxEntries];
    int32_t entries;
};

// What the lists are made from; it lies where the ring's stages come later.
struct Scratch {
    int32_t ids[kMaxPairs];
    uint32_t tokens[2][kGateMaxExperts];  // of each expert, a bit each
    uint16_t first[kGateMaxExperts];      // of each expert in `pair`
    GateSlot slot[kThreads / kGateLanes];
};

// W->ids holds T * k IDs, every expert at most once for a token.  The pairs of
// an expert are ordered by token, in every workgroup alike: its entries are
// worked on by different ones.
template <int kCols>
__device__ void build_lists(Lists *L, Scratch *W, int T, int k, int E) {
    static_assert(kMaxTokens == 64, "a bit for each token");
    for (int e = threadIdx.x; e < E; e += kThreads) W->tokens[0][e] = W->tokens[1][e] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < T * k; p += kThreads) {
        const int t = p / k;
        if (W->ids[p] >= 0) atomicOr(&W->tokens[t / 32][W->ids[p]], 1u << (t % 32));
    }
    __syncthreads();
    if (threadIdx.x < kWave) {
        int entries = 0, first = 0;
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int e = e0 + (int)threadIdx.x;
            const int c = e < E ? __popc(W->tokens[0][e]) + __popc(W->tokens[1][e]) : 0;
            const int n = (c + kCols - 1) / kCols;
            const int places = wave_incl_scan_i32(c), slots = wave_incl_scan_i32(n);
            for (int i = 0; i < n; i++) {
                const int a = entries + slots - n + i;
                L->expert[a] = (uint16_t)e;
                L->start[a] = (uint16_t)(first + places - c + i * kCols);
                L->count[a] = (uint8_t)min(kCols, c - i * kCols);
            }
            if (e < E) W->first[e] = (uint16_t)(first + places - c);
            entries += __builtin_amdgcn_readlane(slots, kWave - 1);
            first += __builtin_amdgcn_readlane(places, kWave - 1);
        }
        if (threadIdx.x == 0) L->entries = entries;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < T * k; p += kThreads) {
        const int e = W->ids[p], t = p / k;
        if (e < 0) continue;
        const uint64_t all = ((uint64_t)W->tokens[1][e] << 32) | W->tokens[0][e];
        L->pair[W->first[e] + __popcll(all & ((1ull << t) - 1))] = (uint16_t)p;
    }
    __syncthreads();
}

template <bool kFp8>
__host__ __device__ __forceinline__ int windows_of(int K) {
    return kFp8 ? (K + 127) / 128 : (K + 63) / 64;
}

template <bool kFp8>
__device__ __forceinline__ int64_t row_bytes(int K) {
    return kFp8 ? (int64_t)((K + 127) / 128) * 128 : (int64_t)K * 2;
}

// Waits until at most n of this wave's loads are in flight; n is the same in
// every lane.  The instruction's count is a constant, hence the cases.
__device__ __forceinline__ void wait_loads_but_n(int n) {
    switch (n) {
#define EP_WAIT(N) \
    case N: asm volatile("s_waitcnt vmcnt(" #N ")" ::: "memory"); break;
        EP_WAIT(2) EP_WAIT(3) EP_WAIT(4) EP_WAIT(5) EP_WAIT(6)
#undef EP_WAIT
        default: wait_loads();
    }
}

// The ring of one workgroup.  kParts: arrays of column values (x, or h's high
// and low parts).  A column's window is kHalves rows of 128 bytes.  LDS rows are
// 128 bytes, their 16-byte chunks exchanged by the row's low 3 bits.
template <bool kFp8, int kCols, int kParts>
struct Ring {
    static constexpr int kHalves = kFp8 ? 2 : 1;
    static constexpr int kColRows = kCols * kParts * kHalves;  // row of column c, part p, half h: (p * kHalves + h) * kCols + c
    static constexpr int kColLoads = kColRows / 8;             // loads of 1 KiB
    static constexpr int kMine = (kColLoads + kWaves - 1) / kWaves;
    static constexpr int kStage = (kRows + kColRows) * 128;
    static constexpr int kStages = 3;  // more would leave room for fewer workgroups: slower in every case measured
    static constexpr int kTiles = kParts == 2 ? kCols / 8 : (kCols + 15) / 16;

    uint8_t *lds;
    int wave, K;
    const uint8_t *w[2];  // this lane's source of the wave's loads, at window 0
    const uint8_t *col[kMine];
    int n;                     // columns of the windows being fetched
    int flying;  // loads of the newest window

    __device__ __forceinline__ static int chunk() { return (lane_id() & 7) ^ (lane_id() >> 3); }
    // row of the weights that load i fetches for this lane, and its row of columns
    __device__ __forceinline__ int weight_row(int i) const { return (wave + i * kWaves) * 8 + lane_id() / 8; }
    __device__ __forceinline__ int column_row(int i) const { return (wave + i * kWaves) * 8 + lane_id() / 8; }

    // Only the groups of 8 columns that the entry has are fetched.
    __device__ __forceinline__ void issue(int slot, int win, bool partial) {
        uint8_t *s = lds + slot * kStage;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint8_t *p = w[i] + win * kWindowBytes;
            if (!kFp8 && partial && win * 64 + chunk() * 8 >= K) p = reinterpret_cast<const uint8_t *>(kNothing);
            load_lds_1k(p, s + (wave + i * kWaves) * 1024);
        }
        int count = 2;
#pragma unroll
        for (int i = 0; i < kMine; i++) {
            const int load = wave + i * kWaves;
            if (load >= kColLoads || load % (kCols / 8) * 8 >= n) continue;
            const uint8_t *p = col[i] + win * kWindowBytes * kHalves;
            const int h = load / (kCols / 8) % kHalves;
            if (partial && (win * kHalves + h) * 64 + chunk() * 8 >= K) p = reinterpret_cast<const uint8_t *>(kNothing);
            load_lds_1k(p, s + kRows * 128 + load * 1024);
            count++;
        }
        flying = count;
    }

    // waits until all but the newest window's loads are there
    __device__ __forceinline__ void arrive() const {
        static_assert(kStages == 3 && 2 + kMine <= 6, "one window stays in flight, its loads have a case");
        wait_loads_but_n(flying);
        __syncthreads();
    }

    // acc[t] += this wave's 16 rows x the columns of tile t, for n columns
    __device__ __forceinline__ void multiply(int slot, int n, float scale, f32x4 (&acc)[kTiles]) const {
        const uint8_t *tw = lds + slot * kStage + wave * 16 * 128, *tc = lds + slot * kStage + kRows * 128;
        const int l = lane_id(), r = l & 15, q = l >> 4;
        auto at = [](const uint8_t *t, int row, int c) {
            return *reinterpret_cast<const u32x4 *>(t + row * 128 + ((c ^ (row & 7)) << 4));
        };
        constexpr int kPer = kParts == 2 ? 8 : 16;  // pairs of a tile
        auto column = [&](int t, int h, int c) {
            const int pair = kParts == 2 ? t * 8 + (r & 7) : (t * 16 + r) % kCols;
            const int part = kParts == 2 ? r >> 3 : 0;
            return __builtin_bit_cast(bf16x8, at(tc, (part * kHalves + h) * kCols + pair, c));
        };
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const u32x4 raw = at(tw, r, q + 4 * h);
            if constexpr (kFp8) {
                // 16 values at k = 16 (q + 4 h), as two steps of 8
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    union {
                        bf16x2 h2[4];
                        bf16x8 v;
                    } a;
                    a.h2[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * j], scale, false);
                    a.h2[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * j], scale, true);
                    a.h2[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * j + 1], scale, false);
                    a.h2[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * j + 1], scale, true);
#pragma unroll
                    for (int t = 0; t < kTiles; t++)
                        if (t * kPer < n)
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, column(t, h, 2 * q + j), acc[t], 0, 0, 0);
                }
            } else {
                // 8 values at k = 8 (q + 4 h)
                const bf16x8 a = __builtin_bit_cast(bf16x8, raw);
#pragma unroll
                for (int t = 0; t < kTiles; t++)
                    if (t * kPer < n)
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, column(t, 0, q + 4 * h), acc[t], 0, 0, 0);
            }
        }
    }
};

template <bool kFp8, int kCols, int V>
__global__ __launch_bounds__(kThreads) void up_kernel(const FewArgs A) {
    typedef Ring<kFp8, kCols, 1> R;
    __shared__ __align__(16) uint8_t stages[R::kStages * R::kStage];
    __shared__ Lists L;
    __shared__ uint8_t scales[kFp8 ? 2 * kScaleUnits : 2];
    static_assert(sizeof(Scratch) <= sizeof(stages), "the scratch fits the stages");
    Scratch *W = reinterpret_cast<Scratch *>(stages);
    // every workgroup chooses for itself, and the first one writes the choice
    constexpr int kPass = kThreads / kGateLanes;
    if (A.chosen)
        for (int p = threadIdx.x; p < A.T * A.k; p += kThreads) W->ids[p] = A.ids[p];
    for (int t0 = 0; t0 < A.T && !A.chosen; t0 += kPass) {
        const int s = threadIdx.x / kGateLanes, j = threadIdx.x % kGateLanes, t = t0 + s;
        int id;
        float w;
        gate_token<V>(A.gate, min(t, A.T - 1), &W->slot[s], id, w);
        if (t < A.T && j < A.k) {
            W->ids[t * A.k + j] = id;
            if (blockIdx.x == 0) {
                A.ids[t * A.k + j] = id;
                A.weights[t * A.k + j] = w;
            }
        }
    }
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < (A.H + kRows - 1) / kRows; i += kThreads) A.arrivals[i] = 0;
    __syncthreads();
    build_lists<kCols>(&L, W, A.T, A.k, A.gate.E);

    // this workgroup's items (an entry's 32 rows of gate and of up), each nw windows
    const int tiles = (A.I + kUpRows - 1) / kUpRows, items = L.entries * tiles, nw = windows_of<kFp8>(A.H);
    if ((int)blockIdx.x >= items) return;
    const int units = ((items - 1 - (int)blockIdx.x) / (int)gridDim.x + 1) * nw;
    const bool partial = A.H % (64 * R::kHalves) != 0;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), l = lane_id(), r = l & 15, q = l >> 4;
    R ring;
    ring.lds = stages;
    ring.wave = wave;
    ring.K = A.H;

    int pu = 0, pit = blockIdx.x, pwin = 0;  // the next window to fetch
    auto sources = [&] {
        const int a = pit / tiles, i0 = (pit - a * tiles) * kUpRows, e = L.expert[a], first = L.start[a];
        const int n = ring.n = __builtin_amdgcn_readfirstlane(L.count[a]);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            // rows 16 w .. + 7 are gate's 8 w .. + 7, the next 8 up's
            const int row = ring.weight_row(i), o = min(i0 + row / 16 * 8 + row % 8, A.I - 1);
            const uint8_t *m = row % 16 < 8 ? A.wg.data + e * A.wg.stride : A.wu.data + e * A.wu.stride;
            ring.w[i] = m + o * row_bytes<kFp8>(A.H) + R::chunk() * 16;
        }
#pragma unroll
        for (int i = 0; i < R::kMine; i++) {
            const int c = ring.column_row(i) % kCols, h = ring.column_row(i) / kCols;
            const int t = L.pair[first + min(c, n - 1)] / A.k;  // columns past the end repeat the last
            ring.col[i] = reinterpret_cast<const uint8_t *>(A.x + t * A.x_stride) + (h % R::kHalves) * 128 + R::chunk() * 16;
        }
    };
    // past the last window that one is fetched again: the count of loads stays
    auto produce = [&](int slot) {
        ring.issue(slot, pwin, partial);
        pu++;
        if (pu < units && ++pwin == nw) {
            pwin = 0;
            pit += gridDim.x;
            sources();
        }
    };
    sources();
#pragma unroll
    for (int s = 0; s < R::kStages - 1; s++) produce(s);

    f32x4 acc[R::kTiles];
#pragma unroll
    for (int t = 0; t < R::kTiles; t++) acc[t] = f32x4{0, 0, 0, 0};
    int slot = 0, it = blockIdx.x, win = 0;
    for (int u = 0; u < units; u++) {
        if (kFp8 && u % kScaleUnits == 0) {
            if (u > 0) __syncthreads();  // those before have been read
            for (int i = threadIdx.x; i < 2 * min(kScaleUnits, units - u); i += kThreads) {
                const int un = u + i / 2, b = blockIdx.x + un / nw * gridDim.x, a = b / tiles, e = L.expert[a];
                const int block = (b - a * tiles) * kUpRows / kScaleBlock;
                const uint8_t *m = i % 2 ? A.wu.scale + e * A.wu.scale_stride : A.wg.scale + e * A.wg.scale_stride;
                scales[i] = m[(int64_t)block * nw + un % nw];
            }
        }
        ring.arrive();
        produce(slot == 0 ? R::kStages - 1 : slot - 1);
        const int a = it / tiles, n = __builtin_amdgcn_readfirstlane(L.count[a]);
        float scale = 1.0f;
        if constexpr (kFp8) scale = pow2_of(scales[u % kScaleUnits * 2 + (r >> 3)]);
        ring.multiply(slot, n, scale, acc);
        slot = slot == R::kStages - 1 ? 0 : slot + 1;
        if (++win < nw) continue;
        // lanes 0 .. 31 have gate's 4 rows of a column, lanes 32 .. 63 up's
        const int i0 = (it - a * tiles) * kUpRows + wave * 8 + (q & 1) * 4;
#pragma unroll
        for (int t = 0; t < R::kTiles; t++) {
            if (t * 16 >= n) break;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float g = acc[t][i], up = __shfl_xor(acc[t][i], 32);
                const float h = g / (1.0f + expf(-g)) * up;
                hi[i] = to_bf16(h);
                const float rest = h - __builtin_bit_cast(float, hi[i] << 16);
                // an h that is infinite as bf16, or NaN, has no rest
                lo[i] = to_bf16(fabsf(rest) < INFINITY ? rest : 0.0f);
            }
            const int c = t * 16 + r;
            if (q < 2 && c < n && i0 < A.I) {  // I is a multiple of 8
                const int64_t at = (int64_t)L.pair[L.start[a] + c] * A.I + i0;
                *reinterpret_cast<u32x2 *>(A.hhi + at) = u32x2{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16};
                *reinterpret_cast<u32x2 *>(A.hlo + at) = u32x2{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16};
            }
            acc[t] = f32x4{0, 0, 0, 0};
        }
        win = 0;
        it += gridDim.x;
    }
    wait_loads();  // those that nobody reads
}

// Shares of the weights that the workgroups of one block of output rows take, at
// most: about 512 workgroups in all, shares of 4 windows at least.
int most_shares(int T, int k, int H, int I) {
    const int64_t blocks = ceil_div(H, kRows), windows = (int64_t)T * k * ceil_div(I, 64);
    const int64_t want = 512 / blocks < windows / 4 ? 512 / blocks : windows / 4;
    return want < 1 ? 1 : want > 32 ? 32 : (int)want;
}

// The shares of a call.  A block's W windows of 8 KiB take W / s of a share's
// time, and adding s shares of 256 T bytes takes s T / 32: their sum is least at
// s = sqrt(32 W / T).  (63 tokens, 16 experts, 416 x 384: 22.6 us with the rule above
// alone, 19.8 with this one.)
int down_shares(const FewArgs &A, int windows, int cols) {
    const int pairs = A.T * A.k, entries = (A.gate.E < pairs ? A.gate.E : pairs) + pairs / cols;
    const int best = (int)sqrt(32.0 * entries * windows / A.T), most = most_shares(A.T, A.k, A.H, A.I);
    return best < 1 ? 1 : best < most ? best : most;
}

__device__ __forceinline__ void store_past_l2(uint64_t *p, float a, float b) {
    const uint64_t v = __builtin_bit_cast(uint32_t, a) | (uint64_t)__builtin_bit_cast(uint32_t, b) << 32;
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <bool kFp8, int kCols>
__global__ __launch_bounds__(kThreads) void down_kernel(const FewArgs A) {
    typedef Ring<kFp8, kCols, 2> R;
    __shared__ __align__(16) uint8_t stages[R::kStages * R::kStage];
    __shared__ Lists L;
    __shared__ float weights[kMaxPairs];
    __shared__ uint8_t scales[kFp8 ? kScaleUnits : 1];
    __shared__ int arrived;
    extern __shared__ __align__(16) float part[];  // [kWaves][T][16], read four at a time
    static_assert(sizeof(Scratch) <= sizeof(stages), "the scratch fits the stages");
    Scratch *W = reinterpret_cast<Scratch *>(stages);
    for (int p = threadIdx.x; p < A.T * A.k; p += kThreads) {
        W->ids[p] = A.ids[p];
        weights[p] = A.weights[p];
    }
    for (int i = threadIdx.x; i < kWaves * A.T * 16; i += kThreads) part[i] = 0.0f;
    __syncthreads();
    build_lists<kCols>(&L, W, A.T, A.k, A.gate.E);

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), l = lane_id(), r = l & 15, q = l >> 4;
    const int o0 = blockIdx.x * kRows, nw = windows_of<kFp8>(A.I);
    const int64_t every = (int64_t)L.entries * nw;
    const int u0 = (int)(every * blockIdx.y / gridDim.y), units = (int)(every * (blockIdx.y + 1) / gridDim.y) - u0;
    if (units > 0) {
        const bool partial = A.I % (64 * R::kHalves) != 0;
        R ring;
        ring.lds = stages;
        ring.wave = wave;
        ring.K = A.I;
        int pu = 0, pa = u0 / nw, pwin = u0 - pa * nw;
        auto sources = [&] {
            const int e = L.expert[pa], first = L.start[pa];
            const int n = ring.n = __builtin_amdgcn_readfirstlane(L.count[pa]);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int o = min(o0 + ring.weight_row(i), A.H - 1);
                ring.w[i] = A.wd.data + e * A.wd.stride + o * row_bytes<kFp8>(A.I) + R::chunk() * 16;
            }
#pragma unroll
            for (int i = 0; i < R::kMine; i++) {
                const int c = ring.column_row(i) % kCols, ph = ring.column_row(i) / kCols;
                const uint16_t *h = ph / R::kHalves ? A.hlo : A.hhi;
                h += (int64_t)L.pair[first + min(c, n - 1)] * A.I;  // columns past the end repeat the last
                ring.col[i] = reinterpret_cast<const uint8_t *>(h) + (ph % R::kHalves) * 128 + R::chunk() * 16;
            }
        };
        auto produce = [&](int slot) {
            ring.issue(slot, pwin, partial);
            pu++;
            if (pu < units && ++pwin == nw) {
                pwin = 0;
                pa++;
                sources();
            }
        };
        sources();
#pragma unroll
        for (int s = 0; s < R::kStages - 1; s++) produce(s);

        f32x4 acc[R::kTiles];
#pragma unroll
        for (int t = 0; t < R::kTiles; t++) acc[t] = f32x4{0, 0, 0, 0};
        int slot = 0, a = u0 / nw, win = u0 - a * nw;
        float *mine = part + wave * A.T * 16;
        for (int u = 0; u < units; u++) {
            if (kFp8 && u % kScaleUnits == 0) {
                if (u > 0) __syncthreads();
                for (int i = threadIdx.x; i < min(kScaleUnits, units - u); i += kThreads) {
                    const int un = u0 + u + i, e = L.expert[un / nw];
                    scales[i] = A.wd.scale[e * A.wd.scale_stride + (int64_t)(o0 / kScaleBlock) * nw + un % nw];
                }
            }
            ring.arrive();
            produce(slot == 0 ? R::kStages - 1 : slot - 1);
            const int n = __builtin_amdgcn_readfirstlane(L.count[a]);
            float scale = 1.0f;
            if constexpr (kFp8) scale = pow2_of(scales[u % kScaleUnits]);
            ring.multiply(slot, n, scale, acc);
            slot = slot == R::kStages - 1 ? 0 : slot + 1;
            if (++win < nw && u + 1 < units) continue;
            // the wave's own sums: an entry has a token once, so lanes do not meet
#pragma unroll
            for (int t = 0; t < R::kTiles; t++) {
                if (t * 8 >= n) break;
                f32x4 both;
#pragma unroll
                for (int i = 0; i < 4; i++) both[i] = acc[t][i] + __shfl_xor(acc[t][i], 8);
                const int c = t * 8 + r;
                if (r < 8 && c < n) {
                    const int p = L.pair[L.start[a] + c];
                    f32x4 *d = reinterpret_cast<f32x4 *>(mine + (p / A.k) * 16 + 4 * q);
                    f32x4 v = *d;
#pragma unroll
                    for (int i = 0; i < 4; i++) v[i] += weights[p] * both[i];
                    *d = v;
                }
                acc[t] = f32x4{0, 0, 0, 0};
            }
            wave_lds_fence();  // the next entry adds to sums that other lanes wrote
            win = 0;
            a++;
        }
        wait_loads();  // those that nobody reads
    }
    __syncthreads();
    const int rows = min(kRows, A.H - o0);
    auto value = [&](int t, int o) { return part[(o / 16 * A.T + t) * 16 + o % 16]; };
    if (gridDim.y == 1) {
        for (int i = threadIdx.x; i < A.T * rows; i += kThreads) {
            const int t = i / rows, o = i - t * rows;
            A.out[t * A.out_stride + o0 + o] = to_bf16(value(t, o));
        }
        return;
    }
    // Shares meet in memory: each writes its sums, and the last of a block of
    // rows to arrive adds them in the shares' order.  The sums are written and
    // read past the L2s, which the XCDs do not share (relaxed atomics of device
    // scope), so that waiting for the stores orders them before the arrival; a
    // fence would write back a whole L2 from every workgroup (70 us measured).
    // Four outputs a thread at a time (rows and H are multiples of 8).
    float *sums = A.sums + o0;
    const int64_t share = (int64_t)A.T * A.H;
    const int quads = rows / 4;
    for (int i = threadIdx.x; i < A.T * quads; i += kThreads) {
        const int t = i / quads, o = (i - t * quads) * 4;
        uint64_t *p = reinterpret_cast<uint64_t *>(sums + blockIdx.y * share + (int64_t)t * A.H + o);
        const f32x4 v = *reinterpret_cast<const f32x4 *>(part + (o / 16 * A.T + t) * 16 + o % 16);
        store_past_l2(p, v[0], v[1]);
        store_past_l2(p + 1, v[2], v[3]);
    }
    wait_loads();  // stores count too
    __syncthreads();
    if (threadIdx.x == 0)
        arrived = __hip_atomic_fetch_add(A.arrivals + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (arrived != (int)gridDim.y - 1) return;
    for (int i = threadIdx.x; i < A.T * quads; i += kThreads) {
        const int t = i / quads, o = (i - t * quads) * 4;
        const uint64_t *p = reinterpret_cast<const uint64_t *>(sums + (int64_t)t * A.H + o);
        float v[4] = {0, 0, 0, 0};
        for (int s0 = 0; s0 < (int)gridDim.y; s0 += 8) {
            uint64_t f[8][2];  // 16 loads in flight
#pragma unroll
            for (int s = 0; s < 8; s++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    f[s][h] = s0 + s < (int)gridDim.y
                                  ? __hip_atomic_load(p + (s0 + s) * (share / 2) + h, __ATOMIC_RELAXED,
                                                      __HIP_MEMORY_SCOPE_AGENT)
                                  : 0;
#pragma unroll
            for (int s = 0; s < 8; s++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    v[2 * h] += __builtin_bit_cast(float, (uint32_t)f[s][h]);
                    v[2 * h + 1] += __builtin_bit_cast(float, (uint32_t)(f[s][h] >> 32));
                }
        }
        uint16_t *out = A.out + t * A.out_stride + o0 + o;
#pragma unroll
        for (int j = 0; j < 4; j++) out[j] = to_bf16(v[j]);
    }
}

template <bool kFp8, int kCols>
const void *up_function(int E) {
    const int per = (E + kGateLanes - 1) / kGateLanes;
    return per <= 8    ? (const void *)up_kernel<kFp8, kCols, 8>
           : per <= 16 ? (const void *)up_kernel<kFp8, kCols, 16>
           : per <= 24 ? (const void *)up_kernel<kFp8, kCols, 24>
           : per <= 32 ? (const void *)up_kernel<kFp8, kCols, 32>
                       : (const void *)up_kernel<kFp8, kCols, 64>;
}

template <bool kFp8, int kUpCols, int kDownCols>
hipError_t launch(const FewArgs &A, hipStream_t s) {
    const int64_t most = ((int64_t)(A.gate.E < A.T * A.k ? A.gate.E : A.T * A.k) + A.T * A.k / kUpCols) *
                         ceil_div(A.I, kUpRows);
    const void *up = up_function<kFp8, kUpCols>(A.gate.E);
    const int64_t resident = resident_blocks(up, kThreads, 0);
    const int64_t blocks = resident > 0 && resident < most ? resident : most;
    void *args[] = {const_cast<FewArgs *>(&A)};
    const hipError_t e = hipLaunchKernel(up, dim3((uint32_t)blocks), dim3(kThreads), args, 0, s);
    if (e != hipSuccess) return e;
    const dim3 grid((uint32_t)ceil_div(A.H, kRows), down_shares(A, windows_of<kFp8>(A.I), kDownCols));
    return hipLaunchKernel((const void *)down_kernel<kFp8, kDownCols>, grid, dim3(kThreads), args,
                           (size_t)kWaves * A.T * 16 * sizeof(float), s);
}

template <bool kFp8>
hipError_t launch(const FewArgs &A, hipStream_t s) {
    // a token takes an expert once: with 8 tokens no expert has more than 8 pairs
    return A.T <= kFew ? launch<kFp8, kFew, kFew>(A, s) : launch<kFp8, kUpMany, kDownMany>(A, s);
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

namespace {

// Parts of the workspace, in bytes from its start
struct Parts {
    size_t low, arrivals, sums, total;
};

Parts parts_of(int32_t T, int32_t k, int32_t H, int32_t I) {
    Parts p;
    p.low = (size_t)T * k * I * sizeof(uint16_t);  // a multiple of 16: I is one of 8
    p.arrivals = align256(2 * p.low);
    p.sums = p.arrivals + align256((size_t)ceil_div(H, kRows) * sizeof(int32_t));
    p.total = p.sums + (size_t)most_shares(T, k, H, I) * T * H * sizeof(float);
    return p;
}

bool sizes_ok(int32_t T, int32_t k, int32_t H, int32_t I) {
    return T >= 0 && T <= kMaxTokens && k >= 1 && k <= kGateMaxK && H >= 8 && I >= 8 && H % 8 == 0 && I % 8 == 0 &&
           H <= kMaxWidth && I <= kMaxWidth;
}

}  // namespace

extern "C" size_t ep_few_tokens_workspace_bytes(int32_t num_tokens, int32_t top_k, int32_t hidden, int32_t inter) {
    if (!sizes_ok(num_tokens, top_k, hidden, inter) || num_tokens == 0) return 0;
    return parts_of(num_tokens, top_k, hidden, inter).total;
}

extern "C" int ep_moe_few_tokens(const void *x, int64_t x_stride, int32_t num_tokens, const void *logits,
                                 int64_t logits_stride, const ep_gate_t *gate, const ep_experts_t *experts, void *out,
                                 int64_t out_stride, int32_t *ids, float *weights, void *ws, size_t ws_bytes,
                                 ep_stream_t stream) {
    if (!gate_ok(gate) || !experts || !sizes_ok(num_tokens, gate->top_k, experts->hidden, experts->inter))
        return EP_ERR_INVALID_ARG;
    const int32_t H = experts->hidden, I = experts->inter, E = gate->num_experts;
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
    const Parts parts = parts_of(num_tokens, gate->top_k, H, I);
    if (!ws || !is_aligned(ws, 16) || ws_bytes < parts.total) return EP_ERR_INVALID_ARG;
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
    uint8_t *w = static_cast<uint8_t *>(ws);
    A.hhi = reinterpret_cast<uint16_t *>(w);
    A.hlo = reinterpret_cast<uint16_t *>(w + parts.low);
    A.arrivals = reinterpret_cast<int32_t *>(w + parts.arrivals);
    A.sums = reinterpret_cast<float *>(w + parts.sums);
    // With many tokens the gate runs by itself first, where each workgroup would take
    // 3 us for every 16 of them.  Measured, in the first kernel or before it: 63 tokens
    // 25 us, 6 + 10; 40 tokens 35, 5 + 29; 24 tokens 25, 4 + 21.
    A.chosen = num_tokens > kGateAlone;
    if (A.chosen) {
        const int rc = ep_gate_topk(logits, logits_stride, num_tokens, gate, ids, weights, stream);
        if (rc != EP_OK) return rc;
    }
    return rc_of(fp8 ? launch<true>(A, to_stream(stream)) : launch<false>(A, to_stream(stream)));
}
