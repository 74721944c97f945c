// Groups of consecutive rows (one per expert or physical slot) and the tiles
// that cover them, for the grouped products.
#pragma once

#include "layer.h"

namespace ep {

constexpr int64_t kMaxRows = 0x7fffffffll - 1024;  // a tile past the last row still counts in 32 bits

// Rows [start, end) of group g; the offsets come from device memory and are
// brought into [0, M] and into order here, so that no value of theirs reaches
// past a buffer.  Null offsets: one group of all rows.
struct Groups {
    const int32_t *offsets;
    int32_t G, M;
    __device__ __forceinline__ int start(int g) const {
        return offsets ? min(max(offsets[g], 0), M) : 0;
    }
    __device__ __forceinline__ int end(int g) const { return offsets ? max(min(offsets[g + 1], M), start(g)) : M; }
};

// Where a group's matrix lives: row g of `own`, or, with a layout, the native
// expert's row or the spare slot's row of the slot buffer.
struct GroupRows {
    const int32_t *slot_home, *slot_spare;  // null: row g
    __device__ __forceinline__ bool spare(int g, int *row) const {
        if (!slot_home) {
            *row = g;
            return false;
        }
        const int home = slot_home[g];
        *row = home >= 0 ? home : slot_spare[g];
        return home < 0;
    }
};

// Fills *where; false if the layout does not have that many physical slots, or
// has spare slots where the call has no buffer for them.
bool layout_groups(const ep_layout_t *layout, int32_t groups, bool slots, GroupRows *where);

// The tile-th tile of T rows over the groups in order, found by every wave for
// itself: *g its group, *first the tiles before that group.  Returns false past
// the last tile; total_tiles is their number.
__device__ __forceinline__ int group_tiles(const Groups &R, int g, int T) {
    return g < R.G ? (R.end(g) - R.start(g) + T - 1) / T : 0;
}

__device__ __forceinline__ int total_tiles(const Groups &R, int T) {
    int total = 0;
    for (int g0 = 0; g0 < R.G; g0 += kWave) total += wave_sum_i32(group_tiles(R, g0 + lane_id(), T));
    return total;
}

__device__ __forceinline__ bool find_tile(const Groups &R, int T, int tile, int *g, int *first) {
    int before = 0;
    for (int g0 = 0; g0 < R.G; g0 += kWave) {
        const int c = group_tiles(R, g0 + lane_id(), T);
        const int incl = wave_incl_scan_i32(c);
        const int sum = __builtin_amdgcn_readlane(incl, kWave - 1);
        if (tile < before + sum) {
            const uint64_t past = __ballot(before + incl > tile);
            const int l = __builtin_ctzll(past);
            *g = g0 + l;
            *first = before + __builtin_amdgcn_readlane(incl - c, l);
            return true;
        }
        before += sum;
    }
    return false;
}

// Starts a load of 1 KiB from memory into LDS: lane i's 16 bytes go to
// `lds` + 16 i, `lds` the same in every lane.  It has no register result and
// is counted in vmcnt; wait_loads() waits for this wave's.  Written in asm
// because the compiler would wait for every such load before any later read
// of LDS, also of the other stage.  The forms below take 4 bytes a lane, or one
// byte that gets 4 in LDS: lane i's at `lds` + 4 i.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is named as changed on purpose
__device__ __forceinline__ uint32_t lds_address(void *lds) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) void *)lds);
}
__device__ __forceinline__ void load_lds_1k(const void *g, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(g) : "m0", "memory");
}
__device__ __forceinline__ void load_lds_1k(const void *g, void *lds) { load_lds_1k(g, lds_address(lds)); }
__device__ __forceinline__ void load_lds_dwords(const void *g, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(g) : "m0", "memory");
}
__device__ __forceinline__ void load_lds_bytes(const void *g, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_ubyte %1, off" ::"s"(lds), "v"(g) : "m0", "memory");
}
#pragma clang diagnostic pop

// Waits until at most N of this wave's loads are in flight.
template <int N>
__device__ __forceinline__ void wait_loads_but() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

}  // namespace ep
