// Operands of a product that sums over the rows of both: bf16 rows in LDS, read
// transposed.  Shared by the weight gradients.
#pragma once

#include "groups.h"

namespace ep {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// what stands for rows and columns that a tile does not have
static __device__ __align__(16) const uint32_t kZeros[4] = {0, 0, 0, 0};

// the 16-byte chunk of an LDS row that holds chunk c of the matrix row
__device__ __forceinline__ int swizzle(int row, int c) { return c ^ ((row & 3) << 2); }

// rows t .. t + 7 (this lane's half of 16) of column c0 + l % 32, as 8 bf16
template <int kCols>
__device__ __forceinline__ bf16x8 read_columns(const uint16_t *tile, int t0, int c0) {
    const int l = lane_id(), i = l & 15, c = c0 + ((l >> 4) & 1) * 16 + (i & 3) * 4;
    union {
        s16x4 h[2];
        bf16x8 v;
    } u;
#pragma unroll
    for (int p = 0; p < 2; p++) {
        const int t = t0 + (l >> 5) * 8 + p * 4 + (i >> 2);
        const uint16_t *a = tile + t * kCols + swizzle(t, c / 8) * 8 + c % 8;
        u.h[p] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)a);
    }
    return u.v;
}

}  // namespace ep
