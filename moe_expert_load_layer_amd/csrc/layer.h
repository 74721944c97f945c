// Device helpers shared by the operators around the balancer: bf16 and scale
// byte conversions, reductions over the 16 lanes of a DPP row.
#pragma once

#include "ep_internal.h"

namespace ep {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// Vectors in memory at any address that their elements may have: the card takes
// them in one access, so rows of odd lengths cost no more instructions.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kScaleBlock = 128;  // values that share one scale byte
// workgroups of 256 threads in one launch: the runtime counts threads in 32 bits
constexpr int64_t kMaxBlocks = 0xffffffffll / 256;

inline hipStream_t to_stream(ep_stream_t s) { return reinterpret_cast<hipStream_t>(s); }
inline bool is_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline int rc_of(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_HIP; }
inline bool float_dtype(int32_t d) { return d == EP_DTYPE_F32 || d == EP_DTYPE_BF16; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }

// to nearest, ties to even; NaN stays NaN
__device__ __forceinline__ uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return (uint32_t)to_bf16(a) | ((uint32_t)to_bf16(b) << 16);
}

// 2^(c - 127) for c in 1..254
__device__ __forceinline__ float pow2_of(int c) { return __builtin_bit_cast(float, (uint32_t)c << 23); }

// The scale byte of a block in 8 bits whose largest finite magnitude is amax: the
// smallest c with amax <= 448 * 2^(c - 127)
__device__ __forceinline__ int fp8_scale_code(float amax) {
    const uint32_t b = __builtin_bit_cast(uint32_t, amax);
    const int c = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u);
    return min(max(c, 1), 254);
}

// One DPP step: the value of the lane that `ctrl` names, in the row of 16
template <int ctrl>
__device__ __forceinline__ float dpp_f32(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), ctrl, 0xF, 0xF, true));
}

// Maximum over the 16 lanes of a DPP row, in every lane (the steps as in
// wave_max_i32; all lanes of the row active).  NaN operands are ignored.
__device__ __forceinline__ float row_max_f32(float v) {
    v = fmaxf(v, dpp_f32<0xB1>(v));
    v = fmaxf(v, dpp_f32<0x4E>(v));
    v = fmaxf(v, dpp_f32<0x141>(v));
    return fmaxf(v, dpp_f32<0x140>(v));
}

// Sum over the 16 lanes of a DPP row, in every lane; the tree is fixed
__device__ __forceinline__ float row_sum_f32(float v) {
    v += dpp_f32<0xB1>(v);
    v += dpp_f32<0x4E>(v);
    v += dpp_f32<0x141>(v);
    return v + dpp_f32<0x140>(v);
}

}  // namespace ep
