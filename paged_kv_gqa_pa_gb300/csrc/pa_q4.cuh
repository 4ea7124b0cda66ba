// pa_q4.cuh -- the 4-bit cache's layout and arithmetic (include/pa_q4.h),
// shared by the kernels that write it, read it back and attend over it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/pa_q4.h"
#include "pa_common.cuh"

namespace pa {

constexpr int kQ4Group = 32;  // dims that share a scale and an offset

__host__ __device__ constexpr bool q4_head_dim_ok(int D) {
    return D == 64 || D == 96 || D == 128 || D == 256;
}

// Byte offsets inside the block of one (page, KV head); see pa_q4.h for why
// the V codes lie in the order of a warp's lanes.
template <int D>
struct Q4Layout {
    static constexpr int kPageBytes = 20 * D;
    static constexpr int kVCodes = 8 * D;
    static constexpr int kKParams = 16 * D;
    static constexpr int kVParams = 18 * D;
    static constexpr int kSlice = D < 128 ? D : 128;          // dims of a K slice
    static constexpr int kSlices = D / kSlice;
    static constexpr int kGroups = D / kQ4Group;
    static constexpr int kSliceGroups = kSlice / kQ4Group;
    static constexpr int kWords = D / 32;                      // V words per lane and token pair
    static constexpr int kVec = D % 128 == 0 ? 4 : (D == 64 ? 2 : 1);  // words of one read
    static_assert(kPageBytes % 128 == 0, "page blocks keep 16-byte alignment");

    // K codes of dims d .. d + 7 (d a multiple of 8) of token r: one 32-bit word.
    __host__ __device__ static constexpr int k_codes(int r, int d) {
        return (d / kSlice) * (8 * kSlice) + r * (kSlice / 2) + (d % kSlice) / 2;
    }
    // V codes of dims d .. d + 3 (d a multiple of 4) of token r: 16 bits.
    __host__ __device__ static constexpr int v_codes(int r, int d) {
        const int col = D == 96 ? (d % 32) / 4 : d / (D / 8);
        const int w = D == 96 ? d / 32 : (d % (D / 8)) / 4;
        const int j = r / 2;
        return kVCodes + (j / 4) * (4 * D) + (w / kVec) * (128 * kVec) +
               (4 * col + j % 4) * (4 * kVec) + (w % kVec) * 4 + (r % 2) * 2;
    }
    // (s, z) of token r, group n: K's 32-bit cell; V's s (z lies 4 bytes on).
    __host__ __device__ static constexpr int k_params(int r, int n) {
        return kKParams + 4 * (((n / kSliceGroups) * kPageSize + r) * kSliceGroups +
                               n % kSliceGroups);
    }
    __host__ __device__ static constexpr int v_params(int r, int n) {
        return kVParams + ((r / 2) * kGroups + n) * 8 + (r % 2) * 2;
    }
};

// (x & mask) | bits as one lop3: written with & and | the compiler keeps both
// constants immediate and spends two.
__device__ __forceinline__ uint32_t q4_join(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "r"(mask), "r"(bits));
    return d;
}

// Element-type specifics.  A code c becomes the 16-bit float 16 + c: 16 has a
// zero mantissa, and its unit in the last place is 2^-6 (fp16) or 2^-3
// (bf16), so c is shifted to bit 6 (3) and joined to 16's bits.
template <typename T>
struct Q4Type;

template <>
struct Q4Type<__half> {
    static constexpr float kLimit = 16384.f;
    // A 32-bit word holds four codes in each half; the pair at bits 4 P of both.
    template <int P>
    __device__ static __forceinline__ uint32_t code16(uint32_t w) {
        const uint32_t x = P == 0 ? w << 6 : (P == 1 ? w << 2 : (P == 2 ? w >> 2 : w >> 6));
        return q4_join(x, 0x03C003C0u, 0x4C004C00u);
    }
    __device__ static __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t d;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
        return d;
    }
    __device__ static __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ static __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ static __forceinline__ float to_float(uint32_t bits) {
        return __half2float(__ushort_as_half((unsigned short)bits));
    }
    __device__ static __forceinline__ uint32_t from_float(float v) {
        return __half_as_ushort(__float2half_rn(v));
    }
    __device__ static __forceinline__ uint32_t from_double(double v) {
        return __half_as_ushort(__double2half(v));
    }
    // Whether rounding q >= 0, itself a rounded quotient, to T may differ from
    // rounding the exact quotient: q within a few of its own units of the
    // middle between two values of T, or in T's subnormal range.
    __device__ static __forceinline__ bool near_tie(float q) {
        const uint32_t low = __float_as_uint(q) & 0x1FFFu;
        return (low - (0x1000u - 4u) <= 8u || q < 6.103515625e-05f) && q != 0.f;
    }
};

template <>
struct Q4Type<__nv_bfloat16> {
    static constexpr float kLimit = 1.329227995784916e36f;  // 2^120
    template <int P>
    __device__ static __forceinline__ uint32_t code16(uint32_t w) {
        const uint32_t x = P == 0 ? w << 3 : (P == 1 ? w >> 1 : (P == 2 ? w >> 5 : w >> 9));
        return q4_join(x, 0x00780078u, 0x41804180u);
    }
    __device__ static __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t d;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
        return d;
    }
    __device__ static __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ static __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ static __forceinline__ float to_float(uint32_t bits) {
        return __uint_as_float(bits << 16);
    }
    __device__ static __forceinline__ uint32_t from_float(float v) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
    // A double rounded once: to fp32 with a sticky last bit (toward zero, then
    // odd if anything was lost), which leaves the second rounding exact.
    __device__ static __forceinline__ uint32_t from_double(double v) {
        float f = __double2float_rz(v);
        if ((double)f != v) f = __uint_as_float(__float_as_uint(f) | 1u);
        return from_float(f);
    }
    __device__ static __forceinline__ bool near_tie(float q) {
        const uint32_t low = __float_as_uint(q) & 0xFFFFu;
        return (low - (0x8000u - 4u) <= 8u || q < 1.1754943508222875e-38f) && q != 0.f;
    }
};

}  // namespace pa
