// pa_rope.cuh -- what the kernels that rotate rows share (pa_rope.cu, pa_append.cu):
// 16 bytes of elements as fp32 and back, and the frequency table.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace pa {

// Frequencies theta^(-2 i / R) as 64-bit fractions of a turn; the table of the last
// (base, rotary dim) this thread used is kept.  (A model whose layers alternate
// between two bases pays the table, up to 1 us of host time, in every call.)
const unsigned long long* rope_frequency_table(float theta, int R);

// Cosine and sine of position * frequency.  The product modulo 2^64 is the angle
// modulo one turn; its top 32 bits, as a signed fraction, go to fp32 and sincospif.  (pa_rope.cu's;
// pa_append.cu has one that is off by half as much.)
__device__ __forceinline__ void rope_angle(int pos, unsigned long long freq, float& cs, float& sn) {
    const unsigned long long turns = (unsigned long long)(long long)pos * freq;
    sincospif((float)(int)(turns >> 32) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31: half turns
}

template <typename T>
struct RopeElem;
template <>
struct RopeElem<__half> {
    static constexpr int kN = 8;  // elements of 16 bytes
    __device__ static __forceinline__ void load(const uint4& u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
    __device__ static __forceinline__ uint4 store(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct RopeElem<__nv_bfloat16> {
    static constexpr int kN = 8;
    __device__ static __forceinline__ void load(const uint4& u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static __forceinline__ uint4 store(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct RopeElem<float> {
    static constexpr int kN = 4;
    __device__ static __forceinline__ void load(const uint4& u, float (&f)[4]) {
        f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
    }
    __device__ static __forceinline__ uint4 store(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};

}  // namespace pa
