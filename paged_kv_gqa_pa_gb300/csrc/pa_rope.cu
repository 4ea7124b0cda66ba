// pa_rope.cu -- rotary embedding of q and k with positions on several axes
// (pa_rope_axes of include/pa_q4.h).
//
// Bound by memory: every element is read and written once.  A CTA serves one
// token: its threads first request their elements, then work out the R / 2
// sines and cosines together (shared memory; all heads use the same), then
// rotate and store.  A work item is 16 bytes of a head's first half and the
// 16 bytes of their partners R / 2 dims on, or 16 bytes behind dim R, which
// are copied.
//
// Measured on GB300: 16384 bf16 tokens of 28 heads at D 256 70.8 us, 6.64 TB/s
// (0.98 of the measured copy rate).  Two items a thread and 48 registers, five
// CTAs of 256 threads per SM, keep the loads in flight; with four items (71
// registers) it took 88.1 us, with two and four CTAs 77.0.  64 tokens of 40
// heads at D 128: 2.3 us, a launch.
//
// Angles: the frequency as a fraction of a turn is a 64-bit fixed-point
// number f = round(2^64 theta^(-2 i / R) / (2 pi)), so position * f modulo
// 2^64 is the angle modulo one turn, exactly but for f's rounding (2^-34 of a
// turn at the largest position).  Its top 32 bits (2^-32 of a turn), as a signed
// fraction, go to fp32 (half a step: 2^-26 of a turn next to half a turn, less
// nearer to 0) and sincospif.  f has to be good to 64 bits, more than a double
// holds: the host works it out in pairs of doubles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "pa_q4.cuh"

namespace pa {

constexpr int kRopeThreads = 256;  // at most
constexpr int kRopeItems = 2;  // items a thread requests before it waits for the angles

struct RopeAxesParams {
    const unsigned char* q;
    const unsigned char* k;
    unsigned char* q_out;
    unsigned char* k_out;
    long long q_stride, k_stride, q_out_stride, k_out_stride;  // bytes
    const int* positions;
    int n, Hq, Hkv, D, R;
    int inverse;
    unsigned long long freq[kMaxRopePairs];
    unsigned char axis[kMaxRopePairs];
};

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

template <typename T>
__global__ void __launch_bounds__(kRopeThreads, 5) rope_axes_kernel(const RopeAxesParams p) {
    constexpr int N = RopeElem<T>::kN;
    constexpr int ES = 16 / N;
    __shared__ float s_cos[kMaxRopePairs];
    __shared__ float s_sin[kMaxRopePairs];
    const int tid = threadIdx.x, nt = blockDim.x;
    const long long t = blockIdx.x;
    const int half = p.R / 2;
    const int turn = half / N;                // rotated items of a head
    const int per_head = turn + (p.D - p.R) / N;
    const int items = (p.Hq + p.Hkv) * per_head;
    allow_dependent_launch();
    wait_for_prerequisite_grid();

    // Item i: chunk c of head h; src and dst of its first 16 bytes.
    auto locate = [&](int i, int& c, const unsigned char*& src, unsigned char*& dst) {
        const int h = i / per_head;
        c = i - h * per_head;
        const int dim = c < turn ? c * N : p.R + (c - turn) * N;
        const bool is_q = h < p.Hq;
        const size_t off = ((size_t)(is_q ? h : h - p.Hq) * p.D + dim) * ES;
        src = (is_q ? p.q + t * p.q_stride : p.k + t * p.k_stride) + off;
        dst = (is_q ? p.q_out + t * p.q_out_stride : p.k_out + t * p.k_out_stride) + off;
    };
    auto finish = [&](int c, const uint4& a, const uint4& b, unsigned char* dst) {
        if (c >= turn) {
            *reinterpret_cast<uint4*>(dst) = a;
            return;
        }
        float x[N], y[N], xr[N], yr[N];
        RopeElem<T>::load(a, x);
        RopeElem<T>::load(b, y);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float cs = s_cos[c * N + j], sn = s_sin[c * N + j];
            xr[j] = fmaf(x[j], cs, -(y[j] * sn));
            yr[j] = fmaf(y[j], cs, x[j] * sn);
        }
        *reinterpret_cast<uint4*>(dst) = RopeElem<T>::store(xr);
        *reinterpret_cast<uint4*>(dst + (size_t)half * ES) = RopeElem<T>::store(yr);
    };

    uint4 a[kRopeItems], b[kRopeItems];
    int c[kRopeItems];
    unsigned char* dst[kRopeItems];
#pragma unroll
    for (int u = 0; u < kRopeItems; ++u) {
        const int i = tid + u * nt;
        c[u] = -1;
        if (i < items) {
            const unsigned char* src;
            locate(i, c[u], src, dst[u]);
            a[u] = *reinterpret_cast<const uint4*>(src);
            if (c[u] < turn) b[u] = *reinterpret_cast<const uint4*>(src + (size_t)half * ES);
        }
    }
    for (int i = tid; i < half; i += nt) {
        const int pos = p.positions[(size_t)p.axis[i] * p.n + t];
        const unsigned long long turns = (unsigned long long)(long long)pos * p.freq[i];
        const float fr = (float)(int)(turns >> 32) * 4.656612873077393e-10f;  // 2^-31: half turns
        float sn, cs;
        sincospif(fr, &sn, &cs);
        s_cos[i] = cs;
        s_sin[i] = p.inverse ? -sn : sn;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kRopeItems; ++u)
        if (c[u] >= 0) finish(c[u], a[u], b[u], dst[u]);
    for (int i = tid + kRopeItems * nt; i < items; i += nt) {
        int ci;
        const unsigned char* src;
        unsigned char* d;
        locate(i, ci, src, d);
        const uint4 va = *reinterpret_cast<const uint4*>(src);
        uint4 vb = va;
        if (ci < turn) vb = *reinterpret_cast<const uint4*>(src + (size_t)half * ES);
        finish(ci, va, vb, d);
    }
}

// A number as the unevaluated sum of two doubles, about 104 bits.  (Written with
// explicit fma, so that every compiler gives the same bits.)
struct Pair {
    double hi, lo;
};

static Pair mul(const Pair& a, const Pair& b) {
    const double p = a.hi * b.hi;
    const double e = fma(a.hi, b.lo, fma(a.lo, b.hi, fma(a.hi, b.hi, -p)));
    const double s = p + e;
    return {s, e - (s - p)};
}

// 2^64 times x modulo one turn, rounded down, and what that leaves (0 <= rest < 1).
static unsigned long long turn64(double x, double* rest) {
    const double a = (x - rint(x)) * 18446744073709551616.0;  // exact, -2^63 .. 2^63
    const double whole = floor(a);
    *rest = a - whole;
    return whole >= 9223372036854775808.0 ? 1ull << 63 : (unsigned long long)(long long)whole;
}

// round(2^64 theta^(-2 i / R) / (2 pi)) modulo 2^64, i < R / 2: all 64 bits for bases
// from 1e-3 on (below, a position is so many turns that fewer are left behind the
// point).  On the Grace host 1.0 us for 128 frequencies; with a pow for each it
// was 1.8.
static void rope_frequencies(float theta, int R, unsigned long long* freq) {
    const int half = R / 2;
    // r = theta^(-1 / half): the double r0 and one step of Newton's method,
    // r0 (1 + (1 - theta r0^half) / half), whose error is the square of r0's.
    const double r0 = pow((double)theta, -1.0 / half);
    Pair power = {1.0, 0.0}, base = {r0, 0.0};
    for (int n = half; n; n >>= 1) {
        if (n & 1) power = mul(power, base);
        base = mul(base, base);
    }
    const Pair one = mul(power, {(double)theta, 0.0});
    const double step = ((1.0 - one.hi) - one.lo) / half * r0;
    const double r_hi = r0 + step;
    const Pair r = {r_hi, step - (r_hi - r0)};
    Pair f = {0.15915494309189535, -9.839338337591243e-18};  // 1 / (2 pi)
    for (int i = 0; i < half; ++i) {
        double rest_hi, rest_lo;
        freq[i] = turn64(f.hi, &rest_hi);
        freq[i] += turn64(f.lo, &rest_lo);
        freq[i] += (unsigned long long)rint(rest_hi + rest_lo);
        f = mul(f, r);
    }
}

}  // namespace pa

using namespace pa;

extern "C" int pa_rope_axes(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                            int rotary_dim, int num_axes, const int* sections, int interleaved,
                            int inverse, float theta, int dtype, const void* q,
                            long long q_stride, const void* k, long long k_stride,
                            const int32_t* positions, void* q_out, long long q_out_stride,
                            void* k_out, long long k_out_stride, void* stream) {
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 || head_dim <= 0 ||
        rotary_dim <= 0 || rotary_dim > head_dim || num_axes < 1 || num_axes > PA_ROPE_MAX_AXES ||
        !sections || interleaved < 0 || interleaved > 1 || inverse < 0 || inverse > 1 ||
        !(theta > 0.f) || theta == INFINITY)
        return PA_ERR_INVALID_ARG;
    if (dtype != PA_DTYPE_F16 && dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_F32)
        return PA_ERR_INVALID_ARG;
    if (head_dim > 2 * kMaxRopePairs || head_dim % 16 != 0 || rotary_dim % 16 != 0 ||
        (long long)num_q_heads + num_kv_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    const int half = rotary_dim / 2;
    long long sum = 0;
    for (int a = 0; a < num_axes; ++a) {
        if (sections[a] < 0) return PA_ERR_INVALID_ARG;
        sum += sections[a];
    }
    if (sum != half) return PA_ERR_INVALID_ARG;
    RopeAxesParams p;
    if (interleaved) {
        // Every axis but the first finds its pairs among i % num_axes == a.
        for (int a = 1; a < num_axes; ++a)
            if (sections[a] > 0 && num_axes * (sections[a] - 1) + a >= half)
                return PA_ERR_INVALID_ARG;
        for (int i = 0; i < half; ++i) {
            const int a = i % num_axes;
            p.axis[i] = (unsigned char)(i < num_axes * sections[a] ? a : 0);
        }
    } else {
        int i = 0;
        for (int a = 0; a < num_axes; ++a)
            for (int j = 0; j < sections[a]; ++j) p.axis[i++] = (unsigned char)a;
    }
    const bool has_q = num_q_heads > 0, has_k = num_kv_heads > 0;
    const int es = dtype == PA_DTYPE_F32 ? 4 : 2, vec = 16 / es;
    const long long lim = 1ll << 40;
    if (has_q && (q_stride < (long long)num_q_heads * head_dim || q_stride % vec || q_stride > lim ||
                  q_out_stride < (long long)num_q_heads * head_dim || q_out_stride % vec ||
                  q_out_stride > lim || (q == q_out && q_stride != q_out_stride)))
        return PA_ERR_INVALID_ARG;
    if (has_k && (k_stride < (long long)num_kv_heads * head_dim || k_stride % vec || k_stride > lim ||
                  k_out_stride < (long long)num_kv_heads * head_dim || k_out_stride % vec ||
                  k_out_stride > lim || (k == k_out && k_stride != k_out_stride)))
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0 || (!has_q && !has_k)) return PA_OK;
    if (!positions || (has_q && (!q || !q_out)) || (has_k && (!k || !k_out)))
        return PA_ERR_INVALID_ARG;
    // (in place with k = q, or into one output, q's rows and k's would be written over one another)
    if (has_q && has_k && q_out == k_out) return PA_ERR_INVALID_ARG;
    uintptr_t bits = 0;
    if (has_q) bits |= (uintptr_t)q | (uintptr_t)q_out;
    if (has_k) bits |= (uintptr_t)k | (uintptr_t)k_out;
    if ((bits & 15u) || ((uintptr_t)positions & 3u)) return PA_ERR_INVALID_ARG;
    // Frequencies as 64-bit fractions of a turn; the table of the last (base,
    // rotary dim) this thread used is kept.  (A model whose layers alternate
    // between two bases pays the table, up to 1 us of host time, in every call.)
    thread_local float t_theta = 0.f;
    thread_local int t_R = 0;
    thread_local unsigned long long t_freq[kMaxRopePairs];
    if (t_theta != theta || t_R != rotary_dim) {
        rope_frequencies(theta, rotary_dim, t_freq);
        t_theta = theta;
        t_R = rotary_dim;
    }
    memcpy(p.freq, t_freq, sizeof(unsigned long long) * half);
    p.q = static_cast<const unsigned char*>(q);
    p.k = static_cast<const unsigned char*>(k);
    p.q_out = static_cast<unsigned char*>(q_out);
    p.k_out = static_cast<unsigned char*>(k_out);
    p.q_stride = q_stride * es;
    p.k_stride = k_stride * es;
    p.q_out_stride = q_out_stride * es;
    p.k_out_stride = k_out_stride * es;
    p.positions = positions;
    p.n = num_tokens;
    p.Hq = num_q_heads;
    p.Hkv = num_kv_heads;
    p.D = head_dim;
    p.R = rotary_dim;
    p.inverse = inverse;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)num_tokens);
    // Threads for kRopeItems items each.
    const int items = (num_q_heads + num_kv_heads) * (half / vec + (head_dim - rotary_dim) / vec);
    const int threads = (items + kRopeItems * 32 - 1) / (kRopeItems * 32) * 32;
    cfg.blockDim = dim3(std::min(kRopeThreads, threads));
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    switch (dtype) {
        case PA_DTYPE_F32: e = cudaLaunchKernelEx(&cfg, rope_axes_kernel<float>, p); break;
        case PA_DTYPE_BF16: e = cudaLaunchKernelEx(&cfg, rope_axes_kernel<__nv_bfloat16>, p); break;
        default: e = cudaLaunchKernelEx(&cfg, rope_axes_kernel<__half>, p); break;
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return PA_OK;
}
