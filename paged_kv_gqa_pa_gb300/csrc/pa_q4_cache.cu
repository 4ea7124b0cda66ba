// pa_q4_cache.cu -- rows of K and V into the 4-bit paged cache and back
// (pa_q4_write, pa_q4_read of include/pa_q4.h).
//
// A row of D elements (2 D bytes) is read and leaves as 0.625 D bytes of codes
// and parameters, or the reverse.  A thread has 8 consecutive dims (16 bytes)
// of a token and goes through its share of the KV heads, K and V, so that the
// slot and the addresses are worked out once; the four lanes of an aligned
// quad hold a group of 32 dims, and D / 8 consecutive lanes a row.  The next
// head's rows are requested before the present ones are worked on.
//
// Measured on GB300, 16384 bf16 rows of 4 heads at D 256 (88 MB either way, 13
// us at the measured copy rate): the writer 27.3 us, bound by what it issues
// (71 % of the slots; the borders of exact codes are most of it), the reader
// 19.1 us, bound by memory latency (0.68 of the copy rate); one behind the
// other 43.2, since the cells just written are still in L2.  64 rows of 8 heads
// at D 128: 1.9 and 1.4 us, a launch.
#include <algorithm>

#include "pa_q4.cuh"

namespace pa {

constexpr int kQ4Threads = 256;

struct Q4CacheParams {
    const int64_t* slots;
    unsigned char* cache;
    unsigned char* k;      // rows (read by the writer, written by the reader)
    unsigned char* v;
    long long k_stride;    // bytes from token to token
    long long v_stride;
    unsigned* err;
    int n, Hkv;
    int heads;             // KV heads a thread serves (blockIdx.y: which)
    long long num_slots;   // num_pages * 16
};

// The fp64 steps, taken where an fp32 quotient lies close to a rounding border
// of T or 1 / s overflows.  Out of line: inlined, their conversions ran for
// every element and kept the fp64 pipe 78 % busy (16384 bf16 rows of 4 x 256:
// 74 us).
template <typename T>
__device__ __noinline__ uint32_t exact_scale(float mx, float mn) {
    return Q4Type<T>::from_double(((double)mx - (double)mn) / 15.0);
}

__device__ __noinline__ float exact_code(float x, float z, float s) {
    return (float)rint(((double)x - (double)z) / (double)s);
}

// Quantise the 8 elements of a lane (the quad's 32 form the group): codes of
// dims 4 i .. 4 i + 3 in the low half of code[i], first dim lowest.
//
// With d = x - z the code is rint(d / s) - 16.  v = fma(d, 1 / s, 1.5 2^23)
// rounds the quotient to an integer r in one step, wrong only where d / s lies
// within 2^-16 of the middle between two integers; there the residual
// d - r s, which is exact, decides.  Such middles are common, not rare: values
// and scales of T are coarse, so about one bf16 element in 300 is an exact
// tie.  They are looked for four elements at a time: of all eight together, three
// warps in five had one.
template <typename T>
__device__ __forceinline__ void quantise8(const uint4& raw, uint32_t (&code)[2], uint32_t& s16,
                                          uint32_t& z16) {
    using Q = Q4Type<T>;
    constexpr float kMagic = 12582912.f;  // 1.5 2^23
    const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
    // (max, -min) of the quad as one packed pair, NaN kept.
    const uint32_t hi = Q::max2_nan(Q::max2_nan(x[0], x[1]), Q::max2_nan(x[2], x[3]));
    const uint32_t lo =
        Q::min2_nan(Q::min2_nan(x[0], x[1]), Q::min2_nan(x[2], x[3])) ^ 0x80008000u;
    uint32_t ext = Q::max2_nan(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
    ext = Q::max2_nan(ext, __shfl_xor_sync(0xffffffffu, ext, 1));
    ext = Q::max2_nan(ext, __shfl_xor_sync(0xffffffffu, ext, 2));
    float mx = Q::to_float(ext & 0xffffu);
    float mn = -Q::to_float(ext >> 16);
    const bool nan = mx != mx || mn != mn;
    const float most = mx, least = mn;
    mx = fminf(fmaxf(mx, -Q::kLimit), Q::kLimit);
    mn = fminf(fmaxf(mn, -Q::kLimit), Q::kLimit);
    const float qs = (mx - mn) * (1.f / 15.f);  // (within 2 of its units)
    s16 = Q::from_float(qs);
    if (Q::near_tie(qs)) s16 = exact_scale<T>(mx, mn);
    // z = RN_T(mn - 16 s): mn is a value of T, so this is one fma of T.
    z16 = Q::fma2(Q::from_float(-16.f), s16, Q::from_float(mn)) & 0xffffu;
    const float s = Q::to_float(s16), z = Q::to_float(z16);
    float inv;  // within 1 unit (s = 0: inf, and the codes are dropped below)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const float half = 0.5f * s, close = half * 0.99996f;
    float v[8];
    const float2 inv2 = make_float2(inv, inv), s2 = make_float2(s, s), nz2 = make_float2(-z, -z);
    const float2 magic2 = make_float2(kMagic, kMagic), minus2 = make_float2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        float2 xv[2], d[2], res[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t w = x[i / 2 + k];
            xv[k] = make_float2(Q::to_float(w & 0xffffu), Q::to_float(w >> 16));
            d[k] = __fadd2_rn(xv[k], nz2);
            // Off by less than 2^-17 before it is rounded, for quotients up to 32:
            // d, 1 / s and its use, 32 (2^-24 + 2^-23).
            const float2 r = __ffma2_rn(d[k], inv2, magic2);
            res[k] = __ffma2_rn(__ffma2_rn(r, minus2, magic2), s2, d[k]);
            v[i + 2 * k] = r.x;
            v[i + 2 * k + 1] = r.y;
        }
        const float worst = fmaxf(fmaxf(fabsf(res[0].x), fabsf(res[0].y)),
                                  fmaxf(fabsf(res[1].x), fabsf(res[1].y)));
        if (__any_sync(0xffffffffu, worst > close)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // what d lost: x - z = d + e (packed: 16384 bf16 rows of 4 heads at
                // D 256, written and read, 44.1 -> 43.1 us)
                const float2 back = __ffma2_rn(xv[k / 2], minus2, d[k / 2]);
                const float2 kept = __ffma2_rn(__ffma2_rn(back, minus2, d[k / 2]), minus2, xv[k / 2]);
                const float2 e2 = __ffma2_rn(__fadd2_rn(back, make_float2(z, z)), minus2, kept);
                const float rk = k & 1 ? res[k / 2].y : res[k / 2].x;
                const float e = k & 1 ? e2.y : e2.x;
                const float over = (fabsf(rk) - half) +
                                   __uint_as_float(__float_as_uint(e) ^
                                                   (__float_as_uint(rk) & 0x80000000u));
                // above the middle, or on it with r odd
                const float bar = __uint_as_float((__float_as_uint(v[i + k]) & 1u) * 0x80000001u);
                if (over > bar) v[i + k] += copysignf(1.f, rk);
            }
        }
    }
    if (s < 1e-37f && s16 != 0) {  // 1 / s overflows (bf16 only)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = kMagic +
                   exact_code(Q::to_float(i & 1 ? x[i / 2] >> 16 : x[i / 2] & 0xffffu), z, s);
    }
    // Codes below 0 or above 15 come from values beyond the limits, or spaced
    // wider than the step: seen from the group's least and greatest.
    constexpr float kLow = kMagic + 16.f, kHigh = kMagic + 31.f;
    if (__any_sync(0xffffffffu,
                   !((least - z) * inv >= 15.625f && (most - z) * inv <= 31.375f))) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], kLow), kHigh);
    }
    // The bits of kMagic + 16 + c, each moved to its place and added up; what
    // all eight constants add up to is taken off again.
    constexpr uint32_t kOne = 0x4B400010u;
    constexpr uint32_t kSum = kOne + (kOne << 4) + (kOne << 8) + (kOne << 12);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t sum = 0u - kSum;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += __float_as_uint(v[4 * k + i]) << (4 * i);
        code[k] = nan || s16 == 0 ? 0u : sum;
    }
    if (nan) {
        s16 = 0;
        z16 = 0x7FFFu;  // NaN in fp16 and bf16
    }
}

// Byte offsets of a thread's cells in a page block, and where its rows lie.
template <int D>
struct Q4Lane {
    using L = Q4Layout<D>;
    static constexpr int kLanes = D / 8;  // of a row
    long long tok;
    int c8;            // first dim
    long long slot;    // -1: left out (or no token)
    bool bad;
    size_t block0;     // byte offset of KV head 0's block of the slot's page
    int k_codes, v_codes0, v_codes1, k_par, v_par;

    __device__ __forceinline__ explicit Q4Lane(const Q4CacheParams& p) {
        const long long idx = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
        tok = idx / kLanes;
        c8 = (int)(idx % kLanes) * 8;
        slot = tok < p.n ? p.slots[tok] : -1;
        bad = slot < -1 || slot >= p.num_slots;
        if (bad) slot = -1;
        if (bad && p.err && blockIdx.y == 0 && c8 == 0) atomicOr(p.err, PA_DEVERR_BAD_SLOT);
        const int r = slot < 0 ? 0 : (int)(slot % kPageSize);
        block0 = slot < 0 ? 0
                          : (size_t)(slot / kPageSize) * p.Hkv * (size_t)L::kPageBytes;
        k_codes = L::k_codes(r, c8);
        v_codes0 = L::v_codes(r, c8);
        v_codes1 = L::v_codes(r, c8 + 4);
        k_par = L::k_params(r, c8 / kQ4Group);
        v_par = L::v_params(r, c8 / kQ4Group);
    }
};

template <int D, typename T>
__global__ void __launch_bounds__(kQ4Threads) q4_write_kernel(const Q4CacheParams p) {
    using L = Q4Layout<D>;
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    const Q4Lane<D> ln(p);
    const bool has = ln.tok < p.n, keep = ln.slot >= 0;
    const int h0 = blockIdx.y * p.heads, h1 = min(p.Hkv, h0 + p.heads);
    const bool first = (ln.c8 & (kQ4Group - 1)) == 0;  // the quad's lane that stores s and z
    const uint4 none = make_uint4(0, 0, 0, 0);
    const unsigned char* kr = p.k + ln.tok * p.k_stride + ((size_t)h0 * D + ln.c8) * 2;
    const unsigned char* vr = p.v + ln.tok * p.v_stride + ((size_t)h0 * D + ln.c8) * 2;
    unsigned char* block = p.cache + ln.block0 + (size_t)h0 * L::kPageBytes;
    uint4 k = has ? *reinterpret_cast<const uint4*>(kr) : none;
    uint4 v = has ? *reinterpret_cast<const uint4*>(vr) : none;
    for (int h = h0; h < h1; ++h) {
        uint4 k_next = none, v_next = none;
        if (has && h + 1 < h1) {
            k_next = *reinterpret_cast<const uint4*>(kr += 2 * D);
            v_next = *reinterpret_cast<const uint4*>(vr += 2 * D);
        }
        uint32_t code[2], s16, z16;
        quantise8<T>(k, code, s16, z16);  // (every lane takes part in the quad's shuffles)
        if (keep) {
            *reinterpret_cast<uint32_t*>(block + ln.k_codes) = code[0] | (code[1] << 16);
            if (first) *reinterpret_cast<uint32_t*>(block + ln.k_par) = s16 | (z16 << 16);
        }
        quantise8<T>(v, code, s16, z16);
        if (keep) {
            *reinterpret_cast<uint16_t*>(block + ln.v_codes0) = (uint16_t)code[0];
            *reinterpret_cast<uint16_t*>(block + ln.v_codes1) = (uint16_t)code[1];
            if (first) {
                *reinterpret_cast<uint16_t*>(block + ln.v_par) = (uint16_t)s16;
                *reinterpret_cast<uint16_t*>(block + ln.v_par + 4) = (uint16_t)z16;
            }
        }
        block += L::kPageBytes;
        k = k_next;
        v = v_next;
    }
}

// The 8 values of two words of codes (dims 4 i .. 4 i + 3 in word half i).
template <typename T>
__device__ __forceinline__ uint4 dequantise8(uint32_t codes, uint32_t s16, uint32_t z16) {
    using Q = Q4Type<T>;
    const uint32_t s2 = s16 * 0x10001u, z2 = z16 * 0x10001u;
    // The pair at bits 4 P of both halves is dims (P, P + 4).
    const uint32_t y0 = Q::fma2(s2, Q::template code16<0>(codes), z2);
    const uint32_t y1 = Q::fma2(s2, Q::template code16<1>(codes), z2);
    const uint32_t y2 = Q::fma2(s2, Q::template code16<2>(codes), z2);
    const uint32_t y3 = Q::fma2(s2, Q::template code16<3>(codes), z2);
    return make_uint4(__byte_perm(y0, y1, 0x5410), __byte_perm(y2, y3, 0x5410),
                      __byte_perm(y0, y1, 0x7632), __byte_perm(y2, y3, 0x7632));
}

template <int D, typename T>
__global__ void __launch_bounds__(kQ4Threads) q4_read_kernel(const Q4CacheParams p) {
    using L = Q4Layout<D>;
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    const Q4Lane<D> ln(p);
    if (ln.tok >= p.n) return;
    const bool keep = ln.slot >= 0;
    const int h0 = blockIdx.y * p.heads, h1 = min(p.Hkv, h0 + p.heads);
    unsigned char* kr = p.k + ln.tok * p.k_stride + ((size_t)h0 * D + ln.c8) * 2;
    unsigned char* vr = p.v + ln.tok * p.v_stride + ((size_t)h0 * D + ln.c8) * 2;
    const unsigned char* block = p.cache + ln.block0 + (size_t)h0 * L::kPageBytes;
    const uint32_t fill = ln.bad ? 0x7FFFu : 0u;  // the offset of a row that is not there
    struct Cells {
        uint32_t kc, kp, v0, v1, vs, vz;
    };
    auto fetch = [&](const unsigned char* b) {
        Cells c = {0, fill << 16, 0, 0, 0, fill};
        if (keep) {
            c.kc = *reinterpret_cast<const uint32_t*>(b + ln.k_codes);
            c.kp = *reinterpret_cast<const uint32_t*>(b + ln.k_par);
            c.v0 = *reinterpret_cast<const uint16_t*>(b + ln.v_codes0);
            c.v1 = *reinterpret_cast<const uint16_t*>(b + ln.v_codes1);
            c.vs = *reinterpret_cast<const uint16_t*>(b + ln.v_par);
            c.vz = *reinterpret_cast<const uint16_t*>(b + ln.v_par + 4);
        }
        return c;
    };
    Cells c = fetch(block);
    for (int h = h0; h < h1; ++h) {
        Cells next = c;
        if (h + 1 < h1) next = fetch(block += L::kPageBytes);
        *reinterpret_cast<uint4*>(kr) = dequantise8<T>(c.kc, c.kp & 0xffffu, c.kp >> 16);
        *reinterpret_cast<uint4*>(vr) = dequantise8<T>(c.v0 | (c.v1 << 16), c.vs, c.vz);
        kr += 2 * D;
        vr += 2 * D;
        c = next;
    }
}

template <typename T>
static cudaError_t launch_q4_cache(bool write, int D, const Q4CacheParams& p, cudaStream_t stream) {
    const long long lanes = (long long)p.n * (D / 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((lanes + kQ4Threads - 1) / kQ4Threads),
                       (p.Hkv + p.heads - 1) / p.heads);
    cfg.blockDim = dim3(kQ4Threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (D) {
        case 64:
            return write ? cudaLaunchKernelEx(&cfg, q4_write_kernel<64, T>, p)
                         : cudaLaunchKernelEx(&cfg, q4_read_kernel<64, T>, p);
        case 96:
            return write ? cudaLaunchKernelEx(&cfg, q4_write_kernel<96, T>, p)
                         : cudaLaunchKernelEx(&cfg, q4_read_kernel<96, T>, p);
        case 128:
            return write ? cudaLaunchKernelEx(&cfg, q4_write_kernel<128, T>, p)
                         : cudaLaunchKernelEx(&cfg, q4_read_kernel<128, T>, p);
        default:
            return write ? cudaLaunchKernelEx(&cfg, q4_write_kernel<256, T>, p)
                         : cudaLaunchKernelEx(&cfg, q4_read_kernel<256, T>, p);
    }
}

static int q4_cache_call(bool write, int num_tokens, int num_kv_heads, int head_dim,
                         int page_size, int num_pages, int dtype, void* k, long long k_stride,
                         void* v, long long v_stride, const int64_t* slots, void* cache,
                         uint32_t* device_error, void* stream) {
    if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 || num_pages <= 0)
        return PA_ERR_INVALID_ARG;
    if (dtype != PA_DTYPE_F16 && dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_F32)
        return PA_ERR_INVALID_ARG;
    if (dtype == PA_DTYPE_F32 || !q4_head_dim_ok(head_dim) || page_size != kPageSize ||
        num_kv_heads > 32767)
        return PA_ERR_UNSUPPORTED;
    const long long row = (long long)num_kv_heads * head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        k_stride > (1ll << 40) || v_stride > (1ll << 40))
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!k || !v || !slots || !cache) return PA_ERR_INVALID_ARG;
    if (!write && k == v) return PA_ERR_INVALID_ARG;  // (two outputs)
    if (((uintptr_t)k & 15u) || ((uintptr_t)v & 15u) || ((uintptr_t)cache & 15u) ||
        ((uintptr_t)slots & 7u) || ((uintptr_t)device_error & 3u))
        return PA_ERR_INVALID_ARG;
    Q4CacheParams p;
    p.slots = slots;
    p.cache = static_cast<unsigned char*>(cache);
    p.k = static_cast<unsigned char*>(k);
    p.v = static_cast<unsigned char*>(v);
    p.k_stride = k_stride * 2;
    p.v_stride = v_stride * 2;
    p.err = device_error;
    p.n = num_tokens;
    p.Hkv = num_kv_heads;
    p.num_slots = (long long)num_pages * kPageSize;
    // As many heads in one thread as leave 608 CTAs (four for each of GB300's 152
    // SMs): what is worked out once per token is then shared, and short inputs still
    // spread out.
    // 16384 rows of 4 heads at D 256, written and read: 4 heads a thread 45.4
    // us, 2 heads 49.1, 1 head 61.7.
    const long long ctas = ((long long)num_tokens * (head_dim / 8) + kQ4Threads - 1) / kQ4Threads;
    p.heads = (int)std::max(1ll, std::min<long long>(num_kv_heads, ctas * num_kv_heads / 608));
    const cudaError_t e =
        dtype == PA_DTYPE_BF16
            ? launch_q4_cache<__nv_bfloat16>(write, head_dim, p, static_cast<cudaStream_t>(stream))
            : launch_q4_cache<__half>(write, head_dim, p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return PA_OK;
}

}  // namespace pa

extern "C" {

int pa_q4_page_bytes(int head_dim) { return pa::q4_head_dim_ok(head_dim) ? 20 * head_dim : 0; }

int pa_q4_write(int num_tokens, int num_kv_heads, int head_dim, int page_size, int num_pages,
                int dtype, const void* k, long long k_stride, const void* v, long long v_stride,
                const int64_t* slots, void* cache, uint32_t* device_error, void* stream) {
    return pa::q4_cache_call(true, num_tokens, num_kv_heads, head_dim, page_size, num_pages, dtype,
                             const_cast<void*>(k), k_stride, const_cast<void*>(v), v_stride, slots,
                             cache, device_error, stream);
}

int pa_q4_read(int num_tokens, int num_kv_heads, int head_dim, int page_size, int num_pages,
               int dtype, const void* cache, const int64_t* slots, void* k, long long k_stride,
               void* v, long long v_stride, uint32_t* device_error, void* stream) {
    return pa::q4_cache_call(false, num_tokens, num_kv_heads, head_dim, page_size, num_pages, dtype,
                             k, k_stride, v, v_stride, slots, const_cast<void*>(cache),
                             device_error, stream);
}

}  // extern "C"
