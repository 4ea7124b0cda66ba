// pa_q4_cache.cu -- rows of K and V into the 4-bit paged cache and back
// (pa_q4_write, pa_q4_read of include/pa_q4.h).
//
// Both kernels are bound by memory: a row of D elements is read (2 D bytes)
// and leaves as 0.625 D bytes of codes and parameters, or the reverse.  A
// thread has 8 consecutive dims (16 bytes) of a row, so the four lanes of an
// aligned quad hold a group of 32 dims, and D / 8 consecutive lanes a row.
// blockIdx.y is K or V of a KV head; along x the rows follow each other.
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
    long long num_slots;   // num_pages * 16
};

// Quantise the 8 elements of a lane (the quad's 32 form the group).  The
// codes, scale and offset are those of exact arithmetic: where an fp32
// result lies close to a rounding border the step is repeated in fp64.
template <typename T>
__device__ __forceinline__ void quantise8(const uint32_t (&x)[4], uint32_t (&code)[2], uint32_t& s16,
                                          uint32_t& z16) {
    using Q = Q4Type<T>;
    // (max, -min) of the quad as one packed pair, NaN kept.
    constexpr uint32_t kSign = 0x80008000u;
    uint32_t hi = Q::max2_nan(Q::max2_nan(x[0], x[1]), Q::max2_nan(x[2], x[3]));
    uint32_t lo = Q::max2_nan(Q::max2_nan(x[0] ^ kSign, x[1] ^ kSign),
                              Q::max2_nan(x[2] ^ kSign, x[3] ^ kSign));
    uint32_t ext = Q::max2_nan(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
    ext = Q::max2_nan(ext, __shfl_xor_sync(0xffffffffu, ext, 1));
    ext = Q::max2_nan(ext, __shfl_xor_sync(0xffffffffu, ext, 2));
    float mx = Q::to_float(ext & 0xffffu);
    float mn = -Q::to_float(ext >> 16);
    if (mx != mx || mn != mn) {
        s16 = 0;
        z16 = 0x7FFFu;  // NaN in fp16 and bf16
        code[0] = code[1] = 0;
        return;
    }
    mx = fminf(fmaxf(mx, -Q::kLimit), Q::kLimit);
    mn = fminf(fmaxf(mn, -Q::kLimit), Q::kLimit);
    const float qs = __fdiv_rn(mx - mn, 15.f);
    s16 = Q::near_tie(qs) ? Q::from_double(((double)mx - (double)mn) / 15.0) : Q::from_float(qs);
    // z = RN_T(mn - 16 s): mn is a value of T, so this is one fma of T.
    z16 = Q::fma2(Q::from_float(-16.f), s16, Q::from_float(mn)) & 0xffffu;
    const float s = Q::to_float(s16), z = Q::to_float(z16);
    code[0] = code[1] = 0;
    if (s16 == 0) return;
    const float inv = __frcp_rn(s);
    // (1 / s overflows for the smallest bf16 scales: those go by fp64)
    const bool tiny = s < 1e-37f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float xv = Q::to_float(i & 1 ? x[i / 2] >> 16 : x[i / 2] & 0xffffu);
        // u = 16 + c before rounding; its error is below 2^-17 for u <= 32
        // (the subtraction, 1 / s and the product: 3 * 2^-24 * 32).
        const float u = (xv - z) * inv;
        float r = rintf(u);
        if (tiny || fabsf(fabsf(u - r) - 0.5f) < 1.52587890625e-05f)
            r = (float)rint(((double)xv - (double)z) / (double)s);
        const float c = fminf(fmaxf(r - 16.f, 0.f), 15.f);
        code[i / 4] |= (uint32_t)(int)c << (4 * (i % 4));
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kQ4Threads) q4_write_kernel(const Q4CacheParams p) {
    using L = Q4Layout<D>;
    constexpr int LPR = D / 8;  // lanes per row
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    const int head = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const long long idx = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
    const long long tok = idx / LPR;
    const int c8 = (int)(idx % LPR) * 8;
    long long slot = -1;
    uint32_t x[4] = {0, 0, 0, 0};
    if (tok < p.n) {
        slot = p.slots[tok];
        const unsigned char* row =
            (is_v ? p.v + tok * p.v_stride : p.k + tok * p.k_stride) + ((size_t)head * D + c8) * 2;
        const uint4 raw = *reinterpret_cast<const uint4*>(row);
        x[0] = raw.x, x[1] = raw.y, x[2] = raw.z, x[3] = raw.w;
    }
    uint32_t code[2], s16, z16;
    quantise8<T>(x, code, s16, z16);  // (every lane takes part in the quad's shuffles)
    if (slot < 0 || slot >= p.num_slots) {
        if (p.err && slot != -1 && blockIdx.y == 0 && c8 == 0) atomicOr(p.err, PA_DEVERR_BAD_SLOT);
        return;
    }
    unsigned char* block =
        p.cache + ((size_t)(slot / kPageSize) * p.Hkv + head) * (size_t)L::kPageBytes;
    const int r = (int)(slot % kPageSize);
    if (!is_v) {
        *reinterpret_cast<uint32_t*>(block + L::k_codes(r, c8)) = code[0] | (code[1] << 16);
        if ((c8 & (kQ4Group - 1)) == 0)
            *reinterpret_cast<uint32_t*>(block + L::k_params(r, c8 / kQ4Group)) = s16 | (z16 << 16);
    } else {
        *reinterpret_cast<uint16_t*>(block + L::v_codes(r, c8)) = (uint16_t)code[0];
        *reinterpret_cast<uint16_t*>(block + L::v_codes(r, c8 + 4)) = (uint16_t)code[1];
        if ((c8 & (kQ4Group - 1)) == 0) {
            unsigned char* cell = block + L::v_params(r, c8 / kQ4Group);
            *reinterpret_cast<uint16_t*>(cell) = (uint16_t)s16;
            *reinterpret_cast<uint16_t*>(cell + 4) = (uint16_t)z16;
        }
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kQ4Threads) q4_read_kernel(const Q4CacheParams p) {
    using L = Q4Layout<D>;
    using Q = Q4Type<T>;
    constexpr int LPR = D / 8;
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    const int head = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const long long idx = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
    const long long tok = idx / LPR;
    const int c8 = (int)(idx % LPR) * 8;
    if (tok >= p.n) return;
    const long long slot = p.slots[tok];
    uint32_t codes = 0, s16 = 0, z16 = 0;
    if (slot >= 0 && slot < p.num_slots) {
        const unsigned char* block =
            p.cache + ((size_t)(slot / kPageSize) * p.Hkv + head) * (size_t)L::kPageBytes;
        const int r = (int)(slot % kPageSize);
        if (!is_v) {
            codes = *reinterpret_cast<const uint32_t*>(block + L::k_codes(r, c8));
            const uint32_t sz =
                *reinterpret_cast<const uint32_t*>(block + L::k_params(r, c8 / kQ4Group));
            s16 = sz & 0xffffu;
            z16 = sz >> 16;
        } else {
            codes = *reinterpret_cast<const uint16_t*>(block + L::v_codes(r, c8)) |
                    ((uint32_t) * reinterpret_cast<const uint16_t*>(block + L::v_codes(r, c8 + 4))
                     << 16);
            const unsigned char* cell = block + L::v_params(r, c8 / kQ4Group);
            s16 = *reinterpret_cast<const uint16_t*>(cell);
            z16 = *reinterpret_cast<const uint16_t*>(cell + 4);
        }
    } else if (slot != -1) {
        z16 = 0x7FFFu;
        if (p.err && blockIdx.y == 0 && c8 == 0) atomicOr(p.err, PA_DEVERR_BAD_SLOT);
    }
    const uint32_t s2 = s16 * 0x10001u, z2 = z16 * 0x10001u;
    // The pair at bits 4 P of both halves is dims (P, P + 4).
    const uint32_t y0 = Q::fma2(s2, Q::template code16<0>(codes), z2);
    const uint32_t y1 = Q::fma2(s2, Q::template code16<1>(codes), z2);
    const uint32_t y2 = Q::fma2(s2, Q::template code16<2>(codes), z2);
    const uint32_t y3 = Q::fma2(s2, Q::template code16<3>(codes), z2);
    uint4 o;
    o.x = __byte_perm(y0, y1, 0x5410);
    o.y = __byte_perm(y2, y3, 0x5410);
    o.z = __byte_perm(y0, y1, 0x7632);
    o.w = __byte_perm(y2, y3, 0x7632);
    unsigned char* row =
        (is_v ? p.v + tok * p.v_stride : p.k + tok * p.k_stride) + ((size_t)head * D + c8) * 2;
    *reinterpret_cast<uint4*>(row) = o;
}

template <typename T>
static cudaError_t launch_q4_cache(bool write, int D, const Q4CacheParams& p, cudaStream_t stream) {
    const long long lanes = (long long)p.n * (D / 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((lanes + kQ4Threads - 1) / kQ4Threads), 2 * p.Hkv);
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
