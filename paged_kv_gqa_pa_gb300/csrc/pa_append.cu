// pa_append.cu -- new rows of q, K and V normalised, rotated and appended to the
// paged cache, of 16 or 32 bits (pa_append) or of 8 (pa_q8_append), and rows of the
// 8-bit cache read back (pa_q8_read); include/pa_q8.h.
//
// A lane has two runs of 16 bytes of a head's row whose elements are rotation
// partners (i and i + R / 2), or that lie side by side behind dim R; the lanes of a
// row, a power of two of them, sum its squares by shuffles.  Everything between
// load and store stays in registers.
#include <float.h>

#include <algorithm>
#include <cstring>

#include "../../include/pa_q8.h"
#include "pa_common.cuh"
#include "pa_rope.cuh"

namespace pa {

constexpr int kAppendThreads = 256;  // at most, of pa_append
constexpr int kAppendItems = 2;      // items a thread requests before it waits for the angles
constexpr int kAppendCtas = 608;     // CTAs that fill the GPU: four for each of 152 SMs

struct AppendParams {
    const unsigned char *q, *k, *v;
    const unsigned char *q_norm, *k_norm;  // null: not normalised
    unsigned char *q_out, *k_cache, *v_cache;
    float *k_scales, *v_scales;  // 8-bit cache
    long long q_stride, k_stride, v_stride, q_out_stride;  // bytes
    const int* positions;
    const int64_t* slots;
    unsigned* err;
    int n, Hq, Hkv;
    int R;                 // 0: not rotated
    long long num_slots;   // num_pages * 16
    float eps;
    // 8-bit cache: CTAs in front that serve runs of rows, rows of such a CTA's tile, KV
    // heads that it goes through and groups of them
    int kv_ctas, tile, heads, groups;
    unsigned long long freq[kMaxRopePairs];
};

// Rows of D elements of T: lanes and what each has.
template <int D, typename T>
struct RowLanes {
    using E = RopeElem<T>;
    static constexpr int N = E::kN;          // elements of 16 bytes
    static constexpr int ES = 16 / N;
    static constexpr int kHave = D / (2 * N);  // lanes that have elements
    static constexpr int kLanes = kHave <= 4 ? 4 : kHave <= 8 ? 8 : kHave <= 16 ? 16 : 32;
    // First dims of lane c's two runs.
    __device__ static __forceinline__ int first(int c, int R) {
        const int turn = R / (2 * N);
        return c < turn ? c * N : R + (c - turn) * 2 * N;
    }
    __device__ static __forceinline__ int second(int c, int R) {
        const int turn = R / (2 * N);
        return c < turn ? c * N + R / 2 : R + (c - turn) * 2 * N + N;
    }
    // x, y times w / sqrt(mean square + eps), w the weights as fp32 in shared memory; every
    // lane of the warp takes part.
    __device__ static __forceinline__ void normalise(float (&x)[N], float (&y)[N], const float* w,
                                                     int d0, int d1, bool has, float eps) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) sum = fmaf(x[j], x[j], fmaf(y[j], y[j], sum));
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const float f = rsqrtf(sum * (1.f / D) + eps);
        if (!has) return;
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const float4 a = *reinterpret_cast<const float4*>(w + d0 + j);
            const float4 b = *reinterpret_cast<const float4*>(w + d1 + j);
            x[j] *= f * a.x, x[j + 1] *= f * a.y, x[j + 2] *= f * a.z, x[j + 3] *= f * a.w;
            y[j] *= f * b.x, y[j + 1] *= f * b.y, y[j + 2] *= f * b.z, y[j + 3] *= f * b.w;
        }
    }
    // Norm weights into shared memory (the caller's barrier follows).
    __device__ static __forceinline__ void stage(const unsigned char* w, float* to) {
        if (!w) return;
        for (int i = threadIdx.x; i < D / N; i += blockDim.x) {
            float f[N];
            E::load(__ldg(reinterpret_cast<const uint4*>(w) + i), f);
#pragma unroll
            for (int j = 0; j < N; ++j) to[i * N + j] = f[j];
        }
    }
};

// The slot of token t, -1 where its K and V are left out; reported by `tell`.
__device__ __forceinline__ long long append_slot(const AppendParams& p, long long t, bool tell) {
    const long long s = p.slots[t];
    const bool bad = s < -1 || s >= p.num_slots;
    if (bad && tell && p.err) atomicOr(p.err, PA_DEVERR_BAD_SLOT);
    return bad ? -1 : s;
}

// What a CTA of a token has in shared memory.
template <int D>
struct AppendShared {
    alignas(16) float cos[kMaxRopePairs];
    alignas(16) float sin[kMaxRopePairs];
    alignas(16) float w[2][D];  // norm weights of q and k
};

// The q heads of token t, or all its heads (ALL: q's, K's, then V's, into the cache too).
template <int D, typename T, bool ALL>
__device__ __forceinline__ void append_token(const AppendParams& p, long long t,
                                             AppendShared<D>& sh) {
    using Rw = RowLanes<D, T>;
    using E = RopeElem<T>;
    constexpr int N = Rw::N, ES = Rw::ES, L = Rw::kLanes;
    const int tid = threadIdx.x, nt = blockDim.x;
    const int n_rows = p.Hq + (ALL ? 2 * p.Hkv : 0);
    const int items = n_rows * L;
    const int c = tid % L;  // (blockDim is a multiple of 32)
    const bool has_lane = c < Rw::kHave;
    const int d0 = Rw::first(c, p.R), d1 = Rw::second(c, p.R);
    const bool turn = c < p.R / (2 * N);
    const long long slot = ALL ? append_slot(p, t, tid == 0) : -1;
    for (int i0 = 0; i0 < items; i0 += kAppendItems * nt) {
        uint4 a[kAppendItems], b[kAppendItems];
#pragma unroll
        for (int u = 0; u < kAppendItems; ++u) {
            const int h = (i0 + u * nt + tid) / L;
            a[u] = b[u] = make_uint4(0, 0, 0, 0);
            if (has_lane && h < n_rows) {  // (rows that are left out too: nobody waits for the slot)
                const unsigned char* src =
                    h < p.Hq ? p.q + t * p.q_stride + (size_t)h * D * ES
                    : h < p.Hq + p.Hkv
                        ? p.k + t * p.k_stride + (size_t)(h - p.Hq) * D * ES
                        : p.v + t * p.v_stride + (size_t)(h - p.Hq - p.Hkv) * D * ES;
                a[u] = *reinterpret_cast<const uint4*>(src + d0 * ES);
                b[u] = *reinterpret_cast<const uint4*>(src + d1 * ES);
            }
        }
        if (i0 == 0) {  // (while the rows are on their way)
            Rw::stage(p.q_norm, sh.w[0]);
            if (ALL) Rw::stage(p.k_norm, sh.w[1]);
            if (p.R > 0) {
                const int pos = p.positions[t];
                for (int i = tid; i < p.R / 2; i += nt)
                    rope_angle(pos, p.freq[i], sh.cos[i], sh.sin[i]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kAppendItems; ++u) {
            const int h = (i0 + u * nt + tid) / L;
            const bool is_q = !ALL || h < p.Hq, is_v = ALL && h >= p.Hq + p.Hkv;
            const bool has = has_lane && h < n_rows && (is_q || slot >= 0);
            float x[N], y[N];
            E::load(a[u], x);
            E::load(b[u], y);
            // (rows of one warp may be q's and k's: the shuffles are for all of them)
            if (p.q_norm || (ALL && p.k_norm))
                Rw::normalise(x, y, sh.w[is_q ? 0 : 1], d0, d1,
                              has && !is_v && (is_q ? p.q_norm : p.k_norm), p.eps);
            if (!has) continue;
            if (turn && !is_v) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float cs = sh.cos[c * N + j], sn = sh.sin[c * N + j];
                    const float xr = fmaf(x[j], cs, -(y[j] * sn));
                    y[j] = fmaf(y[j], cs, x[j] * sn);
                    x[j] = xr;
                }
            }
            unsigned char* dst;
            if (is_q) {
                dst = p.q_out + t * p.q_out_stride + (size_t)h * D * ES;
            } else {
                const size_t block = (size_t)(slot / kPageSize) * p.Hkv +
                                     (is_v ? h - p.Hq - p.Hkv : h - p.Hq);
                dst = (is_v ? p.v_cache : p.k_cache) +
                      (block * kPageSize + (int)(slot % kPageSize)) * (size_t)(D * ES);
            }
            *reinterpret_cast<uint4*>(dst + d0 * ES) = is_v ? a[u] : E::store(x);
            *reinterpret_cast<uint4*>(dst + d1 * ES) = is_v ? b[u] : E::store(y);
        }
    }
}

// A CTA for each token.
template <int D, typename T>
__global__ void __launch_bounds__(kAppendThreads, 5) append_kernel(const AppendParams p) {
    __shared__ AppendShared<D> sh;
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    append_token<D, T, true>(p, blockIdx.x, sh);
}

// ---- The 8-bit cache.

// Codes of N values times f (non-finite ones become NaN), first one lowest.
template <int N>
__device__ __forceinline__ void q8_codes(const float (&x)[N], float f, uint32_t (&c)[N / 4]) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fabsf(x[j + i]) <= FLT_MAX ? x[j + i] * f : NAN;
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
        c[j / 4] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
}

// The values of four codes.
__device__ __forceinline__ void q8_values(uint32_t c, float (&v)[4]) {
    uint32_t lo, hi;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
        " cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// The least 2^e, e >= -120, with amax <= 448 * 2^e = 1.75 * 2^(e + 8); amax finite.
__device__ __forceinline__ float q8_scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, -120) + 127) << 23);
}

template <int W>
__device__ __forceinline__ void q8_load_codes(uint32_t (&c)[W], const unsigned char* p) {
    if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        c[0] = v.x, c[1] = v.y;
    } else {
        c[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

template <int W>
__device__ __forceinline__ void q8_store_codes(unsigned char* p, const uint32_t (&c)[W]) {
    if constexpr (W == 2)
        *reinterpret_cast<uint2*>(p) = make_uint2(c[0], c[1]);
    else
        *reinterpret_cast<uint32_t*>(p) = c[0];
}

// The first kv_ctas CTAs go by (tile of rows, group of KV heads, K or V): in its tile a
// CTA finds the rows that begin a run (rows at consecutive slots of a page), and for
// each run and head every thread has its two pieces of one of the page's 16 rows: a
// new one, one that was there, or none.  The largest magnitude goes through the CTA,
// the scale follows, codes are stored.  The other CTAs serve a token's q each.
template <int D, typename T>
__global__ void __launch_bounds__(16 * (RowLanes<D, T>::kLanes), 64 / RowLanes<D, T>::kLanes)
    q8_append_kernel(const AppendParams p) {
    using Rw = RowLanes<D, T>;
    using E = RopeElem<T>;
    constexpr int N = Rw::N, ES = Rw::ES, L = Rw::kLanes, W = N / 4;
    constexpr int kWarpsHere = 16 * L / 32;
    __shared__ AppendShared<D> sh;
    __shared__ uint32_t s_max[2][kWarpsHere];
    __shared__ unsigned long long s_freq[kMaxRopePairs];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    if ((int)blockIdx.x >= p.kv_ctas) {
        append_token<D, T, false>(p, blockIdx.x - p.kv_ctas, sh);
        return;
    }
    const int is_v = blockIdx.x & 1, group = (blockIdx.x >> 1) % p.groups;
    const long long row0 = (long long)((blockIdx.x >> 1) / p.groups) * p.tile;
    const int h0 = group * p.heads, h1 = min(p.Hkv, h0 + p.heads);
    // Lane j looks at row row0 - 1 + j: runs begin at lanes 1 .. tile and have at most 16
    // rows.
    const long long at = row0 - 1 + lane;
    long long slot = -1;
    if (at >= 0 && at < p.n)
        slot = append_slot(p, at, !is_v && group == 0 && warp == 0 && lane >= 1 && lane <= p.tile);
    const long long before = __shfl_up_sync(0xffffffffu, slot, 1);
    const bool goes_on = lane > 0 && slot >= 0 && before >= 0 && slot == before + 1 &&
                         slot % kPageSize != 0;
    const uint32_t on = __ballot_sync(0xffffffffu, goes_on);
    uint32_t leads = __ballot_sync(0xffffffffu, slot >= 0 && !goes_on && lane >= 1 && lane <= p.tile);
    if (!leads) return;
    const bool rotate = !is_v && p.R > 0, norm = !is_v && p.k_norm;
    if (norm) Rw::stage(p.k_norm, sh.w[1]);
    if (rotate)
        for (int i = tid; i < p.R / 2; i += blockDim.x) s_freq[i] = p.freq[i];
    if (norm || rotate) __syncthreads();
    const unsigned char* src0 = is_v ? p.v : p.k;
    const long long stride = is_v ? p.v_stride : p.k_stride;
    unsigned char* cache = is_v ? p.v_cache : p.k_cache;
    float* scales = is_v ? p.v_scales : p.k_scales;
    const int r = tid / L, c = tid % L;
    const int d0 = Rw::first(c, p.R), d1 = Rw::second(c, p.R);
    const bool turn = rotate && c < p.R / (2 * N);
    int turn_of = 0;  // buffer of s_max
    for (; leads; leads &= leads - 1) {
        const int j = __ffs(leads) - 1;
        const uint32_t rest = j == 31 ? 0u : on >> (j + 1);
        const int cnt = __ffs(~rest);  // 1 + the rows that go on
        const long long first = __shfl_sync(0xffffffffu, slot, j);
        const int r0 = (int)(first % kPageSize);
        const size_t page = (size_t)(first / kPageSize);
        const bool have = c < Rw::kHave;
        const bool fresh = have && r >= r0 && r < r0 + cnt, kept = have && r < r0;
        const long long row = row0 - 1 + j + (r - r0);
        const unsigned char* src = src0 + row * stride + (size_t)h0 * D * ES;
        const size_t block0 = page * p.Hkv + h0;
        unsigned char* dst = cache + (block0 * kPageSize + r) * D;
        float cs[N], sn[N];
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        uint32_t ca[W] = {}, cb[W] = {};
        float old = 0.f;
        auto request = [&](int h, uint4& a_, uint4& b_, uint32_t (&ca_)[W], uint32_t (&cb_)[W],
                           float& old_) {
            const size_t step = h - h0;
            if (fresh) {
                a_ = *reinterpret_cast<const uint4*>(src + step * D * ES + d0 * ES);
                b_ = *reinterpret_cast<const uint4*>(src + step * D * ES + d1 * ES);
            }
            if (kept) {
                q8_load_codes(ca_, dst + step * (kPageSize * D) + d0);
                q8_load_codes(cb_, dst + step * (kPageSize * D) + d1);
            }
            if (r0 > 0) old_ = scales[block0 + step];
        };
        request(h0, a, b, ca, cb, old);
        if (turn && fresh) {
            const int pos = p.positions[row];
#pragma unroll
            for (int i = 0; i < N; ++i) rope_angle(pos, s_freq[c * N + i], cs[i], sn[i]);
        }
        for (int h = h0; h < h1; ++h) {
            uint4 an = a, bn = b;
            uint32_t can[W] = {}, cbn[W] = {};
            float old_n = 0.f;
            if (h + 1 < h1) request(h + 1, an, bn, can, cbn, old_n);
            float x[N], y[N];
            E::load(a, x);
            E::load(b, y);
            if (norm) Rw::normalise(x, y, sh.w[1], d0, d1, fresh, p.eps);
            if (turn && fresh) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float xr = fmaf(x[i], cs[i], -(y[i] * sn[i]));
                    y[i] = fmaf(y[i], cs[i], x[i] * sn[i]);
                    x[i] = xr;
                }
            }
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float ax = fabsf(x[i]), ay = fabsf(y[i]);
                most = fmaxf(most, fmaxf(ax <= FLT_MAX ? ax : 0.f, ay <= FLT_MAX ? ay : 0.f));
            }
            if (!fresh) most = 0.f;
            const uint32_t wmax = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
            if (lane == 0) s_max[turn_of][warp] = wmax;
            __syncthreads();
            uint32_t all = 0;
#pragma unroll
            for (int i = 0; i < kWarpsHere; ++i) all = max(all, s_max[turn_of][i]);
            turn_of ^= 1;
            if (!(old > 0.f && old <= FLT_MAX)) old = 0.f;
            const float scale = fmaxf(old, q8_scale_for(__uint_as_float(all)));
            const size_t step = h - h0;
            unsigned char* to = dst + step * (kPageSize * D);
            if (fresh) {
                const float inv = 1.f / scale;
                q8_codes(x, inv, ca);
                q8_codes(y, inv, cb);
            } else if (kept && scale != old) {
                const float ratio = old / scale;
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    float v[4];
                    uint32_t one[1];
                    q8_values(ca[i], v);
                    q8_codes(v, ratio, one);
                    ca[i] = one[0];
                    q8_values(cb[i], v);
                    q8_codes(v, ratio, one);
                    cb[i] = one[0];
                }
            }
            if (fresh || (kept && scale != old)) {
                q8_store_codes(to + d0, ca);
                q8_store_codes(to + d1, cb);
            }
            if (tid == 0 && scale != old) scales[block0 + step] = scale;
            a = an, b = bn, old = old_n;
#pragma unroll
            for (int i = 0; i < W; ++i) ca[i] = can[i], cb[i] = cbn[i];
        }
    }
}

struct Q8ReadParams {
    const unsigned char *k_cache, *v_cache;
    const float *k_scales, *v_scales;
    const int64_t* slots;
    unsigned char *k, *v;
    long long k_stride, v_stride;  // bytes
    unsigned* err;
    int n, Hkv;
    int heads;  // KV heads a thread serves (blockIdx.y: which)
    long long num_slots;
};

constexpr int kReadThreads = 256;

// A thread has 16 bytes of a row (its codes' values), goes through its KV heads, K and
// V; the next head's codes are requested before the present ones are worked on.
template <int D, typename T>
__global__ void __launch_bounds__(kReadThreads) q8_read_kernel(const Q8ReadParams p) {
    using E = RopeElem<T>;
    constexpr int N = E::kN, W = N / 4, ES = 16 / N;
    constexpr int kLanes = D / N;
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    const long long idx = (long long)blockIdx.x * kReadThreads + threadIdx.x;
    const long long tok = idx / kLanes;
    const int d = (int)(idx % kLanes) * N;
    if (tok >= p.n) return;
    long long slot = p.slots[tok];
    const bool bad = slot < -1 || slot >= p.num_slots;
    if (bad) slot = -1;
    if (bad && p.err && blockIdx.y == 0 && d == 0) atomicOr(p.err, PA_DEVERR_BAD_SLOT);
    const bool keep = slot >= 0;
    const int h0 = blockIdx.y * p.heads, h1 = min(p.Hkv, h0 + p.heads);
    size_t block = keep ? (size_t)(slot / kPageSize) * p.Hkv + h0 : 0;
    const size_t off = (size_t)(keep ? slot % kPageSize : 0) * D + d;
    unsigned char* kr = p.k + tok * p.k_stride + ((size_t)h0 * D + d) * ES;
    unsigned char* vr = p.v + tok * p.v_stride + ((size_t)h0 * D + d) * ES;
    struct Cells {
        uint32_t k[W], v[W];
        float ks, vs;
    };
    auto fetch = [&]() {
        Cells c = {};
        c.ks = c.vs = bad ? NAN : 0.f;
        if (keep) {
            q8_load_codes(c.k, p.k_cache + block * (kPageSize * D) + off);
            q8_load_codes(c.v, p.v_cache + block * (kPageSize * D) + off);
            c.ks = p.k_scales[block];
            c.vs = p.v_scales[block];
        }
        ++block;
        return c;
    };
    auto values = [&](const uint32_t (&c)[W], float s) {
        float f[N];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float v[4];
            q8_values(c[i], v);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[4 * i + j] = s * v[j];
        }
        return E::store(f);
    };
    Cells c = fetch();
    for (int h = h0; h < h1; ++h) {
        Cells next = c;
        if (h + 1 < h1) next = fetch();
        *reinterpret_cast<uint4*>(kr) = values(c.k, c.ks);
        *reinterpret_cast<uint4*>(vr) = values(c.v, c.vs);
        kr += D * ES;
        vr += D * ES;
        c = next;
    }
}

// ---- Launches and checks.

template <typename... A>
static cudaError_t launch_step(void (*kernel)(A...), dim3 grid, int threads, cudaStream_t stream,
                               const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, typename T>
static cudaError_t launch_append(const AppendParams& p, bool q8, cudaStream_t stream) {
    constexpr int L = RowLanes<D, T>::kLanes;
    if (!q8) {
        // Threads for kAppendItems items each.
        const int items = (p.Hq + 2 * p.Hkv) * L;
        const int threads = (items + kAppendItems * 32 - 1) / (kAppendItems * 32) * 32;
        return launch_step(append_kernel<D, T>, dim3(p.n), std::min(kAppendThreads, threads),
                           stream, p);
    }
    return launch_step(q8_append_kernel<D, T>, dim3(p.kv_ctas + (p.Hq > 0 ? p.n : 0)), 16 * L,
                       stream, p);
}

template <typename T>
static cudaError_t launch_append_t(int D, const AppendParams& p, bool q8, cudaStream_t stream) {
    switch (D) {
        case 64: return launch_append<64, T>(p, q8, stream);
        case 96: return launch_append<96, T>(p, q8, stream);
        case 128: return launch_append<128, T>(p, q8, stream);
        default: return launch_append<256, T>(p, q8, stream);
    }
}

template <typename T>
static cudaError_t launch_read_t(int D, const Q8ReadParams& p, dim3 grid, cudaStream_t stream) {
    switch (D) {
        case 64: return launch_step(q8_read_kernel<64, T>, grid, kReadThreads, stream, p);
        case 96: return launch_step(q8_read_kernel<96, T>, grid, kReadThreads, stream, p);
        case 128: return launch_step(q8_read_kernel<128, T>, grid, kReadThreads, stream, p);
        default: return launch_step(q8_read_kernel<256, T>, grid, kReadThreads, stream, p);
    }
}

// What the calls' sizes must satisfy.
static int check_rows(int num_tokens, int num_kv_heads, int head_dim, int page_size,
                      int num_pages, int dtype) {
    if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 || num_pages <= 0)
        return PA_ERR_INVALID_ARG;
    if (dtype != PA_DTYPE_F16 && dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_F32)
        return PA_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 256) ||
        page_size != kPageSize || num_kv_heads > 32767)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

static bool bad_stride(long long stride, long long row, int vec) {
    return stride < row || stride % vec != 0 || stride > (1ll << 40);
}

static int append_call(bool q8, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                       int rotary_dim, int page_size, int num_pages, int dtype, float theta,
                       float eps, const void* q, long long q_stride, const void* k,
                       long long k_stride, const void* v, long long v_stride, const void* q_norm,
                       const void* k_norm, const int32_t* positions, const int64_t* slots,
                       void* q_out, long long q_out_stride, void* k_cache, void* v_cache,
                       float* k_scales, float* v_scales, uint32_t* device_error, void* stream) {
    const int st = check_rows(num_tokens, num_kv_heads, head_dim, page_size, num_pages, dtype);
    if (st == PA_ERR_INVALID_ARG) return st;
    const bool rotate = theta != 0.f, norm = q_norm || k_norm, has_q = num_q_heads > 0;
    if (num_q_heads < 0 || !(theta >= 0.f) || theta == INFINITY ||
        (rotate && (rotary_dim <= 0 || rotary_dim > head_dim)) ||
        (norm && (!(eps >= 0.f) || eps == INFINITY)))
        return PA_ERR_INVALID_ARG;
    if (st != PA_OK) return st;
    if (num_q_heads > 32767 || (rotate && rotary_dim % 16 != 0)) return PA_ERR_UNSUPPORTED;
    const int es = dtype == PA_DTYPE_F32 ? 4 : 2, vec = 16 / es;
    const long long kv_row = (long long)num_kv_heads * head_dim;
    const long long q_row = (long long)num_q_heads * head_dim;
    if (bad_stride(k_stride, kv_row, vec) || bad_stride(v_stride, kv_row, vec) ||
        (has_q && (bad_stride(q_stride, q_row, vec) || bad_stride(q_out_stride, q_row, vec) ||
                   (q == q_out && q_stride != q_out_stride))))
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!k || !v || !slots || !k_cache || !v_cache || (has_q && (!q || !q_out)) ||
        (rotate && !positions) || (q8 && (!k_scales || !v_scales)))
        return PA_ERR_INVALID_ARG;
    // (two outputs, or an output that another row's input is)
    if (k_cache == v_cache || k_cache == k || k_cache == v || v_cache == k || v_cache == v ||
        (has_q && (q_out == k || q_out == v || q_out == k_cache || q_out == v_cache ||
                   q == k_cache || q == v_cache)) ||
        (q8 && k_scales == v_scales))
        return PA_ERR_INVALID_ARG;
    uintptr_t bits = (uintptr_t)k | (uintptr_t)v | (uintptr_t)k_cache | (uintptr_t)v_cache |
                     (uintptr_t)q_norm | (uintptr_t)k_norm;
    if (has_q) bits |= (uintptr_t)q | (uintptr_t)q_out;
    uintptr_t words = (uintptr_t)device_error;
    if (rotate) words |= (uintptr_t)positions;
    if (q8) words |= (uintptr_t)k_scales | (uintptr_t)v_scales;
    if ((bits & 15u) || (words & 3u) || ((uintptr_t)slots & 7u)) return PA_ERR_INVALID_ARG;
    AppendParams p = {};
    p.q = static_cast<const unsigned char*>(q);
    p.k = static_cast<const unsigned char*>(k);
    p.v = static_cast<const unsigned char*>(v);
    p.q_norm = has_q ? static_cast<const unsigned char*>(q_norm) : nullptr;
    p.k_norm = static_cast<const unsigned char*>(k_norm);
    p.q_out = static_cast<unsigned char*>(q_out);
    p.k_cache = static_cast<unsigned char*>(k_cache);
    p.v_cache = static_cast<unsigned char*>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.q_stride = q_stride * es;
    p.k_stride = k_stride * es;
    p.v_stride = v_stride * es;
    p.q_out_stride = q_out_stride * es;
    p.positions = positions;
    p.slots = slots;
    p.err = device_error;
    p.n = num_tokens;
    p.Hq = num_q_heads;
    p.Hkv = num_kv_heads;
    p.num_slots = (long long)num_pages * kPageSize;
    p.eps = eps;
    if (rotate) {
        p.R = rotary_dim;
        memcpy(p.freq, rope_frequency_table(theta, rotary_dim),
               sizeof(unsigned long long) * (rotary_dim / 2));
    }
    if (q8) {
        // Tiles of 16 rows where they fill the GPU (a prompt's tile then is a run or two,
        // and no CTA starts for nothing), else of one row; as many heads in one CTA as
        // leave kAppendCtas of them, so that angles are worked out once for several.
        const long long tiles16 = ((long long)num_tokens + 15) / 16;
        p.tile = tiles16 * 2 * num_kv_heads >= kAppendCtas ? 16 : 1;
        const long long tiles = p.tile == 16 ? tiles16 : num_tokens;
        p.heads = (int)std::max(1ll, std::min<long long>(num_kv_heads,
                                                         tiles * 2 * num_kv_heads / kAppendCtas));
        p.groups = (num_kv_heads + p.heads - 1) / p.heads;
        const long long ctas = tiles * 2 * p.groups;
        if (ctas + num_tokens > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
        p.kv_ctas = (int)ctas;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (dtype) {
        case PA_DTYPE_F32: e = launch_append_t<float>(head_dim, p, q8, s); break;
        case PA_DTYPE_BF16: e = launch_append_t<__nv_bfloat16>(head_dim, p, q8, s); break;
        default: e = launch_append_t<__half>(head_dim, p, q8, s); break;
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" {

int pa_append(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
              int page_size, int num_pages, int dtype, float theta, float eps, const void* q,
              long long q_stride, const void* k, long long k_stride, const void* v,
              long long v_stride, const void* q_norm, const void* k_norm,
              const int32_t* positions, const int64_t* slots, void* q_out,
              long long q_out_stride, void* k_cache, void* v_cache, uint32_t* device_error,
              void* stream) {
    return append_call(false, num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim,
                       page_size, num_pages, dtype, theta, eps, q, q_stride, k, k_stride, v,
                       v_stride, q_norm, k_norm, positions, slots, q_out, q_out_stride, k_cache,
                       v_cache, nullptr, nullptr, device_error, stream);
}

int pa_q8_append(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
                 int page_size, int num_pages, int dtype, float theta, float eps, const void* q,
                 long long q_stride, const void* k, long long k_stride, const void* v,
                 long long v_stride, const void* q_norm, const void* k_norm,
                 const int32_t* positions, const int64_t* slots, void* q_out,
                 long long q_out_stride, void* k_cache, void* v_cache, float* k_scales,
                 float* v_scales, uint32_t* device_error, void* stream) {
    return append_call(true, num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim,
                       page_size, num_pages, dtype, theta, eps, q, q_stride, k, k_stride, v,
                       v_stride, q_norm, k_norm, positions, slots, q_out, q_out_stride, k_cache,
                       v_cache, k_scales, v_scales, device_error, stream);
}

int pa_q8_read(int num_tokens, int num_kv_heads, int head_dim, int page_size, int num_pages,
               int dtype, const void* k_cache, const void* v_cache, const float* k_scales,
               const float* v_scales, const int64_t* slots, void* k, long long k_stride, void* v,
               long long v_stride, uint32_t* device_error, void* stream) {
    const int st = check_rows(num_tokens, num_kv_heads, head_dim, page_size, num_pages, dtype);
    if (st != PA_OK) return st;
    const int es = dtype == PA_DTYPE_F32 ? 4 : 2, vec = 16 / es;
    const long long row = (long long)num_kv_heads * head_dim;
    if (bad_stride(k_stride, row, vec) || bad_stride(v_stride, row, vec)) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!k || !v || !slots || !k_cache || !v_cache || !k_scales || !v_scales || k == v ||
        k == k_cache || k == v_cache || v == k_cache || v == v_cache)
        return PA_ERR_INVALID_ARG;
    if ((((uintptr_t)k | (uintptr_t)v | (uintptr_t)k_cache | (uintptr_t)v_cache) & 15u) ||
        (((uintptr_t)k_scales | (uintptr_t)v_scales | (uintptr_t)device_error) & 3u) ||
        ((uintptr_t)slots & 7u))
        return PA_ERR_INVALID_ARG;
    Q8ReadParams p = {};
    p.k_cache = static_cast<const unsigned char*>(k_cache);
    p.v_cache = static_cast<const unsigned char*>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.slots = slots;
    p.k = static_cast<unsigned char*>(k);
    p.v = static_cast<unsigned char*>(v);
    p.k_stride = k_stride * es;
    p.v_stride = v_stride * es;
    p.err = device_error;
    p.n = num_tokens;
    p.Hkv = num_kv_heads;
    p.num_slots = (long long)num_pages * kPageSize;
    // As many heads in one thread as leave kAppendCtas CTAs.
    const long long ctas = ((long long)num_tokens * (head_dim / vec) + kReadThreads - 1) / kReadThreads;
    p.heads = (int)std::max(1ll, std::min<long long>(num_kv_heads, ctas * num_kv_heads / kAppendCtas));
    const dim3 grid((unsigned)ctas, (num_kv_heads + p.heads - 1) / p.heads);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (dtype) {
        case PA_DTYPE_F32: e = launch_read_t<float>(head_dim, p, grid, s); break;
        case PA_DTYPE_BF16: e = launch_read_t<__nv_bfloat16>(head_dim, p, grid, s); break;
        default: e = launch_read_t<__half>(head_dim, p, grid, s); break;
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return PA_OK;
}

}  // extern "C"
