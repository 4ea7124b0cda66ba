// pa_verify.cu -- verification of drafted tokens (pa_verify_drafts of
// include/pa_q8.h).
//
// A cluster of CTAs serves a sequence.  Every CTA works out for itself where the
// drafts stop (a warp, a draft a lane), then sums the weights of its share of the
// vocabulary in whole units of 2^-44; the sums meet in distributed shared memory, and
// the CTA whose share holds the drawn token looks for it: by its warps' sums, then
// all its threads within that warp's stretch.  Sums are of whole numbers, so no order
// changes them.
//
// Bound by memory where rows are many and long: one row of the target's probabilities, and
// one of the draft's where a draft was not accepted, are read once (128 sequences of 131072 in
// fp32 26.7 us of a floor of 19); else by a fixed part of 5 to 6 us, the launch, the gather of
// the drafts' probabilities, the exchange of sums and the search (1 of 32003: 5.3 us).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/pa_q8.h"
#include "pa_common.cuh"

namespace pa {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;    // CTAs of a sequence, at most
// CTAs of 152 SMs at four each.  Up to so many have four 16-byte loads of a row in flight a
// lane; more of them two, and run seven at a time on an SM (128 sequences of 131072: 28.5
// and 26.7 us, 64: 16.0 and 16.4).
constexpr int kVerifyWave = 608;
// Up to so many run two at a time on an SM with eight loads in flight (8 sequences of 131072 8.2
// -> 6.8 us, 23 of 199880 14.8 -> 12.4, 32 of 131072 11.9 -> 10.4; 38 of 128000, 304 CTAs, whose
// clusters no longer fit at once, 10.4 -> 14.3).
constexpr int kVerifyFew = 256;
constexpr int kVerifyMaxVocab = 1 << 19;  // (sums of 2^19 weights of 1 fit 64 bits)

struct VerifyParams {
    const void* target;
    const void* draft;  // null: certain drafts
    const int* draft_tokens;
    const int* num_drafts;  // null: T each
    const float* accept_u;
    const float* sample_u;
    int* accepted;
    int* tokens;
    unsigned* err;
    int T, V;
    int cluster;
    int stretch;  // elements of a warp (a multiple of 8)
    int vec;      // 1: rows lie at multiples of 16 bytes
};

template <typename T>
__device__ __forceinline__ float verify_float(T x);
template <>
__device__ __forceinline__ float verify_float(float x) {
    return x;
}
template <>
__device__ __forceinline__ float verify_float(__half x) {
    return __half2float(x);
}
template <>
__device__ __forceinline__ float verify_float(__nv_bfloat16 x) {
    return __bfloat162float(x);
}

// A weight in units of 2^-44, to nearest, as two numbers: the multiple of 2^-21 next to
// it and what that leaves, each made an integer by adding 1.5 times the power of two
// whose unit in the last place it counts in.  Sums of the floats' bits, modulo 2^32, are
// sums of those integers and of the constants' bits.
struct VerifySum {
    static constexpr float kHigh = 6.f;        // 1.5 * 2^2: unit 2^-21
    static constexpr float kLow = 12582912.f;  // 1.5 * 2^23: unit 1
    uint32_t hi = 0, lo = 0;
    __device__ __forceinline__ void add(float w) {
        const float a = w + kHigh;
        const float rest = w - (a - kHigh);  // exact, at most 2^-22
        hi += __float_as_uint(a);
        lo += __float_as_uint(fmaf(rest, 17592186044416.f, kLow));
    }
    // Of n weights, at most 256 (so that the sums of 2^21 and 2^22 at most fit 32 bits).
    __device__ __forceinline__ unsigned long long units(int n) const {
        const int h = (int)(hi - (uint32_t)n * __float_as_uint(kHigh));
        const int l = (int)(lo - (uint32_t)n * __float_as_uint(kLow));
        return (unsigned long long)((long long)h * (1ll << 23) + l);
    }
};

__device__ __forceinline__ unsigned long long verify_warp_sum(unsigned long long x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// Rows of weights: p, less q where there is one, and none at `hole`.  (Saturating
// limits a number to [0, 1], NaN to 0.)
template <typename T, int LOADS>
struct VerifyRow {
    const T* p;
    const T* q;  // null: p itself
    int hole;    // -1: none
    __device__ __forceinline__ unsigned long long at(int i) const {
        float w = __saturatef(verify_float(p[i]));
        if (q) w = __saturatef(w - __saturatef(verify_float(q[i])));
        VerifySum s;
        s.add(i == hole ? 0.f : w);
        return s.units(1);
    }
    // This lane's share of elements lo .. hi - 1 (a hole counted like the others).
    template <bool Q>
    __device__ __forceinline__ unsigned long long sum(int lo, int hi, int lane, bool vec) const {
        VerifySum s;
        int n = 0;
        constexpr int N = 16 / sizeof(T), U = LOADS;
        int i = lo;
        if (vec) {  // (lo is a multiple of 8)
            for (; i + 32 * N * U <= hi; i += 32 * N * U) {
                uint4 a[U], b[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    a[u] = __ldcs(reinterpret_cast<const uint4*>(p + i + (u * 32 + lane) * N));
                    if (Q) b[u] = __ldcs(reinterpret_cast<const uint4*>(q + i + (u * 32 + lane) * N));
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const T* x = reinterpret_cast<const T*>(&a[u]);
                    const T* y = reinterpret_cast<const T*>(&b[u]);
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        float w = __saturatef(verify_float(x[k]));
                        if (Q) w = __saturatef(w - __saturatef(verify_float(y[k])));
                        s.add(w);
                    }
                }
                n += N * U;
            }
        }
        constexpr int M = 8;
        for (; i + 32 * M <= hi; i += 32 * M) {
            T a[M], b[M];
#pragma unroll
            for (int u = 0; u < M; ++u) {
                a[u] = p[i + u * 32 + lane];
                if (Q) b[u] = q[i + u * 32 + lane];
            }
#pragma unroll
            for (int u = 0; u < M; ++u) {
                float w = __saturatef(verify_float(a[u]));
                if (Q) w = __saturatef(w - __saturatef(verify_float(b[u])));
                s.add(w);
            }
            n += M;
        }
        for (i += lane; i < hi; i += 32) {
            float w = __saturatef(verify_float(p[i]));
            if (Q) w = __saturatef(w - __saturatef(verify_float(q[i])));
            s.add(w);
            ++n;
        }
        return s.units(n);
    }
    // Of a warp's elements lo .. hi - 1.
    __device__ __forceinline__ unsigned long long warp_sum(int lo, int hi, int lane, bool vec) const {
        unsigned long long x = q ? sum<true>(lo, hi, lane, vec) : sum<false>(lo, hi, lane, vec);
        if (lane == 0 && hole >= lo && hole < hi) {
            VerifyRow all = *this;
            all.hole = -1;
            x -= all.at(hole);
        }
        return verify_warp_sum(x);
    }
};

template <typename T, int LOADS>
__global__ void __launch_bounds__(kVerifyThreads, (LOADS > 4 ? 2 : LOADS > 2 ? 4 : 7))
    verify_kernel(const VerifyParams p) {
    __shared__ int s_stop[2];                                // j, and the draft there
    __shared__ unsigned long long s_warp[kVerifyWarps];      // sums of the warps' stretches
    __shared__ unsigned long long s_cta[2][kVerifyCluster];  // of the cluster's CTAs (by pass)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
    const int lo = min(p.V, (rank * kVerifyWarps + warp) * p.stretch);
    const int hi = min(p.V, lo + p.stretch);
    allow_dependent_launch();
    // (a peer's shared memory is written only once all CTAs of the cluster have begun)
    if (p.cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    wait_for_prerequisite_grid();

    const T* target = static_cast<const T*>(p.target) + (size_t)b * (p.T + 1) * p.V;
    const T* draft = static_cast<const T*>(p.draft);
    if (draft) draft += (size_t)b * p.T * p.V;
    const float u = p.sample_u[b];
    const int asked = p.num_drafts ? p.num_drafts[b] : p.T;
    const int n = min(max(asked, 0), p.T);
    if (warp == 0) {  // (at most 32 drafts)
        int x = -1;
        float ua = 0.f, px = 0.f, qx = 1.f;
        if (lane < p.T) {  // (before the number of drafts is there)
            x = p.draft_tokens[(size_t)b * p.T + lane];
            ua = p.accept_u[(size_t)b * p.T + lane];
        }
        const bool known = x >= 0 && x < p.V;
        if (lane < p.T && known) {
            px = __saturatef(verify_float(target[(size_t)lane * p.V + x]));
            if (draft) qx = __saturatef(verify_float(draft[(size_t)lane * p.V + x]));
        }
        const bool ok = lane < n && known && (double)ua * (double)qx < (double)px;
        const unsigned no = __ballot_sync(0xffffffffu, !ok);
        const int j = no ? min(n, __ffs(no) - 1) : n;
        const int xj = __shfl_sync(0xffffffffu, x, j & 31);
        if (lane == 0) {
            s_stop[0] = j;
            s_stop[1] = j < n ? xj : -1;
        }
        if (rank == 0) {
            // (a draft behind the first that is not accepted is not looked at)
            if (p.err && (n != asked || (lane == j && lane < n && !known)))
                atomicOr(p.err, PA_DEVERR_BAD_TOKEN);
            for (int i = lane; i <= p.T; i += 32)
                if (i != j) p.tokens[(size_t)b * (p.T + 1) + i] = i < j ? x : -1;  // (i < j: lane i)
            if (lane == 0) p.accepted[b] = j;
        }
    }
    __syncthreads();
    const int j = s_stop[0];
    VerifyRow<T, LOADS> row;
    row.p = target + (size_t)j * p.V;
    row.q = j < n && draft ? draft + (size_t)j * p.V : nullptr;
    row.hole = j < n && !draft ? s_stop[1] : -1;

    // A second pass only where the first has found no weight: then p itself.
    unsigned long long total = 0, mine = 0, front = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2 && total == 0; ++pass) {
        if (pass == 1) {
            if (!row.q && row.hole < 0) break;
            row.q = nullptr;
            row.hole = -1;
        }
        const unsigned long long sum = row.warp_sum(lo, hi, lane, p.vec != 0);
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        mine = 0;
#pragma unroll
        for (int w = 0; w < kVerifyWarps; ++w) mine += s_warp[w];
        if (p.cluster > 1) {
            if (pass == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
            if (tid < p.cluster) {
                uint32_t at;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(at)
                             : "r"(smem_u32(&s_cta[pass][rank])), "r"(tid));
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(mine) : "memory");
            }
            asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                         "barrier.cluster.wait.acquire.aligned;" ::: "memory");
            total = front = 0;
            for (int i = 0; i < p.cluster; ++i) {
                const unsigned long long c = s_cta[pass][i];
                total += c;
                if (i < rank) front += c;
            }
        } else {
            total = mine;
            __syncthreads();  // (s_warp is written again in a second pass)
        }
    }
    int* out = p.tokens + (size_t)b * (p.T + 1) + j;
    if (total == 0) {
        if (rank == 0 && tid == 0) {
            *out = -1;
            if (p.err) atomicOr(p.err, PA_DEVERR_BAD_TOKEN);
        }
        return;
    }
    unsigned long long at = 0;
    if (u > 0.f) {
        const double x = floor((double)u * (double)total);
        at = x < (double)total ? min((unsigned long long)x, total - 1) : total - 1;
    }
    if (at < front || at >= front + mine) return;
    at -= front;
    // The warp's stretch that holds it, then its elements, a run of them a thread.
    int w = 0;
    while (at >= s_warp[w]) at -= s_warp[w++];
    const int w0 = min(p.V, (rank * kVerifyWarps + w) * p.stretch);
    const int w1 = min(p.V, w0 + p.stretch);
    const int each = (w1 - w0 + kVerifyThreads - 1) / kVerifyThreads;
    const int e0 = min(w1, w0 + tid * each), e1 = min(w1, e0 + each);
    unsigned long long own = 0;
    for (int e = e0; e < e1; ++e) own += row.at(e);
    unsigned long long inc = own;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m) inc += o;
    }
    __syncthreads();  // (s_warp has been read)
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    for (int i = 0; i < warp; ++i) inc += s_warp[i];
    if (at < inc && at >= inc - own) {
        at -= inc - own;
        int e = e0;
        for (unsigned long long x; at >= (x = row.at(e)); ++e) at -= x;
        *out = e;
    }
}

template <typename T>
static cudaError_t launch_verify(const VerifyParams& p, int batch, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(batch * p.cluster));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    if (batch * p.cluster <= kVerifyFew) return cudaLaunchKernelEx(&cfg, verify_kernel<T, 8>, p);
    return batch * p.cluster <= kVerifyWave ? cudaLaunchKernelEx(&cfg, verify_kernel<T, 4>, p)
                                            : cudaLaunchKernelEx(&cfg, verify_kernel<T, 2>, p);
}

}  // namespace pa

using namespace pa;

extern "C" int pa_verify_drafts(int batch, int max_drafts, int vocab, int dtype,
                                const void* target_probs, const void* draft_probs,
                                const int32_t* draft_tokens, const int32_t* num_drafts,
                                const float* accept_u, const float* sample_u, int32_t* accepted,
                                int32_t* tokens, uint32_t* device_error, void* stream) {
    if (batch < 0 || max_drafts < 0 || vocab <= 0) return PA_ERR_INVALID_ARG;
    if (dtype != PA_DTYPE_F16 && dtype != PA_DTYPE_BF16 && dtype != PA_DTYPE_F32)
        return PA_ERR_INVALID_ARG;
    if (max_drafts > PA_VERIFY_MAX_DRAFTS || vocab > kVerifyMaxVocab || batch > (1 << 24))
        return PA_ERR_UNSUPPORTED;
    if (batch == 0) return PA_OK;
    if (!target_probs || !sample_u || !accepted || !tokens ||
        (max_drafts > 0 && (!draft_tokens || !accept_u)))
        return PA_ERR_INVALID_ARG;
    const int es = dtype == PA_DTYPE_F32 ? 4 : 2;
    uintptr_t words = (uintptr_t)sample_u | (uintptr_t)accepted | (uintptr_t)tokens |
                      (uintptr_t)num_drafts | (uintptr_t)device_error;
    if (max_drafts > 0) words |= (uintptr_t)draft_tokens | (uintptr_t)accept_u;
    if ((words & 3u) || (((uintptr_t)target_probs | (uintptr_t)draft_probs) & (es - 1u)))
        return PA_ERR_INVALID_ARG;
    if (accepted == tokens || accepted == num_drafts || accepted == draft_tokens ||
        tokens == num_drafts || tokens == draft_tokens)
        return PA_ERR_INVALID_ARG;
    VerifyParams p;
    p.target = target_probs;
    p.draft = max_drafts > 0 ? draft_probs : nullptr;
    p.draft_tokens = draft_tokens;
    p.num_drafts = num_drafts;
    p.accept_u = accept_u;
    p.sample_u = sample_u;
    p.accepted = accepted;
    p.tokens = tokens;
    p.err = device_error;
    p.T = max_drafts;
    p.V = vocab;
    p.vec = (long long)vocab * es % 16 == 0 &&
            (((uintptr_t)target_probs | (uintptr_t)draft_probs) & 15u) == 0;
    // CTAs of a sequence: with 2048 elements each at least, and no more than leave one wave
    // of CTAs where they have 16384 at most (128 sequences of 32003: by 8 CTAs each 13.7
    // us, by 4 9.8; of 131072: 28.5 and 30.0).
    p.cluster = 1;
    while (p.cluster < kVerifyCluster && vocab >= p.cluster * 2 * 2048) p.cluster *= 2;
    while (p.cluster > 1 && (long long)batch * p.cluster > kVerifyWave &&
           vocab <= p.cluster / 2 * 16384)
        p.cluster /= 2;
    const int parts = p.cluster * kVerifyWarps;
    p.stretch = ((vocab + parts - 1) / parts + 7) / 8 * 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (dtype) {
        case PA_DTYPE_F32: e = launch_verify<float>(p, batch, s); break;
        case PA_DTYPE_BF16: e = launch_verify<__nv_bfloat16>(p, batch, s); break;
        default: e = launch_verify<__half>(p, batch, s); break;
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return PA_OK;
}
