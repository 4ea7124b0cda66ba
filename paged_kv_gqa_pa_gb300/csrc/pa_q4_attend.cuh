// pa_q4_attend.cuh -- decode attention over the 4-bit paged cache
// (pa_q4_decode of include/pa_q4.h).
//
// For sequence b and the G <= 8 query heads of a KV head's chunk:
//   S^T[16 tokens x 8] = K[16 x D] Q^T, p = 2^(scale log2(e) S - m),
//   O^T[D x 8] += V^T[D x 16] P^T, out = O / sum p, lse = ln 2 (m + log2 sum p)
// page by page with a running maximum m, where K and V are the values the
// cache's codes stand for, made in registers right in front of the
// mma.sync m16n8k16 that takes them.
//
//  * What bounds it.  A page of one KV head is 20 D bytes against 64 D for
//    fp16, so memory could deliver about 38 elements per clock and SM at D 128.
//    Each pair of elements costs a shift, a logic op and a packed fma (the
//    code becomes the float 16 + c, the fma applies s and z with one
//    rounding); with the softmax and the ring that is about 2 issue slots per
//    element-pair and thread, 60-70 % of the issue rate at full memory speed.
//    So the layout spends nothing else: codes and parameters lie as the
//    mma fragments want them (no ldmatrix, no transposition, no bank
//    conflict), both halves of a register come from one fma.
//  * Copies.  K, V and parameters of a page are one block, fetched by one
//    cp.async.bulk into the warp's ring; each of the four warps streams every
//    fourth page of the CTA's range.
//  * Maximum.  m is raised, and O rescaled, only when a score exceeds it by
//    more than 2^8 (weights then stay below 2^8, far from fp16's limit); so
//    most pages need no shuffle, just one vote.
//  * Split.  The pages the batch attends, all sequences end to end, are cut
//    into equal ranges, one per CTA of the group (blockIdx.x), whatever the
//    lengths; a range may hold many short sequences or part of a long one.
//    A sequence cut by a range border leaves a partial (o, m, sum) per CTA in
//    the workspace, and the last of its CTAs to arrive merges them in order,
//    so results do not depend on which one that is.
#pragma once

#include <math.h>

#include <atomic>
#include <climits>
#include <type_traits>

#include "pa_q4.cuh"

namespace pa {

constexpr int kQ4StagedPages = 1024;  // page ids staged at a time
constexpr int kQ4MinPages = 8;        // pages of the shortest range

struct Q4AttendParams {
    const void* q;
    const unsigned char* cache;
    const int* block_tables;
    const int* context_lens;
    void* out;
    float* lse;
    float* ws_o;         // [groups][X][2][G][D] partial outputs, normalised
    float* ws_ml;        // [groups][X][2][G][2] their maximum (log2 domain) and exp-sum
    unsigned* counters;  // [groups][B] arrivals of cut sequences
    unsigned* err;
    int B, Hq, Hkv, g, num_pages, maxp, max_ctx, window;
    int nchunk, G, X;
    int stall_tx;        // test hook
    float scale_log2;
};

template <int D>
struct Q4Cfg {
    // Pages of a ring slot: two where a page is little work (what a page costs
    // beside its elements -- the wait, the vote, the request -- is then paid
    // once for two, and two chains of mma overlap), one at D 256.
    static constexpr int kPair = D == 256 ? 1 : 2;
    static constexpr int kSlotBytes = kPair * Q4Layout<D>::kPageBytes;
    static constexpr int kStages = D == 64 ? 6 : (D == 96 ? 4 : 3);
    static constexpr int kRingBytes = kWarps * kStages * kSlotBytes;
    // The warps' O meet in shared memory so many dims at a time.
    static constexpr int kRoundDims = D == 96 ? 32 : 64;
    static constexpr int kRounds = D / kRoundDims;
    static constexpr int kXStride = kRoundDims + 4;
    static constexpr int kXBytes = kWarps * kMaxHeadsPerCta * kXStride * 4;
    static constexpr int kSmemBytes = kRingBytes + kXBytes + kQ4StagedPages * 4 +
                                      kWarps * kMaxHeadsPerCta * 3 * 4 + kWarps * kStages * 8;
    static constexpr int kMinBlocks = 3;
    static_assert(kMinBlocks * (kSmemBytes + 1024 + 128) <= 228 * 1024, "CTAs per SM");
    // (the sums over the batch, B + 1 words, follow)
    static int smem(int B) { return kSmemBytes + (B + 1) * 4; }
};

// mma.sync m16n8k16, 16-bit in, fp32 accumulate; and fp32 pairs to 16 bits.
template <typename T>
struct Q4Mma;

template <>
struct Q4Mma<__half> {
    static constexpr uint32_t kOnes = 0x3C003C00u;
    static constexpr bool kSplitP = false;
    __device__ static __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
            " {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static __forceinline__ float2 unpack(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
};

template <>
struct Q4Mma<__nv_bfloat16> {
    static constexpr uint32_t kOnes = 0x3F803F80u;
    // bf16 weights would cost 8 significant bits: P goes in as two bf16, its
    // head and the rest, about 16 bits.
    static constexpr bool kSplitP = true;
    __device__ static __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
            " {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static __forceinline__ float2 unpack(uint32_t u) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
    }
};

__device__ __forceinline__ uint32_t q4_movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// N consecutive 32-bit words of shared memory in one read.
template <int N>
__device__ __forceinline__ void q4_lds(uint32_t (&r)[N], const unsigned char* p) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r[0] = v.x, r[1] = v.y;
    } else {
        r[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// Dims of word w (8 of them) of lane column t in q.K: the contraction may
// take the dims in any order as long as q follows, so a lane's words are one
// read of the token's row.
template <int D>
__device__ __forceinline__ int q4_k_dim(int t, int w) {
    if constexpr (D == 96) return 32 * w + 8 * t;
    if constexpr (D == 256) return 128 * (w / 4) + 32 * t + 8 * (w % 4);
    return (D / 4) * t + 8 * w;
}

// First of the 4 dims of word w of lane column g in P.V.
template <int D>
__device__ __forceinline__ int q4_v_dim(int g, int w) {
    return D == 96 ? 32 * w + 4 * g : (D / 8) * g + 4 * w;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, Q4Cfg<D>::kMinBlocks)
    q4_attend_kernel(const Q4AttendParams p) {
    using L = Q4Layout<D>;
    using Q = Q4Type<T>;
    using M = Q4Mma<T>;
    using Cfg = Q4Cfg<D>;
    constexpr int NS = Cfg::kStages;
    constexpr int PB = L::kPageBytes;
    constexpr int W = L::kWords;   // 32-bit words of K per lane and token, of V per token pair
    constexpr int V = L::kVec;

    extern __shared__ __align__(128) unsigned char q4_smem[];
    unsigned char* ring = q4_smem;
    float* xbuf = reinterpret_cast<float*>(ring + Cfg::kRingBytes);
    int* s_pid = reinterpret_cast<int*>(xbuf + Cfg::kXBytes / 4);
    float* s_ml = reinterpret_cast<float*>(s_pid + kQ4StagedPages);  // [warps][8][m, sum, weight sum]
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_ml + kWarps * kMaxHeadsPerCta * 3);
    int* s_base = reinterpret_cast<int*>(bars + kWarps * NS);  // pages in front of sequence b
    __shared__ int s_red[kWarps];
    __shared__ int s_last;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int G = p.G;
    const int kvh = blockIdx.y / p.nchunk;
    const int h0 = kvh * p.g + (blockIdx.y % p.nchunk) * G;
    const uint32_t bar_w = smem_u32(bars) + warp * NS * 8;
    unsigned char* ring_w = ring + warp * NS * Cfg::kSlotBytes;
    const uint32_t ring_u = smem_u32(ring_w);

    allow_dependent_launch();
    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < NS; ++s) mbar_init(bar_w + s * 8, 1);
        fence_mbar_init();
    }
    wait_for_prerequisite_grid();

    // ---- The batch's pages end to end: s_base[b] of them lie before sequence
    // b (s_base[B] in all).  A thread sums a run of sequences, a scan over the
    // CTA joins the runs.
    const int per_thread = (p.B + kThreads - 1) / kThreads;
    {
        const int b0 = min(p.B, (int)threadIdx.x * per_thread), b1 = min(p.B, b0 + per_thread);
        int sum = 0;
        for (int b = b0; b < b1; ++b) {
            const int n = balanced_seq_pages(p.context_lens[b], p.window, p.max_ctx, p.maxp);
            s_base[b] = n;
            sum += n;
        }
        int inc = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, m);
            if (lane >= m) inc += o;
        }
        if (lane == 31) s_red[warp] = inc;
        __syncthreads();
        for (int w = 0; w < warp; ++w) inc += s_red[w];
        int at = inc - sum;
        for (int b = b0; b < b1; ++b) {
            const int n = s_base[b];
            s_base[b] = at;
            at += n;
        }
        if (threadIdx.x == kThreads - 1) s_base[p.B] = inc;
        __syncthreads();
    }
    const int total = s_base[p.B];
    const int pp = max(kQ4MinPages, (total + p.X - 1) / p.X);
    const long long lo_ll = (long long)blockIdx.x * pp;
    const int lo = (int)min((long long)total, lo_ll);
    const int hi = (int)min((long long)total, lo_ll + pp);

    // ---- Sequences that attend nothing: out 0 and lse -inf, or NaN where the
    // length is out of bounds.
    T* const out = reinterpret_cast<T*>(p.out);
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (s_base[b + 1] != s_base[b]) continue;
        const bool valid = seq_span(p.context_lens[b], p.window, p.max_ctx, p.maxp, 1).valid;
        if (!valid && threadIdx.x == 0) atomicOr(p.err, PA_DEVERR_BAD_LENGTH);
        const uint32_t fill = valid ? 0u : 0x7FFF7FFFu;
        uint32_t* row = reinterpret_cast<uint32_t*>(out + ((size_t)b * p.Hq + h0) * D);
        for (int i = threadIdx.x; i < G * D / 2; i += kThreads) row[i] = fill;
        if (threadIdx.x < G)
            p.lse[(size_t)b * p.Hq + h0 + threadIdx.x] = valid ? -INFINITY : NAN;
    }
    if (lo >= hi) return;

    // Sequence of the range's first page: the last b with s_base[b] <= lo
    // (behind any empty ones that share that number).
    int b = 0;
    {
        int a = 0, z = p.B - 1;
        while (a < z) {
            const int m = (a + z + 1) >> 1;
            if (s_base[m] <= lo)
                a = m;
            else
                z = m - 1;
        }
        b = a;
    }

    // ---- Registers of a sequence: q as the mma's B operand, O^T, the sums.
    uint32_t qf[W][4];          // word w: pairs (P, P + 4) of its 8 dims, P = 0..3
    float acc[W][2][4];         // O^T: dims q4_v_dim(g, w) + 2u (rows g), + 2u + 1, heads 2t, 2t + 1
    float lacc[4];              // sums of the rounded weights (all rows alike)
    float m0, m1, l0, l1;       // running maximum (log2 domain), sums of this lane's weights
    int seq_L = 0, seq_start = 0, seq_page0 = 0;
    bool dead = false;          // a copy timed out
    bool bad = false;           // this sequence met a bad page id or a timeout

    auto begin_sequence = [&]() {
        const SeqSpan sp = seq_span(p.context_lens[b], p.window, p.max_ctx, p.maxp, 1);
        seq_L = sp.L;
        seq_start = sp.start;
        seq_page0 = sp.first_page;
        const T* qrow = reinterpret_cast<const T*>(p.q) + ((size_t)b * p.Hq + h0 + g) * D;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (g < G) x = *reinterpret_cast<const uint4*>(qrow + q4_k_dim<D>(t, w));
            qf[w][0] = __byte_perm(x.x, x.z, 0x5410);
            qf[w][1] = __byte_perm(x.x, x.z, 0x7632);
            qf[w][2] = __byte_perm(x.y, x.w, 0x5410);
            qf[w][3] = __byte_perm(x.y, x.w, 0x7632);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[w][u][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) lacc[i] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
        bad = dead;
    };

    // ---- N consecutive pages in shared memory; MASK: some of their tokens may
    // lie outside the attended range (their cells may hold anything).
    auto pages = [&](const unsigned char* blk0, int tok0, auto n_pages, auto mask) {
        constexpr int N = decltype(n_pages)::value;
        constexpr bool MASK = decltype(mask)::value;
        float s[N][4];
        // K: tokens g and g + 8 of this lane's dims.
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned char* blk = blk0 + j * PB;
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] = 0.f;
#pragma unroll
            for (int sl = 0; sl < W / V; ++sl) {  // runs of V words that one read takes
                uint32_t ka[V], kb[V];
                uint32_t pa_, pb_;  // (s, z) of the run's group
                if constexpr (D == 96) {
                    q4_lds<V>(ka, blk + g * (D / 2) + 16 * sl + 4 * t);
                    q4_lds<V>(kb, blk + (g + 8) * (D / 2) + 16 * sl + 4 * t);
                    pa_ = *reinterpret_cast<const uint32_t*>(blk + L::k_params(0, sl) + g * 12);
                    pb_ = *reinterpret_cast<const uint32_t*>(blk + L::k_params(8, sl) + g * 12);
                } else {
                    const unsigned char* row = blk + sl * (8 * L::kSlice) + lane * (4 * V);
                    q4_lds<V>(ka, row);
                    q4_lds<V>(kb, row + 8 * (L::kSlice / 2));
                    const int n = D == 64 ? t >> 1 : t;
                    const unsigned char* par =
                        blk + L::kKParams + sl * (kPageSize * 4 * L::kSliceGroups) +
                        (g * L::kSliceGroups + n) * 4;
                    pa_ = *reinterpret_cast<const uint32_t*>(par);
                    pb_ = *reinterpret_cast<const uint32_t*>(par + 8 * L::kSliceGroups * 4);
                }
                const uint32_t sa = __byte_perm(pa_, pa_, 0x1010), za = __byte_perm(pa_, pa_, 0x3232);
                const uint32_t sb = __byte_perm(pb_, pb_, 0x1010), zb = __byte_perm(pb_, pb_, 0x3232);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int w = sl * V + i;
                    M::mma(s[j], Q::fma2(sa, Q::template code16<0>(ka[i]), za),
                           Q::fma2(sb, Q::template code16<0>(kb[i]), zb),
                           Q::fma2(sa, Q::template code16<1>(ka[i]), za),
                           Q::fma2(sb, Q::template code16<1>(kb[i]), zb), qf[w][0], qf[w][1]);
                    M::mma(s[j], Q::fma2(sa, Q::template code16<2>(ka[i]), za),
                           Q::fma2(sb, Q::template code16<2>(kb[i]), zb),
                           Q::fma2(sa, Q::template code16<3>(ka[i]), za),
                           Q::fma2(sb, Q::template code16<3>(kb[i]), zb), qf[w][2], qf[w][3]);
                }
            }
        }
        // e: the scores in the log2 domain, above the running maximum.  `out`
        // marks tokens g and g + 8 that are not attended.
        const float sc = p.scale_log2;
        bool out_a = false, out_b = false;
        if constexpr (MASK) {
            static_assert(!MASK || N == 1, "masked pages go one at a time");
            const int ta = tok0 + g, tb = ta + 8;
            out_a = ta < seq_start || ta >= seq_L;
            out_b = tb < seq_start || tb >= seq_L;
        }
        float e[N][4];
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[j][i] = fmaf(s[j][i], sc, i & 1 ? -m1 : -m0);
                if (MASK && (i < 2 ? out_a : out_b)) e[j][i] = -INFINITY;
                top = fmaxf(top, e[j][i]);
            }
        if (__any_sync(0xffffffffu, top > 8.f)) {
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[j][i] = s[j][i] * sc;
                    if (MASK && (i < 2 ? out_a : out_b)) e[j][i] = -INFINITY;
                    if (i & 1)
                        x1 = fmaxf(x1, e[j][i]);
                    else
                        x0 = fmaxf(x0, e[j][i]);
                }
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, k));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, k));
            }
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
            const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - n0);
            const float f1 = m1 == -INFINITY ? 0.f : ex2(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= f0;
            l1 *= f1;
            lacc[0] *= f0;
            lacc[1] *= f1;
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    acc[w][u][0] *= f0;
                    acc[w][u][1] *= f1;
                    acc[w][u][2] *= f0;
                    acc[w][u][3] *= f1;
                }
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) e[j][i] -= i & 1 ? m1 : m0;
        }
        // Weights; P^T's fragments are S^T's, each 8 x 8 block transposed.
        uint32_t b0[N], b1[N];
        [[maybe_unused]] uint32_t r0[N], r1[N];  // the rest of a split P
#pragma unroll
        for (int j = 0; j < N; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) e[j][i] = ex2(e[j][i]);
            l0 += e[j][0] + e[j][2];
            l1 += e[j][1] + e[j][3];
            const uint32_t ha = M::pack(e[j][0], e[j][1]), hb = M::pack(e[j][2], e[j][3]);
            b0[j] = q4_movmatrix(ha);
            b1[j] = q4_movmatrix(hb);
            M::mma(lacc, M::kOnes, M::kOnes, M::kOnes, M::kOnes, b0[j], b1[j]);
            if constexpr (M::kSplitP) {
                const float2 fa = M::unpack(ha), fb = M::unpack(hb);
                r0[j] = q4_movmatrix(M::pack(e[j][0] - fa.x, e[j][1] - fa.y));
                r1[j] = q4_movmatrix(M::pack(e[j][2] - fb.x, e[j][3] - fb.y));
                M::mma(lacc, M::kOnes, M::kOnes, M::kOnes, M::kOnes, r0[j], r1[j]);
            }
        }
        // V: token pairs t and t + 4 (tokens 2t, 2t + 1, 2t + 8, 2t + 9).  A token
        // that is not attended gets scale and offset 0: 0 * NaN would be NaN.
        uint32_t keep_a = 0xffffffffu, keep_b = 0xffffffffu;
        if constexpr (MASK) {
            auto in = [&](int k) { return k >= seq_start && k < seq_L; };
            const int k0 = tok0 + 2 * t;
            keep_a = (in(k0) ? 0xffffu : 0u) | (in(k0 + 1) ? 0xffff0000u : 0u);
            keep_b = (in(k0 + 8) ? 0xffffu : 0u) | (in(k0 + 9) ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned char* blk = blk0 + j * PB;
#pragma unroll
            for (int sl = 0; sl < W / V; ++sl) {
                uint32_t va[V], vb[V], pa2[2], pb2[2];
                const unsigned char* at = blk + L::kVCodes + sl * (128 * V) + lane * (4 * V);
                q4_lds<V>(va, at);
                q4_lds<V>(vb, at + 4 * D);
                const int n = D == 96 ? sl : (D == 64 ? g >> 2 : (D == 128 ? g >> 1 : g));
                const unsigned char* par = blk + L::kVParams + (t * L::kGroups + n) * 8;
                q4_lds<2>(pa2, par);
                q4_lds<2>(pb2, par + 4 * L::kGroups * 8);
                const uint32_t sa = pa2[0] & keep_a, za = pa2[1] & keep_a;
                const uint32_t sb = pb2[0] & keep_b, zb = pb2[1] & keep_b;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int w = sl * V + i;
                    const uint32_t a00 = Q::fma2(sa, Q::template code16<0>(va[i]), za);
                    const uint32_t a01 = Q::fma2(sa, Q::template code16<1>(va[i]), za);
                    const uint32_t a02 = Q::fma2(sb, Q::template code16<0>(vb[i]), zb);
                    const uint32_t a03 = Q::fma2(sb, Q::template code16<1>(vb[i]), zb);
                    M::mma(acc[w][0], a00, a01, a02, a03, b0[j], b1[j]);
                    if constexpr (M::kSplitP) M::mma(acc[w][0], a00, a01, a02, a03, r0[j], r1[j]);
                    const uint32_t a10 = Q::fma2(sa, Q::template code16<2>(va[i]), za);
                    const uint32_t a11 = Q::fma2(sa, Q::template code16<3>(va[i]), za);
                    const uint32_t a12 = Q::fma2(sb, Q::template code16<2>(vb[i]), zb);
                    const uint32_t a13 = Q::fma2(sb, Q::template code16<3>(vb[i]), zb);
                    M::mma(acc[w][1], a10, a11, a12, a13, b0[j], b1[j]);
                    if constexpr (M::kSplitP) M::mma(acc[w][1], a10, a11, a12, a13, r0[j], r1[j]);
                }
            }
        }
    };

    // ---- The end of a sequence in this CTA: the warps' states meet in shared
    // memory; a sequence that lies in the range altogether is written, a cut
    // one leaves its partial, and the last of its CTAs merges.
    auto end_sequence = [&]() {
        const int first = s_base[b], end = s_base[b + 1];
        const bool cut = first < lo || end > hi;
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, k);
            l1 += __shfl_xor_sync(0xffffffffu, l1, k);
        }
        __syncthreads();  // the last use of xbuf and s_ml is over
        if (g == 0) {
            float* ml = s_ml + (warp * kMaxHeadsPerCta + 2 * t) * 3;
            ml[0] = m0, ml[1] = bad ? NAN : l0, ml[2] = lacc[0];
            ml[3] = m1, ml[4] = bad ? NAN : l1, ml[5] = lacc[1];
        }
        const int group = blockIdx.y;
        const size_t part =
            ((size_t)group * gridDim.x + blockIdx.x) * 2 + (max(first, lo) > lo ? 1 : 0);
#pragma unroll
        for (int rd = 0; rd < Cfg::kRounds; ++rd) {
            constexpr int RD = Cfg::kRoundDims;
            if (rd > 0) __syncthreads();
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int dim = q4_v_dim<D>(g, w) - rd * RD;
                if (Cfg::kRounds == 1 || (dim >= 0 && dim < RD)) {
                    float* x = xbuf + (warp * kMaxHeadsPerCta + 2 * t) * Cfg::kXStride + dim;
                    if (2 * t < G)
                        *reinterpret_cast<float4*>(x) =
                            make_float4(acc[w][0][0], acc[w][0][2], acc[w][1][0], acc[w][1][2]);
                    if (2 * t + 1 < G)
                        *reinterpret_cast<float4*>(x + Cfg::kXStride) =
                            make_float4(acc[w][0][1], acc[w][0][3], acc[w][1][1], acc[w][1][3]);
                }
            }
            __syncthreads();
            for (int it = threadIdx.x; it < G * (RD / 4); it += kThreads) {
                const int h = it / (RD / 4), dd = (it % (RD / 4)) * 4;
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    mx = fmaxf(mx, s_ml[(w * kMaxHeadsPerCta + h) * 3]);
                float sum = 0.f, wsum = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float* ml = s_ml + (w * kMaxHeadsPerCta + h) * 3;
                    const float4 x = *reinterpret_cast<const float4*>(
                        xbuf + (w * kMaxHeadsPerCta + h) * Cfg::kXStride + dd);
                    // (a sum of 0: this warp had no page; NaN is kept)
                    const float f = ml[1] == 0.f ? 0.f : (ml[1] != ml[1] ? NAN : ex2(ml[0] - mx));
                    sum += f * ml[1];
                    wsum += f * ml[2];
                    o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
                }
                const float inv = 1.f / wsum;
                o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
                const int dim = rd * RD + dd;
                if (!cut) {
                    const size_t bh = (size_t)b * p.Hq + h0 + h;
                    uint2 u;
                    u.x = M::pack(o.x, o.y);
                    u.y = M::pack(o.z, o.w);
                    *reinterpret_cast<uint2*>(out + bh * D + dim) = u;
                    if (dim == 0) p.lse[bh] = (mx + log2f(sum)) * 0.69314718055994531f;
                } else {
                    *reinterpret_cast<float4*>(p.ws_o + (part * G + h) * D + dim) = o;
                    if (dim == 0)
                        *reinterpret_cast<float2*>(p.ws_ml + (part * G + h) * 2) =
                            make_float2(mx, sum);
                }
            }
        }
        if (!cut) return;
        // Arrival, as in the 16-bit kernel's last-CTA merge: the barrier orders
        // the CTA's stores before thread 0's acquire-release atomic.
        const int x0 = first / pp, x1 = (end - 1) / pp;
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned* ctr = p.counters + (size_t)group * p.B + b;
            unsigned prev;
            asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                         : "=r"(prev)
                         : "l"(ctr)
                         : "memory");
            s_last = (int)prev == x1 - x0;
            if (s_last) atomicExch(ctr, 0u);  // ready for the next call
        }
        __syncthreads();
        if (!s_last) return;
        // The first of its CTAs holds the sequence in its second slot unless
        // its range begins with it; every later one in its first.
        const int slot0 = first > x0 * pp ? 1 : 0;
        auto row_of = [&](int x) {
            return ((size_t)group * gridDim.x + x) * 2 + (x == x0 ? slot0 : 0);
        };
        for (int it = threadIdx.x; it < G * (D / 4); it += kThreads) {
            const int h = it / (D / 4), dim = (it % (D / 4)) * 4;
            float mx = -INFINITY, sum = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            constexpr int U = 8;  // partials in flight
            for (int xb = x0; xb <= x1; xb += U) {
                float2 ml[U];
                float4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const size_t r = row_of(min(xb + u, x1)) * G + h;
                    ml[u] = __ldcg(reinterpret_cast<const float2*>(p.ws_ml + r * 2));
                    v[u] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + r * D + dim));
                }
                float nm = mx;
#pragma unroll
                for (int u = 0; u < U; ++u) nm = fmaxf(nm, ml[u].x);
                const float f = mx == -INFINITY ? 0.f : ex2(mx - nm);
                sum *= f;
                o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (xb + u > x1) continue;
                    const float wgt = ml[u].y != ml[u].y ? NAN : ex2(ml[u].x - nm) * ml[u].y;
                    sum += wgt;
                    o.x += wgt * v[u].x, o.y += wgt * v[u].y;
                    o.z += wgt * v[u].z, o.w += wgt * v[u].w;
                }
                mx = nm;
            }
            const float inv = 1.f / sum;
            const size_t bh = (size_t)b * p.Hq + h0 + h;
            uint2 u;
            u.x = M::pack(o.x * inv, o.y * inv);
            u.y = M::pack(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2*>(out + bh * D + dim) = u;
            if (dim == 0) p.lse[bh] = (mx + log2f(sum)) * 0.69314718055994531f;
        }
    };

    // ---- The range, kQ4StagedPages at a time.  Slots of kPair pages go to the
    // warps in turn; a warp's copies take its ring slots round.
    constexpr int NP = Cfg::kPair;
    constexpr int SB = Cfg::kSlotBytes;
    using One = std::integral_constant<int, 1>;
    using Slot = std::integral_constant<int, NP>;
    int in_slot = 0, out_slot = 0;    // ring slots of the next copy and of the next page
    uint32_t out_phase = 0;
    int pending = 0;                  // slots requested and not yet waited for
    int stall = p.stall_tx;
    begin_sequence();
    for (int c0 = lo; c0 < hi; c0 += kQ4StagedPages) {
        const int c1 = min(hi, c0 + kQ4StagedPages);
        __syncthreads();  // the previous stretch's ids have been used
        bool bad_id = false;
        for (int f = c0 + threadIdx.x; f < c1; f += kThreads) {
            int a = 0, z = p.B - 1;  // the sequence of page f
            while (a < z) {
                const int m = (a + z + 1) >> 1;
                if (s_base[m] <= f)
                    a = m;
                else
                    z = m - 1;
            }
            int first_page = 0;
            if (p.window > 0) {
                const int Lb = p.context_lens[a];
                first_page = (p.window < Lb ? Lb - p.window : 0) / kPageSize;
            }
            int id = p.block_tables[(size_t)a * p.maxp + first_page + (f - s_base[a])];
            if (id < 0 || id >= p.num_pages) {
                id = -1;
                bad_id = true;
            }
            s_pid[f - c0] = id;
        }
        if (bad_id) atomicOr(p.err, PA_DEVERR_BAD_PAGE);
        // With a bad id in the stretch its pages are looked at one by one.
        const bool careful = __syncthreads_or(bad_id);

        int ask = NP * warp;  // first page (from c0) of the next slot to request
        auto request = [&]() {
            int id = -1;
            if (lane < NP && ask + lane < c1 - c0) id = s_pid[ask + lane];
            const uint32_t n_ids = __popc(__ballot_sync(0xffffffffu, id >= 0));
            const uint32_t bar = bar_w + in_slot * 8;
            if (lane == 0) mbar_arrive_expect_tx(bar, n_ids * PB + stall);
            __syncwarp();
            if (id >= 0)
                bulk_g2s(ring_u + in_slot * SB + lane * PB,
                         p.cache + ((size_t)id * p.Hkv + kvh) * (size_t)PB, PB, bar);
            stall = 0;
            ask += NP * kWarps;
            in_slot = in_slot + 1 == NS ? 0 : in_slot + 1;
            ++pending;
        };
        if (!dead)
            for (int i = 0; i < NS && ask < c1 - c0; ++i) request();

        int f = dead ? c1 : c0 + NP * warp;  // next page of this warp
        while (true) {
            const int seg_end = min(c1, s_base[b + 1]);
            // Pages that are attended whole lie in [whole0, whole1).
            const int base = s_base[b] - seq_page0;  // page of token 0
            const int whole0 = careful ? INT_MAX : base + (seq_start + kPageSize - 1) / kPageSize;
            const int whole1 = min(seg_end, base + seq_L / kPageSize);
            while (f < seg_end) {
                const int sub = (f - c0) & (NP - 1);
                if (sub == 0) {
                    const bool ok = mbar_wait_bounded(bar_w + out_slot * 8, out_phase);
                    if (!__all_sync(0xffffffffu, ok)) {
                        if (lane == 0) atomicOr(p.err, PA_DEVERR_TIMEOUT);
                        dead = bad = true;
                        f = c1;
                        break;
                    }
                    --pending;
                }
                const unsigned char* blk = ring_w + out_slot * SB + sub * PB;
                const int tok0 = (f - base) * kPageSize;
                if (sub == 0 && f >= whole0 && f + NP <= whole1) {
                    pages(blk, tok0, Slot{}, std::false_type{});
                    f += NP;
                } else {
                    if (careful && s_pid[f - c0] < 0)
                        bad = true;
                    else
                        pages(blk, tok0, One{}, std::true_type{});
                    ++f;
                }
                if (((f - c0) & (NP - 1)) == 0 || f == c1) {  // the slot is used up
                    f += NP * (kWarps - 1);
                    __syncwarp();  // every lane has read it
                    if (ask < c1 - c0) request();
                    if (++out_slot == NS) {
                        out_slot = 0;
                        out_phase ^= 1;
                    }
                }
            }
            if (s_base[b + 1] > c1) break;  // goes on in the next stretch or CTA
            end_sequence();
            ++b;
            while (b < p.B && s_base[b + 1] == s_base[b]) ++b;
            if (b >= p.B || s_base[b] >= hi) break;
            begin_sequence();
            if (s_base[b] >= c1) break;
        }
    }
    if (b < p.B && s_base[b] < hi && s_base[b + 1] > hi) end_sequence();
    // After a timeout: copies still on their way must not outlive the CTA's
    // shared memory.
    for (; dead && pending > 0; --pending) {
        mbar_wait_bounded(bar_w + out_slot * 8, out_phase);
        if (++out_slot == NS) {
            out_slot = 0;
            out_phase ^= 1;
        }
    }
}

template <int D, typename T>
cudaError_t launch_q4_attend_d(const Q4AttendParams& p, dim3 grid, cudaStream_t stream) {
    const int smem = Q4Cfg<D>::smem(p.B);
    // The kernel's shared-memory limit, raised once per device to the most a
    // plan can ask for.
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!bit || !(done.load() & bit)) {
        e = cudaFuncSetAttribute(q4_attend_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Q4Cfg<D>::smem(4096));
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, q4_attend_kernel<D, T>, p);
}

}  // namespace pa
