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
//  * What bounds it.  A page of one KV head is 20 D bytes (64 D in fp16), so
//    memory could deliver about 38 elements per clock and SM at D 128.  A pair
//    of elements costs a shift, a logic op and a packed fma (the code becomes
//    the float 16 + c, the fma applies s and z with one rounding); with the
//    softmax and the ring a page of D 128 is about 290 warp instructions, 65 %
//    of what an SM issues in the 112 cycles that memory needs for it.  So the
//    layout spends nothing else: codes and parameters lie as the mma fragments
//    want them (no ldmatrix, no transposition, no bank conflict), both halves of
//    a register come from one fma.  tcgen05 would take its operands from shared
//    memory, where the values would first have to be stored; at up to 8 query
//    heads mma.sync is a fifth busy.
//    Measured on GB300: 4 sequences of 100K tokens, 24/4 heads at D 256, 90 us,
//    5.68 TB/s (0.84 of the measured copy rate).  From 128K to 512K tokens at D
//    128 each further byte goes at 0.9-1.0 of that rate (bf16, whose weights take
//    two mma, at 0.8); what is lost is a fixed part of 8 us and more: the start,
//    warps of an SM that end unevenly, joining and merging.
//  * Copies.  K, V and parameters of a page are one block, fetched by one
//    cp.async.bulk into the ring of the warp that works on it; the pages of a
//    CTA's range go to its four warps in turn.
//  * Maximum.  m is raised, and O rescaled, only when a score exceeds it by
//    more than 8 in the log2 domain (weights then stay below 2^8, far from
//    fp16's limit); so most pages need no shuffle, just one vote.
//  * Split.  Where every sequence is short (q4_short pages) and there are CTAs
//    enough, each has one to itself.  Where clusters of CTAs, one per sequence,
//    fit the GPU at once and leave no CTA many pages more than equal ranges do
//    (pa_q4_plan has the figures), a cluster shares a sequence evenly and merges
//    its CTAs' states through distributed shared memory: 4 sequences of 1000
//    tokens 9.5 -> 7.6 us.  Otherwise the pages the batch attends, all sequences
//    end to end, are cut into ranges of equal cost (kQ4Start), one per CTA of the
//    group, whatever the lengths; a range may hold many short sequences or part of
//    a long one.  At a sequence's end the warps' states meet in shared memory.  A
//    sequence inside the range is written; one cut by a border leaves a partial
//    (o, maximum, sum) per CTA in the workspace.  Who merges a sequence's
//    partials, always in order: the last CTA to leave one, or, in plans where a
//    sequence may leave many, a second kernel that has them all in flight.
#pragma once

#include <math.h>

#include <atomic>
#include <climits>
#include <type_traits>

#include "pa_q4.cuh"

namespace pa {

// The kernel's state is captured by reference: a lambda that is not inlined
// puts the accumulators into local memory.
#define PA_INLINE_LAMBDA __attribute__((always_inline))

// Pages up to which a sequence goes to one CTA where there is one for each: 40
// sequences of up to 40 tokens 13.2 -> 4.3 us.  Against clusters at 16 and 24
// pages: D 64 ragged 5.0 and 6.0, 5.7 and 6.1 us, D 128 5.4 and 6.0, 6.2 and 5.8
// (ragged 7.0 and 7.4), D 256 7.5 and 7.3, 9.0 and 7.5.
constexpr int q4_short(int D) { return D == 256 ? 16 : 24; }
// What a sequence's start and end cost a CTA, in pages: equal ranges are equal
// in this cost, not in pages.  0, 4, 8, 12, 16, 24: 64 ragged sequences up to
// 4096 tokens (bf16, D 128) 50.0, 49.5, 48.7, 47.7, 48.0, 48.1 us, 4 of 4096 at D
// 256 15.5, 14.6, 12.7, 12.8, 12.7, 13.2, 32 of 4096 (fp16) 39.7, 39.8, 38.7, 37.9,
// 37.8, 37.8, 256 of up to 512 45.5, 41.0, 39.7, 39.3, 38.4, 38.4.
constexpr int kQ4Start = 12;
constexpr int kQ4StagedPages = 512;  // page ids a CTA stages at a time
// The running maximum (log2 domain) before any score: below every score that
// counts, and finite, so that a score of -inf (a product beyond fp32) is further
// below it and weighs nothing.
constexpr float kQ4NoMax = -3e38f;

struct Q4AttendParams {
    const void* q;
    const unsigned char* cache;
    const int* block_tables;
    const int* context_lens;
    void* out;
    float* lse;
    float* ws_o;    // [groups][X][2] partial outputs, normalised, [unit][lane][4]
    float* ws_ml;   // [groups][X][2][8][2] their maximum (log2 domain) and exp-sum
    int* ws_info;   // for the merge kernel: cost of a range, then s_base and s_rank [B + 1]
    unsigned* counters;  // [groups][B] partials left so far
    unsigned* err;
    int B, Hq, Hkv, g, num_pages, maxp, max_ctx, window;
    int nchunk, G, X;
    int merge_kernel;  // 1: q4_merge_kernel merges, 0: the last to leave a partial
    int cluster;       // > 0: CTAs of a sequence's cluster (X = B clusters of them)
    int stall_tx;   // test hook
    float scale_log2;
};

template <int D>
struct Q4Cfg {
    // Pages of a ring slot: two where a page is little work (what a page costs
    // beside its elements -- the wait, the vote, the request -- is then paid
    // once for two, and two chains of mma overlap), one at D 256.
    static constexpr int kPair = D == 256 ? 1 : 2;
    static constexpr int kSlotBytes = kPair * Q4Layout<D>::kPageBytes;
    // Two slots are enough: a warp's next one streams in while it works on the
    // other (one sequence of 128K tokens at D 128: 39.9 us with two, 41.0 with
    // three).
    static constexpr int kStages = D == 64 ? 4 : 2;
    static constexpr int kRingBytes = kWarps * kStages * kSlotBytes;
    // q's fragments: in registers, or in shared memory where the accumulators
    // leave no room for them.
    static constexpr bool kQShared = D == 256;
    static constexpr int kQBytes = kQShared ? D * 16 : 0;
    // Units of O: a word of dims of one head of a lane, 16 bytes a lane.  At a
    // sequence's end every warp owns a quarter of them and gets the other
    // warps' shares through shared memory.
    static constexpr int kUnits = 2 * Q4Layout<D>::kWords;
    static_assert(kUnits * 512 <= kRingBytes, "a cluster's CTA leaves its state in the ring");
    static constexpr int kXBytes = kUnits * (kWarps - 1) * 512;
    static constexpr int kSmemBytes = kRingBytes + kQBytes + kXBytes + kQ4StagedPages * 4 +
                                      kWarps * kMaxHeadsPerCta * 3 * 4 + kWarps * kStages * 8;
    // CTAs per SM by registers: 64 sequences of 4096 tokens at D 64 take 46.9 us
    // with 4 and 49.9 with 3; at D 128 four did not pay (40.1 and 40.4 us).
    static constexpr int kMinBlocks = D <= 96 ? 4 : 3;
    static_assert(kMinBlocks * (kSmemBytes + 1024 + 128) <= 228 * 1024, "CTAs per SM");
    // (four words per sequence follow: s_base, s_rank, s_page0, s_len)
    static int smem(int B) { return kSmemBytes + (4 * B + 2) * 4; }
};

// mma.sync m16n8k16, 16-bit in, fp32 accumulate; and fp32 pairs to 16 bits.
template <typename T>
struct Q4Mma;

template <>
struct Q4Mma<__half> {
    static constexpr uint32_t kOnes = 0x3C003C00u;
    // fp16 weights keep 11 bits in P.V, as in the 16-bit kernel; they are
    // normalised by the sum of the rounded ones.  Relative error of rows against
    // 64 bits: 2.4e-4 (256 tokens) to 2.9e-4 (4096 and more), where rounding
    // the exact rows to fp16 makes 1.9e-4 to 2.1e-4.  Split as for bf16 nothing is
    // added to that, but it costs a tenth: 32 sequences of 4096 tokens at D 128
    // 37.4 and 41.3 us, at D 96 33.8 and 38.0, 64 at D 64 44.7 and 50.2, 4 of 32K
    // at D 256 36.9 and 39.8, one of 256 tokens 4.5 and 4.7.
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
    // The same from zero accumulators.
    __device__ static __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1,
                                                uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
            " {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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
    // The same from zero accumulators.
    __device__ static __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1,
                                                uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
            " {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

// The partial rows of one sequence, pages [first, end) and `rank` sequences
// with pages before it, with ranges of the cost `range`: one per CTA whose range
// has pages of it.  A CTA's second row holds a sequence that
// begins inside its range, its first row any other.
struct Q4Rows {
    int x0, n;  // first CTA, rows
    int slot0;  // which row of x0
    __device__ __forceinline__ Q4Rows(int range, int first, int end, int rank) {
        first += kQ4Start * (rank + 1), end += kQ4Start * (rank + 1);
        x0 = first / range;
        n = (end - 1) / range - x0 + 1;
        slot0 = first > x0 * range ? 1 : 0;
    }
    // Row i of the sequence, in order, among its group's rows.
    __device__ __forceinline__ int row(int i) const { return (x0 + i) * 2 + (i == 0 ? slot0 : 0); }
};

template <int D, typename T>
__device__ __forceinline__ void q4_store_unit(const Q4AttendParams& p, int b, int h0, int u,
                                              int lane, float4 o, float inv) {
    const int h = 2 * (lane & 3) + (u & 1);
    uint2 r;
    r.x = Q4Mma<T>::pack(o.x * inv, o.y * inv);
    r.y = Q4Mma<T>::pack(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.out) + ((size_t)b * p.Hq + h0 + h) * D +
                              q4_v_dim<D>(lane >> 2, u >> 1)) = r;
}

// A cluster's barrier, and reads of a peer's shared memory.
__device__ __forceinline__ void q4_cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t q4_peer(const void* p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 q4_ld_peer4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float2 q4_ld_peer2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Log-sum-exp merge of rows i, i + step, ... for this lane's heads and dims of
// NU units, u, u + du, ...: NR rows of them in flight.
struct Q4Merge {
    float top, sum;
    float4 o;
};

template <int D, int NU, int NR>
__device__ __forceinline__ void q4_merge_run(const Q4AttendParams& p, const Q4Rows& rows,
                                             int group, int u, int du, int lane, int i, int step,
                                             Q4Merge (&r)[NU]) {
    const size_t row0 = (size_t)group * p.X * 2;
#pragma unroll
    for (int j = 0; j < NU; ++j) r[j] = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (; i < rows.n; i += NR * step) {
        float2 ml[NU][NR];
        float4 v[NU][NR];
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            const size_t row = row0 + rows.row(min(i + k * step, rows.n - 1));
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                const int uj = u + j * du, h = 2 * (lane & 3) + (uj & 1);
                ml[j][k] = make_float2(-INFINITY, 0.f);
                v[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (h < p.G && uj < Q4Cfg<D>::kUnits && i + k * step < rows.n) {
                    ml[j][k] = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) +
                                      row * kMaxHeadsPerCta + h);
                    v[j][k] = __ldcg(reinterpret_cast<const float4*>(p.ws_o) +
                                     (row * Q4Cfg<D>::kUnits + uj) * 32 + lane);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            float top = r[j].top;
#pragma unroll
            for (int k = 0; k < NR; ++k) top = fmaxf(top, ml[j][k].x);
            const float f = r[j].top == -INFINITY ? 0.f : ex2(r[j].top - top);
            r[j].sum *= f;
            r[j].o.x *= f, r[j].o.y *= f, r[j].o.z *= f, r[j].o.w *= f;
#pragma unroll
            for (int k = 0; k < NR; ++k) {
                // (a sum of 0: no row.  NaN is kept.)
                const float s = ml[j][k].y;
                const float w = s == 0.f ? 0.f : (s != s ? NAN : ex2(ml[j][k].x - top) * s);
                r[j].sum += w;
                r[j].o.x += w * v[j][k].x, r[j].o.y += w * v[j][k].y;
                r[j].o.z += w * v[j][k].z, r[j].o.w += w * v[j][k].w;
            }
            r[j].top = top;
        }
    }
}

template <int D, typename T>
__device__ __forceinline__ void q4_finish_unit(const Q4AttendParams& p, int b, int h0, int u,
                                               int lane, float top, float sum, float4 o) {
    if (2 * (lane & 3) + (u & 1) >= p.G || u >= Q4Cfg<D>::kUnits) return;
    q4_store_unit<D, T>(p, b, h0, u, lane, o, sum == 0.f ? 0.f : 1.f / sum);
    if (u < 2 && lane < 4)
        p.lse[(size_t)b * p.Hq + h0 + 2 * lane + u] = (top + log2f(sum)) * 0.69314718055994531f;
}

// Units u, u + du, ... of sequence b by one warp.
template <int D, typename T, int NU, int NR>
__device__ __forceinline__ void q4_merge_units(const Q4AttendParams& p, const Q4Rows& rows, int b,
                                               int group, int h0, int u, int du) {
    const int lane = threadIdx.x & 31;
    for (; u < Q4Cfg<D>::kUnits; u += NU * du) {
        Q4Merge r[NU];
        q4_merge_run<D, NU, NR>(p, rows, group, u, du, lane, 0, 1, r);
#pragma unroll
        for (int j = 0; j < NU; ++j)
            q4_finish_unit<D, T>(p, b, h0, u + j * du, lane, r[j].top, r[j].sum, r[j].o);
    }
}

// One more partial of a sequence is in place (the caller's barrier has ordered
// its stores before this); how many were there before.
__device__ __forceinline__ int q4_arrive(unsigned* counter) {
    unsigned prev;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                 : "=r"(prev)
                 : "l"(counter)
                 : "memory");
    return (int)prev;
}

// The merge as a kernel of its own: a CTA per (sequence, group, unit), whose
// warps take the rows in turn, so all of them are in flight at once.
constexpr int kQ4MergeWarps = 8;

template <int D, typename T>
__global__ void __launch_bounds__(kQ4MergeWarps * 32) q4_merge_kernel(const Q4AttendParams p) {
    __shared__ float s_top[kQ4MergeWarps][32];
    __shared__ float s_sum[kQ4MergeWarps][32];
    __shared__ float4 s_o[kQ4MergeWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x, group = blockIdx.y, u = blockIdx.z;
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    const int range = p.ws_info[0], first = p.ws_info[1 + b], end = p.ws_info[2 + b];
    if (end <= first) return;
    const Q4Rows rows(range, first, end, p.ws_info[p.B + 2 + b]);
    if (rows.n == 1) return;  // not cut
    const int h0 = (group / p.nchunk) * p.g + (group % p.nchunk) * p.G;
    Q4Merge r[1];
    q4_merge_run<D, 1, 8>(p, rows, group, u, 1, lane, warp, kQ4MergeWarps, r);
    s_top[warp][lane] = r[0].top;
    s_sum[warp][lane] = r[0].sum;
    s_o[warp][lane] = r[0].o;
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kQ4MergeWarps; ++w) top = fmaxf(top, s_top[w][lane]);
#pragma unroll
    for (int w = 0; w < kQ4MergeWarps; ++w) {
        const float ws = s_sum[w][lane];
        const float f = ws == 0.f ? 0.f : (ws != ws ? NAN : ex2(s_top[w][lane] - top));
        const float4 v = s_o[w][lane];
        sum += f * ws;
        o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
    }
    q4_finish_unit<D, T>(p, b, h0, u, lane, top, sum, o);
}

// kCluster: X is B clusters of p.cluster CTAs, one for each sequence (instances
// of their own: with the merge of a cluster in the same code, bf16's spilled 32
// bytes and 64 ragged sequences took 50.3 us for 49.3).
template <int D, typename T, bool kCluster>
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
    constexpr int NP = Cfg::kPair;

    extern __shared__ __align__(128) unsigned char q4_smem[];
    unsigned char* ring = q4_smem;
    float4* xbuf = reinterpret_cast<float4*>(ring + Cfg::kRingBytes);
    uint4* s_q = reinterpret_cast<uint4*>(xbuf + Cfg::kXBytes / 16);  // [word][lane]
    int* s_pid = reinterpret_cast<int*>(s_q + Cfg::kQBytes / 16);
    float* s_ml = reinterpret_cast<float*>(s_pid + kQ4StagedPages);  // [warp][8][m, sum, weights]
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_ml + kWarps * kMaxHeadsPerCta * 3);
    int* s_base = reinterpret_cast<int*>(bars + kWarps * NS);
    int* s_rank = s_base + p.B + 1;
    int* s_page0 = s_rank + p.B + 1;
    int* s_len = s_page0 + p.B;
    __shared__ int s_red[2];
    __shared__ long long s_scan[kWarps];
    __shared__ float2 s_sum[kMaxHeadsPerCta];  // cluster: this CTA's maximum and sum of each head

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

    // ---- The batch's pages end to end: s_base[b] of them lie before sequence
    // b (s_base[B] in all); page f of them is logical page f + s_page0[b] of
    // its sequence.  A thread sums a run of sequences, a scan over the CTA
    // joins the runs.
    const int tid = threadIdx.x;
    // Returns whether a sequence is longer than q4_short pages.
    auto scan = [&](bool one, int len) {  // one: B <= kThreads, and len is sequence tid's length
        const int per = one ? 1 : (p.B + kThreads - 1) / kThreads;
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        int longest = 0;
        long long sum = 0;  // sequences with pages << 32 | pages
        for (int b = b0; b < b1; ++b) {
            const SeqSpan sp =
                seq_span(one ? len : p.context_lens[b], p.window, p.max_ctx, p.maxp, 1);
            const int n = sp.valid ? sp.end_page - sp.first_page : 0;
            s_base[b] = n;
            s_page0[b] = sp.first_page;
            s_len[b] = sp.L;
            sum += n > 0 ? (1ll << 32) + n : 0;
            longest = max(longest, n);
        }
        long long inc = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, inc, m);
            if (lane >= m) inc += o;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        for (int w = 0; w < warp; ++w) inc += s_scan[w];
        int at = (int)(inc - sum), rank = (int)((inc - sum) >> 32);
        for (int b = b0; b < b1; ++b) {
            const int n = s_base[b];
            s_base[b] = at;
            s_rank[b] = rank;
            s_page0[b] -= at;
            at += n;
            rank += n > 0;
        }
        if (tid == kThreads - 1) {
            s_base[p.B] = (int)inc;
            s_rank[p.B] = (int)(inc >> 32);
        }
        return __syncthreads_or(longest > q4_short(D)) != 0;
    };
    // Sequence of page f: the last b with s_base[b] <= f (behind any empty ones
    // that share that number).
    auto sequence_of = [&](int f) {
        int a = 0, z = p.B - 1;
        while (a < z) {
            const int m = (a + z + 1) >> 1;
            if (s_base[m] <= f)
                a = m;
            else
                z = m - 1;
        }
        return a;
    };
    // Page at which cost x falls: the pages of b have the costs behind
    // s_base[b] + kQ4Start (s_rank[b] + 1), its start the kQ4Start before them.
    auto page_at = [&](long long x) {
        int a = 0, z = p.B;
        while (a < z) {
            const int m = (a + z + 1) >> 1;
            if (s_base[m] + kQ4Start * s_rank[m] <= x)
                a = m;
            else
                z = m - 1;
        }
        if (a == p.B) return s_base[a];
        const int in = (int)(x - s_base[a] - kQ4Start * (s_rank[a] + 1));
        return s_base[a] + min(s_base[a + 1] - s_base[a], max(0, in));
    };
    // This CTA's range [lo, hi) of the pages, the cost it begins at, and its
    // first sequence b.
    int range, from = 0, lo, hi, b;
    auto locate = [&](bool any_long) {
        const int total = s_base[p.B];
        if constexpr (kCluster) {  // an even share of a sequence
            b = blockIdx.x / p.cluster;
            const int first = s_base[b], n = s_base[b + 1] - first;
            range = max(NP, ((n + p.cluster - 1) / p.cluster + NP - 1) / NP * NP);
            const int at = (int)(blockIdx.x - b * p.cluster) * range;
            lo = first + min(n, at);
            hi = first + min(n, at + range);
            return;
        }
        if (!any_long && p.B <= p.X) {  // a CTA for each sequence
            range = max(1, total + kQ4Start * s_rank[p.B]);  // (no border cuts anything)
            b = min((int)blockIdx.x, p.B - 1);
            lo = (int)blockIdx.x < p.B ? s_base[b] : total;
            hi = (int)blockIdx.x < p.B ? s_base[b + 1] : total;
            return;
        }
        const int cost = total + kQ4Start * s_rank[p.B];
        range = max(NP * kWarps, (cost + p.X - 1) / p.X);
        from = (int)min((long long)cost, (long long)blockIdx.x * range);
        lo = page_at(from);
        hi = page_at((long long)from + range);
        b = lo < hi ? sequence_of(lo) : 0;
    };
    auto table_entry = [&](int f) {
        const int a = f < s_base[b + 1] ? b : sequence_of(f);
        return p.block_tables + (size_t)a * p.maxp + (f + s_page0[a]);
    };

    // Up to kThreads sequences: all this is worked out before the wait for the
    // previous grid, from lengths that may still change, and the first pages
    // are requested into L2 (addresses checked as ever; a stale one only
    // fetches a page that is not used).  After the wait the lengths and the
    // first ids are read again, in one round trip, and the work stands if no
    // length has changed.  Steps one behind the other: 32 sequences of 4096
    // tokens 41.2 -> 39.5 us, one of 128K 38.8 -> 37.5.
    const bool early = p.B <= kThreads;
    int len = 0;
    if (early) {
        if (tid < p.B) len = __ldcg(p.context_lens + tid);
        locate(scan(true, len));
        const int f = lo + (lane / NP) * (NP * kWarps) + NP * warp + lane % NP;
        if (lane < NS * NP && f < hi) {
            const int id = __ldcg(table_entry(f));
            if (id >= 0 && id < p.num_pages)
                prefetch_l2(p.cache + ((size_t)id * p.Hkv + kvh) * (size_t)PB, PB);
        }
    }
    wait_for_prerequisite_grid();
    constexpr int kIds = kQ4StagedPages / kThreads;  // ids of a stretch per thread
    int ids[kIds];
    bool again = true;
    if (early) {
        const int now = tid < p.B ? __ldcg(p.context_lens + tid) : 0;
#pragma unroll
        for (int i = 0; i < kIds; ++i) {
            const int f = lo + tid + i * kThreads;
            ids[i] = f < hi ? *table_entry(f) : 0;
        }
        again = __syncthreads_or(now != len);
    }
    if (again) {
        len = early && tid < p.B ? p.context_lens[tid] : 0;
        locate(scan(early, len));
    }
    if (p.merge_kernel && blockIdx.x == 0 && blockIdx.y == 0) {
        if (tid == 0) p.ws_info[0] = range;
        for (int i = tid; i <= p.B; i += kThreads) {
            p.ws_info[1 + i] = s_base[i];
            p.ws_info[p.B + 2 + i] = s_rank[i];
        }
    }

    // ---- Sequences that attend nothing: out 0 and lse -inf, or NaN where the
    // length is out of bounds.
    T* const out = reinterpret_cast<T*>(p.out);
    for (int e = blockIdx.x; e < p.B; e += gridDim.x) {
        if (s_base[e + 1] != s_base[e]) continue;
        const bool valid = seq_span(s_len[e], p.window, p.max_ctx, p.maxp, 1).valid;
        if (!valid && tid == 0) atomicOr(p.err, PA_DEVERR_BAD_LENGTH);
        const uint32_t fill = valid ? 0u : 0x7FFF7FFFu;
        uint32_t* row = reinterpret_cast<uint32_t*>(out + ((size_t)e * p.Hq + h0) * D);
        for (int i = tid; i < G * D / 2; i += kThreads) row[i] = fill;
        if (tid < G) p.lse[(size_t)e * p.Hq + h0 + tid] = valid ? -INFINITY : NAN;
    }
    // (A cluster whose sequence attends anything needs all its CTAs below.)
    if (lo >= hi && (!kCluster || s_base[b + 1] == s_base[b])) return;

    // ---- Registers of a sequence: q as the mma's B operand, O^T, the sums.
    // q, word w: pairs (P, P + 4) of its 8 dims, P = 0..3
    // (kQShared: this warp's share of it on its way to shared memory)
    uint4 qf[Cfg::kQShared ? W / kWarps : W];
    float acc[W][2][4];         // O^T: dims q4_v_dim(g, w) + 2u (rows g), + 2u + 1, heads 2t, 2t + 1
    float lacc[4];              // sums of the rounded weights (all rows alike)
    float m0, m1, l0, l1;       // running maximum (log2 domain), sums of this lane's weights
    int seq_L = 0, seq_start = 0;
    bool dead = false;          // a copy timed out
    bool bad = false;           // this sequence met a bad page id or a timeout

    // The q of a sequence is requested first, and again for the next sequence
    // before the states of the present one are joined, which hides the loads.
    constexpr int QL = Cfg::kQShared ? W / kWarps : W;  // words of q this warp loads
    auto load_q = [&](int seq) PA_INLINE_LAMBDA {
        const T* qrow = reinterpret_cast<const T*>(p.q) + ((size_t)seq * p.Hq + h0 + g) * D;
#pragma unroll
        for (int i = 0; i < QL; ++i) {
            const int w = Cfg::kQShared ? warp + i * kWarps : i;
            qf[i] = make_uint4(0, 0, 0, 0);
            if (g < G) qf[i] = *reinterpret_cast<const uint4*>(qrow + q4_k_dim<D>(t, w));
        }
    };
    auto begin_sequence = [&]() PA_INLINE_LAMBDA {
        seq_L = s_len[b];
        seq_start = (p.window > 0 && p.window < seq_L) ? seq_L - p.window : 0;
#pragma unroll
        for (int i = 0; i < QL; ++i) {
            const uint4 x = qf[i];
            qf[i] = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                               __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
            if (Cfg::kQShared) s_q[(warp + i * kWarps) * 32 + lane] = qf[i];
        }
        if (Cfg::kQShared) __syncthreads();  // (no warp still reads the previous sequence's)
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[w][u][i] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) lacc[i] = 0.f;
        m0 = m1 = kQ4NoMax;
        l0 = l1 = 0.f;
        bad = dead;
    };

    // ---- N consecutive pages in shared memory; MASK: some of their tokens may
    // lie outside the attended range (their cells may hold anything).
    auto pages = [&](const unsigned char* blk0, int tok0, auto n_pages, auto mask) PA_INLINE_LAMBDA {
        constexpr int N = decltype(n_pages)::value;
        constexpr bool MASK = decltype(mask)::value;
        float s[N][4];
        // K: tokens g and g + 8 of this lane's dims.
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned char* blk = blk0 + j * PB;
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
                    const uint4 q = Cfg::kQShared ? s_q[(sl * V + i) * 32 + lane]
                                                  : qf[Cfg::kQShared ? 0 : sl * V + i];
                    const uint32_t a0 = Q::fma2(sa, Q::template code16<0>(ka[i]), za);
                    const uint32_t a1 = Q::fma2(sb, Q::template code16<0>(kb[i]), zb);
                    const uint32_t a2 = Q::fma2(sa, Q::template code16<1>(ka[i]), za);
                    const uint32_t a3 = Q::fma2(sb, Q::template code16<1>(kb[i]), zb);
                    if (sl == 0 && i == 0)
                        M::mma0(s[j], a0, a1, a2, a3, q.x, q.y);
                    else
                        M::mma(s[j], a0, a1, a2, a3, q.x, q.y);
                    M::mma(s[j], Q::fma2(sa, Q::template code16<2>(ka[i]), za),
                           Q::fma2(sb, Q::template code16<2>(kb[i]), zb),
                           Q::fma2(sa, Q::template code16<3>(ka[i]), za),
                           Q::fma2(sb, Q::template code16<3>(kb[i]), zb), q.z, q.w);
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
            const float f0 = ex2(m0 - n0), f1 = ex2(m1 - n1);
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

    const int group = blockIdx.y;
    const size_t row0 = ((size_t)group * p.X + blockIdx.x) * 2;
    auto unit_of = [&](int u, float f) PA_INLINE_LAMBDA {  // (u a constant where this is called)
        const int w = u >> 1, k = u & 1;
        return make_float4(acc[w][0][k] * f, acc[w][0][2 + k] * f, acc[w][1][k] * f,
                           acc[w][1][2 + k] * f);
    };

    // ---- The end of sequence b in this CTA.  Sequences that a border cuts (at
    // most two) are noted.  The one at the range's head is counted at once,
    // long before the CTA that has its front gets there; thread 0 looks at the
    // count when it is done.
    int cut_head = -1, cut_tail = -1, head_count = 0;
    unsigned* counters = p.counters + (size_t)group * p.B;
    auto end_sequence = [&]() PA_INLINE_LAMBDA {
        const bool cut = !kCluster && (s_base[b] < lo || s_base[b + 1] > hi);
        const bool tail = s_base[b] + kQ4Start * (s_rank[b] + 1) > from;
        const size_t row = row0 + (tail ? 1 : 0);
        if (cut) (tail ? cut_tail : cut_head) = b;
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, k);
            l1 += __shfl_xor_sync(0xffffffffu, l1, k);
        }
        if (bad) l0 = l1 = NAN;
        __syncthreads();  // the last use of xbuf and s_ml is over
        if (g == 0) {
            float* ml = s_ml + (warp * kMaxHeadsPerCta + 2 * t) * 3;
            ml[0] = m0, ml[1] = l0, ml[2] = lacc[0];
            ml[3] = m1, ml[4] = l1, ml[5] = lacc[1];
        }
        __syncthreads();
        // Maximum and sums over the warps of heads 2t, 2t + 1, and this warp's
        // factor.  (A sum of 0: the warp had no page.  NaN is kept.)
        float top[2], sum[2], inv[2], own[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float* ml = s_ml + (2 * t + k) * 3;
            top[k] = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                top[k] = fmaxf(top[k], ml[w * kMaxHeadsPerCta * 3]);
            sum[k] = 0.f;
            float wsum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* x = ml + w * kMaxHeadsPerCta * 3;
                const float f = x[1] == 0.f ? 0.f : (x[1] != x[1] ? NAN : ex2(x[0] - top[k]));
                sum[k] += f * x[1];
                wsum += f * x[2];
                if (w == warp) own[k] = f;
            }
            inv[k] = wsum == 0.f ? 0.f : 1.f / wsum;  // (0: no score above -inf)
        }
#pragma unroll
        for (int u = 0; u < Cfg::kUnits; ++u)
            if (2 * t + (u & 1) < G && (u & 3) != warp)
                xbuf[(u * (kWarps - 1) + ((warp - u - 1) & 3)) * 32 + lane] =
                    unit_of(u, own[u & 1]);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < Cfg::kUnits; ++u) {
            const int k = u & 1;
            if (2 * t + k >= G || (u & 3) != warp) continue;
            float4 o = unit_of(u, own[k]);
#pragma unroll
            for (int x = 0; x < kWarps - 1; ++x) {
                const float4 v = xbuf[(u * (kWarps - 1) + x) * 32 + lane];
                o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
            }
            if (!cut && !kCluster) {
                q4_store_unit<D, T>(p, b, h0, u, lane, o, inv[k]);
            } else {
                o.x *= inv[k], o.y *= inv[k], o.z *= inv[k], o.w *= inv[k];
                if (kCluster)  // (the ring is idle: this is the range's end)
                    reinterpret_cast<float4*>(ring)[u * 32 + lane] = o;
                else
                    reinterpret_cast<float4*>(p.ws_o)[(row * Cfg::kUnits + u) * 32 + lane] = o;
            }
        }
        if (warp == 0 && g == 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int h = 2 * t + k;
                if (h >= G) continue;
                if (kCluster)
                    s_sum[h] = make_float2(top[k], sum[k]);
                else if (!cut)
                    p.lse[(size_t)b * p.Hq + h0 + h] =
                        (top[k] + log2f(sum[k])) * 0.69314718055994531f;
                else
                    reinterpret_cast<float2*>(p.ws_ml)[row * kMaxHeadsPerCta + h] =
                        make_float2(top[k], sum[k]);
            }
        }
        if (cut && !tail && !p.merge_kernel) {
            __syncthreads();
            if (threadIdx.x == 0) head_count = q4_arrive(counters + b);
        }
    };

    // ---- The range, kQ4StagedPages at a time.  Slots of NP pages go to the
    // warps in turn; a warp's copies take its ring slots round.
    constexpr int SB = Cfg::kSlotBytes;
    using One = std::integral_constant<int, 1>;
    using Slot = std::integral_constant<int, NP>;
    int in_slot = 0, out_slot = 0;    // ring slots of the next copy and of the next page
    uint32_t out_phase = 0;
    int pending = 0;                  // slots requested and not yet waited for
    int stall = p.stall_tx;
    for (int c0 = lo; c0 < hi; c0 += kQ4StagedPages) {
        const int c1 = min(hi, c0 + kQ4StagedPages);
        __syncthreads();  // the previous stretch's ids have been used
        bool bad_id = false;
#pragma unroll
        for (int i = 0; i < kIds; ++i) {
            const int f = c0 + tid + i * kThreads;
            if (f >= c1) continue;
            int id = again || c0 != lo ? *table_entry(f) : ids[i];
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
        const int n_ids = c1 - c0;
        auto request = [&]() PA_INLINE_LAMBDA {
            if (lane == 0) {
                const uint32_t bar = bar_w + in_slot * 8, dst = ring_u + in_slot * SB;
                int id[NP], n = 0;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    id[j] = j == 0 || ask + j < n_ids ? s_pid[ask + j] : -1;
                    n += id[j] >= 0 ? PB : 0;
                }
                mbar_arrive_expect_tx(bar, n + stall);
#pragma unroll
                for (int j = 0; j < NP; ++j)
                    if (id[j] >= 0)
                        bulk_g2s(dst + j * PB,
                                 p.cache + ((size_t)id[j] * p.Hkv + kvh) * (size_t)PB, PB, bar);
                stall = 0;
            }
            ask += NP * kWarps;
            in_slot = in_slot + 1 == NS ? 0 : in_slot + 1;
            ++pending;
        };
        // The next slot's pages are there (or the wait for them ran out).
        auto wait = [&]() PA_INLINE_LAMBDA {
            const uint32_t bar = bar_w + out_slot * 8;
            if (!__all_sync(0xffffffffu, mbar_try_wait(bar, out_phase)) &&
                !__all_sync(0xffffffffu, mbar_wait_bounded(bar, out_phase))) {
                if (lane == 0) atomicOr(p.err, PA_DEVERR_TIMEOUT);
                dead = bad = true;
            }
        };
        auto release = [&]() PA_INLINE_LAMBDA {
            --pending;
            __syncwarp();  // every lane has read the slot
            if (ask < n_ids) request();
            if (++out_slot == NS) {
                out_slot = 0;
                out_phase ^= 1;
            }
        };
        if (!dead)
            for (int i = 0; i < NS && ask < n_ids; ++i) request();
        // (the first q is fetched while the first pages are on their way)
        if (c0 == lo) {
            load_q(b);
            begin_sequence();
        }

        int f = dead ? c1 : c0 + NP * warp;  // next page of this warp
        while (true) {
            const int seg_end = min(c1, s_base[b + 1]);
            // Pages that are attended whole lie in [whole0, whole1).
            const int base = -s_page0[b];  // page of token 0
            const int whole0 = careful ? INT_MAX : base + (seq_start + kPageSize - 1) / kPageSize;
            const int whole1 = min(seg_end, base + seq_L / kPageSize);
            while (f < seg_end) {
                if (((f - c0) & (NP - 1)) == 0) {
                    // Slots of whole pages, the bulk of a long sequence.
                    if (f >= whole0) {
                        for (; f + NP <= whole1; f += NP * kWarps) {
                            wait();
                            if (dead) break;
                            pages(ring_w + out_slot * SB, 0, Slot{}, std::false_type{});
                            release();
                        }
                        if (!dead && f >= seg_end) break;
                    }
                    if (!dead) wait();
                    if (dead) {
                        f = c1;
                        break;
                    }
                }
                // One page, with some of its tokens masked or a bad id near.
                if (careful && s_pid[f - c0] < 0)
                    bad = true;
                else
                    pages(ring_w + out_slot * SB + ((f - c0) & (NP - 1)) * PB,
                          (f - base) * kPageSize, One{}, std::true_type{});
                ++f;
                if (((f - c0) & (NP - 1)) == 0 || f == c1) {  // the slot is used up
                    f += NP * (kWarps - 1);
                    release();
                }
            }
            if (s_base[b + 1] > c1 && c1 < hi) break;  // goes on in the next stretch
            if (s_base[b + 1] >= hi) {  // the range's last
                end_sequence();
                break;
            }
            int next = b + 1;
            while (s_base[next + 1] == s_base[next]) ++next;
            load_q(next);
            end_sequence();
            b = next;
            begin_sequence();
            if (s_base[b] >= c1) break;
        }
    }
    if constexpr (kCluster) {
        // The state of every CTA with pages is in its ring and s_sum; each warp of
        // the cluster merges units of all of them, whose reads go out together.
        // The second barrier keeps the shared memory until all have read it.
        __syncthreads();
        q4_cluster_barrier();
        const int rank = blockIdx.x - b * p.cluster;
        const int rows = (s_base[b + 1] - s_base[b] + range - 1) / range;
        for (int u = rank * kWarps + warp; u < Cfg::kUnits; u += p.cluster * kWarps) {
            const int h = 2 * t + (u & 1);
            float m = -INFINITY, sum = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            constexpr int N = 8;  // peers in flight
            for (int r0 = 0; r0 < rows; r0 += N) {
                float2 ml[N];
                float4 v[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int r = min(r0 + i, rows - 1);
                    ml[i] = q4_ld_peer2(q4_peer(s_sum + h, r));
                    v[i] = q4_ld_peer4(q4_peer(ring + (u * 32 + lane) * 16, r));
                    if (r0 + i >= rows) ml[i] = make_float2(-INFINITY, 0.f);
                }
                float top = m;
#pragma unroll
                for (int i = 0; i < N; ++i) top = fmaxf(top, ml[i].x);
                const float f = m == -INFINITY ? 0.f : ex2(m - top);
                sum *= f;
                o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float l = ml[i].y;
                    const float w = l == 0.f ? 0.f : (l != l ? NAN : ex2(ml[i].x - top) * l);
                    if (w == 0.f) continue;
                    sum += w;
                    o.x += w * v[i].x, o.y += w * v[i].y, o.z += w * v[i].z, o.w += w * v[i].w;
                }
                m = top;
            }
            q4_finish_unit<D, T>(p, b, h0, u, lane, m, sum, o);
        }
        q4_cluster_barrier();
    }
    // After a timeout: copies still on their way must not outlive the CTA's
    // shared memory.
    for (; dead && pending > 0; --pending) {
        mbar_wait_bounded(bar_w + out_slot * 8, out_phase);
        if (++out_slot == NS) {
            out_slot = 0;
            out_phase ^= 1;
        }
    }
    if (kCluster || p.merge_kernel) return;
    // (here, behind the loop: in it the merge's loads in flight made the
    // accumulators spill, 64 ragged sequences 51 -> 88 us)
    if (cut_head < 0 && cut_tail < 0) return;
    __syncthreads();
    if (threadIdx.x == 0) {
        auto last = [&](int c, int before) {
            const bool is = before == Q4Rows(range, s_base[c], s_base[c + 1], s_rank[c]).n - 1;
            if (is) counters[c] = 0;  // ready for the next call
            return is;
        };
        s_red[0] = cut_head >= 0 && last(cut_head, head_count);
        s_red[1] = cut_tail >= 0 && last(cut_tail, q4_arrive(counters + cut_tail));
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int c = i == 0 ? cut_head : cut_tail;
        if (s_red[i])
            q4_merge_units<D, T, 2, 4>(p, Q4Rows(range, s_base[c], s_base[c + 1], s_rank[c]), c, group, h0,
                                       warp, kWarps);
    }
}

// The kernel's shared memory limit raised to what the largest batch asks for.
template <int D, typename T, bool kCluster>
cudaError_t q4_attend_attributes() {
    return cudaFuncSetAttribute(q4_attend_kernel<D, T, kCluster>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Q4Cfg<D>::smem(4096));
}

// Clusters of c CTAs that the current device holds at once.
template <int D, typename T>
cudaError_t q4_attend_clusters(int c, int batch, int* held) {
    cudaError_t e = q4_attend_attributes<D, T, true>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Q4Cfg<D>::smem(batch);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(held, q4_attend_kernel<D, T, true>, &cfg);
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
        e = q4_attend_attributes<D, T, false>();
        if (e == cudaSuccess) e = q4_attend_attributes<D, T, true>();
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster ? 2 : 1;
    e = p.cluster ? cudaLaunchKernelEx(&cfg, q4_attend_kernel<D, T, true>, p)
                  : cudaLaunchKernelEx(&cfg, q4_attend_kernel<D, T, false>, p);
    if (e != cudaSuccess || !p.merge_kernel) return e;
    cfg.gridDim = dim3(p.B, grid.y, Q4Cfg<D>::kUnits);
    cfg.blockDim = dim3(kQ4MergeWarps * 32);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, q4_merge_kernel<D, T>, p);
}

}  // namespace pa
