// pa_q8_attend.cuh -- attention of one or several query tokens per sequence
// over the 8-bit paged cache (pa_q8_decode of include/pa_q8.h).
//
// For sequence b and the R = G T_b query rows (G heads, T_b tokens) of a KV
// head's chunk, in NT tiles of 8 rows:
//   S^T[16 tokens x 8] = K[16 x D] Q^T, p = 2^(scale log2(e) k_scale S - m),
//   O^T[D x 8] += V^T[D x 16] (v_scale P)^T in two parts, out = O / sum p,
//   lse = ln 2 (m + log2 sum p)
// page by page with a running maximum m; the codes of K and V become fp16 (every
// e4m3 value is one) in registers in front of the mma.sync m16n8k16.
//
// Tokens are the products' rows, so a step with one query row wastes no more than seven of
// eight columns, and a page of 16 tokens is one tile.  A warp takes whole pages, one after the
// other of its CTA's range, with a ring of its own (a tensor copy for K and one for V, whose
// swizzle makes every ldmatrix free of conflicts), an own maximum and own accumulators: no
// barrier until the sequence ends.  V's codes come out of ldmatrix.trans with two tokens' bytes
// of a dim pair in a word, one byte_perm from what the product takes.
//
// Bound by: the copies, where there is one tile of rows (4 sequences of 100000 tokens, 24/4
// heads, D 256: 127 us, 0.95 of the copy rate; 16 of 8192 with two queries, 32/8, D 128: 49.2,
// 0.81); with more the latency of a warp's page (four tiles of rows, eight queries: 102.6 us,
// 0.39), whose accumulators leave two warps a scheduler; in short steps the start, of about
// 1.3 us, and the joining of a sequence's states (16 of a 4096 window, five queries: 46.9 us
// of a floor of 20).  Slots of a warp's ring, 2, 3, 4: 64 ragged sequences 47.8, 48.8, 48.9 us.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>
#include <climits>
#include <type_traits>

#include "../../include/pa_q8.h"
#include "pa_common.cuh"

namespace pa {

#define PA_INLINE_LAMBDA __attribute__((always_inline))

// Pages up to which a plan gives each sequence one CTA, if so many run at once, and no
// cluster (48 sequences of 24 pages 10.0 us, in ranges 15.1; beyond, see kQ8Whole).
constexpr int q8_short(int D) { return D == 256 ? 16 : 24; }
// What a sequence's start and end cost a CTA, in pages: equal ranges are equal
// in this cost, not in pages.  (6, 12, 20: 64 ragged sequences 47.7, 47.4, 47.6 us, 16 with
// five queries 48.7, 46.9, 46.9.)
constexpr int kQ8Start = 12;
// Where there is a CTA for each sequence, each has one unless the longest has so many pages
// more than an equal range costs: that many are as long as cutting and joining.  (48 of 57
// CTAs a head, head_dim 128, sequences of 560 tokens 18.4 -> 13.1 us, of 2000 39.2 -> 35.6; with
// 48 pages instead, 30 of up to 1000 tokens 13.1 -> 16.2.)
constexpr int kQ8Whole = 24;
// The running maximum (log2 domain) before any score: below every score that
// counts, and finite, so that a score of -inf is further below it.
constexpr float kQ8NoMax = -3e38f;
// Weights are 2^(score - m).  m is set kQ8Room below a new greatest score and left
// until a score exceeds it by kQ8Most: p stays below 2^15 (fp16 ends at 2^16) and
// the least weight fp16 holds is 2^-24 / 2^kQ8Room of the greatest's.
constexpr float kQ8Room = 8.f, kQ8Most = 15.f;
// A page whose V scale is at least this share of the reference has it applied to
// its weights; below, to its products.
constexpr float kQ8LeastRatio = 0x1p-8f;
constexpr int kQ8MaxRows = 32;  // query rows of a CTA (NT tiles of 8)

constexpr int q8_max_rows(int D) { return D == 256 ? 16 : kQ8MaxRows; }

struct Q8Maps {
    CUtensorMap k, v;
};

struct Q8AttendParams {
    const void* q;
    const int* starts;       // null: one row per sequence
    const unsigned char* k;  // (for prefetches; copies go by the maps)
    const unsigned char* v;
    const float* k_scales;
    const float* v_scales;
    const int* block_tables;
    const int* context_lens;
    void* out;
    float* lse;
    float* ws_o;    // [groups][X][2] partial outputs, normalised, [unit][lane][4]
    float* ws_ml;   // [groups][X][2][8 NT][2] their maximum (log2 domain) and exp-sum
    int* ws_info;   // for the merge kernel: cost of a range, then s_base, s_rank, s_row [B + 1]
    unsigned* counters;  // [groups][B] partials left so far
    unsigned* err;
    int B, Hq, Hkv, g, num_pages, maxp, max_ctx, window, max_t, rows;
    int nchunk, G, X;
    int ginv;          // 65536 / G + 1: r / G = r ginv >> 16 for rows r below kQ8MaxRows
    int merge_kernel;  // 1: q8_merge_kernel merges, 0: the last to leave a partial
    int cluster;       // > 0: CTAs of a sequence's cluster (X = B clusters of them)
    int stall_tx;      // test hook
    int bf16;          // q and out are bf16
    float scale_log2;
};

template <int D, int NT>
struct Q8Cfg {
    static constexpr int kPage = 16 * D;           // bytes of a page of K, or of V
    static constexpr int kSlotBytes = 2 * kPage;   // a ring slot: a page's K and V
    static constexpr int kStages = D == 64 ? 4 : (NT > 2 ? 3 : 2);
    static constexpr int kRingBytes = kWarps * kStages * kSlotBytes;
    // q's fragments: in registers, or in shared memory where the accumulators
    // leave no room for them.
    static constexpr bool kQShared = NT > 1;
    static constexpr int kQBytes = kQShared ? NT * D * 16 : 0;
    // Units of O: 4 dims of one row of a lane, 16 bytes a lane.
    static constexpr int kTileUnits = D / 16;
    static constexpr int kUnits = NT * kTileUnits;
    static constexpr int kRows = 8 * NT;
    static_assert(kUnits * 512 <= kRingBytes, "a cluster's CTA leaves its state in the ring");
    static constexpr int kXBytes = kTileUnits * kWarps * 512;
    // Page ids and scales that a CTA stages at a time.
    static constexpr int kStaged = NT == 2 && D == 256 ? 256 : 512;
    static constexpr int kSmemBytes = 1024 + kRingBytes + kXBytes + kQBytes + kStaged * 12 +
                                      kWarps * kRows * 8 + kRows * 4 + kWarps * kStages * 8;
    // CTAs per SM by registers.
    static constexpr int kMinBlocks = D == 256 || NT > 2 ? 2 : 3;
    static constexpr int kStaticBytes = kRows * 8 + 128;  // (beside the dynamic ones)
    static_assert(kMinBlocks * (kSmemBytes + kStaticBytes + 1024) <= 228 * 1024, "CTAs per SM");
    // (five words per sequence follow: s_base, s_rank, s_row, s_page0, s_len)
    static int smem(int B) { return kSmemBytes + (5 * B + 3) * 4; }
};

__device__ __forceinline__ void q8_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero accumulators.
__device__ __forceinline__ void q8_mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t q8_pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 q8_unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

__device__ __forceinline__ uint32_t q8_movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void q8_ldmatrix(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void q8_ldmatrix_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// The fp16 values of two e4m3 codes: bytes 0 and 1 (low), or 2 and 3 (high).
__device__ __forceinline__ uint32_t q8_low(uint32_t x) {
    uint32_t y;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}"
        : "=r"(y)
        : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t q8_high(uint32_t x) {
    uint32_t y;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}"
        : "=r"(y)
        : "r"(x));
    return y;
}

// 0x80 in every byte that is the code of a NaN (0x7F, 0xFF).
__device__ __forceinline__ uint32_t q8_nan_bytes(uint32_t x) {
    return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Byte of 16-byte chunk c of token r of a page in shared memory.  A page arrives
// through one tensor copy whose swizzle lays the eight rows that an ldmatrix phase
// reads into eight different bank groups: D 128 and 256 as slabs of 128 bytes a
// row (128-byte swizzle), D 64 as rows of 64 (64-byte swizzle), D 96 as units of 32
// bytes, three a row (32-byte swizzle; three is odd, so eight rows' units cover
// all groups).
template <int D>
__device__ __forceinline__ uint32_t q8_chunk(int r, int c) {
    if constexpr (D == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    if constexpr (D == 96) {
        const int u = 3 * r + (c >> 1);
        return u * 32 + (((c & 1) ^ ((u >> 2) & 1)) << 4);
    }
    return (c >> 3) * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void q8_tma(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                       uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void q8_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void prefetch_l2_line(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

template <int D>
__device__ __forceinline__ void q8_load_page(uint32_t dst, const CUtensorMap* map, int row,
                                             uint32_t bar) {
    if constexpr (D == 96)
        q8_tma(dst, map, 0, 0, row, bar);
    else
        q8_tma(dst, map, 0, row, 0, bar);
}

// The partial rows of one sequence, pages [first, end) and `rank` sequences
// with pages before it, with ranges of the cost `range`: one per CTA whose range
// has pages of it.  A CTA's second row holds a sequence that
// begins inside its range, its first row any other.
struct Q8Rows {
    int x0, n;  // first CTA, rows
    int slot0;  // which row of x0
    __device__ __forceinline__ Q8Rows(int range, int first, int end, int rank) {
        first += kQ8Start * (rank + 1), end += kQ8Start * (rank + 1);
        x0 = first / range;
        n = (end - 1) / range - x0 + 1;
        slot0 = first > x0 * range ? 1 : 0;
    }
    // Row i of the sequence, in order, among its group's rows.
    __device__ __forceinline__ int row(int i) const { return (x0 + i) * 2 + (i == 0 ? slot0 : 0); }
};

// Row (of the CTA's 8 NT) and first dim of unit u in this lane: dims d, d + 1,
// d + 16, d + 17.
template <int D, int NT>
__device__ __forceinline__ int q8_unit_row(int u, int lane) {
    return 8 * (u / Q8Cfg<D, NT>::kTileUnits) + 2 * (lane & 3) + (u & 1);
}
template <int D, int NT>
__device__ __forceinline__ int q8_unit_dim(int u, int lane) {
    return 32 * ((u % Q8Cfg<D, NT>::kTileUnits) >> 1) + 2 * (lane >> 2);
}

__device__ __forceinline__ uint32_t q8_out2(int bf16, float x, float y) {
    if (bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return q8_pack(x, y);
}

// Row r of those that begin at row0, head h0: its place among out's and lse's rows.
__device__ __forceinline__ size_t q8_out_row(const Q8AttendParams& p, int row0, int h0, int r) {
    const int t = (r * p.ginv) >> 16;
    return (size_t)(row0 + t) * p.Hq + h0 + (r - t * p.G);
}

// Unit u of the rows that begin at row0, head h0.
template <int D, int NT>
__device__ __forceinline__ void q8_store_unit(const Q8AttendParams& p, int row0, int h0, int u,
                                              int lane, float4 o) {
    uint32_t* at = reinterpret_cast<uint32_t*>(
        reinterpret_cast<__half*>(p.out) +
        q8_out_row(p, row0, h0, q8_unit_row<D, NT>(u, lane)) * D + q8_unit_dim<D, NT>(u, lane));
    at[0] = q8_out2(p.bf16, o.x, o.y);
    at[8] = q8_out2(p.bf16, o.z, o.w);
}

__device__ __forceinline__ void q8_store_lse(const Q8AttendParams& p, int row0, int h0, int r,
                                             float top, float sum) {
    p.lse[q8_out_row(p, row0, h0, r)] = (top + log2f(sum)) * 0.69314718055994531f;
}

// 1 / x (a sum of weights), 0 for 0.
__device__ __forceinline__ float q8_inverse(float x) { return x == 0.f ? 0.f : __fdividef(1.f, x); }

// A cluster's barrier, and reads of a peer's shared memory.
__device__ __forceinline__ void q8_cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t q8_peer(const void* p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 q8_ld_peer4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float2 q8_ld_peer2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(addr)
                 : "memory");
    return v;
}

// A log-sum-exp merge: N more partials (a sum of 0: none; NaN is kept).  o is an average
// throughout, so that it is no larger than the largest of V, which may be next to fp32's end.
struct Q8Merge {
    float top, sum;
    float4 o;
    __device__ __forceinline__ Q8Merge() : top(-INFINITY), sum(0.f), o(make_float4(0, 0, 0, 0)) {}
    template <int N>
    __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&v)[N]) {
        float most = top;
#pragma unroll
        for (int i = 0; i < N; ++i) most = fmaxf(most, ml[i].x);
        float w[N];
        const float before = top == -INFINITY ? 0.f : sum * ex2(top - most);
        sum = before;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float l = ml[i].y;
            w[i] = l == 0.f ? 0.f : (l != l ? NAN : ex2(ml[i].x - most) * l);
            sum += w[i];
        }
        const float inv = q8_inverse(sum), f = before * inv;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (w[i] == 0.f) continue;
            w[i] *= inv;
            o.x += w[i] * v[i].x, o.y += w[i] * v[i].y, o.z += w[i] * v[i].z, o.w += w[i] * v[i].w;
        }
        top = most;
    }
};

// Rows i, i + step, ... of unit u: NR of them in flight.
template <int D, int NT, int NR>
__device__ __forceinline__ void q8_merge_run(const Q8AttendParams& p, const Q8Rows& rows,
                                             int group, int u, int lane, int i, int step,
                                             Q8Merge& r) {
    using Cfg = Q8Cfg<D, NT>;
    const size_t row0 = (size_t)group * p.X * 2;
    const int hr = q8_unit_row<D, NT>(u, lane);
    for (; i < rows.n; i += NR * step) {
        float2 ml[NR];
        float4 v[NR];
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            const size_t row = row0 + rows.row(min(i + k * step, rows.n - 1));
            ml[k] = make_float2(-INFINITY, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i + k * step < rows.n) {
                ml[k] = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + row * Cfg::kRows + hr);
                v[k] = __ldcg(reinterpret_cast<const float4*>(p.ws_o) +
                              (row * Cfg::kUnits + u) * 32 + lane);
            }
        }
        r.add(ml, v);
    }
}

template <int D, int NT>
__device__ __forceinline__ void q8_finish_unit(const Q8AttendParams& p, int row0, int nrows,
                                               int h0, int u, int lane, const Q8Merge& m) {
    const int r = q8_unit_row<D, NT>(u, lane);
    if (r >= nrows) return;
    q8_store_unit<D, NT>(p, row0, h0, u, lane, m.o);
    if (u % Q8Cfg<D, NT>::kTileUnits < 2 && lane < 4) q8_store_lse(p, row0, h0, r, m.top, m.sum);
}

// One more partial of a sequence is in place (the caller's barrier has ordered
// its stores before this); how many were there before.
__device__ __forceinline__ int q8_arrive(unsigned* counter) {
    unsigned prev;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                 : "=r"(prev)
                 : "l"(counter)
                 : "memory");
    return (int)prev;
}

// The merge as a kernel of its own: a CTA per (sequence, group, unit), whose
// warps take the rows in turn, so all of them are in flight at once.
constexpr int kQ8MergeWarps = 8;

template <int D, int NT>
__global__ void __launch_bounds__(kQ8MergeWarps * 32) q8_merge_kernel(const Q8AttendParams p) {
    __shared__ float2 s_ml[kQ8MergeWarps][32];
    __shared__ float4 s_o[kQ8MergeWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x, group = blockIdx.y, u = blockIdx.z;
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    const int* info = p.ws_info + 1;
    const int range = p.ws_info[0], first = info[b], end = info[b + 1];
    if (end <= first) return;
    const Q8Rows rows(range, first, end, info[p.B + 1 + b]);
    if (rows.n == 1) return;  // not cut
    const int row0 = info[2 * p.B + 2 + b], nrows = (info[2 * p.B + 3 + b] - row0) * p.G;
    const int h0 = (group / p.nchunk) * p.g + (group % p.nchunk) * p.G;
    Q8Merge r;
    if (q8_unit_row<D, NT>(u, lane) < nrows)
        q8_merge_run<D, NT, 8>(p, rows, group, u, lane, warp, kQ8MergeWarps, r);
    s_ml[warp][lane] = make_float2(r.top, r.sum);
    s_o[warp][lane] = r.o;
    __syncthreads();
    if (warp != 0) return;
    float2 ml[kQ8MergeWarps];
    float4 v[kQ8MergeWarps];
#pragma unroll
    for (int w = 0; w < kQ8MergeWarps; ++w) {
        ml[w] = s_ml[w][lane];
        v[w] = s_o[w][lane];
    }
    Q8Merge all;
    all.add(ml, v);
    q8_finish_unit<D, NT>(p, row0, nrows, h0, u, lane, all);
}

// A sequence's query rows and attended pages.
struct Q8Span {
    int L, row0, t, first_page, pages;
    bool valid;
};

__device__ __forceinline__ Q8Span q8_span(const Q8AttendParams& p, int L, int s0, int s1) {
    Q8Span s;
    const bool ordered = s0 >= 0 && s1 >= s0 && s1 <= p.rows;
    s.valid = L >= 0 && L <= p.max_ctx && (L + kPageSize - 1) / kPageSize <= p.maxp && ordered &&
              s1 - s0 <= p.max_t;
    s.row0 = min(max(s0, 0), p.rows);
    s.t = ordered ? s1 - s0 : 0;
    s.L = s.valid ? L : -1;
    const int end0 = s.valid ? L - s.t + 1 : 0;  // behind the last token that row 0 sees
    const int start = p.window > 0 && end0 > p.window ? end0 - p.window : 0;
    s.first_page = start / kPageSize;
    s.pages = s.valid && s.t > 0 ? (L + kPageSize - 1) / kPageSize - s.first_page : 0;
    return s;
}

// kCluster: X is B clusters of p.cluster CTAs, one for each sequence.
template <int D, int NT, bool kCluster>
__global__ void __launch_bounds__(kThreads, (Q8Cfg<D, NT>::kMinBlocks))
    q8_attend_kernel(const Q8AttendParams p, const __grid_constant__ Q8Maps maps) {
    using Cfg = Q8Cfg<D, NT>;
    constexpr int NS = Cfg::kStages;
    constexpr int PB = Cfg::kPage;
    constexpr int NC = D / 16;  // 16-byte chunks of a token: k steps of q.K, m tiles of P.V

    extern __shared__ __align__(128) unsigned char q8_smem[];
    // (the swizzle goes by the address: pages begin at multiples of its period)
    unsigned char* ring = q8_smem + ((1024u - (smem_u32(q8_smem) & 1023u)) & 1023u);
    float4* xbuf = reinterpret_cast<float4*>(ring + Cfg::kRingBytes);
    uint2* s_q = reinterpret_cast<uint2*>(xbuf + Cfg::kXBytes / 16);  // [tile][chunk][lane]
    float2* s_sc = reinterpret_cast<float2*>(s_q + Cfg::kQBytes / 8);  // K's and V's scale
    float2* s_ml = s_sc + Cfg::kStaged;                                // [warp][row] m, sum
    float2* s_c = s_ml + kWarps * Cfg::kRows;                          // [row pair] see crow
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_c + Cfg::kRows / 2);
    float* s_qmax = reinterpret_cast<float*>(xbuf);  // [warp][row] (while xbuf is idle)
    int* s_pid = reinterpret_cast<int*>(bars + kWarps * NS);
    int* s_base = s_pid + Cfg::kStaged;  // (s_pid: first row of the page in the cache's maps)
    int* s_rank = s_base + p.B + 1;
    int* s_row = s_rank + p.B + 1;
    int* s_page0 = s_row + p.B + 1;
    int* s_len = s_page0 + p.B;
    __shared__ int s_red[2];
    __shared__ long long s_scan[kWarps];
    __shared__ float2 s_sum[Cfg::kRows];  // cluster: this CTA's maximum and sum of each row

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int kvh = blockIdx.y / p.nchunk;
    const int h0 = kvh * p.g + (blockIdx.y % p.nchunk) * p.G;
    const uint32_t bar_w = smem_u32(bars) + warp * NS * 8;
    const uint32_t ring_u = smem_u32(ring) + warp * NS * Cfg::kSlotBytes;

    allow_dependent_launch();
    if (threadIdx.x == 0) {  // (the first copies would wait for them)
        q8_prefetch_map(&maps.k);
        q8_prefetch_map(&maps.v);
    }
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
    auto read_sequence = [&](int b, int& len, int& s0, int& s1) {
        len = __ldcg(p.context_lens + b);
        s0 = p.starts ? __ldcg(p.starts + b) : b;
        s1 = p.starts ? __ldcg(p.starts + b + 1) : b + 1;
    };
    auto range_of = [&](int pages, int sequences) {
        return max(kWarps, (pages + kQ8Start * sequences + p.X - 1) / p.X);
    };
    // Returns whether a sequence is too long for a CTA of its own.  (one: B <= kThreads,
    // and len, s0, s1 are sequence tid's)
    auto scan = [&](bool one, int len, int s0, int s1) {
        const int per = one ? 1 : (p.B + kThreads - 1) / kThreads;
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        int longest = 0;
        long long sum = 0;  // sequences with pages << 32 | pages
        for (int b = b0; b < b1; ++b) {
            if (!one) read_sequence(b, len, s0, s1);
            const Q8Span sp = q8_span(p, len, s0, s1);
            s_base[b] = sp.pages;
            s_page0[b] = sp.first_page;
            s_len[b] = sp.L;
            s_row[b] = sp.row0;
            if (b == p.B - 1) s_row[p.B] = sp.row0 + sp.t;
            sum += sp.pages > 0 ? (1ll << 32) + sp.pages : 0;
            longest = max(longest, sp.pages);
        }
        long long inc = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, inc, m);
            if (lane >= m) inc += o;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        long long all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) inc += s_scan[w];
            all += s_scan[w];
        }
        const int whole = range_of((int)all, (int)(all >> 32)) + kQ8Whole;
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
        return __syncthreads_or(longest > whole) != 0;
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
    // s_base[b] + kQ8Start (s_rank[b] + 1), its start the kQ8Start before them.
    auto page_at = [&](long long x) {
        int a = 0, z = p.B;
        while (a < z) {
            const int m = (a + z + 1) >> 1;
            if (s_base[m] + kQ8Start * s_rank[m] <= x)
                a = m;
            else
                z = m - 1;
        }
        if (a == p.B) return s_base[a];
        const int in = (int)(x - s_base[a] - kQ8Start * (s_rank[a] + 1));
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
            range = max(1, (n + p.cluster - 1) / p.cluster);
            const int at = (int)(blockIdx.x - b * p.cluster) * range;
            lo = first + min(n, at);
            hi = first + min(n, at + range);
            return;
        }
        if (!any_long && p.B <= p.X) {  // a CTA for each sequence
            range = max(1, total + kQ8Start * s_rank[p.B]);  // (no border cuts anything)
            b = min((int)blockIdx.x, p.B - 1);
            lo = (int)blockIdx.x < p.B ? s_base[b] : total;
            hi = (int)blockIdx.x < p.B ? s_base[b + 1] : total;
            return;
        }
        const int cost = total + kQ8Start * s_rank[p.B];
        range = range_of(total, s_rank[p.B]);
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
    // length has changed.
    const bool early = p.B <= kThreads;
    constexpr int kIds = Cfg::kStaged / kThreads;  // ids of a stretch per thread
    const int* entry[kIds];  // where the ids of the first stretch lie
    int len = 0, s0 = 0, s1 = 0;
    if (early) {
        if (tid < p.B) read_sequence(tid, len, s0, s1);
        locate(scan(true, len, s0, s1));
        int hint[kIds];
#pragma unroll
        for (int i = 0; i < kIds; ++i) {
            const int f = lo + tid + i * kThreads;
            entry[i] = f < hi ? table_entry(f) : nullptr;
            hint[i] = entry[i] ? __ldcg(entry[i]) : -1;
        }
#pragma unroll
        for (int i = 0; i < kIds; ++i) {
            if (hint[i] < 0 || hint[i] >= p.num_pages) continue;
            const size_t at = (size_t)hint[i] * p.Hkv + kvh;
            prefetch_l2_line(p.k_scales + at);
            prefetch_l2_line(p.v_scales + at);
            if (i == 0 && tid < NS * kWarps) {  // the ring's first pages
                prefetch_l2(p.k + at * PB, PB);
                prefetch_l2(p.v + at * PB, PB);
            }
        }
    }
    wait_for_prerequisite_grid();
    int ids[kIds];
    bool again = true;
    if (early) {
        int now = 0, now0 = 0, now1 = 0;
        if (tid < p.B) read_sequence(tid, now, now0, now1);
#pragma unroll
        for (int i = 0; i < kIds; ++i) ids[i] = entry[i] ? __ldcg(entry[i]) : 0;
        again = __syncthreads_or(now != len || now0 != s0 || now1 != s1);
        if (again) len = now, s0 = now0, s1 = now1;
    }
    if (again) locate(scan(early, len, s0, s1));
    if (p.merge_kernel && blockIdx.x == 0 && blockIdx.y == 0) {
        if (tid == 0) p.ws_info[0] = range;
        for (int i = tid; i <= p.B; i += kThreads) {
            p.ws_info[1 + i] = s_base[i];
            p.ws_info[p.B + 2 + i] = s_rank[i];
            p.ws_info[2 * p.B + 3 + i] = s_row[i];
        }
    }
    // (rows of a valid sequence end where the next one's begin)
    auto tokens_of = [&](int e) { return s_row[e + 1] - s_row[e]; };

    // ---- Sequences that attend nothing: out 0 and lse -inf, or NaN where a
    // length or start is out of bounds.
    for (int e = blockIdx.x; e < p.B; e += gridDim.x) {
        if (s_base[e + 1] != s_base[e]) continue;
        int l2, a0, a1;
        read_sequence(e, l2, a0, a1);
        const Q8Span sp = q8_span(p, l2, a0, a1);
        if (!sp.valid && tid == 0) atomicOr(p.err, PA_DEVERR_BAD_LENGTH);
        const uint32_t fill = sp.valid ? 0u : 0x7FFF7FFFu;
        for (int r = 0; r < sp.t; ++r) {
            const size_t at = (size_t)(sp.row0 + r) * p.Hq + h0;
            uint32_t* row = reinterpret_cast<uint32_t*>(reinterpret_cast<__half*>(p.out) + at * D);
            for (int i = tid; i < p.G * D / 2; i += kThreads) row[i] = fill;
            if (tid < p.G) p.lse[at + tid] = sp.valid ? -INFINITY : NAN;
        }
    }
    // (A cluster whose sequence attends anything needs all its CTAs below.)
    if (lo >= hi && (!kCluster || s_base[b + 1] == s_base[b])) return;

    // ---- Registers of a sequence: q as the mma's B operand, O^T, the sums.
    // Chunk c of tile n: dims 16 c + 4 t .. + 3 of row 8 n + g, as two fp16 pairs
    // (kQShared: this warp's share of it on its way to shared memory).
    constexpr int QL = Cfg::kQShared ? (NC + kWarps - 1) / kWarps : NC;
    uint2 qf[Cfg::kQShared ? NT * QL : QL];
    float acc[NT][NC][4];  // O^T: dims 16 c + 2 g (0, 1) and the next (2, 3) of rows 2 t, 2 t + 1
    float m[NT][2];        // running maximum (log2 domain) of rows 2 t, 2 t + 1 of a tile
    float l[NT][2];        // sums of this lane's weights
    float crow[NT][2];     // what a row's products are multiplied by, beside the page's scale
                           // (kQShared: in s_c, for want of registers)
    float vref;            // acc counts in units of it
    int seq_L = 0, seq_end0 = 0, seq_rows = 0, row0 = 0;
    bool dead = false;     // a copy timed out
    bool bad = false;      // this sequence met a bad page id or a timeout

    // The q of a sequence is requested before the states of the one before it are joined,
    // which hides the loads.
    auto load_q = [&](int seq) PA_INLINE_LAMBDA {
        const int n_rows = tokens_of(seq) * p.G, first = s_row[seq];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + g;
            const __half* row = reinterpret_cast<const __half*>(p.q) +
                                q8_out_row(p, first, h0, r) * D + 4 * t;
#pragma unroll
            for (int i = 0; i < QL; ++i) {
                const int c = Cfg::kQShared ? warp + i * kWarps : i;
                uint2 x = make_uint2(0, 0);
                if (r < n_rows && c < NC) x = *reinterpret_cast<const uint2*>(row + 16 * c);
                qf[n * QL + i] = x;
            }
        }
    };
    // bf16 rows become fp16 by the power of two that brings the row's largest element to
    // 2^14 .. 2^15: exactly, where an element is within 28 octaves of it (so far down fp16
    // has normal numbers); smaller ones are rounded to multiples of 2^-38 of it at most.
    auto begin_sequence = [&]() PA_INLINE_LAMBDA {
        seq_L = s_len[b];
        row0 = s_row[b];
        const int T = tokens_of(b);
        seq_end0 = seq_L - T + 1;
        seq_rows = T * p.G;
#pragma unroll
        for (int n = 0; n < NT; ++n) crow[n][0] = crow[n][1] = p.scale_log2;
        if (Cfg::kQShared) __syncthreads();  // (the previous sequence's q and xbuf are done with)
        if (p.bf16) {
            float most[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                most[n] = 0.f;
#pragma unroll
                for (int i = 0; i < QL; ++i) {
                    const uint2 x = qf[n * QL + i];
                    most[n] = fmaxf(most[n], fmaxf(fabsf(__uint_as_float(x.x << 16)),
                                                   fabsf(__uint_as_float(x.x & 0xffff0000u))));
                    most[n] = fmaxf(most[n], fmaxf(fabsf(__uint_as_float(x.y << 16)),
                                                   fabsf(__uint_as_float(x.y & 0xffff0000u))));
                }
                most[n] = fmaxf(most[n], __shfl_xor_sync(0xffffffffu, most[n], 1));
                most[n] = fmaxf(most[n], __shfl_xor_sync(0xffffffffu, most[n], 2));
            }
            if (Cfg::kQShared) {
                if (t == 0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) s_qmax[warp * Cfg::kRows + 8 * n + g] = most[n];
                }
                __syncthreads();
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        most[n] = fmaxf(most[n], s_qmax[w * Cfg::kRows + 8 * n + g]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // (a row of zeros or of the least numbers: as if its largest were 2^-110)
                const int e = max((int)(__float_as_uint(most[n]) >> 23) - 127, -110);
                const float f = __uint_as_float((uint32_t)(14 - e + 127) << 23);
                const float back = __uint_as_float((uint32_t)max(e - 14 + 127, 1) << 23);
#pragma unroll
                for (int i = 0; i < QL; ++i) {
                    const uint2 x = qf[n * QL + i];
                    qf[n * QL + i] = make_uint2(
                        q8_pack(__uint_as_float(x.x << 16) * f,
                                __uint_as_float(x.x & 0xffff0000u) * f),
                        q8_pack(__uint_as_float(x.y << 16) * f,
                                __uint_as_float(x.y & 0xffff0000u) * f));
                }
                // row g's factor, for the lanes that have it as column 2 t or 2 t + 1
                const float mine = p.scale_log2 * back;
                crow[n][0] = __shfl_sync(0xffffffffu, mine, 8 * t);
                crow[n][1] = __shfl_sync(0xffffffffu, mine, 8 * t + 4);
            }
        }
        if (Cfg::kQShared) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < QL; ++i)
                    if (warp + i * kWarps < NC)
                        s_q[(n * NC + warp + i * kWarps) * 32 + lane] = qf[n * QL + i];
            if (warp == 0 && g == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n) s_c[4 * n + t] = make_float2(crow[n][0], crow[n][1]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][c][i] = 0.f;
            m[n][0] = m[n][1] = kQ8NoMax;
            l[n][0] = l[n][1] = 0.f;
        }
        vref = 0.f;
        bad = dead;
    };

    // This lane's place in an ldmatrix: token and half of a pair of chunks.
    const int lm_row = (lane & 7) + (lane & 8), lm_half = lane >> 4;

    // ---- What a page needs before its products where some of its tokens are hidden
    // from some rows (their cells may hold anything): V's rows of tokens that no row
    // sees become zeros, for 0 * NaN would be NaN; and where rows see different tokens, a
    // NaN among V's codes of a token that only some of them see becomes NaN in those
    // rows' sums at once (found by a product of indicators) and a zero.  Returns which
    // scores count: bit 4 n + i for score i of tile n.
    auto prepare_masked = [&](uint32_t kat, int tok0) PA_INLINE_LAMBDA {
        uint32_t seen = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * n + 2 * t + i;
                const int end = r < seq_rows ? seq_end0 + ((r * p.ginv) >> 16) : 0;
                const int begin = p.window > 0 ? end - p.window : 0;
                const int ta = tok0 + g, tb = ta + 8;
                if (ta < end && ta >= begin) seen |= 1u << (4 * n + i);
                if (tb < end && tb >= begin) seen |= 1u << (4 * n + i + 2);
            }
        const uint32_t vat = kat + PB;
        const int begin0 = p.window > 0 ? seq_end0 - p.window : 0;  // the first row's
        bool nan = false;
#pragma unroll 1
        for (int i = lane; i < 16 * NC; i += 32) {  // 16-byte chunks
            const int r = i / NC, tok = tok0 + r;
            const uint32_t at = vat + q8_chunk<D>(r, i - r * NC);
            if (tok < begin0 || tok >= seq_L)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
            else if (seq_rows > p.G) {
                uint4 x;
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                             : "r"(at)
                             : "memory");
                nan |= (q8_nan_bytes(x.x) | q8_nan_bytes(x.y) | q8_nan_bytes(x.z) | q8_nan_bytes(x.w)) != 0;
            }
        }
        __syncwarp();
        if (__any_sync(0xffffffffu, nan)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t on = seen >> (4 * n);
                const uint32_t b0 = q8_movmatrix((on & 1 ? 0x3C00u : 0u) | (on & 2 ? 0x3C000000u : 0u));
                const uint32_t b1 = q8_movmatrix((on & 4 ? 0x3C00u : 0u) | (on & 8 ? 0x3C000000u : 0u));
#pragma unroll
                for (int c = 0; c < NC; c += 2) {
                    uint32_t x[4];
                    q8_ldmatrix_trans(x, vat + q8_chunk<D>(lm_row, c + lm_half));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // (the code of 1 where there is a NaN)
                        const uint32_t ya = (q8_nan_bytes(__byte_perm(x[2 * k], 0, 0x3120)) >> 7) * 0x38u;
                        const uint32_t yb = (q8_nan_bytes(__byte_perm(x[2 * k + 1], 0, 0x3120)) >> 7) * 0x38u;
                        float d[4];
                        q8_mma0(d, q8_low(ya), q8_high(ya), q8_low(yb), q8_high(yb), b0, b1);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (d[i] > 0.f) acc[n][c + k][i] = NAN;
                    }
                }
            }
            __syncwarp();
#pragma unroll 1
            for (int i = lane; i < 16 * D / 4; i += 32) {  // (words, in whatever order they lie)
                uint32_t x;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(vat + 4 * i) : "memory");
                x &= ~((q8_nan_bytes(x) >> 7) * 0xffu);
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(vat + 4 * i), "r"(x) : "memory");
            }
            __syncwarp();
        }
        fence_proxy_async_smem();  // (a copy writes here next)
        return seen;
    };

    // ---- A page in shared memory, K at `at`, V PB behind it; `masked`: see above.
    auto page = [&](uint32_t at, float2 sc, int tok0, bool masked) PA_INLINE_LAMBDA {
        uint32_t seen = 0xffffffffu;
        if (masked) seen = prepare_masked(at, tok0);
        float s[NT][4];
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
            uint32_t x[4];
            q8_ldmatrix(x, at + q8_chunk<D>(lm_row, c + lm_half));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t a0 = q8_low(x[2 * k]), a1 = q8_low(x[2 * k + 1]);
                const uint32_t a2 = q8_high(x[2 * k]), a3 = q8_high(x[2 * k + 1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint2 q = Cfg::kQShared ? s_q[(n * NC + c + k) * 32 + lane]
                                                  : qf[Cfg::kQShared ? 0 : c + k];
                    if (c + k == 0)
                        q8_mma0(s[n], a0, a1, a2, a3, q.x, q.y);
                    else
                        q8_mma(s[n], a0, a1, a2, a3, q.x, q.y);
                }
            }
        }
        // e: the scores in the log2 domain, above the running maximum.
        float e[NT][4], most = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 by = Cfg::kQShared ? s_c[4 * n + t] : make_float2(crow[n][0], crow[n][1]);
            const float k0 = sc.x * by.x, k1 = sc.x * by.y;
#pragma unroll
            for (int i = 0; i < 4; ++i) e[n][i] = fmaf(s[n][i], i & 1 ? k1 : k0, -m[n][i & 1]);
        }
        if (masked) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!(seen >> (4 * n + i) & 1)) e[n][i] = -INFINITY;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) most = fmaxf(most, e[n][i]);
        if (__any_sync(0xffffffffu, most > kQ8Most)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // (again from the products: against no maximum yet, e has lost them)
                    const float2 by = Cfg::kQShared ? s_c[4 * n + t] : make_float2(crow[n][0], crow[n][1]);
                    const float k = sc.x * (i ? by.y : by.x);
                    const float xa = e[n][i] == -INFINITY ? -INFINITY : s[n][i] * k;
                    const float xb = e[n][i + 2] == -INFINITY ? -INFINITY : s[n][i + 2] * k;
                    float x = fmaxf(xa, xb);
#pragma unroll
                    for (int k2 = 4; k2 < 32; k2 <<= 1)
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k2));
                    const float top = fmaxf(m[n][i], x - kQ8Room);
                    const float f = ex2(m[n][i] - top);
                    m[n][i] = top;
                    e[n][i] = xa - top;
                    e[n][i + 2] = xb - top;
                    l[n][i] *= f;
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        acc[n][c][i] *= f;
                        acc[n][c][i + 2] *= f;
                    }
                }
        }
        // The page's V scale against the reference, which only rises.
        if (!(sc.y <= vref)) {
            const float f = vref == 0.f ? 0.f : __fdividef(vref, sc.y);
            vref = sc.y;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][c][i] *= f;
        }
        const float ratio = sc.y == vref ? 1.f : __fdividef(sc.y, vref);
        const bool direct = ratio >= kQ8LeastRatio;
        const float on_weights = direct ? ratio : 1.f;
        // Weights, times the page's ratio, as two fp16 numbers each, a head and a rest: 22 bits, and
        // 2^-33 of the greatest at least.  P^T's fragments are S^T's, each 8 x 8 block transposed.
        // (Heads alone, 11 bits, move rows across roundings' borders.  The rests cost nothing with
        // one tile of rows; with two 32 ragged sequences of four queries, head_dim 96, go 24.5 ->
        // 26.5 us, 16 of two, 128, stay at 49.1; with three 16 of five behind a window of 4096 go
        // 41.8 -> 46.9, with four 16 of eight 91.6 -> 102.6: 8 cycles a product.)
        uint32_t b0[NT][2], b1[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ex2(e[n][i]);
            l[n][0] += w[0] + w[2];
            l[n][1] += w[1] + w[3];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] *= on_weights;
            const uint32_t ha = q8_pack(w[0], w[1]), hb = q8_pack(w[2], w[3]);
            const float2 fa = q8_unpack(ha), fb = q8_unpack(hb);
            b0[n][0] = q8_movmatrix(ha);
            b1[n][0] = q8_movmatrix(hb);
            b0[n][1] = q8_movmatrix(q8_pack(w[0] - fa.x, w[1] - fa.y));
            b1[n][1] = q8_movmatrix(q8_pack(w[2] - fb.x, w[3] - fb.y));
        }
        // V: tokens 2 t, 2 t + 1 and 8 on, dims 2 g and 2 g + 1 of a chunk.
        auto products = [&](auto straight) PA_INLINE_LAMBDA {
            constexpr bool STRAIGHT = decltype(straight)::value;
#pragma unroll
            for (int c = 0; c < NC; c += 2) {
                uint32_t x[4], a[2][4];
                q8_ldmatrix_trans(x, at + PB + q8_chunk<D>(lm_row, c + lm_half));
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t ya = __byte_perm(x[2 * k], 0, 0x3120);
                    const uint32_t yb = __byte_perm(x[2 * k + 1], 0, 0x3120);
                    a[k][0] = q8_low(ya), a[k][1] = q8_high(ya);
                    a[k][2] = q8_low(yb), a[k][3] = q8_high(yb);
                }
                if constexpr (STRAIGHT) {  // (rests first: two products of one sum lie far apart)
#pragma unroll
                    for (int h = 1; h >= 0; --h)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                q8_mma(acc[n][c + k], a[k][0], a[k][1], a[k][2], a[k][3], b0[n][h], b1[n][h]);
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float d[4];
                            q8_mma0(d, a[k][0], a[k][1], a[k][2], a[k][3], b0[n][1], b1[n][1]);
                            q8_mma(d, a[k][0], a[k][1], a[k][2], a[k][3], b0[n][0], b1[n][0]);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[n][c + k][i] = fmaf(ratio, d[i], acc[n][c + k][i]);
                        }
                }
            }
        };
        if (direct)
            products(std::true_type{});
        else
            products(std::false_type{});
    };

    const int group = blockIdx.y;
    const size_t wrow0 = ((size_t)group * p.X + blockIdx.x) * 2;
    // ---- The end of sequence b in this CTA.  Sequences that a border cuts (at
    // most two) are noted.  The one at the range's head is counted at once,
    // long before the CTA that has its front gets there; thread 0 looks at the
    // count when it is done.
    int cut_head = -1, cut_tail = -1, head_count = 0;
    unsigned* counters = p.counters + (size_t)group * p.B;
    auto end_sequence = [&]() PA_INLINE_LAMBDA {
        const bool cut = !kCluster && (s_base[b] < lo || s_base[b + 1] > hi);
        const bool tail = s_base[b] + kQ8Start * (s_rank[b] + 1) > from;
        const size_t wrow = wrow0 + (tail ? 1 : 0);
        if (cut) (tail ? cut_tail : cut_head) = b;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], k);
                if (bad) l[n][i] = NAN;
            }
        __syncthreads();  // the last use of xbuf and s_ml is over
        if (g == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    s_ml[warp * Cfg::kRows + 8 * n + 2 * t + i] = make_float2(m[n][i], l[n][i]);
        }
        __syncthreads();
        // A lane for each row: maximum and sum over the warps, and this warp's factor, its share
        // of a weight of 1: times the greatest V scale only then, for that may be next to fp32's
        // end.  (A sum of 0: the warp had no page.  NaN is kept.)
        float top = -INFINITY, sum = 0.f, own = 0.f;
        {
            float2 ml[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ml[w] = s_ml[w * Cfg::kRows + min(lane, Cfg::kRows - 1)];
                if (ml[w].y != 0.f) top = fmaxf(top, ml[w].x);
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ml[w].y == 0.f ? 0.f : (ml[w].y != ml[w].y ? NAN : ex2(ml[w].x - top));
                sum += f * ml[w].y;
                if (w == warp) own = f;
            }
            own *= q8_inverse(sum);
        }
        if (warp == 0 && lane < seq_rows) {
            if (kCluster)
                s_sum[lane] = make_float2(top, sum);
            else if (!cut)
                q8_store_lse(p, row0, h0, lane, top, sum);
            else
                reinterpret_cast<float2*>(p.ws_ml)[wrow * Cfg::kRows + lane] = make_float2(top, sum);
        }
        // Tile by tile the warps' shares meet in shared memory; a warp adds up units of it.
        // (Rolled: this runs once a sequence, from instructions that have to be fetched.)
#pragma unroll 1
        for (int n = 0; n < NT; ++n) {
            if (n > 0) __syncthreads();
            const float f0 = __shfl_sync(0xffffffffu, own, 8 * n + 2 * t);
            const float f1 = __shfl_sync(0xffffffffu, own, 8 * n + 2 * t + 1);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if (i != n) continue;
#pragma unroll
                for (int u = 0; u < Cfg::kTileUnits; ++u) {
                    const int c = u >> 1 << 1, k = u & 1;
                    const float f = k ? f1 : f0;
                    xbuf[(u * kWarps + warp) * 32 + lane] =
                        make_float4(acc[i][c][k] * f * vref, acc[i][c][2 + k] * f * vref,
                                    acc[i][c + 1][k] * f * vref, acc[i][c + 1][2 + k] * f * vref);
                }
            }
            __syncthreads();
#pragma unroll 1
            for (int u = warp; u < Cfg::kTileUnits; u += kWarps) {
                const int r = 8 * n + 2 * t + (u & 1), un = n * Cfg::kTileUnits + u;
                if (r >= seq_rows) continue;
                float4 o = xbuf[u * kWarps * 32 + lane];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 v = xbuf[(u * kWarps + w) * 32 + lane];
                    o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
                }
                if (!cut && !kCluster)
                    q8_store_unit<D, NT>(p, row0, h0, un, lane, o);
                else if (kCluster)  // (the ring is idle: this is the range's end)
                    reinterpret_cast<float4*>(ring)[un * 32 + lane] = o;
                else
                    reinterpret_cast<float4*>(p.ws_o)[(wrow * Cfg::kUnits + un) * 32 + lane] = o;
            }
        }
        if (cut && !tail && !p.merge_kernel) {
            __syncthreads();
            if (threadIdx.x == 0) head_count = q8_arrive(counters + b);
        }
    };

    // ---- The range, kStaged pages at a time.  Pages go to the warps in turn; a warp's
    // copies take its ring slots round.
    constexpr int SB = Cfg::kSlotBytes;
    int in_slot = 0, out_slot = 0;    // ring slots of the next copy and of the next page
    uint32_t out_phase = 0;
    int pending = 0;                  // slots requested and not yet waited for
    int stall = p.stall_tx;
    bool have = false;   // the registers hold sequence b
    int next = b;        // the sequence whose turn it is at the next border, -1: none
    bool border = true;  // a sequence ends or the first begins
    for (int c0 = lo; c0 < hi; c0 += Cfg::kStaged) {
        const int c1 = min(hi, c0 + Cfg::kStaged);
        __syncthreads();  // the previous stretch's ids have been used
        bool bad_id = false;
        int mine[kIds];
#pragma unroll
        for (int i = 0; i < kIds; ++i) {
            const int f = c0 + tid + i * kThreads;
            mine[i] = -1;
            if (f >= c1) continue;
            int id = again || c0 != lo ? *table_entry(f) : ids[i];
            if (id < 0 || id >= p.num_pages) {
                id = -1;
                bad_id = true;
            }
            mine[i] = id;
            s_pid[f - c0] = id < 0 ? -1 : (id * p.Hkv + kvh) * kPageSize;  // (below 2^31: checked)
        }
        if (bad_id) atomicOr(p.err, PA_DEVERR_BAD_PAGE);
        __syncthreads();

        int ask = warp;  // page (from c0) of the next request
        const int n_ids = c1 - c0;
        auto request = [&]() PA_INLINE_LAMBDA {
            if (lane == 0) {
                const uint32_t bar = bar_w + in_slot * 8, dst = ring_u + in_slot * SB;
                const int row = s_pid[ask];
                mbar_arrive_expect_tx(bar, (row >= 0 ? 2 * PB : 0) + stall);
                if (row >= 0) {
                    q8_load_page<D>(dst, &maps.k, row, bar);
                    q8_load_page<D>(dst + PB, &maps.v, row, bar);
                }
                stall = 0;
            }
            ask += kWarps;
            in_slot = in_slot + 1 == NS ? 0 : in_slot + 1;
            ++pending;
        };
        // Scales and the first q are asked for before the first pages: behind them they
        // would wait for all that the ring holds.
        float2 scales[kIds];
#pragma unroll
        for (int i = 0; i < kIds; ++i)
            if (mine[i] >= 0) {
                const size_t at = (size_t)mine[i] * p.Hkv + kvh;
                scales[i] = make_float2(__ldcg(p.k_scales + at), __ldcg(p.v_scales + at));
            }
        if (border && next >= 0) load_q(next);
        if (!dead) {
#pragma unroll 1
            for (int i = 0; i < NS && ask < n_ids; ++i) request();
        }
        bool staged = false;

        int f = dead ? c1 : c0 + warp;  // next page of this warp
        while (true) {
            if (border && next >= 0 && staged) load_q(next);
            if (!staged) {
#pragma unroll
                for (int i = 0; i < kIds; ++i)
                    if (mine[i] >= 0) s_sc[tid + i * kThreads] = scales[i];
                __syncthreads();
                staged = true;
            }
            if (border) {
                if (have) end_sequence();
                if (next < 0) break;
                b = next;
                begin_sequence();
                have = true;
                border = false;
            }
            const int seg_end = min(c1, s_base[b + 1]);
            // Pages that all rows see whole lie in [whole0, whole1).
            const int base = -s_page0[b];  // page of token 0
            const int begin = p.window > 0 ? max(0, seq_L - p.window) : 0;  // the last row's
            const int whole0 = base + (begin + kPageSize - 1) / kPageSize;
            const int whole1 = base + max(seq_end0, 0) / kPageSize;
            while (f < seg_end) {
                // The page is there (or the wait for it ran out).
                const uint32_t bar = bar_w + out_slot * 8;
                const float2 sc = s_sc[f - c0];
                const int row = s_pid[f - c0];
                if (!__all_sync(0xffffffffu, mbar_try_wait(bar, out_phase)) &&
                    !__all_sync(0xffffffffu, mbar_wait_bounded(bar, out_phase))) {
                    if (lane == 0) atomicOr(p.err, PA_DEVERR_TIMEOUT);
                    dead = bad = true;
                    f = c1;
                    break;
                }
                if (row < 0)
                    bad = true;
                else
                    page(ring_u + out_slot * SB, sc, (f - base) * kPageSize,
                         f < whole0 || f >= whole1);
                f += kWarps;
                --pending;
                __syncwarp();  // every lane has read the slot
                if (ask < n_ids) request();
                if (++out_slot == NS) {
                    out_slot = 0;
                    out_phase ^= 1;
                }
            }
            if (s_base[b + 1] > c1 && c1 < hi) break;  // goes on in the next stretch
            border = true;
            if (s_base[b + 1] >= hi) {  // the range's last
                next = -1;
                continue;
            }
            next = b + 1;
            while (s_base[next + 1] == s_base[next]) ++next;
            if (s_base[next] >= c1) break;  // begins in the next stretch
        }
    }
    if constexpr (kCluster) {
        // The state of every CTA with pages is in its ring and s_sum; each warp of
        // the cluster merges units of all of them, whose reads go out together.
        // The second barrier keeps the shared memory until all have read it.
        __syncthreads();
        q8_cluster_barrier();
        const int rank = blockIdx.x - b * p.cluster;
        const int rows = (s_base[b + 1] - s_base[b] + range - 1) / range;
#pragma unroll 1
        for (int u = rank * kWarps + warp; u < Cfg::kUnits; u += p.cluster * kWarps) {
            const int r = q8_unit_row<D, NT>(u, lane), n_rows = tokens_of(b) * p.G;
            Q8Merge mg;
            constexpr int N = 8;  // peers in flight
            for (int r0 = 0; r0 < rows; r0 += N) {
                float2 ml[N];
                float4 v[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    ml[i] = make_float2(-INFINITY, 0.f);
                    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (r0 + i < rows && r < n_rows) {
                        ml[i] = q8_ld_peer2(q8_peer(s_sum + r, r0 + i));
                        v[i] = q8_ld_peer4(q8_peer(ring + (u * 32 + lane) * 16, r0 + i));
                    }
                }
                mg.add(ml, v);
            }
            q8_finish_unit<D, NT>(p, s_row[b], n_rows, h0, u, lane, mg);
        }
        q8_cluster_barrier();
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
    // (behind the loop: in it the merge's loads in flight make accumulators spill)
    if (cut_head < 0 && cut_tail < 0) return;
    __syncthreads();
    if (threadIdx.x == 0) {
        auto last = [&](int c, int before) {
            const bool is = before == Q8Rows(range, s_base[c], s_base[c + 1], s_rank[c]).n - 1;
            if (is) counters[c] = 0;  // ready for the next call
            return is;
        };
        s_red[0] = cut_head >= 0 && last(cut_head, head_count);
        s_red[1] = cut_tail >= 0 && last(cut_tail, q8_arrive(counters + cut_tail));
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int c = i == 0 ? cut_head : cut_tail;
        if (!s_red[i]) continue;
        const Q8Rows rows(range, s_base[c], s_base[c + 1], s_rank[c]);
#pragma unroll 1
        for (int u = warp; u < Cfg::kUnits; u += kWarps) {
            const int n_rows = tokens_of(c) * p.G;
            Q8Merge mg;
            if (q8_unit_row<D, NT>(u, lane) < n_rows)
                q8_merge_run<D, NT, 4>(p, rows, group, u, lane, 0, 1, mg);
            q8_finish_unit<D, NT>(p, s_row[c], n_rows, h0, u, lane, mg);
        }
    }
}

// The kernel's shared memory limit raised to what the largest batch asks for.
template <int D, int NT, bool kCluster>
cudaError_t q8_attend_attributes() {
    return cudaFuncSetAttribute(q8_attend_kernel<D, NT, kCluster>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Q8Cfg<D, NT>::smem(4096));
}

// Clusters of c CTAs that the current device holds at once.
template <int D, int NT>
cudaError_t q8_attend_clusters(int c, int batch, int* held) {
    cudaError_t e = q8_attend_attributes<D, NT, true>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Q8Cfg<D, NT>::smem(batch);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(held, q8_attend_kernel<D, NT, true>, &cfg);
}

template <int D, int NT>
cudaError_t launch_q8_attend(const Q8AttendParams& p, const Q8Maps& maps, dim3 grid,
                             cudaStream_t stream) {
    // The kernel's shared-memory limit, raised once per device to the most a
    // plan can ask for.
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!bit || !(done.load() & bit)) {
        e = q8_attend_attributes<D, NT, false>();
        if (e == cudaSuccess) e = q8_attend_attributes<D, NT, true>();
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Q8Cfg<D, NT>::smem(p.B);
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
    e = p.cluster ? cudaLaunchKernelEx(&cfg, q8_attend_kernel<D, NT, true>, p, maps)
                  : cudaLaunchKernelEx(&cfg, q8_attend_kernel<D, NT, false>, p, maps);
    if (e != cudaSuccess || !p.merge_kernel) return e;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(p.B, grid.y, Q8Cfg<D, NT>::kUnits);
    cfg.blockDim = dim3(kQ8MergeWarps * 32);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, q8_merge_kernel<D, NT>, p);
}

// Shared memory of a CTA, and CTAs per SM that the registers allow.
template <int D, int NT>
void q8_attend_size(int batch, int* smem, int* most) {
    *smem = Q8Cfg<D, NT>::smem(batch);
    *most = Q8Cfg<D, NT>::kMinBlocks;
}

// What pa_q8_api.cu calls of an instance.
struct Q8Instance {
    cudaError_t (*launch)(const Q8AttendParams&, const Q8Maps&, dim3, cudaStream_t);
    cudaError_t (*clusters)(int, int, int*);
    void (*size)(int, int*, int*);
};

template <int D, int NT>
constexpr Q8Instance q8_instance() {
    return {launch_q8_attend<D, NT>, q8_attend_clusters<D, NT>, q8_attend_size<D, NT>};
}

extern const Q8Instance kQ8D64[4], kQ8D96[4], kQ8D128a[2], kQ8D128b[2], kQ8D256[2];

}  // namespace pa
