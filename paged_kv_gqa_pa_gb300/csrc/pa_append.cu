// pa_append.cu -- new rows of q, K and V normalised, rotated and appended to the
// paged cache, of 16 or 32 bits (pa_append) or of 8 (pa_q8_append), and rows of the
// 8-bit cache read back (pa_q8_read); include/pa_q8.h.
//
// A lane has two runs of 16 bytes of a head's row whose elements are rotation
// partners (i and i + R / 2), or that lie side by side behind dim R; the lanes of a
// row, a power of two of them, sum its squares by shuffles.  Everything between
// load and store stays in registers.
//
// Three kernels put rows away.  Few tokens, or small ones: threads for each token, whose loads
// go out before the angles are worked out (64 tokens of 32 + 2 x 8 heads of 128 3.5 us, the
// launch and three dependent reads; 16384 of 16 + 2 x 4 39.4, 0.75 of the copy rate: bound by
// instructions).  Many large ones: rings in shared memory (16384 tokens of 24 + 2 x 4 heads of
// 256, bf16: 84.6 us, 0.94 of the copy rate).  8 bits: tiles of rows (the same tokens and their
// read back 113 us, about 63 of them q's rows, 31 the runs', which are bound by instructions:
// norm, angles, the largest, codes; 19 the reading, bound by latency).
#include <float.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "../../include/pa_q8.h"
#include "pa_common.cuh"
#include "pa_rope.cuh"

namespace pa {

constexpr int kAppendThreads = 256;  // at most, of pa_append
constexpr int kMaxTileBytes = 48 << 10;  // of rows that a CTA holds at a time
// Tokens whose q a CTA beside 8-bit runs serves, at most (16384 tokens of 8 + 2 x 2 heads of 64,
// appended and read back: 1 26.1 us, 4 18.2, 8 the same).
constexpr int kQTokens = 4;
// Tiles have 16 rows where that makes so many of them, times KV heads, times two; see append_call.
constexpr int kAppendTiles = 38;
// Runs of a tile from which they are served side by side (a step of 64 sequences, 32 + 2 x 8
// heads of 128, with the q rows and read back: 6.9 -> 6.1 us, of 776 with 16 + 2 x 4 14.1 -> 9.2,
// of 6615 with 48 + 2 x 8 of 64 194 -> 61; two runs of a prompt's chunks are faster one after
// the other, 7707 rows 72.5 and 79.7).  That path's registers cost the others: 4093 rows of
// 16 + 2 x 4 heads of 96 in chunks, with their read back, 14.4 -> 16.0 us.
constexpr int kSideBySide = 3;
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
    int q_shift, q_tokens;  // of the other CTAs: log2 of the threads for a token's q, tokens
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
        const float2 f2 = make_float2(f, f);
        auto times = [&](float* v, const float* by) {
            const float4 w4 = *reinterpret_cast<const float4*>(by);
            const float2 lo = __fmul2_rn(__fmul2_rn(make_float2(v[0], v[1]), f2), make_float2(w4.x, w4.y));
            const float2 hi = __fmul2_rn(__fmul2_rn(make_float2(v[2], v[3]), f2), make_float2(w4.z, w4.w));
            v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
        };
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            times(x + j, w + d0 + j);
            times(y + j, w + d1 + j);
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

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Cosine and sine of position * frequency.  The product modulo 2^64 is the angle modulo one
// turn.  Its quarters are taken off first, so that at most an eighth of a turn goes to fp32
// (half a step: 2^-28 of a turn; without that 2^-26 next to half a turn), x half turns, and to
// the Taylor series of sin(pi x) and cos(pi x), whose next terms are below 2^-28 there.  Both
// are then off by 2^-23.6 at most.  (By sincospif of the same x: the same, and a step of 776
// sequences of 16 + 2 x 4 heads stored and read back 9.9 -> 10.2 us.)
__device__ __forceinline__ void append_angle(int pos, unsigned long long freq, float& cs, float& sn) {
    // (an eighth further: the top two bits are the nearest quarter)
    const uint32_t turn = (uint32_t)(((unsigned long long)(long long)pos * freq) >> 32) + 0x20000000u;
    const float x = (float)((int)(turn & 0x3fffffffu) - 0x20000000) * 4.656612873077393e-10f;  // 2^-31
    const float z = x * x;
    float s = fmaf(z, 0.0821458866f, -0.599264529f);
    s = fmaf(z, fmaf(z, s, 2.55016404f), -5.16771278f);
    s = fmaf(x, 3.14159274f, x * fmaf(z, s, -8.74227766e-8f));  // (pi as two numbers)
    float c = fmaf(z, -0.0258068913f, 0.235330630f);
    c = fmaf(z, fmaf(z, fmaf(z, c, -1.33526277f), 4.05871213f), -4.93480220f);
    c = fmaf(z, c, 1.f);
    const bool odd = turn & 0x40000000u;
    cs = __uint_as_float(__float_as_uint(odd ? s : c) ^ ((turn + 0x40000000u) & 0x80000000u));
    sn = __uint_as_float(__float_as_uint(odd ? c : s) ^ (turn & 0x80000000u));
}

// A token's slot, -1 where its K and V are left out; reported by `tell`.
__device__ __forceinline__ long long append_slot(const AppendParams& p, long long s, bool tell) {
    const bool bad = s < -1 || s >= p.num_slots;
    if (bad && tell && p.err) atomicOr(p.err, PA_DEVERR_BAD_SLOT);
    return bad ? -1 : s;
}

// What a CTA of TOKENS tokens has in shared memory.
template <int D, int TOKENS>
struct AppendShared {
    alignas(16) float cos[TOKENS][D / 2];
    alignas(16) float sin[TOKENS][D / 2];
    alignas(16) float w[2][D];  // norm weights of q and k
};

// The q heads of token t, or all its heads (ALL: q's, K's, then V's, into the cache too), by
// nt threads, ITEMS of whose items are requested before the wait for the angles; of the CTA's
// tokens this one has number `part`.
template <int D, typename T, bool ALL, int ITEMS, int TOKENS>
__device__ __forceinline__ void append_token(const AppendParams& p, long long t, int part, int tid,
                                             int nt, AppendShared<D, TOKENS>& sh) {
    using Rw = RowLanes<D, T>;
    using E = RopeElem<T>;
    constexpr int N = Rw::N, ES = Rw::ES, L = Rw::kLanes;
    const bool real = TOKENS == 1 || t < p.n;  // (behind the last token: only the barrier)
    if (!real) t = 0;
    const int all_rows = p.Hq + (ALL ? 2 * p.Hkv : 0), n_rows = real ? all_rows : 0;
    const int items = all_rows * L;
    const int c = tid % L;  // (nt is a multiple of 32)
    const bool has_lane = c < Rw::kHave;
    const int d0 = Rw::first(c, p.R), d1 = Rw::second(c, p.R);
    const bool turn = c < p.R / (2 * N);
    const long long slot = ALL ? append_slot(p, p.slots[t], real && tid == 0) : -1;
    for (int i0 = 0; i0 < items; i0 += ITEMS * nt) {
        uint4 a[ITEMS], b[ITEMS];
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
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
            if (p.R > 0 && real) {
                const int pos = p.positions[t];
                for (int i = tid; i < p.R / 2; i += nt)
                    append_angle(pos, p.freq[i], sh.cos[part][i], sh.sin[part][i]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
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
                    const float cs = sh.cos[part][c * N + j], sn = sh.sin[part][c * N + j];
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

// TOKENS tokens a CTA, nt threads for each.  (Four CTAs an SM: 512 tokens of 32 + 2 x 8 heads
// 5.15 us, five, with fewer registers, 5.53.)
template <int D, typename T, int ITEMS, int TOKENS>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(const AppendParams p, const int nt) {
    __shared__ AppendShared<D, TOKENS> sh;
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    if (TOKENS == 1) {
        append_token<D, T, true, ITEMS>(p, blockIdx.x, 0, threadIdx.x, blockDim.x, sh);
    } else {
        const int part = threadIdx.x / nt;
        append_token<D, T, true, ITEMS>(p, (long long)blockIdx.x * TOKENS + part, part,
                                        threadIdx.x - part * nt, nt, sh);
    }
}

// ---- Many tokens: persistent CTAs whose groups of four warps each have a ring of tokens in
// shared memory, filled by bulk copies.

// (16384 tokens of 16 KB: 3 groups with 96 KB on their way 85 us, 4 groups with 128 KB 92, with
// 256 KB 94: more on their way is slower.)
constexpr int kRingGroups = 3;     // groups of a CTA
constexpr int kRingThreads = 128;  // threads of a group
constexpr int kRingStages = 8;     // tokens of a group's ring, at most
constexpr int kRingFill = 96 << 10;  // bytes of the CTA's rings, about
// Bytes of a token's rows from which the ring pays, for a token costs its group about 1 us
// whatever its size (16384 tokens of 6 KB 53.4 us, directly 39.4; 8000 of 12 KB 36.3 and
// 43.6), and bytes of all rows (1024 tokens of 16 KB 8.3 us, directly 10.1; 4 MB 5.8 and 4.5).
// For the q rows of pa_q8_append it is one more launch (2048 tokens of 16 KB 25.0 us, directly
// 23.3; 4096 equal).
constexpr int kRingToken = 8 << 10;
constexpr long long kRingBytes = 12 << 20, kRingBytesQ8 = 48 << 20;

// What turns a row's pairs, weights included: (x, y) becomes (x a + y b, y c + x d) times
// the norm's factor.  Entry i is element i % N of lane i / N; four consecutive elements lie
// side by side, those of the next lane behind them.
template <int D>
struct RingTable {
    float a[D / 2], b[D / 2], c[D / 2], d[D / 2];
};

template <int D>
struct RingShared {
    alignas(16) RingTable<D> table[2][2];  // [token, alternating][q, k]
    alignas(8) uint64_t full[kRingStages];
    int dead[2];  // a copy timed out, seen at a token (alternating)
};

__device__ __forceinline__ void ring_barrier(int group) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(kRingThreads) : "memory");
}

// ALL: rows are q's, K's and V's, as in append_token; otherwise q's alone.
template <int D, typename T, bool ALL>
__global__ void __launch_bounds__(kRingGroups * kRingThreads, 1)
    append_ring_kernel(const AppendParams p, const int stages, const int token_bytes) {
    using Rw = RowLanes<D, T>;
    using E = RopeElem<T>;
    constexpr int N = Rw::N, ES = Rw::ES, L = Rw::kLanes, F = N / 2;
    constexpr int kRows = kRingThreads / L;  // rows of a pass
    extern __shared__ __align__(128) unsigned char ring_smem[];
    __shared__ RingShared<D> shared[kRingGroups];
    const int group = threadIdx.x / kRingThreads, tid = threadIdx.x % kRingThreads;
    RingShared<D>& sh = shared[group];
    unsigned char* ring = ring_smem + (size_t)group * stages * token_bytes;
    const long long step = gridDim.x * kRingGroups, t0 = blockIdx.x * kRingGroups + group;
    const uint32_t full = smem_u32(sh.full);
    allow_dependent_launch();
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(full + 8 * i, 1);
        fence_mbar_init();
        sh.dead[0] = sh.dead[1] = 0;
    }
    __syncthreads();
    // Entry tid of the tables: its pair's weights and frequency.
    const bool has_pair = tid < D / 2;
    const bool turns = tid < p.R / 2;
    const unsigned long long freq = turns ? p.freq[tid] : 0;
    const int at = (tid % N) / 4 * (D * 2 / N) + tid / N * 4 + tid % 4;  // (its place in a table)
    wait_for_prerequisite_grid();
    float w[2][2];  // [q, k][x, y]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned char* wp = i == 0 ? p.q_norm : p.k_norm;
        w[i][0] = w[i][1] = 1.f;
        if (wp && has_pair) {
            const int c = tid / N, j = tid % N;
            w[i][0] = to_float(reinterpret_cast<const T*>(wp)[Rw::first(c, p.R) + j]);
            w[i][1] = to_float(reinterpret_cast<const T*>(wp)[Rw::second(c, p.R) + j]);
        }
    }
    const uint32_t q_bytes = p.Hq * D * ES, kv_bytes = ALL ? p.Hkv * D * ES : 0;
    auto request = [&](long long t, int slot) {  // (one thread)
        const uint32_t dst = smem_u32(ring + (size_t)slot * token_bytes), bar = full + 8 * slot;
        mbar_arrive_expect_tx(bar, q_bytes + 2 * kv_bytes);
        if (q_bytes) bulk_g2s(dst, p.q + t * p.q_stride, q_bytes, bar);
        if (ALL) {
            bulk_g2s(dst + q_bytes, p.k + t * p.k_stride, kv_bytes, bar);
            bulk_g2s(dst + q_bytes + kv_bytes, p.v + t * p.v_stride, kv_bytes, bar);
        }
    };
    if (tid == 0)
        for (int i = 0; i < stages && t0 + i * step < p.n; ++i)
            request(t0 + i * step, i);
    const int n_rows = p.Hq + (ALL ? 2 * p.Hkv : 0);
    const int c = tid % L, r0 = tid / L;
    const bool has_lane = c < Rw::kHave, turn = c < p.R / (2 * N);
    const int d0 = Rw::first(c, p.R) * ES, d1 = Rw::second(c, p.R) * ES;
    int pos = 0;
    long long row_slot = -1;
    auto look = [&](long long t) {  // (a token ahead)
        if (p.R > 0) pos = p.positions[t];
        if (ALL) row_slot = p.slots[t];
    };
    if (t0 < p.n) look(t0);
    int slot = 0, before = -1, k = 0;  // ring slot, the one of the token before, tokens so far
    uint32_t phase = 0;
    bool dead = false;
    for (long long t = t0; t < p.n; t += step, ++k) {
        float cs = 1.f, sn = 0.f;
        if (turns) append_angle(pos, freq, cs, sn);
        if (has_pair) {
#pragma unroll
            for (int i = 0; i < (ALL ? 2 : 1); ++i) {
                RingTable<D>& tb = sh.table[k & 1][i];
                tb.a[at] = w[i][0] * cs, tb.b[at] = -w[i][1] * sn;
                tb.c[at] = w[i][1] * cs, tb.d[at] = w[i][0] * sn;
            }
        }
        const long long cell = ALL ? append_slot(p, row_slot, tid == 0) : -1;
        if (t + step < p.n) look(t + step);
        if (!mbar_wait_bounded(full + 8 * slot, phase)) sh.dead[k & 1] = 1;
        ring_barrier(group);
        if (sh.dead[k & 1]) {
            dead = true;
            break;
        }
        // (all are through with the token before: its slot takes the next one)
        if (tid == 0 && before >= 0 && t + step * (stages - 1) < p.n)
            request(t + step * (stages - 1), before);
        const unsigned char* rows = ring + (size_t)slot * token_bytes;
        float2 ta[F], tb[F], tc[F], td[F];
        auto table = [&](int i) {
            const RingTable<D>& s = sh.table[k & 1][i];
#pragma unroll
            for (int f = 0; f < F; f += 2) {
                const int e = f / 2 * (D * 2 / N) + c * 4;
                const float4 va = *reinterpret_cast<const float4*>(s.a + e);
                const float4 vb = *reinterpret_cast<const float4*>(s.b + e);
                const float4 vc = *reinterpret_cast<const float4*>(s.c + e);
                const float4 vd = *reinterpret_cast<const float4*>(s.d + e);
                ta[f] = make_float2(va.x, va.y), ta[f + 1] = make_float2(va.z, va.w);
                tb[f] = make_float2(vb.x, vb.y), tb[f + 1] = make_float2(vb.z, vb.w);
                tc[f] = make_float2(vc.x, vc.y), tc[f + 1] = make_float2(vc.z, vc.w);
                td[f] = make_float2(vd.x, vd.y), td[f + 1] = make_float2(vd.z, vd.w);
            }
        };
        int kind = -1;  // whose table the registers hold
#pragma unroll 1
        for (int h0 = 0; h0 < n_rows; h0 += kRows) {
            const int h = h0 + r0;
            const bool is_q = !ALL || h < p.Hq, is_v = ALL && h >= p.Hq + p.Hkv;
            const bool has = has_lane && h < n_rows && (is_q || cell >= 0);
            uint4 ra = make_uint4(0, 0, 0, 0), rb = ra;
            if (has) {
                ra = *reinterpret_cast<const uint4*>(rows + (size_t)h * (D * ES) + d0);
                rb = *reinterpret_cast<const uint4*>(rows + (size_t)h * (D * ES) + d1);
                const int want = is_q ? 0 : 1;
                if (!is_v && kind != want) {
                    table(want);
                    kind = want;
                }
            }
            float2 x[F], y[F];
            E::load(ra, reinterpret_cast<float(&)[N]>(x));
            E::load(rb, reinterpret_cast<float(&)[N]>(y));
            float factor = 1.f;
            if (p.q_norm || (ALL && p.k_norm)) {  // (the shuffles are for all rows of the warp)
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int f = 0; f < F; ++f) sum = __ffma2_rn(x[f], x[f], __ffma2_rn(y[f], y[f], sum));
                float ss = sum.x + sum.y;
#pragma unroll
                for (int m = 1; m < L; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                if (is_q ? p.q_norm : p.k_norm) factor = rsqrtf(ss * (1.f / D) + p.eps);
            }
            if (!has) continue;
            if (!is_v) {
                const float2 f2 = make_float2(factor, factor);
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    const float2 xf = __fmul2_rn(x[f], f2), yf = __fmul2_rn(y[f], f2);
                    x[f] = __fmul2_rn(xf, ta[f]);
                    y[f] = __fmul2_rn(yf, tc[f]);
                    if (turn) {
                        x[f] = __ffma2_rn(yf, tb[f], x[f]);
                        y[f] = __ffma2_rn(xf, td[f], y[f]);
                    }
                }
                ra = E::store(reinterpret_cast<const float(&)[N]>(x));
                rb = E::store(reinterpret_cast<const float(&)[N]>(y));
            }
            unsigned char* dst;
            if (is_q) {
                dst = p.q_out + t * p.q_out_stride + (size_t)h * (D * ES);
            } else {
                const size_t block = (size_t)(cell / kPageSize) * p.Hkv +
                                     (is_v ? h - p.Hq - p.Hkv : h - p.Hq);
                dst = (is_v ? p.v_cache : p.k_cache) +
                      (block * kPageSize + (int)(cell % kPageSize)) * (size_t)(D * ES);
            }
            *reinterpret_cast<uint4*>(dst + d0) = ra;
            *reinterpret_cast<uint4*>(dst + d1) = rb;
        }
        before = slot;
        if (++slot == stages) {
            slot = 0;
            phase ^= 1;
        }
    }
    if (dead && tid == 0) {  // (copies on their way must not outlive the shared memory)
        if (p.err) atomicOr(p.err, PA_DEVERR_TIMEOUT);
        for (int i = 0; i < stages; ++i) mbar_wait_bounded(full + 8 * i, i < slot ? phase ^ 1 : phase);
    }
}

// ---- The 8-bit cache.

// Codes of N values times f, first one lowest (NaN stays NaN, beyond 448: 448).
template <int F>
__device__ __forceinline__ void q8_codes(const float2 (&x)[F], float f, uint32_t (&c)[F / 2]) {
    const float2 f2 = make_float2(f, f);
#pragma unroll
    for (int j = 0; j < F; j += 2) {
        const float2 a = __fmul2_rn(x[j], f2), b = __fmul2_rn(x[j + 1], f2);
        asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n"
            " cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}"
            : "=r"(c[j / 2])
            : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
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
// CTA finds the rows that begin a run (rows at consecutive slots of a page).  Several runs
// that end in the tile are served side by side, see below.  Otherwise, for each
// run and head, a thread has its two pieces of a new row, and of a row that was there
// before, if there are so many.  The largest magnitude goes through the CTA, the scale
// follows, codes are stored.  The rows of the tile come by bulk copies, asked for beside
// the slots; those of a run that goes on behind the tile (it is the tile's last) take the
// places of rows before it, which are done with.  The other CTAs serve the q of a token or
// a few.
template <int D, typename T>
__global__ void __launch_bounds__(16 * (RowLanes<D, T>::kLanes), 64 / RowLanes<D, T>::kLanes)
    q8_append_kernel(const AppendParams p) {
    using Rw = RowLanes<D, T>;
    using E = RopeElem<T>;
    constexpr int N = Rw::N, ES = Rw::ES, L = Rw::kLanes, W = N / 4, F = N / 2;
    constexpr int kWarpsHere = 16 * L / 32;
    __shared__ AppendShared<D, kQTokens> sh;
    __shared__ uint32_t s_max[2][kWarpsHere];
    __shared__ float s_row[2][kPageSize];  // rows' largest magnitudes, by turns of heads
    __shared__ unsigned long long s_freq[kMaxRopePairs];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    allow_dependent_launch();
    wait_for_prerequisite_grid();
    if ((int)blockIdx.x >= p.kv_ctas) {
        const int part = tid >> p.q_shift, nt = 1 << p.q_shift;
        const long long t = (long long)(blockIdx.x - p.kv_ctas) * p.q_tokens + part;
        // (threads that are left over: a token behind the last)
        append_token<D, T, false, 1>(p, part < p.q_tokens ? t : p.n, min(part, p.q_tokens - 1),
                                     tid & (nt - 1), nt, sh);
        return;
    }
    const int is_v = blockIdx.x & 1, group = (blockIdx.x >> 1) % p.groups;
    const long long row0 = (long long)((blockIdx.x >> 1) / p.groups) * p.tile;
    const int h0 = group * p.heads, h1 = min(p.Hkv, h0 + p.heads);
    const unsigned char* rows = is_v ? p.v : p.k;
    const long long stride = is_v ? p.v_stride : p.k_stride;
    unsigned char* cache = is_v ? p.v_cache : p.k_cache;
    float* scales = is_v ? p.v_scales : p.k_scales;
    const bool rotate = !is_v && p.R > 0, norm = !is_v && p.k_norm;
    const int i_row = tid / L, c = tid % L;  // row of a run, and lane of the row
    const bool have = c < Rw::kHave;
    const int d0 = Rw::first(c, p.R), d1 = Rw::second(c, p.R);
    const bool turn = rotate && c < p.R / (2 * N);
    // Row i of the tile, heads h0 .. h1 - 1, at i modulo 16.
    extern __shared__ __align__(128) unsigned char tile_smem[];
    __shared__ __align__(8) uint64_t s_full;
    const int row_bytes = (h1 - h0) * D * ES;
    const uint32_t full = smem_u32(&s_full);
    auto fetch = [&](int from, int to) {  // (warp 0)
        if (lane == 0) mbar_arrive_expect_tx(full, (to - from) * row_bytes);
        __syncwarp();
        if (from + lane < to)
            bulk_g2s(smem_u32(tile_smem) + (from + lane) % kPageSize * row_bytes,
                     rows + (row0 + from + lane) * stride + (size_t)h0 * D * ES, row_bytes, full);
    };
    if (warp == 0) {
        if (lane == 0) {
            mbar_init(full, 1);
            fence_mbar_init();
        }
        __syncwarp();
        fetch(0, (int)min((long long)p.tile, p.n - row0));
    }
    uint32_t phase = 0;
    auto arrived = [&]() {  // (every thread; false: the wait ran out)
        const bool late = !mbar_wait_bounded(full, phase);
        if (late) {  // (a copy on its way must not outlive the shared memory)
            if (p.err) atomicOr(p.err, PA_DEVERR_TIMEOUT);
            mbar_wait_bounded(full, phase);
        }
        phase ^= 1;
        return !__syncthreads_or(late);
    };
    const int first_pos = rotate && row0 + i_row < p.n ? p.positions[row0 + i_row] : 0;
    // Lane j looks at row row0 - 1 + j: runs begin at lanes 1 .. tile and have at most 16
    // rows.
    const long long at = row0 - 1 + lane;
    long long slot = -1;
    if (at >= 0 && at < p.n)
        slot = append_slot(p, p.slots[at], !is_v && group == 0 && warp == 0 && lane >= 1 && lane <= p.tile);
    if (norm) Rw::stage(p.k_norm, sh.w[1]);
    if (rotate)
        for (int i = tid; i < p.R / 2; i += blockDim.x) s_freq[i] = p.freq[i];
    __syncthreads();  // (the barrier's initial state as well)
    const long long before = __shfl_up_sync(0xffffffffu, slot, 1);
    const bool goes_on = lane > 0 && slot >= 0 && before >= 0 && slot == before + 1 &&
                         slot % kPageSize != 0;
    const uint32_t on = __ballot_sync(0xffffffffu, goes_on);
    uint32_t leads = __ballot_sync(0xffffffffu, slot >= 0 && !goes_on && lane >= 1 && lane <= p.tile);
    // Rows of the last run behind the tile; fetched at once where no other run is in the
    // way, else when the others are done.
    const int last = 31 - __clz(leads);
    const int last_end = leads ? last - 1 + __ffs(~(last == 31 ? 0u : on >> (last + 1))) : 0;
    bool behind = last_end > p.tile;
    if (!arrived()) return;
    if (!leads) return;
    // A row of the run (x, y) normalised and rotated.
    float2 cs[F], sn[F];
    auto angles = [&](int pos) {
#pragma unroll
        for (int i = 0; i < F; ++i) {
            append_angle(pos, s_freq[c * N + 2 * i], cs[i].x, sn[i].x);
            append_angle(pos, s_freq[c * N + 2 * i + 1], cs[i].y, sn[i].y);
        }
    };
    float2 x[F], y[F];
    auto load_row = [&](const unsigned char* from, bool fresh) {  // (the whole warp)
        float(&xs)[N] = reinterpret_cast<float(&)[N]>(x);
        float(&ys)[N] = reinterpret_cast<float(&)[N]>(y);
        uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
        if (fresh) {
            xa = *reinterpret_cast<const uint4*>(from + d0 * ES);
            xb = *reinterpret_cast<const uint4*>(from + d1 * ES);
        }
        E::load(xa, xs);
        E::load(xb, ys);
        if (norm) Rw::normalise(xs, ys, sh.w[1], d0, d1, fresh, p.eps);
        if (turn && fresh) {
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const float2 minus = make_float2(-sn[i].x, -sn[i].y);
                const float2 xr = __ffma2_rn(x[i], cs[i], __fmul2_rn(y[i], minus));
                y[i] = __ffma2_rn(y[i], cs[i], __fmul2_rn(x[i], sn[i]));
                x[i] = xr;
            }
        }
    };
    auto largest_here = [&]() {  // (NaN does not count)
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < F; ++i)
            most = fmaxf(fmaxf(most, fmaxf(fabsf(x[i].x), fabsf(x[i].y))),
                         fmaxf(fabsf(y[i].x), fabsf(y[i].y)));
        return most;
    };
    auto no_infinities = [&]() {
#pragma unroll
        for (int i = 0; i < F; ++i) {
            if (fabsf(x[i].x) > FLT_MAX) x[i].x = NAN;
            if (fabsf(x[i].y) > FLT_MAX) x[i].y = NAN;
            if (fabsf(y[i].x) > FLT_MAX) y[i].x = NAN;
            if (fabsf(y[i].y) > FLT_MAX) y[i].y = NAN;
        }
    };
    auto store_row = [&](unsigned char* to, float scale) {
        const float inv = __frcp_rn(scale);
        uint32_t ca[W], cb[W];
        q8_codes(x, inv, ca);
        q8_codes(y, inv, cb);
        q8_store_codes(to + d0, ca);
        q8_store_codes(to + d1, cb);
    };
    auto recode = [&](uint32_t (&k)[W], float ratio) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float2 v[2];
            uint32_t one[1];
            q8_values(k[i], reinterpret_cast<float(&)[4]>(v));
            q8_codes(v, ratio, one);
            k[i] = one[0];
        }
    };
    const uint32_t within = behind ? leads & ~(1u << last) : leads;
    if (__popc(within) >= kSideBySide) {
        // Several runs that end in the tile (a step's rows, one or a few of each sequence): the
        // lanes of a row serve it, and a share of the rows that were in its page before.
        const int j = i_row + 1;
        const uint32_t upto = leads & ((2u << j) - 1);
        const int begin = upto ? 31 - __clz(upto) : 0;  // where its run begins
        const bool mine = (within >> begin & 1) && (begin == j || (on >> j & 1));
        const bool fresh = have && mine, alone = (on >> 1 & within) == 0;  // (alone: in every run)
        const long long first = __shfl_sync(0xffffffffu, slot, begin);
        const int cnt = __ffs(~(on >> (begin + 1)));
        const int r0 = mine ? (int)(first % kPageSize) : 0;
        const size_t block0 = mine ? (size_t)(first / kPageSize) * p.Hkv : 0;
        if (turn && fresh) angles(first_pos);
        float next = r0 > 0 ? scales[block0 + h0] : 0.f;
#pragma unroll 1
        for (int h = h0; h < h1; ++h) {
            const float was = next;
            if (r0 > 0 && h + 1 < h1) next = scales[block0 + h + 1];
            unsigned char* page = cache + (block0 + h) * (size_t)(kPageSize * D);
            load_row(tile_smem + i_row * row_bytes + (h - h0) * (D * ES), fresh);
            float most;
#pragma unroll 1
            for (bool again = false;; again = true) {
                most = fresh ? largest_here() : 0.f;
#pragma unroll
                for (int m = 1; m < L; m <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
                if (again || !__any_sync(0xffffffffu, most > FLT_MAX)) break;
                no_infinities();
            }
            if (!alone) {
                float* of_rows = s_row[h & 1];
                if (c == 0) of_rows[i_row] = most;
                __syncthreads();
                if (mine)
                    for (int i = begin - 1; i < begin - 1 + cnt; ++i) most = fmaxf(most, of_rows[i]);
            }
            const float old = was > 0.f && was <= FLT_MAX ? was : 0.f;
            const float scale = fmaxf(old, q8_scale_for(most));
            if (!mine) continue;
            if (have) store_row(page + (r0 + j - begin) * D, scale);
            if (scale == old) continue;
            if (c == 0 && j == begin) scales[block0 + h] = scale;
            const float ratio = __fdiv_rn(old, scale);
            if (!have) continue;
#pragma unroll 1
            for (int r = j - begin; r < r0; r += cnt) {
                uint32_t ka[W], kb[W];
                q8_load_codes(ka, page + r * D + d0);
                q8_load_codes(kb, page + r * D + d1);
                recode(ka, ratio);
                recode(kb, ratio);
                q8_store_codes(page + r * D + d0, ka);
                q8_store_codes(page + r * D + d1, kb);
            }
        }
        if (!behind) return;
        leads = 1u << last;
        __syncthreads();  // (every thread has read the rows whose places the last run's take)
    }
    if (behind && (leads & (leads - 1)) == 0) {
        if (warp == 0) fetch(p.tile, last_end);
        if (!arrived()) return;
        behind = false;
    }
    int turn_of = 0;  // buffer of s_max
    for (; leads; leads &= leads - 1) {
        const int j = __ffs(leads) - 1;
        const uint32_t rest = j == 31 ? 0u : on >> (j + 1);
        const int cnt = __ffs(~rest);  // 1 + the rows that go on
        const long long first = __shfl_sync(0xffffffffu, slot, j), run = row0 - 1 + j;
        if (behind && j == last) {
            __syncthreads();  // (every thread has read the rows whose places these take)
            if (warp == 0) fetch(p.tile, last_end);
            if (!arrived()) return;
        }
        const int r0 = (int)(first % kPageSize);
        const bool fresh = have && i_row < cnt, kept = have && i_row < r0;
        const size_t block0 = (size_t)(first / kPageSize) * p.Hkv;
        const unsigned char* src = tile_smem + (j - 1 + i_row) % kPageSize * row_bytes;
        if (turn && fresh) angles(j == 1 ? first_pos : p.positions[run + i_row]);
        for (int h = h0; h < h1; ++h) {
            unsigned char* page = cache + (block0 + h) * (size_t)(kPageSize * D);
            uint32_t ka[W] = {}, kb[W] = {};
            if (kept) {  // (asked for now, wanted if the scale rises)
                q8_load_codes(ka, page + i_row * D + d0);
                q8_load_codes(kb, page + i_row * D + d1);
            }
            const float was = r0 > 0 ? scales[block0 + h] : 0.f;
            load_row(src + (h - h0) * (D * ES), fresh);
            auto largest = [&]() {
                const float most = largest_here();
                // over the CTA, as bits: numbers from 0 on are in the order of their bits
                uint32_t all = __reduce_max_sync(0xffffffffu, __float_as_uint(fresh ? most : 0.f));
                if (lane == 0) s_max[turn_of][warp] = all;
                __syncthreads();
                all = __reduce_max_sync(0xffffffffu, s_max[turn_of][lane % kWarpsHere]);
                turn_of ^= 1;
                return all;
            };
            uint32_t all = largest();
            if (all == 0x7F800000u) {  // an infinity somewhere: NaN in its place, and again
                no_infinities();
                all = largest();
            }
            const float old = was > 0.f && was <= FLT_MAX ? was : 0.f;
            const float scale = fmaxf(old, q8_scale_for(__uint_as_float(all)));
            if (fresh) store_row(page + (r0 + i_row) * D, scale);
            if (kept && scale != old) {
                const float ratio = __fdiv_rn(old, scale);
                recode(ka, ratio);
                recode(kb, ratio);
                q8_store_codes(page + i_row * D + d0, ka);
                q8_store_codes(page + i_row * D + d1, kb);
            }
            if (tid == 0 && scale != old) scales[block0 + h] = scale;
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

template <typename... A, typename... B>
static cudaError_t launch_step_smem(void (*kernel)(A...), dim3 grid, int threads, int smem,
                                    cudaStream_t stream, const B&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, A(args)...);
}

template <typename... A>
static cudaError_t launch_step(void (*kernel)(A...), dim3 grid, int threads, cudaStream_t stream,
                               const A&... args) {
    return launch_step_smem(kernel, grid, threads, 0, stream, args...);
}

// Tokens a group of the ring kernel holds in rows of `heads` heads; 0: not two.
template <int D, typename T>
static int ring_stages(int heads) {
    const long long token = (long long)heads * D * (int)sizeof(T);
    const long long room = 227 * 1024 - (long long)sizeof(RingShared<D>) * kRingGroups - 256;
    if (heads == 0 || room < 2 * token * kRingGroups) return 0;
    const long long want = (kRingFill + token * kRingGroups / 2) / (token * kRingGroups);
    return (int)std::max(2ll, std::min<long long>({want, room / (token * kRingGroups), kRingStages}));
}

template <int D, typename T, bool ALL>
static cudaError_t launch_ring(const AppendParams& p, cudaStream_t stream) {
    const int heads = p.Hq + (ALL ? 2 * p.Hkv : 0), stages = ring_stages<D, T>(heads);
    const int token = heads * D * (int)sizeof(T), smem = stages * token * kRingGroups;
    // The kernel's shared-memory limit, raised once per device, and the device's SMs.
    static std::atomic<int> sms[64];
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64) n = sms[dev].load();
    if (n == 0) {
        e = cudaFuncSetAttribute(append_ring_kernel<D, T, ALL>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 227 * 1024 - (int)sizeof(RingShared<D>) * kRingGroups - 256);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (dev < 64) sms[dev].store(n);
    }
    const int ctas = std::min(n, (p.n + kRingGroups - 1) / kRingGroups);
    return launch_step_smem(append_ring_kernel<D, T, ALL>, dim3(ctas), kRingGroups * kRingThreads,
                            smem, stream, p, stages, token);
}

template <int D, typename T>
static cudaError_t launch_append(const AppendParams& p, bool q8, cudaStream_t stream) {
    constexpr int L = RowLanes<D, T>::kLanes;
    const int heads = p.Hq + (q8 ? 0 : 2 * p.Hkv);
    const long long token = (long long)heads * D * (int)sizeof(T);
    const bool ring = token >= kRingToken && p.n * token >= (q8 ? kRingBytesQ8 : kRingBytes) &&
                      ring_stages<D, T>(heads) > 0;
    if (!q8) {
        if (ring) return launch_ring<D, T, true>(p, stream);
        auto direct = [&](auto kernel, int items, int tokens) {
            const int nt = std::min(kAppendThreads, (heads * L + items * 32 - 1) / (items * 32) * 32);
            return launch_step(kernel, dim3((p.n + tokens - 1) / tokens), nt * tokens, stream, p, nt);
        };
        // Few tokens: more threads for each.  Many: three items a thread, and two tokens a CTA
        // where a warp is enough for one (16384 tokens of 16 + 2 x 4 heads: D 128 two items
        // 44.5 us, three 39.4, in pairs 42.5; D 64 28.1, 23.7, 23.3; 512 tokens of 32 + 2 x 8
        // heads, D 128: two 5.2, three 5.8).
        if (p.n <= kAppendCtas) return direct(append_kernel<D, T, 2, 1>, 2, 1);
        if (heads * L <= 2 * 32) return direct(append_kernel<D, T, 2, 2>, 2, 2);
        if (heads * L <= 3 * 32) return direct(append_kernel<D, T, 3, 2>, 3, 2);
        return direct(append_kernel<D, T, 3, 1>, 3, 1);
    }
    // (a tile's rows: at most kMaxTileBytes, see append_call)
    static std::atomic<unsigned long long> raised{0};  // the shared-memory limit, by device
    const int smem = kPageSize * p.heads * D * (int)sizeof(T);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !(raised.load() >> dev & 1))) {
        e = cudaFuncSetAttribute(q8_append_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMaxTileBytes);
        if (e == cudaSuccess && dev < 64) raised.fetch_or(1ull << dev);
    }
    if (e != cudaSuccess) return e;
    AppendParams with_q = p;
    with_q.q_shift = 5;
    while (2 << with_q.q_shift <= 16 * L && 1 << with_q.q_shift < heads * L) ++with_q.q_shift;
    int q_ctas = 0;
    if (heads > 0 && !ring) {
        with_q.q_tokens = std::min(kQTokens, 16 * L >> with_q.q_shift);
        q_ctas = (p.n + with_q.q_tokens - 1) / with_q.q_tokens;
    }
    e = launch_step_smem(q8_append_kernel<D, T>, dim3(p.kv_ctas + q_ctas), 16 * L, smem, stream, with_q);
    return e == cudaSuccess && ring ? launch_ring<D, T, false>(p, stream) : e;
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
    const bool rotate = theta != 0.f, has_q = num_q_heads > 0;
    if (!has_q) q_norm = nullptr;
    const bool norm = q_norm || k_norm;
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
    p.q_norm = static_cast<const unsigned char*>(q_norm);
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
        // Tiles of 16 rows but for the smallest calls (300 rows of 8 + 2 heads of 96: from 152
        // CTAs on 6.2 us, from 38 5.4), whose runs get a CTA each; as many heads in one CTA as
        // leave kAppendCtas of them, so that angles are worked out once for several.
        const long long tiles16 = ((long long)num_tokens + 15) / 16;
        p.tile = tiles16 * 2 * num_kv_heads >= kAppendTiles ? 16 : 1;
        const long long tiles = p.tile == 16 ? tiles16 : num_tokens;
        p.heads = (int)std::max(1ll, std::min<long long>(num_kv_heads,
                                                         tiles * 2 * num_kv_heads / kAppendCtas));
        p.heads = std::min(p.heads, kMaxTileBytes / (kPageSize * head_dim * es));
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
