// pa_q4_api.cu -- planning, argument checks and launch of the decode
// attention over the 4-bit cache (include/pa_q4.h).
#include <limits.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "pa_q4_attend.cuh"

namespace pa {

#define PA_Q4_EXTERN(D)                                                                          \
    extern template cudaError_t launch_q4_attend_d<D, __half>(const Q4AttendParams&, dim3,       \
                                                              cudaStream_t);                     \
    extern template cudaError_t launch_q4_attend_d<D, __nv_bfloat16>(const Q4AttendParams&, dim3, \
                                                                     cudaStream_t);              \
    extern template cudaError_t q4_attend_clusters<D, __half>(int, int, int*);                   \
    extern template cudaError_t q4_attend_clusters<D, __nv_bfloat16>(int, int, int*);
PA_Q4_EXTERN(64)
PA_Q4_EXTERN(96)
PA_Q4_EXTERN(128)
PA_Q4_EXTERN(256)
#undef PA_Q4_EXTERN

constexpr int kQ4MaxBatch = 4096;
constexpr int kQ4MinRun = 2;    // pages of a warp, at least
constexpr int kQ4MaxCluster = 8;  // (the largest that every launch may have)
constexpr int kQ4ClusterExtra = 12;  // pages of head_dim 128, see pa_q4_plan
constexpr int kQ4KernelRows = 4;  // partials per sequence beyond which a kernel merges

// Workspace: [control block | counters of the partials left, groups x B | run
// size and page sums for the merge kernel | (max, sum) of the partials | their
// outputs], each 256-byte aligned; two partials per CTA.
struct Q4WsLayout {
    size_t ctr_off, ctrl_bytes, info_off, ml_off, o_off, total;
};

static size_t q4_align256(size_t x) { return (x + 255) & ~(size_t)255; }

static Q4WsLayout q4_ws_layout(int B, int D, long long groups, int X) {
    Q4WsLayout w;
    const size_t rows = (size_t)groups * X * 2;
    w.ctr_off = kCtrlBytes;
    w.ctrl_bytes = kCtrlBytes + q4_align256((size_t)groups * B * 4);
    w.info_off = w.ctrl_bytes;
    w.ml_off = w.info_off + q4_align256((2 * (size_t)B + 4) * 4);
    w.o_off = w.ml_off + q4_align256(rows * kMaxHeadsPerCta * 8);
    w.total = w.o_off + q4_align256(rows * kMaxHeadsPerCta * D * 4);
    return w;
}

static int q4_ctas_per_sm(int D, int B) {
    int smem = 0, most = 0;  // shared memory of a CTA, CTAs that the registers allow
    switch (D) {
        case 64: smem = Q4Cfg<64>::smem(B), most = Q4Cfg<64>::kMinBlocks; break;
        case 96: smem = Q4Cfg<96>::smem(B), most = Q4Cfg<96>::kMinBlocks; break;
        case 128: smem = Q4Cfg<128>::smem(B), most = Q4Cfg<128>::kMinBlocks; break;
        default: smem = Q4Cfg<256>::smem(B), most = Q4Cfg<256>::kMinBlocks; break;
    }
    return std::max(1, std::min(most, 228 * 1024 / (smem + 1024 + 128)));
}

// Clusters of c CTAs held at once: the current device's answer (asked for once
// per device and CTAs per SM), or for a plan made for an SM count a low estimate
// (a cluster must lie within one GPC, so up to a third of the slots stay unused).
static long long q4_clusters_held(bool this_device, int D, int dtype, int batch, int c,
                                  long long slots) {
    constexpr int kMaxDevices = 64, kMaxPerSm = 8;
    static std::atomic<int> cache[kMaxDevices][4][2][kMaxPerSm][kQ4MaxCluster];  // value + 1
    const long long estimate = slots * 2 / (3 * c);
    const int per_sm = q4_ctas_per_sm(D, batch);
    int dev = 0;
    if (!this_device || per_sm > kMaxPerSm) return estimate;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return estimate;
    }
    const int di = D == 64 ? 0 : D == 96 ? 1 : D == 128 ? 2 : 3;
    const int ti = dtype == PA_DTYPE_BF16 ? 1 : 0;
    std::atomic<int>& slot = cache[dev][di][ti][per_sm - 1][c - 1];
    const int known = slot.load();
    if (known > 0) return known - 1;
    int held = 0;
    cudaError_t e;
#define PA_HELD(DD)                                                  \
    e = ti ? q4_attend_clusters<DD, __nv_bfloat16>(c, batch, &held) \
           : q4_attend_clusters<DD, __half>(c, batch, &held)
    switch (D) {
        case 64: PA_HELD(64); break;
        case 96: PA_HELD(96); break;
        case 128: PA_HELD(128); break;
        default: PA_HELD(256); break;
    }
#undef PA_HELD
    if (e != cudaSuccess || held < 0) {
        cudaGetLastError();
        return estimate;
    }
    slot.store(held + 1);
    return held;
}

// What a plan's shapes must satisfy; the automatic fields are checked by the caller.
static int q4_check_shapes(const pa_q4_plan_t* p) {
    if (p->batch < 0 || p->num_q_heads <= 0 || p->num_kv_heads <= 0 ||
        p->num_q_heads % p->num_kv_heads != 0 || p->head_dim <= 0 || p->page_size <= 0 ||
        p->num_pages <= 0 || p->max_pages_per_seq <= 0 || p->max_context_len < 0 ||
        p->window < 0 || p->num_sms < 0)
        return PA_ERR_INVALID_ARG;
    if (p->dtype != PA_DTYPE_F16 && p->dtype != PA_DTYPE_BF16 && p->dtype != PA_DTYPE_F32)
        return PA_ERR_INVALID_ARG;
    if ((long long)p->max_context_len > (long long)p->max_pages_per_seq * p->page_size)
        return PA_ERR_INVALID_ARG;
    if (p->dtype == PA_DTYPE_F32 || !q4_head_dim_ok(p->head_dim) || p->page_size != kPageSize ||
        p->batch > kQ4MaxBatch)
        return PA_ERR_UNSUPPORTED;
    // Positions, and lengths rounded up to whole pages, are counted in 32 bits.
    if (p->max_context_len > INT_MAX - (kPageSize - 1)) return PA_ERR_UNSUPPORTED;
    // So are the batch's pages end to end.
    const long long span = ((long long)p->max_context_len + kPageSize - 1) / kPageSize;
    if (span * std::max(1, p->batch) > (1ll << 30)) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" {

int pa_q4_plan(int batch, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
               int num_pages, int max_pages_per_seq, int max_context_len, int window,
               int num_sms, int dtype, pa_q4_plan_t* plan) {
    if (!plan) return PA_ERR_INVALID_ARG;
    memset(plan, 0, sizeof(*plan));
    pa_q4_plan_t p = {};
    p.batch = batch;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_pages_per_seq = max_pages_per_seq;
    p.max_context_len = max_context_len;
    p.window = window;
    p.num_sms = num_sms;
    p.dtype = dtype;
    const int st = q4_check_shapes(&p);
    if (st != PA_OK) return st;
    const int g = num_q_heads / num_kv_heads;
    // The fewest equal chunks of at most kMaxHeadsPerCta heads: each reads the cache
    // once.  (One head at a time, what a prime above that comes to, is refused.)
    int nchunk = (g + kMaxHeadsPerCta - 1) / kMaxHeadsPerCta;
    while (g % nchunk != 0) ++nchunk;
    if (nchunk > 1 && nchunk == g) return PA_ERR_UNSUPPORTED;
    const long long groups = (long long)num_kv_heads * nchunk;
    if (groups > 65535) return PA_ERR_UNSUPPORTED;
    const bool this_device = p.num_sms == 0;
    if (this_device) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&p.num_sms, cudaDevAttrMultiProcessorCount, dev) !=
                cudaSuccess) {
            cudaGetLastError();
            return PA_ERR_CUDA;
        }
    }
    p.heads_per_cta = g / nchunk;
    // One wave of resident CTAs over all groups, filled to a little under its
    // slots (a grid that needs every slot had CTAs starting in a second wave),
    // but no more than give every sequence one and every warp kQ4MinRun pages
    // of the longest batch.
    const int span = attended_pages(max_context_len, window);
    const long long cost = std::max(1ll, (long long)std::max(1, batch) * (span + kQ4Start));
    const long long slots = (long long)p.num_sms * q4_ctas_per_sm(head_dim, batch);
    long long x = std::max(1ll, (slots - slots / 64) / groups);
    if (span <= q4_short(head_dim) && batch <= x)
        x = std::max(1, batch);  // one for each sequence
    else
        x = std::min(x, std::max<long long>(batch, (cost + kWarps * kQ4MinRun - 1) /
                                                      (kWarps * kQ4MinRun)));
    // A cluster for each sequence, which saves the partials' way through the L2
    // (2 to 4 us) but gives the CTAs of the longest sequence more pages than equal
    // ranges do: the largest cluster of which one wave holds all, with a page for
    // every warp, where that is at most kQ4ClusterExtra pages of head_dim 128 more.
    // Clusters against equal ranges, head_dim 128, 8 KV heads: one sequence of 1000
    // tokens 6.2 and 7.2 us, of 2500 7.9 and 7.9, of 4000 9.3 and 8.4; 4 of 1000 7.6
    // and 9.5, of 4000 11.9 and 12.0, of 6000 14.9 and 14.0; 16 of 2500 (bf16) 19.2
    // and 20.7.  Lengths are known on the device only, so every sequence counts as
    // the longest: a ragged batch pays for that.  One longer than the rest, 8 in
    // all, of 2000 8.9 and 9.0, of 4000 11.5 and 9.3 (a caller that knows better
    // sets cluster 0).  Clusters that one wave does not hold cost 5 to 10 us (16
    // sequences of 1000 tokens, bf16, by 4 CTAs 18.8, by 3 12.5).
    if (batch > 0 && span > q4_short(head_dim)) {
        int c = std::min(kQ4MaxCluster, (span + kWarps - 1) / kWarps);
        while (c > 1 && (groups * batch * c > slots ||
                         q4_clusters_held(this_device, head_dim, dtype, batch, c, slots) <
                             groups * batch))
            --c;
        const long long extra = (span + c - 1) / c - (cost + x - 1) / x;
        if (c > 1 && extra * head_dim <= kQ4ClusterExtra * 128) {
            p.cluster = c;
            x = (long long)c * batch;
        }
    }
    p.ctas_per_group = (int)x;
    p.ctas = (int)std::min<long long>(x * groups, INT_MAX);
    const Q4WsLayout wl = q4_ws_layout(batch, head_dim, groups, p.ctas_per_group);
    if (wl.ctrl_bytes > (size_t)INT_MAX) return PA_ERR_UNSUPPORTED;
    p.workspace_bytes = wl.total;
    p.ctrl_bytes = (int)wl.ctrl_bytes;
    *plan = p;
    return PA_OK;
}

int pa_q4_decode(const pa_q4_plan_t* plan, const void* q, const void* cache,
                 const int32_t* block_tables, const int32_t* context_lens, float scale,
                 int window, void* out, float* lse, void* workspace, void* stream) {
    if (!plan) return PA_ERR_INVALID_ARG;
    const int st = q4_check_shapes(plan);
    if (st != PA_OK) return st;
    const int g = plan->num_q_heads / plan->num_kv_heads;
    const int G = plan->heads_per_cta, X = plan->ctas_per_group, D = plan->head_dim;
    if (G < 1 || G > kMaxHeadsPerCta || g % G != 0 || X < 1 || X > (1 << 20) ||
        (plan->cluster != 0 && (plan->cluster < 2 || plan->cluster > kQ4MaxCluster ||
                                (long long)plan->cluster * plan->batch != X)) ||
        window != plan->window || plan->test_stall_bytes < 0 || plan->test_stall_bytes > 4096)
        return PA_ERR_INVALID_ARG;
    const long long groups = (long long)plan->num_kv_heads * (g / G);
    if (groups > 65535) return PA_ERR_UNSUPPORTED;
    const Q4WsLayout wl = q4_ws_layout(plan->batch, D, groups, X);
    if (plan->workspace_bytes < wl.total || plan->ctrl_bytes < 0 ||
        (size_t)plan->ctrl_bytes < wl.ctrl_bytes)
        return PA_ERR_INVALID_ARG;
    if (!workspace) return PA_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 15u) return PA_ERR_INVALID_ARG;
    if (plan->batch == 0) return PA_OK;
    if (!q || !cache || !block_tables || !context_lens || !out || !lse) return PA_ERR_INVALID_ARG;
    if (((uintptr_t)q & 15u) || ((uintptr_t)cache & 15u) || ((uintptr_t)out & 15u) ||
        (((uintptr_t)block_tables | (uintptr_t)context_lens | (uintptr_t)lse) & 3u))
        return PA_ERR_INVALID_ARG;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    Q4AttendParams p;
    p.q = q;
    p.cache = static_cast<const unsigned char*>(cache);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.out = out;
    p.lse = lse;
    p.ws_o = reinterpret_cast<float*>(ws + wl.o_off);
    p.ws_ml = reinterpret_cast<float*>(ws + wl.ml_off);
    p.err = reinterpret_cast<unsigned*>(ws);
    p.ws_info = reinterpret_cast<int*>(ws + wl.info_off);
    p.cluster = plan->cluster;
    // A sequence of a batch of B cut into equal ranges leaves about X / B
    // partials: beyond kQ4KernelRows a kernel of its own gathers them.  By the last
    // CTA to leave one, and by the kernel: 16 sequences of 20000 tokens (3.5 each)
    // 76.5 and 79.8 us, 8 ragged ones up to 30000 (7) 34.9 and 32.8, 4 of 9000 (14)
    // 20.4 and 17.6; at 4 to 5 of them D 96 would do with the CTA (26.4 and 28.1),
    // D 256 does not (45.1 and 42.7).
    p.merge_kernel = !p.cluster && X > kQ4KernelRows * plan->batch ? 1 : 0;
    p.counters = reinterpret_cast<unsigned*>(ws + wl.ctr_off);
    p.B = plan->batch;
    p.Hq = plan->num_q_heads;
    p.Hkv = plan->num_kv_heads;
    p.g = g;
    p.num_pages = plan->num_pages;
    p.maxp = plan->max_pages_per_seq;
    p.max_ctx = plan->max_context_len;
    p.window = plan->window;
    p.nchunk = g / G;
    p.G = G;
    p.X = X;
    p.stall_tx = plan->test_stall_bytes;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    const dim3 grid(X, (unsigned)groups);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf = plan->dtype == PA_DTYPE_BF16;
    cudaError_t e;
    switch (D) {
        case 64:
            e = bf ? launch_q4_attend_d<64, __nv_bfloat16>(p, grid, s)
                   : launch_q4_attend_d<64, __half>(p, grid, s);
            break;
        case 96:
            e = bf ? launch_q4_attend_d<96, __nv_bfloat16>(p, grid, s)
                   : launch_q4_attend_d<96, __half>(p, grid, s);
            break;
        case 128:
            e = bf ? launch_q4_attend_d<128, __nv_bfloat16>(p, grid, s)
                   : launch_q4_attend_d<128, __half>(p, grid, s);
            break;
        default:
            e = bf ? launch_q4_attend_d<256, __nv_bfloat16>(p, grid, s)
                   : launch_q4_attend_d<256, __half>(p, grid, s);
            break;
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return PA_OK;
}

}  // extern "C"
