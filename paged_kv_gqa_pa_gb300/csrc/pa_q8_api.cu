// pa_q8_api.cu -- planning, argument checks and launch of the attention over
// the 8-bit cache (include/pa_q8.h).
#include <limits.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include <cudaTypedefs.h>

#include "pa_q8_attend.cuh"

namespace pa {

constexpr int kQ8MaxBatch = 4096;
constexpr int kQ8MaxQuery = 16;     // query tokens of a sequence
// Pages of a warp, at least (one sequence of 4000 tokens, one KV head: 2 7.9 us, 4 8.9, 8 10.3; of
// 16000: 1 11.6, 2 9.7, 4 9.3, 8 11.7).
constexpr int kQ8MinRun = 2;
constexpr int kQ8MaxCluster = 8;    // (the largest that every launch may have)
// Pages of head_dim 128, see pa_q8_plan (16 sequences of 4096 tokens' window, five queries: 4
// pages 48.0 us, 12 46.9; with 24, 12 of 10000 tokens each go 48.0 -> 44.4, but 12 of up to
// 10000 25.7 -> 37.2).
constexpr int kQ8ClusterExtra = 12;
// Partials per sequence beyond which a kernel merges (20 sequences of 6000 tokens: 2 50.4 us, 4
// 45.3; 6 of 20000: 4 46.1, 12 47.5).
constexpr int kQ8KernelRows = 4;

static bool q8_head_dim_ok(int D) { return D == 64 || D == 96 || D == 128 || D == 256; }

static const Q8Instance& q8_pick(int D, int tiles) {
    switch (D) {
        case 64: return kQ8D64[tiles - 1];
        case 96: return kQ8D96[tiles - 1];
        case 128: return tiles <= 2 ? kQ8D128a[tiles - 1] : kQ8D128b[tiles - 3];
        default: return kQ8D256[tiles - 1];
    }
}

// Workspace: [control block | counters of the partials left, groups x B | cost of a
// range, page and rank sums and first rows for the merge kernel | (max, sum) of the
// partials | their outputs], each 256-byte aligned; two partials per CTA.
struct Q8WsLayout {
    size_t ctr_off, ctrl_bytes, info_off, ml_off, o_off, total;
};

static size_t q8_align256(size_t x) { return (x + 255) & ~(size_t)255; }

static Q8WsLayout q8_ws_layout(int B, int D, int tiles, long long groups, int X) {
    Q8WsLayout w;
    const size_t rows = (size_t)groups * X * 2;
    w.ctr_off = kCtrlBytes;
    w.ctrl_bytes = kCtrlBytes + q8_align256((size_t)groups * B * 4);
    w.info_off = w.ctrl_bytes;
    w.ml_off = w.info_off + q8_align256((3 * (size_t)B + 4) * 4);
    w.o_off = w.ml_off + q8_align256(rows * 8 * tiles * 8);
    w.total = w.o_off + q8_align256(rows * 8 * tiles * D * 4);
    return w;
}

static int q8_ctas_per_sm(int D, int tiles, int B) {
    int smem = 0, most = 0;  // shared memory of a CTA, CTAs that the registers allow
    q8_pick(D, tiles).size(B, &smem, &most);
    return std::max(1, std::min(most, 228 * 1024 / (smem + 1024 + 384)));
}

// Clusters of c CTAs held at once: the current device's answer (asked for once
// per device and CTAs per SM), or for a plan made for an SM count a low estimate
// (a cluster must lie within one GPC, so up to a third of the slots stay unused).
static long long q8_clusters_held(bool this_device, int D, int tiles, int batch, int c,
                                  long long slots) {
    constexpr int kMaxDevices = 64, kMaxPerSm = 8;
    static std::atomic<int> cache[kMaxDevices][4][4][kMaxPerSm][kQ8MaxCluster];  // value + 1
    const long long estimate = slots * 2 / (3 * c);
    const int per_sm = q8_ctas_per_sm(D, tiles, batch);
    int dev = 0;
    if (!this_device || per_sm > kMaxPerSm) return estimate;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return estimate;
    }
    const int di = D == 64 ? 0 : D == 96 ? 1 : D == 128 ? 2 : 3;
    std::atomic<int>& slot = cache[dev][di][tiles - 1][per_sm - 1][c - 1];
    const int known = slot.load();
    if (known > 0) return known - 1;
    int held = 0;
    if (q8_pick(D, tiles).clusters(c, batch, &held) != cudaSuccess || held < 0) {
        cudaGetLastError();
        return estimate;
    }
    slot.store(held + 1);
    return held;
}

// What a plan's shapes must satisfy; the automatic fields are checked by the caller.
static int q8_check_shapes(const pa_q8_plan_t* p) {
    if (p->batch < 0 || p->num_q_heads <= 0 || p->num_kv_heads <= 0 ||
        p->num_q_heads % p->num_kv_heads != 0 || p->head_dim <= 0 || p->page_size <= 0 ||
        p->num_pages <= 0 || p->max_pages_per_seq <= 0 || p->max_context_len < 0 ||
        p->window < 0 || p->num_sms < 0 || p->max_query_len < 1)
        return PA_ERR_INVALID_ARG;
    if (p->dtype != PA_DTYPE_F16 && p->dtype != PA_DTYPE_BF16 && p->dtype != PA_DTYPE_F32)
        return PA_ERR_INVALID_ARG;
    if ((long long)p->max_context_len > (long long)p->max_pages_per_seq * p->page_size)
        return PA_ERR_INVALID_ARG;
    if (p->dtype == PA_DTYPE_F32 || !q8_head_dim_ok(p->head_dim) || p->page_size != kPageSize ||
        p->batch > kQ8MaxBatch || p->max_query_len > kQ8MaxQuery)
        return PA_ERR_UNSUPPORTED;
    // Positions, and lengths rounded up to whole pages, are counted in 32 bits.
    if (p->max_context_len > INT_MAX - (kPageSize - 1)) return PA_ERR_UNSUPPORTED;
    // So are the batch's pages end to end, and the rows of the cache's tensor maps.
    const long long span = ((long long)p->max_context_len + kPageSize - 1) / kPageSize;
    if (span * std::max(1, p->batch) > (1ll << 30)) return PA_ERR_UNSUPPORTED;
    if ((long long)p->num_pages * p->num_kv_heads > INT_MAX / kPageSize) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// Pages that a sequence can attend: those of its query tokens' windows together.
static int q8_attended_pages(int max_context_len, int window, int max_query_len) {
    if (window > 0 && window > INT_MAX - max_query_len) window = 0;  // (holds everything)
    return attended_pages(max_context_len, window > 0 ? window + max_query_len - 1 : 0);
}

// K's or V's cache as a tensor of bytes whose boxes are pages; see q8_chunk.
static bool q8_page_map(CUtensorMap* map, const void* base, long long rows, int D) {
    static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
        else
            cudaGetLastError();
    });
    if (!enc) return false;
    const cuuint32_t estr[3] = {1, 1, 1};
    auto encode = [&](const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                      const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle) {
        return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t n = (cuuint64_t)rows, row = (cuuint64_t)D;
    if (D == 96)
        return encode({32, 3, n}, {32, row}, {32, 3, kPageSize}, CU_TENSOR_MAP_SWIZZLE_32B);
    if (D == 64)
        return encode({64, n, 1}, {row, row}, {64, kPageSize, 1}, CU_TENSOR_MAP_SWIZZLE_64B);
    return encode({128, n, row / 128}, {row, 128}, {128, kPageSize, (cuuint32_t)D / 128},
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// The maps of the last pools this thread used: a map is a pure function of the
// address, the rows and the head dim.
static bool q8_cached_map(CUtensorMap* map, const void* base, long long rows, int D) {
    struct Entry {
        alignas(64) CUtensorMap map;
        const void* base;
        long long rows;
        int D;
        bool valid;
    };
    constexpr int kEntries = 8;
    thread_local Entry cache[kEntries] = {};
    thread_local int next = 0;
    for (const Entry& e : cache)
        if (e.valid && e.base == base && e.rows == rows && e.D == D) {
            *map = e.map;
            return true;
        }
    if (!q8_page_map(map, base, rows, D)) return false;
    Entry& e = cache[next];
    next = (next + 1) % kEntries;
    e.map = *map;
    e.base = base;
    e.rows = rows;
    e.D = D;
    e.valid = true;
    return true;
}

}  // namespace pa

using namespace pa;

extern "C" {

int pa_q8_plan(int batch, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
               int num_pages, int max_pages_per_seq, int max_context_len, int window,
               int max_query_len, int num_sms, int dtype, pa_q8_plan_t* plan) {
    if (!plan) return PA_ERR_INVALID_ARG;
    memset(plan, 0, sizeof(*plan));
    pa_q8_plan_t p = {};
    p.batch = batch;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_pages_per_seq = max_pages_per_seq;
    p.max_context_len = max_context_len;
    p.window = window;
    p.max_query_len = max_query_len;
    p.num_sms = num_sms;
    p.dtype = dtype;
    const int st = q8_check_shapes(&p);
    if (st != PA_OK) return st;
    const int g = num_q_heads / num_kv_heads;
    // The fewest equal chunks whose rows fit the tiles: each reads the cache once.
    int nchunk = 1;
    while (g % nchunk != 0 || (long long)(g / nchunk) * max_query_len > q8_max_rows(head_dim))
        ++nchunk;
    const int G = g / nchunk, tiles = (G * max_query_len + 7) / 8;
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
    p.heads_per_cta = G;
    // One wave of resident CTAs over all groups, filled to a little under its
    // slots (a grid that needs every slot has CTAs starting in a second wave),
    // but no more than give every sequence one and every warp kQ8MinRun pages
    // of the longest batch.
    const int span = q8_attended_pages(max_context_len, window, max_query_len);
    const long long cost = std::max(1ll, (long long)std::max(1, batch) * (span + kQ8Start));
    const long long slots = (long long)p.num_sms * q8_ctas_per_sm(head_dim, tiles, batch);
    long long x = std::max(1ll, (slots - slots / 64) / groups);
    if (span <= q8_short(head_dim) && batch <= x)
        x = std::max(1, batch);  // one for each sequence
    else
        x = std::min(x, std::max<long long>(batch, (cost + kWarps * kQ8MinRun - 1) /
                                                      (kWarps * kQ8MinRun)));
    // A cluster for each sequence saves the partials' way through the L2 but gives
    // the CTAs of the longest sequence more pages than equal ranges do: the largest
    // cluster of which one wave holds all, with a page for every warp, where that is
    // at most kQ8ClusterExtra pages of head_dim 128 more.  (Lengths are known on the
    // device only, so every sequence counts as the longest.)
    if (batch > 0 && span > q8_short(head_dim)) {
        int c = std::min(kQ8MaxCluster, (span + kWarps - 1) / kWarps);
        while (c > 1 && (groups * batch * c > slots ||
                         q8_clusters_held(this_device, head_dim, tiles, batch, c, slots) <
                             groups * batch))
            --c;
        const long long extra = (span + c - 1) / c - (cost + x - 1) / x;
        if (c > 1 && extra * head_dim <= kQ8ClusterExtra * 128) {
            p.cluster = c;
            x = (long long)c * batch;
        }
    }
    p.ctas_per_group = (int)x;
    p.ctas = (int)std::min<long long>(x * groups, INT_MAX);
    const Q8WsLayout wl = q8_ws_layout(batch, head_dim, tiles, groups, p.ctas_per_group);
    if (wl.ctrl_bytes > (size_t)INT_MAX) return PA_ERR_UNSUPPORTED;
    p.workspace_bytes = wl.total;
    p.ctrl_bytes = (int)wl.ctrl_bytes;
    *plan = p;
    return PA_OK;
}

int pa_q8_decode(const pa_q8_plan_t* plan, int num_rows, const void* q, const int32_t* starts,
                 const void* k_cache, const void* v_cache, const float* k_scales,
                 const float* v_scales, const int32_t* block_tables,
                 const int32_t* context_lens, float scale, int window, void* out, float* lse,
                 void* workspace, void* stream) {
    if (!plan) return PA_ERR_INVALID_ARG;
    const int st = q8_check_shapes(plan);
    if (st != PA_OK) return st;
    const int g = plan->num_q_heads / plan->num_kv_heads;
    const int G = plan->heads_per_cta, X = plan->ctas_per_group, D = plan->head_dim;
    if (G < 1 || g % G != 0 || G * plan->max_query_len > q8_max_rows(D) || X < 1 ||
        X > (1 << 20) ||
        (plan->cluster != 0 && (plan->cluster < 2 || plan->cluster > kQ8MaxCluster ||
                                (long long)plan->cluster * plan->batch != X)) ||
        window != plan->window || plan->test_stall_bytes < 0 || plan->test_stall_bytes > 4096 ||
        num_rows < 0 || (!starts && num_rows < plan->batch))
        return PA_ERR_INVALID_ARG;
    const long long groups = (long long)plan->num_kv_heads * (g / G);
    if (groups > 65535) return PA_ERR_UNSUPPORTED;
    const int tiles = (G * plan->max_query_len + 7) / 8;
    const Q8WsLayout wl = q8_ws_layout(plan->batch, D, tiles, groups, X);
    if (plan->workspace_bytes < wl.total || plan->ctrl_bytes < 0 ||
        (size_t)plan->ctrl_bytes < wl.ctrl_bytes)
        return PA_ERR_INVALID_ARG;
    if (!workspace) return PA_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 15u) return PA_ERR_INVALID_ARG;
    if (plan->batch == 0 || num_rows == 0) return PA_OK;
    if (!q || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables || !context_lens ||
        !out || !lse)
        return PA_ERR_INVALID_ARG;
    if ((((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out) & 15u) ||
        (((uintptr_t)block_tables | (uintptr_t)context_lens | (uintptr_t)lse |
          (uintptr_t)starts | (uintptr_t)k_scales | (uintptr_t)v_scales) & 3u))
        return PA_ERR_INVALID_ARG;
    Q8Maps maps;
    const long long map_rows = (long long)plan->num_pages * plan->num_kv_heads * kPageSize;
    if (!q8_cached_map(&maps.k, k_cache, map_rows, D) ||
        !q8_cached_map(&maps.v, v_cache, map_rows, D))
        return PA_ERR_CUDA;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    Q8AttendParams p;
    p.q = q;
    p.starts = starts;
    p.k = static_cast<const unsigned char*>(k_cache);
    p.v = static_cast<const unsigned char*>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
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
    // partials: beyond kQ8KernelRows a kernel of its own gathers them.
    p.merge_kernel = !p.cluster && X > kQ8KernelRows * plan->batch ? 1 : 0;
    p.counters = reinterpret_cast<unsigned*>(ws + wl.ctr_off);
    p.B = plan->batch;
    p.Hq = plan->num_q_heads;
    p.Hkv = plan->num_kv_heads;
    p.g = g;
    p.num_pages = plan->num_pages;
    p.maxp = plan->max_pages_per_seq;
    p.max_ctx = plan->max_context_len;
    // (a window that holds everything is none; sums with it stay in 32 bits)
    p.window = plan->window > plan->max_context_len ? 0 : plan->window;
    p.max_t = plan->max_query_len;
    p.rows = num_rows;
    p.nchunk = g / G;
    p.G = G;
    p.ginv = 65536 / G + 1;
    p.X = X;
    p.stall_tx = plan->test_stall_bytes;
    p.bf16 = plan->dtype == PA_DTYPE_BF16;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    if (q8_pick(D, tiles).launch(p, maps, dim3(X, (unsigned)groups),
                                 static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return PA_OK;
}

}  // extern "C"
