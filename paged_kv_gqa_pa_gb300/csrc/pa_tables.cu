// pa_tables.cu -- block tables, lengths, slots and positions of a step from
// the requests' lengths and a list of free pages (pa_extend_tables of
// include/pa_q4.h).
//
// The sums over the requests (packed rows, pages needed) are small, the
// tokens many, so every CTA works the sums out for itself in shared memory
// and then serves its share of the tokens: one launch, no CTA waits for
// another, and no output depends on their order.  A token finds its request
// by bisection of the sums.  The token at the start of a page writes that
// page's table entry; CTA 0 writes what there is per request.
//
// Measured on GB300: one request with one token 2.4 us, 512 requests with 52K
// new tokens 5.3 us: a launch, the two dependent reads (lengths, then table or
// free list) and the scans between them; memory would need 0.2 us.
#include <climits>

#include "pa_q4.cuh"

namespace pa {

constexpr int kTableThreads = 256;
constexpr int kTableTokens = 4;        // tokens per thread
constexpr int kTableMaxBatch = 8192;

struct TablesParams {
    const int* past;
    const int* fresh;       // new_lens
    const int* free_pages;
    int* block_tables;
    int* context_lens;
    int* starts;
    long long* slots;
    int* positions;
    int* taken;
    unsigned* err;
    int B, maxp, num_pages, num_free, cap;
};

// Exclusive sum over the CTA of one 64-bit value per thread; *total: the whole.
__device__ __forceinline__ long long cta_exclusive(long long v, long long* s_red,
                                                   long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long inc = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m) inc += o;
    }
    __syncthreads();  // earlier reads of s_red are done
    if (lane == 31) s_red[warp] = inc;
    __syncthreads();
    long long sum = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kTableThreads / 32; ++w) {
        if (w == warp) before = sum;
        sum += s_red[w];
    }
    *total = sum;
    return before + inc - v;
}

__global__ void __launch_bounds__(kTableThreads) extend_tables_kernel(const TablesParams p) {
    extern __shared__ int s_dyn[];
    int* s_start = s_dyn;            // [B + 1] first packed row (limited to INT_MAX)
    int* s_first = s_dyn + p.B + 1;  // [B] first free page, -1: the request is refused
    __shared__ long long s_red[kTableThreads / 32];
    const int tid = threadIdx.x;
    allow_dependent_launch();
    wait_for_prerequisite_grid();

    const int per = (p.B + kTableThreads - 1) / kTableThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    const long long room = (long long)p.maxp * kPageSize;
    // Packed rows: a negative new length has none.
    long long rows = 0;
    for (int b = b0; b < b1; ++b) rows += max(0, p.fresh[b]);
    long long all_rows, all_pages;
    long long row = cta_exclusive(rows, s_red, &all_rows);
    // Pages of the requests that are in order; the others take none.
    long long pages = 0;
    unsigned err = 0;
    {
        long long r = row;
        for (int b = b0; b < b1; ++b) {
            const int past = p.past[b], n = p.fresh[b];
            s_start[b] = (int)min(r, (long long)INT_MAX);
            r += max(0, n);
            const bool ok = past >= 0 && n >= 0 && (long long)past + n <= room && r <= p.cap;
            int add = -1;
            if (ok) {
                add = (past + n + kPageSize - 1) / kPageSize - (past + kPageSize - 1) / kPageSize;
                pages += add;
            } else {
                err |= PA_DEVERR_BAD_LENGTH;
            }
            s_first[b] = add;  // (for the pass below)
        }
    }
    long long page = cta_exclusive(pages, s_red, &all_pages);
    // The free list serves requests in order as far as it reaches; what is
    // taken ends with the last request served.
    long long used = 0;
    for (int b = b0; b < b1; ++b) {
        const int add = s_first[b];
        int first = -1;
        if (add >= 0) {
            if (add == 0) {
                first = 0;
            } else if (page + add <= p.num_free) {
                first = (int)page;
                used += add;
            } else {
                err |= PA_DEVERR_NO_PAGES;
            }
            page += add;
        }
        s_first[b] = first;
    }
    if (blockIdx.x == 0) {
        for (int b = b0; b < b1; ++b) {
            p.context_lens[b] = p.past[b] + (s_first[b] >= 0 ? p.fresh[b] : 0);
            p.starts[b] = s_start[b];
        }
        long long all_used;
        cta_exclusive(used, s_red, &all_used);
        if (tid == 0) {
            p.taken[0] = (int)all_used;
            p.starts[p.B] = (int)min(all_rows, (long long)INT_MAX);
        }
        if (err && p.err) atomicOr(p.err, err);
    }
    if (tid == 0) s_start[p.B] = (int)min(all_rows, (long long)INT_MAX);
    __syncthreads();

    const int end = s_start[p.B];
#pragma unroll
    for (int u = 0; u < kTableTokens; ++u) {
        const long long t = ((long long)blockIdx.x * kTableTokens + u) * kTableThreads + tid;
        if (t >= p.cap) return;
        long long slot = -1;
        int pos = 0;
        if (t < end) {
            int a = 0, z = p.B - 1;  // the last request whose rows begin at or before t
            while (a < z) {
                const int m = (a + z + 1) >> 1;
                if (s_start[m] <= t)
                    a = m;
                else
                    z = m - 1;
            }
            const int past = p.past[a];
            const long long at = (long long)past + (t - s_start[a]);
            if (past >= 0 && at < room) pos = (int)at;
            const int first = s_first[a];
            if (first >= 0) {
                const int have = (past + kPageSize - 1) / kPageSize;
                const int col = pos / kPageSize;
                int* cell = p.block_tables + (size_t)a * p.maxp + col;
                // (L2 loads: CTAs write other entries of the same rows)
                const int id = col < have ? __ldcg(cell) : __ldcg(p.free_pages + first + col - have);
                const bool good = id >= 0 && id < p.num_pages;
                if (good)
                    slot = (long long)id * kPageSize + pos % kPageSize;
                else if (p.err)
                    atomicOr(p.err, PA_DEVERR_BAD_PAGE);
                if (col >= have && pos % kPageSize == 0) *cell = good ? id : -1;
            }
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
}

}  // namespace pa

using namespace pa;

extern "C" int pa_extend_tables(int batch, int max_pages_per_seq, int page_size, int num_pages,
                                int num_free, int token_capacity, const int32_t* past_lens,
                                const int32_t* new_lens, const int32_t* free_pages,
                                int32_t* block_tables, int32_t* context_lens, int32_t* starts,
                                int64_t* slots, int32_t* positions, int32_t* pages_taken,
                                uint32_t* device_error, void* stream) {
    if (batch < 0 || max_pages_per_seq <= 0 || page_size <= 0 || num_pages <= 0 || num_free < 0 ||
        token_capacity < 0)
        return PA_ERR_INVALID_ARG;
    if (page_size != kPageSize || batch > kTableMaxBatch ||
        (long long)max_pages_per_seq * kPageSize > INT_MAX)
        return PA_ERR_UNSUPPORTED;
    if (!starts || !pages_taken || (batch > 0 && (!past_lens || !new_lens || !block_tables ||
                                                  !context_lens)) ||
        (num_free > 0 && !free_pages) || (token_capacity > 0 && (!slots || !positions)))
        return PA_ERR_INVALID_ARG;
    const uintptr_t words = (uintptr_t)past_lens | (uintptr_t)new_lens | (uintptr_t)free_pages |
                            (uintptr_t)block_tables | (uintptr_t)context_lens |
                            (uintptr_t)starts | (uintptr_t)positions | (uintptr_t)pages_taken |
                            (uintptr_t)device_error;
    if ((words & 3u) || ((uintptr_t)slots & 7u)) return PA_ERR_INVALID_ARG;
    // Other CTAs still read the lengths while one writes the results.
    if (batch > 0 && (context_lens == past_lens || context_lens == new_lens ||
                      starts == past_lens || starts == new_lens))
        return PA_ERR_INVALID_ARG;
    TablesParams p;
    p.past = past_lens;
    p.fresh = new_lens;
    p.free_pages = free_pages;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.starts = starts;
    p.slots = reinterpret_cast<long long*>(slots);
    p.positions = positions;
    p.taken = pages_taken;
    p.err = device_error;
    p.B = batch;
    p.maxp = max_pages_per_seq;
    p.num_pages = num_pages;
    p.num_free = num_free;
    p.cap = token_capacity;
    const int smem = (2 * batch + 1) * 4;
    // (48 KB without asking, the kernel's own s_red among them)
    if (smem > 47 * 1024 &&
        cudaFuncSetAttribute(extend_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (2 * kTableMaxBatch + 1) * 4) != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    const int per_cta = kTableThreads * kTableTokens;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)token_capacity + per_cta - 1) / per_cta));
    if (cfg.gridDim.x == 0) cfg.gridDim.x = 1;  // (the lengths are still written)
    cfg.blockDim = dim3(kTableThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, extend_tables_kernel, p) != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return PA_OK;
}
