// step_tables.cu -- a step's page table, slots and positions from the requests'
// lengths, on the device.
//
// Integer work: prefix sums over the requests (CSR rows, tokens, pages to take)
// and then one independent entry per page-table cell and per token.  Two
// launches: a single block scans the requests and leaves one record per request
// in the workspace, then a grid fills the entries.  The fill reads only the
// records, so the length and free-count outputs may be the inputs' own arrays.
// Bytes: 16 per page-table entry (id and tag, in and out) and 12 per token; at
// decode sizes both launches are bound by latency.
#include "fkv_common.cuh"

namespace fkv {

constexpr int kTabThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kListed = 1, kGranted = 2;        // record flags

struct StepRecord {
    int32_t cached, fresh;    // tokens held and new (0 when refused as invalid)
    int32_t top;              // free-list index of the request's first new page
    int32_t flags;
};

struct StepParams {
    const int32_t *cached, *fresh;
    int32_t *table;
    uint32_t *table_tags;
    const int32_t *free_pages, *free_count;
    const uint32_t *page_tags;
    int32_t *step_lens, *cached_out;
    uint8_t *refused;
    int32_t *page_indptr, *page_indices;
    uint32_t *expected;
    int32_t *token_indptr;
    int64_t *slots;
    int32_t *positions, *free_left;
    StepRecord *rec;
    uint32_t *err;
    int32_t batch, max_blocks, num_free, num_pages, page, nnz, n_tokens;
};

__device__ __forceinline__ int32_t pages_of(int64_t tokens, int32_t page) {
    return static_cast<int32_t>((tokens + page - 1) / page);
}

// Inclusive prefix sum over the block's threads, plus the block's total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t &total, int64_t *s_warp) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) s_warp[wid] = v;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int i = 0; i < kTabThreads / 32; ++i) {
        const int64_t x = s_warp[i];
        if (i < wid) before += x;
        total += x;
    }
    __syncthreads();                           // s_warp is free again
    return before + v;
}

__global__ void __launch_bounds__(kTabThreads)
step_plan_kernel(const StepParams p) {
    grid_dep_wait();
    grid_dep_launch();
    __shared__ int64_t s_warp[kTabThreads / 32];
    const int64_t free = min(max(*p.free_count, 0), p.num_free);
    int64_t rows = 0, toks = 0, taken = 0;     // sums over the requests before this chunk
    bool any_refused = false;
    for (int base = 0; base < p.batch; base += kTabThreads) {
        const int r = base + threadIdx.x;
        const bool in = r < p.batch;
        const int32_t c = in ? p.cached[r] : 0, n = in ? p.fresh[r] : 0;
        const int64_t len = static_cast<int64_t>(c) + n;
        const bool valid = c >= 0 && n >= 0 && len <= 0x7FFFFFFF && pages_of(len, p.page) <= p.max_blocks;
        const int32_t pages = valid ? pages_of(len, p.page) : 0;
        const int32_t count = max(n, 0);
        int64_t sum;
        const int64_t row_end = rows + block_scan(pages, sum, s_warp);
        rows += sum;
        const int64_t tok_end = toks + block_scan(count, sum, s_warp);
        toks += sum;
        const bool fits = valid && row_end <= p.nnz && tok_end <= p.n_tokens;
        const int32_t need = fits ? pages - pages_of(c, p.page) : 0;
        const int64_t need_end = taken + block_scan(need, sum, s_warp);
        taken += sum;
        const bool granted = fits && (need == 0 || need_end <= free);
        if (in) {
            p.page_indptr[r + 1] = static_cast<int32_t>(min(row_end, static_cast<int64_t>(p.nnz)));
            p.token_indptr[r + 1] = static_cast<int32_t>(min(tok_end, static_cast<int64_t>(p.n_tokens)));
            p.step_lens[r] = granted ? static_cast<int32_t>(len) : 0;
            p.cached_out[r] = granted ? static_cast<int32_t>(len) : c;
            p.refused[r] = granted ? 0 : 1;
            StepRecord rec;
            rec.cached = valid ? c : 0;
            rec.fresh = valid ? n : 0;
            rec.top = granted ? static_cast<int32_t>(free - 1 - (need_end - need)) : -1;
            rec.flags = (valid ? kListed : 0) | (granted ? kGranted : 0);
            p.rec[r] = rec;
        }
        any_refused |= in && !granted;
    }
    // pages granted: every request up to the first that found too few
    const int refused = __syncthreads_or(any_refused);
    __shared__ unsigned long long s_used;
    if (threadIdx.x == 0) s_used = 0;
    __syncthreads();
    unsigned long long used = 0;
    for (int r = threadIdx.x; r < p.batch; r += kTabThreads) {
        const StepRecord rec = p.rec[r];
        if (rec.flags & kGranted)
            used += pages_of(static_cast<int64_t>(rec.cached) + rec.fresh, p.page) - pages_of(rec.cached, p.page);
    }
    atomicAdd(&s_used, used);                  // whole numbers: any order gives the same sum
    __syncthreads();
    if (threadIdx.x == 0) {
        p.page_indptr[0] = 0;
        p.token_indptr[0] = 0;
        *p.free_left = static_cast<int32_t>(free - static_cast<int64_t>(s_used));
        if (refused) atomicOr(p.err, FKV_DEVERR_TABLES);
    }
}

// The request whose part of a prefix table holds entry i: the last one with
// indptr[r] <= i (requests without entries are passed over).
__device__ __forceinline__ int find_row(const int32_t *indptr, int batch, int32_t i) {
    int a = 0, z = batch;                      // indptr[a] <= i < indptr[z]
    while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (__ldg(indptr + mid) <= i) a = mid; else z = mid;
    }
    return a;
}

// Page `col` of a request: from its table where it held it already, else from
// the free list.  -1 (and the error bit) for an id outside the pool, -1 for a
// page it was not granted.
__device__ __forceinline__ int32_t page_at(const StepParams &p, const StepRecord &rec, int r, int32_t col) {
    const int32_t have = pages_of(rec.cached, p.page);
    int32_t id;
    if (col < have) {
        id = __ldg(p.table + static_cast<int64_t>(r) * p.max_blocks + col);
    } else {
        if (!(rec.flags & kGranted)) return -1;
        id = __ldg(p.free_pages + (rec.top - (col - have)));
    }
    if (id < 0 || id >= p.num_pages) {
        atomicOr(p.err, FKV_DEVERR_TABLES);
        return -1;
    }
    return id;
}

__global__ void __launch_bounds__(kFillThreads)
step_fill_kernel(const StepParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kFillThreads;
    const int64_t start = static_cast<int64_t>(blockIdx.x) * kFillThreads + threadIdx.x;
    const int32_t rows = p.page_indptr[p.batch], toks = p.token_indptr[p.batch];
    for (int64_t j = start; j < rows; j += stride) {
        const int r = find_row(p.page_indptr, p.batch, static_cast<int32_t>(j));
        const StepRecord rec = p.rec[r];
        const int32_t col = static_cast<int32_t>(j) - p.page_indptr[r];
        const int64_t cell = static_cast<int64_t>(r) * p.max_blocks + col;
        const int32_t id = page_at(p, rec, r, col);
        uint32_t tag = 0;
        if (col < pages_of(rec.cached, p.page)) {
            tag = p.table_tags[cell];
        } else if (id >= 0) {
            tag = __ldg(p.page_tags + id);
            p.table_tags[cell] = tag;
        }
        if (col >= pages_of(rec.cached, p.page) && (rec.flags & kGranted)) p.table[cell] = id;
        p.page_indices[j] = id;
        p.expected[j] = tag;
    }
    for (int64_t i = start; i < p.n_tokens; i += stride) {
        int64_t slot = -1;
        int32_t pos = 0;
        if (i < toks) {
            const int r = find_row(p.token_indptr, p.batch, static_cast<int32_t>(i));
            const StepRecord rec = p.rec[r];
            if (rec.flags & kListed) {
                pos = rec.cached + (static_cast<int32_t>(i) - p.token_indptr[r]);
                const int32_t id = rec.flags & kGranted ? page_at(p, rec, r, pos / p.page) : -1;
                if (id >= 0) slot = static_cast<int64_t>(id) * p.page + pos % p.page;
            }
        }
        p.slots[i] = slot;
        p.positions[i] = pos;
    }
}

}  // namespace fkv

using namespace fkv;

extern "C" size_t kv_step_tables_workspace_size(int32_t batch) {
    if (batch < 0) return 0;
    const size_t n = sizeof(StepRecord) * static_cast<size_t>(batch);
    return (n + 255) / 256 * 256 + 256;
}

extern "C" fkv_status kv_step_tables(const int32_t *cached_lens, const int32_t *new_lens, int32_t batch,
                                     int32_t *block_table, uint32_t *block_tags, int32_t max_blocks,
                                     const int32_t *free_pages, int32_t num_free, const int32_t *free_count,
                                     const uint32_t *page_tags, int32_t num_pages, int32_t page_size,
                                     int32_t *step_lens, int32_t *cached_lens_out, uint8_t *refused,
                                     int32_t *page_indptr, int32_t *page_indices, uint32_t *expected_tags,
                                     int32_t nnz, int32_t *token_indptr, int64_t *slot_mapping,
                                     int32_t *positions, int32_t n_tokens, int32_t *free_left, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    if (batch < 0 || max_blocks <= 0 || num_free < 0 || num_pages <= 0 || page_size <= 0 || nnz < 0 || n_tokens < 0)
        return FKV_ERR_INVALID_ARG;
    if (!free_count || !free_left || !page_indptr || !token_indptr || !page_tags || !workspace)
        return FKV_ERR_INVALID_ARG;
    if (batch > 0 && (!cached_lens || !new_lens || !block_table || !block_tags || !step_lens || !cached_lens_out ||
                      !refused))
        return FKV_ERR_INVALID_ARG;
    if (num_free > 0 && !free_pages) return FKV_ERR_INVALID_ARG;
    if (nnz > 0 && (!page_indices || !expected_tags)) return FKV_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!slot_mapping || !positions)) return FKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < kv_step_tables_workspace_size(batch))
        return FKV_ERR_INVALID_ARG;
    uint32_t *err = device_error_word();
    const int sms = device_sm_count();
    if (!err || sms <= 0) return FKV_ERR_CUDA;
    const StepParams p{cached_lens, new_lens, block_table, block_tags, free_pages, free_count, page_tags, step_lens,
                       cached_lens_out, refused, page_indptr, page_indices, expected_tags, token_indptr, slot_mapping,
                       positions, free_left, static_cast<StepRecord *>(workspace), err, batch, max_blocks, num_free,
                       num_pages, page_size, nnz, n_tokens};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_pdl(step_plan_kernel, dim3(1), dim3(kTabThreads), 0, st, p) != cudaSuccess) return FKV_ERR_CUDA;
    const int64_t most = nnz > n_tokens ? nnz : n_tokens;
    int64_t blocks = (most + kFillThreads - 1) / kFillThreads;
    if (blocks > 8 * sms) blocks = 8 * sms;
    if (blocks == 0) return FKV_OK;
    return launch_pdl(step_fill_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kFillThreads), 0, st, p) ==
                   cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}
