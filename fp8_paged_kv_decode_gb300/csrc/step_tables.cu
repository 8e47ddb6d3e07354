// step_tables.cu -- a step's page table, slots and positions from the requests'
// lengths, on the device.
//
// Integer work: prefix sums over the requests (CSR rows, tokens, pages to take)
// and then one independent entry per page-table cell and per token.  Two
// launches: a single block scans the requests and leaves one record per request
// in the workspace, then a grid fills the entries, four neighbours to a thread
// (one search for their request, 16-byte stores).  The fill reads only the
// records, so the length and free-count outputs may be the inputs' own arrays.
// Bytes: 16 per page-table entry (id and tag, in and out) and 12 per token; both
// launches are bound by latency: the scan's two block-wide steps, and the
// fill's chain of search, record, page id, tag.  64 requests (20 thousand
// entries) take 6.4 us, one request 4.7, 256 prompt chunks (524 thousand tokens)
// 8.7; one launch of a cluster of eight blocks that scan for themselves took 6.8,
// 4.8 and 33.6 us, and 9.1 against 6.0 on 64 requests of 1024 pages each.
#include "fkv_common.cuh"

namespace fkv {

constexpr int kTabThreads = 1024;               // most threads of the scan's block
constexpr int kFillThreads = 256;
constexpr int kListed = 1, kGranted = 2;        // record flags

struct alignas(16) StepRecord {
    int32_t cached, have;     // tokens and pages held (0 for lengths that are not valid)
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
    int32_t batch, max_blocks, num_free, num_pages, nnz, n_tokens;
    uint32_t page;
    int32_t page_shift;       // log2 of the page size, -1 if it is not a power of two
    bool wide;                // the entry and token arrays are 16-byte aligned
    int32_t token_run;        // tokens of a thread's run: kRun, or 1 where requests have few each
};

// Pages that hold so many tokens (below 2^31).
__device__ __forceinline__ int32_t pages_of(const StepParams &p, uint32_t tokens) {
    const uint32_t up = tokens + (p.page - 1);                 // below 2^32
    return static_cast<int32_t>(p.page_shift >= 0 ? up >> p.page_shift : up / p.page);
}

// Inclusive prefix sums of v[0 .. K - 1] over the block's threads and their
// totals, with one barrier: every warp scans the warps' totals for itself.
template <int K>
__device__ __forceinline__ void block_scan(int64_t (&v)[K], int64_t (&total)[K], int64_t (*s_warp)[32]) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t y = __shfl_up_sync(0xffffffffu, v[k], o);
            if (lane >= o) v[k] += y;
        }
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < K; ++k) s_warp[k][wid] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t own = lane < warps ? s_warp[k][lane] : 0;
        int64_t x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        v[k] += __shfl_sync(0xffffffffu, x - own, wid);
        total[k] = __shfl_sync(0xffffffffu, x, 31);
    }
}

__global__ void __launch_bounds__(kTabThreads)
step_plan_kernel(const StepParams p) {
    __shared__ int64_t s_one[2][32], s_two[1][32];
    __shared__ int s_used, s_refused;
    if (threadIdx.x == 0) s_used = s_refused = 0;
    grid_dep_wait();
    grid_dep_launch();
    const int32_t free = min(max(*p.free_count, 0), p.num_free);
    int64_t rows = 0, toks = 0, taken = 0;     // sums over the requests before this chunk
    int used = 0, refused = 0;
    for (int base = 0; base < p.batch; base += blockDim.x) {
        const int r = base + threadIdx.x;
        const bool in = r < p.batch;
        const int32_t c = in ? p.cached[r] : 0, n = in ? p.fresh[r] : 0;
        const bool lens = c >= 0 && n >= 0 && static_cast<uint32_t>(c) + static_cast<uint32_t>(n) <= 0x7FFFFFFFu;
        const int32_t len = lens ? c + n : 0;
        int32_t pages = pages_of(p, len);
        const bool valid = lens && pages <= p.max_blocks;
        if (!valid) pages = 0;
        int64_t one[2] = {pages, max(n, 0)}, sum[2];
        block_scan<2>(one, sum, s_one);
        const int64_t row_end = rows + one[0], tok_end = toks + one[1];
        rows += sum[0];
        toks += sum[1];
        const bool fits = valid && row_end <= p.nnz && tok_end <= p.n_tokens;
        const int32_t need = fits ? pages - pages_of(p, c) : 0;
        int64_t two[1] = {need}, sum2[1];
        block_scan<1>(two, sum2, s_two);
        const int64_t need_end = taken + two[0];
        taken += sum2[0];
        const bool granted = fits && (need == 0 || need_end <= free);
        if (in) {
            p.page_indptr[r + 1] = static_cast<int32_t>(min(row_end, static_cast<int64_t>(p.nnz)));
            p.token_indptr[r + 1] = static_cast<int32_t>(min(tok_end, static_cast<int64_t>(p.n_tokens)));
            p.step_lens[r] = granted ? len : 0;
            p.cached_out[r] = granted ? len : c;
            p.refused[r] = granted ? 0 : 1;
            StepRecord rec;
            rec.cached = valid ? c : 0;
            rec.have = valid ? pages_of(p, c) : 0;
            rec.top = granted ? static_cast<int32_t>(free - 1 - (need_end - need)) : -1;
            rec.flags = (valid ? kListed : 0) | (granted ? kGranted : 0);
            *reinterpret_cast<int4 *>(p.rec + r) = *reinterpret_cast<const int4 *>(&rec);
            // Pages are granted to every request up to the first that found too
            // few: the last granted one's sum is what was taken.
            if (granted && need > 0) used = max(used, static_cast<int>(need_end));
            if (!granted) refused = 1;
        }
    }
    used = __reduce_max_sync(0xffffffffu, used);
    refused = __reduce_or_sync(0xffffffffu, refused);
    __syncthreads();                           // s_used, s_refused are set (and an empty batch's too)
    if ((threadIdx.x & 31) == 0) {
        atomicMax(&s_used, used);              // whole numbers: any order gives the same
        atomicOr(&s_refused, refused);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        p.page_indptr[0] = 0;
        p.token_indptr[0] = 0;
        *p.free_left = free - s_used;
        if (s_refused) atomicOr(p.err, FKV_DEVERR_TABLES);
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

__device__ __forceinline__ StepRecord load_record(const StepParams &p, int r) {
    const int4 v = __ldg(reinterpret_cast<const int4 *>(p.rec + r));
    return StepRecord{v.x, v.y, v.z, v.w};
}

// Page `col` of a request: from its table where it held it already, else from
// the free list.  -1 (and the error bit) for an id outside the pool, -1 for a
// page it was not granted.
__device__ __forceinline__ int32_t page_at(const StepParams &p, const StepRecord &rec, int r, int32_t col) {
    int32_t id;
    if (col < rec.have) {
        id = __ldg(p.table + static_cast<int64_t>(r) * p.max_blocks + col);
    } else {
        if (!(rec.flags & kGranted)) return -1;
        id = __ldg(p.free_pages + (rec.top - (col - rec.have)));
    }
    if (id < 0 || id >= p.num_pages) {
        atomicOr(p.err, FKV_DEVERR_TABLES);
        return -1;
    }
    return id;
}

// A thread's run of neighbouring entries: the request of the first by search,
// then onwards.  The following request's record is loaded with the first one's,
// so a run that passes one border waits for nothing more.
constexpr int kRun = 4;
struct Walk {
    int r;
    int32_t first, next, next2;       // the request's entries are [first, next), its successor's [next, next2)
    StepRecord rec, rec2;
};
__device__ __forceinline__ Walk walk_from(const StepParams &p, const int32_t *indptr, int32_t i) {
    Walk w;
    w.r = find_row(indptr, p.batch, i);
    const int r2 = min(w.r + 1, p.batch - 1);
    w.first = __ldg(indptr + w.r);
    w.next = __ldg(indptr + w.r + 1);
    w.next2 = __ldg(indptr + r2 + 1);
    w.rec = load_record(p, w.r);
    w.rec2 = load_record(p, r2);
    return w;
}
// On to the request of entry i >= w.next.
__device__ __forceinline__ void walk_on(const StepParams &p, const int32_t *indptr, Walk &w, int32_t i) {
    ++w.r;
    w.first = w.next;
    w.next = w.next2;
    w.rec = w.rec2;
    if (i < w.next) {                                          // the successor's successor, should the run reach it
        const int r2 = min(w.r + 1, p.batch - 1);
        w.next2 = __ldg(indptr + r2 + 1);
        w.rec2 = load_record(p, r2);
        return;
    }
    do {                                                       // requests without entries are passed over
        ++w.r;
        w.first = w.next;
        w.next = __ldg(indptr + w.r + 1);
    } while (i >= w.next);
    const int r2 = min(w.r + 1, p.batch - 1);
    w.rec = load_record(p, w.r);
    w.next2 = __ldg(indptr + r2 + 1);
    w.rec2 = load_record(p, r2);
}

__global__ void __launch_bounds__(kFillThreads)
step_fill_kernel(const StepParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int32_t rows = __ldg(p.page_indptr + p.batch), toks = __ldg(p.token_indptr + p.batch);
    const uint32_t row_runs = (static_cast<uint32_t>(rows) + kRun - 1) / kRun;
    const uint32_t tok_runs = (static_cast<uint32_t>(p.n_tokens) + p.token_run - 1) / p.token_run;
    const uint32_t stride = gridDim.x * kFillThreads;
    // runs of page-table entries first, then runs of tokens
    for (uint64_t run = blockIdx.x * kFillThreads + threadIdx.x; run < static_cast<uint64_t>(row_runs) + tok_runs;
         run += stride) {
        if (run < row_runs) {
            const int32_t j0 = static_cast<int32_t>(run) * kRun, m = min(kRun, rows - j0);
            Walk w = walk_from(p, p.page_indptr, j0);
            int32_t id[kRun];
            uint32_t tag[kRun];
            int64_t cell[kRun];
            bool fresh[kRun];
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                const int32_t j = j0 + e;
                id[e] = -1;
                tag[e] = 0;
                fresh[e] = false;
                if (e >= m) continue;
                if (j >= w.next) walk_on(p, p.page_indptr, w, j);
                const int32_t col = j - w.first;
                cell[e] = static_cast<int64_t>(w.r) * p.max_blocks + col;
                id[e] = page_at(p, w.rec, w.r, col);
                fresh[e] = col >= w.rec.have && (w.rec.flags & kGranted);
                if (col < w.rec.have) tag[e] = __ldg(p.table_tags + cell[e]);
                else if (id[e] >= 0) tag[e] = __ldg(p.page_tags + id[e]);
            }
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                if (!fresh[e]) continue;
                p.table[cell[e]] = id[e];
                if (id[e] >= 0) p.table_tags[cell[e]] = tag[e];
            }
            if (m == kRun && p.wide) {
                reinterpret_cast<int4 *>(p.page_indices)[run] = make_int4(id[0], id[1], id[2], id[3]);
                reinterpret_cast<uint4 *>(p.expected)[run] = make_uint4(tag[0], tag[1], tag[2], tag[3]);
            } else {
#pragma unroll
                for (int e = 0; e < kRun; ++e) {
                    if (e >= m) continue;
                    p.page_indices[j0 + e] = id[e];
                    p.expected[j0 + e] = tag[e];
                }
            }
        } else {
            const uint32_t run_t = static_cast<uint32_t>(run - row_runs);
            const int32_t i0 = static_cast<int32_t>(run_t) * p.token_run, m = min(p.token_run, p.n_tokens - i0);
            int64_t slot[kRun] = {-1, -1, -1, -1};
            int32_t pos[kRun] = {0, 0, 0, 0};
            if (i0 < toks) {
                Walk w = walk_from(p, p.token_indptr, i0);
                int32_t col_at = -1, id = -1;                  // the page looked up last
#pragma unroll
                for (int e = 0; e < kRun; ++e) {
                    const int32_t i = i0 + e;
                    if (e >= m || i >= toks) continue;
                    if (i >= w.next) {
                        walk_on(p, p.token_indptr, w, i);
                        col_at = -1;
                    }
                    if (!(w.rec.flags & kListed)) continue;
                    pos[e] = w.rec.cached + (i - w.first);
                    if (!(w.rec.flags & kGranted)) continue;
                    const uint32_t at = static_cast<uint32_t>(pos[e]);
                    const uint32_t col = p.page_shift >= 0 ? at >> p.page_shift : at / p.page;
                    if (static_cast<int32_t>(col) != col_at) {
                        col_at = static_cast<int32_t>(col);
                        id = page_at(p, w.rec, w.r, col_at);
                    }
                    if (id >= 0) slot[e] = static_cast<int64_t>(id) * p.page + (at - col * p.page);
                }
            }
            if (m == kRun && p.wide) {
                longlong2 *s = reinterpret_cast<longlong2 *>(p.slots) + 2 * static_cast<uint64_t>(run_t);
                s[0] = make_longlong2(slot[0], slot[1]);
                s[1] = make_longlong2(slot[2], slot[3]);
                reinterpret_cast<int4 *>(p.positions)[run_t] = make_int4(pos[0], pos[1], pos[2], pos[3]);
            } else {
#pragma unroll
                for (int e = 0; e < kRun; ++e) {
                    if (e >= m) continue;
                    p.slots[i0 + e] = slot[e];
                    p.positions[i0 + e] = pos[e];
                }
            }
        }
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
    const uint32_t page = static_cast<uint32_t>(page_size);
    const bool wide = aligned16(page_indices) && aligned16(expected_tags) && aligned16(slot_mapping) && aligned16(positions);
    // A decode step's tokens are each a request of their own: one to a thread.
    const int32_t token_run = n_tokens <= kRun * static_cast<int64_t>(batch) ? 1 : kRun;
    const StepParams p{cached_lens, new_lens, block_table, block_tags, free_pages, free_count, page_tags, step_lens,
                       cached_lens_out, refused, page_indptr, page_indices, expected_tags, token_indptr, slot_mapping,
                       positions, free_left, static_cast<StepRecord *>(workspace), err, batch, max_blocks, num_free,
                       num_pages, nnz, n_tokens, page, (page & (page - 1)) ? -1 : __builtin_ctz(page), wide, token_run};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned scan = batch >= kTabThreads ? kTabThreads : batch <= 32 ? 32u : (static_cast<unsigned>(batch) + 31u) & ~31u;
    if (launch_pdl(step_plan_kernel, dim3(1), dim3(scan), 0, st, p) != cudaSuccess) return FKV_ERR_CUDA;
    const int64_t runs = (static_cast<int64_t>(nnz) + kRun - 1) / kRun + (static_cast<int64_t>(n_tokens) + token_run - 1) / token_run;
    int64_t blocks = (runs + kFillThreads - 1) / kFillThreads;
    if (blocks > 8 * sms) blocks = 8 * sms;
    if (blocks == 0) return FKV_OK;
    return launch_pdl(step_fill_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kFillThreads), 0, st, p) ==
                   cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}
