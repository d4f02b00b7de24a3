// A serving step's bookkeeping on the GPU: offsets, positions, page tables and slots from request
// lengths (the integer formulas stand at cdr_build_page_tables in chunk_dr.h).
//
// A new page's first position is always one of the request's new tokens, so the token at it writes
// the table entry and everything after the prefix sums is one independent step a token.  What it
// costs is latency: the sums over the requests are one workgroup's work, and up to PAGES_ONE tokens the
// same workgroup goes on with the tokens, one launch in all.  Beyond that a second launch spreads the
// tokens over the device.  256 requests, one launch against two: 256 tokens 6.7 and 8.0 us, 1024 tokens
// 7.1 and 8.9, 4096 tokens 11.0 and 8.9, 16384 tokens 30 and 9.6.
#include "chunk_dr.h"
#include "cdr_common.h"

namespace cdr {

namespace {

constexpr int PAGES_THREADS = 1024;
constexpr int PAGES_ONE = 2048;     // tokens that the scanning workgroup handles by itself
constexpr int PAGES_LDS = 4096;     // requests whose offsets fit the copy in LDS

struct PageArgs {
    const int32_t* query;
    const int32_t* context;
    int32_t* table;
    const int32_t* free_pages;
    const int32_t* head_in;
    int32_t* head_out;
    int32_t* cu;
    int32_t* lens;
    int32_t* pos;
    int32_t* slot;
    int32_t* shortage;
    int32_t* first;      // workspace [N]: index into free_pages of a request's first new page
    int n, cols, num_free, page, cap;
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int page) { return (tokens + page - 1) / page; }

// inclusive sums of two values over the workgroup; `tot` gets the totals
__device__ __forceinline__ void scan2(int64_t& a, int64_t& b, int64_t (*buf)[2], int64_t (&tot)[2]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int64_t x = __shfl_up(a, m, 64), y = __shfl_up(b, m, 64);
        if (lane >= m) a += x, b += y;
    }
    if (lane == 63) buf[wave][0] = a, buf[wave][1] = b;
    __syncthreads();
    int64_t pa = 0, pb = 0, ta = 0, tb = 0;
#pragma unroll 2
    for (int i = 0; i < PAGES_THREADS / 64; ++i) {
        if (i < wave) pa += buf[i][0], pb += buf[i][1];
        ta += buf[i][0], tb += buf[i][1];
    }
    a += pa, b += pb;
    tot[0] = ta, tot[1] = tb;
    __syncthreads();
}

// one token's position, slot and, where it opens a page, table entry; cu is the offsets' copy
__device__ __forceinline__ void one_token(const PageArgs& a, const int32_t* cu, int t) {
    int lo = 0, hi = a.n;   // the first request whose end lies behind t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    int p = 0, slot = -1;
    if (lo < a.n) {
        const int ctx = max(a.context[lo], 0);
        const int64_t at = (int64_t)ctx + t - cu[lo];
        p = (int)min(at, (int64_t)INT32_MAX);
        const int64_t j = at / a.page;
        if (j < a.cols) {
            const int held = (int)min(pages_of(ctx, a.page), (int64_t)a.cols);
            int32_t* entry = a.table + (size_t)lo * a.cols + j;
            int page;
            if (j < held) {
                page = *entry;
            } else {
                const int64_t f = (int64_t)a.first[lo] + j - held;
                page = f < a.num_free ? a.free_pages[f] : -1;
                if (at == j * a.page) *entry = page;
            }
            if (page >= 0) {
                const int64_t s = (int64_t)page * a.page + (at - j * a.page);
                if (s <= INT32_MAX) slot = (int)s;
            }
        }
    }
    a.pos[t] = p;
    a.slot[t] = slot;
}

__global__ __launch_bounds__(PAGES_THREADS) void page_scan_kernel(PageArgs a, int tokens_too) {
    __shared__ int64_t buf[PAGES_THREADS / 64][2];
    __shared__ int32_t cu_lds[PAGES_LDS + 1];
    const int tid = threadIdx.x;
    const int64_t head = min(max(a.head_in[0], 0), a.num_free);
    int64_t tokens = 0;    // before this chunk of requests, not yet cut at cap
    int64_t pages = head;
    int64_t beyond = 0;
    if (tid == 0) a.cu[0] = 0, cu_lds[0] = 0;
    for (int base = 0; base < a.n; base += PAGES_THREADS) {
        const int i = base + tid;
        const bool live = i < a.n;
        const int64_t q = live ? max(a.query[i], 0) : 0, ctx = live ? max(a.context[i], 0) : 0;
        int64_t ends = q, none = 0, tot[2];
        scan2(ends, none, buf, tot);
        const int64_t end = min(tokens + ends, (int64_t)a.cap), start = min(tokens + ends - q, (int64_t)a.cap);
        const int64_t len = ctx + end - start;
        const int64_t full = pages_of(len, a.page);
        const int64_t held = min(pages_of(ctx, a.page), (int64_t)a.cols), upto = min(full, (int64_t)a.cols);
        int64_t need = upto - held, over = full - upto;
        int64_t sum = need, oversum = over, ptot[2];
        scan2(sum, oversum, buf, ptot);
        if (live) {
            a.cu[i + 1] = (int32_t)end;
            if (i < PAGES_LDS) cu_lds[i + 1] = (int32_t)end;
            a.lens[i] = (int32_t)min(len, (int64_t)INT32_MAX);
            a.first[i] = (int32_t)min(pages + sum - need, (int64_t)INT32_MAX);
        }
        tokens += tot[0];
        pages += ptot[0];
        beyond += ptot[1];
    }
    __syncthreads();   // every thread has read head_in
    if (tid == 0) {
        a.head_out[0] = (int32_t)min(pages, (int64_t)a.num_free);
        const int64_t missing = max(pages - a.num_free, (int64_t)0) + beyond;
        a.shortage[0] = (int32_t)min(missing, (int64_t)INT32_MAX);
    }
    if (!tokens_too) return;
    __threadfence_block();
    __syncthreads();
    const int32_t* cu = a.n <= PAGES_LDS ? cu_lds : a.cu;
    for (int t = tid; t < a.cap; t += PAGES_THREADS) one_token(a, cu, t);
}

__global__ __launch_bounds__(256) void page_token_kernel(PageArgs a) {
    __shared__ int32_t cu_lds[PAGES_LDS + 1];
    const int32_t* cu = a.cu;
    if (a.n <= PAGES_LDS) {
        for (int i = threadIdx.x; i <= a.n; i += 256) cu_lds[i] = a.cu[i];
        __syncthreads();
        cu = cu_lds;
    }
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < a.cap; t += (int64_t)gridDim.x * 256)
        one_token(a, cu, (int)t);
}

}  // namespace

}  // namespace cdr

extern "C" {

size_t cdr_page_tables_workspace_bytes(int32_t N) { return N > 0 ? (size_t)N * sizeof(int32_t) : 0; }

cdr_status cdr_build_page_tables(int32_t N, int32_t table_cols, int32_t num_free, int32_t page_size, int32_t max_tokens,
                                 const int32_t* query_lens, const int32_t* context_lens, int32_t* block_table,
                                 const int32_t* free_pages, const int32_t* free_head, int32_t* free_head_out,
                                 int32_t* cu_seqlens, int32_t* seq_lens, int32_t* positions, int32_t* slot_map,
                                 int32_t* shortage, void* workspace, size_t workspace_bytes, void* stream) {
    if (N <= 0 || table_cols <= 0 || num_free < 0 || page_size <= 0 || max_tokens < 0) return CDR_ERR_BAD_SHAPE;
    if (!query_lens || !context_lens || !block_table || !free_head || !free_head_out || !cu_seqlens || !seq_lens ||
        !shortage || (num_free > 0 && !free_pages) || (max_tokens > 0 && (!positions || !slot_map)))
        return CDR_ERR_NULL_ARG;
    if (!workspace || workspace_bytes < cdr_page_tables_workspace_bytes(N)) return CDR_ERR_WORKSPACE;
    cdr::PageArgs a;
    a.query = query_lens;
    a.context = context_lens;
    a.table = block_table;
    a.free_pages = free_pages;
    a.head_in = free_head;
    a.head_out = free_head_out;
    a.cu = cu_seqlens;
    a.lens = seq_lens;
    a.pos = positions;
    a.slot = slot_map;
    a.shortage = shortage;
    a.first = static_cast<int32_t*>(workspace);
    a.n = N;
    a.cols = table_cols;
    a.num_free = num_free;
    a.page = page_size;
    a.cap = max_tokens;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool one = max_tokens <= cdr::PAGES_ONE;
    hipLaunchKernelGGL(cdr::page_scan_kernel, dim3(1), dim3(cdr::PAGES_THREADS), 0, s, a, one ? 1 : 0);
    if (hipGetLastError() != hipSuccess) return CDR_ERR_HIP;
    if (!one) {
        const int64_t wgs = ((int64_t)max_tokens + 255) / 256;
        hipLaunchKernelGGL(cdr::page_token_kernel, dim3((unsigned)(wgs < 2048 ? wgs : 2048)), dim3(256), 0, s, a);
        if (hipGetLastError() != hipSuccess) return CDR_ERR_HIP;
    }
    return CDR_OK;
}

}  // extern "C"
