// Block tables, slots and sequence bounds of a step from the rows' lengths (include/pkv.h, pkv_tables_grow,
// pkv_tables_release).
//
// Row b holds L_b tokens in ceil(L_b / 16) pages and gets n_b more. With need_b = ceil((L_b + n_b) / 16) - ceil(L_b / 16), page j
// of a row's new ones is entry count - 1 - (sum of need over the rows before it) - j of the stack of free pages, and its tokens'
// packed rows begin at the sum of n over the rows before it: two prefix sums over the rows, of which everything else follows
// independently, so nothing is read that the same call writes. Every CTA makes both sums (at most 4096 rows, 8 bytes a row) and
// takes a share of the tokens and pages, for each of which it finds the row by bisection; what may be updated in place (lengths,
// the stack's height) is written by the CTA that ends last, when all have read it.
//
// Bound: latency (two dependent round trips, lengths, then table or stack, and the scan between them), then the
// 12 bytes a token that are written. Measured on a GB300, in a captured graph: 256 rows of one new token 4.1-5.5 us, 64 rows of up to
// 4096 (130k tokens) 6.0-7.9 us, 128 of 256 rows released (130k pages) 4.8 us; as calls 8.5-11 us, which the binding takes.
#include <algorithm>

#include "pkv_internal.h"
#include "pkv_launch.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct Two {
    int64_t a, b;
};

// Exclusive sums over the CTA's threads, and the totals. Uses (and leaves) the CTA synchronised.
__device__ __forceinline__ Two scan(Two x, Two& total, Two* s_warp) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Two incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, incl.a, o), b = __shfl_up_sync(0xffffffffu, incl.b, o);
        if (lane >= o) {
            incl.a += a;
            incl.b += b;
        }
    }
    __syncthreads();  // the sums of a scan before this one have been read
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    Two before{incl.a - x.a, incl.b - x.b};
    total = Two{0, 0};
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const Two y = s_warp[i];
        if (i < warp) {
            before.a += y.a;
            before.b += y.b;
        }
        total.a += y.a;
        total.b += y.b;
    }
    return before;
}

__device__ __forceinline__ int pages_of(int64_t tokens) { return (int)((tokens + kPageSize - 1) / kPageSize); }

// The last row r of [0, rows) with first[r] <= i (rows of nothing lie before others that begin at the same place).
__device__ __forceinline__ int row_of(const int32_t* first, int rows, int i) {
    int lo = 0, hi = rows - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// True in the CTA that is the last to get here, when all others have read what it is to overwrite.
__device__ __forceinline__ bool last_cta(pkv_ws_header* hdr) {
    __shared__ bool s_last;
    __syncthreads();
    if (threadIdx.x == 0) {
        s_last = true;
        if (gridDim.x > 1) {
            __threadfence();
            s_last = atomicAdd(&hdr->ctas_done, 1u) == gridDim.x - 1;
            if (s_last) atomicExch(&hdr->ctas_done, 0u);
        }
    }
    __syncthreads();
    return s_last;
}

__global__ void __launch_bounds__(kThreads) grow_kernel(const TablesParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    extern __shared__ int32_t s_rows[];  // of every row: first packed token, first of the new pages, tokens held
    __shared__ Two s_warp[kWarps];
    int32_t* s_tok = s_rows;
    int32_t* s_page = s_rows + p.B;
    int32_t* s_len = s_rows + 2 * p.B;
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    const int given = *p.free_count;
    const int count = min(max(given, 0), p.num_pages);
    uint32_t status = given == count ? 0u : PKV_STATUS_BAD_LEN;
    auto row = [&](int b, int& n) {  // tokens held and, where the row is in order, new ones
        const int len = p.seq_lens[b];
        n = p.new_tokens[b];
        if (len < 0 || n < 0 || (int64_t)len + n > (int64_t)p.max_pages * kPageSize) {
            status |= PKV_STATUS_BAD_LEN;
            n = 0;
        }
        return len;
    };
    auto need = [](int len, int n) { return n == 0 ? 0 : pages_of((int64_t)len + n) - pages_of(len); };
    Two mine{0, 0}, total;
    int len0 = 0, n0 = 0;  // the thread's first row (up to 512 rows its only one) is read once
    if (b0 < b1) len0 = row(b0, n0);
    auto again = [&](int b, int& n) {
        if (b > b0) return row(b, n);
        n = n0;
        return len0;
    };
    for (int b = b0; b < b1; ++b) {
        int n;
        const int len = again(b, n);
        mine.a += n;
        mine.b += need(len, n);
    }
    Two before = scan(mine, total, s_warp);
    // Rows that do not fit get nothing: tokens behind the slots' number, pages behind the stack's.
    const int64_t capacity = p.slots || p.positions ? p.capacity : INT32_MAX;
    const bool all = total.a <= capacity && total.b <= count;
    Two at = before;
    auto served = [&](int len, int n, Two& upto) {  // upto: sums up to the row
        const int m = need(len, n);
        upto.a += n;
        upto.b += m;
        return n > 0 && upto.a <= capacity && (m == 0 || upto.b <= count);
    };
    if (!all) {  // the packed rows of those that are served
        Two upto = before, x{0, 0}, sum;
        for (int b = b0; b < b1; ++b) {
            int n;
            const int len = again(b, n);
            if (served(len, n, upto)) {
                x.a += n;
                x.b += need(len, n);
            } else if (n > 0) {
                status |= PKV_STATUS_NO_PAGES;
            }
        }
        at.a = scan(x, sum, s_warp).a;
        total = sum;
    }
    {
        Two upto = before;
        for (int b = b0; b < b1; ++b) {
            int n;
            const int len = again(b, n);
            s_tok[b] = (int32_t)at.a;
            s_page[b] = (int32_t)min(at.b, (int64_t)INT32_MAX);
            s_len[b] = len;
            if (!served(len, n, upto)) n = 0;
            at.a += n;
            at.b = upto.b;
            if (blockIdx.x == 0) {
                if (p.cu_seqlens) p.cu_seqlens[b] = s_tok[b];
                if (p.start) p.start[b] = len;
            }
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.cu_seqlens) p.cu_seqlens[p.B] = (int32_t)total.a;
    if (status && blockIdx.x == 0) atomicOr(&p.hdr->status, status);
    __syncthreads();
    // Pages of the stack, the uppermost first. One that is not of the pool is handed out as it is: whoever reads its entry in the
    // table says so.
    auto free_page = [&](int64_t i) { return p.free_pages[count - 1 - i]; };
    const int64_t self = (int64_t)blockIdx.x * kThreads + threadIdx.x, all_threads = (int64_t)gridDim.x * kThreads;
    auto next_token = [&](int b) { return b + 1 < p.B ? s_tok[b + 1] : (int32_t)total.a; };
    if (p.slots || p.positions)
        for (int64_t i = self; i < total.a; i += all_threads) {
            const int b = row_of(s_tok, p.B, (int)i);
            const int pos = s_len[b] + ((int)i - s_tok[b]), held = pages_of(s_len[b]), lp = pos / kPageSize;
            if (p.slots) {
                const int64_t page = lp < held ? p.block_table[(int64_t)b * p.max_pages + lp] : free_page((int64_t)s_page[b] + lp - held);
                p.slots[i] = page * kPageSize + pos % kPageSize;
            }
            if (p.positions) p.positions[i] = pos;
        }
    // The new entries, row by row: those of a row are as many as its tokens need, whatever the sums of rows that got nothing say.
    for (int b = blockIdx.x * kWarps + (threadIdx.x >> 5); b < p.B; b += gridDim.x * kWarps) {
        const int n = next_token(b) - s_tok[b];
        const int m = need(s_len[b], n), held = pages_of(s_len[b]);
        for (int j = threadIdx.x & 31; j < m; j += 32)
            p.block_table[(int64_t)b * p.max_pages + held + j] = free_page((int64_t)s_page[b] + j);
    }
    if (last_cta(p.hdr)) {
        for (int b = threadIdx.x; b < p.B; b += kThreads) p.seq_lens_out[b] = s_len[b] + (next_token(b) - s_tok[b]);
        if (threadIdx.x == 0) *p.free_count_out = count - (int32_t)total.b;
    }
}

__global__ void __launch_bounds__(kThreads) release_kernel(const TablesParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    extern __shared__ int32_t s_rows[];  // of every row: first of the released pages; its length afterwards
    __shared__ Two s_warp[kWarps];
    int32_t* s_page = s_rows;
    int32_t* s_len = s_rows + p.B;
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    const int count = *p.free_count;
    uint32_t status = 0;
    auto row = [&](int b, int& len) {  // pages that the row gives back
        len = p.seq_lens[b];
        if (p.released[b] == 0) return 0;
        if (len < 0 || len > (int64_t)p.max_pages * kPageSize) {
            status |= PKV_STATUS_BAD_LEN;
            return 0;
        }
        return pages_of(len);
    };
    Two mine{0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        int len;
        mine.a += row(b, len);
    }
    Two at = scan(mine, total, s_warp);
    // More than the stack holds: the tables are not those of this stack, and nothing is released.
    const bool fits = count >= 0 && count + total.a <= p.num_pages;
    if (!fits) status |= PKV_STATUS_BAD_LEN;
    for (int b = b0; b < b1; ++b) {
        int len;
        const int m = row(b, len);
        s_page[b] = (int32_t)min(at.a, (int64_t)INT32_MAX);
        at.a += m;
        s_len[b] = fits && m > 0 ? 0 : len;
    }
    if (status && blockIdx.x == 0) atomicOr(&p.hdr->status, status);
    __syncthreads();
    if (fits) {
        const int64_t all_threads = (int64_t)gridDim.x * kThreads;
        for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total.a; i += all_threads) {
            const int b = row_of(s_page, p.B, (int)i);
            p.free_out[count + i] = p.block_table[(int64_t)b * p.max_pages + ((int)i - s_page[b])];
        }
    }
    if (last_cta(p.hdr)) {
        for (int b = threadIdx.x; b < p.B; b += kThreads) p.seq_lens_out[b] = s_len[b];
        if (threadIdx.x == 0) *p.free_count_out = fits ? count + (int32_t)total.a : count;
    }
}

// CTAs for `items` tokens or pages: one a thread, as every CTA's scan takes the same time side by side (130k tokens: 9.3 us with 8 a
// thread, 7.2 with 4, 6.0 with one; 256 tokens 5.0, 4.5, 4.1-4.6).
int grid_for(int64_t items, int num_sms) {
    return (int)std::max<int64_t>(1, std::min<int64_t>((items + kThreads - 1) / kThreads, num_sms));
}

}  // namespace

int launch_tables_grow(const TablesParams& p, int num_sms, void* stream) {
    static int configured_mask = 0;  // one bit per device ordinal (< 32)
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 32 || !(__atomic_load_n(&configured_mask, __ATOMIC_ACQUIRE) & (1 << dev))) {
        // with the static part more than the 48 KB that a launch gets without asking
        const cudaError_t e = cudaFuncSetAttribute(grow_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * PKV_MAX_BATCH * 4);
        if (e != cudaSuccess) return e;
        if (dev < 32) __atomic_fetch_or(&configured_mask, 1 << dev, __ATOMIC_ACQ_REL);
    }
    const int64_t items = std::max<int64_t>(p.slots || p.positions ? p.capacity : 0, (int64_t)p.B * 32);
    return launch_behind(grow_kernel, dim3(grid_for(items, num_sms)), dim3(kThreads), 3 * p.B * 4, static_cast<cudaStream_t>(stream), p);
}

int launch_tables_release(const TablesParams& p, int num_sms, void* stream) {
    const int64_t items = std::min<int64_t>((int64_t)p.B * p.max_pages, p.num_pages);
    return launch_behind(release_kernel, dim3(grid_for(items, num_sms)), dim3(kThreads), 2 * p.B * 4, static_cast<cudaStream_t>(stream), p);
}

}  // namespace pkv
