// The pages whose bounds promise a KV head's queries the greatest scores (include/pkv.h, pkv_select_pages).
//
// score(page) = max over the G query heads of sum_d max(q_d lo_d, q_d hi_d), lo and hi the least and greatest key of the page in
// dim d: no key of the page has a greater product with the query. With q- = min(q, 0), q+ = max(q, 0) the sum is q-.lo +
// q+.hi, one product over 256 dims, so a tile of 16 pages takes 16 mma.sync m16n8k16 (pages on the 16-row side, the heads on the
// 8-column side; tcgen05 needs 64 rows of either). The order of a contraction is free: a lane takes 16 bytes of a page's bounds
// at a time, which are its fragments of two steps, and holds the same dims of the queries.
//
// The row's last page is always selected (it holds the newest tokens), and the select - 1 greatest of the others; equal scores
// go to the lowest page. The definition is exact: sums of products of fp16 values. The fp32 scores are off by at most
// delta = 2^-15 max_g |q_g|_1 max |bound|: 16 instructions add 16 products and the sum before, each of which may lose 2^-23 of the
// greatest magnitude (17 * 16 * 2^-23 = 2^-14.9 of the sum of magnitudes, half of which are zeros of q- or q+). With T the
// (select - 1)-th greatest fp32 score, pages above T + 2 delta are in and those below T - 2 delta out whatever their exact scores
// are; those between are scored again exactly, in integers (one to four of 2048 with normal values), and ranked by those (by their sums
// rounded to 64 bits where more than 256 pages lie between).
// Bounds or queries that are not finite make a score of +inf: such pages come first.
//
// Two kernels: scores, bound by HBM (512 bytes a (page, KV head)), a warp per KV head and 16 pages, so that the heads of a page
// are read together; and a CTA per (row, KV head) that selects, bound by latency.
// Measured on a GB300 (32 query heads, 8 KV heads): one row of 2048 pages 11.8 us, 32 rows of 250-2048 pages 36 us, of which the
// bounds' 133 MB take 24 (5.6 TB/s). A selection takes 12000-14000 cycles: scores from L2 2500, the border 2000, what lies next to it
// 1500, exact scores 4000-5000 (two dependent loads), the list 1500. What moved it: the threshold bit by bit from counts of all keys
// took 10 us, the histogram takes 1; 512 threads 36 us for the 32 rows, 256 41, 1024 (one CTA an SM) 45; half a warp an exact score
// 41, a warp 43.
// Where this is weak: delta takes the row's greatest bound, so one page with a bound of 6e4 among normal ones puts all pages next to the
// border, and the selection of 32 rows of 2048 pages takes 665 us instead of 58. And a scoring CTA has a warp a KV head: 32 rows of 2048
// pages take 58 us with 8 KV heads, 44 with 4, 38 with 2 or 1, where most warps have nothing to read (0.9 TB/s with one).
#include <cuda_fp16.h>

#include <algorithm>

#include "pkv_internal.h"
#include "pkv_launch.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kTile = 16;                 // pages of a tile
constexpr int kBoundBytes = 2 * kRowBytes;  // of a (page, KV head)
constexpr int kScoreWarps = 8;
constexpr int kThreads = 512;             // of the selection
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 8192;               // keys in shared memory
constexpr int kBins = 1024;
constexpr int kList = 256;                // pages next to the border that are ranked in shared memory

__device__ __forceinline__ int row_pages(const SelectParams& p, int b, bool& bad) {
    const int len = p.seq_lens[b];
    bad = len < 0 || len > (int64_t)p.max_pages * kPageSize;
    return bad ? 0 : (len + kPageSize - 1) / kPageSize;
}

__device__ __forceinline__ int page_of(const SelectParams& p, int b, int lp) {
    const int e = p.block_table[(int64_t)b * p.max_pages + lp];
    return e >= 0 && e < p.num_pages ? e : -1;
}

__device__ __forceinline__ uint32_t bits(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }

// ---- scores --------------------------------------------------------------------------------------------------------
template <int G>
__global__ void __launch_bounds__(kScoreWarps * 32) score_kernel(const SelectParams p) {
    constexpr int kNT = (G + 7) / 8;
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const int b = blockIdx.y, first = blockIdx.x * p.tiles;
    bool bad;
    const int pages = row_pages(p, b, bad);
    if (first * kTile >= pages || pages <= p.select || p.select == 1) return;  // nothing there, or nothing to be compared
    const int tiles = min(p.tiles, (pages + kTile - 1) / kTile - first);
    // the lane's two pages of a tile; -1: none (its bounds count as 0)
    auto entry = [&](int tile, int i) {
        const int lp = (first + tile) * kTile + r + 8 * i;
        if (tile >= tiles || lp >= pages) return -1;
        const int page = page_of(p, b, lp);
        if (page < 0) atomicOr(&p.hdr->status, PKV_STATUS_BAD_PAGE);
        return page;
    };
    for (int h = warp; h < p.Hkv; h += kScoreWarps) {
        int next[2] = {entry(0, 0), entry(0, 1)};
        uint4 q[kNT][4];  // dims 32 j + 8 t .. + 7 of head r (+ 8)
        bool infinite = false;  // a query of the group
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                q[n][j] = make_uint4(0u, 0u, 0u, 0u);
                if (8 * n + r < G)
                    q[n][j] = *reinterpret_cast<const uint4*>(static_cast<const __half*>(p.q) +
                                                              ((int64_t)b * p.Hq + h * G + 8 * n + r) * kHeadDim + 32 * j + 8 * t);
                const uint32_t* w = reinterpret_cast<const uint32_t*>(&q[n][j]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    infinite = infinite || (w[e] & 0x7c00u) == 0x7c00u || (w[e] & 0x7c000000u) == 0x7c000000u;
            }
        infinite = __any_sync(kAll, infinite);
        for (int tile = 0; tile < tiles; ++tile) {
            uint4 x[2][8];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.bounds) +
                                                                 ((int64_t)max(next[i], 0) * p.Hkv + h) * kBoundBytes) + t;
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = next[i] >= 0 ? __ldcs(at + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
            }
            next[0] = entry(tile + 1, 0);
            next[1] = entry(tile + 1, 1);
            float d[kNT][4] = {};
            __half2 top[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                __half2 m = __float2half2_rn(0.f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const __half2* y = reinterpret_cast<const __half2*>(&x[i][j]);
                    m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(__habs2(y[0]), __habs2(y[1])), __hmax2_nan(__habs2(y[2]), __habs2(y[3]))));
                }
                top[i] = m;
            }
            const __half2 zero = __float2half2_rn(0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t* a = reinterpret_cast<const uint32_t*>(&x[0][j]);
                const uint32_t* c = reinterpret_cast<const uint32_t*>(&x[1][j]);
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                    uint32_t f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2 y = half2_of(reinterpret_cast<const uint32_t*>(&q[n][j & 3])[e]);
                        f[e] = bits(j < 4 ? __hmin2(y, zero) : __hmax2(y, zero));
                    }
                    mma_16816(d[n], a[0], c[0], a[1], c[1], f[0], f[1]);
                    mma_16816(d[n], a[2], c[2], a[3], c[3], f[2], f[3]);
                }
            }
            float score[2] = {-INFINITY, -INFINITY}, mag = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (8 * n + 2 * t + e < G) score[i] = fmaxf(score[i], d[n][2 * i + e]);
                float m = fmaxf(__low2float(top[i]), __high2float(top[i]));
                bool finite = isfinite(__low2float(top[i])) && isfinite(__high2float(top[i]));
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    score[i] = fmaxf(score[i], __shfl_xor_sync(kAll, score[i], o));
                    m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
                    finite = __shfl_xor_sync(kAll, (int)finite, o) && finite;
                }
                if (!finite || infinite) score[i] = INFINITY;
                if (finite) mag = fmaxf(mag, m);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mag = fmaxf(mag, __shfl_xor_sync(kAll, mag, o));
            const int64_t pair = (int64_t)b * p.Hkv + h;
            if (t == 0)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if ((first + tile) * kTile + r + 8 * i < pages) p.scores[pair * p.max_pages + (first + tile) * kTile + r + 8 * i] = score[i];
            if (lane == 0) p.tops[pair * ((p.max_pages + kTile - 1) / kTile) + first + tile] = mag;
        }
    }
}

// ---- selection -----------------------------------------------------------------------------------------------------
// Keys in the order of the scores, from their bits. (Those of decided pages are not numbers, and what a float of such bits is loaded
// and has its sign set as need not keep them.)
__device__ __forceinline__ uint32_t key_of(uint32_t u) { return u & 0x80000000u ? ~u : u | 0x80000000u; }

__device__ __forceinline__ float from_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// A sum of products of two fp16 values, exact: these are multiples of 2^-48 below 2^32, here hi * 2^-19 + lo * 2^-48 with 0 <= lo <
// 2^29. (In 64-bit floating point, of which an SM adds two a cycle, a page takes 2 us.)
struct Exact {
    int64_t hi;
    uint32_t lo;
};
__device__ __forceinline__ bool operator>(const Exact& a, const Exact& b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ bool operator==(const Exact& a, const Exact& b) { return a.hi == b.hi && a.lo == b.lo; }
__device__ __forceinline__ double rounded(const Exact& x) { return (double)x.hi * 0x1p-19 + (double)x.lo * 0x1p-48; }
constexpr int64_t kMost = INT64_MAX;         // of a score of +inf
constexpr uint32_t kInfinite = 0xff800000u;  // its key

// The exact score of a page for query heads g0 <= g < g1 of the group, by half a warp: lane l sums dims 8 l .. 8 l + 7. Both halves
// are in it together.
__device__ __forceinline__ Exact exact_score(const SelectParams& p, int b, int h, int lp, int g0, int g1) {
    const int lane = threadIdx.x & 15, G = p.Hq / p.Hkv;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __half*>(p.q) + ((int64_t)b * p.Hq + h * G) * kHeadDim) + lane;
    uint4 next = q[g0 * 16];  // on its way together with the table's entry
    const int page = page_of(p, b, lp);
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (page >= 0) {
        const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.bounds) + ((int64_t)page * p.Hkv + h) * kBoundBytes);
        lo = at[lane];
        hi = at[16 + lane];
    }
    Exact best{0, 0};
    for (int g = g0; g < g1; ++g) {
        const uint4 now = next;
        if (g + 1 < g1) next = q[(g + 1) * 16];
        int64_t x = 0, y = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            auto at = [&](const uint4& u) { return reinterpret_cast<const uint32_t*>(&u)[i >> 1] >> (16 * (i & 1)) & 0xffffu; };
            // |value| = mantissa (11 bits) * 2^(exponent - 25), exponent 1 .. 30. The greater product is with the greatest key where the
            // query is positive, with the least one where it is negative.
            auto mantissa = [](uint32_t u) { return (int)((u & 0x3ffu) + (min(u >> 10 & 31u, 1u) << 10)); };
            auto exponent = [](uint32_t u) { return (int)max(u >> 10 & 31u, 1u); };
            const uint32_t a = at(now), c = a & 0x8000u ? at(lo) : at(hi);
            const int m = mantissa(a) * mantissa(c), product = (a ^ c) & 0x8000u ? -m : m;
            const int shift = exponent(a) + exponent(c) - 2;  // in units of 2^-48: 0 .. 58
            const bool upper = shift >= 29;
            const int power = 1 << (upper ? shift - 29 : shift);
            x += (int64_t)(upper ? product : 0) * power;
            y += (int64_t)(upper ? 0 : product) * power;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            x += __shfl_xor_sync(kAll, x, o);
            y += __shfl_xor_sync(kAll, y, o);
        }
        const Exact s{x + (y >> 29), (uint32_t)y & 0x1fffffffu};
        if (g == g0 || s > best) best = s;
    }
    return best;
}

// Sum over the CTA, in every thread, and of the threads before it. s_sum is free again after the next barrier.
__device__ __forceinline__ int block_scan(int x, int& before, int* s_sum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    before = incl - x;
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    return total;
}

struct SelectSmem {
    uint32_t keys[kHeld];
    int bins[kBins];
    int sum[2][kWarps];
    float l1[kWarps], mag[kWarps];
    uint32_t low[kWarps], high[kWarps];
    int near, bin, above;
    int list[kList];
    Exact exact[kList];
};

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
    __shared__ SelectSmem sm;
    // Behind a kernel of scores lengths and queries may be read at once: it began when every CTA of that one had waited itself.
    if (p.max_pages <= p.select) grid_dependency_wait();
    const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t pair = (int64_t)b * p.Hkv + h;
    bool bad;
    const int pages = row_pages(p, b, bad);
    int32_t* out = p.pages + pair * p.select;
    if (bad && h == 0 && threadIdx.x == 0) atomicOr(&p.hdr->status, PKV_STATUS_BAD_LEN);
    if (pages <= p.select || p.select == 1) {
        grid_dependency_wait();  // what comes behind this grid comes behind the scores, too
        for (int i = threadIdx.x; i < p.select; i += kThreads) out[i] = p.select == 1 ? pages - 1 : i < pages ? i : -1;
        return;
    }
    const int n = pages - 1, want = p.select - 1;  // candidates, and how many of them
    if (threadIdx.x == 0) {
        sm.near = 0;
        out[want] = n;  // the last page
    }
    for (int i = threadIdx.x; i < kBins; i += kThreads) sm.bins[i] = 0;
    float l1 = 0.f;  // of the query heads of this warp: the greatest sum of magnitudes
    const int G = p.Hq / p.Hkv;
    for (int g = warp; g < G; g += kWarps) {
        const uint2 q = reinterpret_cast<const uint2*>(static_cast<const __half*>(p.q) + ((int64_t)b * p.Hq + h * G + g) * kHeadDim)[lane];
        const float2 x = __half22float2(half2_of(q.x)), y = __half22float2(half2_of(q.y));
        float s = fabsf(x.x) + fabsf(x.y) + fabsf(y.x) + fabsf(y.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        l1 = fmaxf(l1, isfinite(s) ? s : INFINITY);
    }
    grid_dependency_wait();
    uint32_t* scores = reinterpret_cast<uint32_t*>(p.scores) + pair * p.max_pages;
    double* exact = p.exact + pair * p.max_pages;
    const int tiles = (p.max_pages + kTile - 1) / kTile;
    const float* tops = p.tops + pair * tiles;
    float mag = (int)threadIdx.x * kTile < pages ? __ldcg(tops + threadIdx.x) : 0.f;  // (on its way together with the scores)
    uint32_t low = 0xffffffffu, high = 0u;
#pragma unroll 8
    for (int j = threadIdx.x; j < n; j += kThreads) {
        const uint32_t k = key_of(__ldcg(scores + j));
        if (j < kHeld) sm.keys[j] = k;
        low = min(low, k);
        high = max(high, k);
    }
    for (int i = threadIdx.x + kThreads; i * kTile < pages; i += kThreads) mag = fmaxf(mag, __ldcg(tops + i));
    low = __reduce_min_sync(kAll, low);
    high = __reduce_max_sync(kAll, high);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mag = fmaxf(mag, __shfl_xor_sync(kAll, mag, o));
    if (lane == 0) {
        sm.l1[warp] = l1;
        sm.mag[warp] = mag;
        sm.low[warp] = low;
        sm.high[warp] = high;
    }
    __syncthreads();
    float q1 = 0.f, top = 0.f;
    for (int w = 0; w < kWarps; ++w) {
        q1 = fmaxf(q1, sm.l1[w]);
        top = fmaxf(top, sm.mag[w]);
        low = min(low, sm.low[w]);
        high = max(high, sm.high[w]);
    }
    // Keys of longer rows than shared memory holds are read again, and decided ones written back as what gives 0 and ~0.
    auto key = [&](int j) { return j < kHeld ? sm.keys[j] : key_of(__ldcg(scores + j)); };
    auto decide = [&](int j, bool in) {
        if (j < kHeld)
            sm.keys[j] = in ? 0xffffffffu : 0u;
        else
            __stcg(scores + j, in ? 0x7fffffffu : 0xffffffffu);
    };
    // The border, the greatest key that `want` keys reach, lies in one of 1024 equal parts of the keys' range, found from a
    // histogram; where that part has many keys, in one of 1024 parts of it, and so on.
    for (int above = 0;;) {
        const int shift = max(0, 22 - __clz(high - low));
        for (int j = threadIdx.x; j < n; j += kThreads) {
            const uint32_t k = key(j);
            if (k >= low && k <= high) atomicAdd(&sm.bins[(k - low) >> shift], 1);
        }
        __syncthreads();
        int c[kBins / kThreads], sum = 0, before;  // thread 0 has the uppermost bins
        const int first = kBins - (kBins / kThreads) * (threadIdx.x + 1);
#pragma unroll
        for (int i = 0; i < kBins / kThreads; ++i) sum += c[i] = sm.bins[first + i];
        block_scan(sum, before, sm.sum[0]);
        before += above;
#pragma unroll
        for (int i = kBins / kThreads - 1; i >= 0; --i) {
            if (before < want && before + c[i] >= want) {
                sm.bin = first + i;
                sm.above = before;
                sm.near = c[i];
            }
            before += c[i];
            sm.bins[first + i] = 0;
        }
        __syncthreads();
        above = sm.above;
        low += (uint32_t)sm.bin << shift;
        high = min(high, low + ((1u << shift) - 1u));
        const bool done = shift == 0 || sm.near <= kList / 4;
        __syncthreads();
        if (done) break;
    }
    // Next to the border: scores within twice their error of it. (Queries that are not finite give scores of +inf alone.)
    const float delta = isfinite(q1) ? 0x1p-14f * q1 * top : 0.f;
    auto moved = [&](uint32_t k, float by, bool up) {
        const float x = from_key(k);
        return isfinite(x) ? key_of(__float_as_uint(up ? __fadd_ru(x, by) : __fadd_rd(x, -by))) : k;
    };
    const uint32_t above = moved(high, delta, true), below = moved(low, delta, false);
    if (threadIdx.x == 0) sm.near = 0;
    __syncthreads();
    int in = 0;
    for (int j = threadIdx.x; j < n; j += kThreads) {
        const uint32_t k = key(j);
        in += k > above;
        if (k >= below && k <= above) {
            const int i = atomicAdd(&sm.near, 1);
            if (i < kList) sm.list[i] = j;
        }
    }
    int unused;
    in = block_scan(in, unused, sm.sum[1]);
    const int room = want - in, near = sm.near;  // pages next to the border that are selected; all of them
    auto score = [&](int j, int g0, int g1) {  // by half a warp
        const Exact e = exact_score(p, b, h, j, g0, g1);
        return key(j) == kInfinite ? Exact{kMost, 0} : e;
    };
    const int half = (int)threadIdx.x >> 4, first_lane = (lane & 15) == 0;
    const int run = (n + kThreads - 1) / kThreads, p0 = min(n, (int)threadIdx.x * run), p1 = min(n, p0 + run);
    if (near <= kList) {
        if (near > room) {
            if (near * G <= kList) {  // half a warp for every head of every page
                for (int i0 = 0; i0 + 2 * warp < near * G; i0 += 2 * kWarps) {
                    const int i = min(i0 + half, near * G - 1), g = i % G;
                    const Exact e = score(sm.list[i / G], g, g + 1);
                    if (first_lane && i0 + half < near * G) sm.exact[i] = e;
                }
                __syncthreads();
                Exact best{0, 0};
                if ((int)threadIdx.x < near)
                    for (int g = 0; g < G; ++g) {
                        const Exact e = sm.exact[threadIdx.x * G + g];
                        if (g == 0 || e > best) best = e;
                    }
                __syncthreads();
                if ((int)threadIdx.x < near) sm.exact[threadIdx.x] = best;
            } else {
                for (int i0 = 0; i0 + 2 * warp < near; i0 += 2 * kWarps) {
                    const int i = min(i0 + half, near - 1);
                    const Exact e = score(sm.list[i], 0, G);
                    if (first_lane && i0 + half < near) sm.exact[i] = e;
                }
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < near; i += kThreads) {
            int rank = 0;
            if (near > room)
                for (int y = 0; y < near; ++y)
                    rank += sm.exact[y] > sm.exact[i] || (sm.exact[y] == sm.exact[i] && sm.list[y] < sm.list[i]);
            decide(sm.list[i], rank < room);
        }
        __syncthreads();
    } else {
        // Many equal or nearly equal scores: the border among the exact ones (rounded to 64 bits), bit by bit, then the lowest of
        // the pages at it.
        for (int j0 = 0; j0 < n; j0 += 2 * kWarps) {
            const int j = min(j0 + half, n - 1);
            const uint32_t k = key(j);
            const bool wanted = k >= below && k <= above;
            if (!__any_sync(kAll, wanted)) continue;
            const Exact e = score(j, 0, G);
            if (first_lane && wanted && j0 + half < n) __stcg(exact + j, rounded(e));
        }
        __syncthreads();
        auto key64 = [&](int j) {
            const uint64_t u = (uint64_t)__double_as_longlong(__ldcg(exact + j));
            return u >> 63 ? ~u : u | 1ull << 63;
        };
        uint64_t border = 0;
        auto count = [&](auto f, int turn) {
            int c = 0, ahead;
            for (int j = p0; j < p1; ++j) {
                const uint32_t k = key(j);
                c += k >= below && k <= above && f(key64(j));
            }
            const int total = block_scan(c, ahead, sm.sum[turn]);
            return make_int2(total, ahead);
        };
        for (int bit = 63; bit >= 0; --bit) {
            const uint64_t x = border | 1ull << bit;
            if (count([&](uint64_t y) { return y >= x; }, bit & 1).x >= room) border = x;
        }
        const int greater = count([&](uint64_t y) { return y > border; }, 1).x;
        int left = room - greater - count([&](uint64_t y) { return y == border; }, 0).y;
        for (int j = p0; j < p1; ++j) {
            const uint32_t k = key(j);
            if (k < below || k > above) continue;
            const uint64_t y = key64(j);
            decide(j, y > border || (y == border && left-- > 0));
        }
        __syncthreads();
    }
    // The selected pages, in order.
    int mine = 0, at;
    for (int j = p0; j < p1; ++j) mine += key(j) > above;
    block_scan(mine, at, sm.sum[0]);
    if (mine > 0)
        for (int j = p0; j < p1; ++j)
            if (key(j) > above) out[at++] = j;
}

template <int G>
int launch_scores(const SelectParams& p, cudaStream_t stream) {
    const int tiles = (p.max_pages + kTile - 1) / kTile;
    return launch_behind(score_kernel<G>, dim3((unsigned)((tiles + p.tiles - 1) / p.tiles), (unsigned)p.B), dim3(kScoreWarps * 32), 0,
                         stream, p);
}

}  // namespace

SelectLayout select_layout(const pkv_problem& pr) {
    auto up = [](size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; };
    const size_t n = (size_t)pr.batch * pr.num_kv_heads, tiles = ((size_t)pr.max_pages_per_seq + kTile - 1) / kTile;
    SelectLayout l;
    l.scores = sizeof(pkv_ws_header);
    l.exact = l.scores + up(n * pr.max_pages_per_seq * sizeof(float));
    l.tops = l.exact + up(n * pr.max_pages_per_seq * sizeof(double));
    l.bytes = l.tops + up(n * tiles * sizeof(float));
    return l;
}

int launch_select_pages(const SelectParams& in, int num_sms, void* stream) {
    SelectParams p = in;
    // Tiles a CTA: one while that leaves the GPU idle, and more where the CTAs of one would come in waves, each of which begins with
    // three dependent round trips (32 rows of up to 2048 pages: 36 us with one, 28 with 8).
    const int64_t all = (int64_t)p.B * ((p.max_pages + kTile - 1) / kTile);
    p.tiles = (int)std::max<int64_t>(1, std::min<int64_t>(8, all / (3 * num_sms)));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int e = cudaSuccess;
    if (p.max_pages > p.select) {
        switch (p.Hq / p.Hkv) {
            case 1: e = launch_scores<1>(p, s); break;
            case 2: e = launch_scores<2>(p, s); break;
            case 4: e = launch_scores<4>(p, s); break;
            case 8: e = launch_scores<8>(p, s); break;
            case 16: e = launch_scores<16>(p, s); break;
            default: e = cudaErrorInvalidValue;
        }
    }
    if (e != cudaSuccess) return e;
    return launch_behind(select_kernel, dim3((unsigned)p.Hkv, (unsigned)p.B), dim3(kThreads), 0, s, p);
}

}  // namespace pkv
