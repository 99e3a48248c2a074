// The pages whose bounds promise a KV head's queries the greatest scores (include/pkv.h, pkv_select_pages).
//
// score(page) = max over the G query heads of sum_d max(q_d lo_d, q_d hi_d), lo and hi the least and greatest key of the page in
// dim d: no key of the page has a greater product with the query. With q- = min(q, 0), q+ = max(q, 0) the sum is q-.lo +
// q+.hi, one product over 256 dims, so a tile of 16 pages takes 16 mma.sync m16n8k16 (pages on the 16-row side, the heads on the
// 8-column side; tcgen05 needs 64 rows of either). The order of a contraction is free: a lane takes 16 bytes of a page's bounds
// at a time, which are its fragments of two steps, and holds the same dims of the queries.
//
// The row's last page is always selected (it holds the newest tokens), and the select - 1 greatest of the others; equal scores
// go to the lowest page. The definition is exact: products of fp16 values summed in 64 bits. The fp32 scores are off by at most
// delta = 2^-15 max_g |q_g|_1 max |bound|: 16 instructions add 16 products and the sum before, each of which may lose 2^-23 of the
// greatest magnitude (17 * 16 * 2^-23 = 2^-14.9 of the sum of magnitudes, half of which are zeros of q- or q+). With T the
// (select - 1)-th greatest fp32 score, pages above T + 2 delta are in and those below T - 2 delta out whatever their exact scores
// are; those between are scored again in 64 bits (one or two of 2048 with normal values) and ranked by those.
// Bounds or queries that are not finite make a score of +inf: such pages come first.
//
// Two kernels: scores, bound by HBM (512 bytes a (page, KV head)), a warp per KV head and 16 pages, so that the heads of a page
// are read together; and a CTA per (row, KV head) that selects, bound by latency (the threshold is found two bits at a time,
// 16 counts over the CTA). Measured: @@MEASURED@@
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
constexpr int kThreads = 256;             // of the selection
constexpr int kWarps = kThreads / 32;

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
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const int b = blockIdx.y, tile = blockIdx.x;
    bool bad;
    const int pages = row_pages(p, b, bad);
    if (tile * kTile >= pages || pages <= p.select || p.select == 1) return;  // nothing there, or nothing to be compared
    // the lane's two pages; -1: none (its bounds count as 0)
    int page[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int lp = tile * kTile + r + 8 * i;
        page[i] = lp < pages ? page_of(p, b, lp) : -1;
        if (lp < pages && page[i] < 0) atomicOr(&p.hdr->status, PKV_STATUS_BAD_PAGE);
    }
    for (int h = warp; h < p.Hkv; h += kScoreWarps) {
        uint4 x[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.bounds) +
                                                             ((int64_t)max(page[i], 0) * p.Hkv + h) * kBoundBytes) + t;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = page[i] >= 0 ? __ldcs(at + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
        }
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
                if (tile * kTile + r + 8 * i < pages) p.scores[pair * p.max_pages + tile * kTile + r + 8 * i] = score[i];
        if (lane == 0) p.tops[pair * ((p.max_pages + kTile - 1) / kTile) + tile] = mag;
    }
}

// ---- selection -----------------------------------------------------------------------------------------------------
// Keys in the order of the scores.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float from_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// The exact score of a page, by a warp: lane l sums dims 4 l .. 4 l + 3.
__device__ __forceinline__ double exact_score(const SelectParams& p, int b, int h, int lp) {
    const int lane = threadIdx.x & 31, G = p.Hq / p.Hkv, page = page_of(p, b, lp);
    uint2 lo = make_uint2(0u, 0u), hi = lo;
    if (page >= 0) {
        const uint2* at = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.bounds) + ((int64_t)page * p.Hkv + h) * kBoundBytes);
        lo = at[lane];
        hi = at[32 + lane];
    }
    double best = 0.;
    for (int g = 0; g < G; ++g) {
        const uint2 q = reinterpret_cast<const uint2*>(static_cast<const __half*>(p.q) + ((int64_t)b * p.Hq + h * G + g) * kHeadDim)[lane];
        double s = 0.;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            auto at = [&](const uint2& u) { return __half2float(__ushort_as_half((unsigned short)((i < 2 ? u.x : u.y) >> (16 * (i & 1))))); };
            const float y = at(q);
            s += (double)fmaxf(y * at(lo), y * at(hi));  // a product of two fp16 values is exact in fp32
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        if (g == 0 || s > best) best = s;
    }
    return best;
}

// Sums of N numbers over the CTA, in every thread. `turn` alternates: a slot of s_sum is written again two sums later.
template <int N>
__device__ __forceinline__ void block_sums(int (&x)[N], int (*s_sum)[kWarps][3], int turn) {
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __reduce_add_sync(kAll, x[i]);
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) s_sum[turn][warp][i] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x[i] += s_sum[turn][w][i];
    }
}

// The greatest key that at least `want` keys reach, two bits at a time; count(x, c): c[i] = this thread's keys of at least
// x[i]. Uses s_sum[0] last.
template <typename Key, typename Count>
__device__ __forceinline__ Key border_of(int want, Count count, int (*s_sum)[kWarps][3]) {
    Key border = 0;
    int turn = 1;
    for (int shift = 8 * (int)sizeof(Key) - 2; shift >= 0; shift -= 2, turn ^= 1) {
        const Key x[3] = {border | (Key)1 << shift, border | (Key)2 << shift, border | (Key)3 << shift};
        int c[3] = {0, 0, 0};
        count(x, c);
        block_sums(c, s_sum, turn);
        border |= (Key)(c[2] >= want ? 3 : c[1] >= want ? 2 : c[0] >= want ? 1 : 0) << shift;
    }
    return border;
}

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
    constexpr int kHeld = 16;   // keys that a thread holds; of rows of more pages the others are read each time
    constexpr int kList = 256;  // pages next to the border that are ranked in shared memory
    const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t pair = (int64_t)b * p.Hkv + h;
    __shared__ int s_sum[2][kWarps][3];
    __shared__ float s_float[2][kWarps];
    __shared__ int s_near, s_list[kList];
    __shared__ double s_exact[kList];
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
        s_near = 0;
        out[want] = n;  // the last page
    }
    float l1 = 0.f;  // of the query heads of this thread's warp: the greatest sum of magnitudes
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
    const float* scores = p.scores + pair * p.max_pages;
    double* exact = p.exact + pair * p.max_pages;
    // A thread's candidates are a run of pages, in order.
    const int run = (n + kThreads - 1) / kThreads, p0 = min(n, (int)threadIdx.x * run), p1 = min(n, p0 + run);
    uint32_t held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = p0 + i < p1 ? key_of(__ldcg(scores + p0 + i)) : 0u;
    float mag = 0.f;
    const int tiles = (p.max_pages + kTile - 1) / kTile;
    for (int i = threadIdx.x; i * kTile < pages; i += kThreads) mag = fmaxf(mag, __ldcg(p.tops + pair * tiles + i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mag = fmaxf(mag, __shfl_xor_sync(kAll, mag, o));
    if (lane == 0) {
        s_float[0][warp] = l1;
        s_float[1][warp] = mag;
    }
    auto for_keys = [&](auto f) {  // f(page, key) for this thread's candidates
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (p0 + i < p1) f(p0 + i, held[i]);
        for (int j = p0 + kHeld; j < p1; ++j) f(j, key_of(__ldcg(scores + j)));
    };
    const uint32_t border = border_of<uint32_t>(
        want,
        [&](const uint32_t (&x)[3], int (&c)[3]) {
            for_keys([&](int, uint32_t k) {
#pragma unroll
                for (int i = 0; i < 3; ++i) c[i] += k >= x[i];
            });
        },
        s_sum);
    float q1 = 0.f, top = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        q1 = fmaxf(q1, s_float[0][w]);
        top = fmaxf(top, s_float[1][w]);
    }
    // Next to the border: scores within twice their error of it. (Queries that are not finite give scores of +inf alone.)
    const float edge = from_key(border), delta = isfinite(q1) ? 0x1p-14f * q1 * top : 0.f;
    const uint32_t above = key_of(edge == INFINITY ? edge : __fadd_ru(edge, delta));
    const uint32_t below = key_of(edge == INFINITY ? edge : __fadd_rd(edge, -delta));
    int c2[2] = {0, 0};
    for_keys([&](int, uint32_t k) {
        c2[0] += k > above;
        c2[1] += k >= below && k <= above;
    });
    block_sums(c2, s_sum, 1);
    const int room = want - c2[0], near = c2[1];  // pages next to the border that are selected; all of them
    int ties = 0;       // of those whose exact score is the last one's: how many, the lowest pages, are selected
    uint64_t last = 0;  // the key of that score
    const bool listed = near <= kList;
    if (near > room) {
        auto score = [&](int j, uint32_t k) { return k == key_of(INFINITY) ? (double)INFINITY : exact_score(p, b, h, j); };
        if (listed) {
            for_keys([&](int j, uint32_t k) {
                if (k >= below && k <= above) s_list[atomicAdd(&s_near, 1)] = j;
            });
            __syncthreads();
            for (int i = warp; i < near; i += kWarps) {
                const double e = score(s_list[i], key_of(__ldcg(scores + s_list[i])));
                if (lane == 0) s_exact[i] = e;
            }
            __syncthreads();
        } else {
            for (int j = warp; j < n; j += kWarps) {
                const uint32_t k = key_of(__ldcg(scores + j));
                if (k < below || k > above) continue;
                const double e = score(j, k);
                if (lane == 0) exact[j] = e;
            }
            __syncthreads();
            auto key64 = [&](int j) {
                const uint64_t u = (uint64_t)__double_as_longlong(exact[j]);
                return u >> 63 ? ~u : u | 1ull << 63;
            };
            last = border_of<uint64_t>(
                room,
                [&](const uint64_t (&x)[3], int (&c)[3]) {
                    for_keys([&](int j, uint32_t k) {
                        if (k >= below && k <= above) {
                            const uint64_t y = key64(j);
#pragma unroll
                            for (int i = 0; i < 3; ++i) c[i] += y >= x[i];
                        }
                    });
                },
                s_sum);
            int c[2] = {0, 0};  // greater scores; equal ones
            for_keys([&](int j, uint32_t k) {
                if (k >= below && k <= above) {
                    const uint64_t y = key64(j);
                    c[0] += y > last;
                    c[1] += y == last;
                }
            });
            // the equal ones of the threads before this one
            int incl = c[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += y;
            }
            int ahead = incl - c[1], greater[1] = {c[0]};
            __syncthreads();
            if (lane == 31) s_sum[1][warp][1] = incl;
            block_sums(greater, s_sum, 1);
            for (int w = 0; w < warp; ++w) ahead += s_sum[1][w][1];
            ties = room - greater[0] - ahead;
        }
    }
    int seen = 0;  // equal ones of this thread's run
    auto selected = [&](int j, uint32_t k) {
        if (k > above) return true;
        if (k < below) return false;
        if (near <= room) return true;
        if (listed) {
            double e = 0.;
            for (int i = 0; i < near; ++i)
                if (s_list[i] == j) e = s_exact[i];
            int rank = 0;
            for (int i = 0; i < near; ++i) rank += s_exact[i] > e || (s_exact[i] == e && s_list[i] < j);
            return rank < room;
        }
        const uint64_t u = (uint64_t)__double_as_longlong(exact[j]), y = u >> 63 ? ~u : u | 1ull << 63;
        return y > last || (y == last && seen++ < ties);
    };
    // Which of the run's first 64 pages, and how many; then the places, in the order of the pages.
    uint64_t mask = 0;
    int mine = 0;
    for_keys([&](int j, uint32_t k) {
        const bool yes = selected(j, k);
        mine += yes;
        if (yes && j - p0 < 64) mask |= 1ull << (j - p0);
    });
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[0][warp][0] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int w = 0; w < warp; ++w) at += s_sum[0][w][0];
    for (; mask; mask &= mask - 1) out[at++] = p0 + __ffsll((long long)mask) - 1;
    if (run > 64) {
        seen = 0;
        for (int j = p0; j < p1; ++j) {
            const bool yes = selected(j, key_of(__ldcg(scores + j)));
            if (yes && j - p0 >= 64) out[at++] = j;
        }
    }
}

template <int G>
int launch_scores(const SelectParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.max_pages + kTile - 1) / kTile), (unsigned)p.B);
    cfg.blockDim = dim3(kScoreWarps * 32);
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, score_kernel<G>, p);
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

int launch_select_pages(const SelectParams& p, int num_sms, void* stream) {
    (void)num_sms;
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.Hkv, (unsigned)p.B);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.max_pages > p.select ? 1 : 0;  // it may overlap the scores alone
    return cudaLaunchKernelEx(&cfg, select_kernel, p);
}

}  // namespace pkv
