// Packed prompts' K/V into pages and back (include/pkv.h, pkv_prompt_append, pkv_q4_prompt_append, pkv_q4_read), and the bounds of
// pages that they went to (pkv_page_bounds).
//
// Bound: HBM (a token and KV head: 512 bytes read and written; 512 and 144 with the 4-bit pages), and latency where it
// quantises: nothing is full there (ALU 56 %, issue 59 %, HBM 60 %), a warp has no load in flight while it quantises, and
// its longest stall is on its loads. Measured on a GB300, 8 KV heads: FP16 append of 17k tokens 25 us, 5.7 TB/s; 4-bit
// append of 50k tokens 65 us, 4.0 TB/s (0.60 of the copy bandwidth; 980 instructions for the K or V of a page and KV
// head); read-back 48 us, 5.4 TB/s; a few tokens 7.5 and 4.7 us. Warps are the unit of work: a token for the FP16
// pages, the K or V of a (page, KV head) for the 4-bit append, a (page, KV head) for the read-back. All warps of the
// grid share the items of all sequences evenly, whatever their lengths: each warp looks at 32 sequences at a time (a
// lane each), scans their item counts, and takes every W-th item of the running line (W = warps of the grid).
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "pkv_internal.h"
#include "pkv_launch.h"
#include "pkv_tcgen05.cuh"
#include "q4.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

// One sequence: its first packed row, its tokens, and the position in its row's pages that they begin at.
struct Seq {
    int32_t s, first, n, start;
};

__device__ __forceinline__ int first_page(const Seq& q) { return q.start / kPageSize; }
__device__ __forceinline__ int page_count(const Seq& q) {
    return q.n == 0 ? 0 : (q.start + q.n - 1) / kPageSize - q.start / kPageSize + 1;
}

// Calls item(sequence, index within the sequence) for every item of this warp; count(sequence) is how many it has.
// (An index fits 32 bits: the packed rows of 2^32 items would take more memory than there is.) Sequences whose bounds
// are not ordered inside [0, total_tokens], or that would outgrow their block table, have none.
template <typename Count, typename Item>
__device__ __forceinline__ void for_items(const PagesParams& p, Count count, Item item) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * kWarps;
    const int64_t self = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    int64_t next = self;  // this warp's next item, from the first of the 32 sequences
    for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
        Seq q{s0 + lane, 0, 0, 0};
        if (q.s < p.num_seqs) {
            q.first = p.cu_seqlens[q.s];
            const int last = p.cu_seqlens[q.s + 1];
            q.start = p.start ? p.start[q.s] : 0;
            const bool ok = q.first >= 0 && last >= q.first && last <= p.total_tokens && q.start >= 0 &&
                            (int64_t)q.start + (last - q.first) <= (int64_t)p.max_pages * kPageSize;
            if (ok)
                q.n = last - q.first;
            else if (self == 0)
                atomicOr(&p.hdr->status, PKV_STATUS_BAD_LEN);
        }
        const int64_t mine = count(q);
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += y;
        }
        const int64_t total = __shfl_sync(kAll, incl, 31);
        int64_t t = next;
        for (; t < total; t += warps) {
            const int src = __ffs(__ballot_sync(kAll, incl > t)) - 1;
            const Seq w{__shfl_sync(kAll, q.s, src), __shfl_sync(kAll, q.first, src), __shfl_sync(kAll, q.n, src),
                        __shfl_sync(kAll, q.start, src)};
            item(w, (uint32_t)(t - __shfl_sync(kAll, incl - mine, src)));
        }
        next = t - total;
    }
}

// Physical page of logical page lp of row s; -1 (and a status bit) where the entry is outside the pool.
__device__ __forceinline__ int64_t page_of(const PagesParams& p, int s, int lp) {
    const int32_t e = p.block_table[(int64_t)s * p.max_pages + lp];
    if (e >= 0 && e < p.num_pages) return e;
    if ((threadIdx.x & 31) == 0) atomicOr(&p.hdr->status, PKV_STATUS_BAD_PAGE);
    return -1;
}

// FP16 pages: a warp per token, 16 bytes a lane, the token's K and V in flight together.
__global__ void __launch_bounds__(kThreads) append_kernel(const PagesParams p) {
    const int lane = threadIdx.x & 31;
    const int per = p.Hkv * 16;  // 16-byte pieces of a token's K
    for_items(
        p, [](const Seq& q) { return (int64_t)q.n; },
        [&](const Seq& q, uint32_t i) {
            const int pos = q.start + (int)i;
            const int64_t page = page_of(p, q.s, pos / kPageSize);
            if (page < 0) return;
            const uint4* k = reinterpret_cast<const uint4*>(static_cast<const __half*>(p.k) + (int64_t)(q.first + i) * p.k_stride);
            const uint4* v = reinterpret_cast<const uint4*>(static_cast<const __half*>(p.v) + (int64_t)(q.first + i) * p.v_stride);
            const int64_t dst = (page * kPageSize + pos % kPageSize) * per;
            uint4* ko = static_cast<uint4*>(p.k_pool) + dst;
            uint4* vo = static_cast<uint4*>(p.v_pool) + dst;
            for (int c = lane; c < per; c += 128) {
                uint4 a[4], b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + 32 * j < per) {
                        a[j] = __ldcs(k + c + 32 * j);
                        b[j] = __ldcs(v + c + 32 * j);
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + 32 * j < per) {
                        ko[c + 32 * j] = a[j];
                        vo[c + 32 * j] = b[j];
                    }
            }
        });
}

// Bounds of pages: a warp per (page, 32 pieces of 16 bytes of a token's K), a lane per piece, all 16 tokens in flight. Bound:
// HBM (the pages' K is read once, 512 bytes a (page, KV head) written). Measured on a GB300: 33k tokens of 8 KV heads 11.8 us (5.8
// TB/s), the pages of 48 single tokens 4.4 us. (The table's entries read 32 items ahead: 0.5 us slower.)
__global__ void __launch_bounds__(kThreads) bounds_kernel(const PagesParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int per = p.Hkv * 16, parts = (per + 31) / 32;
    for_items(
        p, [&](const Seq& q) { return (int64_t)page_count(q) * parts; },
        [&](const Seq& q, uint32_t i) {
            const int lp = first_page(q) + (int)(i / (uint32_t)parts), c = (int)(i % (uint32_t)parts) * 32 + lane;
            const int64_t page = page_of(p, q.s, lp);
            if (page < 0 || c >= per) return;
            const int n = min(kPageSize, q.start + q.n - lp * kPageSize);
            const uint4* k = static_cast<const uint4*>(p.k_pool) + page * kPageSize * per + c;
            uint4 x[kPageSize];
#pragma unroll
            for (int t = 0; t < kPageSize; ++t) x[t] = __ldcs(k + min(t, n - 1) * per);
            __half2 lo[4], hi[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) lo[j] = hi[j] = reinterpret_cast<const __half2*>(&x[0])[j];
#pragma unroll
            for (int t = 1; t < kPageSize; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __half2 y = reinterpret_cast<const __half2*>(&x[t])[j];
                    lo[j] = __hmin2_nan(lo[j], y);
                    hi[j] = __hmax2_nan(hi[j], y);
                }
            // [page][head][least, greatest][16 pieces]
            uint4* out = static_cast<uint4*>(p.pool) + (page * p.Hkv + c / 16) * 32 + c % 16;
            out[0] = *reinterpret_cast<const uint4*>(lo);
            out[16] = *reinterpret_cast<const uint4*>(hi);
        });
}

// ---- quantising a whole (page, KV head) ----------------------------------------------------------------------------
// Lane l holds dims 8 c .. 8 c + 7 (c = l % 16) of tokens 2 i + l / 16, i < 8: coalesced rows. A group is 8 lanes.

// (min, -max) of 8 values; a NaN stays one.
__device__ __forceinline__ __half2 extremes8(const uint4& x) {
    const __half2 neg = __float2half2_rn(-1.f);
    const __half2* h = reinterpret_cast<const __half2*>(&x);
    __half2 lo = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
    __half2 hi = __hmul2(__hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3])), neg);
    return __hmin2_nan(__lows2half2(lo, hi), __highs2half2(lo, hi));
}

// One step of the reduction of N tokens' extremes over the lanes that differ in bit N / 2: each half of the lanes keeps
// half of the tokens.
template <int N>
__device__ __forceinline__ void reduce_half(__half2 (&m)[8], bool upper) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        const __half2 keep = upper ? m[N / 2 + j] : m[j], give = upper ? m[j] : m[N / 2 + j];
        m[j] = __hmin2_nan(keep, __shfl_xor_sync(kAll, give, N / 2));
    }
}

// The codes of 8 values by the definition's division, one byte each. Out of line: rare, and long.
__device__ __noinline__ uint2 codes8_exact(uint4 x, float scale, float offset) {
    const __half* h = reinterpret_cast<const __half*>(&x);
    uint32_t y[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i >> 2] |= q4_code(__half2float(h[i]), scale, offset) << (8 * (i & 3));
    return make_uint2(y[0], y[1]);
}

// What the lanes need of a group: its parameters, the reciprocal of the scale, and the constant that the quotient is
// added to; exact: the definition's division decides every code.
struct __align__(16) Group {
    __half2 par;
    float inv, add;
    uint32_t exact;
};

__device__ __forceinline__ Group group_of(__half2 extremes) {  // (min, -max)
    const float mn = __low2float(extremes), mx = -__high2float(extremes);
    Group g;
    const bool finite = isfinite(mn) && isfinite(mx);
    g.par = q4_params(mn, mx, finite);
    const float scale = __low2float(g.par);
    const bool some = scale > 0.f;  // neither equal values (codes 0) nor a group that stands for NaN
    g.inv = some ? __frcp_rn(scale) : 0.f;
    const float off = some ? mn * g.inv : 0.f;
    g.add = 192.5f + 0x1p-15f - off;
    g.exact = some ? fabsf(off) > 60.f || scale < 6.2e-5f : !finite;  // (codes 0 for a group that stands for NaN)
    return g;
}

// The codes of 8 values, one byte each: two words. x / scale - offset / scale + 192.5 + 2^-15, one fused operation for
// two values, lies in [128, 256), where an fp32 has 16 fraction bits: byte 2 holds the code (192 is 0 modulo 16, and
// 0.5 makes the truncation a rounding), and the low 16 bits are the quotient's distance above the last tie, plus 2.
// The reciprocal, the constant and the sum are off by less than 2 of those units together (|offset / scale| <= 60), so
// where the distance is below 4 the true quotient could round the other way (doubt): the definition's division decides.
__device__ __forceinline__ uint2 codes8(const uint4& x, const Group& g, bool& doubt) {
    const __half2* h = reinterpret_cast<const __half2*>(&x);
    const uint64_t inv2 = pack_f32x2(g.inv, g.inv), add2 = pack_f32x2(g.add, g.add);
    uint32_t k[8], least = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        float a, b;
        unpack_f32x2(fma_f32x2(pack_f32x2(f.x, f.y), inv2, add2), a, b);
        k[2 * i] = __float_as_uint(a);
        k[2 * i + 1] = __float_as_uint(b);
        least = __vminu2(least, __byte_perm(k[2 * i], k[2 * i + 1], 0x5410));
    }
    doubt = g.exact || (least & 0xffffu) < 4u || least < 0x40000u;
    uint2 y;
    y.x = __byte_perm(__byte_perm(k[0], k[1], 0x0062), __byte_perm(k[2], k[3], 0x0062), 0x5410) & 0x0f0f0f0fu;
    y.y = __byte_perm(__byte_perm(k[4], k[5], 0x0062), __byte_perm(k[6], k[7], 0x0062), 0x5410) & 0x0f0f0f0fu;
    return y;
}

// Staging of one warp: the 16 rows of K (or V) as the lanes will take them, the half block being made, and the
// groups.
struct Quant {
    uint4 rows[8][32];
    uint8_t half[kQ4Half];
    Group groups[32];
};

// The staged rows of K or V into their half block. Rolled over the tokens: unrolled, the code of one page is 24 KB, and
// a call of a few pages spends most of its time on fetching instructions.
template <bool kV>
__device__ __forceinline__ void quantise_page(Quant& w, int lane) {
    const int c = lane & 15, odd = lane >> 4, c7 = c & 7, hi = c >> 3;
    // The extremes of the 8 tokens, reduced over the group's 8 lanes so that lane c7 ends with token i = c7; it works out
    // that token's parameters and the reciprocal of its scale for all of them.
    __half2 m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = extremes8(w.rows[i][lane]);
    reduce_half<8>(m, c7 & 4);
    reduce_half<4>(m, c7 & 2);
    reduce_half<2>(m, c7 & 1);
    {
        const Group g = group_of(m[0]);
        const int at = 2 * (2 * c7 + odd) + hi;
        reinterpret_cast<__half2*>(w.half + kQ4Codes)[at] = g.par;
        w.groups[at] = g;
    }
    __syncwarp();
    // Group 1's codes go into the high 4 bits of group 0's bytes. The lane of group 0 keeps dims 8 c7 .. + 3, that of group
    // 1 dims + 4 .. + 7: four bytes each, e = 4 hi + byte.
    auto put = [&](int i, uint2 code) {
        const uint32_t got = __shfl_xor_sync(kAll, hi ? code.x : code.y, 8);
        const uint32_t own = hi ? got | code.y << 4 : code.x | got << 4;
        uint32_t word;
        int at;
        if (!kV) {
            // word (r, t, ks): bytes dim 2t of lane c7 even, of c7 odd, dim 2t + 1 of even, of odd
            const uint32_t far = __shfl_xor_sync(kAll, c7 & 1 ? own : own >> 16, 1);
            word = c7 & 1 ? __byte_perm(far, own, 0x7160) : __byte_perm(own, far, 0x5140);
            at = i * 128 + odd * 64 + (2 * hi + (c7 & 1)) * 16 + (c7 >> 1) * 4;
        } else {
            // word (i, e, ks): bytes token 2i of lane c7 even, of odd, token 2i + 1 of even, of odd. Four lanes with four
            // e each transpose their 4 x 4 bytes in two exchanges; lane (odd, c7 & 1) keeps e = 4 hi + 2 odd + (c7 & 1).
            const uint32_t far = __shfl_xor_sync(kAll, own, 1);
            const uint32_t two = c7 & 1 ? __byte_perm(far, own, 0x7351) : __byte_perm(own, far, 0x6240);
            const uint32_t other = __shfl_xor_sync(kAll, two, 16);
            word = odd ? __byte_perm(other, two, 0x7632) : __byte_perm(two, other, 0x5410);
            at = (i >> 2) * 512 + (4 * hi + 2 * odd + (c7 & 1)) * 64 + (i & 3) * 16 + (c7 >> 1) * 4;
        }
        *reinterpret_cast<uint32_t*>(w.half + at) = word;
    };
    uint32_t doubts = 0;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
        bool doubt;
        put(i, codes8(w.rows[i][lane], w.groups[2 * (2 * i + odd) + hi], doubt));
        doubts |= (doubt ? 1u : 0u) << i;
    }
    // tokens with a quotient in doubt again, after the others (a branch for each token would cost all of them)
    for (uint32_t left = __reduce_or_sync(kAll, doubts); left; left &= left - 1) {
        const int i = __ffs(left) - 1;
        const Group g = w.groups[2 * (2 * i + odd) + hi];
        bool doubt;
        uint2 code = codes8(w.rows[i][lane], g, doubt);
        if (doubt) code = codes8_exact(w.rows[i][lane], __low2float(g.par), __high2float(g.par));
        __syncwarp();
        put(i, code);
    }
}

// 16 bytes global -> shared, asynchronously; zeros where there is nothing to read.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(read ? 16 : 0) : "memory");
}

__global__ void __launch_bounds__(kThreads, 4) q4_append_kernel(const PagesParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31;
    Quant& w = reinterpret_cast<Quant*>(smem)[threadIdx.x >> 5];
    const uint8_t* blk = w.half;
    const int c = lane & 15, odd = lane >> 4;
    // an item is the K or the V of a (page, KV head): K, V, K, ...
    for_items(
        p, [&](const Seq& q) { return (int64_t)page_count(q) * p.Hkv * 2; },
        [&](const Seq& q, uint32_t it) {
            const uint32_t v = it & 1u, pg = (it >> 1) / (uint32_t)p.Hkv, h = (it >> 1) - pg * p.Hkv;
            const int lp = first_page(q) + (int)pg;
            const int64_t page = page_of(p, q.s, lp);
            if (page < 0) return;
            uint8_t* dst = static_cast<uint8_t*>(p.pool) + (page * p.Hkv + h) * kQ4Block + v * kQ4Half;
            const int64_t row = (int64_t)lp * kPageSize - q.start;  // of the page's slot 0, within the sequence
            const int lo = (int)max((int64_t)0, -row), hi = (int)min((int64_t)kPageSize, q.n - row);
            const __half* x = static_cast<const __half*>(v ? p.v : p.k) + h * kHeadDim + c * 8;
            const int64_t stride = v ? p.v_stride : p.k_stride;
            const bool whole = lo == 0 && hi == kPageSize;
            if (whole) {
                const __half* at = x + (q.first + row + odd) * stride;
#pragma unroll
                for (int i = 0; i < 8; ++i, at += 2 * stride) copy16(&w.rows[i][lane], at, true);
            } else {
                for (int i = 0; i < 8; ++i) {
                    const int r = 2 * i + odd;
                    const bool in = r >= lo && r < hi;
                    copy16(&w.rows[i][lane], x + (q.first + (in ? row + r : 0)) * stride, in);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (v == 0)
                quantise_page<false>(w, lane);
            else
                quantise_page<true>(w, lane);
            __syncwarp();
            if (whole) {
                for (int j = lane; j < kQ4Half / 16; j += 32)
                    reinterpret_cast<uint4*>(dst)[j] = reinterpret_cast<const uint4*>(blk)[j];
            } else {  // a page that the sequence fills in part: its tokens' bytes, the other slots keep theirs
                auto in = [&](int r) { return r >= lo && r < hi; };
                auto put = [&](int at, auto* type) {
                    using T = std::remove_pointer_t<decltype(type)>;
                    *reinterpret_cast<T*>(dst + at) = *reinterpret_cast<const T*>(blk + at);
                };
                if (lane < 16 && in(lane)) put(kQ4Codes + lane * 8, static_cast<uint2*>(nullptr));
                if (v == 0) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)  // 64 bytes of codes a token
                        if (in((lane + 32 * j) / 4)) put((lane + 32 * j) * 16, static_cast<uint4*>(nullptr));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {  // a word of codes is two bytes of each of two tokens
                        const int at = (lane + 32 * j) * 4, r = (at >> 9) * 8 + ((at >> 4) & 3) * 2;
                        if (in(r) && in(r + 1))
                            put(at, static_cast<uint32_t*>(nullptr));
                        else if (in(r) || in(r + 1))
                            put(at + (in(r) ? 0 : 2), static_cast<uint16_t*>(nullptr));
                    }
                }
            }
            __syncwarp();
        });
}

// ---- reading back ----------------------------------------------------------------------------------------------------
// Eight codes (as 4-bit values in the low bits of the two halves of four words) times scale plus offset, one rounding.
__device__ __forceinline__ uint4 dequantise8(const uint32_t (&pairs)[4], __half2 par) {
    const __half2 sc = __low2half2(par), off = __high2half2(par), bias = __float2half2_rn(-1024.f);
    uint4 y;
    uint32_t* o = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = pairs[i] | 0x64006400u;  // 1024 + code
        const __half2 v = __hfma2(__hadd2(*reinterpret_cast<const __half2*>(&u), bias), sc, off);
        o[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return y;
}

__global__ void __launch_bounds__(kThreads) q4_read_kernel(const PagesParams p) {
    __shared__ __align__(16) uint8_t s_blk[kWarps][kQ4Block];
    const int lane = threadIdx.x & 31;
    uint8_t* blk = s_blk[threadIdx.x >> 5];
    // lane: dims 8 c .. 8 c + 7 (c = lane % 16) of tokens 2 i + lane / 16
    const int c = lane & 15, odd = lane >> 4, c7 = c & 7, hi = c >> 3, ks = c7 >> 1;
    for_items(
        p, [&](const Seq& q) { return (int64_t)page_count(q) * p.Hkv; },
        [&](const Seq& q, uint32_t it) {
            const uint32_t pg = it / (uint32_t)p.Hkv, h = it - pg * p.Hkv;
            const int lp = first_page(q) + (int)pg;
            const int64_t page = page_of(p, q.s, lp);
            if (page < 0) return;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.pool) + (page * p.Hkv + h) * kQ4Block);
            for (int j = lane; j < kQ4Block / 16; j += 32) reinterpret_cast<uint4*>(blk)[j] = __ldcs(src + j);
            __syncwarp();
            const int64_t row = (int64_t)lp * kPageSize - q.start;
            __half* k = static_cast<__half*>(p.k_pool) + (q.first + row) * p.k_stride + h * kHeadDim + c * 8;
            __half* v = static_cast<__half*>(p.v_pool) + (q.first + row) * p.v_stride + h * kHeadDim + c * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 2 * i + odd;
                if (row + r < 0 || row + r >= q.n) continue;
                uint32_t pairs[4];
                const int sh = 8 * (c7 & 1) + 4 * hi;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    pairs[t] = *reinterpret_cast<const uint32_t*>(blk + r * 64 + t * 16 + ks * 4) >> sh & 0x000f000fu;
                *reinterpret_cast<uint4*>(k + r * p.k_stride) =
                    dequantise8(pairs, reinterpret_cast<const __half2*>(blk + kQ4Codes)[2 * r + hi]);
                const uint8_t* vb = blk + kQ4Half + (i >> 2) * 512 + (i & 3) * 16 + ks * 4 + 2 * odd + (c7 & 1);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    pairs[t] = (vb[(2 * t) * 64] >> (4 * hi) & 15u) | (uint32_t)(vb[(2 * t + 1) * 64] >> (4 * hi) & 15u) << 16;
                *reinterpret_cast<uint4*>(v + r * p.v_stride) =
                    dequantise8(pairs, reinterpret_cast<const __half2*>(blk + kQ4Half + kQ4Codes)[2 * r + hi]);
            }
            __syncwarp();
        });
}

int grid_for(int num_sms, int64_t items) {
    return (int)std::max<int64_t>(1, std::min<int64_t>((items + kWarps - 1) / kWarps, 8 * (int64_t)num_sms));
}

// At most this many (page, KV head) items.
int64_t page_items(const PagesParams& p) { return ((int64_t)p.total_tokens / kPageSize + 2 * (int64_t)p.num_seqs) * p.Hkv; }

}  // namespace

int launch_prompt_append(const PagesParams& p, int num_sms, void* stream) {
    return launch_kernel(append_kernel, grid_for(num_sms, p.total_tokens), kThreads, 0, static_cast<cudaStream_t>(stream), p);
}

int launch_page_bounds(const PagesParams& p, int num_sms, void* stream) {
    // The number of new tokens is not known here, so more CTAs than are resident would start to find nothing; four an SM are. (33k
    // tokens: 14.8 us with two an SM, 11.8 with four, 12.1 with eight.) No row has more pages than its table.
    const int64_t items = std::min(page_items(p) / p.Hkv, (int64_t)p.num_seqs * p.max_pages) * ((p.Hkv + 1) / 2);
    return launch_behind(bounds_kernel, dim3(std::min(grid_for(num_sms, items), 4 * num_sms)), dim3(kThreads), 0,
                         static_cast<cudaStream_t>(stream), p);
}

int launch_q4_append(const PagesParams& p, int num_sms, void* stream) {
    static int configured_mask = 0;  // one bit per device ordinal (< 32)
    constexpr int smem = kWarps * (int)sizeof(Quant);
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 32 || !(__atomic_load_n(&configured_mask, __ATOMIC_ACQUIRE) & (1 << dev))) {
        const cudaError_t e = cudaFuncSetAttribute(q4_append_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 32) __atomic_fetch_or(&configured_mask, 1 << dev, __ATOMIC_ACQ_REL);
    }
    return launch_kernel(q4_append_kernel, grid_for(num_sms, 2 * page_items(p)), kThreads, smem, static_cast<cudaStream_t>(stream), p);
}

int launch_q4_read(const PagesParams& p, int num_sms, void* stream) {
    return launch_kernel(q4_read_kernel, grid_for(num_sms, page_items(p)), kThreads, 0, static_cast<cudaStream_t>(stream), p);
}

}  // namespace pkv
