// One decode step over the 4-bit pages (include/pkv.h, pkv_q4_decode_step).
//
// Per row b, KV head h and query head: x_j = scale * log2(e) * q.k_j, out = sum 2^(x_j - m) v_j / sum 2^(x_j - m), with
// k_j = sum over the two groups of (scale_j code_j + offset_j). Everything that is one number per (token, group) stays
// out of the matrix products and in fp32:
//   q.k_j   = sum_g scale_jg (q.code_jg) + offset_jg (sum of q over the group)
//   out     = sum_g sum_j (w_j scale_jg) code_jg + sum_j w_j offset_jg
// so the products (mma.sync m16n8k16, tokens or dims on the 16-row side, the G <= 16 query heads on the 8-column side)
// take the codes as they lie in memory: one mask makes two codes into two fp16 subnormals (q4.cuh), no conversion.
// tcgen05 needs 64 or 128 rows of query heads, of which a KV head has G. The weights w_j scale_jg enter as two fp16 parts;
// the exponent that w_j is taken relative to includes V's scale (ref, below), so that V of any magnitude keeps its
// precision.
//
// Bound: HBM; a (token, KV head) is 144 bytes against 512 in fp16. A unit is 4 pages (64 tokens) of one (row, KV head),
// four bulk copies of 2304 bytes into one ring stage, and goes to one consumer warp. Measured on a GB300 (G = 4): 48 rows
// of 900-32768 tokens, 765 MB, 143 us: 5.4 TB/s, 0.80 of the copy bandwidth; copies alone 125 us, arithmetic alone
// 120 us; eight rows, 154 MB, 37 us; one row of 512 tokens 8.8 us (from L2 7.9).
// Division: the units of all (row, KV head) pairs form one line, and each CTA takes an equal piece of it, whatever the
// rows' lengths; every CTA finds its piece itself from a scan of seq_lens, so there is no plan. A pair that lies in one
// piece is written out at once. The others leave a state (m, l, accumulator) per piece, and the last of a pair's
// pieces to arrive at its counter merges them in the order of the pieces (so results do not depend on the arrival
// order); nobody waits for another CTA.
//
// Warp roles: consumers (NC), loader (walks the piece, issues the copies, publishes segments = a piece's part of one
// pair), epilogue (combines the consumers' partial results of a segment and writes it).
// Every wait is bounded (pkv_wait.cuh).
#include <cuda_fp16.h>

#include <algorithm>

#include "pkv_internal.h"
#include "pkv_launch.h"
#include "pkv_ptx.cuh"
#include "pkv_wait.cuh"
#include "q4.cuh"

namespace pkv {
namespace {

constexpr int kUnitPages = 4;
constexpr int kUnitTokens = kUnitPages * kPageSize;
constexpr int kStageBytes = kUnitPages * kQ4Block;
constexpr int kChunk = 32 / kUnitPages;  // units whose block-table entries one warp-wide read brings
constexpr int kCombRow = kHeadDim + 4;  // floats per partial output row: rows land 4 banks apart
constexpr uint32_t kAllPages = (1u << kUnitPages) - 1u;
// Arrival counters behind the workspace's header, one a piece. They are zero between steps, so they lie where no step of
// other heads or of a grid of another size puts its states: their place and number depend on nothing.
constexpr int kMaxPieces = 2 * 4 * kCombRow;
// Units per CTA below which fewer CTAs take part: with fewer, short rows are spread wider and more states are merged. Batches
// of one to eight rows of 40 to 32768 tokens, geometric mean of 24 at (query heads, KV heads) of (8, 8), (32, 8), (32, 4),
// (16, 1), pages in L2, in us: 4 units 10.1, 10.8, 12.6, 13.4; 8 units 11.3, 11.9, 12.6, 14.6; but one row of 32768 takes
// 16.2, 17.4, 22, 29 with 4 and 16.2, 17.2, 19, 23 with 8. (Pieces that are whole pairs need no merge: 512 tokens of 8 KV
// heads 7.9 with 8, 8.8 with 4; 300 tokens 12.1 and 11.7.)
constexpr int kMinUnits = 8;

// A piece's part of one (row, KV head) pair.
struct Segment {
    int32_t b, h, units;  // units < 0: no more segments
    int32_t out;          // -1: the whole pair, written to out; else the state that it leaves
    int32_t first_cta, ctas;  // the pair's pieces
    int32_t len;              // tokens of the row
    int32_t append;           // 1: the new token is in this piece
};

// Consumers, stages, partial-result buffers, resident CTAs. Two CTAs an SM share its registers (four consumers of up to 168)
// and its shared memory (8 units of 9 KB in flight each); at G = 16 the query fragments and accumulators of one CTA's
// consumers take more than half. With 6 consumers of 128 registers and units of 3 pages a CTA the 48-row step took 148 us
// when this shape took 141.
template <int G>
struct Shape {
    static constexpr int NC = G >= 16 ? 6 : 4;
    static constexpr int NS = 2 * NC;
    static constexpr int NB = G >= 8 ? 1 : 2;
    static constexpr int kSlots = G >= 8 ? 2 : 4;  // segments published ahead
    static constexpr int per_sm = G >= 16 ? 1 : 2;
    static constexpr int threads = (NC + 2) * 32;
    static constexpr int off_q = NS * kStageBytes;
    static constexpr int off_comb = off_q + kSlots * G * kRowBytes;
    static constexpr int off_comb_ml = off_comb + NB * NC * G * kCombRow * 4;
    static constexpr int off_seg = off_comb_ml + NB * NC * G * 8;
    static constexpr int off_meta = off_seg + (kSlots + 2) * (int)sizeof(Segment);  // and two pairs to merge
    static constexpr int off_bars = off_meta + NS * 4;
    static constexpr int nbars = 2 * NS + 3 * kSlots + 2 * NB + 2;
    static constexpr int off_misc = off_bars + nbars * 8;
    static constexpr int off_new = (off_misc + 64 + 15) / 16 * 16;  // a block with the new token in its slot
    static constexpr int smem = off_new + kQ4Block;
    static_assert(off_bars % 8 == 0 && off_comb % 16 == 0 && smem <= 227 * 1024, "layout");
    static constexpr int kFactors = NB * NC * kCombRow;  // pieces of a pair whose factors fit (the grid is smaller)
    static_assert(kFactors <= kMaxPieces, "an arrival counter for every piece");
};

__device__ __forceinline__ int row_length(const Q4Params& p, int b) {
    const int len = p.seq_lens[b];
    return len < 0 || len > p.max_pages * kPageSize ? 0 : len;
}

__device__ __forceinline__ int row_units(int len) { return (len + kUnitTokens - 1) / kUnitTokens; }

// Piece of the line of `total` units that unit u lies in; piece i begins at i * total / ctas.
__device__ __forceinline__ int cta_of(int64_t u, int64_t total, int ctas) {
    return (int)(((u + 1) * ctas + total - 1) / total) - 1;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

// The bytes of one token of a block, K and V: 64 code bytes and 8 of parameters each.
__device__ __forceinline__ void copy_token(uint8_t* dst, const uint8_t* src, int r, int lane) {
#pragma unroll
    for (int d = lane; d < 64; d += 32) {
        const int kb = q4_k_byte(r, d), vb = kQ4Half + q4_v_byte(r, d);
        dst[kb] = src[kb];
        dst[vb] = src[vb];
    }
    if (lane < 4) {
        const int at = (lane >> 1) * kQ4Half + kQ4Codes + r * 8 + (lane & 1) * 4;
        *reinterpret_cast<uint32_t*>(dst + at) = *reinterpret_cast<const uint32_t*>(src + at);
    }
}

__device__ __forceinline__ float2 half2_of(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }

template <int G>
__global__ void __launch_bounds__(Shape<G>::threads, Shape<G>::per_sm) q4_decode_kernel(const Q4Params p) {
    using L = Shape<G>;
    constexpr int NC = L::NC, NS = L::NS, NB = L::NB, kSlots = L::kSlots, kNT = (G + 7) / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_scan[L::threads / 32];
    __shared__ int32_t s_row, s_len;  // where the piece begins: row, its length,
    __shared__ int64_t s_unit;  // unit of the row's Hkv * units
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::off_bars);
    uint64_t* empty = full + NS;
    uint64_t* seg_full = empty + NS;
    uint64_t* seg_q = seg_full + kSlots;
    uint64_t* seg_empty = seg_q + kSlots;
    uint64_t* part_full = seg_empty + kSlots;
    uint64_t* part_empty = part_full + NB;
    uint64_t* merged = part_empty + NB;
    uint64_t* new_full = merged + 1;
    uint8_t* new_blk = smem + L::off_new;
    Segment* segs = reinterpret_cast<Segment*>(smem + L::off_seg);
    Segment* merges = segs + kSlots;
    uint32_t* meta = reinterpret_cast<uint32_t*>(smem + L::off_meta);
    float* comb = reinterpret_cast<float*>(smem + L::off_comb);
    float2* comb_ml = reinterpret_cast<float2*>(smem + L::off_comb_ml);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::off_misc);
    volatile int* n_merges = abort_flag + 1;
    const WaitCtx ctx{abort_flag, &p.hdr->status};

    // The line of units: every thread sums a run of rows (the first row's length is on its way while the barriers are set
    // up), the CTA scans the sums, and the thread whose run holds the piece's first unit finds its row.
    const int per = (p.B + L::threads - 1) / L::threads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    const int len0 = b0 < b1 ? row_length(p, b0) : 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_q[i], 1);
            mbar_init(&seg_empty[i], NC + 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&part_full[i], NC);
            mbar_init(&part_empty[i], 1);
        }
        mbar_init(merged, 1);
        mbar_init(new_full, 1);
        *abort_flag = 0;
        *n_merges = 0;
        mbar_fence_init();
    }
    int64_t mine = row_units(len0);
    for (int b = b0 + 1; b < b1; ++b) mine += row_units(row_length(p, b));
    mine *= p.Hkv;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    for (int i = 0; i < L::threads / 32; ++i) {
        if (i < warp) before += s_scan[i];
        total += s_scan[i];
    }
    const int ctas = (int)min((int64_t)gridDim.x, max((int64_t)1, (total + kMinUnits - 1) / kMinUnits));
    const int cta = blockIdx.x;
    const int64_t lo = cta < ctas ? cta * total / ctas : 0, hi = cta < ctas ? (cta + 1) * total / ctas : 0;
    if (lo < hi && before <= lo && lo < before + mine) {
        int64_t at = before;
        for (int b = b0; b < b1; ++b) {
            const int len = b == b0 ? len0 : row_length(p, b);
            const int64_t n = (int64_t)row_units(len) * p.Hkv;
            if (lo < at + n) {
                s_row = b;
                s_len = len;
                s_unit = lo - at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();

    if (warp == NC) {
        // ------------------------------------------------------------------------------------------ loader
        const __half* q = static_cast<const __half*>(p.q);
        const uint8_t* pool = static_cast<const uint8_t*>(p.pool);
        const uint64_t pol = policy_evict_first();
        int seq = 0, k = 0;
        uint32_t issued = 0;  // after a time-out: units behind seq whose copies were issued
        bool ok = true;
        int b = 0, h = 0, u = 0, len = 0, units = 0;
        if (lo < hi) {
            b = s_row;
            len = s_len;
            units = row_units(len);
            h = (int)(s_unit / units);
            u = (int)(s_unit - (int64_t)h * units);
        }
        for (int64_t pos = lo; ok; ++k) {
            const int slot = k % kSlots;
            if (!warp_wait(&seg_empty[slot], ((k / kSlots) & 1) ^ 1, ctx)) break;
            if (pos >= hi || b == p.B || u >= units) {  // the last two: seq_lens changed under the kernel
                if (lane == 0) {
                    segs[slot].units = -1;
                    mbar_arrive(&seg_full[slot]);
                }
                break;
            }
            const int n = (int)min((int64_t)(units - u), hi - pos);
            const int32_t* bt = p.block_table + (int64_t)b * p.max_pages;
            const int pages = (len + kPageSize - 1) / kPageSize;
            const int p0 = u * kUnitPages;  // the segment's first page; lanes hold 32 entries (kChunk units) at a time
            int ent = p0 + lane < pages ? bt[p0 + lane] : -1;  // on its way while the segment is published
            if (lane == 0) {
                Segment s;
                s.b = b;
                s.h = h;
                s.units = n;
                s.out = n == units ? -1 : 2 * cta + (u == 0 ? 1 : 0);
                s.first_cta = cta_of(pos - u, total, ctas);
                s.ctas = cta_of(pos - u + units - 1, total, ctas) - s.first_cta + 1;
                s.len = len;
                s.append = p.k_new && u + n == units ? 1 : 0;
                segs[slot] = s;
                mbar_arrive(&seg_full[slot]);
                mbar_arrive_expect_tx(&seg_q[slot], G * kRowBytes);
                bulk_g2s(smem + L::off_q + slot * G * kRowBytes, q + ((int64_t)b * p.Hq + (int64_t)h * G) * kHeadDim,
                         G * kRowBytes, &seg_q[slot]);
            }
            __syncwarp();
            // Eight units (kChunk) at a time, a lane each: the warp sleeps on the first stage that is still in use, then every
            // lane whose stage is free announces its unit and issues its copies (one unit after the other, a loader
            // needs 600 cycles a unit, which halves the bandwidth).
            for (int c0 = 0; c0 < n && ok; c0 += kChunk) {
                const int cnt = min(kChunk, n - c0);
                int page[kUnitPages];
#pragma unroll
                for (int i = 0; i < kUnitPages; ++i)
                    page[i] = __shfl_sync(0xffffffffu, ent, (lane * kUnitPages + i) & 31);
                const int at = p0 + (c0 + kChunk) * kUnitPages + lane;
                ent = c0 + kChunk < n && at < pages ? bt[at] : -1;
                const int unit = u + c0 + lane;  // of the pair
                const int np = min(kUnitPages, pages - unit * kUnitPages);
                uint32_t okmask = 0;
#pragma unroll
                for (int i = 0; i < kUnitPages; ++i)
                    if (i < np && page[i] >= 0 && page[i] < p.num_pages) okmask |= 1u << i;
                const int st = (seq + lane) % NS;
                const uint32_t parity = (((seq + lane) / NS) & 1) ^ 1;
                bool pending = lane < cnt;
                if (pending && okmask != (1u << np) - 1u) raise_status(ctx.status, PKV_STATUS_BAD_PAGE);
                for (unsigned left; (left = __ballot_sync(0xffffffffu, pending)) != 0;) {
                    const int first = __ffs(left) - 1;
                    if (!warp_wait(&empty[(seq + first) % NS], (((seq + first) / NS) & 1) ^ 1, ctx)) {
                        ok = false;
                        break;
                    }
                    if (pending && mbar_test_wait(&empty[st], parity)) {
                        pending = false;
                        const int nv = min(kUnitTokens, len - unit * kUnitTokens);
                        const bool append = p.k_new && unit == units - 1;
                        meta[st] = (uint32_t)nv | okmask << 8 | (append ? 1u << 12 : 0u);
                        if (okmask)
                            mbar_arrive_expect_tx(&full[st], __popc(okmask) * kQ4Block);
                        else
                            mbar_arrive(&full[st]);
#pragma unroll
                        for (int i = 0; i < kUnitPages; ++i)
                            if ((okmask >> i) & 1)
                                bulk_g2s_hint(smem + st * kStageBytes + i * kQ4Block,
                                              pool + ((int64_t)page[i] * p.Hkv + h) * kQ4Block, kQ4Block, &full[st], pol);
                    }
                    __syncwarp();
                }
                if (ok) {
                    seq += cnt;
                } else {  // gave up: these units' copies in flight are waited for, too
                    issued = __ballot_sync(0xffffffffu, lane < cnt && !pending);
                }
            }
            pos += n;
            u = 0;
            if (++h == p.Hkv && pos < hi) {
                h = 0;
                do {
                    if (++b == p.B) break;
                    len = row_length(p, b);
                } while (len == 0);
                units = row_units(len);
            }
        }
        // every copy that this warp issued lands before the CTA may end
        for (int j = max(0, seq - NS); j < seq + kChunk; ++j) {
            const bool mine = j < seq ? j + NS >= seq + 32 || !((issued >> (j + NS - seq)) & 1) : (issued >> (j - seq)) & 1;
            if (mine) warp_drain(&full[j % NS], (j / NS) & 1);
        }
        for (int j = max(0, k - kSlots); j < k; ++j) warp_drain(&seg_q[j % kSlots], (j / kSlots) & 1);
    } else if (warp == NC + 1) {
        // ---------------------------------------------------------------------------------------- epilogue
        for (int k = 0;; ++k) {
            const int slot = k % kSlots, e = k % NB;
            if (!warp_wait(&seg_full[slot], (k / kSlots) & 1, ctx)) break;
            const Segment s = segs[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[slot]);
            if (s.units < 0) break;
            if (s.append) {
                // The new token, quantised while the pages are on their way: into the pool, and into a block that the
                // consumer of the pair's last unit takes it from (what the page's copy brings of its slot is not used).
                const int r = (s.len - 1) % kPageSize;
                const int32_t phys = p.block_table[(int64_t)s.b * p.max_pages + (s.len - 1) / kPageSize];
                const int64_t src = ((int64_t)s.b * p.Hkv + s.h) * kHeadDim;
                q4_quantise_row(static_cast<const __half*>(p.k_new) + src, new_blk, r, false, lane);
                q4_quantise_row(static_cast<const __half*>(p.v_new) + src, new_blk + kQ4Half, r, true, lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(new_full);
                if (phys >= 0 && phys < p.num_pages)
                    copy_token(static_cast<uint8_t*>(p.pool) + ((int64_t)phys * p.Hkv + s.h) * kQ4Block, new_blk, r, lane);
            }
            if (!warp_wait(&part_full[e], (k / NB) & 1, ctx)) break;
            const float* co = comb + e * NC * G * kCombRow;
            const float2* cml = comb_ml + e * NC * G;
            for (int g = 0; g < G; ++g) {
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < NC; ++w) M = fmaxf(M, cml[w * G + g].x);
                const float ref = M == -INFINITY ? 0.f : M;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                float l = 0.f;
#pragma unroll
                for (int w = 0; w < NC; ++w) {
                    const float2 ml = cml[w * G + g];
                    const float f = fast_exp2(ml.x - ref);
                    const float4 v = *reinterpret_cast<const float4*>(co + (w * G + g) * kCombRow + lane * 4);
                    l += f * ml.y;
                    a.x += f * v.x;
                    a.y += f * v.y;
                    a.z += f * v.z;
                    a.w += f * v.w;
                }
                if (s.out < 0) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    uint2 y;
                    y.x = pack_half2(a.x * inv, a.y * inv);
                    y.y = pack_half2(a.z * inv, a.w * inv);
                    *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + ((int64_t)s.b * p.Hq + s.h * G + g) * kHeadDim +
                                              lane * 4) = y;
                } else {
                    const int64_t state = (int64_t)s.out * G + g;
                    if (lane == 0) p.ml[state] = make_float2(M, l);
                    reinterpret_cast<float4*>(p.acc + state * kHeadDim)[lane] = a;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_empty[e]);
            if (s.out >= 0) {
                fence_acq_rel_gpu();  // this lane's part of the state is performed before the arrival
                __syncwarp();
                if (lane == 0) {
                    uint32_t* cnt = p.counters + s.first_cta;
                    if (atomicAdd(cnt, 1u) + 1u == (uint32_t)s.ctas) {
                        fence_acq_rel_gpu();  // the other pieces' states, published before their arrivals
                        atomicExch(cnt, 0u);  // re-armed for the next step
                        merges[*n_merges] = s;
                        *n_merges = *n_merges + 1;
                    }
                }
                __syncwarp();
            }
        }
        // rows without tokens
        for (int b = cta; b < p.B; b += gridDim.x) {
            const int len = p.seq_lens[b];
            if (row_length(p, b) == 0) {
                if (len != 0 && lane == 0) raise_status(ctx.status, PKV_STATUS_BAD_LEN);
                uint4* o = reinterpret_cast<uint4*>(static_cast<__half*>(p.out) + (int64_t)b * p.Hq * kHeadDim);
                for (int i = lane; i < p.Hq * kHeadDim / 8; i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    } else {
        // --------------------------------------------------------------------------------------- consumers
        const int g8 = lane >> 2;  // token row of S^T, dim row of O^T, head column of the B operand
        const int t4 = lane & 3;   // head columns 2 t4, 2 t4 + 1 of S^T and O^T
        // Up to four query heads leave half of the 8 columns empty. They get the heads a second time (kFold), and their lanes
        // take over the scores of tokens 8-15 of a page: every lane has one token instead of two, half of the scalar work.
        // In the second product those columns carry the weights' second part.
        constexpr bool kFold = G <= 4;
        constexpr int kTok = kFold ? 1 : 2;  // tokens of a page that this lane scores: tok0, and tok0 + 8
        const int tok0 = kFold ? g8 + ((t4 >> 1) << 3) : g8;
        const int col = kFold ? 2 * (t4 & 1) : 2 * t4;  // this lane's heads: 8 nt + col, + 1
        constexpr int kFirstLane = kFold ? 2 : 4;       // lanes that differ in bits from here on share their heads
        // of a score: sum_g scale_g (q.code_g) 2^-24 + offset_g (sum of q over g) 2^-24
        const float xk = fabsf(p.scale_log2) * 16777216.f;
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale turns q's signs
        int seq = 0, new_seen = 0;  // units, new tokens of the segments before
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int slot = k % kSlots, e = k % NB;
            if (!warp_wait(&seg_full[slot], (k / kSlots) & 1, ctx)) break;
            const int n = segs[slot].units, seg_append = segs[slot].append;
            if (n < 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&seg_empty[slot]);
                break;
            }
            if (!warp_wait(&seg_q[slot], (k / kSlots) & 1, ctx)) break;
            // Q^T as the B operand: b0 = Q[head][16 ks + 2 t4, + 1], b1 = + 8, + 9; head = 8 nt + g8
            uint32_t qb[kNT][8][2];
            float qs[kNT][2][2];  // [nt][group][head]: sum of q over the group, times xk 2^-24
            const uint8_t* qrow = smem + L::off_q + slot * G * kRowBytes;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const int head = kFold ? g8 & 3 : nt * 8 + g8;
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = head < G ? *reinterpret_cast<const uint32_t*>(qrow + head * kRowBytes +
                                                                                         (ks * 16 + 2 * t4 + 8 * i) * 2) ^ flip
                                                    : 0u;
                        qb[nt][ks][i] = w;
                        const float2 f = half2_of(w);
                        (ks < 4 ? s0 : s1) += f.x + f.y;
                    }
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    s0 += __shfl_xor_sync(0xffffffffu, s0, o);
                    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // from the lanes of that head
                    qs[nt][0][i] = __shfl_sync(0xffffffffu, s0, (col + i) * 4) * (xk * 5.9604644775390625e-8f);
                    qs[nt][1][i] = __shfl_sync(0xffffffffu, s1, (col + i) * 4) * (xk * 5.9604644775390625e-8f);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[slot]);

            float o[kNT][8][4];  // O^T: tile dt < 4 dims 16 dt + g8, + 8 of group 0; 4 + dt the same of group 1
            // Weights are 2^(x - ref) with ref chosen per head so that weight * V's scale stays below 2^14 and its
            // largest values above 1; ref is raised only when a unit would go beyond, then by what brings it to 2^7.
            float osum[kNT][2][2], taken[kNT][2][2], ref[kNT][2], l[kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
                for (int d = 0; d < 8; ++d) o[nt][d][0] = o[nt][d][1] = o[nt][d][2] = o[nt][d][3] = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ref[nt][i] = -INFINITY;
                    l[nt][i] = osum[nt][0][i] = osum[nt][1][i] = taken[nt][0][i] = taken[nt][1][i] = 0.f;
                }
            }
            // Unit j of the piece lives in stage j % NS and goes to warp j % NC; NS is a multiple of NC, so a stage
            // always has the same consumer.
            for (int i = (warp - seq % NC + NC) % NC; i < n; i += NC) {
                const int j = seq + i, st = j % NS;
                if (!warp_wait(&full[st], (j / NS) & 1, ctx)) {
                    ok = false;
                    break;
                }
                uint8_t* stage = smem + st * kStageBytes;
                const uint32_t mt = meta[st];
                const int nv = mt & 0xff;
                const uint32_t okmask = (mt >> 8) & kAllPages;
                const bool append = (mt >> 12) & 1;
                if (append) {
                    if (!warp_wait(new_full, new_seen & 1, ctx)) {
                        ok = false;
                        break;
                    }
                    const int pg = (nv - 1) / kPageSize;
                    if ((okmask >> pg) & 1) copy_token(stage + pg * kQ4Block, new_blk, (nv - 1) % kPageSize, lane);
                    __syncwarp();
                }
                const bool whole = nv == kUnitTokens && okmask == kAllPages;
                if (!whole) {  // tokens that the row does not have get parameters of 0, and scores of -inf below
                    for (int tok = lane; tok < kUnitTokens; tok += 32) {
                        const int pg = tok / kPageSize;
                        if (!((okmask >> pg) & 1) || tok >= nv) {
                            uint8_t* blk = stage + pg * kQ4Block + kQ4Codes + (tok % kPageSize) * 8;
                            *reinterpret_cast<uint2*>(blk) = make_uint2(0u, 0u);
                            *reinterpret_cast<uint2*>(blk + kQ4Half) = make_uint2(0u, 0u);
                        }
                    }
                    __syncwarp();
                }
                // scores of the unit's tokens: [page][token][head]
                float x[kNT][kUnitPages][kTok][2];
                __half2 top = __float2half2_rn(0.f);  // V's scales of this lane's tokens
#pragma unroll
                for (int p0 = 0; p0 < kUnitPages; p0 += 2) {  // two pages at a time: four chains of products in flight
                    uint32_t wa[2][4], wb[2][4];
                    float c0[2][kNT][4], c1[2][kNT][4];
#pragma unroll
                    for (int y = 0; y < (kUnitPages - p0 < 2 ? 1 : 2); ++y) {
                        const uint8_t* blk = stage + (p0 + y) * kQ4Block;
                        const uint4 ka = *reinterpret_cast<const uint4*>(blk + lane * 16);
                        const uint4 kb = *reinterpret_cast<const uint4*>(blk + 512 + lane * 16);
                        wa[y][0] = ka.x, wa[y][1] = ka.y, wa[y][2] = ka.z, wa[y][3] = ka.w;
                        wb[y][0] = kb.x, wb[y][1] = kb.y, wb[y][2] = kb.z, wb[y][3] = kb.w;
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                            for (int i2 = 0; i2 < 4; ++i2) c0[y][nt][i2] = c1[y][nt][i2] = 0.f;
                    }
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                        for (int y = 0; y < (kUnitPages - p0 < 2 ? 1 : 2); ++y) {
                            const uint32_t a8 = wa[y][ks] >> 8, b8 = wb[y][ks] >> 8;
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt) {
                                mma_16816(c0[y][nt], wa[y][ks] & 0x000F000Fu, wb[y][ks] & 0x000F000Fu, a8 & 0x000F000Fu,
                                          b8 & 0x000F000Fu, qb[nt][ks][0], qb[nt][ks][1]);
                                mma_16816(c1[y][nt], wa[y][ks] & 0x00F000F0u, wb[y][ks] & 0x00F000F0u, a8 & 0x00F000F0u,
                                          b8 & 0x00F000F0u, qb[nt][4 + ks][0], qb[nt][4 + ks][1]);
                            }
                        }
#pragma unroll
                    for (int y = 0; y < (kUnitPages - p0 < 2 ? 1 : 2); ++y) {
                        const int pg = p0 + y;
#pragma unroll
                        for (int u2 = 0; u2 < kTok; ++u2) {
                            const uint8_t* blk = stage + pg * kQ4Block + kQ4Codes + (tok0 + 8 * u2) * 8;
                            const uint2 pk = *reinterpret_cast<const uint2*>(blk);
                            const uint2 pv = *reinterpret_cast<const uint2*>(blk + kQ4Half);
                            const uint32_t sv = __byte_perm(pv.x, pv.y, 0x5410);
                            top = __hmax2(top, *reinterpret_cast<const __half2*>(&sv));
                            const float2 a0 = half2_of(pk.x), a1 = half2_of(pk.y);
                            const float a0s = a0.x * xk, a1s = a1.x * (0.0625f * xk);  // group 1's codes lie 4 bits higher
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                                for (int i2 = 0; i2 < 2; ++i2) {
                                    float d0 = c0[y][nt][2 * u2 + i2], d1 = c1[y][nt][2 * u2 + i2];
                                    if (kFold && t4 >= 2) {  // tokens 8-15
                                        d0 = c0[y][nt][2 + i2];
                                        d1 = c1[y][nt][2 + i2];
                                    }
                                    x[nt][pg][u2][i2] = fmaf(d0, a0s, fmaf(d1, a1s, fmaf(a0.y, qs[nt][0][i2], a1.y * qs[nt][1][i2])));
                                }
                        }
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int pg = 0; pg < kUnitPages; ++pg)
#pragma unroll
                        for (int u2 = 0; u2 < kTok; ++u2)
                            if (!((okmask >> pg) & 1) || pg * kPageSize + tok0 + 8 * u2 >= nv)
#pragma unroll
                                for (int nt = 0; nt < kNT; ++nt) x[nt][pg][u2][0] = x[nt][pg][u2][1] = -INFINITY;
                }
                // does a weight * scale of this unit go beyond 2^14? (per lane: its largest score and its largest scale)
                const __half peak = __hmax(__hmax(__low2half(top), __high2half(top)), __ushort_as_half(1));
                float need = __log2f(__half2float(peak)) - 7.f;
                float mx[kNT][2];
                bool raise = false;
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int i2 = 0; i2 < 2; ++i2) {
                        float v = -INFINITY;
#pragma unroll
                        for (int pg = 0; pg < kUnitPages; ++pg)
#pragma unroll
                            for (int u2 = 0; u2 < kTok; ++u2) v = fmaxf(v, x[nt][pg][u2][i2]);
                        mx[nt][i2] = v;
                        raise = raise || (v - ref[nt][i2]) + need > 7.f;
                    }
                if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                    for (int s = kFirstLane; s < 32; s <<= 1) need = fmaxf(need, __shfl_xor_sync(0xffffffffu, need, s));
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2) {
                            float v = mx[nt][i2];
#pragma unroll
                            for (int s = kFirstLane; s < 32; s <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
                            if ((v - ref[nt][i2]) + need > 7.f) {
                                // a score of which an fp32 has no fractions is the reference itself: the weights' exponents
                                // (x - ref) are then exact, and the largest weight is 1
                                if (fabsf(v) < 16777216.f) v += need;
                                const float f = fast_exp2(ref[nt][i2] - v);
                                ref[nt][i2] = v;
                                l[nt][i2] *= f;
                                osum[nt][0][i2] *= f;
                                osum[nt][1][i2] *= f;
                                taken[nt][0][i2] *= f;
                                taken[nt][1][i2] *= f;
#pragma unroll
                                for (int d = 0; d < 8; ++d) {
                                    o[nt][d][i2] *= f;
                                    o[nt][d][2 + i2] *= f;
                                }
                            }
                        }
                }
                float nref[kNT][2];
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int i2 = 0; i2 < 2; ++i2) nref[nt][i2] = ref[nt][i2] == -INFINITY ? 0.f : -ref[nt][i2];
                // Weights * scale as the B operand, in two fp16 parts, the second what the first's rounding left: the codes
                // are all positive, so a rounding of the weights would meet their common offset of 7.5 steps and cost three
                // times the output's own rounding. Folded, the two parts share the columns (0-3, 4-7) and take no
                // more products than one.
                uint32_t pb[kUnitPages][kNT][2][kFold ? 1 : 2][2];  // [page][nt][group][part][tokens 0-7, 8-15]
                float ws[kNT][2][2];  // weights * scale of this lane's tokens of the first page: [nt][group][head]
#pragma unroll
                for (int pg = 0; pg < kUnitPages; ++pg)
#pragma unroll
                    for (int u2 = 0; u2 < kTok; ++u2) {
                        const uint2 pv = *reinterpret_cast<const uint2*>(stage + pg * kQ4Block + kQ4Half + kQ4Codes + (tok0 + 8 * u2) * 8);
                        const float2 par[2] = {half2_of(pv.x), half2_of(pv.y)};
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            float w[2];
#pragma unroll
                            for (int i2 = 0; i2 < 2; ++i2) {
                                w[i2] = fast_exp2(x[nt][pg][u2][i2] + nref[nt][i2]);
                                l[nt][i2] += w[i2];
                                osum[nt][0][i2] = fmaf(w[i2], par[0].y, osum[nt][0][i2]);
                                osum[nt][1][i2] = fmaf(w[i2], par[1].y, osum[nt][1][i2]);
                            }
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                const float v0 = w[0] * par[g].x, v1 = w[1] * par[g].x;
                                if (pg == 0) {
                                    ws[nt][g][0] = u2 ? ws[nt][g][0] + v0 : v0;
                                    ws[nt][g][1] = u2 ? ws[nt][g][1] + v1 : v1;
                                }
                                const uint32_t hi = pack_half2(v0, v1);
                                const float2 hf = half2_of(hi);
                                const uint32_t th = transpose8x8(hi), tl = transpose8x8(pack_half2(v0 - hf.x, v1 - hf.y));
                                if (kFold) {
                                    // rows 0-3 of the transposes are tokens 0-7, rows 4-7 tokens 8-15 of the same heads;
                                    // columns 0-3 take the first part of all 16 tokens, columns 4-7 the second
                                    const uint32_t got = __shfl_xor_sync(0xffffffffu, g8 < 4 ? tl : th, 16);
                                    pb[pg][nt][g][0][0] = g8 < 4 ? th : got;
                                    pb[pg][nt][g][0][1] = g8 < 4 ? got : tl;
                                } else {
                                    pb[pg][nt][g][0][u2] = th;
                                    pb[pg][nt][g][kFold ? 0 : 1][u2] = tl;
                                }
                            }
                        }
                    }
                // The matrix instructions cut their sums to fp32 towards zero, which over a long row of codes of one sign adds
                // up (48 rows, 54 units a warp: 5.2e-4 of the output, its own rounding is 2.1e-4). So every unit
                // takes the codes' common offset out of the accumulators in advance, and the end puts it back: 8 times the
                // weights * scale, which this lane estimates from its own tokens of the first page (any amount would be
                // right; from its tokens of all pages: 1 % slower, and the same error).
                {
                    const float k0 = !kFold || t4 < 2 ? 8.f * kUnitTokens / kTok * 5.9604644775390625e-8f : 0.f;  // (not part 2)
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2) {
                            const float t0 = ws[nt][0][i2] * k0, t1 = ws[nt][1][i2] * (16.f * k0);
                            taken[nt][0][i2] += t0;
                            taken[nt][1][i2] += t1;
#pragma unroll
                            for (int d = 0; d < 4; ++d) {
                                o[nt][d][i2] -= t0;
                                o[nt][d][2 + i2] -= t0;
                                o[nt][4 + d][i2] -= t1;
                                o[nt][4 + d][2 + i2] -= t1;
                            }
                        }
                }
#pragma unroll
                for (int pg = 0; pg < kUnitPages; ++pg) {
                    const uint8_t* blk = stage + pg * kQ4Block + kQ4Half;
                    const uint4 va = *reinterpret_cast<const uint4*>(blk + lane * 16);
                    const uint4 vb = *reinterpret_cast<const uint4*>(blk + 512 + lane * 16);
                    const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
                    for (int dt = 0; dt < 4; ++dt) {
                        const uint32_t a8 = wa[dt] >> 8, b8 = wb[dt] >> 8;
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                            for (int part = 0; part < (kFold ? 1 : 2); ++part) {
                                mma_16816(o[nt][dt], wa[dt] & 0x000F000Fu, a8 & 0x000F000Fu, wb[dt] & 0x000F000Fu,
                                          b8 & 0x000F000Fu, pb[pg][nt][0][part][0], pb[pg][nt][0][part][1]);
                                mma_16816(o[nt][4 + dt], wa[dt] & 0x00F000F0u, a8 & 0x00F000F0u, wb[dt] & 0x00F000F0u,
                                          b8 & 0x00F000F0u, pb[pg][nt][1][part][0], pb[pg][nt][1][part][1]);
                            }
                    }
                }
                if (append || !whole) fence_proxy_async_smem();  // our stores into the stage before the next copy into it
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }
            if (!ok) break;
            seq += n;
            // every consumer sees every phase of this barrier (a parity two phases on would pass at once)
            if (seg_append && !warp_wait(new_full, new_seen & 1, ctx)) break;
            new_seen += seg_append;
            // hand this warp's partial result of the segment to the epilogue warp
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2) {
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        o[nt][d][i2] += taken[nt][d >> 2][i2];
                        o[nt][d][2 + i2] += taken[nt][d >> 2][i2];
                    }
                    if (kFold)
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            o[nt][d][i2] += __shfl_xor_sync(0xffffffffu, o[nt][d][i2], 2);
                            o[nt][d][2 + i2] += __shfl_xor_sync(0xffffffffu, o[nt][d][2 + i2], 2);
                        }
#pragma unroll
                    for (int s = kFirstLane; s < 32; s <<= 1) {
                        l[nt][i2] += __shfl_xor_sync(0xffffffffu, l[nt][i2], s);
                        osum[nt][0][i2] += __shfl_xor_sync(0xffffffffu, osum[nt][0][i2], s);
                        osum[nt][1][i2] += __shfl_xor_sync(0xffffffffu, osum[nt][1][i2], s);
                    }
                }
            if (!warp_wait(&part_empty[e], ((k / NB) & 1) ^ 1, ctx)) break;
            float* co = comb + (e * NC + warp) * G * kCombRow;
            float2* cml = comb_ml + (e * NC + warp) * G;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2) {
                    const int head = nt * 8 + col + i2;
                    if (head < G && (!kFold || t4 < 2)) {
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            const float f = d < 4 ? 16777216.f : 1048576.f;
                            co[head * kCombRow + d * 16 + g8] = fmaf(o[nt][d][i2], f, osum[nt][d >> 2][i2]);
                            co[head * kCombRow + d * 16 + g8 + 8] = fmaf(o[nt][d][2 + i2], f, osum[nt][d >> 2][i2]);
                        }
                        if (g8 == 0) cml[head] = make_float2(ref[nt][i2], l[nt][i2]);
                    }
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_full[e]);
        }
    }

    // The pairs whose last piece arrived here. The states of a pair come through the ring's memory by bulk copies, all in
    // flight together (read with loads, 8 a warp at a time, 38 states of 4 heads took 8 us); meanwhile a warp per head
    // takes the maximum of the references and turns them into factors.
    __syncthreads();
    const int nm = *abort_flag ? 0 : *n_merges;
    constexpr int kStateBytes = G * kHeadDim * 4;
    constexpr int kHeld = NS * kStageBytes / kStateBytes;  // states that the ring's memory holds
    float* factor = comb;                                  // [state][head]
    float* sums = reinterpret_cast<float*>(comb_ml);       // [head]
    uint32_t phase = 0;
    for (int i = 0; i < nm; ++i) {
        const Segment s = merges[i];
        const int64_t first = 2 * (int64_t)s.first_cta;  // state c of the pair: 2 (first_cta + c), + 1 for c = 0
        auto fetch = [&](int c0) {                       // warp 0: states c0 .. + kHeld - 1
            const int n = min(kHeld, s.ctas - c0);
            if (lane == 0) mbar_arrive_expect_tx(merged, n * kStateBytes);
            __syncwarp();
            for (int c = c0 + lane; c < c0 + n; c += 32)
                bulk_g2s(smem + (c - c0) * kStateBytes, p.acc + (first + 2 * c + (c == 0)) * (G * kHeadDim), kStateBytes, merged);
        };
        if (warp == 0) {
            fence_proxy_async_global();
            fetch(0);
        }
        for (int g = warp; g < G; g += NC + 2) {
            auto state = [&](int c) { return __ldcg(p.ml + (first + 2 * c + (c == 0)) * G + g); };
            float M = -INFINITY, l = 0.f;
            float2 kept[2];  // of the first 64 pieces
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = lane + 32 * i;
                kept[i] = c < s.ctas ? state(c) : make_float2(-INFINITY, 0.f);
            }
            M = fmaxf(kept[0].x, kept[1].x);
            for (int c = lane + 64; c < s.ctas; c += 32) M = fmaxf(M, state(c).x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            const float ref = M == -INFINITY ? 0.f : M;
            auto put = [&](int c, float2 ml) {
                const float f = fast_exp2(ml.x - ref);
                factor[c * G + g] = f;
                l += f * ml.y;
            };
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (lane + 32 * i < s.ctas) put(lane + 32 * i, kept[i]);
            for (int c = lane + 64; c < s.ctas; c += 32) put(c, state(c));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) sums[g] = l;
        }
        constexpr int kPer = (G + NC + 1) / (NC + 2);  // heads a warp
        float4 acc[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        bool here = true;
        for (int c0 = 0; c0 < s.ctas && here; c0 += kHeld) {
            __syncthreads();  // the factors are there; the states before have been used
            if (c0 > 0 && warp == 0) {
                fence_proxy_async_smem();
                fetch(c0);
            }
            here = warp_wait(merged, phase, ctx);
            phase ^= 1;
            const int n = here ? min(kHeld, s.ctas - c0) : 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int g = warp + j * (NC + 2);
                if (g < G) {
#pragma unroll 4
                    for (int c = 0; c < n; ++c) {
                        const float f = factor[(c0 + c) * G + g];
                        const float4 v = reinterpret_cast<const float4*>(smem + c * kStateBytes + g * kHeadDim * 4)[lane];
                        acc[j].x += f * v.x;
                        acc[j].y += f * v.y;
                        acc[j].z += f * v.z;
                        acc[j].w += f * v.w;
                    }
                }
            }
            here = __syncthreads_and(here);  // all leave together after a time-out
        }
        if (!here) break;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int g = warp + j * (NC + 2);
            if (g < G) {
                const float l = sums[g], inv = l == 0.f ? 0.f : 1.f / l;
                uint2 y;
                y.x = pack_half2(acc[j].x * inv, acc[j].y * inv);
                y.y = pack_half2(acc[j].z * inv, acc[j].w * inv);
                *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + ((int64_t)s.b * p.Hq + s.h * G + g) * kHeadDim + lane * 4) = y;
            }
        }
        __syncthreads();
        if (warp == 0) fence_proxy_async_smem();
    }
}

int64_t align_ws(int64_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }

int max_ctas(int group, int num_sms) { return (group >= 16 ? 1 : 2) * num_sms; }

template <int G>
int launch(Q4Params p, int num_sms, cudaStream_t stream) {
    using L = Shape<G>;
    static int configured_mask = 0;  // one bit per device ordinal (< 32)
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 32 || !(__atomic_load_n(&configured_mask, __ATOMIC_ACQUIRE) & (1 << dev))) {
        const cudaError_t e = cudaFuncSetAttribute(q4_decode_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::smem);
        if (e != cudaSuccess) return e;
        if (dev < 32) __atomic_fetch_or(&configured_mask, 1 << dev, __ATOMIC_ACQ_REL);
    }
    const int ctas = std::min(L::per_sm * num_sms, L::kFactors);
    char* ws = reinterpret_cast<char*>(p.hdr);
    int64_t off = sizeof(pkv_ws_header);
    p.counters = reinterpret_cast<uint32_t*>(ws + off);
    off += align_ws(4 * kMaxPieces);
    p.ml = reinterpret_cast<float2*>(ws + off);
    off += align_ws(8 * 2 * (int64_t)ctas * G);
    p.acc = reinterpret_cast<float*>(ws + off);
    // no more CTAs than the block table can feed
    const int64_t most = ((int64_t)p.B * p.Hkv * ((p.max_pages + kUnitPages - 1) / kUnitPages) + kMinUnits - 1) / kMinUnits;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(ctas, most));
    return launch_kernel(q4_decode_kernel<G>, grid, L::threads, L::smem, stream, p);
}

}  // namespace

size_t q4_workspace_bytes(const pkv_problem& pr, int num_sms) {
    const int g = pr.num_q_heads / pr.num_kv_heads;
    const int64_t ctas = max_ctas(g, num_sms);
    return sizeof(pkv_ws_header) + align_ws(4 * kMaxPieces) + align_ws(16 * ctas * g) + 2 * ctas * g * kHeadDim * 4;
}

int launch_q4_decode(const Q4Params& p, int num_sms, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (p.Hq / p.Hkv) {
        case 1: return launch<1>(p, num_sms, s);
        case 2: return launch<2>(p, num_sms, s);
        case 4: return launch<4>(p, num_sms, s);
        case 8: return launch<8>(p, num_sms, s);
        case 16: return launch<16>(p, num_sms, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
