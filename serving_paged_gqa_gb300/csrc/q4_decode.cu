// One decode step over the 4-bit pages (include/pkv.h, pkv_q4_decode_step).
//
// Per row b, KV head h and query head: x_j = scale * log2(e) * q.k_j, out = sum 2^(x_j - m) v_j / sum 2^(x_j - m), with
// k_j = sum over the two groups of (scale_j code_j + offset_j). Everything that is one number per (token, group) stays
// out of the matrix products and in fp32:
//   q.k_j   = sum_g scale_jg (q.code_jg) + offset_jg (sum of q over the group)
//   out     = sum_g sum_j (w_j scale_jg) code_jg + sum_j w_j offset_jg
// so the products (mma.sync m16n8k16, tokens or dims on the 16-row side, the G <= 16 query heads on the 8-column side)
// take the codes as they lie in memory: one mask makes two codes into two fp16 subnormals (q4.cuh), no conversion. The
// weights w_j scale_jg are rounded to fp16 once, relative to R_g, the largest V scale that the warp has met in the
// group (kept like a running maximum), so that V of any magnitude keeps its 11 bits. tcgen05 needs 64 or 128 rows of
// query heads, of which a KV head has G.
//
// Bound: HBM; a (token, KV head) is 144 bytes against 512 in fp16. A unit is 4 pages (64 tokens) of one (row, KV head),
// four bulk copies of 2304 bytes into one ring stage, and goes to one consumer warp.
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
#include "pkv_ptx.cuh"
#include "pkv_wait.cuh"
#include "q4.cuh"

namespace pkv {
namespace {

constexpr int kUnitPages = 4;
constexpr int kUnitTokens = kUnitPages * kPageSize;
constexpr int kStageBytes = kUnitPages * kQ4Block;
constexpr int kCombRow = kHeadDim + 4;  // floats per partial output row: rows land 4 banks apart
constexpr int kMinUnits = 4;            // units per CTA below which fewer CTAs take part

// A piece's part of one (row, KV head) pair.
struct Segment {
    int32_t b, h, units;  // units < 0: no more segments
    int32_t out;          // -1: the whole pair, written to out; else the state that it leaves
    int32_t first_cta, ctas;  // the pair's pieces
    int32_t pad[2];
};

// consumers, stages, partial-result buffers, resident CTAs
template <int G>
struct Shape {
    static constexpr int NC = G >= 16 ? 6 : 4;
    static constexpr int NS = 2 * NC;
    static constexpr int NB = G >= 8 ? 1 : 2;
    static constexpr int kSlots = G >= 16 ? 2 : 4;  // segments published ahead
    static constexpr int per_sm = G >= 16 ? 1 : 2;
    static constexpr int threads = (NC + 2) * 32;
    static constexpr int off_q = NS * kStageBytes;
    static constexpr int off_comb = off_q + kSlots * G * kRowBytes;
    static constexpr int off_comb_ml = off_comb + NB * NC * G * kCombRow * 4;
    static constexpr int off_seg = off_comb_ml + NB * NC * G * 8;
    static constexpr int off_meta = off_seg + (kSlots + 2) * (int)sizeof(Segment);  // and two pairs to merge
    static constexpr int off_bars = off_meta + NS * 4;
    static constexpr int nbars = 2 * NS + 3 * kSlots + 2 * NB;
    static constexpr int off_misc = off_bars + nbars * 8;
    static constexpr int smem = off_misc + 64;
    static_assert(off_bars % 8 == 0 && off_comb % 16 == 0 && smem <= 227 * 1024, "layout");
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

__device__ __forceinline__ float2 half2_of(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }

template <int G>
__global__ void __launch_bounds__(Shape<G>::threads, Shape<G>::per_sm) q4_decode_kernel(const Q4Params p) {
    using L = Shape<G>;
    constexpr int NC = L::NC, NS = L::NS, NB = L::NB, kSlots = L::kSlots, kNT = (G + 7) / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_scan[L::threads / 32];
    __shared__ int32_t s_row;   // where the piece begins: row,
    __shared__ int64_t s_unit;  // unit of the row's Hkv * units
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::off_bars);
    uint64_t* empty = full + NS;
    uint64_t* seg_full = empty + NS;
    uint64_t* seg_q = seg_full + kSlots;
    uint64_t* seg_empty = seg_q + kSlots;
    uint64_t* part_full = seg_empty + kSlots;
    uint64_t* part_empty = part_full + NB;
    Segment* segs = reinterpret_cast<Segment*>(smem + L::off_seg);
    Segment* merges = segs + kSlots;
    uint32_t* meta = reinterpret_cast<uint32_t*>(smem + L::off_meta);
    float* comb = reinterpret_cast<float*>(smem + L::off_comb);
    float2* comb_ml = reinterpret_cast<float2*>(smem + L::off_comb_ml);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::off_misc);
    volatile int* n_merges = abort_flag + 1;
    const WaitCtx ctx{abort_flag, &p.hdr->status};

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
        *abort_flag = 0;
        *n_merges = 0;
        mbar_fence_init();
    }
    // The line of units: every thread sums a run of rows, the CTA scans the sums, and the thread whose run holds the
    // piece's first unit finds its row.
    const int per = (p.B + L::threads - 1) / L::threads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += row_units(row_length(p, b));
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
            const int64_t n = (int64_t)row_units(row_length(p, b)) * p.Hkv;
            if (lo < at + n) {
                s_row = b;
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
        bool ok = true;
        int b = 0, h = 0, u = 0, len = 0, units = 0;
        if (lo < hi) {
            b = s_row;
            len = row_length(p, b);
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
            if (lane == 0) {
                Segment s;
                s.b = b;
                s.h = h;
                s.units = n;
                s.out = n == units ? -1 : 2 * cta + (u == 0 ? 1 : 0);
                s.first_cta = cta_of(pos - u, total, ctas);
                s.ctas = cta_of(pos - u + units - 1, total, ctas) - s.first_cta + 1;
                s.pad[0] = s.pad[1] = 0;
                segs[slot] = s;
                mbar_arrive(&seg_full[slot]);
                mbar_arrive_expect_tx(&seg_q[slot], G * kRowBytes);
                bulk_g2s(smem + L::off_q + slot * G * kRowBytes, q + ((int64_t)b * p.Hq + (int64_t)h * G) * kHeadDim,
                         G * kRowBytes, &seg_q[slot]);
            }
            __syncwarp();
            const int32_t* bt = p.block_table + (int64_t)b * p.max_pages;
            const int pages = (len + kPageSize - 1) / kPageSize;
            const int p0 = u * kUnitPages;  // the segment's first page; lanes hold 32 entries (8 units) at a time
            int ent = p0 + lane < pages ? bt[p0 + lane] : -1, ent_next = -1;
            for (int i = 0; i < n; ++i) {
                if ((i & 7) == 0) {
                    if (i > 0) ent = ent_next;
                    const int at = p0 + (i + 8) * kUnitPages + lane;
                    ent_next = i + 8 < n && at < pages ? bt[at] : -1;
                }
                const int first = (u + i) * kUnitPages;
                const int np = min(kUnitPages, pages - first);
                const int mine_ent = __shfl_sync(0xffffffffu, ent, (i & 7) * kUnitPages + (lane & 3));
                const bool good = lane < np && mine_ent >= 0 && mine_ent < p.num_pages;
                const unsigned okmask = __ballot_sync(0xffffffffu, good);
                const int st = seq % NS;
                if (!warp_wait(&empty[st], ((seq / NS) & 1) ^ 1, ctx)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const int nv = min(kUnitTokens, len - (u + i) * kUnitTokens);
                    const bool append = p.k_new && u + i == units - 1;
                    meta[st] = (uint32_t)nv | okmask << 8 | (append ? 1u << 12 : 0u);
                    if (okmask != (1u << np) - 1u) raise_status(ctx.status, PKV_STATUS_BAD_PAGE);
                    if (okmask)
                        mbar_arrive_expect_tx(&full[st], __popc(okmask) * kQ4Block);
                    else
                        mbar_arrive(&full[st]);
                }
                __syncwarp();
                if (good)
                    bulk_g2s_hint(smem + st * kStageBytes + lane * kQ4Block,
                                  pool + ((int64_t)mine_ent * p.Hkv + h) * kQ4Block, kQ4Block, &full[st], pol);
                __syncwarp();
                ++seq;
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
        for (int j = max(0, seq - NS); j < seq; ++j) warp_drain(&full[j % NS], (j / NS) & 1);
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
        const float sl2 = p.scale_log2;
        int seq = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int slot = k % kSlots, e = k % NB;
            if (!warp_wait(&seg_full[slot], (k / kSlots) & 1, ctx)) break;
            const int n = segs[slot].units, sb = segs[slot].b, sh = segs[slot].h;
            if (n < 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&seg_empty[slot]);
                break;
            }
            if (!warp_wait(&seg_q[slot], (k / kSlots) & 1, ctx)) break;
            // Q^T as the B operand: b0 = Q[head][16 ks + 2 t4, + 1], b1 = + 8, + 9; head = 8 nt + g8
            uint32_t qb[kNT][8][2];
            float qs[kNT][2][2];  // [nt][group][head 2 t4, 2 t4 + 1]: sum of q over the group, times scale * log2(e)
            const uint8_t* qrow = smem + L::off_q + slot * G * kRowBytes;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const int head = nt * 8 + g8;
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = head < G ? *reinterpret_cast<const uint32_t*>(qrow + head * kRowBytes +
                                                                                         (ks * 16 + 2 * t4 + 8 * i) * 2)
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
                for (int i = 0; i < 2; ++i) {  // from the lanes of head 2 t4 + i
                    qs[nt][0][i] = __shfl_sync(0xffffffffu, s0, (2 * t4 + i) * 4) * sl2;
                    qs[nt][1][i] = __shfl_sync(0xffffffffu, s1, (2 * t4 + i) * 4) * sl2;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[slot]);

            float o[kNT][8][4];  // O^T: tile dt < 4 dims 16 dt + g8, + 8 of group 0; 4 + dt the same of group 1
            float osum[kNT][2][2], m[kNT][2], l[kNT][2], R[2] = {0.f, 0.f};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
                for (int d = 0; d < 8; ++d) o[nt][d][0] = o[nt][d][1] = o[nt][d][2] = o[nt][d][3] = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    m[nt][i] = -INFINITY;
                    l[nt][i] = osum[nt][0][i] = osum[nt][1][i] = 0.f;
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
                const uint32_t okmask = (mt >> 8) & 0xf;
                const bool append = (mt >> 12) & 1;
                if (append) {
                    const int r = (nv - 1) % kPageSize, pg = (nv - 1) / kPageSize;
                    if ((okmask >> pg) & 1) {
                        uint8_t* blk = stage + pg * kQ4Block;
                        const int64_t src = ((int64_t)sb * p.Hkv + sh) * kHeadDim;
                        q4_quantise_row(static_cast<const __half*>(p.k_new) + src, blk, r, false, lane);
                        q4_quantise_row(static_cast<const __half*>(p.v_new) + src, blk + kQ4Half, r, true, lane);
                        __syncwarp();
                        // the token's bytes into the pool: 64 code bytes and 8 parameter bytes of K and of V
                        const int32_t phys = p.block_table[(int64_t)sb * p.max_pages + (row_length(p, sb) - 1) / kPageSize];
                        uint8_t* dst = static_cast<uint8_t*>(p.pool) + ((int64_t)phys * p.Hkv + sh) * kQ4Block;
#pragma unroll
                        for (int d = lane; d < 64; d += 32) {
                            const int kb = q4_k_byte(r, d), vb = kQ4Half + q4_v_byte(r, d);
                            dst[kb] = blk[kb];
                            dst[vb] = blk[vb];
                        }
                        if (lane < 4) {
                            const int at = (lane >> 1) * kQ4Half + kQ4Codes + r * 8 + (lane & 1) * 4;
                            *reinterpret_cast<uint32_t*>(dst + at) = *reinterpret_cast<const uint32_t*>(blk + at);
                        }
                    }
                }
                const bool whole = nv == kUnitTokens && okmask == 0xf;
                // scores of the unit's 64 tokens: this lane holds tokens 16 pg + g8, + 8 of heads 2 t4, 2 t4 + 1
                float x[kNT][kUnitPages][4];
                uint32_t vpar[kUnitPages][2][2];  // [page][token g8, + 8][group]: V's (scale, offset)
                __half2 top = __float2half2_rn(0.f);
#pragma unroll
                for (int pg = 0; pg < kUnitPages; ++pg) {
                    const uint8_t* blk = stage + pg * kQ4Block;
                    const uint4 ka = *reinterpret_cast<const uint4*>(blk + lane * 16);
                    const uint4 kb = *reinterpret_cast<const uint4*>(blk + 512 + lane * 16);
                    const uint2 pa = *reinterpret_cast<const uint2*>(blk + kQ4Codes + g8 * 8);
                    const uint2 pb = *reinterpret_cast<const uint2*>(blk + kQ4Codes + 64 + g8 * 8);
                    uint2 va = *reinterpret_cast<const uint2*>(blk + kQ4Half + kQ4Codes + g8 * 8);
                    uint2 vb = *reinterpret_cast<const uint2*>(blk + kQ4Half + kQ4Codes + 64 + g8 * 8);
                    bool oka = true, okb = true;
                    if (!whole) {
                        const bool pgok = (okmask >> pg) & 1;
                        oka = pgok && pg * kPageSize + g8 < nv;
                        okb = pgok && pg * kPageSize + g8 + 8 < nv;
                        if (!oka) va = make_uint2(0u, 0u);
                        if (!okb) vb = make_uint2(0u, 0u);
                    }
                    vpar[pg][0][0] = va.x;
                    vpar[pg][0][1] = va.y;
                    vpar[pg][1][0] = vb.x;
                    vpar[pg][1][1] = vb.y;
                    const uint32_t sa = __byte_perm(va.x, va.y, 0x5410), sb2 = __byte_perm(vb.x, vb.y, 0x5410);
                    top = __hmax2(top, __hmax2(*reinterpret_cast<const __half2*>(&sa), *reinterpret_cast<const __half2*>(&sb2)));
                    float c0[kNT][4], c1[kNT][4];
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int i2 = 0; i2 < 4; ++i2) c0[nt][i2] = c1[nt][i2] = 0.f;
                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint32_t a8 = wa[ks] >> 8, b8 = wb[ks] >> 8;
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            mma_16816(c0[nt], wa[ks] & 0x000F000Fu, wb[ks] & 0x000F000Fu, a8 & 0x000F000Fu,
                                      b8 & 0x000F000Fu, qb[nt][ks][0], qb[nt][ks][1]);
                            mma_16816(c1[nt], wa[ks] & 0x00F000F0u, wb[ks] & 0x00F000F0u, a8 & 0x00F000F0u,
                                      b8 & 0x00F000F0u, qb[nt][4 + ks][0], qb[nt][4 + ks][1]);
                        }
                    }
                    const float2 a0 = half2_of(pa.x), a1 = half2_of(pa.y), b0f = half2_of(pb.x), b1f = half2_of(pb.y);
                    const float k24 = sl2 * 16777216.f, k20 = sl2 * 1048576.f;
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2) {
                            const float va_ = fmaf(c0[nt][i2], a0.x * k24, fmaf(c1[nt][i2], a1.x * k20,
                                                   fmaf(a0.y, qs[nt][0][i2], a1.y * qs[nt][1][i2])));
                            const float vb_ = fmaf(c0[nt][2 + i2], b0f.x * k24, fmaf(c1[nt][2 + i2], b1f.x * k20,
                                                   fmaf(b0f.y, qs[nt][0][i2], b1f.y * qs[nt][1][i2])));
                            x[nt][pg][i2] = oka ? va_ : -INFINITY;
                            x[nt][pg][2 + i2] = okb ? vb_ : -INFINITY;
                        }
                    }
                }
                // running maxima: scores per head, V's scales per group
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) top = __hmax2(top, __shfl_xor_sync(0xffffffffu, top, s));
                const float2 tf = __half22float2(top);
                bool change = tf.x > R[0] || tf.y > R[1];
                float mx[kNT][2];
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
                    for (int i2 = 0; i2 < 2; ++i2) {
                        float v = fmaxf(x[nt][0][i2], x[nt][0][2 + i2]);
#pragma unroll
                        for (int pg = 1; pg < kUnitPages; ++pg) v = fmaxf(v, fmaxf(x[nt][pg][i2], x[nt][pg][2 + i2]));
#pragma unroll
                        for (int s = 4; s < 32; s <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
                        mx[nt][i2] = fmaxf(v, m[nt][i2]);
                        change = change || mx[nt][i2] != m[nt][i2];
                    }
                }
                if (__any_sync(0xffffffffu, change)) {
                    float fr[2];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float r = fmaxf(R[g], g ? tf.y : tf.x);
                        fr[g] = R[g] > 0.f ? R[g] / r : 0.f;
                        R[g] = r;
                    }
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2) {
                            const float f = mx[nt][i2] == -INFINITY ? 1.f : fast_exp2(m[nt][i2] - mx[nt][i2]);
                            m[nt][i2] = mx[nt][i2];
                            l[nt][i2] *= f;
                            osum[nt][0][i2] *= f;
                            osum[nt][1][i2] *= f;
#pragma unroll
                            for (int d = 0; d < 8; ++d) {
                                o[nt][d][i2] *= f * fr[d >> 2];
                                o[nt][d][2 + i2] *= f * fr[d >> 2];
                            }
                        }
                    }
                }
                const float ir0 = R[0] > 0.f ? 1.f / R[0] : 0.f, ir1 = R[1] > 0.f ? 1.f / R[1] : 0.f;
#pragma unroll
                for (int pg = 0; pg < kUnitPages; ++pg) {
                    const uint8_t* blk = stage + pg * kQ4Block + kQ4Half;
                    const uint4 va = *reinterpret_cast<const uint4*>(blk + lane * 16);
                    const uint4 vb = *reinterpret_cast<const uint4*>(blk + 512 + lane * 16);
                    const float2 a0 = half2_of(vpar[pg][0][0]), a1 = half2_of(vpar[pg][0][1]);
                    const float2 b0f = half2_of(vpar[pg][1][0]), b1f = half2_of(vpar[pg][1][1]);
                    uint32_t pb[kNT][2][2];  // [nt][group]: weights * scale as the B operand
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
                        float w[4];
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2) {
                            const float ref = m[nt][i2] == -INFINITY ? 0.f : m[nt][i2];
                            w[i2] = fast_exp2(x[nt][pg][i2] - ref);
                            w[2 + i2] = fast_exp2(x[nt][pg][2 + i2] - ref);
                            l[nt][i2] += w[i2] + w[2 + i2];
                            osum[nt][0][i2] = fmaf(w[i2], a0.y, fmaf(w[2 + i2], b0f.y, osum[nt][0][i2]));
                            osum[nt][1][i2] = fmaf(w[i2], a1.y, fmaf(w[2 + i2], b1f.y, osum[nt][1][i2]));
                        }
                        const float s0 = a0.x * ir0, s1 = a1.x * ir1, u0 = b0f.x * ir0, u1 = b1f.x * ir1;
                        pb[nt][0][0] = transpose8x8(pack_half2(w[0] * s0, w[1] * s0));
                        pb[nt][0][1] = transpose8x8(pack_half2(w[2] * u0, w[3] * u0));
                        pb[nt][1][0] = transpose8x8(pack_half2(w[0] * s1, w[1] * s1));
                        pb[nt][1][1] = transpose8x8(pack_half2(w[2] * u1, w[3] * u1));
                    }
                    const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
                    for (int dt = 0; dt < 4; ++dt) {
                        const uint32_t a8 = wa[dt] >> 8, b8 = wb[dt] >> 8;
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            mma_16816(o[nt][dt], wa[dt] & 0x000F000Fu, a8 & 0x000F000Fu, wb[dt] & 0x000F000Fu,
                                      b8 & 0x000F000Fu, pb[nt][0][0], pb[nt][0][1]);
                            mma_16816(o[nt][4 + dt], wa[dt] & 0x00F000F0u, a8 & 0x00F000F0u, wb[dt] & 0x00F000F0u,
                                      b8 & 0x00F000F0u, pb[nt][1][0], pb[nt][1][1]);
                        }
                    }
                }
                if (append) fence_proxy_async_smem();  // our stores into the stage before the next copy into it
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }
            if (!ok) break;
            seq += n;
            // hand this warp's partial result of the segment to the epilogue warp
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
                    for (int s = 4; s < 32; s <<= 1) {
                        l[nt][i2] += __shfl_xor_sync(0xffffffffu, l[nt][i2], s);
                        osum[nt][0][i2] += __shfl_xor_sync(0xffffffffu, osum[nt][0][i2], s);
                        osum[nt][1][i2] += __shfl_xor_sync(0xffffffffu, osum[nt][1][i2], s);
                    }
            if (!warp_wait(&part_empty[e], ((k / NB) & 1) ^ 1, ctx)) break;
            float* co = comb + (e * NC + warp) * G * kCombRow;
            float2* cml = comb_ml + (e * NC + warp) * G;
            const float f0 = R[0] * 16777216.f, f1 = R[1] * 1048576.f;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2) {
                    const int head = nt * 8 + 2 * t4 + i2;
                    if (head < G) {
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            const float f = d < 4 ? f0 : f1;
                            co[head * kCombRow + d * 16 + g8] = fmaf(o[nt][d][i2], f, osum[nt][d >> 2][i2]);
                            co[head * kCombRow + d * 16 + g8 + 8] = fmaf(o[nt][d][2 + i2], f, osum[nt][d >> 2][i2]);
                        }
                        if (g8 == 0) cml[head] = make_float2(m[nt][i2], l[nt][i2]);
                    }
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_full[e]);
        }
    }

    // The pairs whose last piece arrived here: warps take their states in turn, eight loads of one head in flight.
    __syncthreads();
    const int nm = *abort_flag ? 0 : *n_merges;
    for (int i = 0; i < nm; ++i) {
        const Segment s = merges[i];
        if (warp < NC) {
            for (int g = 0; g < G; ++g) {
                float M = -INFINITY, l = 0.f;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c0 = warp; c0 < s.ctas; c0 += 8 * NC) {
                    float2 ml[8];
                    float4 v[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int at = c0 + c * NC;
                        const int64_t state = (int64_t)(2 * (s.first_cta + at) + (at == 0 ? 1 : 0)) * G + g;
                        ml[c] = at < s.ctas ? __ldcg(p.ml + state) : make_float2(-INFINITY, 0.f);
                        v[c] = at < s.ctas ? __ldcg(reinterpret_cast<const float4*>(p.acc + state * kHeadDim) + lane)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    float mn = M;
#pragma unroll
                    for (int c = 0; c < 8; ++c) mn = fmaxf(mn, ml[c].x);
                    const float ref = mn == -INFINITY ? 0.f : mn;
                    const float f = fast_exp2(M - ref);
                    M = mn;
                    l *= f;
                    a.x *= f;
                    a.y *= f;
                    a.z *= f;
                    a.w *= f;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float e = fast_exp2(ml[c].x - ref);
                        l += e * ml[c].y;
                        a.x += e * v[c].x;
                        a.y += e * v[c].y;
                        a.z += e * v[c].z;
                        a.w += e * v[c].w;
                    }
                }
                *reinterpret_cast<float4*>(comb + (warp * G + g) * kCombRow + lane * 4) = a;
                if (lane == 0) comb_ml[warp * G + g] = make_float2(M, l);
            }
        }
        __syncthreads();
        for (int g = warp; g < G; g += NC + 2) {
            float M = -INFINITY, l = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NC; ++w) M = fmaxf(M, comb_ml[w * G + g].x);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < NC; ++w) {
                const float2 ml = comb_ml[w * G + g];
                const float f = fast_exp2(ml.x - ref);
                const float4 v = *reinterpret_cast<const float4*>(comb + (w * G + g) * kCombRow + lane * 4);
                l += f * ml.y;
                a.x += f * v.x;
                a.y += f * v.y;
                a.z += f * v.z;
                a.w += f * v.w;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint2 y;
            y.x = pack_half2(a.x * inv, a.y * inv);
            y.y = pack_half2(a.z * inv, a.w * inv);
            *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + ((int64_t)s.b * p.Hq + s.h * G + g) * kHeadDim + lane * 4) = y;
        }
        __syncthreads();
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
    const int ctas = L::per_sm * num_sms;
    char* ws = reinterpret_cast<char*>(p.hdr);
    int64_t off = sizeof(pkv_ws_header);
    p.counters = reinterpret_cast<uint32_t*>(ws + off);
    off += align_ws(4 * (int64_t)ctas);
    p.ml = reinterpret_cast<float2*>(ws + off);
    off += align_ws(8 * 2 * (int64_t)ctas * G);
    p.acc = reinterpret_cast<float*>(ws + off);
    // no more CTAs than the block table can feed
    const int64_t most = ((int64_t)p.B * p.Hkv * ((p.max_pages + kUnitPages - 1) / kUnitPages) + kMinUnits - 1) / kMinUnits;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(ctas, most));
    q4_decode_kernel<G><<<grid, L::threads, L::smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t q4_workspace_bytes(const pkv_problem& pr, int num_sms) {
    const int g = pr.num_q_heads / pr.num_kv_heads;
    const int64_t ctas = max_ctas(g, num_sms);
    return sizeof(pkv_ws_header) + align_ws(4 * ctas) + align_ws(16 * ctas * g) + 2 * ctas * g * kHeadDim * 4;
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
