// Attention of packed new tokens over the FP16 pages that hold them and their sequences' earlier tokens (include/pkv.h,
// pkv_chunk_attention), and of one token a row over selected pages (pkv_sparse_decode_step).
//
// For token i of a sequence (position start + i) and query head hq of KV head h: out = sum_j p_j v_j / sum_j p_j over the
// positions j <= start + i, p_j = 2^(x_j - ref), x_j = scale * log2(e) * q_i.k_j. Products on the 5th-generation tensor
// cores, tiles of 128 rows = 128 / G tokens x G heads, two tiles (A, B: a pair) a CTA at a time over 128 keys a step;
// references and precision of the weights as in prompt_attention.cu. What differs is where keys come from and who does what.
//
// Keys: a step is 8 pages of 16 tokens. A page of one KV head is two TMA boxes (64 dims x 16 tokens) for K and two for V;
// boxes of consecutive pages lie one behind the other in a stage, which gives the same operand layout as one box of 128
// rows. Block-table entries are read 32 at a time ahead of their use. An entry outside the pool becomes a coordinate
// outside the tensor: the copy brings zeros. (A box of 128 rows would take 4 % less: 32 boxes a step keep the copy engine busy.)
//
// Division: a pair of tiles of one (sequence, KV head) has as many steps as its last token has keys. Neither one long
// context with a few new tokens (one pair a KV head) nor a batch of unequal ones fills the GPU pair by pair, so the steps
// of all pairs form one line, in the order (sequence, KV heads, pair, step), and it is cut into equal pieces wherever the
// cuts fall, but for what lies next to a pair's ends. A piece belongs to `lanes` CTAs, one for each of `lanes` neighbouring KV
// heads, so that they read the same pages at the same time (a token's heads are contiguous in a page). Every CTA finds its piece
// from a scan of the sequences' lengths; there is no plan, and one captured graph serves every step. A pair that lies in one
// piece is written out at once. The others leave a state a piece (ref, sum, accumulator, in fp32; a CTA leaves two at most), and a
// second kernel, launched to overlap this one's end, adds them up in the order of the pieces: results do not depend on timing.
//
// Two forms of the kernel: sequences of more than one tile of new tokens (pairs, bound by the tensor core), and sequences of one
// tile (few rows, bound by HBM or latency: see softmax_tile). Warp roles of both:
//   warps 0-15      softmax and output rows, thread = row; warps 0-3 and 4-7 the first and second 64 keys of tile A, 8-15 of B
//   warp 16         one (elected) thread waits for and issues the matrix instructions
//   warps 17, 19    copies of queries and K, and of V, whose rows behind the last key warp 19 clears
//   warp 18         walks the piece and publishes its pairs, two ahead
// Every wait is bounded (pkv_wait.cuh).
//
// Precision: sums, references and states are fp32; the second product takes its weights as fp16, like the values, as both of its operands
// have one type. Relative error 2.9e-4 (the output's rounding alone 2.1e-4), in tiles of at most 64 rows 2.1e-4 from a second fp16 part:
// a token's error depends on how many tokens come with it. Either way the largest weight of a row is about 2^5 and fp16's least 2^-24:
// weights below 2^-30 of the row's largest are 0, and those below 2^-19 have less than 11 bits. Where a row's values are those of such weights
// alone (6000 equal keys next to one 16 / 18 / 20 nats above them whose value is 0), the error is 1.8e-3 / 5.4e-3 / 2.3e-2.
//
// Measured on GB300s (32 query heads, 8 KV heads): 4096 tokens behind 28672 1.38 ms, 1490 TFLOP/s, 0.79 of the
// measured cuBLAS burst under the power cap; 16384 without a prefix 1.40 ms (1570 TFLOP/s; prompt_attention.cu 1.30-1.39); 512
// behind 8192 64 us, of which 28 steps take 46; 16 sequences of 2-8 tokens behind 1000-32000 204 us, 5.75 TB/s; 5 tokens behind 700
// 14.6 us. Under ncu (512 behind 8192, cold) the tensor pipe is active 49 % of the time, warps wait for TMEM loads and for
// instructions; a step of a pair takes 3060 cycles, of which the tensor core's share is 2048 (prompt_attention.cu 2820, which spills no
// register; here, at the same 96 a thread, the kernel for pairs spills 52 bytes and loads 284, that for few rows 64 and 84).
// Tried and dropped: the next pair's first scores issued before the current pair's last products (nothing, and 3-6 % slower with
// short pairs); a grid of merging blocks that share the items they count (2 us slower); both kinds of sequences in one
// kernel (its registers spill: 8192 tokens 371 us, 420); one box of 4 KB a page, its halves side by side (16 sequences of 2-8 tokens
// 205 -> 203 us, 12 of 1-1024 600 -> 610); the next pair's table entries read ahead, its queries behind its first keys, rows of few
// written out in rolled loops (nothing, or 1 us more a call).
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "pkv_internal.h"
#include "pkv_launch.h"
#include "pkv_tcgen05.cuh"
#include "pkv_tensormap.h"
#include "pkv_wait.cuh"

namespace pkv {
namespace {

constexpr uint64_t kFinishNs = 32 * 1000;    // a warp's 32 rows, by the key that they are computed from again, at most
constexpr uint64_t kFinishMostNs = 30000000000ull;  // (a million keys)
constexpr int kRows = 128;                   // rows of a tile, keys of a step
constexpr unsigned kAllLanes = 0xffffffffu;
constexpr int kStepPages = kRows / kPageSize;
constexpr int kTileBytes = kRows * kRowBytes;  // 32 KB: two halves of 64 dims
constexpr int kBoxBytes = kTileBytes / 2;
constexpr int kPageBox = kPageSize * 128;    // one page's part of a half
constexpr int kMostStages = 5;
constexpr int kSoftmax = 512;                // threads of the softmax
constexpr int kThreads = kSoftmax + 128;
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;  // 512 * 104 + 128 * 64 = 640 * 96, what the launch has
constexpr float kMost = 65504.f;             // sum of 64 weights above which the row's reference is raised
constexpr float kLift = 5.f;                 // the largest weight where the reference was set, in powers of two
// What a pair takes beside its steps (its queries' way in, its rows' way out, during which the tensor core or the copies run dry), in
// steps. (Many: 8192 tokens without a prefix 405 us with 0, 394 with 2. Few: 64 sequences of one token behind 1023 75 us with 2, 72
// with 3.)
template <bool kFew>
constexpr int kPairCost = kFew ? 3 : 2;
constexpr int kMinCost = 2;                  // of a piece, at least
constexpr int kWhole = 5;                    // cost of a pair that is not cut where a piece has no more

// One sequence: its first packed row, its new tokens, and how many it holds before them.
struct Seq {
    int32_t first, n, start;
};

struct Work {
    Seq q;
    int32_t s, t0, h;  // sequence; first new token of tile A; KV head (-1: no more work)
    int32_t j0, j1;    // steps of this piece
    int32_t state;     // -1: the whole pair, written to out; else the state that it leaves
};

// A pair whose states are to be added up: `pieces` of them, the first in slot 2 cta + 1 of the CTA that has this entry, the
// others in slots 2 (cta + i lanes).
struct Merge {
    Seq q;
    int32_t s, t0, h, pieces, reserved;
};
static_assert(sizeof(Merge) == kChunkMergeBytes, "workspace layout");

// Barriers of the CTA, in shared memory.
struct Bars {
    uint64_t kv_full[kMostStages], kv_empty[kMostStages];
    uint64_t w_full[2], w_empty[2];  // a work has been published; every warp is done with what it needs of it
    uint64_t q_full[2], q_empty[2];  // like those below: tile A, tile B
    uint64_t s_full[2];              // the tile's scores are in TMEM
    uint64_t p_full[2][2];           // its weights of the step's first, second 64 keys are
    uint64_t o_full[2];              // its accumulator is complete
    uint64_t lo_done[2];             // the products of a step's first 64 keys are in the accumulator
    uint64_t o_free[2];              // the accumulator has been read; few, of A: and the second half is done with the tile
    uint64_t first_ref[2][4];        // [tile][warp of the half]: the tile's first references are in shared memory
    uint64_t half_done[2][4];        // [tile][warp of the half]: the second half has settled its weights of the step
    uint64_t low_full[8], low_empty[8];  // few: [tile][half][warp of rows 0-63] second parts' accumulators are there, have been read
    uint64_t told[8];                // few: [half][warp of the half] so are the rows that B's warp has found
    uint64_t tail_full;              // a tile of V with rows behind the pair's last key has come
    uint64_t drain;
};

// Shared memory. Few: the kernel of sequences whose new tokens are one tile.
template <bool kFew>
struct Layout {
    static constexpr int kStages = kFew ? 5 : 4;  // K and V tiles in flight
    static constexpr int q = 0;
    static constexpr int ring = (kFew ? 1 : 2) * kTileBytes;
    static constexpr int work = ring + kStages * kTileBytes;
    static constexpr int bars = work + 2 * (int)sizeof(Work);
    static constexpr int ref = bars + (int)sizeof(Bars);         // float [tile][row]: ref
    static constexpr int parts = ref + 2 * kRows * 4;            // float2 (ref, l) [work & 1][tile][half][row]
    static constexpr int late = parts + 2 * 2 * 2 * kRows * 8;   // int [tile][warp of the half]: the second half raises
    static constexpr int scan = late + 8 * 4;                    // int64 [warp]: cost of the sequences of a warp's threads
    static constexpr int begin = scan + kThreads / 32 * 8;       // int64, int32: where the piece begins
    static constexpr int low = begin + 16;                       // few: uint32 [tile][half][64][17]: second parts' accumulators
    static constexpr int told = low + (kFew ? 4 * 64 * 17 * 4 : 0);  // few: uint32 [half][warp]: rows to be finished
    static constexpr int misc = told + 8 * 4;                    // abort flag, TMEM address
    static constexpr int bytes = misc + 16 + 1024;               // slack to align the base to 1024 bytes
    static_assert(sizeof(Work) % 4 == 0 && bars % 8 == 0 && parts % 8 == 0 && scan % 8 == 0, "alignment");
    static_assert(kStages <= kMostStages && bytes <= 227 * 1024, "shared memory");
};

struct Params {
    CUtensorMap q, q64, k, v;  // q: 128 rows a box; q64: 64
    ChunkParams p;
};

// ---- sequences, pairs of tiles and their steps ---------------------------------------------------------------------
// Sequence s; nothing (n = 0) where its bounds or lengths are not inside the tensors.
__device__ __forceinline__ Seq load_seq(const ChunkParams& p, int s, bool& bad) {
    Seq q;
    if (p.seq_lens) {  // one token a row, behind the keys of its selected pages; the last of them ends with the row
        const int len = p.seq_lens[s];
        bad = len < 0 || len > (int64_t)p.max_pages * kPageSize;
        q.first = s;
        q.n = bad || len == 0 ? 0 : 1;
        q.start = (min((len + kPageSize - 1) / kPageSize, p.select) - 1) * kPageSize + (len - 1) % kPageSize;
    } else {
        q.first = p.cu_seqlens[s];
        const int last = p.cu_seqlens[s + 1];
        q.start = p.start ? p.start[s] : 0;
        bad = q.first < 0 || last < q.first || last > p.total_tokens || q.start < 0 ||
              (int64_t)q.start + (last - q.first) > (int64_t)p.max_pages * kPageSize;
        q.n = bad ? 0 : last - q.first;
    }
    if (q.n == 0) q.start = 0;
    return q;
}

// The same for a kernel: nothing where the sequence is the other one's.
template <int G, bool kFew>
__device__ __forceinline__ Seq own_seq(const ChunkParams& p, int s, bool& bad) {
    Seq q = load_seq(p, s, bad);
    if (p.split && (q.n <= kRows / G) != kFew) q = Seq{0, 0, 0};
    return q;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((unsigned)a + b - 1) / b); }

template <int G>
__device__ __forceinline__ int pairs_of(const Seq& q) {
    return ceil_div(q.n, 2 * kRows / G);
}

// Keys of the pair that begins at new token t0: those up to its last token.
template <int G>
__device__ __forceinline__ int keys_of(const Seq& q, int t0) {
    return q.start + (int)min((int64_t)q.n, (int64_t)t0 + 2 * kRows / G);
}

// Cost of the first m pairs, all of them whole: sum over i = 1..m of ceil((start + i T) / 128) + kPairCost, T = 256 / G tokens.
// For G > 1 the quotient is ceil((c + i) / r) with c = ceil(start / T), r = 128 / T.
template <int G, bool kFew>
__device__ __forceinline__ int64_t cost_before(const Seq& q, int m) {
    constexpr int T = 2 * kRows / G;
    if constexpr (T > kRows) {
        return (int64_t)m * (ceil_div(q.start, kRows) + kPairCost<kFew>) + (int64_t)m * (m + 1);
    } else {
        constexpr int r = kRows / T;
        const int64_t c = ceil_div(q.start, T);
        auto upto = [](int64_t x) {  // sum over i = 1..x of ceil(i / r)
            const int64_t a = x / r, b = x % r;
            return r * (a * (a + 1) / 2) + b * (a + 1);
        };
        return upto(c + m) - upto(c) + (int64_t)m * kPairCost<kFew>;
    }
}

template <int G, bool kFew>
__device__ __forceinline__ int64_t cost_of(const Seq& q) {  // of one KV head
    const int m = pairs_of<G>(q);
    return m == 0 ? 0 : cost_before<G, kFew>(q, m - 1) + kPairCost<kFew> + ceil_div(q.start + q.n, kRows);
}

// Keys of tile x (0: A, 1: B) of a pair; 0: it has no rows.
template <typename W>
__device__ __forceinline__ int tile_end(const W& w, int x, int tokens) {
    const int t = w.t0 + x * tokens, n = w.q.n;
    return t < n ? w.q.start + min(t + tokens, n) : 0;
}

// Piece of the line of cost `total` that its unit u lies in; piece i begins at i * total / pieces.
__device__ __forceinline__ int piece_of(int64_t u, int64_t total, int pieces) {
    return (int)(((u + 1) * pieces + total - 1) / total) - 1;
}

// The pool's page that holds the keys 16 lp .. of row s (for KV head h, where the row's pages are selected ones); num_pages
// where there is none.
__device__ __forceinline__ int page_of(const ChunkParams& p, int s, int h, int lp) {
    if (p.pages) {
        lp = p.pages[((int64_t)s * p.Hkv + h) * p.select + lp];
        if (lp < 0 || lp >= p.max_pages) return p.num_pages;
    }
    const int e = p.block_table[(int64_t)s * p.max_pages + lp];
    return e >= 0 && e < p.num_pages ? e : p.num_pages;
}

// ---- rows on the CUDA cores ----------------------------------------------------------------------------------------
struct Row4 {
    float x[4];
};

__device__ __forceinline__ uint2 load4(const __half* p) { return *reinterpret_cast<const uint2*>(p); }

__device__ __forceinline__ Row4 floats4(const uint2& u) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return Row4{{a.x, a.y, b.x, b.y}};
}

// The reference for a largest score. Scores of which an fp32 has no fractions are it themselves: nothing is then added to
// their rounding.
__device__ __forceinline__ float ref_for(float top) { return fabsf(top) < 16777216.f ? top - kLift : top; }

// One warp, one (token, query head): online softmax over the keys 0..pos of its sequence, 4 at a time; lane l holds dims
// 4l..4l+3. Stores dims 64 half .. + 63. Factors of the numerator stay at 2^-126 or above, which is nothing to finite values,
// and keeps infinities of V that no weight is too small for: 0 times one would be NaN.
__device__ __forceinline__ void row_attention(const ChunkParams& p, const Seq& sq, int s, int t, int hq, int half, int lane) {
    constexpr int kKeys = 4;
    constexpr float kLeast = 0x1p-126f;
    const int h = hq / (p.Hq / p.Hkv), pos = sq.start + t;
    const int64_t token = (int64_t)p.Hkv * kHeadDim;
    const int64_t at = h * kHeadDim + lane * 4;
    const Row4 q = floats4(load4(static_cast<const __half*>(p.q) + (int64_t)(sq.first + t) * p.q_stride + hq * kHeadDim + lane * 4));
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j <= pos; j += kKeys) {
        const int page = page_of(p, s, h, j / kPageSize);
        const int64_t row = ((int64_t)page * kPageSize + j % kPageSize) * token + at;
        uint2 a[kKeys], b[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            a[i] = b[i] = make_uint2(0u, 0u);
            if (page < p.num_pages && j + i <= pos) {
                a[i] = load4(static_cast<const __half*>(p.k_pool) + row + i * token);
                b[i] = load4(static_cast<const __half*>(p.v_pool) + row + i * token);
            }
        }
        float x[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const Row4 y = floats4(a[i]);
            x[i] = q.x[0] * y.x[0] + q.x[1] * y.x[1] + q.x[2] * y.x[2] + q.x[3] * y.x[3];
        }
#pragma unroll
        for (int z = 16; z > 0; z >>= 1)
#pragma unroll
            for (int i = 0; i < kKeys; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], z);
        float mn = m;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            x[i] = j + i <= pos ? x[i] * p.scale_log2 : -INFINITY;
            mn = fmaxf(mn, x[i]);
        }
        const float ref = mn == -INFINITY ? 0.f : mn, f = exp2f(m - ref);
        l *= f;
#pragma unroll
        for (int z = 0; z < 4; ++z) o[z] *= fmaxf(f, kLeast);
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
            if (j + i <= pos) {
                const float e = exp2f(x[i] - ref);
                const Row4 y = floats4(b[i]);
                l += e;
#pragma unroll
                for (int z = 0; z < 4; ++z) o[z] += fmaxf(e, kLeast) * y.x[z];
            }
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : NAN;  // NaN: a score is, or all of them are -inf
    uint2 u;
    u.x = pack_half2(o[0] * inv, o[1] * inv);
    u.y = pack_half2(o[2] * inv, o[3] * inv);
    if (lane >> 4 == half)
        *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + (int64_t)(sq.first + t) * p.out_stride + hq * kHeadDim + lane * 4) = u;
}

// One warp; rows: a bit for each of its 32 rows (row r is head h * G + r % G of new token t0 + r / G of the sequence) whose
// tensor-core result, dims 64 half .. + 63 of it in out, is not finite, redo: those among them that are wrong for
// certain. Lane l looks at dims 2l, 2l + 1. Infinities of V that the row attends to add up to an infinity, of both signs (or
// with a NaN) to a NaN, whatever their weights; a row that has other dims that are not finite is computed again.
template <int G>
__device__ __noinline__ void finish_rows(const ChunkParams& p, const Seq& sq, int s, int t0, int h, int half, uint32_t rows,
                                         uint32_t redo) {
    const int lane = threadIdx.x & 31;
    const int64_t token = (int64_t)p.Hkv * kHeadDim;
    const __half* v = static_cast<const __half*>(p.v_pool) + h * kHeadDim + half * 64 + lane * 2;
    __half2 top = __float2half2_rn(0.f), low = top, nan = top;  // of the values of the keys before `keys`
    int keys = 0;
    for (; rows; rows &= rows - 1) {  // in the order of their tokens
        const int r = __ffs(rows) - 1, pos = sq.start + t0 + r / G;
        if ((redo >> r) & 1) continue;
        while (keys <= pos) {
            const int page = page_of(p, s, h, keys / kPageSize), lim = min(pos + 1, (keys | (kPageSize - 1)) + 1);
            if (page == p.num_pages) {
                keys = lim;
                continue;
            }
            const __half* at = v + (int64_t)page * kPageSize * token;
#pragma unroll 16
            for (; keys < lim; ++keys) {
                const __half2 x = *reinterpret_cast<const __half2*>(at + (keys % kPageSize) * token);
                top = __hmax2(top, x);
                low = __hmin2(low, x);
                nan = __hmax2_nan(nan, x);
            }
        }
        const uint32_t t = *reinterpret_cast<const uint32_t*>(&top), w = *reinterpret_cast<const uint32_t*>(&low),
                       n = *reinterpret_cast<const uint32_t*>(&nan);
        uint32_t* at = reinterpret_cast<uint32_t*>(static_cast<__half*>(p.out) + (int64_t)(sq.first + t0 + r / G) * p.out_stride +
                                                   (h * G + r % G) * kHeadDim + half * 64 + lane * 2);
        uint32_t y = *at;
        bool other = false;
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
            const bool up = ((t >> i) & 0xffffu) == 0x7c00u, down = ((w >> i) & 0xffffu) == 0xfc00u;
            const bool any = ((n >> i) & 0x7fffu) > 0x7c00u;
            if (any || up || down)
                y = (y & ~(0xffffu << i)) | (any || (up && down) ? 0x7fffu : up ? 0x7c00u : 0xfc00u) << i;
            else
                other = other || ((y >> i) & 0x7c00u) == 0x7c00u;
        }
        *at = y;
        if (__any_sync(0xffffffffu, other)) redo |= 1u << r;
    }
    for (; redo; redo &= redo - 1) {
        const int r = __ffs(redo) - 1;
        row_attention(p, sq, s, t0 + r / G, h * G + r % G, half, lane);
    }
}

// ---- softmax and output rows -----------------------------------------------------------------------------------------
// What a warp of the softmax has counted: its tile's steps; works with a tile A, with a tile B; steps with keys in the second
// half, as the first half counts them; few: tiles with second parts, and tiles that went to out.
struct Counts {
    int ns, na, nb, step2, low, told;
};

__device__ __forceinline__ float scaled(float y, float f) { return y == INFINITY && f == 0.f ? 0.f : y * f; }  // NaN only where a score is

// A row's reference and sum from those of both halves of its keys, relative to the last reference (they only rise).
__device__ __forceinline__ float2 sum_of(const float2* at, bool second_half) {
    const float2 lo = at[0], hi = at[kRows];
    if (!second_half) return lo;
    const float top = fmaxf(lo.x, hi.x);
    return make_float2(top, scaled(lo.y, lo.x == top ? 1.f : fast_exp2(lo.x - top)) +
                                scaled(hi.y, hi.x == top ? 1.f : fast_exp2(hi.x - top)));
}

// A wait for another warp of the softmax that is as far as this one (done with the tile before: see o_free): warp_wait's clock would take
// registers that the rows need.
__device__ __forceinline__ bool short_wait(uint64_t* bar, uint32_t parity, const WaitCtx& ctx) {
    for (uint32_t it = 0; it < 1u << 20; ++it) {
        if (__all_sync(kAllLanes, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(kAllLanes, *ctx.abort_flag != 0)) return false;
    }
    *ctx.abort_flag = 1;
    raise_status(ctx.status, PKV_STATUS_TIMEOUT);
    return false;
}

// The rows of a tile that is alone, by the warps of both tiles: dims 64 h + 32 x .. + 31. keys: the piece's; own: this thread's row
// is one to be stored; low: it holds second parts.
template <int G>
__device__ __forceinline__ bool few_rows_out(const ChunkParams& p, uint8_t* smem, uint32_t tmem, const volatile Work& w,
                                             const WaitCtx& ctx, Counts& cnt, int keys, bool both, bool dup, bool idle) {
    using L = Layout<true>;
    Bars& bars = *reinterpret_cast<Bars*>(smem + L::bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = warp >> 3, h = (warp >> 2) & 1;
    const int lane_row = threadIdx.x & 127, row = dup ? lane_row & 63 : lane_row;
    const bool low = dup && lane_row >= 64, mine = !low && row / G < w.q.n;
    if (!warp_wait(&bars.o_full[0], cnt.na & 1, ctx) || (both && !warp_wait(&bars.o_full[1], cnt.nb & 1, ctx))) return false;
    auto have_read = [&]() {  // the next tile's products may overwrite them (A's second half says so when it is done with the tile)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (x == 1 || h == 0) mbar_arrive(&bars.o_free[0]);
            if (both) mbar_arrive(&bars.o_free[1]);
        }
    };
    const int na = cnt.na++, nb = cnt.nb;
    cnt.nb += both;
    if (idle) {
        have_read();
        return true;
    }
    tc_fence_after();
    const float2* parts = reinterpret_cast<const float2*>(smem + L::parts) + lane_row;
    float2 y = sum_of(parts + (na & 1) * 4 * kRows, keys > 64);
    float fa = 1.f, fb = 0.f;  // factors of the accumulators; of one without a key that the row attends to, nothing is taken
    bool some_a = true, some_b = false;
    if (both) {
        const float2 yb = sum_of(parts + (nb & 1) * 4 * kRows + 2 * kRows, keys - kRows > 64);
        some_a = y.y != 0.f;
        some_b = yb.y != 0.f;
        const float top = some_b && (!some_a || yb.x > y.x) ? yb.x : y.x;
        fa = y.x == top ? 1.f : fast_exp2(y.x - top);
        fb = yb.x == top ? 1.f : fast_exp2(yb.x - top);
        y = make_float2(top, (some_a ? scaled(y.y, fa) : 0.f) + (some_b ? scaled(yb.y, fb) : 0.f));
    }
    uint32_t o[32];
    const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256 + h * 64 + x * 32;
    tmem_ld32(at, o);
    if (both) {
        uint32_t ob[32];
        tmem_ld32(at + 128, ob);
        tmem_wait_ld();
        tmem_use32(o);
        tmem_use32(ob);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint((some_a ? __uint_as_float(o[i]) * fa : 0.f) + (some_b ? __uint_as_float(ob[i]) * fb : 0.f));
    } else {
        tmem_wait_ld();
        tmem_use32(o);
    }
    have_read();
    if (dup) {
        // Rows 64-127 hand over what they have, 2^-11 of the rows' values and less, in bfloat16 (17 words a row: lanes are in
        // different banks).
        uint32_t* to = reinterpret_cast<uint32_t*>(smem + L::low) + ((x * 2 + h) * 64 + row) * 17;
        uint64_t* full = &bars.low_full[x * 4 + h * 2 + (warp & 1)];
        uint64_t* empty = &bars.low_empty[x * 4 + h * 2 + (warp & 1)];
        const int n = cnt.low++;
        if (low) {
            if (!short_wait(empty, (n & 1) ^ 1, ctx)) return false;
#pragma unroll
            for (int i = 0; i < 16; ++i) to[i] = pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
            return true;
        }
        if (!short_wait(full, n & 1, ctx)) return false;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t u = to[i];
            o[2 * i] = __float_as_uint(__uint_as_float(o[2 * i]) + __uint_as_float(u << 16));
            o[2 * i + 1] = __float_as_uint(__uint_as_float(o[2 * i + 1]) + __uint_as_float(u & 0xffff0000u));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty);
    }
    const int state = w.state;
    if (state >= 0) {  // columns in fours, rows side by side
        float4* acc = reinterpret_cast<float4*>(p.acc) + ((int64_t)state * 32 + h * 16 + x * 8) * kRows + row;
        if (mine) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i * kRows] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                                             __uint_as_float(o[4 * i + 3]));
            if (h == 0 && x == 0) p.ml[(int64_t)state * kRows + row] = y;
        }
        return true;
    }
    const float inv = 1.f / y.y;
    __half2 probe = __float2half2_rn(0.f);  // stays 0 while every value is finite
    const __half2 zero = probe;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(p.out) + (int64_t)(w.q.first + row / G) * p.out_stride +
                                          (w.h * G + row % G) * kHeadDim + h * 64 + x * 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            u[e] = pack_half2(__uint_as_float(o[8 * i + 2 * e]) * inv, __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
            probe = __hfma2(*reinterpret_cast<const __half2*>(&u[e]), zero, probe);
        }
        if (mine) dst[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    // As in softmax_tile; B's warps tell A's, which finish the 64 dims of both. A's have read a word before the next tile's accumulator is
    // complete (the first half has made its weights, and the second half's arrivals are part of o_free), so no word is overwritten early.
    const bool low_sum = !(y.y >= 0.25f);
    const bool odd = __low2float(probe) != 0.f || __high2float(probe) != 0.f || low_sum;
    unsigned again = __ballot_sync(kAllLanes, mine && odd && !isnan(y.y));
    const unsigned redo = __ballot_sync(kAllLanes, low_sum);
    uint32_t* told = reinterpret_cast<uint32_t*>(smem + L::told) + h * 4 + (warp & 3);
    uint64_t* told_full = &bars.told[h * 4 + (warp & 3)];
    __syncwarp();  // finish_rows reads rows that other lanes have stored; of B's warp they are told behind its lane 0
    if (x == 1) {
        if (lane == 0) {
            *told = again;
            mbar_arrive(told_full);
        }
        __syncwarp();
        return true;
    }
    if (!short_wait(told_full, cnt.told++ & 1, ctx)) return false;
    again |= *told;
    if (again)
        finish_rows<G>(p, Seq{w.q.first, w.q.n, w.q.start}, w.s, (row & ~31) / G, w.h, h, again, redo & again);
    return true;
}

// The tile of one work. Few: the tile is alone, and its rows are worked on by both tiles' warps, which take its even and odd steps
// and the accumulators of A and B (few rows wait for K and V, and for one step's scores, weights and products after the
// other). Where it has at most 64 rows, lanes 64-127 hold the same queries again: their warps make the same weights and store
// what the rounding to fp16 left of them, so that one product takes both parts, and the two halves of the accumulators are added
// in the end. The relative error is then that of the output's rounding, 2.1e-4 (with one part 2.9e-4).
template <int G, bool kFew>
__device__ __forceinline__ bool softmax_tile(const ChunkParams& p, uint8_t* smem, uint32_t tmem, const volatile Work& w,
                                             const WaitCtx& ctx, Counts& cnt) {
    constexpr int kTokens = kRows / G, kTiles = kFew ? 1 : 2;
    using L = Layout<kFew>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Bars& bars = *reinterpret_cast<Bars*>(smem + L::bars);
    const int x = warp >> 3, h = (warp >> 2) & 1;  // tile, half of the keys (and of the output's dims)
    const int lane_row = threadIdx.x & 127;
    const bool dup = kFew && w.q.n <= kRows / 2 / G, low = dup && lane_row >= 64;
    const int row = dup ? lane_row & 63 : lane_row;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + x * 128 + h * 64;  // this half's scores, and its weights over the first 32
    const uint32_t o_at = tmem + lanes + 256 + x * 128;
    volatile float* ref_at = reinterpret_cast<volatile float*>(smem + L::ref) + x * kRows + lane_row;
    float2* parts = reinterpret_cast<float2*>(smem + L::parts) + x * 2 * kRows + lane_row;  // + buffer * 4 kRows + half * kRows
    uint64_t* settled = &bars.first_ref[x][warp & 3];
    uint64_t* second = &bars.half_done[x][warp & 3];
    volatile int* late_at = reinterpret_cast<volatile int*>(smem + L::late) + x * 4 + (warp & 3);
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = pack_f32x2(sl2, sl2);
    constexpr int kNext = kFew ? 2 * kRows : kRows;  // from one of the tile's steps to the next
    const bool both = !kFew || w.j1 - w.j0 > 1;      // B's warps have something to do
    const int skip = kFew ? x * kRows : 0;
    // Positions are counted from the tile's first key of the piece.
    const int end = tile_end(w, kFew ? 0 : x, kTokens) - w.j0 * kRows - skip;
    const int all = min(w.j1 - w.j0, ceil_div(max(end + skip, 0), kRows));
    const int steps = kFew ? (all + 1 - x) >> 1 : all;
    auto first_token = [&]() { return w.q.start - w.j0 * kRows + w.t0 + (kFew ? 0 : x * kTokens) - skip; };
    const int no = kFew && x == 1 ? cnt.nb : cnt.na;  // of this tile
    const bool idle = first_token() + (row & ~31) / G >= end;  // none of the warp's rows is one
    if (!kFew && steps == 0) {  // tile A may end before the piece begins, and B is not always there
        if (w.state >= 0 && h == 0 && first_token() + row / G < end)
            p.ml[((int64_t)w.state * kTiles + x) * kRows + row] = make_float2(-INFINITY, 0.f);
        return true;
    }
    if (idle) {
        // Nothing reads the weights and accumulators of the warp's rows: it keeps the count of arrivals.
        for (int j = 0; j < steps; ++j) {
            const int step = cnt.ns++, last = end - j * kNext - h * 64;
            if (last <= 0) continue;
            if (!warp_wait(&bars.s_full[x], step & 1, ctx)) return false;
            if (last > 64) ++cnt.step2;
            if (lane == 0) {
                if (h == 0 && j == 0) mbar_arrive(settled);
                if (h == 1) mbar_arrive(second);
                mbar_arrive(&bars.p_full[x][h]);
            }
            __syncwarp();
        }
        if constexpr (!kFew) {
            if (!warp_wait(&bars.o_full[x], no & 1, ctx)) return false;
            if (lane == 0) mbar_arrive(&bars.o_free[x]);
            __syncwarp();
            ++cnt.na;
            return true;
        }
    }
    // Keys from `masked` on are in steps with keys behind the tile's first token; the others are whole. (It may begin before the
    // piece.)
    const int masked = max(first_token(), 0) / kRows * kRows;
    const int seen = min(first_token() + row / G, end - 1) - h * 64;  // the row's last key, from the half's first on
    float ref = -INFINITY, l = 0.f;
    for (int j = 0; j < steps && !(kFew && idle); ++j) {
        const int step = cnt.ns++;
        const int last = end - j * kNext - h * 64;  // keys of this half, counted from its first
        // The tile's last step ends in the first half: the second does not wait for its scores (nothing would keep
        // the next tile's from coming before it looks, and a parity two phases on does not pass). They have come
        // when the tile's accumulator is complete, for which it waits below.
        if (last <= 0) continue;
        if (!warp_wait(&bars.s_full[x], step & 1, ctx)) return false;
        tc_fence_after();
        // Keys behind the row's token: -inf in TMEM, before anything reads the scores, so that what reads them has no form with a mask.
        if (j * kNext >= masked) {
            const int lim = seen - j * kNext;
#pragma unroll 1
            for (int c = 0; c < 2 && c * 32 < last; ++c) {
                uint32_t r[32];
                tmem_ld32(s_at + c * 32, r);
                tmem_wait_ld();
                tmem_use32(r);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (c * 32 + i > lim) r[i] = 0xff800000u;
                tmem_st32(s_at + c * 32, r);
            }
            tmem_wait_st();
        }
        auto fetch = [&](int c, uint32_t* r) {  // 32 of the row's scores
            tmem_ld32(s_at + c * 32, r);
            tmem_wait_ld();
            tmem_use32(r);
        };
        auto greatest = [&]() {
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (c * 32 < last) {
                    uint32_t r[32];
                    fetch(c, r);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        m0 = fmaxf(m0, __uint_as_float(r[i]));
                        m1 = fmaxf(m1, __uint_as_float(r[i + 1]));
                    }
                }
            }
            return fmaxf(m0, m1);
        };
        uint32_t ph[32];  // the weights, in fp16
        auto weights = [&]() {  // returns their sum
            const float nref = ref == -INFINITY ? 0.f : -ref;
            const uint64_t refx2 = pack_f32x2(nref, nref);
            uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (c * 32 < last) {
                    uint32_t r[32];
                    fetch(c, r);
                    const float* f = reinterpret_cast<const float*>(r);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float a, b;
                        unpack_f32x2(fma_f32x2(pack_f32x2(f[2 * i], f[2 * i + 1]), sl2x2, refx2), a, b);
                        a = fast_exp2(a);
                        b = fast_exp2(b);
                        if (i & 1)
                            sum1 = add_f32x2(sum1, pack_f32x2(a, b));
                        else
                            sum0 = add_f32x2(sum0, pack_f32x2(a, b));
                        uint32_t y = pack_half2(a, b);
                        if (kFew && low) {
                            const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&y));
                            y = pack_half2(a - hi.x, b - hi.y);
                        }
                        ph[c * 16 + i] = y;
                    }
                }
            }
            float a, b;
            unpack_f32x2(add_f32x2(sum0, sum1), a, b);
            return a + b;
        };
        // Scales what has been accumulated up to now (this thread's sum; the row's accumulator).
        auto scale_sum = [&](float to) {
            if (to != ref) {
                const float f = ref == -INFINITY ? 0.f : fast_exp2(ref - to);
                l = l == INFINITY && f == 0.f ? 0.f : l * f;  // NaN only where a score is
            }
        };
        auto scale_acc = [&](float f) {
            const uint64_t ff = pack_f32x2(f, f);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t t[32];
                tmem_ld32(o_at + c * 32, t);
                tmem_wait_ld();
                tmem_use32(t);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float a, b;
                    unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(t[i]), __uint_as_float(t[i + 1])), ff), a, b);
                    t[i] = __float_as_uint(a);
                    t[i + 1] = __float_as_uint(b);
                }
                tmem_st32(o_at + c * 32, t);
            }
        };
        // The reference that this half's keys ask for: above the present one by a whole number.
        auto raised = [&]() {
            const float to = ref_for(greatest() * sl2);
            return ref == -INFINITY ? to : to > ref ? ref + ceilf(to - ref) : ref;
        };
        if (j > 0) {  // the other half may have raised it in the step before
            const float r = *ref_at;
            scale_sum(r);
            ref = r;
        } else if (h == 0) {
            ref = ref_for(greatest() * sl2);
            *ref_at = ref;
            __syncwarp();
            if (lane == 0) mbar_arrive(settled);
        } else {
            if (!warp_wait(settled, no & 1, ctx)) return false;
            ref = *ref_at;
        }
        float sum = weights();
        // (A row without a finite score has no reference yet, and asks for one. One whose scores are NaN, such as those
        // of garbage behind the sequence's end, has none to ask for, and would do so in every step.)
        const bool ask = ref == -INFINITY ? !isnan(sum) : sum > kMost;
        const bool raise = (j > 0 || h == 1) && __any_sync(0xffffffffu, ask);
        if (h == 0 && raise) {
            // The second half's weights of this step are in TMEM already, unless it raises, too, after this.
            float f2 = 1.f;
            const float to = raised();
            const float f = to == ref ? 1.f : ref == -INFINITY ? 0.f : fast_exp2(ref - to);
            if (last > 64) {
                if (!warp_wait(second, cnt.step2 & 1, ctx)) return false;
                if (*late_at == 0) f2 = f;
            }
            tc_fence_after();
            if (__any_sync(0xffffffffu, f2 != 1.f)) {
                uint32_t t[32];
                tmem_ld32(s_at + 64, t);
                tmem_wait_ld();
                tmem_use32(t);
#pragma unroll
                for (int i = 0; i < 32; ++i) {  // in fp32: weights of up to 2^16 times a power of two that fp16 may not have
                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&t[i]));
                    t[i] = pack_half2(v.x * f2, v.y * f2);
                }
                tmem_st32(s_at + 64, t);
            }
            scale_sum(to);
            ref = to;
            *ref_at = ref;
            scale_acc(f);
            sum = weights();
        } else if (h == 1) {
            if (raise) {
                if (lane == 0) *late_at = 1;
                __syncwarp();
                if (lane == 0) mbar_arrive(second);
                // the first half's products must be in the accumulator before it is scaled
                if (!warp_wait(&bars.lo_done[x], step & 1, ctx)) return false;
                tc_fence_after();
                const float r = *ref_at;  // the first half may have raised it in this step
                scale_sum(r);
                ref = r;
                const float to = raised();
                const float f = to == ref ? 1.f : ref == -INFINITY ? 0.f : fast_exp2(ref - to);
                scale_sum(to);
                ref = to;
                *ref_at = ref;
                scale_acc(f);
                sum = weights();
            } else if (lane == 0) {
                *late_at = 0;
            }
        }
        if (last > 64) ++cnt.step2;
        l += sum;
        parts[(no & 1) * 4 * kRows + h * kRows] = make_float2(ref, l);
        tmem_st32(s_at, ph);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (h == 1 && !raise) mbar_arrive(second);  // before the one that lets the first half's next step begin
            mbar_arrive(&bars.p_full[x][h]);
        }
    }
    if constexpr (kFew) return few_rows_out<G>(p, smem, tmem, w, ctx, cnt, end + skip, both, dup, idle);
    if (!warp_wait(&bars.o_full[x], no & 1, ctx)) return false;
    tc_fence_after();
    const float2 y = sum_of(parts + (no & 1) * 4 * kRows, end > 64);
    const float total = y.y;
    auto fetch_o = [&](int c, uint32_t* o) {  // 32 of this half's dims
        tmem_ld32(o_at + h * 64 + c * 32, o);
        tmem_wait_ld();
        tmem_use32(o);
        if (c == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.o_free[x]);  // the next tile's products may overwrite it
        }
    };
    const bool mine = first_token() + row / G < end;
    const int state = w.state;
    if (state >= 0) {  // columns in fours, rows side by side
        float4* acc = reinterpret_cast<float4*>(p.acc) + (((int64_t)state * kTiles + x) * 32 + h * 16) * kRows + row;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t o[32];
            fetch_o(c, o);
            if (mine) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[(c * 8 + i) * kRows] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                           __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
            }
        }
        if (h == 0 && mine) p.ml[((int64_t)state * kTiles + x) * kRows + row] = y;
        ++cnt.na;
        return true;
    }
    const float inv = 1.f / total;
    __half2 probe = __float2half2_rn(0.f);  // stays 0 while every value is finite
    const __half2 zero = probe;
    // Four lanes exchange 16-byte pieces of their rows, so that they store 64 consecutive bytes of one row at a time
    // (16 bytes of 32 rows an instruction took 1.7 us a tile).
    const int q4 = lane & 3;
    __half* dst[4];
    bool in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (row & ~3) + i, t = w.t0 + x * kTokens + r / G;
        in[i] = first_token() + r / G < end;
        dst[i] = static_cast<__half*>(p.out) + (int64_t)(w.q.first + t) * p.out_stride + (w.h * G + r % G) * kHeadDim +
                 h * 64 + q4 * 8;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t o[32], y[4][4];
        fetch_o(c, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float a = __uint_as_float(o[2 * i]) * inv, b = __uint_as_float(o[2 * i + 1]) * inv;
            const uint32_t u = pack_half2(a, b);
            probe = __hfma2(*reinterpret_cast<const __half2*>(&u), zero, probe);
            y[i >> 2][i & 3] = u;
        }
#pragma unroll
        for (int s = 1; s < 4; s <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!(i & s))
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, q4 & s ? y[i][e] : y[i + s][e], s);
                        (q4 & s ? y[i][e] : y[i + s][e]) = got;
                    }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (in[i]) *reinterpret_cast<uint4*>(dst[i] + c * 32) = make_uint4(y[i][0], y[i][1], y[i][2], y[i][3]);
    }
    ++cnt.na;
    // The largest weight is 2^kLift, or half of that where the reference was raised, and next to scores that are it
    // themselves 1, or above 1/2.
    const bool low_sum = !(total >= 0.25f);
    const bool odd = __low2float(probe) != 0.f || __high2float(probe) != 0.f || low_sum;
    const unsigned again = __ballot_sync(0xffffffffu, mine && odd && !isnan(total));
    if (again) {
        const unsigned redo = __ballot_sync(0xffffffffu, low_sum) & again;
        __syncwarp();  // the rows were stored by other lanes
        finish_rows<G>(p, Seq{w.q.first, w.q.n, w.q.start}, w.s, w.t0 + x * kTokens + (row & ~31) / G, w.h, h, again, redo);
    }
    return true;
}

// ---- the tensor-core kernel ---------------------------------------------------------------------------------------
template <int G, bool kFew>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ Params prm) {
    constexpr int kTokens = kRows / G;  // tokens of a tile
    using L = Layout<kFew>;
    constexpr int kStages = L::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const ChunkParams& p = prm.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    Bars& bars = *reinterpret_cast<Bars*>(smem + L::bars);
    const Work* work = reinterpret_cast<const Work*>(smem + L::work);  // [2]
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::misc);
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + L::misc + 4);
    int64_t* scan = reinterpret_cast<int64_t*>(smem + L::scan);
    int64_t* begin_off = reinterpret_cast<int64_t*>(smem + L::begin);
    int32_t* begin_seq = reinterpret_cast<int32_t*>(smem + L::begin + 8);
    const WaitCtx ctx{abort_flag, &p.hdr->status, p.wait_ns};

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.kv_full[i], 1);
            mbar_init(&bars.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.w_full[i], 1);
            mbar_init(&bars.w_empty[i], kSoftmax / 32 + 3);  // and warps 16, 17, 19
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.q_empty[i], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i][0], 4);  // one arrival a warp
            mbar_init(&bars.p_full[i][1], 4);
            mbar_init(&bars.o_full[i], 1);
            mbar_init(&bars.lo_done[i], 1);
            mbar_init(&bars.o_free[i], kFew ? 16 : 8);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&bars.first_ref[0][i], 1);
            mbar_init(&bars.half_done[0][i], 1);
        }
        mbar_init(&bars.tail_full, 1);
        mbar_init(&bars.drain, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (kFew && threadIdx.x >= 32 && threadIdx.x < 40) {
        mbar_init(&bars.low_full[threadIdx.x - 32], 1);
        mbar_init(&bars.low_empty[threadIdx.x - 32], 1);
        mbar_init(&bars.told[threadIdx.x - 32], 1);
    }
    // Everything before this kernel on the stream has completed, and what comes behind it may begin to begin. (Not so the second of
    // two kernels: begun in the gaps of the first, 30 sequences of 64 tokens behind 1000 took 74 us, 66 one behind the other.)
    grid_dependency_wait();
    if (!(kFew && p.split)) grid_launch_dependents();
    // The line: up to 32 sequences are scanned by the warp that walks the piece, a lane each. Of more, every thread sums a run
    // (the first one's bounds are on their way while the barriers are set up), the CTA scans the sums, and the thread whose
    // run holds the piece's first unit finds its sequence.
    const bool few = p.num_seqs <= 32;
    if (few && p.split) {  // nothing for this kernel: every warp sees it
        bool b = false;
        const Seq q = lane < p.num_seqs ? own_seq<G, kFew>(p, lane, b) : Seq{0, 0, 0};
        if (!__any_sync(0xffffffffu, q.n > 0)) {
            if (b && warp == 0 && blockIdx.x == 0) raise_status(ctx.status, PKV_STATUS_BAD_LEN);
            if (threadIdx.x == 0) static_cast<Merge*>(p.merges)[blockIdx.x] = Merge{};
            return;
        }
    }
    const int per = few ? 1 : ceil_div(p.num_seqs, kThreads);
    const int self = few ? (warp == 18 ? lane : p.num_seqs) : (int)threadIdx.x * per;
    const int s0 = min(p.num_seqs, self), s1 = min(p.num_seqs, s0 + per);
    bool bad = false;
    Seq sq0{0, 0, 0};
    if (s0 < s1) sq0 = own_seq<G, kFew>(p, s0, bad);
    if (few && warp == 16) tmem_alloc(tmem_at, 512);
    int64_t mine = s0 < s1 ? cost_of<G, kFew>(sq0) : 0;
    for (int s = s0 + 1; s < s1; ++s) {
        bool b;
        mine += cost_of<G, kFew>(own_seq<G, kFew>(p, s, b));
        bad |= b;
    }
    if (bad && blockIdx.x == 0) raise_status(ctx.status, PKV_STATUS_BAD_LEN);
    const int head_groups = p.Hkv / p.lanes, group = blockIdx.x / p.lanes;
    mine *= head_groups;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t before = incl - mine, total = 0;
    for (int i = few ? 18 : 0; i < (few ? 19 : kThreads / 32); ++i) {
        if (i < warp) before += scan[i];
        total += scan[i];
    }
    const int pieces = (int)min((int64_t)(gridDim.x / p.lanes), (total + kMinCost - 1) / kMinCost);
    const int64_t lo = group < pieces ? group * total / pieces : 0, hi = group < pieces ? (group + 1) * total / pieces : 0;
    if (!few) {
        if (total == 0 && p.split) {  // nothing for this kernel
            if (threadIdx.x == 0) static_cast<Merge*>(p.merges)[blockIdx.x] = Merge{};
            return;
        }
        if (warp == 16) tmem_alloc(tmem_at, 512);
        if (lo < hi && before <= lo && lo < before + mine) {
            int64_t at = before;
            for (int s = s0; s < s1; ++s) {
                bool b;
                const int64_t n = cost_of<G, kFew>(s == s0 ? sq0 : own_seq<G, kFew>(p, s, b)) * head_groups;
                if (lo < at + n) {
                    *begin_seq = s;
                    *begin_off = lo - at;
                    break;
                }
                at += n;
            }
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    const uint32_t tmem = *tmem_at;
    int oldest = -1;  // of an odd number of stages: ring position of a copy that may be in flight after a wait that ran out
    if (p.seq_lens) {  // rows without a token get 0
        for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x) {
            bool b;
            if (load_seq(p, s, b).n == 0)
                for (int i = threadIdx.x; i < p.Hq * 16; i += kThreads)
                    reinterpret_cast<uint4*>(static_cast<__half*>(p.out) + (int64_t)s * p.out_stride)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }

    if (warp >= kSoftmax / 32) {
        regs_shrink<kOtherRegs>();
        if (warp == 18) {
            // ---------------------------------------------------------------------- the piece, pair after pair
            auto publish = [&](int k, const Work& w) {
                if (!warp_wait(&bars.w_empty[k & 1], ((k >> 1) & 1) ^ 1, ctx)) return false;
                if (lane == 0) {
                    const_cast<Work*>(work)[k & 1] = w;
                    mbar_arrive(&bars.w_full[k & 1]);
                }
                __syncwarp();
                return true;
            };
            // Where a cut at `u` of a pair of cost `len` goes: to the pair's beginning or end where it is next to one (or where pieces
            // are no more than a short pair).
            const int near = total <= (int64_t)kWhole * pieces ? kWhole : 0;
            auto snap = [&](int u, int len) {
                if (len <= near) return 2 * u <= len ? 0 : len;
                return u <= kPairCost<kFew> ? 0 : u >= len - 1 ? len : u;
            };
            Merge merge{};
            int k = 0;
            bool ok = true;
            if (lo < hi) {
                bool b;
                int s;
                int64_t rest;
                auto take = [&](int i) {  // sequence i
                    if (!few) return own_seq<G, kFew>(p, i, b);
                    return Seq{__shfl_sync(0xffffffffu, sq0.first, i), __shfl_sync(0xffffffffu, sq0.n, i),
                               __shfl_sync(0xffffffffu, sq0.start, i)};
                };
                if (few) {
                    s = __ffs(__ballot_sync(0xffffffffu, before <= lo && lo < before + mine)) - 1;
                    rest = lo - __shfl_sync(0xffffffffu, before, s);
                } else {
                    s = *begin_seq;
                    rest = *begin_off;
                }
                Seq q = take(s);
                int hg = 0;
                if (head_groups > 1) {
                    const int64_t of_head = cost_of<G, kFew>(q);
                    hg = (int)(rest / of_head);
                    rest -= hg * of_head;
                }
                int left = 0, right = pairs_of<G>(q) - 1;  // the last pair that begins at or before `rest`
                while (left < right) {
                    const int mid = (left + right + 1) >> 1;
                    if (cost_before<G, kFew>(q, mid) <= rest)
                        left = mid;
                    else
                        right = mid - 1;
                }
                int pair = left, u = (int)(rest - cost_before<G, kFew>(q, pair));
                bool first = true;
                // The last steps of the first pair: where about a whole pair follows they are kept for the end. CTAs that begin with
                // whole pairs read a head's keys at the same time, once from HBM for all of them where a context does not fit L2 (4096
                // tokens behind 28672: 1.46-1.48 ms in order, 1.38-1.39 so).
                Work tail;
                tail.h = -1;
                for (int64_t at = lo - u; ok; first = false) {  // where the pair begins
                    Work w;
                    w.q = q;
                    w.s = s;
                    w.t0 = pair * 2 * kTokens;
                    w.h = hg * p.lanes + (int)(blockIdx.x % p.lanes);
                    const int steps = ceil_div(keys_of<G>(q, w.t0), kRows), len = steps + kPairCost<kFew>;
                    if (first) u = snap(u, len);
                    const int end = at + len <= hi ? len : snap((int)(hi - at), len);
                    if (end > u) {
                        w.j0 = max(0, u - kPairCost<kFew>);  // (a cut leaves the pair's own cost to its first piece)
                        w.j1 = end - kPairCost<kFew>;
                        const bool whole = w.j0 == 0 && w.j1 == steps;
                        w.state = whole ? -1 : 2 * (int)blockIdx.x + (w.j0 == 0);
                        if (!whole && w.j0 == 0) {
                            int e = piece_of(at + len - 1, total, pieces);
                            while (e > group && snap((int)((int64_t)e * total / pieces - at), len) == len) --e;
                            merge = Merge{q, s, w.t0, w.h, e - group + 1, 0};
                        }
                        if (!kFew && w.j0 > 0 && hi - (at + len) >= len)
                            tail = w;
                        else
                            ok = publish(k++, w);
                    }
                    at += len;
                    u = 0;
                    if (at >= hi) break;
                    if (++pair == pairs_of<G>(q)) {
                        pair = 0;
                        if (++hg == head_groups) {
                            hg = 0;
                            do {
                                if (++s >= p.num_seqs) break;
                                q = take(s);
                            } while (q.n == 0);
                            if (s >= p.num_seqs) break;  // (only where the lengths change under the kernel)
                        }
                    }
                }
                if (!kFew && ok && tail.h >= 0) ok = publish(k++, tail);
            }
            if (ok) {
                Work w{};
                w.h = -1;
                publish(k, w);
            }
            if (lane == 0) static_cast<Merge*>(p.merges)[blockIdx.x] = merge;
        } else if (warp == 17 || warp == 19) {
            // ----------------------------------------------- copies: of queries and K (warp 17), of V (warp 19)
            // (A page is four boxes, and a warp issues the boxes of its lanes one after the other: one warp for all of them leaves
            // the tensor core waiting.)
            const bool of_v = warp == 19;
            const CUtensorMap* map = of_v ? &prm.v : &prm.k;
            if (lane == 0) {
                prefetch_tensormap(map);
                if (!of_v) prefetch_tensormap(&prm.q);
                if (!of_v) prefetch_tensormap(&prm.q64);
            }
            uint64_t ordinary;
            asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(ordinary));
            const uint64_t stream = policy_evict_first();
            int seq = of_v ? 1 : 0, nq[2] = {0, 0}, nc = 0;  // ring position; tiles of queries; tiles that were cleared
            const int seq0 = seq;
            bool stop = false;
            for (int k = 0; !stop; ++k) {
                if (!warp_wait(&bars.w_full[k & 1], (k >> 1) & 1, ctx)) break;
                const Work w = work[k & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.w_empty[k & 1]);
                if (w.h < 0) break;
                const int end = max(tile_end(w, 0, kTokens), tile_end(w, 1, kTokens));
                const int npages = ceil_div(end, kPageSize);
                auto entries = [&](int lp) { return lp < npages ? page_of(p, w.s, w.h, lp) : 0; };
                int next = entries(w.j0 * kStepPages + lane), ent = 0;
                auto load_q = [&](int x) {
                    if (tile_end(w, x, kTokens) <= w.j0 * kRows) return true;
                    if (!warp_wait(&bars.q_empty[x], (nq[x] & 1) ^ 1, ctx)) return false;
                    if (lane == 0) {
                        uint8_t* dst = smem + L::q + x * kTileBytes;
                        const bool dup = kFew && w.q.n <= kRows / 2 / G;
                        mbar_arrive_expect_tx(&bars.q_full[x], kTileBytes);
                        for (int b = 0; b < 2; ++b)
                            for (int i = 0; i <= dup; ++i)
                                tma_load_3d(dst + b * kBoxBytes + i * kBoxBytes / 2, dup ? &prm.q64 : &prm.q, b * 64, w.h * G,
                                            w.q.first + w.t0 + x * kTokens, &bars.q_full[x], stream);
                    }
                    __syncwarp();
                    ++nq[x];
                    return true;
                };
                for (int j = w.j0; j < w.j1; ++j) {
                    if (((j - w.j0) & 3) == 0) {  // 32 entries serve four steps; the next 32 are on their way meanwhile
                        ent = next;
                        if (ent == p.num_pages) raise_status(ctx.status, PKV_STATUS_BAD_PAGE);
                        if (j + 4 < w.j1) next = entries((j + 4) * kStepPages + lane);
                    }
                    stop = !of_v && j == w.j0 && !load_q(0);
                    const int st = seq % kStages, n = min(kStepPages, npages - j * kStepPages);
                    stop = stop || !warp_wait(&bars.kv_empty[st], ((seq / kStages) & 1) ^ 1, ctx);
                    if (stop) break;
                    // The products' last step of 16 keys reads rows behind the pair's last key, which may hold anything: in V they are
                    // cleared before the tile counts as loaded.
                    const bool tail = of_v && (j + 1) * kRows >= end && (end & 15);
                    uint64_t* bar = tail ? &bars.tail_full : &bars.kv_full[st];
                    uint8_t* dst = smem + L::ring + st * kTileBytes;
                    // lane 2 i + half: half of the dims of the step's page i
                    const int page = __shfl_sync(0xffffffffu, ent, ((j - w.j0) & 3) * kStepPages + ((lane >> 1) & 7));
                    if (lane == 0) mbar_arrive_expect_tx(bar, n * 2 * kPageBox);
                    __syncwarp();
                    if (lane < 2 * n)
                        tma_load_3d(dst + (lane & 1) * kBoxBytes + (lane >> 1) * kPageBox, map, (lane & 1) * 64, w.h, page * kPageSize,
                                    bar, ordinary);
                    __syncwarp();
                    seq += 2;
                    if (tail) {
                        nc += 1;
                        stop = !warp_wait(&bars.tail_full, (nc - 1) & 1, ctx);
                        if (stop) break;
                        const int first = end - j * kRows, last = (first + 15) & ~15;
                        for (int i = first * 16 + lane; i < last * 16; i += 32)
                            *reinterpret_cast<uint4*>(dst + ((i >> 3) & 1) * kBoxBytes + (i >> 4) * 128 + (i & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars.kv_full[st]);
                    }
                    stop = !of_v && j == w.j0 && !load_q(1);
                    if (stop) break;
                }
            }
            // every copy that this warp issued lands before the CTA may end
            if (nc > 0) warp_drain(&bars.tail_full, (nc - 1) & 1);
            for (int j = max(seq0, seq - kStages / 2 * 2); j < seq; j += 2) warp_drain(&bars.kv_full[j % kStages], (j / kStages) & 1);
            if (kStages % 2 && seq - (kStages + 1) >= seq0) oldest = seq - (kStages + 1);
            for (int x = 0; x < 2; ++x)
                if (nq[x] > 0) warp_drain(&bars.q_full[x], (nq[x] - 1) & 1);
        } else if (warp == 16) {
            // ------------------------------------------------------------------------- matrix instructions
            if (elect_one()) {  // one thread waits for and issues everything
                int kv = 0;                        // ring position of the next K tile of the current work
                int nq[2] = {0, 0}, no[2] = {0, 0};  // tiles begun; accumulators begun
                int np[2][2] = {{0, 0}, {0, 0}};     // halves of steps taken
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    if (!thread_wait(&bars.w_full[k & 1], (k >> 1) & 1, ctx)) break;
                    const Work w = work[k & 1];
                    mbar_arrive(&bars.w_empty[k & 1]);
                    if (w.h < 0) break;
                    // keys from the piece's first on, up to its last
                    const int steps = w.j1 - w.j0, most = steps * kRows;
                    const int end0 = min(tile_end(w, 0, kTokens) - w.j0 * kRows, most);
                    const int end1 = min(tile_end(w, 1, kTokens) - w.j0 * kRows, most);
                    // ring positions: K_j at kv + 2j, V_j one behind it
                    const uint32_t ring = smem_addr(smem + L::ring);
                    auto stage_addr = [&](int pos) { return ring + (pos % kStages) * kTileBytes; };
                    auto wait_stage = [&](int pos) { return thread_wait(&bars.kv_full[pos % kStages], (pos / kStages) & 1, ctx); };
                    auto release = [&](int pos) { mma_commit(&bars.kv_empty[pos % kStages]); };
                    constexpr uint32_t idesc_v = mma_idesc(kHeadDim, true);
                    if constexpr (!kFew) {
                        // keys of the piece's step j that tile x needs (0: none)
                        auto keys = [&](int x, int j) { return max(0, min(kRows, (x ? end1 : end0) - j * kRows)); };
                        auto scores = [&](int x, int j) {  // S_x(j) = Q_x K_j^T
                            const int n = (keys(x, j) + 15) & ~15;
                            if (n == 0) return;
                            const uint64_t q = smem_desc_k_major(smem_addr(smem + L::q + x * kTileBytes));
                            const uint64_t kd = smem_desc_k_major(stage_addr(kv + 2 * j));
                            const uint32_t idesc = mma_idesc(n, false);
                            const bool last = keys(x, j + 1) == 0;  // the tile's last use of its queries
                            mma_ss_128<kBoxBytes / 16>(tmem + x * 128, q, kd, idesc);
                            mma_commit(&bars.s_full[x]);
                            if (last) mma_commit(&bars.q_empty[x]);
                        };
                        auto values = [&](int x, int j) {  // O_x += P_x(j) V_j
                            const int n = (keys(x, j) + 15) >> 4;
                            if (n == 0) return true;
                            const uint64_t v = smem_desc_mn_major(stage_addr(kv + 2 * j + 1), kBoxBytes);
                            const uint32_t o = tmem + 256 + x * 128, pw = tmem + x * 128;
                            const bool last = keys(x, j + 1) == 0;
                            if (j == 0) {  // the previous tile's rows have been read
                                if (!thread_wait(&bars.o_free[x], (no[x] & 1) ^ 1, ctx)) return false;
                                ++no[x];
                            }
#pragma unroll
                            for (int half = 0; half < 2; ++half) {  // 64 keys each
                                const int c = min(4, n - 4 * half);  // steps of 16 keys
                                if (c <= 0) break;
                                if (!thread_wait(&bars.p_full[x][half], np[x][half] & 1, ctx)) return false;
                                ++np[x][half];
                                tc_fence_after();
                                if (c == 4)
                                    mma_ts_64(o, pw + 64 * half, v + 512 * half, idesc_v, j > 0 || half > 0);
                                else
                                    for (int i = 0; i < c; ++i)
                                        mma_ts(o, pw + 64 * half + 8 * i, v + 512 * half + 128 * i, idesc_v, j > 0 || half > 0 || i > 0);
                                if (half == 0) mma_commit(&bars.lo_done[x]);
                                if (last && n - 4 * half <= 4) mma_commit(&bars.o_full[x]);
                            }
                            return true;
                        };
                        ok = wait_stage(kv);
                        for (int x = 0; x < 2 && ok; ++x) {
                            if (keys(x, 0) == 0) continue;
                            ok = thread_wait(&bars.q_full[x], nq[x] & 1, ctx);
                            ++nq[x];
                            tc_fence_after();
                            if (ok) scores(x, 0);
                        }
                        if (!ok) break;
                        release(kv);
                        for (int j = 0; j < steps && ok; ++j) {
                            ok = wait_stage(kv + 2 * j + 1) && values(0, j);
                            if (ok && j + 1 < steps) {
                                ok = wait_stage(kv + 2 * j + 2);
                                if (ok) scores(0, j + 1);
                            }
                            ok = ok && values(1, j);
                            if (!ok) break;
                            release(kv + 2 * j + 1);
                            if (j + 1 < steps) {
                                scores(1, j + 1);
                                release(kv + 2 * j + 2);
                            }
                        }
                    } else {
                        // One tile: its even steps are A's, its odd ones B's.
                        ok = thread_wait(&bars.q_full[0], nq[0] & 1, ctx);
                        ++nq[0];
                        tc_fence_after();
                        const uint64_t q = smem_desc_k_major(smem_addr(smem + L::q));
                        for (int i = 0; i < steps + 2 && ok; ++i) {  // values of step i - 2, scores of step i
                            const int x = i & 1, j = i - 2;
                            if (j >= 0) {
                                const int n = (min(kRows, end0 - j * kRows) + 15) >> 4;
                                ok = wait_stage(kv + 2 * j + 1);
                                if (ok && j < 2) {
                                    ok = thread_wait(&bars.o_free[x], (no[x] & 1) ^ 1, ctx);
                                    ++no[x];
                                }
                                const uint64_t v = smem_desc_mn_major(stage_addr(kv + 2 * j + 1), kBoxBytes);
                                for (int half = 0; half < 2 && 4 * half < n && ok; ++half) {
                                    ok = thread_wait(&bars.p_full[x][half], np[x][half] & 1, ctx);
                                    ++np[x][half];
                                    tc_fence_after();
                                    const uint32_t o = tmem + 256 + x * 128, pw = tmem + x * 128 + 64 * half;
                                    const int c = min(4, n - 4 * half);
                                    if (c == 4)
                                        mma_ts_64(o, pw, v + 512 * half, idesc_v, j > 1 || half > 0);
                                    else
                                        for (int k16 = 0; k16 < c; ++k16)
                                            mma_ts(o, pw + 8 * k16, v + 512 * half + 128 * k16, idesc_v, j > 1 || half > 0 || k16 > 0);
                                    if (half == 0) mma_commit(&bars.lo_done[x]);
                                    if (j + 2 >= steps && n - 4 * half <= 4) mma_commit(&bars.o_full[x]);
                                }
                                if (!ok) break;
                                release(kv + 2 * j + 1);
                            }
                            if (i < steps) {
                                ok = wait_stage(kv + 2 * i);
                                const uint64_t kd = smem_desc_k_major(stage_addr(kv + 2 * i));
                                mma_ss_128<kBoxBytes / 16>(tmem + x * 128, q, kd, mma_idesc((min(kRows, end0 - i * kRows) + 15) & ~15, false));
                                mma_commit(&bars.s_full[x]);
                                release(kv + 2 * i);
                                if (i + 1 == steps) mma_commit(&bars.q_empty[0]);
                            }
                        }
                    }
                    kv += 2 * steps;
                }
                mma_commit(&bars.drain);
            }
            __syncwarp();
            // every matrix instruction has completed before the TMEM is freed and the CTA ends
            warp_drain(&bars.drain, 0);
        }
    } else {
        // ---------------------------------------------------------------------------- softmax and output rows
        regs_grow<kSoftmaxRegs>();
        Counts counts{};
        for (int k = 0;; ++k) {
            // The slot is kept while it is worked on: what a step does not need is not kept in registers.
            __syncwarp();
            if (k > 0 && lane == 0) {
                mbar_arrive(&bars.w_empty[(k - 1) & 1]);
                // A tile of 64 keys or fewer takes no weights from A's second half: without this its accumulator would be complete,
                // and B's warps tell of its rows, while A's have not read what they told of the tile before, or finish its rows.
                if (kFew && warp >> 2 == 1) mbar_arrive(&bars.o_free[0]);
            }
            if (!warp_wait(&bars.w_full[k & 1], (k >> 1) & 1, ctx)) break;
            const volatile Work& w = reinterpret_cast<const volatile Work*>(work)[k & 1];
            if (w.h < 0) break;
            if (!softmax_tile<G, kFew>(p, smem, tmem, w, ctx, counts)) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (kStages % 2 && *abort_flag && oldest >= 0) warp_drain(&bars.kv_full[oldest % kStages], (oldest / kStages) & 1);
    if (warp == 16) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

// ---- adding up the states of pairs that were cut ---------------------------------------------------------------------
// A block: 32 rows of the pair that began in CTA blockIdx.x and went on in the pieces behind it. Warp w takes dims 16 w ..
// + 15. Where few rows are valid, the lanes of the others take every 2nd, 4th, .. state of them, and the sums are added
// over the lanes.
constexpr int kMergeWarps = 8;

template <int G>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const ChunkParams first, const ChunkParams second) {
    constexpr int kTokens = kRows / G;
    __shared__ uint32_t s_bad[2], s_redo;  // rows with a value that is not finite, by half of the dims; wrong for certain
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();  // (and no dependents launched: the next step's kernels in the way, 32 sparse rows take 127 us, 117 without)
    const bool is_first = (int)blockIdx.x < first.grid;
    const ChunkParams& p = is_first ? first : second;
    const int cta = blockIdx.x - (is_first ? 0 : first.grid), tiles = p.tiles;
    const Merge m = static_cast<const Merge*>(p.merges)[cta];
    const int r0 = (int)blockIdx.y * 32;  // of the pair's 256 rows
    const int valid = min(32, (min(m.q.n, m.t0 + 2 * kTokens) - m.t0) * G - r0);
    if (m.pieces <= 1 || valid <= 0) return;
    if (threadIdx.x < 2) s_bad[threadIdx.x] = 0;
    if (threadIdx.x == 2) s_redo = 0;
    __syncthreads();
    int span = 1;  // lanes a row takes: a power of two
    while (32 / (2 * span) >= valid) span *= 2;
    const int rows = 32 / span, row = r0 + lane % rows, turn = lane / rows;
    const float2* ml = p.ml + row;
    const float4* acc = reinterpret_cast<const float4*>(p.acc) + ((row >> 7) * 32 + warp * 4) * kRows + (row & 127);
    auto slot = [&](int i) { return (int64_t)(i == 0 ? 2 * cta + 1 : 2 * (cta + i * p.lanes)); };
    // Four states at a time, all of their loads in flight together.
    constexpr int kBatch = 4;
    float top = -INFINITY, total = 0.f;
    float4 sum[4] = {};
    bool nan = false;
    auto scaled = [](float l, float f) { return l == INFINITY && f == 0.f ? 0.f : l * f; };  // NaN only where a score is
    auto rescale = [&](float to) {
        const float f = top == to ? 1.f : fast_exp2(top - to);
        top = to;
        total = scaled(total, f);
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[c] = make_float4(sum[c].x * f, sum[c].y * f, sum[c].z * f, sum[c].w * f);
    };
    for (int i0 = turn; i0 < m.pieces; i0 += kBatch * span) {
        float2 x[kBatch];
        float4 a[kBatch][4];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int i = i0 + e * span;
            x[e] = make_float2(0.f, 0.f);
            if (i < m.pieces) {
                x[e] = __ldcg(ml + slot(i) * tiles * kRows);
#pragma unroll
                for (int c = 0; c < 4; ++c) a[e][c] = __ldcg(acc + slot(i) * tiles * 32 * kRows + c * kRows);
            }
        }
        float to = top;
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            nan |= isnan(x[e].y);
            if (x[e].y > 0.f) to = fmaxf(to, x[e].x);
        }
        rescale(to);
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
            if (x[e].y > 0.f) {  // 0: keys behind the row's token alone
                const float f = x[e].x == top ? 1.f : fast_exp2(x[e].x - top);
                total += scaled(x[e].y, f);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    sum[c] = make_float4(sum[c].x + a[e][c].x * f, sum[c].y + a[e][c].y * f, sum[c].z + a[e][c].z * f,
                                         sum[c].w + a[e][c].w * f);
            }
    }
    float to = top;
    for (int o = rows; o < 32; o *= 2) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
    rescale(to);
    if (nan) total = NAN;
    for (int o = rows; o < 32; o *= 2) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            sum[c].x += __shfl_xor_sync(0xffffffffu, sum[c].x, o);
            sum[c].y += __shfl_xor_sync(0xffffffffu, sum[c].y, o);
            sum[c].z += __shfl_xor_sync(0xffffffffu, sum[c].z, o);
            sum[c].w += __shfl_xor_sync(0xffffffffu, sum[c].w, o);
        }
    }
    const int t = m.t0 + row / G;
    const bool mine = turn == 0 && row - r0 < valid;
    const float inv = 1.f / total;
    uint32_t y[8];
    __half2 probe = __float2half2_rn(0.f);  // stays 0 while every value is finite
    const __half2 zero = probe;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        y[2 * c] = pack_half2(sum[c].x * inv, sum[c].y * inv);
        y[2 * c + 1] = pack_half2(sum[c].z * inv, sum[c].w * inv);
        probe = __hfma2(*reinterpret_cast<const __half2*>(&y[2 * c]), zero, probe);
        probe = __hfma2(*reinterpret_cast<const __half2*>(&y[2 * c + 1]), zero, probe);
    }
    if (mine) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(p.out) + (int64_t)(m.q.first + t) * p.out_stride +
                                              (m.h * G + row % G) * kHeadDim + warp * 16);
        dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
        dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
        const bool low_sum = !(total >= 0.25f);
        if ((__low2float(probe) != 0.f || __high2float(probe) != 0.f || low_sum) && !isnan(total)) {
            atomicOr(&s_bad[warp >> 2], 1u << (row - r0));
            if (low_sum) atomicOr(&s_redo, 1u << (row - r0));
        }
    }
    __syncthreads();
    if (warp < 2 && s_bad[warp]) finish_rows<G>(p, m.q, m.s, m.t0 + r0 / G, m.h, warp, s_bad[warp], s_redo & s_bad[warp]);
}

template <int G, bool kFew>
int launch_one(const Params& prm, cudaStream_t stream) {
    static int configured_mask = 0;  // one bit per device ordinal (< 32)
    constexpr int smem = Layout<kFew>::bytes;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 32 || !(__atomic_load_n(&configured_mask, __ATOMIC_ACQUIRE) & (1 << dev))) {
        cudaFuncAttributes a{};
        cudaError_t e = cudaFuncGetAttributes(&a, chunk_kernel<G, kFew>);
        if (e != cudaSuccess) return e;
        // the warpgroups' register shares come out of what the launch gives them
        if (a.numRegs * kThreads < kSoftmax * kSoftmaxRegs + 128 * kOtherRegs) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(chunk_kernel<G, kFew>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 32) __atomic_fetch_or(&configured_mask, 1 << dev, __ATOMIC_ACQ_REL);
    }
    return launch_behind(chunk_kernel<G, kFew>, dim3((unsigned)prm.p.grid), dim3(kThreads), smem, stream, prm);
}

// Sequences of one tile of new tokens go to one kernel, those of more to another behind it; both where the host cannot tell (the
// lengths are on the device). A kernel that has no sequences ends at once: 5 us.
template <int G>
int launch(const Params& prm, const Params& prm_few, cudaStream_t stream) {
    const ChunkParams& p = prm.p;
    const bool only_few = p.seq_lens || p.total_tokens <= kRows / G, only_many = !only_few && p.num_seqs == 1;
    int e = cudaSuccess;
    Params x = prm, y = prm_few;
    x.p.split = y.p.split = !only_few && !only_many;
    if (!only_many) e = launch_one<G, true>(y, stream);
    if (e == cudaSuccess && !only_few) e = launch_one<G, false>(x, stream);
    if (e != cudaSuccess) return e;
    // 32 rows a block, of the most that a pair may have
    const int64_t most = only_few ? kRows : 2 * kRows, rows = p.seq_lens ? G : std::min<int64_t>(most, (int64_t)p.total_tokens * G);
    const dim3 grid((unsigned)(x.p.split ? 2 * p.grid : p.grid), (unsigned)((rows + 31) / 32));
    return launch_behind(merge_kernel<G>, grid, dim3(kMergeWarps * 32), 0, stream, only_few ? y.p : x.p, y.p);
}

// KV heads whose CTAs read the same pages at the same time: of the divisors of Hkv up to 8 (a token's K of 8 heads are 2 KB
// of a page) the one that leaves the fewest SMs without a piece, the largest of these.
int head_lanes(int hkv, int num_sms) {
    int best = 1;
    for (int d = 2; d <= 8; ++d)
        if (hkv % d == 0 && d <= num_sms && num_sms / d * d >= num_sms / best * best) best = d;
    return best;
}

// The workspace behind its header: a Merge a CTA of both kernels, then the states of both, two a CTA.
struct ChunkLayout {
    size_t merges, states, few, bytes;
};

ChunkLayout chunk_layout(int num_sms) {
    const size_t row = sizeof(float2) + kRowBytes * 2, n = (size_t)num_sms;
    ChunkLayout l;
    l.merges = sizeof(pkv_ws_header);
    l.states = l.merges + (2 * n * kChunkMergeBytes + kWsAlign - 1) / kWsAlign * kWsAlign;
    l.few = l.states + n * 2 * 2 * kRows * row;
    l.bytes = l.few + n * 2 * kRows * row;
    return l;
}

}  // namespace

size_t chunk_workspace_bytes(int num_sms) { return chunk_layout(num_sms).bytes; }

int launch_chunk_attention(const ChunkParams& in, int num_sms, void* stream) {
    Params prm;
    ChunkParams& p = prm.p;
    p = in;
    p.lanes = head_lanes(p.Hkv, num_sms);
    p.grid = num_sms / p.lanes * p.lanes;
    p.tiles = 2;
    uint8_t* ws = reinterpret_cast<uint8_t*>(p.hdr);
    const ChunkLayout l = chunk_layout(num_sms);
    p.merges = ws + l.merges;
    p.ml = reinterpret_cast<float2*>(ws + l.states);
    p.acc = reinterpret_cast<float*>(p.ml + (size_t)num_sms * 2 * 2 * kRows);
    p.wait_ns = kWaitLimitNs + std::min(kFinishMostNs, kFinishNs * kPageSize * (uint64_t)p.max_pages);
    const int g = p.Hq / p.Hkv;
    const int64_t token = (int64_t)p.Hkv * kHeadDim;
    if (!encode_rows(&prm.q, p.q, p.Hq, p.total_tokens, p.q_stride, g, kRows / g) ||
        !encode_rows(&prm.q64, p.q, p.Hq, p.total_tokens, p.q_stride, g, kRows / 2 / g) ||
        !encode_rows(&prm.k, p.k_pool, p.Hkv, (int64_t)p.num_pages * kPageSize, token, 1, kPageSize) ||
        !encode_rows(&prm.v, p.v_pool, p.Hkv, (int64_t)p.num_pages * kPageSize, token, 1, kPageSize))
        return cudaErrorInvalidValue;
    Params few = prm;
    few.p.tiles = 1;
    few.p.merges = ws + l.merges + (size_t)num_sms * kChunkMergeBytes;
    few.p.ml = reinterpret_cast<float2*>(ws + l.few);
    few.p.acc = reinterpret_cast<float*>(few.p.ml + (size_t)num_sms * 2 * kRows);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (g) {
        case 1: return launch<1>(prm, few, s);
        case 2: return launch<2>(prm, few, s);
        case 4: return launch<4>(prm, few, s);
        case 8: return launch<8>(prm, few, s);
        case 16: return launch<16>(prm, few, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
