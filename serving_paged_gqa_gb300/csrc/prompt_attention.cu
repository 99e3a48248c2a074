// Causal grouped-query attention over packed prompts on the 5th-generation tensor cores (include/pkv.h,
// pkv_prompt_attention).
//
// For token i of a sequence and query head hq of KV head h: out = sum_{j <= i} p_j v_j / sum p_j with p_j = 2^(x_j - m),
// x_j = scale * log2(e) * q_i.k_j, one pass over the keys with a running m and sum (online softmax).
//
// Work: a tile is 128 rows of the score matrix: the G query heads of 128 / G consecutive tokens of one KV head (row =
// token * G + head, which one TMA box of q gives), so that short and ragged prompts fill tiles G times better than
// tiles of one head would and K and V are read once for all G heads. A CTA works on two neighbouring tiles (A, B) at
// a time, over 128 keys per step. Causality cuts the keys of a tile at its last token, so only its last step is
// masked, and that step's matrix products are cut to the 16-key steps that it needs.
//
// One CTA per SM, persistent; pairs of tiles are claimed from an atomic counter, longest sequences and latest tokens
// first. Warp roles:
//   warps 0-15      softmax: warps 0-3 and 4-7 the first and second 64 keys of every step of tile A, 8-15 those of tile
//                   B; thread = row. The scores come from TMEM into registers (tcgen05.ld), the weights go back as fp16
//                   over them. (With one thread for all 128 keys of a row the softmax of a step takes 2000 cycles, and
//                   the tensor core, which has 1024 cycles of the other tile's work meanwhile, waits.) Finally they
//                   divide, round and store the output rows, 64 dims each.
//   warp 16         one (elected) thread waits for and issues the matrix instructions: S = Q K^T (both from shared memory),
//                   O += P V (P from TMEM). While tile A's softmax runs, the tensor core works on B's products, and the
//                   other way round: order PV_A(j), S_A(j+1), PV_B(j), S_B(j+1).
//   warp 17         one lane issues the TMA copies: q tiles, and K, V tiles of 128 tokens through a ring of 4 stages.
//   warp 18         claims work, two steps before the end of the current pair, and publishes it.
//   warp 19         clears the rows behind a sequence's end in its last tile of V, before the tile counts as loaded (in
//                   the other warps it costs 2-4 %).
// TMEM (512 columns): S_A, S_B (P over columns 0-31 and 64-95 of each), O_A, O_B. Instructions of one thread run in
// order, so S(j+1) may be issued over P(j) right after PV(j).
//
// Weights are 2^(x - ref), one ref a row, and enter the second product as fp16, the type of V, which both operands must
// have: the relative error of 16384 normal tokens' outputs is 2.9e-4, with 32-bit weights 2.1e-4, of which the output's
// rounding is most; a second fp16 part would be half as many matrix products again. Sums and accumulators are fp32.
// ref is the maximum of the row's first 64 keys less kLift, and stays as it is while the sum of 64 keys' weights, needed
// anyway, fits fp16: an ordinary step has no search for a maximum. A thread whose keys fail the test (before their
// weights are announced) raises ref by a whole number to its keys' maximum less kLift, scales what has been accumulated,
// and computes its weights again.
// kLift divides fp16's 40 powers of two between weights that are small beside a row's largest and scores that grow behind
// its first 64 keys. Weights below 2^-(14 + kLift) of the largest lose bits, and below 2^-(25 + kLift) are 0, which shows
// where a token whose V is 0 takes most of the weight. Relative error with such a first token 16 / 18 / 20 nats above
// 16384 others, and us of 2048 tokens whose scores have a standard deviation of 1-2 / 3 / 4 / 6 nats: kLift 0 1.3e-3,
// 0.27, 0.93; 30, 30, 35, 53. 4: 2.1e-4, 4.4e-4, 6.6e-2; 30, 35, 46, 67. 5: 2.1e-4, 2.5e-4, 9e-3; 31, 37, 51, 69. 6: 2.1e-4,
// 2.1e-4, 9e-4; 31, 40, 57, 71. (32-bit weights 1.7-2.1e-4. 16384 tokens take 4, 11, 23 % longer with 5 than with 0 at
// 3, 4, 6 nats.)
// The two threads of a row do not wait for each other in ordinary steps (that cost 450 cycles a step): products of a
// step's second half never begin before those of its first, so where the first half raises, it scales the second half's
// weights in TMEM as well, and where the second half does, it first waits for the first half's products. Each sees what the
// other has raised at the next step.
//
// A value that a row does not attend to is multiplied by a weight of 0, which does not remove an infinity or a NaN of
// V. Rows behind the sequence's end are therefore cleared in V's last tile (they may hold anything, and most tiles that
// end a sequence have some). What is left are infinities and NaN among the tile's own tokens, and scores beyond 2^27, of
// which the fp32 reference is off by more than the weights' range: an output row that is not finite, or whose weights
// add up to less than any reference allows, is finished by its warp (finish_rows): dimensions in which V's attended
// values are not finite get what those add up to, and if others are left, the row is computed again from its own
// keys alone (row_attention). A row whose weights' sum is NaN has a NaN score that it attends to: it stays NaN.
//
// Bound: the tensor core and the paths of its operands. Measured on GB300s (32 query heads, 8 KV heads): 16384 tokens
// 1.34-1.47 ms, 1500-1640 TFLOP/s as the power cap of the GPU at hand allows (0.78-0.86 of the measured cuBLAS burst,
// 0.87-0.95 of its sustained rate); 2048 tokens 30-32 us; one prompt of 17 tokens 6.3 us. The tensor pipe is active 69 %
// of the time at 4096 tokens.
//
// Every wait is bounded (pkv_wait.cuh): on a time-out the kernel sets PKV_STATUS_TIMEOUT, the warps drain what they
// have in flight, and the CTA frees its TMEM and returns. The limit grows with the prompt: a warp may finish 32 rows from
// all keys before them (0.16 us a key), while the others wait for it.
#include <cuda_fp16.h>

#include <algorithm>

#include "pkv_internal.h"
#include "pkv_launch.h"
#include "pkv_tcgen05.cuh"
#include "pkv_tensormap.h"
#include "pkv_wait.cuh"

namespace pkv {
namespace {

constexpr uint64_t kFinishNs = 32 * 1000;    // a warp's 32 rows, by the key that they are computed from again, at most
constexpr int kRows = 128;                   // rows of a tile, keys of a step
constexpr int kTileBytes = kRows * kRowBytes;  // 32 KB: two boxes of 64 dims
constexpr int kBoxBytes = kTileBytes / 2;
constexpr int kStages = 4;                   // K and V tiles in flight; loads are not what the tensor core waits for
constexpr int kSoftmax = 512;                // threads of the softmax
constexpr int kThreads = kSoftmax + 128;
// 512 * 104 + 128 * 64 = 640 * 96, what the launch has; equal shares of 96 are 1-3 % slower
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;
constexpr float kMost = 65504.f;             // sum of 64 weights above which the row's reference is raised
constexpr float kLift = 5.f;                 // the largest weight where the reference was set, in powers of two

struct Work {
    int32_t first, n, t0, h;  // sequence's first packed row and length; first token of tile A; KV head (-1: no more work)
};

constexpr int off_q = 0;
constexpr int off_ring = 2 * kTileBytes;
constexpr int off_prefix = off_ring + kStages * kTileBytes;  // work pairs before the i-th sequence of the order
constexpr int off_order = off_prefix + (PKV_MAX_BATCH + 1) * 4 + 12;
constexpr int off_work = off_order + PKV_MAX_BATCH * 2;
constexpr int off_hist = off_work + (int)sizeof(Work);
constexpr int off_bars = off_hist + 32 * 4;
constexpr int kBars = 2 * kStages + 2 + 2 + 2 + 2 + 4 + 2 + 2 + 2 + 8 + 8 + 2 + 1;
constexpr int off_ref = off_bars + kBars * 8;            // float [tile][row]: ref
constexpr int off_parts = off_ref + 2 * kRows * 4;       // float2 (ref, l) [work & 1][tile][half][row]
constexpr int off_late = off_parts + 2 * 2 * 2 * kRows * 8;  // int [tile][warp of the half]: the second half raises
constexpr int off_misc = off_late + 8 * 4;  // abort flag, TMEM address
constexpr int kSmem = off_misc + 16 + 1024;     // slack to align the base to 1024 bytes
static_assert(off_order % 16 == 0 && off_work % 16 == 0 && off_bars % 8 == 0 && off_parts % 8 == 0, "alignment");
static_assert(kSmem <= 227 * 1024, "shared memory");

struct Params {
    CUtensorMap q, k, v;
    PromptParams p;
};

// ---- one row on the CUDA cores ------------------------------------------------------------------------------------
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
// 4l..4l+3. Stores dims 64 half .. + 63. (With 8 at a time the kernel's ordinary steps spill registers.) Factors of the
// numerator stay at 2^-126 or above, which is nothing to finite values, and keeps infinities of V that no weight is too
// small for: 0 times one would be NaN.
__device__ __forceinline__ void row_attention(const PromptParams& p, int64_t first, int pos, int hq, int half, int lane) {
    constexpr int kKeys = 4;
    constexpr float kLeast = 0x1p-126f;
    const int h = hq / (p.Hq / p.Hkv);
    const __half* k = static_cast<const __half*>(p.k) + first * p.k_stride + h * kHeadDim + lane * 4;
    const __half* v = static_cast<const __half*>(p.v) + first * p.v_stride + h * kHeadDim + lane * 4;
    const Row4 q = floats4(load4(static_cast<const __half*>(p.q) + (first + pos) * p.q_stride + hq * kHeadDim + lane * 4));
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j <= pos; j += kKeys) {
        uint2 a[kKeys], b[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            a[i] = load4(k + min(j + i, pos) * p.k_stride);
            b[i] = load4(v + min(j + i, pos) * p.v_stride);
        }
        float s[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const Row4 x = floats4(a[i]);
            s[i] = q.x[0] * x.x[0] + q.x[1] * x.x[1] + q.x[2] * x.x[2] + q.x[3] * x.x[3];
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
#pragma unroll
            for (int i = 0; i < kKeys; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], x);
        float mn = m;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            s[i] = j + i <= pos ? s[i] * p.scale_log2 : -INFINITY;
            mn = fmaxf(mn, s[i]);
        }
        const float ref = mn == -INFINITY ? 0.f : mn, f = exp2f(m - ref);
        l *= f;
#pragma unroll
        for (int x = 0; x < 4; ++x) o[x] *= fmaxf(f, kLeast);
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
            if (j + i <= pos) {
                const float e = exp2f(s[i] - ref);
                const Row4 x = floats4(b[i]);
                l += e;
#pragma unroll
                for (int y = 0; y < 4; ++y) o[y] += fmaxf(e, kLeast) * x.x[y];
            }
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : NAN;  // NaN: a score is, or all of them are -inf
    uint2 u;
    u.x = pack_half2(o[0] * inv, o[1] * inv);
    u.y = pack_half2(o[2] * inv, o[3] * inv);
    if (lane >> 4 == half)
        *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + (first + pos) * p.out_stride + hq * kHeadDim + lane * 4) = u;
}

// One warp; rows: a bit for each of its 32 rows (row r is head h * G + r % G of token t0 + r / G of the sequence that
// begins at row `first`) whose tensor-core result, dims 64 half .. + 63 of it in out, is not finite, redo: those among them
// that are wrong for certain. Lane l looks at dims 2l, 2l + 1. Infinities of V that the row attends to add up to an
// infinity, of both signs (or with a NaN) to a NaN, whatever their weights; a row that has other dims that are not
// finite is computed again.
template <int G>
__device__ __noinline__ void finish_rows(const PromptParams& p, int first, int t0, int h, int half, uint32_t rows, uint32_t redo) {
    const int lane = threadIdx.x & 31;
    const __half* v = static_cast<const __half*>(p.v) + (int64_t)first * p.v_stride + h * kHeadDim + half * 64 + lane * 2;
    __half2 top = __float2half2_rn(0.f), low = top, nan = top;  // of the values of the keys before `keys`
    int64_t keys = 0;
    for (; rows; rows &= rows - 1) {  // in the order of their tokens
        const int r = __ffs(rows) - 1, pos = t0 + r / G;
        if ((redo >> r) & 1) continue;
#pragma unroll 16
        for (; keys <= pos; ++keys) {
            const __half2 x = *reinterpret_cast<const __half2*>(v + keys * p.v_stride);
            top = __hmax2(top, x);
            low = __hmin2(low, x);
            nan = __hmax2_nan(nan, x);
        }
        const uint32_t t = *reinterpret_cast<const uint32_t*>(&top), w = *reinterpret_cast<const uint32_t*>(&low),
                       n = *reinterpret_cast<const uint32_t*>(&nan);
        uint32_t* at = reinterpret_cast<uint32_t*>(static_cast<__half*>(p.out) + (int64_t)(first + pos) * p.out_stride +
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
        row_attention(p, first, t0 + r / G, h * G + r % G, half, lane);
    }
}

// ---- the tensor-core kernel ---------------------------------------------------------------------------------------
__device__ __forceinline__ int tiles_of(int n, int pair_tokens) { return (n + pair_tokens - 1) / pair_tokens; }

// Tokens that tile x (0: A, 1: B) of a work pair ends at (its keys are the tokens before that); <= its start: no row.
__device__ __forceinline__ int tile_end(const Work& w, int x, int tokens) {
    const int start = w.t0 + x * tokens;
    return start < w.n ? min(start + tokens, w.n) : 0;
}

// Length of sequence s, 0 where its bounds are not ordered inside [0, total_tokens].
__device__ __forceinline__ int seq_length(const PromptParams& p, int s, int& first, bool& bad) {
    first = p.cu_seqlens[s];
    const int last = p.cu_seqlens[s + 1];
    bad = first < 0 || last < first || last > p.total_tokens;
    return bad ? 0 : last - first;
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Params prm) {
    constexpr int kTokens = kRows / G;  // tokens of a tile
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const PromptParams& p = prm.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + off_bars);
    uint64_t* kv_empty = kv_full + kStages;
    uint64_t* w_full = kv_empty + kStages;  // the CTA's next work has been published
    uint64_t* w_empty = w_full + 1;         // every warp has taken it, and its copies have been issued
    uint64_t* q_full = w_empty + 1;       // [2], like those below: tile A, tile B
    uint64_t* q_empty = q_full + 2;
    uint64_t* s_full = q_empty + 2;       // the tile's scores are in TMEM
    uint64_t* p_full = s_full + 2;        // [2][2]: its weights of the step's first, second 64 keys are
    uint64_t* o_full = p_full + 4;        // its accumulator is complete
    uint64_t* lo_done = o_full + 2;       // the products of a step's first 64 keys are in the accumulator
    uint64_t* o_free = lo_done + 2;       // the accumulator has been read
    uint64_t* first_ref = o_free + 2;     // [tile][warp of the half]: the tile's first references are in shared memory
    uint64_t* half_done = first_ref + 8;  // [tile][warp of the half]: the second half has settled its weights of the step
    uint64_t* tail_full = half_done + 8;  // [2]: a tile of V with rows behind the sequence's end has come
    uint64_t* drain = tail_full + 2;
    Work* work = reinterpret_cast<Work*>(smem + off_work);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + off_misc);
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + off_misc + 4);
    const WaitCtx ctx{abort_flag, &p.hdr->status, p.wait_ns};

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        mbar_init(w_full, 1);
        mbar_init(w_empty, kSoftmax / 32 + 3);  // and warps 16, 17, 19
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);  // one arrival a warp
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&lo_done[i], 1);
            mbar_init(&o_free[i], 8);
            mbar_init(&tail_full[i], 1);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&first_ref[i], 1);
            mbar_init(&half_done[i], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 16) tmem_alloc(tmem_at, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;

    if (warp >= kSoftmax / 32) {
        regs_shrink<kOtherRegs>();
        auto claim = [&](int k, int64_t& at) {  // the index of the CTA's k-th work, once the warps have taken the one before
            at = blockIdx.x;
            if (k == 0) return true;
            if (!warp_wait(w_empty, (k - 1) & 1, ctx)) return false;
            uint32_t c = 0;
            if (lane == 0) c = atomicAdd(&p.hdr->queue_head, 1u);
            at = (int64_t)gridDim.x + __shfl_sync(0xffffffffu, c, 0);
            return true;
        };
        auto publish = [&](const Work& w) {  // false: it was the last
            if (lane == 0) {
                *work = w;
                mbar_arrive(w_full);
            }
            __syncwarp();
            return w.h >= 0;
        };
        auto rearm = [&]() {  // the last CTA to end claiming re-arms the counter for the next call
            if (lane == 0) {
                __threadfence();
                if (atomicAdd(&p.hdr->ctas_done, 1u) == gridDim.x - 1) {
                    atomicExch(&p.hdr->queue_head, 0u);
                    atomicExch(&p.hdr->ctas_done, 0u);
                }
            }
        };
        if (warp == 18 && p.num_seqs <= 32) {
            // -------------------------------------------------------------- work claims, up to 32 sequences
            // A lane holds a sequence. Most tile pairs first; within a sequence the last tokens (most keys) first. The
            // pairs before a lane's sequence are a sum over the lanes, so nothing is sorted or stored (the general form
            // below takes 1.4 us longer to the first claim).
            int first = 0, n = 0;
            bool bad = false;
            if (lane < p.num_seqs) n = seq_length(p, lane, first, bad);
            if (bad && blockIdx.x == 0) raise_status(ctx.status, PKV_STATUS_BAD_LEN);
            const int t = tiles_of(n, 2 * kTokens);
            int before = 0, all = 0;
            for (int i = 0; i < p.num_seqs; ++i) {
                const int y = __shfl_sync(0xffffffffu, t, i);
                before += y > t || (y == t && i < lane) ? y : 0;
                all += y;
            }
            const int64_t total = (int64_t)all * p.Hkv;
            for (int k = 0;; ++k) {
                int64_t at;
                if (!claim(k, at)) break;
                Work w{0, 0, 0, -1};
                if (at < total) {
                    const int pair = (int)(at / p.Hkv);
                    const int src = __ffs(__ballot_sync(0xffffffffu, before <= pair && pair < before + t)) - 1;
                    w.first = __shfl_sync(0xffffffffu, first, src);
                    w.n = __shfl_sync(0xffffffffu, n, src);
                    w.t0 = __shfl_sync(0xffffffffu, (t - 1 - (pair - before)) * 2 * kTokens, src);
                    w.h = (int)(at - (int64_t)pair * p.Hkv);
                }
                if (!publish(w)) break;
            }
            rearm();
        } else if (warp == 18) {
            // ---------------------------------------------------------------------------------- work claims
            // Sequences in descending order of the power of two of their tile pairs; within one, the last tokens
            // (most keys) first.
            int* prefix = reinterpret_cast<int*>(smem + off_prefix);
            uint16_t* order = reinterpret_cast<uint16_t*>(smem + off_order);
            int* hist = reinterpret_cast<int*>(smem + off_hist);
            const int chunks = (p.num_seqs + 31) / 32;
            hist[lane] = 0;
            __syncwarp();
            for (int c = 0; c < chunks; ++c) {
                const int s = c * 32 + lane;
                int first, n = 0;
                bool bad = false;
                if (s < p.num_seqs) n = seq_length(p, s, first, bad);
                if (bad && blockIdx.x == 0) raise_status(ctx.status, PKV_STATUS_BAD_LEN);
                const int t = tiles_of(n, 2 * kTokens);
                if (t > 0) atomicAdd(&hist[__clz(t)], 1);
            }
            __syncwarp();
            int incl = hist[lane];  // by leading zeros: the most tiles first
            const int mine = incl;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const int seqs = __shfl_sync(0xffffffffu, incl, 31);
            __syncwarp();
            hist[lane] = incl - mine;
            __syncwarp();
            for (int c = 0; c < chunks; ++c) {
                const int s = c * 32 + lane;
                int first, n = 0;
                bool bad;
                if (s < p.num_seqs) n = seq_length(p, s, first, bad);
                const int t = tiles_of(n, 2 * kTokens);
                const int key = t > 0 ? __clz(t) : 32;
                const unsigned same = __match_any_sync(0xffffffffu, key);
                const int base = t > 0 ? hist[key] : 0;
                __syncwarp();
                if (t > 0) {
                    order[base + __popc(same & ((1u << lane) - 1))] = (uint16_t)s;
                    if (lane == __ffs(same) - 1) hist[key] = base + __popc(same);
                }
                __syncwarp();
            }
            int run = 0;
            for (int c = 0; c * 32 < seqs; ++c) {
                const int i = c * 32 + lane;
                int first, t = 0;
                bool bad;
                if (i < seqs) t = tiles_of(seq_length(p, order[i], first, bad), 2 * kTokens);
                int sum = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                if (i < seqs) prefix[i] = run + sum - t;
                run += __shfl_sync(0xffffffffu, sum, 31);
            }
            __syncwarp();
            const int64_t total = (int64_t)run * p.Hkv;
            for (int k = 0;; ++k) {
                int64_t t;
                if (!claim(k, t)) break;
                Work w{0, 0, 0, -1};
                if (t < total) {
                    const int pair = (int)(t / p.Hkv);
                    int lo = 0, hi = seqs - 1;
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (prefix[mid] <= pair)
                            lo = mid;
                        else
                            hi = mid - 1;
                    }
                    bool bad;
                    w.n = seq_length(p, order[lo], w.first, bad);
                    w.t0 = (tiles_of(w.n, 2 * kTokens) - 1 - (pair - prefix[lo])) * 2 * kTokens;
                    w.h = (int)(t - (int64_t)pair * p.Hkv);
                }
                if (!publish(w)) break;
            }
            rearm();
        } else if (warp == 17) {
            // ------------------------------------------------------------------------------------- copies
            if (lane == 0) {
                prefetch_tensormap(&prm.q);
                prefetch_tensormap(&prm.k);
                prefetch_tensormap(&prm.v);
            }
            // K and V take L2's ordinary policy: kept first (evict_last) they are no faster (2048 tokens 30.1 us, 16384 1.41
            // ms either way), and the kernels that follow find less of L2 (a copy of 40 MB behind 16384 tokens: 15.5 us
            // instead of 13.4); evicted first they take 3 % longer.
            uint64_t ordinary;
            asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(ordinary));
            const uint64_t stream = policy_evict_first();
            int seq = 0, nq[2] = {0, 0}, nc = 0;
            bool stop = false;
            for (int k = 0; !stop; ++k) {
                if (!warp_wait(w_full, k & 1, ctx)) break;
                const Work w = *work;
                __syncwarp();
                if (w.h < 0) break;
                const int end = max(tile_end(w, 0, kTokens), tile_end(w, 1, kTokens));
                const int steps = (end + kRows - 1) / kRows;
                auto load_q = [&](int x) {
                    if (tile_end(w, x, kTokens) == 0) return true;
                    if (!warp_wait(&q_empty[x], (nq[x] & 1) ^ 1, ctx)) return false;
                    if (lane == 0) {
                        uint8_t* dst = smem + off_q + x * kTileBytes;
                        mbar_arrive_expect_tx(&q_full[x], kTileBytes);
                        for (int b = 0; b < 2; ++b)
                            tma_load_3d(dst + b * kBoxBytes, &prm.q, b * 64, w.h * G, w.first + w.t0 + x * kTokens,
                                        &q_full[x], stream);
                    }
                    __syncwarp();
                    ++nq[x];
                    return true;
                };
                auto load_kv = [&](const CUtensorMap* map, int j, bool tail = false) {  // tail: comes by way of warp 19
                    const int st = seq % kStages;
                    uint64_t* bar = tail ? &tail_full[nc & 1] : &kv_full[st];
                    if (!warp_wait(&kv_empty[st], ((seq / kStages) & 1) ^ 1, ctx)) return false;
                    if (lane == 0) {
                        uint8_t* dst = smem + off_ring + st * kTileBytes;
                        mbar_arrive_expect_tx(bar, kTileBytes);
                        for (int b = 0; b < 2; ++b)
                            tma_load_3d(dst + b * kBoxBytes, map, b * 64, w.h, w.first + j * kRows, bar, ordinary);
                    }
                    __syncwarp();
                    ++seq;
                    nc += tail;
                    return true;
                };
                auto load_v = [&](int j) { return load_kv(&prm.v, j, j == steps - 1 && (end & 15)); };
                stop = !load_q(0) || !load_kv(&prm.k, 0) || !load_q(1) || !load_v(0);
                for (int j = 1; j < steps && !stop; ++j) stop = !load_kv(&prm.k, j) || !load_v(j);
                // The next claim, about two steps before this pair's end. (Claimed when this one begins, a pair may go to a
                // CTA that is not done for long: 4096 tokens of 4 KV heads took 77 us, the longest pair takes 60.)
                if (lane == 0) mbar_arrive(w_empty);
            }
            // every copy that this warp issued lands before the CTA may end
            for (int j = max(0, nc - 2); j < nc; ++j) warp_drain(&tail_full[j & 1], (j >> 1) & 1);
            for (int j = max(0, seq - kStages); j < seq; ++j) warp_drain(&kv_full[j % kStages], (j / kStages) & 1);
            for (int x = 0; x < 2; ++x)
                if (nq[x] > 0) warp_drain(&q_full[x], (nq[x] - 1) & 1);
        } else if (warp == 19) {
            // --------------------------------------------------------------------- rows behind the sequence's end
            // The products' last step of 16 keys reads them (a pair of tiles ends at a multiple of 16 tokens elsewhere).
            int kv = 0, nc = 0;
            for (int k = 0;; ++k) {
                if (!warp_wait(w_full, k & 1, ctx)) break;
                const Work w = *work;
                __syncwarp();
                if (lane == 0) mbar_arrive(w_empty);
                if (w.h < 0) break;
                const int end = max(tile_end(w, 0, kTokens), tile_end(w, 1, kTokens));
                const int steps = (end + kRows - 1) / kRows;
                kv += 2 * steps;
                if ((end & 15) == 0) continue;
                const int pos = kv - 1;
                // (Two barriers: the loader may be one such tile ahead, but not two, as it gets a work when every warp has
                // taken the one before.)
                if (!warp_wait(&tail_full[nc & 1], (nc >> 1) & 1, ctx)) break;
                ++nc;
                uint8_t* v = smem + off_ring + (pos % kStages) * kTileBytes;
                const int first = end - (steps - 1) * kRows, last = (first + 15) & ~15;
                for (int i = first * 16 + lane; i < last * 16; i += 32)
                    *reinterpret_cast<uint4*>(v + ((i >> 3) & 1) * kBoxBytes + (i >> 4) * 128 + (i & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&kv_full[pos % kStages]);
            }
        } else if (warp == 16) {
            // ------------------------------------------------------------------------- matrix instructions
            // One thread does everything: the step's six waits are then 40 cycles each where there is nothing to wait for, and
            // 100 as votes of a warp, during which the tensor core runs dry (16384 tokens: 1440 TFLOP/s, now 1600).
            if (elect_one()) {
                int kv = 0;                        // ring position of the next K tile of the current work
                int nq[2] = {0, 0}, no[2] = {0, 0};  // tiles begun; accumulators begun
                int np[2][2] = {{0, 0}, {0, 0}};     // halves of steps taken
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    if (!thread_wait(w_full, k & 1, ctx)) break;
                    const Work w = *work;
                    mbar_arrive(w_empty);
                    if (w.h < 0) break;
                    const int end0 = tile_end(w, 0, kTokens), end1 = tile_end(w, 1, kTokens);
                    const int steps = (max(end0, end1) + kRows - 1) / kRows;
                    // ring positions: K_j at kv + 2j, V_j one behind it
                    const uint32_t ring = smem_addr(smem + off_ring);
                    auto stage_addr = [&](int pos) { return ring + (pos % kStages) * kTileBytes; };
                    auto wait_stage = [&](int pos) { return thread_wait(&kv_full[pos % kStages], (pos / kStages) & 1, ctx); };
                    // keys of step j that tile x needs (0: none)
                    auto keys = [&](int x, int j) { return max(0, min(kRows, (x ? end1 : end0) - j * kRows)); };
                    auto scores = [&](int x, int j) {  // S_x(j) = Q_x K_j^T
                        const int n = (keys(x, j) + 15) & ~15;
                        if (n == 0) return;
                        const uint64_t q = smem_desc_k_major(smem_addr(smem + off_q + x * kTileBytes));
                        const uint64_t kd = smem_desc_k_major(stage_addr(kv + 2 * j));
                        const uint32_t idesc = mma_idesc(n, false);
                        const bool last = keys(x, j + 1) == 0;  // the tile's last use of its queries
                        mma_ss_128<kBoxBytes / 16>(tmem + x * 128, q, kd, idesc);
                        mma_commit(&s_full[x]);
                        if (last) mma_commit(&q_empty[x]);
                    };
                    auto values = [&](int x, int j) {  // O_x += P_x(j) V_j
                        const int n = (keys(x, j) + 15) >> 4;
                        if (n == 0) return true;
                        constexpr uint32_t idesc = mma_idesc(kHeadDim, true);
                        const uint64_t v = smem_desc_mn_major(stage_addr(kv + 2 * j + 1), kBoxBytes);
                        const uint32_t o = tmem + 256 + x * 128, pw = tmem + x * 128;
                        const bool last = keys(x, j + 1) == 0;
                        if (j == 0) {  // the previous tile's rows have been read
                            if (!thread_wait(&o_free[x], (no[x] & 1) ^ 1, ctx)) return false;
                            ++no[x];
                        }
#pragma unroll
                        for (int half = 0; half < 2; ++half) {  // 64 keys each
                            const int c = min(4, n - 4 * half);  // steps of 16 keys
                            if (c <= 0) break;
                            if (!thread_wait(&p_full[2 * x + half], np[x][half] & 1, ctx)) return false;
                            ++np[x][half];
                            tc_fence_after();
                            if (c == 4)
                                mma_ts_64(o, pw + 64 * half, v + 512 * half, idesc, j > 0 || half > 0);
                            else
                                for (int i = 0; i < c; ++i)
                                    mma_ts(o, pw + 64 * half + 8 * i, v + 512 * half + 128 * i, idesc, j > 0 || half > 0 || i > 0);
                            if (half == 0) mma_commit(&lo_done[x]);
                            if (last && n - 4 * half <= 4) mma_commit(&o_full[x]);
                        }
                        return true;
                    };
                    auto release = [&](int pos) { mma_commit(&kv_empty[pos % kStages]); };
                    ok = wait_stage(kv);
                    for (int x = 0; x < 2 && ok; ++x) {
                        if (keys(x, 0) == 0) continue;
                        ok = thread_wait(&q_full[x], nq[x] & 1, ctx);
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
                    kv += 2 * steps;
                }
                mma_commit(drain);
            }
            __syncwarp();
            // every matrix instruction has completed before the TMEM is freed and the CTA ends
            warp_drain(drain, 0);
        }
    } else {
        // ---------------------------------------------------------------------------- softmax and output rows
        regs_grow<kSoftmaxRegs>();
        const int x = warp >> 3, h = (warp >> 2) & 1;  // tile, half of the keys (and of the output's dims)
        const int row = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + x * 128 + h * 64;  // this half's scores, and its weights over the first 32
        const uint32_t o_at = tmem + lanes + 256 + x * 128;
        volatile float* ref_at = reinterpret_cast<volatile float*>(smem + off_ref) + x * kRows + row;
        float2* parts = reinterpret_cast<float2*>(smem + off_parts) + x * 2 * kRows + row;  // + buffer * 4 kRows + half * kRows
        uint64_t* settled = &first_ref[x * 4 + (warp & 3)];
        uint64_t* second = &half_done[x * 4 + (warp & 3)];
        volatile int* late_at = reinterpret_cast<volatile int*>(smem + off_late) + x * 4 + (warp & 3);
        const float sl2 = p.scale_log2;
        const uint64_t sl2x2 = pack_f32x2(sl2, sl2);
        int ns = 0, no = 0;  // steps, tiles taken
        int step2 = 0;       // steps with keys in the second half, as the first half counts them
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!warp_wait(w_full, k & 1, ctx)) break;
            const Work w = *work;
            __syncwarp();
            if (lane == 0) mbar_arrive(w_empty);
            if (w.h < 0) break;
            const int end = tile_end(w, x, kTokens);
            if (end == 0) continue;
            const int steps = (end + kRows - 1) / kRows;
            const int token = w.t0 + x * kTokens + row / G;
            float ref = -INFINITY, l = 0.f;
            for (int j = 0; j < steps; ++j) {
                const int step = ns++;
                const int last = end - j * kRows - h * 64;  // keys of this half, counted from its first
                // The tile's last step ends in the first half: the second does not wait for its scores (nothing would keep
                // the next tile's from coming before it looks, and a parity two phases on does not pass). They have come
                // when the tile's accumulator is complete, for which it waits below.
                if (last <= 0) continue;
                if (!warp_wait(&s_full[x], step & 1, ctx)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // The step with the diagonal and the sequence's end is masked; the others are whole.
                const bool tail = j == steps - 1;
                const int lim = tail ? min(token, end - 1) - j * kRows - h * 64 : 64;
                auto fetch = [&](int c, uint32_t* r) {  // 32 of the row's scores
                    tmem_ld32(s_at + c * 32, r);
                    tmem_wait_ld();
                    tmem_use32(r);
                    if (tail) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c * 32 + i > lim) r[i] = 0xff800000u;  // -inf
                    }
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
                                ph[c * 16 + i] = pack_half2(a, b);
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
                    if (!warp_wait(settled, no & 1, ctx)) {
                        ok = false;
                        break;
                    }
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
                        if (!warp_wait(second, step2 & 1, ctx)) {
                            ok = false;
                            break;
                        }
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
                        if (!warp_wait(&lo_done[x], step & 1, ctx)) {
                            ok = false;
                            break;
                        }
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
                if (last > 64) ++step2;
                l += sum;
                parts[(no & 1) * 4 * kRows + h * kRows] = make_float2(ref, l);
                tmem_st32(s_at, ph);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (h == 1 && !raise) mbar_arrive(second);  // before the one that lets the first half's next step begin
                    mbar_arrive(&p_full[2 * x + h]);
                }
            }
            if (!ok) break;
            if (!warp_wait(&o_full[x], no & 1, ctx)) break;
            tc_fence_after();
            // the row's sum: both halves', relative to the last reference (they only rise)
            const float2 lo = parts[(no & 1) * 4 * kRows], hi = parts[(no & 1) * 4 * kRows + kRows];
            float total = lo.y;
            if (end > 64) {
                const float top = fmaxf(lo.x, hi.x);
                auto part = [&](const float2& x) {
                    const float f = x.x == top ? 1.f : fast_exp2(x.x - top);
                    return x.y == INFINITY && f == 0.f ? 0.f : x.y * f;
                };
                total = part(lo) + part(hi);
            }
            const bool mine = token < w.n;
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
                in[i] = t < w.n;
                dst[i] = static_cast<__half*>(p.out) + (int64_t)(w.first + t) * p.out_stride + (w.h * G + r % G) * kHeadDim +
                         h * 64 + q4 * 8;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t o[32], y[4][4];
                tmem_ld32(o_at + h * 64 + c * 32, o);
                tmem_wait_ld();
                tmem_use32(o);
                if (c == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_free[x]);  // the next tile's products may overwrite it
                }
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
            ++no;
            // The largest weight is 2^kLift, or half of that where the reference was raised, and next to scores that are it
            // themselves 1, or above 1/2.
            const bool low_sum = !(total >= 0.25f);
            const bool odd = __low2float(probe) != 0.f || __high2float(probe) != 0.f || low_sum;
            const unsigned again = __ballot_sync(0xffffffffu, mine && odd && !isnan(total));
            if (again) {
                const unsigned redo = __ballot_sync(0xffffffffu, low_sum) & again;
                __syncwarp();  // the rows were stored by other lanes
                finish_rows<G>(p, w.first, w.t0 + x * kTokens + (row & ~31) / G, w.h, h, again, redo);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

template <int G>
int launch(const Params& prm, int num_sms, cudaStream_t stream) {
    static int configured_mask = 0;  // one bit per device ordinal (< 32)
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 32 || !(__atomic_load_n(&configured_mask, __ATOMIC_ACQUIRE) & (1 << dev))) {
        cudaFuncAttributes a{};
        cudaError_t e = cudaFuncGetAttributes(&a, prompt_kernel<G>);
        if (e != cudaSuccess) return e;
        // the warpgroups' register shares come out of what the launch gives them
        if (a.numRegs * kThreads < kSoftmax * kSoftmaxRegs + 128 * kOtherRegs) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(prompt_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 32) __atomic_fetch_or(&configured_mask, 1 << dev, __ATOMIC_ACQ_REL);
    }
    // at most this many pairs of tiles: every sequence begins one, and the rest are full
    const int64_t pairs =
        ((int64_t)prm.p.total_tokens * G / (2 * kRows) + std::min(prm.p.num_seqs, prm.p.total_tokens)) * prm.p.Hkv;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(pairs, num_sms));
    return launch_kernel(prompt_kernel<G>, grid, kThreads, kSmem, stream, prm);
}

}  // namespace

int launch_prompt_attention(const PromptParams& p, int num_sms, void* stream) {
    Params prm;
    prm.p = p;
    prm.p.wait_ns = kWaitLimitNs + kFinishNs * p.total_tokens;
    const int g = p.Hq / p.Hkv;
    // one box is half of a tile's dims
    if (!encode_rows(&prm.q, p.q, p.Hq, p.total_tokens, p.q_stride, g, kRows / g) ||
        !encode_rows(&prm.k, p.k, p.Hkv, p.total_tokens, p.k_stride, 1, kRows) ||
        !encode_rows(&prm.v, p.v, p.Hkv, p.total_tokens, p.v_stride, 1, kRows))
        return cudaErrorInvalidValue;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (g) {
        case 1: return launch<1>(prm, num_sms, s);
        case 2: return launch<2>(prm, num_sms, s);
        case 4: return launch<4>(prm, num_sms, s);
        case 8: return launch<8>(prm, num_sms, s);
        case 16: return launch<16>(prm, num_sms, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
