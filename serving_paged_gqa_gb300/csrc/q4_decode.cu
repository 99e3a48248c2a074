// One decode step over the 4-bit pages (include/pkv.h, pkv_q4_decode_step).
#include <cuda_fp16.h>

#include <algorithm>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "q4.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;

// The newest token's K and V of every (row, KV head), quantised into its slot: warp per (row, KV head, K or V).
__global__ void __launch_bounds__(128) q4_new_token_kernel(const Q4Params p) {
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (i >= p.B * p.Hkv * 2) return;
    const int v = i & 1, h = (i >> 1) % p.Hkv, b = (i >> 1) / p.Hkv;
    const int len = p.seq_lens[b];
    if (len <= 0 || len > p.max_pages * kPageSize) return;
    const int page = p.block_table[(int64_t)b * p.max_pages + (len - 1) / kPageSize];
    if (page < 0 || page >= p.num_pages) return;
    uint8_t* blk = static_cast<uint8_t*>(p.pool) + ((int64_t)page * p.Hkv + h) * kQ4Block + v * kQ4Half;
    q4_quantise_row(static_cast<const __half*>(v ? p.v_new : p.k_new) + ((int64_t)b * p.Hkv + h) * kHeadDim, blk,
                    (len - 1) % kPageSize, v != 0, lane);
}

__global__ void __launch_bounds__(kWarps * 32) q4_decode_kernel(const Q4Params p) {
    __shared__ float s_o[kWarps][kHeadDim];
    __shared__ float s_m[kWarps], s_l[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / p.Hq, hq = blockIdx.x % p.Hq, h = hq / (p.Hq / p.Hkv);
    int len = p.seq_lens[b];
    if (len < 0 || len > p.max_pages * kPageSize) {
        if (threadIdx.x == 0) atomicOr(&p.hdr->status, PKV_STATUS_BAD_LEN);
        len = 0;
    }
    const __half* q = static_cast<const __half*>(p.q) + ((int64_t)b * p.Hq + hq) * kHeadDim;
    float qv[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    for (int i = 0; i < 4; ++i) qv[i] = __half2float(q[4 * lane + i]);
    for (int j = warp; j < len; j += kWarps) {
        const int page = p.block_table[(int64_t)b * p.max_pages + j / kPageSize];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) atomicOr(&p.hdr->status, PKV_STATUS_BAD_PAGE);
            continue;
        }
        const uint8_t* blk = static_cast<const uint8_t*>(p.pool) + ((int64_t)page * p.Hkv + h) * kQ4Block;
        float x[4];
        q4_dequantise4(blk, j % kPageSize, false, lane, x);
        float s = qv[0] * x[0] + qv[1] * x[1] + qv[2] * x[2] + qv[3] * x[3];
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - ref), e = exp2f(s - ref);
        q4_dequantise4(blk + kQ4Half, j % kPageSize, true, lane, x);
        l = l * f + e;
        for (int i = 0; i < 4; ++i) o[i] = o[i] * f + e * x[i];
        m = mn;
    }
    for (int i = 0; i < 4; ++i) s_o[warp][4 * lane + i] = o[i];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, L = 0.f, a = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    const float ref = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(s_m[w] - ref);
        L += f * s_l[w];
        a += f * s_o[w][threadIdx.x];
    }
    static_cast<__half*>(p.out)[((int64_t)b * p.Hq + hq) * kHeadDim + threadIdx.x] = __float2half_rn(L == 0.f ? 0.f : a / L);
}

}  // namespace

size_t q4_workspace_bytes(const pkv_problem&, int) { return sizeof(pkv_ws_header); }

int launch_q4_decode(const Q4Params& p, int num_sms, void* stream) {
    (void)num_sms;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.k_new) q4_new_token_kernel<<<(p.B * p.Hkv * 2 + 3) / 4, 128, 0, s>>>(p);
    q4_decode_kernel<<<p.B * p.Hq, kWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
