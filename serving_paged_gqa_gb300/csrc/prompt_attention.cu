// Causal grouped-query attention over packed prompts (include/pkv.h, pkv_prompt_attention).
#include <cuda_fp16.h>

#include <algorithm>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 8;

struct Row4 {
    float x[4];
};

__device__ __forceinline__ Row4 load4(const __half* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return Row4{{a.x, a.y, b.x, b.y}};
}

// One warp, one (token, query head): online softmax over the keys 0..pos of its sequence, lane l holds dims 4l..4l+3.
__device__ __forceinline__ void row_attention(const PromptParams& p, int64_t first, int pos, int hq, int lane) {
    const int h = hq / (p.Hq / p.Hkv);
    const __half* k = static_cast<const __half*>(p.k) + first * p.k_stride + h * kHeadDim + lane * 4;
    const __half* v = static_cast<const __half*>(p.v) + first * p.v_stride + h * kHeadDim + lane * 4;
    const Row4 q = load4(static_cast<const __half*>(p.q) + (first + pos) * p.q_stride + hq * kHeadDim + lane * 4);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j <= pos; ++j) {
        const Row4 a = load4(k + j * p.k_stride);
        float s = q.x[0] * a.x[0] + q.x[1] * a.x[1] + q.x[2] * a.x[2] + q.x[3] * a.x[3];
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - ref), e = exp2f(s - ref);
        const Row4 b = load4(v + j * p.v_stride);
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = o[i] * f + e * b.x[i];
        m = mn;
    }
    const float inv = 1.f / l;
    uint2 u;
    u.x = pack_half2(o[0] * inv, o[1] * inv);
    u.y = pack_half2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + (first + pos) * p.out_stride + hq * kHeadDim + lane * 4) = u;
}

__global__ void __launch_bounds__(kWarps * 32) prompt_attention_kernel(const PromptParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int s = blockIdx.y; s < p.num_seqs; s += gridDim.y) {
        const int first = p.cu_seqlens[s], last = p.cu_seqlens[s + 1];
        if (first < 0 || last < first || last > p.total_tokens) {
            if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&p.hdr->status, PKV_STATUS_BAD_LEN);
            continue;
        }
        const int64_t rows = (int64_t)(last - first) * p.Hq;
        for (int64_t r = (int64_t)blockIdx.x * kWarps + warp; r < rows; r += (int64_t)gridDim.x * kWarps)
            row_attention(p, first, (int)(r / p.Hq), (int)(r % p.Hq), lane);
    }
}

}  // namespace

int launch_prompt_attention(const PromptParams& p, int num_sms, void* stream) {
    const dim3 grid(num_sms * 8, std::min(p.num_seqs, 64));
    prompt_attention_kernel<<<grid, kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
