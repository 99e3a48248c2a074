// Packed prompts' K/V into pages and back (include/pkv.h, pkv_prompt_append, pkv_q4_prompt_append, pkv_q4_read).
#include <cuda_fp16.h>

#include <algorithm>

#include "pkv_internal.h"
#include "q4.cuh"

namespace pkv {
namespace {

// The packed rows of sequence s, or nothing where cu_seqlens is not monotone inside [0, total_tokens].
__device__ __forceinline__ bool seq_rows(const PagesParams& p, int s, int& first, int& n, int& start) {
    first = p.cu_seqlens[s];
    n = p.cu_seqlens[s + 1] - first;
    start = p.start ? p.start[s] : 0;
    if (first < 0 || n < 0 || n > p.total_tokens - first || start < 0 ||
        (int64_t)start + n > (int64_t)p.max_pages * kPageSize) {
        if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&p.hdr->status, PKV_STATUS_BAD_LEN);
        return false;
    }
    return true;
}

__device__ __forceinline__ int64_t page_of(const PagesParams& p, int s, int pos) {
    const int32_t e = p.block_table[(int64_t)s * p.max_pages + pos / kPageSize];
    if (e >= 0 && e < p.num_pages) return e;
    atomicOr(&p.hdr->status, PKV_STATUS_BAD_PAGE);
    return -1;
}

constexpr int kThreads = 256;

// FP16 pages: thread per 16 bytes of a (token, KV head, K or V).
__global__ void __launch_bounds__(kThreads) append_kernel(const PagesParams p) {
    for (int s = blockIdx.y; s < p.num_seqs; s += gridDim.y) {
        int first, n, start;
        if (!seq_rows(p, s, first, n, start)) continue;
        const int per = p.Hkv * 16;  // 16-byte pieces of one token's K
        for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (int64_t)n * per; i += (int64_t)gridDim.x * kThreads) {
            const int j = (int)(i / per), c = (int)(i % per);
            const int64_t page = page_of(p, s, start + j);
            if (page < 0) continue;
            const int64_t dst = (page * kPageSize + (start + j) % kPageSize) * per + c;
            static_cast<uint4*>(p.k_pool)[dst] =
                *reinterpret_cast<const uint4*>(static_cast<const __half*>(p.k) + (first + j) * p.k_stride + c * 8);
            static_cast<uint4*>(p.v_pool)[dst] =
                *reinterpret_cast<const uint4*>(static_cast<const __half*>(p.v) + (first + j) * p.v_stride + c * 8);
        }
    }
}

// 4-bit pages: warp per (token, KV head).
__global__ void __launch_bounds__(kThreads) q4_append_kernel(const PagesParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int s = blockIdx.y; s < p.num_seqs; s += gridDim.y) {
        int first, n, start;
        if (!seq_rows(p, s, first, n, start)) continue;
        for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + warp; i < (int64_t)n * p.Hkv; i += (int64_t)gridDim.x * (kThreads / 32)) {
            const int j = (int)(i / p.Hkv), h = (int)(i % p.Hkv);
            const int64_t page = page_of(p, s, start + j);
            if (page < 0) continue;
            uint8_t* blk = static_cast<uint8_t*>(p.pool) + (page * p.Hkv + h) * kQ4Block;
            const int r = (start + j) % kPageSize;
            q4_quantise_row(static_cast<const __half*>(p.k) + (first + j) * p.k_stride + h * kHeadDim, blk, r, false, lane);
            q4_quantise_row(static_cast<const __half*>(p.v) + (first + j) * p.v_stride + h * kHeadDim, blk + kQ4Half, r, true, lane);
        }
    }
}

__device__ __forceinline__ void dequantise_row(const uint8_t* half_block, __half* y, int r, bool is_v, int lane) {
    float f[4];
    q4_dequantise4(half_block, r, is_v, lane, f);
    __half2 a = __floats2half2_rn(f[0], f[1]), b = __floats2half2_rn(f[2], f[3]);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t*>(&a);
    u.y = *reinterpret_cast<uint32_t*>(&b);
    *reinterpret_cast<uint2*>(y + lane * 4) = u;
}

__global__ void __launch_bounds__(kThreads) q4_read_kernel(const PagesParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int s = blockIdx.y; s < p.num_seqs; s += gridDim.y) {
        int first, n, start;
        if (!seq_rows(p, s, first, n, start)) continue;
        for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + warp; i < (int64_t)n * p.Hkv; i += (int64_t)gridDim.x * (kThreads / 32)) {
            const int j = (int)(i / p.Hkv), h = (int)(i % p.Hkv);
            const int64_t page = page_of(p, s, start + j);
            if (page < 0) continue;
            const uint8_t* blk = static_cast<const uint8_t*>(p.pool) + (page * p.Hkv + h) * kQ4Block;
            const int r = (start + j) % kPageSize;
            dequantise_row(blk, static_cast<__half*>(p.k_pool) + (first + j) * p.k_stride + h * kHeadDim, r, false, lane);
            dequantise_row(blk + kQ4Half, static_cast<__half*>(p.v_pool) + (first + j) * p.v_stride + h * kHeadDim, r, true, lane);
        }
    }
}

dim3 grid_for(const PagesParams& p, int num_sms, int64_t items, int per_cta) {
    const int64_t want = (items + per_cta - 1) / per_cta;
    return dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(want, 8 * (int64_t)num_sms)), std::min(p.num_seqs, 64));
}

}  // namespace

int launch_prompt_append(const PagesParams& p, int num_sms, void* stream) {
    append_kernel<<<grid_for(p, num_sms, (int64_t)p.total_tokens * p.Hkv * 16, kThreads), kThreads, 0,
                    static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError();
}

int launch_q4_append(const PagesParams& p, int num_sms, void* stream) {
    q4_append_kernel<<<grid_for(p, num_sms, (int64_t)p.total_tokens * p.Hkv, kThreads / 32), kThreads, 0,
                       static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError();
}

int launch_q4_read(const PagesParams& p, int num_sms, void* stream) {
    q4_read_kernel<<<grid_for(p, num_sms, (int64_t)p.total_tokens * p.Hkv, kThreads / 32), kThreads, 0,
                     static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
