// The 4-bit page format (include/pkv.h, "4-bit pages") as the kernels see it.
//
// One block of kQ4Block bytes per (page, KV head): K codes, K parameters, V codes, V parameters. A group is 64 dims
// of one token: value = code * scale + offset with offset = min, scale = fp16((max - min) / 15) and code =
// clamp(round((x - offset) / scale), 0, 15). The code bytes lie in the order in which the decode's matrix
// instructions take them (mma m16n8k16, A operand; lane = 4 * g + t), so that a lane's share of a page is two 16-byte
// reads for K and two for V and no bank is hit twice. A byte holds one token's dims d (low 4 bits) and d + 64 (high):
// masking a word with 0x000F000F gives two fp16 subnormals code * 2^-24 (0x00F000F0: code * 2^-20), which the matrix
// instructions multiply exactly, so unpacking costs one logical instruction per pair and the power of two goes into
// the group's scale.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "pkv_internal.h"

namespace pkv {

constexpr int kQ4Codes = kPageSize * kHeadDim / 2;  // 1024: one page's codes of K (or V), one KV head
constexpr int kQ4Params = kPageSize * 2 * 4;        // 128: (scale, offset) fp16 per token and group
constexpr int kQ4Half = kQ4Codes + kQ4Params;       // 1152
constexpr int kQ4Block = 2 * kQ4Half;               // 2304
static_assert(kQ4Block == PKV_Q4_BLOCK_BYTES, "block size");

// Byte of K codes that holds dims d and d + 64 (d < 64) of token r: word (r, t, ks) has dims 16 ks + 2t, + 8, + 1, + 9.
__host__ __device__ __forceinline__ int q4_k_byte(int r, int d) {
    const int ks = d >> 4, j0 = (d >> 3) & 1, t = (d >> 1) & 3, j1 = d & 1;
    return r * 64 + t * 16 + ks * 4 + 2 * j1 + j0;
}

// Byte of V codes: word (r / 8, d % 8, (r % 8) / 2, d / 16) has tokens r, r + 1 (r even) of dims d, d + 8.
__host__ __device__ __forceinline__ int q4_v_byte(int r, int d) {
    const int dt = d >> 4, j0 = (d >> 3) & 1, g = d & 7, t = (r >> 1) & 3, j1 = r & 1;
    return (r >> 3) * 512 + (4 * g + t) * 16 + dt * 4 + 2 * j1 + j0;
}

// (scale, offset) of a group from its extremes. A group with a NaN or an infinity is stored as NaN: every value that
// it stands for is NaN, as a decode over such a token is.
__device__ __forceinline__ __half2 q4_params(float mn, float mx, bool finite) {
    if (!finite) return __halves2half2(__ushort_as_half(0x7fff), __ushort_as_half(0x7fff));
    return __halves2half2(__float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.f)), __float2half_rn(mn));
}

// Code of x in a group; the same division and rounding for every writer, so that a token has one 4-bit form.
__device__ __forceinline__ uint32_t q4_code(float x, float scale, float offset) {
    if (!(scale > 0.f)) return 0u;
    const float c = rintf(__fdiv_rn(__fsub_rn(x, offset), scale));
    return static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f));
}

// One warp quantises token r of a block half from 128 fp16 values: lane l holds dims 4l..4l+3, a group is 16 lanes.
__device__ __forceinline__ void q4_quantise_row(const __half* x, uint8_t* half_block, int r, bool is_v, int lane) {
    const uint2 u = *reinterpret_cast<const uint2*>(x + lane * 4);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    const float f[4] = {a.x, a.y, b.x, b.y};
    float mn = f[0], mx = f[0];
    bool fin = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mn = fminf(mn, f[i]);
        mx = fmaxf(mx, f[i]);
        fin = fin && isfinite(f[i]);
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    const unsigned all = __ballot_sync(0xffffffffu, fin);
    const int grp = lane >> 4;
    const __half2 par = q4_params(mn, mx, ((all >> (16 * grp)) & 0xffffu) == 0xffffu);
    const float sc = __low2float(par), off = __high2float(par);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = q4_code(f[i], sc, off);
        const uint32_t hi = __shfl_down_sync(0xffffffffu, c, 16);
        const int d = 4 * lane + i;
        if (lane < 16) half_block[is_v ? q4_v_byte(r, d) : q4_k_byte(r, d)] = (uint8_t)(c | (hi << 4));
    }
    if ((lane & 15) == 0) reinterpret_cast<__half2*>(half_block + kQ4Codes)[2 * r + grp] = par;
}

}  // namespace pkv
