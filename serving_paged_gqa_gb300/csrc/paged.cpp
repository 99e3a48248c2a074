// C-ABI entry points of the calls over a paged cache that grows and is read piece by piece: argument validation and kernel
// launches (include/pkv.h, "chunks, tables and selected pages").
#include <cuda_runtime.h>

#include <cmath>

#include "pkv_internal.h"

namespace {

using namespace pkv;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_rc(int e) { return e == cudaSuccess ? PKV_OK : PKV_E_CUDA; }

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
    if (!ws) return PKV_E_NULLPTR;
    if (!aligned(ws, kWsAlign)) return PKV_E_ALIGN;
    return ws_bytes < need ? PKV_E_WS_TOO_SMALL : PKV_OK;
}

bool good_sms(int32_t num_sms) { return num_sms > 0 && num_sms <= PKV_MAX_SMS; }

// Times a score of fp16 rows (at most 128 * 65504^2) it stays inside fp32.
bool good_scale(float scale) { return scale >= 0.f && scale <= 1e12f; }

// Above 0, so that a masked score of -inf stays one; 1e-30 times any fp16 score is a weight of 1 all the same.
float scale_log2(float scale) { return std::fmax(scale * 1.4426950408889634f, 1e-30f); }

// The pools' tokens are the rows of a TMA tensor, whose coordinates have 32 bits.
bool good_pool(const pkv_problem* pr) { return pr->num_pages <= 0x7fffffff / kPageSize; }

}  // namespace

extern "C" int pkv_chunk_workspace_bytes(int32_t num_sms, size_t* bytes) {
    if (!bytes) return PKV_E_NULLPTR;
    if (!good_sms(num_sms)) return PKV_E_INVAL;
    *bytes = chunk_workspace_bytes(num_sms);
    return PKV_OK;
}

extern "C" int pkv_chunk_attention(const pkv_problem* pr, const pkv_prompt* pm, const void* q, const void* k_pool,
                                   const void* v_pool, const int32_t* cu_seqlens, const int32_t* start,
                                   const int32_t* block_table, float scale, int32_t num_sms, void* ws, size_t ws_bytes,
                                   void* out, void* stream) {
    if (!pr || !pm) return PKV_E_NULLPTR;
    int rc = pkv_check_problem(pr);
    if (rc == PKV_OK) rc = pkv_check_prompt(pm);
    if (rc != PKV_OK) return rc;
    if (pr->batch != pm->num_seqs || pr->num_kv_heads != pm->num_kv_heads || pr->num_q_heads != pm->num_q_heads ||
        !good_sms(num_sms) || !good_scale(scale))
        return PKV_E_INVAL;
    if (!good_pool(pr)) return PKV_E_UNSUPPORTED;
    rc = check_ws(ws, ws_bytes, chunk_workspace_bytes(num_sms));
    if (rc != PKV_OK) return rc;
    if (pm->num_seqs == 0 || pm->total_tokens == 0) return PKV_OK;
    if (!q || !k_pool || !v_pool || !cu_seqlens || !block_table || !out) return PKV_E_NULLPTR;
    if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16) || !aligned(cu_seqlens, 4) ||
        !aligned(start, 4) || !aligned(block_table, 4))
        return PKV_E_ALIGN;
    // tiles are read while others are written; a pool without pages has no tensor
    if (out == q || out == k_pool || out == v_pool || pr->num_pages == 0) return PKV_E_INVAL;
    ChunkParams p{};
    p.q = q;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.out = out;
    p.cu_seqlens = cu_seqlens;
    p.start = start;
    p.block_table = block_table;
    p.hdr = static_cast<pkv_ws_header*>(ws);
    p.q_stride = pm->q_stride;
    p.out_stride = pm->out_stride;
    p.num_seqs = pm->num_seqs;
    p.total_tokens = pm->total_tokens;
    p.Hq = pm->num_q_heads;
    p.Hkv = pm->num_kv_heads;
    p.num_pages = pr->num_pages;
    p.max_pages = pr->max_pages_per_seq;
    p.scale_log2 = scale_log2(scale);
    return cuda_rc(launch_chunk_attention(p, num_sms, stream));
}
