// C-ABI entry points of the prompt and 4-bit-cache calls: argument validation and kernel launches (include/pkv.h).
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

// A GPU's SM count: the workspace's size and the grids are multiples of it.
bool good_sms(int32_t num_sms) { return num_sms > 0 && num_sms <= PKV_MAX_SMS; }

// Times a score of fp16 rows (at most 128 * 65504^2), or a 4-bit group's scale and 2^24, it stays inside fp32.
bool good_scale(float scale) { return std::fabs(scale) <= 1e12f; }

bool good_stride(int64_t stride, int64_t heads, int64_t rows) {
    return stride >= heads * kHeadDim && stride % 8 == 0 && stride < (int64_t(1) << 32) &&
           (rows <= 1 || stride <= INT64_MAX / 4 / rows);
}

// The checks that the three page calls share.
int check_pages(const pkv_problem* pr, const pkv_prompt* pm, const int32_t* cu_seqlens, const int32_t* start,
                const int32_t* block_table, int32_t num_sms, const void* ws, size_t ws_bytes) {
    if (!pr || !pm) return PKV_E_NULLPTR;
    int rc = pkv_check_problem(pr);
    if (rc == PKV_OK) rc = pkv_check_prompt(pm);
    if (rc != PKV_OK) return rc;
    if (pr->batch != pm->num_seqs || pr->num_kv_heads != pm->num_kv_heads || !good_sms(num_sms)) return PKV_E_INVAL;
    rc = check_ws(ws, ws_bytes, PKV_PROMPT_WS_BYTES);
    if (rc != PKV_OK) return rc;
    if (!aligned(cu_seqlens, 4) || !aligned(start, 4) || !aligned(block_table, 4)) return PKV_E_ALIGN;
    return PKV_OK;
}

PagesParams pages_params(const pkv_problem* pr, const pkv_prompt* pm, const int32_t* cu_seqlens, const int32_t* start,
                         const int32_t* block_table, void* ws) {
    PagesParams p{};
    p.cu_seqlens = cu_seqlens;
    p.start = start;
    p.block_table = block_table;
    p.hdr = static_cast<pkv_ws_header*>(ws);
    p.k_stride = pm->k_stride;
    p.v_stride = pm->v_stride;
    p.num_seqs = pm->num_seqs;
    p.total_tokens = pm->total_tokens;
    p.Hkv = pm->num_kv_heads;
    p.num_pages = pr->num_pages;
    p.max_pages = pr->max_pages_per_seq;
    return p;
}

bool nothing(const pkv_prompt* pm) { return pm->num_seqs == 0 || pm->total_tokens == 0; }

int q4_step(const pkv_problem* pr, const void* q, const void* k_new, const void* v_new, void* pool,
            const int32_t* block_table, const int32_t* seq_lens_dev, float scale, int32_t num_sms, void* ws,
            size_t ws_bytes, void* out, void* stream) {
    size_t need = 0;
    int rc = pkv_q4_workspace_bytes(pr, num_sms, &need);
    if (rc == PKV_OK) rc = check_ws(ws, ws_bytes, need);
    if (rc != PKV_OK) return rc;
    if (!good_scale(scale)) return PKV_E_INVAL;
    if (pr->batch == 0) return PKV_OK;
    if (!q || !pool || !block_table || !seq_lens_dev || !out) return PKV_E_NULLPTR;
    if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) ||
        !aligned(block_table, 4) || !aligned(seq_lens_dev, 4))
        return PKV_E_ALIGN;
    // the pieces of a row read q, k_new and v_new when others are done, and the pool's pages all the time
    if (out == q || out == k_new || out == v_new || out == pool) return PKV_E_INVAL;
    Q4Params p{};
    p.q = q;
    p.k_new = k_new;
    p.v_new = v_new;
    p.pool = pool;
    p.block_table = block_table;
    p.seq_lens = seq_lens_dev;
    p.out = out;
    p.hdr = static_cast<pkv_ws_header*>(ws);
    p.B = pr->batch;
    p.Hq = pr->num_q_heads;
    p.Hkv = pr->num_kv_heads;
    p.num_pages = pr->num_pages;
    p.max_pages = pr->max_pages_per_seq;
    // not 0, so that a masked score of -inf stays one (see pkv_prompt_attention)
    p.scale_log2 = scale * 1.4426950408889634f;
    if (std::fabs(p.scale_log2) < 1e-30f) p.scale_log2 = 1e-30f;
    return cuda_rc(launch_q4_decode(p, num_sms, stream));
}

}  // namespace

extern "C" int pkv_check_prompt(const pkv_prompt* pm) {
    if (!pm) return PKV_E_NULLPTR;
    if (pm->num_seqs < 0 || pm->total_tokens < 0 || pm->num_q_heads <= 0 || pm->num_kv_heads <= 0 || pm->reserved != 0)
        return PKV_E_INVAL;
    if (pm->head_dim != kHeadDim || pm->num_q_heads % pm->num_kv_heads != 0) return PKV_E_UNSUPPORTED;
    const int g = pm->num_q_heads / pm->num_kv_heads;
    if (g != 1 && g != 2 && g != 4 && g != 8 && g != 16) return PKV_E_UNSUPPORTED;
    if (pm->num_seqs > PKV_MAX_BATCH || pm->num_kv_heads > 0x7fff) return PKV_E_UNSUPPORTED;
    if (!good_stride(pm->q_stride, pm->num_q_heads, pm->total_tokens) ||
        !good_stride(pm->out_stride, pm->num_q_heads, pm->total_tokens) ||
        !good_stride(pm->k_stride, pm->num_kv_heads, pm->total_tokens) ||
        !good_stride(pm->v_stride, pm->num_kv_heads, pm->total_tokens))
        return PKV_E_INVAL;
    return PKV_OK;
}

extern "C" int pkv_prompt_attention(const pkv_prompt* pm, const void* q, const void* k, const void* v,
                                    const int32_t* cu_seqlens, float scale, int32_t num_sms, void* ws, size_t ws_bytes,
                                    void* out, void* stream) {
    int rc = pkv_check_prompt(pm);
    if (rc == PKV_OK) rc = check_ws(ws, ws_bytes, PKV_PROMPT_WS_BYTES);
    if (rc != PKV_OK) return rc;
    if (!good_scale(scale) || scale < 0.f || !good_sms(num_sms)) return PKV_E_INVAL;
    if (nothing(pm)) return PKV_OK;
    if (!q || !k || !v || !cu_seqlens || !out) return PKV_E_NULLPTR;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu_seqlens, 4))
        return PKV_E_ALIGN;
    if (out == q || out == k || out == v) return PKV_E_INVAL;  // tiles are read while others are written
    PromptParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.out = out;
    p.cu_seqlens = cu_seqlens;
    p.hdr = static_cast<pkv_ws_header*>(ws);
    p.q_stride = pm->q_stride;
    p.k_stride = pm->k_stride;
    p.v_stride = pm->v_stride;
    p.out_stride = pm->out_stride;
    p.num_seqs = pm->num_seqs;
    p.total_tokens = pm->total_tokens;
    p.Hq = pm->num_q_heads;
    p.Hkv = pm->num_kv_heads;
    // above 0, so that a masked score of -inf stays one; 1e-30 times any fp16 score is a weight of 1 all the same
    p.scale_log2 = std::fmax(scale * 1.4426950408889634f, 1e-30f);
    return cuda_rc(launch_prompt_attention(p, num_sms, stream));
}

extern "C" int pkv_prompt_append(const pkv_problem* pr, const pkv_prompt* pm, const void* k, const void* v,
                                 const int32_t* cu_seqlens, const int32_t* start, void* k_pool, void* v_pool,
                                 const int32_t* block_table, int32_t num_sms, void* ws, size_t ws_bytes, void* stream) {
    int rc = check_pages(pr, pm, cu_seqlens, start, block_table, num_sms, ws, ws_bytes);
    if (rc != PKV_OK) return rc;
    if (nothing(pm)) return PKV_OK;
    if (!k || !v || !cu_seqlens || !k_pool || !v_pool || !block_table) return PKV_E_NULLPTR;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16)) return PKV_E_ALIGN;
    if (k_pool == v_pool) return PKV_E_INVAL;
    PagesParams p = pages_params(pr, pm, cu_seqlens, start, block_table, ws);
    p.k = k;
    p.v = v;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    return cuda_rc(launch_prompt_append(p, num_sms, stream));
}

extern "C" int pkv_q4_prompt_append(const pkv_problem* pr, const pkv_prompt* pm, const void* k, const void* v,
                                    const int32_t* cu_seqlens, const int32_t* start, void* pool,
                                    const int32_t* block_table, int32_t num_sms, void* ws, size_t ws_bytes,
                                    void* stream) {
    int rc = check_pages(pr, pm, cu_seqlens, start, block_table, num_sms, ws, ws_bytes);
    if (rc != PKV_OK) return rc;
    if (nothing(pm)) return PKV_OK;
    if (!k || !v || !cu_seqlens || !pool || !block_table) return PKV_E_NULLPTR;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pool, 16)) return PKV_E_ALIGN;
    PagesParams p = pages_params(pr, pm, cu_seqlens, start, block_table, ws);
    p.k = k;
    p.v = v;
    p.pool = pool;
    return cuda_rc(launch_q4_append(p, num_sms, stream));
}

extern "C" int pkv_q4_read(const pkv_problem* pr, const pkv_prompt* pm, const int32_t* cu_seqlens,
                           const int32_t* start, const void* pool, const int32_t* block_table, void* k_out,
                           void* v_out, int32_t num_sms, void* ws, size_t ws_bytes, void* stream) {
    int rc = check_pages(pr, pm, cu_seqlens, start, block_table, num_sms, ws, ws_bytes);
    if (rc != PKV_OK) return rc;
    if (nothing(pm)) return PKV_OK;
    if (!k_out || !v_out || !cu_seqlens || !pool || !block_table) return PKV_E_NULLPTR;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(pool, 16)) return PKV_E_ALIGN;
    if (k_out == v_out || k_out == pool || v_out == pool) return PKV_E_INVAL;
    PagesParams p = pages_params(pr, pm, cu_seqlens, start, block_table, ws);
    p.k_pool = k_out;
    p.v_pool = v_out;
    p.pool = const_cast<void*>(pool);
    return cuda_rc(launch_q4_read(p, num_sms, stream));
}

extern "C" int pkv_q4_pool_bytes(const pkv_problem* pr, size_t* bytes) {
    if (!pr || !bytes) return PKV_E_NULLPTR;
    int rc = pkv_check_problem(pr);
    if (rc != PKV_OK) return rc;
    *bytes = (size_t)pr->num_pages * pr->num_kv_heads * PKV_Q4_BLOCK_BYTES;
    return PKV_OK;
}

extern "C" int pkv_q4_workspace_bytes(const pkv_problem* pr, int32_t num_sms, size_t* bytes) {
    if (!pr || !bytes) return PKV_E_NULLPTR;
    int rc = pkv_check_problem(pr);
    if (rc != PKV_OK) return rc;
    if (!good_sms(num_sms)) return PKV_E_INVAL;
    *bytes = q4_workspace_bytes(*pr, num_sms);
    return PKV_OK;
}

extern "C" int pkv_q4_decode_step(const pkv_problem* pr, const void* q, const void* pool, const int32_t* block_table,
                                  const int32_t* seq_lens_dev, float scale, int32_t num_sms, void* ws,
                                  size_t ws_bytes, void* out, void* stream) {
    return q4_step(pr, q, nullptr, nullptr, const_cast<void*>(pool), block_table, seq_lens_dev, scale, num_sms, ws,
                   ws_bytes, out, stream);
}

extern "C" int pkv_q4_decode_step_append(const pkv_problem* pr, const void* q, const void* k_new, const void* v_new,
                                         void* pool, const int32_t* block_table, const int32_t* seq_lens_dev,
                                         float scale, int32_t num_sms, void* ws, size_t ws_bytes, void* out,
                                         void* stream) {
    if (pr && pr->batch > 0 && (!k_new || !v_new)) return PKV_E_NULLPTR;
    return q4_step(pr, q, k_new, v_new, pool, block_table, seq_lens_dev, scale, num_sms, ws, ws_bytes, out, stream);
}
