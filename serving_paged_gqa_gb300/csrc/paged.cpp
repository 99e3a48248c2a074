// C-ABI entry points of the calls over a paged cache that grows and is read piece by piece: argument validation and kernel
// launches (include/pkv.h, "chunks, tables and selected pages").
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

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

extern "C" int pkv_tables_grow(const pkv_problem* pr, const int32_t* new_tokens, const int32_t* seq_lens,
                               int32_t* block_table, const int32_t* free_pages, const int32_t* free_count,
                               int32_t* cu_seqlens, int32_t* start, int64_t* slots, int32_t* positions, int64_t capacity,
                               int32_t* seq_lens_out, int32_t* free_count_out, int32_t num_sms, void* ws, size_t ws_bytes,
                               void* stream) {
    if (!pr) return PKV_E_NULLPTR;
    int rc = pkv_check_problem(pr);
    if (rc == PKV_OK) rc = check_ws(ws, ws_bytes, PKV_PROMPT_WS_BYTES);
    if (rc != PKV_OK) return rc;
    if (!good_sms(num_sms) || capacity < 0 || capacity > INT32_MAX) return PKV_E_INVAL;
    if (!free_count || !free_count_out) return PKV_E_NULLPTR;
    if (pr->batch > 0 && (!new_tokens || !seq_lens || !seq_lens_out)) return PKV_E_NULLPTR;
    if (pr->batch > 0 && pr->max_pages_per_seq > 0 && !block_table) return PKV_E_NULLPTR;
    if (pr->num_pages > 0 && !free_pages) return PKV_E_NULLPTR;
    for (const void* p : {(const void*)new_tokens, (const void*)seq_lens, (const void*)block_table, (const void*)free_pages,
                          (const void*)free_count, (const void*)cu_seqlens, (const void*)start, (const void*)positions,
                          (const void*)seq_lens_out, (const void*)free_count_out})
        if (!aligned(p, 4)) return PKV_E_ALIGN;
    if (!aligned(slots, 8)) return PKV_E_ALIGN;
    // Lengths and the stack's height may be updated in place: they are written when all have been read. Nothing else may.
    const void* in[] = {new_tokens, seq_lens, free_pages, free_count};
    const void* out[] = {block_table, cu_seqlens, start, slots, positions, seq_lens_out, free_count_out};
    for (int i = 0; i < 7; ++i) {
        for (const void* x : in)
            if (out[i] && out[i] == x && !(x == seq_lens && i == 5) && !(x == free_count && i == 6)) return PKV_E_INVAL;
        for (int j = 0; j < i; ++j)
            if (out[i] && out[i] == out[j]) return PKV_E_INVAL;
    }
    TablesParams p{};
    p.new_tokens = new_tokens;
    p.seq_lens = seq_lens;
    p.block_table = block_table;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.cu_seqlens = cu_seqlens;
    p.start = start;
    p.slots = slots;
    p.positions = positions;
    p.capacity = capacity;
    p.seq_lens_out = seq_lens_out;
    p.free_count_out = free_count_out;
    p.hdr = static_cast<pkv_ws_header*>(ws);
    p.B = pr->batch;
    p.num_pages = pr->num_pages;
    p.max_pages = pr->max_pages_per_seq;
    return cuda_rc(launch_tables_grow(p, num_sms, stream));
}

extern "C" int pkv_tables_release(const pkv_problem* pr, const int32_t* released, const int32_t* seq_lens,
                                  const int32_t* block_table, int32_t* free_pages, const int32_t* free_count,
                                  int32_t* seq_lens_out, int32_t* free_count_out, int32_t num_sms, void* ws, size_t ws_bytes,
                                  void* stream) {
    if (!pr) return PKV_E_NULLPTR;
    int rc = pkv_check_problem(pr);
    if (rc == PKV_OK) rc = check_ws(ws, ws_bytes, PKV_PROMPT_WS_BYTES);
    if (rc != PKV_OK) return rc;
    if (!good_sms(num_sms)) return PKV_E_INVAL;
    if (!free_count || !free_count_out) return PKV_E_NULLPTR;
    if (pr->batch > 0 && (!released || !seq_lens || !seq_lens_out)) return PKV_E_NULLPTR;
    if (pr->batch > 0 && pr->max_pages_per_seq > 0 && !block_table) return PKV_E_NULLPTR;
    if (pr->num_pages > 0 && !free_pages) return PKV_E_NULLPTR;
    for (const void* p : {(const void*)released, (const void*)seq_lens, (const void*)block_table, (const void*)free_pages,
                          (const void*)free_count, (const void*)seq_lens_out, (const void*)free_count_out})
        if (!aligned(p, 4)) return PKV_E_ALIGN;
    const void* in[] = {released, seq_lens, block_table, free_count};
    const void* out[] = {free_pages, seq_lens_out, free_count_out};
    for (int i = 0; i < 3; ++i) {
        for (const void* x : in)
            if (out[i] && out[i] == x && !(x == seq_lens && i == 1) && !(x == free_count && i == 2)) return PKV_E_INVAL;
        for (int j = 0; j < i; ++j)
            if (out[i] && out[i] == out[j]) return PKV_E_INVAL;
    }
    TablesParams p{};
    p.released = released;
    p.seq_lens = seq_lens;
    p.block_table = const_cast<int32_t*>(block_table);
    p.free_out = free_pages;
    p.free_count = free_count;
    p.seq_lens_out = seq_lens_out;
    p.free_count_out = free_count_out;
    p.hdr = static_cast<pkv_ws_header*>(ws);
    p.B = pr->batch;
    p.num_pages = pr->num_pages;
    p.max_pages = pr->max_pages_per_seq;
    return cuda_rc(launch_tables_release(p, num_sms, stream));
}

extern "C" int pkv_page_bounds(const pkv_problem* pr, const pkv_prompt* pm, const int32_t* cu_seqlens, const int32_t* start,
                               const void* k_pool, const int32_t* block_table, void* bounds, int32_t num_sms, void* ws,
                               size_t ws_bytes, void* stream) {
    if (!pr || !pm) return PKV_E_NULLPTR;
    int rc = pkv_check_problem(pr);
    if (rc == PKV_OK) rc = pkv_check_prompt(pm);
    if (rc == PKV_OK) rc = check_ws(ws, ws_bytes, PKV_PROMPT_WS_BYTES);
    if (rc != PKV_OK) return rc;
    if (pr->batch != pm->num_seqs || pr->num_kv_heads != pm->num_kv_heads || !good_sms(num_sms)) return PKV_E_INVAL;
    if (pm->num_seqs == 0 || pm->total_tokens == 0) return PKV_OK;
    if (!cu_seqlens || !k_pool || !block_table || !bounds) return PKV_E_NULLPTR;
    if (!aligned(k_pool, 16) || !aligned(bounds, 16) || !aligned(cu_seqlens, 4) || !aligned(start, 4) || !aligned(block_table, 4))
        return PKV_E_ALIGN;
    if (bounds == k_pool) return PKV_E_INVAL;
    // the kernel counts a row's pages, 32 pieces of 16 bytes at a time, in 32 bits
    if ((int64_t)pr->max_pages_per_seq * ((pm->num_kv_heads + 1) / 2) > UINT32_MAX) return PKV_E_UNSUPPORTED;
    PagesParams p{};
    p.k_pool = const_cast<void*>(k_pool);
    p.pool = bounds;
    p.cu_seqlens = cu_seqlens;
    p.start = start;
    p.block_table = block_table;
    p.hdr = static_cast<pkv_ws_header*>(ws);
    p.num_seqs = pm->num_seqs;
    p.total_tokens = pm->total_tokens;
    p.Hkv = pm->num_kv_heads;
    p.num_pages = pr->num_pages;
    p.max_pages = pr->max_pages_per_seq;
    return cuda_rc(launch_page_bounds(p, num_sms, stream));
}

extern "C" int pkv_sparse_workspace_bytes(const pkv_problem* pr, int32_t num_sms, size_t* bytes) {
    if (!pr || !bytes) return PKV_E_NULLPTR;
    const int rc = pkv_check_problem(pr);
    if (rc != PKV_OK) return rc;
    if (!good_sms(num_sms)) return PKV_E_INVAL;
    *bytes = std::max(chunk_workspace_bytes(num_sms), select_layout(*pr).bytes);
    return PKV_OK;
}

extern "C" int pkv_select_pages(const pkv_problem* pr, const void* q, const void* bounds, const int32_t* block_table,
                                const int32_t* seq_lens_dev, int32_t select, int32_t num_sms, void* ws, size_t ws_bytes,
                                int32_t* pages, void* stream) {
    size_t need = 0;
    int rc = pkv_sparse_workspace_bytes(pr, num_sms, &need);
    if (rc == PKV_OK) rc = check_ws(ws, ws_bytes, need);
    if (rc != PKV_OK) return rc;
    if (select < 1) return PKV_E_INVAL;
    if (pr->batch == 0) return PKV_OK;
    if (!q || !bounds || !block_table || !seq_lens_dev || !pages) return PKV_E_NULLPTR;
    if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(block_table, 4) || !aligned(seq_lens_dev, 4) || !aligned(pages, 4))
        return PKV_E_ALIGN;
    if (pages == q || pages == bounds || pages == block_table || pages == seq_lens_dev) return PKV_E_INVAL;
    const SelectLayout l = select_layout(*pr);
    uint8_t* base = static_cast<uint8_t*>(ws);
    SelectParams p{};
    p.q = q;
    p.bounds = bounds;
    p.block_table = block_table;
    p.seq_lens = seq_lens_dev;
    p.pages = pages;
    p.hdr = static_cast<pkv_ws_header*>(ws);
    p.scores = reinterpret_cast<float*>(base + l.scores);
    p.exact = reinterpret_cast<double*>(base + l.exact);
    p.tops = reinterpret_cast<float*>(base + l.tops);
    p.B = pr->batch;
    p.Hq = pr->num_q_heads;
    p.Hkv = pr->num_kv_heads;
    p.num_pages = pr->num_pages;
    p.max_pages = pr->max_pages_per_seq;
    p.select = select;
    return cuda_rc(launch_select_pages(p, num_sms, stream));
}

extern "C" int pkv_sparse_decode_step(const pkv_problem* pr, const void* q, const void* k_pool, const void* v_pool,
                                      const int32_t* block_table, const int32_t* seq_lens_dev, const int32_t* pages,
                                      int32_t select, float scale, int32_t num_sms, void* ws, size_t ws_bytes, void* out,
                                      void* stream) {
    size_t need = 0;
    int rc = pkv_sparse_workspace_bytes(pr, num_sms, &need);
    if (rc == PKV_OK) rc = check_ws(ws, ws_bytes, need);
    if (rc != PKV_OK) return rc;
    if (select < 1 || select > 0x7fffffff / kPageSize || !good_scale(scale)) return PKV_E_INVAL;
    if (!good_pool(pr)) return PKV_E_UNSUPPORTED;
    if (pr->batch == 0) return PKV_OK;
    if (!q || !k_pool || !v_pool || !block_table || !seq_lens_dev || !pages || !out) return PKV_E_NULLPTR;
    if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
        !aligned(seq_lens_dev, 4) || !aligned(pages, 4))
        return PKV_E_ALIGN;
    if (out == q || out == k_pool || out == v_pool || pr->num_pages == 0) return PKV_E_INVAL;
    ChunkParams p{};
    p.q = q;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.out = out;
    p.block_table = block_table;
    p.seq_lens = seq_lens_dev;
    p.pages = pages;
    p.select = select;
    p.hdr = static_cast<pkv_ws_header*>(ws);
    p.q_stride = p.out_stride = (int64_t)pr->num_q_heads * kHeadDim;
    p.num_seqs = p.total_tokens = pr->batch;
    p.Hq = pr->num_q_heads;
    p.Hkv = pr->num_kv_heads;
    p.num_pages = pr->num_pages;
    p.max_pages = pr->max_pages_per_seq;
    p.scale_log2 = scale_log2(scale);
    return cuda_rc(launch_chunk_attention(p, num_sms, stream));
}
