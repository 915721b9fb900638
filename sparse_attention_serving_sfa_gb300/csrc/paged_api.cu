// C ABI of the paged KV cache (paged_append, paged_read), of dense attention
// over it (paged_run) and over packed rows (varlen_run): argument checks,
// layout -> stride resolution, choice of path.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "paged.h"

using namespace sfa;

namespace {

bool al(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool is16(int t) { return t == SFA_DTYPE_F16 || t == SFA_DTYPE_BF16; }
bool is8(int t) { return t == SFA_DTYPE_E4M3 || t == SFA_DTYPE_E5M2; }

sfa_status check_heads(int Hq, int Hkv, int D) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return SFA_ERR_INVALID_ARG;
    if (D < 1 || D % 64 != 0) return SFA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return SFA_ERR_UNSUPPORTED;
    return SFA_OK;
}

// Checks a cache description and fills `kv`.
sfa_status resolve_cache(const paged_kv* c, SeqKV& kv) {
    if (!c || !c->k || !c->v || !c->page_table || !c->kv_lens) return SFA_ERR_INVALID_ARG;
    if (c->num_seqs < 1 || c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1)
        return SFA_ERR_INVALID_ARG;
    sfa_status st = check_heads(c->num_kv_heads, c->num_kv_heads, c->head_dim);
    if (st != SFA_OK) return st;
    if (!is16(c->dtype) && !is8(c->dtype)) return SFA_ERR_INVALID_ARG;
    if (c->kv_layout != SFA_KV_LAYOUT_NHD && c->kv_layout != SFA_KV_LAYOUT_HND)
        return SFA_ERR_INVALID_ARG;
    if (!al(c->k, 16) || !al(c->v, 16) || !al(c->page_table, 4) || !al(c->kv_lens, 4) ||
        !al(c->scale_k, 4) || !al(c->scale_v, 4))
        return SFA_ERR_INVALID_ARG;
    // per-head scales belong to 8-bit caches (as in bsr_run_scaled)
    if (is16(c->dtype) && (c->scale_k || c->scale_v)) return SFA_ERR_UNSUPPORTED;
    // token positions are 32-bit
    if ((int64_t)c->max_pages * c->page_size > 0x7fffffffLL / 2) return SFA_ERR_UNSUPPORTED;
    kv = SeqKV{};
    kv.k = c->k; kv.v = c->v;
    kv.page_table = c->page_table;
    kv.kv_lens = c->kv_lens;
    kv.num_seqs = c->num_seqs; kv.num_pages = c->num_pages;
    kv.page_size = c->page_size; kv.max_pages = c->max_pages;
    kv.Hkv = c->num_kv_heads; kv.D = c->head_dim;
    const int64_t H = kv.Hkv, D = kv.D, P = kv.page_size;
    kv.s_page = P * H * D;
    kv.s_tok = c->kv_layout == SFA_KV_LAYOUT_NHD ? H * D : D;
    kv.s_head = c->kv_layout == SFA_KV_LAYOUT_NHD ? D : P * D;
    kv.f8 = is16(c->dtype) ? 0 : (c->dtype == SFA_DTYPE_E4M3 ? 1 : 2);
    kv.scale_k = c->scale_k; kv.scale_v = c->scale_v;
    kv.by_page = divide_by(c->page_size);
    return SFA_OK;
}

// A token stride (elements) of packed rows of `heads` heads.
bool bad_stride(int64_t stride, int heads, int D) {
    return stride < (int64_t)heads * D || stride % 8 != 0 || stride > (int64_t)1 << 38;
}

// 16-row tiles read the keys at HBM's pace and begin early; the 128-row
// tensor-core tiles stand mostly empty with few rows, but more rows cost them
// nothing.  So 16-row tiles take (times: 16-row tiles, 128-row tiles; head_dim
// 128, 8 kv heads unless said otherwise)
//   - up to 16 rows a kv head (by the longest sequence): 16 rows, 64 sequences
//     of 4,096 keys 174 and 171 us, one sequence of 8,192 keys 15.4 and 22.7 us;
//     but 32 rows, 64 sequences 333 and 173 us.  Over an 8-bit cache, which
//     128-row tiles must convert first, up to 32: 16 rows, 64 sequences 93 and
//     226 us, 32 rows 170 and 230 us, 48 rows 245 and 232 us.
//   - where they are few and read few keys over again.  One sequence, 48 rows
//     (24 tiles): of 2,000 keys 12.5 and 18.2 us, of 8,192 keys 19.9 and 22.8 us,
//     of 65,536 keys 85 and 58 us; 96 rows (48 tiles) of 8,192 keys 29.0 and
//     23.5 us.  2 kv heads, 128 rows (16 tiles) of 8,192 keys 16.8 and 40.1 us.  4
//     sequences of 500 keys, 64 tiles 11.3 and 12.2 us, 128 tiles 13.6 and 12.3
//     us.  8-bit: one sequence of 8,192 keys, 128 rows (64 tiles) 27.7 and 28.5
//     us; 4 of 16,384 keys, 2 kv heads, 64 rows (32 tiles) 28.2 and 31.7 us, 96
//     rows 36.3 and 32.2 us; 16 of 1,000 keys, 2 kv heads, 128 tiles 15.2 and 18.5
//     us, 192 tiles 19.6 and 19.2 us.
bool few_rows(const SeqAttn& p) {
    const bool f8 = p.kv.f8 != 0;
    const int64_t rows = (int64_t)p.max_q_len * p.G;
    const int64_t tiles = (rows + 15) / 16 * p.kv.num_seqs * p.kv.Hkv;
    // (keys: what the table or the packed rows can hold, the lengths are on the device)
    const int64_t keys = p.kv.page_table ? (int64_t)p.kv.max_pages * p.kv.page_size : p.kv.rows;
    return rows <= (f8 ? 32 : 16) || (tiles <= (f8 ? 128 : 64) && tiles * keys <= (f8 ? 524288 : 196608));
}

// Workspace of either path.
size_t attention_ws_bytes(int Hq, int Hkv, int D) {
    const size_t r = attn_rows_ws_bytes(D), t = attn_tc_ws_bytes(Hq / Hkv, D);
    return r > t ? r : t;
}

sfa_status run_attention(SeqAttn& p, int num_tokens, int num_qo_heads, int max_q_len, float scale,
                         int causal, sfa_dtype dtype, const void* q, int64_t q_stride,
                         const int32_t* cu_q, void* out, float* lse, void* ws, size_t ws_bytes,
                         sfa_stream_t stream) {
    if (num_tokens < 0 || max_q_len < 0 || !cu_q || !al(cu_q, 4)) return SFA_ERR_INVALID_ARG;
    sfa_status st = check_heads(num_qo_heads, p.kv.Hkv, p.kv.D);
    if (st != SFA_OK) return st;
    if (!is16(dtype) || !isfinite(scale)) return SFA_ERR_INVALID_ARG;
    if (bad_stride(q_stride, num_qo_heads, p.kv.D)) return SFA_ERR_INVALID_ARG;
    if ((int64_t)num_tokens * num_qo_heads > 0x7fffffffLL / 2) return SFA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return SFA_OK;
    if (!q || !out || !al(q, 16) || !al(out, 16) || !al(lse, 4)) return SFA_ERR_INVALID_ARG;
    const size_t need = attention_ws_bytes(num_qo_heads, p.kv.Hkv, p.kv.D);
    if (!ws || ws_bytes < need) return SFA_ERR_WORKSPACE;
    if (!al(ws, 16)) return SFA_ERR_INVALID_ARG;
    p.q = q; p.out = out; p.lse = lse; p.cu_q = cu_q;
    p.tokens = num_tokens; p.Hq = num_qo_heads; p.G = num_qo_heads / p.kv.Hkv;
    p.causal = causal ? 1 : 0;
    p.max_q_len = max_q_len > 0 && max_q_len < num_tokens ? max_q_len : num_tokens;
    p.q_stride = q_stride;
    p.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)p.kv.D)) * kLog2e;
    p.by_group = divide_by(p.G);
    p.by_heads = divide_by(p.kv.Hkv);
    p.ws = ws;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (!few_rows(p) && attn_tc_supported(p.kv, p.G)) {
        p.err_word = device_error_word();
        if (!p.err_word) return SFA_ERR_CUDA;
        err = launch_attn_tc(p, dtype, num_sms(), s);
    } else {
        err = launch_attn_rows(p, dtype, num_sms(), s);
    }
    return err == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

}  // namespace

extern "C" {

sfa_status paged_append(const paged_kv* cache, const void* k_new, const void* v_new,
                        int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens,
                        int num_tokens, sfa_dtype dtype, sfa_stream_t stream) {
    SeqKV kv;
    sfa_status st = resolve_cache(cache, kv);
    if (st != SFA_OK) return st;
    if (num_tokens < 0 || !cu_seqlens || !al(cu_seqlens, 4) || !is16(dtype)) return SFA_ERR_INVALID_ARG;
    if (kv.f8 == 0 && dtype != cache->dtype) return SFA_ERR_INVALID_ARG;
    if (bad_stride(k_stride, kv.Hkv, kv.D) || bad_stride(v_stride, kv.Hkv, kv.D)) return SFA_ERR_INVALID_ARG;
    if ((int64_t)num_tokens * kv.Hkv > 0x7fffffffLL / 2) return SFA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return SFA_OK;
    if (!k_new || !v_new || !al(k_new, 16) || !al(v_new, 16)) return SFA_ERR_INVALID_ARG;
    return launch_paged_append(kv, k_new, v_new, k_stride, v_stride, cu_seqlens, num_tokens, dtype,
                               reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SFA_OK : SFA_ERR_CUDA;
}

sfa_status paged_read(const paged_kv* cache, const int32_t* cu_seqlens, int num_tokens,
                      sfa_dtype dtype, void* k_out, void* v_out, sfa_stream_t stream) {
    SeqKV kv;
    sfa_status st = resolve_cache(cache, kv);
    if (st != SFA_OK) return st;
    if (num_tokens < 0 || !cu_seqlens || !al(cu_seqlens, 4) || !is16(dtype)) return SFA_ERR_INVALID_ARG;
    if (kv.f8 == 0 && dtype != cache->dtype) return SFA_ERR_INVALID_ARG;
    if ((int64_t)num_tokens * kv.Hkv > 0x7fffffffLL / 2) return SFA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return SFA_OK;
    if (!k_out || !v_out || !al(k_out, 16) || !al(v_out, 16)) return SFA_ERR_INVALID_ARG;
    return launch_paged_read(kv, cu_seqlens, num_tokens, dtype, k_out, v_out,
                             reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SFA_OK : SFA_ERR_CUDA;
}

sfa_status varlen_workspace_size(int num_seqs, int num_tokens, int num_qo_heads, int num_kv_heads,
                                 int head_dim, size_t* bytes) {
    if (!bytes || num_seqs < 1 || num_tokens < 0) return SFA_ERR_INVALID_ARG;
    sfa_status st = check_heads(num_qo_heads, num_kv_heads, head_dim);
    if (st != SFA_OK) return st;
    *bytes = attention_ws_bytes(num_qo_heads, num_kv_heads, head_dim);
    return SFA_OK;
}

sfa_status paged_workspace_size(int num_seqs, int num_tokens, int num_qo_heads, int num_kv_heads,
                                int head_dim, size_t* bytes) {
    return varlen_workspace_size(num_seqs, num_tokens, num_qo_heads, num_kv_heads, head_dim, bytes);
}

sfa_status paged_run(const paged_kv* cache, const void* q, int64_t q_stride,
                     const int32_t* cu_seqlens_q, int num_tokens, int num_qo_heads, int max_q_len,
                     float scale, int causal, sfa_dtype dtype, void* out, float* lse,
                     void* workspace, size_t workspace_bytes, sfa_stream_t stream) {
    SeqAttn p{};
    sfa_status st = resolve_cache(cache, p.kv);
    if (st != SFA_OK) return st;
    if (p.kv.f8 == 0 && dtype != cache->dtype) return SFA_ERR_INVALID_ARG;
    return run_attention(p, num_tokens, num_qo_heads, max_q_len, scale, causal, dtype, q, q_stride,
                         cu_seqlens_q, out, lse, workspace, workspace_bytes, stream);
}

sfa_status varlen_run(const void* q, const void* k, const void* v, int64_t q_stride,
                      int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens_q,
                      const int32_t* cu_seqlens_k, int num_seqs, int num_tokens, int num_keys,
                      int num_qo_heads, int num_kv_heads, int head_dim, int max_q_len, float scale,
                      int causal, sfa_dtype dtype, void* out, float* lse, void* workspace,
                      size_t workspace_bytes, sfa_stream_t stream) {
    if (num_seqs < 1 || num_keys < 0 || !cu_seqlens_k || !al(cu_seqlens_k, 4)) return SFA_ERR_INVALID_ARG;
    sfa_status st = check_heads(num_qo_heads, num_kv_heads, head_dim);
    if (st != SFA_OK) return st;
    if (bad_stride(k_stride, num_kv_heads, head_dim) || bad_stride(v_stride, num_kv_heads, head_dim))
        return SFA_ERR_INVALID_ARG;
    if (num_keys > 0x7fffffff / 2) return SFA_ERR_UNSUPPORTED;
    // with no key at all the (then unused) pointers may be NULL
    if (num_keys > 0 && (!k || !v || !al(k, 16) || !al(v, 16))) return SFA_ERR_INVALID_ARG;
    SeqAttn p{};
    p.kv.k = num_keys > 0 ? k : q;
    p.kv.v = num_keys > 0 ? v : q;
    p.kv.cu_k = cu_seqlens_k;
    p.kv.num_seqs = num_seqs;
    p.kv.rows = num_keys;
    p.kv.Hkv = num_kv_heads;
    p.kv.D = head_dim;
    p.kv.s_tok = k_stride;
    p.kv.sv_tok = v_stride;
    p.kv.s_head = p.kv.sv_head = head_dim;
    return run_attention(p, num_tokens, num_qo_heads, max_q_len, scale, causal, dtype, q, q_stride,
                         cu_seqlens_q, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
