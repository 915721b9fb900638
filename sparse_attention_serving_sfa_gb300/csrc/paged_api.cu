// C ABI of the paged KV cache (paged_append, paged_append_rotated, paged_read), of
// dense attention over it (paged_run, paged_run_window, paged_run_shared) and over
// packed rows (varlen_run, varlen_run_window): argument checks, layout -> stride
// resolution, choice of path.
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

// Rows of one call, `width` elements of 16 bits each.
struct Rows {
    const void* at;
    int64_t stride;
    int64_t width;
};

// Whether `n` rows of x and of y have an element in common.
bool rows_meet(Rows x, Rows y, int64_t n) {
    // y's first element counted from x's (both begin at 16 bytes)
    const int64_t d = (int64_t)(reinterpret_cast<intptr_t>(y.at) - reinterpret_cast<intptr_t>(x.at)) / 2;
    if (d >= (n - 1) * x.stride + x.width || -d >= (n - 1) * y.stride + y.width) return false;
    if (x.stride == y.stride) {
        // row j of y lies d + (j - i) stride behind row i of x: a row or two nearest to it
        for (int64_t t = -d / x.stride - 1; t <= -d / x.stride + 1; ++t) {
            const int64_t off = d + t * x.stride;
            if (t > -n && t < n && off < x.width && -off < y.width) return true;
        }
        return false;
    }
    for (int64_t i = 0; i < n; ++i) {
        // the first row of y that ends behind the beginning of row i of x
        const int64_t from = i * x.stride - d;               // counted from y's first element
        const int64_t j = from < y.width ? 0 : (from - y.width) / y.stride + 1;
        if (j < n && j * y.stride < from + x.width) return true;
    }
    return false;
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
bool few_rows(int64_t rows, int64_t tiles, int64_t keys, bool f8) {
    return rows <= (f8 ? 32 : 16) || (tiles <= (f8 ? 128 : 64) && tiles * keys <= (f8 ? 524288 : 196608));
}

// Keys that the longest sequence can have (below 2^30).
int64_t most_keys(const SeqKV& kv) { return kv.page_table ? (int64_t)kv.max_pages * kv.page_size : kv.rows; }

// The same for a call as described.  (The lengths are on the device; what counts is
// what the table or the packed rows can hold and a window can show.)
bool few_rows(const SeqAttn& p) {
    int64_t keys = most_keys(p.kv);
    int64_t rows = (int64_t)p.max_q_len * p.G, seqs = p.kv.num_seqs;
    if (p.parts.phase == PHASE_PREFIX) {
        // all rows of a group are one sequence's
        rows = (int64_t)p.tokens * p.G;
        return few_rows(rows, ((rows + 15) / 16 + p.parts.groups - 1) * p.kv.Hkv, keys, p.kv.f8 != 0);
    }
    const int64_t seen = (int64_t)p.parts.window + p.parts.sinks + p.max_q_len;
    if (p.parts.window > 0 && seen < keys) keys = seen;
    return few_rows(rows, (rows + 15) / 16 * seqs * p.kv.Hkv, keys, p.kv.f8 != 0);
}

// Workspace of either path.
size_t attention_ws_bytes(int Hq, int Hkv, int D) {
    const size_t r = attn_rows_ws_bytes(D), t = attn_tc_ws_bytes(Hq / Hkv, D);
    return r > t ? r : t;
}

// A call's arguments besides keys and values.
struct Call {
    const void* q;
    int64_t q_stride;
    const int32_t* cu_q;
    int tokens, Hq, max_q_len;
    float scale;
    int causal;
    sfa_dtype dtype;
    void* out;
    float* lse;
    void* ws;
    size_t ws_bytes;
    sfa_stream_t stream;
};

// Checks a call and fills `p` (its keys are filled); `need` bytes of workspace.
// Nothing is to be done if there are no rows.
sfa_status resolve_call(SeqAttn& p, const Call& c, size_t need) {
    if (c.tokens < 0 || c.max_q_len < 0 || !c.cu_q || !al(c.cu_q, 4)) return SFA_ERR_INVALID_ARG;
    sfa_status st = check_heads(c.Hq, p.kv.Hkv, p.kv.D);
    if (st != SFA_OK) return st;
    if (!is16(c.dtype) || !isfinite(c.scale)) return SFA_ERR_INVALID_ARG;
    if (bad_stride(c.q_stride, c.Hq, p.kv.D)) return SFA_ERR_INVALID_ARG;
    if ((int64_t)c.tokens * c.Hq > 0x7fffffffLL / 2) return SFA_ERR_UNSUPPORTED;
    if (c.tokens == 0) return SFA_OK;
    if (!c.q || !c.out || !al(c.q, 16) || !al(c.out, 16) || !al(c.lse, 4)) return SFA_ERR_INVALID_ARG;
    if (!c.ws || c.ws_bytes < need) return SFA_ERR_WORKSPACE;
    if (!al(c.ws, 16)) return SFA_ERR_INVALID_ARG;
    p.q = c.q; p.out = c.out; p.lse = c.lse; p.cu_q = c.cu_q;
    p.tokens = c.tokens; p.Hq = c.Hq; p.G = c.Hq / p.kv.Hkv;
    p.causal = c.causal ? 1 : 0;
    p.max_q_len = c.max_q_len > 0 && c.max_q_len < c.tokens ? c.max_q_len : c.tokens;
    p.q_stride = c.q_stride;
    p.scale_log2 = (c.scale > 0.f ? c.scale : 1.0f / sqrtf((float)p.kv.D)) * kLog2e;
    p.by_group = divide_by(p.G);
    p.by_heads = divide_by(p.kv.Hkv);
    p.ws = c.ws;
    return SFA_OK;
}

// Whether the keys of a call's pass leave L2 first (KeyParts::once): in the two passes
// of 16-row tiles, and on the tensor cores in the prefixes' where its items are fewer
// than SMs.  Then each key is read once, or by a few items next to one another.  32/8
// heads of 128, us with and without: 64 requests behind 16,384 tokens (one item a kv
// head) 57 and 65; 300 behind them (5 items) and 300 own tokens each 160 and 167, and
// 2,000 own 484 and 477; 200 behind 60,000 241 and 248.  40 requests of 16 heads behind
// 4,900, one kv head (40 16-row tiles), 33.7 and 33.7.
bool leaves_l2_first(const SeqAttn& p, bool tc) {
    if (p.parts.phase == PHASE_PREFIX) return !tc || tc_prefix_items(p) < num_sms();
    return p.parts.phase == PHASE_OWN && !tc;
}

// One pass of a resolved call; `parts`: over parts of the keys.
sfa_status launch_attention(SeqAttn& p, bool parts, const Call& c) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(c.stream);
    cudaError_t err;
    const bool tc = !few_rows(p) && attn_tc_supported(p.kv, p.G);
    p.parts.once = leaves_l2_first(p, tc);
    if (tc) {
        p.err_word = device_error_word();
        if (!p.err_word) return SFA_ERR_CUDA;
        err = parts ? launch_attn_tc_parts(p, c.dtype, num_sms(), s) : launch_attn_tc(p, c.dtype, num_sms(), s);
    } else {
        err = parts ? launch_attn_rows_parts(p, c.dtype, num_sms(), s) : launch_attn_rows(p, c.dtype, num_sms(), s);
    }
    return err == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

sfa_status launch_rows_parts(const SeqAttn& p, const Call& c) {
    const cudaError_t err = launch_attn_rows_parts(p, c.dtype, num_sms(), reinterpret_cast<cudaStream_t>(c.stream));
    return err == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
}

// Packed keys and values as `kv`.
sfa_status resolve_packed(SeqKV& kv, const void* q, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                          const int32_t* cu_seqlens_k, int num_seqs, int num_keys, int Hq, int Hkv, int D) {
    if (num_seqs < 1 || num_keys < 0 || !cu_seqlens_k || !al(cu_seqlens_k, 4)) return SFA_ERR_INVALID_ARG;
    sfa_status st = check_heads(Hq, Hkv, D);
    if (st != SFA_OK) return st;
    if (bad_stride(k_stride, Hkv, D) || bad_stride(v_stride, Hkv, D)) return SFA_ERR_INVALID_ARG;
    if (num_keys > 0x7fffffff / 2) return SFA_ERR_UNSUPPORTED;
    // with no key at all the (then unused) pointers may be NULL
    if (num_keys > 0 && (!k || !v || !al(k, 16) || !al(v, 16))) return SFA_ERR_INVALID_ARG;
    kv.k = num_keys > 0 ? k : q;
    kv.v = num_keys > 0 ? v : q;
    kv.cu_k = cu_seqlens_k;
    kv.num_seqs = num_seqs;
    kv.rows = num_keys;
    kv.Hkv = Hkv;
    kv.D = D;
    kv.s_tok = k_stride;
    kv.sv_tok = v_stride;
    kv.s_head = kv.sv_head = D;
    return SFA_OK;
}

constexpr int kNoWindow = 1 << 30;     // (no position is larger)

// The pass over all keys, or through a window.
sfa_status run_attention(SeqAttn& p, const Call& c, int window, int sinks) {
    sfa_status st = resolve_call(p, c, attention_ws_bytes(c.Hq, p.kv.Hkv, p.kv.D));
    if (st != SFA_OK || c.tokens == 0) return st;
    // (nothing lies between the two where they reach over all that the call can hold)
    if (window == 0 || (int64_t)window + sinks >= most_keys(p.kv)) return launch_attention(p, false, c);
    p.parts.window = window;
    p.parts.sinks = sinks;
    return launch_attention(p, true, c);
}

// Where every sequence reading the shared keys for itself moves no more than this (by
// what the table can hold, and few rows each), one pass over all keys is faster than
// two passes and their joins.  Two passes and one, us: 8 sequences behind 500 keys (20
// MB) 15.1 and 9.8, behind 2,000 (66 MB) 17.0 and 14.4, behind 8,000 (254 MB) 22.8 and
// 35.7; 16 behind 2,000 (133 MB) 19.4 and 21.5; 32 behind 500 (80 MB) 18.9 and 17.8,
// behind 2,000 (266 MB) 24.7 and 36.4; E4M3, 8 behind 8,000 (127 MB) 26.4 and 27.3, 32
// behind 1,000 (71 MB) 23.0 and 21.5; 2 kv heads, 8 behind 4,000 (32 MB) 17.8 and 11.8.
// (Tables as wide as the sequences.  One with room for 32,768 tokens counts as that much:
// 5 behind 1,500 take two passes then, 22.2 us instead of 11.2.)
constexpr int64_t kDirectBytes = 96 << 20;
int64_t direct_bytes(const SeqAttn& p) {
    return p.kv.num_seqs * most_keys(p.kv) * p.kv.Hkv * p.kv.D * (p.kv.f8 ? 2 : 4);
}

// Results of a shared prefix's pass, behind the workspace of a pass.
size_t prefix_bytes(int64_t tokens, int Hq, int D) { return (size_t)tokens * Hq * (D + 2) * 4; }

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

sfa_status paged_append_rotated(const paged_kv* cache, const void* q, const void* k_new, const void* v_new,
                                void* q_out, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                int64_t q_out_stride, const int32_t* cu_seqlens, int num_tokens,
                                int num_qo_heads, const float* inv_freq, int rotary_dim, int interleaved,
                                sfa_dtype dtype, sfa_stream_t stream) {
    RotateAppend p{};
    sfa_status st = resolve_cache(cache, p.kv);
    if (st != SFA_OK) return st;
    if (num_tokens < 0 || !cu_seqlens || !al(cu_seqlens, 4) || !is16(dtype)) return SFA_ERR_INVALID_ARG;
    if (p.kv.f8 == 0 && dtype != cache->dtype) return SFA_ERR_INVALID_ARG;
    if (!inv_freq || !al(inv_freq, 4) || rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > p.kv.D)
        return SFA_ERR_INVALID_ARG;
    if (rotary_dim % 16 != 0) return SFA_ERR_UNSUPPORTED;
    if (bad_stride(k_stride, p.kv.Hkv, p.kv.D) || bad_stride(v_stride, p.kv.Hkv, p.kv.D)) return SFA_ERR_INVALID_ARG;
    if (q && (num_qo_heads < 1 || bad_stride(q_stride, num_qo_heads, p.kv.D) ||
              bad_stride(q_out_stride, num_qo_heads, p.kv.D)))
        return SFA_ERR_INVALID_ARG;
    p.Hq = q ? num_qo_heads : 0;
    // 16-element pieces of the call, and of a block's tokens, are counted in 31 bits
    if (((int64_t)p.Hq + 2LL * p.kv.Hkv) > (1 << 20) ||
        (int64_t)num_tokens * ((int64_t)p.Hq + 2LL * p.kv.Hkv) > 0x7fffffffLL / 2)
        return SFA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return SFA_OK;
    if (!k_new || !v_new || !al(k_new, 16) || !al(v_new, 16)) return SFA_ERR_INVALID_ARG;
    if (q && (!q_out || !al(q, 16) || !al(q_out, 16))) return SFA_ERR_INVALID_ARG;
    if (q) {
        // in place, or over no row that is still to be read
        const Rows to{q_out, q_out_stride, (int64_t)num_qo_heads * p.kv.D}, from{q, q_stride, to.width};
        const Rows k{k_new, k_stride, (int64_t)p.kv.Hkv * p.kv.D}, v{v_new, v_stride, k.width};
        const bool in_place = q_out == q && (q_out_stride == q_stride || num_tokens == 1);
        if ((!in_place && rows_meet(to, from, num_tokens)) || rows_meet(to, k, num_tokens) || rows_meet(to, v, num_tokens))
            return SFA_ERR_INVALID_ARG;
    }
    p.q = q; p.k = k_new; p.v = v_new; p.q_out = q_out;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride; p.q_out_stride = q_out_stride;
    p.cu = cu_seqlens;
    p.inv_freq = inv_freq;
    p.tokens = num_tokens;
    p.rotary = rotary_dim;
    p.interleaved = interleaved ? 1 : 0;
    return launch_paged_rotate(p, dtype, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SFA_OK : SFA_ERR_CUDA;
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

sfa_status paged_shared_workspace_size(int num_seqs, int num_tokens, int num_qo_heads, int num_kv_heads,
                                       int head_dim, size_t* bytes) {
    sfa_status st = varlen_workspace_size(num_seqs, num_tokens, num_qo_heads, num_kv_heads, head_dim, bytes);
    if (st != SFA_OK) return st;
    if ((int64_t)num_tokens * num_qo_heads > 0x7fffffffLL / 2) return SFA_ERR_UNSUPPORTED;
    *bytes += prefix_bytes(num_tokens, num_qo_heads, head_dim);
    return SFA_OK;
}

sfa_status paged_run(const paged_kv* cache, const void* q, int64_t q_stride,
                     const int32_t* cu_seqlens_q, int num_tokens, int num_qo_heads, int max_q_len,
                     float scale, int causal, sfa_dtype dtype, void* out, float* lse,
                     void* workspace, size_t workspace_bytes, sfa_stream_t stream) {
    SeqAttn p{};
    sfa_status st = resolve_cache(cache, p.kv);
    if (st != SFA_OK) return st;
    if (p.kv.f8 == 0 && dtype != cache->dtype) return SFA_ERR_INVALID_ARG;
    return run_attention(p, Call{q, q_stride, cu_seqlens_q, num_tokens, num_qo_heads, max_q_len, scale, causal, dtype, out,
                                 lse, workspace, workspace_bytes, stream}, 0, 0);
}

sfa_status paged_run_window(const paged_kv* cache, const void* q, int64_t q_stride,
                            const int32_t* cu_seqlens_q, int num_tokens, int num_qo_heads, int max_q_len,
                            int window, int sinks, float scale, sfa_dtype dtype, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, sfa_stream_t stream) {
    SeqAttn p{};
    sfa_status st = resolve_cache(cache, p.kv);
    if (st != SFA_OK) return st;
    if (window < 1 || sinks < 0) return SFA_ERR_INVALID_ARG;
    if (p.kv.f8 == 0 && dtype != cache->dtype) return SFA_ERR_INVALID_ARG;
    return run_attention(p, Call{q, q_stride, cu_seqlens_q, num_tokens, num_qo_heads, max_q_len, scale, 1, dtype, out, lse,
                                 workspace, workspace_bytes, stream}, window, sinks);
}

sfa_status paged_run_shared(const paged_kv* cache, const void* q, int64_t q_stride,
                            const int32_t* cu_seqlens_q, int num_tokens, int num_qo_heads, int max_q_len,
                            const int32_t* cu_shared, const int32_t* shared_lens, int num_groups,
                            float scale, int causal, sfa_dtype dtype, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, sfa_stream_t stream) {
    SeqAttn p{};
    sfa_status st = resolve_cache(cache, p.kv);
    if (st != SFA_OK) return st;
    if (num_groups < 1 || !cu_shared || !shared_lens || !al(cu_shared, 4) || !al(shared_lens, 4)) return SFA_ERR_INVALID_ARG;
    if (p.kv.f8 == 0 && dtype != cache->dtype) return SFA_ERR_INVALID_ARG;
    const Call c{q, q_stride, cu_seqlens_q, num_tokens, num_qo_heads, max_q_len, scale, causal, dtype, out, lse, workspace,
                 workspace_bytes, stream};
    const size_t pass = attention_ws_bytes(num_qo_heads, p.kv.Hkv, p.kv.D);
    st = resolve_call(p, c, pass + prefix_bytes(num_tokens, num_qo_heads, p.kv.D));
    if (st != SFA_OK || num_tokens == 0) return st;
    p.parts.cu_shared = cu_shared;
    p.parts.shared_lens = shared_lens;
    p.parts.groups = num_groups;
    p.parts.window = kNoWindow;
    p.parts.px_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + pass);
    p.parts.px_ml = p.parts.px_o + (int64_t)num_tokens * num_qo_heads * p.kv.D;
    p.parts.phase = PHASE_DIRECT;
    if (few_rows(p) && (int64_t)direct_bytes(p) <= kDirectBytes) return launch_rows_parts(p, c);
    SeqAttn prefix = p;
    prefix.parts.phase = PHASE_PREFIX;
    prefix.causal = 0;
    prefix.max_q_len = num_tokens;
    st = launch_attention(prefix, true, c);
    if (st != SFA_OK) return st;
    p.parts.phase = PHASE_OWN;
    return launch_attention(p, true, c);
}

sfa_status varlen_run(const void* q, const void* k, const void* v, int64_t q_stride,
                      int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens_q,
                      const int32_t* cu_seqlens_k, int num_seqs, int num_tokens, int num_keys,
                      int num_qo_heads, int num_kv_heads, int head_dim, int max_q_len, float scale,
                      int causal, sfa_dtype dtype, void* out, float* lse, void* workspace,
                      size_t workspace_bytes, sfa_stream_t stream) {
    SeqAttn p{};
    sfa_status st = resolve_packed(p.kv, q, k, v, k_stride, v_stride, cu_seqlens_k, num_seqs, num_keys, num_qo_heads,
                                   num_kv_heads, head_dim);
    if (st != SFA_OK) return st;
    return run_attention(p, Call{q, q_stride, cu_seqlens_q, num_tokens, num_qo_heads, max_q_len, scale, causal, dtype, out,
                                 lse, workspace, workspace_bytes, stream}, 0, 0);
}

sfa_status varlen_run_window(const void* q, const void* k, const void* v, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens_q,
                             const int32_t* cu_seqlens_k, int num_seqs, int num_tokens, int num_keys,
                             int num_qo_heads, int num_kv_heads, int head_dim, int max_q_len, int window,
                             int sinks, float scale, sfa_dtype dtype, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, sfa_stream_t stream) {
    if (window < 1 || sinks < 0) return SFA_ERR_INVALID_ARG;
    SeqAttn p{};
    sfa_status st = resolve_packed(p.kv, q, k, v, k_stride, v_stride, cu_seqlens_k, num_seqs, num_keys, num_qo_heads,
                                   num_kv_heads, head_dim);
    if (st != SFA_OK) return st;
    return run_attention(p, Call{q, q_stride, cu_seqlens_q, num_tokens, num_qo_heads, max_q_len, scale, 1, dtype, out, lse,
                                 workspace, workspace_bytes, stream}, window, sinks);
}

}  // extern "C"
