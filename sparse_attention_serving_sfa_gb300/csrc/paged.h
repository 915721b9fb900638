// Internal interface of the paged KV cache and of dense attention over it and
// over packed rows.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sfa.h"

namespace sfa {

// x / d = x * mul >> shift for 0 <= x < 2^31 (the multiplier rounded up at
// 2^(31 + ceil(log2 d))): a division takes a few hundred cycles of a call's
// first look-ups, this a few.
struct Divisor {
    uint32_t mul;
    int shift;
};
inline Divisor divide_by(uint32_t d) {
    int up = 0;
    while (((uint64_t)1 << up) < d) ++up;
    return {(uint32_t)((((uint64_t)1 << (31 + up)) + d - 1) / d), 31 + up};
}

// Keys and values of a batch of sequences.  Token j of sequence b lies
//   paged  (page_table set): in page page_table[b][j / page_size], place
//          j % page_size, kv_lens[b] tokens in all;
//   packed (page_table NULL): in row cu_k[b] + j, cu_k[b + 1] - cu_k[b] in all.
// Element (page, place, head, dim) is at page * s_page + place * s_tok +
// head * s_head + dim (packed: page 0, place = row).  What the device arrays
// hold is never trusted: lengths and rows are clamped to the sizes given here
// and tokens of a page outside [0, num_pages) count as absent.
struct SeqKV {
    const void* k;
    const void* v;
    const int32_t* page_table;   // [num_seqs][max_pages]
    const int32_t* kv_lens;      // [num_seqs]
    const int32_t* cu_k;         // [num_seqs + 1]
    int num_seqs, num_pages, page_size, max_pages, rows;   // rows: packed rows of k / v
    int Hkv, D;
    Divisor by_page;                 // page_size
    int64_t s_page, s_tok, s_head;   // of k, and of v when paged
    int64_t sv_tok, sv_head;         // of v when packed
    int f8;                          // 0: 16-bit, 1: E4M3, 2: E5M2
    const float* scale_k;            // [Hkv] or NULL (= 1)
    const float* scale_v;
};

// What attention over parts of the keys takes besides: a row at position p sees
// keys lo <= j < lim and j < min(sinks, lim), lim as without (the sequence's
// length, causally p + 1) and
//     lo = max(first, p - window + 1)        (no window: first),
// first = 0, or behind a shared prefix its length.
// A call with shared prefixes runs twice.  PREFIX: the line's sequences are the
// groups, whose rows are those of all sequences of the group and whose keys are the
// first shared_lens[g] of its first sequence, all visible; results stay
// unnormalised in px_o and px_ml, a row a row.  OWN: each sequence's rows over its
// keys from `first` on, joined with those results at the end.  Or, where there is
// little to share, once (DIRECT, few rows only): each sequence's rows over the shared
// keys, from the pages of the group's first sequence, and its own.
enum { PHASE_ALL = 0, PHASE_PREFIX = 1, PHASE_OWN = 2, PHASE_DIRECT = 3 };
struct KeyParts {
    int phase;
    int once;                    // loads of keys leave L2 first: the pass reads each about once (no
                                 // matter where the tensor-core kernel gathers pages row by row)
    int window, sinks;           // at most 2^30; window 2^30: none
    const int32_t* cu_shared;    // [groups + 1]: group g is sequences cu_shared[g] .. cu_shared[g + 1] - 1
    const int32_t* shared_lens;  // [groups]
    int groups;
    float* px_o;                 // [tokens][Hq][D] unnormalised
    float* px_ml;                // [tokens][Hq][2] (m in log2 units, sum)
};

// One attention call over SeqKV.
struct SeqAttn {
    SeqKV kv;
    const void* q;               // row t, head h at t * q_stride + h * D
    void* out;                   // [tokens][Hq][D]
    float* lse;                  // [tokens][Hq] or NULL
    const int32_t* cu_q;         // [num_seqs + 1]
    int tokens, Hq, G, causal, max_q_len;
    int64_t q_stride;
    float scale_log2;            // scale * log2(e)
    Divisor by_group, by_heads;  // G, kv heads
    void* ws;                    // attn_rows_ws_bytes() / attn_tc_ws_bytes() bytes
    int* err_word;
    KeyParts parts;
};

// Items of a prefixes' pass on the tensor-core path, at most (G up to 128).
inline int64_t tc_prefix_items(const SeqAttn& p) {
    return ((int64_t)p.tokens / (2 * (128 / p.G)) + p.parts.groups) * p.kv.Hkv;
}

// Row-tile path (16 rows of one kv head per tile, warp MMAs): any page size
// and group size.
size_t attn_rows_ws_bytes(int D);
cudaError_t launch_attn_rows(const SeqAttn& p, sfa_dtype dtype, int num_sms, cudaStream_t stream);
// the same over parts of the keys (SeqAttn::parts)
cudaError_t launch_attn_rows_parts(const SeqAttn& p, sfa_dtype dtype, int num_sms, cudaStream_t stream);

// Tensor-core path (two tiles of 128 rows of one kv head per CTA): groups of
// up to 128 heads, packed rows or pages of any size.
bool attn_tc_supported(const SeqKV& kv, int G);
size_t attn_tc_ws_bytes(int G, int D);
cudaError_t launch_attn_tc(const SeqAttn& p, sfa_dtype dtype, int num_sms, cudaStream_t stream);
cudaError_t launch_attn_tc_parts(const SeqAttn& p, sfa_dtype dtype, int num_sms, cudaStream_t stream);

cudaError_t launch_paged_append(const SeqKV& kv, const void* k_new, const void* v_new,
                                int64_t k_stride, int64_t v_stride, const int32_t* cu, int tokens,
                                sfa_dtype dtype, cudaStream_t stream);
cudaError_t launch_paged_read(const SeqKV& kv, const int32_t* cu, int tokens, sfa_dtype dtype,
                              void* k_out, void* v_out, cudaStream_t stream);

// One append with rotation.
struct RotateAppend {
    SeqKV kv;
    const void* q;               // NULL: Hq = 0
    const void* k;
    const void* v;
    void* q_out;
    int64_t q_stride, q_out_stride, k_stride, v_stride;
    const int32_t* cu;
    const float* inv_freq;       // [rotary / 2]
    int tokens, Hq, rotary, interleaved;
    int block_tokens;            // tokens of a block
    Divisor by_heads;            // heads of a token: queries, keys, values
};
cudaError_t launch_paged_rotate(RotateAppend p, sfa_dtype dtype, cudaStream_t stream);

#ifdef __CUDACC__
__device__ __forceinline__ int over(int x, Divisor d) { return (int)(((uint64_t)(uint32_t)x * d.mul) >> d.shift); }
// Rows [first, last) of sequence b in packed rows described by cu, clamped to
// [0, rows].
__device__ __forceinline__ int2 seq_rows(const int32_t* cu, int b, int rows) {
    const int lo = min(max(cu[b], 0), rows);
    return make_int2(lo, min(max(cu[b + 1], lo), rows));
}
// Tokens of sequence b, and its first packed row (0 when paged).
__device__ __forceinline__ int2 seq_keys(const SeqKV& kv, int b) {
    if (kv.page_table)
        return make_int2(0, (int)min((int64_t)max(kv.kv_lens[b], 0), (int64_t)kv.max_pages * kv.page_size));
    const int2 r = seq_rows(kv.cu_k, b, kv.rows);
    return make_int2(r.x, r.y - r.x);
}

// Sequence b of the line of a call: its rows [q_row, q_row + n_q) and keys (k_row and
// kv_len as seq_keys).  With parts: its rows see none before `first`; the pages of the
// first `shared` are in row `table` of the page table, and all rows see those.
struct LineSeq {
    int q_row, n_q, k_row, kv_len, first, shared, table;
};
template <bool PARTS>
__device__ __forceinline__ int line_seqs(const SeqAttn& p) {
    return PARTS && p.parts.phase == PHASE_PREFIX ? p.parts.groups : p.kv.num_seqs;
}
template <bool PARTS>
__device__ __forceinline__ LineSeq line_seq(const SeqAttn& p, int b) {
    LineSeq s;
    s.first = s.shared = 0;
    s.table = b;
    const KeyParts& x = p.parts;
    if (PARTS && x.phase == PHASE_PREFIX) {
        const int2 in = seq_rows(x.cu_shared, b, p.kv.num_seqs);
        s.table = min(in.x, p.kv.num_seqs - 1);
        s.q_row = min(max(p.cu_q[in.x], 0), p.tokens);
        s.n_q = in.x < in.y ? min(max(p.cu_q[in.y], s.q_row), p.tokens) - s.q_row : 0;
        s.k_row = 0;
        s.kv_len = s.shared = (int)min((int64_t)max(x.shared_lens[b], 0), (int64_t)p.kv.max_pages * p.kv.page_size);
        return s;
    }
    const int2 q = seq_rows(p.cu_q, b, p.tokens);
    const int2 k = seq_keys(p.kv, b);
    s.q_row = q.x;
    s.n_q = q.y - q.x;
    s.k_row = k.x;
    s.kv_len = k.y;
    if (PARTS && x.phase >= PHASE_OWN) {
        // its group: the last that begins at or before b
        int lo = 0, hi = x.groups;                       // lo: cu_shared[1 .. lo] <= b
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (x.cu_shared[mid + 1] <= b) lo = mid + 1;
            else hi = mid;
        }
        if (lo < x.groups && x.cu_shared[lo] <= b) {
            s.first = (int)min((int64_t)max(x.shared_lens[lo], 0), (int64_t)p.kv.max_pages * p.kv.page_size);
            if (x.phase == PHASE_DIRECT) {
                s.shared = s.first;
                s.first = 0;
                s.kv_len = max(s.kv_len, s.shared);
                s.table = max(x.cu_shared[lo], 0);
            }
        }
    }
    return s;
}
#endif

}  // namespace sfa
