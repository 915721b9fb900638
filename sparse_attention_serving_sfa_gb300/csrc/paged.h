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
};

// Row-tile path (16 rows of one kv head per tile, warp MMAs): any page size
// and group size.
size_t attn_rows_ws_bytes(int D);
cudaError_t launch_attn_rows(const SeqAttn& p, sfa_dtype dtype, int num_sms, cudaStream_t stream);

// Tensor-core path (two tiles of 128 rows of one kv head per CTA): groups of
// up to 128 heads, packed rows or pages of any size.
bool attn_tc_supported(const SeqKV& kv, int G);
size_t attn_tc_ws_bytes(int G, int D);
cudaError_t launch_attn_tc(const SeqAttn& p, sfa_dtype dtype, int num_sms, cudaStream_t stream);

cudaError_t launch_paged_append(const SeqKV& kv, const void* k_new, const void* v_new,
                                int64_t k_stride, int64_t v_stride, const int32_t* cu, int tokens,
                                sfa_dtype dtype, cudaStream_t stream);
cudaError_t launch_paged_read(const SeqKV& kv, const int32_t* cu, int tokens, sfa_dtype dtype,
                              void* k_out, void* v_out, cudaStream_t stream);

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
#endif

}  // namespace sfa
