// What the kernels that move rows into and out of a paged cache have in common:
// finding a row's place, rounding to 8-bit codes and back.
//
// Rounding to codes: x times the scale's rounded reciprocal is within 2 units
// in the last place of the quotient.  A border between two codes has 19 zero
// bits at the end (formats of at most 3 fraction bits), so a product whose
// last 19 bits are further than that from zero has the quotient's code.
// Where one of a thread's 16 is not, they are divided: the quotient rounded
// to fp32, and if that has 19 zeros, the exact remainder x - q * scale (one
// fma) tells on which side the true quotient lies, and q moves off the border
// by one unit in that direction.  So the code is always that of the exact
// quotient, for 5 instructions an element instead of about 18 (which took
// longer than the memory did).  A power of two divides exactly.
#pragma once

#include "common.cuh"
#include "paged.h"

namespace sfa {
namespace {

// Number of entries of cu[1 .. B] that are <= t: the sequence holding row t
// (B if it is past the last).  The whole warp takes part; t is uniform.
__device__ __forceinline__ int find_seq(const int32_t* cu, int B, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int i = lo + (lane + 1) * step - 1;
        const bool below = i < lo + n && cu[1 + i] <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, below));
        const int left = n - c * step;
        lo += c * step;
        n = min(step - 1, left);
        if (n < 0) n = 0;
    }
    return min(lo, B);
}

// Element offset of token row t's place (head 0) in the pools, or -1.  Lists
// are read as attention reads them (seq_rows, seq_keys), so that a row is the
// same token to both.
__device__ __forceinline__ int64_t place_of(const SeqKV& kv, const int32_t* cu, int b, int t, int tokens) {
    if (b >= kv.num_seqs || t < cu[b]) return -1;
    const int pos = seq_keys(kv, b).y - (seq_rows(cu, b, tokens).y - t);
    if (pos < 0) return -1;
    const int slot = over(pos, kv.by_page);
    const int page = kv.page_table[(int64_t)b * kv.max_pages + slot];
    if ((unsigned)page >= (unsigned)kv.num_pages) return -1;
    return page * kv.s_page + (pos - slot * kv.page_size) * kv.s_tok;
}

__device__ __forceinline__ float quotient(float x, float s) {
    float q = __fdiv_rn(x, s);
    if ((__float_as_uint(q) & 0x7ffffu) == 0u) {
        // Exact; its sign is the true quotient's side (s > 0).  (Of a small scale and its value
        // both times 2^64, that the remainder is not below the smallest number.)
        const float up = s < 5.4210109e-20f ? 18446744073709551616.f : 1.f;
        const float r = fmaf(-q, s * up, x * up);
        if (r != 0.f && q != 0.f && isfinite(q))
            q = __uint_as_float(__float_as_uint(q) + (((r > 0.f) == (q > 0.f)) ? 1u : ~0u));
    }
    return q;
}

// Eight values as the nearest codes.
template <bool E5>
__device__ __forceinline__ uint2 codes8(const float (&q)[8]) {
    return make_uint2(f8_pack2<E5>(q[0], q[1]) | (f8_pack2<E5>(q[2], q[3]) << 16),
                      f8_pack2<E5>(q[4], q[5]) | (f8_pack2<E5>(q[6], q[7]) << 16));
}
// Codes of eight values' quotients.
template <bool E5>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float s, float inv) {
    float q[8];
    const bool normal = inv >= 1.1754944e-38f && inv < INFINITY;
    bool near = !normal;                     // (a reciprocal out of the normal range is less exact)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = x[i] * inv;
        near |= ((__float_as_uint(q[i]) + 2u) & 0x7ffffu) <= 4u;
    }
    // an exact reciprocal (a power of two, normal) gives exact quotients
    if (near && ((__float_as_uint(s) & 0x7fffffu) != 0u || !normal)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = quotient(x[i], s);
    }
    return codes8<E5>(q);
}
template <class E>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = E::unpack2(in[i]);
        x[2 * i] = a.x;
        x[2 * i + 1] = a.y;
    }
}
template <class E, bool E5>
__device__ __forceinline__ uint2 encode8(uint4 v, float s, float inv) {
    float x[8];
    unpack8<E>(v, x);
    return encode8<E5>(x, s, inv);
}
template <class E, bool E5>
__device__ __forceinline__ uint4 encode16(const uint4 (&x)[2], float s, float inv) {
    const uint2 lo = encode8<E, E5>(x[0], s, inv), hi = encode8<E, E5>(x[1], s, inv);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

template <class E, bool E5>
__device__ __forceinline__ void decode16(uint4 c, float s, uint4 (&y)[2]) {
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = f8_unpack2<E5>(in[i] & 0xffffu), b = f8_unpack2<E5>(in[i] >> 16);
        o[2 * i] = E::pack2(a.x * s, a.y * s);
        o[2 * i + 1] = E::pack2(b.x * s, b.y * s);
    }
    y[0] = make_uint4(o[0], o[1], o[2], o[3]);
    y[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace
}  // namespace sfa
