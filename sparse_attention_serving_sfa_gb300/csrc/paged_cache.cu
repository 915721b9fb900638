// Writing a paged KV cache and reading it back.
//
// append: row t of sequence b (cu[b] <= t < cu[b + 1]) is token
//     pos = kv_lens[b] - (cu[b + 1] - t)       (lists clamped to the sizes given)
// and goes to page page_table[b][pos / P], place pos % P, either as it is or as
//     code = sat(rne(x / scale[head]))           (E4M3 / E5M2);
// read: x = code * scale[head] in fp32, rounded to 16 bits.  Both move every
// element once (read 2 bytes, write 1 or 2 per element of K and of V).  A thread moves 16 consecutive elements of a head's row of K and of V
// (two 16-byte loads each, and one 16-byte store each for 8-bit codes), so a
// warp covers 512 elements of a token and the loads of K and V are in flight
// together.  (Two pieces a thread, of one token or of several, and pieces of 8
// elements measured slower on most calls: 47.4 -> 50.6 and 54.9 us for 261 MB
// read back.)  The sequence of a warp's first token is found by a 32-way search
// of cu (one load per factor of 32 in the number of sequences), then each lane
// walks to its own token's.  Measured: 261 MB read back from E4M3 pages 48 to
// 49 us (5.3 to 5.4 TB/s, 0.79 to 0.80 of the measured copy rate), bound by HBM;
// 12,800 tokens of 8 heads of 128 quantised into E4M3 pages 16.2 to 16.5 us (4.8
// TB/s; 17.9 at half the warps an SM), bound by nothing alone: issue slots 68%
// and the ALUs 60% busy, HBM 39%, half the warps waiting for memory; 12,500 of 4
// heads of 64 copied into 24-token pages 6.2 us (from and into L2); a decode
// step's 64 tokens 2.9 to 3.1 us, a launch's latency.
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
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "ptx.cuh"

namespace sfa {
namespace {

constexpr int kThreads = 128;   // (256: a decode step 0.1 us longer)
constexpr int kVec = 16;   // elements of a thread's piece

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
        const float r = fmaf(-q, s, x);      // exact; its sign is the true quotient's side (s > 0)
        if (r != 0.f && q != 0.f && isfinite(q))
            q = __uint_as_float(__float_as_uint(q) + (((r > 0.f) == (q > 0.f)) ? 1u : ~0u));
    }
    return q;
}

template <class E, bool E5>
__device__ __forceinline__ uint2 encode8(uint4 x, float s, float inv) {
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    float q[8];
    const bool normal = inv >= 1.1754944e-38f && inv < INFINITY;
    bool near = !normal;                     // (a reciprocal out of the normal range is less exact)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = E::unpack2(in[i]);
        q[2 * i] = a.x * inv;
        q[2 * i + 1] = a.y * inv;
        near |= ((__float_as_uint(q[2 * i]) + 2u) & 0x7ffffu) <= 4u;
        near |= ((__float_as_uint(q[2 * i + 1]) + 2u) & 0x7ffffu) <= 4u;
    }
    // an exact reciprocal (a power of two, normal) gives exact quotients
    if (near && ((__float_as_uint(s) & 0x7fffffu) != 0u || !normal)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = E::unpack2(in[i]);
            q[2 * i] = quotient(a.x, s);
            q[2 * i + 1] = quotient(a.y, s);
        }
    }
    return make_uint2(f8_pack2<E5>(q[0], q[1]) | (f8_pack2<E5>(q[2], q[3]) << 16),
                      f8_pack2<E5>(q[4], q[5]) | (f8_pack2<E5>(q[6], q[7]) << 16));
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

// F8: 0 the pools hold E's 16-bit elements, 1 E4M3, 2 E5M2.
template <class E, int F8, bool READ>
__global__ void __launch_bounds__(kThreads, READ ? 16 : 12)
paged_move_kernel(const SeqKV kv, const void* src_k, const void* src_v, void* dst_k, void* dst_v,
                  int64_t k_stride, int64_t v_stride, const int32_t* cu, int tokens, Divisor by_token) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int head_shift = kv.D == 128 ? 3 : 2, per_token = kv.Hkv << head_shift;
    const int64_t total = (int64_t)tokens * per_token;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t first = id - (threadIdx.x & 31);
    if (first >= total) return;
    // (a 64-bit division took longer than the search)
    const bool small = (total >> 31) == 0;
    auto token_of = [&](int64_t i) { return small ? over((int)i, by_token) : (int)(i / per_token); };
    const int t = id < total ? token_of(id) : tokens;
    const int piece = (int)(id - (int64_t)t * per_token);
    const int h = piece >> head_shift, d = (piece - (h << head_shift)) * kVec;
    uint4 k[2] = {}, v[2] = {};
    if (!READ && t < tokens) {
        // new rows are on their way while their place is looked up
        const uint4* pk = reinterpret_cast<const uint4*>(static_cast<const char*>(src_k) +
                                                         ((int64_t)t * k_stride + h * kv.D + d) * 2);
        const uint4* pv = reinterpret_cast<const uint4*>(static_cast<const char*>(src_v) +
                                                         ((int64_t)t * v_stride + h * kv.D + d) * 2);
        k[0] = __ldcs(pk);
        k[1] = __ldcs(pk + 1);
        v[0] = __ldcs(pv);
        v[1] = __ldcs(pv + 1);
    }
    int b = find_seq(cu, kv.num_seqs, token_of(first));
    if (t >= tokens) return;
    while (b < kv.num_seqs && cu[b + 1] <= t) ++b;
    const int64_t at = place_of(kv, cu, b, t, tokens);
    const int64_t cell = at + h * kv.s_head + d;
    const float sk = F8 && kv.scale_k ? kv.scale_k[h] : 1.f;
    const float sv = F8 && kv.scale_v ? kv.scale_v[h] : 1.f;
    constexpr int EB = F8 ? 1 : 2;
    if constexpr (READ) {
        // rows without a place read as zero; rows past the last sequence are left alone
        if (b >= kv.num_seqs || t < cu[b]) return;
        if (at >= 0) {
            const uint4* pk = reinterpret_cast<const uint4*>(static_cast<const char*>(src_k) + cell * EB);
            const uint4* pv = reinterpret_cast<const uint4*>(static_cast<const char*>(src_v) + cell * EB);
            if constexpr (F8) {
                const uint4 ck = __ldcs(pk), cv = __ldcs(pv);
                decode16<E, F8 == 2>(ck, sk, k);
                decode16<E, F8 == 2>(cv, sv, v);
            } else {
                k[0] = __ldcs(pk); k[1] = __ldcs(pk + 1);
                v[0] = __ldcs(pv); v[1] = __ldcs(pv + 1);
            }
        }
        uint4* ok = reinterpret_cast<uint4*>(static_cast<char*>(dst_k) + ((int64_t)t * k_stride + h * kv.D + d) * 2);
        uint4* ov = reinterpret_cast<uint4*>(static_cast<char*>(dst_v) + ((int64_t)t * v_stride + h * kv.D + d) * 2);
        __stcs(ok, k[0]); __stcs(ok + 1, k[1]);
        __stcs(ov, v[0]); __stcs(ov + 1, v[1]);
    } else {
        if (at < 0) return;
        uint4* ok = reinterpret_cast<uint4*>(static_cast<char*>(dst_k) + cell * EB);
        uint4* ov = reinterpret_cast<uint4*>(static_cast<char*>(dst_v) + cell * EB);
        if constexpr (F8) {
            *ok = encode16<E, F8 == 2>(k, sk, __frcp_rn(sk));
            *ov = encode16<E, F8 == 2>(v, sv, __frcp_rn(sv));
        } else {
            ok[0] = k[0]; ok[1] = k[1];
            ov[0] = v[0]; ov[1] = v[1];
        }
    }
}

template <bool READ>
cudaError_t launch_move(const SeqKV& kv, const void* sk, const void* sv, void* dk, void* dv,
                        int64_t k_stride, int64_t v_stride, const int32_t* cu, int tokens,
                        sfa_dtype dtype, cudaStream_t stream) {
    const int per_token = kv.Hkv * (kv.D / kVec);
    const int64_t total = (int64_t)tokens * per_token;
    const Divisor by_token = divide_by(per_token);
    const dim3 grid((unsigned)((total + kThreads - 1) / kThreads));
    auto go = [&](auto kern) {
        cudaError_t err = launch_pdl(kern, grid, dim3(kThreads), 0, stream, kv, sk, sv, dk, dv,
                                     k_stride, v_stride, cu, tokens, by_token);
        if (err == cudaSuccess) count_launches(1);
        return err;
    };
    const bool bf16 = dtype == SFA_DTYPE_BF16;
    switch (kv.f8) {
        case 0: return go(paged_move_kernel<BF16, 0, READ>);   // 16-bit elements move as they are
        case 1: return bf16 ? go(paged_move_kernel<BF16, 1, READ>) : go(paged_move_kernel<F16, 1, READ>);
        default: return bf16 ? go(paged_move_kernel<BF16, 2, READ>) : go(paged_move_kernel<F16, 2, READ>);
    }
}

}  // namespace

cudaError_t launch_paged_append(const SeqKV& kv, const void* k_new, const void* v_new,
                                int64_t k_stride, int64_t v_stride, const int32_t* cu, int tokens,
                                sfa_dtype dtype, cudaStream_t stream) {
    return launch_move<false>(kv, k_new, v_new, const_cast<void*>(kv.k), const_cast<void*>(kv.v),
                              k_stride, v_stride, cu, tokens, dtype, stream);
}

cudaError_t launch_paged_read(const SeqKV& kv, const int32_t* cu, int tokens, sfa_dtype dtype,
                              void* k_out, void* v_out, cudaStream_t stream) {
    const int64_t stride = (int64_t)kv.Hkv * kv.D;
    return launch_move<true>(kv, kv.k, kv.v, k_out, v_out, stride, stride, cu, tokens, dtype, stream);
}

}  // namespace sfa
