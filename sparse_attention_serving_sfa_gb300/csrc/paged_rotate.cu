// Appending to a paged KV cache with the position rotation on the way, and the
// queries rotated beside it.
//
// Row t of sequence b is token pos = kv_lens[b] - (cu[b + 1] - t), as in append.
// With angle = pos * inv_freq[i], pair i (i < r / 2) of a query or key head,
//     (x, y) -> (x cos - y sin, x sin + y cos),
// in fp32, rounded once: to 16 bits (q, a 16-bit cache) or to the code nearest to the
// quotient by the head's scale.  Pair i is dims (i, i + r / 2), or (2i, 2i + 1)
// interleaved; dims from r on, and values, move as they are.
//
// Angles are kept in turns, as 64-bit fractions: inv_freq / (2 pi) in units of
// 2^-64 turns, times pos, wraps by itself.  The quotient comes from fp64 (a relative
// 2^-53), so an angle is off by at most 2^-53 of itself and 2^-64 |pos| turns, the
// fraction is rounded to fp32 (2^-25 of half a turn), and sincospif does the rest: far
// positions cost no accuracy.
//
// Bound: HBM, every element once in and once out (2 bytes in, 2 or 1 out); a
// decode step by latency.  A block takes a few tokens: their angles once into shared
// memory for all heads (the float4 of two angles lie by piece, so that the eight
// threads of a head read side by side), then a thread moves 16 elements of a head at
// a time, in two 16-byte pieces that hold both halves of its eight pairs.
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_move.cuh"
#include "ptx.cuh"

namespace sfa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;      // of a block

// inv_freq / (2 pi) as a fraction of a turn in units of 2^-64 (whole turns drop out).
__device__ __forceinline__ uint64_t turns_of(float f) {
    double t = (double)f * 0.15915494309189535;
    t -= rint(t);
    return (uint64_t)__double2ll_rn(t * 18446744073709551616.0);
}

// F8: 0 the pools hold E's 16-bit elements, 1 E4M3, 2 E5M2.  PAIRS: interleaved.
template <class E, int F8, bool PAIRS>
__global__ void __launch_bounds__(kThreads) paged_rotate_kernel(const RotateAppend p) {
    __shared__ float4 turn[kMaxTokens][32];       // [token][(j / 2) * pieces + piece]: angles 8 piece + j, + 1
    __shared__ int64_t cell_of[kMaxTokens];       // its place in the pools, or -1
    __shared__ int in_seq[kMaxTokens];            // the row belongs to a sequence
    grid_dependency_wait();
    grid_launch_dependents();
    const SeqKV& kv = p.kv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int half = p.rotary / 2, turned = p.rotary / 16;      // angles, and pieces that turn
    const int t0 = blockIdx.x * p.block_tokens, n = min(p.block_tokens, p.tokens - t0);
    // a warp a token: its place, then its angles
    for (int x = warp; x < n; x += kThreads / 32) {
        const int t = t0 + x;
        const int b = find_seq(p.cu, kv.num_seqs, t);
        const bool in = b < kv.num_seqs && t >= p.cu[b];
        const int pos = in ? seq_keys(kv, b).y - (seq_rows(p.cu, b, p.tokens).y - t) : 0;
        if (lane == 0) {
            in_seq[x] = in;
            cell_of[x] = place_of(kv, p.cu, b, t, p.tokens);
        }
        for (int i = lane; i < half; i += 32) {
            const uint64_t phase = turns_of(p.inv_freq[i]) * (uint64_t)(int64_t)pos;
            float s, c;
            sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);    // 2^-31
            reinterpret_cast<float2*>(&turn[x][(i & 7) / 2 * turned + (i >> 3)])[i & 1] = make_float2(c, s);
        }
    }
    __syncthreads();
    const int head_shift = kv.D == 128 ? 3 : 2, pieces = 1 << head_shift;
    const int per_token = (p.Hq + 2 * kv.Hkv) << head_shift;
    for (int id = tid; id < n * per_token; id += kThreads) {
        const int x = over(id, p.by_token), rest = id - x * per_token;
        if (!in_seq[x]) continue;
        const int h = rest >> head_shift, piece = rest & (pieces - 1);
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + kv.Hkv;
        const int hh = is_q ? h : (is_v ? h - p.Hq - kv.Hkv : h - p.Hq);
        const int64_t cell = cell_of[x];
        if (!is_q && cell < 0) continue;
        const bool turns = !is_v && piece < turned;
        // the two 8-element pieces
        const bool apart = turns && !PAIRS;
        const int da = apart ? 8 * piece : 16 * piece, db = apart ? da + half : da + 8;
        const int64_t t = t0 + x;
        const uint16_t* src = static_cast<const uint16_t*>(is_q ? p.q : (is_v ? p.v : p.k)) +
                              t * (is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride)) + hh * kv.D;
        const uint4 va = *reinterpret_cast<const uint4*>(src + da), vb = *reinterpret_cast<const uint4*>(src + db);
        float a[8], b[8];
        unpack8<E>(va, a);
        unpack8<E>(vb, b);
        if (turns) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float4 cs = turn[x][j / 2 * turned + piece];
                if constexpr (PAIRS) {
                    float* y = j < 4 ? a + 2 * j : b + 2 * (j - 4);
                    const float y0 = y[0], y1 = y[1], y2 = y[2], y3 = y[3];
                    y[0] = y0 * cs.x - y1 * cs.y;
                    y[1] = y0 * cs.y + y1 * cs.x;
                    y[2] = y2 * cs.z - y3 * cs.w;
                    y[3] = y2 * cs.w + y3 * cs.z;
                } else {
                    const float x0 = a[j], x1 = a[j + 1], y0 = b[j], y1 = b[j + 1];
                    a[j] = x0 * cs.x - y0 * cs.y;
                    b[j] = x0 * cs.y + y0 * cs.x;
                    a[j + 1] = x1 * cs.z - y1 * cs.w;
                    b[j + 1] = x1 * cs.w + y1 * cs.z;
                }
            }
        }
        auto pack = [](const float (&y)[8]) {
            return make_uint4(E::pack2(y[0], y[1]), E::pack2(y[2], y[3]), E::pack2(y[4], y[5]), E::pack2(y[6], y[7]));
        };
        // what does not turn keeps its bits (NaN payloads, too)
        const uint4 wa = turns ? pack(a) : va, wb = turns ? pack(b) : vb;
        if (is_q) {
            uint16_t* dst = static_cast<uint16_t*>(p.q_out) + t * p.q_out_stride + hh * kv.D;
            *reinterpret_cast<uint4*>(dst + da) = wa;
            *reinterpret_cast<uint4*>(dst + db) = wb;
            continue;
        }
        void* pool = const_cast<void*>(is_v ? kv.v : kv.k);
        const int64_t at = cell + hh * kv.s_head;
        if constexpr (F8) {
            const float* scales = is_v ? kv.scale_v : kv.scale_k;
            const float s = scales ? scales[hh] : 1.f, inv = __frcp_rn(s);
            uint8_t* dst = static_cast<uint8_t*>(pool) + at;
            *reinterpret_cast<uint2*>(dst + da) = encode8<F8 == 2>(a, s, inv);
            *reinterpret_cast<uint2*>(dst + db) = encode8<F8 == 2>(b, s, inv);
        } else {
            uint16_t* dst = static_cast<uint16_t*>(pool) + at;
            *reinterpret_cast<uint4*>(dst + da) = wa;
            *reinterpret_cast<uint4*>(dst + db) = wb;
        }
    }
}

}  // namespace

cudaError_t launch_paged_rotate(RotateAppend p, sfa_dtype dtype, cudaStream_t stream) {
    const int per_token = (p.Hq + 2 * p.kv.Hkv) * (p.kv.D / 16);
    p.by_token = divide_by(per_token);
    p.block_tokens = 1;
    while (p.block_tokens < kMaxTokens && p.block_tokens * per_token < 4 * kThreads && p.tokens / p.block_tokens > 2048)
        p.block_tokens *= 2;
    const dim3 grid((unsigned)((p.tokens + p.block_tokens - 1) / p.block_tokens));
    auto go = [&](auto kern) {
        cudaError_t err = launch_pdl(kern, grid, dim3(kThreads), 0, stream, p);
        if (err == cudaSuccess) count_launches(1);
        return err;
    };
#define SFA_ROTATE(E_, F8_) (p.interleaved ? go(paged_rotate_kernel<E_, F8_, true>) : go(paged_rotate_kernel<E_, F8_, false>))
    const bool bf16 = dtype == SFA_DTYPE_BF16;
    switch (p.kv.f8) {
        case 0: return bf16 ? SFA_ROTATE(BF16, 0) : SFA_ROTATE(F16, 0);
        case 1: return bf16 ? SFA_ROTATE(BF16, 1) : SFA_ROTATE(F16, 1);
        default: return bf16 ? SFA_ROTATE(BF16, 2) : SFA_ROTATE(F16, 2);
    }
#undef SFA_ROTATE
}

}  // namespace sfa
