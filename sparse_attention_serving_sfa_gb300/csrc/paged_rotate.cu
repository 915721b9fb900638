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
// 2^-64 turns (turns_of), times pos, wraps by itself.  What is left within an
// eighth of a turn goes to fp32 (2^-24 of itself) and sincospif, the quarters are put
// back by swaps and signs: far positions cost no accuracy.
//
// Bound: HBM, every element once in and once out (2 bytes in, 2 or 1 out); a
// decode step by latency.  A block takes a few tokens: their angles once into shared
// memory for all heads (the float4 of two angles lie by piece, so that the eight
// threads of a head read side by side), then a thread moves 16 elements of a head at
// a time, in two 16-byte halves that hold both sides of eight pairs, the next under
// way.  Measured: 12,837 tokens of 32 / 8 heads of 128 into E4M3 pages 62 to 63.5 us
// (289 MB, 4.6 TB/s, 0.69 of the measured copy rate; a fetch not under way 67 us, four
// blocks an SM with spills 68, a warp a token with its angles in registers 71);
// 7,210 of 16 / 4 heads of 64 into 16-bit pages 12 to 13.7 us; one token each of 64
// requests 4.7 to 5.1 us, 3.5 of them where no code has to be found in 64 bits.
#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "paged_move.cuh"
#include "ptx.cuh"

namespace sfa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;      // of a block

// f / (2 pi) as a fraction of a turn in units of 2^-64 (whole turns drop out), to 3
// units (five roundings) and 1.6e-4 |f| of one: 1 / (2 pi) as three floats, the first
// two products with their remainders, the third rounded.  So an angle is off by 2^-59
// of a radian a position for frequencies up to 1, and by 2^-24 at any position (below
// 2^30) for those up to 2^20.
// (In fp64 arithmetic this took up to 58% of that pipe's time, and the kernel up to
// 25% more.)
__device__ __forceinline__ uint64_t turns_of(float f) {
    constexpr float kHigh = 0.15915493667125702f, kMid = 6.4206382432985265e-09f, kLow = 7.342738699078887e-17f;
    const float a = f * kHigh, b = f * kMid;
    auto units = [](float x) { return (uint64_t)__float2ll_rn((x - rintf(x)) * 18446744073709551616.f); };
    return units(a) + units(fmaf(f, kHigh, -a)) + units(b) + units(fmaf(f, kMid, -b)) + units(f * kLow);
}

// The code nearest to the exact quotient y / scale.  A float near it decides, unless
// it lies within 8 units in the last place of a border between codes (which has zeros
// behind its fourth fraction bit): then the border times the scale, exact in 64 bits,
// does.  (Three roundings make the float, of y, the reciprocal and their product; where
// one could be out of the normal numbers it is the 64-bit quotient rounded.)
template <bool E5>
__device__ __forceinline__ uint32_t nearest_code(double y, float scale) {
    const float f = (float)y;
    float q = f * __frcp_rn(scale);
    auto middling = [](float v) { return fabsf(v) >= 1e-30f && fabsf(v) < 1e30f; };
    if (!(middling(f) && middling(q))) q = (float)(y / (double)scale);
    const uint32_t bits = __float_as_uint(q), border = (bits + 0x40000u) & ~0x7ffffu;
    if (bits - border + 8u <= 16u) {
        const double d = fabs(y) - (double)fabsf(__uint_as_float(border)) * (double)scale;
        q = __uint_as_float(d == 0.0 ? border : (d > 0.0 ? border + 1u : border - 1u));
    }
    return f8_pack2<E5>(q, 0.f) & 0xffu;
}

// The codes of a pair's rotation by the scale (low byte: the first), found in 64 bits:
// sine and cosine of the angle within an eighth of a turn by their Taylor series in
// fixed point, of which 7 and 8 terms leave 2^-45.  (t = angle / (pi / 4) in [0, 1];
// coefficients (pi / 4)^n / n! in units of 2^-64.  What counts is how long it takes: with
// the series in fp64 a decode step took 5.2 us instead of 5.0.)
template <bool E5>
__device__ __noinline__ uint32_t exact_codes(float x, float y, uint64_t phase, float scale) {
    const int quarter = (int)((phase + (1ull << 61)) >> 62) & 3;
    const int64_t r = (int64_t)(phase - ((uint64_t)quarter << 62));
    const uint64_t t = (uint64_t)(r < 0 ? -r : r) << 2, z = __umul64hi(t, t) << 1;          // 2^-63
    constexpr uint64_t kSin[7] = {0xc90fdaa22168c235, 0x14abbce625be52bf, 0xa335e33bad570f, 0x265a599cc57b1,
                                  0x541e0d21fba, 0x78c1d3f7a, 0x7a3d0d3};
    constexpr uint64_t kCos[7] = {0x4ef4f326f9177969, 0x40f07c206d6b0ed, 0x155d3c7e3cbffa, 0x3c3ea0d12375,
                                  0x69b47ca881, 0x7e74e28e, 0x6db894};
    uint64_t ps = kSin[6], pc = kCos[6];
#pragma unroll
    for (int k = 5; k >= 0; --k) {
        ps = kSin[k] - 2 * __umul64hi(ps, z);
        pc = kCos[k] - 2 * __umul64hi(pc, z);
    }
    auto fraction = [](uint64_t v) {              // of 2^63
        const double d = __ull2double_rn(v);
        return v ? __hiloint2double(__double2hiint(d) - (63 << 20), __double2loint(d)) : 0.0;
    };
    const double sa = fraction(__umul64hi(ps, t)), s = r < 0 ? -sa : sa, c = fraction((1ull << 63) - __umul64hi(pc, z));
    const double co = quarter & 1 ? s : c, si = quarter & 1 ? c : s;
    const double cs = quarter == 1 || quarter == 2 ? -co : co, sn = quarter >= 2 ? -si : si;
    return nearest_code<E5>((double)x * cs - (double)y * sn, scale) | nearest_code<E5>((double)x * sn + (double)y * cs, scale) << 8;
}

// F8: 0 the pools hold E's 16-bit elements, 1 E4M3, 2 E5M2.  PAIRS: interleaved.
template <class E, int F8, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 3) paged_rotate_kernel(const RotateAppend p) {
    __shared__ float4 turn[kMaxTokens][32];       // [token][(j / 2) * pieces + piece]: angles 8 piece + j, + 1
    __shared__ int64_t cell_of[kMaxTokens];       // its place in the pools, -1 without, kNoRow for a row of no sequence
    __shared__ int pos_of[kMaxTokens];
    constexpr int64_t kNoRow = -2;
    grid_dependency_wait();
    grid_launch_dependents();
    const SeqKV& kv = p.kv;
    const int tid = threadIdx.x, lane = tid & 31;
    const int half = p.rotary / 2, turning = p.rotary / 16;     // angles, and pieces that turn
    const int t0 = blockIdx.x * p.block_tokens, n = min(p.block_tokens, p.tokens - t0);
    const int head_shift = kv.D == 128 ? 3 : 2, heads = p.Hq + 2 * kv.Hkv;

    // This thread's piece of every head it comes to: its two 8-element halves (a
    // value's lie side by side).
    const int piece = tid & ((1 << head_shift) - 1);
    const bool turned = piece < turning;
    const int at_a = turned && !PAIRS ? 8 * piece : 16 * piece, at_b = turned && !PAIRS ? at_a + half : at_a + 8;
    const int first = (blockIdx.y * kThreads + tid) >> head_shift, step = (kThreads * gridDim.y) >> head_shift;
    const int last = n * heads;
    const uint16_t *const q = static_cast<const uint16_t*>(p.q), *const k = static_cast<const uint16_t*>(p.k),
                   *const v = static_cast<const uint16_t*>(p.v);
    // head i of the block's tokens, one token's queries, keys and values after the other
    auto fetch = [&](int i, uint4& va, uint4& vb) {
        if (i >= last) return;
        const int x = over(i, p.by_heads), h = i - x * heads, hk = h - p.Hq, hv = hk - kv.Hkv;
        const int64_t t = t0 + x;
        const uint16_t* src = hk < 0 ? q + t * p.q_stride + h * kv.D : (hv < 0 ? k + t * p.k_stride + hk * kv.D : v + t * p.v_stride + hv * kv.D);
        va = *reinterpret_cast<const uint4*>(src + (hv < 0 ? at_a : 16 * piece));
        vb = *reinterpret_cast<const uint4*>(src + (hv < 0 ? at_b : 16 * piece + 8));
    };
    // the first ones are on their way while their tokens' places and angles are found
    uint4 next_a = {}, next_b = {};
    fetch(first, next_a, next_b);

    // half a warp's worth of angles at least to a warp: the warps go round the tokens
    for (int x = tid >> 5; x < 2 * n; x += kThreads / 32) {
        const int tk = x >> 1, t = t0 + tk;
        const int b = find_seq(p.cu, kv.num_seqs, t);
        const bool in = b < kv.num_seqs && t >= p.cu[b];
        const int pos = in ? seq_keys(kv, b).y - (seq_rows(p.cu, b, p.tokens).y - t) : 0;
        for (int i = lane + 32 * (x & 1); i < half; i += 64) {
            const uint64_t phase = turns_of(p.inv_freq[i]) * (uint64_t)(int64_t)pos;
            const int quarter = (int)((phase + (1ull << 61)) >> 62) & 3;
            const int32_t r = (int32_t)((int64_t)(phase - ((uint64_t)quarter << 62)) >> 30);
            float sr, cr;
            sincospif((float)r * 1.1641532182693481e-10f, &sr, &cr);                     // 2^-33
            const float co = quarter & 1 ? sr : cr, si = quarter & 1 ? cr : sr;
            reinterpret_cast<float2*>(&turn[tk][(i & 7) / 2 * turning + (i >> 3)])[i & 1] =
                make_float2(quarter == 1 || quarter == 2 ? -co : co, quarter >= 2 ? -si : si);
        }
        if (lane == 0 && (x & 1) == 0) {
            pos_of[tk] = pos;
            cell_of[tk] = in ? place_of(kv, p.cu, b, t, p.tokens) : kNoRow;
        }
    }
    __syncthreads();

    for (int i = first; i < last; i += step) {
        const uint4 raw_a = next_a, raw_b = next_b;
        fetch(i + step, next_a, next_b);
        const int x = over(i, p.by_heads), h = i - x * heads;
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + kv.Hkv, turns = turned && !is_v;
        const int64_t cell = cell_of[x], t = t0 + x;
        if (cell < (is_q ? -1 : 0)) continue;
        const int head = is_q ? h : (is_v ? h - p.Hq - kv.Hkv : h - p.Hq);
        const int to_a = is_v ? 16 * piece : at_a, to_b = is_v ? 16 * piece + 8 : at_b;
        float a[8], b[8];
        unpack8<E>(raw_a, a);
        unpack8<E>(raw_b, b);
        if (turns) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float4 cs = turn[x][j / 2 * turning + piece];
                float& x0 = PAIRS ? (j < 4 ? a : b)[2 * (j & 3)] : a[j];
                float& y0 = PAIRS ? (j < 4 ? a : b)[2 * (j & 3) + 1] : b[j];
                float& x1 = PAIRS ? (j < 4 ? a : b)[2 * (j & 3) + 2] : a[j + 1];
                float& y1 = PAIRS ? (j < 4 ? a : b)[2 * (j & 3) + 3] : b[j + 1];
                const float u0 = x0 * cs.x - y0 * cs.y, v0 = x0 * cs.y + y0 * cs.x;
                const float u1 = x1 * cs.z - y1 * cs.w, v1 = x1 * cs.w + y1 * cs.z;
                x0 = u0;
                y0 = v0;
                x1 = u1;
                y1 = v1;
            }
        }
        const int64_t at = cell + head * kv.s_head;
        if (F8 && !is_q) {
            const float* scales = is_v ? kv.scale_v : kv.scale_k;
            const float s = scales ? scales[head] : 1.f, inv = __frcp_rn(s);
            uint8_t* dst = static_cast<uint8_t*>(const_cast<void*>(is_v ? kv.v : kv.k)) + at;
            uint2 ca, cb;
            if (turns) {
                // The codes, if they are the same 5.25 2^-24 of the sum of the pair's magnitudes
                // to either side.  That is a bound: in units of 2^-24 of an element's magnitude,
                // at t within an eighth of a turn, the cosine is off by 1 and by 0.4 sin t for its
                // angle's rounding (the sine by less than 1 and by 0.4 cos t), and the product
                // rounded by itself, the sum, the reciprocal and the quotient add cos t (sin t)
                // each; 5.02 at most, at t = 0.08.  So it mostly is; the other pairs' are found in
                // 64 bits, and so is every pair whose scale is beyond 2^100 or below 2^-100: there
                // the rotation could leave the normal numbers and its error that margin.
                auto codes = [&](const float (&v)[8], uint4 raw, uint4 other, uint2& differ) {
                    float m[8], lo[8], hi[8];
                    unpack8<E>(raw, m);
                    if constexpr (!PAIRS) unpack8<E>(other, hi);
#pragma unroll
                    for (int j = 0; j < 8; ++j) lo[j] = fabsf(m[j]) + fabsf(PAIRS ? m[j ^ 1] : hi[j]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float e = lo[j] * inv * 3.1292439e-07f;
                        lo[j] = v[j] * inv - e;
                        hi[j] = v[j] * inv + e;
                    }
                    const uint2 c = codes8<F8 == 2>(lo), o = codes8<F8 == 2>(hi);
                    const bool middling = inv >= 7.8886091e-31f && inv <= 1.2676506e30f;
                    differ = middling ? make_uint2(c.x ^ o.x, c.y ^ o.y) : make_uint2(~0u, ~0u);
                    return c;
                };
                uint2 da, db;
                ca = codes(a, raw_a, raw_b, da);
                cb = codes(b, raw_b, raw_a, db);
                if (da.x | da.y | db.x | db.y) {
#pragma unroll 1
                    for (int j = 0; j < 8; ++j) {
                        // pair j: byte j of both halves, or bytes 2 j and 2 j + 1 of one after the other
                        const int at = PAIRS ? 16 * (j & 1) : 8 * (j & 3);
                        const uint32_t bytes = (PAIRS ? 0xffffu : 0xffu) << at;
                        uint32_t& wa = PAIRS ? (j < 4 ? (j < 2 ? ca.x : ca.y) : (j < 6 ? cb.x : cb.y)) : (j < 4 ? ca.x : ca.y);
                        uint32_t& wb = j < 4 ? cb.x : cb.y;
                        const uint32_t d = PAIRS ? (j < 4 ? (j < 2 ? da.x : da.y) : (j < 6 ? db.x : db.y))
                                                 : (j < 4 ? da.x | db.x : da.y | db.y);
                        if (!(d & bytes)) continue;
                        auto word = [](uint4 v, int i) { return i < 2 ? (i ? v.y : v.x) : (i == 2 ? v.z : v.w); };
                        float ex, ey;
                        if constexpr (PAIRS) {
                            const float2 e = E::unpack2(word(j < 4 ? raw_a : raw_b, j & 3));
                            ex = e.x;
                            ey = e.y;
                        } else {
                            const float2 e = E::unpack2(word(raw_a, j >> 1)), f = E::unpack2(word(raw_b, j >> 1));
                            ex = j & 1 ? e.y : e.x;
                            ey = j & 1 ? f.y : f.x;
                        }
                        const uint64_t phase = turns_of(p.inv_freq[8 * piece + j]) * (uint64_t)(int64_t)pos_of[x];
                        const uint32_t c = exact_codes<F8 == 2>(ex, ey, phase, s);
                        if constexpr (PAIRS) {
                            wa = (wa & ~bytes) | (c << at);
                        } else {
                            wa = (wa & ~bytes) | ((c & 0xffu) << at);
                            wb = (wb & ~bytes) | ((c >> 8) << at);
                        }
                    }
                }
            } else {
                ca = encode8<F8 == 2>(a, s, inv);
                cb = encode8<F8 == 2>(b, s, inv);
            }
            *reinterpret_cast<uint2*>(dst + to_a) = ca;
            *reinterpret_cast<uint2*>(dst + to_b) = cb;
            continue;
        }
        auto pack = [](const float (&y)[8]) {
            return make_uint4(E::pack2(y[0], y[1]), E::pack2(y[2], y[3]), E::pack2(y[4], y[5]), E::pack2(y[6], y[7]));
        };
        // what does not turn keeps its bits (NaN payloads, too)
        uint16_t* dst = is_q ? static_cast<uint16_t*>(p.q_out) + t * p.q_out_stride + head * kv.D
                             : static_cast<uint16_t*>(const_cast<void*>(is_v ? kv.v : kv.k)) + at;
        *reinterpret_cast<uint4*>(dst + to_a) = turns ? pack(a) : raw_a;
        *reinterpret_cast<uint4*>(dst + to_b) = turns ? pack(b) : raw_b;
    }
}

}  // namespace

cudaError_t launch_paged_rotate(RotateAppend p, sfa_dtype dtype, cudaStream_t stream) {
    // As many tokens a block as leave some blocks for every SM; where tokens are few
    // a token's heads are dealt out over several.
    const int heads = p.Hq + 2 * p.kv.Hkv, want = 3 * num_sms();
    p.by_heads = divide_by(heads);
    p.block_tokens = 1;
    while (p.block_tokens < kMaxTokens && p.block_tokens * heads * (p.kv.D / 16) < 4 * kThreads &&
           p.tokens / (2 * p.block_tokens) >= want)
        p.block_tokens *= 2;
    const int blocks = (p.tokens + p.block_tokens - 1) / p.block_tokens;
    const int passes = (p.block_tokens * heads * (p.kv.D / 16) + kThreads - 1) / kThreads;
    const int split = blocks >= want ? 1 : min(passes, (want + blocks - 1) / blocks);
    const dim3 grid((unsigned)blocks, (unsigned)split);
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
