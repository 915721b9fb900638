// Dense attention of a few query rows over a paged cache or packed rows, on
// warp-level MMAs.
//
// A tile is 16 rows of one kv head: row r is query token r / G of the
// sequence and head r % G of the group (one decode step of up to 16 grouped
// heads is one tile).  Its keys come in chunks of 4 warps x KS keys.  For a
// row with visible keys j (j < kv_len, and j <= i + kv_len - q_len when causal)
//     s_j = scale * q.k_j,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
// one pass with the running maximum m and sum in fp32 per warp, the four
// warps' states merged at the end of the tile.
//
// Bound: HBM, each cached K / V row of a kv head read once per 16-row tile;
// over an 8-bit cache also the issue slots of the conversions; a small batch by
// latency (two launches, three dependent look-ups).  Measured: 64 sequences of
// 2,000 to 8,192 keys, 32/8 heads of 128, bf16 183 to 186 us, 6.4 to 6.5 TB/s
// (0.94 to 0.96 of the measured copy rate); 16 of 3,001 to 65,536 keys, 64/8
// heads, E4M3 114 to 127 us, 5.2 to 5.8 TB/s; 4 of 100 to 1,024 keys 8 us on the
// device.
// All tiles lie on one line, each as long as its chunks plus a fixed charge
// for what a tile costs besides, and the line is cut into equal ranges, one
// per CTA (two CTAs per SM), whatever the mix of lengths.  A cut falls on a
// chunk; tiles of fewer than kMinCut chunks stay whole (a part costs its way
// through the workspace).  A tile cut by a range border leaves its parts
// (O unnormalised, m, sum; fp32) in the workspace: a CTA has at most two, the
// one it ends and the one it begins.  attn_rows_merge, launched behind with
// programmatic dependent launch, joins them in order of their keys, so results do not
// depend on timing.
//
// Each warp fetches its own keys (16-byte cp.async into a private ring, rows
// swizzled by 16-byte pieces) and never waits for another warp until the end
// of the tile.  Rows without a key (past kv_len, pages out of range) are
// filled with zeros, never fetched, so whatever a page holds behind the last
// token cannot reach the output.
//
// P is carried to P.V as a 16-bit high part plus the 16-bit rounding of the
// remainder (two MMAs; the tensor pipe is idle most of the time here), the
// 8-bit cache's in fp16 alone (its V are exact in fp16): at most half a step,
// 2^-11 of a weight.  fp16 P carries a factor 2^7 (at most 2^15 in all, as m lags
// by up to 2^8), so a weight below 2^-21 of the one at m, where fp16's steps no
// longer shrink, is off by at most 2^-32 of that one.  8-bit K / V
// become fp16 in registers (exact); q is then scaled by a power of two per row
// to a largest magnitude in [2^14, 2^15), so that bf16 q fits fp16: elements
// down to 2^-31 of the row's largest are exact, smaller ones off by at most
// 2^-39 of it.  The power leaves with the scores.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "ptx.cuh"

namespace sfa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;            // rows of a tile
constexpr int kMaxCtas = 320;        // ranges (the workspace's size goes by it)
constexpr int kCharge = 2;           // a tile's fixed cost, in chunks
// Tiles of kMinCut chunks or more are cut, anywhere.  (Parts of two chunks at
// least: 4 requests of up to 1,024 keys 8.7 instead of 8.3 us, 19 of up to 1,231
// over E4M3 9.5 instead of 8.2; shorter tiles cut, too: 4 of up to 99 keys 6.0
// instead of 4.8 us, a join's launch.)
constexpr int kMinCut = 4;
constexpr float kRescale = 8.f;      // log2 growth of m that rescales O

// log2 of the factor that P, and with it O and the sums, carries: in fp16 the
// small weights of many keys would be lost without.
template <class E, int F8>
constexpr float kPShift = F8 || std::is_same<E, F16>::value ? 7.f : 0.f;

template <int D, int F8>
struct RowsCfg {
    static constexpr int EB = F8 ? 1 : 2;
    static constexpr int RB = D * EB;                         // bytes of a K (or V) row
    static constexpr int KS = RB >= 256 ? 16 : 32;            // keys of a warp's step
    static constexpr int tile = KS * RB;
    static constexpr int stage = 2 * tile;                    // K, V
    static constexpr int NS = 24576 / stage;                  // ring stages (3 or 6)
    static constexpr int warp_bytes = NS * stage;
    static constexpr int masks = kWarps * warp_bytes;         // valid-key bits of each stage
    static constexpr int ml = masks + kWarps * NS * 4;
    static constexpr int total = ml + kWarps * kRows * 2 * 4;
    static constexpr int chunk = kWarps * KS;
    // A warp's O in shared memory (over its ring): dim d of a row at o_at(d).
    // Rows and, where a thread holds D / 4 dims on end, those are spread over
    // the banks (without that the writes of a part took 8,000 cycles).
    static constexpr int o_row = F8 ? D + 16 : D + 8;
    __device__ static constexpr int o_at(int d) { return F8 ? d + d / (D / 4) * 4 : d; }
    static_assert(kRows * o_row * 4 <= warp_bytes, "a warp's O fits its ring");
};

// A sequence on the line: tiles * Hkv pieces of chunks + kCharge units, a tile's
// kv heads side by side.
struct Seq {
    int q_row, n_q, k_row, kv_len, tiles, chunks;
};

__device__ __forceinline__ Seq seq_of(const SeqAttn& p, int b, int chunk) {
    const int2 q = seq_rows(p.cu_q, b, p.tokens);
    const int2 k = seq_keys(p.kv, b);
    Seq s;
    s.q_row = q.x;
    s.n_q = q.y - q.x;
    s.k_row = k.x;
    s.kv_len = k.y;
    s.tiles = (s.n_q * p.G + kRows - 1) / kRows;             // (tokens * heads fits 30 bits)
    s.chunks = max(1, (s.kv_len + chunk - 1) / chunk);
    return s;
}

// The line's length, a range's length, the unit range (blockIdx.x + shift)
// begins at, and the sequence (and its first unit) that holds it.  One warp;
// every lane gets the answer.
struct Line {
    int64_t total, per, at, start;
    int b;
    Seq seq;
};

__device__ __forceinline__ Line line_at(const SeqAttn& p, int chunk, uint64_t ctas_mul, int shift) {
    const int lane = threadIdx.x & 31, B = p.kv.num_seqs;
    Seq mine_seq{};
    auto length = [&](int b) -> int64_t {
        if (b >= B) return 0;
        mine_seq = seq_of(p, b, chunk);
        return (int64_t)mine_seq.tiles * (mine_seq.chunks + kCharge) * p.kv.Hkv;
    };
    Line l;
    const int64_t first = length(lane);
    const Seq first_seq = mine_seq;
    int64_t sum = first;
    for (int b = lane + 32; b < B; b += 32) sum += length(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l.total = sum;
    l.per = (int64_t)__umul64hi((uint64_t)l.total, ctas_mul) + 1;
    l.at = ((int64_t)blockIdx.x + shift) * l.per;
    l.b = B;
    l.start = 0;
    if (l.at >= l.total) return l;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int64_t mine = b0 == 0 ? first : length(b0 + lane);
        if (b0 == 0) mine_seq = first_seq;
        int64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned above = __ballot_sync(0xffffffffu, l.start + inc > l.at);
        if (above) {
            const int w = __ffs(above) - 1;
            l.start += __shfl_sync(0xffffffffu, inc - mine, w);
            l.b = b0 + w;
            l.seq.q_row = __shfl_sync(0xffffffffu, mine_seq.q_row, w);
            l.seq.n_q = __shfl_sync(0xffffffffu, mine_seq.n_q, w);
            l.seq.k_row = __shfl_sync(0xffffffffu, mine_seq.k_row, w);
            l.seq.kv_len = __shfl_sync(0xffffffffu, mine_seq.kv_len, w);
            l.seq.tiles = __shfl_sync(0xffffffffu, mine_seq.tiles, w);
            l.seq.chunks = __shfl_sync(0xffffffffu, mine_seq.chunks, w);
            return l;
        }
        l.start += __shfl_sync(0xffffffffu, inc, 31);
    }
    return l;
}

// Tile-and-head number of unit `rel` of a sequence, and the unit within it.
__device__ __forceinline__ void split_unit(int64_t rel, int len, int& x, int64_t& th) {
    if ((rel >> 32) == 0) {
        const uint32_t q = (uint32_t)rel / (uint32_t)len;
        th = q;
        x = (int)((uint32_t)rel - q * (uint32_t)len);
    } else {
        th = rel / len;
        x = (int)(rel - th * len);
    }
}

// Chunks of a tile of n before unit x of its n + kCharge.
__device__ __forceinline__ int cut(int64_t x, int n) {
    if (x >= n + kCharge) return n;
    const int c = (int)min(x - kCharge / 2, (int64_t)n);
    if (n < kMinCut) return 2 * c < n ? 0 : n;
    return max(c, 0);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two 8-bit codes (low 16 bits of x) -> two fp16.
template <bool E5>
__device__ __forceinline__ uint32_t f8_to_h2(uint32_t x) {
    const uint16_t in = (uint16_t)x;
    uint32_t h;
    if constexpr (E5) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(in));
    else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
    return h;
}

// 16-byte piece `ch` of row `key` of a K / V tile.  16-bit rows (ldmatrix
// reads eight rows' pieces at one column) and 8-bit rows (a thread reads whole
// pieces: of keys g, columns lane % 4 for K; of keys 2c, columns g for V) want
// different spreads over the banks.
template <int RB, int F8>
__device__ __forceinline__ int piece_at(int key, int ch) {
    if constexpr (!F8) return key * RB + ((ch ^ (key & 7)) << 4);
    else if constexpr (RB == 128) return key * RB + ((ch ^ (((key ^ (key >> 2)) & 1) << 2 ^ (key & 2))) << 4);
    else return key * RB + ((ch ^ ((key >> 1) & 3)) << 4);
}

template <class E, int D, int F8, bool PAGED>
__global__ void __launch_bounds__(kThreads, 2) attn_rows_kernel(const SeqAttn p, uint64_t ctas_mul) {
    using C = RowsCfg<D, F8>;
    constexpr int KS = C::KS, RB = C::RB, NS = C::NS;
    constexpr bool BF = std::is_same<E, BF16>::value && F8 == 0;    // MMA element type
    constexpr int NT = KS / 8;                                      // key n-tiles of a step
    constexpr int KK = D / 16;                                      // k-steps of Q.K^T
    constexpr int ND = D / 8;                                       // dim n-tiles
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    unsigned char* ring = smem + warp * C::warp_bytes;
    const uint32_t ring_u = smem_u32(ring);
    volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + C::masks) + warp * NS;
    float* ml = reinterpret_cast<float*>(smem + C::ml);
    grid_dependency_wait();
    grid_launch_dependents();

    const Line line = line_at(p, C::chunk, ctas_mul, 0);
    int64_t u = line.at;
    const int64_t u_end = min(line.total, u + line.per);
    if (u >= u_end) return;
    int b = line.b;
    int64_t seq_start = line.start;
    Seq sq = line.seq;

    float* ws_o = static_cast<float*>(p.ws);
    float* ws_ml = ws_o + (int64_t)2 * kMaxCtas * kRows * D;

    while (u < u_end) {
        // ---- the tile ----
        const int64_t seq_units = (int64_t)sq.tiles * (sq.chunks + kCharge) * p.kv.Hkv;
        if (u >= seq_start + seq_units) {
            seq_start += seq_units;
            if (++b >= p.kv.num_seqs) return;
            sq = seq_of(p, b, C::chunk);
            continue;
        }
        int x0;
        int64_t th;
        split_unit(u - seq_start, sq.chunks + kCharge, x0, th);
        const int tile = over((int)th, p.by_heads), h = (int)th - tile * p.kv.Hkv;
        const int64_t x1 = min((int64_t)sq.chunks + kCharge, x0 + (u_end - u));
        const int c0 = cut(x0, sq.chunks), c1 = cut(x1, sq.chunks);
        u += x1 - x0;
        if (c0 == c1) continue;
        const int n_q = sq.n_q, kv_len = sq.kv_len;
        const int rows = n_q * p.G, row_base = tile * kRows;
        // number of visible keys of a row (rows past the tile: all, unused)
        auto limit = [&](int r) -> int {
            if (!p.causal || row_base + r >= rows) return kv_len;
            const int i = over(row_base + r, p.by_group);
            return max(0, min(kv_len, i + kv_len - n_q + 1));
        };
        const int last_row = min(kRows, rows - row_base) - 1;
        const int tile_lim = limit(last_row);
        const int lim0 = limit(g), lim1 = limit(g + 8);

        // ---- K / V fetch: step st of this warp is keys key0(st) .. + KS - 1 ----
        const int nsteps = min(c1 - c0, max(0, (tile_lim - c0 * C::chunk + C::chunk - 1) / C::chunk));
        auto key0 = [&](int st) { return (c0 + st) * C::chunk + warp * KS; };
        const char* kb = static_cast<const char*>(p.kv.k) + h * p.kv.s_head * C::EB;
        const char* vb = static_cast<const char*>(p.kv.v) + h * (PAGED ? p.kv.s_head : p.kv.sv_head) * C::EB;
        // page of this lane's key of step st, or -1: looked up a step early, and
        // left as loaded, so that nothing waits for the load
        auto page_of = [&](int st) -> int {
            const int key = key0(st) + lane;
            if (st >= nsteps || lane >= KS || key >= kv_len) return -1;
            if constexpr (!PAGED) return 0;
            return p.kv.page_table[(int64_t)b * p.kv.max_pages + over(key, p.kv.by_page)];
        };
        auto issue = [&](int st, int page) {
            if (PAGED && (unsigned)page >= (unsigned)p.kv.num_pages) page = -1;
            if (st < nsteps) {
                const int s = st % NS;
                const int key = key0(st) + lane;
                int64_t ko = -1, vo = -1;
                if (page >= 0) {
                    if constexpr (PAGED) {
                        ko = (int64_t)page * p.kv.s_page + (int64_t)(key - over(key, p.kv.by_page) * p.kv.page_size) * p.kv.s_tok;
                    } else {
                        ko = (int64_t)(sq.k_row + key) * p.kv.s_tok;
                        vo = (int64_t)(sq.k_row + key) * p.kv.sv_tok;
                    }
                }
                const uint32_t ok = __ballot_sync(0xffffffffu, page >= 0);
                if (lane == 0) masks[s] = ok;
                constexpr int PIECES = RB / 16, PER = 32 / PIECES;    // rows of a warp-wide copy
                const int ch = lane % PIECES;
#pragma unroll
                for (int i = 0; i < KS / PER; ++i) {
                    const int key_i = i * PER + lane / PIECES;
                    const int64_t o = __shfl_sync(0xffffffffu, ko, key_i);
                    int64_t o2 = o;
                    if constexpr (!PAGED) o2 = __shfl_sync(0xffffffffu, vo, key_i);
                    unsigned char* dst = ring + s * C::stage + piece_at<RB, F8>(key_i, ch);
                    cp_async_16_zfill(dst, kb + (o < 0 ? 0 : o * C::EB + ch * 16), o < 0 ? 0 : 16);
                    cp_async_16_zfill(dst + C::tile, vb + (o < 0 ? 0 : o2 * C::EB + ch * 16), o < 0 ? 0 : 16);
                }
            }
            cp_async_commit();
        };

        int page_next = page_of(0);
        for (int st = 0; st < NS - 1; ++st) {
            const int pg = page_next;
            page_next = page_of(st + 1);
            issue(st, pg);
        }

        // ---- Q fragments ----
        uint32_t qf[KK][4];
        float rs0 = p.scale_log2, rs1 = p.scale_log2;   // multipliers of the two rows' scores
        {
            const uint16_t* qb = static_cast<const uint16_t*>(p.q);
            auto q_row = [&](int r) -> const uint16_t* {
                if (row_base + r >= rows) return nullptr;
                const int i = over(row_base + r, p.by_group);
                return qb + (sq.q_row + i) * p.q_stride + (h * p.G + (row_base + r) - i * p.G) * D;
            };
            const uint16_t* q0 = q_row(g);
            const uint16_t* q1 = q_row(g + 8);
            auto ld = [](const uint16_t* q, int d) {
                return q ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
            };
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                // 8-bit rows: k-step kk of thread column c holds dims
                // 64 (kk / 4) + 16 c + 4 (kk % 4) .. + 3 (one 16-byte piece of
                // a K row serves four k-steps)
                const int d = F8 ? 64 * (kk / 4) + 16 * c + 4 * (kk % 4) : 16 * kk + 2 * c;
                const int d2 = F8 ? d + 2 : d + 8;
                qf[kk][0] = ld(q0, d);
                qf[kk][1] = ld(q1, d);
                qf[kk][2] = ld(q0, d2);
                qf[kk][3] = ld(q1, d2);
            }
            if constexpr (F8) {
                if constexpr (std::is_same<E, BF16>::value) {
                    // scale each row by a power of two into fp16's range
                    float a0 = 0.f, a1 = 0.f;
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f = E::unpack2(qf[kk][i]);
                            float& a = (i & 1) ? a1 : a0;
                            a = fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) {
                        a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, o));
                        a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, o));
                    }
                    // exponent of the row's largest, kept where both 2^x and 2^-x are normal
                    auto expo = [](float a) {
                        const int e = (int)((__float_as_uint(a) >> 23) & 255u) - 127;
                        return (a == 0.f || e > 127) ? 0 : max(e - 14, -120);
                    };
                    const int e0 = expo(a0), e1 = expo(a1);
                    const float f0 = __uint_as_float((uint32_t)(127 - e0) << 23);
                    const float f1 = __uint_as_float((uint32_t)(127 - e1) << 23);
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f = E::unpack2(qf[kk][i]);
                            const float m = (i & 1) ? f1 : f0;
                            qf[kk][i] = F16::pack2(f.x * m, f.y * m);
                        }
                    rs0 *= __uint_as_float((uint32_t)(127 + e0) << 23);
                    rs1 *= __uint_as_float((uint32_t)(127 + e1) << 23);
                }
                if (p.kv.scale_k) {
                    rs0 *= p.kv.scale_k[h];
                    rs1 *= p.kv.scale_k[h];
                }
            }
        }

        float o[ND][4];
#pragma unroll
        for (int i = 0; i < ND; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        for (int st = 0; st < nsteps; ++st) {
            {
                const int pg = page_next;
                page_next = page_of(st + NS);
                issue(st + NS - 1, pg);
            }
            cp_async_wait<NS - 1>();
            __syncwarp();
            const int s = st % NS;
            const uint32_t kt = ring_u + s * C::stage, vt = kt + C::tile;
            const uint32_t valid = masks[s];
            // ---- S = Q K^T ----
            float sc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
                if constexpr (F8) {
#pragma unroll
                    for (int half = 0; half < D / 64; ++half) {
                        const uint4 w = lds16(kt + piece_at<RB, F8>(nt * 8 + g, 4 * half + c));
                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma<BF>(sc[nt], qf[4 * half + i], f8_to_h2<F8 == 2>(x[i]), f8_to_h2<F8 == 2>(x[i] >> 16));
                    }
                } else {
#pragma unroll
                    for (int kk = 0; kk < KK / 2; ++kk) {
                        uint32_t r[4];
                        ldsm4(kt + piece_at<RB, F8>(nt * 8 + (lane & 7), 4 * kk + (lane >> 3)), r);
                        mma<BF>(sc[nt], qf[2 * kk], r[0], r[1]);
                        mma<BF>(sc[nt], qf[2 * kk + 1], r[2], r[3]);
                    }
                }
            }
            // ---- scale, mask, running maximum ----
            const int kfirst = key0(st);
            const bool whole = valid == (KS == 32 ? 0xffffffffu : (1u << KS) - 1u) &&
                               kfirst + KS <= min(lim0, lim1);
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float a = sc[nt][j] * rs0, d = sc[nt][2 + j] * rs1;
                    if (!whole) {
                        const int kk = nt * 8 + 2 * c + j;
                        const bool in = (valid >> kk) & 1u;
                        if (!in || kfirst + kk >= lim0) a = -INFINITY;
                        if (!in || kfirst + kk >= lim1) d = -INFINITY;
                    }
                    sc[nt][j] = a;
                    sc[nt][2 + j] = d;
                    x0 = fmaxf(x0, a);
                    x1 = fmaxf(x1, d);
                }
#pragma unroll
            for (int of = 1; of < 4; of <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, of));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, of));
            }
            // O keeps its scale until a row's maximum has grown by 2^8
            const bool grow = x0 > m0 + kRescale || x1 > m1 + kRescale;
            if (__any_sync(0xffffffffu, grow)) {
                const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                const float f0 = rescale_factor(m0, n0), f1 = rescale_factor(m1, n1);
                m0 = n0;
                m1 = n1;
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int i = 0; i < ND; ++i) {
                    o[i][0] *= f0;
                    o[i][1] *= f0;
                    o[i][2] *= f1;
                    o[i][3] *= f1;
                }
            }
            // a row that has seen no key has only -inf scores: subtracting 0 gives P = 0
            constexpr float kShift = kPShift<E, F8>;
            const float z0 = m0 == -INFINITY ? 0.f : m0 - kShift, z1 = m1 == -INFINITY ? 0.f : m1 - kShift;
            // ---- P, O += P V ----
#pragma unroll
            for (int ks = 0; ks < KS / 16; ++ks) {
                uint32_t ph[4], pl[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // A fragment i: row g (i even) or g + 8, keys of n-tile 2 ks + i / 2
                    const int nt = 2 * ks + (i >> 1), r = (i & 1) * 2;
                    const float z = (i & 1) ? z1 : z0;
                    const float pa = fast_exp2(sc[nt][r] - z), pb = fast_exp2(sc[nt][r + 1] - z);
                    if (i & 1) l1 += pa + pb;
                    else l0 += pa + pb;
                    if constexpr (F8) {
                        ph[i] = F16::pack2(pa, pb);
                    } else {
                        ph[i] = E::pack2(pa, pb);
                        const float2 hf = E::unpack2(ph[i]);
                        pl[i] = E::pack2(pa - hf.x, pb - hf.y);
                    }
                }
                if constexpr (F8) {
                    // keys 16 ks + 2c, + 1, + 8, + 9; dims PB g .. of each: n-tile i
                    // of this thread's column g is dim PB g + i
                    constexpr int PB = D / 8;          // 16 or 8 dims a thread reads of a row
                    uint32_t w[4][PB / 4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = 16 * ks + 2 * c + (i & 1) + 8 * (i >> 1);
                        if constexpr (PB == 16) {
                            const uint4 t = lds16(vt + piece_at<RB, F8>(key, g));
                            w[i][0] = t.x; w[i][1] = t.y; w[i][2] = t.z; w[i][3] = t.w;
                        } else {
                            const uint2 t = lds8(vt + piece_at<RB, F8>(key, g >> 1) + 8 * (g & 1));
                            w[i][0] = t.x; w[i][1] = t.y;
                        }
                    }
#pragma unroll
                    for (int q4 = 0; q4 < PB / 4; ++q4) {
                        const uint32_t a = __byte_perm(w[0][q4], w[1][q4], 0x5140), a2 = __byte_perm(w[0][q4], w[1][q4], 0x7362);
                        const uint32_t e = __byte_perm(w[2][q4], w[3][q4], 0x5140), e2 = __byte_perm(w[2][q4], w[3][q4], 0x7362);
                        mma<BF>(o[4 * q4 + 0], ph, f8_to_h2<F8 == 2>(a), f8_to_h2<F8 == 2>(e));
                        mma<BF>(o[4 * q4 + 1], ph, f8_to_h2<F8 == 2>(a >> 16), f8_to_h2<F8 == 2>(e >> 16));
                        mma<BF>(o[4 * q4 + 2], ph, f8_to_h2<F8 == 2>(a2), f8_to_h2<F8 == 2>(e2));
                        mma<BF>(o[4 * q4 + 3], ph, f8_to_h2<F8 == 2>(a2 >> 16), f8_to_h2<F8 == 2>(e2 >> 16));
                    }
                } else {
#pragma unroll
                    for (int np = 0; np < ND / 2; ++np) {
                        uint32_t r[4];
                        ldsm4t(vt + piece_at<RB, F8>(16 * ks + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * np + (lane >> 4)), r);
                        mma<BF>(o[2 * np], ph, r[0], r[1]);
                        mma<BF>(o[2 * np], pl, r[0], r[1]);
                        mma<BF>(o[2 * np + 1], ph, r[2], r[3]);
                        mma<BF>(o[2 * np + 1], pl, r[2], r[3]);
                    }
                }
            }
            __syncwarp();      // every lane has read the stage before it is filled again
        }
        cp_async_wait<0>();
        __syncwarp();

        // ---- merge the four warps (in order), write the tile or its part ----
#pragma unroll
        for (int of = 1; of < 4; of <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, of);
            l1 += __shfl_xor_sync(0xffffffffu, l1, of);
        }
        float* wo = reinterpret_cast<float*>(ring);
        const int rows_here = rows - row_base;     // (rows behind the last need no result)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (8 * half >= rows_here) continue;
            float* to = wo + (g + 8 * half) * C::o_row;
            if constexpr (F8) {
                // dims D / 8 (2c + j) .. + D / 8 - 1
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < ND; i += 4)
                        *reinterpret_cast<float4*>(to + C::o_at((D / 8) * (2 * c + j) + i)) =
                            make_float4(o[i][2 * half + j], o[i + 1][2 * half + j], o[i + 2][2 * half + j], o[i + 3][2 * half + j]);
            } else {
#pragma unroll
                for (int i = 0; i < ND; ++i)
                    *reinterpret_cast<float2*>(to + 8 * i + 2 * c) = make_float2(o[i][2 * half], o[i][2 * half + 1]);
            }
        }
        if (c == 0) {
            float* mw = ml + warp * kRows * 2;
            mw[2 * g] = m0;
            mw[2 * g + 1] = l0;
            mw[2 * (g + 8)] = m1;
            mw[2 * (g + 8) + 1] = l1;
        }
        __syncthreads();
        const int r = tid >> 3;
        if (r < rows_here) {
            // dims 32 i + d0 .. + 3: the eight threads of a row read side by side
            constexpr int N = D / 32;
            const int d0 = (tid & 7) * 4;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[(w * kRows + r) * 2]);
            float L = 0.f;
            float4 acc[N];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = ml[(w * kRows + r) * 2];
                const float f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
                L += f * ml[(w * kRows + r) * 2 + 1];
                const float* src = reinterpret_cast<const float*>(smem + w * C::warp_bytes) + r * C::o_row;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float4 t = *reinterpret_cast<const float4*>(src + C::o_at(32 * i + d0));
                    acc[i].x += f * t.x;
                    acc[i].y += f * t.y;
                    acc[i].z += f * t.z;
                    acc[i].w += f * t.w;
                }
            }
            if (c0 == 0 && c1 == sq.chunks) {
                const float vs = F8 && p.kv.scale_v ? p.kv.scale_v[h] : 1.f;
                const bool none = L == 0.f;        // no visible key (a NaN sum is not that)
                const float inv = none ? 0.f : vs / L;
                const int i = over(row_base + r, p.by_group);
                const int64_t row = (int64_t)(sq.q_row + i) * p.Hq + h * p.G + (row_base + r) - i * p.G;
                typename E::T* dst = static_cast<typename E::T*>(p.out) + row * D + d0;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    *reinterpret_cast<uint2*>(dst + 32 * i) =
                        none ? make_uint2(0u, 0u)
                             : make_uint2(E::pack2(acc[i].x * inv, acc[i].y * inv), E::pack2(acc[i].z * inv, acc[i].w * inv));
                if (p.lse && (tid & 7) == 0) p.lse[row] = none ? -INFINITY : (M + __log2f(L) - kPShift<E, F8>) * kLn2;
            } else {
                const int slot = 2 * blockIdx.x + (c0 == 0 ? 1 : 0);
                float* dst = ws_o + ((int64_t)slot * kRows + r) * D + d0;
#pragma unroll
                for (int i = 0; i < N; ++i) *reinterpret_cast<float4*>(dst + 32 * i) = acc[i];
                if ((tid & 7) == 0)
                    *reinterpret_cast<float2*>(ws_ml + ((int64_t)slot * kRows + r) * 2) = make_float2(M, L);
            }
        }
        __syncthreads();       // the rings are free for the next tile
    }
}

// Block x joins the parts of the tile that border x (between the ranges of
// CTAs x and x + 1) cuts first: a warp per row, the parts' (m, sum) a lane
// each, eight parts of O in flight.
template <class E, int D, int F8>
__global__ void __launch_bounds__(32 * kRows, 1) attn_rows_merge(const SeqAttn p, uint64_t ctas_mul) {
    constexpr int chunk = RowsCfg<D, F8>::chunk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // The lists are older than the main kernel, which waited for them before
    // this one could start; its parts are not.  (Every block waits, also those
    // with nothing to do: this grid must not be over before the main one.)
    const Line line = line_at(p, chunk, ctas_mul, 1);
    int x = 0;
    int64_t th = 0;
    Seq sq{};
    if (line.b < p.kv.num_seqs) {
        sq = line.seq;
        split_unit(line.at - line.start, sq.chunks + kCharge, x, th);
    }
    grid_dependency_wait();
    const int n = sq.chunks, c = cut(x, n);
    // not cut here, or first cut earlier
    if (c == 0 || c == n || cut(x - line.per, n) > 0) return;
    const int tile = over((int)th, p.by_heads), h = (int)th - tile * p.kv.Hkv;
    const int rows = sq.n_q * p.G, row_base = tile * kRows;
    // one before this border and one behind each border that still cuts
    const int parts = 2 + (int)((uint32_t)(n - 1 + kCharge / 2 - x) / (uint32_t)min(line.per, (int64_t)0x7fffffff));
    const float* ws_o = static_cast<const float*>(p.ws);
    const float* ws_ml = ws_o + (int64_t)2 * kMaxCtas * kRows * D;
    auto slot_of = [&](int i) { return i == 0 ? 2 * (int)blockIdx.x + 1 : 2 * ((int)blockIdx.x + i); };

    constexpr int W = D / 32;                     // dims of a lane
    // (as many warps as the longest sequence is said to have rows)
    for (int r = warp; r < kRows && row_base + r < rows; r += blockDim.x >> 5) {
        float M = -INFINITY, L = 0.f, acc[W];
#pragma unroll
        for (int i = 0; i < W; ++i) acc[i] = 0.f;
        for (int i0 = 0; i0 < parts; i0 += 32) {
            const int m = min(32, parts - i0);
            float v[8][W];
            auto load = [&](int j0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float* src = ws_o + ((int64_t)slot_of(i0 + min(j0 + j, m - 1)) * kRows + r) * D + lane * W;
#pragma unroll
                    for (int i = 0; i < W; i += 2)
                        *reinterpret_cast<float2*>(&v[j][i]) = *reinterpret_cast<const float2*>(src + i);
                }
            };
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < m) ml = *reinterpret_cast<const float2*>(ws_ml + ((int64_t)slot_of(i0 + lane) * kRows + r) * 2);
            load(0);
            const float m_new = fmaxf(M, warp_max(ml.x));
            const float old = rescale_factor(M, m_new), f = rescale_factor(ml.x, m_new);
            M = m_new;
            L = L * old + warp_sum(ml.y * f);
#pragma unroll
            for (int i = 0; i < W; ++i) acc[i] *= old;
            for (int j0 = 0; j0 < m; j0 += 8) {
                if (j0 > 0) load(j0);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float g = __shfl_sync(0xffffffffu, f, (j0 + j) & 31);
                    if (j0 + j < m) {
#pragma unroll
                        for (int i = 0; i < W; ++i) acc[i] += g * v[j][i];
                    }
                }
            }
        }
        const bool none = L == 0.f;
        const float vs = F8 && p.kv.scale_v ? p.kv.scale_v[h] : 1.f;
        const float inv = none ? 0.f : vs / L;
        const int i = over(row_base + r, p.by_group);
        const int64_t row = (int64_t)(sq.q_row + i) * p.Hq + h * p.G + (row_base + r) - i * p.G;
        typename E::T* out = static_cast<typename E::T*>(p.out) + row * D + lane * W;
#pragma unroll
        for (int k = 0; k < W; k += 2)
            *reinterpret_cast<uint32_t*>(out + k) = none ? 0u : E::pack2(acc[k] * inv, acc[k + 1] * inv);
        if (p.lse && lane == 0) p.lse[row] = none ? -INFINITY : (M + __log2f(L) - kPShift<E, F8>) * kLn2;
    }
}

template <class E, int D, int F8, bool PAGED>
cudaError_t launch_rows_t(const SeqAttn& p, int num_sms, cudaStream_t stream) {
    using C = RowsCfg<D, F8>;
    auto kern = attn_rows_kernel<E, D, F8, PAGED>;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::total);
    if (err != cudaSuccess) return err;
    const int ctas = 2 * num_sms < kMaxCtas ? 2 * num_sms : kMaxCtas;
    const uint64_t mul = ~uint64_t(0) / (uint64_t)ctas + 1;        // x / ctas = high word of x * mul
    err = launch_pdl(kern, dim3(ctas), dim3(kThreads), C::total, stream, p, mul);
    if (err != cudaSuccess) return err;
    count_launches(1);
    // shorter tiles are never cut
    const int64_t longest = p.kv.page_table ? (int64_t)p.kv.max_pages * p.kv.page_size : p.kv.rows;
    if (longest > (int64_t)(kMinCut - 1) * C::chunk) {
        const int64_t most = (int64_t)p.max_q_len * p.G;           // rows of a kv head
        err = launch_pdl(attn_rows_merge<E, D, F8>, dim3(ctas - 1), dim3(32 * (int)min(most, (int64_t)kRows)), 0, stream, p,
                         mul);
        if (err == cudaSuccess) count_launches(1);
    }
    return err;
}

template <class E, int D>
cudaError_t launch_rows_d(const SeqAttn& p, int num_sms, cudaStream_t stream) {
    if (!p.kv.page_table) return launch_rows_t<E, D, 0, false>(p, num_sms, stream);
    switch (p.kv.f8) {
        case 0: return launch_rows_t<E, D, 0, true>(p, num_sms, stream);
        case 1: return launch_rows_t<E, D, 1, true>(p, num_sms, stream);
        default: return launch_rows_t<E, D, 2, true>(p, num_sms, stream);
    }
}

}  // namespace

size_t attn_rows_ws_bytes(int D) { return (size_t)2 * kMaxCtas * kRows * (D + 2) * 4; }

cudaError_t launch_attn_rows(const SeqAttn& p, sfa_dtype dtype, int num_sms, cudaStream_t stream) {
    const bool bf16 = dtype == SFA_DTYPE_BF16;
    if (p.kv.D == 128)
        return bf16 ? launch_rows_d<BF16, 128>(p, num_sms, stream) : launch_rows_d<F16, 128>(p, num_sms, stream);
    return bf16 ? launch_rows_d<BF16, 64>(p, num_sms, stream) : launch_rows_d<F16, 64>(p, num_sms, stream);
}

}  // namespace sfa
