// Dense attention of many query rows over packed rows or a paged cache on the
// 5th-generation tensor cores.
//
//     s_j = scale * q.k_j  (j < kv_len; causal: j <= i + kv_len - q_len)
//     out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  m the running maximum
//
// A work item is one kv head and 2 x TR query tokens of a sequence, TR =
// 128 / G: two M-tiles of 128 rows (row r of a tile: token r / G, head r % G,
// so a K / V tile serves all G heads), against its visible keys in steps of
// 128.  CTAs are persistent, one per SM.  All items lie on one line, each as
// long as its visible keys plus a fixed charge for what an item costs besides,
// and the line is cut into equal ranges, one per CTA, whatever the mix of
// lengths: a cut inside an item falls on a step (never within kMinShare steps
// of an item's end) and leaves the item in parts, fp32 in the workspace, at
// most two of them from a CTA (the item it ends and the one it begins), which
// attn_tc_merge joins in order of their keys.
//
// Warp roles, 384 threads (512 with movers):
//   - softmax warpgroups 0, 1: tile t, thread = row = TMEM lane.  Read the
//     128 scores of a step, mask them (only where a row's limit or a missing
//     page falls into the step), update m (O is rescaled only when m grows by
//     more than 2^8), write P = exp2(s - m) rounded to 16 bits over S.  At the
//     end divide and store.
//   - MMA thread: S_t = Q_t K^T into TMEM, O_t += P_t V with P from TMEM and
//     V an MN-major operand; tile 0's P.V and next Q.K^T run while the
//     softmax works on tile 1, and the other way round.
//   - loader: Q tiles and a ring of 128-key K and V tiles in the order the
//     MMAs use them, running ahead across items.  Packed rows and 16-bit pages
//     of a multiple of 16 tokens come by TMA (one warp; a page is a box of a
//     4-D map).  8-bit pages (of a multiple of 8) come by TMA into two swizzled
//     staging tiles, from which four mover warps write them out as fp16 (exact)
//     into the tiles the MMA reads.  Pages of other sizes come row by row
//     through the movers' 16-byte cp.async.  Rows without a key are zeros.
// TMEM: tile t at column 256 t: S / P in [0, 128), O in [128, 128 + D).
//
// With an 8-bit cache both products run in fp16.  bf16 rows of q are scaled to
// a largest magnitude in [2^14, 2^15) by a power of two each, which leaves with
// the scores: elements down to 2^-31 of the row's largest are exact, smaller
// ones off by at most 2^-39 of it.
//
// P is rounded once to 16 bits (at most half a step of the output's type per
// weight, so the output moves by no more than its own rounding of
// sum_j p_j |v_j|); a second P.V on the remainders would cost half as many
// MMAs again.  fp16 P carries a factor 2^7 so that weights down to 2^-21 of the
// largest stay normal.  Sums of P use the unrounded fp32 values.
//
// V rows behind kv_len (the next sequence's, or whatever a page holds) would
// turn 0 x NaN into NaN: where TMA brought them the loader waits for such a
// tile itself, writes zeros over those rows and then hands it on.
//
// Bound: the way from one barrier to the next.  S, softmax, P and P.V of a step
// follow one another; two tiles of a CTA hide the one behind the other, and
// still nothing is busy throughout (tensor pipe, issue slots, exponentials' unit:
// long prompt 72%, 41%, 36%; chunks over 16-bit pages 60%, 40%, 30%, over E4M3
// 48%, 44%, 24%, whose conversion takes slots; short prompts 12%, 23%, 13%).  208
// registers a softmax thread hold a row's 128 scores, so that S is read from
// TMEM once.  Measured: one causal prompt of 16,384 tokens, 32/8 heads of 128,
// 1.38 to 1.53 ms, 1.43 to 1.59 PFLOP/s (0.85 to 0.94 of a sustained library
// product's rate); chunks of 200 to 1,024 tokens over up to 8,192 keys in
// 32-token pages 200 to 214 us, 1.17 to 1.25 PFLOP/s; over E4M3 pages 386 to 417
// us, 1.01 to 1.09 PFLOP/s; 40 prompts of up to 700 tokens, 12/4 heads of 64, 31 us.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace sfa {
namespace {

constexpr int kTileM = 128;
constexpr int kStep = 128;                  // keys of a step
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kMoveWarp = 12, kMovers = 128; // the movers: warps 12 to 15
constexpr int kTmemCols = 512, kTileCols = 256, kOCol = 128;
constexpr float kRescale = 8.0f;            // log2 units
constexpr int kItemRows = 2 * kTileM;
constexpr int kMinShare = 2;                // fewest steps of a part (1: 8 prompts of 300 tokens 22.7 instead of 14.9 us)
// Pages of a multiple of this many tokens come by TMA, others row by row.  8
// sequences' chunks of 512 tokens over 4,096 keys, 32/8 heads of 128: 16-bit
// pages of 32 tokens 195 us, of 16 217, of 8 317 (row by row 302); E4M3 pages of
// 16 tokens 290 us, of 8 300 (row by row 415).
constexpr int kMinBox = 16, kMinBox8 = 8;
constexpr int kMinRange = kStep;            // shortest range of a CTA, in keys
constexpr int kMaxCtas = 160;               // ranges (the workspace's size goes by it)

// Where K and V come from: packed rows, or pages by TMA; or gathered rows of
// 16-bit, E4M3 or E5M2 pages.
enum { SRC_PACKED = 0, SRC_PAGES = 1, SRC_G16 = 2, SRC_E4M3 = 3, SRC_E5M2 = 4 };

// Block size and registers a thread: at launch, then of the control warps and
// of the softmax warps.  The movers come as a warpgroup of their own.
template <int SRC>
struct TcBlock {
    static constexpr bool movers = SRC >= SRC_G16;
    static constexpr int threads = movers ? 512 : 384;
    static constexpr int launch = movers ? 128 : 168, control = movers ? 64 : 80, softmax = movers ? 192 : 208;
    static_assert(softmax * kSoftWarps * 32 + control * (threads - kSoftWarps * 32) <= launch * threads,
                  "the register split fits what the block was launched with");
};

template <int D, int SRC>
struct TcSmem {
    static constexpr bool f8 = SRC >= SRC_E4M3, gather = SRC >= SRC_G16;
    static constexpr int panels = D / 64;
    static constexpr int panel = kStep * 128;              // 128 rows x 128 bytes
    static constexpr int tile = panels * panel;            // Q, K or V tile
    static constexpr int slots = D == 128 ? (f8 ? 4 : 5) : 8;
    static constexpr int q = 0;
    static constexpr int ring = 2 * tile;
    static constexpr int staging = ring + slots * tile;    // two tiles of 8-bit rows
    static constexpr int rows = staging + (f8 ? 2 * kStep * D : 0);   // row numbers of two steps
    static constexpr int bars = rows + (gather ? 2 * kStep * 4 : 0);
    static constexpr int items = bars + 8 * 38;            // the two items being worked on
    static constexpr int abort = items + 2 * 48;
    static constexpr int tmem_slot = abort + 4;
    static constexpr int total = abort + 16;
    static constexpr int alloc = total + 1024;             // room to align the base to 1024
    static_assert(alloc <= 232448, "dynamic shared memory per block");
};

enum {
    B_Q = 0,            // + t: Q tile t of the item there
    B_Q_FREE = 2,       // every Q.K^T of the item done
    B_S = 3,            // + t: S_t written (and the P.V before it done)
    B_P = 5,            // + t: all of P_t written (one arrival a warp)
    B_PH = 7,           // + t: P_t of keys 0..63 written
    B_O = 9,            // + t: O_t of the item complete
    B_TAIL = 11,        // V tile landed whose tail is still to be cleared
    B_DRAIN = 12,
    B_ROWS = 13,        // the movers met (one arrival a warp)
    B_FULL = 14,        // + slot (gathered: one arrival a mover warp that fills it)
    B_FREE = 22,        // + slot
    B_ITEM = 30,        // + i: item slot i written
    B_ITEM_FREE = 32,   // + i: item slot i read by the MMA, softmax and mover warps
    B_STAGE = 34,       // + i: staging tile i landed
    B_STAGE_FREE = 36   // + i: staging tile i read (one arrival a mover warp that does)
};

struct TcParams {
    SeqAttn a;
    int TR, hnd;
    Divisor by_unit;                    // tokens of an item, 2 TR
    uint64_t ctas_mul;                  // x / ctas = high word of x * ctas_mul for x < 2^56
    int charge;                         // an item's fixed cost, in keys
    int out32;                          // out is 32-byte aligned
    int box, box_shift, boxes;          // keys of a TMA box (and its log2), boxes of a step
    float* ws_o;                        // [2 * kMaxCtas][D / 4][kItemRows][4] parts
    float* ws_ml;                       // [2 * kMaxCtas][kItemRows][2] (m, sum)
    struct CutItem* ws_cut;             // [kMaxCtas] the item that each range cuts first
};

// An item whose first part a range holds: what attn_tc_merge has to join.
// Written by every CTA, cut or not.
struct CutItem {
    int N, c;                           // steps (0: none) and length of the item
    int h, q_row, n_q, tok0;            // as in Item
    int64_t x, per;                     // end of the range within the item, length of a range
};

// A sequence on the line.  Tile j holds tokens [j U, (j + 1) U), U = 2 TR, and
// sees max(0, min((j + 1) U, n_q) + off) keys, off = kv_len - n_q, when causal,
// else kv_len.
struct Seq {
    int q_row, n_q, k_row, kv_len, tiles;
};

// x / (2 TR)
__device__ __forceinline__ int units(const TcParams& p, int x) {
    return over(x, p.by_unit);
}

// x / page_size
__device__ __forceinline__ int page_slot(const TcParams& p, int x) {
    return over(x, p.a.kv.by_page);
}

__device__ __forceinline__ Seq seq_of(const TcParams& p, int b) {
    const int2 q = seq_rows(p.a.cu_q, b, p.a.tokens);
    const int2 k = seq_keys(p.a.kv, b);
    Seq s;
    s.q_row = q.x;
    s.n_q = q.y - q.x;
    s.k_row = k.x;
    s.kv_len = k.y;
    s.tiles = units(p, s.n_q + 2 * p.TR - 1);
    return s;
}

// Keys visible to the last of the tokens before tok_end.
__device__ __forceinline__ int visible(const TcParams& p, const Seq& s, int tok_end) {
    if (!p.a.causal) return s.kv_len;
    return max(0, min(tok_end, s.n_q) + s.kv_len - s.n_q);
}

__device__ __forceinline__ int cost(const TcParams& p, const Seq& s, int j) {
    return visible(p, s, (j + 1) * 2 * p.TR) + p.charge;
}

// Cost of one kv head's tiles before tile j.
__device__ __forceinline__ int64_t cost_before(const TcParams& p, const Seq& s, int j) {
    int64_t sum = (int64_t)j * p.charge;
    if (!p.a.causal) return sum + (int64_t)j * s.kv_len;
    const int64_t U = 2 * p.TR, off = s.kv_len - s.n_q;
    int64_t full = j;                                  // tiles of U tokens among them
    if (j == s.tiles && j > 0) {
        sum += s.kv_len;                               // the last one ends at n_q
        --full;
    }
    const int64_t first = off < 0 ? min(full, (int64_t)units(p, (int)-off)) : 0;    // tiles that see no key
    return sum + (full - first) * off + U * (full * (full + 1) - first * (first + 1)) / 2;
}

// Steps of an item of N steps before point x of its length c.
__device__ __forceinline__ int cut(int64_t x, int c, int N) {
    if (x <= 0) return 0;
    if (x >= c) return N;
    // (fp32: monotonic in x, and the same wherever a border is looked at)
    const int st = (int)__fdividef(__ll2float_rn(x) * (float)N, (float)c);
    return st < kMinShare ? 0 : (st > N - kMinShare ? N : st);
}

// The line: its length, the length of a range, the point this CTA's range
// begins at, and the sequence (and its first point) that holds it.  One warp;
// every lane gets the answer.
struct Line {
    int64_t total, per, at, start;
    int b;
    Seq seq;
};

__device__ __forceinline__ Line line_at(const TcParams& p) {
    const int lane = threadIdx.x & 31, B = p.a.kv.num_seqs;
    Seq mine_seq{};
    auto length = [&](int b) -> int64_t {
        if (b >= B) return 0;
        mine_seq = seq_of(p, b);
        return cost_before(p, mine_seq, mine_seq.tiles) * p.a.kv.Hkv;
    };
    Line l;
    const int64_t first = length(lane);
    const Seq first_seq = mine_seq;
    int64_t sum = first;
    for (int b = lane + 32; b < B; b += 32) sum += length(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l.total = sum;
    l.per = max((int64_t)__umul64hi((uint64_t)l.total, p.ctas_mul) + 1, (int64_t)kMinRange);
    l.at = (int64_t)blockIdx.x * l.per;
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
            return l;
        }
        l.start += __shfl_sync(0xffffffffu, inc, 31);
    }
    return l;
}

// Tile and kv head that hold point `rel` of a sequence (tile by tile, its
// heads one after the other), and the point within the item.  One warp.
__device__ __forceinline__ void find_item(const TcParams& p, const Seq& s, int64_t rel, int& j, int& h, int64_t& x) {
    const int lane = threadIdx.x & 31, H = p.a.kv.Hkv;
    // the last of tiles j .. j + n that begins at or before rel, 32 tried at a time
    j = 0;
    for (int n = s.tiles - 1; n > 0;) {
        const int step = (n + 31) / 32, i = j + (lane + 1) * step;
        const bool below = (lane + 1) * step <= n && cost_before(p, s, i) * H <= rel;
        const int c = __popc(__ballot_sync(0xffffffffu, below));
        j += c * step;
        n = min(step - 1, n - c * step);
    }
    rel -= cost_before(p, s, j) * H;
    const int c = cost(p, s, j);
    h = min(H - 1, (int)__fdividef(__ll2float_rn(rel), (float)c));     // within one of the quotient
    if ((int64_t)h * c > rel) --h;
    if (h + 1 < H && (int64_t)(h + 1) * c <= rel) ++h;
    x = rel - (int64_t)h * c;
}

// A share of an item.
struct Item {
    int b, h;                   // b < 0: the end of the range
    int q_row, n_q, tok0;       // packed row of the sequence's first token, its rows, the item's first token
    int k_row, kv_len;
    int s0, n[2];               // first step, steps of each tile
    int whole;                  // all of the item's keys
    int pad;
};
static_assert(sizeof(Item) == 48, "TcSmem::items");

// Walks the shares of this CTA's range: the producer does, and hands each item
// to the MMA thread and the softmax through two slots in shared memory.
struct Walk {
    int64_t left, per;          // of the range: what is left, its length
    int64_t x;                  // point within the item (j, h)
    int b, j, h;
    Seq s;

    __device__ __forceinline__ void begin(const TcParams& p, const Line& l) {
        left = x = 0;
        per = l.per;
        b = l.b;
        j = h = 0;
        if (b >= p.a.kv.num_seqs) return;
        left = min(l.per, l.total - l.at);
        s = l.seq;
        find_item(p, s, l.at - l.start, j, h, x);
    }

    __device__ __forceinline__ bool next(const TcParams& p, Item& it) {
        const int U = 2 * p.TR;
        while (left > 0) {
            if (j == s.tiles) {                        // on to the next sequence with rows
                do {
                    if (++b >= p.a.kv.num_seqs) return false;
                    s = seq_of(p, b);
                } while (s.tiles == 0);
                j = h = 0;
            }
            const int c = cost(p, s, j);
            const int64_t x0 = x, x1 = min((int64_t)c, x + left);
            const int v1 = visible(p, s, (j + 1) * U), N = (v1 + kStep - 1) / kStep;
            const int s0 = cut(x0, c, N), s1 = cut(x1, c, N);
            it.b = b;
            it.h = h;
            it.q_row = s.q_row;
            it.n_q = s.n_q;
            it.tok0 = j * U;
            it.k_row = s.k_row;
            it.kv_len = s.kv_len;
            it.s0 = s0;
            it.whole = s0 == 0 && s1 == N;
            const bool two = it.tok0 + p.TR < s.n_q;   // the second tile has rows
            const int v0 = two ? visible(p, s, it.tok0 + p.TR) : v1;
            it.n[0] = max(0, min((v0 + kStep - 1) / kStep, s1) - s0);
            it.n[1] = two ? s1 - s0 : 0;
            if (s0 == 0 && s1 > 0 && s1 < N && (threadIdx.x & 31) == 0)
                p.ws_cut[blockIdx.x] = CutItem{N, c, h, s.q_row, s.n_q, j * U, x1, per};
            left -= x1 - x0;
            x = x1;
            if (x1 == c) {
                x = 0;
                if (++h == p.a.kv.Hkv) {
                    h = 0;
                    ++j;
                }
            }
            // (an item without keys belongs to the range it begins in)
            if (s1 > s0 || (N == 0 && x0 == 0)) return true;
        }
        return false;
    }
};

// Two 8-bit codes (low 16 bits of x) as two fp16.
template <bool E5>
__device__ __forceinline__ uint32_t codes_h2(uint32_t x) {
    const uint16_t in = (uint16_t)x;
    uint32_t h;
    if constexpr (E5) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(in));
    else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
    return h;
}

// Hands item number i (counting from 0) on; the end of the range as b < 0.  One thread.
template <class L>
__device__ __forceinline__ bool put_item(unsigned char* smem, uint32_t sbase, int i, const Item& it, int* err,
                                         volatile int* abort_flag) {
    const uint32_t bars = sbase + L::bars;
    if (i >= 2 && !mbar_wait(bars + 8 * (B_ITEM_FREE + (i & 1)), ((i >> 1) - 1) & 1, err, abort_flag)) return false;
    reinterpret_cast<Item*>(smem + L::items)[i & 1] = it;
    mbar_arrive(bars + 8 * (B_ITEM + (i & 1)));
    return true;
}
// Waits for item i; false if the wait gave up.
template <class L>
__device__ __forceinline__ bool get_item(unsigned char* smem, uint32_t sbase, int i, Item& it, int* err,
                                         volatile int* abort_flag) {
    if (!mbar_wait(sbase + L::bars + 8 * (B_ITEM + (i & 1)), (i >> 1) & 1, err, abort_flag)) return false;
    const int4* src = reinterpret_cast<const int4*>(smem + L::items + (i & 1) * sizeof(Item));
    int4* dst = reinterpret_cast<int4*>(&it);
    dst[0] = src[0];
    dst[1] = src[1];
    dst[2] = src[2];
    return true;
}

// Two fp32 in a register pair: packed arithmetic, each half rounded as alone.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float low(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float high(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// 32 bytes at once (a full sector a thread).
__device__ __forceinline__ void st_32(void* to, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// MMA issue by a whole converged warp, one lane elected in the instruction:
// with every operand the same in all lanes the descriptors stay in uniform
// registers.  Issued from one lane's branch instead, 16 MMAs took twice as long
// next to busy softmax warps.  Descriptors as low words (address in 16-byte units
// and leading offset) over a constant high word.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 a, b;\nsetp.ne.b32 p, %5, 0;\nelect.sync _|q, 0xffffffff;\n"
        "mov.b64 a, {%1, %3};\nmov.b64 b, {%2, %3};\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 b;\nsetp.ne.b32 p, %5, 0;\nelect.sync _|q, 0xffffffff;\n"
        "mov.b64 b, {%2, %3};\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrive on `bar` when every MMA the elected lane issued so far has completed.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n.reg .pred q;\nelect.sync _|q, 0xffffffff;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
        : "memory");
}

// 16-byte piece `ch` of 8-bit row r in a staging tile: TMA's swizzle for rows
// of 128 or 64 bytes.
template <int D>
__device__ __forceinline__ int staged(int r, int ch) {
    return r * D + ((ch ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4);
}

// The movers, thread x of kMovers: K and V tiles that TMA does not bring into
// the ring by itself.
template <int D, int SRC>
__device__ __forceinline__ void move_rows(const TcParams& p, unsigned char* smem, uint32_t sbase, int x) {
    using L = TcSmem<D, SRC>;
    constexpr bool F8 = L::f8, E5 = SRC == SRC_E5M2;
    constexpr int EB = F8 ? 1 : 2, RB = D * EB;
    constexpr int PR = RB / 16;                              // 16-byte pieces of a row
    const SeqAttn& a = p.a;
    int* err = a.err_word;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::abort);
    auto bar = [&](int i) { return sbase + L::bars + 8 * i; };
    auto all = [](bool v) { return __all_sync(0xffffffffu, v) != 0; };
    // one arrival for this warp, behind what all its lanes did
    auto arrive = [&](int b) {
        __syncwarp();
        if ((x & 31) == 0) mbar_arrive(bar(b));
    };
    static_assert(kMovers == kStep, "a thread a row number");
    uint32_t* rows = reinterpret_cast<uint32_t*>(smem + L::rows);
    const bool tma = F8 && p.box >= kMinBox8;                     // staging tiles filled by the loader's TMA
    int loads = 0, meetings = 0, steps = 0;    // tiles, barrier phases, steps of the items before
    bool ok = true;
    // the four mover warps are here (with what they wrote to shared memory)
    auto together = [&]() -> bool {
        arrive(B_ROWS);
        return all(mbar_wait(bar(B_ROWS), meetings++ & 1, err, abort_flag));
    };
    for (int number = 0; ok; ++number) {
        Item it;
        ok = all(get_item<L>(smem, sbase, number, it, err, abort_flag));
        if (!ok) break;
        arrive(B_ITEM_FREE + (number & 1));
        if (it.b < 0) break;
        const int n = max(it.n[0], it.n[1]), s0 = it.s0, kv_len = it.kv_len, h = it.h;
        const int32_t* table = a.kv.page_table + (int64_t)it.b * a.kv.max_pages;
        // page of this thread's key of a step, looked up a step ahead (left as
        // loaded, so that nothing waits for the load)
        int ahead;
        auto look_up = [&](int st) {
            const int key = (s0 + st) * kStep + x;
            ahead = st < n && key < kv_len ? table[page_slot(p, key)] : -1;
        };
        // Row numbers (in units of D elements) of step st's keys, in the two
        // tables by turns over all steps of the range, whatever the item: a
        // table is written again two steps later, and by then every warp has
        // met the others in the step between, after its last read.  (Turns
        // that began anew with each item would write the table that a slower
        // warp still reads for the last step of an odd number.)
        auto table_of = [&](int st) { return rows + ((steps + st) & 1) * kStep; };
        auto find_rows = [&](int st) -> bool {
            const int key = (s0 + st) * kStep + x, place = key - page_slot(p, key) * a.kv.page_size;
            const uint32_t pg = (uint32_t)ahead;
            table_of(st)[x] = pg >= (uint32_t)a.kv.num_pages ? 0xffffffffu
                              : p.hnd ? (pg * a.kv.Hkv + h) * a.kv.page_size + place
                                      : (pg * a.kv.page_size + place) * a.kv.Hkv + h;
            return together();
        };
        auto wait_free = [&](int load) {
            return load < L::slots ||
                   all(mbar_wait(bar(B_FREE + load % L::slots), (load / L::slots - 1) & 1, err, abort_flag));
        };
        // starts the copy of tile y, ring index `load`, row by row
        auto copy = [&](int y, int load) -> bool {
            if (y < 2 * n) {
                const int st = y >> 1;
                // (here, too: all have read what the staging tile held)
                if (!(y & 1)) {
                    if (!find_rows(st)) return false;
                    look_up(st + 1);
                } else if (F8) {
                    if (!together()) return false;
                }
                if (!F8 && !wait_free(load)) return false;
                const char* src = static_cast<const char*>((y & 1) ? a.kv.v : a.kv.k);
                unsigned char* stage = smem + L::staging + (load & 1) * kStep * D;
                unsigned char* slot = smem + L::ring + (load % L::slots) * L::tile;
                const uint32_t* row_of = table_of(st);
                const int ch = x % PR;
                // kMovers / PR rows at a time, a row's pieces side by side
#pragma unroll 8
                for (int r = x / PR; r < kStep; r += kMovers / PR) {
                    const uint32_t row = row_of[r];
                    const bool in = row != 0xffffffffu;
                    unsigned char* dst = F8 ? stage + staged<D>(r, ch)
                                            : slot + (ch >> 3) * L::panel + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
                    cp_async_16_zfill(dst, src + (in ? (int64_t)row * RB + ch * 16 : 0), in ? 16 : 0);
                }
            }
            cp_async_commit();
            return true;
        };
        if (!tma && n > 0) {
            look_up(0);
            ok = copy(0, loads);
        }
        // Rows r0, r0 + stride, .. of tile `load`, from its staging tile into its
        // slot.  A page goes on behind the last token: rows from `real` on are
        // written as zeros.
        auto widen = [&](int load, int r0, int stride, int real) {
            const unsigned char* stage = smem + L::staging + (load & 1) * kStep * D;
            unsigned char* slot = smem + L::ring + (load % L::slots) * L::tile;
            for (int r = r0; r < kStep; r += stride) {
                // lanes = rows: the swizzle puts neighbours on different banks on both sides
                uint4 c[PR];
#pragma unroll
                for (int i = 0; i < PR; ++i) c[i] = *reinterpret_cast<const uint4*>(stage + staged<D>(r, i));
                if (r >= real) {
#pragma unroll
                    for (int i = 0; i < PR; ++i) c[i] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < PR; ++i) {
                    const int to = (i >> 2) * L::panel + r * 128 + ((((i & 3) * 2) ^ (r & 7)) << 4);
                    *reinterpret_cast<uint4*>(slot + to) = make_uint4(codes_h2<E5>(c[i].x), codes_h2<E5>(c[i].x >> 16),
                                                                      codes_h2<E5>(c[i].y), codes_h2<E5>(c[i].y >> 16));
                    *reinterpret_cast<uint4*>(slot + (to ^ 16)) = make_uint4(codes_h2<E5>(c[i].z), codes_h2<E5>(c[i].z >> 16),
                                                                             codes_h2<E5>(c[i].w), codes_h2<E5>(c[i].w >> 16));
                }
            }
        };
        if (tma) {
            // Warps 0, 1 do the K tiles, 2, 3 the V tiles: each pair goes at its own pace.
            const int g = x >> 6;
            for (int st = 0; st < n && ok; ++st) {
                const int load = loads + 2 * st + g;
                ok = all(mbar_wait(bar(B_STAGE + g), (load >> 1) & 1, err, abort_flag)) && wait_free(load);
                if (!ok) break;
                widen(load, x & 63, kMovers / 2, kv_len - (s0 + st) * kStep);
                arrive(B_STAGE_FREE + g);
                fence_proxy_async_smem();
                arrive(B_FULL + load % L::slots);
            }
            loads += 2 * n;
            continue;
        }
        for (int y = 0; y < 2 * n && ok; ++y) {
            // the next tile on its way, this one landed
            ok = copy(y + 1, loads + 1);
            cp_async_wait<1>();
            if (!ok) break;
            if constexpr (F8) {
                // (pieces are read by other threads than copied them)
                ok = together() && wait_free(loads);
                if (!ok) break;
                widen(loads, x, kMovers, kStep);
            }
            fence_proxy_async_smem();
            arrive(B_FULL + loads % L::slots);
            ++loads;
        }
        steps += n;
    }
    cp_async_wait<0>();
}

template <class E, int D, int SRC>
__global__ void __launch_bounds__(TcBlock<SRC>::threads, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const TcParams p) {
    using L = TcSmem<D, SRC>;
    constexpr bool PAGED = SRC != SRC_PACKED, F8 = L::f8;
    constexpr bool kScaledQ = F8 && std::is_same<E, BF16>::value;    // q's rows go to fp16
    using M = typename std::conditional<F8, F16, E>::type;           // element type of the MMAs
    constexpr bool kBf16 = std::is_same<M, BF16>::value;
    constexpr uint32_t kIdescQK = idesc_f16(kTileM, kStep, kBf16, false, false);
    constexpr uint32_t kIdescPV = idesc_f16(kTileM, D, kBf16, false, true);
    constexpr float kPShift = kBf16 ? 0.f : 7.f;

    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) { return sbase + L::bars + 8 * i; };
    const SeqAttn& a = p.a;
    const int G = a.G;
    int* err = a.err_word;

    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::abort);
    if (tid == 0) {
        *abort_flag = 0;
        mbar_init(bar(B_ROWS), kMovers / 32);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_ITEM + i), 1);
            mbar_init(bar(B_ITEM_FREE + i), kSoftWarps + 1 + (L::gather ? kMovers / 32 : 0));
            mbar_init(bar(B_STAGE + i), 1);
            mbar_init(bar(B_STAGE_FREE + i), kMovers / 64);
        }
        mbar_init(bar(B_Q_FREE), 1);
        mbar_init(bar(B_TAIL), 1);
        mbar_init(bar(B_DRAIN), 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(B_S + t), 1);
            mbar_init(bar(B_P + t), 4);
            mbar_init(bar(B_PH + t), 4);
            mbar_init(bar(B_O + t), 1);
            mbar_init(bar(B_Q + t), kScaledQ ? 4 : 1);
        }
        for (int s = 0; s < L::slots; ++s) {
            mbar_init(bar(B_FULL + s), !L::gather ? 1 : (L::f8 && p.box >= kMinBox8 ? kMovers / 64 : kMovers / 32));
            mbar_init(bar(B_FREE + s), 1);
        }
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(sbase + L::tmem_slot, kTmemCols);
    Item next_item;                     // the loader: found while the others set up
    bool more = false;
    Walk walk;
    if (warp == kLoadWarp) {
        if (lane == 0) {
            tma_prefetch_map(&mq);
            tma_prefetch_map(&mk);
            tma_prefetch_map(&mv);
        }
        grid_dependency_wait();
        walk.begin(p, line_at(p));
        if (lane == 0) p.ws_cut[blockIdx.x].N = 0;
        more = walk.next(p, next_item);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::tmem_slot);
    grid_dependency_wait();
    grid_launch_dependents();

    if (warp >= kSoftWarps) {
        regs_release<TcBlock<SRC>::control>();
        if (L::gather && warp >= kMoveWarp) {
            if constexpr (L::gather) move_rows<D, SRC>(p, smem, sbase, tid - kMoveWarp * 32);
        } else if (warp == kLoadWarp) {
            // ============================ loader ============================
            int number = 0;
            int items = 0, loads = 0, tails = 0;   // items with keys, tiles loaded, tiles cleared
            int qs[2] = {0, 0};                    // Q tiles loaded
            const bool tma = !L::gather || (L::f8 && p.box >= kMinBox8);
            bool ok = true;
            for (;; more = walk.next(p, next_item)) {
                if (!more) next_item.b = -1;
                if (lane == 0) ok = put_item<L>(smem, sbase, number, next_item, err, abort_flag);
                ++number;
                ok = __all_sync(0xffffffffu, ok);
                if (!more || !ok) break;
                const Item& it = next_item;
                const int n = max(it.n[0], it.n[1]);
                if (n == 0) continue;
                if constexpr (!kScaledQ) {
                    if (items > 0) ok = mbar_wait(bar(B_Q_FREE), (items - 1) & 1, err, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (it.n[t] == 0) continue;
                        ++qs[t];
                        if (lane != 0) continue;
                        mbar_arrive_expect_tx(bar(B_Q + t), L::panels * p.TR * G * 128);
                        for (int pn = 0; pn < L::panels; ++pn)
                            tma_load_3d(sbase + L::q + t * L::tile + pn * L::panel, &mq, pn * 64, it.h * G,
                                        it.q_row + it.tok0 + t * p.TR, bar(B_Q + t));
                    }
                }
                ++items;
                if (!tma) continue;
                // page of this lane's box of a step, -1 if there is none to read
                // (left as loaded, so that nothing waits for the load)
                auto page_of = [&](int st) -> int {
                    const int key = (it.s0 + st) * kStep + lane * p.box;
                    if (st >= n || lane >= p.boxes || key >= it.kv_len) return -1;
                    return a.kv.page_table[(int64_t)it.b * a.kv.max_pages + page_slot(p, key)];
                };
                int page = 0;
                if constexpr (PAGED) page = page_of(0);
                for (int st = 0; st < n && ok; ++st) {
                    const int key0 = (it.s0 + st) * kStep;
                    const int pg = (unsigned)page < (unsigned)a.kv.num_pages ? page : -1;
                    if constexpr (PAGED) page = page_of(st + 1);
                    for (int kv = 0; kv < 2 && ok; ++kv) {
                        // 16-bit tiles go into the ring, 8-bit ones into the staging tiles
                        constexpr int kDepth = L::gather ? 2 : L::slots;
                        const int s = loads % kDepth;
                        if (loads >= kDepth)
                            ok = mbar_wait(bar((L::gather ? B_STAGE_FREE : B_FREE) + s), (loads / kDepth - 1) & 1, err, abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        const uint32_t dst = sbase + (L::gather ? L::staging + s * kStep * D : L::ring + s * L::tile);
                        const int real = it.kv_len - key0;             // keys of this tile that exist
                        const bool tail = !L::gather && kv == 1 && real < kStep;
                        const uint32_t b = bar(tail ? B_TAIL : (L::gather ? B_STAGE : B_FULL) + s);
                        const CUtensorMap* map = kv ? &mv : &mk;
                        if (lane == 0) mbar_arrive_expect_tx(b, L::gather ? kStep * D : L::tile);
                        __syncwarp();
                        if constexpr (PAGED) {
                            if (lane < p.boxes) {
                                // a box without a page reads page num_pages: outside, zeros
                                const int at = pg < 0 ? a.kv.num_pages : pg;
                                const int key = key0 + lane * p.box;
                                const int place = pg < 0 ? 0 : key - page_slot(p, key) * a.kv.page_size;
                                constexpr int kRow = L::gather ? D : 128;          // bytes of a box's row
                                for (int pn = 0; pn < (L::gather ? 1 : L::panels); ++pn) {
                                    const uint32_t to = dst + pn * L::panel + lane * p.box * kRow;
                                    if (p.hnd) tma_load_4d(to, map, pn * 64, place, it.h, at, b);
                                    else tma_load_4d(to, map, pn * 64, it.h, place, at, b);
                                }
                            }
                        } else if (lane == 0) {
                            for (int pn = 0; pn < L::panels; ++pn)
                                tma_load_3d(dst + pn * L::panel, map, pn * 64, it.h, it.k_row + key0, b);
                        }
                        if (tail) {
                            __syncwarp();
                            ok = mbar_wait(b, tails & 1, err, abort_flag);
                            ++tails;
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            unsigned char* row = smem + L::ring + s * L::tile;
                            for (int x = real * 8 + lane; x < kStep * 8; x += 32)
                                for (int pn = 0; pn < L::panels; ++pn)
                                    *reinterpret_cast<uint4*>(row + pn * L::panel + x * 16) = make_uint4(0, 0, 0, 0);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(B_FULL + s));
                        }
                        ++loads;
                    }
                }
                if (!ok) break;
            }
            if (!ok && lane == 0) {
                // a wait gave up: let the copies in flight land (bounded) before leaving
                for (int t = 0; t < 2; ++t)
                    if (qs[t] > 0) mbar_wait(bar(B_Q + t), (qs[t] - 1) & 1, nullptr, nullptr, 100000000ull);
                constexpr int kDepth = L::gather ? 2 : L::slots;
                for (int x = max(0, loads - kDepth); x < loads; ++x)
                    mbar_wait(bar((L::gather ? B_STAGE : B_FULL) + x % kDepth), (x / kDepth) & 1, nullptr, nullptr, 100000000ull);
            }
        } else if (warp == kMmaWarp) {
            // ============================ MMA ============================
            constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);    // stride 1024, version 1, 128-byte swizzle
            const uint32_t k_lo = ((sbase + L::ring) >> 4) | (1u << 16);
            const uint32_t v_lo = ((sbase + L::ring) >> 4) | ((uint32_t)(L::panel >> 4) << 16);
            const uint32_t q_lo = ((sbase + L::q) >> 4) | (1u << 16);
            Item it;
            int x = 0;                      // tiles of the ring used so far
            int qs0 = 0, qs1 = 0;           // Q tiles used
            int slot = 0;                   // x % slots
            int done0 = 0, done1 = 0;       // P tiles consumed
            bool ok = true;
            auto full = [&](int sl, int tile) {
                return __all_sync(0xffffffffu, mbar_wait(bar(B_FULL + sl), (tile / L::slots) & 1, err, abort_flag)) != 0;
            };
            auto after = [&](int sl) { return sl + 1 == L::slots ? 0 : sl + 1; };
            auto qk = [&](int t, int sl) {
                const uint32_t kb = k_lo + sl * (L::tile >> 4), qb = q_lo + t * (L::tile >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * L::panel + (kk & 3) * 32) >> 4;
                    mma_ss(tmem + t * kTileCols, qb + off, kb + off, kHi, kIdescQK, kk > 0 ? 1u : 0u);
                }
                commit(bar(B_S + t));
            };
            // keys 64 half .. + 63
            auto pv = [&](int t, int sl, int half, bool first) {
                const uint32_t vb = v_lo + sl * (L::tile >> 4);
#pragma unroll
                for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                    mma_ts(tmem + t * kTileCols + kOCol, tmem + t * kTileCols + 8 * kk, vb + kk * (16 * 128 >> 4), kHi,
                           kIdescPV, first && kk == 0 ? 0u : 1u);
            };
            for (int number = 0; ok; ++number) {
                ok = __all_sync(0xffffffffu, get_item<L>(smem, sbase, number, it, err, abort_flag)) != 0;
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_ITEM_FREE + (number & 1)));
                __syncwarp();
                if (__shfl_sync(0xffffffffu, it.b, 0) < 0) break;
                const int n0 = __shfl_sync(0xffffffffu, it.n[0], 0), n1 = __shfl_sync(0xffffffffu, it.n[1], 0);
                const int n = max(n0, n1);
                if (n == 0) continue;
                ok = full(slot, x);
                if (ok && n0 > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(B_Q), qs0++ & 1, err, abort_flag)) != 0;
                    tc_fence_after();
                    if (ok) qk(0, slot);
                }
                if (ok && n1 > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(B_Q + 1), qs1++ & 1, err, abort_flag)) != 0;
                    tc_fence_after();
                    if (ok) qk(1, slot);
                }
                if (!ok) break;
                for (int i = 0; i < n; ++i) {
                    // V of step i, K of step i + 1
                    const int vs = after(slot), ks = after(vs);
                    ok = full(vs, x + 1);
                    if (!ok) break;
                    bool have_k = false;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int nt = t ? n1 : n0;
                        if (i >= nt) continue;
                        int& done = t ? done1 : done0;
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_PH + t), done & 1, err, abort_flag)) != 0;
                        if (!ok) break;
                        tc_fence_after();
                        pv(t, vs, 0, i == 0);
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_P + t), done & 1, err, abort_flag)) != 0;
                        if (!ok) break;
                        ++done;
                        tc_fence_after();
                        pv(t, vs, 1, false);
                        if (i == nt - 1) {
                            commit(bar(B_O + t));
                        } else {
                            if (!have_k) {
                                ok = full(ks, x + 2);
                                if (!ok) break;
                                tc_fence_after();
                                have_k = true;
                            }
                            qk(t, ks);
                        }
                    }
                    if (!ok) break;
                    slot = ks;
                    x += 2;
                }
            }
            if (!ok) {
                __syncwarp();
                commit(bar(B_DRAIN));
                mbar_wait(bar(B_DRAIN), 0, nullptr, nullptr, 100000000ull);
            }
            __syncwarp();
        }
    } else {
        // ============================ softmax ============================
        regs_acquire<TcBlock<SRC>::softmax>();
        const int t = warp >> 2;
        const int r = tid & 127;                            // row of the tile = TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + t * kTileCols;
        int steps = 0, outs = 0;                            // barrier phases of this tile so far
        int base = 0;                                       // ring index of the item's first tile
        Item it;
        bool ok = true;
        for (int number = 0; ok; ++number) {
            ok = get_item<L>(smem, sbase, number, it, err, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_ITEM_FREE + (number & 1)));
            if (it.b < 0) break;
            const int n = t ? it.n[1] : it.n[0], n_all = max(it.n[0], it.n[1]);
            // The last tile issued sees every step; when its S of a step (or
            // its O) is there, everything issued before is done too, and its
            // thread 0 gives the tiles read by that back to the producer.
            // (A commit on the MMA side for each of them cost ~500 cycles of
            // the issuing thread.)
            const bool frees = n == n_all && (t == 1 || it.n[1] == 0) && r == 0;
            const int tok = it.tok0 + t * p.TR + r / G, head = it.h * G + r % G;
            const bool valid = r < p.TR * G && tok < it.n_q;
            // keys this row sees (a row of no token: all, its result is dropped)
            const int lim = a.causal && valid ? max(0, min(it.kv_len, tok + it.kv_len - it.n_q + 1)) : it.kv_len;
            const int lim_min = __reduce_min_sync(0xffffffffu, lim);
            float rs = a.scale_log2;
            if constexpr (kScaledQ) {
                // This thread's row of q as fp16, scaled by 2^-e.  (The last
                // Q.K^T that read the tile was done before the S of the item
                // before was there.)
                if (n > 0) {
                    uint32_t w[D / 2];
                    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                                      (int64_t)(it.q_row + tok) * a.q_stride + head * D);
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
                        reinterpret_cast<uint4*>(w)[c] = valid ? src[c] : make_uint4(0, 0, 0, 0);
                    float top = 0.f;
#pragma unroll
                    for (int c = 0; c < D / 2; ++c) {
                        const float2 f = BF16::unpack2(w[c]);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                    const int e8 = (int)((__float_as_uint(top) >> 23) & 255u) - 127;
                    const int e = (top == 0.f || e8 > 127) ? 0 : max(e8 - 14, -120);
                    const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                    for (int c = 0; c < D / 2; ++c) {
                        const float2 y = BF16::unpack2(w[c]);
                        w[c] = F16::pack2(y.x * f, y.y * f);
                    }
                    unsigned char* to = smem + L::q + t * L::tile + r * 128;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
                        *reinterpret_cast<uint4*>(to + (c >> 3) * L::panel + (((c & 7) ^ (r & 7)) << 4)) =
                            reinterpret_cast<const uint4*>(w)[c];
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_Q + t));
                    rs *= __uint_as_float((uint32_t)(127 + e) << 23);
                }
            }
            if constexpr (F8) {
                if (a.kv.scale_k) rs *= a.kv.scale_k[it.h];
                // Scores are masked before they are scaled, and -inf * 0 is NaN:
                // where the product of the scales underflows the smallest number
                // serves, under which every score is still nothing.
                rs = fmaxf(rs, __uint_as_float(1u));
            }
            float m_used = -INFINITY, l = 0.f;
            // Pages of the boxes (runs of p.box keys that no page border cuts)
            // lane + 32 i of step st, looked up a step ahead; left as loaded, so
            // that nothing waits for the load.
            constexpr int kWords = L::gather ? 4 : 1;
            int ahead[kWords];
            auto look_up = [&](int st) {
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    const int box = lane + 32 * i, key = (it.s0 + st) * kStep + box * p.box;
                    ahead[i] = 0;
                    if (i > 0 && 32 * i >= p.boxes) continue;          // (the same for all lanes)
                    if (st < n && box < p.boxes && key < it.kv_len)
                        ahead[i] = a.kv.page_table[(int64_t)it.b * a.kv.max_pages + page_slot(p, key)];
                }
            };
            if constexpr (PAGED) look_up(0);
            for (int st = 0; st < n; ++st) {
                unsigned bad = 0;                // bit i: the page of box lane + 32 i is out of range
                bool missing = false;
                if constexpr (PAGED) {
#pragma unroll
                    for (int i = 0; i < kWords; ++i) bad |= ((unsigned)ahead[i] >= (unsigned)a.kv.num_pages ? 1u : 0u) << i;
                    missing = __any_sync(0xffffffffu, bad != 0);
                    look_up(st + 1);
                }
                ok = mbar_wait(bar(B_S + t), steps & 1, err, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                ++steps;
                if (frees) {
                    mbar_arrive(bar(B_FREE + (base + 2 * st) % L::slots));                    // K of this step
                    if (st > 0) mbar_arrive(bar(B_FREE + (base + 2 * st - 1) % L::slots));    // V of the one before
                    if (st == n - 1) mbar_arrive(bar(B_Q_FREE));
                }
                tc_fence_after();
                uint32_t sv[128];
                tmem_ld128_sync(lane_base, sv);
                const int key0 = (it.s0 + st) * kStep;
                if (lim_min < key0 + kStep || missing) {
                    const int rel = lim - key0, rel_min = lim_min - key0;
                    // 32 keys at a time, where a row of this warp ends before or in them
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (rel_min < 32 * (q + 1)) {
#pragma unroll
                            for (int j = 32 * q; j < 32 * (q + 1); ++j)
                                if (j >= rel) sv[j] = __float_as_uint(-INFINITY);
                        }
                    if (PAGED && missing) {
                        // 128 bits, one a key: the words' bits spread over their boxes
                        unsigned gone[4] = {0, 0, 0, 0};
#pragma unroll
                        for (int i = 0; i < kWords; ++i) {
                            const unsigned w = __ballot_sync(0xffffffffu, (bad >> i) & 1u);
                            for (unsigned x = w; x; x &= x - 1) {
                                const int key = (__ffs(x) - 1 + 32 * i) << p.box_shift;
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const int lo = max(key - 32 * q, 0), hi = min(key + p.box - 32 * q, 32);
                                    if (lo < hi) gone[q] |= (hi - lo == 32 ? 0xffffffffu : ((1u << (hi - lo)) - 1u)) << lo;
                                }
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 128; ++j)
                            if ((gone[j >> 5] >> (j & 31)) & 1u) sv[j] = __float_as_uint(-INFINITY);
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 128; j += 2)
                    mx[(j >> 1) & 3] = fmaxf(fmaxf(mx[(j >> 1) & 3], __uint_as_float(sv[j])), __uint_as_float(sv[j + 1]));
                // the scale is positive and rounding monotonic: max of scaled = scaled max
                const float m_new = fmaxf(m_used, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * rs);
                const bool need = m_new > m_used + kRescale;
                // the P.V before this step's Q.K^T is complete: O is settled
                if (st > 0 && __any_sync(0xffffffffu, need)) {
                    const float f = need ? fast_exp2(m_used - m_new) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t ov[32];
                        tmem_ld32_sync(lane_base + kOCol + 32 * c, ov);
#pragma unroll
                        for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * f);
                        tmem_st32(lane_base + kOCol + 32 * c, ov);
                    }
                    l *= f;
                }
                if (need) m_used = m_new;
                // (a row that has seen no key has only -inf scores: subtracting 0 gives P = 0)
                const float sub = m_used == -INFINITY ? 0.f : m_used - kPShift;
                const uint64_t rs2 = pair(rs, rs), sub2 = pair(-sub, -sub);
                uint64_t ls[2] = {0, 0};
                auto weights = [&](int k) {              // keys 2 k, 2 k + 1
                    const uint64_t u = fma2(pair(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1])), rs2, sub2);
                    const float p0 = fast_exp2(low(u)), p1 = fast_exp2(high(u));
                    ls[k & 1] = add2(ls[k & 1], pair(p0, p1));
                    sv[k] = M::pack2(p0, p1);
                };
#pragma unroll
                for (int k = 0; k < 32; ++k) weights(k);
                tmem_st32(lane_base, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                // (the first half's store completes under the next weights)
#pragma unroll
                for (int k = 32; k < 44; ++k) weights(k);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_PH + t));
#pragma unroll
                for (int k = 44; k < 64; ++k) weights(k);
                tmem_st32(lane_base + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                const uint64_t l2 = add2(ls[0], ls[1]);
                l += low(l2) + high(l2);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_P + t));
            }
            if (!ok) break;
            // ---- epilogue ----
            if (n > 0) {
                ok = mbar_wait(bar(B_O + t), outs & 1, err, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                ++outs;
                if (frees) mbar_arrive(bar(B_FREE + (base + 2 * n - 1) % L::slots));
                tc_fence_after();
            }
            base += 2 * n_all;
            const bool none = l == 0.f;          // no visible key (a NaN sum is not that)
            const int64_t row = (int64_t)(it.q_row + tok) * a.Hq + head;
            const float vs = F8 && a.kv.scale_v ? a.kv.scale_v[it.h] : 1.f;
            const float inv = none ? 0.f : vs / l;
            // parts: [D / 4][row][4], so that the lanes (rows) write side by side
            const int64_t slot = 2 * blockIdx.x + (it.s0 == 0 ? 1 : 0);
            float* part = p.ws_o + slot * kItemRows * D + (t * kTileM + r) * 4;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t ov[32];
                if (n > 0) {
                    tmem_ld32_sync(lane_base + kOCol + 32 * c, ov);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) ov[j] = 0u;
                }
                if (!valid) continue;
                if (it.whole) {
                    typename E::T* dst = static_cast<typename E::T*>(a.out) + row * D + 32 * c;
#pragma unroll
                    for (int j = 0; j < 32; j += 16) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w[i] = none ? 0u : E::pack2(__uint_as_float(ov[j + 2 * i]) * inv, __uint_as_float(ov[j + 2 * i + 1]) * inv);
                        if (p.out32) {
                            st_32(dst + j, w);
                        } else {
                            reinterpret_cast<uint4*>(dst + j)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4*>(dst + j)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<uint4*>(part + (32 * c + j) * kItemRows) = make_uint4(ov[j], ov[j + 1], ov[j + 2], ov[j + 3]);
                }
            }
            // O has been read: the MMAs of the next item may overwrite it (they wait for its P)
            tc_fence_before();
            if (valid) {
                if (!it.whole)
                    *reinterpret_cast<float2*>(p.ws_ml + (slot * kItemRows + t * kTileM + r) * 2) = make_float2(m_used, l);
                else if (a.lse)
                    a.lse[row] = none ? -INFINITY : (m_used + __log2f(l) - kPShift) * kLn2;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Block (x, y) joins rows 32 y .. 32 y + 31 of the parts of the item that range
// x cuts first: lane = row, each warp some of the dims; the result crosses over
// in shared memory to be written row by row.  (Finding the cuts here again took
// longer than joining: 16 us where nothing was cut.)  Most blocks have nothing
// to do, so what counts is how many fit an SM: 512 threads, or 4 parts in flight at
// 118 registers, took 3 to 6 and 1 to 2 us longer.
constexpr int kMergeThreads = 256;

template <class E, int D>
__global__ void __launch_bounds__(kMergeThreads, 4) attn_tc_merge(const TcParams p) {
    constexpr int kWarps = kMergeThreads / 32;
    constexpr int Q = D / 4 / kWarps;                    // 4-dim groups of a warp
    constexpr int kBatch = 2;
    __shared__ uint2 turn[32][D / 4 + 1];
    const SeqAttn& a = p.a;
    const float kPShift = std::is_same<E, BF16>::value && a.kv.f8 == 0 ? 0.f : 7.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    const CutItem it = p.ws_cut[blockIdx.x];
    const int N = it.N, h = it.h;
    if (N == 0) return;
    const int r = blockIdx.y * 32 + lane, rr = r % kTileM, tok = it.tok0 + r / kTileM * p.TR + rr / a.G;
    const bool valid = rr < p.TR * a.G && tok < it.n_q;
    if (!__any_sync(0xffffffffu, valid)) return;         // (the same in every warp)
    float M = -INFINITY, l = 0.f;
    float4 acc[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    // kBatch parts in flight (`last`: steps before part i)
    for (int i = 0, last = 0; last < N; i += kBatch) {
        float2 ml[kBatch];
        float4 v[kBatch][Q];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int end = last < N ? cut(it.x + (i + j) * it.per, it.c, N) : last;
            const bool some = valid && end != last;      // (two borders can move to the same step)
            last = end;
            const int64_t slot = i + j == 0 ? 2 * (int)blockIdx.x + 1 : 2 * ((int)blockIdx.x + i + j);
            ml[j] = some ? *reinterpret_cast<const float2*>(p.ws_ml + (slot * kItemRows + r) * 2) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int q = 0; q < Q; ++q)
                v[j][q] = some ? *reinterpret_cast<const float4*>(p.ws_o + slot * kItemRows * D + ((q * kWarps + warp) * kItemRows + r) * 4)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // (a part without a visible key: m = -inf, everything else 0)
        float m_new = M;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) m_new = fmaxf(m_new, ml[j].x);
        const float old = rescale_factor(M, m_new);
        M = m_new;
        l *= old;
#pragma unroll
        for (int q = 0; q < Q; ++q) acc[q] = make_float4(acc[q].x * old, acc[q].y * old, acc[q].z * old, acc[q].w * old);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const float f = rescale_factor(ml[j].x, M);
            l += ml[j].y * f;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                acc[q].x += v[j][q].x * f;
                acc[q].y += v[j][q].y * f;
                acc[q].z += v[j][q].z * f;
                acc[q].w += v[j][q].w * f;
            }
        }
    }
    const bool none = l == 0.f;
    const float vs = a.kv.f8 && a.kv.scale_v ? a.kv.scale_v[h] : 1.f;
    const float inv = none ? 0.f : vs / l;
    const int64_t row = (int64_t)(it.q_row + tok) * a.Hq + h * a.G + rr % a.G;
#pragma unroll
    for (int q = 0; q < Q; ++q)
        turn[lane][q * kWarps + warp] = none ? make_uint2(0u, 0u)
                                             : make_uint2(E::pack2(acc[q].x * inv, acc[q].y * inv),
                                                          E::pack2(acc[q].z * inv, acc[q].w * inv));
    if (warp == 0 && valid && a.lse) a.lse[row] = none ? -INFINITY : (M + __log2f(l) - kPShift) * kLn2;
    __syncthreads();
    // D / 4 threads a row
    for (int i = warp; i < 32; i += kWarps) {
        const int64_t to = __shfl_sync(0xffffffffu, row, i);
        if (!__shfl_sync(0xffffffffu, (int)valid, i)) continue;
        if (lane < D / 4) *reinterpret_cast<uint2*>(static_cast<typename E::T*>(a.out) + to * D + lane * 4) = turn[i][lane];
    }
}

// q, or packed k / v: [rows][heads][D] with rows `stride` elements apart; box
// 64 dims x hb heads x rb rows, 128-byte swizzle.
bool rows_map(CUtensorMap* m, const void* base, bool bf16, int D, int heads, int rows, int64_t stride, int hb, int rb) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t st[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)hb, (cuuint32_t)rb};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
              dim, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A page pool: (dim, head, place, page) or, HND, (dim, place, head, page); box
// 64 dims x `box` places.
bool pool_map(CUtensorMap* m, const void* base, bool bf16, const SeqKV& kv, bool hnd, int box_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t D = kv.D, H = kv.Hkv, P = kv.page_size;
    const cuuint64_t dim[4] = {D, hnd ? P : H, hnd ? H : P, (cuuint64_t)kv.num_pages};
    const cuuint64_t st[3] = {D * 2, (hnd ? P : H) * D * 2, H * P * D * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(hnd ? box_rows : 1), (cuuint32_t)(hnd ? 1 : box_rows), 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(base),
              dim, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A pool of 8-bit codes likewise; box D bytes x `box_rows` places, swizzled over a row (see staged()).
bool codes_map(CUtensorMap* m, const void* base, const SeqKV& kv, bool hnd, int box_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t D = kv.D, H = kv.Hkv, P = kv.page_size;
    const cuuint64_t dim[4] = {D, hnd ? P : H, hnd ? H : P, (cuuint64_t)kv.num_pages};
    const cuuint64_t st[3] = {D, (hnd ? P : H) * D, H * P * D};
    const cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)(hnd ? box_rows : 1), (cuuint32_t)(hnd ? 1 : box_rows), 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dim, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              kv.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class E, int D, int SRC>
cudaError_t launch_tc_t(const TcParams& p, int64_t longest, int num_sms, cudaStream_t stream) {
    using L = TcSmem<D, SRC>;
    const SeqAttn& a = p.a;
    const bool bf16 = std::is_same<E, BF16>::value;
    CUtensorMap mq, mk, mv;
    if (!rows_map(&mq, a.q, bf16, D, a.Hq, a.tokens, a.q_stride, a.G, p.TR)) return cudaErrorInvalidValue;
    if (L::gather) {
        mk = mv = mq;              // (unused where rows are gathered without maps)
        if (L::f8 && p.box >= kMinBox8 && (!codes_map(&mk, a.kv.k, a.kv, p.hnd, p.box) || !codes_map(&mv, a.kv.v, a.kv, p.hnd, p.box)))
            return cudaErrorInvalidValue;
    } else if (SRC == SRC_PAGES ? (!pool_map(&mk, a.kv.k, bf16, a.kv, p.hnd, p.box) || !pool_map(&mv, a.kv.v, bf16, a.kv, p.hnd, p.box))
              : (!rows_map(&mk, a.kv.k, bf16, D, a.kv.Hkv, max(a.kv.rows, 1), a.kv.s_tok, 1, kStep) ||
                 !rows_map(&mv, a.kv.v, bf16, D, a.kv.Hkv, max(a.kv.rows, 1), a.kv.sv_tok, 1, kStep))) {
        return cudaErrorInvalidValue;
    }
    auto kern = attn_tc_kernel<E, D, SRC>;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::alloc);
    if (err != cudaSuccess) return err;
    // the register split assumes a launch with that many registers a thread
    static const bool regs_ok = [&] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, kern) == cudaSuccess && fa.numRegs == TcBlock<SRC>::launch;
    }();
    if (!regs_ok) return cudaErrorInvalidConfiguration;
    const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    err = launch_pdl(kern, dim3(ctas), dim3(TcBlock<SRC>::threads), L::alloc, stream, mq, mk, mv, p);
    if (err != cudaSuccess) return err;
    count_launches(1);
    // items of fewer than 2 kMinShare steps are never cut
    if (longest >= 2 * kMinShare * kStep - kStep + 1) {
        err = launch_pdl(attn_tc_merge<E, D>, dim3(ctas - 1, kItemRows / 32), dim3(kMergeThreads), 0, stream, p);
        if (err == cudaSuccess) count_launches(1);
    }
    return err;
}

}  // namespace

bool attn_tc_supported(const SeqKV& kv, int G) {
    // (a gathered row is named by a 32-bit number)
    return G <= kTileM &&
           (!kv.page_table || (int64_t)kv.num_pages * kv.page_size * kv.Hkv < 0xffffffffLL);
}

size_t attn_tc_ws_bytes(int G, int D) {
    return G <= kTileM ? (size_t)2 * kMaxCtas * kItemRows * (D + 2) * 4 + kMaxCtas * sizeof(CutItem) : 0;
}

cudaError_t launch_attn_tc(const SeqAttn& a, sfa_dtype dtype, int num_sms, cudaStream_t stream) {
    TcParams p{};
    p.a = a;
    p.TR = kTileM / a.G;
    p.hnd = a.kv.s_tok == a.kv.D && a.kv.Hkv > 1 ? 1 : 0;
    p.box = kStep;
    if (a.kv.page_table)
        while (a.kv.page_size % p.box != 0) p.box /= 2;
    p.boxes = kStep / p.box;
    while ((1 << p.box_shift) < p.box) ++p.box_shift;
    p.by_unit = divide_by(2 * p.TR);
    p.ctas_mul = ~uint64_t(0) / (uint64_t)(num_sms < kMaxCtas ? num_sms : kMaxCtas) + 1;
    // Measured (448 / 576): chunks of 200 to 1,024 tokens over 16-bit pages 199.8 /
    // 202.0 us, 4 causal prompts of 2,048 tokens 139.6 / 145.5 us; 64-dim ones (320 /
    // 448) 101.2 / 103.8 us, prompts of up to 700 tokens 30.9 / 31.2 us; chunks over
    // E4M3 pages (512 / 640) 399 / 394 us.  A step of 128 keys takes about 2,700
    // cycles (64-dim 2,400, 8-bit 3,900).
    p.charge = a.kv.f8 ? 640 : (a.kv.D == 128 ? 448 : 320);
    p.out32 = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    p.ws_o = static_cast<float*>(a.ws);
    p.ws_ml = p.ws_o + (int64_t)2 * kMaxCtas * kItemRows * a.kv.D;
    p.ws_cut = reinterpret_cast<CutItem*>(p.ws_ml + (int64_t)2 * kMaxCtas * kItemRows * 2);
    // no sequence has more keys than this
    const int64_t longest = a.kv.page_table ? (int64_t)a.kv.max_pages * a.kv.page_size : a.kv.rows;
    const bool bf16 = dtype == SFA_DTYPE_BF16;
    const int src = !a.kv.page_table ? SRC_PACKED
                    : a.kv.f8        ? (a.kv.f8 == 1 ? SRC_E4M3 : SRC_E5M2)
                                     : (a.kv.page_size % kMinBox == 0 ? SRC_PAGES : SRC_G16);
#define SFA_ATTN_TC(D_, SRC_)                                                        \
    if (a.kv.D == D_ && src == SRC_)                                                 \
        return bf16 ? launch_tc_t<BF16, D_, SRC_>(p, longest, num_sms, stream)         \
                    : launch_tc_t<F16, D_, SRC_>(p, longest, num_sms, stream);
#define SFA_ATTN_TC_D(D_)                                                            \
    SFA_ATTN_TC(D_, SRC_PACKED)                                                      \
    SFA_ATTN_TC(D_, SRC_PAGES)                                                       \
    SFA_ATTN_TC(D_, SRC_G16)                                                         \
    SFA_ATTN_TC(D_, SRC_E4M3)                                                        \
    SFA_ATTN_TC(D_, SRC_E5M2)
    SFA_ATTN_TC_D(128)
    SFA_ATTN_TC_D(64)
#undef SFA_ATTN_TC_D
#undef SFA_ATTN_TC
    return cudaErrorInvalidValue;
}

}  // namespace sfa
