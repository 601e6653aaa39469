// pi_paged_attn.cu -- causal attention of new tokens over a paged cache.
//
// The query heads that share a KV head go through its keys together: a tile of
// rows is as many whole tokens as fit 128 rows (row = token * group + head in
// the group), so one pass over the keys serves the whole group.  An item is up
// to two such tiles of one request and KV head; its keys come in tiles of 128.
// For a tile, on the tcgen05 tensor cores,
//     S = Q K^T         (fp16/bf16 products, fp32 sums in tensor memory)
//     P = 2^(c S - m)   (a thread per row; running m and l = sum P)
//     O += P V          (P as the A operand in tensor memory)
// where c = scale / ln 2 and m trails the running maximum: it moves only when
// the weights of some row outgrow it (fp16: a score 2^8 above it, looked for in
// every tile, since a weight must fit 16 bits; bf16: a tile's weights adding up
// to more than 2^30, seen after the tile), and then O and l are scaled.  P
// carries a factor 2^7, which l and O share: no fp16 weight is above 2^15, those
// of the largest scores are 2^7 or more, and weights down to 2^-31 of theirs
// survive the rounding.
//
// Warps: 0-3 and 4-7 softmax (a thread per row), 8 key copies, 9 MMA issue, 10
// value copies, 11 the work list and the query copies.  Items of two tiles of
// rows give each softmax group one (both use every key tile: "pair"); smaller
// items, decode steps among them, give the two groups alternate key tiles and
// merge at the end: one group's exponentials run beside the other's products.
//
// Work split: the (item x key tile) space is cut into equal contiguous ranges
// per block, whatever the lengths; an item cut by a border leaves unnormalised
// partials (m, l, O) in the workspace, and the block that arrives last adds
// them in block order (the order is fixed, who does it is not: same bits).
//
// Rows whose outputs are not finite are taken again in fp32 over the keys they
// see, by the block that wrote them, once it is done with everything else.
//
// Bounds and figures (GB300, 64 query and 8 KV heads of 128 unless said):
//  - few rows per key (decoding): HBM.  Four sequences with 120-131 thousand
//    keys, bf16: 300-308 us, 6.7-6.9 TB/s.  32 sequences with 500-8000 keys, fp16: 80
//    us, 5.7 TB/s; DRAM reads are 1.006 of the keys and values, the start and
//    the joins of cut items are the rest.  One sequence with 1001 keys: 13.3
//    us of latency, two key tiles per block and a join.
//  - many rows (a chunk of 4096 tokens behind 12288, bf16): the tensor cores.
//    1.11-1.22 ms, 1.58-1.73 PFLOP/s.  Two tiles of rows keep them busy for
//    2048 cycles per key tile, which takes 2900: each group's chain of S, the
//    softmax (1350 for both, 1170 of them for 2 x 128 x 128 exponentials) and
//    P V is longer than the other's products beside it, and tensor memory has
//    no room for a second S.  The copies of a tile's eight pages take 600 on
//    each of two warps.
//  - prompts of some thousand tokens and mixed steps: 29 us for a prompt of
//    1999 tokens (12 heads of 64), 118 us for 16 sequences that decode or take
//    100-700 tokens (32 heads, window of 2000).  A block has its SM to itself,
//    so nothing hides its start, its items' outputs and the joins.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "pi_common.cuh"
#include "pi_internal.h"
#include "pi_pipe.cuh"
#include "pi_umma.cuh"

namespace pi {
namespace {

using namespace pipe;

constexpr int kKeys = 128;             // keys of a tile
constexpr int kTileRows = 128;         // rows of a tile at most
constexpr int kPagedThreads = 384;
constexpr int kListDepth = 4;          // pieces the work list runs ahead
constexpr int kConsumers = 11;         // warps that read the work list: all but the one that writes it
constexpr int kWalk = 64;              // items of a request that are counted one by one, not by formula: one prompt of
                                       // 16-32 items 22-40 us so, 26-44 by formula (63 items 84.5 and 88.5); of 125 items
                                       // 61.7 by formula and 73.9 one by one (16 heads of 64), since the walk grows with it
// What the work split counts, in units of half a microsecond or so: a key tile
// for one tile of rows (memory), for two (products), an item besides its tiles
// (kLead before them, the rest after: a border that falls there does not cut the
// item).  Without these weights a mixed step of 16 sequences that decode or take
// 100-700 tokens took 131 us instead of 119.  Over 18 cases (four of the listed ones
// of perf/operators.py and 14 drawn from its ranges) the geometric mean is 2 % below that of 6 units all before the tiles, 0.6 % below
// 3 + 3 and 5 + 5, 0.7 % above 6 + 6 (32 decoding sequences 83 us instead of
// 80); pair costs of 3.5 and 4 add 1 or 2 %.
constexpr int kTileCost = 2, kPairCost = 3, kItemCost = 8, kLead = 4;
// Units of a block at least (a tile's cost or more): 18 cases' mean 30.5 us, one
// sequence with 1001 keys 13.4 us; with 3 units 31.1 and 13.8, 4 30.8 and 12.7,
// 6 30.5 and 13.5, 9 30.7 and 14.5.
constexpr int kMinUnits = 5;
constexpr float kLift = 7.f;           // log2 of the factor that P, l and O share
constexpr float kGrow = 8.f;           // fp16: growth (log2) of a maximum before m follows
constexpr float kSum = 1073741824.f;   // bf16: sum of a tile's weights from which m follows
constexpr float kSink = 31.f;          // rows taken again: -log2 of the factor of their weights
constexpr float kLn2 = 0.69314718055994531f;

template <int DH>
struct PagedCfg {
    static constexpr int HALVES = DH / 64;               // 64-element column blocks of a row
    static constexpr int TILE = kKeys * DH * 2;          // bytes of a key or value tile
    static constexpr int QTILE = kTileRows * DH * 2;
    static constexpr int Q = 2 * QTILE;
    static constexpr int SK = DH == 128 ? 3 : 6;         // ring slots for keys: one more than for values, since
    static constexpr int SV = DH == 128 ? 2 : 6;         // a key tile is used a step before its values
    static constexpr int GROUP = HALVES * 1024;          // bytes of 8 keys or values: a 64-element block after the other
    static constexpr int MISC = 3 * 1024;
    static constexpr int SMEM = Q + (SK + SV) * TILE + MISC;
    static constexpr unsigned O_COL = 2 * kKeys;         // tensor memory: S0 S1 | O0 O1
    static_assert(SMEM <= 232448, "shared memory of a block");
};

struct PagedArgs {
    // a page as {64 elements, 8 positions, 64-element blocks, groups of 8 positions, page}:
    // a head is dh / 64 blocks from block head * head_blocks on, the box the head's part of a page
    CUtensorMap kmap, vmap;
    CUtensorMap qmap;         // {dh, head, token}, box 64 x group x tile_tokens
    const void *q, *k, *v;
    const int32_t *table, *cu, *kv;
    void* out;
    float* lse;
    long long q_stride, o_stride, page_stride, head_stride, token_stride;
    int heads, kv_heads, batch, max_tokens, max_new, max_pages, window, page_size, num_pages;
    int group;                // query heads per KV head
    int tile_tokens;          // tokens of a tile, 128 / group
    int head_blocks;          // head stride in blocks of 64 elements
    int part_rows;            // rows of a partial
    float scale;
    int* counters;            // [blocks][8] arrivals at a cut item
    float* part_ml;           // [blocks][2][2][part_rows][2]
    float* part_o;            // [blocks][2][DH / 4][part_rows][4]
    int* status;
    long long timeout_ns;
};

// A range of key tiles of one item.
struct Piece {
    int nt;          // key tiles (0: end of the list)
    int j0;          // first key tile
    int lo, hi;      // keys that some row of the item sees: lo <= t < hi
    int b, g;        // request, KV head
    int tok0, toks;  // tokens of the request
    int first;       // position of the request's first new token (negative: it sees nothing)
    int cu;          // the request's first row of q and out
    int block0;      // first block that holds a part of the item
    int parts;       // blocks that do (1: this one alone)
    int own;         // this block's partial: 1 where the item starts here
    int pad[3];
};

struct Request {
    int cu, n, first;   // first row of q, tokens, position of the first token
};

// What the work list goes by, as values: behind a function's reference to the
// kernel's arguments each look is a load from memory, not from the constant bank
// (31 requests of short and long items 58 us so, 62 by reference).
struct Lengths {
    const int32_t *cu, *kv;
    int batch, kv_heads, max_tokens, max_new, max_pages, page_size, window, group, tile_tokens;

    PI_DEV explicit Lengths(const PagedArgs& a)
        : cu(a.cu), kv(a.kv), batch(a.batch), kv_heads(a.kv_heads), max_tokens(a.max_tokens), max_new(a.max_new),
          max_pages(a.max_pages), page_size(a.page_size), window(a.window), group(a.group), tile_tokens(a.tile_tokens) {}
};

// Where a block's range of units starts, and how far its pieces have been walked.
struct Walk {
    Request r;
    long long u, u1, U;   // unit reached, the range's end, units in all
    int G, b, g, tok0, off;   // blocks with work; request, KV head, first token and unit within the item at u

    template <typename A>
    PI_DEV Piece next(const A& a);   // nt = 0: none is left
};

template <int DH>
struct PagedShared {
    unsigned long long kfull[6], kempty[6], vfull[6], vempty[6], qfull, qempty, sfull[2], pready[2][2], odone[2], lfull[kListDepth],
        lempty[kListDepth], merge[2], merged, drain;
    Piece list[kListDepth];
    float ml[2][kKeys][2];
    Walk walk;   // from this block's first unit
    unsigned tmem;
    int abort_flag;
    int redo;            // some row that this block has written is not finite
    int joined[2];       // warps that have written the outputs of a cut item (by Piece::own), a bit each
    int odd_rows, redo_rows;   // rows of a piece that are not finite, and those of them to be taken again
    int bad_keys, bad_k;       // keys of a piece with values that are not finite, and whether a key itself has one
};

template <typename A>
PI_DEV Request request(const A& a, int b, bool* bad) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    int kv = a.kv[b];
    Request r{lo, hi - lo, 0};
    if (lo < 0 || hi < lo || hi > a.max_tokens || hi - lo > a.max_new) {
        *bad = true;
        r.n = 0;
    }
    if (kv < 0 || kv > a.max_pages * a.page_size) {
        *bad = true;
        kv = 0;
    }
    r.first = kv - r.n;
    return r;
}

// Keys that an item's tokens (from tok0 on) see, as key tiles (one tile, with
// nothing to see in it, where they see none: it writes the zeros).
template <typename A>
PI_DEV int item_tiles(const A& a, const Request& r, int tok0, int* toks, int* lo, int* hi) {
    *toks = min(2 * a.tile_tokens, r.n - tok0);
    *hi = r.first + tok0 + *toks;
    *lo = a.window > 0 ? max(0, r.first + tok0 - a.window + 1) : 0;
    if (*hi <= *lo) {
        *lo = *hi = 0;
        return 1;
    }
    return (*hi + kKeys - 1) / kKeys - *lo / kKeys;
}

// sum of floor((a i + b) / m) over 0 <= i < n, for a, b >= 0 (Euclid's steps)
PI_DEV long long floor_sum(long long n, long long m, long long a, long long b) {
    long long sum = 0;
    for (;;) {
        if (a >= m) {
            sum += n * (n - 1) / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            sum += n * (b / m);
            b %= m;
        }
        const long long y = a * n + b;
        if (y < m) return sum;
        n = y / m;
        b = y % m;
        const long long t = m;
        m = a;
        a = t;
    }
}

template <typename A>
PI_DEV int tile_cost(const A& a, int toks) { return toks > a.tile_tokens ? kPairCost : kTileCost; }

// Cost of the first x items of one KV head of a request: kItemCost each, and
// their tiles (as item_tiles counts them).
__device__ __noinline__ long long units_before(const PagedArgs& a, const Request& r, int x) {
    const int d = 2 * a.tile_tokens, items = (r.n + d - 1) / d;
    if (x <= 0) return 0;
    long long u = (long long)kItemCost * x;
    int y = x;   // items before the last of all, which may be shorter
    if (x == items) {
        int toks, lo, hi;
        const int nt = item_tiles(a, r, (x - 1) * d, &toks, &lo, &hi);
        u += nt * tile_cost(a, toks);
        --y;
    }
    // items whose last token sees nothing: a tile each
    const int none = r.first < 0 ? min(y, -r.first / d) : 0;
    // ceil(hi / 128) with hi = first + (i + 1) d
    long long tiles = none + floor_sum(y - none, kKeys, d, (long long)r.first + (long long)(none + 1) * d + kKeys - 1);
    if (a.window > 0) {
        // floor(lo / 128) with lo = first + i d - window + 1 once that is positive
        const int gap = a.window - 1 - r.first;
        const int from = max(none, gap < 0 ? 0 : gap / d + 1);
        if (from < y) tiles -= floor_sum(y - from, kKeys, d, (long long)from * d - gap);
    }
    return u + kPairCost * tiles;
}
PI_DEV long long request_units(const PagedArgs& a, const Request& r) {   // of one KV head
    const int d = 2 * a.tile_tokens;
    if (r.n > kWalk * d) return units_before(a, r, (r.n + d - 1) / d);
    long long u = 0;
    int toks, lo, hi;
    for (int t = 0; t < r.n; t += d) {
        const int nt = item_tiles(a, r, t, &toks, &lo, &hi);
        u += kItemCost + nt * tile_cost(a, toks);
    }
    return u;
}

PI_DEV bool warp_wait(unsigned long long* b, unsigned parity, const Ctl& c) {
    if (__all_sync(FULL, bar_test(b, parity))) return true;
    return __all_sync(FULL, bar_wait(b, parity, c));
}

PI_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
PI_DEV float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
// the lowest n bits (none below 0, all from 32 on)
PI_DEV uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }
template <int N>
PI_DEV float largest(const uint32_t* s) {
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = max3(m[k], __uint_as_float(s[i + k]), __uint_as_float(s[i + 4 + k]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
PI_DEV float to_f(__half v) { return __half2float(v); }
PI_DEV float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
PI_DEV uint32_t pack2(float a, float b, __half) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
PI_DEV uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// Whether outputs are finite, after their rounding (the weights are rounded and
// their sum is not, so a mean of the largest fp16 values may round past them):
// 0 x both values of w + acc, which stays at zeros until an infinity or a NaN
PI_DEV uint32_t times0(uint32_t w, uint32_t acc, __half) {
    const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&w), __half2half2(__half(0.f)), *reinterpret_cast<const __half2*>(&acc));
    return *reinterpret_cast<const uint32_t*>(&v);
}
PI_DEV uint32_t times0(uint32_t w, uint32_t acc, __nv_bfloat16) {
    const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w), __bfloat162bfloat162(__nv_bfloat16(0.f)),
                                     *reinterpret_cast<const __nv_bfloat162*>(&acc));
    return *reinterpret_cast<const uint32_t*>(&v);
}
PI_DEV bool is_odd(uint32_t acc) { return (acc & 0x7fff7fffu) != 0; }   // zeros of either sign are not
// two fp32 values in one 64-bit register pair: a * b + c on both
PI_DEV uint64_t pair2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
PI_DEV void split2(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
PI_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
PI_DEV uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
PI_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// a / b for positive numbers, in 32 bits where they fit (a 64-bit division is a call)
PI_DEV long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
    return a / b;
}

// ------------------------------------------------------------ work list (warp 11)
//
// Units u of the block's range run through the items: kLead, the tiles' costs,
// the rest of kItemCost.  A block does the tiles that begin in its range (a range is
// longer than a tile's cost, so every block between an item's first and last
// has one).
template <typename A>
PI_DEV Piece Walk::next(const A& a) {
    Piece p{};
    while (u < u1 && p.nt == 0) {   // again where only an item's cost falls into this block
        int toks, lo, hi;
        const int nt = item_tiles(a, r, tok0, &toks, &lo, &hi);
        const int c = tile_cost(a, toks);
        const long long i0 = u - off;   // the item's first unit
        const int stop = (int)min((long long)(kItemCost + nt * c), u1 - i0);
        const int from = min((max(off - kLead, 0) + c - 1) / c, nt), to = min((max(stop - kLead, 0) + c - 1) / c, nt);
        p.nt = max(to - from, 0);
        p.j0 = lo / kKeys + from;
        p.lo = lo;
        p.hi = hi;
        p.b = b;
        p.g = g;
        p.tok0 = tok0;
        p.toks = toks;
        p.first = r.first;
        p.cu = r.cu;
        p.parts = 1;
        p.own = from == 0;
        // Blocks that own its first and its last tile.  Whatever the lengths become
        // under the kernel, block0 is this block or one before it; parts may pass the
        // blocks there are, and then no block finds that many arrivals.
        if (p.nt != nt) {
            p.block0 = (int)quotient((i0 + kLead + 1) * G - 1, U);
            p.parts = (int)quotient((i0 + kLead + (nt - 1) * c + 1) * G - 1, U) - p.block0 + 1;
        }
        u = stop > off ? i0 + stop : u1;   // (off past the item: the lengths changed under the kernel)
        off = 0;
        tok0 += 2 * a.tile_tokens;
        if (u < u1 && tok0 >= r.n) {
            tok0 = 0;
            if (++g == a.kv_heads) {
                g = 0;
                // u < u1 <= U: a later request has tokens
                do {
                    if (++b >= a.batch) {   // the lengths changed under the kernel: stop
                        u = u1;
                        break;
                    }
                    bool bad = false;
                    r = request(a, b, &bad);
                } while (r.n == 0);
            }
        }
    }
    return p;
}

// With a piece go its query tiles, once the scores of the piece before are
// done; tokens past the request's end or the last row come along or read as
// zeros: a row of S depends on its own query alone.  A function of its own: in
// line, its registers cost the other roles theirs (4096-token chunk 1.12-1.16 ms so,
// 1.21-1.26 in line).
template <int DH>
__device__ __noinline__ void list_role(Lengths a, const CUtensorMap* qmap, PagedShared<DH>& sh, unsigned char* qs, Walk walk, Ctl ctl) {
    using C = PagedCfg<DH>;
    int n = 0;
    for (;;) {
        const Piece p = walk.next(a);
        const int s = n % kListDepth;
        if (n >= kListDepth && !bar_wait(&sh.lempty[s], (n / kListDepth - 1) & 1, ctl)) break;
        sh.list[s] = p;
        bar_arrive(&sh.lfull[s]);
        if (p.nt == 0) break;
        if (n >= 1 && !bar_wait(&sh.qempty, (n - 1) & 1, ctl)) break;
        const int tiles = p.toks > a.tile_tokens ? 2 : 1;
        bar_arrive_expect_tx(&sh.qfull, (unsigned)(tiles * C::HALVES * a.tile_tokens * a.group) * 128u);
        for (int w = 0; w < tiles; ++w)
            for (int h = 0; h < C::HALVES; ++h)
                tma_load_3d(qs + w * C::QTILE + h * (kTileRows * 128), qmap, 64 * h, p.g * a.group,
                            p.cu + p.tok0 + w * a.tile_tokens, &sh.qfull);
        ++n;
    }
    // the last copy has landed before the block may exit
    if (n > 0) bar_drain(&sh.qfull, (n - 1) & 1, kDrainTimeoutNs);
}

// Next piece for a consumer warp; nt = 0 at the end or after an abort.
template <int DH>
PI_DEV Piece next_piece(PagedShared<DH>& sh, int n, const Ctl& ctl) {
    const int s = n % kListDepth;
    Piece p;
    if (!warp_wait(&sh.lfull[s], (n / kListDepth) & 1, ctl)) {
        p.nt = 0;
        return p;
    }
    p = sh.list[s];
    warp_arrive(&sh.lempty[s]);
    return p;
}

// ------------------------------------------------------------ key tiles (warp 8), value tiles (warp 10)
//
// A lane per page of a tile, one copy each.  A copy takes 70 cycles to issue:
// keys and values from one warp, 16 pages of 16 positions and their table
// entries, would take most of the 2048 cycles of a step's products, so a warp
// for each ring.  Pages outside the keys the item sees are not read (their rows
// of the slot are stale: scores there are masked, value rows are cleared by the
// MMA warp).
template <int DH, bool VALUES>
PI_DEV void tile_role(const PagedArgs& a, PagedShared<DH>& sh, unsigned char* ring, const Ctl& ctl) {
    using C = PagedCfg<DH>;
    constexpr int S = VALUES ? C::SV : C::SK;
    unsigned long long* const full = VALUES ? sh.vfull : sh.kfull;
    unsigned long long* const empty = VALUES ? sh.vempty : sh.kempty;
    const CUtensorMap* const map = VALUES ? &a.vmap : &a.kmap;
    const int lane = threadIdx.x & 31;
    const int pages = kKeys / a.page_size;   // of a tile
    int slot = 0, phase = 1, used = 0;       // phase of the slot's release before this use (none before the first)
    bool ok = true;
    for (int n = 0; ok; ++n) {
        const Piece p = next_piece<DH>(sh, n, ctl);
        if (p.nt == 0) break;
        const int32_t* row = a.table + (size_t)p.b * a.max_pages;
        // this lane's page in tile t: whether it is needed, and its table entry
        auto need = [&](int t) {
            const int key = (p.j0 + t) * kKeys + lane * a.page_size;
            return t < p.nt && lane < pages && key < p.hi && key + a.page_size > p.lo;
        };
        auto entry = [&](int t) { return need(t) ? row[(p.j0 + t) * pages + lane] : 0; };
        int id = entry(0), id1 = entry(1), id2 = entry(2);   // on their way two tiles ahead
        for (int t = 0; t < p.nt; ++t) {
            if (used >= S && !(ok = warp_wait(&empty[slot], phase, ctl))) break;
            const bool copy = need(t);
            const unsigned boxes = __popc(__ballot_sync(FULL, copy));
            if (lane == 0) bar_arrive_expect_tx(&full[slot], boxes * (unsigned)(a.page_size * DH * 2));
            __syncwarp();
            if (copy) {
                if (id < 0 || id >= a.num_pages) {
                    atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
                    id = a.num_pages;   // past the last page: the copy fills zeros
                }
                tma_load_5d(ring + (size_t)slot * C::TILE + lane * (a.page_size >> 3) * C::GROUP, map, 0, 0,
                            p.g * a.head_blocks, 0, id, &full[slot]);
            }
            id = id1;
            id1 = id2;
            id2 = entry(t + 3);
            ++used;
            if (++slot == S) {
                slot = 0;
                phase ^= 1;
            }
        }
    }
    // every copy issued has landed before the block may exit
    for (int s = 0; s < S && s < used; ++s) {
        const int last = s + ((used - 1 - s) / S) * S;
        bar_drain(&full[s], (last / S) & 1, kDrainTimeoutNs);
    }
}

// ------------------------------------------------------------ products (warp 9)
//
// The tensor core takes four or so MMAs ahead of the one it runs, so this warp
// has about 250 cycles from the last MMA of one product to the first of the
// next: its waits are for things that are there already.
template <typename T, int DH>
PI_DEV void mma_role(const PagedArgs& a, PagedShared<DH>& sh, unsigned char* qs, unsigned char* kring,
                     unsigned char* vring, unsigned tmem, const Ctl& ctl) {
    using C = PagedCfg<DH>;
    constexpr unsigned kType = std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10);   // A and B: fp16 or bf16
    const unsigned id_s = idesc_f16(128, kKeys, false) | kType;
    const unsigned id_o = idesc_f16(128, DH, false) | kType | (1u << 16);   // B (values) MN-major
    const uint64_t qd = sdesc_sw128(su32(qs)), kd = sdesc_sw128(su32(kring), C::GROUP),
                   vd = sdesc_sw128_mn(su32(vring), 1024, C::GROUP);
    int ks = 0, kph = 0, vs = 0, vph = 0;   // ring slots to use next, and the phases of their copies
    int done0 = 0, done1 = 0;               // tiles of each group so far
    bool ok = true;
    auto next_k = [&]() {
        if (++ks == C::SK) {
            ks = 0;
            kph ^= 1;
        }
    };
    auto next_v = [&]() {
        if (++vs == C::SV) {
            vs = 0;
            vph ^= 1;
        }
    };
    auto keys_in = [&]() { return warp_wait(&sh.kfull[ks], kph, ctl); };
    auto values_in = [&]() { return warp_wait(&sh.vfull[vs], vph, ctl); };
    // S_w = Q_qw K^T
    auto scores = [&](int w, int qw, int i) {
        const uint64_t x = qd + (uint64_t)(qw * (C::QTILE >> 4)), y = kd + (uint64_t)(i * (C::TILE >> 4));
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
            const unsigned b = (unsigned)((kk & 3) * 32);
            mma_f16_warp(tmem + (unsigned)(w * kKeys), x + (((unsigned)((kk >> 2) * (kTileRows * 128)) + b) >> 4),
                         y + (((unsigned)((kk >> 2) * 1024) + b) >> 4), id_s, kk > 0 ? 1u : 0u);
        }
        mma_commit_warp(&sh.sfull[w]);
    };
    // O_w (+)= P_w V, half of the keys at a time as their weights arrive
    auto values = [&](int w, int i, unsigned add, int& done, bool last) {
        const unsigned d = tmem + C::O_COL + (unsigned)(w * DH), x = tmem + (unsigned)(w * kKeys);
        const uint64_t y = vd + (uint64_t)(i * (C::TILE >> 4));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (!warp_wait(&sh.pready[w][half], done & 1, ctl)) return false;
            tc_after();
#pragma unroll
            for (int k = 0; k < kKeys / 32; ++k) {
                const int kk = half * (kKeys / 32) + k;
                mma_f16_ta_warp(d, x + (unsigned)(kk * 8), y + (uint64_t)(kk * (2 * C::GROUP >> 4)), id_o, kk > 0 ? 1u : add);
            }
        }
        ++done;
        if (last) mma_commit_warp(&sh.odone[w]);
        return true;
    };
    // value rows outside the keys the item sees (in an item's first and last
    // tile): zeros, not what the cache or the slot holds there, since 0 x NaN
    // would reach every row
    auto clear = [&](const Piece& p, int t, int i) {
        const int base = (p.j0 + t) * kKeys;
        if (base >= p.lo && base + kKeys <= p.hi) return;
        const int z = min(max(p.lo - base, 0), kKeys), e = min(max(p.hi - base, z), kKeys);
        unsigned char* v = vring + (size_t)i * C::TILE;
        const int dead = kKeys - (e - z);
#pragma unroll 1
        for (int x = threadIdx.x & 31; x < dead * (DH / 8); x += 32) {
            const int d = x / (DH / 8), c = x % (DH / 8);
            const int r = d < z ? d : d + (e - z);
            *reinterpret_cast<uint4*>(v + (r >> 3) * C::GROUP + (c >> 3) * 1024 + (r & 7) * 128 + (c & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_smem();
        __syncwarp();
    };
    for (int n = 0; ok; ++n) {
        const Piece p = next_piece<DH>(sh, n, ctl);
        if (p.nt == 0) break;
        const int nt = __shfl_sync(FULL, p.nt, 0);
        const bool pair = __shfl_sync(FULL, (int)(p.toks > a.tile_tokens), 0);
        if (!(ok = warp_wait(&sh.qfull, n & 1, ctl))) break;
        if (!(ok = keys_in())) break;
        if (pair) {
            // both groups use every tile; step t takes V(t) and K(t + 1), and
            // looks for the next step's between the two groups' products
            scores(0, 0, ks);
            scores(1, 1, ks);
            mma_commit_warp(&sh.kempty[ks]);
            if (nt == 1) mma_commit_warp(&sh.qempty);
            next_k();
            bool there = false;
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
                const bool more = t + 1 < nt;
                if (!there && !((ok = values_in()) && (!more || (ok = keys_in())))) break;
                clear(p, t, vs);
                if (!(ok = values(0, vs, t > 0, done0, !more))) break;
                const int iv = vs, ik = ks;
                next_v();
                if (more) {
                    scores(0, 0, ik);
                    next_k();
                    there = __all_sync(FULL, bar_test(&sh.vfull[vs], vph) & (t + 2 >= nt || bar_test(&sh.kfull[ks], kph)));
                }
                if (!(ok = values(1, iv, t > 0, done1, !more))) break;
                mma_commit_warp(&sh.vempty[iv]);
                if (more) {
                    scores(1, 1, ik);
                    mma_commit_warp(&sh.kempty[ik]);
                    if (t + 2 == nt) mma_commit_warp(&sh.qempty);
                }
            }
        } else {
            // the groups take alternate tiles
#pragma unroll 1
            for (int t = -2; t < nt; ++t) {
                const int w = t & 1;
                if (t >= 0) {
                    if (!(ok = values_in())) break;
                    clear(p, t, vs);
                    int& done = w ? done1 : done0;
                    if (!(ok = values(w, vs, t > 1, done, t + 2 >= nt))) break;
                    mma_commit_warp(&sh.vempty[vs]);
                    next_v();
                }
                if (t + 2 < nt) {
                    if (!(ok = keys_in())) break;
                    scores(w, 0, ks);
                    mma_commit_warp(&sh.kempty[ks]);
                    next_k();
                    if (t + 3 == nt) mma_commit_warp(&sh.qempty);
                }
            }
        }
    }
    // every product has completed before the block may exit
    __syncwarp();
    mma_commit_warp(&sh.drain);
    bar_drain(&sh.drain, 0, kDrainTimeoutNs);
}

// The weights 2^(c s + bias) of 64 scores into P (32 columns at `at`), and their sum.
template <typename T>
PI_DEV float take_weights(const uint32_t* s, unsigned at, uint64_t c2, uint64_t bias2) {
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kKeys / 2; i += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            float u, v;
            split2(fma2(pair2(__uint_as_float(s[i + e]), __uint_as_float(s[i + e + 1])), c2, bias2), u, v);
            u = ex2(u);
            v = ex2(v);
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair2(u, v));
            pk[e >> 1] = pack2(u, v, T());
        }
        tmem_st16(at + (unsigned)(i >> 1), pk);
    }
    float u, v;
    split2(add2(sum[0], sum[1]), u, v);
    return u + v;
}

// 1 / l, 0 for a row that sees nothing, NaN for a sum that is not finite (the row is taken again)
PI_DEV float inverse(float l) { return l < INFINITY ? (l > 0.f ? 1.f / l : 0.f) : NAN; }

PI_DEV int arrive_gpu(int* p) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
    return old;
}

PI_DEV int peek_gpu(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Adds the parts of rows r0 .. r0 + rows - 1 (at most 32) of an item's tile,
// whose first token is tok0, columns c0 .. c0 + cols - 1, in block order and
// writes the outputs: one warp, once all parts have arrived.  A lane keeps one
// row and every (32 / rows)-th group of 4 columns, so that a few rows still use
// the whole warp, and asks for CS column groups of KS parts and for their m and
// l at a time (what other blocks have just written takes 1500 cycles to come;
// one sequence with 1001 keys: 13.3 us so, 14.0 with m and l fetched first; 24
// loads at a time spill, here or in the caller).  True: some output is not finite.
template <typename T, int DH>
__device__ __noinline__ bool join_parts(const PagedArgs& a, const Piece& p, bool pair, int w, int r0, int rows, int tok0,
                                        int c0, int cols) {
    constexpr int CS = 4, KS = 4;
    const int lane = threadIdx.x & 31;
    const int span = rows > 16 ? 32 : rows > 8 ? 16 : rows > 4 ? 8 : rows > 2 ? 4 : rows;   // power of two
    const int tr = r0 + (lane & (span - 1));   // row of the tile
    const int cg = lane / span, step = 32 / span;
    if ((lane & (span - 1)) >= rows) return false;
    const int r = (pair ? w * kTileRows : 0) + tr;
    const size_t ml_step = (size_t)2 * 2 * a.part_rows, o_step = (size_t)2 * DH / 4 * a.part_rows;
    // partial of block block0 + k: its second slot (k = 0, where the item starts) or its first
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + (size_t)p.block0 * ml_step +
                       (size_t)(pair ? 0 : w) * a.part_rows + r;
    const float4* po = reinterpret_cast<const float4*>(a.part_o) + (size_t)p.block0 * o_step + r;
    const size_t ml_first = (size_t)2 * a.part_rows, o_first = (size_t)DH / 4 * a.part_rows;
    const int tok = tr / a.group, head = p.g * a.group + tr - tok * a.group;
    const long long orow = p.cu + tok0 + tok;
    T* dst = static_cast<T*>(a.out) + orow * a.o_stride + (long long)head * DH;
    const int end = (c0 + cols) / 4;
    float M = -INFINITY, L = 0.f, use = 0.f, inv = 0.f;
    bool first = true;
    uint32_t odd = 0;
    for (int c = c0 / 4 + cg; c < end; c += CS * step) {
        float4 v[CS];
#pragma unroll
        for (int j = 0; j < CS; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < p.parts; k0 += KS) {
            // loads without conditions, so that all of them are in flight at once
            // (past the end: once more the last one, left out below)
            float2 s[KS];
            float4 x[KS][CS];
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const int k = min(k0 + i, p.parts - 1);
                s[i] = __ldcg(ml + k * ml_step + (k == 0 ? ml_first : 0));
                const float4* src = po + k * o_step + (k == 0 ? o_first : 0);
#pragma unroll
                for (int j = 0; j < CS; ++j) x[i][j] = __ldcg(src + (size_t)min(c + j * step, end - 1) * a.part_rows);
            }
            if (first) {   // m and l of all parts, while those are on their way
                first = false;
                auto add = [&](float2 y) {
                    const float top = fmaxf(M, y.x);
                    use = top == -INFINITY ? 0.f : top;
                    L = fmaf(y.y, ex2(y.x - use), L * ex2(M - use));
                    M = top;
                };
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    if (i < p.parts) add(s[i]);
#pragma unroll 1
                for (int k = KS; k < p.parts; ++k) add(__ldcg(ml + k * ml_step));
                inv = inverse(L);
            }
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                if (k0 + i >= p.parts) break;
                const float g = ex2(s[i].x - use);
#pragma unroll
                for (int j = 0; j < CS; ++j) {
                    v[j].x = fmaf(x[i][j].x, g, v[j].x);
                    v[j].y = fmaf(x[i][j].y, g, v[j].y);
                    v[j].z = fmaf(x[i][j].z, g, v[j].z);
                    v[j].w = fmaf(x[i][j].w, g, v[j].w);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < CS; ++j)
            if (c + j * step < end) {
                const uint2 y = make_uint2(pack2(v[j].x * inv, v[j].y * inv, T()), pack2(v[j].z * inv, v[j].w * inv, T()));
                *reinterpret_cast<uint2*>(dst + 4 * (c + j * step)) = y;
                odd = times0(y.y, times0(y.x, odd, T()), T());
            }
    }
    if (a.lse != nullptr && c0 == 0 && cg == 0)
        a.lse[orow * a.heads + head] = L == 0.f ? -INFINITY : (M - kLift + log2f(L)) * kLn2;
    return is_odd(odd);
}

// ------------------------------------------------------------ softmax (warps 0-7)
//
// Thread = row.  Group w holds S in columns 128 w of its lanes, writes P over
// its first 64 columns, and owns O_w.
template <typename T, int DH>
PI_DEV void softmax_role(const PagedArgs& a, PagedShared<DH>& sh, unsigned tmem, const Ctl& ctl) {
    using C = PagedCfg<DH>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = warp >> 2, quad = warp & 3;
    const unsigned lanes = tmem + ((unsigned)(32 * quad) << 16);
    const unsigned s_at = lanes + (unsigned)(w * kKeys), o_at = lanes + C::O_COL + (unsigned)(w * DH);
    const float c = a.scale / kLn2;
    const uint64_t c2 = pair2(c, c);
    int ns = 0, np = 0, nm = 0;   // tiles of this group so far, pieces with any, merges
    for (int n = 0;; ++n) {
        // the piece stays in its slot until it is done
        if (!warp_wait(&sh.lfull[n % kListDepth], (n / kListDepth) & 1, ctl)) return;
        const Piece& p = sh.list[n % kListDepth];
        const int nt = p.nt, j0 = p.j0;
        if (nt == 0) return;
        const bool pair = p.toks > a.tile_tokens;
        const int tok0 = p.tok0 + (pair ? w * a.tile_tokens : 0);              // of this group's tile of rows
        const int tile_rows = min(a.tile_tokens, p.tok0 + p.toks - tok0) * a.group;
        const int tr = 32 * quad + lane;                                       // row of the tile
        const bool live = tr < tile_rows;
        const bool any = 32 * quad < tile_rows;
        // keys this row sees (a row of nothing: all, so that it does not ask for masking)
        int lo = 0, hi = 0x7fffffff;
        if (live) {
            const int pos = p.first + tok0 + tr / a.group;
            hi = max(pos + 1, 0);
            lo = a.window > 0 ? min(max(0, pos - a.window + 1), hi) : 0;
        }
        const int lo_most = __reduce_max_sync(FULL, lo), hi_least = __reduce_min_sync(FULL, hi);
        float m = -INFINITY, l = 0.f;
        bool fresh = true;    // some row of the warp has seen nothing yet
        float over = 0.f;     // bf16: the last tile's weights, and whether some row's add up to too much
        bool outgrown = false;
        int mine = 0;         // tiles of this piece that this group has done
        for (int t = pair ? 0 : w; t < nt; t += pair ? 1 : 2) {
            if (!warp_wait(&sh.sfull[w], ns & 1, ctl)) return;
            tc_after();
            if (any) {
                uint32_t s[kKeys];
#pragma unroll
                for (int i = 0; i < kKeys; i += 32) tmem_ld32(s_at + (unsigned)i, s + i);
                tmem_wait_ld();
                tmem_loaded<kKeys>(s);
                const int base = (j0 + t) * kKeys;
                if (base < lo_most || base + kKeys > hi_least) {
#pragma unroll
                    for (int i = 0; i < kKeys; i += 32) {
                        // bits of the keys that the row sees
                        const uint32_t see = low_bits(hi - base - i) & ~low_bits(lo - base - i);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(see & (1u << e))) s[i + e] = 0xff800000u;   // -inf
                    }
                }
                // m, where it has to move: to the maximum where some row has seen
                // nothing yet and for fp16 weights, above the last tile's for bf16
                constexpr bool kHalfType = std::is_same<T, __half>::value;
                float to = m;
                bool move = fresh;
                if (kHalfType || fresh) {
                    to = fmaxf(m, largest<kKeys>(s) * c);
                    if (!fresh) move = __any_sync(FULL, live && to > m + kGrow);
                }
                if (!kHalfType && outgrown) {
                    if (over > kSum) to = fmaxf(to, m + log2f(over) - kLift);
                    move = true;
                }
                if (move) {
                    const float f = to > m ? ex2(m - to) : 1.f;
                    m = to;
                    l *= f;
                    fresh = __any_sync(FULL, live && m == -INFINITY);
                    if (mine > 0) {
                        // O holds the sums over this group's earlier tiles: all in,
                        // since their products came before this tile's S
#pragma unroll 1
                        for (int i = 0; i < DH; i += 16) {
                            float o[16];
                            tmem_ld16(o_at + (unsigned)i, o);
                            tmem_wait_ld();
                            tmem_loaded<16>(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f;
                            tmem_st16(o_at + (unsigned)i, o);
                        }
                    }
                }
                // the weights, half of the keys at a time, each handed over once done
                const float bias = kLift - (m == -INFINITY ? 0.f : m);
                const uint64_t bias2 = pair2(bias, bias);
                const float u = take_weights<T>(s, s_at, c2, bias2);
                tmem_wait_st();
                tc_before();
                warp_arrive(&sh.pready[w][0]);
                const float v = take_weights<T>(s + kKeys / 2, s_at + kKeys / 4, c2, bias2);
                tmem_wait_st();
                tc_before();
                warp_arrive(&sh.pready[w][1]);
                l += u + v;
                if (!kHalfType) {
                    over = live ? u + v : 0.f;
                    outgrown = __any_sync(FULL, over > kSum);
                }
            } else {
                tc_before();
                warp_arrive(&sh.pready[w][0]);
                warp_arrive(&sh.pready[w][1]);
            }
            ++ns;
            ++mine;
        }
        if (mine > 0) {
            if (!warp_wait(&sh.odone[w], np & 1, ctl)) return;
            ++np;
            tc_after();
        }
        // what the merge adds: this group's columns [c0, c0 + cols) of O_w, and of the other group's O
        float f_own = 1.f, f_other = 0.f;
        unsigned o_other = 0;
        int c0 = 0, cols = DH;
        if (!pair) {
            sh.ml[w][32 * quad + lane][0] = m;
            sh.ml[w][32 * quad + lane][1] = l;
            tc_before();
            warp_arrive(&sh.merge[w]);
            if (!warp_wait(&sh.merge[w ^ 1], nm & 1, ctl)) return;
            tc_after();
            const float m2 = sh.ml[w ^ 1][32 * quad + lane][0], l2 = sh.ml[w ^ 1][32 * quad + lane][1];
            const float M = fmaxf(m, m2), use = M == -INFINITY ? 0.f : M;
            f_own = ex2(m - use);
            f_other = ex2(m2 - use);
            l = l * f_own + l2 * f_other;
            m = M;
            o_other = lanes + C::O_COL + (unsigned)((w ^ 1) * DH);
            cols = DH / 2;
            c0 = w * cols;
            ++nm;
        }
        const int r = (pair ? w * kTileRows : 0) + tr;   // row of a partial
        const int tok = tok0 + tr / a.group, h = tr % a.group;
        const long long orow = (long long)(p.cu + tok);
        const int head = p.g * a.group + h;
        const bool own_any = mine > 0;                  // O_w holds something
        const bool other_any = !pair && (w == 1 || p.nt > 1);
        if (any) {
            const bool whole = p.parts == 1;
            const int blk = (int)blockIdx.x * 2 + p.own;
            float* po = a.part_o + (size_t)blk * DH * a.part_rows;
            int* const arrivals = a.counters + p.block0 * 8 + warp;
            // Of two parts, the one that finds the other there adds the two on the
            // spot (in block order, as join_parts does); where both finish together,
            // the last to arrive does so with its sums still in tensor memory.
            bool spot = p.parts == 2, last = false;
            if (spot) {
                int seen = 0;
                if (lane == 0) seen = peek_gpu(arrivals);
                last = __shfl_sync(FULL, seen, 0) == 1;
                __syncwarp();   // the other part, which lane 0 has acquired, is there for every lane (a shuffle orders no memory)
            }
            const int mine_k = (int)blockIdx.x - p.block0;
            const int there = (p.block0 + 1 - mine_k) * 2 + mine_k;   // the other's partial: its second slot is of part 0
            const float m_own = m, l_own = l;
            float f_here = 1.f, f_there = 0.f;
            for (;;) {
                m = m_own;
                l = l_own;
                if (last) {
                    const float2 x = __ldcg(reinterpret_cast<const float2*>(
                        a.part_ml + ((size_t)(there * 2 + (pair ? 0 : w)) * a.part_rows + (live ? r : 0)) * 2));
                    const float M = fmaxf(m, x.x), use = M == -INFINITY ? 0.f : M;
                    f_here = ex2(m - use);
                    f_there = ex2(x.x - use);
                    l = mine_k == 0 ? fmaf(x.y, f_there, l * f_here) : fmaf(l, f_here, x.y * f_there);
                    m = M;
                }
                uint32_t odd = 0;   // not 0: some output is not finite
                const float inv = inverse(l);
                const float4* pt = reinterpret_cast<const float4*>(a.part_o + (size_t)there * DH * a.part_rows) + (live ? r : 0);
                // a whole item's 1 / l goes into what the groups' O count for
                const bool both = own_any && other_any;
                const unsigned from = own_any ? o_at : o_other;
                const float g1 = (own_any ? f_own : f_other) * (whole ? inv : 1.f), g2 = f_other * (whole ? inv : 1.f);
                const uint64_t gg1 = pair2(g1, g1), gg2 = pair2(g2, g2);
#pragma unroll 1
                for (int i = c0; i < c0 + cols; i += 32) {
                    float v[32];
                    uint32_t o[32], q[32];
                    tmem_ld32(from + (unsigned)i, o);
                    if (both) tmem_ld32(o_other + (unsigned)i, q);
                    tmem_wait_ld();
                    tmem_loaded<32>(o);
                    if (both) {
                        tmem_loaded<32>(q);
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            split2(fma2(pair2(__uint_as_float(q[e]), __uint_as_float(q[e + 1])), gg2,
                                        mul2(pair2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), gg1)), v[e], v[e + 1]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            split2(mul2(pair2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), gg1), v[e], v[e + 1]);
                    }
                    if (last) {
                        float4 y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = __ldcg(pt + (size_t)(i / 4 + e) * a.part_rows);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float z = e % 4 == 0 ? y[e / 4].x : e % 4 == 1 ? y[e / 4].y : e % 4 == 2 ? y[e / 4].z : y[e / 4].w;
                            v[e] = (mine_k == 0 ? fmaf(z, f_there, fmaf(v[e], f_here, 0.f))
                                                : fmaf(v[e], f_here, fmaf(z, f_there, 0.f))) * inv;
                        }
                    }
                    if (live && (whole || last)) {
                        T* dst = static_cast<T*>(a.out) + orow * a.o_stride + (long long)head * DH + i;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            const uint4 y = make_uint4(pack2(v[e], v[e + 1], T()), pack2(v[e + 2], v[e + 3], T()),
                                                       pack2(v[e + 4], v[e + 5], T()), pack2(v[e + 6], v[e + 7], T()));
                            *reinterpret_cast<uint4*>(dst + e) = y;
                            odd = times0(y.w, times0(y.z, times0(y.y, times0(y.x, odd, T()), T()), T()), T());
                        }
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(po + ((size_t)((i + e) / 4) * a.part_rows + r) * 4) =
                                make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                }
                if (whole || last) {
                    if (live && a.lse != nullptr && c0 == 0)
                        a.lse[orow * a.heads + head] = l == 0.f ? -INFINITY : (m - kLift + log2f(l)) * kLn2;
                    const bool again = __any_sync(FULL, is_odd(odd));
                    if (lane == 0 && again) sh.redo = 1;
                    if (lane == 0 && last) {
                        *arrivals = 0;
                        atomicOr(&sh.joined[p.own], 1 << warp);
                    }
                    break;
                }
                float* ml = a.part_ml + ((size_t)(blk * 2 + (pair ? 0 : w)) * a.part_rows + r) * 2;
                if (live) *reinterpret_cast<float2*>(ml) = make_float2(m, l);
                // the lanes' stores happen before lane 0's arrival (__syncwarp, then
                // release), the other blocks' before what any lane reads after it
                // (acquire, then __syncwarp)
                __syncwarp();
                int seen = 0;
                if (lane == 0) seen = arrive_gpu(arrivals);
                seen = __shfl_sync(FULL, seen, 0);
                __syncwarp();
                if (seen != p.parts - 1) break;
                if (spot) {
                    last = true;
                    continue;
                }
                const int rows = min(32, tile_rows - 32 * quad);
                const bool again = __any_sync(FULL, join_parts<T, DH>(a, p, pair, w, 32 * quad, rows, tok0, c0, cols));
                if (lane == 0) {
                    *arrivals = 0;
                    atomicOr(&sh.joined[p.own], 1 << warp);
                    if (again) sh.redo = 1;
                }
                break;
            }
        }
        if (!pair) {
            // both groups have read both O before either may be written again
            tc_before();
            warp_arrive(&sh.merged);
            if (!warp_wait(&sh.merged, (nm - 1) & 1, ctl)) return;
            tc_after();
        }
        warp_arrive(&sh.lempty[n % kListDepth]);
    }
}

// ------------------------------------------------------------ rows taken again (warps 0-7, after the block's pieces)
//
// Rows whose outputs are not finite, once more over all keys they see and only
// those, in fp32.  On the tensor cores 0 x value lets a non-finite value of a
// key that a row does not see into its sum (P is 0 there, but 0 x inf is NaN);
// weights, or the parts' sums together, may have outgrown fp32 before m
// followed; or the row sees such a value and stays as it is.  A block looks
// through what it has written itself: the halves of a cut item's rows may have
// been joined by different blocks, and each takes its half again.  No role waits
// on this, so a long cache cannot make a wait run out.
//
// Most such rows see the value themselves, and then it settles them without
// their sums: a score of NaN or infinity makes the row NaN, and a weight is above
// 0, so an element of the output is the sum of the infinities and NaN that its
// column holds.  One pass over the piece's keys and values finds those (the first
// kBadKeys of them, and per column which kinds there are); rows that it leaves
// open (a value that the row does not see, an overflow) are taken again.  A chunk
// of 4096 tokens behind 12288 with a NaN at its request's fourth position takes
// 5.0 ms so and 209 with all rows taken again (1.13 without the NaN); a token
// behind 131 thousand keys 7.0 ms, 16.5 and 0.33: one block reads its keys again.
//
// Weights carry a factor 2^-kSink, so that the sum of 2^30 of them, each 2^-31 at
// most, times the largest bf16 value stays in fp32; weights down to 2^-118 of the
// largest count in full.
//
// A warp per row, eight rows at a time over tiles of 64 keys in shared memory, a
// lane per key for the scores and per column for the sums.  A tile starts at a
// multiple of 64 whatever rows share it: same bits every time.
PI_DEV void sync_softmax() { asm volatile("bar.sync 1, 256;" ::: "memory"); }   // warps 0-7
PI_DEV void widen2(uint32_t w, float& x, float& y, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    x = f.x;
    y = f.y;
}
PI_DEV void widen2(uint32_t w, float& x, float& y, __nv_bfloat16) {
    x = __uint_as_float(w << 16);
    y = __uint_as_float(w & 0xffff0000u);
}
// keys that the row of the t-th token of a piece sees (none: hi <= lo)
PI_DEV void row_sees(const PagedArgs& a, const Piece& p, int t, int* lo, int* hi) {
    const int pos = p.first + p.tok0 + t;
    *hi = pos + 1;
    *lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
}

// where a key's elements are, or -1 for a page outside the cache (reads as zeros)
PI_DEV long long key_at(const PagedArgs& a, const int32_t* pages, int g, int key, int shift) {
    const int page = pages[key >> shift];
    if (page < 0 || page >= a.num_pages) return -1;
    return page * a.page_stride + g * a.head_stride + (key & (a.page_size - 1)) * a.token_stride;
}

constexpr int kBadKeys = 32;
template <int DH>
struct Bad {
    uint32_t key[kBadKeys];   // 4 x position + 1 (the key is bad) + 2 (the value)
    int kinds[DH];            // per column of the values: 1 NaN, 2 +inf, 4 -inf
};

// Finds the keys lo .. hi - 1 of one request and KV head that hold something not finite.
template <typename T, int DH>
PI_DEV void find_bad(const PagedArgs& a, PagedShared<DH>& sh, Bad<DH>& bad, const Piece& p, int shift) {
    constexpr int CHUNKS = DH / 8, AT_ONCE = 256 / CHUNKS, N = 4;
    const int tid = threadIdx.x, lane = tid & 31, chunk = tid % CHUNKS;
    const int32_t* pages = a.table + (size_t)p.b * a.max_pages;
    for (int base = p.lo; base < p.hi; base += N * AT_ONCE) {
        uint4 k[N], v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int key = base + i * AT_ONCE + tid / CHUNKS;
            k[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
            const long long at = key < p.hi ? key_at(a, pages, p.g, key, shift) : -1;
            if (at < 0) continue;
            k[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + at + chunk * 8);
            v[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + at + chunk * 8);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool bk = is_odd(times0(k[i].w, times0(k[i].z, times0(k[i].y, times0(k[i].x, 0u, T()), T()), T()), T()));
            const bool bv = is_odd(times0(v[i].w, times0(v[i].z, times0(v[i].y, times0(v[i].x, 0u, T()), T()), T()), T()));
            // the lanes of a key
            const unsigned of = (CHUNKS == 16 ? 0xffffu : 0xffu) << (lane & ~(CHUNKS - 1));
            const unsigned mk = __ballot_sync(FULL, bk) & of, mv = __ballot_sync(FULL, bv) & of;
            if (bv) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float f[2];
                    widen2(w[e / 2], f[0], f[1], T());
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (!(fabsf(f[j]) < INFINITY))
                            atomicOr(&bad.kinds[chunk * 8 + e + j], f[j] != f[j] ? 1 : f[j] > 0.f ? 2 : 4);
                }
            }
            if ((mk | mv) != 0 && lane == __ffs(mk | mv) - 1) {
                const int n = atomicAdd(&sh.bad_keys, 1);
                if (n < kBadKeys)
                    bad.key[n] = 4u * (uint32_t)(base + i * AT_ONCE + tid / CHUNKS) + (mk != 0 ? 1u : 0u) + (mv != 0 ? 2u : 0u);
                if (mk != 0) sh.bad_k = 1;
            }
        }
    }
}

// Settles a row (a warp; entry: 4 x row of the piece + halves) from the bad keys
// that it sees.  False: it has to be taken again.
template <typename T, int DH>
PI_DEV bool settle_row(const PagedArgs& a, const PagedShared<DH>& sh, const Bad<DH>& bad, const Piece& p,
                                        int entry, int shift) {
    constexpr int E = DH / 32;
    const int lane = threadIdx.x & 31, x = entry >> 2;
    const long long row = p.cu + p.tok0 + x / a.group;
    const int head = p.g * a.group + x % a.group;
    const int32_t* pages = a.table + (size_t)p.b * a.max_pages;
    const T* src = static_cast<const T*>(a.q) + row * a.q_stride + (long long)head * DH + lane * E;
    T* dst = static_cast<T*>(a.out) + row * a.o_stride + (long long)head * DH + lane * E;
    float q[E], o[E];
    bool nan = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = to_f(src[e]);
        nan |= q[e] != q[e];
        o[e] = 0.f;
    }
    int lo, hi;
    row_sees(a, p, x / a.group, &lo, &hi);
    const bool all = sh.bad_keys <= kBadKeys;
    bool none = __any_sync(FULL, nan) && lo < hi;   // a score of NaN or +inf: no element is a number
    for (int i = 0; i < min(sh.bad_keys, kBadKeys) && !none; ++i) {
        const uint32_t what = bad.key[i];
        const int key = (int)(what >> 2);
        if (key < lo || key >= hi) continue;
        const long long at = key_at(a, pages, p.g, key, shift) + lane * E;
        float s = 0.f;
        if (what & 1u) {
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(q[e], to_f(static_cast<const T*>(a.k)[at + e]), s);
            s = warp_sum(s) * a.scale;
            none = !(s < INFINITY);
        }
        if (what & 2u) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float v = to_f(static_cast<const T*>(a.v)[at + e]);
                if (!(fabsf(v) < INFINITY)) o[e] += s == -INFINITY ? NAN : v;
            }
        }
    }
    const bool own = (entry >> (lane >> 4)) & 1;
    bool open = false, every = true;
    bool put[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        put[e] = !(fabsf(to_f(dst[e])) < INFINITY);   // the element is not finite
        every &= put[e];
        // its kind is known: NaN, or one infinity that is the only kind there is
        const int kinds = bad.kinds[lane * E + e];
        const bool known = o[e] != o[e] || (!(fabsf(o[e]) < INFINITY) && (all || (kinds & (kinds - 1)) == 0));
        open |= put[e] && !known;
    }
    // where all elements are not finite, the row's sum of weights need not be
    if (!none && (__any_sync(FULL, own && open) || __all_sync(FULL, !own || every) || (!all && sh.bad_k != 0))) return false;
    if (own) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (none || put[e]) dst[e] = T(none ? NAN : o[e]);
    }
    if (none && a.lse != nullptr && (entry & 1) && lane == 0) a.lse[row * a.heads + head] = NAN;
    return true;
}

template <typename T, int DH>
__device__ __noinline__ void redo_rows(const PagedArgs& a, PagedShared<DH>& sh, unsigned char* smem, Walk walk) {
    constexpr int KT = 64, CHUNKS = DH / 8, ROW = DH * 2 + 16, E = DH / 32, EACH = KT * CHUNKS / 256;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float* const q = reinterpret_cast<float*>(smem) + warp * DH;   // this warp's query
    unsigned char* const kt = smem + 8 * DH * 4;                    // keys, rows 16 bytes apart in banks
    unsigned char* const vt = kt + KT * ROW;
    int* const odd = reinterpret_cast<int*>(vt + KT * DH * 2);      // 4 x row + halves (bits)
    int* const list = odd + 2 * kTileRows;                          // those that are taken again
    Bad<DH>& bad = *reinterpret_cast<Bad<DH>*>(list + 2 * kTileRows);
    const int shift = __ffs(a.page_size) - 1;
    const float c = a.scale / kLn2;
    for (;;) {
        sync_softmax();
        if (tid == 0) {
            sh.list[0] = walk.next(a);
            sh.odd_rows = sh.redo_rows = sh.bad_keys = sh.bad_k = 0;
        }
        if (tid < DH) bad.kinds[tid] = 0;
        sync_softmax();
        const Piece p = sh.list[0];
        if (p.nt == 0) return;
        const bool pair = p.toks > a.tile_tokens;
        const int bits = p.parts == 1 ? 0xff : sh.joined[p.own];   // warps whose outputs this block wrote
        for (int x = warp; x < p.toks * a.group; x += 8) {
            const int t = x / a.group, w = t >= a.tile_tokens, quad = (x - w * a.tile_tokens * a.group) >> 5;
            const int own = pair ? 3 * ((bits >> (4 * w + quad)) & 1) : ((bits >> quad) & 1) | 2 * ((bits >> (4 + quad)) & 1);
            if (own == 0) continue;
            const T* o = static_cast<const T*>(a.out) + (long long)(p.cu + p.tok0 + t) * a.o_stride +
                         (long long)(p.g * a.group + x % a.group) * DH + lane * E;
            bool some = false;
#pragma unroll
            for (int e = 0; e < E; ++e) some |= !(fabsf(to_f(o[e])) < INFINITY);
            const unsigned who = __ballot_sync(FULL, some);
            const int halves = own & ((who & 0xffffu ? 1 : 0) | (who >> 16 ? 2 : 0));
            if (halves != 0 && lane == 0) odd[atomicAdd(&sh.odd_rows, 1)] = 4 * x + halves;
        }
        sync_softmax();
        if (sh.odd_rows == 0) continue;
        find_bad<T, DH>(a, sh, bad, p, shift);
        sync_softmax();
        for (int i = warp; i < sh.odd_rows; i += 8)
            if (!settle_row<T, DH>(a, sh, bad, p, odd[i], shift) && lane == 0) list[atomicAdd(&sh.redo_rows, 1)] = odd[i];
        sync_softmax();
        const int n = sh.redo_rows;
        const int32_t* pages = a.table + (size_t)p.b * a.max_pages;
        for (int i0 = 0; i0 < n; i0 += 8) {
            // the rows' keys together, and this warp's
            int from = 0x7fffffff, to = 0, lo = 0, hi = 0;
            for (int i = i0; i < min(i0 + 8, n); ++i) {
                int l, h;
                row_sees(a, p, (list[i] >> 2) / a.group, &l, &h);
                if (l < h) {
                    from = min(from, l);
                    to = max(to, h);
                }
                if (i == i0 + warp) {
                    lo = l;
                    hi = h;
                }
            }
            const bool mine = i0 + warp < n;
            const int entry = mine ? list[i0 + warp] : 0, x = entry >> 2;
            const long long row = p.cu + p.tok0 + x / a.group;
            const int head = p.g * a.group + x % a.group;
            if (mine) {
                const T* src = static_cast<const T*>(a.q) + row * a.q_stride + (long long)head * DH + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) q[lane * E + e] = to_f(src[e]);
            }
            __syncwarp();
            float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = 0.f;
            uint4 k[EACH], v[EACH];   // this thread's part of the next tile
            auto fetch = [&](int base) {
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    const int at = tid + 256 * i, key = base + at / CHUNKS;
                    k[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
                    const long long e = key >= from && key < to ? key_at(a, pages, p.g, key, shift) : -1;
                    if (e < 0) continue;
                    k[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + e + at % CHUNKS * 8);
                    v[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + e + at % CHUNKS * 8);
                }
            };
            int base = from / KT * KT;
            if (from < to) fetch(base);
            for (; base < to; base += KT) {
                sync_softmax();   // the last tile has been read
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    const int at = tid + 256 * i;
                    *reinterpret_cast<uint4*>(kt + at / CHUNKS * ROW + at % CHUNKS * 16) = k[i];
                    *reinterpret_cast<uint4*>(vt + at * 16) = v[i];
                }
                sync_softmax();
                if (base + KT < to) fetch(base + KT);
                if (!mine || hi <= base || lo >= base + KT) continue;
                float s[2] = {0.f, 0.f};
#pragma unroll
                for (int d = 0; d < CHUNKS; ++d) {
                    const float4 q0 = *reinterpret_cast<const float4*>(q + 8 * d), q1 = *reinterpret_cast<const float4*>(q + 8 * d + 4);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 y = *reinterpret_cast<const uint4*>(kt + (lane + 32 * j) * ROW + d * 16);
                        float f[8];
                        widen2(y.x, f[0], f[1], T());
                        widen2(y.y, f[2], f[3], T());
                        widen2(y.z, f[4], f[5], T());
                        widen2(y.w, f[6], f[7], T());
                        s[j] = fmaf(q0.x, f[0], fmaf(q0.y, f[1], fmaf(q0.z, f[2], fmaf(q0.w, f[3], s[j]))));
                        s[j] = fmaf(q1.x, f[4], fmaf(q1.y, f[5], fmaf(q1.z, f[6], fmaf(q1.w, f[7], s[j]))));
                    }
                }
                float top = m;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int key = base + lane + 32 * j;
                    s[j] = key >= lo && key < hi ? s[j] * c : -INFINITY;
                    top = fmaxf(top, s[j]);
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, d));
                const float use = top == -INFINITY ? 0.f : top, f = exp2f(m - use);
                const float w[2] = {exp2f(s[0] - use - kSink), exp2f(s[1] - use - kSink)};
                m = top;
                l = l * f + (w[0] + w[1]);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] *= f;
                const int x0 = max(lo - base, 0), x1 = min(hi - base, KT);
                auto value = [&](int x, float (&y)[E]) {
                    const uint32_t* src = reinterpret_cast<const uint32_t*>(vt + (x * DH + lane * E) * 2);
#pragma unroll
                    for (int e = 0; e < E; e += 2) widen2(src[e / 2], y[e], y[e + 1], T());
                };
                if (!__any_sync(FULL, (w[0] == 0.f && s[0] > -INFINITY) || (w[1] == 0.f && s[1] > -INFINITY))) {
#pragma unroll 8
                    for (int x = x0; x < x1; ++x) {
                        const float wx = __shfl_sync(FULL, x < 32 ? w[0] : w[1], x & 31);
                        float y[E];
                        value(x, y);
#pragma unroll
                        for (int e = 0; e < E; ++e) o[e] = fmaf(wx, y[e], o[e]);
                    }
                } else {
                    // e^a is not 0 but for a = -inf, so infinities count although the weight's fp32 is 0
#pragma unroll 1
                    for (int x = x0; x < x1; ++x) {
                        const float wx = __shfl_sync(FULL, x < 32 ? w[0] : w[1], x & 31);
                        const float sx = __shfl_sync(FULL, x < 32 ? s[0] : s[1], x & 31);
                        float y[E];
                        value(x, y);
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            o[e] = wx == 0.f && sx > -INFINITY && !(fabsf(y[e]) < INFINITY) ? o[e] + y[e] : fmaf(wx, y[e], o[e]);
                    }
                }
            }
            l = warp_sum(l);
            if (mine) {
                if ((entry >> (lane >> 4)) & 1) {
                    T* dst = static_cast<T*>(a.out) + row * a.o_stride + (long long)head * DH + lane * E;
#pragma unroll
                    for (int e = 0; e < E; ++e) dst[e] = T(l == 0.f ? 0.f : o[e] / l);
                }
                if (a.lse != nullptr && (entry & 1) && lane == 0)
                    a.lse[row * a.heads + head] = l == 0.f ? -INFINITY : (m + log2f(l * exp2f(kSink))) * kLn2;
            }
            __syncwarp();
        }
    }
}

template <typename T, int DH>
__global__ void __launch_bounds__(kPagedThreads, 1) k_paged_attn(const __grid_constant__ PagedArgs a) {
    pdl_entry();
    using C = PagedCfg<DH>;
    extern __shared__ __align__(1024) unsigned char paged_smem[];
    unsigned char* qs = paged_smem;
    unsigned char* ring = qs + C::Q;
    unsigned char* vring = ring + C::SK * C::TILE;
    PagedShared<DH>& sh = *reinterpret_cast<PagedShared<DH>*>(vring + C::SV * C::TILE);
    static_assert(sizeof(PagedShared<DH>) <= C::MISC, "bookkeeping");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((su32(paged_smem) & 1023u) != 0) {   // the tiles' swizzle needs it; the whole block leaves
        if (tid == 0) atomicExch(a.status, (int)PI_ERR_UNSUPPORTED);
        return;
    }
    if (warp == 9) {
        if (lane == 0) {
            for (int s = 0; s < 6; ++s) {
                bar_init(&sh.kfull[s], 1);
                bar_init(&sh.kempty[s], 1);
                bar_init(&sh.vfull[s], 1);
                bar_init(&sh.vempty[s], 1);
            }
            bar_init(&sh.qfull, 1);
            bar_init(&sh.qempty, 1);
            for (int w = 0; w < 2; ++w) {
                bar_init(&sh.sfull[w], 1);
                bar_init(&sh.pready[w][0], 4);
                bar_init(&sh.pready[w][1], 4);
                bar_init(&sh.odone[w], 1);
                bar_init(&sh.merge[w], 4);
            }
            for (int s = 0; s < kListDepth; ++s) {
                bar_init(&sh.lfull[s], 1);
                bar_init(&sh.lempty[s], kConsumers);
            }
            bar_init(&sh.merged, 8);
            bar_init(&sh.drain, 1);
            sh.abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        tmem_alloc(&sh.tmem, 512);
    }
    if (tid == 0) {   // no work, unless a thread finds this block's start below
        sh.walk = Walk{};
        sh.walk.u = 0x7fffffffffffffffll;
        sh.redo = sh.joined[0] = sh.joined[1] = 0;
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_map(&a.kmap);
        tma_prefetch_map(&a.vmap);
        tma_prefetch_map(&a.qmap);
    }
    // units of all requests: each thread sums a run of them, then a prefix over
    // the threads (scratch in the ring, which nothing uses yet)
    long long* sums = reinterpret_cast<long long*>(ring);
    const int per = (a.batch + kPagedThreads - 1) / kPagedThreads;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    long long own = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) own += a.kv_heads * request_units(a, request(a, b, &bad));
    if (bad && blockIdx.x == 0) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
    long long pre = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(FULL, pre, o);
        if (lane >= o) pre += x;
    }
    if (lane == 31) sums[warp] = pre;
    tc_before();
    __syncthreads();
    tc_after();
    long long U = 0, before = 0;
    for (int i = 0; i < kPagedThreads / 32; ++i) {
        if (i < warp) before += sums[i];
        U += sums[i];
    }
    pre += before - own;   // units before this thread's requests
    const unsigned tmem = sh.tmem;
    // blocks with work: about two tiles each at least, one for each softmax group
    // (a part costs a join, the second tile runs beside the first); U / G is
    // kMinUnits or more, or all
    const int G = (int)min((long long)gridDim.x, max(U / kMinUnits, U > 0 ? 1ll : 0ll));
    const int blk = blockIdx.x;
    const long long u0 = G > 0 ? quotient(U * blk, G) : 0, u1 = G > 0 ? quotient(U * (blk + 1), G) : 0;
    const bool work = blk < G;
    if (tid == 0) {
        sh.walk.u1 = u1;
        sh.walk.U = U;
        sh.walk.G = G;
    }
    if (work && pre <= u0 && u0 < pre + own) {
        // this block's range starts in this thread's requests
        long long left = u0 - pre;
        int b = b0;
        for (; b < b1; ++b) {
            const Request r = request(a, b, &bad);
            const long long u = request_units(a, r);
            if (left >= a.kv_heads * u) {
                left -= a.kv_heads * u;
                continue;
            }
            const int g = (int)quotient(left, u);
            left -= g * u;
            // the item: the last one that starts at or before `left`
            const int d = 2 * a.tile_tokens;
            int i0 = 0, i1 = (r.n + d - 1) / d;
            if (i1 > kWalk) {
                while (i1 - i0 > 1) {
                    const int mid = (i0 + i1) / 2;
                    if (units_before(a, r, mid) <= left) i0 = mid;
                    else i1 = mid;
                }
                left -= units_before(a, r, i0);
            } else {
                int toks, lo, hi;
                for (;; ++i0) {
                    const int nt = item_tiles(a, r, i0 * d, &toks, &lo, &hi);
                    const int cost = kItemCost + nt * tile_cost(a, toks);
                    if (left < cost) break;
                    left -= cost;
                }
            }
            const int tok0 = i0 * d;
            sh.walk.u = u0;
            sh.walk.b = b;
            sh.walk.g = g;
            sh.walk.tok0 = tok0;
            sh.walk.off = (int)left;
            sh.walk.r = r;
            break;
        }
    }
    fence_async_smem();   // the scratch in the ring, before copies land there
    __syncthreads();
    const Ctl ctl{a.status, a.timeout_ns, &sh.abort_flag};
    if (work) {
        // 384 threads x 168 registers at launch = 256 x 200 + 128 x 104
        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
            softmax_role<T, DH>(a, sh, tmem, ctl);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
            if (warp == 8)
                tile_role<DH, false>(a, sh, ring, ctl);
            else if (warp == 9)
                mma_role<T, DH>(a, sh, qs, ring, vring, tmem, ctl);
            else if (warp == 10)
                tile_role<DH, true>(a, sh, vring, ctl);
            else if (lane == 0)
                list_role<DH>(Lengths(a), &a.qmap, sh, qs, sh.walk, ctl);
        }
    }
    tc_before();
    __syncthreads();
    if (warp == 9) {
        tc_after();
        tmem_free(tmem, 512);
    }
    // all copies and products are in, the tiles' shared memory is free
    if (warp < 8 && sh.redo != 0 && sh.abort_flag == 0) redo_rows<T, DH>(a, sh, qs, sh.walk);
}

bool paged_ok(const pi_paged_desc& d, const pi_page_desc& c) {
    return page_desc_ok(c) && d.heads >= 1 && d.heads <= 1024 && d.heads % c.kv_heads == 0 &&
           d.heads / c.kv_heads <= 128 && d.batch >= 1 && d.batch <= 4096 && d.max_tokens >= 0 &&
           d.max_tokens <= (1 << 24) && d.max_new >= 1 && (d.max_tokens == 0 || d.max_new <= d.max_tokens) &&
           d.max_pages >= 1 && (long long)d.max_pages * c.page_size <= (1ll << 30) && d.window >= 0 &&
           d.scale >= 0.f && isfinite(d.scale);
}

// SMs of the current device (the grid is one block on each), 0 on failure.
int paged_blocks() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

// Workspace: arrival counters at offset 0 (the same place for every
// descriptor), then the partials of two items per block.
struct PagedLayout {
    size_t ml, o, total;
    int rows;
    PagedLayout(const pi_paged_desc& d, const pi_page_desc& c, int blocks) {
        const int group = d.heads / c.kv_heads, tile_tokens = kTileRows / group;
        rows = d.max_new > tile_tokens ? 2 * kTileRows : (d.max_new * group + 31) / 32 * 32;
        auto up = [](size_t v) { return (v + 255) / 256 * 256; };
        ml = up((size_t)blocks * 8 * sizeof(int));
        o = up(ml + (size_t)blocks * 2 * 2 * rows * 2 * sizeof(float));
        total = up(o + (size_t)blocks * 2 * c.head_dim * rows * sizeof(float));
    }
};

bool cache_map(CUtensorMap* m, const void* base, const pi_page_desc& c) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t blocks = (cuuint64_t)((c.kv_heads - 1) * (c.head_stride / 64) + c.head_dim / 64);
    const cuuint64_t dims[5] = {64, 8, blocks, (cuuint64_t)(c.page_size / 8), (cuuint64_t)c.num_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)c.token_stride * 2, 128, (cuuint64_t)c.token_stride * 16,
                                   (cuuint64_t)c.page_stride * 2};
    const cuuint32_t box[5] = {64u, 8u, (cuuint32_t)(c.head_dim / 64), (cuuint32_t)(c.page_size / 8), 1u};
    const cuuint32_t es[5] = {1u, 1u, 1u, 1u, 1u};
    return fn(m, c.dtype == PI_T_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
              const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool query_map(CUtensorMap* m, const void* base, const PagedArgs& a, int dh, int dtype) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)dh, (cuuint64_t)a.heads, (cuuint64_t)a.max_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)dh * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)a.group, (cuuint32_t)a.tile_tokens};
    const cuuint32_t es[3] = {1u, 1u, 1u};
    return fn(m, dtype == PI_T_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DH>
cudaError_t launch_paged(const PagedArgs& a, int blocks, cudaStream_t s) {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            e = cudaFuncSetAttribute(k_paged_attn<T, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, PagedCfg<DH>::SMEM);
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    return launch_pdl(k_paged_attn<T, DH>, blocks, kPagedThreads, PagedCfg<DH>::SMEM, s, a);
}

}  // namespace
}  // namespace pi

using namespace pi;

extern "C" {

size_t pi_paged_workspace_bytes(const pi_paged_desc* desc, const pi_page_desc* cache) {
    if (!desc || !cache || !paged_ok(*desc, *cache)) return 0;
    // without a device (descriptors checked on a host), as for one SM
    return PagedLayout(*desc, *cache, std::max(1, paged_blocks())).total;
}

pi_status pi_paged_attn(const pi_paged_desc* desc, const pi_page_desc* cache, const void* q, long long q_stride,
                        const void* kcache, const void* vcache, const int32_t* block_table, const int32_t* cu_new,
                        const int32_t* kv_len, void* out, long long out_stride, float* lse, void* workspace,
                        size_t ws_bytes, void* stream) {
    if (!desc || !cache || !paged_ok(*desc, *cache)) return PI_ERR_INVALID_ARG;
    const long long width = (long long)desc->heads * cache->head_dim;
    if (q_stride % 8 != 0 || q_stride < width || out_stride % 8 != 0 || out_stride < width) return PI_ERR_INVALID_ARG;
    if (desc->max_tokens == 0) return PI_OK;
    auto aligned = [](const void* p, size_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    if (!aligned(q, 16) || !aligned(kcache, 16) || !aligned(vcache, 16) || !aligned(out, 16) ||
        !aligned(block_table, 4) || !aligned(cu_new, 4) || !aligned(kv_len, 4) || (lse && !aligned(lse, 4)))
        return PI_ERR_INVALID_ARG;
    const int blocks = paged_blocks();
    const PagedLayout lay(*desc, *cache, std::max(1, blocks));
    if (!aligned(workspace, 16) || ws_bytes < lay.total) return PI_ERR_WORKSPACE;
    // rows that are not finite are computed again from q after outputs are written
    if (rows_overlap(q, 2 * q_stride, 2 * width, out, 2 * out_stride, 2 * width, desc->max_tokens)) return PI_ERR_INVALID_ARG;
    PagedArgs a{};
    char* ws = static_cast<char*>(workspace);
    a.q = q;
    a.k = kcache;
    a.v = vcache;
    a.table = block_table;
    a.cu = cu_new;
    a.kv = kv_len;
    a.out = out;
    a.lse = lse;
    a.q_stride = q_stride;
    a.o_stride = out_stride;
    a.page_stride = cache->page_stride;
    a.head_stride = cache->head_stride;
    a.token_stride = cache->token_stride;
    a.heads = desc->heads;
    a.kv_heads = cache->kv_heads;
    a.batch = desc->batch;
    a.max_tokens = desc->max_tokens;
    a.max_new = desc->max_new;
    a.max_pages = desc->max_pages;
    // a window of all positions a row can hold, or more, is none; below that,
    // sums with first positions (down to -2^24) stay far from the ends of int
    a.window = (long long)desc->window >= (long long)desc->max_pages * cache->page_size ? 0 : desc->window;
    a.page_size = cache->page_size;
    a.num_pages = cache->num_pages;
    a.group = desc->heads / cache->kv_heads;
    a.tile_tokens = kTileRows / a.group;
    a.head_blocks = (int)(cache->head_stride / 64);
    a.part_rows = lay.rows;
    a.scale = desc->scale > 0.f ? desc->scale : 1.0f / sqrtf((float)cache->head_dim);
    a.counters = reinterpret_cast<int*>(ws);
    a.part_ml = reinterpret_cast<float*>(ws + lay.ml);
    a.part_o = reinterpret_cast<float*>(ws + lay.o);
    a.status = status_word();
    a.timeout_ns = wait_timeout_ns();
    if (blocks < 1 || a.status == nullptr || !cache_map(&a.kmap, kcache, *cache) || !cache_map(&a.vmap, vcache, *cache) ||
        !query_map(&a.qmap, q, a, cache->head_dim, cache->dtype))
        return PI_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (cache->dtype == PI_T_F16)
        e = cache->head_dim == 128 ? launch_paged<__half, 128>(a, blocks, s) : launch_paged<__half, 64>(a, blocks, s);
    else
        e = cache->head_dim == 128 ? launch_paged<__nv_bfloat16, 128>(a, blocks, s)
                                   : launch_paged<__nv_bfloat16, 64>(a, blocks, s);
    return e == cudaSuccess ? PI_OK : PI_ERR_CUDA;
}

}  // extern "C"
