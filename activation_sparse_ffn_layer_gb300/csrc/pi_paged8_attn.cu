// pi_paged8_attn.cu -- causal attention of new tokens over the 8-bit paged cache.
//
// Requests of few rows (tokens x query heads of a KV head; decode steps among
// them) are bound by the bytes of codes, and k_attn8_few takes them straight from
// the codes.  Requests of many rows are bound by products: the pages that they
// see are widened to 16 bits in the workspace once (widen_pages, in the same
// launch), and the 16-bit cache's kernel takes them from there on the tcgen05
// tensor cores.  A step may hold both.
//
// k_attn8_few: an item is up to 8 or 16 rows of one request and KV head (row =
// token * group + head in the group).  A warp takes 32 keys at a time, two blocks
// of the cache:
//     S = Q K^T           (codes as fp16, which holds them exactly; fp32 sums)
//     x = c 2^ek S        (c = scale / ln 2; ek the exponent of the keys' block)
//     P = 2^(x + ev - m)  (ev the exponent of the values' block)
//     O += P V            (codes as fp16 again), l += 2^-ev sum P
// so that P counts how much a key adds to the output, whatever its block's
// exponent, and m trails the largest of those: it moves only where a weight
// would pass 2^15 (fp16 holds P, which carries a factor 2^7 that l and O share;
// weights down to 2^-32 of the largest survive the rounding).  A mma.sync
// fragment wants 2 elements of a row at a time and has the lanes' columns
// interleaved; which element of a head is which column is free as long as queries
// and keys, or values and outputs, agree, so a lane takes 16 bytes in a row.  With
// 8 rows of work for each key the products are a quarter of what mma.sync can do
// here, and tcgen05 would not pay: its smallest M is 64.
//
// Work split: the (item x tile of 32 keys) space is cut into equal contiguous
// ranges per block and then per warp, whatever the lengths; a warp goes through its
// range by itself, with a ring of tiles of its own.  Items that warps of a block
// share are added up once at its end; of an item that blocks share each leaves
// unnormalised partials (m, l, O) in the workspace, and the block that arrives last
// adds them in block order (the order is fixed, who does it is not: same bits).
//
// Bounds and figures (GB300, 64 query and 8 KV heads of 128 unless said):
//  - four sequences with 120-131 thousand keys, bf16: 185-204 us, 5.1-5.6 TB/s; the
//    memory and 10 us of start and joins.  Copies alone take 171 us of 182 (heads first).
//  - 32 sequences with 500-8000 keys, fp16: 57 us, 4.0 TB/s.  The first tile is there
//    after 10 us (3 to know the work, then every SM asks for 190 KB at once), the last
//    after 50 (5.0 TB/s meanwhile), the joins take 8.
//  - five tokens of each of 24 sequences, 200-6000 keys, bf16: 92 us.  40 rows are three
//    items, each of which copies the keys from L2: 450 MB, which at the 22 bytes a cycle
//    of an SM's copies take 70 us.
//  - one sequence with 1001 keys: 14-15 us of latency: 3 to know the work, 1.5 for page and
//    copies each, 1 for a tile, 5 for the two joins.  (Codes straight into registers took 11 us here,
//    and 73 instead of 57 for the 32 sequences, 261 instead of 190 for the long ones.)
//  - requests of many rows add the widening to the 16-bit kernel's time: 4096 tokens behind
//    12288, 17 us of 1160; a prompt of 1999 (12 heads of 64) 5 of 39; in a mixed step of 16
//    sequences (32 heads, window of 2000) 38 of 175, 0.92 of the memory's rate.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "pi_common.cuh"
#include "pi_e4m3.cuh"
#include "pi_internal.h"
#include "pi_pipe.cuh"
#include "pi_umma.cuh"

namespace pi {
namespace {

using namespace e4m3;
using namespace pipe;

constexpr int kRows = 16;            // rows of an item
constexpr int kFewRows = 64;         // rows of a request up to which it goes through k_attn8_few (or one token's)
constexpr int kTile = 32;            // keys of a unit of the work split
// Units that an item counts besides its tiles.  Of 2, 3, 5 and 8 (replayed, L2 flushed) a mixed
// step of 16 sequences takes 176, 174, 173 and 170 us, 32 decoding sequences 62.2, 61.2, 60.7 and
// 60.7, 16 of 32 heads 111, 111, 110.5 and 110, five tokens of 24 sequences 95.6, 92.7, 92.7 and
// 93.0, one sequence 14.6, 15.6, 15.1 and 14.1: fewer cost the steps of many items, more than 5
// gain 2 % of the mixed step and of the shortest call and nothing elsewhere.
constexpr int kLead = 5;
// Units of a block at least: with 2, 3, 4, 6 and 8 one sequence with 1001 keys takes 17.7, 16.7,
// 15.1, 15.6 and 16.2 us (replayed); steps that fill the blocks anyway do not change.
constexpr int kMinUnits = 4;
constexpr float kLift = 7.f;         // log2 of the factor that P, l and O share
constexpr float kGrow = 8.f;         // growth (log2) of a maximum before m follows
constexpr float kLn2 = 0.69314718055994531f;

struct Few8Args {
    // {dh / 4 words, positions of a page, heads, pages, arrays}, box dh / 4 x 16 or 32 positions
    // of every array: keys and values of the lower address first, where `both`, else an array each
    CUtensorMap kmap, vmap;
    int both;
    int k_at, v_at, block_step;   // bytes: keys, values of a slot's first block, and the second block behind the first
    Cache8 c;
    const void* q;
    const int32_t *table, *cu, *kv;
    void* out;
    float* lse;
    long long q_stride, o_stride;
    int heads, batch, max_tokens, max_new, max_pages, window, group, few, rows;   // rows of an item: 8 or 16
    float scale;
    int* counters;     // [blocks] arrivals at an item that blocks share
    float* part_ml;    // [blocks][2][16][2]: a block's sums of such items
    float4* part_o;    // [blocks][2][chunks][32]
    float4* warp_o;    // [blocks][warps][2][chunks][32]: a warp's sums of items that warps share
    void *wide_k, *wide_v;   // [num_pages, kv_heads, page_size, dh] in 16 bits, or null: no long requests
    int* status;
    long long timeout_ns;
};

struct Request8 {
    int cu, n, first;   // first row of q, tokens, position of the first token
};

// A request as the 16-bit cache's attention takes it: inconsistent lengths count as none.
template <typename A>
PI_DEV Request8 request8(const A& a, int b, bool* bad) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    int kv = a.kv[b];
    Request8 r{lo, hi - lo, 0};
    if (lo < 0 || hi < lo || hi > a.max_tokens || hi - lo > a.max_new) {
        *bad = true;
        r.n = 0;
    }
    if (kv < 0 || kv > a.max_pages << a.c.page_shift) {
        *bad = true;
        kv = 0;
    }
    r.first = kv - r.n;
    return r;
}

// Sum of v over the threads before this one, and over all (in *all); scratch: 33 values.
template <int THREADS>
PI_DEV long long scan_before(long long v, long long* scratch, long long* all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long pre = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(FULL, pre, o);
        if (lane >= o) pre += x;
    }
    if (lane == 31) scratch[warp] = pre;
    __syncthreads();
    long long before = 0, sum = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) before += scratch[i];
        sum += scratch[i];
    }
    *all = sum;
    return before + pre - v;
}

// Keys that rows 16 rt .. of a request see together, and their tiles (one, with
// nothing to see in it, where there are none: it writes the zeros).
PI_DEV int item_range(const Few8Args& a, const Request8& r, int rt, int* lo, int* hi) {
    const int t0 = rt * a.rows / a.group, t1 = min(rt * a.rows + a.rows - 1, r.n * a.group - 1) / a.group;
    *hi = r.first + t1 + 1;
    *lo = a.window > 0 ? max(0, r.first + t0 - a.window + 1) : 0;
    if (*hi <= *lo) {
        *lo = *hi = 0;
        return 1;
    }
    return (*hi + kTile - 1) / kTile - *lo / kTile;
}
PI_DEV int row_tiles(const Few8Args& a, const Request8& r) { return r.n > a.few ? 0 : (r.n * a.group + a.rows - 1) / a.rows; }
PI_DEV long long request_units(const Few8Args& a, const Request8& r) {   // of one KV head
    long long u = 0;
    int lo, hi;
    for (int rt = 0; rt < row_tiles(a, r); ++rt) u += kLead + item_range(a, r, rt, &lo, &hi);
    return u;
}

// A range of key tiles of one item.
struct Piece8 {
    long long i0;    // the item's first unit
    int nt;          // key tiles (0: end)
    int from, all;   // the first of them and how many there are, counted from the item's first
    int lo, hi;      // keys that some row of the item sees
    int b, g, rt;
    int rows;        // of the item
    int first, cu;   // of the request
};

struct Walk8 {
    Request8 r;
    long long u, u1;        // unit reached, the range's end
    int b, g, rt, off;      // request, KV head, row tile and unit within the item at u

    PI_DEV Piece8 next(const Few8Args& a) {
        Piece8 p{};
        while (u < u1 && p.nt == 0) {   // again where only an item's lead falls into this range
            int lo, hi;
            const int nt = item_range(a, r, rt, &lo, &hi);
            p.i0 = u - off;
            const int stop = (int)min((long long)(kLead + nt), u1 - p.i0);
            p.from = max(off - kLead, 0);
            p.nt = max(max(stop - kLead, 0) - p.from, 0);
            p.all = nt;
            p.lo = lo;
            p.hi = hi;
            p.b = b;
            p.g = g;
            p.rt = rt;
            p.rows = min(a.rows, r.n * a.group - rt * a.rows);
            p.first = r.first;
            p.cu = r.cu;
            u = stop > off ? p.i0 + stop : u1;   // (off past the item: the lengths changed under the kernel)
            off = 0;
            if (u < u1 && ++rt >= row_tiles(a, r)) {
                rt = 0;
                if (++g == a.c.kv_heads) {
                    g = 0;
                    do {
                        if (++b >= a.batch) {   // the lengths changed under the kernel: stop
                            u = u1;
                            break;
                        }
                        bool bad = false;
                        r = request8(a, b, &bad);
                    } while (row_tiles(a, r) == 0);
                }
            }
        }
        return p;
    }
};

// a / b for positive numbers, in 32 bits where they fit (a 64-bit division is a call)
PI_DEV long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
    return a / b;
}

PI_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
PI_DEV uint32_t half2_of(float x, float y) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// d += a b: 16 x 16 by 16 x 8, fp16 with fp32 sums
PI_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
PI_DEV int arrive_gpu(int* p) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
    return old;
}

// Two queries as fp16: fp16 as they are, bf16 (8 bits of significand) times a
// power of two that brings the row's largest to 2^14: exact but for elements
// below 2^-28 of it.
PI_DEV uint32_t query2(uint32_t w, float f, __nv_bfloat16) {
    return half2_of(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
}
PI_DEV uint32_t query2(uint32_t w, float, __half) { return w; }

// The codes of a tile of 32 keys, a row a position, 16-byte pieces in the order that the
// copies' swizzle gives them.  One copy brings keys and values of 32 positions (of 16 where
// pages hold no more; with copies of their own for keys and for values 32 decoding sequences
// take 58.4 us, so 57.4).  Plain asynchronous copies by the lanes, 16 bytes each, bring 5.2
// TB/s at most, and some SMs get a third less than others: 68 us.  Of the keys of a block a
// lane uses 8 j + lane / 4, elements 16 q .. and 64 + 16 q .. (q = lane % 4); of the values
// 2 q, 2 q + 1, 2 q + 8, 2 q + 9, elements (dh / 8) (lane / 4) ..
template <int DH>
struct Slot8 {
    static constexpr int KC = DH / 64, VW = DH / 32;   // 16-byte pieces of a lane's key, words of its value
    unsigned char bytes[2 * kTile * DH];

    static PI_DEV int at(int row, int piece) {
        return row * DH + ((DH == 128 ? piece ^ (row & 7) : piece ^ ((row >> 1) & 3)) * 16);
    }
    // (block: where the block's keys, or its values, begin)
    PI_DEV uint4 key(int block, int j, int c) const {
        const int lane = threadIdx.x & 31;
        return *reinterpret_cast<const uint4*>(bytes + block + at(8 * j + (lane >> 2), (lane & 3) + 4 * c));
    }
    PI_DEV void value(int block, int x, uint32_t (&w)[VW]) const {
        const int lane = threadIdx.x & 31, row = 2 * (lane & 3) + (x & 1) + 8 * (x >> 1), r8 = lane >> 2;
        if (DH == 128) {
            const uint4 z = *reinterpret_cast<const uint4*>(bytes + block + at(row, r8));
            w[0] = z.x;
            w[1] = z.y;
            w[VW - 2] = z.z;
            w[VW - 1] = z.w;
        } else {
            const uint2 z = *reinterpret_cast<const uint2*>(bytes + block + at(row, r8 >> 1) + (r8 & 1) * 8);
            w[0] = z.x;
            w[1] = z.y;
        }
    }
};

// Warps of a block, one block on an SM: what registers leave room for.  (Items of 8 rows for
// 24 x 40 rows: 116 us, of 16 rows 92; items of 16 on 12 warps, which spill: 97.)
template <int DH, bool HALF>
struct Few8Cfg {
    static constexpr int WARPS = HALF ? 12 : 8, THREADS = 32 * WARPS;
    static constexpr int CHUNKS = HALF ? DH / 16 : DH / 8;   // float4 of a lane's part of O
    static constexpr int STAGES = DH == 64 ? 4 : HALF ? 2 : 3;   // slots of a warp's ring
};
constexpr int kMostWarps = 12;

template <int DH, bool HALF>
struct Few8Shared {
    using C = Few8Cfg<DH, HALF>;
    Slot8<DH> ring[C::WARPS][C::STAGES];
    unsigned long long full[C::WARPS][C::STAGES];   // a slot's codes are there
    int abort_flag;
    float2 ml[C::WARPS][2][kRows];     // m and l of pieces that warps share, as of their O in warp_o
    long long scratch[C::WARPS + 1];
    long long before[C::THREADS];      // units of the requests before those that a thread has counted
    Walk8 walk[C::WARPS];
    Piece8 piece[C::WARPS][2];         // a warp's next pieces
    Piece8 cut[C::WARPS][2];           // those that it shares: the one it does not begin, the one it does not end
    bool stays[C::WARPS][2];           // their sums are in the warp's ring (else in warp_o)
    Piece8 open[2];                    // items that the block shares with others, by whether it begins them
    int parts[2], seen[2];
};

// This lane's rows r = lane / 4 and r + 8 of an item.
struct Rows8 {
    int lo[2], hi[2];      // keys they see
    float c[2];            // scale / ln 2 (times the power of two taken out of the queries)
    float m[2], l[2];
};

// One tile: two blocks of 16 keys from kb on, with exponents ek and ev.
// HALF: rows 8 .. 15 hold nothing.
template <int DH, bool HALF>
PI_DEV void step(const Few8Args& a, const Piece8& p, const Slot8<DH>& s, const int (&ek)[2], const int (&ev)[2], int kb, bool edge,
                 const uint32_t (&q)[DH / 16][4], Rows8& w, float (&o)[DH / 8][4]) {
    constexpr int KC = Slot8<DH>::KC, VW = Slot8<DH>::VW, RH = HALF ? 1 : 2, NB = 2;
    const int lane = threadIdx.x & 31, q4 = lane & 3;
    float acc[NB][2][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b][j][e] = 0.f;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
        uint4 y[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) y[b][j] = s.key(a.k_at + b * a.block_step, j, c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t word = i == 0 ? y[b][j].x : i == 1 ? y[b][j].y : i == 2 ? y[b][j].z : y[b][j].w;
                    mma16816(acc[b][j], q[4 * c + i], widen2(word & 0xffffu), widen2(word >> 16));
                }
    }
    // x = c 2^ek S of this lane's keys kb + 16 b + 8 j + 2 q + e
    float x[NB][2][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const float fk = pow2(ek[b]);
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            const float f = fminf(w.c[h] * fk, 3e38f);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 2 * h; e < 2 * h + 2; ++e)
                    x[b][j][e] = acc[b][j][e] * f;
        }
    }
    uint32_t see = ~0u;    // bit 8 b + 4 j + 2 h + e: the row sees the key
    if (edge) {
        see = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < RH; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = kb + 16 * b + 8 * j + 2 * q4 + e;
                        if (key >= w.lo[h] && key < w.hi[h]) see |= 1u << (8 * b + 4 * j + 2 * h + e);
                        else x[b][j][2 * h + e] = -INFINITY;
                    }
    }
    // m, where it has to move
    bool grown = false;
    float top[2];
#pragma unroll
    for (int h = 0; h < RH; ++h) {
        top[h] = -INFINITY;
#pragma unroll
        for (int b = 0; b < NB; ++b)
            top[h] = fmaxf(top[h], fmaxf(fmaxf(x[b][0][2 * h], x[b][0][2 * h + 1]), fmaxf(x[b][1][2 * h], x[b][1][2 * h + 1])) + (float)ev[b]);
        grown |= top[h] > w.m[h] + kGrow;
    }
    if (__any_sync(FULL, grown)) {
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(FULL, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(FULL, top[h], 2));
            const float to = fmaxf(w.m[h], top[h]), f = to > w.m[h] ? ex2(w.m[h] - to) : 1.f;
            w.m[h] = to;
            w.l[h] *= f;
#pragma unroll
            for (int i = 0; i < DH / 8; ++i) {
                o[i][2 * h] *= f;
                o[i][2 * h + 1] *= f;
            }
        }
    }
    uint32_t pk[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (HALF) pk[b][1] = pk[b][3] = 0u;
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            const float bias = kLift + (float)ev[b] - (w.m[h] == -INFINITY ? 0.f : w.m[h]);
            float y[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) y[j][e] = ex2(x[b][j][2 * h + e] + bias);
            w.l[h] = fmaf((y[0][0] + y[0][1]) + (y[1][0] + y[1][1]), pow2(-ev[b]), w.l[h]);
            pk[b][h] = half2_of(y[0][0], y[0][1]);
            pk[b][2 + h] = half2_of(y[1][0], y[1][1]);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        uint32_t v[4][VW];
#pragma unroll
        for (int y = 0; y < 4; ++y) s.value(a.v_at + b * a.block_step, y, v[y]);
        if (edge) {
            // values of keys that no row sees are not used, whatever they are; and 0 x NaN
            // would reach rows that do not see the value: such codes leave the product, and
            // the rows that see one become NaN there
            bool nan = false;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int key = kb + 16 * b + 8 * (y >> 1) + 2 * q4 + (y & 1);
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    if (key < p.lo || key >= p.hi) v[y][i] = 0u;
                    nan |= (((v[y][i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                }
            }
            if (__any_sync(FULL, nan)) {
                uint32_t seen[4];   // 1 where the row sees the key
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = 8 * b + 4 * (i >> 1) + 2 * (i & 1);
                    seen[i] = HALF && (i & 1) ? 0u : ((see >> at) & 1 ? 0x3c00u : 0u) | ((see >> (at + 1)) & 1 ? 0x3c000000u : 0u);
                }
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    uint32_t one[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t is = (((v[y][i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
                        v[y][i] &= ~(is * 255u);
                        one[y] = is * 0x38u;   // the code of 1
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float n[4] = {0.f, 0.f, 0.f, 0.f};
                        const int sh = 8 * c;
                        mma16816(n, seen, widen2(((one[0] >> sh) & 255u) | ((one[1] >> sh) & 255u) << 8),
                                 widen2(((one[2] >> sh) & 255u) | ((one[3] >> sh) & 255u) << 8));
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n[e] > 0.f) o[4 * i + c][e] = NAN;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            // bytes of two keys side by side: elements 4 i, 4 i + 1 and 4 i + 2, 4 i + 3
            const uint32_t a0 = __byte_perm(v[0][i], v[1][i], 0x5140), a1 = __byte_perm(v[0][i], v[1][i], 0x7362);
            const uint32_t b0 = __byte_perm(v[2][i], v[3][i], 0x5140), b1 = __byte_perm(v[2][i], v[3][i], 0x7362);
            mma16816(o[4 * i], pk[b], widen2(a0 & 0xffffu), widen2(b0 & 0xffffu));
            mma16816(o[4 * i + 1], pk[b], widen2(a0 >> 16), widen2(b0 >> 16));
            mma16816(o[4 * i + 2], pk[b], widen2(a1 & 0xffffu), widen2(b1 & 0xffffu));
            mma16816(o[4 * i + 3], pk[b], widen2(a1 >> 16), widen2(b1 >> 16));
        }
    }
}

// 4 outputs, rounded once (fp16: finite ones past 65504 are that)
PI_DEV void put4(__half* p, float4 v) {
    auto in = [](float x) { return fabsf(x) > 65504.f && fabsf(x) < INFINITY ? copysignf(65504.f, x) : x; };
    *reinterpret_cast<uint2*>(p) = make_uint2(half2_of(in(v.x), in(v.y)), half2_of(in(v.z), in(v.w)));
}
PI_DEV void put4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// The key tiles of a warp's piece.  Pages and exponents of its blocks are looked up 32 at a
// time (16 tiles), a lane each; those of the 32 behind them come while these run.
template <int DH, bool HALF>
struct Run8 {
    static constexpr int STAGES = Few8Cfg<DH, HALF>::STAGES;
    int first, tiles;            // first block (of the request, even), tiles
    int asked, taken;            // tiles asked for, and those of them that have been waited for
    int slot, ask_slot, phase;   // of the ring: next to use, next to fill, the phase of the next's copies
    int id, id_next, ex, ex_next;   // page of this lane's block (past the cache: zeros), ek * 256 + ev

    PI_DEV int page_of(const Few8Args& a, const Piece8& p, int i) const {
        if (i >= 2 * tiles || (first + i) * kBlock >= p.hi) return a.c.num_pages;
        const int page = a.table[(size_t)p.b * a.max_pages + ((first + i) >> (a.c.page_shift - 4))];
        if (page >= 0 && page < a.c.num_pages) return page;
        if ((first + i + 1) * kBlock > p.lo) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
        return a.c.num_pages;   // past the last page: the copy fills zeros
    }
    PI_DEV int exponents_of(const Few8Args& a, const Piece8& p, int i, int page) const {
        if (page >= a.c.num_pages) return 0;
        const int in_page = (first + i) & ((1 << (a.c.page_shift - 4)) - 1);
        const long long at = (((long long)page * a.c.kv_heads + p.g) << (a.c.page_shift - 4)) + in_page;
        return bounded(a.c.ke[at]) * 256 + bounded(a.c.ve[at]);
    }
    // asks for the next tile, if there is one (the lanes are done with its slot)
    PI_DEV void ask(const Few8Args& a, const Piece8& p, Few8Shared<DH, HALF>& sh, int batch) {
        if (asked >= tiles) return;
        const int i = 2 * (asked - batch);   // 0 .. 62
        const int page = __shfl_sync(FULL, i & 32 ? id_next : id, i & 31), page1 = __shfl_sync(FULL, i & 32 ? id_next : id, (i + 1) & 31);
        if ((threadIdx.x & 31) == 0) {
            Slot8<DH>& to = sh.ring[threadIdx.x >> 5][ask_slot];
            unsigned long long* const bar = &sh.full[threadIdx.x >> 5][ask_slot];
            const int pos = ((first + 2 * asked) & ((1 << (a.c.page_shift - 4)) - 1)) * kBlock;
            bar_arrive_expect_tx(bar, 2 * kTile * DH);
            tma_load_5d(to.bytes, &a.kmap, 0, pos, p.g, page, 0, bar);
            if (!a.both) tma_load_5d(to.bytes + a.v_at, &a.vmap, 0, pos, p.g, page, 0, bar);
            if (a.c.page_shift == 4) {
                tma_load_5d(to.bytes + a.block_step, &a.kmap, 0, 0, p.g, page1, 0, bar);
                if (!a.both) tma_load_5d(to.bytes + a.v_at + a.block_step, &a.vmap, 0, 0, p.g, page1, 0, bar);
            }
        }
        ++asked;
        if (++ask_slot == STAGES) ask_slot = 0;
    }
    // waits (bounded) for the next tile in the ring; false: gave up
    PI_DEV bool take(Few8Shared<DH, HALF>& sh, const Ctl& ctl, const Slot8<DH>** at) {
        const int warp = threadIdx.x >> 5;
        *at = &sh.ring[warp][slot];
        unsigned long long* const bar = &sh.full[warp][slot];
        if (!__all_sync(FULL, bar_test(bar, phase)) && !__all_sync(FULL, bar_wait(bar, phase, ctl))) return false;
        ++taken;
        if (++slot == STAGES) {
            slot = 0;
            phase ^= 1;
        }
        return true;
    }
    // every copy asked for has landed before the block may exit
    PI_DEV void drain(Few8Shared<DH, HALF>& sh) {
        for (; taken < asked; ++taken) {
            bar_drain(&sh.full[threadIdx.x >> 5][slot], phase, kDrainTimeoutNs);
            if (++slot == STAGES) {
                slot = 0;
                phase ^= 1;
            }
        }
    }
    PI_DEV void start(const Few8Args& a, const Piece8& p, Few8Shared<DH, HALF>& sh) {
        const int lane = threadIdx.x & 31;
        first = 2 * (p.lo / kTile + p.from);
        tiles = p.lo < p.hi ? p.nt : 0;
        asked = taken = 0;
        id = page_of(a, p, lane);
        id_next = page_of(a, p, 32 + lane);
        for (int i = 0; i < STAGES; ++i) ask(a, p, sh, 0);
        ex = exponents_of(a, p, lane, id);
        ex_next = 0;
    }
};

// 1 / l (a sum of 0: the row sees nothing; one that is not a number stays one), and log sum e^a
PI_DEV float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
PI_DEV float log_sum(float m, float l) { return l == 0.f ? -INFINITY : (m - kLift + log2f(l)) * kLn2; }

// ------------------------------------------------ pages of long requests in 16 bits
//
// A unit is one KV head of one page that a request of many rows sees; a warp takes a
// contiguous range of units, once it is done with the items of few rows.  Page p of the
// cache is page p of the copy.  (In a launch of its own: a prompt of 1999 tokens 41.9 us a
// call, so 38.8.)

// pages of a request that are widened: first and how many
PI_DEV int seen_pages(const Few8Args& a, const Request8& r, int* first) {
    const int hi = r.first + r.n, lo = a.window > 0 ? max(0, r.first - a.window + 1) : 0;
    *first = lo >> a.c.page_shift;
    if (r.n <= a.few || hi <= lo) return 0;
    return ((hi + (1 << a.c.page_shift) - 1) >> a.c.page_shift) - *first;
}

// 8 codes times `scale` in 16 bits (fp16: finite ones past 65504 are that)
PI_DEV void put_wide(__half* p, const uint2& c, float scale) {
    const uint32_t w[2] = {c.x, c.y};
    uint32_t o[4];
    auto in = [](float x) { return fabsf(x) > 65504.f ? copysignf(65504.f, x) : x; };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = values2((w[i / 2] >> (16 * (i & 1))) & 0xffffu);
        o[i] = half2_of(in(u.x * scale), in(u.y * scale));
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}
PI_DEV void put_wide(__nv_bfloat16* p, const uint2& c, float scale) {
    const uint32_t w[2] = {c.x, c.y};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = values2((w[i / 2] >> (16 * (i & 1))) & 0xffffu);
        const __nv_bfloat162 y = __floats2bfloat162_rn(u.x * scale, u.y * scale);
        o[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename T, int DH, int THREADS>
PI_DEV void widen_pages(const Few8Args& a, long long* scratch, long long* before) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int per = (a.batch + THREADS - 1) / THREADS, b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    long long own = 0, U = 0;
    bool bad = false;
    int first;
    for (int b = b0; b < b1; ++b) own += (long long)a.c.kv_heads * seen_pages(a, request8(a, b, &bad), &first);
    before[tid] = scan_before<THREADS>(own, scratch, &U);
    __syncthreads();
    const long long warps = (long long)gridDim.x * (THREADS / 32), w = (long long)blockIdx.x * (THREADS / 32) + (tid >> 5);
    const long long u0 = quotient(U * w, warps), u1 = quotient(U * (w + 1), warps);
    if (u0 >= u1) return;
    // where the range starts: the last thread whose requests' units start at or before u0, then its requests
    int t = 0;
    for (int d = 256; d > 0; d >>= 1)
        if (t + d < THREADS && before[t + d] <= u0) t += d;
    int b = min(t * per, a.batch), count = 0;
    long long left = u0 - before[t];
    for (; b < a.batch; ++b) {
        count = seen_pages(a, request8(a, b, &bad), &first);
        if (left < (long long)a.c.kv_heads * count) break;
        left -= (long long)a.c.kv_heads * count;
    }
    if (b >= a.batch) return;   // (the lengths changed under the kernel)
    int page = (int)quotient(left, a.c.kv_heads), head = (int)(left - (long long)page * a.c.kv_heads);
    constexpr int POS = DH / 8, N = 16;                // pieces of 8 codes of a position; of a lane in flight
    const int chunks = POS << a.c.page_shift;          // of a head
    int id = -1, at = -1;        // page of the cache, and the column it was looked up for
    for (long long u = u0; u < u1; ++u) {
        const int col = first + page;
        if (col != at) {
            id = col < a.max_pages ? a.table[(size_t)b * a.max_pages + col] : -1;
            at = col;
        }
        if (id >= 0 && id < a.c.num_pages) {   // (others read as zeros and are reported by the attention)
            const long long src = id * a.c.page_stride + head * a.c.head_stride;
            const long long ex = ((long long)id * a.c.kv_heads + head) << (a.c.page_shift - 4);
            const long long dst = ((long long)id * a.c.kv_heads + head) * ((long long)DH << a.c.page_shift);
            for (int i0 = lane; i0 < 2 * chunks; i0 += N * 32) {
                uint2 y[N];
                int e[N];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int i = i0 + 32 * j, x = i & (chunks - 1), pos = x / POS, c = x % POS;
                    if (i >= 2 * chunks) break;
                    const bool values = i >= chunks;
                    y[j] = ld_stream8((values ? a.c.v : a.c.k) + src + pos * a.c.token_stride + c * 8);
                    e[j] = (values ? a.c.ve : a.c.ke)[ex + pos / kBlock];
                }
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int i = i0 + 32 * j;
                    if (i >= 2 * chunks) break;
                    put_wide(static_cast<T*>(i >= chunks ? a.wide_v : a.wide_k) + dst + (long long)(i & (chunks - 1)) * 8, y[j], pow2(bounded(e[j])));
                }
            }
        }
        if (++head == a.c.kv_heads) {
            head = 0;
            if (++page >= count) {
                page = 0;
                at = -1;
                do {
                    if (++b >= a.batch) return;
                    count = seen_pages(a, request8(a, b, &bad), &first);
                } while (count == 0);
            }
        }
    }
}

// ------------------------------------------------ items of few rows
template <typename T, int DH, bool HALF>
PI_DEV void few_items(const Few8Args& a, Few8Shared<DH, HALF>& sh) {
    using C = Few8Cfg<DH, HALF>;
    constexpr int KC = Slot8<DH>::KC, OC = DH / 8, CHUNKS = C::CHUNKS, RH = HALF ? 1 : 2, STAGES = C::STAGES;
    constexpr int W = C::WARPS, THREADS = C::THREADS;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q4 = lane & 3, r8 = lane >> 2;

    if (lane == 0) {
        for (int i = 0; i < STAGES; ++i) bar_init(&sh.full[warp][i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) {
        sh.abort_flag = 0;
        tma_prefetch_map(&a.kmap);
    }

    // units of all requests, and where the warps' ranges start
    const int per = (a.batch + THREADS - 1) / THREADS, b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    long long own = 0, U = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) own += a.c.kv_heads * request_units(a, request8(a, b, &bad));
    if (bad && blockIdx.x == 0) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
    if (tid < W) sh.cut[tid][0].nt = sh.cut[tid][1].nt = 0;
    if (tid < 2) sh.open[tid].nt = 0;
    const long long pre = scan_before<THREADS>(own, sh.scratch, &U);
    const int G = (int)min((long long)gridDim.x, max(U / kMinUnits, U > 0 ? 1ll : 0ll));
    if ((int)blockIdx.x >= G) return;
    const long long u0 = quotient(U * blockIdx.x, G), u1 = quotient(U * (blockIdx.x + 1), G);
    sh.before[tid] = pre;
    __syncthreads();
    if (lane == 0) {
        const long long v0 = u0 + (u1 - u0) * warp / W, v1 = u0 + (u1 - u0) * (warp + 1) / W;
        Walk8 walk{};
        if (v0 < v1) {
            // the last thread whose requests' units start at or before v0
            int t = 0;
            for (int d = 256; d > 0; d >>= 1)
                if (t + d < THREADS && sh.before[t + d] <= v0) t += d;
            long long left = v0 - sh.before[t];
            const int e = min(min((t + 1) * per, a.batch), a.batch);
            for (int b = min(t * per, a.batch); b < e; ++b) {
                const Request8 r = request8(a, b, &bad);
                const long long u = request_units(a, r);
                if (left >= a.c.kv_heads * u) {
                    left -= a.c.kv_heads * u;
                    continue;
                }
                const int g = (int)quotient(left, u);
                left -= g * u;
                int rt = 0, lo, hi;
                for (;; ++rt) {
                    const int cost = kLead + item_range(a, r, rt, &lo, &hi);
                    if (left < cost) break;
                    left -= cost;
                }
                walk = Walk8{r, v0, v1, b, g, rt, (int)left};
                break;
            }
        }
        sh.walk[warp] = walk;
        sh.piece[warp][0] = sh.walk[warp].next(a);
    }
    __syncwarp();
    const Ctl ctl{a.status, a.timeout_ns, &sh.abort_flag};
    Run8<DH, HALF> run;
    run.slot = run.ask_slot = run.phase = 0;
    run.start(a, sh.piece[warp][0], sh);
    if (lane == 0) sh.piece[warp][1] = sh.walk[warp].next(a);
    __syncwarp();
    bool ok = true;

    for (int n = 0;; ++n) {
        const Piece8 p = sh.piece[warp][n & 1];
        if (p.nt == 0) break;

        // queries, and what the rows see (rows of nothing: all, so that they do not ask for masking)
        uint32_t q[DH / 16][4];
        Rows8 w;
        int lo_most = 0, hi_least = 0x7fffffff;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w.lo[h] = 0;
            w.hi[h] = 0x7fffffff;
            w.c[h] = a.scale / kLn2;
            w.m[h] = -INFINITY;
            w.l[h] = 0.f;
            if (h >= RH) {
#pragma unroll
                for (int i = 0; i < DH / 16; ++i) q[i][h] = q[i][2 + h] = 0u;
                continue;
            }
            const int tr = r8 + 8 * h, row = p.rt * a.rows + tr;
            uint32_t raw[DH / 8];
#pragma unroll
            for (int i = 0; i < DH / 8; ++i) raw[i] = 0u;
            if (tr < p.rows) {
                const int tok = row / a.group, head = p.g * a.group + row - tok * a.group, pos = p.first + tok;
                w.hi[h] = max(pos + 1, 0);
                w.lo[h] = a.window > 0 ? min(max(0, pos - a.window + 1), w.hi[h]) : 0;
                const T* const src = static_cast<const T*>(a.q) + (long long)(p.cu + tok) * a.q_stride + (long long)head * DH + q4 * 16;
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 v = *reinterpret_cast<const uint4*>(src + 64 * c + 8 * i);
                        raw[8 * c + 4 * i] = v.x;
                        raw[8 * c + 4 * i + 1] = v.y;
                        raw[8 * c + 4 * i + 2] = v.z;
                        raw[8 * c + 4 * i + 3] = v.w;
                    }
            }
            lo_most = max(lo_most, w.lo[h]);
            hi_least = min(hi_least, w.hi[h]);
            float f = 1.f;
            if (!std::is_same<T, __half>::value) {
                uint32_t most = 0;   // bits of the row's largest finite magnitude (bf16)
#pragma unroll
                for (int i = 0; i < DH / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t v = (raw[i] >> (16 * e)) & 0x7fffu;
                        if (v < 0x7f80u) most = max(most, v);
                    }
                most = max(most, __shfl_xor_sync(FULL, most, 1));
                most = max(most, __shfl_xor_sync(FULL, most, 2));
                // its exponent to 14 (of 2^-113 or less: as far as a power of two goes)
                const int up = min(14 + 127 - (int)(most >> 7), 126);
                f = pow2(up);
                w.c[h] = w.c[h] * pow2(-up);
            }
#pragma unroll
            for (int i = 0; i < DH / 16; ++i) {
                q[i][h] = query2(raw[2 * i], f, T());
                q[i][2 + h] = query2(raw[2 * i + 1], f, T());
            }
        }
        lo_most = __reduce_max_sync(FULL, lo_most);
        hi_least = __reduce_min_sync(FULL, hi_least);
        float o[OC][4];
#pragma unroll
        for (int i = 0; i < OC; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

        for (int i = 0; i < run.tiles; ++i) {
            const int batch = i & ~15, x = 2 * (i & 15);
            if (x == 0 && i > 0) {
                run.id = run.id_next;
                run.ex = run.ex_next;
                run.id_next = run.page_of(a, p, 2 * i + 32 + lane);
            }
            if (x == 16) run.ex_next = run.exponents_of(a, p, 2 * batch + 32 + lane, run.id_next);
            const int e0 = __shfl_sync(FULL, run.ex, x), e1 = __shfl_sync(FULL, run.ex, x + 1);
            const int v0 = (int)(signed char)(e0 & 255), v1 = (int)(signed char)(e1 & 255);
            const int kb = (run.first + 2 * i) * kBlock, ek[2] = {(e0 - v0) >> 8, (e1 - v1) >> 8}, ev[2] = {v0, v1};
            const Slot8<DH>* at;
            if (!(ok = run.take(sh, ctl, &at))) break;
            step<DH, HALF>(a, p, *at, ek, ev, kb, kb < lo_most || kb + kTile > hi_least, q, w, o);
            __syncwarp();
            run.ask(a, p, sh, batch);
        }
        if (!ok) {
            run.drain(sh);
            break;
        }

        // the next piece's first blocks are on their way while this one is put away
        run.start(a, sh.piece[warp][(n + 1) & 1], sh);
        __syncwarp();   // (every lane has its copy of this piece)
        if (lane == 0) sh.piece[warp][n & 1] = sh.walk[warp].next(a);   // the piece after the next
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            w.l[h] += __shfl_xor_sync(FULL, w.l[h], 1);
            w.l[h] += __shfl_xor_sync(FULL, w.l[h], 2);
        }
        if (p.nt == p.all) {
#pragma unroll
            for (int h = 0; h < RH; ++h) {
                const int tr = r8 + 8 * h, row = p.rt * a.rows + tr;
                if (tr >= p.rows) continue;
                const int tok = row / a.group, head = p.g * a.group + row - tok * a.group;
                T* const dst = static_cast<T*>(a.out) + (long long)(p.cu + tok) * a.o_stride + (long long)head * DH + 2 * q4 * (DH / 8);
                const float f = inverse(w.l[h]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < OC; i += 4)
                        put4(dst + e * (DH / 8) + i, make_float4(o[i][2 * h + e] * f, o[i + 1][2 * h + e] * f, o[i + 2][2 * h + e] * f, o[i + 3][2 * h + e] * f));
                if (a.lse != nullptr && q4 == 0) a.lse[(long long)(p.cu + tok) * a.heads + head] = log_sum(w.m[h], w.l[h]);
            }
        } else {
            const int slot = p.from == 0;   // a warp begins at most one piece that it does not end
            // the last piece's sums stay in the ring, which holds nothing any more
            static_assert(CHUNKS * 32 * sizeof(float4) <= sizeof(sh.ring[0]), "a ring holds a piece's sums");
            // (an item of no keys asks for nothing either, but others may follow it)
            const bool stays = sh.piece[warp][(n + 1) & 1].nt == 0;
            float4* const po = (stays ? reinterpret_cast<float4*>(&sh.ring[warp][0]) : a.warp_o + (((size_t)blockIdx.x * W + warp) * 2 + slot) * CHUNKS * 32) + lane;
#pragma unroll
            for (int h = 0; h < RH; ++h) {
                if (q4 == 0) sh.ml[warp][slot][r8 + 8 * h] = make_float2(w.m[h], w.l[h]);
                // chunk (2 h + e) DH / 32 + i: elements 4 i .. of this lane's run e, of row r8 + 8 h
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < DH / 32; ++i)
                        po[((2 * h + e) * (DH / 32) + i) * 32] = make_float4(o[4 * i][2 * h + e], o[4 * i + 1][2 * h + e], o[4 * i + 2][2 * h + e], o[4 * i + 3][2 * h + e]);
            }
            if (lane == 0) {
                sh.cut[warp][slot] = p;
                sh.stays[warp][slot] = stays;
            }
        }
        __syncwarp();
    }

    // ---- items that warps of this block share: each of them takes its share of the chunks
    auto write = [&](const Piece8& p, int c, float4 v, const float (&inv)[2]) {
        const int h = c / (DH / 16), e = c / (DH / 32) % 2, tr = r8 + 8 * h, row = p.rt * a.rows + tr;
        if (tr >= p.rows) return;
        const int tok = row / a.group, head = p.g * a.group + row - tok * a.group;
        const float f = inv[h];
        put4(static_cast<T*>(a.out) + (long long)(p.cu + tok) * a.o_stride + (long long)head * DH + (2 * q4 + e) * (DH / 8) + c % (DH / 32) * 4,
             make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
    };
    auto write_lse = [&](const Piece8& p, const float (&m)[2], const float (&l)[2]) {
        if (a.lse == nullptr || q4 != 0) return;
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            const int tr = r8 + 8 * h, row = p.rt * a.rows + tr;
            if (tr >= p.rows) continue;
            const int tok = row / a.group, head = p.g * a.group + row - tok * a.group;
            a.lse[(long long)(p.cu + tok) * a.heads + head] = log_sum(m[h], l[h]);
        }
    };
    __syncthreads();
    if (*(volatile int*)&sh.abort_flag) return;
    const Piece8* const cuts = &sh.cut[0][0];
    for (int slot = 0; slot < 2; ++slot) {
        const Piece8& p = sh.cut[warp][slot];
        if (p.nt == 0) continue;
        const unsigned who = __ballot_sync(FULL, lane < 2 * W && cuts[lane].nt > 0 && cuts[lane].i0 == p.i0);   // in the order of the keys
        const int k = __popc(who), mine = __popc(who & ((1u << (2 * warp + slot)) - 1u));
        const Piece8 &first = cuts[__ffs(who) - 1], &last = cuts[31 - __clz(who)];
        const bool begun = first.from == 0, whole = begun && last.from + last.nt == last.all;
        float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f}, use[2] = {0.f, 0.f};
        for (unsigned x = who; x != 0; x &= x - 1)
#pragma unroll
            for (int h = 0; h < RH; ++h) M[h] = fmaxf(M[h], (&sh.ml[0][0][0])[(__ffs(x) - 1) * kRows + r8 + 8 * h].x);
#pragma unroll
        for (int h = 0; h < RH; ++h) use[h] = M[h] == -INFINITY ? 0.f : M[h];
        const float4* const po = a.warp_o + (size_t)blockIdx.x * W * 2 * CHUNKS * 32 + lane;
        const size_t at = (size_t)blockIdx.x * 2 + begun;
        for (unsigned x = who; x != 0; x &= x - 1)
#pragma unroll
            for (int h = 0; h < RH; ++h) {
                const float2 y = (&sh.ml[0][0][0])[(__ffs(x) - 1) * kRows + r8 + 8 * h];
                L[h] = fmaf(y.y, ex2(y.x - use[h]), L[h]);
            }
        const float inv[2] = {inverse(L[0]), inverse(L[1])};
        for (int c = mine; c < CHUNKS; c += k) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (unsigned x = who; x != 0;) {   // four parts at a time (past the end: the last once more, left out below)
                float4 z[4];
                float f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int part = x != 0 ? __ffs(x) - 1 : 31 - __clz(who);
                    z[i] = sh.stays[part >> 1][part & 1] ? reinterpret_cast<const float4*>(&sh.ring[part >> 1][0])[c * 32 + lane]
                                                         : __ldcg(po + ((size_t)part * CHUNKS + c) * 32);
                    f[i] = x != 0 ? ex2((&sh.ml[0][0][0])[part * kRows + r8 + (HALF || c < DH / 16 ? 0 : 8)].x - use[HALF || c < DH / 16 ? 0 : 1]) : -1.f;
                    x &= x - 1;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!(f[i] < 0.f)) v = make_float4(fmaf(z[i].x, f[i], v.x), fmaf(z[i].y, f[i], v.y), fmaf(z[i].z, f[i], v.z), fmaf(z[i].w, f[i], v.w));
            }
            if (whole) write(p, c, v, inv);
            else a.part_o[(at * CHUNKS + c) * 32 + lane] = v;
        }
        if (mine == 0) {
            if (whole) {
                write_lse(p, M, L);
            } else {
                if (q4 == 0)
#pragma unroll
                    for (int h = 0; h < RH; ++h) reinterpret_cast<float2*>(a.part_ml)[at * kRows + r8 + 8 * h] = make_float2(M[h], L[h]);
                if (lane == 0) {
                    // blocks that hold its first and its last tile, in range whatever the lengths become under the kernel
                    const long long f = quotient((p.i0 + kLead + 1) * G - 1, U), l = quotient((p.i0 + kLead + p.all) * G - 1, U);
                    const int block0 = (int)min(max(f, 0ll), (long long)G - 1);
                    sh.parts[begun] = (int)min(max(l - f + 1, 1ll), (long long)(G - block0));
                    sh.open[begun] = p;
                    sh.open[begun].from = block0;
                }
            }
        }
    }
    // the block's stores happen before thread 0's arrivals (barrier, then release), the other
    // blocks' before what any thread reads after them (acquire, then barrier)
    __syncthreads();
    if (sh.open[0].nt == 0 && sh.open[1].nt == 0) return;
    if (lane == 0 && warp < 2 && sh.open[warp].nt != 0) {
        int* const count = a.counters + sh.open[warp].from;
        sh.seen[warp] = arrive_gpu(count);
        if (sh.seen[warp] == sh.parts[warp] - 1) *count = 0;
    }
    __syncthreads();
    for (int x = 0; x < 2; ++x) {
        if (sh.open[x].nt == 0 || sh.seen[x] != sh.parts[x] - 1) continue;
        const Piece8& p = sh.open[x];
        const int parts = sh.parts[x], block0 = p.from;
        constexpr int SHARE = (CHUNKS + W - 1) / W;   // chunks of a warp (some have none)
        constexpr int AT_ONCE = 8 / SHARE;            // parts whose loads are in flight together
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float4 v[SHARE];
#pragma unroll
        for (int i = 0; i < SHARE; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < parts; k += AT_ONCE) {
            float4 z[AT_ONCE][SHARE];
            float2 y[AT_ONCE][RH];
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {   // past the end: the last one once more, left out below
                // partial of block block0 + k: its second place (k = 0, where the item begins) or its first
                const int part = min(k + j, parts - 1);
                const size_t at = (size_t)(block0 + part) * 2 + (part == 0 ? 1 : 0);
#pragma unroll
                for (int h = 0; h < RH; ++h) y[j][h] = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + at * kRows + r8 + 8 * h);
#pragma unroll
                for (int i = 0; i < SHARE; ++i) z[j][i] = __ldcg(a.part_o + (at * CHUNKS + min(warp + i * W, CHUNKS - 1)) * 32 + lane);
            }
            float use[2];
#pragma unroll
            for (int h = 0; h < RH; ++h) {
                float top = m[h];
#pragma unroll
                for (int j = 0; j < AT_ONCE; ++j) top = fmaxf(top, y[j][h].x);
                use[h] = top == -INFINITY ? 0.f : top;
                const float f = ex2(m[h] - use[h]);   // of what the parts before these have summed
                m[h] = top;
                l[h] *= f;
#pragma unroll
                for (int i = 0; i < SHARE; ++i)
                    if ((!HALF && warp + i * W >= DH / 16) == (h == 1)) v[i] = make_float4(v[i].x * f, v[i].y * f, v[i].z * f, v[i].w * f);
            }
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
                if (k + j >= parts) break;
                float f[2] = {0.f, 0.f};
#pragma unroll
                for (int h = 0; h < RH; ++h) {
                    f[h] = ex2(y[j][h].x - use[h]);
                    l[h] = fmaf(y[j][h].y, f[h], l[h]);
                }
#pragma unroll
                for (int i = 0; i < SHARE; ++i) {
                    const float g = HALF || warp + i * W < DH / 16 ? f[0] : f[1];
                    v[i] = make_float4(fmaf(z[j][i].x, g, v[i].x), fmaf(z[j][i].y, g, v[i].y), fmaf(z[j][i].z, g, v[i].z), fmaf(z[j][i].w, g, v[i].w));
                }
            }
        }
        const float inv[2] = {inverse(l[0]), inverse(l[1])};
#pragma unroll
        for (int i = 0; i < SHARE; ++i)
            if (warp + i * W < CHUNKS) write(p, warp + i * W, v[i], inv);
        if (warp == 0) write_lse(p, m, l);
    }
}

template <typename T, int DH, bool HALF>
__global__ void __launch_bounds__(Few8Cfg<DH, HALF>::THREADS, 1) k_attn8_few(const __grid_constant__ Few8Args a) {
    pdl_entry();
    extern __shared__ __align__(1024) unsigned char few_smem[];
    Few8Shared<DH, HALF>& sh = *reinterpret_cast<Few8Shared<DH, HALF>*>(few_smem);
    if ((su32(few_smem) & 1023u) != 0) {   // the copies' swizzle needs it; the whole block leaves
        if (threadIdx.x == 0) atomicExch(a.status, (int)PI_ERR_UNSUPPORTED);
        return;
    }
    few_items<T, DH, HALF>(a, sh);
    if (a.wide_k == nullptr) return;
    __syncthreads();
    widen_pages<T, DH, Few8Cfg<DH, HALF>::THREADS>(a, sh.scratch, sh.before);
}

// ------------------------------------------------ host

bool paged8_ok(const pi_paged_desc& d, const pi_page8_desc& c) {
    return page8_desc_ok(c) && d.heads >= 1 && d.heads <= 1024 && d.heads % c.kv_heads == 0 &&
           d.heads / c.kv_heads <= 128 && d.batch >= 1 && d.batch <= 4096 && d.max_tokens >= 0 &&
           d.max_tokens <= (1 << 24) && d.max_new >= 1 && (d.max_tokens == 0 || d.max_new <= d.max_tokens) &&
           d.max_pages >= 1 && (long long)d.max_pages * c.page_size <= (1ll << 30) && d.window >= 0 &&
           d.scale >= 0.f && isfinite(d.scale);
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

bool codes_map(CUtensorMap* m, const void* base, const pi_page8_desc& c, int arrays, unsigned long long apart) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[5] = {(cuuint64_t)c.head_dim / 4, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads, (cuuint64_t)c.num_pages,
                                (cuuint64_t)arrays};
    const cuuint64_t strides[4] = {(cuuint64_t)c.token_stride, (cuuint64_t)c.head_stride, (cuuint64_t)c.page_stride, apart};
    const cuuint32_t box[5] = {(cuuint32_t)c.head_dim / 4, (cuuint32_t)std::min(c.page_size, kTile), 1u, 1u, (cuuint32_t)arrays};
    const cuuint32_t es[5] = {1u, 1u, 1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 5, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Both arrays as one tensor, the distance of their addresses a stride (16 .. 2^40 bytes), or one each.
bool codes_maps(Few8Args* a, const void* k, const void* v, const pi_page8_desc& c) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(k), y = reinterpret_cast<uintptr_t>(v), apart = x < y ? y - x : x - y;
    const int block = kBlock * c.head_dim, box = std::min(c.page_size, kTile) * c.head_dim;   // bytes of an array
    a->both = apart > 0 && apart < (1ull << 40);
    const bool keys_first = !a->both || x < y;
    // boxes of 32 positions: 32 rows of one array, then of the other; of 16: a block of one, of the other, twice
    a->k_at = keys_first ? 0 : box;
    a->v_at = keys_first ? box : 0;
    a->block_step = c.page_size < kTile ? 2 * block : block;
    return a->both ? codes_map(&a->kmap, keys_first ? k : v, c, 2, apart)
                   : codes_map(&a->kmap, k, c, 1, 16) && codes_map(&a->vmap, v, c, 1, 16);
}

// Whether a step may hold requests for the 16-bit kernel, and the tokens up to which one goes
// through k_attn8_few: 64 rows (or a token) where all requests are that short (24 sequences
// with 64 rows each: 113 us so, 161 over widened pages; with 128 rows 194 and 164), else 8, so
// that decode steps beside prompts take the 8-row items (16 sequences that decode or take
// 100-700 tokens, a head to a KV head: 173 us so, 184 with items of 16 rows for up to 64).
//   The one border stands for two things, the height of the items and who goes over widened
// pages, and where requests of a few tokens stand beside a prompt it is low: their caches are
// widened for 9-64 rows.  24 sequences with 1, 2, 5 and 8 tokens behind 200-6000 beside a chunk
// of 512 (64 query and 8 KV heads): 122, 207, 206 and 208 us so; 126, 129, 174 and 196 with 64
// rows and items of 16; 122, 139, 204 and 267 with 64 rows and items of 8.  16 sequences with 8,
// 16, 40 and 64 tokens beside one (32 heads): 185, 418, 424 and 426 so, 196, 191, 300 and 393, 184,
// 244, 370 and 574.  What gives both its gains is a height of the items by request.
bool has_long(int max_new, int group) { return max_new > std::max(1, kFewRows / group); }
int few_tokens(int max_new, int group) { return std::max(1, (has_long(max_new, group) ? 8 : kFewRows) / group); }

// The copy's description: [pages, heads, positions, elements].
pi_page_desc wide_desc(const pi_page8_desc& c, int dtype) {
    return pi_page_desc{c.kv_heads, c.head_dim, c.page_size, c.num_pages, dtype, (long long)c.kv_heads * c.page_size * c.head_dim,
                        (long long)c.page_size * c.head_dim, c.head_dim};
}

// Workspace: the arrival counters of both kernels first, in the same place for every descriptor
// (they have to be zeros between calls, and what lies behind them goes by head width, max_new
// and pages); then the partials of two items per block and per warp; for steps with long requests
// the 16-bit attention's workspace and the copies of the caches' pages.
struct Layout8 {
    size_t arrivals, ml, o, warps, wide, wide_bytes, k, v, total;
    Layout8(const pi_paged_desc& d, const pi_page8_desc& c, int sms) {
        auto up = [](size_t v) { return (v + 255) / 256 * 256; };
        const size_t blocks = std::max(1, sms), item = (size_t)kRows * c.head_dim * sizeof(float);
        arrivals = up(blocks * sizeof(int));
        ml = up(arrivals + blocks * kPagedArrivals * sizeof(int));
        o = up(ml + blocks * 2 * kRows * sizeof(float2));
        warps = up(o + blocks * 2 * item);
        wide = up(warps + blocks * kMostWarps * 2 * item);
        k = v = total = wide;
        wide_bytes = 0;
        if (has_long(d.max_new, d.heads / c.kv_heads)) {
            const pi_page_desc w = wide_desc(c, PI_T_F16);
            wide_bytes = pi_paged_workspace_bytes(&d, &w);
            const size_t pages = up((size_t)c.num_pages * w.page_stride * 2);
            k = up(wide + wide_bytes);
            v = k + pages;
            total = v + pages;
        }
    }
};

template <typename T, int DH, bool HALF>
cudaError_t launch_few(const Few8Args& a, int sms, cudaStream_t s) {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr int smem = (int)sizeof(Few8Shared<DH, HALF>);
    static_assert(smem <= 232448, "shared memory of a block");
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            e = cudaFuncSetAttribute(k_attn8_few<T, DH, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    return launch_pdl(k_attn8_few<T, DH, HALF>, sms, Few8Cfg<DH, HALF>::THREADS, smem, s, a);
}
template <typename T>
cudaError_t launch_few(const Few8Args& a, int dh, bool half, int sms, cudaStream_t s) {
    if (dh == 128) return half ? launch_few<T, 128, true>(a, sms, s) : launch_few<T, 128, false>(a, sms, s);
    return half ? launch_few<T, 64, true>(a, sms, s) : launch_few<T, 64, false>(a, sms, s);
}

}  // namespace
}  // namespace pi

using namespace pi;

extern "C" {

size_t pi_paged8_workspace_bytes(const pi_paged_desc* desc, const pi_page8_desc* cache) {
    if (!desc || !cache || !paged8_ok(*desc, *cache)) return 0;
    // without a device (descriptors checked on a host), as for one SM
    return Layout8(*desc, *cache, sm_count()).total;
}

pi_status pi_paged_attn8(const pi_paged_desc* desc, const pi_page8_desc* cache, int dtype, const void* q, long long q_stride,
                         const void* kcache, const void* vcache, const int8_t* kexp, const int8_t* vexp,
                         const int32_t* block_table, const int32_t* cu_new, const int32_t* kv_len, void* out,
                         long long out_stride, float* lse, void* workspace, size_t ws_bytes, void* stream) {
    if (!desc || !cache || !paged8_ok(*desc, *cache) || (dtype != PI_T_F16 && dtype != PI_T_BF16)) return PI_ERR_INVALID_ARG;
    const long long width = (long long)desc->heads * cache->head_dim;
    if (q_stride % 8 != 0 || q_stride < width || out_stride % 8 != 0 || out_stride < width) return PI_ERR_INVALID_ARG;
    if (desc->max_tokens == 0) return PI_OK;
    auto aligned = [](const void* p, size_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    if (!aligned(q, 16) || !aligned(kcache, 16) || !aligned(vcache, 16) || !kexp || !vexp || !aligned(out, 16) ||
        !aligned(block_table, 4) || !aligned(cu_new, 4) || !aligned(kv_len, 4) || (lse && !aligned(lse, 4)))
        return PI_ERR_INVALID_ARG;
    const int sms = sm_count();
    const Layout8 lay(*desc, *cache, sms);
    if (!aligned(workspace, 16) || ws_bytes < lay.total) return PI_ERR_WORKSPACE;
    // queries are read while other rows' outputs are written
    if (rows_overlap(q, 2 * q_stride, 2 * width, out, 2 * out_stride, 2 * width, desc->max_tokens)) return PI_ERR_INVALID_ARG;
    char* const ws = static_cast<char*>(workspace);
    Few8Args a{};
    a.c = Cache8{static_cast<const uint8_t*>(kcache), static_cast<const uint8_t*>(vcache), kexp, vexp, cache->page_stride,
                 cache->head_stride, cache->token_stride, cache->kv_heads, __builtin_ctz((unsigned)cache->page_size),
                 cache->num_pages};
    a.q = q;
    a.table = block_table;
    a.cu = cu_new;
    a.kv = kv_len;
    a.out = out;
    a.lse = lse;
    a.q_stride = q_stride;
    a.o_stride = out_stride;
    a.heads = desc->heads;
    a.batch = desc->batch;
    a.max_tokens = desc->max_tokens;
    a.max_new = desc->max_new;
    a.max_pages = desc->max_pages;
    // a window of all positions a row can hold, or more, is none; below that,
    // sums with first positions (down to -2^24) stay far from the ends of int
    a.window = (long long)desc->window >= (long long)desc->max_pages * cache->page_size ? 0 : desc->window;
    a.group = desc->heads / cache->kv_heads;
    a.few = few_tokens(desc->max_new, a.group);
    const bool half = std::min(desc->max_new, a.few) * a.group <= 8;   // no item has more than 8 rows
    a.rows = half ? 8 : 16;
    a.scale = desc->scale > 0.f ? desc->scale : 1.0f / sqrtf((float)cache->head_dim);
    a.counters = reinterpret_cast<int*>(ws);
    a.part_ml = reinterpret_cast<float*>(ws + lay.ml);
    a.part_o = reinterpret_cast<float4*>(ws + lay.o);
    a.warp_o = reinterpret_cast<float4*>(ws + lay.warps);
    a.status = status_word();
    a.timeout_ns = wait_timeout_ns();
    if (sms < 1 || a.status == nullptr || !codes_maps(&a, kcache, vcache, *cache)) return PI_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f16 = dtype == PI_T_F16;
    const bool some_long = has_long(desc->max_new, a.group);
    if (some_long) {
        a.wide_k = ws + lay.k;
        a.wide_v = ws + lay.v;
    }
    const cudaError_t e = f16 ? launch_few<__half>(a, cache->head_dim, half, sms, s)
                              : launch_few<__nv_bfloat16>(a, cache->head_dim, half, sms, s);
    if (e != cudaSuccess) return PI_ERR_CUDA;
    if (!some_long) return PI_OK;
    const pi_page_desc wide = wide_desc(*cache, dtype);
    return paged_attn(desc, &wide, q, q_stride, a.wide_k, a.wide_v, block_table, cu_new, kv_len, out, out_stride, lse, ws + lay.wide,
                      lay.wide_bytes, reinterpret_cast<int*>(ws + lay.arrivals), a.few, stream);
}

}  // extern "C"
