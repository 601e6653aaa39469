// pi_paged8_attn.cu -- causal attention of new tokens over the 8-bit paged cache.
//
// Requests of few rows (tokens x query heads of a KV head; decode steps among
// them) are bound by the bytes of codes, and go through k_attn8_few.  Requests
// of many rows are bound by products: the pages that they see are widened to 16
// bits in the workspace once (k_widen8), and the 16-bit cache's kernel takes
// them from there on the tcgen05 tensor cores.  A step may hold both.
//
// k_attn8_few: an item is up to 16 rows of one request and KV head (row = token *
// group + head in the group).  A warp takes 16 keys at a time, one block of the
// cache, through a ring of its own in shared memory, three steps ahead:
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
// and keys, or values and outputs, agree, so a lane takes 16 bytes in a row.
//
// Work split: the (item x tile of 64 keys) space is cut into equal contiguous
// ranges per block, whatever the lengths; the four warps of a block share a
// piece's keys.  An item cut by a border leaves unnormalised partials (m, l, O)
// in the workspace, and the block that arrives last adds them in block order
// (the order is fixed, who does it is not: same bits).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "pi_common.cuh"
#include "pi_e4m3.cuh"
#include "pi_internal.h"

namespace pi {
namespace {

using namespace e4m3;

constexpr int kRows = 16;            // rows of an item
constexpr int kFewRows = 64;         // rows of a request up to which it goes through k_attn8_few (or one token's)
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16 * kWarps;   // keys of a unit of the work split
constexpr int kLead = 2;             // units that an item counts besides its tiles
constexpr int kMinUnits = 2;         // units of a block at least
constexpr int kMostBlocks = 3;       // of an SM
constexpr float kLift = 7.f;         // log2 of the factor that P, l and O share
constexpr float kGrow = 8.f;         // growth (log2) of a maximum before m follows
constexpr float kLn2 = 0.69314718055994531f;

struct Few8Args {
    Cache8 c;
    const void* q;
    const int32_t *table, *cu, *kv;
    void* out;
    float* lse;
    long long q_stride, o_stride;
    int heads, batch, max_tokens, max_new, max_pages, window, group, few;
    float scale;
    int* counters;     // [blocks] arrivals at a cut item
    float* part_ml;    // [blocks][2][16][2]
    float* part_o;     // [blocks][2][chunks][32][4]
    int* status;
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
    const int t0 = rt * kRows / a.group, t1 = min(rt * kRows + kRows - 1, r.n * a.group - 1) / a.group;
    *hi = r.first + t1 + 1;
    *lo = a.window > 0 ? max(0, r.first + t0 - a.window + 1) : 0;
    if (*hi <= *lo) {
        *lo = *hi = 0;
        return 1;
    }
    return (*hi + kTile - 1) / kTile - *lo / kTile;
}
PI_DEV int row_tiles(const Few8Args& a, const Request8& r) { return r.n > a.few ? 0 : (r.n * a.group + kRows - 1) / kRows; }
PI_DEV long long request_units(const Few8Args& a, const Request8& r) {   // of one KV head
    long long u = 0;
    int lo, hi;
    for (int rt = 0; rt < row_tiles(a, r); ++rt) u += kLead + item_range(a, r, rt, &lo, &hi);
    return u;
}

// A range of key tiles of one item.
struct Piece8 {
    int nt;          // key tiles (0: end)
    int j0;          // first key tile
    int lo, hi;      // keys that some row of the item sees
    int b, g, rt;
    int rows;        // of the item
    int first, cu;   // of the request
    int block0, parts;   // blocks that hold a part of the item: the first, and how many
    int own;         // this block's partial: 1 where the item starts here
};

struct Walk8 {
    Request8 r;
    long long u, u1, U;   // unit reached, the range's end, units in all
    int G, b, g, rt, off;   // blocks with work; request, KV head, row tile and unit within the item at u

    PI_DEV Piece8 next(const Few8Args& a) {
        Piece8 p{};
        while (u < u1 && p.nt == 0) {
            int lo, hi;
            const int nt = item_range(a, r, rt, &lo, &hi);
            const long long i0 = u - off;
            const int stop = (int)min((long long)(kLead + nt), u1 - i0);
            const int from = max(off - kLead, 0), to = max(stop - kLead, 0);
            p.nt = max(to - from, 0);
            p.j0 = lo / kTile + from;
            p.lo = lo;
            p.hi = hi;
            p.b = b;
            p.g = g;
            p.rt = rt;
            p.rows = min(kRows, r.n * a.group - rt * kRows);
            p.first = r.first;
            p.cu = r.cu;
            p.parts = 1;
            p.own = from == 0;
            if (p.nt != nt) {
                // blocks that own its first and its last tile, in range whatever the lengths become under the kernel
                const long long b0 = ((i0 + kLead + 1) * G - 1) / U, b1 = ((i0 + kLead + nt) * G - 1) / U;
                p.block0 = (int)min(max(b0, 0ll), (long long)G - 1);
                p.parts = (int)min(max(b1 - b0 + 1, 1ll), (long long)(G - p.block0));
            }
            u = stop > off ? i0 + stop : u1;
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

// The codes of 16 keys, as a lane uses them.  Keys: keys 8 j + lane / 4, elements 16 q ..
// and 64 + 16 q .. (q = lane % 4).  Values: keys 2 q, 2 q + 1, 2 q + 8, 2 q + 9, elements
// (dh / 8) (lane / 4) ...  A lane copies what it uses itself, so a ring's slot is ordered
// by lane and nothing but the lane's own wait is needed before it is read.
template <int DH>
struct Slot8 {
    static constexpr int KC = DH / 64, VW = DH / 32;   // 16-byte chunks of a key, words of a value
    uint4 k[2 * KC][32];
    uint32_t v[4][32][VW];
};

template <int BYTES>
PI_DEV void copy_async(void* to, const void* from, bool there) {   // zeros where not there
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    const int n = there ? BYTES : 0;
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(at), "l"(from), "r"(n) : "memory");
}
PI_DEV void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
PI_DEV void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Asks for the codes of keys kb .. kb + 15 (page `id`, negative: zeros).
template <int DH>
PI_DEV void fetch(const Few8Args& a, Slot8<DH>& to, int id, int kb, int g) {
    const int lane = threadIdx.x & 31, q4 = lane & 3, r8 = lane >> 2;
    const bool there = id >= 0;
    const long long at = there ? id * a.c.page_stride + g * a.c.head_stride + (kb & ((1 << a.c.page_shift) - 1)) * a.c.token_stride : 0;
    const uint8_t* const k = a.c.k + at + r8 * a.c.token_stride + q4 * 16;
    const uint8_t* const v = a.c.v + at + 2 * q4 * a.c.token_stride + r8 * (DH / 8);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int c = 0; c < Slot8<DH>::KC; ++c)
            copy_async<16>(&to.k[j * Slot8<DH>::KC + c][lane], k + 8 * j * a.c.token_stride + 64 * c, there);
#pragma unroll
    for (int x = 0; x < 4; ++x) copy_async<DH / 8>(to.v[x][lane], v + ((x & 1) + 8 * (x >> 1)) * a.c.token_stride, there);
}

constexpr int kStages = 4;           // slots of a warp's ring

template <int DH>
struct Few8Shared {
    static constexpr int CHUNKS = DH / 8;     // float4 of a thread's part of O
    union {
        Slot8<DH> ring[kWarps][kStages];
        float4 o[kWarps][CHUNKS][32];         // a piece's sums, once its rings are empty
    };
    float ml[kWarps][kRows][2];
    long long scratch[kWarps + 1];
    Walk8 walk;
    Piece8 piece;
    int seen;
};

// This lane's rows r = lane / 4 and r + 8 of an item.
struct Rows8 {
    int lo[2], hi[2];      // keys they see
    float c[2];            // scale / ln 2 (times the power of two taken out of the queries)
    float m[2], l[2];
};

// One step of 16 keys from kb on, whose blocks have exponents ek and ev.
// HALF: rows 8 .. 15 hold nothing.
template <int DH, bool HALF>
PI_DEV void step(const Piece8& p, const Slot8<DH>& s, int ek, int ev, int kb, bool edge, const uint32_t (&q)[DH / 16][4],
                 Rows8& w, float (&o)[DH / 8][4]) {
    constexpr int KC = Slot8<DH>::KC, VW = Slot8<DH>::VW, RH = HALF ? 1 : 2;
    const int lane = threadIdx.x & 31, q4 = lane & 3;
    float acc[2][2][4];   // two chains for each 8 keys
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][i][e] = 0.f;
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 y = s.k[j * KC + c][lane];
                const uint32_t word = i == 0 ? y.x : i == 1 ? y.y : i == 2 ? y.z : y.w;
                mma16816(acc[j][i & 1], q[4 * c + i], widen2(word & 0xffffu), widen2(word >> 16));
            }
    uint32_t v[4][VW];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        if (DH == 128) {
            const uint4 y = *reinterpret_cast<const uint4*>(s.v[x][lane]);
            v[x][0] = y.x;
            v[x][1] = y.y;
            v[x][VW - 2] = y.z;
            v[x][VW - 1] = y.w;
        } else {
            const uint2 y = *reinterpret_cast<const uint2*>(s.v[x][lane]);
            v[x][0] = y.x;
            v[x][1] = y.y;
        }
    }
    // x = c 2^ek S of this lane's keys kb + 8 j + 2 q + e
    float x[2][4];
    const float fk = pow2(ek), fev = (float)ev;
#pragma unroll
    for (int h = 0; h < RH; ++h) {
        const float f = fminf(w.c[h] * fk, 3e38f);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) x[j][2 * h + e] = (acc[j][0][2 * h + e] + acc[j][1][2 * h + e]) * f;
    }
    uint32_t see = ~0u;    // bit 4 j + 2 h + e: the row sees the key
    if (edge) {
        see = 0;
#pragma unroll
        for (int h = 0; h < RH; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = kb + 8 * j + 2 * q4 + e;
                    if (key >= w.lo[h] && key < w.hi[h]) see |= 1u << (4 * j + 2 * h + e);
                    else x[j][2 * h + e] = -INFINITY;
                }
        // values of keys that no row sees are not used, whatever they are
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int key = kb + 8 * (y >> 1) + 2 * q4 + (y & 1);
            if (key < p.lo || key >= p.hi)
#pragma unroll
                for (int i = 0; i < VW; ++i) v[y][i] = 0u;
        }
    }
    // m, where it has to move
    bool grown = false;
    float top[2];
#pragma unroll
    for (int h = 0; h < RH; ++h) {
        top[h] = fmaxf(fmaxf(x[0][2 * h], x[0][2 * h + 1]), fmaxf(x[1][2 * h], x[1][2 * h + 1])) + fev;
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
    uint32_t pk[4] = {0u, 0u, 0u, 0u};
    const float back = pow2(-ev);
#pragma unroll
    for (int h = 0; h < RH; ++h) {
        const float bias = kLift + fev - (w.m[h] == -INFINITY ? 0.f : w.m[h]);
        float y[2][2], sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) sum += y[j][e] = ex2(x[j][2 * h + e] + bias);
        w.l[h] = fmaf(sum, back, w.l[h]);
        pk[h] = half2_of(y[0][0], y[0][1]);
        pk[2 + h] = half2_of(y[1][0], y[1][1]);
    }
    if (edge) {
        // 0 x NaN would reach rows that do not see the value: such codes leave the
        // product, and the rows that see one become NaN there
        bool nan = false;
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int i = 0; i < VW; ++i) nan |= (((v[y][i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
        if (__any_sync(FULL, nan)) {
            uint32_t seen[4];   // 1 where the row sees the key
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = 4 * (i >> 1) + 2 * (i & 1);
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
        mma16816(o[4 * i], pk, widen2(a0 & 0xffffu), widen2(b0 & 0xffffu));
        mma16816(o[4 * i + 1], pk, widen2(a0 >> 16), widen2(b0 >> 16));
        mma16816(o[4 * i + 2], pk, widen2(a1 & 0xffffu), widen2(b1 & 0xffffu));
        mma16816(o[4 * i + 3], pk, widen2(a1 >> 16), widen2(b1 >> 16));
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

// Blocks of an SM: what registers and rings leave room for.
template <int DH, bool HALF>
constexpr int few_blocks() { return DH == 64 || HALF ? 3 : 2; }

template <typename T, int DH, bool HALF>
__global__ void __launch_bounds__(kThreads, few_blocks<DH, HALF>()) k_attn8_few(const __grid_constant__ Few8Args a) {
    pdl_entry();
    constexpr int KC = Slot8<DH>::KC, OC = DH / 8, CHUNKS = HALF ? DH / 16 : DH / 8, RH = HALF ? 1 : 2;
    extern __shared__ __align__(16) unsigned char few_smem[];
    Few8Shared<DH>& sh = *reinterpret_cast<Few8Shared<DH>*>(few_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q4 = lane & 3, r8 = lane >> 2;

    // units of all requests, and where this block's range starts
    const int per = (a.batch + kThreads - 1) / kThreads, b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    long long own = 0, U = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) own += a.c.kv_heads * request_units(a, request8(a, b, &bad));
    if (bad && blockIdx.x == 0) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
    if (tid == 0) {
        sh.walk = Walk8{};
        sh.walk.u = 0x7fffffffffffffffll;
    }
    const long long pre = scan_before<kThreads>(own, sh.scratch, &U);
    const int G = (int)min((long long)gridDim.x, max(U / kMinUnits, U > 0 ? 1ll : 0ll));
    if ((int)blockIdx.x >= G) return;
    const long long u0 = U * blockIdx.x / G, u1 = U * (blockIdx.x + 1) / G;
    if (tid == 0) {
        sh.walk.u1 = u1;
        sh.walk.U = U;
        sh.walk.G = G;
    }
    if (pre <= u0 && u0 < pre + own) {
        long long left = u0 - pre;
        for (int b = b0; b < b1; ++b) {
            const Request8 r = request8(a, b, &bad);
            const long long u = request_units(a, r);
            if (left >= a.c.kv_heads * u) {
                left -= a.c.kv_heads * u;
                continue;
            }
            const int g = (int)(left / u);
            left -= g * u;
            int rt = 0, lo, hi;
            for (;; ++rt) {
                const int cost = kLead + item_range(a, r, rt, &lo, &hi);
                if (left < cost) break;
                left -= cost;
            }
            sh.walk.u = u0;
            sh.walk.b = b;
            sh.walk.g = g;
            sh.walk.rt = rt;
            sh.walk.off = (int)left;
            sh.walk.r = r;
            break;
        }
    }
    __syncthreads();

    for (;;) {
        if (tid == 0) sh.piece = sh.walk.next(a);
        __syncthreads();
        const Piece8 p = sh.piece;
        if (p.nt == 0) return;
        const int32_t* const pages = a.table + (size_t)p.b * a.max_pages;
        // this warp's steps: keys 16 s of the piece's tiles that some row sees
        const int s_end = (min(p.hi, (p.j0 + p.nt) * kTile) + kBlock - 1) / kBlock;
        const int s0 = max(p.lo, p.j0 * kTile) / kBlock + warp;
        const int steps = s0 < s_end ? (s_end - s0 + kWarps - 1) / kWarps : 0;
        // Pages and exponents of the warp's next 32 steps, a lane each; those of the 32
        // behind them come while these run.
        auto page_of = [&](int i) {
            if (i >= steps) return -1;
            const int id = pages[(s0 + i * kWarps) >> (a.c.page_shift - 4)];
            if (id >= 0 && id < a.c.num_pages) return id;
            atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
            return -1;
        };
        auto exponents_of = [&](int i, int id) {
            if (id < 0) return 0;
            const long long at = (((long long)id * a.c.kv_heads + p.g) << (a.c.page_shift - 4)) + ((s0 + i * kWarps) & ((1 << (a.c.page_shift - 4)) - 1));
            return bounded(a.c.ke[at]) * 256 + bounded(a.c.ve[at]);
        };
        int id = page_of(lane), id_next = page_of(32 + lane);
        Slot8<DH>* const ring = sh.ring[warp];
        auto ask = [&](int i) {   // step i of the piece, at most 31 ahead of the one that runs
            const int mine = __shfl_sync(FULL, i & 32 ? id_next : id, i & 31);
            if (i < steps) fetch<DH>(a, ring[i % kStages], mine, (s0 + i * kWarps) * kBlock, p.g);
            copies_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) ask(i);
        int ex = exponents_of(lane, id), ex_next = 0;

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
            const int tr = r8 + 8 * h, row = p.rt * kRows + tr;
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

        for (int i = 0; i < steps; ++i) {
            const int in_32 = i & 31;
            if (in_32 == 0 && i > 0) {
                id = id_next;
                ex = ex_next;
                id_next = page_of(i + 32 + lane);
            }
            if (in_32 == 16) ex_next = exponents_of((i & ~31) + 32 + lane, id_next);
            {   // the step kStages - 1 ahead
                const int n = in_32 + kStages - 1;
                const int mine = __shfl_sync(FULL, n & 32 ? id_next : id, n & 31);
                if (i + kStages - 1 < steps)
                    fetch<DH>(a, ring[(i + kStages - 1) % kStages], mine, (s0 + (i + kStages - 1) * kWarps) * kBlock, p.g);
                copies_commit();
            }
            copies_wait<kStages - 1>();
            const int e = __shfl_sync(FULL, ex, in_32), ev = (int)(signed char)(e & 255), ek = (e - ev) >> 8;
            const int kb = (s0 + i * kWarps) * kBlock;
            step<DH, HALF>(p, ring[i % kStages], ek, ev, kb, kb < lo_most || kb + kBlock > hi_least, q, w, o);
        }
        copies_wait<0>();
        __syncthreads();   // the rings are empty: their place is the sums'

        // the warps' sums, each scaled to the block's maximum
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            w.l[h] += __shfl_xor_sync(FULL, w.l[h], 1);
            w.l[h] += __shfl_xor_sync(FULL, w.l[h], 2);
            if (q4 == 0) {
                sh.ml[warp][r8 + 8 * h][0] = w.m[h];
                sh.ml[warp][r8 + 8 * h][1] = w.l[h];
            }
        }
        __syncthreads();
        float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f};   // of this lane's rows, over the block
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            float m[kWarps], l[kWarps];
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                m[i] = sh.ml[i][r8 + 8 * h][0];
                l[i] = sh.ml[i][r8 + 8 * h][1];
                M[h] = fmaxf(M[h], m[i]);
            }
            const float use = M[h] == -INFINITY ? 0.f : M[h], f = ex2(w.m[h] - use);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) L[h] = fmaf(l[i], ex2(m[i] - use), L[h]);
            // chunk (2 h + e) DH / 32 + i: elements 4 i .. of this lane's run e, of row r8 + 8 h
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < DH / 32; ++i)
                    sh.o[warp][(2 * h + e) * (DH / 32) + i][lane] =
                        make_float4(o[4 * i][2 * h + e] * f, o[4 * i + 1][2 * h + e] * f, o[4 * i + 2][2 * h + e] * f, o[4 * i + 3][2 * h + e] * f);
        }
        __syncthreads();

        // a thread's share: chunks warp, warp + 4, ... of its lane's rows
        auto write = [&](int c, float4 v, const float (&inv)[2]) {
            const int h = c / (DH / 16), e = c / (DH / 32) % 2, tr = r8 + 8 * h, row = p.rt * kRows + tr;
            if (tr >= p.rows) return;
            const int tok = row / a.group, head = p.g * a.group + row - tok * a.group;
            const float f = inv[h];
            put4(static_cast<T*>(a.out) + (long long)(p.cu + tok) * a.o_stride + (long long)head * DH + (2 * q4 + e) * (DH / 8) + c % (DH / 32) * 4,
                 make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
        };
        auto write_lse = [&](const float (&m)[2], const float (&l)[2]) {
            if (a.lse == nullptr || warp != 0 || q4 != 0) return;
#pragma unroll
            for (int h = 0; h < RH; ++h) {
                const int tr = r8 + 8 * h, row = p.rt * kRows + tr;
                if (tr >= p.rows) continue;
                const int tok = row / a.group, head = p.g * a.group + row - tok * a.group;
                a.lse[(long long)(p.cu + tok) * a.heads + head] = l[h] == 0.f ? -INFINITY : (m[h] - kLift + log2f(l[h])) * kLn2;
            }
        };
        // (a sum of 0: the row sees nothing; one that is not a number stays one)
        auto inverse = [](float l) { return l == 0.f ? 0.f : 1.f / l; };
        if (p.parts == 1) {
            const float inv[2] = {inverse(L[0]), inverse(L[1])};
#pragma unroll
            for (int c = warp; c < CHUNKS; c += kWarps) {
                float4 v = sh.o[0][c][lane];
#pragma unroll
                for (int i = 1; i < kWarps; ++i) {
                    const float4 z = sh.o[i][c][lane];
                    v = make_float4(v.x + z.x, v.y + z.y, v.z + z.z, v.w + z.w);
                }
                write(c, v, inv);
            }
            write_lse(M, L);
        } else {
            const int slot = (int)blockIdx.x * 2 + p.own;
            float4* const po = reinterpret_cast<float4*>(a.part_o) + (size_t)slot * Few8Shared<DH>::CHUNKS * 32;
            float2* const pm = reinterpret_cast<float2*>(a.part_ml) + slot * kRows;
#pragma unroll
            for (int c = warp; c < CHUNKS; c += kWarps) {
                float4 v = sh.o[0][c][lane];
#pragma unroll
                for (int i = 1; i < kWarps; ++i) {
                    const float4 z = sh.o[i][c][lane];
                    v = make_float4(v.x + z.x, v.y + z.y, v.z + z.z, v.w + z.w);
                }
                po[c * 32 + lane] = v;
            }
            if (warp == 0 && q4 == 0)
#pragma unroll
                for (int h = 0; h < RH; ++h) pm[r8 + 8 * h] = make_float2(M[h], L[h]);
            // the block's stores happen before thread 0's arrival (barrier, then release), the
            // other blocks' before what any thread reads after it (acquire, then barrier)
            __syncthreads();
            if (tid == 0) {
                sh.seen = arrive_gpu(a.counters + p.block0);
                if (sh.seen == p.parts - 1) a.counters[p.block0] = 0;
            }
            __syncthreads();
            if (sh.seen == p.parts - 1) {
                // partial of block block0 + k: its second slot (k = 0, where the item starts) or its first
                auto slot_of = [&](int k) { return (p.block0 + k) * 2 + (k == 0 ? 1 : 0); };
                const float4* const all = reinterpret_cast<const float4*>(a.part_o);
                // m and l of all parts beside each other, up to as many as the rings' place holds at a time
                const int most = kWarps * kStages * (int)sizeof(Slot8<DH>) / (kRows * (int)sizeof(float2));
                float2* const ml = reinterpret_cast<float2*>(&sh.ring[0][0]);
                float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, use[2] = {0.f, 0.f};
                float4 v[CHUNKS / kWarps];
#pragma unroll
                for (int i = 0; i < CHUNKS / kWarps; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k0 = 0; k0 < p.parts; k0 += most) {
                    const int n = min(most, p.parts - k0);
                    __syncthreads();
                    for (int i = tid; i < n * kRows; i += kThreads)
                        ml[i] = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot_of(k0 + i / kRows) * kRows + i % kRows);
                    __syncthreads();
#pragma unroll
                    for (int h = 0; h < RH; ++h) {
                        float top = m[h];
#pragma unroll 4
                        for (int k = 0; k < n; ++k) top = fmaxf(top, ml[k * kRows + r8 + 8 * h].x);
                        use[h] = top == -INFINITY ? 0.f : top;
                        const float f = ex2(m[h] - use[h]);   // of what the parts before these have summed
                        m[h] = top;
                        l[h] *= f;
#pragma unroll
                        for (int i = 0; i < CHUNKS / kWarps; ++i)
                            if (HALF || (warp + i * kWarps) / (DH / 16) == h) {
                                v[i].x *= f;
                                v[i].y *= f;
                                v[i].z *= f;
                                v[i].w *= f;
                            }
                    }
                    constexpr int AT_ONCE = 16 / (CHUNKS / kWarps);   // parts whose loads are in flight together
                    for (int k = 0; k < n; k += AT_ONCE) {
                        float4 z[AT_ONCE][CHUNKS / kWarps];
#pragma unroll
                        for (int x = 0; x < AT_ONCE; ++x) {   // past the end: the last one once more, left out below
                            const int at = slot_of(k0 + min(k + x, n - 1));
#pragma unroll
                            for (int i = 0; i < CHUNKS / kWarps; ++i)
                                z[x][i] = __ldcg(all + ((size_t)at * Few8Shared<DH>::CHUNKS + warp + i * kWarps) * 32 + lane);
                        }
#pragma unroll
                        for (int x = 0; x < AT_ONCE; ++x) {
                            if (k + x >= n) break;
                            float f[2] = {0.f, 0.f};
#pragma unroll
                            for (int h = 0; h < RH; ++h) {
                                const float2 y = ml[(k + x) * kRows + r8 + 8 * h];
                                f[h] = ex2(y.x - use[h]);
                                l[h] = fmaf(y.y, f[h], l[h]);
                            }
#pragma unroll
                            for (int i = 0; i < CHUNKS / kWarps; ++i) {
                                const float g = HALF || warp + i * kWarps < DH / 16 ? f[0] : f[1];
                                v[i] = make_float4(fmaf(z[x][i].x, g, v[i].x), fmaf(z[x][i].y, g, v[i].y), fmaf(z[x][i].z, g, v[i].z),
                                                   fmaf(z[x][i].w, g, v[i].w));
                            }
                        }
                    }
                }
                const float inv[2] = {inverse(l[0]), inverse(l[1])};
#pragma unroll
                for (int i = 0; i < CHUNKS / kWarps; ++i) write(warp + i * kWarps, v[i], inv);
                write_lse(m, l);
            }
        }
        // (the next piece's sums are written behind its own barriers)
    }
}

// ------------------------------------------------ pages of long requests in 16 bits
//
// A unit is one KV head of one page that a request of many rows sees; a block
// takes a contiguous range of units.  Page p of the cache is page p of the copy.
constexpr int kWidenThreads = 256;

struct Widen8Args {
    Cache8 c;
    const int32_t *table, *cu, *kv;
    void *k, *v;       // [num_pages, kv_heads, page_size, dh] in 16 bits
    int batch, max_tokens, max_new, max_pages, window, few, dh;
    int* status;
};

// pages of a request that are widened: first and how many
PI_DEV int seen_pages(const Widen8Args& a, const Request8& r, int* first) {
    const int hi = r.first + r.n, lo = a.window > 0 ? max(0, r.first - a.window + 1) : 0;
    *first = lo >> a.c.page_shift;
    if (r.n <= a.few || hi <= lo) return 0;
    return ((hi + (1 << a.c.page_shift) - 1) >> a.c.page_shift) - *first;
}

PI_DEV void put16(__half* p, const uint4& c, float scale) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
    auto in = [](float x) { return fabsf(x) > 65504.f ? copysignf(65504.f, x) : x; };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 u = values2((w[i / 2] >> (16 * (i & 1))) & 0xffffu);
        o[i] = half2_of(in(u.x * scale), in(u.y * scale));
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
}
PI_DEV void put16(__nv_bfloat16* p, const uint4& c, float scale) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 u = values2((w[i / 2] >> (16 * (i & 1))) & 0xffffu);
        const __nv_bfloat162 y = __floats2bfloat162_rn(u.x * scale, u.y * scale);
        o[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

template <typename T>
__global__ void __launch_bounds__(kWidenThreads) k_widen8(const __grid_constant__ Widen8Args a) {
    pdl_entry();
    __shared__ long long scratch[kWidenThreads / 32 + 1];
    __shared__ int at_b, at_page, at_head;
    const int tid = threadIdx.x;
    const int per = (a.batch + kWidenThreads - 1) / kWidenThreads, b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    long long own = 0, U = 0;
    bool bad = false;
    int first;
    for (int b = b0; b < b1; ++b) own += (long long)a.c.kv_heads * seen_pages(a, request8(a, b, &bad), &first);
    const long long pre = scan_before<kWidenThreads>(own, scratch, &U);
    const long long u0 = U * blockIdx.x / gridDim.x, u1 = U * (blockIdx.x + 1) / gridDim.x;
    if (u0 >= u1) return;
    if (tid == 0) at_b = a.batch;
    __syncthreads();
    if (pre <= u0 && u0 < pre + own) {
        long long left = u0 - pre;
        for (int b = b0; b < b1; ++b) {
            const long long u = (long long)a.c.kv_heads * seen_pages(a, request8(a, b, &bad), &first);
            if (left < u) {
                at_page = (int)(left / a.c.kv_heads);
                at_head = (int)(left % a.c.kv_heads);
                at_b = b;
                break;
            }
            left -= u;
        }
    }
    __syncthreads();
    int b = at_b, page = at_page, head = at_head;
    if (b >= a.batch) return;   // (the lengths changed under the kernel)
    const int per_pos = a.dh / 16, chunks = per_pos << a.c.page_shift;
    int count = seen_pages(a, request8(a, b, &bad), &first);
    for (long long u = u0; u < u1; ++u) {
        const int col = first + page;
        const int id = col < a.max_pages ? a.table[(size_t)b * a.max_pages + col] : -1;
        if (id >= 0 && id < a.c.num_pages) {   // (others read as zeros and are reported by the attention)
            const long long src = id * a.c.page_stride + head * a.c.head_stride;
            const long long ex = ((long long)id * a.c.kv_heads + head) << (a.c.page_shift - 4);
            const long long dst = ((long long)id * a.c.kv_heads + head) * ((long long)a.dh << a.c.page_shift);
            for (int i = tid; i < 2 * chunks; i += kWidenThreads) {
                const bool values = i >= chunks;
                const int x = values ? i - chunks : i, pos = x / per_pos, c = x % per_pos;
                const uint4 y = ld_stream16((values ? a.c.v : a.c.k) + src + pos * a.c.token_stride + c * 16);
                const float f = pow2(bounded((values ? a.c.ve : a.c.ke)[ex + pos / kBlock]));
                put16(static_cast<T*>(values ? a.v : a.k) + dst + (long long)x * 16, y, f);
            }
        }
        if (++head == a.c.kv_heads) {
            head = 0;
            if (++page >= count) {
                page = 0;
                do {
                    if (++b >= a.batch) return;
                    count = seen_pages(a, request8(a, b, &bad), &first);
                } while (count == 0);
            }
        }
    }
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

// tokens up to which a request goes through k_attn8_few
int few_tokens(int group) { return std::max(1, kFewRows / group); }

// The copy's description: [pages, heads, positions, elements].
pi_page_desc wide_desc(const pi_page8_desc& c, int dtype) {
    return pi_page_desc{c.kv_heads, c.head_dim, c.page_size, c.num_pages, dtype, (long long)c.kv_heads * c.page_size * c.head_dim,
                        (long long)c.page_size * c.head_dim, c.head_dim};
}

// Workspace: arrival counters at offset 0 (the same place for every descriptor),
// the partials of two items per block; for steps with long requests the 16-bit
// attention's workspace and the copies of the caches' pages.
struct Layout8 {
    size_t ml, o, wide, wide_bytes, k, v, total;
    int blocks;
    Layout8(const pi_paged_desc& d, const pi_page8_desc& c, int sms) {
        auto up = [](size_t v) { return (v + 255) / 256 * 256; };
        blocks = kMostBlocks * std::max(1, sms);
        ml = up((size_t)blocks * sizeof(int));
        o = up(ml + (size_t)blocks * 2 * kRows * 2 * sizeof(float));
        wide = up(o + (size_t)blocks * 2 * kRows * c.head_dim * sizeof(float));
        k = v = total = wide;
        wide_bytes = 0;
        if (d.max_new > few_tokens(d.heads / c.kv_heads)) {
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
    constexpr int smem = (int)sizeof(Few8Shared<DH>);
    static_assert(few_blocks<DH, HALF>() * (smem + 1024) <= 228 * 1024, "shared memory of an SM");
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            e = cudaFuncSetAttribute(k_attn8_few<T, DH, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    return launch_pdl(k_attn8_few<T, DH, HALF>, few_blocks<DH, HALF>() * sms, kThreads, smem, s, a);
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
    a.few = few_tokens(a.group);
    a.scale = desc->scale > 0.f ? desc->scale : 1.0f / sqrtf((float)cache->head_dim);
    a.counters = reinterpret_cast<int*>(ws);
    a.part_ml = reinterpret_cast<float*>(ws + lay.ml);
    a.part_o = reinterpret_cast<float*>(ws + lay.o);
    a.status = status_word();
    if (sms < 1 || a.status == nullptr) return PI_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool half = std::min(desc->max_new, a.few) * a.group <= 8;   // no item has more than 8 rows
    const bool f16 = dtype == PI_T_F16;
    cudaError_t e = f16 ? launch_few<__half>(a, cache->head_dim, half, sms, s)
                        : launch_few<__nv_bfloat16>(a, cache->head_dim, half, sms, s);
    if (e != cudaSuccess) return PI_ERR_CUDA;
    if (desc->max_new <= a.few) return PI_OK;
    Widen8Args w{a.c, block_table, cu_new, kv_len, ws + lay.k, ws + lay.v, desc->batch, desc->max_tokens, desc->max_new,
                 desc->max_pages, a.window, a.few, cache->head_dim, a.status};
    e = f16 ? launch_pdl(k_widen8<__half>, 4 * sms, kWidenThreads, 0, s, w)
            : launch_pdl(k_widen8<__nv_bfloat16>, 4 * sms, kWidenThreads, 0, s, w);
    if (e != cudaSuccess) return PI_ERR_CUDA;
    const pi_page_desc wide = wide_desc(*cache, dtype);
    return paged_attn(desc, &wide, q, q_stride, w.k, w.v, block_table, cu_new, kv_len, out, out_stride, lse, ws + lay.wide,
                      lay.wide_bytes, a.few, stream);
}

}  // extern "C"
