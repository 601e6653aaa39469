// pi_paged_attn.cu -- causal attention of new tokens over a paged cache.
//
// A request's new tokens and the query heads that share a KV head form rows
// (row = token * group + head in the group), so one pass over the keys serves
// the whole group.  An item is up to 256 rows of one request and KV head; its
// keys come in tiles of 128.  For a tile, on the tcgen05 tensor cores,
//     S = Q K^T         (fp16/bf16 products, fp32 sums in tensor memory)
//     P = 2^(c S - m)   (a thread per row; running m and l = sum P)
//     O += P V          (P as the A operand in tensor memory)
// where c = scale / ln 2 and m trails the running maximum: it moves only when
// a row's maximum has grown by more than 2^8 (then O and l are scaled), so O is
// touched rarely.  P carries a factor 2^7, which l and O share: the largest
// weights are then 2^7 .. 2^15, within fp16, and weights down to 2^-31 of the
// largest survive the rounding.
//
// Warps: 0-3 and 4-7 softmax (a thread per row), 8 TMA, 9 MMA issue, 10 query
// rows, 11 the work list.  Items of more than 128 rows give each softmax group
// 128 of them (both use every key tile: "pair"); smaller items, decode steps
// among them, give the two groups alternate key tiles and merge at the end, so
// that one group's exponentials run beside the other's products.
//
// Work split: the (item x key tile) space is cut into equal contiguous ranges
// per block, whatever the lengths; an item cut by a border leaves unnormalised
// partials (m, l, O) in the workspace, and the block that arrives last adds
// them in block order (the order is fixed, who does it is not: same bits).
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
constexpr int kRows = 256;             // rows of an item at most
constexpr int kPagedThreads = 384;
constexpr int kListDepth = 4;          // pieces the work list runs ahead
constexpr int kConsumers = 11;         // warps that read the work list
constexpr float kLift = 7.f;           // log2 of the factor that P, l and O share
constexpr float kSlack = 8.f;          // growth (log2) of a maximum before m follows
constexpr float kLn2 = 0.69314718055994531f;

template <int DH>
struct PagedCfg {
    static constexpr int HALVES = DH / 64;               // 64-element column blocks of a row
    static constexpr int TILE = kKeys * DH * 2;          // bytes of a key or value tile
    static constexpr int Q = kRows * DH * 2;
    static constexpr int S = DH == 128 ? 5 : 12;         // ring slots
    static constexpr int MISC = 3072;
    static constexpr int SMEM = Q + S * TILE + MISC;
    static constexpr unsigned O_COL = 2 * kKeys;         // tensor memory: S0 S1 | O0 O1
    static_assert(SMEM <= 232448, "shared memory of a block");
};

struct PagedArgs {
    CUtensorMap kmap, vmap;   // {dh, position, head, page}, box 64 x page_size
    const void *q, *k, *v;
    const int32_t *table, *cu, *kv;
    void* out;
    float* lse;
    long long q_stride, o_stride, page_stride, head_stride, token_stride;
    int heads, kv_heads, batch, max_tokens, max_new, max_pages, window, page_size, num_pages;
    int group;                // query heads per KV head
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
    int row0, rows;  // rows of the request's (token, head in group) rows
    int first;       // position of the request's first new token (negative: it sees nothing)
    int cu;          // the request's first row of q and out
    int block0;      // first block that holds a part of the item
    int parts;       // blocks that do (1: this one alone)
    int own;         // this block's partial: 1 where the item starts here
    int pad[3];
};

template <int DH>
struct PagedShared {
    unsigned long long full[12], empty[12], qfull, qempty, sfull[2], pready[2], odone[2], lfull[kListDepth],
        lempty[kListDepth], merge[2], merged, drain;
    Piece list[kListDepth];
    float ml[2][kKeys][2];
    long long start_u;   // this block's first unit, and where it is
    int start_b, start_g, start_row0, start_off;
    unsigned tmem;
    int abort_flag;
};

struct Request {
    int cu, n, first, rows;
};

PI_DEV Request request(const PagedArgs& a, int b, bool* bad) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    int kv = a.kv[b];
    Request r{lo, hi - lo, 0, 0};
    if (lo < 0 || hi < lo || hi > a.max_tokens || hi - lo > a.max_new) {
        *bad = true;
        r.n = 0;
    }
    if (kv < 0 || kv > a.max_pages * a.page_size) {
        *bad = true;
        kv = 0;
    }
    r.first = kv - r.n;
    r.rows = r.n * a.group;
    return r;
}

// Keys that rows row0 .. row0 + rows - 1 of a request see, as key tiles (one
// tile, with nothing to see in it, where they see none: it writes the zeros).
PI_DEV int item_tiles(const PagedArgs& a, const Request& r, int row0, int* rows, int* lo, int* hi) {
    *rows = min(kRows, r.rows - row0);
    const int t0 = row0 / a.group, t1 = (row0 + *rows - 1) / a.group;
    *hi = r.first + t1 + 1;
    *lo = a.window > 0 ? max(0, r.first + t0 - a.window + 1) : 0;
    if (*hi <= *lo) {
        *lo = *hi = 0;
        return 1;
    }
    return (*hi + kKeys - 1) / kKeys - *lo / kKeys;
}

PI_DEV long long request_units(const PagedArgs& a, const Request& r) {   // of one KV head
    long long u = 0;
    int rows, lo, hi;
    for (int row0 = 0; row0 < r.rows; row0 += kRows) u += item_tiles(a, r, row0, &rows, &lo, &hi);
    return u;
}

PI_DEV bool warp_wait(unsigned long long* b, unsigned parity, const Ctl& c) {
    return __all_sync(FULL, bar_wait(b, parity, c));
}

PI_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
PI_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// One row over keys lo .. hi - 1 by the whole warp, key by key, keeping only
// what the row sees.  For rows whose tensor-core result is not finite: there
// 0 x value has let a non-finite value of a key that this row does not see
// into the sum (P is 0 there, but 0 x inf is NaN), or the row sees such a
// value itself.  Same convention as the tiles: m in log2 units, l and o with
// the factor 2^kLift.
template <typename T, int DH>
__device__ __noinline__ void careful_row(const PagedArgs& a, int b, int g, long long q_at, int lo, int hi, float& m_out,
                                         float& l_out, float (&o)[DH / 32]) {
    constexpr int E = DH / 32;
    const int lane = threadIdx.x & 31;
    const T* qp = static_cast<const T*>(a.q) + q_at + lane * E;
    const float c = a.scale / kLn2;
    float q[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = to_f(qp[e]);
        o[e] = 0.f;
    }
    for (int x = lo; x < hi; ++x) {
        const int page = a.table[(size_t)b * a.max_pages + x / a.page_size];
        const bool ok = page >= 0 && page < a.num_pages;
        const long long at = (ok ? page : 0) * a.page_stride + g * a.head_stride +
                             (x % a.page_size) * a.token_stride + lane * E;
        const T *kp = static_cast<const T*>(a.k) + at, *vp = static_cast<const T*>(a.v) + at;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], ok ? to_f(kp[e]) : 0.f, s);
        s = warp_sum(s) * c;
        const float mn = fmaxf(m, s), use = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - use), w = exp2f(s - use + kLift);
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], f, w * (ok ? to_f(vp[e]) : 0.f));
        m = mn;
    }
    m_out = m;
    l_out = l;
}

// ------------------------------------------------------------ work list (warp 11)
template <int DH>
PI_DEV void list_role(const PagedArgs& a, PagedShared<DH>& sh, long long u1, long long U, int G, const Ctl& ctl) {
    int b = sh.start_b, g = sh.start_g, row0 = sh.start_row0, off = sh.start_off;
    long long u = sh.start_u;
    bool bad = false;
    Request r = request(a, b, &bad);
    int n = 0;
    for (;; ++n) {
        const int s = n % kListDepth;
        if (n >= kListDepth && !bar_wait(&sh.lempty[s], (n / kListDepth - 1) & 1, ctl)) return;
        Piece p{};
        if (u < u1) {
            int rows, lo, hi;
            const int nt = item_tiles(a, r, row0, &rows, &lo, &hi);
            p.nt = (int)min((long long)(nt - off), u1 - u);
            p.j0 = lo / kKeys + off;
            p.lo = lo;
            p.hi = hi;
            p.b = b;
            p.g = g;
            p.row0 = row0;
            p.rows = rows;
            p.first = r.first;
            p.cu = r.cu;
            p.parts = 1;
            p.own = off == 0;
            if (p.nt != nt) {
                const long long i0 = u - off;   // the item's first unit, and the blocks that own its ends
                p.block0 = (int)(((i0 + 1) * G - 1) / U);
                p.parts = (int)(((i0 + nt) * G - 1) / U) - p.block0 + 1;
            }
            u += p.nt;
            off = 0;
            row0 += kRows;
            if (u < u1 && row0 >= r.rows) {
                row0 = 0;
                if (++g == a.kv_heads) {
                    g = 0;
                    // u < u1 <= U: a later request has rows
                    do {
                        if (++b >= a.batch) {   // the lengths changed under the kernel: stop
                            u = u1;
                            break;
                        }
                        r = request(a, b, &bad);
                    } while (r.rows == 0);
                }
            }
        }
        sh.list[s] = p;
        bar_arrive(&sh.lfull[s]);
        if (p.nt == 0) return;
    }
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

// ------------------------------------------------------------ key and value tiles (warp 8)
//
// Slots go out in the order the products need them: K0, then K(t+1), V(t).  A
// lane per (page, column block) of a tile; pages outside the keys the item
// sees are not read (their rows of the slot are stale: scores there are
// masked, value rows are cleared by the MMA warp).
template <int DH>
PI_DEV void tile_role(const PagedArgs& a, PagedShared<DH>& sh, unsigned char* ring, const Ctl& ctl) {
    using C = PagedCfg<DH>;
    const int lane = threadIdx.x & 31;
    const int ppt = kKeys / a.page_size;
    const int pl = lane % ppt, half = lane / ppt;
    const bool has = half < C::HALVES;
    int it = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
        const Piece p = next_piece<DH>(sh, n, ctl);
        if (p.nt == 0) break;
        const int32_t* row = a.table + (size_t)p.b * a.max_pages;
        // page of this lane in tile t: -1 where it is not needed
        auto page_of = [&](int t) {
            const int key = (p.j0 + t) * kKeys + pl * a.page_size;
            if (t >= p.nt || !has || key >= p.hi || key + a.page_size <= p.lo) return -1;
            const int id = row[key / a.page_size];
            if (id >= 0 && id < a.num_pages) return id;
            atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
            return a.num_pages;   // past the last page: the copy fills zeros
        };
        auto issue = [&](const CUtensorMap* map, int id) {
            const int s = it % C::S;
            if (it >= C::S && !warp_wait(&sh.empty[s], (it / C::S - 1) & 1, ctl)) return false;
            const unsigned boxes = __popc(__ballot_sync(FULL, id >= 0));
            if (lane == 0) bar_arrive_expect_tx(&sh.full[s], boxes * (unsigned)a.page_size * 128u);
            __syncwarp();
            if (id >= 0)
                tma_load_4d(ring + (size_t)s * C::TILE + half * (kKeys * 128) + pl * a.page_size * 128, map, 64 * half, 0,
                            p.g, id, &sh.full[s]);
            ++it;
            return true;
        };
        int cur = page_of(0), nxt = page_of(1);
        ok = issue(&a.kmap, cur);
        for (int t = 0; t < p.nt && ok; ++t) {
            const int after = page_of(t + 2);
            if (t + 1 < p.nt) ok = issue(&a.kmap, nxt);
            if (ok) ok = issue(&a.vmap, cur);
            cur = nxt;
            nxt = after;
        }
    }
    // every copy issued has landed before the block may exit
    for (int s = 0; s < C::S && s < it; ++s) {
        const int last = s + ((it - 1 - s) / C::S) * C::S;
        bar_drain(&sh.full[s], (last / C::S) & 1, kDrainTimeoutNs);
    }
}

// ------------------------------------------------------------ query rows (warp 10)
//
// Rows of the item in the MMA's K-major layout (128 bytes per row and column
// block, 16-byte chunk c of row r at c ^ (r % 8)); rows past the item's stay
// as they are: a row of S depends on its own query alone.
template <typename T, int DH>
PI_DEV void query_role(const PagedArgs& a, PagedShared<DH>& sh, unsigned char* qs, const Ctl& ctl) {
    constexpr int CH = DH / 8, STEP = 32 / CH;   // 16-byte chunks of a row; rows per step
    const int lane = threadIdx.x & 31;
    const int c = lane % CH;
    for (int n = 0;; ++n) {
        const Piece p = next_piece<DH>(sh, n, ctl);
        if (p.nt == 0) return;
        if (n >= 1 && !warp_wait(&sh.qempty, (n - 1) & 1, ctl)) return;
        int tok = (p.row0 + lane / CH) / a.group, h = (p.row0 + lane / CH) % a.group;
        for (int r = lane / CH; r < p.rows; r += STEP) {
            const T* src = static_cast<const T*>(a.q) + (long long)(p.cu + tok) * a.q_stride +
                           (long long)(p.g * a.group + h) * DH + 8 * c;
            cp16(qs + (r >> 7) * (kKeys * DH * 2) + (c >> 3) * (kKeys * 128) + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4),
                 src);
            for (h += STEP; h >= a.group; h -= a.group) ++tok;
        }
        cp_commit();
        cp_wait_all();
        fence_async_smem();
        warp_arrive(&sh.qfull);
    }
}

// ------------------------------------------------------------ products (warp 9)
template <typename T, int DH>
PI_DEV void mma_role(const PagedArgs& a, PagedShared<DH>& sh, unsigned char* qs, unsigned char* ring, unsigned tmem,
                     const Ctl& ctl) {
    using C = PagedCfg<DH>;
    const int lane = threadIdx.x & 31;
    constexpr unsigned kType = std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10);   // A and B: fp16 or bf16
    const unsigned id_s = idesc_f16(128, kKeys, false) | kType;
    const unsigned id_o = idesc_f16(128, DH, false) | kType | (1u << 16);   // B (values) MN-major
    int it = 0;               // next ring slot to use
    int np[2] = {0, 0};       // products P V asked of each softmax group
    bool ok = true;
    auto slot = [&](int i) { return su32(ring) + (unsigned)((i % C::S) * C::TILE); };
    auto wait_full = [&](int i) {
        const bool r = warp_wait(&sh.full[i % C::S], (i / C::S) & 1, ctl);
        tc_after();
        return r;
    };
    auto scores = [&](int w, int qw, int i) {   // S_w = Q_qw K^T of slot i
        if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk) {
                const unsigned o = (unsigned)((kk >> 2) * (kKeys * 128) + (kk & 3) * 32);
                mma_f16(tmem + (unsigned)(w * kKeys), sdesc_sw128(su32(qs) + (unsigned)(qw * kKeys * DH * 2) + o),
                        sdesc_sw128(slot(i) + o), id_s, kk > 0 ? 1u : 0u);
            }
            mma_commit(&sh.sfull[w]);
        }
    };
    auto values = [&](int w, int i, bool add) {   // O_w (+)= P_w V of slot i
        if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_f16_ta(tmem + C::O_COL + (unsigned)(w * DH), tmem + (unsigned)(w * kKeys + kk * 8),
                           sdesc_sw128_mn(slot(i) + (unsigned)(kk * 2048), kKeys * 128, 1024), id_o,
                           (add || kk > 0) ? 1u : 0u);
            mma_commit(&sh.odone[w]);
        }
    };
    auto release = [&](unsigned long long* bar) {
        if (lane == 0) mma_commit(bar);
    };
    // value rows outside the keys the item sees: zeros, not what the cache or the slot holds there
    auto clear = [&](const Piece& p, int t, int i) {
        const int base = (p.j0 + t) * kKeys;
        const int z = min(max(p.lo - base, 0), kKeys), e = min(max(p.hi - base, z), kKeys);
        if (z == 0 && e == kKeys) return;
        unsigned char* v = ring + (size_t)(i % C::S) * C::TILE;
        const int dead = kKeys - (e - z);
        for (int x = lane; x < dead * (DH / 8); x += 32) {
            const int d = x / (DH / 8), c = x % (DH / 8);
            const int r = d < z ? d : d + (e - z);
            *reinterpret_cast<uint4*>(v + (c >> 3) * (kKeys * 128) + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_smem();
        __syncwarp();
    };
    auto wait_p = [&](int w) {
        const bool r = warp_wait(&sh.pready[w], np[w] & 1, ctl);
        ++np[w];
        tc_after();
        return r;
    };
    for (int n = 0; ok; ++n) {
        const Piece p = next_piece<DH>(sh, n, ctl);
        if (p.nt == 0) break;
        ok = warp_wait(&sh.qfull, n & 1, ctl) && wait_full(it);
        if (!ok) break;
        if (p.rows > kKeys) {   // pair: both groups use every tile
            scores(0, 0, it);
            scores(1, 1, it);
            release(&sh.empty[it % C::S]);
            if (p.nt == 1) release(&sh.qempty);
            ++it;
            for (int t = 0; t < p.nt && ok; ++t) {
                const bool more = t + 1 < p.nt;
                const int ik = it, iv = more ? it + 1 : it;
                ok = (!more || wait_full(ik)) && wait_full(iv);
                if (!ok) break;
                clear(p, t, iv);
                for (int w = 0; w < 2; ++w) {
                    if (!(ok = wait_p(w))) break;
                    values(w, iv, t > 0);
                    if (more) scores(w, w, ik);
                }
                if (!ok) break;
                if (more) release(&sh.empty[ik % C::S]);
                release(&sh.empty[iv % C::S]);
                if (t + 2 == p.nt) release(&sh.qempty);
                it = iv + 1;
            }
        } else {                // the groups take alternate tiles
            scores(0, 0, it);
            release(&sh.empty[it % C::S]);
            ++it;
            if (p.nt > 1) {
                if (!(ok = wait_full(it))) break;
                scores(1, 0, it);
                release(&sh.empty[it % C::S]);
                ++it;
            }
            if (p.nt <= 2) release(&sh.qempty);
            for (int t = 0; t < p.nt && ok; ++t) {
                const int w = t & 1;
                ok = wait_full(it);
                if (!ok) break;
                clear(p, t, it);
                if (!(ok = wait_p(w))) break;
                values(w, it, t > 1);
                release(&sh.empty[it % C::S]);
                ++it;
                if (t + 2 < p.nt) {
                    if (!(ok = wait_full(it))) break;
                    scores(w, 0, it);
                    release(&sh.empty[it % C::S]);
                    ++it;
                    if (t + 3 == p.nt) release(&sh.qempty);
                }
            }
        }
    }
    // every product has completed before the block may exit
    if (lane == 0) {
        mma_commit(&sh.drain);
        bar_drain(&sh.drain, 0, kDrainTimeoutNs);
    }
    __syncwarp();
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
    int ns = 0, nm = 0;   // tiles of this group so far (all pieces); merges
    for (int n = 0;; ++n) {
        // the piece stays in its slot until it is done, so that the tile loop's
        // registers go to the scores
        if (!warp_wait(&sh.lfull[n % kListDepth], (n / kListDepth) & 1, ctl)) return;
        const Piece& p = sh.list[n % kListDepth];
        const int nt = p.nt, j0 = p.j0;
        if (nt == 0) return;
        const bool pair = p.rows > kKeys;
        const int r = (pair ? w * kKeys : 0) + 32 * quad + lane;   // row of the item
        const bool live = r < p.rows;
        int lo, hi;   // keys this row sees
        {
            const int pos = p.first + (p.row0 + r) / a.group;
            hi = live ? max(pos + 1, 0) : 0;
            lo = live && a.window > 0 ? min(max(0, pos - a.window + 1), hi) : 0;
        }
        const bool any = __any_sync(FULL, live);
        float m = -INFINITY, l = 0.f;
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
                if (__any_sync(FULL, base < lo || base + kKeys > hi)) {
#pragma unroll
                    for (int i = 0; i < kKeys; ++i)
                        if (base + i < lo || base + i >= hi) s[i] = 0xff800000u;   // -inf
                }
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(s[i]);
#pragma unroll
                for (int i = 4; i < kKeys; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                const bool grow = top > m + kSlack || (m == -INFINITY && top > m);
                if (__any_sync(FULL, grow)) {
                    const float f = grow ? ex2(m - top) : 1.f;
                    if (grow) m = top;
                    l *= f;
                    if (mine > 0) {
                        // O holds the sums over this group's earlier tiles
                        if (!warp_wait(&sh.odone[w], (ns - 1) & 1, ctl)) return;
                        tc_after();
#pragma unroll
                        for (int i = 0; i < DH; i += 32) {
                            uint32_t o[32];
                            tmem_ld32(o_at + (unsigned)i, o);
                            tmem_wait_ld();
                            tmem_loaded<32>(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(o_at + (unsigned)i, o);
                        }
                    }
                }
                const float bias = kLift - (m == -INFINITY ? 0.f : m);
                const uint64_t bias2 = pair2(bias, bias);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < kKeys; i += 64) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        float x, y;
                        split2(fma2(pair2(__uint_as_float(s[i + e]), __uint_as_float(s[i + e + 1])), c2, bias2), x, y);
                        x = ex2(x);
                        y = ex2(y);
                        sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair2(x, y));
                        pk[e >> 1] = pack2(x, y, T());
                    }
                    tmem_st32(s_at + (unsigned)(i >> 1), pk);
                }
                float x, y;
                split2(add2(sum[0], sum[1]), x, y);
                l += x + y;
                tmem_wait_st();
            }
            tc_before();
            warp_arrive(&sh.pready[w]);
            ++ns;
            ++mine;
        }
        if (mine > 0) {
            if (!warp_wait(&sh.odone[w], (ns - 1) & 1, ctl)) return;
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
        const int tok = (p.row0 + r) / a.group, h = (p.row0 + r) - tok * a.group;
        const long long orow = (long long)(p.cu + tok);
        const int head = p.g * a.group + h;
        const bool own_any = mine > 0;                  // O_w holds something
        const bool other_any = !pair && (w == 1 || p.nt > 1);
        if (any) {
            const bool whole = p.parts == 1;
            const int blk = (int)blockIdx.x * 2 + p.own;
            float* po = a.part_o + (size_t)blk * DH * a.part_rows;
            float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            bool odd = false;
            for (int i = c0; i < c0 + cols; i += 32) {
                float v[32];
                uint32_t o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0.f;
                if (own_any) {
                    tmem_ld32(o_at + (unsigned)i, o);
                    tmem_wait_ld();
                    tmem_loaded<32>(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * f_own;
                }
                if (other_any) {
                    tmem_ld32(o_other + (unsigned)i, o);
                    tmem_wait_ld();
                    tmem_loaded<32>(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = fmaf(__uint_as_float(o[e]), f_other, v[e]);
                }
                float check = 0.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) check = fmaf(v[e], 0.f, check);
                odd |= check != 0.f;   // NaN: some value is not finite
                if (live && whole) {
                    T* dst = static_cast<T*>(a.out) + orow * a.o_stride + (long long)head * DH + i;
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(dst + e) =
                            make_uint4(pack2(v[e] * inv, v[e + 1] * inv, T()), pack2(v[e + 2] * inv, v[e + 3] * inv, T()),
                                       pack2(v[e + 4] * inv, v[e + 5] * inv, T()), pack2(v[e + 6] * inv, v[e + 7] * inv, T()));
                } else if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(po + ((size_t)((i + e) / 4) * a.part_rows + r) * 4) =
                            make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
            }
            // rows whose sums are not finite, once more without the keys they do not see
            const unsigned redo = __ballot_sync(FULL, live && odd);
            __syncwarp();
            for (unsigned left = redo; left; left &= left - 1) {
                const int src = __ffs(left) - 1;
                const int rlo = max(__shfl_sync(FULL, lo, src), p.j0 * kKeys);
                const int rhi = min(__shfl_sync(FULL, hi, src), (p.j0 + p.nt) * kKeys);
                const int rt = __shfl_sync(FULL, tok, src), rh = __shfl_sync(FULL, h, src), rr = __shfl_sync(FULL, r, src);
                float rm, rl, ro[DH / 32];
                careful_row<T, DH>(a, p.b, p.g, (long long)(p.cu + rt) * a.q_stride + (long long)(p.g * a.group + rh) * DH,
                                   rlo, rhi, rm, rl, ro);
                if (lane == src) {
                    m = rm;
                    l = rl;
                }
#pragma unroll
                for (int e = 0; e < DH / 32; ++e) {
                    const int col = lane * (DH / 32) + e;
                    if (col < c0 || col >= c0 + cols) continue;
                    if (whole)
                        static_cast<T*>(a.out)[(long long)(p.cu + rt) * a.o_stride + (long long)(p.g * a.group + rh) * DH +
                                               col] = T(rl > 0.f || rl != rl ? ro[e] / rl : 0.f);
                    else
                        po[((size_t)(col / 4) * a.part_rows + rr) * 4 + col % 4] = ro[e];
                }
            }
            float out_lse = l == 0.f ? -INFINITY : (m - kLift + log2f(l)) * kLn2;
            if (whole) {
                if (live && a.lse != nullptr && c0 == 0) a.lse[orow * a.heads + head] = out_lse;
            } else {
                float* ml = a.part_ml + ((size_t)(blk * 2 + (pair ? 0 : w)) * a.part_rows + r) * 2;
                if (live) *reinterpret_cast<float2*>(ml) = make_float2(m, l);
                __threadfence();
                __syncwarp();
                int seen = 0;
                if (lane == 0) seen = atomicAdd(a.counters + p.block0 * 8 + warp, 1);
                seen = __shfl_sync(FULL, seen, 0);
                if (seen == p.parts - 1) {
                    // all parts are there: add them in block order
                    __threadfence();
                    if (lane == 0) a.counters[p.block0 * 8 + warp] = 0;
                    if (live) {
                        const size_t ml_step = (size_t)2 * 2 * a.part_rows * 2, o_step = (size_t)2 * DH * a.part_rows;
                        // partial of block block0 + k: its second slot (k = 0, where the item starts) or its first
                        auto ml_at = [&](int k) {
                            return a.part_ml + (size_t)(p.block0 + k) * ml_step +
                                   ((size_t)((k == 0 ? 2 : 0) + (pair ? 0 : w)) * a.part_rows + r) * 2;
                        };
                        float M = -INFINITY, L = 0.f;
                        for (int k = 0; k < p.parts; ++k) M = fmaxf(M, __ldcg(ml_at(k)));
                        const float use = M == -INFINITY ? 0.f : M;
                        for (int k = 0; k < p.parts; ++k) {
                            const float2 x = __ldcg(reinterpret_cast<const float2*>(ml_at(k)));
                            L = fmaf(x.y, ex2(x.x - use), L);
                        }
                        inv = L > 0.f || L != L ? 1.f / L : 0.f;
                        T* dst = static_cast<T*>(a.out) + orow * a.o_stride + (long long)head * DH;
                        for (int i = c0; i < c0 + cols; i += 16) {
                            float v[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] = 0.f;
                            for (int k = 0; k < p.parts; ++k) {
                                const float f = ex2(__ldcg(ml_at(k)) - use);
                                const float* src = a.part_o + (size_t)(p.block0 + k) * o_step +
                                                   (k == 0 ? (size_t)DH * a.part_rows : 0);
#pragma unroll
                                for (int e = 0; e < 16; e += 4) {
                                    const float4 x = __ldcg(
                                        reinterpret_cast<const float4*>(src + ((size_t)((i + e) / 4) * a.part_rows + r) * 4));
                                    v[e] = fmaf(x.x, f, v[e]);
                                    v[e + 1] = fmaf(x.y, f, v[e + 1]);
                                    v[e + 2] = fmaf(x.z, f, v[e + 2]);
                                    v[e + 3] = fmaf(x.w, f, v[e + 3]);
                                }
                            }
#pragma unroll
                            for (int e = 0; e < 16; e += 8)
                                *reinterpret_cast<uint4*>(dst + i + e) = make_uint4(
                                    pack2(v[e] * inv, v[e + 1] * inv, T()), pack2(v[e + 2] * inv, v[e + 3] * inv, T()),
                                    pack2(v[e + 4] * inv, v[e + 5] * inv, T()), pack2(v[e + 6] * inv, v[e + 7] * inv, T()));
                        }
                        if (a.lse != nullptr && c0 == 0)
                            a.lse[orow * a.heads + head] = L == 0.f ? -INFINITY : (M - kLift + log2f(L)) * kLn2;
                    }
                }
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

template <typename T, int DH>
__global__ void __launch_bounds__(kPagedThreads, 1) k_paged_attn(const __grid_constant__ PagedArgs a) {
    pdl_entry();
    using C = PagedCfg<DH>;
    extern __shared__ __align__(1024) unsigned char paged_smem[];
    unsigned char* qs = paged_smem;
    unsigned char* ring = qs + C::Q;
    PagedShared<DH>& sh = *reinterpret_cast<PagedShared<DH>*>(ring + C::S * C::TILE);
    static_assert(sizeof(PagedShared<DH>) <= C::MISC, "bookkeeping");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((su32(paged_smem) & 1023u) != 0) {   // the tiles' swizzle needs it; the whole block leaves
        if (tid == 0) atomicExch(a.status, (int)PI_ERR_UNSUPPORTED);
        return;
    }
    if (warp == 9) {
        if (lane == 0) {
            for (int s = 0; s < C::S; ++s) {
                bar_init(&sh.full[s], 1);
                bar_init(&sh.empty[s], 1);
            }
            bar_init(&sh.qfull, 1);
            bar_init(&sh.qempty, 1);
            for (int w = 0; w < 2; ++w) {
                bar_init(&sh.sfull[w], 1);
                bar_init(&sh.pready[w], 4);
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
        sh.start_u = 0x7fffffffffffffffll;
        sh.start_b = sh.start_g = sh.start_row0 = sh.start_off = 0;
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
    const int G = (int)min((long long)gridDim.x, U);   // blocks with work
    const int blk = blockIdx.x;
    const long long u0 = G > 0 ? U * blk / G : 0, u1 = G > 0 ? U * (blk + 1) / G : 0;
    const bool work = blk < G;
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
            const int g = (int)(left / u);
            left -= g * u;
            int row0 = 0, rows, lo, hi;
            for (;; row0 += kRows) {
                const int nt = item_tiles(a, r, row0, &rows, &lo, &hi);
                if (left < nt) break;
                left -= nt;
            }
            sh.start_u = u0;
            sh.start_b = b;
            sh.start_g = g;
            sh.start_row0 = row0;
            sh.start_off = (int)left;
            break;
        }
    }
    fence_async_smem();   // the scratch in the ring, before copies land there
    __syncthreads();
    const Ctl ctl{a.status, a.timeout_ns, &sh.abort_flag};
    if (work) {
        // 384 threads x 168 registers at launch = 256 x 208 + 128 x 88
        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
            softmax_role<T, DH>(a, sh, tmem, ctl);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
            if (warp == 8)
                tile_role<DH>(a, sh, ring, ctl);
            else if (warp == 9)
                mma_role<T, DH>(a, sh, qs, ring, tmem, ctl);
            else if (warp == 10)
                query_role<T, DH>(a, sh, qs, ctl);
            else if (lane == 0)
                list_role<DH>(a, sh, u1, U, G, ctl);
        }
    }
    tc_before();
    __syncthreads();
    if (warp == 9) {
        tc_after();
        tmem_free(tmem, 512);
    }
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
        const long long need = (long long)d.max_new * (d.heads / c.kv_heads);
        rows = (int)std::min<long long>(kRows, (need + 31) / 32 * 32);
        auto up = [](size_t v) { return (v + 255) / 256 * 256; };
        ml = up((size_t)blocks * 8 * sizeof(int));
        o = up(ml + (size_t)blocks * 2 * 2 * rows * 2 * sizeof(float));
        total = up(o + (size_t)blocks * 2 * c.head_dim * rows * sizeof(float));
    }
};

bool cache_map(CUtensorMap* m, const void* base, const pi_page_desc& c) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads,
                                (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride * 2, (cuuint64_t)c.head_stride * 2,
                                   (cuuint64_t)c.page_stride * 2};
    const cuuint32_t box[4] = {64u, (cuuint32_t)c.page_size, 1u, 1u};
    const cuuint32_t es[4] = {1u, 1u, 1u, 1u};
    return fn(m, c.dtype == PI_T_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
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
    a.window = desc->window;
    a.page_size = cache->page_size;
    a.num_pages = cache->num_pages;
    a.group = desc->heads / cache->kv_heads;
    a.part_rows = lay.rows;
    a.scale = desc->scale > 0.f ? desc->scale : 1.0f / sqrtf((float)cache->head_dim);
    a.counters = reinterpret_cast<int*>(ws);
    a.part_ml = reinterpret_cast<float*>(ws + lay.ml);
    a.part_o = reinterpret_cast<float*>(ws + lay.o);
    a.status = status_word();
    a.timeout_ns = wait_timeout_ns();
    if (blocks < 1 || a.status == nullptr || !cache_map(&a.kmap, kcache, *cache) || !cache_map(&a.vmap, vcache, *cache))
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
