// pi_paged8.cu -- the paged cache in 8 bits: rotary positions and the store of
// keys and values as e4m3 codes with an exponent for each block of 16 positions
// and head, and rows read back from it.  The attention over it is in
// pi_paged8_attn.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "pi_common.cuh"
#include "pi_e4m3.cuh"
#include "pi_internal.h"
#include "pi_pipe.cuh"

namespace pi {
namespace {

using namespace e4m3;

// ------------------------------------------------ rotary positions and quantised store
//
// One launch: blocks for keys and values first, then blocks for queries.
//
// Keys and values: a block looks at a window of 1, 4 or 16 tokens, each warp for one KV
// head and array (keys or values).  A token that is the first new one of its block of
// positions stands for all of the block's new tokens, up to 16 rows from it on: the warp
// asks for them all, then takes the largest magnitude, the exponent, the earlier positions'
// codes again where it grew, and the new codes.  A lane holds 4 elements of a token that
// turn together: two pairs (i, i + rot / 2) in the half layout, 4 in a row when interleaved
// or past rot_dim.  The tokens' cos and sin are computed once for the block's heads.
//
// Queries: as pi_rope_store takes them, units of 8 pairs (or 16 elements), the same bits.
//
// 32 decoding tokens (64 + 2 x 8 heads, fp16): 4.4 us, a launch and a chain of three loads.
// 1999 fp32 tokens (32 + 2 x 32 heads): 33 us, 4.0 TB/s; 16384 bf16 tokens: 119 us, 5.3 TB/s,
// 84 of them the queries'.  The keys' and values' 33 us (100 MB) are instructions: 1450 of a
// warp for 16 rows, two thirds of the issue slots, the rows read twice from shared memory (with
// the rows in registers 37 us: two blocks on an SM) and cos and sin a fifth.
constexpr int kStoreWarps = 8, kStoreThreads = 32 * kStoreWarps;
constexpr int kWindow = 16;              // tokens of a window at most
constexpr int kQueryUnits = 2;           // units of a thread whose loads are in flight together
constexpr int kQueryTokens = 16;         // tokens of a block at most
// More blocks of queries than this go through pi_rope_store's kernel, in a launch of their
// own: here they share registers and shared memory with the keys' and values' blocks, three
// of which fit an SM (by registers; of fp32 rows of 128 elements two, by shared memory).  64 + 2 x 8 heads: 32 tokens 4.4 us in one launch, 7.0 in two; 1024
// decoding rows 17 and 21, 16384 prompt tokens 145 and 120.
constexpr int kQueryBlocks = 4096;

struct Store8Args {
    const void *q, *k, *v;
    const int32_t* positions;
    const int64_t* slots;
    void* q_out;
    uint8_t *kc, *vc;
    int8_t *ke, *ve;
    long long q_stride, k_stride, v_stride, out_stride, page_stride, head_stride, token_stride, num_slots;
    int tokens, heads, kv_heads, dh, page_shift;
    int kv_blocks, window, shares;       // blocks for keys and values; tokens of a window; blocks of a window
    int q_tokens;                        // tokens of a block for queries
    int* status;
    pi_rope_plan plan;
};

template <typename T>
PI_DEV float2 widen_pair(uint32_t w);
template <>
PI_DEV float2 widen_pair<__half>(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
template <>
PI_DEV float2 widen_pair<__nv_bfloat16>(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
// two elements in a row
template <typename T>
PI_DEV float2 pair_at(const T* p) { return widen_pair<T>(*reinterpret_cast<const uint32_t*>(p)); }
PI_DEV float2 pair_at(const float* p) { return *reinterpret_cast<const float2*>(p); }

// cos and sin of position x turns in fixed point: the top 32 bits of the turn's
// fraction are a signed fraction of a half turn; what fp32 does not hold of them
// enters to first order, so that the angle is off by 2^-31 half turns.
PI_DEV float2 turn_of(int position, unsigned long long turns, float mscale) {
    const int a = (int)((unsigned long long)(long long)position * turns >> 32);
    const float f = (float)a;
    // a - f: f is a multiple of 2^7 or more wherever it is not a itself, so the low bits tell
    const int whole = f >= 2147483648.f ? (int)0x80000000u : (int)f;   // (2^31 as -2^31: the difference wraps back)
    const float rest = (float)(int)((unsigned)a - (unsigned)whole) * (3.14159265358979f / 2147483648.0f);
    float s, c;
    sincospif(f * (1.0f / 2147483648.0f), &s, &c);
    return make_float2(fmaf(-s, rest, c) * mscale, fmaf(c, rest, s) * mscale);
}

template <typename I, int DH>
PI_DEV void store_codes(const Store8Args& a, float2* table, unsigned long long* turns, I* all_rows) {
    constexpr int LANES = DH / 4;   // lanes of a token: 32 or 16
    constexpr int SIDE = 32 / LANES;   // tokens side by side
    const int tid = threadIdx.x, lane = tid & 31;
    const int share = blockIdx.x % a.shares, t0 = blockIdx.x / a.shares * a.window;
    const int work = share * kStoreWarps + (tid >> 5);
    const bool idle = work >= 2 * a.kv_heads, values = work >= a.kv_heads;
    const int h = values ? work - a.kv_heads : work, half = a.plan.rot_dim / 2;
    // lane i: the slot of token t0 - 1 + i
    long long mine = -2;
    if (t0 - 1 + lane >= 0 && t0 - 1 + lane < a.tokens) mine = a.slots[t0 - 1 + lane];
    if (tid < half) turns[tid] = a.plan.turns[tid];
    const bool in_cache = mine >= 0 && mine < a.num_slots;
    const bool window = lane >= 1 && lane <= a.window && t0 - 1 + lane < a.tokens;
    if (window && !in_cache && mine != -1 && share == 0 && tid < 32) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
    const long long before = __shfl_up_sync(FULL, mine, 1);
    const bool follows = lane >= 1 && in_cache && (mine & (kBlock - 1)) != 0 && before == mine - 1;
    const unsigned chain = __ballot_sync(FULL, follows);
    unsigned heads = __ballot_sync(FULL, window && in_cache && !follows);   // first new tokens of their blocks
    if (heads == 0) return;
    // new tokens of the block that the token at lane i begins
    auto count_at = [&](int i) { return __ffs(~(chain >> i >> 1)); };
    const int first = __ffs(heads) - 1, last = 31 - __clz(heads), end = last + count_at(last);

    const int sub = lane / LANES, l = lane % LANES;
    const bool apart = !values && !a.plan.interleaved && 2 * l < half;
    const int e0 = apart ? 2 * l : 4 * l, e1 = apart ? half + 2 * l : 4 * l + 2;
    // (pairs from half on pass through: 2 l >= half there, so 4 l >= rot_dim)
    const bool turn = !values && 2 * l < half;
    const void* const src = values ? a.v : a.k;
    const long long stride = values ? a.v_stride : a.k_stride;
    I* const rows = all_rows + (tid >> 5) * kBlock * DH;   // this warp's
    auto ask = [&](int at) {
        constexpr int PIECES = DH * (int)sizeof(I) / 16;   // of a row
        const I* const from = static_cast<const I*>(src) + (long long)(t0 - 1 + at) * stride + (long long)h * DH;
        for (int i = lane; i < count_at(at) * PIECES; i += 32)
            pipe::cp16(reinterpret_cast<unsigned char*>(rows) + i * 16, reinterpret_cast<const unsigned char*>(from + (i / PIECES) * stride) + i % PIECES * 16);
        pipe::cp_commit();
    };
    if (!idle) ask(first);
    // cos and sin of the window's tokens, while those are on their way
    if (half > 0 && share * kStoreWarps < a.kv_heads) {
        __syncthreads();
        for (int i = tid; i < (end - first) * half; i += kStoreThreads) {
            const int t = i / half, p = i - t * half;
            table[t * (DH / 2) + p] = turn_of(a.positions[t0 - 1 + first + t], turns[p], a.plan.mscale);
        }
        __syncthreads();
    }
    if (idle) return;
    for (;;) {
        const int at = __ffs(heads) - 1, count = count_at(at);
        heads &= heads - 1;
        const long long slot = __shfl_sync(FULL, mine, at);
        const int r = (int)(slot & (kBlock - 1)), in_page = (int)(slot & ((1 << a.page_shift) - 1)) - r;
        const long long page = slot >> a.page_shift;
        uint8_t* const codes = (values ? a.vc : a.kc) + page * a.page_stride + h * a.head_stride + in_page * a.token_stride;
        int8_t* const exp_at = (values ? a.ve : a.ke) + ((page * a.kv_heads + h) << (a.page_shift - 4)) + in_page / kBlock;
        const int old = r > 0 ? bounded(*exp_at) : kMinExp;
        pipe::cp_wait<0>();
        __syncwarp();
        // this lane's elements of a row, turned
        auto turned = [&](int row, float (&x)[4]) {
            const float2 u = pair_at(rows + row * DH + e0), v = pair_at(rows + row * DH + e1);
            x[0] = u.x;
            x[1] = u.y;
            x[2] = v.x;
            x[3] = v.y;
            if (turn) {
                const float4 cs = *reinterpret_cast<const float4*>(table + (at - first + row) * (DH / 2) + 2 * l);
                if (apart) {   // (0, 2) and (1, 3)
                    x[0] = u.x * cs.x - v.x * cs.y;
                    x[2] = v.x * cs.x + u.x * cs.y;
                    x[1] = u.y * cs.z - v.y * cs.w;
                    x[3] = v.y * cs.z + u.y * cs.w;
                } else {       // (0, 1) and (2, 3)
                    x[0] = u.x * cs.x - u.y * cs.y;
                    x[1] = u.y * cs.x + u.x * cs.y;
                    x[2] = v.x * cs.z - v.y * cs.w;
                    x[3] = v.y * cs.z + v.x * cs.w;
                }
            }
        };
        float top = 0.f, odd = 0.f;   // odd: 0, or NaN where some element is not finite
#pragma unroll 4
        for (int row = sub; row < count; row += SIDE) {
            float x[4];
            turned(row, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                top = fmaxf(top, fabsf(x[e]));
                odd = fmaf(x[e], 0.f, odd);
            }
        }
        const bool some = __any_sync(FULL, odd != 0.f);   // infinities and NaN count as NaN, and not for the exponent
        if (some) {
            top = 0.f;
            for (int row = sub; row < count; row += SIDE) {
                float x[4];
                turned(row, x);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (fabsf(x[e]) < INFINITY) top = fmaxf(top, fabsf(x[e]));
            }
        }
        const int e = max(exponent_of(__reduce_max_sync(FULL, __float_as_uint(top))), old);
        if (r > 0 && e > old) {
            // the earlier positions' codes, 16 at a time
            const float f = pow2(old - e);
            for (int i = lane; i < r * (DH / 16); i += 32) {
                uint4* const w = reinterpret_cast<uint4*>(codes + (i / (DH / 16)) * a.token_stride + i % (DH / 16) * 16);
                uint4 c = *w;
                auto again = [&](uint32_t y) {
                    const float2 u = values2(y & 0xffffu), v = values2(y >> 16);
                    return encode2(u.x * f, u.y * f) | encode2(v.x * f, v.y * f) << 16;
                };
                c = make_uint4(again(c.x), again(c.y), again(c.z), again(c.w));
                *w = c;
            }
        }
        const float f = pow2(-e);
        uint8_t* to = codes + (r + sub) * a.token_stride;
#pragma unroll 4
        for (int row = sub; row < count; row += SIDE, to += SIDE * a.token_stride) {
            float x[4];
            turned(row, x);
            if (some)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = fabsf(x[e]) < INFINITY ? x[e] : NAN;
            const uint32_t lo = encode2(x[0] * f, x[1] * f), hi = encode2(x[2] * f, x[3] * f);
            if (apart) {
                *reinterpret_cast<uint16_t*>(to + e0) = (uint16_t)lo;
                *reinterpret_cast<uint16_t*>(to + e1) = (uint16_t)hi;
            } else {
                *reinterpret_cast<uint32_t*>(to + e0) = lo | hi << 16;
            }
        }
        if (lane == 0) *exp_at = (int8_t)e;
        if (heads == 0) return;
        __syncwarp();   // the rows have been read
        ask(__ffs(heads) - 1);
    }
}

// 8 elements in a row, and back to 16 bits.
template <typename T>
struct Eight {
    uint4 w;
    PI_DEV void load(const void* base, long long at) { w = ld_stream16(static_cast<const T*>(base) + at); }
    PI_DEV void get(float (&f)[8]) const {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 u = widen_pair<T>(x[i]);
            f[2 * i] = u.x;
            f[2 * i + 1] = u.y;
        }
    }
};
template <>
struct Eight<float> {
    uint4 w[2];
    PI_DEV void load(const void* base, long long at) {
        w[0] = ld_stream16(static_cast<const float*>(base) + at);
        w[1] = ld_stream16(static_cast<const float*>(base) + at + 4);
    }
    PI_DEV void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i] = __uint_as_float(w[i].x);
            f[4 * i + 1] = __uint_as_float(w[i].y);
            f[4 * i + 2] = __uint_as_float(w[i].z);
            f[4 * i + 3] = __uint_as_float(w[i].w);
        }
    }
};
PI_DEV uint32_t pack_pair(float x, float y, __half) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
PI_DEV uint32_t pack_pair(float x, float y, __nv_bfloat16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename O>
PI_DEV void put8(O* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_pair(f[0], f[1], O()), pack_pair(f[2], f[3], O()), pack_pair(f[4], f[5], O()), pack_pair(f[6], f[7], O()));
}

template <typename I, typename O>
PI_DEV void turn_queries(const Store8Args& a, float2* table, unsigned long long* turns) {
    const int tid = threadIdx.x, half = a.plan.rot_dim / 2, turning = a.plan.rot_dim / 16, per_head = a.dh / 16;
    const int t0 = (blockIdx.x - a.kv_blocks) * a.q_tokens, n = min(a.q_tokens, a.tokens - t0);
    const int units = a.heads * per_head, all = n * units;
    // where a unit comes from: its token's row and the offsets of its two runs of 8
    auto runs = [&](int u, int* t, int* hu, int* r0, int* r1) {
        *t = u / units;
        const int x = u - *t * units, h = x / per_head;
        *hu = x - h * per_head;
        const bool split = *hu < turning && !a.plan.interleaved;
        *r0 = h * a.dh + (split ? 8 * *hu : 16 * *hu);
        *r1 = h * a.dh + (split ? half + 8 * *hu : 16 * *hu + 8);
    };
    Eight<I> raw[kQueryUnits][2];
    auto ask = [&](int u0) {
#pragma unroll
        for (int i = 0; i < kQueryUnits; ++i) {
            int t, hu, r0, r1;
            if (u0 + i * kStoreThreads >= all) break;
            runs(u0 + i * kStoreThreads, &t, &hu, &r0, &r1);
            const long long row = (long long)(t0 + t) * a.q_stride;
            raw[i][0].load(a.q, row + r0);
            raw[i][1].load(a.q, row + r1);
        }
    };
    ask(tid);
    if (half > 0) {
        if (tid < half) turns[tid] = a.plan.turns[tid];
        __syncthreads();
        for (int i = tid; i < n * half; i += kStoreThreads) {
            const int t = i / half, p = i - t * half;
            // (as pi_rope_store: the angle's top 32 bits as fp32)
            const unsigned long long turn = (unsigned long long)(long long)a.positions[t0 + t] * turns[p];
            float s, c;
            sincospif((float)(int)(turn >> 32) * (1.0f / 2147483648.0f), &s, &c);
            table[t * (a.dh / 2) + p] = make_float2(c * a.plan.mscale, s * a.plan.mscale);
        }
        __syncthreads();
    }
    for (int u0 = tid; u0 < all; u0 += kQueryUnits * kStoreThreads) {
        if (u0 != tid) ask(u0);
#pragma unroll
        for (int i = 0; i < kQueryUnits; ++i) {
            if (u0 + i * kStoreThreads >= all) break;
            int t, hu, r0, r1;
            runs(u0 + i * kStoreThreads, &t, &hu, &r0, &r1);
            float x[8], y[8];
            raw[i][0].get(x);
            raw[i][1].get(y);
            if (hu < turning) {
                const float2* const cs = table + t * (a.dh / 2) + 8 * hu;
                if (a.plan.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 p = cs[e], r = cs[4 + e];
                        const float x1 = x[2 * e], x2 = x[2 * e + 1], y1 = y[2 * e], y2 = y[2 * e + 1];
                        x[2 * e] = x1 * p.x - x2 * p.y;
                        x[2 * e + 1] = x2 * p.x + x1 * p.y;
                        y[2 * e] = y1 * r.x - y2 * r.y;
                        y[2 * e + 1] = y2 * r.x + y1 * r.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 p = cs[e];
                        const float x1 = x[e], x2 = y[e];
                        x[e] = x1 * p.x - x2 * p.y;
                        y[e] = x2 * p.x + x1 * p.y;
                    }
                }
            }
            O* const dst = static_cast<O*>(a.q_out) + (long long)(t0 + t) * a.out_stride;
            put8(dst + r0, x);
            put8(dst + r1, y);
        }
    }
}

template <typename I, typename O, int DH>
__global__ void __launch_bounds__(kStoreThreads, 3) k_rope_store8(const __grid_constant__ Store8Args a) {
    pdl_entry();
    extern __shared__ __align__(16) unsigned char store_rows[];   // a block's rows of each warp
    __shared__ __align__(16) float2 table[(2 * kWindow - 1) * (DH / 2)];
    __shared__ unsigned long long turns[DH / 2];
    if ((int)blockIdx.x < a.kv_blocks) store_codes<I, DH>(a, table, turns, reinterpret_cast<I*>(store_rows));
    else turn_queries<I, O>(a, table, turns);
}

// ------------------------------------------------ rows read back
//
// A block takes up to 32 rows: a lane each finds its row's request (binary search in
// cu_rows) and page, then all threads move 8 codes at a time, four times of a thread in flight.
// Bound by HBM: 48 requests of 100-8000 positions (8 heads of 128, bf16) 150 us, 6.4 TB/s; 1001
// rows of 12 heads of 64 take 5-7 us, a chain of four loads (and a call 9 on the host).
constexpr int kReadRows = 32;
constexpr int kReadBlocks = 4 * 152;   // rows are shared out over this many blocks (four on each SM), where there are enough

struct Read8Args {
    Cache8 c;
    const int32_t *table, *start, *cu;
    void *k_out, *v_out;
    long long k_stride, v_stride;
    int batch, max_pages, max_rows, rows;   // rows of a block
    int head_shift, per_row;                 // pieces of 8 codes: of a head (log2), of a row
    int* status;
};

// values of 8 codes times `scale`, rounded to the output's type: 16 bytes of a 16-bit one, so
// that a warp's stores fill whole sectors (16 codes of a thread, two stores of every other 16
// bytes each: 16384 rows of 2 x 8 heads 27 us, so 17)
PI_DEV void values8(const uint2& c, float scale, float (&f)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 u = values2(w[i] & 0xffffu), v = values2(w[i] >> 16);
        f[4 * i] = u.x * scale;
        f[4 * i + 1] = u.y * scale;
        f[4 * i + 2] = v.x * scale;
        f[4 * i + 3] = v.y * scale;
    }
}
PI_DEV void put_values(__half* p, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)   // past 65504: the largest (a comparison keeps NaN)
        if (fabsf(f[i]) > 65504.f) f[i] = copysignf(65504.f, f[i]);
    put8(p, f);
}
PI_DEV void put_values(__nv_bfloat16* p, float (&f)[8]) { put8(p, f); }
PI_DEV void put_values(float* p, float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

template <typename O>
__global__ void __launch_bounds__(256) k_page_read8(const __grid_constant__ Read8Args a) {
    pdl_entry();
    __shared__ long long code_at[kReadRows], exp_at[kReadRows];   // -1: zeros, -2: no row
    const int row0 = blockIdx.x * a.rows, row = row0 + threadIdx.x;
    const bool mine = (int)threadIdx.x < a.rows && row < a.max_rows;
    auto holds = [&](int b) {   // request b is consistent, and the row one of its
        const int first = a.cu[b], end = a.cu[b + 1];
        return first >= 0 && first <= row && row < end && end <= a.max_rows;
    };
    auto find = [&](int b) {    // where the row's codes are, as one of request b's
        const long long pos = (long long)(a.start ? a.start[b] : 0) + (row - a.cu[b]);
        long long code = -1, ex = 0;
        if (pos >= 0 && pos < (long long)a.max_pages << a.c.page_shift) {
            const int id = a.table[(size_t)b * a.max_pages + (size_t)(pos >> a.c.page_shift)];
            const int in_page = (int)(pos & ((1 << a.c.page_shift) - 1));
            if (id >= 0 && id < a.c.num_pages) {
                code = id * a.c.page_stride + in_page * a.c.token_stride;
                ex = ((long long)id * a.c.kv_heads << (a.c.page_shift - 4)) + in_page / kBlock;
            }
        }
        if (code < 0) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
        code_at[threadIdx.x] = code;
        exp_at[threadIdx.x] = ex;
    };
    bool open = false;   // a row whose request is not found
    if (mine) {
        // the last request that starts at or before the row
        int lo = 0, hi = a.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.cu[mid] <= row) lo = mid;
            else hi = mid;
        }
        open = !holds(lo);
        if (!open) find(lo);
    }
    if ((int)threadIdx.x < a.rows && (!mine || open)) code_at[threadIdx.x] = -2;
    if (__syncthreads_or(open) || blockIdx.x == 0) {
        bool bad = false;
        for (int b = threadIdx.x; b < a.batch; b += 256) bad |= a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.max_rows;
        if (__syncthreads_or(bad)) {
            // cu_rows is not in order everywhere, and the search may have missed: one by one
            if (bad) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
            for (int b = 0; open && b < a.batch; ++b)
                if (holds(b)) {
                    find(b);
                    open = false;
                }
            __syncthreads();
        }
    }
    // a thread keeps its piece of the rows (of keys or values) and goes from row to row
    const int first_array = a.k_out ? 0 : 1, pieces = ((a.k_out ? 1 : 0) + (a.v_out ? 1 : 0)) * a.per_row;
    const int beside = max(1, 256 / pieces), r0 = pieces < 256 ? threadIdx.x / pieces : 0;   // rows that a pass takes
    for (int i = threadIdx.x - r0 * pieces; i < pieces && r0 < beside; i += 256) {
        const bool values = i >= a.per_row || first_array == 1;
        const int piece = i >= a.per_row ? i - a.per_row : i, h = piece >> a.head_shift;
        const uint8_t* const codes = (values ? a.c.v : a.c.k) + h * a.c.head_stride + (piece & ((1 << a.head_shift) - 1)) * 8;
        const int8_t* const exps = (values ? a.c.ve : a.c.ke) + ((long long)h << (a.c.page_shift - 4));
        const long long stride = values ? a.v_stride : a.k_stride;
        O* to = static_cast<O*>(values ? a.v_out : a.k_out) + (row0 + r0) * stride + piece * 8;
        for (int r = r0; r < a.rows; r += 4 * beside) {
            uint2 c[4];
            int e[4];
            long long at[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int row = r + x * beside;
                at[x] = row < a.rows ? code_at[row] : -2;
                c[x] = make_uint2(0u, 0u);
                e[x] = 0;
                if (at[x] >= 0) {
                    c[x] = ld_stream8(codes + at[x]);
                    e[x] = exps[exp_at[row]];
                }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x, to += beside * stride) {
                if (at[x] == -2) continue;
                float f[8];
                values8(c[x], pow2(bounded(e[x])), f);
                put_values(to, f);
            }
        }
    }
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename I, typename O, int DH>
cudaError_t launch_store8(const Store8Args& a, unsigned blocks, cudaStream_t s) {
    static std::mutex mu;
    static bool done[64] = {};
    constexpr int smem = kStoreWarps * kBlock * DH * (int)sizeof(I);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            e = cudaFuncSetAttribute(k_rope_store8<I, O, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    return launch_pdl(k_rope_store8<I, O, DH>, blocks, kStoreThreads, a.kv_blocks > 0 ? smem : 0, s, a);
}
template <typename I, typename O>
cudaError_t launch_store8(const Store8Args& a, cudaStream_t s) {
    const int q_blocks = a.heads > 0 ? (a.tokens + a.q_tokens - 1) / a.q_tokens : 0;
    const unsigned blocks = (unsigned)(a.kv_blocks + q_blocks);
    return a.dh == 128 ? launch_store8<I, O, 128>(a, blocks, s) : launch_store8<I, O, 64>(a, blocks, s);
}
template <typename I>
cudaError_t launch_store8(const Store8Args& a, int out_dtype, cudaStream_t s) {
    return out_dtype == PI_T_F16 ? launch_store8<I, __half>(a, s) : launch_store8<I, __nv_bfloat16>(a, s);
}

}  // namespace

bool page8_desc_ok(const pi_page8_desc& c) {
    if (c.kv_heads < 1 || c.kv_heads > 1024 || (c.head_dim != 64 && c.head_dim != 128) ||
        (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128) || c.num_pages < 1 ||
        c.num_pages > (1 << 26))
        return false;
    for (long long s : {c.page_stride, c.head_stride, c.token_stride})
        if (s < c.head_dim || s % 16 != 0 || s > (1ll << 36)) return false;
    return true;
}

}  // namespace pi

using namespace pi;

extern "C" {

pi_status pi_rope_store8(const pi_rope_plan* plan, const pi_page8_desc* cache, const pi_qkv_desc* desc, int out_dtype,
                         const void* q, const void* k, const void* v, const int32_t* positions, const int64_t* slots,
                         void* q_out, void* kcache, void* vcache, int8_t* kexp, int8_t* vexp, void* stream) {
    if (!plan || !cache || !desc || !page8_desc_ok(*cache) || (out_dtype != PI_T_F16 && out_dtype != PI_T_BF16))
        return PI_ERR_INVALID_ARG;
    const pi_qkv_desc& d = *desc;
    if (plan->head_dim != cache->head_dim || plan->rot_dim < 0 || plan->rot_dim > plan->head_dim ||
        plan->rot_dim % 16 != 0 || (plan->interleaved != 0 && plan->interleaved != 1))
        return PI_ERR_INVALID_ARG;
    if (d.tokens < 0 || d.tokens > (1 << 24) || d.heads < 1 || d.heads > 1024 || d.dtype < PI_T_F16 ||
        d.dtype > PI_T_F32)
        return PI_ERR_INVALID_ARG;
    const bool has_q = q || q_out, has_kv = k || v || kcache || vcache || kexp || vexp || slots;
    if (!has_q && !has_kv) return d.tokens == 0 ? PI_OK : PI_ERR_INVALID_ARG;   // (empty tensors have no address)
    auto stride_ok = [&](long long s, int heads) {
        return s % 8 == 0 && s >= (long long)heads * cache->head_dim && s <= (1ll << 36);
    };
    if (has_q && !(stride_ok(d.q_stride, d.heads) && stride_ok(d.out_stride, d.heads))) return PI_ERR_INVALID_ARG;
    if (has_kv && !(stride_ok(d.k_stride, cache->kv_heads) && stride_ok(d.v_stride, cache->kv_heads)))
        return PI_ERR_INVALID_ARG;
    if (d.tokens == 0) return PI_OK;
    if (!positions || !aligned(positions, 4)) return PI_ERR_INVALID_ARG;
    if (has_q && (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16))) return PI_ERR_INVALID_ARG;
    if (has_kv && (!k || !v || !kcache || !vcache || !kexp || !vexp || !slots || !aligned(k, 16) || !aligned(v, 16) ||
                   !aligned(kcache, 16) || !aligned(vcache, 16) || !aligned(slots, 8)))
        return PI_ERR_INVALID_ARG;
    // Rotated queries go over no input that another thread may still have to
    // read.  In place a thread reads all it writes first, if the elements lie alike.
    const long long in = d.dtype == PI_T_F32 ? 4 : 2, q_width = (long long)d.heads * cache->head_dim,
                    k_width = (long long)cache->kv_heads * cache->head_dim;
    auto over = [&](const void* x, long long stride, long long width) {
        return rows_overlap(x, in * stride, in * width, q_out, 2 * d.out_stride, 2 * q_width, d.tokens);
    };
    const bool in_place = q == q_out && d.dtype == out_dtype && d.q_stride == d.out_stride;
    if (has_q && ((!in_place && over(q, d.q_stride, q_width)) ||
                  (has_kv && (over(k, d.k_stride, k_width) || over(v, d.v_stride, k_width)))))
        return PI_ERR_INVALID_ARG;
    Store8Args a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.kc = static_cast<uint8_t*>(kcache);
    a.vc = static_cast<uint8_t*>(vcache);
    a.ke = kexp;
    a.ve = vexp;
    a.q_stride = d.q_stride;
    a.k_stride = d.k_stride;
    a.v_stride = d.v_stride;
    a.out_stride = d.out_stride;
    a.page_stride = cache->page_stride;
    a.head_stride = cache->head_stride;
    a.token_stride = cache->token_stride;
    a.num_slots = (long long)cache->num_pages * cache->page_size;
    a.tokens = d.tokens;
    a.heads = has_q ? d.heads : 0;
    a.kv_heads = has_kv ? cache->kv_heads : 0;
    a.dh = cache->head_dim;
    a.page_shift = __builtin_ctz((unsigned)cache->page_size);
    a.status = status_word();
    a.plan = *plan;
    if (a.status == nullptr) return PI_ERR_CUDA;
    // Windows of one token while that many blocks run at once (four on each of 152 SMs), of 16
    // where there are many: tokens of a prompt share blocks of positions, and one in 16 begins one.  Windows of 1, 4
    // and 16, two blocks a window: 64 decoding rows 4.9, 7.5 and 21 us, 512 12.6, 10.8 and 23,
    // 4096 68, 58 and 67; eight blocks a window: a chunk of 1999 tokens 73, 42 and 35.
    a.shares = std::max(1, (2 * a.kv_heads + kStoreWarps - 1) / kStoreWarps);
    const long long ones = (long long)d.tokens * a.shares;
    a.window = ones <= 608 ? 1 : ones <= 8192 ? 4 : kWindow;
    a.kv_blocks = has_kv ? (int)((d.tokens + a.window - 1) / a.window) * a.shares : 0;
    a.q_tokens = has_q ? std::min(kQueryTokens, std::max(1, kQueryUnits * kStoreThreads / (d.heads * (a.dh / 16)))) : 1;
    if (a.heads > 0 && (d.tokens + a.q_tokens - 1) / a.q_tokens > kQueryBlocks) {
        const int dh = cache->head_dim;
        const pi_page_desc rows{1, dh, cache->page_size, 1, out_dtype, (long long)dh * cache->page_size,
                                (long long)dh * cache->page_size, dh};
        const pi_status st = pi_rope_store(plan, &rows, desc, q, nullptr, nullptr, positions, nullptr, q_out, nullptr,
                                           nullptr, stream);
        if (st != PI_OK || !has_kv) return st;
        a.heads = 0;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d.dtype == PI_T_F16    ? launch_store8<__half>(a, out_dtype, s)
                          : d.dtype == PI_T_BF16 ? launch_store8<__nv_bfloat16>(a, out_dtype, s)
                                                 : launch_store8<float>(a, out_dtype, s);
    return e == cudaSuccess ? PI_OK : PI_ERR_CUDA;
}

pi_status pi_page_read8(const pi_read8_desc* desc, const pi_page8_desc* cache, const void* kcache, const void* vcache,
                        const int8_t* kexp, const int8_t* vexp, const int32_t* block_table, const int32_t* start,
                        const int32_t* cu_rows, void* k_out, void* v_out, void* stream) {
    if (!desc || !cache || !page8_desc_ok(*cache)) return PI_ERR_INVALID_ARG;
    const pi_read8_desc& d = *desc;
    if (d.batch < 1 || d.batch > 4096 || d.max_pages < 1 || (long long)d.max_pages * cache->page_size > (1ll << 30) ||
        d.max_rows < 0 || d.max_rows > (1 << 30) || d.dtype < PI_T_F16 || d.dtype > PI_T_F32)
        return PI_ERR_INVALID_ARG;
    if (d.max_rows == 0) return PI_OK;   // (empty tensors have no address)
    const long long width = (long long)cache->kv_heads * cache->head_dim;
    auto array_ok = [&](const void* codes, const void* exps, const void* out, long long stride) {
        if (!out) return !codes && !exps;
        return codes && exps && aligned(codes, 16) && aligned(out, 16) && stride % 8 == 0 && stride >= width && stride <= (1ll << 36);
    };
    if (!array_ok(kcache, kexp, k_out, d.k_stride) || !array_ok(vcache, vexp, v_out, d.v_stride) || (!k_out && !v_out))
        return PI_ERR_INVALID_ARG;
    if (!block_table || !cu_rows || !aligned(block_table, 4) || !aligned(cu_rows, 4) || !aligned(start, 4))
        return PI_ERR_INVALID_ARG;
    const long long size = d.dtype == PI_T_F32 ? 4 : 2;
    if (rows_overlap(k_out, size * d.k_stride, size * width, v_out, size * d.v_stride, size * width, d.max_rows))
        return PI_ERR_INVALID_ARG;
    Read8Args a{};
    a.c = Cache8{static_cast<const uint8_t*>(kcache), static_cast<const uint8_t*>(vcache), kexp, vexp, cache->page_stride,
                 cache->head_stride, cache->token_stride, cache->kv_heads, __builtin_ctz((unsigned)cache->page_size),
                 cache->num_pages};
    a.table = block_table;
    a.start = start;
    a.cu = cu_rows;
    a.k_out = k_out;
    a.v_out = v_out;
    a.k_stride = d.k_stride;
    a.v_stride = d.v_stride;
    a.batch = d.batch;
    a.max_pages = d.max_pages;
    a.max_rows = d.max_rows;
    a.head_shift = cache->head_dim == 128 ? 4 : 3;
    a.per_row = cache->kv_heads << a.head_shift;
    a.status = status_word();
    if (a.status == nullptr) return PI_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.rows = std::min(kReadRows, std::max(1, d.max_rows / kReadBlocks));
    const unsigned blocks = (unsigned)((d.max_rows + (long long)a.rows - 1) / a.rows);
    const cudaError_t e = d.dtype == PI_T_F16    ? launch_pdl(k_page_read8<__half>, blocks, 256, 0, s, a)
                          : d.dtype == PI_T_BF16 ? launch_pdl(k_page_read8<__nv_bfloat16>, blocks, 256, 0, s, a)
                                                 : launch_pdl(k_page_read8<float>, blocks, 256, 0, s, a);
    return e == cudaSuccess ? PI_OK : PI_ERR_CUDA;
}

}  // extern "C"
