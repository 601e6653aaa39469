// pi_paged.cu -- block tables and slot maps from request lengths, and rotary
// positions with the store into a paged key/value cache, with their entry
// points.  The attention over that cache is in pi_paged_attn.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "pi_common.cuh"
#include "pi_internal.h"

namespace pi {
namespace {

// ------------------------------------------------------------- block tables
//
// All rows' page needs are known from the lengths alone, so the whole step is
// three prefix sums over the rows (tokens, pages given back, pages wanted) and
// then independent writes: pushed page i, popped page i, token i each find
// their row by binary search in a prefix.  The stack after the pushes is never
// read back: entry x of it is free_list[x] below the old count, else released
// page x - count, still in its row's table entry (releasing rows' entries are
// not overwritten, free-list entries below the old count are not written).
//
// Bound by latency, the chain from lengths over prefixes to table entries and
// slots: 4.7 us for 8 decoding rows, 10.8 us for 2048 rows with 42 thousand
// tokens (1.6 MB, 0.24 us of HBM).  Every block scans all rows
// (three block prefixes) and takes its share of the writes.  Small steps are
// one block.  Large ones are two grids: kTabMoves, as wide as the writes need,
// writes pages, slots and positions; kTabState, one block, writes held_out and
// free_count_out, which may alias the inputs, and the other per-row outputs.
// The second is a programmatic dependent of the first, which lets it go only
// once each of its blocks has read all inputs; so it may overwrite them while
// the first still writes, and waits for the first's end at its own.
constexpr int kTabThreads = 1024;
constexpr int kTabMaxRows = 4096;
constexpr int kTabPer = kTabMaxRows / kTabThreads;
constexpr int kTabAll = 0, kTabMoves = 1, kTabState = 2;

struct TablesArgs {
    const int32_t *cached, *fresh, *held;
    int32_t *held_out, *table, *free_list;
    const int32_t* free_count;
    int32_t *free_count_out, *cu, *kv;
    int64_t* slots;
    int32_t* positions;
    int B, page_shift, num_pages, max_pages, max_tokens;
    int* status;
};

// Exclusive prefix of each thread's v over the block, and the total.
PI_DEV long long block_prefix(long long v, long long* warp_sums, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(FULL, s, o);
        if (lane >= o) s += t;
    }
    __syncthreads();   // warp_sums may still be read from the last prefix
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    long long w = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : 0;
    const long long mine = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(FULL, w, o);
        if (lane >= o) w += t;
    }
    *total = __shfl_sync(FULL, w, 31);
    return __shfl_sync(FULL, w - mine, warp) + s - v;
}

// The same out of line, for a case that hardly occurs
__device__ __noinline__ long long block_prefix_again(long long v, long long* warp_sums, long long* total) {
    return block_prefix(v, warp_sums, total);
}

// The row b with first[b] <= x < first[b + 1] (first[0] <= x < first[n]).
template <typename T>
PI_DEV int row_of(const T* first, int n, T x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int PART>
__global__ void __launch_bounds__(kTabThreads) k_block_tables(const TablesArgs a) {
    if (PART != kTabState) asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ long long warp_sums[32];
    __shared__ int free_in;
    extern __shared__ long long tab_smem[];
    const int B = a.B;
    // prefixes [B + 1]: tokens, pages given back, pages wanted; then per row
    long long* gfirst = tab_smem;
    long long* wfirst = gfirst + B + 1;
    int* tfirst = reinterpret_cast<int*>(wfirst + B + 1);
    int* scached = tfirst + B + 1;
    int* sheld = scached + B;
    int* sneed = sheld + B;        // pages needed, -1: not served
    const int per = (B + kTabThreads - 1) / kTabThreads;
    int c[kTabPer], n[kTabPer], h[kTabPer];
    bool bad[kTabPer], over[kTabPer];
    // this thread's tokens (at most 2^42 over all rows), and from bit 44 on its
    // rows whose positions leave their table row
    constexpr long long kOver = 1ll << 44;
    long long tok = 0;
    bool any_bad = false;
    const int page = 1 << a.page_shift;
    const long long capacity = (long long)a.max_pages << a.page_shift;
#pragma unroll
    for (int i = 0; i < kTabPer; ++i) {
        const int b = threadIdx.x * per + i;
        c[i] = n[i] = h[i] = 0;
        bad[i] = over[i] = false;
        if (i < per && b < B) {
            c[i] = a.cached[b];
            n[i] = a.fresh[b];
            h[i] = a.held[b];
            bad[i] = n[i] < 0 || h[i] < 0 || h[i] > a.max_pages || n[i] > capacity;
            if (bad[i]) n[i] = 0;
            over[i] = !bad[i] && (c[i] < 0 || (long long)c[i] + n[i] > capacity);
            bad[i] |= over[i];
            tok += n[i] + (over[i] ? kOver : 0);
        }
        any_bad |= bad[i];
    }
    if (threadIdx.x == 0) free_in = *a.free_count;
    long long total_tok;
    long long tp = block_prefix(tok, warp_sums, &total_tok);
    // the packed rows hold the tokens of such rows as well, so those are counted
    // (the rows after them would be moved); where the tokens do not all fit, the
    // packed rows cannot hold them, and the others' are
    if (total_tok >= kOver) {
        if ((total_tok & (kOver - 1)) > a.max_tokens) {
            tok = 0;
#pragma unroll
            for (int i = 0; i < kTabPer; ++i) {
                if (over[i]) n[i] = 0;
                tok += n[i];
            }
            tp = block_prefix_again(tok, warp_sums, &total_tok);
        }
        total_tok &= kOver - 1;
        tp &= kOver - 1;
    }
    const int f = min(max(free_in, 0), a.num_pages);
    any_bad |= f != free_in;
    long long give = 0, want = 0;
    int need[kTabPer];
#pragma unroll
    for (int i = 0; i < kTabPer; ++i) {
        const int b = threadIdx.x * per + i;
        need[i] = -1;
        if (i < per && b < B) {
            const long long end = tp + n[i];
            tfirst[b] = (int)min(tp, (long long)a.max_tokens);
            scached[b] = c[i];
            sheld[b] = h[i];
            const bool past = n[i] > 0 && end > a.max_tokens;
            any_bad |= past;
            if (!bad[i] && !past) need[i] = (c[i] + n[i] + page - 1) >> a.page_shift;
            if (need[i] >= 0) {
                give += max(0, h[i] - need[i]);
                want += max(0, need[i] - h[i]);
            }
            tp = end;
        }
    }
    long long R, all_want;
    long long gp = block_prefix(give, warp_sums, &R);
    long long wp = block_prefix(want, warp_sums, &all_want);
    long long taken = 0;   // most pages that the served rows of this thread end at
#pragma unroll
    for (int i = 0; i < kTabPer; ++i) {
        const int b = threadIdx.x * per + i;
        if (i < per && b < B) {
            gfirst[b] = gp;
            wfirst[b] = wp;
            if (need[i] >= 0) {
                gp += max(0, h[i] - need[i]);
                const int w = max(0, need[i] - h[i]);
                wp += w;
                if (w > 0) {
                    if (wp <= f + R) taken = wp;
                    else need[i] = -1;
                }
            }
            sneed[b] = need[i];
        }
    }
    // pages taken: the largest prefix that fits, over all threads
    __syncthreads();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(FULL, taken, o));
    if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = taken;
    if (threadIdx.x == 0) {
        tfirst[B] = (int)min(total_tok, (long long)a.max_tokens);
        gfirst[B] = R;
        wfirst[B] = all_want;
    }
    __syncthreads();
    long long A = warp_sums[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) A = max(A, __shfl_xor_sync(FULL, A, o));
    // the block has its inputs: what a thread read went to shared memory or
    // into a prefix before the barriers above
    if (PART != kTabState) asm volatile("griddepcontrol.launch_dependents;");
    if (PART != kTabMoves) {
        for (int b = threadIdx.x; b < B; b += kTabThreads) {
            const int t0 = tfirst[b];
            a.held_out[b] = sneed[b] >= 0 ? sneed[b] : sheld[b];
            a.kv[b] = sneed[b] >= 0 ? scached[b] + tfirst[b + 1] - t0 : 0;
            a.cu[b] = t0;
        }
        if (threadIdx.x == 0) {
            a.cu[B] = tfirst[B];
            *a.free_count_out = (int)min(f + R - A, (long long)a.num_pages);
        }
        if (any_bad) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
    }
    if (PART == kTabState) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }

    // row that gives back released page j, and the table entry it is in
    auto released = [&](long long j) {
        const int b = row_of(gfirst, B, j);
        return a.table[(size_t)b * a.max_pages + sneed[b] + (int)(j - gfirst[b])];
    };
    // entry x of the stack once all releases are pushed
    auto stacked = [&](long long x) { return x < f ? a.free_list[x] : released(x - f); };

    const long long t0 = (long long)blockIdx.x * kTabThreads + threadIdx.x, step = (long long)gridDim.x * kTabThreads;
    bool dropped = false;
    for (long long j = t0; j < R; j += step) {
        if (f + j < a.num_pages) a.free_list[f + j] = released(j);
        else dropped = true;
    }
    for (long long x = t0; x < A; x += step) {
        const int b = row_of(wfirst, B, x);
        a.table[(size_t)b * a.max_pages + sheld[b] + (int)(x - wfirst[b])] = stacked(f + R - 1 - x);
    }
    const int T = tfirst[B];
    for (long long i = t0; i < a.max_tokens; i += step) {
        long long slot = -1;
        int pos = 0;
        if (i < T) {
            const int b = row_of(tfirst, B, (int)i);
            pos = (int)((unsigned)scached[b] + (unsigned)(i - tfirst[b]));   // (a row that is not served may pass int)
            if (sneed[b] >= 0) {
                const int pi = pos >> a.page_shift, held = sheld[b];
                const int id = pi < held ? a.table[(size_t)b * a.max_pages + pi]
                                         : stacked(f + R - 1 - (wfirst[b] + pi - held));
                slot = ((long long)id << a.page_shift) + (pos & (page - 1));
            }
        }
        a.slots[i] = slot;
        a.positions[i] = pos;
    }
    if (dropped) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
}

// ------------------------------------------------ rotary positions and store
//
// A unit is 16 elements of one head of one token: 8 pairs that turn together
// (two runs of 8 in the half layout, 16 in a row when interleaved), or 16 in a
// row that pass through.  Every unit is two or four 16-byte loads and two
// 16-byte stores, so the kernel is bound by HBM; a block takes one token (a
// share of its units where there are many), asks for all its loads first,
// and computes the token's cos and sin once for all heads while they are on
// their way.  16384 bf16 tokens (64 + 2 x 8 heads of 128): 103 us, 6.5 TB/s;
// 1999 fp32 tokens (32 + 2 x 32 heads) into fp16: 26.2 us, 5.6 TB/s; 32
// decoding tokens: 2.5 us, a launch.
constexpr int kRopeUnits = 2;   // units per thread (1: 134 us for the 16384 tokens, 4: 104, and 28.6 for the 1999: the last wave)
constexpr int kRopeMaxPairs = 64;

struct RopeArgs {
    const void *q, *k, *v;
    const int32_t* positions;
    const int64_t* slots;
    void *q_out, *kcache, *vcache;
    long long q_stride, k_stride, v_stride, out_stride;
    long long page_stride, head_stride, token_stride, num_slots;
    int heads, kv_heads, dh, page_shift, units;   // units of a token
    int* status;
    pi_rope_plan plan;
};

// 8 values as floats from a run of the input type, and back to a 16-bit type.
template <typename T>
PI_DEV void load8(const void* base, long long at, uint4 (&raw)[2]) {
    const T* p = static_cast<const T*>(base) + at;
    raw[0] = ld_stream16(p);
    if (sizeof(T) == 4) raw[1] = ld_stream16(p + 4);
}
template <typename T>
PI_DEV void widen8(const uint4 (&raw)[2], float (&f)[8]);
template <>
PI_DEV void widen8<__half>(const uint4 (&raw)[2], float (&f)[8]) {
    h8_to_f8(raw[0], f);
}
template <>
PI_DEV void widen8<__nv_bfloat16>(const uint4 (&raw)[2], float (&f)[8]) {
    const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <>
PI_DEV void widen8<float>(const uint4 (&raw)[2], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(raw[i].x);
        f[4 * i + 1] = __uint_as_float(raw[i].y);
        f[4 * i + 2] = __uint_as_float(raw[i].z);
        f[4 * i + 3] = __uint_as_float(raw[i].w);
    }
}
PI_DEV uint32_t pack2(float a, float b, __half) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
PI_DEV uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename O>
PI_DEV void store8(O* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1], O()), pack2(f[2], f[3], O()), pack2(f[4], f[5], O()),
                                              pack2(f[6], f[7], O()));
}

template <typename I, typename O>
__global__ void __launch_bounds__(256) k_rope_store(const __grid_constant__ RopeArgs a) {
    pdl_entry();
    __shared__ float2 cs[kRopeMaxPairs];
    const int t = blockIdx.x;
    const int per_head = a.dh / 16, turning = a.plan.rot_dim / 16, half = a.plan.rot_dim / 2;
    // where unit u of the token comes from: offsets of its two runs of 8
    auto runs = [&](int hu, bool turns, int* r0, int* r1) {
        if (turns && hu < turning && !a.plan.interleaved) {
            *r0 = 8 * hu;
            *r1 = half + 8 * hu;
        } else {
            *r0 = 16 * hu;
            *r1 = 16 * hu + 8;
        }
    };
    uint4 raw[kRopeUnits][2][2];
    const int u0 = blockIdx.y * kRopeUnits * blockDim.x + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kRopeUnits; ++i) {
        const int u = u0 + i * blockDim.x;
        if (u >= a.units) continue;
        int h = u / per_head, r0, r1;
        const int hu = u - h * per_head;
        runs(hu, h < a.heads + a.kv_heads, &r0, &r1);
        const void* src = a.q;
        long long at = t * a.q_stride;
        if (h >= a.heads + a.kv_heads) {
            h -= a.heads + a.kv_heads;
            src = a.v;
            at = t * a.v_stride;
        } else if (h >= a.heads) {
            h -= a.heads;
            src = a.k;
            at = t * a.k_stride;
        }
        at += (long long)h * a.dh;
        load8<I>(src, at + r0, raw[i][0]);
        load8<I>(src, at + r1, raw[i][1]);
    }
    // the angle in turns, position x turns[i] mod 1 in fixed point; its top 32
    // bits as a signed fraction of a half turn (off by at most 2^-25 of one in
    // the conversion to fp32)
    if (threadIdx.x < half) {
        const unsigned long long turn = (unsigned long long)(long long)a.positions[t] * a.plan.turns[threadIdx.x];
        float s, c;
        sincospif((float)(int)(turn >> 32) * (1.0f / 2147483648.0f), &s, &c);
        cs[threadIdx.x] = make_float2(c * a.plan.mscale, s * a.plan.mscale);
    }
    const long long slot = a.kv_heads > 0 ? a.slots[t] : -1;
    const bool keep = slot >= 0 && slot < a.num_slots;
    if (slot < -1 || slot >= a.num_slots)
        if (threadIdx.x == 0 && a.kv_heads > 0) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
    const long long cache_at =
        keep ? (slot >> a.page_shift) * a.page_stride + (slot & ((1 << a.page_shift) - 1)) * a.token_stride : 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRopeUnits; ++i) {
        const int u = u0 + i * blockDim.x;
        if (u >= a.units) continue;
        int h = u / per_head, r0, r1;
        const int hu = u - h * per_head;
        const bool turns = h < a.heads + a.kv_heads;
        runs(hu, turns, &r0, &r1);
        float x[8], y[8];
        widen8<I>(raw[i][0], x);
        widen8<I>(raw[i][1], y);
        if (turns && hu < turning) {
            if (a.plan.interleaved) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 p = cs[8 * hu + e], r = cs[8 * hu + 4 + e];
                    const float x1 = x[2 * e], x2 = x[2 * e + 1], y1 = y[2 * e], y2 = y[2 * e + 1];
                    x[2 * e] = x1 * p.x - x2 * p.y;
                    x[2 * e + 1] = x2 * p.x + x1 * p.y;
                    y[2 * e] = y1 * r.x - y2 * r.y;
                    y[2 * e + 1] = y2 * r.x + y1 * r.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 p = cs[8 * hu + e];
                    const float x1 = x[e], x2 = y[e];
                    x[e] = x1 * p.x - x2 * p.y;
                    y[e] = x2 * p.x + x1 * p.y;
                }
            }
        }
        O* dst;
        if (h < a.heads) {
            dst = static_cast<O*>(a.q_out) + t * a.out_stride + (long long)h * a.dh;
        } else {
            if (!keep) continue;
            h -= a.heads;
            dst = static_cast<O*>(a.kcache);
            if (h >= a.kv_heads) {
                h -= a.kv_heads;
                dst = static_cast<O*>(a.vcache);
            }
            dst += cache_at + (long long)h * a.head_stride;
        }
        store8(dst + r0, x);
        store8(dst + r1, y);
    }
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

bool tables_ok(const pi_tables_desc& d) {
    return d.batch >= 1 && d.batch <= kTabMaxRows && page_size_ok(d.page_size) && d.num_pages >= 1 &&
           d.num_pages <= (1 << 26) && d.max_pages >= 1 && d.max_pages <= (1 << 20) &&
           (long long)d.max_pages * d.page_size <= (1ll << 30) && d.max_tokens >= 0 && d.max_tokens <= (1 << 24);
}

size_t tables_smem(int B) { return 16 * (size_t)(B + 1) + 4 * (size_t)(B + 1) + 12 * (size_t)B; }

// One part of a step on `blocks` blocks; the shared memory of the largest
// batch is allowed once per device.
template <int PART>
cudaError_t launch_tables(const TablesArgs& a, int blocks, cudaStream_t s) {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            e = cudaFuncSetAttribute(k_block_tables<PART>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)tables_smem(kTabMaxRows));
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    return launch_pdl(k_block_tables<PART>, blocks, kTabThreads, tables_smem(a.B), s, a);
}

int page_shift(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

}  // namespace

bool rows_overlap(const void* a, long long a_stride, long long a_width, const void* b, long long b_stride,
                  long long b_width, long long n) {
    if (a == nullptr || b == nullptr || n < 1) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    if (x + (uintptr_t)((n - 1) * a_stride + a_width) <= y || y + (uintptr_t)((n - 1) * b_stride + b_width) <= x) return false;
    if (n == 1 || a_stride != b_stride) return true;
    // how far b's rows begin behind a's, within a stride
    const long long d = y >= x ? (long long)((y - x) % a_stride) : (a_stride - (long long)((x - y) % a_stride)) % a_stride;
    return d < a_width || d + b_width > a_stride;
}

bool page_desc_ok(const pi_page_desc& c) {
    if (c.kv_heads < 1 || c.kv_heads > 1024 || (c.head_dim != 64 && c.head_dim != 128) || !page_size_ok(c.page_size) ||
        c.num_pages < 1 || c.num_pages > (1 << 26) || (c.dtype != PI_T_F16 && c.dtype != PI_T_BF16))
        return false;
    for (long long s : {c.page_stride, c.head_stride, c.token_stride})
        if (s < c.head_dim || s % 8 != 0 || s > (1ll << 36)) return false;
    // a head starts on a block of 64 elements, and its last block has a 31-bit number
    return c.head_stride % 64 == 0 && (c.kv_heads - 1) * (c.head_stride / 64) < (1ll << 31) - 2;
}

}  // namespace pi

using namespace pi;

extern "C" {

pi_status pi_block_tables(const pi_tables_desc* desc, const int32_t* cached_len, const int32_t* new_len,
                          const int32_t* held, int32_t* held_out, int32_t* block_table, int32_t* free_list,
                          const int32_t* free_count, int32_t* free_count_out, int32_t* cu_new, int32_t* kv_len,
                          int64_t* slots, int32_t* positions, void* stream) {
    if (!desc || !tables_ok(*desc)) return PI_ERR_INVALID_ARG;
    if (!cached_len || !new_len || !held || !held_out || !block_table || !free_list || !free_count ||
        !free_count_out || !cu_new || !kv_len || (desc->max_tokens > 0 && (!slots || !positions)))
        return PI_ERR_INVALID_ARG;
    for (const void* p : {(const void*)cached_len, (const void*)new_len, (const void*)held, (const void*)held_out,
                          (const void*)block_table, (const void*)free_list, (const void*)free_count,
                          (const void*)free_count_out, (const void*)cu_new, (const void*)kv_len,
                          (const void*)positions})
        if (!aligned(p, 4)) return PI_ERR_INVALID_ARG;
    if (!aligned(slots, 8)) return PI_ERR_INVALID_ARG;
    TablesArgs a{cached_len,     new_len, held,   held_out, block_table, free_list,   free_count,
                 free_count_out, cu_new,  kv_len, slots,    positions,   desc->batch, page_shift(desc->page_size),
                 desc->num_pages, desc->max_pages, desc->max_tokens, status_word()};
    if (a.status == nullptr) return PI_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // writes to expect: a token each, and a few moved pages a row (a decoding
    // row moves one in page_size steps, a row that ends gives all back).  One
    // block takes 4.3 us and 1.2 more per 1024 tokens, two grids 6.8 us: 5.9
    // against 6.7 at 2048 tokens of 64 rows, 4.9 against 7.0 at 512 decoding
    // rows (6.6 against 7.1 if each gives back 4 pages), 10 against 6.9 at 8192
    // tokens, 187 against 10.4 at 2048 rows with 42 thousand tokens.
    const long long writes = desc->max_tokens + 4ll * desc->batch;
    cudaError_t e;
    if (writes <= 5 * kTabThreads / 2) {
        e = launch_tables<kTabAll>(a, 1, s);
    } else {
        // wide enough for tens of moved pages a row (2048 rows: 10.4 us so, 11.4 with blocks for 4 a row)
        const long long most = desc->max_tokens + 32ll * desc->batch;
        e = launch_tables<kTabMoves>(a, (int)std::min<long long>(128, (most + kTabThreads - 1) / kTabThreads), s);
        if (e == cudaSuccess) e = launch_tables<kTabState>(a, 1, s);
    }
    return e == cudaSuccess ? PI_OK : PI_ERR_CUDA;
}

pi_status pi_rope_plan_init(const pi_rope_desc* desc, pi_rope_plan* plan) {
    if (!desc || !plan) return PI_ERR_INVALID_ARG;
    const pi_rope_desc& d = *desc;
    if ((d.head_dim != 64 && d.head_dim != 128) || d.rot_dim < 0 || d.rot_dim > d.head_dim || d.rot_dim % 16 != 0 ||
        (d.interleaved != 0 && d.interleaved != 1) || d.scaling < PI_ROPE_NONE || d.scaling > PI_ROPE_RAMP ||
        !(d.base > 1.0) || !std::isfinite(d.base) || !std::isfinite(d.mscale))
        return PI_ERR_INVALID_ARG;
    if (d.scaling != PI_ROPE_NONE && (!(d.factor > 0.0) || !std::isfinite(d.factor))) return PI_ERR_INVALID_ARG;
    if (d.scaling >= PI_ROPE_BLEND && (!(d.original_max > 0.0) || !std::isfinite(d.original_max) || !(d.low > 0.0) ||
                                       !(d.high > d.low) || !std::isfinite(d.high)))
        return PI_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    pi_rope_plan p{};
    p.head_dim = d.head_dim;
    p.rot_dim = d.rot_dim;
    p.interleaved = d.interleaved;
    p.mscale = (float)d.mscale;
    double first = 0.0, last = 0.0;
    if (d.scaling == PI_ROPE_RAMP) {
        // the (real) pair index that turns r times within original_max positions
        auto index = [&](double r) { return d.rot_dim * log(d.original_max / (two_pi * r)) / (2.0 * log(d.base)); };
        first = std::max(floor(index(d.high)), 0.0);
        last = std::min(ceil(index(d.low)), d.rot_dim - 1.0);
    }
    for (int i = 0; i < d.rot_dim / 2; ++i) {
        double f = pow(d.base, -2.0 * i / d.rot_dim);
        if (d.scaling == PI_ROPE_LINEAR) {
            f /= d.factor;
        } else if (d.scaling == PI_ROPE_BLEND) {
            const double r = d.original_max * f / two_pi;
            const double g = std::min(std::max((r - d.low) / (d.high - d.low), 0.0), 1.0);
            f = (1.0 - g) * f / d.factor + g * f;
        } else if (d.scaling == PI_ROPE_RAMP) {
            const double g = std::min(std::max((i - first) / std::max(last - first, 0.001), 0.0), 1.0);
            f = f / d.factor * g + f * (1.0 - g);
        }
        const double x = f / two_pi;
        p.turns[i] = (uint64_t)ldexp(x - floor(x), 64);   // x - floor(x) < 1, so below 2^64
    }
    *plan = p;
    return PI_OK;
}

pi_status pi_rope_store(const pi_rope_plan* plan, const pi_page_desc* cache, const pi_qkv_desc* desc, const void* q,
                        const void* k, const void* v, const int32_t* positions, const int64_t* slots, void* q_out,
                        void* kcache, void* vcache, void* stream) {
    if (!plan || !cache || !desc || !page_desc_ok(*cache)) return PI_ERR_INVALID_ARG;
    const pi_qkv_desc& d = *desc;
    if (plan->head_dim != cache->head_dim || plan->rot_dim < 0 || plan->rot_dim > plan->head_dim ||
        plan->rot_dim % 16 != 0 || (plan->interleaved != 0 && plan->interleaved != 1))
        return PI_ERR_INVALID_ARG;
    if (d.tokens < 0 || d.tokens > (1 << 24) || d.heads < 1 || d.heads > 1024 || d.dtype < PI_T_F16 ||
        d.dtype > PI_T_F32)
        return PI_ERR_INVALID_ARG;
    const bool has_q = q || q_out, has_kv = k || v || kcache || vcache || slots;
    if (!has_q && !has_kv) return PI_ERR_INVALID_ARG;
    auto stride_ok = [&](long long s, int heads) {
        return s % 8 == 0 && s >= (long long)heads * cache->head_dim && s <= (1ll << 36);
    };
    if (has_q && !(stride_ok(d.q_stride, d.heads) && stride_ok(d.out_stride, d.heads))) return PI_ERR_INVALID_ARG;
    if (has_kv && !(stride_ok(d.k_stride, cache->kv_heads) && stride_ok(d.v_stride, cache->kv_heads)))
        return PI_ERR_INVALID_ARG;
    if (d.tokens == 0) return PI_OK;
    if (!positions || !aligned(positions, 4)) return PI_ERR_INVALID_ARG;
    if (has_q && (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16))) return PI_ERR_INVALID_ARG;
    if (has_kv && (!k || !v || !kcache || !vcache || !slots || !aligned(k, 16) || !aligned(v, 16) ||
                   !aligned(kcache, 16) || !aligned(vcache, 16) || !aligned(slots, 8)))
        return PI_ERR_INVALID_ARG;
    // Rotated queries go over no input that another thread may still have to
    // read.  In place a thread reads all it writes first, if the elements lie alike.
    const long long in = d.dtype == PI_T_F32 ? 4 : 2, q_width = (long long)d.heads * cache->head_dim,
                    k_width = (long long)cache->kv_heads * cache->head_dim;
    auto over = [&](const void* x, long long stride, long long width) {
        return rows_overlap(x, in * stride, in * width, q_out, 2 * d.out_stride, 2 * q_width, d.tokens);
    };
    const bool in_place = q == q_out && d.dtype == cache->dtype && d.q_stride == d.out_stride;
    if (has_q && ((!in_place && over(q, d.q_stride, q_width)) ||
                  (has_kv && (over(k, d.k_stride, k_width) || over(v, d.v_stride, k_width)))))
        return PI_ERR_INVALID_ARG;
    RopeArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.kcache = kcache;
    a.vcache = vcache;
    a.q_stride = d.q_stride;
    a.k_stride = d.k_stride;
    a.v_stride = d.v_stride;
    a.out_stride = d.out_stride;
    a.page_stride = cache->page_stride;
    a.head_stride = cache->head_stride;
    a.token_stride = cache->token_stride;
    a.num_slots = (long long)cache->num_pages * cache->page_size;
    a.heads = has_q ? d.heads : 0;
    a.kv_heads = has_kv ? cache->kv_heads : 0;
    a.dh = cache->head_dim;
    a.page_shift = page_shift(cache->page_size);
    a.units = (a.heads + 2 * a.kv_heads) * (a.dh / 16);
    a.status = status_word();
    a.plan = *plan;
    if (a.status == nullptr) return PI_ERR_CUDA;
    // blocks of at most 256 threads that share the units evenly; at least 64
    // threads, one for each pair's angle
    const int shares = (a.units + 256 * kRopeUnits - 1) / (256 * kRopeUnits);
    const int threads = std::max(64, ((a.units + shares * kRopeUnits - 1) / (shares * kRopeUnits) + 31) / 32 * 32);
    const dim3 grid((unsigned)d.tokens, (unsigned)shares);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (cache->dtype == PI_T_F16) {
        e = d.dtype == PI_T_F16    ? launch_pdl(k_rope_store<__half, __half>, grid, threads, 0, s, a)
            : d.dtype == PI_T_BF16 ? launch_pdl(k_rope_store<__nv_bfloat16, __half>, grid, threads, 0, s, a)
                                   : launch_pdl(k_rope_store<float, __half>, grid, threads, 0, s, a);
    } else {
        e = d.dtype == PI_T_F16    ? launch_pdl(k_rope_store<__half, __nv_bfloat16>, grid, threads, 0, s, a)
            : d.dtype == PI_T_BF16 ? launch_pdl(k_rope_store<__nv_bfloat16, __nv_bfloat16>, grid, threads, 0, s, a)
                                   : launch_pdl(k_rope_store<float, __nv_bfloat16>, grid, threads, 0, s, a);
    }
    return e == cudaSuccess ? PI_OK : PI_ERR_CUDA;
}

}  // extern "C"
