// pi_paged8.cu -- the paged cache in 8 bits: rotary positions and the store of
// keys and values as e4m3 codes with an exponent for each block of 16 positions
// and head, and rows read back from it.  The attention over it is in
// pi_paged8_attn.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "pi_common.cuh"
#include "pi_e4m3.cuh"
#include "pi_internal.h"

namespace pi {
namespace {

using namespace e4m3;

// ------------------------------------------------ quantised store
//
// A warp per token, KV head and array (keys or values); it works if its token
// is the first new one of its block, and then for all of the block's new tokens
// (up to 16), which are the rows behind it: magnitudes, exponent, the earlier
// positions' codes again where the exponent grew, the new codes.  A lane holds 4
// elements of a token that turn together: two pairs (i, i + rot / 2) in the half
// layout, 4 in a row when interleaved or past rot_dim.
constexpr int kStoreWarps = 8;

struct Store8Args {
    const void *k, *v;
    const int32_t* positions;
    const int64_t* slots;
    uint8_t *kc, *vc;
    int8_t *ke, *ve;
    long long k_stride, v_stride, page_stride, head_stride, token_stride, num_slots;
    int tokens, kv_heads, dh, page_shift;
    int* status;
    pi_rope_plan plan;
};

template <typename T>
PI_DEV float2 load2(const void* base, long long at);
template <>
PI_DEV float2 load2<__half>(const void* base, long long at) {
    return __half22float2(*reinterpret_cast<const __half2*>(static_cast<const __half*>(base) + at));
}
template <>
PI_DEV float2 load2<__nv_bfloat16>(const void* base, long long at) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(static_cast<const __nv_bfloat16*>(base) + at));
}
template <>
PI_DEV float2 load2<float>(const void* base, long long at) {
    return *reinterpret_cast<const float2*>(static_cast<const float*>(base) + at);
}

// cos and sin of position x turns in fixed point: the top 32 bits of the turn's
// fraction are a signed fraction of a half turn; what fp32 does not hold of them
// enters to first order, so that the angle is off by 2^-31 half turns.
PI_DEV float2 turn_of(int position, unsigned long long turns, float mscale) {
    const int a = (int)((unsigned long long)(long long)position * turns >> 32);
    const float f = (float)a;
    const float rest = (float)((long long)a - (long long)f) * (3.14159265358979f / 2147483648.0f);
    float s, c;
    sincospif(f * (1.0f / 2147483648.0f), &s, &c);
    return make_float2(fmaf(-s, rest, c) * mscale, fmaf(c, rest, s) * mscale);
}

template <typename I, int DH>
__global__ void __launch_bounds__(32 * kStoreWarps) k_store8(const __grid_constant__ Store8Args a) {
    pdl_entry();
    constexpr int LANES = DH / 4;   // lanes of a token: 32 or 16
    constexpr int SIDE = 32 / LANES, N = kBlock / SIDE;   // tokens side by side, and of a lane at most
    const int lane = threadIdx.x & 31;
    const int work = blockIdx.y * kStoreWarps + (threadIdx.x >> 5);
    if (work >= 2 * a.kv_heads) return;
    const int t = blockIdx.x;
    const bool values = work >= a.kv_heads;
    const int h = values ? work - a.kv_heads : work;
    // the slots of this token, the one before it and the 15 behind it
    long long mine = -2;
    if (lane < kBlock + 1 && t - 1 + lane >= 0 && t - 1 + lane < a.tokens) mine = a.slots[t - 1 + lane];
    const long long slot = __shfl_sync(FULL, mine, 1), before = __shfl_sync(FULL, mine, 0);
    if (slot < 0 || slot >= a.num_slots) {
        if (slot != -1 && lane == 0) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
        return;
    }
    const int r = (int)(slot & (kBlock - 1));
    if (r != 0 && before == slot - 1) return;   // not the block's first new token
    const unsigned next = __ballot_sync(FULL, lane >= 1 && lane <= kBlock && mine == slot + lane - 1);
    const int count = min(__ffs(~(next >> 1)) - 1, kBlock - r);   // new tokens of the block
    const int in_page = (int)(slot & ((1 << a.page_shift) - 1)) - r;
    const long long page = slot >> a.page_shift;
    uint8_t* const codes = (values ? a.vc : a.kc) + page * a.page_stride + h * a.head_stride + in_page * a.token_stride;
    int8_t* const exp_at = (values ? a.ve : a.ke) + ((page * a.kv_heads + h) << (a.page_shift - 4)) + in_page / kBlock;
    const int old = r > 0 ? bounded(*exp_at) : kMinExp;

    // this lane's elements of a token: at e0, e0 + 1 and e1, e1 + 1
    const int sub = lane / LANES, l = lane % LANES, half = a.plan.rot_dim / 2;
    const bool apart = !a.plan.interleaved && 2 * l < half;
    const int e0 = apart ? 2 * l : 4 * l, e1 = apart ? half + 2 * l : 4 * l + 2;
    // (pairs from half on pass through: 2 l >= half there, so 4 l >= rot_dim)
    const bool turns = !values && 2 * l < half;
    unsigned long long w0 = 0, w1 = 0;
    if (turns) {
        w0 = a.plan.turns[2 * l];
        w1 = a.plan.turns[2 * l + 1];
    }
    const void* const src = values ? a.v : a.k;
    const long long stride = values ? a.v_stride : a.k_stride;
    float x[N][4];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = i * SIDE + sub;
        if (i * SIDE >= count) break;
        x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
        if (row >= count) continue;
        const long long at = (long long)(t + row) * stride + (long long)h * DH;
        const float2 u = load2<I>(src, at + e0), v = load2<I>(src, at + e1);
        x[i][0] = u.x;
        x[i][1] = u.y;
        x[i][2] = v.x;
        x[i][3] = v.y;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = i * SIDE + sub;
        if (i * SIDE >= count) break;
        if (turns && row < count) {
            const int pos = a.positions[t + row];
            const float2 p = turn_of(pos, w0, a.plan.mscale), q = turn_of(pos, w1, a.plan.mscale);
            const float x0 = x[i][0], x1 = x[i][1], x2 = x[i][2], x3 = x[i][3];
            if (apart) {   // (0, 2) and (1, 3)
                x[i][0] = x0 * p.x - x2 * p.y;
                x[i][2] = x2 * p.x + x0 * p.y;
                x[i][1] = x1 * q.x - x3 * q.y;
                x[i][3] = x3 * q.x + x1 * q.y;
            } else {       // (0, 1) and (2, 3)
                x[i][0] = x0 * p.x - x1 * p.y;
                x[i][1] = x1 * p.x + x0 * p.y;
                x[i][2] = x2 * q.x - x3 * q.y;
                x[i][3] = x3 * q.x + x2 * q.y;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t bits = __float_as_uint(x[i][e]) & 0x7fffffffu;
            if (bits >= 0x7f800000u) x[i][e] = NAN;
            else most = max(most, bits);
        }
    }
    most = __reduce_max_sync(FULL, most);
    const int e = max(exponent_of(most), old);
    if (r > 0 && e > old) {
        // the earlier positions' codes, 16 at a time
        const float f = pow2(old - e);
        for (int i = lane; i < r * (DH / 16); i += 32) {
            uint4* const at = reinterpret_cast<uint4*>(codes + (i / (DH / 16)) * a.token_stride + i % (DH / 16) * 16);
            uint4 c = *at;
            auto again = [&](uint32_t w) {
                const float2 u = values2(w & 0xffffu), v = values2(w >> 16);
                return encode2(u.x * f, u.y * f) | encode2(v.x * f, v.y * f) << 16;
            };
            c = make_uint4(again(c.x), again(c.y), again(c.z), again(c.w));
            *at = c;
        }
    }
    const float f = pow2(-e);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = i * SIDE + sub;
        if (i * SIDE >= count) break;
        if (row >= count) continue;
        uint8_t* const at = codes + (r + row) * a.token_stride;
        const uint32_t lo = encode2(x[i][0] * f, x[i][1] * f), hi = encode2(x[i][2] * f, x[i][3] * f);
        if (apart) {
            *reinterpret_cast<uint16_t*>(at + e0) = (uint16_t)lo;
            *reinterpret_cast<uint16_t*>(at + e1) = (uint16_t)hi;
        } else {
            *reinterpret_cast<uint32_t*>(at + e0) = lo | hi << 16;
        }
    }
    if (lane == 0) *exp_at = (int8_t)e;
}

// ------------------------------------------------ rows read back
//
// A block takes 32 rows: a lane each finds its row's request (binary search in
// cu_rows) and page, then all threads move 16 codes at a time.
constexpr int kReadRows = 32;

struct Read8Args {
    Cache8 c;
    const int32_t *table, *start, *cu;
    void *k_out, *v_out;
    long long k_stride, v_stride;
    int batch, max_pages, max_rows, dh;
    int* status;
};

// values of 16 codes, rounded to the output's type
PI_DEV void put16(__half* p, const float (&f)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // (past 65504: the largest; a comparison keeps NaN)
        const float x = fabsf(f[2 * i]) > 65504.f ? copysignf(65504.f, f[2 * i]) : f[2 * i];
        const float y = fabsf(f[2 * i + 1]) > 65504.f ? copysignf(65504.f, f[2 * i + 1]) : f[2 * i + 1];
        const __half2 v = __floats2half2_rn(x, y);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
PI_DEV void put16(__nv_bfloat16* p, const float (&f)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
PI_DEV void put16(float* p, const float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}
PI_DEV void values16(const uint4& c, float scale, float (&f)[16]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = values2(w[i] & 0xffffu), v = values2(w[i] >> 16);
        f[4 * i] = u.x * scale;
        f[4 * i + 1] = u.y * scale;
        f[4 * i + 2] = v.x * scale;
        f[4 * i + 3] = v.y * scale;
    }
}

template <typename O>
__global__ void __launch_bounds__(256) k_page_read8(const __grid_constant__ Read8Args a) {
    pdl_entry();
    __shared__ long long code_at[kReadRows], exp_at[kReadRows];   // -1: zeros, -2: no row
    const int row0 = blockIdx.x * kReadRows;
    if (threadIdx.x < kReadRows) {
        const int row = row0 + threadIdx.x;
        long long code = -2, ex = 0;
        if (row < a.max_rows) {
            // the last request that starts at or before the row
            int lo = 0, hi = a.batch;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (a.cu[mid] <= row) lo = mid;
                else hi = mid;
            }
            const int first = a.cu[lo], end = a.cu[lo + 1];
            if (first >= 0 && first <= row && row < end && end <= a.max_rows) {
                const long long pos = (long long)(a.start ? a.start[lo] : 0) + (row - first);
                code = -1;
                if (pos >= 0 && pos < (long long)a.max_pages << a.c.page_shift) {
                    const int id = a.table[(size_t)lo * a.max_pages + (size_t)(pos >> a.c.page_shift)];
                    const int in_page = (int)(pos & ((1 << a.c.page_shift) - 1));
                    if (id >= 0 && id < a.c.num_pages) {
                        code = id * a.c.page_stride + in_page * a.c.token_stride;
                        ex = ((long long)id * a.c.kv_heads << (a.c.page_shift - 4)) + in_page / kBlock;
                    }
                }
                if (code < 0) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
            }
        }
        code_at[threadIdx.x] = code;
        exp_at[threadIdx.x] = ex;
    }
    if (blockIdx.x == 0) {
        bool bad = false;
        for (int b = threadIdx.x; b < a.batch; b += 256) bad |= a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.max_rows;
        if (bad) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
    }
    __syncthreads();
    const int per_head = a.dh / 16, per_row = a.c.kv_heads * per_head;
    const int first_array = a.k_out ? 0 : 1, arrays = (a.k_out ? 1 : 0) + (a.v_out ? 1 : 0);
    for (int i = threadIdx.x; i < arrays * kReadRows * per_row; i += 256) {
        const int chunk = i % per_row, r = i / per_row % kReadRows;
        const bool values = i / per_row / kReadRows + first_array == 1;
        const long long at = code_at[r];
        if (at == -2) continue;
        const int h = chunk / per_head;
        float f[16];
        if (at >= 0) {
            const uint8_t* const codes = values ? a.c.v : a.c.k;
            const int8_t* const exps = values ? a.c.ve : a.c.ke;
            values16(ld_stream16(codes + at + h * a.c.head_stride + chunk % per_head * 16),
                     pow2(bounded(exps[exp_at[r] + ((long long)h << (a.c.page_shift - 4))])), f);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = 0.f;
        }
        put16(static_cast<O*>(values ? a.v_out : a.k_out) + (long long)(row0 + r) * (values ? a.v_stride : a.k_stride) + chunk * 16, f);
    }
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename I>
cudaError_t launch_store8(const Store8Args& a, cudaStream_t s) {
    const dim3 grid((unsigned)a.tokens, (unsigned)((2 * a.kv_heads + kStoreWarps - 1) / kStoreWarps));
    return a.dh == 128 ? launch_pdl(k_store8<I, 128>, grid, 32 * kStoreWarps, 0, s, a)
                       : launch_pdl(k_store8<I, 64>, grid, 32 * kStoreWarps, 0, s, a);
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
    if (!has_q && !has_kv) return PI_ERR_INVALID_ARG;
    auto stride_ok = [&](long long s, int heads) {
        return s % 8 == 0 && s >= (long long)heads * cache->head_dim && s <= (1ll << 36);
    };
    if (has_kv && !(stride_ok(d.k_stride, cache->kv_heads) && stride_ok(d.v_stride, cache->kv_heads)))
        return PI_ERR_INVALID_ARG;
    if (has_kv && d.tokens > 0 &&
        (!k || !v || !kcache || !vcache || !kexp || !vexp || !slots || !aligned(k, 16) || !aligned(v, 16) ||
         !aligned(kcache, 16) || !aligned(vcache, 16) || !aligned(slots, 8)))
        return PI_ERR_INVALID_ARG;
    if (d.tokens > 0 && (!positions || !aligned(positions, 4))) return PI_ERR_INVALID_ARG;
    // rotated queries go over no key or value that another thread may still have to read
    const long long in = d.dtype == PI_T_F32 ? 4 : 2, k_width = (long long)cache->kv_heads * cache->head_dim;
    if (has_q && has_kv)
        for (const void* x : {k, v})
            if (rows_overlap(x, in * (x == k ? d.k_stride : d.v_stride), in * k_width, q_out, 2 * d.out_stride,
                             2ll * d.heads * cache->head_dim, d.tokens))
                return PI_ERR_INVALID_ARG;
    if (has_q) {
        const int dh = cache->head_dim;
        const pi_page_desc rows{1, dh, cache->page_size, 1, out_dtype, (long long)dh * cache->page_size,
                                (long long)dh * cache->page_size, dh};
        const pi_status st = pi_rope_store(plan, &rows, desc, q, nullptr, nullptr, positions, nullptr, q_out, nullptr,
                                           nullptr, stream);
        if (st != PI_OK) return st;
    }
    if (!has_kv || d.tokens == 0) return PI_OK;
    Store8Args a{};
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.slots = slots;
    a.kc = static_cast<uint8_t*>(kcache);
    a.vc = static_cast<uint8_t*>(vcache);
    a.ke = kexp;
    a.ve = vexp;
    a.k_stride = d.k_stride;
    a.v_stride = d.v_stride;
    a.page_stride = cache->page_stride;
    a.head_stride = cache->head_stride;
    a.token_stride = cache->token_stride;
    a.num_slots = (long long)cache->num_pages * cache->page_size;
    a.tokens = d.tokens;
    a.kv_heads = cache->kv_heads;
    a.dh = cache->head_dim;
    a.page_shift = __builtin_ctz((unsigned)cache->page_size);
    a.status = status_word();
    a.plan = *plan;
    if (a.status == nullptr) return PI_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d.dtype == PI_T_F16    ? launch_store8<__half>(a, s)
                          : d.dtype == PI_T_BF16 ? launch_store8<__nv_bfloat16>(a, s)
                                                 : launch_store8<float>(a, s);
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
    const long long width = (long long)cache->kv_heads * cache->head_dim;
    auto array_ok = [&](const void* codes, const void* exps, const void* out, long long stride) {
        if (!out) return !codes && !exps;
        return codes && exps && aligned(codes, 16) && aligned(out, 16) && stride % 8 == 0 && stride >= width && stride <= (1ll << 36);
    };
    if (!array_ok(kcache, kexp, k_out, d.k_stride) || !array_ok(vcache, vexp, v_out, d.v_stride) || (!k_out && !v_out))
        return PI_ERR_INVALID_ARG;
    if (!block_table || !cu_rows || !aligned(block_table, 4) || !aligned(cu_rows, 4) || !aligned(start, 4))
        return PI_ERR_INVALID_ARG;
    if (d.max_rows == 0) return PI_OK;
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
    a.dh = cache->head_dim;
    a.status = status_word();
    if (a.status == nullptr) return PI_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned blocks = (unsigned)((d.max_rows + (long long)kReadRows - 1) / kReadRows);
    const cudaError_t e = d.dtype == PI_T_F16    ? launch_pdl(k_page_read8<__half>, blocks, 256, 0, s, a)
                          : d.dtype == PI_T_BF16 ? launch_pdl(k_page_read8<__nv_bfloat16>, blocks, 256, 0, s, a)
                                                 : launch_pdl(k_page_read8<float>, blocks, 256, 0, s, a);
    return e == cudaSuccess ? PI_OK : PI_ERR_CUDA;
}

}  // extern "C"
