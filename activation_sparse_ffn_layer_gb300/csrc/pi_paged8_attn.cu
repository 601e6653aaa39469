// pi_paged8_attn.cu -- causal attention of new tokens over the 8-bit paged cache.
//
// A block per token and query head: a thread per key of a tile of 128 for the
// scores, a thread per column for the sums, a running maximum and sum; all in
// fp32, and only keys that the token sees are touched.
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

struct Attn8Args {
    Cache8 c;
    const void* q;
    const int32_t *table, *cu, *kv;
    void* out;
    float* lse;
    long long q_stride, o_stride;
    int heads, batch, max_tokens, max_new, max_pages, window, group;
    float scale;
    int* status;
};

PI_DEV float wide(__half v) { return __half2float(v); }
PI_DEV float wide(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T, int DH>
__global__ void __launch_bounds__(128) k_paged_attn8(const __grid_constant__ Attn8Args a) {
    pdl_entry();
    __shared__ float q[DH], w[128], red[4];
    __shared__ long long at[128];
    __shared__ float es[128];
    const int row = blockIdx.x, head = blockIdx.y, g = head / a.group, tid = threadIdx.x;
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.cu[mid] <= row) lo = mid;
        else hi = mid;
    }
    if (row == 0 && head == 0) {
        bool bad = false;
        for (int b = tid; b < a.batch; b += 128)
            bad |= a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.max_tokens || a.cu[b + 1] - a.cu[b] > a.max_new ||
                   a.kv[b] < 0 || a.kv[b] > a.max_pages << a.c.page_shift;
        if (bad) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
    }
    const int first = a.cu[lo], end = a.cu[lo + 1];
    if (first < 0 || row < first || row >= end || end > a.max_tokens || end - first > a.max_new) return;
    int kv = a.kv[lo];
    if (kv < 0 || kv > a.max_pages << a.c.page_shift) kv = 0;
    const int pos = kv - (end - row), from = a.window > 0 ? max(0, pos - a.window + 1) : 0, to = pos + 1;
    if (tid < DH) q[tid] = wide(static_cast<const T*>(a.q)[(long long)row * a.q_stride + head * DH + tid]) * a.scale;
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int base = from; base < to; base += 128) {
        __syncthreads();
        const int key = base + tid;
        float s = -INFINITY;
        if (key < to) {
            const int id = a.table[(size_t)lo * a.max_pages + (key >> a.c.page_shift)];
            const int in_page = key & ((1 << a.c.page_shift) - 1);
            long long where = -1;
            s = 0.f;
            if (id >= 0 && id < a.c.num_pages) {
                where = id * a.c.page_stride + g * a.c.head_stride + in_page * a.c.token_stride;
                const long long ex = (((long long)id * a.c.kv_heads + g) << (a.c.page_shift - 4)) + in_page / kBlock;
                for (int d = 0; d < DH; d += 16) {
                    const uint4 y = *reinterpret_cast<const uint4*>(a.c.k + where + d);
                    const uint32_t words[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 u = values2(words[i] & 0xffffu), v = values2(words[i] >> 16);
                        s = fmaf(q[d + 4 * i], u.x, fmaf(q[d + 4 * i + 1], u.y, fmaf(q[d + 4 * i + 2], v.x, fmaf(q[d + 4 * i + 3], v.y, s))));
                    }
                }
                s *= pow2(bounded(a.c.ke[ex]));
                es[tid] = pow2(bounded(a.c.ve[ex]));
            } else {
                atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
            }
            at[tid] = where;
        }
        float top = s;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, d));
        if ((tid & 31) == 0) red[tid >> 5] = top;
        __syncthreads();
        top = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float use = top == -INFINITY ? 0.f : top, f = expf(m - use);
        w[tid] = key < to ? expf(s - use) : 0.f;
        m = top;
        __syncthreads();
        l *= f;
        o *= f;
        for (int x = 0; x < min(128, to - base); ++x) {
            l += w[x];
            if (tid < DH && at[x] >= 0) o = fmaf(w[x], values2(a.c.v[at[x] + tid]).x * es[x], o);
        }
    }
    if (tid < DH) static_cast<T*>(a.out)[(long long)row * a.o_stride + head * DH + tid] = T(l == 0.f ? 0.f : o / l);
    if (tid == 0 && a.lse) a.lse[(long long)row * a.heads + head] = l == 0.f ? -INFINITY : m + logf(l);
}

bool paged8_ok(const pi_paged_desc& d, const pi_page8_desc& c) {
    return page8_desc_ok(c) && d.heads >= 1 && d.heads <= 1024 && d.heads % c.kv_heads == 0 &&
           d.heads / c.kv_heads <= 128 && d.batch >= 1 && d.batch <= 4096 && d.max_tokens >= 0 &&
           d.max_tokens <= (1 << 24) && d.max_new >= 1 && (d.max_tokens == 0 || d.max_new <= d.max_tokens) &&
           d.max_pages >= 1 && (long long)d.max_pages * c.page_size <= (1ll << 30) && d.window >= 0 &&
           d.scale >= 0.f && isfinite(d.scale);
}

}  // namespace
}  // namespace pi

using namespace pi;

extern "C" {

size_t pi_paged8_workspace_bytes(const pi_paged_desc* desc, const pi_page8_desc* cache) {
    if (!desc || !cache || !paged8_ok(*desc, *cache)) return 0;
    return 256;
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
    if (!aligned(workspace, 16) || ws_bytes < pi_paged8_workspace_bytes(desc, cache)) return PI_ERR_WORKSPACE;
    // queries are read while other rows' outputs are written
    if (rows_overlap(q, 2 * q_stride, 2 * width, out, 2 * out_stride, 2 * width, desc->max_tokens)) return PI_ERR_INVALID_ARG;
    Attn8Args a{};
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
    // a window of all positions a row can hold, or more, is none
    a.window = (long long)desc->window >= (long long)desc->max_pages * cache->page_size ? 0 : desc->window;
    a.group = desc->heads / cache->kv_heads;
    a.scale = desc->scale > 0.f ? desc->scale : 1.0f / sqrtf((float)cache->head_dim);
    a.status = status_word();
    if (a.status == nullptr) return PI_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)desc->max_tokens, (unsigned)desc->heads);
    cudaError_t e;
    if (dtype == PI_T_F16)
        e = cache->head_dim == 128 ? launch_pdl(k_paged_attn8<__half, 128>, grid, 128, 0, s, a)
                                   : launch_pdl(k_paged_attn8<__half, 64>, grid, 128, 0, s, a);
    else
        e = cache->head_dim == 128 ? launch_pdl(k_paged_attn8<__nv_bfloat16, 128>, grid, 128, 0, s, a)
                                   : launch_pdl(k_paged_attn8<__nv_bfloat16, 64>, grid, 128, 0, s, a);
    return e == cudaSuccess ? PI_OK : PI_ERR_CUDA;
}

}  // extern "C"
