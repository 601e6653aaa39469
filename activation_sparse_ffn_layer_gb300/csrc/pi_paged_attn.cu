// pi_paged_attn.cu -- causal attention of new tokens over a paged cache.
//
// The simplest form that is right for every case: a warp per (token, query
// head) walks the visible positions through the block table with a running
// maximum and sum, its lanes holding the head's elements.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pi_common.cuh"
#include "pi_internal.h"

namespace pi {
namespace {

struct PagedArgs {
    const void *q, *k, *v;
    const int32_t *table, *cu, *kv;
    void* out;
    float* lse;
    long long q_stride, o_stride, page_stride, head_stride, token_stride;
    int heads, kv_heads, batch, max_tokens, max_new, max_pages, window, page_size, num_pages;
    float scale;
    int* status;
};

PI_DEV float to_f(__half v) { return __half2float(v); }
PI_DEV float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
PI_DEV void from_f(__half* p, float v) { *p = __float2half_rn(v); }
PI_DEV void from_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T, int DH>
__global__ void __launch_bounds__(128) k_paged_rows(const PagedArgs a) {
    pdl_entry();
    constexpr int E = DH / 32;
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x;
    const int head = blockIdx.y * 4 + (threadIdx.x >> 5);
    if (head >= a.heads) return;
    // the request of row t
    int b = -1, first = 0, n = 0;
    for (int i = 0; i < a.batch; ++i) {
        const int lo = a.cu[i], hi = a.cu[i + 1];
        if (lo < 0 || hi < lo || hi > a.max_tokens || hi - lo > a.max_new) {
            if (lane == 0 && t == 0 && head == 0) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
            continue;
        }
        if (b < 0 && t >= lo && t < hi) {
            b = i;
            first = lo;
            n = hi - lo;
            if (t > 0) break;   // the first row looks at every request
        }
    }
    if (b < 0) return;
    int kv = a.kv[b];
    if (kv < 0 || kv > (long long)a.max_pages * a.page_size) {
        if (lane == 0) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
        kv = 0;
    }
    const int p = kv - n + (t - first);
    const int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
    const int g = head / (a.heads / a.kv_heads);
    const T* qp = static_cast<const T*>(a.q) + t * a.q_stride + (long long)head * DH + lane * E;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = to_f(qp[e]) * a.scale;
        o[e] = 0.f;
    }
    for (int x = lo; x <= p; ++x) {
        const int page = a.table[(size_t)b * a.max_pages + x / a.page_size];
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok && lane == 0) atomicExch(a.status, (int)PI_ERR_INVALID_ARG);
        const long long at = page * a.page_stride + g * a.head_stride + (x % a.page_size) * a.token_stride + lane * E;
        const T *kp = static_cast<const T*>(a.k) + at, *vp = static_cast<const T*>(a.v) + at;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], ok ? to_f(kp[e]) : 0.f, s);
        s = warp_sum(s);
        const float mn = fmaxf(m, s), c = expf(m - mn), w = expf(s - mn);
        l = l * c + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], c, w * (ok ? to_f(vp[e]) : 0.f));
        m = mn;
    }
    T* op = static_cast<T*>(a.out) + t * a.o_stride + (long long)head * DH + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) from_f(op + e, lo <= p ? o[e] / l : 0.f);
    if (a.lse != nullptr && lane == 0) a.lse[(size_t)t * a.heads + head] = lo <= p ? m + logf(l) : -INFINITY;
}

bool paged_ok(const pi_paged_desc& d, const pi_page_desc& c) {
    return page_desc_ok(c) && d.heads >= 1 && d.heads <= 1024 && d.heads % c.kv_heads == 0 &&
           d.heads / c.kv_heads <= 128 && d.batch >= 1 && d.batch <= 4096 && d.max_tokens >= 0 &&
           d.max_tokens <= (1 << 24) && d.max_new >= 1 && (d.max_tokens == 0 || d.max_new <= d.max_tokens) &&
           d.max_pages >= 1 && (long long)d.max_pages * c.page_size <= (1ll << 30) && d.window >= 0 &&
           d.scale >= 0.f && isfinite(d.scale);
}

}  // namespace
}  // namespace pi

using namespace pi;

extern "C" {

size_t pi_paged_workspace_bytes(const pi_paged_desc* desc, const pi_page_desc* cache) {
    if (!desc || !cache || !paged_ok(*desc, *cache)) return 0;
    return 256;
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
    if (!aligned(workspace, 16) || ws_bytes < pi_paged_workspace_bytes(desc, cache)) return PI_ERR_WORKSPACE;
    PagedArgs a{};
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
    a.scale = desc->scale > 0.f ? desc->scale : 1.0f / sqrtf((float)cache->head_dim);
    a.status = status_word();
    if (a.status == nullptr) return PI_ERR_CUDA;
    const dim3 grid((unsigned)desc->max_tokens, (unsigned)((desc->heads + 3) / 4));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (cache->dtype == PI_T_F16)
        e = cache->head_dim == 128 ? launch_pdl(k_paged_rows<__half, 128>, grid, 128, 0, s, a)
                                   : launch_pdl(k_paged_rows<__half, 64>, grid, 128, 0, s, a);
    else
        e = cache->head_dim == 128 ? launch_pdl(k_paged_rows<__nv_bfloat16, 128>, grid, 128, 0, s, a)
                                   : launch_pdl(k_paged_rows<__nv_bfloat16, 64>, grid, 128, 0, s, a);
    return e == cudaSuccess ? PI_OK : PI_ERR_CUDA;
}

}  // extern "C"
