// sq_kv_attention.cu -- attention of the newest tokens over the paged 8-bit
// cache (sq_kv_attention). Included into the library's single translation unit
// after sq_kv.cu, whose cache view and argument checks it uses.
#include <cuda_runtime.h>

#include "sq_device.cuh"
#include "sq_internal.h"

namespace sq {
namespace {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

struct KvAttnArgs {
    KvView c;
    const int32_t *block_table, *seq_len;
    int64_t max_pages, q_stride;
    int n_seqs, q_len, n_q_heads;
    float scale;
    const void* q;
    void* out;
    float* lse;
};

// One warp for each (sequence, query token, query head); a lane holds D / 32
// channels, and the softmax runs along the tokens.
template <typename T, int D>
__global__ void __launch_bounds__(128) kv_attention_kernel(const KvAttnArgs g) {
    constexpr int E = D / 32;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (id >= (int64_t)g.n_seqs * g.q_len * g.n_q_heads) return;
    const int h = (int)(id % g.n_q_heads);
    const int64_t row = id / g.n_q_heads;
    const int b = (int)(row / g.q_len), i = (int)(row % g.q_len);
    int64_t len = __ldg(g.seq_len + b);
    bool bad = len < 0 || len > (g.max_pages << g.c.page_shift);
    len = bad ? 0 : len - g.q_len + 1 + i;
    const T* q = static_cast<const T*>(g.q) + row * g.q_stride + (int64_t)h * D;
    float x[E], o[E];
    for (int e = 0; e < E; ++e) {
        x[e] = to_f32(q[lane * E + e]) * g.scale;
        o[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    const int hk = h / (g.n_q_heads / g.c.n_heads);
    for (int64_t p = 0; p < len; ++p) {
        const int64_t page = __ldg(g.block_table + b * g.max_pages + (p >> g.c.page_shift));
        if ((uint64_t)page >= (uint64_t)g.c.n_pages) { bad = true; break; }
        const int64_t ph = page * g.c.n_heads + hk;
        const int slot = (int)(p & (g.c.page_size - 1));
        const int64_t at = ((ph << g.c.page_shift) + slot) * D + lane * E;
        const int64_t sa = (ph << (g.c.page_shift - g.c.block_shift)) + (slot >> g.c.block_shift);
        float s = 0.0f;
        for (int e = 0; e < E; ++e) s += x[e] * (float)g.c.k[at + e];
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= g.c.k_scale[sa];
        const float mn = fmaxf(m, s);
        const float f = expf(m - mn), w = expf(s - mn);
        m = mn;
        l = l * f + w;
        const float wv = w * g.c.v_scale[sa];
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + wv * (float)g.c.v[at + e];
    }
    if (bad && lane == 0) record_status(SQ_ERR_BOUNDS, SITE_KV_ATTENTION);
    const float nan = __int_as_float(0x7fc00000);
    for (int e = 0; e < E; ++e)
        put(static_cast<T*>(g.out) + (row * g.n_q_heads + h) * D + lane * E + e, bad ? nan : l > 0.0f ? o[e] / l : 0.0f);
    if (g.lse && lane == 0) g.lse[row * g.n_q_heads + h] = bad ? nan : l > 0.0f ? m + logf(l) : -INFINITY;
}

sq_status kv_attention_impl(const void* q, int64_t q_stride, sq_dtype dt, const sq_kv_cache* cache,
                            const int32_t* block_table, int64_t max_pages, const int32_t* seq_len, int64_t n_seqs,
                            int64_t q_len, int64_t n_q_heads, float scale, void* out, float* lse, void* ws,
                            size_t ws_bytes, cudaStream_t st) {
    sq_status r;
    KvAttnArgs g{};
    if ((r = check_kv_dtype(dt)) != SQ_OK) return r;
    if ((r = check_cache(cache, block_table, max_pages, n_seqs, g.c)) != SQ_OK) return r;
    if (q_len < 0 || n_q_heads < 0) { set_error("negative size"); return SQ_ERR_INVALID_ARG; }
    if (!(scale > -3.0e38f && scale < 3.0e38f)) { set_error("scale must be finite"); return SQ_ERR_INVALID_ARG; }
    if (n_q_heads % cache->n_heads != 0) {
        set_error("%lld query heads over %d heads of keys", (long long)n_q_heads, (int)cache->n_heads);
        return SQ_ERR_UNSUPPORTED;
    }
    if (q_len * (n_q_heads / cache->n_heads) > 128 || q_len > 128) {
        set_error("q_len times the query heads of one key head is above 128");
        return SQ_ERR_UNSUPPORTED;
    }
    if (n_seqs == 0 || q_len == 0 || n_q_heads == 0) return SQ_OK;
    const int D = cache->head_dim;
    if ((r = check_rows(q, q_stride, n_q_heads * D, dt == SQ_F32 ? 4 : 2, "q")) != SQ_OK) return r;
    if (!seq_len || !out) { set_error("seq_len or out: NULL pointer"); return SQ_ERR_INVALID_ARG; }
    if (!aligned16(out)) { set_error("out must be 16-byte aligned"); return SQ_ERR_UNSUPPORTED; }
    (void)ws; (void)ws_bytes;
    g.block_table = block_table; g.seq_len = seq_len; g.max_pages = max_pages; g.q_stride = q_stride;
    g.n_seqs = (int)n_seqs; g.q_len = (int)q_len; g.n_q_heads = (int)n_q_heads; g.scale = scale;
    g.q = q; g.out = out; g.lse = lse;
    const dim3 grid((unsigned)((n_seqs * q_len * n_q_heads + 3) / 4)), block(128);
    if (dt == SQ_F32)
        return D == 64 ? launch_pdl("kv_attention_kernel", kv_attention_kernel<float, 64>, grid, block, 0, st, 1, g)
                       : launch_pdl("kv_attention_kernel", kv_attention_kernel<float, 128>, grid, block, 0, st, 1, g);
    return D == 64 ? launch_pdl("kv_attention_kernel", kv_attention_kernel<__nv_bfloat16, 64>, grid, block, 0, st, 1, g)
                   : launch_pdl("kv_attention_kernel", kv_attention_kernel<__nv_bfloat16, 128>, grid, block, 0, st, 1, g);
}

}  // namespace
}  // namespace sq

extern "C" {

size_t sq_kv_attention_workspace_size(const sq_kv_cache* cache, int64_t n_seqs, int64_t q_len, int64_t n_q_heads) {
    (void)cache; (void)n_seqs; (void)q_len; (void)n_q_heads;
    return 0;
}

sq_status sq_kv_attention(const void* q, int64_t q_stride, sq_dtype dt, const sq_kv_cache* cache,
                          const int32_t* block_table, int64_t max_pages, const int32_t* seq_len, int64_t n_seqs,
                          int64_t q_len, int64_t n_q_heads, float scale, void* out, float* lse, void* workspace,
                          size_t ws_bytes, sq_stream_t stream) {
    return sq::kv_attention_impl(q, q_stride, dt, cache, block_table, max_pages, seq_len, n_seqs, q_len, n_q_heads,
                                 scale, out, lse, workspace, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
