// sq_prompt_attention.cu -- attention of packed prompts over themselves
// (sq_prompt_attention). Included into the library's single translation unit
// after sq_kv_attention.cu, some of whose helpers it uses.
#include <cuda_runtime.h>

#include "sq_device.cuh"
#include "sq_internal.h"

namespace sq {
namespace {

struct PromptArgs {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16* out;
    float* lse;
    const int32_t* cu;
    int64_t q_stride, k_stride, v_stride, T;
    int n_seqs, n_q_heads, n_kv_heads;
    float scale;
    bool causal;
};

// One warp for each (token, query head).
template <int D>
__global__ void __launch_bounds__(128) prompt_attention_kernel(const PromptArgs g) {
    constexpr int E = D / 32;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int h = (int)(id % g.n_q_heads);
    const int64_t t = id / g.n_q_heads;
    if (t >= min(g.T, (int64_t)__ldg(g.cu + g.n_seqs))) return;
    const int b = warp_find([&](int i) { return (int64_t)__ldg(g.cu + i); }, g.n_seqs, t);
    if (lane == 0 && (__ldg(g.cu + b) < 0 || __ldg(g.cu + b + 1) > g.T)) record_status(SQ_ERR_BOUNDS, SITE_PROMPT);
    const int64_t u0 = max(0, __ldg(g.cu + b));
    const int64_t u1 = g.causal ? t + 1 : min(g.T, (int64_t)__ldg(g.cu + b + 1));
    const int hk = h / (g.n_q_heads / g.n_kv_heads);
    float x[E], o[E];
    for (int e = 0; e < E; ++e) {
        x[e] = to_f32(g.q[t * g.q_stride + (int64_t)h * D + lane * E + e]) * g.scale;
        o[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int64_t u = u0; u < u1; ++u) {
        float s = 0.0f;
        for (int e = 0; e < E; ++e) s += x[e] * to_f32(g.k[u * g.k_stride + (int64_t)hk * D + lane * E + e]);
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        const float mn = fmaxf(m, s);
        const float f = expf(m - mn), w = expf(s - mn);
        m = mn;
        l = l * f + w;
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * to_f32(g.v[u * g.v_stride + (int64_t)hk * D + lane * E + e]);
    }
    for (int e = 0; e < E; ++e) put(g.out + (t * g.n_q_heads + h) * D + lane * E + e, l > 0.0f ? o[e] / l : 0.0f);
    if (g.lse && lane == 0) g.lse[t * g.n_q_heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

sq_status prompt_attention_impl(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const int32_t* cu, int64_t n_seqs, int64_t T, int64_t n_q_heads,
                                int64_t n_kv_heads, int64_t D, float scale, int causal, void* out, float* lse,
                                cudaStream_t st) {
    sq_status r;
    if (n_seqs < 0 || T < 0 || n_q_heads < 0 || n_kv_heads < 0) { set_error("negative size"); return SQ_ERR_INVALID_ARG; }
    if (D != 64 && D != 128) { set_error("head_dim must be 64 or 128 (got %lld)", (long long)D); return SQ_ERR_UNSUPPORTED; }
    if (!(scale > -3.0e38f && scale < 3.0e38f)) { set_error("scale must be finite"); return SQ_ERR_INVALID_ARG; }
    if (n_seqs > 65536 || n_q_heads > 1024 || T > (int64_t(1) << 30) / (n_q_heads > 0 ? n_q_heads : 1)) {
        set_error("n_seqs, n_q_heads or T too large");
        return SQ_ERR_UNSUPPORTED;
    }
    if (n_seqs == 0 || T == 0 || n_q_heads == 0) return SQ_OK;
    if (n_kv_heads == 0 || n_q_heads % n_kv_heads != 0) {
        set_error("%lld query heads over %lld heads of keys", (long long)n_q_heads, (long long)n_kv_heads);
        return SQ_ERR_UNSUPPORTED;
    }
    if ((r = check_rows(q, q_stride, n_q_heads * D, 2, "q")) != SQ_OK) return r;
    if ((r = check_rows(k, k_stride, n_kv_heads * D, 2, "k")) != SQ_OK) return r;
    if ((r = check_rows(v, v_stride, n_kv_heads * D, 2, "v")) != SQ_OK) return r;
    if (!cu || !out) { set_error("cu_seqlens or out: NULL pointer"); return SQ_ERR_INVALID_ARG; }
    if (!aligned16(out)) { set_error("out must be 16-byte aligned"); return SQ_ERR_UNSUPPORTED; }
    PromptArgs g{static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
                 static_cast<const __nv_bfloat16*>(v), static_cast<__nv_bfloat16*>(out), lse, cu, q_stride, k_stride,
                 v_stride, T, (int)n_seqs, (int)n_q_heads, (int)n_kv_heads, scale, causal != 0};
    const dim3 grid((unsigned)((T * n_q_heads + 3) / 4)), block(128);
    return D == 64 ? launch_pdl("prompt_attention_kernel", prompt_attention_kernel<64>, grid, block, 0, st, 1, g)
                   : launch_pdl("prompt_attention_kernel", prompt_attention_kernel<128>, grid, block, 0, st, 1, g);
}

}  // namespace
}  // namespace sq

extern "C" {

sq_status sq_prompt_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, const int32_t* cu_seqlens, int64_t n_seqs, int64_t T,
                              int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim, float scale, int causal,
                              void* out, float* lse, sq_stream_t stream) {
    return sq::prompt_attention_impl(q, q_stride, k, k_stride, v, v_stride, cu_seqlens, n_seqs, T, n_q_heads, n_kv_heads,
                                     head_dim, scale, causal, out, lse, (cudaStream_t)stream);
}

}  // extern "C"
