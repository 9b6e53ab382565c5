// sq_kv.cu -- what comes behind the QKV projection: the rotary table
// (sq_rope_table), the rotation with the append to the paged 8-bit cache
// (sq_rope_kv_append) and the cache read back as values (sq_kv_read).
// Included into the library's single translation unit after sq_search.cu.
#include <cmath>

#include <cuda_runtime.h>

#include "sq_device.cuh"
#include "sq_internal.h"

namespace sq {

// The caller's cache as the kernels take it.
struct KvView {
    int8_t* k;
    int8_t* v;
    float* k_scale;
    float* v_scale;
    int64_t n_pages;
    int n_heads, page_size, page_shift, block_shift;   // sizes are powers of two
};

namespace {

int log2_of(int64_t v) {
    int s = 0;
    while ((int64_t(1) << s) < v) ++s;
    return s;
}

sq_status check_cache(const sq_kv_cache* c, const int32_t* block_table, int64_t max_pages, int64_t n_seqs, KvView& out) {
    if (!c) { set_error("cache: NULL pointer"); return SQ_ERR_INVALID_ARG; }
    if (n_seqs < 0 || max_pages < 0 || c->n_pages < 0) { set_error("negative size"); return SQ_ERR_INVALID_ARG; }
    if (c->head_dim != 64 && c->head_dim != 128) {
        set_error("head_dim must be 64 or 128 (got %d)", (int)c->head_dim);
        return SQ_ERR_UNSUPPORTED;
    }
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) {
        set_error("page_size must be 16, 32, 64 or 128 (got %d)", (int)c->page_size);
        return SQ_ERR_UNSUPPORTED;
    }
    if (c->scale_block < 1 || c->scale_block > c->page_size || (c->scale_block & (c->scale_block - 1)) != 0) {
        set_error("scale_block must be a power of two up to page_size (got %d)", (int)c->scale_block);
        return SQ_ERR_UNSUPPORTED;
    }
    if (c->n_heads < 1 || c->n_heads > 1024) {
        set_error("the cache must have 1 .. 1024 heads (got %d)", (int)c->n_heads);
        return SQ_ERR_UNSUPPORTED;
    }
    if (n_seqs > 65536) { set_error("more than 65536 sequences"); return SQ_ERR_UNSUPPORTED; }
    if (max_pages * c->page_size > (int64_t(1) << 30) || c->n_pages > 2147483647LL) {
        set_error("block table or cache too large");
        return SQ_ERR_UNSUPPORTED;
    }
    if (c->n_pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) {
        set_error("cache: NULL pointer");
        return SQ_ERR_INVALID_ARG;
    }
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale)) {
        set_error("the cache's arrays must be 16-byte aligned");
        return SQ_ERR_UNSUPPORTED;
    }
    if (n_seqs > 0 && max_pages > 0 && !block_table) { set_error("block_table: NULL pointer"); return SQ_ERR_INVALID_ARG; }
    out = KvView{c->k, c->v, c->k_scale, c->v_scale, c->n_pages, c->n_heads, c->page_size, log2_of(c->page_size),
                 log2_of(c->scale_block)};
    return SQ_OK;
}

sq_status check_rows(const void* p, int64_t stride, int64_t width, int es, const char* name) {
    if (!p) { set_error("%s: NULL pointer", name); return SQ_ERR_INVALID_ARG; }
    if (!aligned16(p) || (stride * es) % 16 != 0) {
        set_error("%s: pointer and token stride must be multiples of 16 bytes", name);
        return SQ_ERR_UNSUPPORTED;
    }
    if (stride < width) { set_error("%s: token stride below the heads' width", name); return SQ_ERR_INVALID_ARG; }
    return SQ_OK;
}

// What an earlier kernel of the stream may have written is read by plain loads behind
// pdl_wait(), never as read-only data (ld.global.nc): these kernels are launched before
// that kernel has ended, and only plain loads are promised to see its writes.
//
// The last b in [0, n) with at(b) <= u, for ascending `at` with at(0) <= u: 32
// candidates at once, so two dependent loads for up to 1024 sequences. Any
// values give a result in [0, n). All lanes of the warp take part.
template <typename F>
__device__ __forceinline__ int warp_find(F at, int n, int64_t u) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + (lane + 1) * step;
        const unsigned m = __ballot_sync(0xffffffffu, i < hi && at(i) <= u);
        lo += __popc(m) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// By all threads of one block of a launch: offsets outside [0, rows] or descending, which the
// kernel cuts, are reported.
__device__ __forceinline__ void check_offsets(const int32_t* cu, int n_seqs, int64_t rows, unsigned int site) {
    for (int b = threadIdx.x; b <= n_seqs; b += blockDim.x) {
        const int64_t a = *(cu + b);
        if (a < 0 || a > rows || (b > 0 && a < *(cu + b - 1))) record_status(SQ_ERR_BOUNDS, site);
    }
}

// ---------------------------------------------------------------- 8 channels of a head
template <typename T> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&x)[8]) {
        const uint4 r = *reinterpret_cast<const uint4*>(p);
        x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x); x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y);
        x[4] = bf16_lo(r.z); x[5] = bf16_hi(r.z); x[6] = bf16_lo(r.w); x[7] = bf16_hi(r.w);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                  pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
};
template <> struct Chunk<float> {
    static __device__ __forceinline__ void load(const float* p, float (&x)[8]) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// The same 8 channels as they lie in memory, so that loads can be far ahead of their use.
template <typename T> struct RawEight {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        if constexpr (sizeof(T) == 2) {
            x[0] = bf16_lo(v[0].x); x[1] = bf16_hi(v[0].x); x[2] = bf16_lo(v[0].y); x[3] = bf16_hi(v[0].y);
            x[4] = bf16_lo(v[0].z); x[5] = bf16_hi(v[0].z); x[6] = bf16_lo(v[0].w); x[7] = bf16_hi(v[0].w);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[4 * i] = __uint_as_float(v[i].x); x[4 * i + 1] = __uint_as_float(v[i].y);
                x[4 * i + 2] = __uint_as_float(v[i].z); x[4 * i + 3] = __uint_as_float(v[i].w);
            }
        }
    }
};

// Lane c of a head's head_dim / 16 lanes holds two chunks of 8 channels: for
// c < rot/16 the chunks c and c + rot/16, which hold each other's partners in the
// half layout (and whole pairs in the interleaved one); the other lanes hold
// the channels behind rot_dim, two chunks each.
__device__ __forceinline__ void lane_chunks(int c, int rot, int& a, int& b) {
    const int r = rot >> 4;
    a = c < r ? c : 2 * c;
    b = c < r ? c + r : 2 * c + 1;
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float y = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = y;
}

// xa, xb: this lane's chunks; cs: the position's table row.
__device__ __forceinline__ void rotate_lane(float (&xa)[8], float (&xb)[8], const float* cs, int c, int rot, bool pairs) {
    if (c >= (rot >> 4)) return;
    if (pairs) {
        const float4* ta = reinterpret_cast<const float4*>(cs + 8 * c);
        const float4* tb = reinterpret_cast<const float4*>(cs + 8 * (c + (rot >> 4)));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 u = ta[i], w = tb[i];
            turn(xa[4 * i], xa[4 * i + 1], u.x, u.y);
            turn(xa[4 * i + 2], xa[4 * i + 3], u.z, u.w);
            turn(xb[4 * i], xb[4 * i + 1], w.x, w.y);
            turn(xb[4 * i + 2], xb[4 * i + 3], w.z, w.w);
        }
    } else {
        const float4* t = reinterpret_cast<const float4*>(cs + 16 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 u = t[i];
            turn(xa[2 * i], xb[2 * i], u.x, u.y);
            turn(xa[2 * i + 1], xb[2 * i + 1], u.z, u.w);
        }
    }
}

__device__ __forceinline__ uint32_t code_of(float x, float s) {
    const int q = __float2int_rn(__fdiv_rn(x, s));
    return (uint32_t)max(-127, min(127, q)) & 0xffu;
}
// clamp(round(RN(x / s))) of 8 values. x RN(1 / s) is within 3 2^-24 of RN(x / s) relatively,
// so below 3e-5 for the |x / s| <= 127.5 that occur here; a value within 2^-13 of a half
// integer is divided, the others cannot round differently. 1.5 2^23 added and
// taken away rounds to the nearest integer, ties to even, and leaves the code in the
// sum's low byte. A scale below 2^-100 (reciprocals near the top of fp32's range,
// quotients that may pass 127) takes the divisions and the clamp.
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float s) {
    if (!(s > 0.0f)) return make_uint2(0u, 0u);
    uint32_t t[8];
    const float r = __frcp_rn(s);
    bool near = !(s >= 7.888609052210118e-31f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = __fmul_rn(x[i], r);
        const float m = __fadd_rn(q, 12582912.0f);
        t[i] = __float_as_uint(m);
        near |= !(fabsf(__fsub_rn(q, __fsub_rn(m, 12582912.0f))) < 0.5f - 1.220703125e-4f);
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = code_of(x[i], s);
    }
    return make_uint2(__byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410));
}
__device__ __forceinline__ float code_at(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }
__device__ __forceinline__ uint2 requantize(uint2 w, float was, float s) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = __fmul_rn(code_at(w.x, i), was);
        x[4 + i] = __fmul_rn(code_at(w.y, i), was);
    }
    return codes_of(x, s);
}

// ================================================================== rotary table
// A thread has one frequency and RUN positions in a row: it works out the first angle's
// cosine and sine and those of one step, and turns by the step from position to
// position, z' = z (cos w + i sin w): four fp64 products an entry in place of a sincos. Each
// turn adds at most some 2^-52, so 32 of them stay far below the one rounding to fp32
// (2^-24). Longer runs amortise the two sincos and the power, shorter ones fill the GPU:
// 131,072 positions x 64
// frequencies (67 MB) take 13.5 us, 0.76 of the measured copy rate; with a sincos for every
// entry they took 32.
struct RopeFreq {
    double theta, factor, low, high, orig, magnitude;
};

template <int RUN>
__global__ void __launch_bounds__(256)
rope_table_kernel(float2* __restrict__ table, int64_t first, int64_t n_pos, int half, RopeFreq f) {
    pdl_wait();
    pdl_trigger();
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int i = (int)(id % half);
    const int64_t p0 = id / half * RUN;
    if (p0 >= n_pos) return;
    double w = pow(f.theta, -(double)i / (double)half);
    if (f.high > 0.0) {
        const double turns = f.orig * w / 6.283185307179586476925286766559;
        const double b = fmin(fmax((turns - f.low) / (f.high - f.low), 0.0), 1.0);
        w = (1.0 - b) * w / f.factor + b * w;
    } else {
        w = w / f.factor;
    }
    double s, c, ds, dc;
    sincos((double)(first + p0) * w, &s, &c);
    sincos(w, &ds, &dc);
    s *= f.magnitude;
    c *= f.magnitude;
    const int n = (int)min((int64_t)RUN, n_pos - p0);
    float2* out = table + p0 * half + i;
    for (int k = 0; k < n; ++k) {
        out[(int64_t)k * half] = make_float2((float)c, (float)s);
        const double t = c * dc - s * ds;
        s = s * dc + c * ds;
        c = t;
    }
}

// ================================================================== rotate and append
// Work is cut into spans of max(scale_block, 16) positions, which lie in one
// page. A sequence of n new tokens touches at most n / span + 2 of them; with
// U_b = cu[b] / span + 2 b the spans of sequence b have the numbers U_b, U_b + 1, ..,
// below U_{b+1}: no scan over the batch, and the host needs only T and n_seqs.
struct AppendArgs {
    KvView c;
    const int32_t *block_table, *ctx_len, *cu;
    int64_t max_pages, n_pos, T, q_stride, k_stride, v_stride;
    int n_seqs, n_q_heads, rot, span_shift;
    bool pairs;
    const void *q, *k, *v;
    void *q_out, *k_out;
    const float* table;
};

constexpr int kQRows = 128;   // (position, query head) rows of one block: 8 heads of 16 positions .. 1 of 128

// A block has a span of one head of K or of V, or of some query heads; NP passes of
// THREADS / (D / 16) rows cover the span. Small blocks, because a block is a chain of
// dependent steps (its sequence, its rows, their maximum, the codes) that only
// other blocks on the SM can hide: 1024 threads of 64 registers an SM take 62 us for five
// prompts of 3,500 tokens and 32 heads, 512 of 126 took 81. Each thread also reads the row
// maxima of its whole scale block from shared memory. The four passes of a span of 128 tokens
// and heads of 128 do not fit 64 registers and spill 624 to 660 bytes a thread.
template <typename T, int D, int THREADS, int NP>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
rope_append_kernel(const AppendArgs g) {
    constexpr int LPR = D / 16;          // lanes of a row
    constexpr int RP = THREADS / LPR;    // rows of a pass
    __shared__ float row_max[128];
    pdl_wait();
    pdl_trigger();
    const int64_t u = blockIdx.x;
    const int32_t* cu = g.cu;
    const int sh = g.span_shift;
    auto start_of = [&](int b) { return (int64_t)(*(cu + b) >> sh) + 2 * (int64_t)b; };
    if (u + 1 == gridDim.x) {   // behind the last span: a block that looks at the offsets and has nothing else in registers
        if (blockIdx.y == 0) check_offsets(cu, g.n_seqs, g.T, SITE_KV_APPEND);
        return;
    }
    if (u >= start_of(g.n_seqs)) return;
    const int b = warp_find(start_of, g.n_seqs, u);
    const int64_t j = u - start_of(b);
    const int64_t t0 = max(0, *(cu + b));
    const int64_t n = min((int64_t)*(cu + b + 1), g.T) - t0;
    const int64_t ctx = *(g.ctx_len + b);
    if (j < 0 || n <= 0) return;
    const int64_t span0 = ctx < 0 ? j << sh : ((ctx >> sh) + j) << sh;      // first position of the span
    const int64_t lo = max(span0, ctx), hi = min(span0 + (1 << sh), max((int64_t)0, ctx) + n);
    if (lo >= hi) return;
    // positions the tables cover; the others give NaN
    const int64_t most = min(g.max_pages << g.c.page_shift, g.rot > 0 ? g.n_pos : (int64_t)1 << 62);
    const int64_t ok = ctx < 0 ? lo : min(hi, most);
    if (ok < hi && threadIdx.x == 0 && blockIdx.y == 0) record_status(SQ_ERR_BOUNDS, SITE_KV_APPEND);
    const int64_t base = max((int64_t)0, ctx);

    if ((int)blockIdx.y >= 2 * g.c.n_heads) {   // ---- query heads
        const int per = kQRows >> sh;
        const int h0 = ((int)blockIdx.y - 2 * g.c.n_heads) * per;
        const int nh = min(per, g.n_q_heads - h0);
        const int rows = (int)(hi - lo) * nh;
        const int c = threadIdx.x % LPR;
        int ca, cb;
        lane_chunks(c, g.rot, ca, cb);
        constexpr int Q = 2, STEP = THREADS / LPR;   // rows in flight; rows apart
        for (int r0 = threadIdx.x / LPR; r0 < rows; r0 += Q * STEP) {
            RawEight<T> ra[Q], rb[Q];
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                const int r = r0 + k * STEP;
                if (r >= rows) break;
                const T* x = static_cast<const T*>(g.q) + (t0 + lo - base + r / nh) * g.q_stride + (int64_t)(h0 + r % nh) * D;
                ra[k].load(x + 8 * ca);
                rb[k].load(x + 8 * cb);
            }
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                const int r = r0 + k * STEP;
                if (r >= rows) break;
                const int64_t p = lo + r / nh;
                T* y = static_cast<T*>(g.q_out) + ((t0 + p - base) * g.n_q_heads + h0 + r % nh) * D;
                float xa[8], xb[8];
                ra[k].get(xa);
                rb[k].get(xb);
                if (p < ok) {
                    rotate_lane(xa, xb, g.table + p * g.rot, c, g.rot, g.pairs);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) xa[i] = xb[i] = __int_as_float(0x7fc00000);
                }
                Chunk<T>::store(y + 8 * ca, xa);
                Chunk<T>::store(y + 8 * cb, xb);
            }
        }
        return;
    }

    // ---- one head of K or of V
    const bool is_v = (int)blockIdx.y >= g.c.n_heads;
    const int h = (int)blockIdx.y - (is_v ? g.c.n_heads : 0);
    const int c = threadIdx.x % LPR;
    const int r0 = threadIdx.x / LPR;
    int64_t page = -1;
    if (lo < ok) {
        page = *(g.block_table + b * g.max_pages + (span0 >> g.c.page_shift));
        if ((uint64_t)page >= (uint64_t)g.c.n_pages) {
            if (threadIdx.x == 0) record_status(SQ_ERR_BOUNDS, SITE_KV_APPEND);
            page = -1;
        }
    }
    int ca, cb;
    lane_chunks(c, is_v ? 0 : g.rot, ca, cb);
    const int span = 1 << sh;
    RawEight<T> ra[NP], rb[NP];
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        const int r = s * RP + r0;
        const int64_t p = span0 + r;
        if (r < span && p >= lo && p < hi) {
            const int64_t t = t0 + p - base;
            const T* x = (is_v ? static_cast<const T*>(g.v) + t * g.v_stride : static_cast<const T*>(g.k) + t * g.k_stride) + (int64_t)h * D;
            ra[s].load(x + 8 * ca);
            rb[s].load(x + 8 * cb);
        }
    }
    float xa[NP][8], xb[NP][8];
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        const int r = s * RP + r0;
        const int64_t p = span0 + r;
        float m = 0.0f;
        if (r < span && p >= lo && p < hi) {
            const int64_t t = t0 + p - base;
            ra[s].get(xa[s]);
            rb[s].get(xb[s]);
            if (p < ok) {
                if (!is_v) rotate_lane(xa[s], xb[s], g.table + p * g.rot, c, g.rot, g.pairs);
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(xa[s][i]), fabsf(xb[s][i])));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) xa[s][i] = xb[s][i] = __int_as_float(0x7fc00000);
            }
            if (!is_v && g.k_out) {
                T* y = static_cast<T*>(g.k_out) + (t * g.c.n_heads + h) * D;
                Chunk<T>::store(y + 8 * ca, xa[s]);
                Chunk<T>::store(y + 8 * cb, xb[s]);
            }
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (c == 0 && r < span) row_max[r] = m;
    }
    if (page < 0) return;   // the whole block
    const int bs = g.c.block_shift, block = 1 << bs;
    const int slot0 = (int)(span0 & (g.c.page_size - 1));
    float* scales = (is_v ? g.c.v_scale : g.c.k_scale) + ((page * g.c.n_heads + h) << (g.c.page_shift - bs));
    int8_t* codes = (is_v ? g.c.v : g.c.k) + ((page * g.c.n_heads + h) << g.c.page_shift) * D;
    float was[NP];
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        const int r = s * RP + r0;
        const int64_t first = span0 + (r >> bs << bs);   // of the row's scale block
        was[s] = r < span && first < ctx && first + block > ctx ? scales[(slot0 + r) >> bs] : 0.0f;
    }
    __syncthreads();   // row maxima are written, old scales are read
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        const int r = s * RP + r0;
        if (r >= span) continue;
        const int64_t p = span0 + r;
        const int g0 = r >> bs << bs;
        const int64_t first = span0 + g0;
        if (p >= ok || first + block <= lo) continue;   // nothing of this row, or of its block, is new
        float m = 0.0f;
        for (int i = 0; i < block; ++i) m = fmaxf(m, row_max[g0 + i]);
        const float scale = fmaxf(was[s], __fdiv_rn(m, 127.0f));
        int8_t* row = codes + (int64_t)(slot0 + r) * D;
        if (p >= lo) {
            *reinterpret_cast<uint2*>(row + 8 * ca) = codes_of(xa[s], scale);
            *reinterpret_cast<uint2*>(row + 8 * cb) = codes_of(xb[s], scale);
            if (c == 0 && p == max(lo, first)) scales[(slot0 + r) >> bs] = scale;
        } else if (scale != was[s]) {   // an earlier token of a block whose scale grew
            uint2* wa = reinterpret_cast<uint2*>(row + 8 * ca);
            uint2* wb = reinterpret_cast<uint2*>(row + 8 * cb);
            *wa = requantize(*wa, was[s], scale);
            *wb = requantize(*wb, was[s], scale);
        }
    }
}

// ================================================================== read back
// A lane has 16 codes of K and of V of one (token, head): 16-byte loads, whole sectors both
// ways. Bound by HBM: 870 MB of sixteen prefixes of 32 heads in 153 us, 0.87 of the
// measured copy rate.
template <typename T, int D>
__global__ void __launch_bounds__(256)
kv_read_kernel(const KvView g, const int32_t* block_table, int64_t max_pages, const int32_t* first, const int32_t* cu, int n_seqs,
               int64_t rows, T* k_out, T* v_out) {
    constexpr int LPR = D / 16;
    pdl_wait();
    pdl_trigger();
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t flat = id / LPR;
    const int c = (int)(id % LPR);
    if (blockIdx.x + 1 == gridDim.x) {   // behind the last row
        check_offsets(cu, n_seqs, rows, SITE_KV_READ);
        return;
    }
    // the block's first row by search, the thread's own from there
    const int64_t total = min(rows, (int64_t)*(cu + n_seqs));
    const int64_t t_block = (int64_t)blockIdx.x * (256 / LPR) / g.n_heads;
    if (t_block >= total) return;
    int b = warp_find([&](int i) { return (int64_t)*(cu + i); }, n_seqs, t_block);
    const int64_t t = flat / g.n_heads;
    if (t >= total) return;
    while (b + 1 < n_seqs && *(cu + b + 1) <= t) ++b;
    if (t < *(cu + b)) return;   // in front of the first sequence
    const int h = (int)(flat % g.n_heads);
    const int64_t p = (int64_t)*(first + b) + t - *(cu + b);
    int64_t page = -1;
    if (p >= 0 && p < (max_pages << g.page_shift)) page = *(block_table + b * max_pages + (p >> g.page_shift));
    const bool ok = (uint64_t)page < (uint64_t)g.n_pages;
    if (!ok && c == 0) record_status(SQ_ERR_BOUNDS, SITE_KV_READ);
    const int64_t ph = ok ? page * g.n_heads + h : 0;
    const int slot = (int)(p & (g.page_size - 1));
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
        float x[2][8];
        if (ok) {
            const uint4 w = *reinterpret_cast<const uint4*>((is_v ? g.v : g.k) + ((ph << g.page_shift) + slot) * D + 16 * c);
            const float s = (is_v ? g.v_scale : g.k_scale)[(ph << (g.page_shift - g.block_shift)) + (slot >> g.block_shift)];
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i >> 3][i & 7] = __fmul_rn(code_at(ws[i >> 2], i & 3), s);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i >> 3][i & 7] = __int_as_float(0x7fc00000);
        }
        T* y = (is_v ? v_out : k_out) + flat * D + 16 * c;
        Chunk<T>::store(y, x[0]);
        Chunk<T>::store(y + 8, x[1]);
    }
}

// ================================================================== host side
sq_status check_kv_dtype(sq_dtype dt) {
    if (dt != SQ_F32 && dt != SQ_BF16) {
        set_error("dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)dt);
        return SQ_ERR_UNSUPPORTED;
    }
    return SQ_OK;
}

template <typename T, int D>
sq_status launch_append(const AppendArgs& g, dim3 grid, cudaStream_t st) {
    constexpr int RP = 4096 / D;   // rows of a pass of 256 threads
    const int span = 1 << g.span_shift;
    if (span <= 2048 / D) return launch_pdl("rope_append_kernel", rope_append_kernel<T, D, 128, 1>, grid, dim3(128), 0, st, 1, g);
    if (span <= RP) return launch_pdl("rope_append_kernel", rope_append_kernel<T, D, 256, 1>, grid, dim3(256), 0, st, 1, g);
    if (D == 64 || span <= 2 * RP) return launch_pdl("rope_append_kernel", rope_append_kernel<T, D, 256, 2>, grid, dim3(256), 0, st, 1, g);
    if constexpr (D == 128)   // a span of 128 tokens
        return launch_pdl("rope_append_kernel", rope_append_kernel<T, D, 256, 4>, grid, dim3(256), 0, st, 1, g);
}

sq_status rope_table_impl(float* table, int64_t first, int64_t n_pos, int64_t rot, double theta,
                          const sq_rope_scaling* sc, cudaStream_t st) {
    if (first < 0 || n_pos < 0) { set_error("negative position or size"); return SQ_ERR_INVALID_ARG; }
    if (rot <= 0 || rot % 16 != 0 || rot > 256) {
        set_error("rot_dim must be a multiple of 16 in 16 .. 256 (got %lld)", (long long)rot);
        return SQ_ERR_UNSUPPORTED;
    }
    if (first > (int64_t(1) << 31) || n_pos > (int64_t(1) << 31) - first) {
        set_error("positions beyond 2^31");
        return SQ_ERR_UNSUPPORTED;
    }
    RopeFreq f{theta, 1.0, 0.0, 0.0, 0.0, 1.0};
    if (sc) f = RopeFreq{theta, sc->factor, sc->low_turns, sc->high_turns, (double)sc->original_len, sc->magnitude};
    if (!(f.theta > 0.0) || !std::isfinite(f.theta) || !(f.factor > 0.0) || !std::isfinite(f.factor) ||
        !std::isfinite(f.magnitude)) {
        set_error("theta and factor must be positive and finite, magnitude finite");
        return SQ_ERR_INVALID_ARG;
    }
    if (f.high != 0.0 && !(f.low >= 0.0 && f.high > f.low && std::isfinite(f.high) && f.orig > 0.0)) {
        set_error("scaling by turns needs high_turns > low_turns >= 0 and original_len > 0");
        return SQ_ERR_INVALID_ARG;
    }
    if (n_pos == 0) return SQ_OK;
    if (!table) { set_error("table: NULL pointer"); return SQ_ERR_INVALID_ARG; }
    if (!aligned16(table)) { set_error("table must be 16-byte aligned"); return SQ_ERR_UNSUPPORTED; }
    const int half = (int)(rot / 2);
    // Runs of 32 where they still fill the GPU's threads, else of 4.
    const bool many = n_pos / 32 * half >= (int64_t)device_info().sm_count * 1024;
    const int run = many ? 32 : 4;
    const int64_t threads = (n_pos + run - 1) / run * half;
    return launch_pdl("rope_table_kernel", many ? rope_table_kernel<32> : rope_table_kernel<4>,
                      dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st, 1, reinterpret_cast<float2*>(table), first,
                      n_pos, half, f);
}

sq_status rope_append_impl(const sq_kv_cache* cache, const int32_t* block_table, int64_t max_pages, const int32_t* ctx_len,
                           const int32_t* cu_new, int64_t n_seqs, int64_t T, const void* q, int64_t q_stride,
                           int64_t n_q_heads, const void* k, int64_t k_stride, const void* v, int64_t v_stride, sq_dtype dt,
                           const float* table, int64_t n_pos, int64_t rot, int interleaved, void* q_out, void* k_out,
                           cudaStream_t st) {
    sq_status r;
    AppendArgs g{};
    if ((r = check_kv_dtype(dt)) != SQ_OK) return r;
    if ((r = check_cache(cache, block_table, max_pages, n_seqs, g.c)) != SQ_OK) return r;
    if (T < 0 || n_q_heads < 0 || n_pos < 0 || rot < 0) { set_error("negative size"); return SQ_ERR_INVALID_ARG; }
    if (T > (int64_t(1) << 30) || n_q_heads > 1024) { set_error("T or n_q_heads too large"); return SQ_ERR_UNSUPPORTED; }
    const int D = cache->head_dim, es = dt == SQ_F32 ? 4 : 2;
    if (rot % 16 != 0 || rot > D) {
        set_error("rot_dim must be a multiple of 16 up to head_dim (got %lld)", (long long)rot);
        return SQ_ERR_UNSUPPORTED;
    }
    if (n_seqs == 0 || T == 0) return SQ_OK;
    if (!ctx_len || !cu_new) { set_error("ctx_len or cu_new: NULL pointer"); return SQ_ERR_INVALID_ARG; }
    if ((r = check_rows(k, k_stride, (int64_t)cache->n_heads * D, es, "k")) != SQ_OK) return r;
    if ((r = check_rows(v, v_stride, (int64_t)cache->n_heads * D, es, "v")) != SQ_OK) return r;
    if (n_q_heads > 0) {
        if ((r = check_rows(q, q_stride, n_q_heads * D, es, "q")) != SQ_OK) return r;
        if (!q_out) { set_error("q_out: NULL pointer"); return SQ_ERR_INVALID_ARG; }
    }
    if (rot > 0 && !table) { set_error("table: NULL pointer"); return SQ_ERR_INVALID_ARG; }
    if (!aligned16(table) || !aligned16(q_out) || !aligned16(k_out)) {
        set_error("table, q_out and k_out must be 16-byte aligned");
        return SQ_ERR_UNSUPPORTED;
    }
    g.block_table = block_table; g.ctx_len = ctx_len; g.cu = cu_new;
    g.max_pages = max_pages; g.n_pos = n_pos; g.T = T;
    g.q_stride = q_stride; g.k_stride = k_stride; g.v_stride = v_stride;
    g.n_seqs = (int)n_seqs; g.n_q_heads = (int)n_q_heads; g.rot = (int)rot; g.pairs = interleaved != 0;
    g.q = q; g.k = k; g.v = v; g.q_out = q_out; g.k_out = k_out; g.table = table;
    const int span = cache->scale_block > 16 ? cache->scale_block : 16;
    g.span_shift = log2_of(span);
    const dim3 grid((unsigned)(T / span + 2 * n_seqs + 1), (unsigned)(2 * cache->n_heads + (n_q_heads + kQRows / span - 1) / (kQRows / span)));
    if (dt == SQ_F32) return D == 64 ? launch_append<float, 64>(g, grid, st) : launch_append<float, 128>(g, grid, st);
    return D == 64 ? launch_append<__nv_bfloat16, 64>(g, grid, st) : launch_append<__nv_bfloat16, 128>(g, grid, st);
}

sq_status kv_read_impl(const sq_kv_cache* cache, const int32_t* block_table, int64_t max_pages, const int32_t* first,
                       const int32_t* cu_out, int64_t n_seqs, int64_t T, void* k_out, void* v_out, sq_dtype dt,
                       cudaStream_t st) {
    sq_status r;
    KvView g;
    if ((r = check_kv_dtype(dt)) != SQ_OK) return r;
    if ((r = check_cache(cache, block_table, max_pages, n_seqs, g)) != SQ_OK) return r;
    if (T < 0) { set_error("negative size"); return SQ_ERR_INVALID_ARG; }
    if (T > (int64_t(1) << 30)) { set_error("T too large"); return SQ_ERR_UNSUPPORTED; }
    if (n_seqs == 0 || T == 0) return SQ_OK;
    if (!first || !cu_out || !k_out || !v_out) { set_error("NULL pointer"); return SQ_ERR_INVALID_ARG; }
    if (!aligned16(k_out) || !aligned16(v_out)) { set_error("outputs must be 16-byte aligned"); return SQ_ERR_UNSUPPORTED; }
    const int D = cache->head_dim;
    const int64_t blocks = (T * cache->n_heads * (D / 16) + 255) / 256;
    if (blocks >= 2147483647LL) { set_error("T too large"); return SQ_ERR_UNSUPPORTED; }
    const dim3 grid((unsigned)blocks + 1), block(256);
#define SQ_READ(TT, DD)                                                                                              \
    launch_pdl("kv_read_kernel", kv_read_kernel<TT, DD>, grid, block, 0, st, 1, g, block_table, max_pages, first,    \
               cu_out, (int)n_seqs, T, static_cast<TT*>(k_out), static_cast<TT*>(v_out))
    if (dt == SQ_F32) return D == 64 ? SQ_READ(float, 64) : SQ_READ(float, 128);
    return D == 64 ? SQ_READ(__nv_bfloat16, 64) : SQ_READ(__nv_bfloat16, 128);
#undef SQ_READ
}

}  // namespace
}  // namespace sq

extern "C" {

sq_status sq_rope_table(float* table, int64_t first_pos, int64_t n_pos, int64_t rot_dim, double theta,
                        const sq_rope_scaling* scaling, sq_stream_t stream) {
    return sq::rope_table_impl(table, first_pos, n_pos, rot_dim, theta, scaling, (cudaStream_t)stream);
}

sq_status sq_rope_kv_append(const sq_kv_cache* cache, const int32_t* block_table, int64_t max_pages,
                            const int32_t* ctx_len, const int32_t* cu_new, int64_t n_seqs, int64_t T,
                            const void* q, int64_t q_stride, int64_t n_q_heads, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, sq_dtype dt, const float* table, int64_t n_pos,
                            int64_t rot_dim, int interleaved, void* q_out, void* k_out, sq_stream_t stream) {
    return sq::rope_append_impl(cache, block_table, max_pages, ctx_len, cu_new, n_seqs, T, q, q_stride, n_q_heads, k,
                                k_stride, v, v_stride, dt, table, n_pos, rot_dim, interleaved, q_out, k_out,
                                (cudaStream_t)stream);
}

sq_status sq_kv_read(const sq_kv_cache* cache, const int32_t* block_table, int64_t max_pages, const int32_t* first,
                     const int32_t* cu_out, int64_t n_seqs, int64_t T, void* k_out, void* v_out, sq_dtype dt,
                     sq_stream_t stream) {
    return sq::kv_read_impl(cache, block_table, max_pages, first, cu_out, n_seqs, T, k_out, v_out, dt, (cudaStream_t)stream);
}

}  // extern "C"
