// sq_kv_attention.cu -- attention of the newest tokens over the paged 8-bit
// cache (sq_kv_attention). Included into the library's single translation unit
// after sq_kv.cu, whose cache view and argument checks it uses.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sq_device.cuh"
#include "sq_internal.h"

namespace sq {
namespace {

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
    long long wait_limit;
    int64_t* border;    // in the workspace: where each CTA's share begins, and the end of the last;
    int4* start;        // what that tile is (sequence, head, tile, tiles of the sequence);
    float2* part_ml;    // and two partial results of each CTA
    float* part_o;
};

// The kernel. Every key/value head's G = n_q_heads / n_heads query heads times q_len query
// tokens are R rows that share its keys: reading the codes is the floor, so
// they go from HBM through a ring of shared-memory stages (TMA, one page
// of one head a copy) once per head, whatever R is.
//   Work: tiles of 128 tokens, numbered by sequence, head, tile. The CTAs, one on each
// SM, take equal shares of all W tiles, wherever the sequences' borders fall, so a
// ragged batch is balanced without the host knowing a length. A (sequence, head)
// that several CTAs share leaves one partial result (reference, sum, accumulator) from
// each in the workspace; a second small kernel joins them in a fixed order.
//   Inside a CTA the consumer warps take groups of 32 tokens in turn (with more than 16
// rows each group is taken once for each of MT row tiles); a warp keeps a softmax
// reference, sum and accumulator of its own, and they meet once at the end of a
// head's piece: no barrier between warps inside the loop.
//   S^T = K Q^T and O^T += V^T P^T are m16n8k16 products with fp32 accumulators: tokens
// and channels make the 16 sides, rows the sides of 8, because R is often 8 or less. The
// channels of a k step may come in any order as long as Q and K agree, and the rows of S^T
// may be any tokens: the orders here are those in which one 16-byte shared-memory
// read gives a lane its codes without bank conflicts. S^T's accumulators become P^T's
// operand by an 8 x 8 transpose in registers.
//   Measured: 697 MB of a ragged batch of 64 sequences and 8 heads in 135 us, 0.79 of the
// measured copy rate (its loads alone take 111); 268 MB of one sequence of 131,072
// tokens in 51 us, 0.80. Some 40 integer and fp16
// instructions for 16 codes keep the warps at about the pace of HBM.
//   A code c becomes fp16 exactly: (c ^ 0x80) under the byte 0x64 is 1024 + c + 128.
//   Scales: a key's scale multiplies its score. A value's scale multiplies its weight:
// w = 2^(s - m) vs goes to the second product, 2^(s - m) into the sum. The reference m is
// moved only when some 2^(s - m) max(vs, 2^-80) is above 2^15 (rare after the first
// groups); then it becomes the largest s + max(floor(log2 vs), -80), less 7, so that the
// largest w is 2^7 .. 2^8 for scales from 2^-80 up: 2^8 below the limit, and 2^-32 of it is
// what fp16's smallest step, 2^-24, leaves of small weights. (Kept at 1 .. 2, weights below 2^-25 of
// the largest were lost: an eighth of a result that 32,767 of them made.)
constexpr int kTile = 128;
// Eight consumer warps of 224 registers, so that every accumulator and a group's codes
// stay in them for bf16 queries, but for 160 bytes a thread with 9 to 16 rows and heads of
// 128; fp32 queries with their second parts spill 44 to 178 bytes with heads of 128, 56
// with 9 to 16 rows and heads of 64. (Twelve warps of 152 spilled with 8 rows too: 148 us
// for the ragged batch of 64 sequences, eight 133 to 135.) And a warpgroup whose first two
// warps load. 168 registers at launch times 12
// warps are as many as 224 times 8 and 56 times 4.
constexpr int kConsumers = 8;
constexpr int kAttnThreads = 32 * (kConsumers + 4);
constexpr int kConsumerRegs = 224, kProducerRegs = 56;
constexpr int kGroup = 32;                    // tokens of a warp's step
constexpr int kGroups = kTile / kGroup;
constexpr float kMaxWeight = 32768.0f;        // fp16 ends at 65504
constexpr int kHeadroom = 7;                  // a new reference makes the largest weight 2^7 .. 2^8
constexpr float kNoReference = -1.0e30f;      // nothing seen yet: 2^(s - m) is infinite for any score, 0 for a masked one
// Scales below 2^-80, zero among them, count as 2^-80 where the reference is chosen and where it
// is found too low: a weight of 2^(s - m) that its value's scale makes small or zero could
// overflow in the sum otherwise. Each stays below 2^95, the sum over 2^30 tokens below 2^125. The
// floor costs 1% and less, but 6% with fp32 queries, heads of 64 and 128 rows (266 against 284 us
// for 64 sequences of 4,096 tokens and 4 heads); looking at the sums, or at them only
// where a scale is that small, cost up to 3% more with 32 to 128 rows.
constexpr float kNoScale = -80.0f, kLeastScale = 0x1p-80f;

// NB sides of 8 rows a warp, MT row tiles. MT == 1: the queries of a piece travel with its first tile.
template <typename T, int D, int NB, int MT>
struct AttnSmem {
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int CODES = kTile * D;                              // bytes of K, and of V
    static constexpr int Q = 2 * CODES + 2 * kTile * 4;                  // behind the codes and their scales
    static constexpr int STAGE = Q + (MT == 1 ? 8 * NB * D * (int)sizeof(T) : 0);
    static constexpr int DB = D / 8;
    static constexpr int ROW = D == 128 ? 164 : 100;                     // floats of a merge row: a gap of 4 behind every DB, and
                                                                         // 4 mod 8, so that the 16-byte accesses meet no conflict
    static constexpr int MERGE = kConsumers * 8 * ROW * 4;
    static constexpr int TOTAL = 1024 + STAGES * STAGE + MERGE;
    static_assert(STAGE % 1024 == 0, "a stage keeps the swizzle's alignment");
    static_assert(TOTAL <= 227 * 1024 - 4096, "");
};

__device__ __forceinline__ uint32_t lop_and_xor(uint32_t x, uint32_t m, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(x), "r"(m), "r"(c));   // (x & m) ^ c
    return r;
}
__device__ __forceinline__ uint32_t sub_1152(uint32_t h) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// Codes (0, 2) and (1, 3) of a word as fp16 pairs.
__device__ __forceinline__ void codes_even_odd(uint32_t w, uint32_t& even, uint32_t& odd) {
    even = sub_1152(lop_and_xor(w, 0x00ff00ffu, 0x64806480u));
    odd = sub_1152(lop_and_xor(w >> 8, 0x00ff00ffu, 0x64806480u));
}
// Code i of a and of b as an fp16 pair.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t a, uint32_t b) {
    return sub_1152(lop_and_xor(__byte_perm(a, b, (4 + I) << 8 | I), 0x00ff00ffu, 0x64806480u));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// What fp16 leaves of a pair, as an fp16 pair.
__device__ __forceinline__ uint32_t rest_f16x2(float lo, float hi, uint32_t packed) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&packed));
    return pack_f16x2(lo - f.x, hi - f.y);
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ float lds32(uint32_t a) {
    float r;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        :: "r"(dst), "l"(tmap), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}

// A sequence's tokens, -1 if its length is impossible.
__device__ __forceinline__ int attn_len(const KvAttnArgs& g, int b) {
    const int n = *(g.seq_len + b);
    return n < 0 || n > (g.max_pages << g.c.page_shift) ? -1 : n;
}
__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + kTile - 1) / kTile : 0; }

// Where a CTA is in the numbering; producer and consumers walk it alike.
struct TileWalk {
    int b, h, tile, nt, len;
    __device__ __forceinline__ void next(const KvAttnArgs& g) {
        if (++tile < nt) return;
        tile = 0;
        if (++h < g.c.n_heads) return;
        h = 0;
        do {
            len = attn_len(g, ++b);
            nt = tiles_of(len);
        } while (nt == 0);   // only called while tiles remain, so a later sequence has some
    }
};

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" :: "n"(32 * kConsumers) : "memory"); }
// An 8 x 8 matrix of 16-bit values, two of a row in each lane, transposed.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Four channels of a finished row.
template <typename T, int D>
__device__ __forceinline__ void attn_result(const KvAttnArgs& g, int b, int h, int row, int G, int d, float4 acc, float M, float L) {
    const int64_t at = ((int64_t)b * g.q_len + row / G) * g.n_q_heads + h * G + row % G;
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;   // NaN stays NaN
    T* o = static_cast<T*>(g.out) + at * D + d;
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(o) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    else
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (g.lse && d == 0) g.lse[at] = L == 0.0f ? -INFINITY : 0.6931471805599453f * (M + log2f(L));
}

template <typename T, int D, int NB, int MT>
__global__ void __launch_bounds__(kAttnThreads, 1)
kv_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const KvAttnArgs g) {
    using S = AttnSmem<T, D, NB, MT>;
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int KS = D / 16, IT = D / 16, DB = D / 8;   // k steps of S, channel tiles of O, codes a lane holds of a value row
    constexpr int TG = kConsumers / MT;                   // warps of a row tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * S::STAGES];
    __shared__ int abort_flag, drain_flag, stage_bad[S::STAGES];
    __shared__ int64_t scan[kAttnThreads / 32 + 1];
    __shared__ int start_b;
    __shared__ int64_t start_prefix;
    __shared__ float2 meet[2][kConsumers][8 * NB];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * S::STAGES;
    float* merge = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)) + S::STAGES * S::STAGE);
    if (tid == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(full + 8 * i, 65);   // the codes' expected bytes; a store and a copy of each lane of the scales' warp
            mbar_init(empty + 8 * i, kGroups * MT);
        }
        abort_flag = 0;
        drain_flag = 0;
        start_b = 0;
        start_prefix = 0;
        fence_barrier_init();
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    pdl_wait();
    pdl_trigger();

    // All tiles, and the sequence in which this CTA's share begins: every thread
    // sums a run of sequences, the run that holds the border is walked again.
    const int run = (g.n_seqs + kAttnThreads - 1) / kAttnThreads;
    const int s0 = min(g.n_seqs, tid * run), s1 = min(g.n_seqs, s0 + run);
    int64_t mine = 0;
    for (int b = s0; b < s1; ++b) mine += tiles_of(attn_len(g, b));
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    if (tid == 0) {
        int64_t sum = 0;
        for (int i = 0; i < kAttnThreads / 32; ++i) {
            const int64_t v = scan[i];
            scan[i] = sum;
            sum += v;
        }
        scan[kAttnThreads / 32] = sum;
    }
    __syncthreads();
    const int H = g.c.n_heads;
    const int64_t W = scan[kAttnThreads / 32] * H;
    const int64_t x0 = W * blockIdx.x / gridDim.x, x1 = W * (blockIdx.x + 1) / gridDim.x;
    {
        int64_t before = (scan[warp] + incl - mine) * H;
        if (x0 >= before && x0 < before + mine * H) {
            for (int b = s0; b < s1; ++b) {
                const int64_t n = (int64_t)tiles_of(attn_len(g, b)) * H;
                if (x0 < before + n) {
                    start_b = b;
                    start_prefix = before;
                    break;
                }
                before += n;
            }
        }
    }
    __syncthreads();
    TileWalk w{start_b, 0, 0, 0, 0};
    w.len = attn_len(g, w.b);
    w.nt = tiles_of(w.len);
    if (w.nt > 0) {
        w.h = (int)((x0 - start_prefix) / w.nt);
        w.tile = (int)((x0 - start_prefix) % w.nt);
    }
    if (tid == 0) {
        g.border[blockIdx.x] = x0;
        if (blockIdx.x + 1 == gridDim.x) g.border[gridDim.x] = W;
        g.start[blockIdx.x] = make_int4(w.b, w.h, x0 < W ? w.tile : 0, w.nt);
    }
    const int G = g.n_q_heads / H, R = G * g.q_len;
    // sequences without tiles: nothing seen, or a length that cannot be
    for (int b = blockIdx.x; b < g.n_seqs; b += gridDim.x) {
        const int len = attn_len(g, b);
        if (tiles_of(len) > 0) continue;
        const float v = len < 0 ? __int_as_float(0x7fc00000) : 0.0f;
        if (len < 0 && tid == 0) record_status(SQ_ERR_BOUNDS, SITE_KV_ATTENTION);
        T* o = static_cast<T*>(g.out) + (int64_t)b * g.q_len * g.n_q_heads * D;
        for (int i = tid; i < g.q_len * g.n_q_heads * D; i += kAttnThreads) put(o + i, v);
        if (g.lse)
            for (int i = tid; i < g.q_len * g.n_q_heads; i += kAttnThreads)
                g.lse[(int64_t)b * g.q_len * g.n_q_heads + i] = len < 0 ? v : -INFINITY;
    }

    const int n_items = (int)(x1 - x0);
    const long long limit = g.wait_limit;
    volatile int* abort = &abort_flag;
    if (warp >= kConsumers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kProducerRegs));
        if (warp > kConsumers + 1) return;
        // ------------------------------------------------------------ producers
        // The first warp sends the pages of codes by TMA, the second the scales, through
        // registers: a lane has four tokens, whose scales are one load of 16, 8 or 4
        // bytes (scale_block 1, 2, more), taken a tile ahead. (Scales sent by 4-byte
        // asynchronous copies, one a token, cost that warp 1550 cycles a tile, which was
        // the whole kernel's pace: 67 us for 128k tokens and 8 heads.)
        const bool sends_codes = warp == kConsumers;
        const int ps = g.c.page_size, sh = g.c.page_shift, bs = g.c.block_shift, per = kTile >> sh;   // pages of a tile
        int held_b = -1, held_from = 0, held = 0;   // 32 entries of a sequence's block table, one a lane
        int st = 0;
        uint32_t parity = 0;
        auto pages_of = [&](const TileWalk& v) {   // makes sure that a tile's entries are held; the place of the first
            const int from = v.tile * per;
            if (v.b != held_b || from < held_from || from + per > held_from + 32) {
                held_b = v.b;
                held_from = from;
                const int64_t e = (int64_t)from + lane;
                held = (e << sh) < v.len ? *(g.block_table + v.b * g.max_pages + e) : 0;
            }
            return from - held_from;
        };
        int issued = 0;
        if (sends_codes) {
            for (int i = 0; i < n_items; ++i) {
                const int at = pages_of(w);
                if (i >= S::STAGES) {
                    const bool go = mbar_wait(empty + 8 * st, parity ^ 1u, limit, abort, SITE_KV_ATTENTION_WAIT);
                    if (!__all_sync(0xffffffffu, go)) break;
                }
                const uint32_t dst = ring + st * S::STAGE;
                const uint32_t bar = full + 8 * st;
                const int page = __shfl_sync(0xffffffffu, held, (at + lane) & 31);
                const bool there = lane < per && (lane << sh) < w.len - w.tile * kTile;
                const bool good = there && (uint32_t)page < (uint64_t)g.c.n_pages;
                const unsigned bad = __ballot_sync(0xffffffffu, there && !good);
                const unsigned n_good = __popc(__ballot_sync(0xffffffffu, good));
                if (lane == 0) {
                    stage_bad[st] = bad != 0;
                    if (bad) record_status(SQ_ERR_BOUNDS, SITE_KV_ATTENTION);
                    mbar_arrive_expect_tx(bar, n_good * 2u * (uint32_t)(ps * D));
                }
                __syncwarp();
                if (good) {
                    const int z = page * H + w.h;
                    tma_load_3d(dst + lane * ps * D, &map_k, bar, 0, 0, z);
                    tma_load_3d(dst + S::CODES + lane * ps * D, &map_v, bar, 0, 0, z);
                }
                ++issued;
                if (i + 1 < n_items) w.next(g);
                if (++st == S::STAGES) {
                    st = 0;
                    parity ^= 1u;
                }
            }
        } else {
            float4 ks = make_float4(0.0f, 0.0f, 0.0f, 0.0f), vs = ks;
            auto take = [&](const TileWalk& v, float4& k, float4& x) {
                const int at = pages_of(v);
                const int t = 4 * lane;
                const int page = __shfl_sync(0xffffffffu, held, (at + (t >> sh)) & 31);
                if (t < v.len - v.tile * kTile && (uint32_t)page < (uint64_t)g.c.n_pages) {
                    const int64_t a = (((int64_t)page * H + v.h) << (sh - bs)) + ((t & (ps - 1)) >> bs);
                    if (bs == 0) {
                        k = *(reinterpret_cast<const float4*>(g.c.k_scale + a));
                        x = *(reinterpret_cast<const float4*>(g.c.v_scale + a));
                    } else if (bs == 1) {
                        const float2 p = *(reinterpret_cast<const float2*>(g.c.k_scale + a));
                        const float2 q = *(reinterpret_cast<const float2*>(g.c.v_scale + a));
                        k.x = p.x; k.y = p.y;
                        x.x = q.x; x.y = q.y;
                    } else {
                        k.x = *(g.c.k_scale + a);
                        x.x = *(g.c.v_scale + a);
                    }
                }
            };
            // one value of each token from what was loaded; not before it is needed, for
            // a use waits for the load
            auto spread = [&](const float4& k) {
                return bs == 0 ? k : bs == 1 ? make_float4(k.x, k.x, k.y, k.y) : make_float4(k.x, k.x, k.x, k.x);
            };
            if (n_items > 0) take(w, ks, vs);
            for (int i = 0; i < n_items; ++i) {
                TileWalk nx = w;
                float4 nk = ks, nv = vs;
                if (i + 1 < n_items) {
                    nx.next(g);
                    take(nx, nk, nv);
                }
                if (i >= S::STAGES) {
                    const bool go = mbar_wait(empty + 8 * st, parity ^ 1u, limit, abort, SITE_KV_ATTENTION_WAIT);
                    if (!__all_sync(0xffffffffu, go)) break;
                }
                const uint32_t bar = full + 8 * st;
                uint8_t* stage = smem_raw + (ring - smem_u32(smem_raw)) + st * S::STAGE;
                *reinterpret_cast<float4*>(stage + 2 * S::CODES + 16 * lane) = spread(ks);
                *reinterpret_cast<float4*>(stage + 2 * S::CODES + kTile * 4 + 16 * lane) = spread(vs);
                if (MT == 1 && (i == 0 || w.tile == 0)) {   // a piece begins: its query rows
                    constexpr int PER = D * (int)sizeof(T) / 16;
                    for (int u = lane; u < R * PER; u += 32) {
                        const int row = u / PER, c = u % PER;
                        const T* q = static_cast<const T*>(g.q) + ((int64_t)w.b * g.q_len + row / G) * g.q_stride +
                                     (int64_t)(w.h * G + row % G) * D;
                        cp_async16(smem_u32(stage) + S::Q + u * 16, reinterpret_cast<const uint8_t*>(q) + c * 16);
                    }
                }
                mbar_arrive(bar);       // the stores above
                cp_async_arrive(bar);   // the copies above, when they are there
                w = nx;
                ks = nk;
                vs = nv;
                if (++st == S::STAGES) {
                    st = 0;
                    parity ^= 1u;
                }
            }
        }
        if (*abort) {   // a wait ran out: the copies in flight end before the shared memory goes
            if (sends_codes) {
                volatile int* drain = &drain_flag;
                if (lane == 0)
                    for (int i = issued > S::STAGES ? issued - S::STAGES : 0; i < issued; ++i)
                        mbar_wait(full + 8 * (i % S::STAGES), (i / S::STAGES) & 1, limit, drain, SITE_KV_ATTENTION_WAIT);
            } else {
                asm volatile("cp.async.wait_all;" ::: "memory");
            }
            __syncwarp();
        }
        return;
    }

    // -------------------------------------------------------------------- consumers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kConsumerRegs));
    const int gr = lane >> 2, t4 = lane & 3;
    const int mt = warp % MT;
    int next_group = warp / MT;   // groups are dealt to the warps of a row tile in turn
    const int pi_g = gr & 1 ? (gr + 4) & 7 : gr;          // the token of row gr of an 8-row block: 0 5 2 7 4 1 6 3
    const int tok_a = 2 * t4, tok_b = (2 * t4 + 5) & 7;   // and of rows 2 t4, 2 t4 + 1
    uint32_t k_off[D / 64], v_off[2];
    if (D == 128) {
        k_off[0] = pi_g * 128 + ((t4 ^ pi_g) << 4);
        k_off[D / 64 - 1] = pi_g * 128 + (((4 + t4) ^ pi_g) << 4);
        v_off[0] = tok_a * 128 + ((gr ^ tok_a) << 4);
        v_off[1] = tok_b * 128 + ((gr ^ tok_b) << 4);
    } else {
        k_off[0] = pi_g * 64 + ((t4 ^ (pi_g >> 1)) << 4);
        v_off[0] = tok_a * 64 + ((((gr >> 1) ^ (tok_a >> 1)) << 4) | ((gr & 1) << 3));
        v_off[1] = tok_b * 64 + ((((gr >> 1) ^ (tok_b >> 1)) << 4) | ((gr & 1) << 3));
    }
    // Of each side of 8 rows: the queries as an operand (row gr); reference, sum, factor and
    // tokens seen of rows 2 t4 and 2 t4 + 1, whose scores a lane holds.
    uint32_t qh[NB][KS][2], ql[F32 ? NB : 1][F32 ? KS : 1][2];
    float o[IT][NB][4], m[NB][2], l[NB][2], qs[NB][2];
    int see[NB][2];
    int see_all = 0;  // tokens that every row sees
    bool spoilt = false, began_before = false;
    int st = 0, piece = 0;
    uint32_t parity = 0;
    for (int i = 0; i < n_items; ++i) {
        const uint32_t base = ring + st * S::STAGE;
        const bool begins = i == 0 || w.tile == 0;
        if (begins || next_group < kGroups) {
            mbar_wait(full + 8 * st, parity, limit, abort, SITE_KV_ATTENTION_WAIT);
            if (stage_bad[st]) spoilt = true;
        }
        if (begins) {   // a new piece: its queries
            spoilt = stage_bad[st] != 0;
            began_before = w.tile > 0;
            see_all = w.len - g.q_len + 1;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
#pragma unroll
                for (int k = 0; k < IT; ++k) o[k][n][0] = o[k][n][1] = o[k][n][2] = o[k][n][3] = 0.0f;
                const int row = (mt * NB + n) * 8 + gr;
                const bool has = row < R;
                const T* q;
                if (MT == 1)
                    q = reinterpret_cast<const T*>(smem_raw + (base - smem_u32(smem_raw)) + S::Q) + (has ? row : 0) * D;
                else
                    q = static_cast<const T*>(g.q) + ((int64_t)w.b * g.q_len + (has ? row / G : 0)) * g.q_stride +
                        (int64_t)(w.h * G + (has ? row % G : 0)) * D;
                float x[KS][4];
                float top = 0.0f;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float v[8];
                        Chunk<T>::load(q + 64 * c + 16 * t4 + 8 * half, v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x[4 * c + 2 * half + (e >> 2)][e & 3] = v[e];
                            top = fmaxf(top, fabsf(v[e]));
                        }
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // a power of two that brings the row's largest value to 1 .. 4 (a subnormal one below 1)
                const int ex = min(126, max(-126, (int)(__float_as_uint(top) >> 23) - 127));
                const float down = __int_as_float((127 - ex) << 23);
                const float up = g.scale * 1.4426950408889634f * __int_as_float((127 + ex) << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[ks][e] *= down;
                    // codes 0 and 2 of a word make the first pair of a k step, 1 and 3 the second
                    qh[n][ks][0] = pack_f16x2(x[ks][0], x[ks][2]);
                    qh[n][ks][1] = pack_f16x2(x[ks][1], x[ks][3]);
                    if (F32) {
                        ql[F32 ? n : 0][F32 ? ks : 0][0] = rest_f16x2(x[ks][0], x[ks][2], qh[n][ks][0]);
                        ql[F32 ? n : 0][F32 ? ks : 0][1] = rest_f16x2(x[ks][1], x[ks][3], qh[n][ks][1]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = (mt * NB + n) * 8 + 2 * t4 + e;
                    m[n][e] = kNoReference;
                    l[n][e] = 0.0f;
                    qs[n][e] = __shfl_sync(0xffffffffu, up, 4 * (2 * t4 + e));
                    see[n][e] = r < R ? max(0, see_all + r / G) : 0;
                }
            }
            // With one row tile half of the warps have no group in this tile and so no say in
            // when its stage is free, but they have read the queries and the flag there:
            // nobody frees it before all have. (With more, every warp has a group.)
            if (MT == 1) consumers_sync();
        }
#pragma unroll 1
        for (; next_group < kGroups; next_group += TG) {
            const int t0 = next_group * kGroup;            // first of the 32 tokens, in the tile
            const int p0 = w.tile * kTile + t0;            // and in the sequence
            if (p0 >= w.len) {
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + 8 * st);
                continue;
            }
            // j: blocks of 8 tokens; j / 2: the 16 tokens of a product
            float s[2][NB][4];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[0][n][e] = s[1][n][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint4 kw[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) kw[j] = lds128(base + (t0 + 8 * j) * D + k_off[c]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t a[4];
                        codes_even_odd(e == 0 ? kw[2 * h].x : e == 1 ? kw[2 * h].y : e == 2 ? kw[2 * h].z : kw[2 * h].w, a[0], a[2]);
                        codes_even_odd(e == 0 ? kw[2 * h + 1].x : e == 1 ? kw[2 * h + 1].y : e == 2 ? kw[2 * h + 1].z : kw[2 * h + 1].w,
                                       a[1], a[3]);
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            mma_f16(s[h][n], a, qh[n][4 * c + e][0], qh[n][4 * c + e][1]);
                            if (F32) mma_f16(s[h][n], a, ql[F32 ? n : 0][F32 ? 4 * c + e : 0][0], ql[F32 ? n : 0][F32 ? 4 * c + e : 0][1]);
                        }
                    }
            }
            float vs[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {   // scores in units of log2, by their keys' scales; the value scales
                const uint32_t a = base + 2 * S::CODES + (t0 + 8 * j + pi_g) * 4;
                const float ks = lds32(a);
                vs[j] = lds32(a + kTile * 4);
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) s[j >> 1][n][2 * (j & 1) + e] *= qs[n][e] * ks;
            }
            uint32_t va[2][4][DB / 4];   // values' codes: of tokens a, b, 8 + a, 8 + b of both k steps
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a = base + S::CODES + (t0 + 16 * half + 8 * (k >> 1)) * D + v_off[k & 1];
                    if constexpr (D == 128) {
                        const uint4 x = lds128(a);
                        va[half][k][0] = x.x; va[half][k][1] = x.y; va[half][k][2] = x.z; va[half][k][3] = x.w;
                    } else {
                        const uint2 x = lds64(a);
                        va[half][k][0] = x.x; va[half][k][1] = x.y;
                    }
                }
            }
            // All of the group is in registers: its part of the stage is free
            // before the weights and the second product.
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * st);
            if (p0 + kGroup > see_all) {   // the end of what some row sees
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int p = p0 + 8 * j + pi_g;
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (p >= see[n][e]) s[j >> 1][n][2 * (j & 1) + e] = -INFINITY;
                    if (p >= w.len) vs[j] = 0.0f;   // its scales were not loaded
                }
            }
            float wt[2][NB][4], sum[NB][2];
            auto weigh = [&](float& most) {
                most = 0.0f;
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    sum[n][0] = sum[n][1] = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float a = exp2_fast(s[j >> 1][n][2 * (j & 1) + e] - m[n][e]);
                            sum[n][e] += a;
                            wt[j >> 1][n][2 * (j & 1) + e] = a * vs[j];
                            most = fmaxf(most, a * fmaxf(fabsf(vs[j]), kLeastScale));
                        }
                }
            };
            float most;
            weigh(most);
            if (__any_sync(0xffffffffu, most > kMaxWeight)) {
                float ex[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    ex[j] = fmaxf((float)((int)((__float_as_uint(vs[j]) >> 23) & 255u) - 127 - kHeadroom), kNoScale - kHeadroom);
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = m[n][e];
#pragma unroll
                        for (int j = 0; j < 4; ++j) x = fmaxf(x, s[j >> 1][n][2 * (j & 1) + e] + ex[j]);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        const float f = exp2_fast(m[n][e] - x);
                        m[n][e] = x;
                        l[n][e] *= f;
#pragma unroll
                        for (int k = 0; k < IT; ++k) {
                            o[k][n][e] *= f;
                            o[k][n][2 + e] *= f;
                        }
                    }
                weigh(most);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                l[n][0] += sum[n][0];
                l[n][1] += sum[n][1];
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {   // 16 tokens a k step
                uint32_t ph[NB][2], pl[F32 ? NB : 1][2];
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float x = wt[half][n][2 * k], y = wt[half][n][2 * k + 1];
                        const uint32_t hi = pack_f16x2(x, y);
                        ph[n][k] = transpose_8x8(hi);
                        if (F32) pl[F32 ? n : 0][k] = transpose_8x8(rest_f16x2(x, y, hi));
                    }
#pragma unroll
                for (int c = 0; c < DB / 4; ++c) {
#define SQ_PV(I)                                                                                                 \
    {                                                                                                            \
        const uint32_t a[4] = {code_pair<2 * I>(va[half][0][c], va[half][1][c]),                                 \
                               code_pair<2 * I + 1>(va[half][0][c], va[half][1][c]),                             \
                               code_pair<2 * I>(va[half][2][c], va[half][3][c]),                                 \
                               code_pair<2 * I + 1>(va[half][2][c], va[half][3][c])};                            \
        _Pragma("unroll") for (int n = 0; n < NB; ++n) {                                                         \
            mma_f16(o[2 * c + I][n], a, ph[n][0], ph[n][1]);                                                     \
            if (F32) mma_f16(o[2 * c + I][n], a, pl[F32 ? n : 0][0], pl[F32 ? n : 0][1]);                        \
        }                                                                                                        \
    }
                    SQ_PV(0) SQ_PV(1)
#undef SQ_PV
                }
            }
        }
        next_group -= kGroups;

        const bool ends = w.tile + 1 == w.nt;
        if (ends || i + 1 == n_items) {   // the end of the piece: the warps' results meet
            float2 (*all)[8 * NB] = meet[piece & 1];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[n][e];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    if (spoilt) x = __int_as_float(0x7fc00000);
                    if (gr == 0) all[warp][n * 8 + 2 * t4 + e] = make_float2(m[n][e], x);
                }
            consumers_sync();
            const bool whole = ends && !began_before;
            const int64_t slot = (2 * (int64_t)blockIdx.x + (began_before ? 0 : 1)) * (8 * NB * MT);
#pragma unroll
            for (int n = 0; n < NB; ++n) {   // 8 rows of each row tile at a time
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int rr = 2 * t4 + e;
                    if ((mt * NB + n) * 8 + rr >= R) continue;
                    float M = kNoReference;
#pragma unroll
                    for (int q = 0; q < TG; ++q) M = fmaxf(M, all[q * MT + mt][n * 8 + rr].x);
                    const float f = exp2_fast(m[n][e] - M);
                    float* dst = merge + (warp * 8 + rr) * S::ROW + (DB + 4) * gr;   // channels DB gr .. + DB - 1
#pragma unroll
                    for (int k = 0; k < IT; k += 2)
                        *reinterpret_cast<float4*>(dst + 2 * k) = make_float4(o[k][n][e] * f, o[k][n][2 + e] * f,
                                                                              o[k + 1][n][e] * f, o[k + 1][n][2 + e] * f);
                }
                consumers_sync();
                for (int u = tid; u < MT * 8 * (D / 4); u += 32 * kConsumers) {
                    const int d = u % (D / 4) * 4, rr = u / (D / 4) % 8, rm = u / (2 * D);
                    const int row = (rm * NB + n) * 8 + rr;
                    if (row >= R) continue;
                    float M = kNoReference, L = 0.0f;
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int q = 0; q < TG; ++q) M = fmaxf(M, all[q * MT + rm][n * 8 + rr].x);
#pragma unroll
                    for (int q = 0; q < TG; ++q) {
                        const float2 ml = all[q * MT + rm][n * 8 + rr];
                        L += ml.y * exp2_fast(ml.x - M);
                        const float4 x = *reinterpret_cast<const float4*>(merge + ((q * MT + rm) * 8 + rr) * S::ROW + d + 4 * (d / DB));
                        acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
                    }
                    if (whole) {
                        attn_result<T, D>(g, w.b, w.h, row, G, d, acc, M, L);
                    } else {
                        if (d == 0) g.part_ml[slot + row] = make_float2(M, L);
                        *reinterpret_cast<float4*>(g.part_o + (slot + row) * D + d) = acc;
                    }
                }
                if (n + 1 < NB) consumers_sync();
            }
            ++piece;
        }
        if (i + 1 < n_items) w.next(g);
        if (++st == S::STAGES) {
            st = 0;
            parity ^= 1u;
        }
    }
}

// Joins the partial results of the (sequence, head)s that several CTAs shared.
// Block i - 1 looks at the border between the shares of CTAs i - 1 and i: if it
// lies inside a (sequence, head) and is the first that does, this block's warps join
// that one's rows. A lane holds the reference and sum of one piece (32 at a time); the
// accumulators are added in the CTAs' order.
template <typename T, int D>
__global__ void __launch_bounds__(128) kv_attention_join_kernel(const KvAttnArgs g, int n_ctas, int slot_rows) {
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x + 1, lane = threadIdx.x & 31;
    const int64_t x = *(g.border + i), x_before = *(g.border + i - 1);
    const int4 at = g.start[i];
    const int64_t begin = x - at.z, end = begin + at.w;
    if (at.z == 0 || x_before > begin) return;
    const int G = g.n_q_heads / g.c.n_heads;
    const int row = blockIdx.y * 4 + (threadIdx.x >> 5);
    if (row >= G * g.q_len) return;
    constexpr int E = D / 32;
    float M = kNoReference, L = 0.0f;
    float acc[E] = {};
    for (int p0 = 0;; p0 += 32) {   // pieces: CTA i - 1 (its slot 1), then i, i + 1, .. (slot 0) that begin inside
        const int c = i - 1 + p0 + lane;
        const bool in = c < n_ctas && *(g.border + min(c, n_ctas)) < end;
        const unsigned inside = __ballot_sync(0xffffffffu, in);
        if (inside == 0) break;
        const bool some = in && *(g.border + c) < *(g.border + c + 1);   // a share may be empty
        const int64_t slot = (2 * (int64_t)c + (c == i - 1 ? 1 : 0)) * slot_rows + row;
        const float2 ml = some ? g.part_ml[slot] : make_float2(kNoReference, 0.0f);
        float m = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = fmaxf(m, M);
        const float old = exp2_fast(M - m), f = exp2_fast(ml.x - m);
        float l = ml.y * f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        M = m;
        L = L * old + l;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= old;
        const unsigned have = __ballot_sync(0xffffffffu, some);
        const int n = 32 - __clz(inside);
#pragma unroll 8
        for (int p = 0; p < n; ++p) {   // no branch, so that several pieces' loads are in flight
            const float fp = __shfl_sync(0xffffffffu, f, p);
            const bool is = (have >> p) & 1u;   // an empty share's slot holds anything
            const int cp = i - 1 + p0 + p;
            const float* o = g.part_o + ((2 * (int64_t)cp + (cp == i - 1 ? 1 : 0)) * slot_rows + row) * D + lane * E;
            float v[E];
            if constexpr (E == 4) {
                const float4 x = *reinterpret_cast<const float4*>(o);
                v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2*>(o);
                v[0] = x.x; v[1] = x.y;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += is ? v[e] * fp : 0.0f;
        }
        if (inside != 0xffffffffu) break;
    }
    const int qi = row / G, h = at.y * G + row % G;
    const int64_t out_row = ((int64_t)at.x * g.q_len + qi) * g.n_q_heads + h;
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int e = 0; e < E; ++e) put(static_cast<T*>(g.out) + out_row * D + lane * E + e, acc[e] * inv);
    if (g.lse && lane == 0) g.lse[out_row] = L == 0.0f ? -INFINITY : 0.6931471805599453f * (M + log2f(L));
}

// Codes [pages * heads][page_size][D] as a map whose box is one page of one head, in the
// swizzle whose rows are D bytes.
sq_status make_map_pages(CUtensorMap* map, const void* base, int64_t slabs, int ps, int D) {
    sq_status r = get_encoder();
    if (r != SQ_OK) return r;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)ps, (cuuint64_t)slabs};
    cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * ps};
    cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)ps, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult cr = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (cr != CUDA_SUCCESS) {
        set_error("cuTensorMapEncodeTiled failed (%d) for %lld pages", (int)cr, (long long)slabs);
        return SQ_ERR_CUDA;
    }
    return SQ_OK;
}

// Rows that the kernel's row tiles hold: 8, or 16 times a power of two.
int padded_rows(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

struct KvAttnLayout {
    size_t start, ml, o, total;
};
KvAttnLayout kv_attn_layout(int ctas, int64_t rows, int D) {
    const size_t slots = (size_t)ctas * 2 * padded_rows(rows);
    KvAttnLayout L{};
    L.start = align256((size_t)(ctas + 1) * sizeof(int64_t));
    L.ml = L.start + align256((size_t)ctas * sizeof(int4));
    L.o = L.ml + align256(slots * sizeof(float2));
    L.total = L.o + slots * D * sizeof(float);
    return L;
}

template <typename T, int D, int NB, int MT>
sq_status launch_kv_attention(const CUtensorMap& mk, const CUtensorMap& mv, const KvAttnArgs& g, cudaStream_t st) {
    static bool attr_done[64] = {};
    const DeviceInfo& di = device_info();
    constexpr size_t smem = AttnSmem<T, D, NB, MT>::TOTAL;
    sq_status r = ensure_smem_attr(kv_attention_kernel<T, D, NB, MT>, smem, attr_done[di.device & 63]);
    if (r != SQ_OK) return r;
    r = launch_pdl("kv_attention_kernel", kv_attention_kernel<T, D, NB, MT>, dim3(di.sm_count), dim3(kAttnThreads), smem, st, 1,
                   mk, mv, g);
    if (r != SQ_OK) return r;
    const int rows = g.n_q_heads / g.c.n_heads * g.q_len;
    return launch_pdl("kv_attention_join_kernel", kv_attention_join_kernel<T, D>, dim3(di.sm_count - 1, (rows + 3) / 4),
                      dim3(128), 0, st, 1, g, di.sm_count, 8 * NB * MT);
}

template <typename T, int D>
sq_status launch_kv_attention_rows(const CUtensorMap& mk, const CUtensorMap& mv, const KvAttnArgs& g, cudaStream_t st) {
    switch (padded_rows((int64_t)g.n_q_heads / g.c.n_heads * g.q_len)) {
    case 8: return launch_kv_attention<T, D, 1, 1>(mk, mv, g, st);
    case 16: return launch_kv_attention<T, D, 2, 1>(mk, mv, g, st);
    case 32: return launch_kv_attention<T, D, 2, 2>(mk, mv, g, st);
    case 64: return launch_kv_attention<T, D, 2, 4>(mk, mv, g, st);
    default: return launch_kv_attention<T, D, 2, 8>(mk, mv, g, st);
    }
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
    if (!(scale >= -1.0e38f && scale <= 1.0e38f)) { set_error("scale must be within +-1e38"); return SQ_ERR_INVALID_ARG; }
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
    const int64_t rows = q_len * (n_q_heads / cache->n_heads);
    const KvAttnLayout L = kv_attn_layout(device_info().sm_count, rows, D);
    if (!ws || ws_bytes < L.total) {
        set_error("workspace too small: %zu bytes given, %zu needed", ws_bytes, L.total);
        return SQ_ERR_INVALID_ARG;
    }
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) { set_error("workspace must be 256-byte aligned"); return SQ_ERR_UNSUPPORTED; }
    g.block_table = block_table; g.seq_len = seq_len; g.max_pages = max_pages; g.q_stride = q_stride;
    g.n_seqs = (int)n_seqs; g.q_len = (int)q_len; g.n_q_heads = (int)n_q_heads; g.scale = scale;
    g.q = q; g.out = out; g.lse = lse;
    uint8_t* base = static_cast<uint8_t*>(ws);
    g.wait_limit = wait_limit_cycles();
    g.border = reinterpret_cast<int64_t*>(base);
    g.start = reinterpret_cast<int4*>(base + L.start);
    g.part_ml = reinterpret_cast<float2*>(base + L.ml);
    g.part_o = reinterpret_cast<float*>(base + L.o);
    // an empty cache has no page to map; any address serves, since no page number is valid
    const int64_t slabs = cache->n_pages > 0 ? cache->n_pages * cache->n_heads : 1;
    if (slabs > 2147483647LL) { set_error("cache too large"); return SQ_ERR_UNSUPPORTED; }
    CUtensorMap mk, mv;
    if ((r = make_map_pages(&mk, cache->n_pages > 0 ? cache->k : out, slabs, cache->page_size, D)) != SQ_OK) return r;
    if ((r = make_map_pages(&mv, cache->n_pages > 0 ? cache->v : out, slabs, cache->page_size, D)) != SQ_OK) return r;
    if (dt == SQ_F32)
        return D == 64 ? launch_kv_attention_rows<float, 64>(mk, mv, g, st) : launch_kv_attention_rows<float, 128>(mk, mv, g, st);
    return D == 64 ? launch_kv_attention_rows<__nv_bfloat16, 64>(mk, mv, g, st)
                   : launch_kv_attention_rows<__nv_bfloat16, 128>(mk, mv, g, st);
}

}  // namespace
}  // namespace sq

extern "C" {

size_t sq_kv_attention_workspace_size(const sq_kv_cache* cache, int64_t n_seqs, int64_t q_len, int64_t n_q_heads) {
    if (!cache || n_seqs <= 0 || q_len <= 0 || n_q_heads <= 0 || cache->n_heads <= 0 || cache->head_dim <= 0) return 0;
    const int64_t rows = q_len * (n_q_heads / cache->n_heads);
    if (q_len > 128 || rows > 128) return 0;
    return sq::kv_attn_layout(sq::device_info().sm_count, rows, cache->head_dim).total;
}

sq_status sq_kv_attention(const void* q, int64_t q_stride, sq_dtype dt, const sq_kv_cache* cache,
                          const int32_t* block_table, int64_t max_pages, const int32_t* seq_len, int64_t n_seqs,
                          int64_t q_len, int64_t n_q_heads, float scale, void* out, float* lse, void* workspace,
                          size_t ws_bytes, sq_stream_t stream) {
    return sq::kv_attention_impl(q, q_stride, dt, cache, block_table, max_pages, seq_len, n_seqs, q_len, n_q_heads,
                                 scale, out, lse, workspace, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
