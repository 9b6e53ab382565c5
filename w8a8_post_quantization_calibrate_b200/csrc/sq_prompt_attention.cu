// sq_prompt_attention.cu -- attention of packed prompts over themselves
// (sq_prompt_attention). Included into the library's single translation unit
// after sq_kv_attention.cu, some of whose helpers it uses.
#include <cuda.h>
#include <cuda_runtime.h>

#include "sq_device.cuh"
#include "sq_internal.h"

namespace sq {
namespace {

struct PromptArgs {
    __nv_bfloat16* out;
    float* lse;
    const int32_t* cu;
    int64_t T, blocks;              // blocks of 256 rows, empty ones among them
    int n_seqs, n_q_heads, group;   // query heads of one key head
    float scale;                    // in units of log2
    bool causal;
    long long wait_limit;
};

// The kernel. A work item is 256 query rows (two tiles of 128) of one sequence and head; the
// CTAs, one on each SM, take the items in turn, each sequence's longest first. With S = Q K^T and
// O += P V as tcgen05 products of 128 x 128 x D and 128 x D x 128 and about as much time
// for the 128 x 128 exponentials of a tile as for its two products, the two query
// tiles alternate: while one's softmax runs, the other's products do.
//   Measured: two prompts of 5,000 and 3,340 tokens, 64 heads over 8, causal (593 GFLOP) in 622 to 647 us,
// 0.92 to 0.95 PFLOP/s; 494 without the softmax. A tile's softmax takes some 1,700 cycles,
// the other tile's two products 1,024, so the tensor cores wait for about half of the time.
//   Tensor memory: the two tiles' scores (128 columns each, the weights in bf16 over them:
// P is read as an operand from there) and accumulators (D columns each).
//   Softmax: a thread has a row. The reference m is moved only when a score is 2^8
// above it (any row of the warp), so the accumulator is rarely rescaled: P is at most 2^8,
// and sums and accumulators in fp32 do not care. P is rounded to bf16 (relative
// 2^-8 at most) because the product takes two bf16 operands.
//   Warp 0 loads (TMA: Q, and K and V tiles of 128 tokens), warp 1 issues the products.
// Warps 4-7 and 8-11: softmax and results of the two tiles.
constexpr int kPThreads = 384;
constexpr int kPSlots = 4;              // tiles in flight: K, V, K, V; key tile number c is in slots 2 (c & 1) and 2 (c & 1) + 1
// registers a thread: 168 at launch times 12 warps are as many as 224 times 8 and 56 times 4
constexpr int kPSoftRegs = 224, kPOtherRegs = 56;
constexpr float kPSlack = 8.0f;

template <int D>
struct PromptSmem {
    static constexpr int BOX = 128 * 128;              // 128 rows of 64 channels
    static constexpr int TILE = BOX * (D / 64);
    static constexpr int RING = 2 * TILE;              // behind the two query tiles
    static constexpr int TOTAL = 1024 + 2 * TILE + kPSlots * TILE;
};

// The products' operands by the low words of their shared-memory descriptors (address and
// leading offset; the high word is the same for every tile here: 8-row groups 1024 bytes
// apart, version 1, 128-byte swizzle). A product takes 64 cycles on the tensor cores, and
// the issuing warp has to keep that pace: with a slot's address worked out for every
// product it took 80 to 120, and two long prompts 735 us. So a step over a key tile is
// compiled twice, for the two places a tile can have, its loop bounds are made uniform to the
// compiler, and its operands are constants in uniform registers: 628 us.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
// Tiles whose rows run along the contraction (leading offset unused, 1), and tiles
// whose rows ARE the contraction (the next 64 columns a box further).
__device__ __forceinline__ uint32_t desc_low(uint32_t smem_addr, uint32_t leading) { return ((smem_addr & 0x3FFFFu) >> 4) | (leading << 16); }
// All lanes call these with the same operands and `lead` says which one issues: no branch
// around them, so that the operands stay in uniform registers.
template <int ACCUMULATE>
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
                 "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
                 "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_low), "r"(b_low), "r"(idesc), "n"(kDescHigh), "n"(ACCUMULATE), "r"(lead) : "memory");
}
template <int ACCUMULATE>
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
                 "mov.b64 db, {%2, %4};\n\t"
                 "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_tmem), "r"(b_low), "r"(idesc), "n"(kDescHigh), "n"(ACCUMULATE), "r"(lead) : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint32_t bar) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                 :: "r"(bar), "r"(lead) : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
        " {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
           "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
           "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// A wait of a whole warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, long long limit, volatile int* abort, unsigned int site) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit, abort, site));
}

template <uint32_t V>
struct Const {
    static constexpr uint32_t v = V;
};

// Work items in order: every role walks them alike, a warp at a time. Sequence b's blocks of 256
// rows have the numbers U_b = cu[b] / 256 + b, U_b + 1, .., below U_{b+1}: at least
// as many as it needs, without a scan over the batch; the rest are empty.
struct PromptWalk {
    int64_t u = 0, next = 0;   // U_b and U_{b+1} of the sequence at hand
    int start = 0, len = 0;
    int h, row;                // head; first query row, in the sequence
    int n0, n1;                // key tiles of the two query tiles, n0 <= n1 unless n1 is 0; n0 = 0: an empty item
    __device__ __forceinline__ bool find(const PromptArgs& g, int64_t id) {
        const int64_t f = id / g.n_q_heads;
        if (f >= g.blocks) return false;
        h = (int)(id % g.n_q_heads);
        if (f < u || f >= next) {
            auto at = [&](int i) { return (int64_t)(*(g.cu + i) >> 8) + i; };
            const int b = warp_find(at, g.n_seqs, f);
            const int64_t a = *(g.cu + b), e = *(g.cu + b + 1);
            u = at(b);
            next = at(b + 1);
            start = (int)min(max(a, (int64_t)0), g.T);
            len = (int)(min(max(e, (int64_t)start), g.T) - start);
        }
        const int nb = (len + 255) / 256;
        n0 = n1 = 0;
        if (f < u || f - u >= nb) return true;
        row = (nb - 1 - (int)(f - u)) * 256;
        n0 = (min(len, g.causal ? row + 128 : len) + 127) / 128;
        n1 = row + 128 >= len ? 0 : (min(len, g.causal ? row + 256 : len) + 127) / 128;
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(kPThreads, 1)
prompt_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const PromptArgs g) {
    using S = PromptSmem<D>;
    constexpr int NBOX = D / 64;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 + 2 * kPSlots + 6 + 1];
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_flag, drain_flag;
    __shared__ uint32_t sent[kPSlots];   // loads into each slot
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform to the compiler
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t q_full = smem_u32(bars), q_empty = q_full + 8, full = q_full + 16, empty = full + 8 * kPSlots;
    const uint32_t s_full = empty + 8 * kPSlots, p_full = s_full + 16, o_full = p_full + 16, drained = o_full + 16;
    if (tid == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < kPSlots; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
            sent[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);
            mbar_init(o_full + 8 * i, 1);
        }
        mbar_init(drained, 1);
        abort_flag = 0;
        drain_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    if (warp == 1) tmem_alloc<512>(smem_u32(&tmem_base_s));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base_s, 0);
    const uint32_t t_s = tmem, t_o = tmem + 256;   // scores at 0, 128; accumulators at 256, 256 + D
    const long long limit = g.wait_limit;
    volatile int* abort = &abort_flag;
    pdl_wait();
    pdl_trigger();
    PromptWalk w;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kPOtherRegs));
        if (warp == 0) {
            // ------------------------------------------------------------ loads
            int work = 0;
            uint32_t count = 0;   // key tiles sent
            bool ok = true;
            if (blockIdx.x == 0)   // once: offsets that the walk cuts
                for (int b = lane; b <= g.n_seqs; b += 32) {
                    const int64_t a = *(g.cu + b);
                    if (a < 0 || a > g.T || (b > 0 && a < *(g.cu + b - 1))) record_status(SQ_ERR_BOUNDS, SITE_PROMPT);
                }
            auto send = [&](const CUtensorMap* map, int slot, int h, int tok) {
                const uint32_t turn = count >> 1;
                if (turn > 0 && !mbar_wait(empty + 8 * slot, (turn - 1) & 1, limit, abort, SITE_PROMPT_WAIT)) return false;
                mbar_arrive_expect_tx(full + 8 * slot, S::TILE);
#pragma unroll
                for (int c = 0; c < NBOX; ++c)
                    tma_load_3d(base + S::RING + slot * S::TILE + c * S::BOX, map, full + 8 * slot, 64 * c, h, tok);
                sent[slot] = turn + 1;
                return true;
            };
            for (int64_t id = blockIdx.x; w.find(g, id); id += gridDim.x) {
                if (w.n0 == 0) continue;
                if (lane == 0) {
                    ok = work == 0 || mbar_wait(q_empty, (work - 1) & 1, limit, abort, SITE_PROMPT_WAIT);
                    if (ok) {
                        const int tiles = w.n1 > 0 ? 2 : 1;
                        mbar_arrive_expect_tx(q_full, tiles * S::TILE);
                        for (int i = 0; i < tiles; ++i)
#pragma unroll
                            for (int c = 0; c < NBOX; ++c)
                                tma_load_3d(base + i * S::TILE + c * S::BOX, &map_q, q_full, 64 * c, w.h, w.start + w.row + 128 * i);
                        ++work;
                        const int n = max(w.n0, w.n1), hk = w.h / g.group;
                        for (int j = 0; ok && j < n; ++j, ++count)
                            ok = send(&map_k, 2 * (count & 1), hk, w.start + 128 * j) && send(&map_v, 2 * (count & 1) + 1, hk, w.start + 128 * j);
                    }
                }
                if (!__shfl_sync(0xffffffffu, (int)ok, 0)) break;
            }
            if (lane == 0 && *abort) {   // a wait ran out: the copies in flight end before the shared memory goes
                volatile int* drain = &drain_flag;
                for (int i = 0; i < kPSlots; ++i)
                    if (sent[i] > 0) mbar_wait(full + 8 * i, (sent[i] - 1) & 1, limit, drain, SITE_PROMPT_WAIT);
                if (work > 0) mbar_wait(q_full, (work - 1) & 1, limit, drain, SITE_PROMPT_WAIT);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ products
            constexpr uint32_t IS = make_idesc_bf16(128, 128);
            constexpr uint32_t IO = make_idesc_bf16(128, D) | (1u << 16);   // V's rows are the contraction
            // All 512 columns are this CTA's, so its tensor memory begins at address 0.
            constexpr uint32_t TS = 0, TO = 256;
            int work = 0;
            uint32_t count = 0, p_turn0 = 0, p_turn1 = 0;   // key tiles begun; weights taken
            const uint32_t lead = lane == 0;
            const uint32_t q_low = desc_low(base, 1), k_low = desc_low(base + S::RING, 1), v_low = desc_low(base + S::RING, S::BOX >> 4);
            constexpr uint32_t STEP = S::TILE >> 4;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return warp_wait(bar, parity, limit, abort, SITE_PROMPT_WAIT);
            };
            // S_i = Q_i K^T from K slot 2 P
            auto scores = [&](auto I_, auto P_) {
                constexpr uint32_t I = decltype(I_)::v, P = decltype(P_)::v;
                const uint32_t a = q_low + I * STEP, b = k_low + 2 * P * STEP;
                mma_ss<0>(lead, TS + 128 * I, a, b, IS);
#pragma unroll
                for (int k = 1; k < D / 16; ++k)
                    mma_ss<1>(lead, TS + 128 * I, a + (((k >> 2) * S::BOX + (k & 3) * 32) >> 4), b + (((k >> 2) * S::BOX + (k & 3) * 32) >> 4), IS);
                commit_if(lead, s_full + 8 * I);
            };
            // O_i += P_i V from V slot 2 P + 1, once the weights are there; on a new item that also
            // says that the same warps have read the last one's accumulator.
            auto outputs = [&](auto I_, auto P_, uint32_t& p_turn, bool first, bool last) {
                constexpr uint32_t I = decltype(I_)::v, P = decltype(P_)::v;
                if (!wait(p_full + 8 * I, p_turn & 1)) return false;
                ++p_turn;
                tc_fence_after();
                const uint32_t b = v_low + (2 * P + 1) * STEP;
                if (first) mma_ts<0>(lead, TO + D * I, TS + 128 * I, b, IO);
                else mma_ts<1>(lead, TO + D * I, TS + 128 * I, b, IO);
#pragma unroll
                for (int k = 1; k < 8; ++k) mma_ts<1>(lead, TO + D * I, TS + 128 * I + 8 * k, b + k * (2048 >> 4), IO);
                if (last) commit_if(lead, o_full + 8 * I);
                return true;
            };
            constexpr Const<0> c0{};
            constexpr Const<1> c1{};
            int n0 = 0, n1 = 0, len = 0;   // of the item, uniform to the compiler
            // Key tile j, in the slots of P; the next one's are those of N.
            auto step = [&](auto P_, auto N_, int j, int n) {
                constexpr uint32_t P = decltype(P_)::v, N = decltype(N_)::v;
                if (!wait(full + 8 * (2 * P + 1), (count >> 1) & 1)) return false;
                const int rows = len - 128 * j;
                if (rows < 128) {   // rows behind the sequence: a weight of 0 times what lies there must be 0
                    uint8_t* v = base_ptr + S::RING + (2 * P + 1) * S::TILE;
                    for (int u = rows * 8 + lane; u < 128 * 8; u += 32)
#pragma unroll
                        for (int c = 0; c < NBOX; ++c) *reinterpret_cast<uint4*>(v + c * S::BOX + u * 16) = make_uint4(0, 0, 0, 0);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (j < n0 && !outputs(c0, P_, p_turn0, j == 0, j + 1 == n0)) return false;
                if (j + 1 < n) {
                    if (!wait(full + 8 * 2 * N, ((count + 1) >> 1) & 1)) return false;
                    if (j + 1 < n0) scores(c0, N_);
                }
                if (j < n1 && !outputs(c1, P_, p_turn1, j == 0, j + 1 == n1)) return false;
                commit_if(lead, empty + 8 * (2 * P + 1));
                if (j + 1 < n) {
                    if (j + 1 < n1) scores(c1, N_);
                    commit_if(lead, empty + 8 * 2 * N);
                    if (j + 2 == n) commit_if(lead, q_empty);
                }
                ++count;
                return true;
            };
            auto begin = [&](auto P_, int n) {
                constexpr uint32_t P = decltype(P_)::v;
                if (!wait(full + 8 * 2 * P, (count >> 1) & 1)) return false;
                scores(c0, P_);
                if (n1 > 0) scores(c1, P_);
                commit_if(lead, empty + 8 * 2 * P);
                if (n == 1) commit_if(lead, q_empty);
                return true;
            };
            bool ok = true;
            for (int64_t id = blockIdx.x; ok && __all_sync(0xffffffffu, w.find(g, id)); id += gridDim.x) {
                n0 = __shfl_sync(0xffffffffu, w.n0, 0);
                if (n0 == 0) continue;
                n1 = __shfl_sync(0xffffffffu, w.n1, 0);
                len = __shfl_sync(0xffffffffu, w.len, 0);
                const int n = max(n0, n1);
                ok = wait(q_full, work & 1) && ((count & 1) ? begin(c1, n) : begin(c0, n));
                for (int j = 0; ok && j < n; ++j) ok = (count & 1) ? step(c1, c0, j, n) : step(c0, c1, j, n);
                ++work;
            }
            if (*abort) {   // products in flight end before the tensor memory goes
                if (lane == 0) {
                    volatile int* drain = &drain_flag;
                    mma_commit(drained);
                    mbar_wait(drained, 0, limit, drain, SITE_PROMPT_WAIT);
                }
            }
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kPSoftRegs));
        const int i = (warp >> 2) - 1;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's 32 lanes of tensor memory
        const uint32_t ts = t_s + 128 * i + lanes, to = t_o + D * i + lanes;
        const float sc = g.scale;
        const bool neg = sc < 0.0f;
        uint32_t s_turn = 0, o_turn = 0;
        bool ok = true;
        for (int64_t id = blockIdx.x; ok && w.find(g, id); id += gridDim.x) {
            const int n = i == 0 ? w.n0 : w.n1;
            if (n == 0) continue;
            const int r = w.row + 128 * i + (tid & 127);      // this thread's row, in the sequence
            const int see = g.causal ? min(r + 1, w.len) : w.len;
            const int sure = g.causal ? min(w.row + 128 * i + 1, w.len) : w.len;   // what every row of the tile sees
            float m = kNoReference, l = 0.0f;
            for (int j = 0; j < n; ++j) {
                ok = warp_wait(s_full + 8 * i, s_turn & 1, limit, abort, SITE_PROMPT_WAIT);
                if (!ok) break;
                ++s_turn;
                tc_fence_after();
                uint32_t x[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(ts + 32 * c, x[c]);
                tmem_wait_ld();
                if (128 * j + 128 > sure) {
                    const int v = see - 128 * j;   // columns this row sees
                    const uint32_t none = neg ? 0x7f800000u : 0xff800000u;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * c + e >= v) x[c][e] = none;
                }
                float t[4];
                if (neg) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        t[c] = fminf(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]));
#pragma unroll
                        for (int e = 2; e < 32; e += 2) t[c] = fminf(t[c], fminf(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])));
                    }
                    t[0] = fminf(fminf(t[0], t[1]), fminf(t[2], t[3]));
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        t[c] = fmaxf(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]));
#pragma unroll
                        for (int e = 2; e < 32; e += 2) t[c] = fmaxf(t[c], fmaxf(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])));
                    }
                    t[0] = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                }
                const float top = t[0] * sc;
                if (__any_sync(0xffffffffu, top > m + kPSlack)) {
                    const float mn = fmaxf(m, top);
                    const float f = exp2_fast(m - mn);
                    m = mn;
                    if (j > 0) {   // the accumulator: the products before these scores are complete
                        l *= f;
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(to + 32 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st_32x32b_x32(to + 32 * c, o);
                        }
                    }
                }
                const uint64_t sc2 = f2_pack(sc, sc), m2 = f2_pack(-m, -m);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int c = 2 * half + (e >> 4), k = (2 * e) & 31;
                        float a, b;
                        f2_unpack(pair_fma(f2_pack(__uint_as_float(x[c][k]), __uint_as_float(x[c][k + 1])), sc2, m2), a, b);
                        a = exp2_fast(a);
                        b = exp2_fast(b);
                        sum[e & 3] = f2_add(sum[e & 3], f2_pack(a, b));
                        pk[e] = pack_bf16x2(a, b);
                    }
                    tmem_st_32x32b_x32(ts + 32 * half, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * i);
                float a, b;
                f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), a, b);
                l += a + b;
            }
            if (!ok) break;
            ok = warp_wait(o_full + 8 * i, o_turn & 1, limit, abort, SITE_PROMPT_WAIT);
            if (!ok) break;
            ++o_turn;
            tc_fence_after();
            const float inv = 1.0f / l;
            const int64_t at = (int64_t)(w.start + r) * g.n_q_heads + w.h;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(to + 32 * c, o);
                tmem_wait_ld();
                if (r < w.len) {
                    uint4* dst = reinterpret_cast<uint4*>(g.out + at * D + 32 * c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            y[k] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * k]) * inv, __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                        dst[e] = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            if (g.lse && r < w.len) g.lse[at] = 0.6931471805599453f * (m + log2f(l));
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<512>(tmem);
    }
}

// Tokens [T][heads][D] bf16, `stride` elements from token to token, as a map whose box is 64
// channels of one head of 128 tokens.
sq_status make_map_tokens(CUtensorMap* map, const void* base, int64_t T, int64_t heads, int64_t D, int64_t stride) {
    sq_status r = get_encoder();
    if (r != SQ_OK) return r;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64u, 1u, 128u};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult cr = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (cr != CUDA_SUCCESS) {
        set_error("cuTensorMapEncodeTiled failed (%d) for %lld tokens of %lld heads", (int)cr, (long long)T, (long long)heads);
        return SQ_ERR_CUDA;
    }
    return SQ_OK;
}

template <int D>
sq_status launch_prompt(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PromptArgs& g, cudaStream_t st) {
    static bool attr_done[64] = {};
    const DeviceInfo& di = device_info();
    constexpr size_t smem = PromptSmem<D>::TOTAL;
    sq_status r = ensure_smem_attr(prompt_attention_kernel<D>, smem, attr_done[di.device & 63]);
    if (r != SQ_OK) return r;
    const int64_t items = g.blocks * g.n_q_heads;
    const unsigned grid = (unsigned)(items < di.sm_count ? items : di.sm_count);
    return launch_pdl("prompt_attention_kernel", prompt_attention_kernel<D>, dim3(grid), dim3(kPThreads), smem, st, 1, mq, mk, mv, g);
}

sq_status prompt_attention_impl(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const int32_t* cu, int64_t n_seqs, int64_t T, int64_t n_q_heads,
                                int64_t n_kv_heads, int64_t D, float scale, int causal, void* out, float* lse,
                                cudaStream_t st) {
    sq_status r;
    if (n_seqs < 0 || T < 0 || n_q_heads < 0 || n_kv_heads < 0) { set_error("negative size"); return SQ_ERR_INVALID_ARG; }
    if (D != 64 && D != 128) { set_error("head_dim must be 64 or 128 (got %lld)", (long long)D); return SQ_ERR_UNSUPPORTED; }
    if (!(scale >= -1.0e38f && scale <= 1.0e38f)) { set_error("scale must be within +-1e38"); return SQ_ERR_INVALID_ARG; }
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
    // A scale of 0 weighs all tokens alike; a smaller factor than any score times it can
    // show keeps masked scores at -infinity.
    const float sc = (scale == 0.0f ? 1.0e-37f : scale) * 1.4426950408889634f;
    PromptArgs g{static_cast<__nv_bfloat16*>(out), lse, cu, T, T / 256 + n_seqs, (int)n_seqs, (int)n_q_heads, (int)(n_q_heads / n_kv_heads), sc,
                 causal != 0, wait_limit_cycles()};
    CUtensorMap mq, mk, mv;
    if ((r = make_map_tokens(&mq, q, T, n_q_heads, D, q_stride)) != SQ_OK) return r;
    if ((r = make_map_tokens(&mk, k, T, n_kv_heads, D, k_stride)) != SQ_OK) return r;
    if ((r = make_map_tokens(&mv, v, T, n_kv_heads, D, v_stride)) != SQ_OK) return r;
    return D == 64 ? launch_prompt<64>(mq, mk, mv, g, st) : launch_prompt<128>(mq, mk, mv, g, st);
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
