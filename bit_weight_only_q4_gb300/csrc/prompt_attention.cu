// Causal attention over whole prompts, packed one behind the other, with grouped heads:
// for query token i of a sequence and a head that shares key head h,
//     s_ij = scale log2(e) (q_i . k_j),  p_ij = 2^(s_ij - m_i)  for j <= i,
//     out_i = sum_j p_ij v_j / sum_j p_ij.
// Products are bf16 with fp32 sums, s, p and its sum fp32; p goes to the second product as bf16, as
// wide as the v that it meets there (at most 2^-8 of each term of the sum).
//
// A tile is 128 rows: T = 128 / G tokens with the G query heads of one key head, token by
// token, so that grouped heads share each tile of keys.  A unit of work is two neighbouring
// tiles A and B (2 T tokens) of one key head; both run over the same tiles of 128 keys, from
// their own tokens back to the first.  The order matters: only the first tile or two are cut by
// the mask, and the reference m_i that they give serves for the others.  m_i need not be the largest
// s_ij: p keeps its relative precision at any size, and only when a tile's sum passes 2^20 is the
// reference raised and what was summed scaled down.  So a tile that is seen whole costs one pass over its scores and no maximum.
// (Of 2^31 tokens, 64 at least to a sum, the sums together stay below 2^45, and with |v| up to 2^80 in fp32's range.)
//
// One CTA per SM, 12 warps: four with the softmax of A (one thread a row), four with that of
// B, one that copies (TMA), one or two that issue the MMAs, one that fetches units.  A step is one tile of
// rows on one tile of keys; A and B take turns, so that the tensor cores work on one while the
// other is in its softmax.
//   Heads of 128: two S and two O fill the tensor memory, and P takes the place of its S, whose MMA for the next step
//   comes behind the one that reads P.  P is handed over in two halves, so that less of a step's softmax lies between two MMAs of
//   its rows (1 to 4% faster than whole; with heads of 64, whose S comes earlier, 15% slower).
//   Heads of 64: P has a place of its own, and S is free for the next step as soon as it has been read: a step's softmax
//   follows that of the rows' last one without a wait.
//
// A masked probability is 0, and 0 times a v that is not finite would be NaN: tiles cut by the
// mask are looked through for such values (by the warp that fetches units), and a tile that has one
// is multiplied by the softmax threads themselves, over the tokens that a row sees.
//
// What bounds it.  Heads of 128, 32 on 8: the tensor cores, whose pipe is busy for 76% of the SMs' time: 7 prompts of 333
// to 8,191 tokens 1,050 us, 1,735 TFLOP/s of what the mask leaves (89% of a large library product's rate); one of 32,768
// 5,000 to 5,300 us, 1,660 to 1,760 TFLOP/s, as the power limit has it.  The rest is tiles that the mask cuts, and a unit's
// beginning and end, some 7,000 cycles, which rule for short prompts: 48 of 37 to 1,501 tokens, 16 heads, 177 us, 895 TFLOP/s.
// Heads of 64: half the products for as many exponentials, so 2^x (4 cycles a warp and scheduler) and what is about it: 3
// prompts of 5,000 to 16,383 tokens, 28 on 4 heads, 1,240 us, 1,220 TFLOP/s.  5 of at most 77 tokens: 6.5 us, latency.
// All of these are calls in a captured graph.
#include "layer_ops.h"
#include "segments.cuh"
#include "tc_device.cuh"
#include "tma.h"

#include <atomic>

namespace q4 {

constexpr int PA_ROWS = 128, PA_KEYS = 128;
constexpr int PA_COPY = 8, PA_MMA = 9, PA_NEXT = 10, PA_ADD = 11, PA_WARPS = 12;
constexpr int PA_QUEUE = 2;                // units that a CTA has been given and not begun
constexpr float PA_SUM_TOP = 0x1p20f;

template <int D>
struct PaSmem {
    static constexpr bool APART = D == 64;                           // P is not in the place of S
    static constexpr int HALVES = APART ? 1 : 2;
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr uint32_t TILE = PA_KEYS * D * 2;
    static constexpr uint32_t RING = 2 * TILE;                       // [Q of A, Q of B][ring][results, 4 KB a warp]
    static constexpr uint32_t STAGE = RING + STAGES * TILE;
    static constexpr uint32_t TOTAL = STAGE + 8 * 4096;
};

// What a unit is.
struct __align__(16) PaUnit {
    int start, len;              // the sequence's first row and tokens
    int first;                   // first token of tile A
    int head;                    // key head
    int na, nb;                  // key tiles of A and of B (0: B has no token; na = 0: no unit)
    int pad[2];
};

// A warp's units.  Units are numbered by sequence, then from the last pair of tiles to the first, then
// by key head.
struct PaWalk {
    const PromptArgs &p;
    SegmentWalk walk;

    __device__ explicit PaWalk(const PromptArgs &args)
        : p(args), walk(Segments{args.offsets, args.batch, args.tokens, 2 * args.tile_tokens, args.kv_heads, args.err}) {}

    __device__ bool find(int number, PaUnit &u)
    {
        SegmentUnit f;
        if (!walk.find(number, f))
            return false;
        const int t = p.tile_tokens, pair = 2 * t, back = f.unit / p.kv_heads;
        u.start = f.start;
        u.len = f.len;
        u.head = f.unit - back * p.kv_heads;
        u.first = ((f.len + pair - 1) / pair - 1 - back) * pair;
        const int rest = u.len - u.first;
        u.na = (u.first + (rest < t ? rest : t) + PA_KEYS - 1) / PA_KEYS;
        u.nb = rest <= t ? 0 : (u.first + (rest < pair ? rest : pair) + PA_KEYS - 1) / PA_KEYS;
        return true;
    }
};

// 32 scores of a row to probabilities: ta, tb += 2^(s sl + neg), p <- the same as bf16.  CUT: columns from `at` on
// past `seen` count as none, and the sum is of the rounded values: where a row sees few tokens, what rounding does to all of
// its probabilities alike goes away with that.
template <bool CUT>
__device__ __forceinline__ void pa_exp(const uint32_t (&s)[32], uint32_t *p, f32x2 sl2, f32x2 neg2, f32x2 &ta, f32x2 &tb,
                                       int at, int seen)
{
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const f32x2 a = fma2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), sl2, neg2);
        const f32x2 b = fma2(pack2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), sl2, neg2);
        float e[4];
        unpack2(a, e[0], e[1]);
        unpack2(b, e[2], e[3]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if (CUT)
                e[y] = at + i + y <= seen ? e[y] : -INFINITY;
            e[y] = ex2(e[y]);
        }
        p[i / 2] = bf16_pair(e[0], e[1]);
        p[i / 2 + 1] = bf16_pair(e[2], e[3]);
        if (CUT) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
                e[y] = __uint_as_float(y & 1 ? p[(i + y) / 2] & 0xffff0000u : p[(i + y) / 2] << 16);
        }
        ta = add2(ta, pack2(e[0], e[1]));
        tb = add2(tb, pack2(e[2], e[3]));
    }
}

// A row's probabilities (N pairs) where the mask cuts: those behind the first `seen` are none, and the sum is of the rounded
// values that are left: where a row sees few tokens, what rounding does to all of its probabilities alike goes away with that.
template <int N>
__device__ __forceinline__ void pa_cut(uint32_t (&p)[N], int seen, f32x2 &ta, f32x2 &tb)
{
    ta = tb = 0ull;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = seen > 2 * i + 1 ? p[i] : seen > 2 * i ? p[i] & 0xffffu : 0u;
        const f32x2 e = pack2(__uint_as_float(p[i] << 16), __uint_as_float(p[i] & 0xffff0000u));
        if (i & 1)
            tb = add2(tb, e);
        else
            ta = add2(ta, e);
    }
}

// 0 v + acc for a pair of bf16: NaN if v is not finite or acc is NaN already, else a zero.
__device__ __forceinline__ uint32_t pa_fma_bf16(uint32_t v, uint32_t acc)
{
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0u), "r"(acc));
    return r;
}

// Asks for a CTA of the grid that has not begun, to have its work instead: 16 bytes at `to`, counted on `bar`.
__device__ __forceinline__ void pa_ask(uint32_t to, uint32_t bar)
{
    mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(to), "r"(bar) : "memory");
}

// The answer: that CTA's number, or -1 (no question may be asked after that).
__device__ __forceinline__ int pa_answer(uint32_t at)
{
    int r;
    asm volatile("{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
                 "ld.shared.b128 h, [%1];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
                 "mov.s32 %0, -1;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
                 : "=r"(r) : "r"(at) : "memory");
    return r;
}

template <int D>
__global__ void __launch_bounds__(PA_WARPS * 32, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                            const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap out_map,
                            const PromptArgs p)
{
    using L = PaSmem<D>;
    constexpr int NS = L::STAGES;
    constexpr bool APART = L::APART;
    constexpr int HALVES = L::HALVES, CH = PA_KEYS / HALVES;
    // tensor memory: S of A and of B, P (where it is apart), O
    constexpr uint32_t TM_S = 0, TM_P = APART ? 256 : TM_S, TM_P_STEP = APART ? 64 : 128, TM_P_HALF = APART ? CH / 2 : CH,
                       TM_O = APART ? 384 : 256, TM_COLS = 512;
    static_assert(TM_O + 2 * D <= TM_COLS, "tensor memory");
    constexpr uint32_t BF16 = (1u << 7) | (1u << 10);
    constexpr uint32_t IDESC_S = (1u << 4) | BF16 | ((uint32_t)(PA_KEYS >> 3) << 17) | (8u << 24);
    constexpr uint32_t IDESC_O = (1u << 4) | BF16 | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ uint64_t s_bar[2 * NS + 9 + 4 * HALVES + 2 * PA_QUEUE + 1 + NS];
    __shared__ uint32_t s_tmem;
    __shared__ __align__(16) uint4 s_answer;
    __shared__ PaUnit s_unit[PA_QUEUE];
    __shared__ int s_dead, s_bad[NS];
    const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
    const uint32_t kv_full = smem_u32(s_bar), kv_free = kv_full + 8u * NS, q_full = kv_free + 8u * NS,   // q_full: A, B
                   q_free = q_full + 16, drained = q_full + 24, pv_done = q_full + 40,      // pv_done: by tile and half
                   s_full = pv_done + 16u * HALVES, s_free = s_full + 16, p_full = s_free + 16,        // by tile (and half)
                   unit_full = p_full + 16u * HALVES, unit_free = unit_full + 8u * PA_QUEUE,
                   answered = unit_free + 8u * PA_QUEUE, v_raw = answered + 8;        // by stage: V that is to be looked through
    pdl_wait();
    PaWalk walk(p);
    PaUnit u;
    if (!walk.find((int)blockIdx.x ^ p.swap, u))
        return;                                            // (the whole CTA)
    if (warp == PA_COPY) {
        if (lane == 0) {
            for (int i = 0; i < NS; ++i) {
                mbar_init(kv_full + 8u * i, 1);
                mbar_init(kv_free + 8u * i, 1);
                mbar_init(v_raw + 8u * i, 1);
            }
            mbar_init(q_free, 1);
            mbar_init(drained, 1);
            mbar_init(drained + 8, 1);
            mbar_init(answered, 1);
            for (int i = 0; i < PA_QUEUE; ++i) {
                mbar_init(unit_full + 8u * i, 1);
                mbar_init(unit_free + 8u * i, APART ? 11 : 10);        // softmax, copies, MMAs
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(q_full + 8u * i, 1);
                for (int half = 0; half < HALVES; ++half)
                    mbar_init(pv_done + 8u * (i * HALVES + half), 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(s_full + 8u * i, 1);
                mbar_init(s_free + 8u * i, 4);
            }
            for (int i = 0; i < 2 * HALVES; ++i)
                mbar_init(p_full + 8u * i, 4);
            s_dead = 0;
        }
        mbar_init_fence();
    } else if (warp == PA_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&s_tmem)), "n"(TM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    const KvDead dead = {p.err, &s_dead, smem_u32(&s_dead)};
    auto gone_all = [&]() { return __any_sync(0xffffffffu, *dead.flag != 0); };
    // The CTA's unit of a round, the first being its own; false: there is none.
    auto unit = [&](int round) {
        if (round == 0)
            return true;
        const int slot = (round - 1) % PA_QUEUE;
        kv_wait(unit_full + 8u * slot, (uint32_t)((round - 1) / PA_QUEUE) & 1u, dead);
        const uint4 e = lds128(smem_u32(&s_unit[slot])), f = lds128(smem_u32(&s_unit[slot]) + 16u);
        u.start = (int)e.x, u.len = (int)e.y, u.first = (int)e.z, u.head = (int)e.w, u.na = (int)f.x, u.nb = (int)f.y;
        __syncwarp();
        if (lane == 0)
            mbar_arrive(unit_free + 8u * slot);
        return u.na > 0;
    };

    if (warp < 8) {
        // ------------------------------------------ softmax and results
        const int x = warp >> 2;                           // tile: A, B
        const int quad = warp & 3;
        const int row = quad * 32 + lane;
        const int row_token = row / p.group, row_head = row - row_token * p.group;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_o = t_lane + TM_O + (uint32_t)(D * x);
        const float sl = p.scale_log2;
        const f32x2 sl2 = pack2(sl, sl);
        const uint32_t t_s = t_lane + TM_S + 128u * x, t_ps = t_lane + TM_P + TM_P_STEP * x;
        uint32_t ring = 0u, steps = 0u, pv_count = 0u;     // copies, this tile's steps and waited-for MMAs before
        const uint32_t pv_first = pv_done + 8u * (uint32_t)(x * HALVES), pv_last = pv_first + 8u * (HALVES - 1);
        // The step before is through its MMAs.  Where P is in the place of S, this step's S came behind them; where it
        // is apart, each step waits for the one before it, so that no barrier is ever two phases from the one that is waited for.
        auto last_step = [&]() {
            if (APART && pv_count > 0) {
                kv_wait(pv_last, (pv_count - 1u) & 1u, dead);
                tc_fence_after();
            }
        };
        // And so are the halves of this step before half `half`.
        auto pv_wait = [&](int half) {
            last_step();
            if (half > 0)
                kv_wait(pv_first, steps & 1u, dead);
            tc_fence_after();
        };
#pragma unroll 1
        for (int round = 0;; ++round) {
            if (!unit(round) || gone_all())
                break;
            const int n = u.nb > 0 ? u.nb : u.na, mine = x ? u.nb : u.na;
            const int first = u.first + x * p.tile_tokens;
            // the row's token within the sequence; -1: there is none
            const int token = row_token < p.tile_tokens && first + row_token < u.len ? first + row_token : -1;
            const int whole = (first + 1) / PA_KEYS;       // key tiles that all rows see wholly
            float m = -INFINITY;
            f32x2 la = 0ull, lb = 0ull;
#pragma unroll 1
            for (int j = mine - 1; j >= 0; --j) {
                const bool masked = j >= whole;
                const int seen = token >= 0 ? token - j * PA_KEYS : PA_KEYS - 1;      // the row's last visible column
                int hi = PA_KEYS - 1;
                const uint32_t v_at = ring + 2u * (uint32_t)(n - 1 - j) + 1u, v_stage = v_at & (NS - 1);
                const uint32_t v_tile = sm + L::RING + v_stage * L::TILE;
                kv_wait(s_full + 8u * x, steps & 1u, dead);
                tc_fence_after();
                if (masked)
                    hi = __reduce_max_sync(0xffffffffu, seen);
#pragma unroll 1
                for (int half = 0; half < HALVES; ++half) {
                    const int c0 = half * CH;
                    uint32_t ph[CH / 2];
                    bool careful = false;
                    if (APART) {
                        // One code for tiles that the mask cuts and for others, for instructions that a unit passes once have to be
                        // fetched anew: 7% faster than two, 48 short texts 10%.  (Heads of 128, with more and shorter parts, are
                        // 1 to 3% slower so.)
                        uint32_t v[2][32];
                        const bool fresh = __any_sync(0xffffffffu, token >= 0 && m == -INFINITY);
                        float neg = -m;
                        tmem_ld32_async(t_s + (uint32_t)c0, v[0]);
                        tmem_wait_ld();
                        if (fresh) {
                            // the first reference: the largest of the first 16 scores that are seen
                            float want = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                want = c0 + i <= seen ? fmaxf(want, __uint_as_float(v[0][i]) * sl) : want;
                            if (m == -INFINITY)
                                m = want;
                            careful = __any_sync(0xffffffffu, token >= 0 && seen >= c0 && m == -INFINITY);
                            neg = m == -INFINITY ? 0.f : -m;
                        }
                        const f32x2 n2 = pack2(neg, neg);
                        f32x2 ta = 0ull, tb = 0ull;
#pragma unroll
                        for (int c = 0; c < CH / 32; ++c) {
                            if (c + 1 < CH / 32)
                                tmem_ld32_async(t_s + (uint32_t)(c0 + 32 * (c + 1)), v[(c + 1) & 1]);
                            pa_exp<false>(v[c & 1], ph + 16 * c, sl2, n2, ta, tb, 0, 0);
                            if (c + 1 < CH / 32)
                                tmem_wait_ld();
                        }
                        if (masked)
                            pa_cut(ph, seen + 1 - c0, ta, tb);
                        float sa, sb;
                        unpack2(add2(ta, tb), sa, sb);
                        careful = careful || __any_sync(0xffffffffu, token >= 0 && !(sa + sb < PA_SUM_TOP));
                        if (!careful) {
                            la = add2(la, ta);
                            lb = add2(lb, tb);
                        }
                    } else if (!masked && !__any_sync(0xffffffffu, token >= 0 && m == -INFINITY)) {
                        uint32_t v[2][32];
                        tmem_ld32_async(t_s + (uint32_t)c0, v[0]);
                        tmem_wait_ld();
                        const f32x2 n2 = pack2(-m, -m);
                        f32x2 ta = 0ull, tb = 0ull;
#pragma unroll
                        for (int c = 0; c < CH / 32; ++c) {
                            if (c + 1 < CH / 32)
                                tmem_ld32_async(t_s + (uint32_t)(c0 + 32 * (c + 1)), v[(c + 1) & 1]);
                            pa_exp<false>(v[c & 1], ph + 16 * c, sl2, n2, ta, tb, 0, 0);
                            if (c + 1 < CH / 32)
                                tmem_wait_ld();
                        }
                        float sa, sb;
                        unpack2(add2(ta, tb), sa, sb);
                        careful = __any_sync(0xffffffffu, token >= 0 && !(sa + sb < PA_SUM_TOP));
                        if (!careful) {
                            la = add2(la, ta);
                            lb = add2(lb, tb);
                        }
                    } else if (c0 > hi) {
#pragma unroll
                        for (int i = 0; i < CH / 2; ++i)
                            ph[i] = 0u;
                    } else {
                        f32x2 ta = 0ull, tb = 0ull;
#pragma unroll
                        for (int c = 0; c < CH / 32; ++c) {
                            const int at = c0 + 32 * c;
                            if (at > hi) {
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    ph[16 * c + i] = 0u;
                                continue;
                            }
                            uint32_t v[32];
                            tmem_ld32_async(t_s + (uint32_t)at, v);
                            tmem_wait_ld();
                            if (c == 0 && __any_sync(0xffffffffu, token >= 0 && m == -INFINITY)) {
                                // the first reference: the largest of the first 16 scores that are seen
                                float want = -INFINITY;
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    want = at + i <= seen ? fmaxf(want, __uint_as_float(v[i]) * sl) : want;
                                if (m == -INFINITY)
                                    m = want;
                                careful = __any_sync(0xffffffffu, token >= 0 && seen >= at && m == -INFINITY);
                            }
                            const float neg = m == -INFINITY ? 0.f : -m;
                            pa_exp<true>(v, ph + 16 * c, sl2, pack2(neg, neg), ta, tb, at, seen);
                        }
                        float sa, sb;
                        unpack2(add2(ta, tb), sa, sb);
                        careful = careful || __any_sync(0xffffffffu, token >= 0 && !(sa + sb < PA_SUM_TOP));
                        if (!careful) {
                            la = add2(la, ta);
                            lb = add2(lb, tb);
                        }
                    }
                    const bool begun = j < mine - 1 || half > 0;       // O holds something
                    if (careful) {
                        // again, with the half's largest score as the reference
                        float want = -INFINITY;
#pragma unroll 1
                        for (int c = c0; c < c0 + CH; c += 32) {
                            uint32_t v[32];
                            tmem_ld32_async(t_s + (uint32_t)c, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float s = __uint_as_float(v[i]) * sl;
                                want = c + i <= seen ? fmaxf(want, s) : want;
                            }
                        }
                        if (__any_sync(0xffffffffu, want > m)) {
                            const float old = m;
                            m = fmaxf(m, want);
                            const float f = old == -INFINITY ? 0.f : ex2(old - m);
                            const f32x2 f2 = pack2(f, f);
                            la = mul2(la, f2);
                            lb = mul2(lb, f2);
                            if (begun) {
                                pv_wait(half);
#pragma unroll 1
                                for (int c = 0; c < D; c += 32) {
                                    uint32_t o[32];
                                    tmem_ld32_async(t_o + c, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                    tmem_st32(t_o + c, o);
                                }
                                tmem_wait_st();
                            }
                        }
                        const float neg = m == -INFINITY ? 0.f : -m;
#pragma unroll
                        for (int c = 0; c < CH / 32; ++c) {
                            uint32_t v[32];
                            tmem_ld32_async(t_s + (uint32_t)(c0 + 32 * c), v);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                float a = ex2(fmaf(__uint_as_float(v[i]), sl, neg)), b = ex2(fmaf(__uint_as_float(v[i + 1]), sl, neg));
                                a = c0 + 32 * c + i <= seen ? a : 0.f;
                                b = c0 + 32 * c + i + 1 <= seen ? b : 0.f;
                                la = add2(la, pack2(a, b));
                                ph[16 * c + i / 2] = bf16_pair(a, b);
                            }
                        }
                    }
                    if (APART) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(s_free + 8u * x);
                        last_step();                       // (its P has been read)
                    }
                    const uint32_t t_p = t_ps + TM_P_HALF * (uint32_t)half;
#pragma unroll
                    for (int c = 0; c < CH / 2; c += 32)
                        tmem_st32(t_p + c, reinterpret_cast<uint32_t(&)[32]>(ph[c]));
                    tmem_wait_st();
                    bool skip = false;
                    if (masked) {
                        // (behind the wait for S: what the ring's stage held before has been loaded by then, so that the
                        // phase is this one or the next)
                        kv_wait(kv_full + 8u * v_stage, (v_at / NS) & 1u, dead);
                        skip = __shfl_sync(0xffffffffu, *(volatile int *)&s_bad[v_stage], 0) != 0;
                    }
                    if (skip) {
                        // O += P V over the tokens that the row sees, 16 columns at a time
                        if (begun)
                            pv_wait(half);
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            float o[16];
                            uint32_t w[16];
                            if (begun)
                                tmem_ld16(t_o + c, w);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = begun ? __uint_as_float(w[i]) : 0.f;
#pragma unroll 1
                            for (int k = c0; k < c0 + CH; ++k) {
                                uint32_t pk;
                                tmem_ld1(t_p + ((k - c0) >> 1), pk);
                                const float pf = __uint_as_float((k & 1) ? pk & 0xffff0000u : pk << 16);
                                const uint32_t r = v_tile + (uint32_t)(c >> 6) * 16384u + (uint32_t)k * 128u;
                                const uint32_t piece = (uint32_t)(c >> 3) & 7u;
                                const uint4 e0 = lds128(r + 16u * (piece ^ ((uint32_t)k & 7u)));
                                const uint4 e1 = lds128(r + 16u * ((piece + 1u) ^ ((uint32_t)k & 7u)));
                                const uint32_t e[8] = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
                                if (k <= seen) {
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {
                                        o[2 * i] = fmaf(pf, __uint_as_float(e[i] << 16), o[2 * i]);
                                        o[2 * i + 1] = fmaf(pf, __uint_as_float(e[i] & 0xffff0000u), o[2 * i + 1]);
                                    }
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = __float_as_uint(o[i]);
                            tmem_st16(t_o + c, w);
                        }
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(p_full + 8u * (uint32_t)(x * HALVES + half));
                }
                if (APART || j == 0)
                    ++pv_count;
                ++steps;
            }
            ring += 2u * (uint32_t)n;
            if (mine == 0)
                continue;
            // ---- the unit's results
            kv_wait(pv_last, (pv_count - 1u) & 1u, dead);
            tc_fence_after();
            float l0, l1;
            unpack2(add2(la, lb), l0, l1);
            const float inv = 1.f / (l0 + l1);             // (a row of no score above -inf: 0 / 0)
            const bool gone = gone_all(), full = p.box_tokens > 0 && __all_sync(0xffffffffu, token >= 0);
            if (full) {
                // All of the warp's rows are results: by way of its 4 KB of shared memory, 64 columns at a time, and from
                // there by TMA (whose rows of 128 bytes have piece c at c ^ (row & 7)).
                const uint32_t st = sm + L::STAGE + (uint32_t)warp * 4096u, st_row = st + (uint32_t)lane * 128u;
#pragma unroll 1
                for (int c = 0; c < D; c += 64) {
                    uint32_t o[2][32];
                    tmem_ld32_async(t_o + c, o[0]);
                    tmem_ld32_async(t_o + c + 32, o[1]);
                    tmem_wait_ld();
                    uint32_t e[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        e[i] = bf16_pair(__uint_as_float(o[i / 16][2 * i % 32]) * inv, __uint_as_float(o[i / 16][2 * i % 32 + 1]) * inv);
                    if (lane == 0)                         // (the last store has read them)
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sts128(st_row + (((uint32_t)i ^ ((uint32_t)lane & 7u)) << 4), e[4 * i], e[4 * i + 1], e[4 * i + 2], e[4 * i + 3]);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0 && !gone) {
                        tma_store_3d(&out_map, c, u.head * p.group, u.start + token, st);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                }
            } else {
                uint16_t *to = p.out + ((int64_t)(u.start + token) * p.q_heads + u.head * p.group + row_head) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32_async(t_o + c, o);
                    tmem_wait_ld();
                    uint32_t e[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        e[i] = bf16_pair(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                    if (token >= 0 && !gone) {
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            *reinterpret_cast<uint4 *>(to + c + 2 * i) = make_uint4(e[i], e[i + 1], e[i + 2], e[i + 3]);
                    }
                }
            }
            tc_fence_before();                             // (the next P of this tile lets its O be written again)
        }
        if (lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else if (warp == PA_COPY) {
        // ------------------------------------------------------- copies
        uint32_t at = 0u;
        uint32_t loads[2] = {0u, 0u}, raw = 0u, raw_uses = 0u;           // stages that v_raw counts now; its parities
#pragma unroll 1
        for (int round = 0; unit(round) && !gone_all(); ++round) {
            const int n = u.nb > 0 ? u.nb : u.na, cut = n - (u.first + 1) / PA_KEYS;       // V is looked through
#pragma unroll 1
            for (int i = 0; i < 2 * n && !gone_all(); ++i, ++at) {
                const uint32_t s = at & (NS - 1);
                if (at >= NS)
                    kv_wait(kv_free + 8u * s, (at / NS - 1u) & 1u, dead);
                if (gone_all())
                    break;
                const bool look = (i & 1) && i / 2 < cut;
                raw = look ? raw | 1u << s : raw & ~(1u << s);
                raw_uses ^= (uint32_t)look << s;
                if (elect_one()) {
                    const CUtensorMap *map = (i & 1) ? &v_map : &k_map;
                    const uint32_t dst = sm + L::RING + s * L::TILE, bar = (look ? v_raw : kv_full) + 8u * s;
                    mbar_arrive_expect_tx(bar, L::TILE);
#pragma unroll
                    for (int c = 0; c < D; c += 64)
                        tma_load_3d(dst + (uint32_t)c * 256u, map, c, u.head, u.start + (n - 1 - i / 2) * PA_KEYS, bar);
                }
                __syncwarp();
                if (i == 0) {                              // (behind the first keys)
                    if (round > 0)
                        kv_wait(q_free, (uint32_t)(round - 1) & 1u, dead);
                    if (gone_all()) {
                        ++at;
                        break;
                    }
                    for (int x = 0; x < (u.nb > 0 ? 2 : 1); ++x, __syncwarp()) {
                        if (elect_one()) {
                            const uint32_t bytes = (uint32_t)(p.tile_tokens * p.group) * D * 2;
                            mbar_arrive_expect_tx(q_full + 8u * x, bytes);
#pragma unroll
                            for (int c = 0; c < D; c += 64)
                                tma_load_3d(sm + (uint32_t)x * L::TILE + (uint32_t)c * 256u, &q_map, c, u.head * p.group,
                                            u.start + u.first + x * p.tile_tokens, q_full + 8u * x);
                        }
                        ++loads[x];
                    }
                }
            }
        }
        if (gone_all()) {
            // copies in flight land before the CTA ends
            for (uint32_t i = at > NS ? at - NS : 0u; i < at; ++i) {
                const uint32_t s = i & (NS - 1);
                if ((raw >> s) & 1u)
                    mbar_wait(v_raw + 8u * s, ~(raw_uses >> s) & 1u, p.err);
                else
                    mbar_wait(kv_full + 8u * s, (i / NS) & 1u, p.err);
            }
            for (int x = 0; x < 2; ++x)
                if (loads[x] > 0)
                    mbar_wait(q_full + 8u * x, (loads[x] - 1u) & 1u, p.err);
        }
    } else if (warp == PA_MMA || (APART && warp == PA_ADD)) {
        // -------------------------------------------------------- MMAs
        // This warp is what the tensor cores wait for, so the two tiles are written out (x is known where it is
        // compiled) and everything that an MMA takes is the warp's: such an MMA takes 30 (PV) and 52 cycles (S) to
        // issue, of the 64 or 32 that it runs.
        uint32_t at = 0u, qn = 0u, sn[2] = {0u, 0u}, pn = 0u;          // copies before this unit; parities of Q loads, S's, parities of P's
        const uint64_t qd = smem_desc_sw128(sm), kd = smem_desc_sw128(sm + L::RING);
        const uint64_t vd = (kd & ~((uint64_t)0x3fff << 16)) | ((uint64_t)(D == 128 ? PA_KEYS * 128 >> 4 : 0) << 16);
        const uint32_t q_lo = (uint32_t)qd, q_hi = (uint32_t)(qd >> 32), k_lo = (uint32_t)kd, k_hi = (uint32_t)(kd >> 32),
                       v_lo = (uint32_t)vd, v_hi = (uint32_t)(vd >> 32);
#pragma unroll 1
        for (int round = 0; unit(round) && !gone_all(); ++round) {
            const int nb = __shfl_sync(0xffffffffu, u.nb, 0), na = __shfl_sync(0xffffffffu, u.na, 0),
                      begin = __shfl_sync(0xffffffffu, u.first, 0);
            const bool pair = nb > 0;
            const int n = pair ? nb : na, late = n - na;   // tiles of keys that A begins behind B
            const int cut[2] = {n - (begin + 1) / PA_KEYS, n - (begin + p.tile_tokens + 1) / PA_KEYS};   // that the mask cuts
            // S of tile x on the t-th tile of keys
            auto score = [&](int x, int t) {
                const uint32_t k = at + 2u * (uint32_t)t, stage = k & (NS - 1);
                if (t == (x ? 0 : late)) {
                    kv_wait(q_full + 8u * x, (qn >> x) & 1u, dead);
                    qn ^= 1u << x;
                }
                if (x == 0 || t == 0)                      // (B's S comes behind A's, but for the first)
                    kv_wait(kv_full + 8u * stage, (k / NS) & 1u, dead);
                if (APART && sn[x] > 0)
                    kv_wait(s_free + 8u * x, (sn[x] - 1u) & 1u, dead);
                ++sn[x];
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t a = q_lo + (uint32_t)x * (L::TILE >> 4), b = k_lo + stage * (L::TILE >> 4),
                                   d = tmem + TM_S + 128u * (uint32_t)x;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t step = (uint32_t)(kk >> 2) * (16384u >> 4) + 2u * (kk & 3);
                        mma_f16_2(d, a + step, q_hi, b + step, k_hi, IDESC_S, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(s_full + 8u * (uint32_t)x);
                    if (x == 1 || !pair) {                 // the last with these keys
                        mma_commit(kv_free + 8u * stage);
                        if (t == n - 1)
                            mma_commit(q_free);
                    }
                }
                __syncwarp();
            };
            // O of tile x += P V
            auto add = [&](int x, int t) {
                const uint32_t k = at + 2u * (uint32_t)t + 1u, stage = k & (NS - 1);
                if (x == 0 || t < late)
                    kv_wait(kv_full + 8u * stage, (k / NS) & 1u, dead);
                const bool masked = t < cut[x], first = t == (x ? 0 : late);
#pragma unroll
                for (int half = 0; half < HALVES; ++half) {
                    kv_wait(p_full + 8u * (uint32_t)(x * HALVES + half), (pn >> x) & 1u, dead);
                    tc_fence_after();
                    const bool skip = masked && __shfl_sync(0xffffffffu, *(volatile int *)&s_bad[stage], 0) != 0;
                    if (elect_one()) {
                        if (!skip) {
                            const uint32_t b = v_lo + stage * (L::TILE >> 4), o = tmem + TM_O + (uint32_t)(D * x),
                                           pm = tmem + TM_P + TM_P_STEP * (uint32_t)x + TM_P_HALF * (uint32_t)half;
#pragma unroll
                            for (int kk = 0; kk < CH / 16; ++kk)
                                mma_f16_tmem_a(o, pm + 8u * kk,
                                               b + (uint32_t)(half * (CH / 16) + kk) * (2048 >> 4), v_hi, IDESC_O,
                                               kk > 0 || half > 0 || !first ? 1u : 0u);
                        }
                        if (APART || half < HALVES - 1 || t == n - 1)          // (the others are waited for by none)
                            mma_commit(pv_done + 8u * (uint32_t)(x * HALVES + half));
                        if (APART && half == HALVES - 1 && (x == 1 || !pair))
                            mma_commit(kv_free + 8u * stage);
                    }
                    __syncwarp();
                }
                pn ^= 1u << x;
            };
            auto release = [&](uint32_t k) {
                if (elect_one())
                    mma_commit(kv_free + 8u * (k & (NS - 1)));
                __syncwarp();
            };
            if constexpr (APART) {
                // S and PV wait for different things: a warp each
                const bool adds = warp == PA_ADD;
#pragma unroll 1
                for (int t = 0; t < n && !gone_all(); ++t) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (x ? !pair : t < late)
                            continue;
                        if (adds)
                            add(x, t);
                        else
                            score(x, t);
                    }
                }
            } else {
                score(0, late);
                if (pair)
                    score(1, 0);
#pragma unroll 1
                for (int t = 0; t < n && !gone_all(); ++t) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (x ? !pair : t < late)
                            continue;
                        add(x, t);
                        if (t + 1 < n)
                            score(x, t + 1);
                    }
                    release(at + 2u * (uint32_t)t + 1u);   // V: behind B's next S (measured: before it, grouped prompts 5% slower)
                }
            }
            at += 2u * (uint32_t)n;
        }
    } else if (warp == PA_NEXT) {
        // ------------------------------------------------- units to come
        // The grid has a CTA for each unit that there may be, and an SM room for one: a CTA takes over the units of those
        // that have not begun, so that units of different lengths are dealt out as SMs come free.  CTAs without a unit
        // are taken over too, and that is all: in whatever order CTAs are given up, the last answer is the one that there is
        // none.  The next unit is fetched before this one's V is looked through.
        bool more = true;
        int asked = 0, told = 0;
        uint32_t at = 0u, uses = 0u;                       // copies before this unit, parities of v_raw
        PaUnit now = u;
#pragma unroll 1
        while ((more || now.na > 0) && !gone_all()) {
            u.na = 0;
            if (more) {
                const int slot = told % PA_QUEUE;
                if (told >= PA_QUEUE)
                    kv_wait(unit_free + 8u * slot, (uint32_t)(told / PA_QUEUE - 1) & 1u, dead);
                if (gone_all())
                    break;
                if (elect_one())
                    pa_ask(smem_u32(&s_answer), answered);
                __syncwarp();
                ++asked;
                kv_wait(answered, (uint32_t)(asked - 1) & 1u, dead);
                const int number = pa_answer(smem_u32(&s_answer));
                fence_proxy_async();                       // (the next answer comes to the same place)
                more = number >= 0;
                if (!more || !walk.find(number ^ p.swap, u))
                    u.na = 0;
                if (!more || u.na > 0) {
                    if (lane == 0) {
                        const uint32_t to = smem_u32(&s_unit[slot]);
                        sts128(to, (uint32_t)u.start, (uint32_t)u.len, (uint32_t)u.first, (uint32_t)u.head);
                        sts128(to + 16u, (uint32_t)u.na, (uint32_t)u.nb, 0u, 0u);
                        mbar_arrive(unit_full + 8u * slot);
                    }
                    ++told;
                }
                __syncwarp();
            }
            if (now.na > 0) {
                // values that are not finite in tiles of V that the mask cuts
                const int n = now.nb > 0 ? now.nb : now.na, cut = n - (now.first + 1) / PA_KEYS;
#pragma unroll 1
                for (int t = 0; t < cut && !gone_all(); ++t) {
                    const uint32_t stage = (at + 2u * (uint32_t)t + 1u) & (NS - 1), v = sm + L::RING + stage * L::TILE;
                    kv_wait(v_raw + 8u * stage, (uses >> stage) & 1u, dead);
                    uses ^= 1u << stage;
                    uint32_t zero[2] = {0u, 0u};
#pragma unroll 8
                    for (uint32_t c = (uint32_t)lane * 16u; c < L::TILE; c += 512u) {
                        const uint4 e = lds128(v + c);
                        zero[0] = pa_fma_bf16(e.x, zero[0]);
                        zero[1] = pa_fma_bf16(e.y, zero[1]);
                        zero[0] = pa_fma_bf16(e.z, zero[0]);
                        zero[1] = pa_fma_bf16(e.w, zero[1]);
                    }
                    const bool any = __any_sync(0xffffffffu, ((zero[0] | zero[1]) & 0x7fff7fffu) != 0u);
                    if (lane == 0) {
                        *(volatile int *)&s_bad[stage] = any;
                        mbar_arrive(kv_full + 8u * stage);
                    }
                    __syncwarp();
                }
                at += 2u * (uint32_t)n;
            }
            now = u;
        }
        if (gone_all() && asked > 0)
            mbar_wait(answered, (uint32_t)(asked - 1) & 1u, p.err);
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (*dead.flag != 0 && (warp == PA_MMA || (APART && warp == PA_ADD)))
        kv_mma_drain(drained + (warp == PA_ADD ? 8u : 0u), dead);
    __syncthreads();
    if (warp == PA_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(TM_COLS) : "memory");
    }
}

template <int D>
static q4_status pa_launch(const PromptArgs &a, int64_t most_units, cudaStream_t st, bool pdl)
{
    CUtensorMap q, k, v, out;
    const uint64_t n = (uint64_t)a.tokens;
    q4_status s = tma_heads(q, a.q, D, a.q_heads, n, a.q_stride, a.group, a.tile_tokens);
    if (s == Q4_OK)
        s = tma_heads(k, a.k, D, a.kv_heads, n, a.k_stride, 1, PA_KEYS);
    if (s == Q4_OK)
        s = tma_heads(v, a.v, D, a.kv_heads, n, a.v_stride, 1, PA_KEYS);
    // (without boxes of whole tokens in 32 rows there are no stores through this map)
    if (s == Q4_OK)
        s = tma_heads(out, a.out, D, a.q_heads, n, (int64_t)a.q_heads * D, a.box_tokens ? a.group : 1, a.box_tokens ? a.box_tokens : 1);
    if (s != Q4_OK)
        return s;
    const size_t smem = PaSmem<D>::TOTAL + 1024;
    cudaError_t e = cudaFuncSetAttribute(prompt_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaFuncSetAttribute(prompt_attention_kernel)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)most_units);
    cfg.blockDim = dim3(PA_WARPS * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, prompt_attention_kernel<D>, q, k, v, out, a);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "launch of prompt_attention_kernel");
}

static std::atomic<int> g_swap{0};

void prompt_set_swap(int ctas) { g_swap.store(ctas); }

q4_status launch_prompt_attention(PromptArgs a, int head_dim, cudaStream_t st, bool pdl)
{
    a.group = a.q_heads / a.kv_heads;
    a.tile_tokens = PA_ROWS / a.group;
    a.err = device_error_flags();
    if (!a.err)                                            // (a wait that runs out writes there)
        return fail(Q4_ERR_CUDA, "the device error word was not found");
    a.swap = g_swap.load();
    a.box_tokens = 32 % a.group == 0 ? 32 / a.group : 0;
    // at most one part-filled pair of tiles a sequence
    int64_t units = ((int64_t)a.tokens / (2 * a.tile_tokens) + a.batch) * a.kv_heads;
    if (a.swap)
        units = (units + 2 * a.swap - 1) / (2 * a.swap) * (2 * a.swap);
    return head_dim == 64 ? pa_launch<64>(a, units, st, pdl) : pa_launch<128>(a, units, st, pdl);
}

}  // namespace q4
