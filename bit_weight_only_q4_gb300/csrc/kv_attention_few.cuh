// Attention over the quantised paged cache for at most 16 query rows per key head (a
// decode step).  Mathematics, work list and the joining of pieces: kv_attention.cuh.
//
// Tokens are the MMA's M dimension and query rows its N = 16:
//     S^T [128 x 16] = K [128 x D] q'^T       O^T [D x 16] += V^T [D x 128] P^T
// so a few rows cost the tensor cores little, each token is one thread's TMEM lane and
// its scales are that thread's scalars, and no row needs a reduction over tokens until
// its reference has to move.  K goes dequantised into tensor memory (A operand), V into
// shared memory (A operand, token rows as they lie: M-major), P^T into shared memory
// (B operand, a token's 16 rows together: N-major).  Of the 16 columns only the first NR
// = 4, 8 or 16, the least that holds the rows, are ever computed.
//
// One CTA per SM, 24 warps: one copies blocks, two issue the MMAs, one loads queries;
// four decode K, four V (a thread a token); two groups of four take the tiles' softmax in turn, each with
// references, sums and an accumulator of its own; four put the two together at the end of
// a unit and store, while the others are at the next one.  A tile's MMAs take some 660
// cycles (D = 128), its decoding and softmax some 2,500 warp instructions.
//
// What bounds it (times in chains of 20 calls of a graph).  int8: HBM on long contexts (eight of
// 131,072 tokens, 8 heads of 128, 4 query heads each: 342 us, 6.5 TB/s).  int4: the decoding
// warps, whose instructions issue one in some four cycles beside the other roles' (the same
// in int4: 312 us, 3.7 TB/s; 3,650 warp instructions a tile use 43 to 49% of the issue slots).
// Heads of 64 in pages of 16 tokens: the starting of copies (308 us; 8 copies a tile).  Short
// contexts: the chain of a unit (queries, first references, sums, results), 3.4 us for one
// tile, partly hidden behind the next unit's (48 streams of 37 to 4,096 tokens: 57 us).
// Tried and left: 32 warps, with K and V decoded by two groups each, gained 10 to 20% on
// units of two to four tiles and lost 14% on long ones to spills (64 registers a thread).
#pragma once

#include "kv_attention.cuh"

namespace q4 {

constexpr int KF_N = 16;
constexpr int KF_COPY = 0, KF_MMA_S = 1, KF_Q = 2, KF_MMA_O = 3, KF_K = 4, KF_V = 8, KF_S = 12, KF_E = 20,
              KF_WARPS = 24;
constexpr int KF_ROW_SLOTS = 8;                    // units whose rows are described at a time

struct KfRows {
    int lim[KF_N];               // tokens that each row sees
    float f[KF_N];               // scale * log2 e over the row's power of two
    float qsum[KF_N];            // sum of q' times f (int4)
    int least;                   // fewest tokens that a row sees
    int pad[3];
};

// A softmax group's sums of one unit.
struct KfSums {
    float l[4][KF_N], off[4][KF_N];                // of each warp
    float m[KF_N];
    int any;
    int pad[3];
};

// What a row's results need: o = ca o_0 + cb o_1 + off, plus cp times the prefix's, goes to
// `at` (elements of the output, of the pieces or of the prefix's results).
struct __align__(16) KfResult {
    float ca, cb, off, cp;
    int64_t at, pad;
};

// Shared memory: [raw ring][V: 2][q: 2][P: 2][token scales: 4]
struct KfSmem {
    uint32_t v, q, p, info, total;
};

template <int FMT, int D>
__host__ __device__ inline KfSmem kf_smem(int stages)
{
    KfSmem s = {};
    uint32_t at = (uint32_t)stages * KT_BLOCKS * KvLayout<FMT, D>::BLOCK;
    at = (at + 1023u) & ~1023u;
    s.v = at, at += 2u * KT_TOKENS * D * 2;
    s.q = at, at += 2u * KF_N * D * 2;
    s.p = at, at += 2u * KF_N * KT_TOKENS * 2;
    s.info = at, at += 4u * KT_TOKENS * 16;
    s.total = at;
    return s;
}

// NR fp32 columns of the warp's lanes (after a wait).
template <int NR>
__device__ __forceinline__ void kf_tmem_ld(uint32_t addr, uint32_t (&v)[NR])
{
    if constexpr (NR == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
    else if constexpr (NR == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "r"(addr));
    else
        tmem_ld16_async(addr, v);
    tmem_wait_ld();
}

template <int NR>
__device__ __forceinline__ void kf_tmem_st(uint32_t addr, const uint32_t (&v)[NR])
{
    if constexpr (NR == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};"
                     ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
    else if constexpr (NR == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    else
        tmem_st16(addr, v);
    tmem_wait_st();
}

template <int FMT, int D, int NR>
__global__ void __launch_bounds__(KF_WARPS * 32, 1) kv_few_rows_kernel(const KvTileParams p)
{
    using L = KvLayout<FMT, D>;
    constexpr uint32_t RAW = KT_BLOCKS * L::BLOCK;
    constexpr uint32_t V_BYTES = KT_TOKENS * D * 2;
    constexpr uint32_t Q_BYTES = KF_N * D * 2;
    constexpr uint32_t P_BYTES = KF_N * KT_TOKENS * 2;
    // tensor memory: two K tiles (D / 2 columns), two S tiles (16), O of two units and groups (16)
    constexpr uint32_t TM_S = D, TM_O = D + 2 * KF_N, TM_COLS = 256;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ uint64_t s_bar[2 * KT_MAX_STAGES + 24 + KT_UNITS];
    __shared__ KvUnit s_unit[KT_UNITS];
    __shared__ __align__(16) KfRows s_rows[KF_ROW_SLOTS];
    __shared__ __align__(16) KfSums s_sums[2][2];          // [unit][group]
    __shared__ __align__(16) float s_nm[2][2][KF_N];       // minus the references: [group][by turns]
    __shared__ __align__(16) float s_zero[KF_N];
    __shared__ float s_red[2][4][KF_N], s_c[2][KF_N];
    __shared__ KfResult s_result[2][KF_N];
    __shared__ uint32_t s_tmem, s_valid[KT_MAX_STAGES], s_vmask[4];
    __shared__ int s_last, s_dead, s_counted;
    const int NS = p.stages;
    const KfSmem off = kf_smem<FMT, D>(NS);
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sm = smem_u32(smem);
    float4 *s_info = reinterpret_cast<float4 *>(smem + off.info);      // [4][128], see kv_scales

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t raw_full = smem_u32(s_bar), raw_empty = raw_full + 8u * KT_MAX_STAGES;
    const uint32_t k_full = raw_empty + 8u * KT_MAX_STAGES, s_full = k_full + 16, s_free = k_full + 32,
                   p_full = k_full + 48, v_full = k_full + 64, pv_done = k_full + 80, q_full = k_full + 96,
                   q_empty = k_full + 112, o_full = k_full + 128, o_empty = k_full + 144, sums_full = k_full + 160,
                   drained = k_full + 176, unit_full = k_full + 192;
    if (warp == KF_COPY) {
        kv_init_bars(raw_full, NS, 1);
        kv_init_bars(raw_empty, NS, 8);                    // K and V warps
        kv_init_bars(k_full, 2, 4);
        kv_init_bars(s_full, 2, 1);                        // commit: S is there, K has been read
        kv_init_bars(s_free, 2, 4);
        kv_init_bars(p_full, 2, 4);
        kv_init_bars(v_full, 2, 4);
        kv_init_bars(pv_done, 2, 1);                       // commit: P and V have been read, O is there
        kv_init_bars(q_full, 2, 1);
        kv_init_bars(q_empty, 2, 1);                       // commit after a unit's last S
        kv_init_bars(o_full, 2, 1);                        // commit after a unit's last O
        kv_init_bars(o_empty, 2, 4);
        kv_init_bars(sums_full, 2, 8);
        kv_init_bars(drained, 2, 1);                       // MMAs of a CTA that has given up
        kv_init_bars(unit_full, KT_UNITS, 1);
        if (lane == 0)
            s_dead = s_counted = 0;
        if (lane < KF_N)
            s_zero[lane] = 0.f;
        mbar_init_fence();
    } else if (warp == KF_MMA_S) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&s_tmem)), "n"(TM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (warp >= KF_S && warp < KF_E) {              // the rows of P that no one writes
        for (uint32_t x = (uint32_t)(tid - KF_S * 32) * 16u; x < 2u * P_BYTES; x += 8u * 32u * 16u)
            sts128(sm + off.p + x, 0u, 0u, 0u, 0u);
        fence_proxy_async();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    pdl_wait();
    const KvShare sh = kv_share<KF_N>(p);
    const KvDead dead = {p.err, &s_dead, smem_u32(&s_dead)};
    auto gone = [&]() { return *dead.flag != 0; };
    // The warps that issue MMAs branch on values that are known to be the warp's, so that
    // descriptors can be kept in uniform registers.
    auto gone_all = [&]() { return __any_sync(0xffffffffu, *dead.flag != 0); };
    const int tiles = __shfl_sync(0xffffffffu, sh.tiles, 0);
    // unit u of this CTA, once it has been described
    auto unit_wait = [&](int u) { kv_wait(unit_full + 8u * (u & (KT_UNITS - 1)), (u / KT_UNITS) & 1, dead); };

    if (warp == KF_COPY) {
        kv_copy_warp<FMT, D, KF_N>(p, sh, s_unit, unit_full, sm, s_valid, raw_full, raw_empty, dead);
    } else if (warp == KF_MMA_S) {
        // -------------------------------------------------- MMAs: S^T = K q'^T
        constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(KF_N >> 3) << 17) | (8u << 24);    // f16, f32 sums, M = 128
        int u = -1, left = 0;
#pragma unroll 1
        for (int i = 0; i < tiles && !gone_all(); ++i) {
            if (left == 0) {
                ++u;
                unit_wait(u);
                const KvUnit &un = s_unit[u & (KT_UNITS - 1)];
                left = __shfl_sync(0xffffffffu, un.k1 - un.k0, 0);
                kv_wait(q_full + 8u * (u & 1), (u >> 1) & 1, dead);
            }
            --left;
            kv_wait(k_full + 8u * (i & 1), (i >> 1) & 1, dead);
            if (i >= 2)
                kv_wait(s_free + 8u * (i & 1), ((i >> 1) - 1) & 1, dead);
            tc_fence_after();
            const uint64_t bd = smem_desc_sw128(sm + off.q + (u & 1) * Q_BYTES);
            const uint32_t blo = (uint32_t)bd, bhi = (uint32_t)(bd >> 32);
            const uint32_t a = tmem + (uint32_t)(i & 1) * (D / 2);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)        // 64-column sub-tiles of q: 16 x 128 bytes
                    mma_f16_tmem_a(tmem + TM_S + (uint32_t)(i & 1) * KF_N, a + 8u * kk,
                                   blo + (uint32_t)(kk >> 2) * (KF_N * 128 >> 4) + 2u * (kk & 3), bhi, idesc,
                                   kk > 0 ? 1u : 0u);
                mma_commit(s_full + 8u * (i & 1));
                if (left == 0)
                    mma_commit(q_empty + 8u * (u & 1));
            }
            __syncwarp();
        }
    } else if (warp == KF_MMA_O) {
        // ------------------------------------------------ MMAs: O^T += V^T P^T
        // A is M-major: 64-column halves 16 KB apart, groups of 8 tokens 1 KB apart (D = 64 has
        // one half; lanes 64 .. 127 of O^T then repeat lanes 0 .. 63).  B is N-major without
        // swizzle: 16 bytes a token, its rows 8 .. 15 2 KB behind.
        constexpr uint32_t idesc = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(KF_N >> 3) << 17) | (8u << 24);
        constexpr uint32_t v_lbo = D == 128 ? KT_TOKENS * 128 >> 4 : 0u;
        int u = -1, left = 0;
        uint32_t begun = 0u;                               // groups that have begun the unit
#pragma unroll 1
        for (int i = 0; i < tiles && !gone_all(); ++i) {
            const int g = i & 1;
            if (left == 0) {
                ++u;
                unit_wait(u);
                const KvUnit &un = s_unit[u & (KT_UNITS - 1)];
                left = __shfl_sync(0xffffffffu, un.k1 - un.k0, 0);
                begun = 0u;
                if (u >= 2)                                // its accumulators have been read
                    kv_wait(o_empty + 8u * (u & 1), ((u >> 1) - 1) & 1, dead);
            }
            --left;
            kv_wait(v_full + 8u * g, (i >> 1) & 1, dead);
            kv_wait(p_full + 8u * g, (i >> 1) & 1, dead);
            tc_fence_after();
            const uint32_t b_at = sm + off.p + (uint32_t)g * P_BYTES;
            const uint32_t blo = ((b_at & 0x3FFFFu) >> 4) | (8u << 16), bhi = (2048u >> 4) | (1u << 14);
            const uint64_t ad = (smem_desc_sw128(sm + off.v + (uint32_t)g * V_BYTES) & ~((uint64_t)0x3fff << 16)) |
                                ((uint64_t)v_lbo << 16);
            const uint32_t alo = (uint32_t)ad, ahi = (uint32_t)(ad >> 32);
            const uint32_t more = (begun >> g) & 1u;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < KT_TOKENS / 16; ++kk)        // 16 tokens: two groups of 8
                    mma_f16_2(tmem + TM_O + (uint32_t)((u & 1) * 2 + g) * KF_N, alo + (uint32_t)kk * (2048 >> 4), ahi,
                              blo + (uint32_t)kk * (256 >> 4), bhi, idesc, kk > 0 ? 1u : more);
                mma_commit(pv_done + 8u * g);
                if (left == 0)
                    mma_commit(o_full + 8u * (u & 1));
            }
            __syncwarp();
            begun |= 1u << g;
        }
    } else if (warp == KF_Q) {
        // ----------------------------------------- q: prescaled fp16, row data
        // (of the first NR rows: a column of S^T or O^T takes nothing from another one's q)
        int done = 0;
#pragma unroll 1
        for (int u = 0; done < sh.tiles; ++u) {
            unit_wait(u);
            if (u >= 2)
                kv_wait(q_empty + 8u * (u & 1), ((u >> 1) - 1) & 1, dead);
            if (gone())
                break;
            const KvUnit un = s_unit[u & (KT_UNITS - 1)];
            done += un.k1 - un.k0;
            KfRows &rows = s_rows[u & (KF_ROW_SLOTS - 1)];
            const int row0 = un.rt * KF_N;
            const int nrows = p.rows - row0 < KF_N ? p.rows - row0 : KF_N;
            const int grow0 = (p.prefix_len > 0 ? 0 : un.b * p.rows) + row0;      // among all rows
            constexpr int LPR = D / 8;                     // lanes of a row, 8 columns each
            constexpr int RPP = 32 / LPR;                  // rows of a step
            const int sub = lane % LPR;
            uint4 v[NR / RPP];
#pragma unroll
            for (int j = 0; j < NR / RPP; ++j) {
                const int n = lane / LPR + j * RPP;
                v[j] = n < nrows ? __ldg(reinterpret_cast<const uint4 *>(kv_q_row(p, grow0 + n, un.h, D)) + sub)
                                 : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int j = 0; j < NR / RPP; ++j) {
                const int n = lane / LPR + j * RPP;
                const uint32_t e[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                uint32_t top = 0u;                         // largest finite |q| of the row
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t lo = e[x] & 0x7fffu, hi = (e[x] >> 16) & 0x7fffu;
                    top = lo < 0x7f80u && lo > top ? lo : top;
                    top = hi < 0x7f80u && hi > top ? hi : top;
                }
#pragma unroll
                for (int y = LPR / 2; y >= 1; y >>= 1) {
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, top, y);
                    top = other > top ? other : top;
                }
                int ex = 141 - (int)(top >> 7);            // the largest goes to [2^14, 2^15)
                ex = ex > 126 ? 126 : ex;
                const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
                const float f = p.scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23);
                if (sub == 0)
                    rows.f[n] = f;
                float x[8], sum = 0.f;
                uint32_t o[4];
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    x[y] = ((y & 1) ? __uint_as_float(e[y / 2] & 0xffff0000u) : bf16_bits_to_f32(e[y / 2] & 0xffffu)) * up;
                    sum += x[y];
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const __half2 h = __floats2half2_rn(x[kv_column<L::I8>(2 * y)], x[kv_column<L::I8>(2 * y + 1)]);
                    o[y] = *reinterpret_cast<const uint32_t *>(&h);
                }
                sts128(sm + off.q + (uint32_t)(u & 1) * Q_BYTES + (uint32_t)(sub >> 3) * (KF_N * 128u) +
                           (uint32_t)n * 128u + (((uint32_t)sub ^ (uint32_t)n) & 7u) * 16u,
                       o[0], o[1], o[2], o[3]);
                if constexpr (!L::I8) {
#pragma unroll
                    for (int y = LPR / 2; y >= 1; y >>= 1)
                        sum += __shfl_xor_sync(0xffffffffu, sum, y);
                    if (sub == 0)
                        rows.qsum[n] = sum * f;
                }
            }
            int least = 0x7fffffff;
            if (lane < NR) {                               // rows that fill the tile up: no limit, never stored
                least = lane < nrows ? kv_row_limit(p, grow0 + lane, un.len) : 0x7fffffff;
                rows.lim[lane] = least;
            }
            least = __reduce_min_sync(0xffffffffu, least);
            if (lane == 0)
                rows.least = least;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full + 8u * (u & 1));
        }
    } else if (warp < KF_V) {
        // ------------------------------------------- K: codes to tensor memory
        const int tok = (warp & 3) * 32 + lane;            // TMEM lane
        const uint32_t t_lane = (uint32_t)((warp & 3) * 32) << 16;
        const int r = tok & (KV_BLOCK - 1);
        const KvRowAt<FMT, D> from(tok);
        int k = 0, k1 = 0, ntok = 0, u = 0, s = 0;
        uint32_t round = 0u;                               // parity of the ring's round
#pragma unroll 1
        for (int i = 0; i < sh.tiles && !gone(); ++i, ++k) {
            if (k == k1) {
                unit_wait(u);
                const KvUnit &un = s_unit[u & (KT_UNITS - 1)];
                k = un.k0, k1 = un.k1, ntok = un.ntok;
                ++u;
            }
            kv_wait(raw_full + 8u * s, round, dead);
            if (i >= 2)
                kv_wait(s_full + 8u * (i & 1), ((i >> 1) - 1) & 1, dead);
            tc_fence_after();
            const uint32_t raw = sm + (uint32_t)s * RAW;
            // blocks of the tile that are there and hold tokens; bit 8: all of them do, wholly
            uint32_t mask = s_valid[s];
            if (mask == 0xffu && (k + 1) * KT_TOKENS <= ntok)
                mask |= 0x100u;
            const bool here = ((mask >> (tok / KV_BLOCK)) & 1u) && k * KT_TOKENS + tok < ntok;
            s_info[(i & 3) * KT_TOKENS + tok] = here ? kv_scales<FMT, D>(raw + (uint32_t)(tok / KV_BLOCK) * L::BLOCK, r)
                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
            if (warp == KF_K && lane == 0)
                s_vmask[i & 3] = mask;
            const uint32_t src = raw + from.base, dst = tmem + t_lane + (uint32_t)(i & 1) * (D / 2);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {             // 32 columns: 16 packed
                uint32_t v[4][4];
                if constexpr (L::I8) {
                    const uint4 a = lds128(src + from.piece[2 * j]), b = lds128(src + from.piece[2 * j + 1]);
                    kv_decode8<true>(a.x, a.y, v[0]);
                    kv_decode8<true>(a.z, a.w, v[1]);
                    kv_decode8<true>(b.x, b.y, v[2]);
                    kv_decode8<true>(b.z, b.w, v[3]);
                } else {
                    const uint4 a = lds128(src + from.piece[j]);
                    kv_decode8<false>(a.x, 0u, v[0]);
                    kv_decode8<false>(a.y, 0u, v[1]);
                    kv_decode8<false>(a.z, 0u, v[2]);
                    kv_decode8<false>(a.w, 0u, v[3]);
                }
                tmem_st16(dst + 16u * j, reinterpret_cast<const uint32_t(&)[16]>(v));
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(k_full + 8u * (i & 1));
                mbar_arrive(raw_empty + 8u * s);
            }
            if (++s == NS)
                s = 0, round ^= 1u;
        }
    } else if (warp < KF_S) {
        // ------------------------------------------- V: fp16 to shared memory
        const int tok = (warp & 3) * 32 + lane;
        const KvRowAt<FMT, D> from(tok);
        const KvRowTo to(tok);
        int s = 0;
        uint32_t round = 0u;
#pragma unroll 1
        for (int i = 0; i < sh.tiles && !gone(); ++i) {
            kv_wait(raw_full + 8u * s, round, dead);
            if (i >= 2)
                kv_wait(pv_done + 8u * (i & 1), ((i >> 1) - 1) & 1, dead);
            kv_row_to_tile<FMT, D>(sm + (uint32_t)s * RAW + L::V_CODES, from, sm + off.v + (uint32_t)(i & 1) * V_BYTES, to);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(v_full + 8u * (i & 1));
                mbar_arrive(raw_empty + 8u * s);
            }
            if (++s == NS)
                s = 0, round ^= 1u;
        }
    } else if (warp < KF_E) {
        // --------------------------------------------------- softmax of a tile
        const int grp = (warp - KF_S) >> 2;                // tiles grp, grp + 2, ...
        const int gw = (warp - KF_S) & 3;
        const int gtid = gw * 32 + lane;
        const int quad = warp & 3;
        const int tok = quad * 32 + lane;                  // TMEM lane
        const uint32_t t_lane = (uint32_t)(quad * 32) << 16;
        const int bar_id = 1 + grp;
        const uint32_t p_dst = sm + off.p + (uint32_t)grp * P_BYTES + (uint32_t)tok * 16u;
        const uint32_t s_at = tmem + t_lane + TM_S + (uint32_t)grp * KF_N;
        const uint32_t nm_at = smem_u32(s_nm[grp]), zero_at = smem_u32(s_zero);
        int nmb = 0;                                       // current half of s_nm
        bool leave = false;                                // a wait has given up: agreed on by vote
        int i = 0;                                         // first tile of the unit
#pragma unroll 1
        for (int u = 0; i < sh.tiles && !leave; ++u) {
            unit_wait(u);
            if (bar_or(bar_id, 128, gone()))               // leave together
                break;
            const KvUnit &un = s_unit[u & (KT_UNITS - 1)];
            const int ntok = un.ntok, k0 = un.k0 - i;
            const int end = i + un.k1 - un.k0;
            const KfRows &rows = s_rows[u & (KF_ROW_SLOTS - 1)];
            f32x2 l2[NR / 2], off2[L::I8 ? 1 : NR / 2];
#pragma unroll
            for (int j = 0; j < NR / 2; ++j)
                l2[j] = 0ull;
#pragma unroll
            for (int j = 0; j < (L::I8 ? 1 : NR / 2); ++j)
                off2[j] = 0ull;
            bool first = true;
#pragma unroll 1
            for (int it = i + ((i ^ grp) & 1); it < end && !leave; it += 2) {
                kv_wait(s_full + 8u * grp, (it >> 1) & 1, dead);
                tc_fence_after();
                const float4 info = s_info[(it & 3) * KT_TOKENS + tok];
                const uint32_t mask = s_vmask[it & 3];
                const bool masked = !(mask & 0x100u) || (k0 + it + 1) * KT_TOKENS > rows.least;
                int pos = (k0 + it) * KT_TOKENS + tok;
                if (masked && (pos >= ntok || !((mask >> (tok / KV_BLOCK)) & 1u)))
                    pos = 0x7fffffff;
                const f32x2 ks2 = pack2(info.x, info.x), vs2 = pack2(info.z, info.z);
                // Products over the references as they are (what = 0).  If one reaches 2^15 (or, for
                // a V scale of 0, its p KT_P_TOP), or the unit begins, the group goes round with scores over zero (1), from which the new
                // references are taken, and then over those (2).
                f32x2 x2[NR / 2];
                uint32_t h[NR / 2];
#pragma unroll 1
                for (int what = first ? 1 : 0; what < 3; ++what) {
                    uint32_t acc[NR];
                    kf_tmem_ld<NR>(s_at, acc);
                    const uint32_t nm = what == 1 ? zero_at : nm_at + (uint32_t)nmb * (KF_N * 4);
#pragma unroll
                    for (int j = 0; j < NR / 4; ++j) {
                        f32x2 na, nb, fa, fb;
                        lds_f32x4(nm + 16u * j, na, nb);
                        lds_f32x4(smem_u32(rows.f) + 16u * j, fa, fb);
                        if constexpr (!L::I8) {
                            f32x2 qa, qb;
                            lds_f32x4(smem_u32(rows.qsum) + 16u * j, qa, qb);
                            na = fma2(pack2(info.y, info.y), qa, na);
                            nb = fma2(pack2(info.y, info.y), qb, nb);
                        }
                        x2[2 * j] = fma2(pack2(__uint_as_float(acc[4 * j]), __uint_as_float(acc[4 * j + 1])), mul2(ks2, fa), na);
                        x2[2 * j + 1] = fma2(pack2(__uint_as_float(acc[4 * j + 2]), __uint_as_float(acc[4 * j + 3])), mul2(ks2, fb), nb);
                    }
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < NR / 2; ++j) {
                            float a, b;
                            unpack2(x2[j], a, b);
                            a = pos >= rows.lim[2 * j] ? -INFINITY : a;
                            b = pos >= rows.lim[2 * j + 1] ? -INFINITY : b;
                            x2[j] = pack2(a, b);
                        }
                    }
                    if (what != 1) {
                        uint32_t high = 0u;
#pragma unroll
                        for (int j = 0; j < NR / 2; ++j) {
                            float a, b;
                            unpack2(x2[j], a, b);
                            x2[j] = pack2(ex2(a), ex2(b));
                            unpack2(mul2(x2[j], vs2), a, b);
                            const __half2 hh = __floats2half2_rn(a, b);
                            h[j] = *reinterpret_cast<const uint32_t *>(&hh);
                            high = __vmaxu2(high, h[j]);
                        }
                        if (info.z == 0.f)
#pragma unroll
                            for (int j = 0; j < NR / 2; ++j) {
                                float a, b;
                                unpack2(x2[j], a, b);
                                high = fmaxf(a, b) >= KT_P_TOP ? 0x7800u : high;
                            }
                        if (what == 0 &&
                            !bar_or(bar_id, 128, (high & 0xffffu) >= 0x7800u || high >= 0x78000000u || gone()))
                            break;
                        continue;
                    }
                    // Move the references; rescale what has been summed.
                    {
                        float z[NR];
                        const float level = kv_scale_level(fabsf(info.z));
#pragma unroll
                        for (int j = 0; j < NR / 2; ++j)
                            unpack2(add2(x2[j], pack2(level, level)), z[2 * j], z[2 * j + 1]);
                        int idx;
                        const float top = warp_max_transpose<NR>(z, lane, idx);
                        s_red[grp][gw][idx] = top;         // lanes of one idx hold one value
                    }
                    leave = bar_or(bar_id, 128, gone());
                    if (gtid < NR) {
                        const float old = first ? -INFINITY : -s_nm[grp][nmb][gtid];
                        const float m = fmaxf(fmaxf(fmaxf(s_red[grp][0][gtid], s_red[grp][1][gtid]),
                                                    fmaxf(s_red[grp][2][gtid], s_red[grp][3][gtid])), old);
                        s_nm[grp][nmb ^ 1][gtid] = -m;
                        s_c[grp][gtid] = old == -INFINITY ? 0.f : ex2(old - m);
                    }
                    bar_sync(bar_id, 128);
                    nmb ^= 1;
                    if (!first) {
                        kv_wait(pv_done + 8u * grp, ((it >> 1) - 1) & 1, dead);
                        tc_fence_after();
                        const uint32_t a = tmem + t_lane + TM_O + (uint32_t)((u & 1) * 2 + grp) * KF_N;
                        kf_tmem_ld<NR>(a, acc);
#pragma unroll
                        for (int j = 0; j < NR / 2; ++j) {
                            const f32x2 c2 = pack2(s_c[grp][2 * j], s_c[grp][2 * j + 1]);
                            l2[j] = mul2(l2[j], c2);
                            if constexpr (!L::I8)
                                off2[j] = mul2(off2[j], c2);
                            float x, y;
                            unpack2(mul2(pack2(__uint_as_float(acc[2 * j]), __uint_as_float(acc[2 * j + 1])), c2), x, y);
                            acc[2 * j] = __float_as_uint(x);
                            acc[2 * j + 1] = __float_as_uint(y);
                        }
                        kf_tmem_st<NR>(a, acc);
                    }
                }
                first = false;
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(s_free + 8u * grp);
#pragma unroll
                for (int j = 0; j < NR / 2; ++j) {
                    l2[j] = add2(l2[j], x2[j]);
                    if constexpr (!L::I8)
                        off2[j] = fma2(x2[j], pack2(info.w, info.w), off2[j]);
                }
                if (it >= 2)                               // the group's last P has been read
                    kv_wait(pv_done + 8u * grp, ((it >> 1) - 1) & 1, dead);
                if constexpr (NR == 4)
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(p_dst), "r"(h[0]), "r"(h[1]) : "memory");
#pragma unroll
                for (int j = 0; j < NR / 8; ++j)
                    sts128(p_dst + 2048u * j, h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full + 8u * grp);
            }
            i = end;
            // ---- the group's sums of the unit, for the warps that put them together
            if (u >= 2)
                kv_wait(o_empty + 8u * (u & 1), ((u >> 1) - 1) & 1, dead);
            KfSums &sums = s_sums[u & 1][grp];
            {
                float z[NR];
                int idx;
#pragma unroll
                for (int j = 0; j < NR / 2; ++j)
                    unpack2(l2[j], z[2 * j], z[2 * j + 1]);
                const float x = warp_sum_transpose<NR>(z, lane, idx);
                sums.l[gw][idx] = x;                       // lanes of one idx hold one value
                if constexpr (!L::I8) {
#pragma unroll
                    for (int j = 0; j < NR / 2; ++j)
                        unpack2(off2[j], z[2 * j], z[2 * j + 1]);
                    const float y = warp_sum_transpose<NR>(z, lane, idx);
                    sums.off[gw][idx] = y;
                }
            }
            if (gw == 0 && lane < NR)
                sums.m[lane] = first ? -INFINITY : -s_nm[grp][nmb][lane];
            if (gw == 0 && lane == 0)
                sums.any = !first;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(sums_full + 8u * (u & 1));
        }
    } else {
        // --------------------------------------------- the results of a unit
        const int quad = warp & 3;
        const int tok = quad * 32 + lane;                  // TMEM lane: a column of O^T
        const uint32_t t_lane = (uint32_t)(quad * 32) << 16;
        const int t = (warp - KF_E) * 32 + lane;
        const int d = kv_column<L::I8>(tok);
        int done = 0;
#pragma unroll 1
        for (int u = 0; done < sh.tiles; ++u) {
            unit_wait(u);
            const KvUnit un = s_unit[u & (KT_UNITS - 1)];
            const int row0 = un.rt * KF_N;
            const int nrows = p.rows - row0 < KF_N ? p.rows - row0 : KF_N;
            const int grow0 = (p.prefix_len > 0 ? 0 : un.b * p.rows) + row0;      // among all rows
            const bool whole = un.k0 == 0 && un.k1 == un.n;
            const int64_t pre = (int64_t)un.h * p.all_rows + grow0;        // the rows' place in the prefix's results
            const bool joins = whole && p.prefix_in_o != nullptr;
            kv_wait(sums_full + 8u * (u & 1), (u >> 1) & 1, dead);
            // A thread a row: the groups' sums together, and what is left to do for the row.
            if (t < NR && t < nrows && !gone()) {
                const KfSums &a = s_sums[u & 1][0], &b = s_sums[u & 1][1];
                const float m = fmaxf(a.m[t], b.m[t]);
                KfResult w;
                w.ca = a.m[t] == -INFINITY ? 0.f : ex2(a.m[t] - m);
                w.cb = b.m[t] == -INFINITY ? 0.f : ex2(b.m[t] - m);
                float l = ((a.l[0][t] + a.l[1][t]) + (a.l[2][t] + a.l[3][t])) * w.ca +
                          ((b.l[0][t] + b.l[1][t]) + (b.l[2][t] + b.l[3][t])) * w.cb;
                w.off = L::I8 ? 0.f
                              : ((a.off[0][t] + a.off[1][t]) + (a.off[2][t] + a.off[3][t])) * w.ca +
                                    ((b.off[0][t] + b.off[1][t]) + (b.off[2][t] + b.off[3][t])) * w.cb;
                w.cp = 0.f;
                const int grow = grow0 + t;
                if (!whole) {
                    const int64_t slot = kv_piece_slot(un) * KF_N + t;
                    *reinterpret_cast<float2 *>(p.piece_ml + slot * 2) = make_float2(m, l);
                    w.at = slot * D;
                } else if (p.prefix_len > 0) {             // a piece for the launch over the sequences' own tokens
                    *reinterpret_cast<float2 *>(p.prefix_out_ml + (pre + t) * 2) = make_float2(m, l);
                    w.at = (pre + t) * D;
                } else {
                    float own = 1.f;
                    if (joins) {
                        const float2 pml = __ldcg(reinterpret_cast<const float2 *>(p.prefix_in_ml + (pre + t) * 2));
                        const float top = fmaxf(m, pml.x);
                        own = m == -INFINITY ? 0.f : ex2(m - top);
                        w.cp = pml.x == -INFINITY ? 0.f : ex2(pml.x - top);
                        l = l * own + pml.y * w.cp;
                    }
                    // a row that sees nothing has l = 0 and gives zeros
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    own *= inv;
                    w.ca *= own, w.cb *= own, w.off *= own, w.cp *= inv;
                    const int token = p.by_group(grow);
                    w.at = ((int64_t)token * p.cache.heads * p.group + un.h * p.group + grow - token * p.group) * D;
                }
                s_result[u & 1][t] = w;
            }
            kv_wait(o_full + 8u * (u & 1), (u >> 1) & 1, dead);
            if (bar_or(3, 128, gone()))                    // leave together
                break;
            done += un.k1 - un.k0;
            tc_fence_after();
            const bool any0 = s_sums[u & 1][0].any, any1 = s_sums[u & 1][1].any;
            uint32_t v0[NR], v1[NR];
            kf_tmem_ld<NR>(tmem + t_lane + TM_O + (uint32_t)((u & 1) * 2) * KF_N, v0);
            kf_tmem_ld<NR>(tmem + t_lane + TM_O + (uint32_t)((u & 1) * 2 + 1) * KF_N, v1);
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(o_empty + 8u * (u & 1));
            // A thread a column: neighbouring lanes store neighbouring columns of a row.
            float x[NR];
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const KfResult &w = s_result[u & 1][j];
                x[j] = any0 ? fmaf(__uint_as_float(v0[j]), w.ca, w.off) : w.off;
                x[j] = any1 ? fmaf(__uint_as_float(v1[j]), w.cb, x[j]) : x[j];
            }
            if (joins && tok < D) {
                const float *src = p.prefix_in_o + pre * D + d;
                float po[NR];
#pragma unroll
                for (int j = 0; j < NR; ++j)               // (all on their way before the first is used)
                    po[j] = j < nrows ? __ldcg(src + j * D) : 0.f;
#pragma unroll
                for (int j = 0; j < NR; ++j)
                    x[j] = fmaf(po[j], s_result[u & 1][j].cp, x[j]);
            }
            if (tok < D) {
                if (!whole || p.prefix_len > 0) {
                    float *dst = (whole ? p.prefix_out_o : p.piece_o) + d;
#pragma unroll
                    for (int j = 0; j < NR; ++j)
                        if (j < nrows)
                            dst[s_result[u & 1][j].at] = x[j];
                } else {
#pragma unroll
                    for (int j = 0; j < NR; ++j)
                        if (j < nrows)
                            p.out[s_result[u & 1][j].at + d] = f32_to_bf16_bits(x[j]);
                }
            }
            if (!whole)                                    // (with more in flight than one it spills, which costs every role)
                kv_join<D, KF_N, 128, 1>(p, sh, un, nrows, grow0, &s_last, &s_counted, t, 3);
        }
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (gone()) {                // (here, not in the warps' roles: there it cost the MMA loops their uniform registers)
        if (warp == KF_COPY)
            kv_arrive_failed<KF_N>(p, s_counted);
        else if (warp == KF_MMA_S || warp == KF_MMA_O)
            kv_mma_drain(drained + (warp == KF_MMA_O ? 8u : 0u), dead);
        tc_fence_before();
        __syncthreads();
    }
    if (warp == KF_MMA_S) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(TM_COLS) : "memory");
    }
}

template <int FMT, int D>
static KvKernel kf_describe(const DeviceInfo &dev, int rows)
{
    KvKernel k = {};
    // The softmax's work goes by the columns that are computed.  With all 16 of them for 1, 4 and 8
    // rows (us, against the least that holds the rows): one stream of 2,047 tokens 15.8 (11.8),
    // 48 streams 95 (57), eight of 131,071 200 (162).
    k.fn = rows <= 4   ? reinterpret_cast<const void *>(&kv_few_rows_kernel<FMT, D, 4>)
           : rows <= 8 ? reinterpret_cast<const void *>(&kv_few_rows_kernel<FMT, D, 8>)
                       : reinterpret_cast<const void *>(&kv_few_rows_kernel<FMT, D, 16>);
    k.tile = KF_N;
    k.threads = KF_WARPS * 32;
    // 1024: alignment; 8192: static arrays
    const size_t budget = dev.smem_optin - 1024 - 8192;
    for (k.stages = KT_MAX_STAGES; k.stages > 1 && kf_smem<FMT, D>(k.stages).total > budget;)
        --k.stages;
    k.smem = kf_smem<FMT, D>(k.stages).total + 1024;
    return k;
}

}  // namespace q4
