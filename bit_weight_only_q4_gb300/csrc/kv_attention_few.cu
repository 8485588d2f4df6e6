// Attention over the quantised paged cache for at most 16 query rows per key head (a
// decode step).  Mathematics, work list and the joining of pieces: kv_attention.cuh.
//
// Tokens are the MMA's M dimension and query rows its N = 16:
//     S^T [128 x 16] = K [128 x D] q'^T       O^T [D x 16] += V^T [D x 128] P^T
// so a few rows cost the tensor cores little, each token is one thread's TMEM lane and
// its scales are that thread's scalars, and no row needs a reduction over tokens until
// its reference has to move.  K goes dequantised into tensor memory (A operand), V into
// shared memory (A operand, token rows as they lie: M-major), P^T into shared memory.
//
// One CTA per SM, 23 warps: one copies blocks, one issues the MMAs, one loads queries;
// four decode K, four V; two groups of four take the tiles' softmax in turn, each with
// references, sums and an accumulator of its own; four put the two together at the end of
// a unit and store, while the others are at the next one.
#include "kv_attention.cuh"

namespace q4 {

constexpr int KF_N = 16;
constexpr int KF_K = 2, KF_V = 6, KF_S = 10, KF_E = 18, KF_Q = 22, KF_WARPS = 23;
constexpr int KF_ROW_SLOTS = 8;                    // units whose rows are described at a time

struct KfRows {
    int lim[KF_N];               // tokens that each row sees
    float qsum[KF_N];            // sum of q' (int4)
    float f;                     // scale * log2 e over the queries' power of two
    int least;                   // fewest tokens that a row sees
    int pad[2];
};

// A softmax group's sums of one unit.
struct KfSums {
    float l[4][KF_N], off[4][KF_N];                // of each warp
    float m[KF_N];
    int any;
    int pad[3];
};

// Shared memory: [raw ring][V: 2][q: 2][P: 2][o][token scales: 4][lengths]
struct KfSmem {
    uint32_t v, q, p, o, info, len, total;
};

template <int FMT, int D>
__host__ __device__ inline KfSmem kf_smem(int stages, int seqs)
{
    KfSmem s = {};
    uint32_t at = (uint32_t)stages * KT_BLOCKS * KvLayout<FMT, D>::BLOCK;
    at = (at + 1023u) & ~1023u;
    s.v = at, at += 2u * KT_TOKENS * D * 2;
    s.q = at, at += 2u * KF_N * D * 2;
    s.p = at, at += 2u * KF_N * KT_TOKENS * 2;
    s.o = at, at += KF_N * D * 4u;
    s.info = at, at += 4u * KT_TOKENS * 16;
    s.len = at, at += ((uint32_t)seqs * 4u + 15u) & ~15u;
    s.total = at;
    return s;
}

template <int FMT, int D>
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
    __shared__ uint64_t s_bar[2 * KT_MAX_STAGES + 20 + KT_UNITS];
    __shared__ KvUnit s_unit[KT_UNITS];
    __shared__ __align__(16) KfRows s_rows[KF_ROW_SLOTS];
    __shared__ __align__(16) KfSums s_sums[2][2];          // [unit][group]
    __shared__ __align__(16) float s_nm[2][2][KF_N];       // minus the references: [group][by turns]
    __shared__ __align__(16) float s_zero[KF_N], s_e[3][KF_N];
    __shared__ float s_red[2][4][KF_N], s_wred[2][4], s_c[2][KF_N];
    __shared__ float2 s_ml[KF_N];
    __shared__ uint32_t s_tmem, s_valid[KT_MAX_STAGES], s_vmask[4];
    __shared__ int s_last, s_dead;
    const int NS = p.stages;
    const KfSmem off = kf_smem<FMT, D>(NS, p.seqs);
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sm = smem_u32(smem);
    float4 *s_info = reinterpret_cast<float4 *>(smem + off.info);      // [4][128], see kv_scales
    int *s_len = reinterpret_cast<int *>(smem + off.len);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t raw_full = smem_u32(s_bar), raw_empty = raw_full + 8u * KT_MAX_STAGES;
    const uint32_t k_full = raw_empty + 8u * KT_MAX_STAGES, s_full = k_full + 16, p_full = k_full + 32,
                   v_full = k_full + 48, pv_done = k_full + 64, q_full = k_full + 80, q_empty = k_full + 96,
                   o_full = k_full + 112, o_empty = k_full + 128, sums_full = k_full + 144,
                   unit_full = k_full + 160;
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(raw_full + 8u * i, 1);
            mbar_init(raw_empty + 8u * i, 8);              // K and V warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full + 8u * i, 4);
            mbar_init(s_full + 8u * i, 1);                 // commit: S is there, K has been read
            mbar_init(p_full + 8u * i, 4);
            mbar_init(v_full + 8u * i, 4);
            mbar_init(pv_done + 8u * i, 1);                // commit: P and V have been read, O is there
            mbar_init(q_full + 8u * i, 1);
            mbar_init(q_empty + 8u * i, 1);                // commit after a unit's last S
            mbar_init(o_full + 8u * i, 1);                 // commit after a unit's last O
            mbar_init(o_empty + 8u * i, 4);
            mbar_init(sums_full + 8u * i, 8);
        }
        for (int i = 0; i < KT_UNITS; ++i)
            mbar_init(unit_full + 8u * i, 1);
        mbar_init_fence();
    }
    if (tid < KF_N)
        s_zero[tid] = 0.f;
    if (tid == 0)
        s_dead = 0;
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&s_tmem)), "n"(TM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    const KvShare sh = kv_share<KF_N, KF_WARPS>(p, s_len);
    const uint32_t tmem = s_tmem;
    const KvDead dead = {p.err, &s_dead};
    auto gone = [&]() { return *dead.flag != 0; };
    // unit u of this CTA, once it has been described
    auto unit_wait = [&](int u) { kv_wait(unit_full + 8u * (u & (KT_UNITS - 1)), (u / KT_UNITS) & 1, dead); };

    if (warp == 0) {
        kv_copy_warp<FMT, D, KF_N>(p, sh, s_len, s_unit, unit_full, sm, s_valid, raw_full, raw_empty, dead);
    } else if (warp == 1) {
        // --------------------------------------------------------------- MMAs
        constexpr uint32_t idesc1 = (1u << 4) | ((uint32_t)(KF_N >> 3) << 17) | (8u << 24);   // f16, f32 sums, M = 128
        constexpr uint32_t idesc2 = idesc1 | (1u << 15);                                      // A is M-major
        // V^T: 64-column halves 16 KB apart, groups of 8 tokens 1 KB apart (D = 64 has one half;
        // lanes 64 .. 127 of O^T then repeat lanes 0 .. 63)
        constexpr uint32_t v_lbo = D == 128 ? KT_TOKENS * 128 >> 4 : 0u;
        int u1 = -1, left1 = 0;                            // unit of the next S, tiles left in it
        int u2 = -1, left2 = 0;                            // unit of the next O
        uint32_t begun = 0u;                               // groups that have begun u2
        auto begin = [&](int &u, int &left) {
            ++u;
            unit_wait(u);
            const KvUnit &un = s_unit[u & (KT_UNITS - 1)];
            left = un.k1 - un.k0;
        };
        auto mma1 = [&](int i) {                           // S(i) = K q^T
            if (left1 == 0) {
                begin(u1, left1);
                kv_wait(q_full + 8u * (u1 & 1), (u1 >> 1) & 1, dead);
            }
            kv_wait(k_full + 8u * (i & 1), (i >> 1) & 1, dead);
            tc_fence_after();
            --left1;
            const uint64_t bd = smem_desc_sw128(sm + off.q + (u1 & 1) * Q_BYTES);
            const uint32_t blo = (uint32_t)bd, bhi = (uint32_t)(bd >> 32);
            const uint32_t a = tmem + (uint32_t)(i & 1) * (D / 2);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)        // 64-column sub-tiles of q: 16 x 128 bytes
                    mma_f16_tmem_a(tmem + TM_S + (uint32_t)(i & 1) * KF_N, a + 8u * kk,
                                   blo + (uint32_t)(kk >> 2) * (KF_N * 128 >> 4) + 2u * (kk & 3), bhi, idesc1,
                                   kk > 0 ? 1u : 0u);
                mma_commit(s_full + 8u * (i & 1));
                if (left1 == 0)
                    mma_commit(q_empty + 8u * (u1 & 1));
            }
            __syncwarp();
        };
        if (sh.tiles > 0)
            mma1(0);
#pragma unroll 1
        for (int i = 0; i < sh.tiles && !gone(); ++i) {
            const int g = i & 1;
            if (i + 1 < sh.tiles)
                mma1(i + 1);
            if (left2 == 0) {
                begin(u2, left2);
                begun = 0u;
                if (u2 >= 2)                               // its accumulators have been read
                    kv_wait(o_empty + 8u * (u2 & 1), ((u2 >> 1) - 1) & 1, dead);
            }
            kv_wait(v_full + 8u * g, (i >> 1) & 1, dead);
            kv_wait(p_full + 8u * g, (i >> 1) & 1, dead);
            tc_fence_after();
            --left2;
            const uint64_t bd = smem_desc_sw128(sm + off.p + (uint32_t)g * P_BYTES);
            const uint32_t blo = (uint32_t)bd, bhi = (uint32_t)(bd >> 32);
            const uint64_t ad = (smem_desc_sw128(sm + off.v + (uint32_t)g * V_BYTES) & ~((uint64_t)0x3fff << 16)) |
                                ((uint64_t)v_lbo << 16);
            const uint32_t alo = (uint32_t)ad, ahi = (uint32_t)(ad >> 32);
            const uint32_t more = (begun >> g) & 1u;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < KT_TOKENS / 16; ++kk)        // 16 tokens: two groups of 8
                    mma_f16_2(tmem + TM_O + (uint32_t)((u2 & 1) * 2 + g) * KF_N, alo + (uint32_t)kk * (2048 >> 4), ahi,
                              blo + (uint32_t)(kk >> 2) * (KF_N * 128 >> 4) + 2u * (kk & 3), bhi, idesc2,
                              kk > 0 ? 1u : more);
                mma_commit(pv_done + 8u * g);
                if (left2 == 0)
                    mma_commit(o_full + 8u * (u2 & 1));
            }
            __syncwarp();
            begun |= 1u << g;
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
            const uint32_t blk = sm + (uint32_t)s * RAW + (uint32_t)(tok / KV_BLOCK) * L::BLOCK;
            const uint32_t src = sm + (uint32_t)s * RAW + from.base;
            // blocks of the tile that are there and hold tokens; bit 8: all of them do, wholly
            uint32_t mask = s_valid[s];
            if (mask == 0xffu && (k + 1) * KT_TOKENS <= ntok)
                mask |= 0x100u;
            const bool here = ((mask >> (tok / KV_BLOCK)) & 1u) && k * KT_TOKENS + tok < ntok;
            s_info[(i & 3) * KT_TOKENS + tok] = here ? kv_scales<FMT, D>(blk, r) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (warp == KF_K && lane == 0)
                s_vmask[i & 3] = mask;
            const uint32_t dst = tmem + t_lane + (uint32_t)(i & 1) * (D / 2);
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
        const int tok = (warp - KF_V) * 32 + lane;
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
    } else if (warp == KF_Q) {
        // ----------------------------------------- q: prescaled fp16, row data
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
            uint4 v[KF_N / RPP];
#pragma unroll
            for (int j = 0; j < KF_N / RPP; ++j) {
                const int n = lane / LPR + j * RPP;
                v[j] = n < nrows ? __ldg(reinterpret_cast<const uint4 *>(kv_q_row(p, grow0 + n, un.h, D)) + sub)
                                 : make_uint4(0u, 0u, 0u, 0u);
            }
            uint32_t top = 0u;                             // largest finite |q| of the tile
#pragma unroll
            for (int j = 0; j < KF_N / RPP; ++j) {
                const uint32_t e[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t lo = e[x] & 0x7fffu, hi = (e[x] >> 16) & 0x7fffu;
                    top = lo < 0x7f80u && lo > top ? lo : top;
                    top = hi < 0x7f80u && hi > top ? hi : top;
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            int ex = 141 - (int)(top >> 7);                // the largest goes to [2^14, 2^15)
            ex = ex > 126 ? 126 : ex;
            const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
            int least = 0x7fffffff;
#pragma unroll
            for (int j = 0; j < KF_N / RPP; ++j) {
                const int n = lane / LPR + j * RPP;
                const uint32_t e[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
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
                        rows.qsum[n] = sum;
                }
            }
            if (lane < KF_N) {                             // rows that fill the tile up: no limit, never stored
                const int lim = lane < nrows ? kv_row_limit(p, grow0 + lane, s_len[un.b]) : 0x7fffffff;
                rows.lim[lane] = lim;
                least = lim;
            }
            least = __reduce_min_sync(0xffffffffu, least);
            if (lane == 0) {
                rows.f = p.scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23);
                rows.least = least;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full + 8u * (u & 1));
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
        const uint32_t p_dst = sm + off.p + (uint32_t)grp * P_BYTES + (uint32_t)(tok >> 6) * (KF_N * 128u) +
                               (uint32_t)(tok & 7) * 2u;
        const uint32_t ch = (uint32_t)(tok & 63) << 1 & 0x70u;
        int nmb = 0;                                       // current half of s_nm
        bool leave = false;                                // a wait has given up: agreed on by vote
        int i = 0;                                         // first tile of the unit
#pragma unroll 1
        for (int u = 0; i < sh.tiles && !leave; ++u) {
            unit_wait(u);
            const KvUnit &un = s_unit[u & (KT_UNITS - 1)];
            const int ntok = un.ntok, k0 = un.k0;
            const int end = i + un.k1 - k0;
            const KfRows &rows = s_rows[u & (KF_ROW_SLOTS - 1)];
            float l[KF_N], sum_off[L::I8 ? 1 : KF_N];
#pragma unroll
            for (int j = 0; j < KF_N; ++j)
                l[j] = 0.f;
#pragma unroll
            for (int j = 0; j < (L::I8 ? 1 : KF_N); ++j)
                sum_off[j] = 0.f;
            float level = -36.f;                           // E - 6
            bool first = true;
            const int i0 = i + ((i ^ grp) & 1);
#pragma unroll 1
            for (int it = i0; it < end && !leave; it += 2) {
                kv_wait(s_full + 8u * grp, (it >> 1) & 1, dead);
                tc_fence_after();
                const float4 info = s_info[(it & 3) * KT_TOKENS + tok];
                const uint32_t mask = s_vmask[it & 3];
                const int k = k0 + it - i;
                const bool masked = !(mask & 0x100u) || (k + 1) * KT_TOKENS > rows.least;
                int pos = k * KT_TOKENS + tok;
                if (pos >= ntok || !((mask >> (tok / KV_BLOCK)) & 1u))
                    pos = 0x7fffffff;
                const float ks = info.x * rows.f, km = info.y * rows.f;
                // Scores over the references (what = 0).  If one is too large, or none are
                // set, the group goes round again: scores over zero (1), from which the new
                // references are taken, then over those (2).
                float s[KF_N];
#pragma unroll 1
                for (int what = 0; what < 3; ++what) {
                    const float *nms = what == 1 ? s_zero : s_nm[grp][nmb];
                    uint32_t acc[KF_N];
                    tmem_ld16(tmem + t_lane + TM_S + (uint32_t)grp * KF_N, acc);
#pragma unroll
                    for (int j = 0; j < KF_N; j += 4) {
                        const float4 nm = *reinterpret_cast<const float4 *>(nms + j);
                        const float base[4] = {nm.x, nm.y, nm.z, nm.w};
                        if constexpr (L::I8) {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                s[j + x] = fmaf(__uint_as_float(acc[j + x]), ks, base[x]);
                        } else {
                            const float4 qs = *reinterpret_cast<const float4 *>(rows.qsum + j);
                            const float q4[4] = {qs.x, qs.y, qs.z, qs.w};
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                s[j + x] = fmaf(__uint_as_float(acc[j + x]), ks, fmaf(km, q4[x], base[x]));
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < KF_N; j += 4) {
                            const int4 lm = *reinterpret_cast<const int4 *>(rows.lim + j);
                            s[j] = pos >= lm.x ? -INFINITY : s[j];
                            s[j + 1] = pos >= lm.y ? -INFINITY : s[j + 1];
                            s[j + 2] = pos >= lm.z ? -INFINITY : s[j + 2];
                            s[j + 3] = pos >= lm.w ? -INFINITY : s[j + 3];
                        }
                    }
                    if (what == 0) {
                        float top = s[0];
#pragma unroll
                        for (int j = 1; j < KF_N; ++j)
                            top = fmaxf(top, s[j]);
                        if (!bar_or(bar_id, 128, first || top + level > 8.f || kv_scale_level(info.z) > level || gone()))
                            break;
                    } else if (what == 1) {
                        // Move the references; rescale what has been summed.
                        int idx;
                        const float z = warp_max_transpose<KF_N>(s, lane, idx);
                        s_red[grp][gw][idx] = z;           // lanes of one idx hold one value
                        float wm = info.z;
#pragma unroll
                        for (int o = 16; o >= 1; o >>= 1)
                            wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
                        if (lane == 0)
                            s_wred[grp][gw] = gone() ? -1.f : wm;
                        bar_sync(bar_id, 128);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            leave = leave || s_wred[grp][w] < 0.f;
                            wm = fmaxf(wm, s_wred[grp][w]);
                        }
                        level = fmaxf(level, kv_scale_level(wm));
                        if (gtid < KF_N) {
                            const float old = first ? -INFINITY : -s_nm[grp][nmb][gtid];
                            const float m = fmaxf(fmaxf(fmaxf(s_red[grp][0][gtid], s_red[grp][1][gtid]),
                                                        fmaxf(s_red[grp][2][gtid], s_red[grp][3][gtid])) + level, old);
                            s_nm[grp][nmb ^ 1][gtid] = -m;
                            s_c[grp][gtid] = old == -INFINITY ? 0.f : ex2(old - m);
                        }
                        bar_sync(bar_id, 128);
                        nmb ^= 1;
                        if (!first) {
                            kv_wait(pv_done + 8u * grp, ((it >> 1) - 1) & 1, dead);
                            tc_fence_after();
                            const uint32_t a = tmem + t_lane + TM_O + (uint32_t)((u & 1) * 2 + grp) * KF_N;
                            tmem_ld16(a, acc);
#pragma unroll
                            for (int j = 0; j < KF_N; ++j) {
                                const float c = s_c[grp][j];
                                l[j] *= c;
                                if constexpr (!L::I8)
                                    sum_off[j] *= c;
                                acc[j] = __float_as_uint(__uint_as_float(acc[j]) * c);
                            }
                            tmem_st16(a, acc);
                            tmem_wait_st();
                        }
                    }
                }
                first = false;
                if (it >= 2)                               // the group's last P has been read
                    kv_wait(pv_done + 8u * grp, ((it >> 1) - 1) & 1, dead);
                // P^T: row n, tokens in 64-token sub-tiles of 16 x 128 bytes
#pragma unroll
                for (int j = 0; j < KF_N; j += 2) {
                    const float p0 = ex2(s[j]), p1 = ex2(s[j + 1]);
                    l[j] += p0;
                    l[j + 1] += p1;
                    if constexpr (!L::I8) {
                        sum_off[j] = fmaf(p0, info.w, sum_off[j]);
                        sum_off[j + 1] = fmaf(p1, info.w, sum_off[j + 1]);
                    }
                    const __half2 h = __floats2half2_rn(p0 * info.z, p1 * info.z);
                    const uint32_t hb = *reinterpret_cast<const uint32_t *>(&h);
                    sts16(p_dst + j * 128u + (ch ^ ((uint32_t)(j & 7) << 4)), hb);
                    sts16(p_dst + (j + 1) * 128u + (ch ^ ((uint32_t)((j + 1) & 7) << 4)), hb >> 16);
                }
                tc_fence_before();
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
                int idx;
                const float x = warp_sum_transpose<KF_N>(l, lane, idx);
                sums.l[gw][idx] = x;                       // lanes of one idx hold one value
                if constexpr (!L::I8) {
                    const float y = warp_sum_transpose<KF_N>(sum_off, lane, idx);
                    sums.off[gw][idx] = y;
                }
            }
            if (gw == 0 && lane < KF_N)
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
        float *s_o = reinterpret_cast<float *>(smem + off.o);
        int done = 0;
#pragma unroll 1
        for (int u = 0; done < sh.tiles; ++u) {
            unit_wait(u);
            kv_wait(sums_full + 8u * (u & 1), (u >> 1) & 1, dead);
            kv_wait(o_full + 8u * (u & 1), (u >> 1) & 1, dead);
            if (bar_or(3, 128, gone()))              // leave together
                break;
            const KvUnit un = s_unit[u & (KT_UNITS - 1)];
            done += un.k1 - un.k0;
            tc_fence_after();
            if (t < KF_N) {
                const KfSums &a = s_sums[u & 1][0], &b = s_sums[u & 1][1];
                const float m = fmaxf(a.m[t], b.m[t]);
                const float ca = a.m[t] == -INFINITY ? 0.f : ex2(a.m[t] - m);
                const float cb = b.m[t] == -INFINITY ? 0.f : ex2(b.m[t] - m);
                s_ml[t] = make_float2(m, ((a.l[0][t] + a.l[1][t]) + (a.l[2][t] + a.l[3][t])) * ca +
                                             ((b.l[0][t] + b.l[1][t]) + (b.l[2][t] + b.l[3][t])) * cb);
                s_e[0][t] = ca;
                s_e[1][t] = cb;
                s_e[2][t] = L::I8 ? 0.f
                                  : ((a.off[0][t] + a.off[1][t]) + (a.off[2][t] + a.off[3][t])) * ca +
                                        ((b.off[0][t] + b.off[1][t]) + (b.off[2][t] + b.off[3][t])) * cb;
            }
            bar_sync(3, 128);
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
                if (!s_sums[u & 1][g].any)
                    continue;
                uint32_t v[KF_N];
                tmem_ld16(tmem + t_lane + TM_O + (uint32_t)((u & 1) * 2 + g) * KF_N, v);
                const bool add = g == 1 && s_sums[u & 1][0].any;
                if (tok < D) {
#pragma unroll
                    for (int j = 0; j < KF_N; ++j) {
                        float *o = s_o + j * D + d;
                        *o = fmaf(__uint_as_float(v[j]), s_e[g][j], add ? *o : s_e[2][j]);
                    }
                }
            }
            tc_fence_before();
            bar_sync(3, 128);
            if (lane == 0)
                mbar_arrive(o_empty + 8u * (u & 1));
            const int row0 = un.rt * KF_N;
            const int nrows = p.rows - row0 < KF_N ? p.rows - row0 : KF_N;
            const int grow0 = (p.prefix_len > 0 ? 0 : un.b * p.rows) + row0;      // among all rows
            const bool whole = un.k0 == 0 && un.k1 == un.n;
            const int64_t slot = kv_piece_slot(un) * KF_N;
#pragma unroll 1
            for (int item = t; item < nrows * (D / 4); item += 128) {
                const int n = item / (D / 4), c4 = item % (D / 4);
                const float4 o = *reinterpret_cast<const float4 *>(s_o + n * D + c4 * 4);
                if (whole) {
                    kv_store4<D>(p, grow0 + n, un.h, c4, KvRowSum{s_ml[n].x, s_ml[n].y, o});
                    continue;
                }
                *reinterpret_cast<float4 *>(p.piece_o + (slot + n) * D + c4 * 4) = o;
                if (c4 == 0)
                    *reinterpret_cast<float2 *>(p.piece_ml + (slot + n) * 2) = s_ml[n];
            }
            if (!whole)
                kv_join<D, KF_N, 128>(p, sh, un, nrows, grow0, &s_last, t, 3);
            bar_sync(3, 128);                              // s_o, s_ml and s_e may be written again
        }
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(TM_COLS) : "memory");
    }
}

template <int FMT, int D>
static KvKernel kf_describe(const DeviceInfo &dev, int seqs)
{
    KvKernel k = {};
    k.fn = reinterpret_cast<const void *>(&kv_few_rows_kernel<FMT, D>);
    k.tile = KF_N;
    k.threads = KF_WARPS * 32;
    // 1024: alignment; 8192: static arrays and the CTA's reserve
    const size_t budget = dev.smem_optin - 1024 - 8192;
    for (k.stages = KT_MAX_STAGES; k.stages > 1 && kf_smem<FMT, D>(k.stages, seqs).total > budget;)
        --k.stages;
    k.smem = kf_smem<FMT, D>(k.stages, seqs).total + 1024;
    return k;
}

KvKernel kv_few_kernel(const DeviceInfo &dev, int format, int head_dim, int seqs)
{
    if (format == Q4_CACHE_INT8)
        return head_dim == 64 ? kf_describe<Q4_CACHE_INT8, 64>(dev, seqs) : kf_describe<Q4_CACHE_INT8, 128>(dev, seqs);
    return head_dim == 64 ? kf_describe<Q4_CACHE_INT4, 64>(dev, seqs) : kf_describe<Q4_CACHE_INT4, 128>(dev, seqs);
}

}  // namespace q4
