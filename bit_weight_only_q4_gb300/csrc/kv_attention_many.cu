// Attention over the quantised paged cache for more than 16 query rows per key head: a
// chunk of a prompt, drafted tokens, or the rows of a whole batch on a prefix that they
// share.  Mathematics, work list and the joining of pieces: kv_attention.cuh.
//
// A tile of 128 query rows is the MMA's M dimension, one row per TMEM lane:
//     S_g [128 x 64] = q' [128 x D] K_g^T       O_g [128 x D] += P_g [128 x 64] V_g
// for the two 64-token halves g of a tile of 128 tokens.  q' and P are A operands in
// tensor memory, K and V dequantised fp16 tiles in shared memory (B operands: K K-major, V
// as its rows lie).  Each half has its softmax group of four warps, one thread per row
// with references, sums and an accumulator of its own: no thread waits for another's
// row, and while one half's scores are turned into probabilities the tensor cores work
// on the other half or the next tile.  The halves are added up at the end of a unit.
//
// One CTA per SM, 20 warps: one copies blocks, two issue the MMAs, four decode K, four
// V, eight do the softmax and the results.  Measured alone, the MMAs of a tile take 1,050
// cycles (D = 128); the softmax issues about 3,000 instructions, the decoding 1,800.
//
// What bounds it.  A tile takes some 3,300 cycles: 509 query tokens of four sequences of up to
// 8,190 (int8, 32 heads on 8, of 128) 321 us, 497 TFLOP/s; 256 rows of 4 on a prefix of
// 32,768 192 us, 716 TFLOP/s.  No single part sets it: without the softmax's arithmetic a chunk takes
// 14% less, without decoding too 21%, and with an eighth of the MMAs besides still 75% --
// the chain of a softmax warp through barriers and tensor memory, which half as much work
// for twice the warps (28 warps, 32 tokens a thread) did not shorten.  Shared memory's port is
// busy half the time with loads and stores, and with the MMAs' operands on top.  The end
// of a unit costs 11,000 cycles: queries 4,400, results about 5,000.
#include "kv_attention.cuh"

namespace q4 {

constexpr int KM_ROWS = 128;
constexpr int KM_HALF = 64;                        // tokens of a half tile
// warps, in groups of four: softmax of the two halves, K, V; copies, S, O (and one idle)
constexpr int KM_K = 8, KM_V = 12, KM_COPY = 16, KM_S = 17, KM_O = 18, KM_WARPS = 20;
// Registers of a softmax thread and of the others: the launch's 20 x 32 x 96 shared out
// (8 x 128 + 12 x 72 <= 20 x 96).  A softmax thread holds 64 scores and 32 packed
// probabilities; at 96 registers its loop ran with too few instructions in flight.
constexpr int KM_REGS_SOFTMAX = 128, KM_REGS_OTHERS = 72;

// Token scales of a tile (see kv_scales), one array each: four tokens are one broadcast load.
struct KmScales {
    float ks[KT_TOKENS], km[KT_TOKENS], vs[KT_TOKENS], vm[KT_TOKENS];
};

// What a whole unit's row needs to be stored: its sums become a sum + b (prefix's sum) and go
// to `at` (elements of the output, or of the prefix's results).
struct __align__(16) KmRow {
    float a, b;
    int64_t at;
};

// Shared memory: [raw ring][K: 2][V: 2][token scales: 4][results: 2 KB a softmax warp]
struct KmSmem {
    uint32_t k, v, scales, stage, total;
};

template <int FMT, int D>
__host__ __device__ inline KmSmem km_smem(int stages)
{
    KmSmem s = {};
    uint32_t at = (uint32_t)stages * KT_BLOCKS * KvLayout<FMT, D>::BLOCK;
    at = (at + 1023u) & ~1023u;
    s.k = at, at += 2u * KT_TOKENS * D * 2;
    s.v = at, at += 2u * KT_TOKENS * D * 2;
    s.scales = at, at += 4u * (uint32_t)sizeof(KmScales);
    s.stage = at, at += 8u * 2048;
    s.total = at;
    return s;
}

template <int FMT, int D>
__global__ void __launch_bounds__(KM_WARPS * 32, 1) kv_many_rows_kernel(const KvTileParams p)
{
    using L = KvLayout<FMT, D>;
    constexpr uint32_t RAW = KT_BLOCKS * L::BLOCK;
    constexpr uint32_t TILE_BYTES = KT_TOKENS * D * 2;
    // tensor memory columns: q' (D / 2), S of two halves (64), P (32), O (D)
    constexpr uint32_t TM_S = D / 2, TM_P = TM_S + 128, TM_O = TM_P + 64, TM_COLS = 512;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ uint64_t s_bar[2 * KT_MAX_STAGES + 19 + KT_UNITS];
    __shared__ KvUnit s_unit[KT_UNITS];
    __shared__ float s_wmax[4][4];                         // largest V scale of 32 tokens, 2^-60 at least
    __shared__ __align__(16) float s_level[4][KT_TOKENS];  // see kv_scale_level
    __shared__ __align__(16) KmRow s_row[KM_ROWS];
    __shared__ uint32_t s_tmem, s_valid[KT_MAX_STAGES], s_vmask[4];
    __shared__ int s_last, s_dead, s_counted;
    const int NS = p.stages;
    const KmSmem off = km_smem<FMT, D>(NS);
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sm = smem_u32(smem);
    KmScales *s_scales = reinterpret_cast<KmScales *>(smem + off.scales);
    // exchanged between a row's two threads, where the results go later.  s_top is read before q_full, which
    // the first S waits for, and may lie where s_sum does; s_qs is read after it and may not.
    uint32_t (*s_top)[KM_ROWS] = reinterpret_cast<uint32_t (*)[KM_ROWS]>(smem + off.stage);
    float4 (*s_sum)[KM_ROWS] = reinterpret_cast<float4 (*)[KM_ROWS]>(smem + off.stage);   // m, l, offset
    float (*s_qs)[KM_ROWS] = reinterpret_cast<float (*)[KM_ROWS]>(smem + off.stage + 2 * sizeof(*s_sum));

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t raw_full = smem_u32(s_bar), raw_empty = raw_full + 8u * KT_MAX_STAGES;
    const uint32_t k_full = raw_empty + 8u * KT_MAX_STAGES, k_done = k_full + 16, v_full = k_full + 32,
                   v_done = k_full + 48, s_full = k_full + 64, s_free = k_full + 80, p_full = k_full + 96,
                   pv_done = k_full + 112, q_full = k_full + 128, drained = k_full + 136, unit_full = k_full + 152;
    if (warp == KM_COPY) {
        kv_init_bars(raw_full, NS, 1);
        kv_init_bars(raw_empty, NS, 8);                    // K and V warps
        kv_init_bars(k_full, 2, 4);                        // K, V: by buffer
        kv_init_bars(k_done, 2, 1);
        kv_init_bars(v_full, 2, 4);
        kv_init_bars(v_done, 2, 1);
        kv_init_bars(s_full, 2, 1);                        // S, P, O: by half
        kv_init_bars(s_free, 2, 4);
        kv_init_bars(p_full, 2, 4);
        kv_init_bars(pv_done, 2, 1);
        kv_init_bars(q_full, 1, 8);
        kv_init_bars(drained, 2, 1);                       // MMAs of a CTA that has given up
        kv_init_bars(unit_full, KT_UNITS, 1);
        if (lane == 0)
            s_dead = s_counted = 0;
        mbar_init_fence();
    } else if (warp == KM_S) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&s_tmem)), "n"(TM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    pdl_wait();
    const KvShare sh = kv_share<KM_ROWS>(p);
    const KvDead dead = {p.err, &s_dead, smem_u32(&s_dead)};
    auto gone = [&]() { return *dead.flag != 0; };
    // The warps that issue MMAs branch on values that are known to be the warp's, so that
    // descriptors can be kept in uniform registers.
    auto gone_all = [&]() { return __any_sync(0xffffffffu, *dead.flag != 0); };
    const int tiles = __shfl_sync(0xffffffffu, sh.tiles, 0);
    auto unit_wait = [&](int u) { kv_wait(unit_full + 8u * (u & (KT_UNITS - 1)), (u / KT_UNITS) & 1, dead); };

    if (warp < KM_K) {
        // ----------------------------------------- softmax, sums and results
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(KM_REGS_SOFTMAX));
        const int g = warp >> 2;                           // half of the tile
        const int quad = warp & 3;
        const int row = quad * 32 + lane;                  // TMEM lane
        const int t = tid;
        const uint32_t t_lane = (uint32_t)(quad * 32) << 16;
        int i = 0;
#pragma unroll 1
        for (int u = 0; i < sh.tiles; ++u) {
            unit_wait(u);
            if (bar_or(1, 256, gone()))                    // leave together
                break;
            const KvUnit &un = s_unit[u & (KT_UNITS - 1)];
            const int end = i + un.k1 - un.k0, k0 = un.k0 - i, ntok = un.ntok;
            const int row0 = un.rt * KM_ROWS;
            const int nrows = p.rows - row0 < KM_ROWS ? p.rows - row0 : KM_ROWS;
            const int grow0 = (p.prefix_len > 0 ? 0 : un.b * p.rows) + row0;      // among all rows
            const bool mine = row < nrows;
            const bool warp_rows = quad * 32 < nrows;      // any row of the warp
            // ---- queries: this thread's half of its row
            float f, qs = 0.f;
            {
                constexpr int V = D / 16;                  // 16-byte pieces of half a row
                uint4 v[V];
                const uint4 *src = mine ? reinterpret_cast<const uint4 *>(kv_q_row(p, grow0 + row, un.h, D)) + g * V : nullptr;
                uint32_t top = 0u;                         // largest finite |q|
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[j] = mine ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const uint32_t e[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t lo = e[x] & 0x7fffu, hi = (e[x] >> 16) & 0x7fffu;
                        top = lo < 0x7f80u && lo > top ? lo : top;
                        top = hi < 0x7f80u && hi > top ? hi : top;
                    }
                }
                s_top[g][row] = top;
                bar_sync(1, 256);
                top = s_top[0][row] > s_top[1][row] ? s_top[0][row] : s_top[1][row];
                int ex = 141 - (int)(top >> 7);            // the largest goes to [2^14, 2^15)
                ex = ex > 126 ? 126 : ex;
                // a negative scale goes to q', so that the largest score is the largest product; f
                // is no zero, which would make NaN of a masked score
                const float up = copysignf(__uint_as_float((uint32_t)(ex + 127) << 23), p.scale_log2);
                f = fmaxf(fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 - ex) << 23), 1e-37f);
#pragma unroll
                for (int j = 0; j < V; j += 4) {           // 32 columns: 16 packed
                    uint32_t o[16];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t e[4] = {v[j + y].x, v[j + y].y, v[j + y].z, v[j + y].w};
                        float x[8];
#pragma unroll
                        for (int z = 0; z < 8; ++z) {
                            x[z] = ((z & 1) ? __uint_as_float(e[z / 2] & 0xffff0000u) : bf16_bits_to_f32(e[z / 2] & 0xffffu)) * up;
                            qs += x[z];
                        }
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const __half2 h = __floats2half2_rn(x[kv_column<L::I8>(2 * z)], x[kv_column<L::I8>(2 * z + 1)]);
                            o[4 * y + z] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                    }
                    tmem_st16(tmem + t_lane + (uint32_t)g * (D / 4) + 4u * j, o);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_full);
                if constexpr (!L::I8) {
                    s_qs[g][row] = qs;
                    bar_sync(1, 256);
                    qs = s_qs[0][row] + s_qs[1][row];
                }
            }
            const int lim = mine ? kv_row_limit(p, grow0 + row, un.len) : 0x7fffffff;
            const int least = __reduce_min_sync(0xffffffffu, lim);
            float m = -INFINITY;                           // reference
            f32x2 l2 = 0ull, l2b = 0ull, off2 = 0ull, off2b = 0ull;        // (two chains each)
            const f32x2 qs2 = pack2(qs, qs), f2 = pack2(f, f);
            bool first = true;
#pragma unroll 1
            for (; i < end; ++i) {
                kv_wait(s_full + 8u * g, i & 1, dead);
                if (!warp_rows) {                          // nothing to do but keep step
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(s_free + 8u * g);
                    if (i > 0)
                        kv_wait(pv_done + 8u * g, (i - 1) & 1, dead);
                    if (lane == 0)
                        mbar_arrive(p_full + 8u * g);
                    continue;
                }
                tc_fence_after();
                uint32_t v[KM_HALF];
#pragma unroll
                for (int j = 0; j < KM_HALF; j += 16)
                    tmem_ld16_async(tmem + t_lane + TM_S + 64u * g + j, reinterpret_cast<uint32_t(&)[16]>(v[j]));
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(s_free + 8u * g);
                const uint32_t sc = smem_u32(&s_scales[i & 3]) + (uint32_t)g * (KM_HALF * 4);
                const int pos0 = (k0 + i) * KT_TOKENS + g * KM_HALF;
                const uint32_t mask = s_vmask[i & 3];
                const bool masked = !(mask & 0x100u) || pos0 + KM_HALF > least;
                uint32_t ph[KM_HALF / 2];
                // With every token seen and every reference set, go by the references as they are;
                // if some product may then be out of range, go again the careful way.
                bool careful = masked || __any_sync(0xffffffffu, m == -INFINITY);
                if (!careful) {
                    const f32x2 n2 = pack2(-m, -m);
                    f32x2 la = 0ull, lb = 0ull, oa = 0ull, ob = 0ull;
#pragma unroll
                    for (int j = 0; j < KM_HALF; j += 4) {
                        f32x2 ka, kb, va, vb;
                        lds_f32x4(sc + 4u * j, ka, kb);
                        f32x2 a = pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                        f32x2 b = pack2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
                        if constexpr (L::I8) {
                            a = fma2(a, mul2(ka, f2), n2);
                            b = fma2(b, mul2(kb, f2), n2);
                        } else {
                            f32x2 ma, mb;
                            lds_f32x4(sc + 512u + 4u * j, ma, mb);
                            a = fma2(fma2(a, ka, mul2(ma, qs2)), f2, n2);
                            b = fma2(fma2(b, kb, mul2(mb, qs2)), f2, n2);
                        }
                        float x[4];
                        unpack2(a, x[0], x[1]);
                        unpack2(b, x[2], x[3]);
                        a = pack2(ex2(x[0]), ex2(x[1]));
                        b = pack2(ex2(x[2]), ex2(x[3]));
                        la = add2(la, a);
                        lb = add2(lb, b);
                        lds_f32x4(sc + 1024u + 4u * j, va, vb);
                        if constexpr (!L::I8) {
                            f32x2 wa, wb;
                            lds_f32x4(sc + 1536u + 4u * j, wa, wb);
                            oa = fma2(a, wa, oa);
                            ob = fma2(b, wb, ob);
                        }
                        a = mul2(a, va);
                        b = mul2(b, vb);
                        unpack2(a, x[0], x[1]);
                        unpack2(b, x[2], x[3]);
                        const __half2 h0 = __floats2half2_rn(x[0], x[1]), h1 = __floats2half2_rn(x[2], x[3]);
                        ph[j / 2] = *reinterpret_cast<const uint32_t *>(&h0);
                        ph[j / 2 + 1] = *reinterpret_cast<const uint32_t *>(&h1);
                    }
                    // (no p vs is above the sum of p times the largest vs, nor a p above KT_P_TOP where that is 0)
                    float sa, sb;
                    unpack2(add2(la, lb), sa, sb);
                    const float wm = fmaxf(s_wmax[i & 3][2 * g], s_wmax[i & 3][2 * g + 1]);
                    careful = __any_sync(0xffffffffu, !((sa + sb) * wm < 65000.f));
                    if (!careful) {
                        l2 = add2(l2, la);
                        l2b = add2(l2b, lb);
                        off2 = add2(off2, oa);
                        off2b = add2(off2b, ob);
                    }
                }
                if (careful) {
                    // scores over f, then what the reference goes by
#pragma unroll
                    for (int j = 0; j < KM_HALF; j += 4) {
                        f32x2 ka, kb;
                        lds_f32x4(sc + 4u * j, ka, kb);
                        f32x2 a = pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                        f32x2 b = pack2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
                        if constexpr (L::I8) {
                            a = mul2(a, ka);
                            b = mul2(b, kb);
                        } else {
                            f32x2 ma, mb;
                            lds_f32x4(sc + 512u + 4u * j, ma, mb);
                            a = fma2(a, ka, mul2(ma, qs2));
                            b = fma2(b, kb, mul2(mb, qs2));
                        }
                        float x[4];
                        unpack2(a, x[0], x[1]);
                        unpack2(b, x[2], x[3]);
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            v[j + y] = __float_as_uint(x[y]);
                    }
                    if (masked) {
                        const uint32_t blocks = mask >> (4 * g);
                        const int lim1 = lim < ntok ? lim : ntok;
#pragma unroll
                        for (int j = 0; j < KM_HALF; ++j)
                            if (pos0 + j >= lim1 || !((blocks >> (j / KV_BLOCK)) & 1u))
                                v[j] = 0xff800000u;
                    }
                    const uint32_t lv = smem_u32(s_level[i & 3]) + (uint32_t)g * (KM_HALF * 4);
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};      // (short chains)
#pragma unroll
                    for (int j = 0; j < KM_HALF; j += 4) {
                        f32x2 a, b;
                        lds_f32x4(lv + 4u * j, a, b);
                        a = fma2(pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), f2, a);
                        b = fma2(pack2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), f2, b);
                        float x[4];
                        unpack2(a, x[0], x[1]);
                        unpack2(b, x[2], x[3]);
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            tops[y] = fmaxf(tops[y], x[y]);
                    }
                    const float want = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    if (__any_sync(0xffffffffu, want > m + 8.f)) {
                        const float old = m;
                        m = fmaxf(m, want);
                        const float c = old == -INFINITY ? 0.f : ex2(old - m);
                        const f32x2 c2 = pack2(c, c);
                        l2 = mul2(l2, c2);
                        l2b = mul2(l2b, c2);
                        off2 = mul2(off2, c2);
                        off2b = mul2(off2b, c2);
                        if (!first) {
                            kv_wait(pv_done + 8u * g, (i - 1) & 1, dead);
                            tc_fence_after();
#pragma unroll 1
                            for (int j = 0; j < D; j += 16) {
                                uint32_t o[16];
                                const uint32_t a = tmem + t_lane + TM_O + (uint32_t)g * D + j;
                                tmem_ld16(a, o);
#pragma unroll
                                for (int x = 0; x < 16; ++x)
                                    o[x] = __float_as_uint(__uint_as_float(o[x]) * c);
                                tmem_st16(a, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float neg = m == -INFINITY ? 0.f : -m;
                    const f32x2 n2 = pack2(neg, neg);
#pragma unroll
                    for (int j = 0; j < KM_HALF; j += 4) {
                        f32x2 a = fma2(pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), f2, n2);
                        f32x2 b = fma2(pack2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), f2, n2);
                        float x[4];
                        unpack2(a, x[0], x[1]);
                        unpack2(b, x[2], x[3]);
                        a = pack2(ex2(x[0]), ex2(x[1]));
                        b = pack2(ex2(x[2]), ex2(x[3]));
                        l2 = add2(l2, a);
                        l2b = add2(l2b, b);
                        f32x2 va, vb;
                        lds_f32x4(sc + 1024u + 4u * j, va, vb);
                        if constexpr (!L::I8) {
                            f32x2 oa, ob;
                            lds_f32x4(sc + 1536u + 4u * j, oa, ob);
                            off2 = fma2(a, oa, off2);
                            off2b = fma2(b, ob, off2b);
                        }
                        a = mul2(a, va);
                        b = mul2(b, vb);
                        unpack2(a, x[0], x[1]);
                        unpack2(b, x[2], x[3]);
                        const __half2 h0 = __floats2half2_rn(x[0], x[1]), h1 = __floats2half2_rn(x[2], x[3]);
                        ph[j / 2] = *reinterpret_cast<const uint32_t *>(&h0);
                        ph[j / 2 + 1] = *reinterpret_cast<const uint32_t *>(&h1);
                    }
                }
                if (i > 0)                                 // the half's last P has been read
                    kv_wait(pv_done + 8u * g, (i - 1) & 1, dead);
                tc_fence_after();
                tmem_st16(tmem + t_lane + TM_P + 32u * g, reinterpret_cast<uint32_t(&)[16]>(ph[0]));
                tmem_st16(tmem + t_lane + TM_P + 32u * g + 16u, reinterpret_cast<uint32_t(&)[16]>(ph[16]));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full + 8u * g);
                first = false;
            }
            // ---- add the two halves up: this thread stores its row's half of the columns
            {
                float a, b, c, d;
                unpack2(add2(l2, l2b), a, b);
                unpack2(add2(off2, off2b), c, d);
                s_sum[g][row] = make_float4(m, a + b, c + d, 0.f);
            }
            kv_wait(pv_done + 8u * g, (i - 1) & 1, dead);
            bar_sync(1, 256);
            tc_fence_after();
            const float4 s0 = s_sum[0][row], s1 = s_sum[1][row];
            KvRowSum r;
            r.m = fmaxf(s0.x, s1.x);
            const float c0 = s0.x == -INFINITY ? 0.f : ex2(s0.x - r.m), c1 = s1.x == -INFINITY ? 0.f : ex2(s1.x - r.m);
            r.l = s0.y * c0 + s1.y * c1;
            const float offset = s0.z * c0 + s1.z * c1;
            const bool whole = un.k0 == 0 && un.k1 == un.n;
            const int64_t slot = kv_piece_slot(un) * KM_ROWS;
            if (g == 0 && mine && whole) {
                const int grow = grow0 + row;
                const int64_t n = (int64_t)un.h * p.all_rows + grow;
                KmRow w = {1.f, 0.f, n * D};
                if (p.prefix_len > 0) {                    // a piece for the launch over the sequences' own tokens
                    *reinterpret_cast<float2 *>(p.prefix_out_ml + n * 2) = make_float2(r.m, r.l);
                } else {
                    float l = r.l;
                    if (p.prefix_in_o) {
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p.prefix_in_ml + n * 2));
                        const float top = fmaxf(r.m, ml.x);
                        w.a = r.m == -INFINITY ? 0.f : ex2(r.m - top);
                        w.b = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
                        l = l * w.a + ml.y * w.b;
                    }
                    // a row that sees nothing has l = 0 and gives zeros
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    w.a *= inv;
                    w.b *= inv;
                    const int token = p.by_group(grow);
                    w.at = ((int64_t)token * p.cache.heads * p.group + un.h * p.group + grow - token * p.group) * D;
                }
                s_row[row] = w;
            }
            const bool leave = bar_or(1, 256, gone());     // (s_sum has been read)
            if (warp_rows && !leave) {
                // 16 columns at a time through the warp's 2 KB of shared memory: written by row,
                // read four lanes to a row, so that a store fills whole sectors.  Float4 c of row
                // n lies at place c ^ (n / 2 & 3): no bank conflicts either way.
                const uint32_t st = sm + off.stage + (uint32_t)warp * 2048u;
                const uint32_t w_at = st + (uint32_t)lane * 64u, w_key = (uint32_t)(lane >> 1) & 3u;
#pragma unroll 1
                for (int j = g * (D / 2); j < (g + 1) * (D / 2); j += 16) {
                    uint32_t a[16], b[16];
                    tmem_ld16_async(tmem + t_lane + TM_O + j, a);
                    tmem_ld16_async(tmem + t_lane + TM_O + D + j, b);
                    tmem_wait_ld();
                    float x[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y)           // place -> column: permuted within 8
                        x[kv_column<L::I8>(y)] = fmaf(__uint_as_float(a[y]), c0, fmaf(__uint_as_float(b[y]), c1, offset));
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        sts128(w_at + ((((uint32_t)y) ^ w_key) << 4), __float_as_uint(x[4 * y]), __float_as_uint(x[4 * y + 1]),
                               __float_as_uint(x[4 * y + 2]), __float_as_uint(x[4 * y + 3]));
                    __syncwarp();
#pragma unroll
                    for (int n = lane >> 2; n < 32; n += 8) {
                        const int nn = quad * 32 + n, c = lane & 3;
                        const uint4 v = lds128(st + (uint32_t)n * 64u + (((uint32_t)c ^ ((uint32_t)n >> 1 & 3u)) << 4));
                        float4 o = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                                               __uint_as_float(v.w));
                        if (nn >= nrows)
                            continue;
                        if (!whole) {
                            *reinterpret_cast<float4 *>(p.piece_o + (slot + nn) * D + j + 4 * c) = o;
                            continue;
                        }
                        const KmRow w = s_row[nn];
                        if (p.prefix_len > 0) {
                            *reinterpret_cast<float4 *>(p.prefix_out_o + w.at + j + 4 * c) = o;
                            continue;
                        }
                        o.x *= w.a, o.y *= w.a, o.z *= w.a, o.w *= w.a;
                        if (p.prefix_in_o) {
                            const float4 x = __ldcg(reinterpret_cast<const float4 *>(
                                p.prefix_in_o + ((int64_t)un.h * p.all_rows + grow0 + nn) * D + j + 4 * c));
                            o.x = fmaf(x.x, w.b, o.x), o.y = fmaf(x.y, w.b, o.y);
                            o.z = fmaf(x.z, w.b, o.z), o.w = fmaf(x.w, w.b, o.w);
                        }
                        *reinterpret_cast<uint2 *>(p.out + w.at + j + 4 * c) =
                            make_uint2((uint32_t)f32_to_bf16_bits(o.x) | ((uint32_t)f32_to_bf16_bits(o.y) << 16),
                                       (uint32_t)f32_to_bf16_bits(o.z) | ((uint32_t)f32_to_bf16_bits(o.w) << 16));
                    }
                    __syncwarp();
                }
            }
            if (!whole && !leave) {
                if (mine && g == 0)
                    *reinterpret_cast<float2 *>(p.piece_ml + (slot + row) * 2) = make_float2(r.m, r.l);
                kv_join<D, KM_ROWS, 256, 4>(p, sh, un, nrows, grow0, &s_last, &s_counted, t, 1);
            }
            tc_fence_before();
            bar_sync(1, 256);                              // O and s_sum may be written again
        }
    } else if (warp < KM_COPY) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(KM_REGS_OTHERS));
        // ------------------------------- K and V: fp16 tiles in shared memory
        const bool is_v = warp >= KM_V;
        const int tok = (warp & 3) * 32 + lane;
        const int r = tok & (KV_BLOCK - 1);
        const KvRowAt<FMT, D> from(tok);
        const KvRowTo to(tok);
        const uint32_t full = is_v ? v_full : k_full, done = is_v ? v_done : k_done;
        const uint32_t dst = sm + (is_v ? off.v : off.k);
        int k = 0, k1 = 0, ntok = 0, u = 0, s = 0;
        uint32_t round = 0u;                               // parity of the ring's round
#pragma unroll 1
        for (int i = 0; i < sh.tiles && !gone(); ++i, ++k) {
            if (!is_v && k == k1) {
                unit_wait(u);
                const KvUnit &un = s_unit[u & (KT_UNITS - 1)];
                k = un.k0, k1 = un.k1, ntok = un.ntok;
                ++u;
            }
            kv_wait(raw_full + 8u * s, round, dead);
            if (i >= 2)
                kv_wait(done + 8u * (i & 1), ((i >> 1) - 1) & 1, dead);
            const uint32_t raw = sm + (uint32_t)s * RAW, blk = raw + (uint32_t)(tok / KV_BLOCK) * L::BLOCK;
            if (!is_v) {
                // blocks of the tile that are there and hold tokens; bit 8: all of them do, wholly
                uint32_t mask = s_valid[s];
                if (mask == 0xffu && (k + 1) * KT_TOKENS <= ntok)
                    mask |= 0x100u;
                const bool here = ((mask >> (tok / KV_BLOCK)) & 1u) && k * KT_TOKENS + tok < ntok;
                const float4 sc = here ? kv_scales<FMT, D>(blk, r) : make_float4(0.f, 0.f, 0.f, 0.f);
                KmScales &out = s_scales[i & 3];
                out.ks[tok] = sc.x;
                out.vs[tok] = sc.z;
                s_level[i & 3][tok] = kv_scale_level(fabsf(sc.z));
                if constexpr (!L::I8) {
                    out.km[tok] = sc.y;
                    out.vm[tok] = sc.w;
                }
                static_assert(KT_P_TOP * 0x1p-60f >= 65000.f, "the range of p ends with that of the products");
                const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(sc.z), 0x1p-60f)));
                if (lane == 0)
                    s_wmax[i & 3][warp & 3] = __uint_as_float(top);
                if (warp == KM_K && lane == 0)
                    s_vmask[i & 3] = mask;
            }
            kv_row_to_tile<FMT, D>(raw + (is_v ? L::V_CODES : 0), from, dst + (uint32_t)(i & 1) * TILE_BYTES, to);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full + 8u * (i & 1));
                mbar_arrive(raw_empty + 8u * s);
            }
            if (++s == NS)
                s = 0, round ^= 1u;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(KM_REGS_OTHERS));
        if (warp == KM_COPY) {
            kv_copy_warp<FMT, D, KM_ROWS>(p, sh, s_unit, unit_full, sm, s_valid, raw_full, raw_empty, dead);
        } else if (warp == KM_S) {
        // ------------------------------------------------------ MMAs: S = q' K^T
        constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(KM_HALF >> 3) << 17) | (8u << 24);       // f16, f32 sums, M = 128
        int u = -1, left = 0;
#pragma unroll 1
        for (int i = 0; i < tiles && !gone_all(); ++i) {
            if (left == 0) {
                ++u;
                unit_wait(u);
                const KvUnit &un = s_unit[u & (KT_UNITS - 1)];
                left = __shfl_sync(0xffffffffu, un.k1 - un.k0, 0);
                kv_wait(q_full, u & 1, dead);
            }
            --left;
            kv_wait(k_full + 8u * (i & 1), (i >> 1) & 1, dead);
            const uint64_t bd = smem_desc_sw128(sm + off.k + (uint32_t)(i & 1) * TILE_BYTES);
            const uint32_t blo = (uint32_t)bd, bhi = (uint32_t)(bd >> 32);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (i > 0)
                    kv_wait(s_free + 8u * g, (i - 1) & 1, dead);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)    // 64-column halves of K 16 KB apart
                        mma_f16_tmem_a(tmem + TM_S + 64u * g, tmem + 8u * kk,
                                       blo + (uint32_t)g * (8192 >> 4) + (uint32_t)(kk >> 2) * (KT_TOKENS * 128 >> 4) +
                                           2u * (kk & 3),
                                       bhi, idesc, kk > 0 ? 1u : 0u);
                    mma_commit(s_full + 8u * g);
                    if (g == 1)
                        mma_commit(k_done + 8u * (i & 1));
                }
                __syncwarp();
            }
        }
        } else if (warp == KM_O) {
        // ------------------------------------------------------- MMAs: O += P V
        constexpr uint32_t idesc = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);   // B is N-major
        int u = -1, left = 0;
#pragma unroll 1
        for (int i = 0; i < tiles && !gone_all(); ++i) {
            const bool first = left == 0;
            if (first) {
                ++u;
                unit_wait(u);
                const KvUnit &un = s_unit[u & (KT_UNITS - 1)];
                left = __shfl_sync(0xffffffffu, un.k1 - un.k0, 0);
            }
            --left;
            kv_wait(v_full + 8u * (i & 1), (i >> 1) & 1, dead);
            const uint64_t bd = (smem_desc_sw128(sm + off.v + (uint32_t)(i & 1) * TILE_BYTES) & ~((uint64_t)0x3fff << 16)) |
                                ((uint64_t)(D == 128 ? KT_TOKENS * 128 >> 4 : 0) << 16);
            const uint32_t blo = (uint32_t)bd, bhi = (uint32_t)(bd >> 32);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                kv_wait(p_full + 8u * g, i & 1, dead);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < KM_HALF / 16; ++kk)          // 16 tokens: two groups of 8
                        mma_f16_tmem_a(tmem + TM_O + (uint32_t)g * D, tmem + TM_P + 32u * g + 8u * kk,
                                       blo + (uint32_t)g * (8192 >> 4) + (uint32_t)kk * (2048 >> 4), bhi, idesc,
                                       kk > 0 || !first ? 1u : 0u);
                    mma_commit(pv_done + 8u * g);
                    if (g == 1)
                        mma_commit(v_done + 8u * (i & 1));
                }
                __syncwarp();
            }
        }
        }
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (gone()) {                // (here, not in the warps' roles: there it cost the MMA loops their uniform registers)
        if (warp == KM_COPY)
            kv_arrive_failed<KM_ROWS>(p, s_counted);
        else if (warp == KM_S || warp == KM_O)
            kv_mma_drain(drained + (warp == KM_O ? 8u : 0u), dead);
        tc_fence_before();
        __syncthreads();
    }
    if (warp == KM_S) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(TM_COLS) : "memory");
    }
}

template <int FMT, int D>
static KvKernel km_describe(const DeviceInfo &dev)
{
    KvKernel k = {};
    k.fn = reinterpret_cast<const void *>(&kv_many_rows_kernel<FMT, D>);
    k.tile = KM_ROWS;
    k.threads = KM_WARPS * 32;
    // 1024: alignment; 6144: static arrays and the CTA's reserve
    const size_t budget = dev.smem_optin - 1024 - 6144;
    for (k.stages = KT_MAX_STAGES; k.stages > 1 && km_smem<FMT, D>(k.stages).total > budget;)
        --k.stages;
    k.smem = km_smem<FMT, D>(k.stages).total + 1024;
    return k;
}

KvKernel kv_many_kernel(const DeviceInfo &dev, int format, int head_dim)
{
    if (format == Q4_CACHE_INT8)
        return head_dim == 64 ? km_describe<Q4_CACHE_INT8, 64>(dev) : km_describe<Q4_CACHE_INT8, 128>(dev);
    return head_dim == 64 ? km_describe<Q4_CACHE_INT4, 64>(dev) : km_describe<Q4_CACHE_INT4, 128>(dev);
}

}  // namespace q4
