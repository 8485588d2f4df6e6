// Adapters for requests of many tokens (see lora.cuh): tiles of up to 128 tokens on tcgen05.
//
//     t [128 x rank] = x [128 x K] A^T,     out [128 x 64] = base + scale (t [128 x rank] B [64 x rank]^T)
// with tokens as the MMA's M.  Eleven warps: eight with the exchange of t and the results, one that copies x, A and base
// (TMA), one that copies B and one that issues the MMAs.  A CTA's share of K comes first, through a ring of x and A
// tiles of 64 columns.  The sums go from tensor memory to shared memory; each CTA of the cluster adds up its share of
// the rows of all and writes them, as bf16, into the second product's operand of all.  Then come the
// CTA's output columns, 64 at a time: base and B through rings, base + product in place, and out by TMA from there,
// or, where a warp's 32 rows are not all the tile's, with plain stores (the next rows are
// another request's).  The two groups of four warps take the pieces of 64 columns in turn.
//
// What bounds it: HBM, 2 bytes of x, and 4 of base and out, a value.  Two CTAs share an SM (112 KB each), so that the
// beginning of one runs beside the columns of another.  Measured: 30,705 tokens, 2048 -> 8192, rank 128, 198 us, 5.7 TB/s
// (84% of a copy's rate; the exchange of t and the last wave are the rest); 9,446 tokens in 79 tiles, 2048 -> 8192,
// rank 32, 63 us, 5.6 TB/s, one wave, whose first 10 us store nothing.  Above some hundred requests the lengths that each
// cluster adds up count, as in lora_few.cu: 64, 256, 1,024 and 4,096 requests of 40 tokens, rank 16, 512 -> 512, take 10.7, 23.7,
// 164 and 2,129 us.
#include "lora.cuh"
#include "tma.h"

namespace q4 {

constexpr int LM_ROWS = 128, LM_COPY = 8, LM_MMA = 9, LM_B = 10, LM_WARPS = 11, LM_COLS = 64;

// WIDE: ranks above 64.  There t goes on into tensor memory, as the second product's A operand, and leaves its
// place to B.  Shared memory, in KB:
//          base ring     weights (A or B)    t             while t is being made: x, A, and its sums
//   narrow 0: 4 x 16     64: 4 x 8           96: 16        0: 4 x 16, 64: 4 x 8, 32: 32
//   wide   0: 4 x 16     64: 3 x 16          80: 32        0: 3 x 16, 48: 3 x 16, 0: 64
template <bool WIDE>
struct LmSmem {
    static constexpr int BASES = 4, WEIGHTS = WIDE ? 3 : 4, STAGES = WIDE ? 3 : 4, DS = WIDE ? 2 : 4;       // DS: D in tensor memory
    // (an even number: a slot's phases are those of one group of warps, which waits for each of them)
    static_assert(BASES % 2 == 0 && DS % 2 == 0, "each slot and each D is one group's");
    static constexpr uint32_t SLOT = 16384, W_SLOT = WIDE ? 16384 : 8192;
    static constexpr uint32_t W = BASES * SLOT, T = W + (WIDE ? 1 : 4) * W_SLOT, A = STAGES * SLOT, SUMS = WIDE ? 0 : 2 * SLOT;
    static constexpr int BASES_EARLY = WIDE ? 0 : 2, WEIGHTS_EARLY = WIDE ? 1 : 4;       // slots beside the sums and t
    static constexpr uint32_t BARS = T + (WIDE ? 32768 : 16384), TOTAL = BARS + 512;
};

template <bool WIDE>
__global__ void __launch_bounds__(LM_WARPS * 32, 2)
    lora_many_kernel(const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap a_map,
                     const __grid_constant__ CUtensorMap b_map, const __grid_constant__ CUtensorMap base_map,
                     const __grid_constant__ CUtensorMap out_map, const LoraArgs p)
{
    using L = LmSmem<WIDE>;
    constexpr uint32_t TM_COLS = 256, TM_T = 128;           // D from column 0 on, t as an operand
    constexpr int LM_D = L::DS;
    constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);    // bf16, fp32 sums, M = 128
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sm = smem_u32(smem);
    const int tid = (int)threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = lr_rank_in_cluster(), size = lr_cluster_size();
    const uint32_t x_full = sm + L::BARS, x_free = x_full + 32, base_full = x_free + 32, base_free = base_full + 32,
                   w_full = base_free + 32, w_free = w_full + 32, d_full = w_free + 32, d_free = d_full + 32,
                   t_full = d_free + 32, drained = t_full + 8, t_ready = drained + 8;
    volatile int *dead_flag = reinterpret_cast<volatile int *>(smem + L::BARS + 384);
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(smem + L::BARS + 388);

    if (warp == LM_COPY && lane == 0) {
        tma_prefetch_map(&x_map);
        tma_prefetch_map(&a_map);
        tma_prefetch_map(&base_map);
        tma_prefetch_map(&b_map);
        tma_prefetch_map(&out_map);
    }
    pdl_wait();
    LoraTile tile;
    if (!lr_tile(p, (int)(blockIdx.x / size), LM_ROWS, tile))
        return;                                            // (the whole cluster)
    if (tile.adapter < 0) {
        lr_copy(p, tile, rank, size);
        return;
    }
    if ((sm & 1023u) != 0u) {                              // (there is no static shared memory in front of it)
        if (p.err && tid == 0)
            atomicOr(p.err, kErrBarrierTimeout);
        return;
    }
    if (warp == LM_COPY) {
        if (lane == 0) {
            for (int i = 0; i < L::STAGES; ++i) {
                mbar_init(x_full + 8u * i, 1);
                mbar_init(x_free + 8u * i, 1);
            }
            for (int i = 0; i < L::BASES; ++i) {
                mbar_init(base_full + 8u * i, 1);
                mbar_init(base_free + 8u * i, 4);
            }
            for (int i = 0; i < L::WEIGHTS; ++i) {
                mbar_init(w_full + 8u * i, 1);
                mbar_init(w_free + 8u * i, 1);
            }
            for (int i = 0; i < LM_D; ++i) {
                mbar_init(d_full + 8u * i, 1);
                mbar_init(d_free + 8u * i, 4);
            }
            mbar_init(t_full, 1);
            mbar_init(drained, 1);
            mbar_init(t_ready, 4);
            *dead_flag = 0;
        }
        mbar_init_fence();
    } else if (warp == LM_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_at)), "n"(TM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_at, 0);
    const KvDead dead = {p.err, dead_flag, smem_u32(const_cast<int *>(dead_flag))};
    auto gone_all = [&]() { return __any_sync(0xffffffffu, *dead.flag != 0); };
    const int ranks = (p.rank + 15) / 16 * 16;
    // Pieces of 64 columns go round the cluster, so that its CTAs are in the same DRAM pages at a time.
    const int nk = lr_round((p.K + 63) / 64, rank, size), nn = lr_round((p.N + 63) / 64, rank, size);
    auto slice = [&](int i) { return (int)rank + i * (int)size; };
    const int groups = (tile.rows + 31) / 32;              // of 32 rows

    if (warp < 8) {
        // ----------------------------------------- exchange of t, results
        const int quad = warp & 3, side = warp >> 2;
        const int row = quad * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        // place of columns j .. j + 3 (7) of row r in t
        auto t_place = [&](int r, int j) {
            return sm + L::T + (uint32_t)(j >> 6) * 16384u + (uint32_t)r * 128u +
                   ((((uint32_t)(j >> 3) & 7u) ^ ((uint32_t)r & 7u)) << 4) + ((uint32_t)j & 7u) * 2u;
        };
        if (nk > 0) {
            kv_wait(t_full, 0u, dead);
            tc_fence_after();
        }
        const uint32_t key = ranks % 32 == 0 ? (uint32_t)row & 7u : (uint32_t)(row >> 1) & 3u;
#pragma unroll 1
        for (int c = side * (ranks / 2); c < (side + 1) * (ranks / 2); c += 8) {
            uint32_t v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            if (nk > 0)
                tmem_ld8(t_lane + c, v);
            const uint32_t at = sm + L::SUMS + (uint32_t)(row * ranks * 4);
            sts128(at + ((((uint32_t)c >> 2) ^ key) << 4), v[0], v[1], v[2], v[3]);
            sts128(at + ((((uint32_t)(c >> 2) + 1u) ^ key) << 4), v[4], v[5], v[6], v[7]);
        }
        tc_fence_before();
        lr_cluster_arrive();
        lr_cluster_wait();
        const int pieces = ranks / 4, part = (LM_ROWS + (int)size - 1) / (int)size;
        for (int i = tid; i < part * pieces; i += 256) {
            const int rr = i / pieces, c = i - rr * pieces, r = part * (int)rank + rr;
            if (r >= tile.rows)                        // (and below 128)
                break;
            const uint32_t k = ranks % 32 == 0 ? (uint32_t)r & 7u : (uint32_t)(r >> 1) & 3u;
            const uint32_t at = sm + L::SUMS + (uint32_t)(r * ranks * 4) + (((uint32_t)c ^ k) << 4);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (uint32_t j = 0; j < LR_CLUSTER; ++j) {
                if (j < size) {
                    const float4 w = lr_load(lr_map(at, j));
                    v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
                }
            }
            const int j = 4 * c;
            const uint32_t lo = j < p.rank ? bf16_pair(v.x, v.y) : 0u, hi = j < p.rank ? bf16_pair(v.z, v.w) : 0u;
            const uint32_t to = t_place(r, j);
#pragma unroll
            for (uint32_t y = 0; y < LR_CLUSTER; ++y)
                if (y < size)
                    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(lr_map(to, y)), "r"(lo), "r"(hi) : "memory");
        }
        asm volatile("fence.proxy.async;" ::: "memory");
        __syncwarp();
        lr_cluster_arrive();
        lr_cluster_wait();
        if (WIDE && side == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 e = lds128(t_place(row, 64 * h + 8 * c));
                    w[4 * c] = e.x, w[4 * c + 1] = e.y, w[4 * c + 2] = e.z, w[4 * c + 3] = e.w;
                }
                tmem_st32(t_lane + TM_T + 32u * h, w);
            }
            tmem_wait_st();
            tc_fence_before();
            fence_proxy_async();                           // (B comes to where they were)
            __syncwarp();
            if (lane == 0)
                mbar_arrive(t_ready);
        }
        const float scale = __ldg(p.scales + tile.adapter);
        const int last = tile.rows - quad * 32;            // the warp's rows, if below 32
#pragma unroll 1
        for (int q = side; q < nn; q += 2) {
            const uint32_t s = (uint32_t)q % L::BASES, d = (uint32_t)q % LM_D;
            kv_wait(d_full + 8u * d, ((uint32_t)q / LM_D) & 1u, dead);
            tc_fence_after();
            const uint32_t mine = sm + s * L::SLOT + (uint32_t)row * 128u, rk = (uint32_t)row & 7u;
            // (warps without rows wait too: their arrival below is to be of this use of the slot)
            kv_wait(base_full + 8u * s, ((uint32_t)q / L::BASES) & 1u, dead);
            if (last > 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[32];
                    tmem_ld32_async(t_lane + LM_COLS * d + 32u * h, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t at = mine + (((uint32_t)(4 * h + c) ^ rk) << 4);
                        const uint4 b = lds128(at);
                        const uint32_t e[4] = {b.x, b.y, b.z, b.w};
                        uint32_t o[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            o[y] = bf16_pair(fmaf(scale, __uint_as_float(v[8 * c + 2 * y]), __uint_as_float(e[y] << 16)),
                                             fmaf(scale, __uint_as_float(v[8 * c + 2 * y + 1]), __uint_as_float(e[y] & 0xffff0000u)));
                        sts128(at, o[0], o[1], o[2], o[3]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(d_free + 8u * d);
            const bool ok = !gone_all();
            if (last >= 32) {
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    if (ok) {
                        tma_store_2d(&out_map, slice(q) * LM_COLS, tile.row + quad * 32, sm + s * L::SLOT + (uint32_t)quad * 4096u);
                        asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
                    }
                    mbar_arrive(base_free + 8u * s);
                }
            } else {
                const int piece = lane & 7, n = slice(q) * LM_COLS + 8 * piece;
                if (ok && n < p.N) {
#pragma unroll 1
                    for (int r = lane >> 3; r < last; r += 4) {
                        const uint4 v = lds128(sm + s * L::SLOT + (uint32_t)(quad * 32 + r) * 128u +
                                               (((uint32_t)piece ^ ((uint32_t)r & 7u)) << 4));
                        *reinterpret_cast<uint4 *>(p.out + (int64_t)(tile.row + quad * 32 + r) * p.out_stride + n) = v;
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(base_free + 8u * s);
            }
            __syncwarp();
        }
        if (lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else if (warp == LM_COPY) {
        // ------------------------------------------------------- copies
        int xs = 0, bs = 0;                                // issued
#pragma unroll 1
        for (int i = 0; i < nk && !gone_all(); ++i) {
            const uint32_t s = (uint32_t)i % L::STAGES;
            if (i >= L::STAGES)
                kv_wait(x_free + 8u * s, ((uint32_t)i / L::STAGES - 1u) & 1u, dead);
            if (gone_all())
                break;
            if (elect_one()) {
                mbar_arrive_expect_tx(x_full + 8u * s, (uint32_t)(groups * 4096 + ranks * 128));
                for (int g = 0; g < groups; ++g)
                    tma_load_2d(sm + s * L::SLOT + 4096u * g, &x_map, 64 * slice(i), tile.row + 32 * g, x_full + 8u * s);
                tma_load_3d(sm + L::A + s * L::W_SLOT, &a_map, 64 * slice(i), 0, tile.adapter, x_full + 8u * s);
            }
            __syncwarp();
            ++xs;
        }
        auto ask_base = [&]() {
            const uint32_t s = (uint32_t)bs % L::BASES;
            if (elect_one()) {
                mbar_arrive_expect_tx(base_full + 8u * s, (uint32_t)groups * 4096u);
                for (int g = 0; g < groups; ++g)
                    tma_load_2d(sm + s * L::SLOT + 4096u * g, &base_map, slice(bs) * LM_COLS, tile.row + 32 * g, base_full + 8u * s);
            }
            __syncwarp();
            ++bs;
        };
        if (nk > 0)
            kv_wait(t_full, 0u, dead);                     // (x and A have been read)
        for (int i = 0; i < L::BASES_EARLY && i < nn && !gone_all(); ++i)
            ask_base();
        lr_cluster_arrive();                               // (every thread passes the same barriers)
        lr_cluster_wait();
        lr_cluster_arrive();
        lr_cluster_wait();
#pragma unroll 1
        for (int q = 0; q < nn && !gone_all(); ++q) {
            if (q >= bs) {
                if (q >= L::BASES)
                    kv_wait(base_free + 8u * ((uint32_t)q % L::BASES), ((uint32_t)q / L::BASES - 1u) & 1u, dead);
                if (gone_all())
                    break;
                ask_base();
            }
        }
        if (gone_all()) {
            // copies in flight land before the CTA ends
            for (int i = xs > L::STAGES ? xs - L::STAGES : 0; i < xs; ++i)
                mbar_wait(x_full + 8u * ((uint32_t)i % L::STAGES), ((uint32_t)i / L::STAGES) & 1u, p.err);
            for (int i = bs > L::BASES ? bs - L::BASES : 0; i < bs; ++i)
                mbar_wait(base_full + 8u * ((uint32_t)i % L::BASES), ((uint32_t)i / L::BASES) & 1u, p.err);
        }
    } else if (warp == LM_B) {
        // ------------------------------------------- B, beside the copies of base
        int ws = 0;
        auto ask = [&]() {
            const uint32_t s = (uint32_t)ws % L::WEIGHTS;
            if (elect_one()) {
                mbar_arrive_expect_tx(w_full + 8u * s, L::W_SLOT);
#pragma unroll
                for (int h = 0; h < (WIDE ? 2 : 1); ++h)
                    tma_load_3d(sm + L::W + s * L::W_SLOT + 8192u * h, &b_map, 64 * h, slice(ws) * LM_COLS, tile.adapter,
                                w_full + 8u * s);
            }
            __syncwarp();
            ++ws;
        };
        if (nk > 0)
            kv_wait(t_full, 0u, dead);                     // (x and A have been read)
        for (int i = 0; i < L::WEIGHTS_EARLY && i < nn && !gone_all(); ++i)
            ask();
        lr_cluster_arrive();
        lr_cluster_wait();
        lr_cluster_arrive();
        lr_cluster_wait();
        if (WIDE)
            kv_wait(t_ready, 0u, dead);
#pragma unroll 1
        while (ws < nn && !gone_all()) {
            if (ws >= L::WEIGHTS)
                kv_wait(w_free + 8u * ((uint32_t)ws % L::WEIGHTS), ((uint32_t)ws / L::WEIGHTS - 1u) & 1u, dead);
            if (gone_all())
                break;
            ask();
        }
        if (gone_all())
            for (int i = ws > L::WEIGHTS ? ws - L::WEIGHTS : 0; i < ws; ++i)
                mbar_wait(w_full + 8u * ((uint32_t)i % L::WEIGHTS), ((uint32_t)i / L::WEIGHTS) & 1u, p.err);
    } else {
        // --------------------------------------------------------- MMAs
        const uint64_t d0 = smem_desc_sw128(sm);
        const uint32_t lo = (uint32_t)d0, hi = (uint32_t)(d0 >> 32);
#pragma unroll 1
        for (int i = 0; i < nk && !gone_all(); ++i) {
            const uint32_t s = (uint32_t)i % L::STAGES;
            kv_wait(x_full + 8u * s, ((uint32_t)i / L::STAGES) & 1u, dead);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f16_2(tmem, lo + s * (L::SLOT >> 4) + 2u * kk, hi, lo + ((L::A + s * L::W_SLOT) >> 4) + 2u * kk, hi,
                              IDESC | ((uint32_t)(ranks >> 3) << 17), i > 0 || kk > 0 ? 1u : 0u);
                mma_commit(x_free + 8u * s);
                if (i == nk - 1)
                    mma_commit(t_full);
            }
            __syncwarp();
        }
        lr_cluster_arrive();                               // (every thread passes the same barriers)
        lr_cluster_wait();
        lr_cluster_arrive();
        lr_cluster_wait();
        asm volatile("fence.proxy.async;" ::: "memory");
        if (WIDE)
            kv_wait(t_ready, 0u, dead);
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < nn && !gone_all(); ++q) {
            const uint32_t s = (uint32_t)q % L::WEIGHTS, d = (uint32_t)q % LM_D;
            kv_wait(w_full + 8u * s, ((uint32_t)q / L::WEIGHTS) & 1u, dead);
            if (q >= LM_D)
                kv_wait(d_free + 8u * d, ((uint32_t)q / LM_D - 1u) & 1u, dead);
            tc_fence_after();
            if (elect_one()) {
                for (int kk = 0; kk < ranks / 16; ++kk) {
                    const uint32_t b = lo + ((L::W + s * L::W_SLOT + (uint32_t)(kk >> 2) * 8192u) >> 4) + 2u * (kk & 3),
                                   idesc = IDESC | ((uint32_t)(LM_COLS >> 3) << 17);
                    if (WIDE)
                        mma_f16_tmem_a(tmem + LM_COLS * d, tmem + TM_T + 8u * kk, b, hi, idesc, kk > 0 ? 1u : 0u);
                    else
                        mma_f16_2(tmem + LM_COLS * d, lo + (L::T >> 4) + 2u * kk, hi, b, hi, idesc, kk > 0 ? 1u : 0u);
                }
                mma_commit(d_full + 8u * d);
                mma_commit(w_free + 8u * s);
            }
            __syncwarp();
        }
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (*dead.flag != 0 && warp == LM_MMA)
        kv_mma_drain(drained, dead);
    __syncthreads();
    if (warp == LM_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(TM_COLS) : "memory");
    }
}

template <bool WIDE>
static q4_status lm_launch(const DeviceInfo &dev, const LoraArgs &a, cudaStream_t st, bool pdl)
{
    CUtensorMap x, wa, wb, base, out;
    const int ranks = (a.rank + 15) / 16 * 16;
    q4_status s = tma_rows(x, a.x, (uint64_t)a.K, (uint64_t)a.tokens, a.x_stride, 32);
    if (s == Q4_OK)
        s = tma_heads(wa, a.a, a.K, a.rank, (uint64_t)a.adapters, (int64_t)a.rank * a.K, ranks, 1);
    if (s == Q4_OK)
        s = tma_heads(wb, a.b, a.rank, a.N, (uint64_t)a.adapters, (int64_t)a.N * a.rank, LM_COLS, 1);
    if (s == Q4_OK)
        s = tma_rows(base, a.base, (uint64_t)a.N, (uint64_t)a.tokens, a.base_stride, 32);
    if (s == Q4_OK)
        s = tma_rows(out, a.out, (uint64_t)a.N, (uint64_t)a.tokens, a.out_stride, 32);
    if (s != Q4_OK)
        return s;
    const size_t smem = LmSmem<WIDE>::TOTAL;
    cudaError_t e = cudaFuncSetAttribute(lora_many_kernel<WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaFuncSetAttribute(lora_many_kernel)");
    // At most one part-filled tile a request.  The cluster is the largest whose CTAs all run at once, two an SM: a CTA
    // that has to wait for a place costs a second wave.  Measured, 79 tiles, 2048 -> 8192, rank 32: sizes 2 .. 8 take 76.6,
    // 62.7, 77.8, 74.5, 68.0, 75.2, 75.6 us (3: 237 CTAs of 304); 13 tiles, rank 64: 48, 36, 29, 26, 24, 22.7, 21.4 us.
    // With more tiles than that two: 248 tiles, rank 128, 199, 213, 205, 227, 227, 243, 241 us, and 282 without clusters.
    // (A cluster behind the last tile, where a request has no tokens, goes through all offsets, as in lora_few.cu.)
    const int64_t tiles = (int64_t)a.tokens / LM_ROWS + a.batch;
    int size = 2;
    while (size < LR_CLUSTER && tiles * (size + 1) <= 2 * (int64_t)dev.sms)
        ++size;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * size));
    cfg.blockDim = dim3(LM_WARPS * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, lora_many_kernel<WIDE>, x, wa, wb, base, out, a);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "launch of lora_many_kernel");
}

q4_status launch_lora_many(const DeviceInfo &dev, const LoraArgs &a, cudaStream_t st, bool pdl)
{
    return a.rank <= 64 ? lm_launch<false>(dev, a, st, pdl) : lm_launch<true>(dev, a, st, pdl);
}

}  // namespace q4
