// Attention of a few query rows per key head over the quantised paged cache: the
// streaming kernel.
//
// Mathematics.  For query row i (a query token and one of the heads that share a key
// head) and token j,
//     s_ij = f_i ks_j (q'_i . c_j)                     int8: K = ks c
//     s_ij = f_i (ks_j (q'_i . (c_j - 8)) + (km_j + 8 ks_j) sum q'_i)     int4: K = ks c + km
// in units of log2 (f_i carries scale * log2 e), p_ij = 2^(s_ij - m_i) with the
// running maximum m_i, and
//     o_i = sum_j p_ij vs_j c_j / sum_j p_ij           (int4: + sum_j p_ij (vm_j + 8 vs_j))
// so the scales never touch the codes: both products run on codes that are exact in
// fp16.  q' is q times a power of two per row that puts its largest value in
// [2^14, 2^15) (every bf16 value is then exact in fp16 down to 2^-28 of that value);
// f undoes it.  p vs enters the second product as fp16, scaled by a power of two so
// that the largest p vs seen so far lies in [2^13, 2^14]: it is rounded to 11 bits, and
// terms 2^-27 times the largest still are.  All sums and statistics are fp32.
//
// Work.  The cached tokens of every (sequence, key head, tile of 16 MT query rows) --
// a unit -- are cut into chunks of 32 tokens, and all chunks of all units, laid end to
// end, are dealt out evenly to the CTAs of one wave, wherever the unit boundaries fall:
// lengths may differ as they like.  A CTA's four warps take its chunks in turn.  Each
// warp keeps its own ring of chunks in shared memory (one 1-D bulk copy per block of 16
// tokens, four kinds of data in one copy), so the loop has no CTA-wide barrier, and its
// own running softmax; at the end of a unit the four are merged through shared memory.
// A unit that several CTAs share is joined by the last of them to arrive, in order of
// the pieces: the result does not depend on timing.  No CTA waits for another.
#include "kv_cache.cuh"

namespace q4 {

constexpr int KA_WARPS = 4;
constexpr int KA_THREADS = KA_WARPS * 32;
constexpr int KA_CHUNK = 32;                      // tokens of a warp's step

struct KvStreamParams {
    KvCache cache;
    const uint16_t *q;
    int64_t q_stride;
    uint16_t *out;
    const int32_t *table;        // pages: [batch][table_width], or of the prefix
    const int32_t *lengths;      // [batch]
    int64_t cap;                 // tokens that a sequence's row of the table can name
    int table_width;
    int seqs;                    // sequences of the work list (1 for the prefix)
    int prefix_len;              // > 0: this launch reads the prefix, for all rows
    int batch, tokens, group;    // group: query heads per key head
    int rows;                    // query rows of a unit's parent (tokens * group, or all)
    int row_tiles;
    float scale_log2;            // scale * log2(e)
    int stages;
    int max_rows;                // row slots of a partial result
    unsigned *tickets;           // one per unit
    float *partial;              // [2 * grid][max_rows][D + 2]
    float *prefix_out;           // [heads][batch * tokens * group][D + 2], written (prefix) ...
    const float *prefix_in;      // ... or joined
    unsigned *err;
};

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t kv_prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// d += a b: 16 x 16 fp16 by 16 x 8 fp16, fp32 sums.  The few query rows of a unit fill
// one or two 16-row tiles, and the cache streams from memory at a fraction of this
// instruction's rate; products over many rows run on tcgen05 (kv_attention_tc.cu).
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}

// int8 codes: bytes with the sign bit flipped are code + 128; as the low byte of an
// fp16 with high byte 0x64 that is 1024 + 128 + code.
constexpr uint32_t kI8Bias = 0xE480E480u;          // (-1152, -1152)
__device__ __forceinline__ uint32_t i8_pair_lo(uint32_t w)   // bytes 0, 1 of the flipped word
{
    return hadd2_rn(kv_prmt(w, 0x64646464u, 0x4140), kI8Bias);
}
__device__ __forceinline__ uint32_t i8_pair_hi(uint32_t w)   // bytes 2, 3
{
    return hadd2_rn(kv_prmt(w, 0x64646464u, 0x4342), kI8Bias);
}
// int4 codes, centred: nibbles 0 and 4 (mask 0x000F000F) or, times 16, nibbles 1 and 5.
__device__ __forceinline__ uint32_t i4_pair_lo(uint32_t w)
{
    return hadd2_rn(int4_pair_f16_biased<0x000F000F>(w), 0xE408E408u);            // -1032
}
__device__ __forceinline__ uint32_t i4_pair_hi(uint32_t w)
{
    return hfma2_rn(int4_pair_f16_biased<0x00F000F0>(w), 0x2C002C00u, 0xD480D480u);   // / 16 - 72
}

// What a CTA needs to know of the work list.
struct KvCursor {
    int b;                       // sequence
    int64_t base;                // first chunk of the sequence in the list
    int nch;                     // chunks of each of its units
};

__device__ __forceinline__ int kv_chunks_of(int len)
{
    return len > KA_CHUNK ? (len + KA_CHUNK - 1) / KA_CHUNK : 1;
}

// Unit (of nch chunks each) that chunk x of a sequence belongs to.
__device__ __forceinline__ int kv_unit_of(int64_t x, int nch)
{
    return (x >> 32) == 0 ? (int)((uint32_t)x / (uint32_t)nch) : (int)(x / nch);
}

template <int FMT, int D, int MT>
__global__ void __launch_bounds__(KA_THREADS) kv_stream_kernel(const KvStreamParams p)
{
    using L = KvLayout<FMT, D>;
    constexpr int ROWS = 16 * MT;
    constexpr int KS = D / 16;                     // k-steps of q K^T
    constexpr int DPL = D / 8;                     // output columns per fragment column
    constexpr int STAGE = 2 * L::BLOCK;
    constexpr int PIECE = D + 2;                   // floats of a partial row: o, m, l
    extern __shared__ __align__(128) unsigned char smem[];
    // [ring: warps x stages][q fragments][merge buffers][lengths]
    unsigned char *ring = smem;
    uint4 *s_qf = reinterpret_cast<uint4 *>(smem + (size_t)KA_WARPS * p.stages * STAGE);
    float4 *s_merge = reinterpret_cast<float4 *>(s_qf + MT * KS * 32);      // [2][warps][ROWS * 8]
    int *s_len = reinterpret_cast<int *>(s_merge + 2 * KA_WARPS * ROWS * 8);
    __shared__ uint64_t s_bar[KA_WARPS * 8];
    __shared__ float s_f[ROWS], s_qsum[ROWS];
    __shared__ int s_lim[ROWS];
    __shared__ float s_m[KA_WARPS][ROWS], s_l[KA_WARPS][ROWS], s_off[KA_WARPS][ROWS];
    __shared__ int64_t s_scan[KA_WARPS], s_start, s_base;
    __shared__ int s_b, s_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int H = p.cache.heads;
    const int upb = H * p.row_tiles;               // units per sequence
    const int NS = p.stages;

    if (tid < KA_WARPS * NS)
        mbar_init(smem_u32(&s_bar[tid]), 1);
    if (tid == 0)
        mbar_init_fence();
    pdl_wait();

    // ---- the work list: chunks in all, and where this CTA's share begins
    int64_t total;
    {
        const int per = (p.seqs + KA_THREADS - 1) / KA_THREADS;
        const int first = tid * per;
        int64_t mine = 0;
        for (int i = first; i < first + per && i < p.seqs; ++i) {
            int64_t len = p.prefix_len > 0 ? p.prefix_len : p.lengths[i];
            if (len > p.cap) {
                len = p.cap;
                if (blockIdx.x == 0)
                    atomicOr(p.err, kErrIndex);
            }
            const int n = len < 0 ? 0 : (int)len;
            s_len[i] = n;
            mine += kv_chunks_of(n);
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += u;
        }
        if (lane == 31)
            s_scan[warp] = incl;
        __syncthreads();
        int64_t before = incl - mine;
        total = 0;
#pragma unroll
        for (int w = 0; w < KA_WARPS; ++w) {
            if (w < warp)
                before += s_scan[w];
            total += s_scan[w];
        }
        total *= upb;
        int64_t share = (total + gridDim.x - 1) / gridDim.x;
        if (share < KA_WARPS)                      // a chunk for each warp: fewer pieces to join
            share = KA_WARPS;
        const int64_t c0 = share * blockIdx.x;
        int64_t at = before * upb;
        if (c0 >= at && c0 < at + mine * upb) {
            int i = first;
            while (at + (int64_t)kv_chunks_of(s_len[i]) * upb <= c0) {
                at += (int64_t)kv_chunks_of(s_len[i]) * upb;
                ++i;
            }
            s_b = i;
            s_base = at;
        }
        s_start = share;
        __syncthreads();
    }
    const int64_t share = s_start;
    const int64_t c0 = share * blockIdx.x;
    const int64_t c1 = c0 + share < total ? c0 + share : total;
    if (c0 >= total) {
        pdl_launch_dependents();
        return;
    }

    // ---- copies: this warp's chunks c0 + warp, + 4, ... through its ring
    KvCursor pc = {s_b, s_base, kv_chunks_of(s_len[s_b])};
    int64_t pf = c0 + warp;                        // next chunk to request
    int p_page = -1, p_blk = 0, p_head = 0;        // its block, looked up one chunk ahead
    const uint32_t ring_base = smem_u32(ring) + (uint32_t)(warp * NS) * STAGE;
    const uint32_t bar_base = smem_u32(&s_bar[warp * NS]);
    auto lookup = [&]() {                          // block of chunk pf for lanes 0 and 1
        p_page = -1;
        if (pf >= c1)
            return;
        while (pf >= pc.base + (int64_t)pc.nch * upb) {
            pc.base += (int64_t)pc.nch * upb;
            ++pc.b;
            pc.nch = kv_chunks_of(s_len[pc.b]);
        }
        const int unit = kv_unit_of(pf - pc.base, pc.nch);
        const int pos = (int)(pf - pc.base - (int64_t)unit * pc.nch) * KA_CHUNK + (lane & 1) * KV_BLOCK;
        p_head = unit / p.row_tiles;
        if (lane < 2 && pos < s_len[pc.b]) {
            p_page = __ldg(p.table + (int64_t)pc.b * p.table_width + (pos >> p.cache.page_shift));
            p_blk = (pos & ((1 << p.cache.page_shift) - 1)) / KV_BLOCK;
            if (p_page < 0 || p_page >= p.cache.pages) {
                p_page = -1;
                atomicOr(p.err, kErrIndex);
            }
        }
    };
    uint32_t have = 0u;                            // two bits per stage: which blocks came
    auto request = [&](int s) {                    // chunk pf into stage s
        const bool any = pf < c1;
        const unsigned bal = __ballot_sync(0xffffffffu, p_page >= 0) & 3u;
        have = (have & ~(3u << (2 * s))) | (bal << (2 * s));
        if (any && lane == 0)
            mbar_arrive_expect_tx(bar_base + 8u * s, (uint32_t)__popc(bal) * L::BLOCK);
        __syncwarp();
        if (p_page >= 0)
            bulk_copy_g2s(ring_base + (uint32_t)s * STAGE + (uint32_t)lane * L::BLOCK,
                          p.cache.block(p_page, p_blk, p_head, L::BLOCK), L::BLOCK, bar_base + 8u * s);
        pf += KA_WARPS;
        lookup();
    };
    lookup();
    for (int s = 0; s < NS; ++s)
        request(s);

    // ---- units
    KvCursor cur = {s_b, s_base, kv_chunks_of(s_len[s_b])};
    int64_t f = c0;                                // first chunk of the current unit segment
    int64_t mine = c0 + warp;                      // this warp's next chunk
    int stage = 0;
    uint32_t parity = 0u;
    bool alive = true;
    int merge_buf = 0;
    while (f < c1) {
        while (f >= cur.base + (int64_t)cur.nch * upb) {
            cur.base += (int64_t)cur.nch * upb;
            ++cur.b;
            cur.nch = kv_chunks_of(s_len[cur.b]);
        }
        const int unit_in = kv_unit_of(f - cur.base, cur.nch);
        const int64_t u0 = cur.base + (int64_t)unit_in * cur.nch;      // the unit's chunks
        const int64_t u1 = u0 + cur.nch;
        const int64_t seg1 = u1 < c1 ? u1 : c1;
        const int h = unit_in / p.row_tiles;
        const int rt = unit_in - h * p.row_tiles;
        const int len = s_len[cur.b];
        const int row0 = rt * ROWS;                // first row of the tile within its parent
        const int nrows = p.rows - row0 < ROWS ? p.rows - row0 : ROWS;
        const int64_t grow0 = (p.prefix_len > 0 ? 0 : (int64_t)cur.b * p.rows) + row0;   // among all rows

        // ---- q: fp16 fragments, per-row factors and limits
        __syncthreads();                           // the last segment's readers are done
        {
            constexpr int TPR = D / 16;            // threads of a row, 16 columns each
            for (int i = tid; i < ROWS * TPR; i += KA_THREADS) {
                const int r = i / TPR, c16 = i % TPR;
                uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
                const int64_t token = (grow0 + r) / p.group;
                const int gq = (int)(grow0 + r - token * p.group);
                if (r < nrows) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        p.q + token * p.q_stride + (int64_t)(h * p.group + gq) * D + c16 * 16);
                    a = __ldg(src);
                    b = __ldg(src + 1);
                }
                const uint32_t e[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                uint32_t mx = 0u;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    mx = __vmaxu2(mx, e[j] & 0x7fff7fffu);
                uint32_t top = (mx & 0xffffu) > (mx >> 16) ? (mx & 0xffffu) : (mx >> 16);
#pragma unroll
                for (int o = TPR / 2; o >= 1; o >>= 1) {
                    const uint32_t v = __shfl_xor_sync(0xffffffffu, top, o);
                    top = v > top ? v : top;
                }
                // power of two that puts the largest |q| in [2^14, 2^15); none for a row
                // that holds an infinity or a NaN (its result is NaN anyway)
                int ex = top >= 0x7f80u ? 0 : 141 - (int)(top >> 7);
                ex = ex > 126 ? 126 : ex;
                const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
                float sum = 0.f;
                __half *fr = reinterpret_cast<__half *>(s_qf);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float x = ((j & 1) ? __uint_as_float(e[j / 2] & 0xffff0000u)
                                             : bf16_bits_to_f32(e[j / 2] & 0xffffu)) * up;
                    sum += x;
                    const int d = c16 * 16 + j;
                    int ft, ks, lo2, half;         // fragment lane, k-step, second register pair, half
                    if constexpr (L::I8) {         // word of four codes: (0, 1), (2, 3)
                        const int c = d / 16;
                        ft = D == 128 ? c >> 1 : c;
                        ks = (D == 128 ? (c & 1) * 4 : 0) + (d % 16) / 4;
                        lo2 = (d & 2) >> 1;
                        half = d & 1;
                    } else {                       // word of eight codes: (0, 4), (1, 5); (2, 6), (3, 7)
                        const int per = D / 4;     // columns of a lane
                        ft = d / per;
                        ks = (d % per) / 8 * 2 + ((d & 3) >> 1);
                        lo2 = d & 1;
                        half = (d & 4) >> 2;
                    }
                    const int rr = r & 15;
                    fr[(((r / 16) * KS + ks) * 32 + (rr & 7) * 4 + ft) * 8 + (lo2 * 2 + (rr >> 3)) * 2 + half] =
                        __float2half_rn(x);
                }
#pragma unroll
                for (int o = TPR / 2; o >= 1; o >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (c16 == 0) {
                    s_f[r] = p.scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23);
                    s_qsum[r] = sum;
                    int lim = 0;                   // cached tokens (of this list) that the row sees
                    if (r < nrows) {
                        const int64_t seq = token / p.tokens;
                        const int tq = (int)(token - seq * p.tokens);
                        int own = len;             // tokens of its own sequence that the row sees
                        if (p.prefix_len > 0)
                            own = p.lengths[seq] > 0 ? p.lengths[seq] : 0;
                        own += tq + 1 - p.tokens;
                        lim = p.prefix_len > 0 ? p.prefix_len + (own < 0 ? own : 0) : own;
                        lim = lim < 0 ? 0 : lim;
                    }
                    s_lim[r] = lim;
                }
            }
        }
        __syncthreads();
        float fr[2 * MT], qs[2 * MT];
        int lim[2 * MT];
        int lim_min = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            fr[i] = s_f[g + 8 * i];
            qs[i] = L::I8 ? 0.f : s_qsum[g + 8 * i];
            lim[i] = s_lim[g + 8 * i];
            if (g + 8 * i < nrows)
                lim_min = lim[i] < lim_min ? lim[i] : lim_min;
        }
#pragma unroll
        for (int o = 16; o >= 4; o >>= 1) {
            const int v = __shfl_xor_sync(0xffffffffu, lim_min, o);
            lim_min = v < lim_min ? v : lim_min;
        }

        float o_acc[MT][DPL][4];
        float m[2 * MT], l[2 * MT], off[2 * MT];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            off[i] = 0.f;
        }
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int j = 0; j < DPL; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o_acc[a][j][i] = 0.f;
        float vup = 0.f;                           // 2^(13 - E), E the exponent of the largest V scale so far

        // ---- the warp's chunks of this segment
        for (; mine < seg1; mine += KA_WARPS) {
            alive = alive && mbar_wait_warp(bar_base + 8u * stage, parity, p.err);
            if (!alive)                            // a copy never came: the error word says so
                continue;
            const uint32_t st = ring_base + (uint32_t)stage * STAGE;
            const int pos0 = (int)(mine - u0) * KA_CHUNK;
            const uint32_t blocks = (have >> (2 * stage)) & 3u;
            const bool masked = blocks != 3u || pos0 + KA_CHUNK > lim_min;

            // s = q K^T: four 8-token tiles
            float s[MT][4][4];
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[a][n][i] = 0.f;
            constexpr int KW = L::RB / 16;         // words of a lane's part of a K row
            uint32_t kw[4][KW];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int r = (n & 1) * 8 + g;
                const uint32_t blk = st + (uint32_t)(n >> 1) * L::BLOCK;
                if constexpr (KW == 8) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 v = lds128(blk + L::place(r, (2 * t + i) * 16));
                        kw[n][4 * i] = v.x, kw[n][4 * i + 1] = v.y, kw[n][4 * i + 2] = v.z, kw[n][4 * i + 3] = v.w;
                    }
                } else if constexpr (KW == 4) {
                    const uint4 v = lds128(blk + L::place(r, t * 16));
                    kw[n][0] = v.x, kw[n][1] = v.y, kw[n][2] = v.z, kw[n][3] = v.w;
                } else {
                    const uint2 v = lds64(blk + L::place(r, t * 8));
                    kw[n][0] = v.x, kw[n][1] = v.y;
                }
            }
            constexpr int SPW = KS / KW;           // k-steps per word: 1 (int8) or 2 (int4)
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                uint32_t qa[MT][SPW][4];
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int x = 0; x < SPW; ++x) {
                        const uint4 v = s_qf[(a * KS + w * SPW + x) * 32 + lane];
                        qa[a][x][0] = v.x, qa[a][x][1] = v.y, qa[a][x][2] = v.z, qa[a][x][3] = v.w;
                    }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if constexpr (L::I8) {
                        const uint32_t wd = kw[n][w] ^ 0x80808080u;
                        const uint32_t b0 = i8_pair_lo(wd), b1 = i8_pair_hi(wd);
#pragma unroll
                        for (int a = 0; a < MT; ++a)
                            mma_16816(s[a][n], qa[a][0], b0, b1);
                    } else {
                        const uint32_t wd = kw[n][w];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t b0 = i4_pair_lo(wd >> (8 * x)), b1 = i4_pair_hi(wd >> (8 * x));
#pragma unroll
                            for (int a = 0; a < MT; ++a)
                                mma_16816(s[a][n], qa[a][x], b0, b1);
                        }
                    }
                }
            }

            // scales of tokens 2t, 2t + 1 of each tile
            float ks[4][2], km[4][2], vs[4][2], vm[4][2];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint32_t blk = st + (uint32_t)(n >> 1) * L::BLOCK;
                const uint32_t r = (uint32_t)((n & 1) * 8 + 2 * t);
                if constexpr (L::I8) {
                    f16x2_to_f32x2(lds32(blk + L::K_SCALES + 2 * r), ks[n][0], ks[n][1]);
                    f16x2_to_f32x2(lds32(blk + L::V_SCALES + 2 * r), vs[n][0], vs[n][1]);
                } else {
                    const uint2 a = lds64(blk + L::K_SCALES + 4 * r), b = lds64(blk + L::V_SCALES + 4 * r);
                    f16x2_to_f32x2(a.x, ks[n][0], km[n][0]);
                    f16x2_to_f32x2(a.y, ks[n][1], km[n][1]);
                    f16x2_to_f32x2(b.x, vs[n][0], vm[n][0]);
                    f16x2_to_f32x2(b.y, vs[n][1], vm[n][1]);
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!((blocks >> (n >> 1)) & 1u) || pos0 + n * 8 + 2 * t + e >= len)
                                km[n][e] = vm[n][e] = 0.f;
                    }
                }
                if (masked) {                      // what lies past the length may be anything
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (!((blocks >> (n >> 1)) & 1u) || pos0 + n * 8 + 2 * t + e >= len)
                            ks[n][e] = vs[n][e] = 0.f;
                }
                if constexpr (!L::I8) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        km[n][e] = fmaf(8.f, ks[n][e], km[n][e]);
                        vm[n][e] = fmaf(8.f, vs[n][e], vm[n][e]);
                    }
                }
            }

            // running maximum
            float mn[2 * MT];
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                mn[i] = m[i];
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = s[i / 2][n][(i & 1) * 2 + e];
                        if constexpr (L::I8)
                            x = x * (ks[n][e] * fr[i]);
                        else
                            x = fr[i] * fmaf(ks[n][e], x, km[n][e] * qs[i]);
                        if (masked && (pos0 + n * 8 + 2 * t + e >= lim[i] || !((blocks >> (n >> 1)) & 1u)))
                            x = -INFINITY;
                        mn[i] = fmaxf(mn[i], x);
                    }
                mn[i] = fmaxf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], 1));
                mn[i] = fmaxf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], 2));
            }
            float vmx = 0.f;
#pragma unroll
            for (int n = 0; n < 4; ++n)
                vmx = fmaxf(vmx, fmaxf(vs[n][0], vs[n][1]));
            vmx = fmaxf(vmx, __shfl_xor_sync(0xffffffffu, vmx, 1));
            vmx = fmaxf(vmx, __shfl_xor_sync(0xffffffffu, vmx, 2));
            // 2^13 / (power of two below the largest V scale); a zero scale asks for nothing
            const float up = vmx > 0.f ? __uint_as_float((uint32_t)(254 + 13 - (int)(__float_as_uint(vmx) >> 23)) << 23)
                                       : 0x1p+60f;
            float vnew = vup > 0.f ? fminf(vup, up) : up;
            bool grown = vnew != vup;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i)
                grown = grown || mn[i] > m[i];
            if (__any_sync(0xffffffffu, grown)) {
                const float vc = vup > 0.f ? vnew / vup : 0.f;     // both powers of two
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) {
                    const float c = m[i] == -INFINITY ? 0.f : ex2(m[i] - mn[i]);
                    l[i] *= c;
                    off[i] *= c;
                    const float cv = c * vc;
#pragma unroll
                    for (int j = 0; j < DPL; ++j) {
                        o_acc[i / 2][j][(i & 1) * 2] *= cv;
                        o_acc[i / 2][j][(i & 1) * 2 + 1] *= cv;
                    }
                    m[i] = mn[i];
                }
                vup = vnew;
            }

            // p and p vs
            uint32_t pa[MT][2][4];
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                const float ref = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    float pv[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = s[i / 2][n][(i & 1) * 2 + e];
                        const float pr = ex2(x - ref);
                        l[i] += pr;
                        pv[e] = pr * (vs[n][e] * vup);
                        if constexpr (!L::I8) {
                            const float w = pr * vm[n][e];
                            off[i] += masked && x == -INFINITY ? 0.f : w;
                        }
                        if (masked && x == -INFINITY)
                            pv[e] = 0.f;
                    }
                    const __half2 hh = __floats2half2_rn(pv[0], pv[1]);
                    pa[i / 2][n >> 1][(n & 1) * 2 + (i & 1)] = *reinterpret_cast<const uint32_t *>(&hh);
                }
            }

            // o += (p vs) c: two 16-token steps
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const uint32_t blk = st + (uint32_t)kb * L::BLOCK + L::V_CODES;
                constexpr int VW = L::RB / 32;     // words of a lane's part of a V row: 4, 2 or 1
                uint32_t vw[4][VW];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 2 * t + (i & 1) + (i >> 1) * 8;
                    if constexpr (VW == 4) {
                        const uint4 v = lds128(blk + L::place(r, g * 16));
                        vw[i][0] = v.x, vw[i][1] = v.y, vw[i][2] = v.z, vw[i][3] = v.w;
                    } else if constexpr (VW == 2) {
                        const uint2 v = lds64(blk + L::place(r, g * 8));
                        vw[i][0] = v.x, vw[i][1] = v.y;
                    } else {
                        vw[i][0] = lds32(blk + L::place(r, g * 4));
                    }
                }
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    if constexpr (L::I8) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {      // byte pairs (0, 1) and (2, 3) of the word
                            const uint32_t sel = y ? 0x7362u : 0x5140u;
                            const uint32_t x0 = kv_prmt(vw[0][w], vw[1][w], sel) ^ 0x80808080u;
                            const uint32_t x1 = kv_prmt(vw[2][w], vw[3][w], sel) ^ 0x80808080u;
                            const uint32_t b00 = i8_pair_lo(x0), b01 = i8_pair_lo(x1);
                            const uint32_t b10 = i8_pair_hi(x0), b11 = i8_pair_hi(x1);
#pragma unroll
                            for (int a = 0; a < MT; ++a) {
                                mma_16816(o_acc[a][w * 4 + 2 * y], pa[a][kb], b00, b01);
                                mma_16816(o_acc[a][w * 4 + 2 * y + 1], pa[a][kb], b10, b11);
                            }
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {      // low and high half words: nibbles 0-3, 4-7
                            const uint32_t sel = y ? 0x7632u : 0x5410u;
                            const uint32_t x0 = kv_prmt(vw[0][w], vw[1][w], sel);
                            const uint32_t x1 = kv_prmt(vw[2][w], vw[3][w], sel);
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const uint32_t lo0 = i4_pair_lo(x0 >> (8 * z)), lo1 = i4_pair_lo(x1 >> (8 * z));
                                const uint32_t hi0 = i4_pair_hi(x0 >> (8 * z)), hi1 = i4_pair_hi(x1 >> (8 * z));
#pragma unroll
                                for (int a = 0; a < MT; ++a) {
                                    mma_16816(o_acc[a][w * 8 + 4 * y + 2 * z], pa[a][kb], lo0, lo1);
                                    mma_16816(o_acc[a][w * 8 + 4 * y + 2 * z + 1], pa[a][kb], hi0, hi1);
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();                          // every lane has read the stage
            request(stage);
            if (++stage == NS) {
                stage = 0;
                parity ^= 1u;
            }
        }

        // ---- merge the four warps
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            off[i] += __shfl_xor_sync(0xffffffffu, off[i], 1);
            off[i] += __shfl_xor_sync(0xffffffffu, off[i], 2);
            if (t == 0) {
                s_m[warp][g + 8 * i] = m[i];
                s_l[warp][g + 8 * i] = l[i];
                s_off[warp][g + 8 * i] = off[i];
            }
        }
        __syncthreads();
        float mine_f[2 * MT];                      // this warp's factor of each row
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < KA_WARPS; ++w)
                top = fmaxf(top, s_m[w][g + 8 * i]);
            mine_f[i] = m[i] == -INFINITY ? 0.f : ex2(m[i] - top) / vup;
        }
        // Thread (row, n) of the tile owns columns DPL n .. + DPL - 1 of its row.
        const bool whole = u0 >= c0 && u1 <= c1;   // no other CTA has a piece of the unit
        const int slot = 2 * (int)blockIdx.x + (u0 >= c0 ? 1 : 0);
        float rm[MT], rl[MT], ro[MT];
        float acc[MT][DPL];
#pragma unroll
        for (int a = 0; a < MT; ++a) {
            const int r = a * 16 + (tid >> 3);
            rm[a] = -INFINITY;
#pragma unroll
            for (int w = 0; w < KA_WARPS; ++w)
                rm[a] = fmaxf(rm[a], s_m[w][r]);
            rl[a] = ro[a] = 0.f;
#pragma unroll
            for (int w = 0; w < KA_WARPS; ++w) {
                const float c = s_m[w][r] == -INFINITY ? 0.f : ex2(s_m[w][r] - rm[a]);
                rl[a] += c * s_l[w][r];
                ro[a] += c * s_off[w][r];
            }
        }
#pragma unroll
        for (int sl = 0; sl < DPL / 4; ++sl) {
            float4 *buf = s_merge + merge_buf * KA_WARPS * ROWS * 8;
            merge_buf ^= 1;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int x = (i & 1) * 2 + e;
                    buf[(warp * ROWS + g + 8 * i) * 8 + 2 * t + e] =
                        make_float4(o_acc[i / 2][4 * sl][x] * mine_f[i], o_acc[i / 2][4 * sl + 1][x] * mine_f[i],
                                    o_acc[i / 2][4 * sl + 2][x] * mine_f[i], o_acc[i / 2][4 * sl + 3][x] * mine_f[i]);
                }
            __syncthreads();
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                float4 v = make_float4(ro[a], ro[a], ro[a], ro[a]);
#pragma unroll
                for (int w = 0; w < KA_WARPS; ++w) {
                    const float4 x = buf[(w * ROWS + a * 16) * 8 + tid];
                    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
                }
                acc[a][4 * sl] = v.x, acc[a][4 * sl + 1] = v.y, acc[a][4 * sl + 2] = v.z, acc[a][4 * sl + 3] = v.w;
            }
        }

        // ---- store a piece, or the result
        bool finish = whole;
        const int n0 = (tid & 7) * DPL;
        if (!whole) {
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                const int r = a * 16 + (tid >> 3);
                if (r < nrows) {
                    float *dst = p.partial + ((int64_t)slot * p.max_rows + r) * PIECE;
                    if ((tid & 7) == 0)
                        *reinterpret_cast<float2 *>(dst + D) = make_float2(rm[a], rl[a]);
#pragma unroll
                    for (int j = 0; j < DPL; j += 2)
                        *reinterpret_cast<float2 *>(dst + n0 + j) = make_float2(acc[a][j], acc[a][j + 1]);
                }
            }
            __threadfence();
            __syncthreads();
            const int64_t unit = (int64_t)cur.b * upb + unit_in;
            const int first = (int)(u0 / share), last = (int)((u1 - 1) / share);
            if (tid == 0) {
                const unsigned old = atomicAdd(&p.tickets[unit], 1u);
                s_last = old == (unsigned)(last - first);
                if (s_last)
                    p.tickets[unit] = 0u;
            }
            __syncthreads();
            finish = s_last != 0;
            if (finish) {
                __threadfence();
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    const int r = a * 16 + (tid >> 3);
                    rm[a] = -INFINITY;
                    rl[a] = 0.f;
#pragma unroll
                    for (int j = 0; j < DPL; ++j)
                        acc[a][j] = 0.f;
                    if (r >= nrows)
                        continue;
                    // first the maximum, then the sum: no load waits for another
                    const float *src = p.partial + (int64_t)r * PIECE;
                    const int64_t step = (int64_t)2 * p.max_rows * PIECE;      // from CTA to CTA
                    auto piece = [&](int k) { return src + k * step + (k == first ? step / 2 : 0); };
#pragma unroll 8
                    for (int k = first; k <= last; ++k)
                        rm[a] = fmaxf(rm[a], __ldcg(piece(k) + D));
#pragma unroll 4
                    for (int k = first; k <= last; ++k) {
                        const float *sp = piece(k);
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(sp + D));
                        const float c = ml.x == -INFINITY ? 0.f : ex2(ml.x - rm[a]);
                        rl[a] += ml.y * c;
#pragma unroll
                        for (int j = 0; j < DPL; j += 2) {
                            const float2 v = __ldcg(reinterpret_cast<const float2 *>(sp + n0 + j));
                            acc[a][j] += v.x * c;
                            acc[a][j + 1] += v.y * c;
                        }
                    }
                }
            }
        }
        if (finish) {
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                const int r = a * 16 + (tid >> 3);
                if (r >= nrows)
                    continue;
                const int64_t grow = grow0 + r;
                if (p.prefix_len > 0) {            // a piece for the launch over the sequences' own tokens
                    float *dst = p.prefix_out + ((int64_t)h * p.rows + grow) * PIECE;
                    if ((tid & 7) == 0)
                        *reinterpret_cast<float2 *>(dst + D) = make_float2(rm[a], rl[a]);
#pragma unroll
                    for (int j = 0; j < DPL; j += 2)
                        *reinterpret_cast<float2 *>(dst + n0 + j) = make_float2(acc[a][j], acc[a][j + 1]);
                    continue;
                }
                if (p.prefix_in) {
                    const float *src = p.prefix_in + ((int64_t)h * p.batch * p.rows + grow) * PIECE;
                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(src + D));
                    const float top = fmaxf(rm[a], ml.x);
                    const float co = rm[a] == -INFINITY ? 0.f : ex2(rm[a] - top);
                    const float cn = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
                    rl[a] = rl[a] * co + ml.y * cn;
#pragma unroll
                    for (int j = 0; j < DPL; j += 2) {
                        const float2 v = __ldcg(reinterpret_cast<const float2 *>(src + n0 + j));
                        acc[a][j] = acc[a][j] * co + v.x * cn;
                        acc[a][j + 1] = acc[a][j + 1] * co + v.y * cn;
                    }
                }
                // a row that sees nothing has l = 0 and gives zeros
                const float inv = rl[a] == 0.f ? 0.f : 1.f / rl[a];
                const int64_t token = grow / p.group;
                const int gq = (int)(grow - token * p.group);
                uint16_t *dst = p.out + (token * ((int64_t)H * p.group) + (int64_t)h * p.group + gq) * D + n0;
#pragma unroll
                for (int j = 0; j < DPL; j += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = (uint32_t)f32_to_bf16_bits(acc[a][j + 2 * i] * inv) |
                               ((uint32_t)f32_to_bf16_bits(acc[a][j + 2 * i + 1] * inv) << 16);
                    *reinterpret_cast<uint4 *>(dst + j) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
        f = seg1;
    }
    if (!alive)                                    // wait once more for what is still in flight
        for (int s = 0; s < NS; ++s) {
            mbar_wait_warp(bar_base + 8u * stage, parity, p.err);
            if (++stage == NS) {
                stage = 0;
                parity ^= 1u;
            }
        }
    pdl_launch_dependents();
}

// ------------------------------------------------------------------ host side
// Tiles of 16 query rows, or 32 where a key head has more than 16 rows.
static int stream_mt(int64_t rows) { return rows > 16 ? 2 : 1; }

struct StreamPlan {
    int mt, row_tiles, stages, per_sm, grid;
    int64_t rows;                // rows of a unit's parent
    int64_t units;
    size_t smem;
};

static size_t stream_smem(int block, int D, int mt, int stages, int seqs)
{
    return (size_t)KA_WARPS * stages * 2 * block + (size_t)mt * (D / 16) * 32 * 16 +
           (size_t)2 * KA_WARPS * 16 * mt * 8 * 16 + ((size_t)seqs * 4 + 15) / 16 * 16;
}

static StreamPlan stream_plan(const DeviceInfo &dev, const KvCacheDesc &c, int seqs, int64_t rows)
{
    StreamPlan s = {};
    s.rows = rows;
    s.mt = stream_mt(rows);
    s.row_tiles = (int)((rows + 16 * s.mt - 1) / (16 * s.mt));
    s.units = (int64_t)seqs * c.heads * s.row_tiles;
    const int block = kv_block_bytes(c.format, c.head_dim);
    // As many CTAs per SM as registers allow (three with one row tile, two with two) and
    // two stages each fit; then as deep a ring as fits.  4096: static arrays and the
    // CTA's reserve.
    for (s.per_sm = s.mt == 1 ? 3 : 2; s.per_sm >= 1; --s.per_sm) {
        const size_t budget = (dev.smem_optin + 1024) / s.per_sm - 4096;
        for (s.stages = 8; s.stages > 2 && stream_smem(block, c.head_dim, s.mt, s.stages, seqs) > budget;)
            --s.stages;
        s.smem = stream_smem(block, c.head_dim, s.mt, s.stages, seqs);
        if (s.smem <= budget || s.per_sm == 1)
            break;
    }
    s.grid = dev.sms * s.per_sm;
    return s;
}

// Workspace: [counters of the units][pieces] of each of the (one or two) launches, then
// the prefix's results.
struct KvWorkspace {
    size_t tickets[2], pieces[2], prefix, total;
};

static KvWorkspace stream_workspace(const KvCacheDesc &c, const StreamPlan *plans, int n, int64_t prefix_rows)
{
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    KvWorkspace w = {};
    for (int i = 0; i < n; ++i) {
        w.tickets[i] = w.total;
        w.total += up((size_t)plans[i].units * 4);
    }
    for (int i = 0; i < n; ++i) {
        w.pieces[i] = w.total;
        w.total += up((size_t)2 * plans[i].grid * 16 * plans[i].mt * (c.head_dim + 2) * 4);
    }
    w.prefix = w.total;
    w.total += up((size_t)prefix_rows * c.heads * (c.head_dim + 2) * 4);
    return w;
}

static int stream_plans(const DeviceInfo &dev, const KvCacheDesc &c, int batch, int tokens, int q_heads,
                        int prefix_len, StreamPlan (&plans)[2])
{
    const int64_t rows = (int64_t)tokens * (q_heads / c.heads);
    plans[0] = stream_plan(dev, c, batch, rows);
    if (prefix_len <= 0)
        return 1;
    plans[1] = stream_plan(dev, c, 1, rows * batch);
    return 2;
}

size_t kv_attention_workspace_bytes(const DeviceInfo &dev, const KvCacheDesc &c, int batch, int tokens,
                                    int q_heads, int prefix_len)
{
    StreamPlan plans[2];
    const int n = stream_plans(dev, c, batch, tokens, q_heads, prefix_len, plans);
    return stream_workspace(c, plans, n, n == 2 ? plans[1].rows : 0).total;
}

template <int FMT, int D>
static const void *stream_kernel(int mt)
{
    return mt == 1 ? reinterpret_cast<const void *>(&kv_stream_kernel<FMT, D, 1>)
                   : reinterpret_cast<const void *>(&kv_stream_kernel<FMT, D, 2>);
}

static q4_status stream_launch(const KvCacheDesc &c, const StreamPlan &plan, KvStreamParams &p, cudaStream_t st,
                               bool pdl)
{
    const void *k = c.format == Q4_CACHE_INT8
                        ? (c.head_dim == 64 ? stream_kernel<Q4_CACHE_INT8, 64>(plan.mt) : stream_kernel<Q4_CACHE_INT8, 128>(plan.mt))
                        : (c.head_dim == 64 ? stream_kernel<Q4_CACHE_INT4, 64>(plan.mt) : stream_kernel<Q4_CACHE_INT4, 128>(plan.mt));
    p.rows = (int)plan.rows;
    p.row_tiles = plan.row_tiles;
    p.stages = plan.stages;
    p.max_rows = 16 * plan.mt;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan.smem);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaFuncSetAttribute(kv_stream_kernel)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.grid);
    cfg.blockDim = dim3(KA_THREADS);
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    void *args[] = {&p};
    e = cudaLaunchKernelExC(&cfg, k, args);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "launch of kv_stream_kernel");
}

q4_status launch_kv_attention(const DeviceInfo &dev, const KvCacheDesc &c, const KvAttnArgs &a, cudaStream_t st,
                              bool pdl)
{
    StreamPlan plans[2];
    const int n = stream_plans(dev, c, a.batch, a.tokens, a.q_heads, a.prefix_len, plans);
    const KvWorkspace w = stream_workspace(c, plans, n, n == 2 ? plans[1].rows : 0);
    unsigned char *ws = static_cast<unsigned char *>(a.ws);
    KvStreamParams p = {};
    p.cache = KvCache{c.data, c.pages, c.heads, c.page_shift, (1 << c.page_shift) / KV_BLOCK};
    p.q = a.q;
    p.q_stride = a.q_stride;
    p.out = a.out;
    p.lengths = a.lengths;
    p.batch = a.batch;
    p.tokens = a.tokens;
    p.group = a.q_heads / c.heads;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.err = device_error_flags();
    q4_status s;
    if (n == 2) {
        KvStreamParams f = p;
        f.table = a.prefix_pages;
        f.table_width = 0;
        f.cap = a.prefix_len;
        f.seqs = 1;
        f.prefix_len = a.prefix_len;
        f.tickets = reinterpret_cast<unsigned *>(ws + w.tickets[1]);
        f.partial = reinterpret_cast<float *>(ws + w.pieces[1]);
        f.prefix_out = reinterpret_cast<float *>(ws + w.prefix);
        if ((s = stream_launch(c, plans[1], f, st, pdl)) != Q4_OK)
            return s;
        p.prefix_in = f.prefix_out;
    }
    p.table = a.table;
    p.table_width = a.table_width;
    p.cap = (int64_t)a.table_width << c.page_shift;
    p.seqs = a.batch;
    p.tickets = reinterpret_cast<unsigned *>(ws + w.tickets[0]);
    p.partial = reinterpret_cast<float *>(ws + w.pieces[0]);
    return stream_launch(c, plans[0], p, st, pdl);
}

}  // namespace q4
