// What the two attention kernels over the paged cache share: parameters, the list of
// work, the copying warp, and the decoding of codes.
//
// kv_attention_few.cuh  at most 16 query rows per key head: tokens are the MMA's M
//                       dimension
// kv_attention_many.cu  more: query rows are its M dimension
//
// Mathematics of both.  For query row i (a query token and one of the heads that share
// a key head) and token j, in units of log2,
//     s_ij = f_i ks_j (q'_i . c_j)                                        int8: K = ks c
//     s_ij = f_i (ks_j (q'_i . (c_j - 8)) + (km_j + 8 ks_j) sum q'_i)     int4: K = ks c + km
// (f carries scale * log2 e), and with p_ij = 2^(s_ij - m_i)
//     o_i = sum_j p_ij vs_j c_j / sum_j p_ij             (int4: c - 8, + p (vm + 8 vs))
// so scales never touch codes, and both products run on codes that are exact in fp16.
// q' is q times a power of two that brings the largest finite value into
// [2^14, 2^15); f undoes it.  p vs enters the second product in fp16 (11 bits).  The
// reference m_i is the largest s_ij + E_j - 6 so far among the tokens that the row sees, with 2^E_j
// the power of two below vs_j: the largest p vs is then about 2^6, whatever scores and scales it is
// made of, and no token that the row does not see has a part in it.  It moves (and what has
// been summed is rescaled) only when that exceeds it by more than 8, so products stay in the
// range of fp16 and keep their 11 bits down to 2^-20 of the largest.  Scores, statistics and sums
// are fp32; pieces of a row are added up by their references, whatever those are.
// A row of the cache whose V scale is not finite counts as one whose K scale is NaN: it
// poisons the query rows that see it and, being kept out of the V operand, no others.
//
// Work.  The cached tokens of every (sequence, tile of query rows, key head) -- a unit --
// are cut into tiles of 128, and all tiles of all units, laid end to end, are dealt out
// evenly to one CTA per SM, wherever the unit boundaries fall: lengths may differ as they
// like, and are read on the device.  A unit that several CTAs share is joined by the last
// of them to arrive, in the order of its pieces, so the result does not depend on timing.
// No CTA waits for another.
#pragma once

#include "kv_cache.cuh"
#include "tc_device.cuh"

namespace q4 {

constexpr int KT_TOKENS = 128;                     // tokens of a tile
constexpr int KT_BLOCKS = KT_TOKENS / KV_BLOCK;
constexpr int KT_UNITS = 32;                       // units described in shared memory at a time (see kv_copy_warp)
constexpr int KT_MAX_STAGES = 8;

struct KvTileParams {
    KvCache cache;
    const uint16_t *q;
    int64_t q_stride;
    uint16_t *out;
    const int32_t *table;        // pages: [seqs][table_width]
    const int32_t *lengths;      // [batch]
    int64_t cap;                 // tokens that a sequence's row of the table can name
    int table_width;
    int seqs;                    // sequences of the work list (1 for the prefix)
    int prefix_len;              // > 0: this launch reads the prefix, for the rows of all sequences
    int tokens, group;           // group: query heads per key head
    KvDivisor by_tokens, by_group;
    int rows;                    // query rows of a sequence (tokens * group), or of all (prefix)
    int all_rows;                // rows of all sequences
    int row_tiles;
    float scale_log2;            // scale * log2(e)
    int stages;
    unsigned *tickets;           // [grid]: of the unit that goes past this CTA's end, if one that begins in it does
    float *piece_o, *piece_ml;   // [2 * grid][tile rows][D], [2 * grid][tile rows][2]: o, and (m, l)
    float *prefix_out_o, *prefix_out_ml;           // [heads][all_rows][D], [..][2]: written (prefix) ...
    const float *prefix_in_o, *prefix_in_ml;       // ... or joined
    unsigned *err;
    int give_up, give_up_tiles;  // (tests) CTA whose copying warp gives up after so many tiles; negative: none
};

// ------------------------------------------------------------------- helpers
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

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t lds16(uint32_t a)
{
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Pairs of fp32 in one 64-bit register: one instruction for two operations.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ void lds_f32x4(uint32_t a, f32x2 &x, f32x2 &y)
{
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(a));
}

// True in one lane of a converged warp.  tcgen05 instructions issued under it take their
// descriptors from uniform registers: an MMA then costs 30 (A in tensor memory) and 52
// cycles (A in shared memory) at N = 16, from a branch of one thread 78 and 119.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Where a wait that has given up is noted: the error word, and a flag of the CTA that
// lets every later wait return at once.  The roles leave their loops when they see it
// (those whose warps meet at barriers by a vote after each wait for a unit: one that was
// never described would not bring them to their end), and nothing is stored after it.
struct KvDead {
    unsigned *err;
    volatile int *flag;
    uint32_t flag_at;            // its shared-memory address
};

// Bounded wait of a whole warp, every lane polling (a phase that is complete costs some 15
// cycles so, and more with one lane polling for the others; waiting warps do not slow
// each other).  Written as one block, for the roles' loops wait in some twenty places
// and have to stay short: the usual way through is two instructions.
__device__ __forceinline__ void kv_wait(uint32_t bar, uint32_t parity, const KvDead &dead)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .u32 n, d;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
                 "@p bra KV_DONE_%=;\n\t"
                 "mov.u32 n, 0;\n"
                 "KV_POLL_%=:\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
                 "@p bra KV_DONE_%=;\n\t"
                 "ld.volatile.shared.u32 d, [%2];\n\t"
                 "setp.ne.u32 p, d, 0;\n\t"
                 "@p bra KV_DONE_%=;\n\t"
                 "add.u32 n, n, 1;\n\t"
                 "setp.lt.u32 p, n, %4;\n\t"
                 "@p bra KV_POLL_%=;\n\t"
                 "st.volatile.shared.u32 [%2], 1;\n\t"
                 "red.global.or.b32 [%3], %5;\n"
                 "KV_DONE_%=:\n\t}"
                 ::"r"(bar), "r"(parity), "r"(dead.flag_at), "l"(dead.err), "n"(kMbarSpinLimit), "n"(kErrBarrierTimeout)
                 : "memory");
    __syncwarp();
}

// A CTA that has given up: the MMAs that this warp's elected lane has issued are waited for,
// so that none runs into the CTA's end.  `bar` has a count of one and is used for this alone.
__device__ __forceinline__ void kv_mma_drain(uint32_t bar, const KvDead &dead)
{
    if (elect_one())
        mma_commit(bar);
    __syncwarp();
    mbar_wait(bar, 0u, dead.err);
}

__device__ __forceinline__ void bar_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ bool bar_or(int id, int threads, bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"(threads), "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// E - 6 for a V scale of v >= 0, see above.  A scale of 0 (a row of one value) makes no product
// that could leave fp16's range, but p alone has a range too: it is added up in l and, times
// vm, in the offset.  At -68 such a p is 2^68 at most, and references move before one reaches 2^76
// (KT_P_TOP): l stays below 2^107 and the offset below 2^123 for any number of tokens.  What weighs
// 2^68 times less than such a row is lost to fp16, no sooner.
__device__ __forceinline__ float kv_scale_level(float v)
{
    return v > 0.f ? (float)((int)(__float_as_uint(v) >> 23) - 133) : -68.f;
}
constexpr float KT_P_TOP = 0x1p76f;

// Largest of each of V values over the 32 lanes (see warp_sum_transpose).
template <int V>
__device__ __forceinline__ float warp_max_transpose(float (&v)[V], int lane, int &idx)
{
    idx = 0;
    int n = V;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        if (n > 1) {
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                if (i < n / 2) {
                    const float send = up ? v[i] : v[i + n / 2];
                    const float keep = up ? v[i + n / 2] : v[i];
                    v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, o));
                }
            }
            if (up)
                idx += n / 2;
            n /= 2;
        } else {
            v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
        }
    }
    return v[0];
}

// Codes as fp16: 16 code bytes (int8: 16 codes, int4: 32) -> 2 or 4 times 8 values.
// int8: a byte with its sign bit flipped is code + 128; as the low byte of an fp16 whose
// high byte is 0x64 that is 1024 + 128 + code.  int4: nibble pairs (0, 4), (1, 5),
// (2, 6), (3, 7) of a word, each minus 8.
template <bool I8>
__device__ __forceinline__ void kv_decode8(uint32_t w0, uint32_t w1, uint32_t (&v)[4])
{
    if constexpr (I8) {
        const uint32_t a = w0 ^ 0x80808080u, b = w1 ^ 0x80808080u;
        v[0] = hadd2_rn(kv_prmt(a, 0x64646464u, 0x4140), 0xE480E480u);         // - 1152
        v[1] = hadd2_rn(kv_prmt(a, 0x64646464u, 0x4342), 0xE480E480u);
        v[2] = hadd2_rn(kv_prmt(b, 0x64646464u, 0x4140), 0xE480E480u);
        v[3] = hadd2_rn(kv_prmt(b, 0x64646464u, 0x4342), 0xE480E480u);
    } else {
        const uint32_t t = w0 >> 8;
        v[0] = hadd2_rn(int4_pair_f16_biased<0x000F000F>(w0), 0xE408E408u);                  // - 1032
        v[1] = hfma2_rn(int4_pair_f16_biased<0x00F000F0>(w0), 0x2C002C00u, 0xD480D480u);     // / 16 - 72
        v[2] = hadd2_rn(int4_pair_f16_biased<0x000F000F>(t), 0xE408E408u);
        v[3] = hfma2_rn(int4_pair_f16_biased<0x00F000F0>(t), 0x2C002C00u, 0xD480D480u);
    }
}

// Column that stands at place x of a decoded row.
template <bool I8>
__host__ __device__ constexpr int kv_column(int x)
{
    return I8 ? x : ((x & ~7) | ((x >> 1) & 3) | ((x & 1) << 2));
}

// A token's scales: ks, km + 8 ks, vs, vm + 8 vs (int8: second and fourth 0).
template <int FMT, int D>
__device__ __forceinline__ float4 kv_scales(uint32_t blk, int r)
{
    using L = KvLayout<FMT, D>;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (L::I8) {
        s.x = f16lo_to_f32(lds16(blk + L::K_SCALES + 2 * r));
        s.z = f16lo_to_f32(lds16(blk + L::V_SCALES + 2 * r));
    } else {
        const uint32_t a = lds32(blk + L::K_SCALES + 4 * r), b = lds32(blk + L::V_SCALES + 4 * r);
        s.x = f16lo_to_f32(a);
        s.y = fmaf(8.f, s.x, f16hi_to_f32(a));
        s.z = f16lo_to_f32(b);
        s.w = fmaf(8.f, s.z, f16hi_to_f32(b));
    }
    if (!(fabsf(s.z) < INFINITY) || !(fabsf(s.w) < INFINITY)) {
        s.x = __uint_as_float(0x7fffffffu);
        s.z = s.w = 0.f;
    }
    return s;
}

// Where a thread finds its token's row of codes in a staged tile, computed once: its 16-byte
// pieces lie at `base` plus the offsets of `piece` (see KvLayout).
template <int FMT, int D>
struct KvRowAt {
    using L = KvLayout<FMT, D>;
    static constexpr int PIECES = L::RB / 16;
    uint32_t base, piece[PIECES];
    __device__ __forceinline__ explicit KvRowAt(int tok)
    {
        const int r = tok & (KV_BLOCK - 1);
        const uint32_t line = (uint32_t)(r * L::RB) & ~127u;
        base = (uint32_t)(tok / KV_BLOCK) * L::BLOCK + line;
#pragma unroll
        for (int j = 0; j < PIECES; ++j)
            piece[j] = (uint32_t)L::place(r, 16 * j) - line;
    }
};

// Where the token's row of fp16 values goes in a tile of 128 tokens: 64-column halves of 128
// rows x 128 bytes, 128-byte swizzle.  As an MMA operand that is K-major with tokens as rows
// and M- or N-major with tokens as K.
struct KvRowTo {
    uint32_t at[8];              // chunks of 8 columns (chunk c + 8 is 16 KB behind chunk c)
    __device__ __forceinline__ explicit KvRowTo(int tok)
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            at[j] = (uint32_t)tok * 128u + ((uint32_t)((j ^ tok) & 7) << 4);
    }
};

template <int FMT, int D>
__device__ __forceinline__ void kv_row_to_tile(uint32_t codes, const KvRowAt<FMT, D> &from, uint32_t tile,
                                               const KvRowTo &to)
{
    using L = KvLayout<FMT, D>;
    constexpr int OUT = L::I8 ? 2 : 4;             // 8-column chunks of a piece
    const uint32_t src = codes + from.base;
#pragma unroll
    for (int j = 0; j < KvRowAt<FMT, D>::PIECES; ++j) {
        const uint4 c = lds128(src + from.piece[j]);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int x = 0; x < OUT; ++x) {
            uint32_t v[4];
            kv_decode8<L::I8>(L::I8 ? w[2 * x] : w[x], L::I8 ? w[2 * x + 1] : 0u, v);
            const int ch = OUT * j + x;
            sts128(tile + to.at[ch & 7] + (uint32_t)(ch >> 3) * (KT_TOKENS * 128u), v[0], v[1], v[2], v[3]);
        }
    }
}

// ------------------------------------------------------------------ work list
// Units in list order: sequence, tile of rows, key head.  A unit's tiles cover the
// tokens that its last row sees.  A sequence's length (len) may go past what its row of the table
// holds (cap): query tokens see by the length, of the tokens that are there.
struct KvWalk {
    int b, rt, len;
    int64_t base;                // first tile of (b, rt, head 0) in the list
    int ntok, nch;               // tokens and tiles of each unit of (b, rt)
};

template <int N>
__device__ __forceinline__ int kv_unit_tokens(const KvTileParams &p, int len, int rt)
{
    int lim = len;
    if (p.prefix_len <= 0 && p.tokens > 1) {
        const int last = (rt + 1) * N < p.rows ? (rt + 1) * N - 1 : p.rows - 1;
        lim += p.by_group(last) + 1 - p.tokens;
    }
    return lim < 0 ? 0 : (lim < p.cap ? lim : (int)p.cap);
}

__device__ __forceinline__ int kv_tiles_of(int ntok)
{
    return ntok > KT_TOKENS ? (ntok + KT_TOKENS - 1) / KT_TOKENS : 1;
}

// What a CTA has of one unit: tiles k0 .. k1 - 1 of its n.
struct KvUnit {
    int b, rt, h, ntok, k0, k1, n;
    int len;                     // length of the sequence (of the prefix)
    int64_t u0;                  // the unit's first tile in the list
};

// This CTA's share of the list.
struct KvShare {
    int64_t share, c0, c1;
    int tiles;
};

__device__ __forceinline__ int kv_length(const KvTileParams &p, int b)
{
    if (p.prefix_len > 0)
        return p.prefix_len;
    const int len = p.lengths[b];
    return len < 0 ? 0 : len;
}

// Tiles of all units of a sequence.
template <int N>
__device__ __forceinline__ int64_t kv_tiles_of_sequence(const KvTileParams &p, int len)
{
    int64_t n = 0;                                 // (a prompt of some millions in one call passes 31 bits)
#pragma unroll 1
    for (int rt = 0; rt < p.row_tiles; ++rt)
        n += kv_tiles_of(kv_unit_tokens<N>(p, len, rt));
    return n * p.cache.heads;
}

// Every warp counts the tiles of all units for itself: no warp waits for another before
// it can start.
template <int N>
__device__ __forceinline__ KvShare kv_share(const KvTileParams &p)
{
    const int lane = threadIdx.x & 31;
    int64_t total = 0;
#pragma unroll 1
    for (int i = lane; i < p.seqs; i += 32)
        total += kv_tiles_of_sequence<N>(p, kv_length(p, i));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        total += __shfl_xor_sync(0xffffffffu, total, o);
    KvShare s;
    s.share = (total >> 31) == 0 ? (int64_t)(((uint32_t)total + gridDim.x - 1) / gridDim.x)
                                 : (total + gridDim.x - 1) / gridDim.x;
    s.c0 = s.share * blockIdx.x;
    s.c1 = s.c0 + s.share < total ? s.c0 + s.share : total;
    s.tiles = s.c1 > s.c0 ? (int)(s.c1 - s.c0) : 0;
    return s;
}

// The sequence that tile c0 of the list lies in (a warp, 32 sequences at a time).
template <int N>
__device__ __forceinline__ KvWalk kv_find(const KvTileParams &p, int64_t c0)
{
    const int lane = threadIdx.x & 31;
    KvWalk w = {};
    int64_t before = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < p.seqs && p.seqs > 1; i0 += 32) {
        const int64_t mine = i0 + lane < p.seqs ? kv_tiles_of_sequence<N>(p, kv_length(p, i0 + lane)) : 0;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += u;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + incl > c0);
        if (past) {
            const int at = __ffs(past) - 1;
            w.b = i0 + at;
            w.base = before + __shfl_sync(0xffffffffu, incl - mine, at);
            break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    w.len = kv_length(p, w.b);
    w.ntok = kv_unit_tokens<N>(p, w.len, 0);
    w.nch = kv_tiles_of(w.ntok);
    return w;
}

// The unit at tile f of the list.
template <int N>
__device__ __forceinline__ KvUnit kv_next_unit(const KvTileParams &p, KvWalk &w, int64_t f, int64_t c1)
{
    const int H = p.cache.heads;
#pragma unroll 1
    while (f >= w.base + (int64_t)w.nch * H) {
        w.base += (int64_t)w.nch * H;
        if (++w.rt == p.row_tiles) {
            w.rt = 0;
            ++w.b;
            w.len = kv_length(p, w.b);
        }
        w.ntok = kv_unit_tokens<N>(p, w.len, w.rt);
        w.nch = kv_tiles_of(w.ntok);
    }
    const uint32_t x = (uint32_t)(f - w.base);     // the host bounds a unit group's tiles
    KvUnit s;
    s.h = (int)(x / (uint32_t)w.nch);
    s.b = w.b;
    s.rt = w.rt;
    s.ntok = w.ntok;
    s.n = w.nch;
    s.len = w.len;
    s.u0 = w.base + (int64_t)s.h * w.nch;
    s.k0 = (int)(f - s.u0);
    s.k1 = c1 - s.u0 < w.nch ? (int)(c1 - s.u0) : w.nch;
    return s;
}

// The copying warp: walks the list, describes each unit to the other warps (slot
// u % KT_UNITS, barrier unit_full), and copies the blocks of each tile into the ring
// (a block is 16 tokens of one head, codes and scales together; the blocks of a page follow
// one another and take one 1-D bulk copy: an SM starts one in some 120 cycles, so that
// single int4 blocks of 2,176 bytes arrive at 5.2 TB/s at most, runs of 8 at 7.1).
// Pages are looked up for four tiles of a unit at once, a block per lane, while the four
// before them are being copied: a look-up takes about as long as the copy of a tile.
// s_valid[stage] says which blocks of the tile there are.
template <int FMT, int D, int N>
__device__ __forceinline__ void kv_copy_warp(const KvTileParams &p, const KvShare &sh, KvUnit *s_unit,
                                             uint32_t unit_full, uint32_t ring, uint32_t *s_valid,
                                             uint32_t raw_full, uint32_t raw_empty, const KvDead &dead)
{
    using L = KvLayout<FMT, D>;
    constexpr uint32_t RAW = KT_BLOCKS * L::BLOCK;
    const int lane = threadIdx.x & 31;
    const int NS = p.stages;
    if (blockIdx.x == 0 && p.prefix_len == 0)      // a length that the table cannot hold
#pragma unroll 1
        for (int b = lane; b < p.seqs; b += 32)
            if (p.lengths[b] > p.cap)
                atomicOr(p.err, kErrIndex);
    if (sh.tiles == 0)
        return;
    KvWalk walk = kv_find<N>(p, sh.c0);
    int64_t f = sh.c0;
    int k = 0, k1 = 0, u = 0, ntok = 0, head = 0;
    const int32_t *table = p.table;
    int page = 0, at_block = 0, at_head = 0, n = 0;        // lane's block of the next tiles, and how many those are
    bool has = false;                              // (not judged by before it is used: the load is on its way)
    const int run = p.cache.blocks < KT_BLOCKS ? p.cache.blocks : KT_BLOCKS;     // blocks of a copy
    const bool starts = (lane & (run - 1)) == 0;
    int s = 0, issued = 0;
    uint32_t round = 1u;                           // parity of the slot's previous release
    const int last = (int)blockIdx.x == p.give_up ? p.give_up_tiles : -1;
    int i = 0;
#pragma unroll 1
    while (i < sh.tiles && i != last && !*dead.flag) {
        // the blocks looked up in the last round
        const uint8_t *from = nullptr;
        if (has && page >= 0 && page < p.cache.pages)
            from = p.cache.block(page, at_block, at_head, L::BLOCK);
        else if (has)
            atomicOr(p.err, kErrIndex);
        const unsigned valid = __ballot_sync(0xffffffffu, from != nullptr);
        const int m = n;
        // the next ones
        if (k == k1 && f < sh.c1) {
            const KvUnit un = kv_next_unit<N>(p, walk, f, sh.c1);
            if (lane == 0) {
                s_unit[u & (KT_UNITS - 1)] = un;
                mbar_arrive(unit_full + 8u * (u & (KT_UNITS - 1)));
            }
            ++u;
            k = un.k0, k1 = un.k1, ntok = un.ntok, head = un.h;
            f += k1 - k;
            table = p.table + (int64_t)un.b * p.table_width;
        }
        n = k1 - k < 4 ? k1 - k : 4;
        const int pos = k * KT_TOKENS + lane * KV_BLOCK;
        has = lane < n * KT_BLOCKS && pos < ntok;
        if (has)
            page = __ldg(table + (pos >> p.cache.page_shift));
        at_block = (pos & ((1 << p.cache.page_shift) - 1)) / KV_BLOCK;
        at_head = head;
        k += n;
#pragma unroll 1
        for (int j = 0; j < m && i != last; ++j, ++i) {
            if (i >= NS)
                kv_wait(raw_empty + 8u * s, round, dead);
            const unsigned blocks = (valid >> (8 * j)) & 0xffu;
            if (lane == 0) {
                s_valid[s] = blocks;
                mbar_arrive_expect_tx(raw_full + 8u * s, (uint32_t)__popc(blocks) * L::BLOCK);
            }
            __syncwarp();
            if (from && starts && (lane >> 3) == j)        // (a run's missing blocks are its last)
                bulk_copy_g2s(ring + (uint32_t)s * RAW + (uint32_t)(lane & 7) * L::BLOCK, from,
                              (uint32_t)__popc((blocks >> (lane & 7)) & ((1u << run) - 1u)) * L::BLOCK, raw_full + 8u * s);
            issued = i + 1;
            if (++s == NS)
                s = 0, round ^= 1u;
        }
    }
    if (i == last) {
        if (lane == 0) {
            *dead.flag = 1;
            atomicOr(p.err, kErrBarrierTimeout);
        }
        __syncwarp();
    }
    // Every copy has been waited for by those who read it, unless one of them has left
    // early: then wait here, once more with a limit, before the CTA can exit.
    if (*dead.flag)
#pragma unroll 1
        for (i = issued > NS ? issued - NS : 0; i < issued; ++i)
#pragma unroll 1
            for (uint32_t w = 0; w < kMbarSpinLimit / 64 && !mbar_try_wait(raw_full + 8u * (i % NS), (i / NS) & 1); ++w)
                ;
}

// A row's sums relative to its reference: add what another piece has.
struct KvRowSum {
    float m, l;
    float4 o;
    __device__ __forceinline__ void add(float2 ml, float4 x)
    {
        const float top = fmaxf(m, ml.x);
        const float ca = m == -INFINITY ? 0.f : ex2(m - top);
        const float cb = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
        o.x = o.x * ca + x.x * cb, o.y = o.y * ca + x.y * cb;
        o.z = o.z * ca + x.z * cb, o.w = o.w * ca + x.w * cb;
        l = l * ca + ml.y * cb;
        m = top;
    }
};

// Stores four columns of a finished row: of the prefix's results, or, with those added, of
// the output.
template <int D>
__device__ __forceinline__ void kv_store4(const KvTileParams &p, int grow, int h, int c4, KvRowSum r)
{
    const int64_t at = (int64_t)h * p.all_rows + grow;
    if (p.prefix_len > 0) {                        // a piece for the launch over the sequences' own tokens
        *reinterpret_cast<float4 *>(p.prefix_out_o + at * D + c4 * 4) = r.o;
        if (c4 == 0)
            *reinterpret_cast<float2 *>(p.prefix_out_ml + at * 2) = make_float2(r.m, r.l);
        return;
    }
    if (p.prefix_in_o)
        r.add(__ldcg(reinterpret_cast<const float2 *>(p.prefix_in_ml + at * 2)),
              __ldcg(reinterpret_cast<const float4 *>(p.prefix_in_o + at * D + c4 * 4)));
    // a row that sees nothing has l = 0 and gives zeros
    const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
    const int token = p.by_group(grow);
    uint16_t *dst = p.out + ((int64_t)token * p.cache.heads * p.group + h * p.group + grow - token * p.group) * D;
    *reinterpret_cast<uint2 *>(dst + c4 * 4) =
        make_uint2((uint32_t)f32_to_bf16_bits(r.o.x * inv) | ((uint32_t)f32_to_bf16_bits(r.o.y * inv) << 16),
                   (uint32_t)f32_to_bf16_bits(r.o.z * inv) | ((uint32_t)f32_to_bf16_bits(r.o.w * inv) << 16));
}

// Where this CTA's piece of a unit that it does not have whole goes.
__device__ __forceinline__ int64_t kv_piece_slot(const KvUnit &un)
{
    return 2 * (int64_t)blockIdx.x + (un.k0 == 0 ? 1 : 0);
}

// The CTA that a unit begins in, and how many share it.
struct KvSharers {
    int64_t first;
    int n;
    __device__ __forceinline__ KvSharers(const KvShare &sh, const KvUnit &un)
        : first(un.u0 / sh.share), n((int)((un.u0 + un.n - 1) / sh.share - first) + 1) {}
};

// Counts this CTA in at a unit that it does not have whole; true if it is the last of them
// and all have their piece.  Every CTA of a unit is counted, one that has given up with a mark
// (bit 16 and up): the counter is zero again when the launch ends, whatever has happened.
__device__ __forceinline__ bool kv_arrive(const KvTileParams &p, const KvSharers &by, bool failed)
{
    unsigned *tk = p.tickets + by.first;           // (of the units that begin in a CTA only its last goes on)
    const unsigned old = atomicAdd(tk, failed ? 0x10001u : 1u);
    if ((old & 0xffffu) != (unsigned)(by.n - 1))
        return false;
    *tk = 0u;
    return !failed && (old >> 16) == 0u;
}

// Which of a CTA's (at most two) pieces have been counted: bit 1 for one that begins its unit, bit 0 for another.
__device__ __forceinline__ int kv_piece_bit(const KvUnit &un) { return un.k0 == 0 ? 2 : 1; }

// A CTA that has given up: counted in, with the mark, where it has not been yet (a warp).
template <int N>
__device__ __forceinline__ void kv_arrive_failed(const KvTileParams &p, int counted)
{
    const KvShare sh = kv_share<N>(p);
    if (sh.tiles == 0)
        return;
    KvWalk walk = kv_find<N>(p, sh.c0);
#pragma unroll 1
    for (int64_t f = sh.c0; f < sh.c1;) {
        const KvUnit un = kv_next_unit<N>(p, walk, f, sh.c1);
        f += un.k1 - un.k0;
        if (un.k1 - un.k0 < un.n && !(counted & kv_piece_bit(un)) && (threadIdx.x & 31) == 0)
            kv_arrive(p, KvSharers(sh, un), true);
    }
}

// The piece is written: if it is the unit's last to arrive, join all of them in order and
// store the rows.  Called by NT threads that meet at barrier `bar`, with IT items a thread in flight.
template <int D, int TILE, int NT, int IT>
__device__ __forceinline__ void kv_join(const KvTileParams &p, const KvShare &sh, const KvUnit &un, int nrows, int grow0,
                                        int *s_last, int *s_counted, int t, int bar)
{
    __threadfence();
    const KvSharers by(sh, un);                    // (before the barrier: two long divisions)
    bar_sync(bar, NT);
    if (t == 0) {
        *s_counted |= kv_piece_bit(un);
        *s_last = kv_arrive(p, by, false);
    }
    bar_sync(bar, NT);
    if (!*s_last)
        return;
    const int64_t first = by.first;
    const int np = by.n;
    __threadfence();
    // IT items (four columns of a row) at a time, two pieces of each: the loads are what
    // this takes, and they have to be in flight together.  Piece j lies in slot
    // 2 (first + j), the first one in the slot behind.
    const int total = nrows * (D / 4);
#pragma unroll 1
    for (int item = t; item < total; item += NT * IT) {
        KvRowSum r[IT];
        const float *so[IT], *sml[IT];
#pragma unroll
        for (int y = 0; y < IT; ++y) {
            const int x = item + y * NT < total ? item + y * NT : item;
            const int64_t at = 2 * first * TILE + x / (D / 4);
            so[y] = p.piece_o + at * D + x % (D / 4) * 4;
            sml[y] = p.piece_ml + at * 2;
            r[y] = KvRowSum{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        }
#pragma unroll 1
        for (int j0 = 0; j0 < np; j0 += 2) {
            float2 ml[2 * IT];
            float4 x[2 * IT];
#pragma unroll
            for (int j = 0; j < 2; ++j) {          // past the end: the last piece again, unused
                const int jj = j0 + j < np ? j0 + j : np - 1;
                const int64_t at = (int64_t)(2 * jj + (jj == 0 ? 1 : 0)) * TILE;
#pragma unroll
                for (int y = 0; y < IT; ++y) {
                    ml[j * IT + y] = __ldcg(reinterpret_cast<const float2 *>(sml[y] + at * 2));
                    x[j * IT + y] = __ldcg(reinterpret_cast<const float4 *>(so[y] + at * D));
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (j0 + j < np)
#pragma unroll
                    for (int y = 0; y < IT; ++y)
                        r[y].add(ml[j * IT + y], x[j * IT + y]);
        }
#pragma unroll
        for (int y = 0; y < IT; ++y) {
            const int x = item + y * NT;
            if (x < total)
                kv_store4<D>(p, grow0 + x / (D / 4), un.h, x % (D / 4), r[y]);
        }
    }
}

// Tokens of the list that row `grow` (among all rows) sees, at most; len: the length of its sequence.
__device__ __forceinline__ int kv_row_limit(const KvTileParams &p, int grow, int len)
{
    const int token = p.by_group(grow);
    const int seq = p.by_tokens(token);
    int own = len;
    if (p.prefix_len > 0)
        own = p.lengths[seq] > 0 ? p.lengths[seq] : 0;
    own += token - seq * p.tokens + 1 - p.tokens;
    const int lim = p.prefix_len > 0 ? p.prefix_len + (own < 0 ? own : 0) : own;
    return lim < 0 ? 0 : lim;
}

__device__ __forceinline__ const uint16_t *kv_q_row(const KvTileParams &p, int grow, int h, int D)
{
    const int token = p.by_group(grow);
    return p.q + token * p.q_stride + (int64_t)(h * p.group + grow - token * p.group) * D;
}

// Initialises barriers first .. first + n - 1 of a CTA with a count each, a lane per
// barrier (at most 32).
__device__ __forceinline__ void kv_init_bars(uint32_t first, int n, uint32_t count)
{
    const int lane = threadIdx.x & 31;
    if (lane < n)
        mbar_init(first + 8u * lane, count);
}

// ------------------------------------------------------------------ host side
struct KvKernel {
    const void *fn;
    int tile;                    // query rows of a tile
    int threads, stages;
    size_t smem;
};

KvKernel kv_few_kernel_int8(const DeviceInfo &dev, int head_dim, int rows);
KvKernel kv_few_kernel_int4(const DeviceInfo &dev, int head_dim, int rows);
KvKernel kv_many_kernel(const DeviceInfo &dev, int format, int head_dim);

}  // namespace q4
