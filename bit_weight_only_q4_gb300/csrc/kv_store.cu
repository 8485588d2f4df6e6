// Quantising K and V rows into the paged cache, and reading cached tokens back.
//
// Both are pure streams: 4 D bytes of bf16 K and V in, 2 D + 4 (int8) or D + 8
// (int4) bytes of cache out per token and head, or the reverse.  Codes and scales are
// those of single IEEE fp32 operations rounded to nearest even:
//   int8   s = fp16(min(amax / 127, 65504)); code = clamp(rint(x / s), -127, 127)
//   int4   s = fp16(min((hi - lo) / 15, 65504)); m = fp16(clamp(lo, +-65504));
//          code = clamp(rint((x - m) / s), 0, 15)
// with code 0 where the fp16 scale is 0.  A row that holds an infinity or a NaN has
// no such scale; its scale (and min) is stored as NaN, so it reads back as NaN.
//
// What bounds them: HBM.  Measured alone in int8, 64,900 tokens of 16 heads of 64 (K and V):
// writing 66 us (402 MB, 6.1 TB/s; 390 warp instructions per 2 KB of rows keep two of three
// issue slots busy, with IEEE divisions it was 148 us), reading 64 us; sixteen contexts of
// 9,000 to 16,384 tokens of 8 heads of 128 read back in 224 us (1.50 GB, 6.7 TB/s).  A
// step's 48 rows of 16 heads of 128: 2.0 us.
#include "kv_cache.cuh"

namespace q4 {

// How the threads of a CTA share the rows of K and V.  The D / 16 threads of a row take 16
// values each, of K and of V, as two chunks of 8: thread j the chunks j and j + D / 16, so
// that a warp's every 16-byte access to bf16 rows and 8- or 4-byte access to codes runs
// through whole sectors (16 neighbouring values a thread left half of each sector to a
// second access).  A CTA takes 16 tokens, one block, of HEADS heads.
template <int D>
struct KvShape {
    static constexpr int TPR = D / 16;                     // threads of a row
    static constexpr int HEADS = 256 / (KV_BLOCK * TPR);
};

struct KvWriteParams {
    const uint16_t *k, *v;       // bf16 rows: token n, head h at n * stride + h * D
    int64_t k_stride, v_stride;
    const int32_t *slots;        // [tokens]; negative: the token is left out
    int tokens;
    int head_groups;             // CTAs that share the heads of 16 tokens
    KvDivisor by_groups;
    KvCache cache;
    unsigned *err;
};

// Elementwise maximum of bf16 pairs, NaN if either is; the larger zero is +0.
__device__ __forceinline__ uint32_t max2_bf16(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t min2_bf16(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// 1 / x to within 2^-22 of itself (x normal).
__device__ __forceinline__ float rcp_near(float x)
{
    float d;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
    return d;
}
__device__ __forceinline__ float bf16_of(const uint32_t (&e)[8], int j)
{
    return (j & 1) ? __uint_as_float(e[j / 2] & 0xffff0000u) : bf16_bits_to_f32(e[j / 2] & 0xffffu);
}

// Quantises 16 values of a row (bf16 pairs e; the row's other threads are the lanes that
// differ in the low bits) and stores codes and, by thread 0 of the row, scales.
//
// The codes are those of IEEE divisions, found with a multiplication by r, which is 1 / s to
// within 2^-22 of itself:
// int8   x has 8 significant bits and s has 11 (S < 2048 in units of its last bit), so x / s
//        is a half-integer or at least 1 / (2 S) > 2^-12 away from every one.  x r is within
//        127 * 2^-22 < 2^-14 of x / s; rounded to a multiple of 2^-12 (by adding 1.5 * 2^11) it
//        is the half-integer where x / s is one, and on the right side of it elsewhere, so the
//        second rounding, to an integer, ends where rint(x / s) does.  In the same way amax / 127
//        is 2^-19 of itself or more away from every value halfway between two of fp16, so that a
//        product with 1 / 127 rounds to the fp16 that the quotient does.
// int4   x - m may have all 24 bits.  n = rint((x - m) r) is right if |(x - m) - n s| < s / 2,
//        which one fused operation judges exactly; else (a tie, or a quotient within an error
//        of one) the thread's codes are computed again with divisions.
// Scales that the fp16 range cuts off leave quotients past the last code: clamped (int8) or
// divided (int4).
template <int FMT, int D>
__device__ __forceinline__ void kv_quantise(const uint32_t (&e)[8], uint8_t *codes, uint8_t *scales, int r, int piece,
                                            bool store)
{
    using L = KvLayout<FMT, D>;
    constexpr int TPR = KvShape<D>::TPR;
    if constexpr (L::I8) {
        uint32_t top = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max2_bf16(top, e[j] & 0x7fff7fffu);
#pragma unroll
        for (int o = TPR / 2; o >= 1; o >>= 1)
            top = max2_bf16(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = max2_bf16(top, top >> 16) & 0xffffu;
        if (!store)
            return;
        const bool bad = top >= 0x7f80u;                   // an infinity or a NaN
        const __half s16 = __float2half_rn(fminf(__fmul_rn(bf16_bits_to_f32(top), 1.f / 127.f), 65504.f));
        const float s = __half2float(s16);
        const float rs = s > 0.f ? rcp_near(s) : 0.f;
        const bool cut = s < 0x1p-14f || s == 65504.f;
        uint32_t w[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                u[j] = __fadd_rn(__fmaf_rn(bf16_of(e, 4 * g + j), rs, 0x1.8p11f), 0x1.8p23f - 0x1.8p11f);
            if (cut)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    u[j] = fminf(fmaxf(u[j], 0x1.8p23f - 127.f), 0x1.8p23f + 127.f);
            w[g] = __byte_perm(__byte_perm(__float_as_uint(u[0]), __float_as_uint(u[1]), 0x0040),
                               __byte_perm(__float_as_uint(u[2]), __float_as_uint(u[3]), 0x0040), 0x5410);
        }
        if (bad)
            w[0] = w[1] = w[2] = w[3] = 0u;
        *reinterpret_cast<uint2 *>(codes + L::place(r, piece * 8)) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(codes + L::place(r, D / 2 + piece * 8)) = make_uint2(w[2], w[3]);
        if (piece == 0)
            *reinterpret_cast<uint16_t *>(scales + 2 * r) = bad ? 0x7fffu : __half_as_ushort(s16);
    } else {
        uint32_t hi2 = e[0], lo2 = e[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            hi2 = max2_bf16(hi2, e[j]);
            lo2 = min2_bf16(lo2, e[j]);
        }
        // [maximum, negated minimum] in one word
        uint32_t both = __byte_perm(max2_bf16(hi2, hi2 >> 16), min2_bf16(lo2, lo2 >> 16), 0x5410) ^ 0x80000000u;
#pragma unroll
        for (int o = TPR / 2; o >= 1; o >>= 1)
            both = max2_bf16(both, __shfl_xor_sync(0xffffffffu, both, o));
        if (!store)
            return;
        const bool bad = (both & 0x7fffu) >= 0x7f80u || (both & 0x7fff0000u) >= 0x7f800000u;
        const float hi = bf16_bits_to_f32(both & 0xffffu), lo = -__uint_as_float(both & 0xffff0000u);
        const __half s16 = __float2half_rn(fminf(__fdiv_rn(__fsub_rn(hi, lo), 15.f), 65504.f));
        const __half m16 = __float2half_rn(fmaxf(fminf(lo, 65504.f), -65504.f));
        const float s = __half2float(s16), m = __half2float(m16);
        uint32_t w[2] = {0u, 0u};
        if (s > 0.f && !bad) {
            const float rs = rcp_near(s);
            float off = 0.f;                               // largest |(x - m) - n s|
#pragma unroll
            for (int g = 0; g < 2; ++g) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = __fsub_rn(bf16_of(e, 8 * g + j), m);
                    const float u = __fmaf_rn(d, rs, 0x1.8p23f);
                    off = fmaxf(off, fabsf(__fmaf_rn(__fsub_rn(0x1.8p23f, u), s, d)));
                    w[g] += __float_as_uint(u) << (4 * j);
                }
                w[g] -= 0x4b400000u * 0x11111111u;         // the bits of 1.5 * 2^23, eight times
            }
            if (!(off < 0.5f * s && s >= 0x1p-14f && s < 65504.f && m == lo)) {
                w[0] = w[1] = 0u;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float q = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(bf16_of(e, j), m), s)), 0.f), 15.f);
                    w[j / 8] |= (uint32_t)(int)q << (4 * (j % 8));
                }
            }
        }
        *reinterpret_cast<uint32_t *>(codes + L::place(r, piece * 4)) = w[0];
        *reinterpret_cast<uint32_t *>(codes + L::place(r, D / 4 + piece * 4)) = w[1];
        if (piece == 0)
            *reinterpret_cast<uint32_t *>(scales + 4 * r) =
                bad ? 0x7fff7fffu : ((uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(m16) << 16));
    }
}

template <int FMT, int D>
__global__ void __launch_bounds__(256) kv_write_kernel(const KvWriteParams p)
{
    using L = KvLayout<FMT, D>;
    using S = KvShape<D>;
    pdl_launch_dependents();
    pdl_wait();
    const int tb = p.by_groups((int)blockIdx.x);           // group of 16 input tokens
    const int piece = threadIdx.x % S::TPR;
    const int h = ((int)blockIdx.x - tb * p.head_groups) * S::HEADS + threadIdx.x / (KV_BLOCK * S::TPR);
    const int64_t n = (int64_t)tb * KV_BLOCK + threadIdx.x / S::TPR % KV_BLOCK;
    const bool here = n < p.tokens && h < p.cache.heads;
    int slot = -1;
    uint32_t ke[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, ve[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (here) {                  // the rows are read beside the slot, not after it
        const uint16_t *k = p.k + n * p.k_stride + h * D + piece * 8, *v = p.v + n * p.v_stride + h * D + piece * 8;
        const uint4 k0 = ld_stream_v4(k), k1 = ld_stream_v4(k + D / 2);
        const uint4 v0 = ld_stream_v4(v), v1 = ld_stream_v4(v + D / 2);
        slot = __ldg(p.slots + n);
        ke[0] = k0.x, ke[1] = k0.y, ke[2] = k0.z, ke[3] = k0.w, ke[4] = k1.x, ke[5] = k1.y, ke[6] = k1.z, ke[7] = k1.w;
        ve[0] = v0.x, ve[1] = v0.y, ve[2] = v0.z, ve[3] = v0.w, ve[4] = v1.x, ve[5] = v1.y, ve[6] = v1.z, ve[7] = v1.w;
        if (slot >= ((int64_t)p.cache.pages << p.cache.page_shift)) {
            slot = -1;
            if (piece == 0 && h == 0)
                atomicOr(p.err, kErrIndex);
        }
    }
    const bool store = slot >= 0;
    const int at = store ? slot : 0;
    const int page = at >> p.cache.page_shift;
    const int tok = at & ((1 << p.cache.page_shift) - 1);
    const int r = tok & (KV_BLOCK - 1);
    uint8_t *blk = const_cast<uint8_t *>(p.cache.block(page, tok / KV_BLOCK, h, L::BLOCK));
    kv_quantise<FMT, D>(ke, blk, blk + L::K_SCALES, r, piece, store);
    kv_quantise<FMT, D>(ve, blk + L::V_CODES, blk + L::V_SCALES, r, piece, store);
}

struct KvReadParams {
    KvCache cache;
    const int32_t *table;        // [batch][table_width] pages of each sequence
    const int32_t *lengths;      // [batch]
    uint16_t *k, *v;             // bf16 [batch][max_len][heads][D]
    int table_width, max_len, block_groups;
    int head_groups;             // CTAs that share the heads of 16 positions
    KvDivisor by_groups, by_blocks;
    unsigned *err;
};

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// 8 values of a row.  int8: byte b = code + 128 in the mantissa of 2^15 + b, from which one
// fused operation takes code * s (2^15 + 128 has 9 bits, so its product with s is exact).
// int4: the code times 16^j in the mantissa of 2^23 (exact), scaled back by s / 16^j.
__device__ __forceinline__ uint4 kv_value8_i8(uint2 c, float s)
{
    const float ms = -32896.f * s;
    const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = __fmaf_rn(__uint_as_float(__byte_perm(w[j / 4], 0x47000000u, 0x7404 | ((j % 4) << 4))), s, ms);
    return make_uint4(bf16x2_of(x[0], x[1]), bf16x2_of(x[2], x[3]), bf16x2_of(x[4], x[5]), bf16x2_of(x[6], x[7]));
}
__device__ __forceinline__ uint4 kv_value8_i4(uint32_t c, float s, float m)
{
    const float sj[4] = {s, s * 0x1p-4f, s * 0x1p-8f, s * 0x1p-12f};
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w = j < 4 ? c : c >> 16;
        x[j] = __fmaf_rn(__fsub_rn(__uint_as_float((w & (15u << (4 * (j % 4)))) | 0x4b000000u), 0x1p23f), sj[j % 4], m);
    }
    return make_uint4(bf16x2_of(x[0], x[1]), bf16x2_of(x[2], x[3]), bf16x2_of(x[4], x[5]), bf16x2_of(x[6], x[7]));
}

// One CTA per (sequence, 16 positions, HEADS heads): it reads that block of its heads and
// writes the 16 rows of bf16 K and V, zeros past the sequence's length.
template <int FMT, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvReadParams p)
{
    using L = KvLayout<FMT, D>;
    using S = KvShape<D>;
    pdl_launch_dependents();
    pdl_wait();
    const int bg = p.by_groups((int)blockIdx.x);
    const int b = p.by_blocks(bg);
    const int pos0 = (bg - b * p.block_groups) * KV_BLOCK;
    const int piece = threadIdx.x % S::TPR;
    const int r = threadIdx.x / S::TPR % KV_BLOCK;
    const int h = ((int)blockIdx.x - bg * p.head_groups) * S::HEADS + threadIdx.x / (KV_BLOCK * S::TPR);
    if (h >= p.cache.heads || pos0 + r >= p.max_len)
        return;
    uint4 k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0, v0 = k0, v1 = k0;
    if (pos0 + r < __ldg(p.lengths + b)) {
        int page = -1;
        if (pos0 < (int64_t)p.table_width << p.cache.page_shift)
            page = __ldg(p.table + (int64_t)b * p.table_width + (pos0 >> p.cache.page_shift));
        if (page >= 0 && page < p.cache.pages) {
            const uint8_t *blk =
                p.cache.block(page, (pos0 & ((1 << p.cache.page_shift) - 1)) / KV_BLOCK, h, L::BLOCK);
            if constexpr (L::I8) {
                const uint8_t *c0 = blk + L::place(r, piece * 8), *c1 = blk + L::place(r, D / 2 + piece * 8);
                const uint2 ck0 = ld_stream_v2(c0), ck1 = ld_stream_v2(c1);
                const uint2 cv0 = ld_stream_v2(c0 + L::V_CODES), cv1 = ld_stream_v2(c1 + L::V_CODES);
                const float ks = f16lo_to_f32(ld_nc_u16(blk + L::K_SCALES + 2 * r));
                const float vs = f16lo_to_f32(ld_nc_u16(blk + L::V_SCALES + 2 * r));
                k0 = kv_value8_i8(ck0, ks), k1 = kv_value8_i8(ck1, ks);
                v0 = kv_value8_i8(cv0, vs), v1 = kv_value8_i8(cv1, vs);
            } else {
                const uint8_t *c0 = blk + L::place(r, piece * 4), *c1 = blk + L::place(r, D / 4 + piece * 4);
                auto word = [](const uint8_t *at) { return __ldg(reinterpret_cast<const uint32_t *>(at)); };
                const uint32_t ck0 = word(c0), ck1 = word(c1);
                const uint32_t cv0 = word(c0 + L::V_CODES), cv1 = word(c1 + L::V_CODES);
                const uint32_t ki = word(blk + L::K_SCALES + 4 * r), vi = word(blk + L::V_SCALES + 4 * r);
                const float ks = f16lo_to_f32(ki), km = f16hi_to_f32(ki), vs = f16lo_to_f32(vi), vm = f16hi_to_f32(vi);
                k0 = kv_value8_i4(ck0, ks, km), k1 = kv_value8_i4(ck1, ks, km);
                v0 = kv_value8_i4(cv0, vs, vm), v1 = kv_value8_i4(cv1, vs, vm);
            }
        } else if (threadIdx.x == 0) {
            atomicOr(p.err, kErrIndex);
        }
    }
    const int64_t at = (((int64_t)b * p.max_len + pos0 + r) * p.cache.heads + h) * D + piece * 8;
    *reinterpret_cast<uint4 *>(p.k + at) = k0;
    *reinterpret_cast<uint4 *>(p.k + at + D / 2) = k1;
    *reinterpret_cast<uint4 *>(p.v + at) = v0;
    *reinterpret_cast<uint4 *>(p.v + at + D / 2) = v1;
}

template <typename P>
static q4_status kv_launch(void (*kernel)(P), const P &p, int64_t blocks, cudaStream_t st, bool pdl,
                           const char *what)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, what);
}

// CTAs that share the heads of 16 tokens (KvShape::HEADS each).
static int kv_head_groups(const KvCacheDesc &c)
{
    const int per = c.head_dim == 64 ? KvShape<64>::HEADS : KvShape<128>::HEADS;
    return (c.heads + per - 1) / per;
}

q4_status launch_kv_write(const KvCacheDesc &c, const uint16_t *k, int64_t k_stride, const uint16_t *v,
                          int64_t v_stride, const int32_t *slots, int tokens, cudaStream_t st, bool pdl)
{
    KvWriteParams p = {};
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.slots = slots;
    p.tokens = tokens;
    p.cache = KvCache{c.data, c.pages, c.heads, c.page_shift, (1 << c.page_shift) / KV_BLOCK};
    p.err = device_error_flags();
    p.head_groups = kv_head_groups(c);
    p.by_groups = KvDivisor((uint32_t)p.head_groups);
    const int64_t blocks = ((int64_t)tokens + KV_BLOCK - 1) / KV_BLOCK * p.head_groups;
    auto *f = c.format == Q4_CACHE_INT8
                  ? (c.head_dim == 64 ? kv_write_kernel<Q4_CACHE_INT8, 64> : kv_write_kernel<Q4_CACHE_INT8, 128>)
                  : (c.head_dim == 64 ? kv_write_kernel<Q4_CACHE_INT4, 64> : kv_write_kernel<Q4_CACHE_INT4, 128>);
    return kv_launch(f, p, blocks, st, pdl, "launch of kv_write_kernel");
}

q4_status launch_kv_read(const KvCacheDesc &c, const int32_t *table, int table_width, const int32_t *lengths,
                         int batch, int max_len, uint16_t *k, uint16_t *v, cudaStream_t st, bool pdl)
{
    KvReadParams p = {};
    p.cache = KvCache{c.data, c.pages, c.heads, c.page_shift, (1 << c.page_shift) / KV_BLOCK};
    p.table = table;
    p.table_width = table_width;
    p.lengths = lengths;
    p.max_len = max_len;
    p.block_groups = (int)(((int64_t)max_len + KV_BLOCK - 1) / KV_BLOCK);
    p.head_groups = kv_head_groups(c);
    p.by_groups = KvDivisor((uint32_t)p.head_groups);
    p.by_blocks = KvDivisor((uint32_t)p.block_groups);
    p.k = k;
    p.v = v;
    p.err = device_error_flags();
    const int64_t blocks = (int64_t)batch * p.block_groups * p.head_groups;
    auto *f = c.format == Q4_CACHE_INT8
                  ? (c.head_dim == 64 ? kv_read_kernel<Q4_CACHE_INT8, 64> : kv_read_kernel<Q4_CACHE_INT8, 128>)
                  : (c.head_dim == 64 ? kv_read_kernel<Q4_CACHE_INT4, 64> : kv_read_kernel<Q4_CACHE_INT4, 128>);
    return kv_launch(f, p, blocks, st, pdl, "launch of kv_read_kernel");
}

}  // namespace q4
