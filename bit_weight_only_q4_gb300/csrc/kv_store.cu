// Quantising K and V rows into the paged cache, and reading cached tokens back.
//
// Both are pure streams: 4 D bytes of bf16 K and V in, 2 D + 4 (int8) or D + 8
// (int4) bytes of cache out per token and head, or the reverse.  Every arithmetic
// step is one IEEE fp32 operation rounded to nearest even, so a row's codes and
// scales are the same whichever kernel or launch shape wrote them:
//   int8   s = fp16(min(amax / 127, 65504)); code = clamp(rint(x / s), -127, 127)
//   int4   s = fp16(min((hi - lo) / 15, 65504)); m = fp16(clamp(lo, +-65504));
//          code = clamp(rint((x - m) / s), 0, 15)
// with code 0 where the fp16 scale is 0.  A row that holds an infinity or a NaN has
// no such scale; its scale (and min) is stored as NaN, so it reads back as NaN.
#include "kv_cache.cuh"

namespace q4 {

struct KvWriteParams {
    const uint16_t *k, *v;       // bf16 rows: token n, head h at n * stride + h * D
    int64_t k_stride, v_stride;
    const int32_t *slots;        // [tokens]; negative: the token is left out
    int64_t items;               // 16-value pieces: tokens * heads * 2 * D / 16
    int tokens;
    KvCache cache;
    unsigned *err;
};

// Sixteen values of a row per thread; the D / 16 threads of a row share its amax or
// min / max by shuffles.  Rows are ordered [head][K, V][token block][token], so a
// block's rows and its 2-byte scales are written by neighbouring threads.
template <int FMT, int D>
__global__ void __launch_bounds__(256) kv_write_kernel(const KvWriteParams p)
{
    using L = KvLayout<FMT, D>;
    constexpr int TPR = D / 16;                    // threads of a row
    pdl_launch_dependents();
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / TPR;
    const int piece = (int)(i % TPR);
    const int64_t per_block = (int64_t)KV_BLOCK * 2 * p.cache.heads;
    const int64_t tb = row / per_block;            // group of 16 input tokens
    const int in = (int)(row - tb * per_block);
    const int64_t n = tb * KV_BLOCK + (in % KV_BLOCK);
    const int kv = (in / KV_BLOCK) & 1;
    const int h = in / (2 * KV_BLOCK);
    int64_t slot = -1;
    if (i < p.items && n < p.tokens) {
        slot = p.slots[n];
        if (slot >= ((int64_t)p.cache.pages << p.cache.page_shift)) {
            slot = -1;
            if (piece == 0 && h == 0 && kv == 0)
                atomicOr(p.err, kErrIndex);
        }
    }
    float x[16];
    uint32_t bad = 0u;
    if (slot >= 0) {
        const uint16_t *src = (kv ? p.v + n * p.v_stride : p.k + n * p.k_stride) + h * D + piece * 16;
        const uint4 a = ld_stream_v4(src), b = ld_stream_v4(src + 8);
        const uint32_t e[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[2 * j] = bf16_bits_to_f32(e[j] & 0xffffu);
            x[2 * j + 1] = __uint_as_float(e[j] & 0xffff0000u);
            bad |= (e[j] & 0x7f80u) == 0x7f80u || (e[j] & 0x7f800000u) == 0x7f800000u;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            x[j] = 0.f;
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) {
        lo = fminf(lo, x[j]);
        hi = fmaxf(hi, x[j]);
    }
#pragma unroll
    for (int o = TPR / 2; o >= 1; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    }
    if (slot < 0)
        return;
    const int page = (int)(slot >> p.cache.page_shift);
    const int tok = (int)(slot & ((1 << p.cache.page_shift) - 1));
    const int r = tok & (KV_BLOCK - 1);
    uint8_t *blk = const_cast<uint8_t *>(p.cache.block(page, tok / KV_BLOCK, h, L::BLOCK));
    uint8_t *codes = blk + (kv ? L::V_CODES : 0);
    uint8_t *scales = blk + (kv ? L::V_SCALES : L::K_SCALES);
    if constexpr (L::I8) {
        const float amax = fmaxf(fabsf(lo), fabsf(hi));
        const __half s16 = __float2half_rn(fminf(__fdiv_rn(amax, 127.f), 65504.f));
        const float s = __half2float(s16);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (s > 0.f && !bad) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float q = fminf(fmaxf(rintf(__fdiv_rn(x[j], s)), -127.f), 127.f);
                w[j / 4] |= ((uint32_t)(int)q & 0xffu) << (8 * (j % 4));
            }
        }
        *reinterpret_cast<uint4 *>(codes + L::place(r, piece * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
        if (piece == 0)
            *reinterpret_cast<uint16_t *>(scales + 2 * r) = bad ? 0x7fffu : __half_as_ushort(s16);
    } else {
        const __half s16 = __float2half_rn(fminf(__fdiv_rn(__fsub_rn(hi, lo), 15.f), 65504.f));
        const __half m16 = __float2half_rn(fmaxf(fminf(lo, 65504.f), -65504.f));
        const float s = __half2float(s16), m = __half2float(m16);
        uint32_t w[2] = {0u, 0u};
        if (s > 0.f && !bad) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float q = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[j], m), s)), 0.f), 15.f);
                w[j / 8] |= (uint32_t)(int)q << (4 * (j % 8));
            }
        }
        *reinterpret_cast<uint2 *>(codes + L::place(r, piece * 8)) = make_uint2(w[0], w[1]);
        if (piece == 0)
            *reinterpret_cast<uint32_t *>(scales + 4 * r) =
                bad ? 0x7fff7fffu : ((uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(m16) << 16));
    }
}

struct KvReadParams {
    KvCache cache;
    const int32_t *table;        // [batch][table_width] pages of each sequence
    const int32_t *lengths;      // [batch]
    uint16_t *k, *v;             // bf16 [batch][max_len][heads][D]
    int table_width, max_len, block_groups;
    unsigned *err;
};

// One CTA per (sequence, 16 positions): it reads that block of every head and
// writes the 16 rows of bf16 K and V, zeros past the sequence's length.
template <int FMT, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvReadParams p)
{
    using L = KvLayout<FMT, D>;
    constexpr int TPR = D / 16;
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.x / p.block_groups;
    const int g = blockIdx.x - b * p.block_groups;         // block of the sequence
    const int pos0 = g * KV_BLOCK;
    const int len = p.lengths[b];
    const int64_t cap = (int64_t)p.table_width << p.cache.page_shift;
    int valid = len - pos0 < p.max_len - pos0 ? len - pos0 : p.max_len - pos0;
    int page = 0;
    if (valid > 0) {
        if (pos0 < cap)
            page = p.table[(int64_t)b * p.table_width + (pos0 >> p.cache.page_shift)];
        if (pos0 >= cap || page < 0 || page >= p.cache.pages) {
            valid = 0;
            if (threadIdx.x == 0)
                atomicOr(p.err, kErrIndex);
        }
    }
    const int blk = (pos0 & ((1 << p.cache.page_shift) - 1)) / KV_BLOCK;
    const int H = p.cache.heads;
    const int rows = p.max_len - pos0 < KV_BLOCK ? p.max_len - pos0 : KV_BLOCK;
    for (int i = threadIdx.x; i < rows * H * TPR * 2; i += 256) {
        const int piece = i % TPR;
        const int h = (i / TPR) % H;
        const int rk = i / (TPR * H);
        const int r = rk % rows, kv = rk / rows;
        uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        if (r < valid) {
            const uint8_t *base = p.cache.block(page, blk, h, L::BLOCK);
            const uint8_t *codes = base + (kv ? L::V_CODES : 0);
            const uint8_t *scales = base + (kv ? L::V_SCALES : L::K_SCALES);
            float x[16];
            if constexpr (L::I8) {
                const uint4 c = ld_stream_v4(codes + L::place(r, piece * 16));
                const float s = f16lo_to_f32(ld_nc_u16(scales + 2 * r));
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    x[j] = __fmul_rn((float)(int8_t)(w[j / 4] >> (8 * (j % 4))), s);
            } else {
                const uint2 c = ld_stream_v2(codes + L::place(r, piece * 8));
                const uint32_t sm = __ldg(reinterpret_cast<const uint32_t *>(scales + 4 * r));
                const float s = f16lo_to_f32(sm), m = f16hi_to_f32(sm);
                const uint32_t w[2] = {c.x, c.y};
#pragma unroll
                for (int j = 0; j < 16; ++j)       // the product is exact in fp32
                    x[j] = __fmaf_rn((float)((w[j / 8] >> (4 * (j % 8))) & 15u), s, m);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = (uint32_t)f32_to_bf16_bits(x[2 * j]) | ((uint32_t)f32_to_bf16_bits(x[2 * j + 1]) << 16);
        }
        uint16_t *dst = (kv ? p.v : p.k) + (((int64_t)b * p.max_len + pos0 + r) * H + h) * D + piece * 16;
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
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
    const int64_t groups = (tokens + KV_BLOCK - 1) / KV_BLOCK;
    p.items = groups * KV_BLOCK * 2 * c.heads * (c.head_dim / 16);
    const int64_t blocks = (p.items + 255) / 256;
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
    p.block_groups = (max_len + KV_BLOCK - 1) / KV_BLOCK;
    p.k = k;
    p.v = v;
    p.err = device_error_flags();
    const int64_t blocks = (int64_t)batch * p.block_groups;
    auto *f = c.format == Q4_CACHE_INT8
                  ? (c.head_dim == 64 ? kv_read_kernel<Q4_CACHE_INT8, 64> : kv_read_kernel<Q4_CACHE_INT8, 128>)
                  : (c.head_dim == 64 ? kv_read_kernel<Q4_CACHE_INT4, 64> : kv_read_kernel<Q4_CACHE_INT4, 128>);
    return kv_launch(f, p, blocks, st, pdl, "launch of kv_read_kernel");
}

}  // namespace q4
