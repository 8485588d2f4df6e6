// The paged key/value cache: its storage layout and the device helpers that the
// cache writer, the cache reader and the attention kernels share.
//
// The cache is a byte array [pages][kv_heads][page_size / 16][block].  One block
// holds 16 consecutive tokens of one head, so a block is one contiguous copy and
// carries everything its 16 tokens need:
//     K codes   16 rows of RB bytes (int8: RB = D; int4: RB = D / 2, low nibble =
//               even column)
//     V codes   the same
//     K scales  16 x fp16 scale (int8) or 16 x (fp16 scale, fp16 min) (int4)
//     V scales  the same
// Values: int8 code * scale, code -127 .. 127; int4 code * scale + min, code 0 .. 15.
//
// The code rows are stored in 128-byte lines of eight 16-byte pieces; piece c of
// the line holding row r sits at place c ^ key(r).  A lane of a 16-bit tensor-core
// fragment reads pieces of rows 2t, 2t + 1, 2t + 8, 2t + 9 (V) or of row g (K); with
// this key every such warp-wide read of the staged block touches each shared-memory
// bank once, for the three row sizes that exist (128, 64 and 32 bytes).
#pragma once

#include "q4_device.cuh"
#include "q4_internal.h"

namespace q4 {

constexpr int KV_BLOCK = 16;               // tokens of a block

template <int FMT, int D>
struct KvLayout {
    static constexpr bool I8 = FMT == Q4_CACHE_INT8;
    static constexpr int RB = I8 ? D : D / 2;              // bytes of a code row
    static constexpr int SB = I8 ? 2 : 4;                  // scale bytes of a row
    static constexpr int PART = KV_BLOCK * RB;             // K (or V) codes of a block
    static constexpr int BLOCK = 2 * PART + 2 * KV_BLOCK * SB;
    static constexpr int V_CODES = PART;
    static constexpr int K_SCALES = 2 * PART;
    static constexpr int V_SCALES = 2 * PART + KV_BLOCK * SB;
    static_assert(RB == 128 || RB == 64 || RB == 32, "code rows of 128, 64 or 32 bytes");

    __host__ __device__ static constexpr int key(int r)
    {
        return RB == 128 ? (r & 7) : (RB == 64 ? (r & 6) : ((r >> 1) & 2));
    }
    // Place of byte b of row r within the codes of its block.
    __host__ __device__ static constexpr int place(int r, int b)
    {
        const int lin = r * RB + b;
        return (lin & ~0x70) | ((((lin >> 4) & 7) ^ key(r)) << 4);
    }
};

// Bytes of a block, 0 for a format or head size that does not exist.
inline int kv_block_bytes(int format, int head_dim)
{
    if (head_dim != 64 && head_dim != 128)
        return 0;
    if (format == Q4_CACHE_INT8)
        return 2 * KV_BLOCK * head_dim + 2 * KV_BLOCK * 2;
    if (format == Q4_CACHE_INT4)
        return 2 * KV_BLOCK * (head_dim / 2) + 2 * KV_BLOCK * 4;
    return 0;
}

// ---- paged key/value cache (kv_store.cu, kv_attention.cu; checked by kv_capi.cu)
struct KvCacheDesc {
    uint8_t *data;
    int format, pages, page_shift, heads, head_dim;
};
struct KvAttnArgs {
    const uint16_t *q;
    int64_t q_stride;
    const int32_t *prefix_pages;
    int prefix_len;
    const int32_t *table;
    int table_width;
    const int32_t *lengths;
    uint16_t *out;
    int batch, tokens, q_heads;
    float scale;
    void *ws;
};
// (tests) The CTA of every later launch whose copying warp gives up after `tiles` tiles.
void kv_set_give_up(int cta, int tiles);
q4_status launch_kv_write(const KvCacheDesc &c, const uint16_t *k, int64_t k_stride, const uint16_t *v,
                          int64_t v_stride, const int32_t *slots, int tokens, cudaStream_t st, bool pdl);
q4_status launch_kv_read(const KvCacheDesc &c, const int32_t *table, int table_width, const int32_t *lengths,
                         int batch, int max_len, uint16_t *k, uint16_t *v, cudaStream_t st, bool pdl);
size_t kv_attention_workspace_bytes(const DeviceInfo &dev, const KvCacheDesc &c, int batch, int tokens,
                                    int q_heads, int prefix_len);
q4_status launch_kv_attention(const DeviceInfo &dev, const KvCacheDesc &c, const KvAttnArgs &a, cudaStream_t st,
                              bool pdl);

// Division of 0 <= n < 2^31 by a divisor that a whole launch shares: with 2^s >= d and
// f = ceil(2^(31 + s) / d) < 2^32 the error of n f / 2^(31 + s) stays below 1 / d.
struct KvDivisor {
    uint32_t f, s;
    __host__ __device__ KvDivisor() : f(0), s(0) {}
    __host__ explicit KvDivisor(uint32_t d) : s(0)
    {
        while ((1u << s) < d)
            ++s;
        f = (uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d);
    }
    __device__ __forceinline__ int operator()(int n) const
    {
        return (int)(((uint64_t)(uint32_t)n * f) >> (31 + s));
    }
};

// What the kernels know of a cache.
struct KvCache {
    uint8_t *data;
    int pages, heads;
    int page_shift;            // log2(page_size)
    int blocks;                // page_size / 16

    // First byte of block blk of a page, of head h.  The number of blocks fits in 31 bits (a
    // check of the host's), their bytes do not.
    __device__ __forceinline__ const uint8_t *block(int page, int blk, int h, int block_bytes) const
    {
        return data + (uint64_t)(uint32_t)((page * heads + h) * blocks + blk) * (uint32_t)block_bytes;
    }
};

}  // namespace q4
