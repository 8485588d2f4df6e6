// C ABI of the paged key/value cache (include/q4.h): host-side validation, then the
// launches of kv_store.cu and kv_attention.cu.
#include <algorithm>

#include "kv_cache.cuh"

namespace q4 {

static bool aligned_to(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxBlocks = 0x7fffffff;

static int log2_exact(int v)
{
    int s = 0;
    while ((1 << s) < v)
        ++s;
    return (1 << s) == v ? s : -1;
}

// Checks and describes a cache.
static q4_status kv_describe(const uint8_t *cache, int format, int pages, int page_size, int kv_heads,
                             int head_dim, KvCacheDesc &d)
{
    if (!cache)
        return fail(Q4_ERR_NULL, "cache must not be NULL");
    if (format != Q4_CACHE_INT8 && format != Q4_CACHE_INT4)
        return fail(Q4_ERR_ARG, "unknown cache format %d", format);
    if (head_dim != 64 && head_dim != 128)
        return fail(Q4_ERR_SHAPE, "head_dim must be 64 or 128 (got %d)", head_dim);
    if (pages < 1 || kv_heads < 1)
        return fail(Q4_ERR_SHAPE, "pages=%d and kv_heads=%d must be >= 1", pages, kv_heads);
    const int shift = page_size >= 16 && page_size <= 1024 ? log2_exact(page_size) : -1;
    if (shift < 0)
        return fail(Q4_ERR_SHAPE, "page_size must be a power of two from 16 to 1024 (got %d)", page_size);
    if ((int64_t)pages * kv_heads > kMaxBlocks >> (shift - 4))
        return fail(Q4_ERR_SHAPE, "the cache has more than 2^31 - 1 blocks of 16 tokens and a head");
    if (!aligned_to(cache, 16))
        return fail(Q4_ERR_ALIGN, "cache must be 16-byte aligned");
    d = KvCacheDesc{const_cast<uint8_t *>(cache), format, pages, shift, kv_heads, head_dim};
    return Q4_OK;
}

static bool pdl_on() { return (q4_get_launch_flags() & Q4_FLAG_PDL) != 0; }

static q4_status kv_attention(const void *q, int64_t q_stride, const uint8_t *cache, int format, int pages,
                              int page_size, int kv_heads, int head_dim, const int32_t *prefix_pages,
                              int prefix_len, const int32_t *table, int table_width, const int32_t *lengths,
                              int batch, int tokens, int q_heads, float scale, void *out, void *ws,
                              size_t ws_bytes, void *stream)
{
    KvCacheDesc c;
    q4_status s = kv_describe(cache, format, pages, page_size, kv_heads, head_dim, c);
    if (s != Q4_OK)
        return s;
    if (!q || !table || !lengths || !out)
        return fail(Q4_ERR_NULL, "q, table, lengths and out must not be NULL");
    if (batch < 1 || batch > 8192 || tokens < 1 || table_width < 1)
        return fail(Q4_ERR_SHAPE, "batch=%d (1 .. 8192), tokens=%d and table_width=%d must be >= 1", batch,
                    tokens, table_width);
    if (q_heads < 1 || q_heads % kv_heads)
        return fail(Q4_ERR_SHAPE, "q_heads=%d must be a multiple of kv_heads=%d", q_heads, kv_heads);
    if (q_stride < (int64_t)q_heads * head_dim || q_stride % 8)
        return fail(Q4_ERR_SHAPE, "q_stride must be a multiple of 8, at least q_heads * head_dim");
    if ((int64_t)batch * tokens * q_heads > kMaxBlocks)
        return fail(Q4_ERR_SHAPE, "batch * tokens * q_heads is too large");
    if (((int64_t)table_width << c.page_shift) > kMaxBlocks - prefix_len)
        return fail(Q4_ERR_SHAPE, "table_width * page_size + prefix_len must stay below 2^31");
    // the units of one (sequence, row tile), in tiles of 128 tokens, are counted in 31 bits
    const int64_t most = std::max((int64_t)table_width << c.page_shift, (int64_t)prefix_len);
    if ((most / 128 + 1) * kv_heads > kMaxBlocks)
        return fail(Q4_ERR_SHAPE, "table_width * page_size * kv_heads or prefix_len * kv_heads is too large");
    if (!(scale - scale == 0.f))
        return fail(Q4_ERR_ARG, "scale must be finite");
    if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(table, 4) || !aligned_to(lengths, 4) ||
        !aligned_to(prefix_pages, 4))
        return fail(Q4_ERR_ALIGN, "q and out must be 16-byte, table, lengths and prefix_pages 4-byte aligned");
    DeviceInfo dev;
    if ((s = current_device(dev)) != Q4_OK)
        return s;
    const size_t need = kv_attention_workspace_bytes(dev, c, batch, tokens, q_heads, prefix_len);
    if (need > 0) {
        if (!ws || ws_bytes < need)
            return fail(Q4_ERR_WORKSPACE, "workspace of %zu bytes required, got %zu", need, ws ? ws_bytes : 0);
        if (!aligned_to(ws, 16))
            return fail(Q4_ERR_ALIGN, "workspace must be 16-byte aligned");
    }
    KvAttnArgs a = {};
    a.q = static_cast<const uint16_t *>(q);
    a.q_stride = q_stride;
    a.prefix_pages = prefix_pages;
    a.prefix_len = prefix_len;
    a.table = table;
    a.table_width = table_width;
    a.lengths = lengths;
    a.out = static_cast<uint16_t *>(out);
    a.batch = batch;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.scale = scale;
    a.ws = ws;
    return launch_kv_attention(dev, c, a, static_cast<cudaStream_t>(stream), pdl_on());
}

}  // namespace q4

using namespace q4;

extern "C" {

size_t q4_kv_block_bytes(int format, int head_dim) { return (size_t)kv_block_bytes(format, head_dim); }

q4_status q4_kv_write(const void *k, int64_t k_stride, const void *v, int64_t v_stride, const int32_t *slots,
                      int tokens, uint8_t *cache, int format, int pages, int page_size, int kv_heads,
                      int head_dim, void *stream)
{
    KvCacheDesc c;
    q4_status s = kv_describe(cache, format, pages, page_size, kv_heads, head_dim, c);
    if (s != Q4_OK)
        return s;
    if (!k || !v || !slots)
        return fail(Q4_ERR_NULL, "k, v and slots must not be NULL");
    if (tokens < 1)
        return fail(Q4_ERR_SHAPE, "tokens=%d must be >= 1", tokens);
    const int64_t row = (int64_t)kv_heads * head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8)
        return fail(Q4_ERR_SHAPE, "k and v strides must be multiples of 8, at least kv_heads * head_dim");
    if (((int64_t)tokens + 15) * row / 8 / 256 >= kMaxBlocks)
        return fail(Q4_ERR_SHAPE, "tokens * kv_heads is too large");
    if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(slots, 4))
        return fail(Q4_ERR_ALIGN, "k and v must be 16-byte, slots 4-byte aligned");
    DeviceInfo dev;
    if ((s = current_device(dev)) != Q4_OK)
        return s;
    return launch_kv_write(c, static_cast<const uint16_t *>(k), k_stride, static_cast<const uint16_t *>(v),
                           v_stride, slots, tokens, static_cast<cudaStream_t>(stream), pdl_on());
}

q4_status q4_kv_read(const uint8_t *cache, int format, int pages, int page_size, int kv_heads, int head_dim,
                     const int32_t *table, int table_width, const int32_t *lengths, int batch, int max_len,
                     void *k, void *v, void *stream)
{
    KvCacheDesc c;
    q4_status s = kv_describe(cache, format, pages, page_size, kv_heads, head_dim, c);
    if (s != Q4_OK)
        return s;
    if (!table || !lengths || !k || !v)
        return fail(Q4_ERR_NULL, "table, lengths, k and v must not be NULL");
    if (batch < 1 || max_len < 1 || table_width < 1)
        return fail(Q4_ERR_SHAPE, "batch=%d, max_len=%d and table_width=%d must be >= 1", batch, max_len,
                    table_width);
    if (((int64_t)max_len + 15) / 16 * batch > kMaxBlocks / kv_heads)
        return fail(Q4_ERR_SHAPE, "batch * max_len * kv_heads is too large");
    if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(table, 4) || !aligned_to(lengths, 4))
        return fail(Q4_ERR_ALIGN, "k and v must be 16-byte, table and lengths 4-byte aligned");
    DeviceInfo dev;
    if ((s = current_device(dev)) != Q4_OK)
        return s;
    return launch_kv_read(c, table, table_width, lengths, batch, max_len, static_cast<uint16_t *>(k),
                          static_cast<uint16_t *>(v), static_cast<cudaStream_t>(stream), pdl_on());
}

void q4_test_kv_give_up(int cta, int tiles) { kv_set_give_up(cta, tiles); }

size_t q4_kv_attention_workspace_bytes(int format, int kv_heads, int head_dim, int batch, int tokens,
                                       int q_heads, int prefix_len)
{
    if (kv_block_bytes(format, head_dim) == 0 || kv_heads < 1 || batch < 1 || tokens < 1 || q_heads < 1 ||
        q_heads % kv_heads || prefix_len < 0)
        return 0;
    DeviceInfo dev;
    if (current_device(dev) != Q4_OK)
        return 0;
    const KvCacheDesc c = {nullptr, format, 1, 4, kv_heads, head_dim};
    return kv_attention_workspace_bytes(dev, c, batch, tokens, q_heads, prefix_len);
}

q4_status q4_kv_attention(const void *q, int64_t q_stride, const uint8_t *cache, int format, int pages,
                          int page_size, int kv_heads, int head_dim, const int32_t *table, int table_width,
                          const int32_t *lengths, int batch, int tokens, int q_heads, float scale, void *out,
                          void *ws, size_t ws_bytes, void *stream)
{
    return kv_attention(q, q_stride, cache, format, pages, page_size, kv_heads, head_dim, nullptr, 0, table,
                        table_width, lengths, batch, tokens, q_heads, scale, out, ws, ws_bytes, stream);
}

q4_status q4_kv_attention_shared(const void *q, int64_t q_stride, const uint8_t *cache, int format, int pages,
                                 int page_size, int kv_heads, int head_dim, const int32_t *prefix_pages,
                                 int prefix_len, const int32_t *table, int table_width, const int32_t *lengths,
                                 int batch, int tokens, int q_heads, float scale, void *out, void *ws,
                                 size_t ws_bytes, void *stream)
{
    if (!prefix_pages)
        return fail(Q4_ERR_NULL, "prefix_pages must not be NULL");
    if (prefix_len < 1)
        return fail(Q4_ERR_SHAPE, "prefix_len=%d must be >= 1", prefix_len);
    return kv_attention(q, q_stride, cache, format, pages, page_size, kv_heads, head_dim, prefix_pages,
                        prefix_len, table, table_width, lengths, batch, tokens, q_heads, scale, out, ws,
                        ws_bytes, stream);
}

}  // extern "C"
