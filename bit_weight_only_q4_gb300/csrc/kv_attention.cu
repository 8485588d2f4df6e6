// Attention of T query tokens per sequence over the quantised paged cache.
#include "kv_cache.cuh"

namespace q4 {

// One CTA per (sequence, query token, query head): a tile of 128 tokens at a time,
// each thread scores one token, then each thread owns output columns.
template <int FMT, int D>
__global__ void __launch_bounds__(128) kv_attention_row_kernel(const KvAttnParams p)
{
    using L = KvLayout<FMT, D>;
    __shared__ float s_q[D], s_p[128], s_red[4], s_red2[4];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x;
    const int hq = blockIdx.x % p.q_heads;
    const int64_t bt = blockIdx.x / p.q_heads;
    const int t = (int)(bt % p.tokens), b = (int)(bt / p.tokens);
    const int h = hq / (p.q_heads / p.cache.heads);
    const int64_t cap = (int64_t)p.table_width << p.cache.page_shift;
    int64_t len = p.lengths[b];
    if (len > cap) {
        len = cap;
        if (tid == 0)
            atomicOr(p.err, kErrIndex);
    }
    if (len < 0)
        len = 0;
    const int64_t limit = p.prefix_len + len - p.tokens + t + 1;
    if (tid < D)
        s_q[tid] = bf16_bits_to_f32(p.q[bt * p.q_stride + (int64_t)hq * D + tid]);
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int64_t base = 0; base < limit; base += 128) {
        const int64_t pos = base + tid;
        float s = -INFINITY;
        const uint8_t *blk = nullptr;
        int r = 0;
        auto find = [&](int64_t x) {
            const bool pre = x < p.prefix_len;
            const int64_t y = pre ? x : x - p.prefix_len;
            const int32_t *tab = pre ? p.prefix_pages : p.table + (int64_t)b * p.table_width;
            const int page = tab[y >> p.cache.page_shift];
            r = (int)(y & (KV_BLOCK - 1));
            if (page < 0 || page >= p.cache.pages) {
                atomicOr(p.err, kErrIndex);
                blk = nullptr;
                return;
            }
            blk = p.cache.block(page, (int)(y & ((1 << p.cache.page_shift) - 1)) / KV_BLOCK, h, L::BLOCK);
        };
        if (pos < limit)
            find(pos);
        if (blk) {
            float a = 0.f;
            for (int d = 0; d < D; ++d) {
                if constexpr (L::I8) {
                    a += s_q[d] * (float)(int8_t)blk[L::place(r, d)];
                } else {
                    a += s_q[d] * (f16lo_to_f32(*reinterpret_cast<const uint16_t *>(blk + L::K_SCALES + 4 * r)) *
                                       (float)((blk[L::place(r, d / 2)] >> (4 * (d & 1))) & 15) +
                                   f16lo_to_f32(*reinterpret_cast<const uint16_t *>(blk + L::K_SCALES + 4 * r + 2)));
                }
            }
            if constexpr (L::I8)
                a *= f16lo_to_f32(*reinterpret_cast<const uint16_t *>(blk + L::K_SCALES + 2 * r));
            s = a * p.scale;
        }
        float mt = s;
        for (int o = 16; o >= 1; o >>= 1)
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        if ((tid & 31) == 0)
            s_red[tid >> 5] = mt;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float e = blk ? expf(s - ref) : 0.f;
        s_p[tid] = e;
        float sum = e;
        for (int o = 16; o >= 1; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if ((tid & 31) == 0)
            s_red2[tid >> 5] = sum;
        __syncthreads();
        const float corr = m == -INFINITY ? 0.f : expf(m - ref);
        l = l * corr + s_red2[0] + s_red2[1] + s_red2[2] + s_red2[3];
        acc *= corr;
        m = mn;
        for (int j = 0; j < 128 && base + j < limit && tid < D; ++j) {
            find(base + j);
            if (!blk)
                continue;
            float v;
            if constexpr (L::I8)
                v = (float)(int8_t)blk[L::V_CODES + L::place(r, tid)] *
                    f16lo_to_f32(*reinterpret_cast<const uint16_t *>(blk + L::V_SCALES + 2 * r));
            else
                v = (float)((blk[L::V_CODES + L::place(r, tid / 2)] >> (4 * (tid & 1))) & 15) *
                        f16lo_to_f32(*reinterpret_cast<const uint16_t *>(blk + L::V_SCALES + 4 * r)) +
                    f16lo_to_f32(*reinterpret_cast<const uint16_t *>(blk + L::V_SCALES + 4 * r + 2));
            acc += s_p[j] * v;
        }
        __syncthreads();
    }
    if (tid < D)
        p.out[(bt * p.q_heads + hq) * D + tid] = f32_to_bf16_bits(l > 0.f || l != l ? acc / l : 0.f);
}

size_t kv_attention_workspace_bytes(const DeviceInfo &dev, const KvCacheDesc &c, int batch, int tokens,
                                    int q_heads, int prefix_len)
{
    (void)dev; (void)c; (void)batch; (void)tokens; (void)q_heads; (void)prefix_len;
    return 0;
}

q4_status launch_kv_attention(const DeviceInfo &dev, const KvCacheDesc &c, const KvAttnArgs &a, cudaStream_t st,
                              bool pdl)
{
    (void)dev;
    KvAttnParams p = {};
    p.cache = KvCache{c.data, c.pages, c.heads, c.page_shift, (1 << c.page_shift) / KV_BLOCK};
    p.q = a.q;
    p.q_stride = a.q_stride;
    p.out = a.out;
    p.table = a.table;
    p.table_width = a.table_width;
    p.lengths = a.lengths;
    p.prefix_pages = a.prefix_pages;
    p.prefix_len = a.prefix_len;
    p.tokens = a.tokens;
    p.q_heads = a.q_heads;
    p.scale = a.scale;
    p.err = device_error_flags();
    auto *f = c.format == Q4_CACHE_INT8
                  ? (c.head_dim == 64 ? kv_attention_row_kernel<Q4_CACHE_INT8, 64> : kv_attention_row_kernel<Q4_CACHE_INT8, 128>)
                  : (c.head_dim == 64 ? kv_attention_row_kernel<Q4_CACHE_INT4, 64> : kv_attention_row_kernel<Q4_CACHE_INT4, 128>);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.batch * a.tokens * a.q_heads));
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, f, p);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "launch of kv_attention_row_kernel");
}

}  // namespace q4
