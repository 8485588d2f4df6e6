// C ABI of the operators around a layer's projections (include/q4.h): host-side validation,
// then the launches of norm_rope.cu, prompt_attention.cu, lora_few.cu,
// lora_shared.cu and lora_many.cu.
#include "layer_ops.h"

namespace q4 {

static bool aligned_to(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
static bool pdl_on() { return (q4_get_launch_flags() & Q4_FLAG_PDL) != 0; }

// Rows of `heads` heads, `stride` elements apart: long enough, and 16-byte accesses.
static bool row_stride_ok(int64_t stride, int64_t row) { return stride >= row && stride % 8 == 0; }

}  // namespace q4

using namespace q4;

extern "C" {

q4_status q4_norm_rope(const void *q, int64_t q_stride, const void *q_weight, void *q_out, int64_t q_out_stride,
                       int q_heads, const void *k, int64_t k_stride, const void *k_weight, void *k_out,
                       int64_t k_out_stride, int kv_heads, const int32_t *positions, const float *inv_freq,
                       int rotary_dim, int interleaved, float eps, int tokens, int head_dim, void *stream)
{
    if (head_dim != 64 && head_dim != 128)
        return fail(Q4_ERR_SHAPE, "head_dim must be 64 or 128 (got %d)", head_dim);
    if (tokens < 1 || q_heads < 0 || kv_heads < 0 || q_heads > 65536 || kv_heads > 65536 || q_heads + kv_heads < 1)
        return fail(Q4_ERR_SHAPE, "tokens=%d must be >= 1, q_heads=%d and kv_heads=%d 0 .. 65536 and not both 0",
                    tokens, q_heads, kv_heads);
    if ((q_heads > 0 && (!q || !q_out)) || (kv_heads > 0 && (!k || !k_out)))
        return fail(Q4_ERR_NULL, "q, q_out, k and k_out must not be NULL where there are heads");
    if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16)
        return fail(Q4_ERR_SHAPE, "rotary_dim must be a multiple of 16, at most head_dim (got %d)", rotary_dim);
    if (rotary_dim > 0 && (!positions || !inv_freq))
        return fail(Q4_ERR_NULL, "positions and inv_freq must not be NULL with a rotation");
    if (interleaved != 0 && interleaved != 1)
        return fail(Q4_ERR_ARG, "interleaved must be 0 or 1 (got %d)", interleaved);
    // (beside squares that leave fp32's range, whose mean is 2.6e36 or more, it has to count for nothing)
    if (!(eps >= 0.f) || !(eps <= 1e30f))
        return fail(Q4_ERR_ARG, "eps must be 0 .. 1e30");
    const int64_t qr = (int64_t)q_heads * head_dim, kr = (int64_t)kv_heads * head_dim;
    if ((q_heads > 0 && (!row_stride_ok(q_stride, qr) || !row_stride_ok(q_out_stride, qr))) ||
        (kv_heads > 0 && (!row_stride_ok(k_stride, kr) || !row_stride_ok(k_out_stride, kr))))
        return fail(Q4_ERR_SHAPE, "strides must be multiples of 8, at least heads * head_dim");
    if ((q_heads > 0 && q == q_out && q_stride != q_out_stride) || (kv_heads > 0 && k == k_out && k_stride != k_out_stride))
        return fail(Q4_ERR_ARG, "in place, input and output have one stride");
    if ((q_heads > 0 && (!aligned_to(q, 16) || !aligned_to(q_out, 16) || !aligned_to(q_weight, 16))) ||
        (kv_heads > 0 && (!aligned_to(k, 16) || !aligned_to(k_out, 16) || !aligned_to(k_weight, 16))) ||
        (rotary_dim > 0 && (!aligned_to(positions, 4) || !aligned_to(inv_freq, 4))))
        return fail(Q4_ERR_ALIGN, "q, k, their outputs and weights must be 16-byte, positions and inv_freq 4-byte aligned");
    if (q_heads > 0 && kv_heads > 0 && (q_out == k_out || q_out == k || k_out == q))
        return fail(Q4_ERR_ARG, "q_out and k_out must be apart from each other and from the other's input");
    DeviceInfo dev;
    const q4_status s = current_device(dev);
    if (s != Q4_OK)
        return s;
    NormRopeArgs a = {};
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.q_out = static_cast<uint16_t *>(q_out);
    a.k_out = static_cast<uint16_t *>(k_out);
    a.q_stride = q_stride, a.k_stride = k_stride, a.q_out_stride = q_out_stride, a.k_out_stride = k_out_stride;
    a.q_weight = static_cast<const uint16_t *>(q_weight);
    a.k_weight = static_cast<const uint16_t *>(k_weight);
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.q_heads = q_heads, a.kv_heads = kv_heads, a.tokens = tokens, a.rotary = rotary_dim;
    a.interleaved = interleaved;
    a.eps = eps;
    return launch_norm_rope(dev, a, head_dim, static_cast<cudaStream_t>(stream), pdl_on());
}

q4_status q4_prompt_attention(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                              int64_t v_stride, const int32_t *offsets, int batch, int tokens, int q_heads, int kv_heads,
                              int head_dim, float scale, void *out, void *stream)
{
    if (!q || !k || !v || !offsets || !out)
        return fail(Q4_ERR_NULL, "q, k, v, offsets and out must not be NULL");
    if (head_dim != 64 && head_dim != 128)
        return fail(Q4_ERR_SHAPE, "head_dim must be 64 or 128 (got %d)", head_dim);
    if (batch < 1 || tokens < 1 || q_heads < 1 || kv_heads < 1)
        return fail(Q4_ERR_SHAPE, "batch=%d, tokens=%d, q_heads=%d and kv_heads=%d must be >= 1", batch, tokens, q_heads,
                    kv_heads);
    if (q_heads % kv_heads || q_heads / kv_heads > 128)
        return fail(Q4_ERR_SHAPE, "q_heads=%d must be a multiple of kv_heads=%d, at most 128 times", q_heads, kv_heads);
    if ((int64_t)tokens * q_heads > 0x7fffffff || (int64_t)batch * kv_heads > 0x3fffffff || batch > 0x7fffff00)
        return fail(Q4_ERR_SHAPE, "tokens * q_heads must stay below 2^31, batch * kv_heads below 2^30");
    const int64_t qr = (int64_t)q_heads * head_dim, kr = (int64_t)kv_heads * head_dim, most = (int64_t)1 << 38;
    if (!row_stride_ok(q_stride, qr) || !row_stride_ok(k_stride, kr) || !row_stride_ok(v_stride, kr) || q_stride > most ||
        k_stride > most || v_stride > most)
        return fail(Q4_ERR_SHAPE, "strides must be multiples of 8, at least heads * head_dim and at most 2^38");
    // (exponents are of 2, so scale log2(e) has to be a number too)
    if (!(scale >= -2e38f) || !(scale <= 2e38f))
        return fail(Q4_ERR_ARG, "scale must be -2e38 .. 2e38");
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(out, 16) || !aligned_to(offsets, 4))
        return fail(Q4_ERR_ALIGN, "q, k, v and out must be 16-byte, offsets 4-byte aligned");
    if (out == q || out == k || out == v)
        return fail(Q4_ERR_ARG, "out must be apart from q, k and v");
    DeviceInfo dev;
    const q4_status s = current_device(dev);
    if (s != Q4_OK)
        return s;
    PromptArgs a = {};
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.out = static_cast<uint16_t *>(out);
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.offsets = offsets;
    a.batch = batch, a.tokens = tokens, a.q_heads = q_heads, a.kv_heads = kv_heads;
    a.scale_log2 = scale * 1.44269504088896341f;
    return launch_prompt_attention(a, head_dim, static_cast<cudaStream_t>(stream), pdl_on());
}

void q4_test_prompt_swap(int blocks)
{
    prompt_set_swap(blocks > 0 && blocks <= 65536 && (blocks & (blocks - 1)) == 0 ? blocks : 0);
}

q4_status q4_lora(const void *x, int64_t x_stride, const void *a, const void *b, const float *scales, int adapters,
                  int rank, const int32_t *offsets, const int32_t *ids, int batch, const void *base,
                  int64_t base_stride, void *out, int64_t out_stride, int tokens, int N, int K, void *stream)
{
    if (!x || !a || !b || !scales || !offsets || !ids || !base || !out)
        return fail(Q4_ERR_NULL, "x, a, b, scales, offsets, ids, base and out must not be NULL");
    if (batch < 1 || tokens < 1 || adapters < 1)
        return fail(Q4_ERR_SHAPE, "batch=%d, tokens=%d and adapters=%d must be >= 1", batch, tokens, adapters);
    if (N < 8 || K < 8 || N % 8 || K % 8)
        return fail(Q4_ERR_SHAPE, "N=%d and K=%d must be multiples of 8", N, K);
    if (rank < 8 || rank > 128 || rank % 8)
        return fail(Q4_ERR_SHAPE, "rank must be a multiple of 8 from 8 to 128 (got %d)", rank);
    if (tokens > 0x07ffffff || batch > 0x07ffffff || N > 0x7fffff00 || K > 0x7fffff00)
        return fail(Q4_ERR_SHAPE, "tokens=%d or batch=%d is above 2^27 - 1, or N=%d or K=%d too large", tokens, batch, N, K);
    const int64_t most = (int64_t)1 << 38;
    if (!row_stride_ok(x_stride, K) || !row_stride_ok(base_stride, N) || !row_stride_ok(out_stride, N) || x_stride > most ||
        base_stride > most || out_stride > most)
        return fail(Q4_ERR_SHAPE, "strides must be multiples of 8, at least K (x) and N (base, out) and at most 2^38");
    if (base == out && base_stride != out_stride)
        return fail(Q4_ERR_ARG, "in place, base and out have one stride");
    if (!aligned_to(x, 16) || !aligned_to(a, 16) || !aligned_to(b, 16) || !aligned_to(base, 16) || !aligned_to(out, 16) ||
        !aligned_to(scales, 4) || !aligned_to(offsets, 4) || !aligned_to(ids, 4))
        return fail(Q4_ERR_ALIGN, "x, a, b, base and out must be 16-byte, scales, offsets and ids 4-byte aligned");
    if (out == x || out == a || out == b)
        return fail(Q4_ERR_ARG, "out must be apart from x, a and b");
    DeviceInfo dev;
    const q4_status s = current_device(dev);
    if (s != Q4_OK)
        return s;
    LoraArgs p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.a = static_cast<const uint16_t *>(a);
    p.b = static_cast<const uint16_t *>(b);
    p.base = static_cast<const uint16_t *>(base);
    p.out = static_cast<uint16_t *>(out);
    p.x_stride = x_stride, p.base_stride = base_stride, p.out_stride = out_stride;
    p.scales = scales;
    p.offsets = offsets, p.ids = ids;
    p.batch = batch, p.tokens = tokens, p.adapters = adapters, p.rank = rank, p.N = N, p.K = K;
    p.err = device_error_flags();
    if (!p.err)                                            // (a wait that runs out writes there)
        return fail(Q4_ERR_CUDA, "the device error word was not found");
    // Which kernel, for the lengths are on the device: the one of eight-token tiles where requests have
    // eight tokens in the mean, or where its CTAs are all on the GPU at once and what their tiles read of the
    // adapters, each anew, stays below 32 MB.  Measured (eight-token tiles, 128-token tiles): 64 requests of 5, rank 64, 14.9
    // against 28 us; 16 of 32, rank 16, 6.4 against 10.8; 16 of 64, rank 64, 18.6 against 12.2; 60 of 50, rank 16, 33
    // against 18.  One kernel has the whole call, also one of single tokens and prompts, where the mean says little:
    // 63 single tokens with an adapter each and a prompt of 400 or of 500 (which goes to the other kernel), K = N = 2048,
    // rank 16, take 10.7 and 15.0 us, the tokens alone 6.4 and the prompts alone 5.6 and 6.4; rank 64 19.5 and 16.5, alone
    // 11.0, 9.9 and 11.3.
    const int64_t tiles = tokens / 8 + batch / 2;
    const bool few = tokens <= 8 * (int64_t)batch ||
                     (tiles <= dev.sms / 2 && tiles * 2 * rank * ((int64_t)N + K) <= 32 << 20);
    if (few && lora_shared_eligible(p))
        return launch_lora_shared(p, static_cast<cudaStream_t>(stream), pdl_on());
    return few ? launch_lora_few(p, static_cast<cudaStream_t>(stream), pdl_on())
               : launch_lora_many(dev, p, static_cast<cudaStream_t>(stream), pdl_on());
}

}  // extern "C"
