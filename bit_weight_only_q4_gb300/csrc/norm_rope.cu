// Norms of queries and keys for each head, and the position rotation, in one pass.
//
// For the D values x of a token's head
//     y = x / sqrt(mean(x^2) + eps) * w
// and of the first R columns the pairs (i, i + R / 2) (or (2 i, 2 i + 1)) are turned by the
// angle position * f_i:
//     (a, b) -> (a cos - b sin, b cos + a sin).
// Everything is fp32 from the bf16 values to one rounding of the result.
//
// Angles.  u = f / 2 pi mod 1 is kept as a 64-bit fraction of a turn; position * u modulo 2^64 is
// then the angle, without the whole turns, by one integer product.  u comes from integers too: f's 24 bits
// times 64 of 1 / 2 pi, cut to 64 behind the point, so that it is off by less than 2^-64 + |f| 2^-67, and the angle by
// 2^31 times that: 2^-24 of a radian at |f| = 256.  The top 32 bits, as fp32 2^-23 at most, go to sincospif.
//
// Layout.  A lane holds eight adjacent columns (one 16-byte access), so a warp takes 256 / D
// heads at a time, and the partner of a pair is a whole lane away: its values come by four
// shuffles of bf16 pairs.  A warp takes one token's heads, or a part of them, for the angles
// are the token's: two a lane, shared through 512 bytes of shared memory.  With them go the weights:
//     y_j = r (x_j (w_j cos_j) + x_p (+-w_p sin_j)),    p the partner,
// and the bracket's factors are worked out once for a token's queries and once for its keys.
//
// What bounds it: HBM, 4 bytes a value (65,000 tokens, 32 and 8 heads of 128: 236 us, 5.6 TB/s), with
// instruction issue close behind (some 130 for 512 bytes).  A few thousand tokens: no one thing (9,446 tokens, 36 heads of 64:
// 20.9 us against 12.9 of HBM).  The SMs are at work for three quarters of the launch; while they are they issue in 68% of
// their cycles, and the rest is the chain that each token begins with, of position, sincospif, factors and
// first loads, which nine passes are too few to hide.  A step: its launch and that chain (48 tokens, 3.0 us).
#include "layer_ops.h"
#include "tc_device.cuh"

namespace q4 {

constexpr int NR_WARPS = 4;
constexpr int NR_BATCH = 2;                // passes over the warp whose loads are in flight together

// u of frequency f (see above) = m 2^(e - 150): 2^64 u = m c 2^(e - 152) with c = 2^66 / 2 pi, rounded to 64 bits; m c has 88.
__device__ __forceinline__ uint64_t nr_turn(float f)
{
    const uint32_t bits = __float_as_uint(f), e = bits >> 23 & 0xffu;
    const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u), c = 0xa2f9836e4e44152aull;
    const uint64_t lo = m * c, hi = __umul64hi(m, c);
    const int right = 152 - (int)(e ? e : 1u);
    uint64_t u;
    if (right >= 64)
        u = right < 128 ? hi >> (right - 64) : 0ull;
    else if (right > 0)
        u = lo >> right | hi << (64 - right);
    else
        u = right > -64 ? lo << -right : 0ull;
    return bits >> 31 ? 0ull - u : u;
}

__device__ __forceinline__ f32x2 nr_widen(uint32_t bf16_pair)
{
    return pack2(__uint_as_float(bf16_pair << 16), __uint_as_float(bf16_pair & 0xffff0000u));
}

__device__ __forceinline__ uint32_t nr_narrow(f32x2 v)
{
    float a, b;
    unpack2(v, a, b);
    return bf16_pair(a, b);
}

template <int LANES>
__device__ __forceinline__ float nr_head_sum(float v)
{
#pragma unroll
    for (int o = LANES / 2; o >= 1; o /= 2)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// What a lane multiplies its columns (own) and their partners (other) by.
struct NrFactors {
    f32x2 own[4], other[4];
};

// Turn and weight of a lane's columns; angle: (cos, sin) of its first column.
template <bool PAIRS>
__device__ __forceinline__ void nr_factors(NrFactors &f, const uint16_t *weight, int l, int partner, bool turned,
                                           float sign, const float2 *angle)
{
    uint4 w = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), p = w;
    if (weight) {
        w = __ldg(reinterpret_cast<const uint4 *>(weight) + l);
        p = PAIRS ? w : __ldg(reinterpret_cast<const uint4 *>(weight) + partner);
    }
    const uint32_t we[4] = {w.x, w.y, w.z, w.w}, pe[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f32x2 c = pack2(1.f, 1.f), s = 0ull;
        if (turned) {
            if (PAIRS) {
                const float2 v = angle[j];
                c = pack2(v.x, v.x), s = pack2(-v.y, v.y);
            } else {
                const float4 v = *reinterpret_cast<const float4 *>(angle + 2 * j);
                c = pack2(v.x, v.z), s = pack2(sign * v.y, sign * v.w);
            }
        }
        const uint32_t o = PAIRS ? __funnelshift_l(pe[j], pe[j], 16) : pe[j];
        f.own[j] = mul2(nr_widen(we[j]), c);
        f.other[j] = mul2(nr_widen(o), s);
    }
}

// PAIRS: adjacent columns are turned together (interleaved).
template <int D, bool PAIRS>
__global__ void __launch_bounds__(NR_WARPS * 32, 6) norm_rope_kernel(const NormRopeArgs a)
{
    constexpr int LANES = D / 8;           // of a head
    constexpr int PER = 32 / LANES;        // heads of a pass
    __shared__ __align__(16) float2 s_angle[NR_WARPS][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % LANES, sub = lane / LANES;
    const int half = a.rotary / 2;

    uint64_t turn[2] = {0ull, 0ull};       // of the lane's two frequencies
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < half)
            turn[i] = nr_turn(__ldg(a.inv_freq + lane + 32 * i));
    // partner lane, and where the lane's angles begin; columns behind R stay as they are
    const bool turned = 8 * l < a.rotary, front = 8 * l < half;
    int partner = lane, first = 4 * l;
    if (!PAIRS && turned) {
        partner = front ? lane + half / 8 : lane - half / 8;
        first = front ? 8 * l : 8 * l - half;
    }
    pdl_wait();

    const int heads = a.q_heads + a.kv_heads;
    const int64_t items = (int64_t)a.tokens * a.parts;
#pragma unroll 1
    for (int64_t item = (int64_t)blockIdx.x * NR_WARPS + warp; item < items; item += (int64_t)gridDim.x * NR_WARPS) {
        const int64_t token = a.parts == 1 ? item : item / a.parts;
        const int part = a.parts == 1 ? 0 : (int)(item - token * a.parts);
        const int h0 = part * a.part_heads, h1 = heads - h0 < a.part_heads ? heads : h0 + a.part_heads;
        if (half > 0) {
            __syncwarp();                  // (the last item's have been read)
            const int position = __ldg(a.positions + token);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (32 * i < half) {
                    const uint64_t t = (uint64_t)(int64_t)position * turn[i];
                    float s, c;
                    sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &s, &c);
                    s_angle[warp][lane + 32 * i] = make_float2(c, s);
                }
            }
            __syncwarp();
        }
        // the part's queries, then its keys
#pragma unroll 1
        for (int kind = 0; kind < 2; ++kind) {
            const int begin = kind ? (h0 > a.q_heads ? h0 - a.q_heads : 0) : h0;
            const int end = kind ? h1 - a.q_heads : (h1 < a.q_heads ? h1 : a.q_heads);
            if (begin >= end)
                continue;
            const uint16_t *weight = kind ? a.k_weight : a.q_weight;
            const uint16_t *in = (kind ? a.k + token * a.k_stride : a.q + token * a.q_stride) + 8 * lane;
            uint16_t *out = (kind ? a.k_out + token * a.k_out_stride : a.q_out + token * a.q_out_stride) + 8 * lane;
            NrFactors f;
            nr_factors<PAIRS>(f, weight, l, partner % LANES, turned, front ? -1.f : 1.f, &s_angle[warp][first]);
            uint4 next[NR_BATCH];
            auto ask = [&](int base) {
#pragma unroll
                for (int i = 0; i < NR_BATCH; ++i) {
                    next[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (base + i * PER + sub < end)
                        next[i] = *reinterpret_cast<const uint4 *>(in + (int64_t)(base + i * PER) * D);
                }
            };
            ask(begin);
#pragma unroll 1
            for (int base = begin; base < end; base += NR_BATCH * PER) {
                uint4 x[NR_BATCH];
#pragma unroll
                for (int i = 0; i < NR_BATCH; ++i)
                    x[i] = next[i];
                ask(base + NR_BATCH * PER);
#pragma unroll
                for (int i = 0; i < NR_BATCH; ++i) {
                    if (base + i * PER >= end)
                        break;             // (the whole warp)
                    uint32_t e[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    float r = 1.f;
                    if (weight) {
                        f32x2 s2 = 0ull;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const f32x2 v = nr_widen(e[j]);
                            s2 = fma2(v, v, s2);
                        }
                        float s, t;
                        unpack2(s2, s, t);
                        const float ss = nr_head_sum<LANES>(s + t);
                        r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
                        const bool large = ss > 3.4e38f, tiny = ss < 0x1p-90f && a.eps < 0x1p-73f;
                        if (__any_sync(0xffffffffu, large || tiny)) {
                            // Squares past fp32's range: their sum from a row 2^100 times smaller, beside which eps is nothing, and
                            // the row 2^34 times smaller, for its products and for bf16's digits of its smaller values; squares that
                            // fp32 has no digits for (beside an eps of 2^-73 they are nothing): a row 2^100 times larger, and
                            // eps 2^200 times, which is below 2^127.
                            const float by = large ? 0x1p-100f : 0x1p100f;
                            s2 = 0ull;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const f32x2 v = mul2(nr_widen(e[j]), pack2(by, by));
                                s2 = fma2(v, v, s2);
                            }
                            unpack2(s2, s, t);
                            const float ss_other = nr_head_sum<LANES>(s + t);
                            if (large || tiny) {
                                const float keep = large ? 0x1p-34f : 0x1p100f;
                                r = rsqrtf(fmaf(ss_other, 1.f / D, large ? 0.f : a.eps * 0x1p100f * 0x1p100f)) *
                                    (large ? 0x1p-66f : 1.f);
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    e[j] = nr_narrow(mul2(nr_widen(e[j]), pack2(keep, keep)));
                            }
                        }
                    }
                    const f32x2 r2 = pack2(r, r);
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        f32x2 y = mul2(nr_widen(e[j]), f.own[j]);
                        if (PAIRS) {
                            if (turned)
                                y = fma2(nr_widen(__funnelshift_l(e[j], e[j], 16)), f.other[j], y);
                        } else {
                            const uint32_t p = __shfl_sync(0xffffffffu, e[j], partner);
                            if (turned)
                                y = fma2(nr_widen(p), f.other[j], y);
                        }
                        o[j] = nr_narrow(mul2(y, r2));
                    }
                    if (base + i * PER + sub < end)
                        *reinterpret_cast<uint4 *>(out + (int64_t)(base + i * PER) * D) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
    pdl_launch_dependents();
}

q4_status launch_norm_rope(const DeviceInfo &dev, NormRopeArgs a, int head_dim, cudaStream_t st, bool pdl)
{
    // A warp takes all heads of a token, or, where that would leave SMs without work, as many as
    // one batch of loads brings.  Measured: 9,446 tokens of 36 heads of 64, whole 20.9, in batches 29.4 us (the angles are
    // worked out for each); 48 tokens of 32 heads of 128 in CTAs of 4 warps 3.3, of 8 warps 4.2 us (with turns from fp64;
    // from integers 3.0).
    const int heads = a.q_heads + a.kv_heads, batch = NR_BATCH * (256 / head_dim);
    a.part_heads = (int64_t)a.tokens >= (int64_t)dev.sms * NR_WARPS * 4 ? heads : batch;
    a.parts = (heads + a.part_heads - 1) / a.part_heads;
    const int64_t ctas = ((int64_t)a.tokens * a.parts + NR_WARPS - 1) / NR_WARPS;
    const int64_t most = (int64_t)dev.sms * 6;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas < most ? ctas : most));
    cfg.blockDim = dim3(NR_WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    void (*kernel)(NormRopeArgs) = nullptr;
    if (a.interleaved)
        kernel = head_dim == 64 ? norm_rope_kernel<64, true> : norm_rope_kernel<128, true>;
    else
        kernel = head_dim == 64 ? norm_rope_kernel<64, false> : norm_rope_kernel<128, false>;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "launch of norm_rope_kernel");
}

}  // namespace q4
