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
// then the angle, without the whole turns, by one integer product.  The error is that of u (f, 1 /
// 2 pi and their product in fp64: 2^-53 of u) times the position: below 2^-24 of a turn for every
// 32-bit position and |f| <= 1.  The top 32 bits go to sincospif.
//
// Layout.  A lane holds eight adjacent columns (one 16-byte access), so a warp takes 256 / D
// heads at a time, and the partner of a pair is a whole lane away: its values come by four
// shuffles of bf16 pairs.  A warp takes one token's heads, or a part of them, for the angles
// are the token's: two a lane, shared through 512 bytes of shared memory.
//
// What bounds it: HBM, 4 bytes a value.
#include "q4_device.cuh"
#include "layer_ops.h"

namespace q4 {

constexpr int NR_WARPS = 8;
constexpr int NR_BATCH = 4;                // passes over the warp whose loads are in flight together

// u of frequency f (see above).
__device__ __forceinline__ uint64_t nr_turn(float f)
{
    double t = (double)f * 0.15915494309189533577;
    t -= floor(t);
    const double hi = floor(t * 4294967296.0);
    const double lo = (t * 4294967296.0 - hi) * 4294967296.0;
    return ((uint64_t)(uint32_t)hi << 32) + (uint64_t)lo;
}

template <int D>
__global__ void __launch_bounds__(NR_WARPS * 32, 3) norm_rope_kernel(const NormRopeArgs a)
{
    constexpr int LANES = D / 8;           // of a head
    constexpr int PER = 32 / LANES;        // heads of a pass
    __shared__ __align__(16) float2 s_angle[NR_WARPS][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % LANES, sub = lane / LANES;
    const int half = a.rotary / 2;

    // what a lane keeps: its columns' weights (and the partner's), its two frequencies
    uint64_t turn[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < half)
            turn[i] = nr_turn(__ldg(a.inv_freq + lane + 32 * i));
    // partner lane and the sign of its part; columns behind R stay as they are
    int partner = lane, first = 0;
    float sign = 0.f;
    const bool turned = 8 * l < a.rotary;
    if (turned && !a.interleaved) {
        const bool front = 8 * l < half;
        partner = front ? lane + half / 8 : lane - half / 8;
        sign = front ? -1.f : 1.f;
        first = front ? 8 * l : 8 * l - half;
    } else if (turned) {
        first = 4 * l;
    }
    const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    const int pl = partner % LANES;
    uint4 wq, wk, pq, pk;
    wq = a.q_weight ? __ldg(reinterpret_cast<const uint4 *>(a.q_weight) + l) : ones;
    wk = a.k_weight ? __ldg(reinterpret_cast<const uint4 *>(a.k_weight) + l) : ones;
    pq = a.q_weight ? __ldg(reinterpret_cast<const uint4 *>(a.q_weight) + pl) : ones;
    pk = a.k_weight ? __ldg(reinterpret_cast<const uint4 *>(a.k_weight) + pl) : ones;
    pdl_wait();

    const int heads = a.q_heads + a.kv_heads;
    const int64_t items = (int64_t)a.tokens * a.parts;
    for (int64_t item = (int64_t)blockIdx.x * NR_WARPS + warp; item < items; item += (int64_t)gridDim.x * NR_WARPS) {
        const int64_t token = a.parts == 1 ? item : item / a.parts;
        const int h0 = (int)(item - token * a.parts) * a.part_heads;
        const int h1 = h0 + a.part_heads < heads ? h0 + a.part_heads : heads;
        const int position = half > 0 ? __ldg(a.positions + token) : 0;
        float cs[8], sn[8];
        bool have = false;
#pragma unroll 1
        for (int base = h0; base < h1; base += NR_BATCH * PER) {
            uint4 x[NR_BATCH];
#pragma unroll
            for (int i = 0; i < NR_BATCH; ++i) {
                const int h = base + i * PER + sub;
                x[i] = make_uint4(0u, 0u, 0u, 0u);
                if (h < h1) {
                    const uint16_t *row = h < a.q_heads ? a.q + token * a.q_stride + (int64_t)h * D
                                                        : a.k + token * a.k_stride + (int64_t)(h - a.q_heads) * D;
                    x[i] = *reinterpret_cast<const uint4 *>(row + 8 * l);
                }
            }
            if (!have && half > 0) {       // (behind the first loads)
                have = true;
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
                if (turned) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i < 2 || !a.interleaved) {
                            const float4 v = *reinterpret_cast<const float4 *>(&s_angle[warp][first + 2 * i]);
                            cs[2 * i] = v.x, sn[2 * i] = v.y, cs[2 * i + 1] = v.z, sn[2 * i + 1] = v.w;
                        }
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < NR_BATCH; ++i) {
                const int h = base + i * PER + sub;
                if (base + i * PER >= h1)  // (the whole warp's)
                    break;
                const bool is_k = h >= a.q_heads;
                uint32_t e[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                float v[8], y[8];
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] = __uint_as_float(e[j] << 16);
                    v[2 * j + 1] = __uint_as_float(e[j] & 0xffff0000u);
                    ss = fmaf(v[2 * j], v[2 * j], ss);
                    ss = fmaf(v[2 * j + 1], v[2 * j + 1], ss);
                }
                const bool norm = is_k ? a.k_weight != nullptr : a.q_weight != nullptr;
#pragma unroll
                for (int o = LANES / 2; o >= 1; o /= 2)
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                float r = rsqrtf(ss * (1.f / D) + a.eps);
                if (__any_sync(0xffffffffu, ss > 3.4e38f)) {
                    // squares past fp32's range: a row 2^100 times smaller, beside which eps is nothing
                    float s2 = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        s2 = fmaf(v[j] * 0x1p-100f, v[j] * 0x1p-100f, s2);
#pragma unroll
                    for (int o = LANES / 2; o >= 1; o /= 2)
                        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
                    if (norm && ss > 3.4e38f) {
                        r = rsqrtf(s2 * (1.f / D));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[2 * j] *= 0x1p-100f, v[2 * j + 1] *= 0x1p-100f;
                            e[j] = (uint32_t)f32_to_bf16_bits(v[2 * j]) | ((uint32_t)f32_to_bf16_bits(v[2 * j + 1]) << 16);
                        }
                    }
                }
                r = norm ? r : 1.f;
                const uint32_t we[4] = {is_k ? wk.x : wq.x, is_k ? wk.y : wq.y, is_k ? wk.z : wq.z, is_k ? wk.w : wq.w};
                const uint32_t pe[4] = {is_k ? pk.x : pq.x, is_k ? pk.y : pq.y, is_k ? pk.z : pq.z, is_k ? pk.w : pq.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y[2 * j] = v[2 * j] * r * __uint_as_float(we[j] << 16);
                    y[2 * j + 1] = v[2 * j + 1] * r * __uint_as_float(we[j] & 0xffff0000u);
                }
                if (half > 0) {
                    if (a.interleaved) {
                        if (turned) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float p = y[2 * j], q = y[2 * j + 1];
                                y[2 * j] = p * cs[j] - q * sn[j];
                                y[2 * j + 1] = q * cs[j] + p * sn[j];
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t o = __shfl_sync(0xffffffffu, e[j], partner);
                            if (turned) {
                                const float p = __uint_as_float(o << 16) * r * __uint_as_float(pe[j] << 16);
                                const float q = __uint_as_float(o & 0xffff0000u) * r * __uint_as_float(pe[j] & 0xffff0000u);
                                y[2 * j] = y[2 * j] * cs[2 * j] + sign * p * sn[2 * j];
                                y[2 * j + 1] = y[2 * j + 1] * cs[2 * j + 1] + sign * q * sn[2 * j + 1];
                            }
                        }
                    }
                }
                if (h < h1) {
                    uint16_t *row = is_k ? a.k_out + token * a.k_out_stride + (int64_t)(h - a.q_heads) * D
                                         : a.q_out + token * a.q_out_stride + (int64_t)h * D;
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[j] = (uint32_t)f32_to_bf16_bits(y[2 * j]) | ((uint32_t)f32_to_bf16_bits(y[2 * j + 1]) << 16);
                    *reinterpret_cast<uint4 *>(row + 8 * l) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
    pdl_launch_dependents();
}

q4_status launch_norm_rope(const DeviceInfo &dev, NormRopeArgs a, int head_dim, cudaStream_t st, bool pdl)
{
    // A warp takes all heads of a token, or, where that would leave SMs without work, as many as
    // one batch of loads brings.
    const int heads = a.q_heads + a.kv_heads, batch = NR_BATCH * (256 / head_dim);
    a.part_heads = (int64_t)a.tokens >= (int64_t)dev.sms * NR_WARPS * 2 ? heads : batch;
    a.parts = (heads + a.part_heads - 1) / a.part_heads;
    const int64_t ctas = ((int64_t)a.tokens * a.parts + NR_WARPS - 1) / NR_WARPS;
    const int64_t most = (int64_t)dev.sms * 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas < most ? ctas : most));
    cfg.blockDim = dim3(NR_WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    const cudaError_t e = head_dim == 64 ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<64>, a)
                                         : cudaLaunchKernelEx(&cfg, norm_rope_kernel<128>, a);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "launch of norm_rope_kernel");
}

}  // namespace q4
