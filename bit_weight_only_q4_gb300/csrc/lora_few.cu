// Adapters for requests of a few tokens each (see lora.cuh): tiles of at most eight tokens.
//
// Both products are small here and each adapter is read for a few tokens, so what counts is how soon its
// bytes are asked for: every load goes straight from global memory to the operand registers of a
// 16 x 8 x 16 MMA of one warp (rank values or output columns as its 16 rows, tokens as its 8 columns; 16
// rows are all that a tcgen05 MMA of 128 would be given).  The columns of K may be taken in any order as
// long as both operands agree: a lane takes eight adjacent ones (16 bytes), which serve two MMAs.
// Output columns lie two to a lane, so that eight lanes store 32 bytes.
//
// What bounds it: the chain of offsets, x and A, the exchange, B (48 single tokens, rank 16: 5.4 us), and where tiles
// share adapters, L2, from which each tile reads its own.  t as two values costs 1 to 4% (64 requests of 5 with an adapter each, rank
// 64: 18.9 -> 19.6 us) and leaves bf16's rounding of the result as the only one that counts.  Each cluster adds up the lengths
// in front of its tile, so that many requests cost more than their number: single tokens, rank 16, 2048 -> 2048, of 64, 256,
// 512, 1,024 and 4,096 requests take 6.1, 25.5, 62, 180 and 2,132 us.
#include "lora.cuh"

namespace q4 {

constexpr int LF_TOKENS = 8, LF_WARPS = 8;

// STEPS: 16s of rank values, rounded up to a power of two.  Four CTAs an SM up to rank 64 (64 registers): 64 requests of
// 5 tokens, 512 CTAs, are one wave then (14.9 us; with 76 registers 20.3).
template <int STEPS>
__global__ void __cluster_dims__(LR_CLUSTER, 1, 1) __launch_bounds__(LF_WARPS * 32, STEPS <= 4 ? 4 : 2) lora_few_kernel(const LoraArgs p)
{
    constexpr int RANKS = 16 * STEPS;
    constexpr int PITCH = RANKS + 8;
    __shared__ __align__(16) float s_part[LF_WARPS][RANKS][LF_TOKENS], s_sum[RANKS][LF_TOKENS];
    __shared__ __align__(16) uint16_t s_t[2][LF_TOKENS][PITCH];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;                  // MMA: row (or token) and place within it
    const uint32_t rank = lr_rank_in_cluster();
    const int r = p.rank;
    pdl_wait();
    LoraTile tile;
    if (!lr_tile(p, (int)(blockIdx.x / LR_CLUSTER), LF_TOKENS, tile))
        return;                                             // (the whole cluster)
    if (tile.adapter < 0) {
        lr_copy(p, tile, rank, LR_CLUSTER);
        return;
    }
    const float scale = __ldg(p.scales + tile.adapter);

    // ---- t over this CTA's columns of K
    {
        // 32 columns at a time for each warp: all rank values against one load of x
        const int k0 = lr_share((p.K + 31) / 32, rank, LR_CLUSTER), k1 = lr_share((p.K + 31) / 32, rank + 1, LR_CLUSTER);
        const uint16_t *a = p.a + ((int64_t)tile.adapter * r + g) * p.K + 8 * t;
        const uint16_t *x = p.x + (int64_t)(tile.row + g) * p.x_stride + 8 * t;
        const bool token = g < tile.rows;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        float c[STEPS][4];
#pragma unroll
        for (int m = 0; m < STEPS; ++m)
            c[m][0] = c[m][1] = c[m][2] = c[m][3] = 0.f;
        constexpr int UNROLL = STEPS <= 2 ? 4 / STEPS : 1;
#pragma unroll UNROLL
        for (int k = k0 + warp; k < k1; k += LF_WARPS) {
            const bool in = 32 * k + 8 * t < p.K;
            const uint4 b = in && token ? *reinterpret_cast<const uint4 *>(x + 32 * k) : zero;
            uint4 w[STEPS][2];
#pragma unroll
            for (int m = 0; m < STEPS; ++m) {
                w[m][0] = in && 16 * m + g < r ? ld_stream_v4(a + (int64_t)(16 * m) * p.K + 32 * k) : zero;
                w[m][1] = in && 16 * m + g + 8 < r ? ld_stream_v4(a + (int64_t)(16 * m + 8) * p.K + 32 * k) : zero;
            }
#pragma unroll
            for (int m = 0; m < STEPS; ++m) {
                lr_mma(c[m], w[m][0].x, w[m][1].x, w[m][0].y, w[m][1].y, b.x, b.y);
                lr_mma(c[m], w[m][0].z, w[m][1].z, w[m][0].w, w[m][1].w, b.z, b.w);
            }
        }
#pragma unroll
        for (int m = 0; m < STEPS; ++m) {
            *reinterpret_cast<float2 *>(&s_part[warp][m * 16 + g][2 * t]) = make_float2(c[m][0], c[m][1]);
            *reinterpret_cast<float2 *>(&s_part[warp][m * 16 + g + 8][2 * t]) = make_float2(c[m][2], c[m][3]);
        }
    }
    // ---- the first of the B rows and base values that this warp needs are on their way during the exchange
    const int n0 = lr_share((p.N + 15) / 16, rank, LR_CLUSTER), n1 = lr_share((p.N + 15) / 16, rank + 1, LR_CLUSTER);
    struct Group {
        uint2 b[2][STEPS];
        uint32_t base[2];
    };
    auto ask = [&](int group, Group &v) {
        const int n = 16 * group + 2 * g;
        const bool in = group < n1 && n < p.N;
        const uint16_t *b = p.b + ((int64_t)tile.adapter * p.N + n) * r + 4 * t;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const bool here = in && 16 * s + 4 * t < r;
            v.b[0][s] = here ? ld_stream_v2(b + 16 * s) : make_uint2(0u, 0u);
            v.b[1][s] = here ? ld_stream_v2(b + r + 16 * s) : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            v.base[i] = in && 2 * t + i < tile.rows
                            ? *reinterpret_cast<const uint32_t *>(p.base + (int64_t)(tile.row + 2 * t + i) * p.base_stride + n)
                            : 0u;
    };
    Group now;
    ask(n0 + warp, now);
    __syncthreads();
    for (int i = tid; i < RANKS * LF_TOKENS / 4; i += LF_WARPS * 32) {
        float4 v = reinterpret_cast<const float4 *>(s_part[0])[i];
#pragma unroll
        for (int k = 1; k < LF_WARPS; ++k) {
            const float4 w = reinterpret_cast<const float4 *>(s_part[k])[i];
            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
        reinterpret_cast<float4 *>(s_sum)[i] = v;
    }
    __syncwarp();
    lr_cluster_arrive();
    lr_cluster_wait();
    for (int i = tid; i < RANKS * LF_TOKENS / 4; i += LF_WARPS * 32) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t at = smem_u32(s_sum) + 16u * (uint32_t)i;
#pragma unroll
        for (uint32_t k = 0; k < LR_CLUSTER; ++k) {
            const float4 w = lr_load(lr_map(at, k));
            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
        const int j = i / (LF_TOKENS / 4), m = (i % (LF_TOKENS / 4)) * 4;
        const bool in = j < r;                              // (what lies behind meets zeros, and is to be one)
        lr_split(in ? v.x : 0.f, s_t[0][m][j], s_t[1][m][j]);
        lr_split(in ? v.y : 0.f, s_t[0][m + 1][j], s_t[1][m + 1][j]);
        lr_split(in ? v.z : 0.f, s_t[0][m + 2][j], s_t[1][m + 2][j]);
        lr_split(in ? v.w : 0.f, s_t[0][m + 3][j], s_t[1][m + 3][j]);
    }
    __syncthreads();
    lr_cluster_arrive();                                    // no CTA leaves while its sums are read
    // ---- this CTA's columns
    uint2 tt[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
        tt[s] = *reinterpret_cast<const uint2 *>(&s_t[0][g][16 * s + 4 * t]);
#pragma unroll 1
    for (int group = n0 + warp; group < n1; group += LF_WARPS) {
        Group next;
        ask(group + LF_WARPS, next);
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const uint2 rest = *reinterpret_cast<const uint2 *>(&s_t[1][g][16 * s + 4 * t]);
            lr_mma(c, now.b[0][s].x, now.b[1][s].x, now.b[0][s].y, now.b[1][s].y, rest.x, rest.y);
            lr_mma(c, now.b[0][s].x, now.b[1][s].x, now.b[0][s].y, now.b[1][s].y, tt[s].x, tt[s].y);
        }
        const int n = 16 * group + 2 * g;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (n < p.N && 2 * t + i < tile.rows)           // (rows n and n + 1 are the lane's rows g and g + 8)
                *reinterpret_cast<uint32_t *>(p.out + (int64_t)(tile.row + 2 * t + i) * p.out_stride + n) =
                    bf16_pair(fmaf(scale, c[i], __uint_as_float(now.base[i] << 16)),
                              fmaf(scale, c[2 + i], __uint_as_float(now.base[i] & 0xffff0000u)));
        now = next;
    }
    __syncwarp();
    lr_cluster_wait();
}

q4_status launch_lora_few(const LoraArgs &a, cudaStream_t st, bool pdl)
{
    // at most one part-filled tile a request; where a request has no tokens that leaves a cluster behind the last tile,
    // which goes through all offsets and notes those that are none
    const int64_t tiles = (int64_t)a.tokens / LF_TOKENS + a.batch, most = (int64_t)a.tokens + 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * LR_CLUSTER));
    cfg.blockDim = dim3(LF_WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    void (*kernel)(LoraArgs) = a.rank <= 16   ? lora_few_kernel<1>
                               : a.rank <= 32 ? lora_few_kernel<2>
                               : a.rank <= 64 ? lora_few_kernel<4>
                                              : lora_few_kernel<8>;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "launch of lora_few_kernel");
}

}  // namespace q4
