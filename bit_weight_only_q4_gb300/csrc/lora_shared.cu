// Adapters for requests of a few tokens each that share them (see lora.cuh): tiles are tokens of one
// adapter, whichever requests they belong to, so that it is read once for eight or sixteen tokens and not once for
// each request.  Products as in lora_few.cu.
//
// Which tokens: every CTA works it out for itself, a request a thread.  Tokens are added up by adapter (the
// requests without one are one more), which gives the adapters' tiles and this cluster's place among them; the
// adapter's requests, laid end to end, then give the tile's rows.
//
// What bounds it: latency, of that and of the loads of A; so tiles are small and CTAs many.  Measured, against a tile for
// each request: 64 requests of 5 tokens on 8 adapters, rank 64, K = 8192, N = 2048, 12.9 against 14.8 us (tiles of 32 tokens:
// 17.4, of 8: 13.4; all with t as one bf16 value, as two 13.4); 48 single tokens on 4 adapters, rank 16, 4.2 against 5.6, on 24 adapters 5.1 against 5.6; 200 of 2
// on 20, rank 64, N = 8192, 28 against 51.
#include "lora.cuh"

namespace q4 {

constexpr int LS_WARPS = 8, LS_THREADS = LS_WARPS * 32;    // and the most requests

// Sum of v over the threads before this one; `all`: over all.  Two barriers.
__device__ __forceinline__ int ls_before(int v, int *s_warp, int &all)
{
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    int sum = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int w = __shfl_up_sync(0xffffffffu, sum, o);
        sum += lane >= o ? w : 0;
    }
    __syncthreads();
    if (lane == 31)
        s_warp[warp] = sum;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < LS_WARPS; ++w) {
        before += w < warp ? s_warp[w] : 0;
        all += s_warp[w];
    }
    return before + sum - v;
}

// STEPS: 16s of rank values, rounded up to a power of two; TILES: groups of eight tokens.
template <int STEPS, int TILES>
__global__ void __cluster_dims__(LR_CLUSTER, 1, 1) __launch_bounds__(LS_THREADS, TILES == 1 ? 4 : 2) lora_shared_kernel(const LoraArgs p)
{
    constexpr int RANKS = 16 * STEPS, TOKENS = 8 * TILES;
    constexpr int KPARTS = LS_WARPS / STEPS;                // warps that share 16 rank values' columns of K
    constexpr int PITCH = RANKS + 8;
    __shared__ __align__(16) float s_part[KPARTS][RANKS][TOKENS], s_sum[RANKS][TOKENS];
    __shared__ __align__(16) uint16_t s_t[2][TOKENS][PITCH];
    __shared__ int s_total[LS_THREADS], s_warp[LS_WARPS], s_top[LS_WARPS], s_row[TOKENS], s_found[2];
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;                  // MMA: row (or token) and place within it
    const uint32_t rank = lr_rank_in_cluster();
    const int r = p.rank, unit = (int)(blockIdx.x / LR_CLUSTER);
    pdl_wait();

    // ---- this thread's request
    int adapter = p.adapters, start = 0, len = 0;           // (p.adapters: none)
    {
        const bool here = tid < p.batch;
        int lo = here ? __ldg(p.offsets + tid) : 0, hi = here ? __ldg(p.offsets + tid + 1) : 0;
        const int id = here ? __ldg(p.ids + tid) : -1;
        s_total[tid] = 0;
        bool bad = lo < 0 || hi < 0 || lo > p.tokens || hi > p.tokens || id >= p.adapters;
        lo = lo < 0 ? 0 : lo > p.tokens ? p.tokens : lo;
        hi = hi < 0 ? 0 : hi > p.tokens ? p.tokens : hi;
        // a request that would begin before the end of one in front of it is left out
        int top = hi;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, top, o);
            top = lane >= o && v > top ? v : top;
        }
        if (lane == 31)
            s_top[warp] = top;
        int under = __shfl_up_sync(0xffffffffu, top, 1);
        under = lane > 0 ? under : 0;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < LS_WARPS; ++w)
            under = w < warp && s_top[w] > under ? s_top[w] : under;
        const bool out = hi < lo || lo < under;
        if (here && (bad || out) && p.err)
            atomicOr(p.err, kErrIndex);
        start = lo;
        len = here && !out ? hi - lo : 0;
        adapter = id < 0 || id >= p.adapters ? p.adapters : id;
        if (len > 0)
            atomicAdd(&s_total[adapter], len);
    }
    __syncthreads();
    // ---- the cluster's tile: which adapter, which of its tokens
    int all;
    const int mine = tid <= p.adapters ? s_total[tid] : 0, units = (mine + TOKENS - 1) / TOKENS;
    const int first = ls_before(units, s_warp, all);
    if (unit >= all)
        return;                                             // (the whole cluster)
    if (unit >= first && unit < first + units) {
        s_found[0] = tid;
        s_found[1] = unit - first;
    }
    __syncthreads();
    const int a_id = s_found[0], skip = s_found[1] * TOKENS;
    const int rows = s_total[a_id] - skip < TOKENS ? s_total[a_id] - skip : TOKENS;
    const int before = ls_before(adapter == a_id ? len : 0, s_warp, all);
    if (adapter == a_id)
        for (int i = before > skip ? before : skip; i < before + len && i < skip + TOKENS; ++i)
            s_row[i - skip] = start + i - before;
    __syncthreads();
    if (a_id == p.adapters) {                               // base as it is
        for (int i = 0; i < rows; ++i)
            lr_copy(p, LoraTile{s_row[i], 1, -1}, rank, LR_CLUSTER);
        return;
    }
    const float scale = __ldg(p.scales + a_id);

    // ---- t over this CTA's columns of K
    {
        const int m = warp % STEPS, part = warp / STEPS;
        const int k0 = lr_share((p.K + 31) / 32, rank, LR_CLUSTER), k1 = lr_share((p.K + 31) / 32, rank + 1, LR_CLUSTER);
        const uint16_t *a = p.a + ((int64_t)a_id * r + m * 16 + g) * p.K + 8 * t;
        const bool row0 = m * 16 + g < r, row1 = m * 16 + g + 8 < r;
        const uint16_t *x[TILES];
#pragma unroll
        for (int i = 0; i < TILES; ++i)
            x[i] = 8 * i + g < rows ? p.x + (int64_t)s_row[8 * i + g] * p.x_stride + 8 * t : nullptr;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        float c[TILES][4];
#pragma unroll
        for (int i = 0; i < TILES; ++i)
            c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
#pragma unroll 4
        for (int k = k0 + part; k < k1; k += KPARTS) {
            const bool in = 32 * k + 8 * t < p.K;
            const uint4 a0 = in && row0 ? ld_stream_v4(a + 32 * k) : zero;
            const uint4 a1 = in && row1 ? ld_stream_v4(a + (int64_t)8 * p.K + 32 * k) : zero;
            uint4 b[TILES];
#pragma unroll
            for (int i = 0; i < TILES; ++i)
                b[i] = in && x[i] ? *reinterpret_cast<const uint4 *>(x[i] + 32 * k) : zero;
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                lr_mma(c[i], a0.x, a1.x, a0.y, a1.y, b[i].x, b[i].y);
                lr_mma(c[i], a0.z, a1.z, a0.w, a1.w, b[i].z, b[i].w);
            }
        }
        // (the results' columns are tokens 2 t and 2 t + 1)
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            *reinterpret_cast<float2 *>(&s_part[part][m * 16 + g][8 * i + 2 * t]) = make_float2(c[i][0], c[i][1]);
            *reinterpret_cast<float2 *>(&s_part[part][m * 16 + g + 8][8 * i + 2 * t]) = make_float2(c[i][2], c[i][3]);
        }
    }
    // ---- the first of the B rows and base values that this warp needs are on their way during the exchange
    const int n0 = lr_share((p.N + 15) / 16, rank, LR_CLUSTER), n1 = lr_share((p.N + 15) / 16, rank + 1, LR_CLUSTER);
    struct Group {
        uint2 b[2][STEPS];
        uint32_t base[TILES][2];
    };
    auto ask = [&](int group, Group &v) {
        const int n = 16 * group + 2 * g;
        const bool in = group < n1 && n < p.N;
        const uint16_t *b = p.b + ((int64_t)a_id * p.N + n) * r + 4 * t;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const bool here = in && 16 * s + 4 * t < r;
            v.b[0][s] = here ? ld_stream_v2(b + 16 * s) : make_uint2(0u, 0u);
            v.b[1][s] = here ? ld_stream_v2(b + r + 16 * s) : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y)
                v.base[i][y] = in && 8 * i + 2 * t + y < rows
                                   ? *reinterpret_cast<const uint32_t *>(p.base + (int64_t)s_row[8 * i + 2 * t + y] * p.base_stride + n)
                                   : 0u;
    };
    Group now;
    ask(n0 + warp, now);
    __syncthreads();
    for (int i = tid; i < RANKS * TOKENS / 4; i += LS_THREADS) {
        float4 v = reinterpret_cast<const float4 *>(s_part[0])[i];
#pragma unroll
        for (int k = 1; k < KPARTS; ++k) {
            const float4 w = reinterpret_cast<const float4 *>(s_part[k])[i];
            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
        reinterpret_cast<float4 *>(s_sum)[i] = v;
    }
    __syncwarp();
    lr_cluster_arrive();
    lr_cluster_wait();
    for (int i = tid; i < RANKS * TOKENS / 4; i += LS_THREADS) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t at = smem_u32(s_sum) + 16u * (uint32_t)i;
#pragma unroll
        for (uint32_t k = 0; k < LR_CLUSTER; ++k) {
            const float4 w = lr_load(lr_map(at, k));
            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
        const int j = i / (TOKENS / 4), m = (i % (TOKENS / 4)) * 4;
        const bool in = j < r;                              // (what lies behind meets zeros, and is to be one)
        lr_split(in ? v.x : 0.f, s_t[0][m][j], s_t[1][m][j]);
        lr_split(in ? v.y : 0.f, s_t[0][m + 1][j], s_t[1][m + 1][j]);
        lr_split(in ? v.z : 0.f, s_t[0][m + 2][j], s_t[1][m + 2][j]);
        lr_split(in ? v.w : 0.f, s_t[0][m + 3][j], s_t[1][m + 3][j]);
    }
    __syncthreads();
    lr_cluster_arrive();                                    // no CTA leaves while its sums are read
    // ---- this CTA's columns
#pragma unroll 1
    for (int group = n0 + warp; group < n1; group += LS_WARPS) {
        Group next;
        ask(group + LS_WARPS, next);
        const int n = 16 * group + 2 * g;
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const uint2 tt = *reinterpret_cast<const uint2 *>(&s_t[0][8 * i + g][16 * s + 4 * t]);
                const uint2 rest = *reinterpret_cast<const uint2 *>(&s_t[1][8 * i + g][16 * s + 4 * t]);
                lr_mma(c, now.b[0][s].x, now.b[1][s].x, now.b[0][s].y, now.b[1][s].y, rest.x, rest.y);
                lr_mma(c, now.b[0][s].x, now.b[1][s].x, now.b[0][s].y, now.b[1][s].y, tt.x, tt.y);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
                if (n < p.N && 8 * i + 2 * t + y < rows)    // (rows n and n + 1 are the lane's rows g and g + 8)
                    *reinterpret_cast<uint32_t *>(p.out + (int64_t)s_row[8 * i + 2 * t + y] * p.out_stride + n) =
                        bf16_pair(fmaf(scale, c[y], __uint_as_float(now.base[i][y] << 16)),
                                  fmaf(scale, c[2 + y], __uint_as_float(now.base[i][y] & 0xffff0000u)));
        }
        now = next;
    }
    __syncwarp();
    lr_cluster_wait();
}

bool lora_shared_eligible(const LoraArgs &a) { return a.batch <= LS_THREADS && a.adapters < LS_THREADS && a.batch >= 2 * a.adapters; }

q4_status launch_lora_shared(const LoraArgs &a, cudaStream_t st, bool pdl)
{
    // at most one part-filled tile an adapter, and one of the tokens without
    const int tile = a.rank <= 32 ? 8 : 16;
    const int64_t tiles = (int64_t)a.tokens / tile + a.adapters + 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tiles < a.tokens ? tiles : a.tokens) * LR_CLUSTER));
    cfg.blockDim = dim3(LS_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    void (*kernel)(LoraArgs) = a.rank <= 16   ? lora_shared_kernel<1, 1>
                               : a.rank <= 32 ? lora_shared_kernel<2, 1>
                               : a.rank <= 64 ? lora_shared_kernel<4, 2>
                                              : lora_shared_kernel<8, 2>;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "launch of lora_shared_kernel");
}

}  // namespace q4
