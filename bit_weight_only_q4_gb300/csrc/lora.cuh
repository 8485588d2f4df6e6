// What the adapter kernels share: the tile that a cluster works on, and clusters.
//
// For token m of a request with adapter a
//     t = x_m A_a^T  (rank values),   out_m = base_m + scale_a (t B_a^T).
// A cluster of up to eight CTAs takes a tile of a request's tokens through both products in one launch:
// each CTA sums t over its share of K, they add their sums up through each other's shared memory, and
// each then has its share of the output columns.  Sums are fp32; t meets B as bf16, as wide as x and B are, and
// in tiles of a few tokens, where another MMA costs nothing, as two bf16 values, t's and what that leaves.
#pragma once

#include "layer_ops.h"
#include "segments.cuh"
#include "tc_device.cuh"

namespace q4 {

constexpr int LR_CLUSTER = 8;              // at most

__device__ __forceinline__ uint32_t lr_rank_in_cluster()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t lr_cluster_size()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void lr_cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void lr_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Address of this CTA's shared-memory address a in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t lr_map(uint32_t a, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 lr_load(uint32_t cluster_address)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_address));
    return v;
}

// First of n things that CTA `rank` of `size` has, when they are shared out evenly.
__device__ __forceinline__ int lr_share(int n, uint32_t rank, uint32_t size) { return (int)((int64_t)n * rank / size); }

// One warp's MMA, for tiles of a few tokens (see lora_few.cu).
__device__ __forceinline__ void lr_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// t as two bf16 values.
__device__ __forceinline__ void lr_split(float v, uint16_t &most, uint16_t &rest)
{
    most = f32_to_bf16_bits(v);
    const float m = __uint_as_float((uint32_t)most << 16);
    rest = m - m == 0.f ? f32_to_bf16_bits(v - m) : 0;
}

// How many of n things dealt round `size` CTAs fall to CTA `rank`.
__device__ __forceinline__ int lr_round(int n, uint32_t rank, uint32_t size) { return (n - (int)rank + (int)size - 1) / (int)size; }

// The tile of tokens that a cluster works on; false: none.
struct LoraTile {
    int row, rows, adapter;                // adapter < 0: base as it is
};

__device__ __forceinline__ bool lr_tile(const LoraArgs &p, int number, int span, LoraTile &t)
{
    // (the first ids are asked for with the first offsets)
    const int lane = (int)(threadIdx.x & 31), id = lane < p.batch ? __ldg(p.ids + lane) : -1;
    SegmentWalk walk(Segments{p.offsets, p.batch, p.tokens, span, 1, p.err});
    SegmentUnit u;
    if (!walk.find(number, u)) {
        // behind the last tile, where a request has no tokens: its id is looked at here
        if (lr_rank_in_cluster() == 0 && threadIdx.x < 32 && p.err)
            for (int b = lane; b < p.batch; b += 32)
                if (__ldg(p.ids + b) >= p.adapters)
                    atomicOr(p.err, kErrIndex);
        return false;
    }
    const int first = u.unit * span;
    t.row = u.start + first;
    t.rows = u.len - first < span ? u.len - first : span;
    t.adapter = __shfl_sync(0xffffffffu, id, u.sequence & 31);
    if (u.sequence >= 32)
        t.adapter = __ldg(p.ids + u.sequence);
    if (t.adapter >= p.adapters) {
        if (p.err && (threadIdx.x & 31) == 0)
            atomicOr(p.err, kErrIndex);
        t.adapter = -1;
    }
    return true;
}

// A tile without an adapter: this CTA's columns of base, where out is not base itself.
__device__ __forceinline__ void lr_copy(const LoraArgs &p, const LoraTile &t, uint32_t rank, uint32_t size)
{
    if (p.out == p.base)
        return;
    const int c0 = lr_share(p.N / 8, rank, size), n = lr_share(p.N / 8, rank + 1, size) - c0;
    const int rows = n <= 1 << 23 ? t.rows : 1;              // at a time: their columns are counted in 32 bits
    for (int r0 = 0; r0 < t.rows; r0 += rows)
        for (int i = (int)threadIdx.x; i < rows * n; i += (int)blockDim.x) {
            const int r = i / n, c = 8 * (c0 + i - r * n), row = t.row + r0 + r;
            *reinterpret_cast<uint4 *>(p.out + (int64_t)row * p.out_stride + c) =
                *reinterpret_cast<const uint4 *>(p.base + (int64_t)row * p.base_stride + c);
        }
}

}  // namespace q4
