// Launch parameters of the operators around a layer's projections: norms and rotation of
// queries and keys, attention over whole prompts, adapters (checked by layer_capi.cu).
#pragma once

#include "q4_internal.h"

namespace q4 {

// ---- norm_rope.cu
struct NormRopeArgs {
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;    // elements from token to token
    const uint16_t *q_weight, *k_weight;                       // NULL: no norm
    const int32_t *positions;
    const float *inv_freq;
    int q_heads, kv_heads, tokens, rotary;                     // rotary = 0: no rotation
    int interleaved;
    float eps;
    int parts, part_heads;                                     // (chosen by the launch)
};
q4_status launch_norm_rope(const DeviceInfo &dev, NormRopeArgs a, int head_dim, cudaStream_t st, bool pdl);

// ---- prompt_attention.cu
struct PromptArgs {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    int64_t q_stride, k_stride, v_stride;                      // elements from token to token
    const int32_t *offsets;                                    // [batch + 1]
    int batch, tokens, q_heads, kv_heads;
    float scale_log2;                                          // scale * log2(e)
    int group, tile_tokens, box_tokens;                        // (by the launch) query heads per key head, tokens of a tile, of 32 rows
    int swap;                                                  // (tests) so many CTAs change places with the next as many; 0: none
    unsigned *err;
};
void prompt_set_swap(int ctas);
q4_status launch_prompt_attention(PromptArgs a, int head_dim, cudaStream_t st, bool pdl);

// ---- lora_few.cu, lora_shared.cu, lora_many.cu
struct LoraArgs {
    const uint16_t *x, *a, *b, *base;
    uint16_t *out;
    int64_t x_stride, base_stride, out_stride;                 // elements from token to token
    const float *scales;                                       // [adapters]
    const int32_t *offsets, *ids;                              // [batch + 1], [batch]
    int batch, tokens, adapters, rank, N, K;
    unsigned *err;
};
q4_status launch_lora_few(const LoraArgs &a, cudaStream_t st, bool pdl);
bool lora_shared_eligible(const LoraArgs &a);
q4_status launch_lora_shared(const LoraArgs &a, cudaStream_t st, bool pdl);
q4_status launch_lora_many(const DeviceInfo &dev, const LoraArgs &a, cudaStream_t st, bool pdl);

}  // namespace q4
