// own_attn.cuh -- split-KV decode attention as a part of a larger call
// (decode_attn.cu; called by prefix_attn.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace fpk {

// Workspace of own_attention with the automatic split count on the current
// device (0: no device).
size_t own_attention_bytes(int32_t B, int32_t Hq, int32_t Hkv);
// The bytes of that workspace that have to be zero when own_attention begins
// (its arrival counters, which lie elsewhere for other shapes): [*from, *to).
void own_attention_counters(int32_t B, int32_t Hq, int32_t Hkv, size_t* from, size_t* to);

// fpk_paged_decode_attn_fp8 / _bf16 with the automatic split count, request r's
// table beginning skip_pages[r] columns to the right (nullable: none), for
// arguments that the caller has checked.
int own_attention(bool fp8, const void* q, const void* kv_pool, const float* k_scale, const float* v_scale,
                  const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                  const int32_t* skip_pages, const uint8_t* abort_mask, float* out, float* lse, void* workspace,
                  size_t workspace_bytes, float sm_scale, int32_t B, int32_t Hq, int32_t Hkv, int32_t page_size,
                  int32_t num_pages, void* stream);

}  // namespace fpk
