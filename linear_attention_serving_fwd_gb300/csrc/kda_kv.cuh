// Parameter blocks of the paged key/value cache's kernels, shared with their
// API layer.
#pragma once

#include "kda_params.cuh"

namespace kda {

struct KvPagesParams {
  int32_t* kv_lens;
  int32_t* table;
  int64_t table_stride;
  int32_t* free_pages;
  int32_t* free_count;
  int n_req, table_cols, n_pages;
  int page_shift;             // page size as a power of two
  const int32_t* lens;        // extend: new_lens, truncate: keep_lens
  int32_t* cu_seqlens;        // extend
  int32_t* slot_map;          // extend, [max_tokens]
  int max_tokens;
  int32_t* step_lens;         // extend
  unsigned* err;
};

// 16-bit storage (bf16 or fp16) throughout; strides in elements.
struct KvAppendParams {
  const __nv_bfloat16 *k, *v;
  int64_t k_st, k_sh, v_st, v_sh;
  __nv_bfloat16 *kc, *vc;
  int64_t kc_sp, kc_st, kc_sh, vc_sp, vc_st, vc_sh;
  const int32_t* slot_map;
  int t_total, hkv, n_pages, page_shift;
  unsigned* err;
};

struct AttentionParams {
  const __nv_bfloat16* q;
  int64_t q_st, q_sh;
  const __nv_bfloat16 *kc, *vc;
  int64_t kc_sp, kc_st, kc_sh, vc_sp, vc_st, vc_sh;
  __nv_bfloat16* out;         // [t_total, hq, 128]
  float* lse;                 // [t_total, hq] or null
  const int32_t* cu_seqlens;  // [n_req + 1]
  const int32_t* kv_lens;     // [n_req]
  const int32_t* table;
  int64_t table_stride;
  int table_cols, n_req, t_total, hq, hkv;
  int n_pages, page_shift;
  float scale;
  int window, sinks;          // window 0: none (sinks then 0)
  unsigned* err;
};

int launch_kv_extend(const KvPagesParams& p, cudaStream_t stream);
int launch_kv_truncate(const KvPagesParams& p, cudaStream_t stream);
int launch_kv_append(const KvAppendParams& p, cudaStream_t stream);
int launch_attention(const AttentionParams& p, bool fp16, void* workspace, cudaStream_t stream);
size_t attention_workspace_bytes();

}  // namespace kda
