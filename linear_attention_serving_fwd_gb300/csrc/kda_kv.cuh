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

// The cache in 8 bits: e4m3 numbers (strides in bytes) and fp32 scales
// [n_pages, hkv, page / 16].
struct KvQuantCache {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  int64_t k_sp, k_st, k_sh, v_sp, v_st, v_sh;
  int hkv, n_pages, page_shift;
};

struct KvQuantAppendParams {
  KvQuantCache c;
  const __nv_bfloat16 *k, *v;
  int64_t k_st, k_sh, v_st, v_sh;
  const int32_t* slot_map;
  int t_total;
  int window;                 // tokens that a warp looks for blocks in
  unsigned* err;
};

// Reads of either cache: 16-bit rows through kc, vc, or 8-bit ones through c.
struct KvReadParams {
  KvQuantCache c;
  const __nv_bfloat16 *kc, *vc;
  int64_t kc_sp, kc_st, kc_sh, vc_sp, vc_st, vc_sh;
  __nv_bfloat16 *k, *v;       // [t_total, hkv, 128]
  const int32_t* slot_map;
  int t_total, hkv, n_pages, page_shift;
  unsigned* err;
};

struct RopeRows {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  int64_t in_st, in_sh, out_st, out_sh;
};
struct RopeParams {
  RopeRows q, k;
  int hq, hk, t_total, pairs;
  const unsigned long long* turns;
  float amplitude;
  const int32_t* positions;   // or null: cu_seqlens and kv_lens
  const int32_t* cu_seqlens;
  const int32_t* kv_lens;
  int n_req;
  int tokens;                 // of a CTA
};

int launch_kv_extend(const KvPagesParams& p, cudaStream_t stream);
int launch_kv_truncate(const KvPagesParams& p, cudaStream_t stream);
int launch_kv_append(const KvAppendParams& p, cudaStream_t stream);
int launch_attention(const AttentionParams& p, bool fp16, void* workspace, cudaStream_t stream);
size_t attention_workspace_bytes();
int launch_kv_quant_append(KvQuantAppendParams p, bool fp16, cudaStream_t stream);
int launch_kv_read(const KvReadParams& p, bool quant, bool fp16, cudaStream_t stream);
// a.kc, a.vc and their strides are not used: the cache is c
int launch_attention_quant(const AttentionParams& a, const KvQuantCache& c, bool fp16, void* workspace, cudaStream_t stream);
size_t attention_quant_workspace_bytes(int t_total, int hq);
int launch_rope(RopeParams p, bool interleaved, bool fp16, cudaStream_t stream);

}  // namespace kda
