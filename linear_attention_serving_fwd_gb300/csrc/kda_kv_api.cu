// Host side of the paged key/value cache's entry points (include/kda.h):
// argument validation and the launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "kda_kv.cuh"

namespace {

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  kda::set_last_error(code, buf);
  return code;
}

int ok() {
  kda::set_last_error(KDA_OK, "");
  return KDA_OK;
}

int cuda_fail(const char* what) {
  return fail(KDA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(cudaGetLastError()));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_page_size(int32_t page_size, int& shift) {
  for (shift = 4; shift <= 8; ++shift)
    if (page_size == 1 << shift) return KDA_OK;
  return fail(KDA_ERR_INVALID_ARGUMENT, "page_size must be 16, 32, 64, 128 or 256 (got %d).", page_size);
}

// Slots are int32.
int check_pages(int32_t n_pages, int32_t page_size) {
  if (n_pages <= 0) return fail(KDA_ERR_INVALID_ARGUMENT, "n_pages must be positive (got %d).", n_pages);
  if ((int64_t)n_pages * page_size > 0x7fffffff)
    return fail(KDA_ERR_INVALID_ARGUMENT, "n_pages * page_size exceeds 2^31.");
  return KDA_OK;
}

int check_table(const void* table, int64_t stride, int32_t cols, int32_t n_req) {
  if (!table) return fail(KDA_ERR_INVALID_ARGUMENT, "block_table must not be NULL.");
  if (cols <= 0) return fail(KDA_ERR_INVALID_ARGUMENT, "block_table needs at least one column.");
  if (stride < cols && n_req > 1)
    return fail(KDA_ERR_INVALID_ARGUMENT, "table_stride must be >= table_cols (%lld < %d).", (long long)stride, cols);
  return KDA_OK;
}

int fill_pages(const kda_kv_pages* g, kda::KvPagesParams& p) {
  memset(&p, 0, sizeof(p));
  if (!g) return fail(KDA_ERR_INVALID_ARGUMENT, "pages must not be NULL.");
  if (g->n_req < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "n_req must be >= 0.");
  int rc = check_page_size(g->page_size, p.page_shift);
  if (rc) return rc;
  if ((rc = check_pages(g->n_pages, g->page_size))) return rc;
  if (!g->free_pages || !g->free_count)
    return fail(KDA_ERR_INVALID_ARGUMENT, "free_pages and free_count must not be NULL.");
  if (g->n_req > 0) {
    if (!g->kv_lens) return fail(KDA_ERR_INVALID_ARGUMENT, "kv_lens must not be NULL.");
    if ((rc = check_table(g->block_table, g->table_stride, g->table_cols, g->n_req))) return rc;
    if ((int64_t)g->table_cols * g->page_size > 0x7fffffff)
      return fail(KDA_ERR_INVALID_ARGUMENT, "table_cols * page_size exceeds 2^31.");
  }
  p.kv_lens = g->kv_lens;
  p.table = g->block_table;
  p.table_stride = g->table_stride;
  p.free_pages = g->free_pages;
  p.free_count = g->free_count;
  p.n_req = g->n_req;
  p.table_cols = g->table_cols;
  p.n_pages = g->n_pages;
  return KDA_OK;
}

int check_cache(const kda_kv_cache* c, int& shift) {
  if (!c) return fail(KDA_ERR_INVALID_ARGUMENT, "cache must not be NULL.");
  if (c->dtype != KDA_DTYPE_BF16 && c->dtype != KDA_DTYPE_FP16)
    return fail(KDA_ERR_UNSUPPORTED_DTYPE, "the cache's dtype must be bfloat16 or float16 (got %d).", c->dtype);
  int rc = check_page_size(c->page_size, shift);
  if (rc) return rc;
  if ((rc = check_pages(c->n_pages, c->page_size))) return rc;
  if (c->hkv <= 0) return fail(KDA_ERR_INVALID_ARGUMENT, "hkv must be positive (got %d).", c->hkv);
  if (!c->k || !c->v) return fail(KDA_ERR_INVALID_ARGUMENT, "the cache's k and v must not be NULL.");
  if (!aligned16(c->k) || !aligned16(c->v))
    return fail(KDA_ERR_INVALID_ARGUMENT, "the cache's k and v must be 16-byte aligned.");
  const int64_t st[6] = {c->k_stride_page, c->k_stride_tok, c->k_stride_head,
                         c->v_stride_page, c->v_stride_tok, c->v_stride_head};
  for (int64_t s : st)
    if (s < kda::D || s % 8 != 0)
      return fail(KDA_ERR_INVALID_ARGUMENT, "the cache's strides must be multiples of 8 elements and >= 128 (got %lld).",
                  (long long)s);
  return KDA_OK;
}

int check_quant_cache(const kda_kv_quant_cache* c, kda::KvQuantCache& g) {
  if (!c) return fail(KDA_ERR_INVALID_ARGUMENT, "cache must not be NULL.");
  if (c->dtype != KDA_DTYPE_BF16 && c->dtype != KDA_DTYPE_FP16)
    return fail(KDA_ERR_UNSUPPORTED_DTYPE, "the cache's dtype must be bfloat16 or float16 (got %d).", c->dtype);
  int rc = check_page_size(c->page_size, g.page_shift);
  if (rc) return rc;
  if ((rc = check_pages(c->n_pages, c->page_size))) return rc;
  if (c->hkv <= 0) return fail(KDA_ERR_INVALID_ARGUMENT, "hkv must be positive (got %d).", c->hkv);
  if (!c->k || !c->v || !c->k_scale || !c->v_scale)
    return fail(KDA_ERR_INVALID_ARGUMENT, "the cache's k, v and their scales must not be NULL.");
  if (!aligned16(c->k) || !aligned16(c->v))
    return fail(KDA_ERR_INVALID_ARGUMENT, "the cache's k and v must be 16-byte aligned.");
  if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3u)
    return fail(KDA_ERR_INVALID_ARGUMENT, "the cache's scales must be 4-byte aligned.");
  const int64_t st[6] = {c->k_stride_page, c->k_stride_tok, c->k_stride_head,
                         c->v_stride_page, c->v_stride_tok, c->v_stride_head};
  for (int64_t s : st)
    if (s < kda::D || s % 16 != 0)
      return fail(KDA_ERR_INVALID_ARGUMENT,
                  "an 8-bit cache's strides must be multiples of 16 elements and >= 128 (got %lld).", (long long)s);
  g.k = static_cast<uint8_t*>(c->k);
  g.v = static_cast<uint8_t*>(c->v);
  g.k_scale = c->k_scale;
  g.v_scale = c->v_scale;
  g.k_sp = c->k_stride_page; g.k_st = c->k_stride_tok; g.k_sh = c->k_stride_head;
  g.v_sp = c->v_stride_page; g.v_st = c->v_stride_tok; g.v_sh = c->v_stride_head;
  g.hkv = c->hkv;
  g.n_pages = c->n_pages;
  return KDA_OK;
}

// [T, H, 128] rows read in 16-byte pieces
int check_rows(const void* x, int64_t st, int64_t sh, const char* name) {
  if (!x) return fail(KDA_ERR_INVALID_ARGUMENT, "%s must not be NULL.", name);
  if (!aligned16(x)) return fail(KDA_ERR_INVALID_ARGUMENT, "%s must be 16-byte aligned.", name);
  if (st < 0 || sh < 0 || st % 8 != 0 || sh % 8 != 0)
    return fail(KDA_ERR_INVALID_ARGUMENT, "%s strides must be non-negative multiples of 8 elements.", name);
  return KDA_OK;
}

// rows of kda_rope: read and written by different threads, so none overlap
int check_turned(const void* x, int64_t st, int64_t sh, int heads, int tokens, const char* name) {
  if (heads == 0) return KDA_OK;
  const int rc = check_rows(x, st, sh, name);
  if (rc) return rc;
  if ((tokens > 1 && st < kda::D) || (heads > 1 && sh < kda::D))
    return fail(KDA_ERR_INVALID_ARGUMENT, "%s rows must not overlap: strides >= 128 elements.", name);
  return KDA_OK;
}

// What the attention calls share.  ``nothing``: no tokens or no requests.
int fill_attention(kda::AttentionParams& p, int32_t page_size, const void* q, int64_t q_stride_tok, int64_t q_stride_head,
                   int32_t hq, int32_t t_total, void* out, float* lse, const int32_t* cu_seqlens, const int32_t* kv_lens,
                   const int32_t* block_table, int64_t table_stride, int32_t table_cols, int32_t n_req, float scale,
                   int32_t window, int32_t sinks, const void* workspace, size_t workspace_bytes, size_t need, bool& nothing) {
  int rc;
  if (hq <= 0 || hq % p.hkv != 0)
    return fail(KDA_ERR_INVALID_ARGUMENT, "query heads must be a multiple of key heads (hq=%d, hkv=%d).", hq, p.hkv);
  if (hq / p.hkv > 128)
    return fail(KDA_ERR_INVALID_ARGUMENT, "at most 128 query heads share a key head (hq=%d, hkv=%d).", hq, p.hkv);
  if (t_total < 0 || n_req < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "t_total and n_req must be >= 0.");
  if (!(scale > 0.f) || !std::isfinite(scale))
    return fail(KDA_ERR_INVALID_ARGUMENT, "scale must be positive and finite (got %g).", (double)scale);
  if (window < 0 || sinks < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "window and sinks must be >= 0.");
  nothing = t_total == 0 || n_req == 0;
  if (nothing) return ok();
  if ((rc = check_rows(q, q_stride_tok, q_stride_head, "q"))) return rc;
  if ((t_total > 1 && q_stride_tok < kda::D) || (hq > 1 && q_stride_head < kda::D))
    return fail(KDA_ERR_INVALID_ARGUMENT, "q rows must not overlap: strides >= 128 elements.");
  if (!out) return fail(KDA_ERR_INVALID_ARGUMENT, "out must not be NULL.");
  if (reinterpret_cast<uintptr_t>(out) & 31u) return fail(KDA_ERR_INVALID_ARGUMENT, "out must be 32-byte aligned.");
  if (!cu_seqlens || !kv_lens) return fail(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens and kv_lens must not be NULL.");
  if ((rc = check_table(block_table, table_stride, table_cols, n_req))) return rc;
  if ((int64_t)table_cols * page_size > 0x7fffffff - 512)
    return fail(KDA_ERR_INVALID_ARGUMENT, "table_cols * page_size must stay below 2^31 - 512.");
  if (!workspace || workspace_bytes < need)
    return fail(KDA_ERR_INVALID_ARGUMENT, "workspace needs %zu bytes (got %zu).", need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned16(workspace)) return fail(KDA_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned.");
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_st = q_stride_tok; p.q_sh = q_stride_head;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.cu_seqlens = cu_seqlens; p.kv_lens = kv_lens;
  p.table = block_table; p.table_stride = table_stride; p.table_cols = table_cols;
  p.n_req = n_req; p.t_total = t_total; p.hq = hq;
  // a window of the whole row is no narrower than any: positions less the
  // window then stay within 32 bits
  const int32_t row = table_cols * page_size;
  p.scale = scale; p.window = window < row ? window : row; p.sinks = window ? sinks : 0;
  p.err = kda::device_error_word();
  if (!p.err) return fail(KDA_ERR_CUDA, "cannot resolve the device error word.");
  return KDA_OK;
}

int read_rows(kda::KvReadParams& p, bool quant, int32_t dtype, const int32_t* slot_map, int32_t t_total, void* k, void* v,
              void* stream) {
  if (t_total < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "t_total must be >= 0.");
  if (t_total == 0) return ok();
  if (!slot_map) return fail(KDA_ERR_INVALID_ARGUMENT, "slot_map must not be NULL.");
  if (!k || !v) return fail(KDA_ERR_INVALID_ARGUMENT, "k and v must not be NULL.");
  if (!aligned16(k) || !aligned16(v)) return fail(KDA_ERR_INVALID_ARGUMENT, "k and v must be 16-byte aligned.");
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  p.slot_map = slot_map;
  p.t_total = t_total;
  p.err = kda::device_error_word();
  if (!p.err) return fail(KDA_ERR_CUDA, "cannot resolve the device error word.");
  if (kda::launch_kv_read(p, quant, dtype == KDA_DTYPE_FP16, static_cast<cudaStream_t>(stream)) != 0)
    return cuda_fail("kda_kv_read launch");
  return ok();
}

}  // namespace

extern "C" {

int kda_kv_extend(const kda_kv_pages* pages, const int32_t* new_lens, int32_t* cu_seqlens,
                  int32_t* slot_map, int32_t max_tokens, int32_t* step_lens, void* stream) {
  kda::KvPagesParams p;
  int rc = fill_pages(pages, p);
  if (rc) return rc;
  if (max_tokens < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "max_tokens must be >= 0.");
  if (!cu_seqlens) return fail(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens must not be NULL.");
  if (p.n_req > 0 && (!new_lens || !step_lens))
    return fail(KDA_ERR_INVALID_ARGUMENT, "new_lens and step_lens must not be NULL.");
  if (max_tokens > 0 && !slot_map) return fail(KDA_ERR_INVALID_ARGUMENT, "slot_map must not be NULL.");
  p.lens = new_lens;
  p.cu_seqlens = cu_seqlens;
  p.slot_map = slot_map;
  p.max_tokens = max_tokens;
  p.step_lens = step_lens;
  p.err = kda::device_error_word();
  if (!p.err) return fail(KDA_ERR_CUDA, "cannot resolve the device error word.");
  if (kda::launch_kv_extend(p, static_cast<cudaStream_t>(stream)) != 0) return cuda_fail("kda_kv_extend launch");
  return ok();
}

int kda_kv_truncate(const kda_kv_pages* pages, const int32_t* keep_lens, void* stream) {
  kda::KvPagesParams p;
  int rc = fill_pages(pages, p);
  if (rc) return rc;
  if (p.n_req == 0) return ok();
  if (!keep_lens) return fail(KDA_ERR_INVALID_ARGUMENT, "keep_lens must not be NULL.");
  p.lens = keep_lens;
  p.err = kda::device_error_word();
  if (!p.err) return fail(KDA_ERR_CUDA, "cannot resolve the device error word.");
  if (kda::launch_kv_truncate(p, static_cast<cudaStream_t>(stream)) != 0) return cuda_fail("kda_kv_truncate launch");
  return ok();
}

int kda_kv_append(const kda_kv_cache* cache, const void* k, int64_t k_stride_tok, int64_t k_stride_head,
                  const void* v, int64_t v_stride_tok, int64_t v_stride_head, const int32_t* slot_map,
                  int32_t t_total, void* stream) {
  kda::KvAppendParams p;
  memset(&p, 0, sizeof(p));
  int rc = check_cache(cache, p.page_shift);
  if (rc) return rc;
  if (t_total < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "t_total must be >= 0.");
  if (t_total == 0) return ok();
  if ((rc = check_rows(k, k_stride_tok, k_stride_head, "k"))) return rc;
  if ((rc = check_rows(v, v_stride_tok, v_stride_head, "v"))) return rc;
  if (!slot_map) return fail(KDA_ERR_INVALID_ARGUMENT, "slot_map must not be NULL.");
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_st = k_stride_tok; p.k_sh = k_stride_head; p.v_st = v_stride_tok; p.v_sh = v_stride_head;
  p.kc = static_cast<__nv_bfloat16*>(cache->k);
  p.vc = static_cast<__nv_bfloat16*>(cache->v);
  p.kc_sp = cache->k_stride_page; p.kc_st = cache->k_stride_tok; p.kc_sh = cache->k_stride_head;
  p.vc_sp = cache->v_stride_page; p.vc_st = cache->v_stride_tok; p.vc_sh = cache->v_stride_head;
  p.slot_map = slot_map;
  p.t_total = t_total; p.hkv = cache->hkv; p.n_pages = cache->n_pages;
  p.err = kda::device_error_word();
  if (!p.err) return fail(KDA_ERR_CUDA, "cannot resolve the device error word.");
  if (kda::launch_kv_append(p, static_cast<cudaStream_t>(stream)) != 0) return cuda_fail("kda_kv_append launch");
  return ok();
}

int kda_kv_append_quant(const kda_kv_quant_cache* cache, const void* k, int64_t k_stride_tok, int64_t k_stride_head,
                        const void* v, int64_t v_stride_tok, int64_t v_stride_head, const int32_t* slot_map,
                        int32_t t_total, void* stream) {
  kda::KvQuantAppendParams p;
  memset(&p, 0, sizeof(p));
  int rc = check_quant_cache(cache, p.c);
  if (rc) return rc;
  if (t_total < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "t_total must be >= 0.");
  if (t_total == 0) return ok();
  if ((rc = check_rows(k, k_stride_tok, k_stride_head, "k"))) return rc;
  if ((rc = check_rows(v, v_stride_tok, v_stride_head, "v"))) return rc;
  if (!slot_map) return fail(KDA_ERR_INVALID_ARGUMENT, "slot_map must not be NULL.");
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_st = k_stride_tok; p.k_sh = k_stride_head; p.v_st = v_stride_tok; p.v_sh = v_stride_head;
  p.slot_map = slot_map;
  p.t_total = t_total;
  p.err = kda::device_error_word();
  if (!p.err) return fail(KDA_ERR_CUDA, "cannot resolve the device error word.");
  if (kda::launch_kv_quant_append(p, cache->dtype == KDA_DTYPE_FP16, static_cast<cudaStream_t>(stream)) != 0)
    return cuda_fail("kda_kv_append_quant launch");
  return ok();
}

int kda_kv_read(const kda_kv_cache* cache, const int32_t* slot_map, int32_t t_total, void* k, void* v, void* stream) {
  kda::KvReadParams p;
  memset(&p, 0, sizeof(p));
  int rc = check_cache(cache, p.page_shift);
  if (rc) return rc;
  p.kc = static_cast<const __nv_bfloat16*>(cache->k);
  p.vc = static_cast<const __nv_bfloat16*>(cache->v);
  p.kc_sp = cache->k_stride_page; p.kc_st = cache->k_stride_tok; p.kc_sh = cache->k_stride_head;
  p.vc_sp = cache->v_stride_page; p.vc_st = cache->v_stride_tok; p.vc_sh = cache->v_stride_head;
  p.hkv = cache->hkv; p.n_pages = cache->n_pages;
  return read_rows(p, false, cache->dtype, slot_map, t_total, k, v, stream);
}

int kda_kv_read_quant(const kda_kv_quant_cache* cache, const int32_t* slot_map, int32_t t_total, void* k, void* v,
                      void* stream) {
  kda::KvReadParams p;
  memset(&p, 0, sizeof(p));
  int rc = check_quant_cache(cache, p.c);
  if (rc) return rc;
  p.hkv = p.c.hkv; p.n_pages = p.c.n_pages; p.page_shift = p.c.page_shift;
  return read_rows(p, true, cache->dtype, slot_map, t_total, k, v, stream);
}

size_t kda_paged_attention_workspace_bytes(void) { return kda::attention_workspace_bytes(); }

int kda_paged_attention(const kda_kv_cache* cache, const void* q, int64_t q_stride_tok,
                        int64_t q_stride_head, int32_t hq, int32_t t_total, void* out, float* lse,
                        const int32_t* cu_seqlens, const int32_t* kv_lens, const int32_t* block_table,
                        int64_t table_stride, int32_t table_cols, int32_t n_req, float scale,
                        int32_t window, int32_t sinks, void* workspace, size_t workspace_bytes,
                        void* stream) {
  kda::AttentionParams p;
  memset(&p, 0, sizeof(p));
  int rc = check_cache(cache, p.page_shift);
  if (rc) return rc;
  p.kc = static_cast<const __nv_bfloat16*>(cache->k);
  p.vc = static_cast<const __nv_bfloat16*>(cache->v);
  p.kc_sp = cache->k_stride_page; p.kc_st = cache->k_stride_tok; p.kc_sh = cache->k_stride_head;
  p.vc_sp = cache->v_stride_page; p.vc_st = cache->v_stride_tok; p.vc_sh = cache->v_stride_head;
  p.hkv = cache->hkv; p.n_pages = cache->n_pages;
  bool nothing = false;
  rc = fill_attention(p, cache->page_size, q, q_stride_tok, q_stride_head, hq, t_total, out, lse, cu_seqlens, kv_lens,
                      block_table, table_stride, table_cols, n_req, scale, window, sinks, workspace, workspace_bytes,
                      kda::attention_workspace_bytes(), nothing);
  if (rc || nothing) return rc;
  if (kda::launch_attention(p, cache->dtype == KDA_DTYPE_FP16, workspace, static_cast<cudaStream_t>(stream)) != 0)
    return cuda_fail("kda_paged_attention launch");
  return ok();
}

size_t kda_paged_attention_quant_workspace_bytes(int32_t t_total, int32_t hq) {
  return kda::attention_quant_workspace_bytes(t_total > 0 ? t_total : 0, hq > 0 ? hq : 0);
}

int kda_paged_attention_quant(const kda_kv_quant_cache* cache, const void* q, int64_t q_stride_tok,
                              int64_t q_stride_head, int32_t hq, int32_t t_total, void* out, float* lse,
                              const int32_t* cu_seqlens, const int32_t* kv_lens, const int32_t* block_table,
                              int64_t table_stride, int32_t table_cols, int32_t n_req, float scale,
                              int32_t window, int32_t sinks, void* workspace, size_t workspace_bytes,
                              void* stream) {
  kda::AttentionParams p;
  kda::KvQuantCache c;
  memset(&p, 0, sizeof(p));
  int rc = check_quant_cache(cache, c);
  if (rc) return rc;
  p.page_shift = c.page_shift; p.hkv = c.hkv; p.n_pages = c.n_pages;
  bool nothing = false;
  rc = fill_attention(p, cache->page_size, q, q_stride_tok, q_stride_head, hq, t_total, out, lse, cu_seqlens, kv_lens,
                      block_table, table_stride, table_cols, n_req, scale, window, sinks, workspace, workspace_bytes,
                      kda_paged_attention_quant_workspace_bytes(t_total, hq), nothing);
  if (rc || nothing) return rc;
  if (kda::launch_attention_quant(p, c, cache->dtype == KDA_DTYPE_FP16, workspace, static_cast<cudaStream_t>(stream)) != 0)
    return cuda_fail("kda_paged_attention_quant launch");
  return ok();
}

int kda_rope(const kda_rotation* rotation, int32_t dtype, const void* q, int64_t q_stride_tok, int64_t q_stride_head,
             int32_t hq, void* q_out, int64_t q_out_stride_tok, int64_t q_out_stride_head, const void* k,
             int64_t k_stride_tok, int64_t k_stride_head, int32_t hk, void* k_out, int64_t k_out_stride_tok,
             int64_t k_out_stride_head, int32_t t_total, const int32_t* positions, const int32_t* cu_seqlens,
             const int32_t* kv_lens, int32_t n_req, void* stream) {
  if (!rotation) return fail(KDA_ERR_INVALID_ARGUMENT, "rotation must not be NULL.");
  if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_FP16)
    return fail(KDA_ERR_UNSUPPORTED_DTYPE, "dtype must be bfloat16 or float16 (got %d).", dtype);
  if (rotation->pairs < 1 || rotation->pairs > kda::D / 2)
    return fail(KDA_ERR_INVALID_ARGUMENT, "pairs must be in 1 .. 64 (got %d).", rotation->pairs);
  if (rotation->interleaved != 0 && rotation->interleaved != 1)
    return fail(KDA_ERR_INVALID_ARGUMENT, "interleaved must be 0 or 1 (got %d).", rotation->interleaved);
  if (!std::isfinite(rotation->amplitude))
    return fail(KDA_ERR_INVALID_ARGUMENT, "amplitude must be finite (got %g).", (double)rotation->amplitude);
  if (!rotation->turns) return fail(KDA_ERR_INVALID_ARGUMENT, "turns must not be NULL.");
  if (reinterpret_cast<uintptr_t>(rotation->turns) & 7u)
    return fail(KDA_ERR_INVALID_ARGUMENT, "turns must be 8-byte aligned.");
  if (hq < 0 || hk < 0 || t_total < 0 || n_req < 0)
    return fail(KDA_ERR_INVALID_ARGUMENT, "hq, hk, t_total and n_req must be >= 0.");
  if (t_total == 0 || (hq == 0 && hk == 0) || (!positions && n_req == 0)) return ok();
  int rc;
  if ((rc = check_turned(q, q_stride_tok, q_stride_head, hq, t_total, "q"))) return rc;
  if ((rc = check_turned(q_out, q_out_stride_tok, q_out_stride_head, hq, t_total, "q_out"))) return rc;
  if ((rc = check_turned(k, k_stride_tok, k_stride_head, hk, t_total, "k"))) return rc;
  if ((rc = check_turned(k_out, k_out_stride_tok, k_out_stride_head, hk, t_total, "k_out"))) return rc;
  if ((q == q_out && hq > 0 && (q_stride_tok != q_out_stride_tok || q_stride_head != q_out_stride_head)) ||
      (k == k_out && hk > 0 && (k_stride_tok != k_out_stride_tok || k_stride_head != k_out_stride_head)))
    return fail(KDA_ERR_INVALID_ARGUMENT, "in place, the strides of input and output must agree.");
  if (!positions && (!cu_seqlens || !kv_lens))
    return fail(KDA_ERR_INVALID_ARGUMENT, "positions, or cu_seqlens and kv_lens, must not be NULL.");
  kda::RopeParams p;
  memset(&p, 0, sizeof(p));
  p.q = {static_cast<const __nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(q_out), q_stride_tok, q_stride_head,
         q_out_stride_tok, q_out_stride_head};
  p.k = {static_cast<const __nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(k_out), k_stride_tok, k_stride_head,
         k_out_stride_tok, k_out_stride_head};
  p.hq = hq; p.hk = hk; p.t_total = t_total; p.pairs = rotation->pairs;
  p.turns = reinterpret_cast<const unsigned long long*>(rotation->turns);
  p.amplitude = rotation->amplitude;
  p.positions = positions; p.cu_seqlens = cu_seqlens; p.kv_lens = kv_lens; p.n_req = n_req;
  if (kda::launch_rope(p, rotation->interleaved != 0, dtype == KDA_DTYPE_FP16, static_cast<cudaStream_t>(stream)) != 0)
    return cuda_fail("kda_rope launch");
  return ok();
}

}  // extern "C"
