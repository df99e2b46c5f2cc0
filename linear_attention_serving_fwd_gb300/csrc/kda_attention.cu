// Causal softmax attention of a step's packed tokens over the paged
// key/value cache, with an optional sliding window and first tokens that
// stay visible.
//
// For the token at position p, query head h and the visible keys j:
//   s_j = scale <q, k_j>,  out = sum_j e^{s_j} v_j / sum_j e^{s_j},
// formed in one pass over the keys with the running maximum m of s, the sum
// l = sum e^{s_j - m} and the accumulator o = sum e^{s_j - m} v_j, both
// multiplied by e^{m_old - m_new} when the maximum grows.
#include <math_constants.h>

#include "kda_kv.cuh"

namespace kda {
namespace {

constexpr int ROW_THREADS = 256;

// One row (token, query head) by one warp, four of the 128 dimensions a lane.
// first, kv: the request's position of its first token and its cached tokens.
template <bool FP16>
__device__ __forceinline__ void attend_row(const AttentionParams& p, int b, int tok, int head, int pos, int kv) {
  const int lane = threadIdx.x & 31;
  const int kvh = head / (p.hq / p.hkv), page = 1 << p.page_shift;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -CUDART_INF_F, l = 0.f;
  load_act4<FP16>(p.q + (int64_t)tok * p.q_st + (int64_t)head * p.q_sh + lane * 4, q);
  const int hi = min(pos + 1, kv), lo = p.window ? max(0, pos + 1 - p.window) : 0;
  const int32_t* table = p.table + (int64_t)b * p.table_stride;
  const __nv_bfloat16* kc = p.kc + (int64_t)kvh * p.kc_sh + lane * 4;
  const __nv_bfloat16* vc = p.vc + (int64_t)kvh * p.vc_sh + lane * 4;
  for (int part = 0; part < 2; ++part) {
    const int end = part == 0 ? min(p.sinks, lo) : hi;
    int j = part == 0 ? 0 : lo;
    while (j < end) {
      const int stop = min(end, ((j >> p.page_shift) + 1) << p.page_shift);
      const int pg = table[j >> p.page_shift];
      if (pg < 0 || pg >= p.n_pages) {
        if (pg >= 0) set_error(p.err, ERR_INDEX);
        j = stop;
        continue;
      }
      for (; j < stop; ++j) {
        const int row = j & (page - 1);
        float k[4], v[4];
        load_act4<FP16>(kc + pg * p.kc_sp + row * p.kc_st, k);
        load_act4<FP16>(vc + pg * p.vc_sp + row * p.vc_st, v);
        const float s = p.scale * warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]);
        const float top = fmaxf(m, s);
        if (top == -CUDART_INF_F && !(s != s)) continue;  // e^s = 0, and no maximum yet
        const float corr = m == -CUDART_INF_F ? 0.f : expf(m - top), w = expf(s - top);
        l = l * corr + w;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = o[i] * corr + w * v[i];
        m = top;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* out = p.out + ((int64_t)tok * p.hq + head) * D + lane * 4;
  *reinterpret_cast<uint2*>(out) = make_uint2(act_pack2<FP16>(o[0] * inv, o[1] * inv), act_pack2<FP16>(o[2] * inv, o[3] * inv));
  if (p.lse && lane == 0) p.lse[(int64_t)tok * p.hq + head] = l == 0.f ? -CUDART_INF_F : m + logf(l);
}

// A request's tokens and lengths, checked; false: no tokens to run.
__device__ __forceinline__ bool request(const AttentionParams& p, int b, int& t0, int& n, int& kv, bool report) {
  t0 = p.cu_seqlens[b];
  const int t1 = p.cu_seqlens[b + 1];
  const int most = p.table_cols << p.page_shift;
  kv = p.kv_lens[b];
  if (t0 < 0 || t1 < t0 || t1 > p.t_total) {
    if (report) set_error(p.err, ERR_INDEX);
    return false;
  }
  n = t1 - t0;
  if (kv < 0 || kv > most) {
    if (report) set_error(p.err, ERR_INDEX);
    kv = kv < 0 ? 0 : most;
  }
  return n > 0;
}

template <bool FP16>
__global__ void __launch_bounds__(ROW_THREADS) attention_rows_kernel(AttentionParams p) {
  const int b = blockIdx.y;
  int t0, n, kv;
  if (!request(p, b, t0, n, kv, blockIdx.x == 0 && threadIdx.x == 0)) return;
  const int64_t rows = (int64_t)n * p.hq;
  for (int64_t r = (int64_t)blockIdx.x * (ROW_THREADS / 32) + (threadIdx.x >> 5); r < rows;
       r += (int64_t)gridDim.x * (ROW_THREADS / 32)) {
    const int i = (int)(r / p.hq), head = (int)(r % p.hq);
    attend_row<FP16>(p, b, t0 + i, head, kv - n + i, kv);
  }
}

}  // namespace

size_t attention_workspace_bytes() { return KDA_ATTENTION_ZEROED_BYTES; }

int launch_attention(const AttentionParams& p, bool fp16, void* workspace, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.t_total * p.hq;
  const int64_t blocks = (rows + ROW_THREADS / 32 - 1) / (ROW_THREADS / 32);
  trace_begin("attention", stream);
  for (int b0 = 0; b0 < p.n_req; b0 += 65535) {
    AttentionParams part = p;
    part.cu_seqlens += b0;
    part.kv_lens += b0;
    part.table += b0 * p.table_stride;
    const int n = p.n_req - b0 < 65535 ? p.n_req - b0 : 65535;
    const dim3 grid((unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), n);
    if (fp16) attention_rows_kernel<true><<<grid, ROW_THREADS, 0, stream>>>(part);
    else attention_rows_kernel<false><<<grid, ROW_THREADS, 0, stream>>>(part);
  }
  trace_end(stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace kda
