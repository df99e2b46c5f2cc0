// Rotary positions: pairs of a row turned by the angle of its token's position.
//
// An angle is a fraction of a turn in 64 bits, position times the pair's turns
// modulo 2^64: exact however far the position, where a product in fp32 (or of
// an fp32 frequency) would have lost the angle.  The top of it, as a signed
// number, is at most half a turn, and its cosine and sine are formed once per
// token and pair for all heads.
//
// Bound by memory: every row is read and written once, 32 bytes a thread.
#include "kda_kv.cuh"

namespace kda {
namespace {

constexpr int THREADS = 256, ROW_THREADS = 8, ROWS = THREADS / ROW_THREADS;
constexpr int MAX_TOKENS = 8;  // of a CTA, a warp each for the search

template <bool FP16>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  return act_f2<FP16>(reinterpret_cast<const __nv_bfloat16*>(&w));
}

// Position of token t, by one warp; false if it belongs to no request.
__device__ __forceinline__ bool find_position(const RopeParams& p, int t, int& pos) {
  if (p.positions) {
    pos = p.positions[t];
    return true;
  }
  // the last request that begins at or before t: 32 probes a round
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.n_req;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const unsigned before = __ballot_sync(0xffffffffu, lane * step < n && p.cu_seqlens[at] <= t);
    const int last = before ? 31 - __clz(before) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  const int t0 = p.cu_seqlens[lo], t1 = p.cu_seqlens[lo + 1];
  pos = p.kv_lens[lo] - (t1 - t);
  return t0 <= t && t < t1;
}

template <bool PAIRS, bool FP16>
__global__ void __launch_bounds__(THREADS) rope_kernel(RopeParams p) {
  __shared__ float2 turn[MAX_TOKENS][D / 2];
  __shared__ int pos[MAX_TOKENS];
  __shared__ bool real[MAX_TOKENS];
  const int warp = threadIdx.x >> 5, t0 = blockIdx.x * p.tokens;
  const int n_tok = min(p.tokens, p.t_total - t0), heads = p.hq + p.hk;
  if (warp < n_tok) {
    int x;
    const bool r = find_position(p, t0 + warp, x);
    if ((threadIdx.x & 31) == 0) {
      pos[warp] = x;
      real[warp] = r;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_tok * p.pairs; i += THREADS) {
    const int tok = i / p.pairs, pair = i % p.pairs;
    // modulo 2^64, as a signed fraction: negative positions turn backwards
    const long long a = (long long)((unsigned long long)(long long)pos[tok] * p.turns[pair]);
    float s, c;
    sincospif((float)a * 0x1p-63f, &s, &c);
    turn[tok][pair] = make_float2(c * p.amplitude, s * p.amplitude);
  }
  __syncthreads();
  const int j = threadIdx.x % ROW_THREADS, rot = 2 * p.pairs;
  for (int row = blockIdx.y * ROWS + threadIdx.x / ROW_THREADS; row < n_tok * heads; row += gridDim.y * ROWS) {
    const int tok = row / heads, head = row % heads;
    if (!real[tok]) continue;
    const RopeRows& r = head < p.hq ? p.q : p.k;
    const int h = head < p.hq ? head : head - p.hq;
    const __nv_bfloat16* in = r.in + (int64_t)(t0 + tok) * r.in_st + (int64_t)h * r.in_sh;
    __nv_bfloat16* out = r.out + (int64_t)(t0 + tok) * r.out_st + (int64_t)h * r.out_sh;
    if (rot % 16 == 0) {
      // 8 pairs, or 16 dimensions that stay
      const bool turned = j * 8 < p.pairs;
      const int a = turned ? (PAIRS ? j * 16 : j * 8) : j * 16, b = turned && !PAIRS ? a + p.pairs : a + 8;
      const uint4 xa = *reinterpret_cast<const uint4*>(in + a), xb = *reinterpret_cast<const uint4*>(in + b);
      uint32_t x[4] = {xa.x, xa.y, xa.z, xa.w}, y[4] = {xb.x, xb.y, xb.z, xb.w};
      if (turned) {
        const float2* w = turn[tok] + j * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 u = unpack<FP16>(x[k]), v = unpack<FP16>(y[k]);
          if constexpr (PAIRS) {
            const float2 cu = w[k], cv = w[k + 4];
            x[k] = act_pack2<FP16>(u.x * cu.x - u.y * cu.y, u.y * cu.x + u.x * cu.y);
            y[k] = act_pack2<FP16>(v.x * cv.x - v.y * cv.y, v.y * cv.x + v.x * cv.y);
          } else {
            const float2 c0 = w[2 * k], c1 = w[2 * k + 1];
            x[k] = act_pack2<FP16>(u.x * c0.x - v.x * c0.y, u.y * c1.x - v.y * c1.y);
            y[k] = act_pack2<FP16>(v.x * c0.x + u.x * c0.y, v.y * c1.x + u.y * c1.y);
          }
        }
      }
      *reinterpret_cast<uint4*>(out + a) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(out + b) = make_uint4(y[0], y[1], y[2], y[3]);
    } else {
      // pieces that do not fill 16 bytes: a pair at a time, both of it by one
      // thread, so that a row may be turned in place
      for (int i = j; i < p.pairs; i += ROW_THREADS) {
        const int a = PAIRS ? 2 * i : i, b = PAIRS ? 2 * i + 1 : i + p.pairs;
        const float2 c = turn[tok][i];
        const float x = act_f<FP16>(in[a]), y = act_f<FP16>(in[b]);
        out[a] = act_from_f(x * c.x - y * c.y, FP16);
        out[b] = act_from_f(y * c.x + x * c.y, FP16);
      }
      for (int i = rot + j; i < D; i += ROW_THREADS) out[i] = in[i];
    }
  }
}

}  // namespace

int launch_rope(RopeParams p, bool interleaved, bool fp16, cudaStream_t stream) {
  const int heads = p.hq + p.hk;
  // a CTA's threads hold 32 rows: tokens of few heads share one
  p.tokens = heads >= ROWS ? 1 : ROWS / heads < MAX_TOKENS ? ROWS / heads : MAX_TOKENS;
  const int64_t ctas = ((int64_t)p.t_total + p.tokens - 1) / p.tokens;
  // few tokens: their heads are shared out as well
  const int passes = (p.tokens * heads + ROWS - 1) / ROWS;
  const dim3 grid((unsigned)ctas, ctas < 152 ? passes : 1);
  trace_begin("rope", stream);
  if (interleaved) {
    if (fp16) rope_kernel<true, true><<<grid, THREADS, 0, stream>>>(p);
    else rope_kernel<true, false><<<grid, THREADS, 0, stream>>>(p);
  } else {
    if (fp16) rope_kernel<false, true><<<grid, THREADS, 0, stream>>>(p);
    else rope_kernel<false, false><<<grid, THREADS, 0, stream>>>(p);
  }
  trace_end(stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace kda
