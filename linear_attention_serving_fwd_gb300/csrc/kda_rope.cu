// Rotary positions: pairs of a row turned by the angle of its token's position.
//
// An angle is a fraction of a turn in 64 bits, position times the pair's turns
// modulo 2^64: exact however far the position, where a product in fp32 (or of
// an fp32 frequency) would have lost the angle.  The top of it, as a signed
// number, is at most half a turn, and its cosine and sine are formed once per
// token and pair for all heads.
//
// Bound by memory: every row is read and written once, 32 bytes a thread.  39,000
// tokens of 32 and 8 heads take 127 us (6.3 TB/s, 92 % of a copy's rate); 155 us with
// one token a CTA and one row a thread, whose loads waited for the angles.  A decode step
// of 16 tokens takes 3.5 us, launch and search.
#include "kda_kv.cuh"

namespace kda {
namespace {

constexpr int THREADS = 256, ROW_THREADS = 8, ROWS = THREADS / ROW_THREADS;
constexpr int MAX_TOKENS = 8;  // of a CTA, a warp each for the search
constexpr int BATCH = 2;       // rows that a thread has under way

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
  auto angles = [&]() {
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
  };
  const int j = threadIdx.x % ROW_THREADS, rot = 2 * p.pairs, rows = n_tok * heads;
  const int first = blockIdx.y * ROWS + threadIdx.x / ROW_THREADS, step = gridDim.y * ROWS;
  auto pointers = [&](int row, const __nv_bfloat16*& in, __nv_bfloat16*& out) {
    const int tok = row / heads, head = row % heads;
    const RopeRows& r = head < p.hq ? p.q : p.k;
    const int h = head < p.hq ? head : head - p.hq;
    in = r.in + (int64_t)(t0 + tok) * r.in_st + (int64_t)h * r.in_sh;
    out = r.out + (int64_t)(t0 + tok) * r.out_st + (int64_t)h * r.out_sh;
    return tok;
  };
  if (rot % 16 == 0) {
    // 8 pairs, or 16 dimensions that stay
    const bool turned = j * 8 < p.pairs;
    const int a = turned ? (PAIRS ? j * 16 : j * 8) : j * 16, b = turned && !PAIRS ? a + p.pairs : a + 8;
    // A batch of rows at once, and the first before the angles are known: the
    // loads are what takes time.
    uint4 x[BATCH][2];
    auto load = [&](int row0) {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int row = row0 + i * step;
        if (row >= rows) continue;
        const __nv_bfloat16* in;
        __nv_bfloat16* out;
        pointers(row, in, out);
        x[i][0] = *reinterpret_cast<const uint4*>(in + a);
        x[i][1] = *reinterpret_cast<const uint4*>(in + b);
      }
    };
    load(first);
    angles();
    for (int row0 = first; row0 < rows; row0 += BATCH * step) {
      if (row0 != first) load(row0);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int row = row0 + i * step;
        if (row >= rows) continue;
        const __nv_bfloat16* in;
        __nv_bfloat16* out;
        const int tok = pointers(row, in, out);
        if (!real[tok]) continue;
        uint32_t u[4] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w}, v[4] = {x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
        if (turned) {
          const float2* w = turn[tok] + j * 8;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack<FP16>(u[k]), g = unpack<FP16>(v[k]);
            if constexpr (PAIRS) {
              const float2 cf = w[k], cg = w[k + 4];
              u[k] = act_pack2<FP16>(f.x * cf.x - f.y * cf.y, f.y * cf.x + f.x * cf.y);
              v[k] = act_pack2<FP16>(g.x * cg.x - g.y * cg.y, g.y * cg.x + g.x * cg.y);
            } else {
              const float2 c0 = w[2 * k], c1 = w[2 * k + 1];
              u[k] = act_pack2<FP16>(f.x * c0.x - g.x * c0.y, f.y * c1.x - g.y * c1.y);
              v[k] = act_pack2<FP16>(g.x * c0.x + f.x * c0.y, g.y * c1.x + f.y * c1.y);
            }
          }
        }
        *reinterpret_cast<uint4*>(out + a) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4*>(out + b) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
    return;
  }
  // pieces that do not fill 16 bytes: a pair at a time, both of it by one
  // thread, so that a row may be turned in place.  2 bytes a load: 39,000 tokens
  // turned in 40 of 128 dimensions take 266 us.
  angles();
  for (int row = first; row < rows; row += step) {
    const __nv_bfloat16* in;
    __nv_bfloat16* out;
    const int tok = pointers(row, in, out);
    if (!real[tok]) continue;
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

}  // namespace

int launch_rope(RopeParams p, bool interleaved, bool fp16, cudaStream_t stream) {
  const int heads = p.hq + p.hk;
  // Few tokens: one a CTA, and their heads shared out as well.  Else as many as
  // make some 160 rows, so that the search and the angles are a small part.
  const bool few = (int64_t)p.t_total * heads <= 152 * 4 * ROWS;
  const int most = few ? (heads >= ROWS ? 1 : ROWS / heads) : (160 + heads - 1) / heads;
  p.tokens = most < MAX_TOKENS ? most : MAX_TOKENS;
  const int64_t ctas = ((int64_t)p.t_total + p.tokens - 1) / p.tokens;
  const dim3 grid((unsigned)ctas, few ? (p.tokens * heads + ROWS - 1) / ROWS : 1);
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
