// The paged key/value cache in 8 bits: the write of keys and values (append)
// and their read-back (read, of the 16-bit cache too).
//
// A block is 16 rows of a page and one head.  With m the largest finite
// magnitude of its new tokens and e the least with m <= 448 2^e, its scale is
// 2^e, or the scale before where that is larger and rows before the new ones
// hold tokens; a number is x 2^-e rounded to e4m3.  Powers of two cost no
// precision (e4m3 has an exponent of its own) and make the second rounding of
// earlier rows, when the scale grows, exact but for numbers below e4m3's normal range.
//
// Both are bound by memory where they are large: 30352 tokens of 8 heads are written
// in 34 us (5.5 TB/s of what is read and written), 75,000 read back in 82 us (5.6
// TB/s, two thirds of it writes).  A decode step's write is a chain of loads: slots,
// then the new row and the block's scale, then its earlier rows where the scale
// grows: 256 tokens 5.65 us.
#include <cuda_fp8.h>

#include "kda_kv.cuh"

namespace kda {
namespace {

constexpr int QB = KDA_KV_BLOCK;
constexpr int LEAST = -48, MOST = 48;  // exponents of the scales

__device__ __forceinline__ float power(int e) { return __int_as_float((e + 127) << 23); }

// Least e with amax <= 448 2^e, within the scales' range: 448 = 1.75 2^8.
__device__ __forceinline__ int exponent(float amax) {
  const int bits = __float_as_int(amax);
  const int e = (bits >> 23) - 127 - ((bits & 0x7fffff) > 0x600000 ? 7 : 8);
  return max(LEAST, min(MOST, e));
}

// a to the lower byte
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 unpack_e4m3(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
template <bool FP16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if constexpr (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// Largest of both halves' magnitudes; as whole numbers they are in order,
// infinities and NaN above all others.
__device__ __forceinline__ uint32_t max_halves(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

// A warp looks for blocks' first tokens among ``window`` tokens and writes one
// head of k or of v of those blocks: lane l holds 8 dimensions of the rows of
// one parity, so that a load or store of the warp is two whole rows.  One warp has
// a block's new rows, its scale and its earlier rows to itself, so nothing is
// agreed on with others.  Four CTAs an SM (64 registers, 48 bytes spilled): 30352 tokens
// 36.3 -> 33.4 us when it was set.
template <bool FP16>
__global__ void __launch_bounds__(256, 4) kv_quant_append_kernel(KvQuantAppendParams p) {
  constexpr uint32_t LARGEST = FP16 ? 0x7bffu : 0x7f7fu;  // finite
  const int lane = threadIdx.x & 31, piece = lane & 15, odd = lane >> 4;
  const int64_t unit = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int per = p.c.hkv * 2, h = (int)(unit % per) >> 1;
  const bool values = unit & 1;
  const int64_t t0 = unit / per * p.window;
  if (t0 >= p.t_total) return;
  const int64_t rows = (int64_t)p.c.n_pages << p.c.page_shift;
  // first tokens of blocks
  bool first = false;
  const int64_t mine = t0 + lane;
  if (lane < p.window && mine < p.t_total) {
    const int slot = p.slot_map[mine];
    if (slot >= rows) {
      set_error(p.err, ERR_INDEX);
    } else if (slot >= 0) {
      const int before = mine > 0 ? p.slot_map[mine - 1] : -1;
      first = before < 0 || before / QB != slot / QB;
      if (!first && slot != before + 1) set_error(p.err, ERR_INDEX);
    }
  }
  const __nv_bfloat16* from = values ? p.v + h * p.v_sh : p.k + h * p.k_sh;
  const int64_t st = values ? p.v_st : p.k_st;
  uint8_t* cache = values ? p.c.v + h * p.c.v_sh : p.c.k + h * p.c.k_sh;
  const int64_t c_sp = values ? p.c.v_sp : p.c.k_sp, c_st = values ? p.c.v_st : p.c.k_st;
  float* scales = values ? p.c.v_scale : p.c.k_scale;
  for (unsigned todo = __ballot_sync(0xffffffffu, first); todo; todo &= todo - 1) {
    const int64_t t = t0 + __ffs(todo) - 1;
    // the block's tokens: those that follow one by one
    int next = -1, near = -1;
    if (lane < QB && t + lane < p.t_total) next = p.slot_map[t + lane];
    if (t - 32 + lane >= 0) near = p.slot_map[t - 32 + lane];
    const int slot = __shfl_sync(0xffffffffu, next, 0);
    // Tokens of the block among the 32 before, that these do not follow: their warp has
    // it.  (256 tokens 5.4 -> 5.65 us, 30352 tokens 33.8 -> 34.05 us.)
    if (__any_sync(0xffffffffu, near >= 0 && near / QB == slot / QB)) {
      if (lane == 0) set_error(p.err, ERR_INDEX);
      continue;
    }
    const int r0 = slot & (QB - 1);
    const unsigned run = __ballot_sync(0xffffffffu, lane < QB - r0 && next == slot + lane);
    const int n = __ffs(~run) - 1;
    const int64_t pg = slot >> p.c.page_shift;
    const int row = slot & ((1 << p.c.page_shift) - 1);
    float* scale = scales + ((pg * p.c.hkv + h) << (p.c.page_shift - 4)) + row / QB;
    const float was = r0 > 0 ? *scale : 0.f;
    uint4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = 2 * j + odd;
      x[j] = i < n ? *reinterpret_cast<const uint4*>(from + (t + i) * st + piece * 8) : make_uint4(0, 0, 0, 0);
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max_halves(max_halves(max_halves(max_halves(m, x[j].x), x[j].y), x[j].z), x[j].w);
    m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    if (m > LARGEST) {  // only finite numbers count
      m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
          if (a <= LARGEST) m = max(m, a);
          if (b <= LARGEST) m = max(m, b);
        }
      }
      m = __reduce_max_sync(0xffffffffu, m);
    }
    const float need = power(exponent(unpack16<FP16>(m).x));
    // earlier tokens keep the larger scale; a scale that is none gives way
    const bool kept = r0 > 0 && was >= need && was <= power(MOST);
    const float now = kept ? was : need, inv = kept ? 1.f / was : power(-exponent(unpack16<FP16>(m).x));
    uint8_t* out = cache + pg * c_sp + (int64_t)row * c_st + piece * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = 2 * j + odd;
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      uint32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = unpack16<FP16>(w[k]);
        y[k] = pack_e4m3(v.x * inv, v.y * inv);
      }
      if (i < n) *reinterpret_cast<uint2*>(out + i * c_st) = make_uint2(y[0] | y[1] << 16, y[2] | y[3] << 16);
    }
    if (r0 > 0 && !kept) {  // all earlier rows at once: one after another took 5 us
      const float ratio = was * inv;
      uint2 old[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (2 * j + odd < r0) old[j] = *reinterpret_cast<const uint2*>(out + (2 * j + odd - r0) * c_st);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = unpack_e4m3((k < 2 ? old[j].x : old[j].y) >> (k & 1) * 16);
          y[k] = pack_e4m3(v.x * ratio, v.y * ratio);
        }
        if (2 * j + odd < r0)
          *reinterpret_cast<uint2*>(out + (2 * j + odd - r0) * c_st) = make_uint2(y[0] | y[1] << 16, y[2] | y[3] << 16);
      }
    }
    if (lane == 0 && !kept) *scale = now;
  }
}

// 16 dimensions of a key and of a value row per thread.
template <bool QUANT, bool FP16>
__global__ void __launch_bounds__(256) kv_read_kernel(KvReadParams p) {
  const int64_t i = blockIdx.x * 256ll + threadIdx.x;
  const int64_t th = i / (D / 16);
  const int c = (int)(i % (D / 16)) * 16;
  const int64_t t = th / p.hkv;
  const int h = (int)(th % p.hkv);
  if (t >= p.t_total) return;
  const int slot = p.slot_map[t];
  const bool bad = slot >= ((int64_t)p.n_pages << p.page_shift);
  if (bad) set_error(p.err, ERR_INDEX);
  uint4 k[2] = {}, v[2] = {};
  if (slot >= 0 && !bad) {
    const int64_t pg = slot >> p.page_shift;
    const int row = slot & ((1 << p.page_shift) - 1);
    if constexpr (QUANT) {
      const int64_t s = ((pg * p.hkv + h) << (p.page_shift - 4)) + row / QB;
      const uint4 a = *reinterpret_cast<const uint4*>(p.c.k + pg * p.c.k_sp + row * p.c.k_st + h * p.c.k_sh + c);
      const uint4 b = *reinterpret_cast<const uint4*>(p.c.v + pg * p.c.v_sp + row * p.c.v_st + h * p.c.v_sh + c);
      const float ks = p.c.k_scale[s], vs = p.c.v_scale[s];
      auto widen = [](uint32_t four, float scale, uint32_t& lo, uint32_t& hi) {
        const float2 x = unpack_e4m3(four), y = unpack_e4m3(four >> 16);
        lo = act_pack2<FP16>(x.x * scale, x.y * scale);
        hi = act_pack2<FP16>(y.x * scale, y.y * scale);
      };
      widen(a.x, ks, k[0].x, k[0].y);
      widen(a.y, ks, k[0].z, k[0].w);
      widen(a.z, ks, k[1].x, k[1].y);
      widen(a.w, ks, k[1].z, k[1].w);
      widen(b.x, vs, v[0].x, v[0].y);
      widen(b.y, vs, v[0].z, v[0].w);
      widen(b.z, vs, v[1].x, v[1].y);
      widen(b.w, vs, v[1].z, v[1].w);
    } else {
      const uint4* a = reinterpret_cast<const uint4*>(p.kc + pg * p.kc_sp + row * p.kc_st + h * p.kc_sh + c);
      const uint4* b = reinterpret_cast<const uint4*>(p.vc + pg * p.vc_sp + row * p.vc_st + h * p.vc_sh + c);
      k[0] = a[0];
      k[1] = a[1];
      v[0] = b[0];
      v[1] = b[1];
    }
  }
  uint4* to = reinterpret_cast<uint4*>(p.k + th * D + c);
  to[0] = k[0];
  to[1] = k[1];
  to = reinterpret_cast<uint4*>(p.v + th * D + c);
  to[0] = v[0];
  to[1] = v[1];
}

}  // namespace

int launch_kv_quant_append(KvQuantAppendParams p, bool fp16, cudaStream_t stream) {
  // Blocks begin at every token of a decode step, at every 16th of a prompt: a
  // warp a token while that fills the machine once, then up to 16 tokens a warp.
  const int64_t all = (int64_t)p.t_total * p.c.hkv * 2;
  p.window = (int)(all >= 152 * 64 * 16 ? 16 : all <= 152 * 64 ? 1 : all / (152 * 64));
  const int64_t units = ((int64_t)p.t_total + p.window - 1) / p.window * p.c.hkv * 2;
  const unsigned blocks = (unsigned)((units + 7) / 8);
  trace_begin("kv_quant_append", stream);
  if (fp16) kv_quant_append_kernel<true><<<blocks, 256, 0, stream>>>(p);
  else kv_quant_append_kernel<false><<<blocks, 256, 0, stream>>>(p);
  trace_end(stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_kv_read(const KvReadParams& p, bool quant, bool fp16, cudaStream_t stream) {
  const int64_t threads = (int64_t)p.t_total * p.hkv * (D / 16);
  const unsigned blocks = (unsigned)((threads + 255) / 256);
  trace_begin(quant ? "kv_quant_read" : "kv_read", stream);
  if (!quant) kv_read_kernel<false, false><<<blocks, 256, 0, stream>>>(p);
  else if (fp16) kv_read_kernel<true, true><<<blocks, 256, 0, stream>>>(p);
  else kv_read_kernel<true, false><<<blocks, 256, 0, stream>>>(p);
  trace_end(stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace kda
