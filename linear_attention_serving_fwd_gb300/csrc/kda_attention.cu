// Causal softmax attention of a step's packed tokens over the paged
// key/value cache, with an optional sliding window and first tokens that
// stay visible.
//
// For the token at position p, query head h and the visible keys j:
//   s_j = scale <q, k_j>,  out = sum_j e^{s_j} v_j / sum_j e^{s_j},
// formed in one pass over the keys with a running reference m of s, the sum
// l = sum e^{s_j - m} and the accumulator o = sum e^{s_j - m} v_j.
//
// Tiles.  The query heads of one key head share every key, so a tile's 128
// rows are (token, head of the group) pairs: 128 / G tokens by G heads.  A
// block is two such tiles.  Keys come in tiles of 128, K and V 32 KB each.
// Per key tile the tensor cores form S = Q K^T (128 x 128 x 128) and
// O += P V (128 x 128 x 128).  S (fp32), the weights P (16 bits, in the columns
// of S that are read first) and O (fp32) of both query tiles fill the 512
// columns of tensor memory; Q, K and V stay in shared memory as the copies left
// them, 64 KB of queries and a ring of five K and V tiles.
//
// Streams.  Each query tile has an S, an O, an issuing warp and two softmax
// warpgroups, one for each half of a tile's keys (a thread: one row, 64 keys):
// while one stream works on its scores, the tensor cores serve the other.  A
// block of one tile (single tokens, short windows) gives both streams the same
// rows and every other key tile, and their results are joined in shared memory;
// the streams lead such blocks in turn, so that two blocks of one key tile run
// side by side (106 requests of at most 17 cached tokens 29.8 -> 23.1 us, mixed
// batches within 2 % either way).
// One warp copies, one lays out the work.  One warpgroup a stream, a thread a
// whole row, was 4 % slower: the steps between the scores' barrier and the
// weights' are a chain that the other stream has to cover.  Steps of 64 keys
// with two S of a stream in tensor memory cover it better, but the products of
// 64 columns read the queries twice as often, at shared memory's full rate, and
// lost 5 % on the whole.
//
// Work.  The (key head, block) pairs in a row, each as long as its key tiles
// (and a lead for what it costs by itself), form one line that is cut into
// equal pieces, one per CTA.  A pair that a cut divides leaves partial results
// (o, m, l) in the workspace; the CTA that finishes the pair last joins them in
// the order of the line, so results do not depend on timing.
//
// Bounds.  Prompt chunks are bound by the chain scores - weights - product of
// two streams on one set of tensor cores: 8192 tokens over 24576 cached, 32
// heads, take 2.77 to 2.97 ms by the chip (1390 to 1295 TFLOP/s) at its power
// limit and 2.5 ms before it; 4096 over 4096 in a short run 1470 to 1515 TFLOP/s,
// tensor cores 64 % busy.  Single tokens are bound by memory: 256 requests over 4.2 GB of keys
// and values take 608 to 626 us (6.9 to 6.75 TB/s).  A single request of 4096
// tokens is a chain of latencies, 14.2 us.
//
// Fewer bits.  The weights are rounded to the values' 16-bit type, which the
// tensor cores ask of both operands: 32-bit weights in two 16-bit parts would
// double the second product.  It takes the outputs' error against 64 bits from
// 1.7e-3 (their own rounding) to 1.8e-3 of their norm in bf16, from 2.1e-4 to
// 2.2e-4 in fp16.  Sums take the weights before they are rounded.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include "kda_kv.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int KT = 128;        // keys per tile
constexpr int ROWS = 128;      // rows per query tile
constexpr int STAGES = 5;      // K or V tiles in shared memory
constexpr int TILE_BYTES = KT * D * 2;
constexpr int HALF_BYTES = TILE_BYTES / 2;  // 64 of the 128 dimensions
constexpr int MERGE_ROWS = 64; // rows whose joining leaves the first query tile alone
constexpr int RING = 4;        // items ahead
constexpr int MASKS = 8;       // page masks of the K tiles in flight
constexpr int THREADS = 640;
constexpr int SOFTMAX_WARPS = 16;  // two warpgroups a stream
constexpr int LOAD_WARP = 16, PLAN_WARP = 17, MMA_WARP = 18;  // MMA_WARP + 1: the second stream's
// Lead of a block of two tiles and of one, in key tiles.  Measured against none:
// prompts of 2048 tokens 246 -> 193 us, a window of 1024 over 8001 tokens 114 ->
// 83 us, 128 single tokens 393 -> 369 us; 6 and 2, or 4 and 1, are 1 to 5 % behind.
constexpr int LEAD_TWO = 4, LEAD_ONE = 2;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// The running reference follows the row's maximum only when 64 weights have
// come to sum to more: until then weights above one stand, and the accumulator
// is left alone.  A weight rounds to 16 bits with the same relative error
// whatever its size.
constexpr float LIMIT = 32768.f;
// fp16 weights are formed 2^7 larger: none passes LIMIT (65504 is the largest
// number), and the smallest normal one (2^-14) is then 2^-21 of the reference.
template <bool FP16>
constexpr float WEIGHT_EXP = FP16 ? 7.f : 0.f;

struct Item {
  int b, kvh;
  int tok, n_tok;      // first packed token, tokens of the block
  int pos, kv;         // position of the first token, cached tokens
  int i0, i1;          // this part's range of the key tile list
  int n_sink, t_lo;    // list: tiles 0 .. n_sink - 1, then t_lo, t_lo + 1, ..
  int lo, hi, sink_hi; // keys that some row sees: [lo, hi) and [0, sink_hi)
  int act[2][3];       // a query tile sees list entries below [0] and in [[1], [2])
  int first, parts;    // CTA of the first part, parts of the pair
  int part;            // this part's number
  int lead;            // block of one tile: the stream that takes its even key tiles and the results
                       // b < 0 ends the work
};

struct Smem {
  uint64_t kv_full[STAGES], kv_empty[STAGES];
  uint64_t ring_full[RING], ring_empty[RING];
  uint64_t q_full, q_empty, q_read, merge_full, merge_free;
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t turn[2], drained[2];
  Item ring[RING];
  int page_mask[MASKS];
  long long sums[SOFTMAX_WARPS];
  long long total;
  int start_b;
  long long start_before;
  uint32_t tmem;
  int dead;
  int beat;    // changes while rows are formed again, which may take longer than a wait
  int joined;  // results of two streams joined so far
  int last[2];
  unsigned poisoned[2][2][4];  // rows whose sum is a number but not their result, by stream and half
  float share[2][2][ROWS];     // what the halves of a row tell each other
};

struct Params {
  AttentionParams a;
  int group, tile_tok;     // G, tokens per query tile
  int n_cta;
  int min_piece;           // least tiles per CTA
  int boxes;               // pages per key tile (1 when a page holds more)
  // K and V tiles in shared memory: rows of 128 bytes (64 of the dimensions) in
  // groups of 8; bytes from group to group and from half to half of a row.  With
  // joined copies a box holds whole rows, half after half in each group, and a
  // page's box begins at group page * page_groups and outer place
  // page * page_outer + head of the map.
  int joined, group_bytes, half_bytes, page_groups, page_outer;
  unsigned* counters;      // [n_cta][2], zero between calls
  float2* part_ml;         // [n_cta][2 slots][2 tiles][ROWS]
  float4* part_o;          // [n_cta][2 slots][2 tiles][ROWS / 8][32][8]: 16-byte pieces of 8 rows side by side
};

// Joined copies halve the number of boxes: with pages of 16, where the copy
// engine's boxes are what limits, single tokens over 4096 cached take 343 us
// instead of 472; with pages of 64 and more the two are alike.

// hardware barriers: a pair of warps that share rows (stream, quarter), a stream's eight warps
constexpr int PAIR_BAR = 1, STREAM_BAR = 9;

// --- waits ---------------------------------------------------------------------
// A wait that expires (bounded as all waits are) marks the CTA: its other waits
// then return at once, and the roles run out.  What they still do stays inside
// the CTA's own memory; only the ring of items is not read on.
// The time since the last sign of life counts: one row has as many keys as the
// request, and 32 of them may be formed again between two waits of the others.
struct Patience {
  uint64_t t0 = 0;
  int beat = 0;
  __device__ __forceinline__ bool over(const volatile Smem& sm) {
    const uint64_t t = globaltimer_ns();
    const int now = sm.beat;
    if (t0 == 0 || now != beat) {
      t0 = t;
      beat = now;
    }
    return t - t0 > WAIT_NS;
  }
};
__device__ __noinline__ void wait_slow(uint64_t* bar, uint32_t parity, volatile Smem& sm, unsigned* err) {
  Patience patience;
  for (uint32_t i = 0; i < WAIT_CAP && !sm.dead; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if (patience.over(sm)) break;
  }
  sm.dead = 1;
  set_error(err, ERR_TIMEOUT);
}
// without a time hint: with one, waking took longer
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n" : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, Smem& sm, unsigned* err) {
  if (!try_wait(bar, parity)) wait_slow(bar, parity, sm, err);
}
__device__ __forceinline__ bool is_dead(const Smem& sm) { return *(const volatile int*)&sm.dead != 0; }
__device__ __forceinline__ void wait_joined(Smem& sm, int count, unsigned* err) {
  Patience patience;
  for (uint32_t i = 0;; ++i) {
    int joined;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(joined) : "r"(smem_u32(&sm.joined)) : "memory");
    if (joined >= count || is_dead(sm)) break;
    __nanosleep(64);
    if (i == WAIT_CAP || patience.over(sm)) {
      *(volatile int*)&sm.dead = 1;
      set_error(err, ERR_TIMEOUT);
      break;
    }
  }
  __syncwarp();
}
// the same; false once the CTA is marked
__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, Smem& sm, unsigned* err) {
  if (try_wait(bar, parity)) return true;
  wait_slow(bar, parity, sm, err);
  return !is_dead(sm);
}
// by a whole warp, which runs warp-wide instructions next
__device__ __forceinline__ void warp_wait(uint64_t* bar, uint32_t parity, Smem& sm, unsigned* err) {
  wait(bar, parity, sm, err);
  __syncwarp();
}

// --- PTX -----------------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// 32 bytes, a whole sector: rows lie far apart, so a warp's store takes the
// memory pipe a cycle a row, whatever its width
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void tma_load5(void* dst, const CUtensorMap* map, int c3, int c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(0), "r"(c3), "r"(c4), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load4(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)) : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], B MN-major
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// 128-byte-swizzled operands as the copies leave them: 64 dimensions (128
// bytes) a row, 8-row groups ``group`` bytes apart, the other 64 dimensions
// ``half`` bytes further.  K-major (the dimensions are summed over; the leading
// offset is not used) or MN-major (the rows are).
__device__ __forceinline__ uint64_t smem_desc_rows(uint32_t saddr, uint32_t group, uint32_t half, bool mn) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(mn ? half >> 4 : 1u) << 16;
  d |= (uint64_t)(group >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// --- rows whose result is not finite -----------------------------------------------
// The tiles' products multiply the values of hidden keys by a weight of 0, which
// is not 0 where such a value is NaN or infinite, and weights against a reference
// that stands may sum to more than fp32 holds.  (Hidden scores never count: a row
// whose sum is NaN is NaN.)  So the rest of the rows that are not finite are
// looked at again: where the values that they see account for it, the result
// stands; else the row is formed again from the keys that it sees alone.
// Bound by latency, groups of 8 keys at once.  A NaN or an infinity early in the
// cache: 8192 tokens over 24576 of 32 heads 13.7 ms (2.6 without it), 512 over
// 7680 of 8 heads 0.3 ms.  A NaN among the tokens themselves, which half a tile's
// rows do not see: 126 ms and 26 ms; 256 over 130,816 of 8 heads 548 ms.
constexpr int GROUP = 8;

// Four dimensions a lane of the rows' values: bits 0-3 NaN, 4-7 inf, 8-11 -inf.
__device__ __forceinline__ unsigned classify(const float (&v)[4]) {
  unsigned f = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (v[i] != v[i]) f |= 1u << i;
    if (v[i] == CUDART_INF_F) f |= 16u << i;
    if (v[i] == -CUDART_INF_F) f |= 256u << i;
  }
  return f;
}

// What the values of keys [from, to) hold (none where from >= to: rows of a narrow
// window may share no key), by a warp that takes every other group of them; ends early where every dimension has a NaN.
template <bool FP16>
__device__ __forceinline__ unsigned scan_values(const AttentionParams& p, Smem& sm, const int32_t* table, int kvh, int from, int to,
                                                int half, unsigned f) {
  if (from >= to) return f;
  const int lane = threadIdx.x & 31, page = 1 << p.page_shift;
  const __nv_bfloat16* vc = p.vc + (int64_t)kvh * p.vc_sh + lane * 4;
#pragma unroll 1
  for (int g = from / GROUP + ((from / GROUP ^ half) & 1); g * GROUP < to; g += 2) {
    if (__all_sync(0xffffffffu, (f & 15) == 15)) break;
    if (lane == 0) *(volatile int*)&sm.beat = (int)clock();
    const int pg = table[(g * GROUP) >> p.page_shift];  // pages hold whole groups
    if (pg < 0 || pg >= p.n_pages) continue;
    float poison = 0.f;
    uint2 raw[GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      const int row = min(max(g * GROUP + i, from), to - 1) & (page - 1);
      raw[i] = *reinterpret_cast<const uint2*>(vc + pg * p.vc_sp + row * p.vc_st);
    }
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      float v[4];
      load_act4<FP16>(reinterpret_cast<const __nv_bfloat16*>(&raw[i]), v);
      poison += v[0] * 0.f + v[1] * 0.f + v[2] * 0.f + v[3] * 0.f;
    }
    if (poison != 0.f) {
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        float v[4];
        load_act4<FP16>(reinterpret_cast<const __nv_bfloat16*>(&raw[i]), v);
        f |= classify(v);
      }
    }
  }
  return f;
}

// The definition row by row, by one warp, four of the 128 dimensions a lane.
template <bool FP16>
__device__ __forceinline__ void attend_row(const AttentionParams& p, Smem& sm, int b, int tok, int head, int pos, int kv) {
  const int lane = threadIdx.x & 31;
  const int kvh = head / (p.hq / p.hkv), page = 1 << p.page_shift;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -CUDART_INF_F, l = 0.f;
  load_act4<FP16>(p.q + (int64_t)tok * p.q_st + (int64_t)head * p.q_sh + lane * 4, q);
  const int hi = min(pos + 1, kv), lo = p.window ? max(0, pos + 1 - p.window) : 0;
  const int32_t* table = p.table + (int64_t)b * p.table_stride;
  const __nv_bfloat16* kc = p.kc + (int64_t)kvh * p.kc_sh + lane * 4;
  const __nv_bfloat16* vc = p.vc + (int64_t)kvh * p.vc_sh + lane * 4;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int from = part == 0 ? 0 : lo, to = part == 0 ? min(min(p.sinks, lo), hi) : hi;
#pragma unroll 1
    for (int g = from / GROUP; g * GROUP < to; ++g) {
      if (lane == 0) *(volatile int*)&sm.beat = (int)clock();
      const int pg = table[(g * GROUP) >> p.page_shift];
      if (pg < 0 || pg >= p.n_pages) continue;
      uint2 raw[GROUP];
      float s[GROUP], top = m;
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        const int row = min(max(g * GROUP + i, from), to - 1) & (page - 1);
        float k[4];
        load_act4<FP16>(kc + pg * p.kc_sp + row * p.kc_st, k);
        raw[i] = *reinterpret_cast<const uint2*>(vc + pg * p.vc_sp + row * p.vc_st);
        s[i] = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
      }
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        s[i] = p.scale * warp_sum(s[i]);
        if (g * GROUP + i >= from && g * GROUP + i < to) top = fmaxf(top, s[i]);
      }
      const float corr = m == -CUDART_INF_F ? 0.f : expf(m - top);
      m = top;
      l *= corr;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] *= corr;
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        if (g * GROUP + i < from || g * GROUP + i >= to) continue;
        // a score of -inf has a weight of 0, whether there is a maximum yet or not
        const float w = s[i] == -CUDART_INF_F ? 0.f : expf(s[i] - top);
        float v[4];
        load_act4<FP16>(reinterpret_cast<const __nv_bfloat16*>(&raw[i]), v);
        l += w;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += w * v[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = l == 0.f ? 0.f : o[j] / l;
  __nv_bfloat16* out = p.out + ((int64_t)tok * p.hq + head) * D + lane * 4;
  *reinterpret_cast<uint2*>(out) = make_uint2(act_pack2<FP16>(o[0], o[1]), act_pack2<FP16>(o[2], o[3]));
  if (p.lse && lane == 0) p.lse[(int64_t)tok * p.hq + head] = l == 0.f ? -CUDART_INF_F : m + logf(l);
}

// Rows ``bad`` of 32 of a tile, whose results stand in memory, by the two warps
// that share them.  A visible value early in a long cache reaches every row after
// it: the values that all of them see are read once for all.
template <bool FP16>
__device__ __forceinline__ void mend_rows(const Params& p, Smem& sm, int s, int half, int quarter, int bar, const Item& it, int tile,
                                          unsigned bad) {
  const int lane = threadIdx.x & 31, r = quarter * 32 + lane;
  const bool mine = (bad >> lane) & 1;
  const int tb = tile * p.tile_tok + r / p.group, pos = it.pos + tb;
  const int hi = __reduce_min_sync(0xffffffffu, mine ? min(pos + 1, it.kv) : 0x7fffffff);
  const int lo = __reduce_max_sync(0xffffffffu, mine && p.a.window ? max(0, pos + 1 - p.a.window) : 0);
  const int32_t* table = p.a.table + (int64_t)it.b * p.a.table_stride;
  unsigned f = 0;
  f = scan_values<FP16>(p.a, sm, table, it.kvh, 0, min(min(p.a.sinks, lo), hi), half, f);
  f = scan_values<FP16>(p.a, sm, table, it.kvh, lo, hi, half, f);
  sm.share[s][half][r] = __uint_as_float(f);
  named_bar_sync(bar, 64);
  f |= __float_as_uint(sm.share[s][half ^ 1][r]);
  int turn = 0;
  while (bad) {
    const int src = __ffs(bad) - 1, row = quarter * 32 + src;
    bad &= bad - 1;
    if ((turn++ & 1) != half) continue;
    const int i = tile * p.tile_tok + row / p.group, tok = it.tok + i, head = it.kvh * p.group + row % p.group;
    float o[4];
    load_act4<FP16>(p.a.out + ((int64_t)tok * p.a.hq + head) * D + lane * 4, o);
    bool stands = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool nan = (f >> j) & 1, inf = (f >> (4 + j)) & 1, neg = (f >> (8 + j)) & 1;
      if (o[j] != o[j]) stands = stands && (nan || (inf && neg));
      else if (o[j] == CUDART_INF_F) stands = stands && inf;
      else if (o[j] == -CUDART_INF_F) stands = stands && neg;
    }
    if (!__all_sync(0xffffffffu, stands)) attend_row<FP16>(p.a, sm, it.b, tok, head, it.pos + i, it.kv);
  }
}

// --- the line of work ----------------------------------------------------------------
// The line's places are 64 bits, but seldom need them: a 64-bit division costs
// several times a 32-bit one, and a single token's call waits for a few.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (unsigned long long)(a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// A request's tokens and lengths, checked; n = 0: no tokens to run.
__device__ __forceinline__ void request(const AttentionParams& p, int b, int& t0, int& n, int& kv, bool report) {
  t0 = p.cu_seqlens[b];
  const int t1 = p.cu_seqlens[b + 1];
  const int most = p.table_cols << p.page_shift;
  kv = p.kv_lens[b];
  n = t1 - t0;
  if (t0 < 0 || t1 < t0 || t1 > p.t_total) {
    if (report) set_error(p.err, ERR_INDEX);
    n = 0;
  }
  if (kv < 0 || kv > most) {
    if (report) set_error(p.err, ERR_INDEX);
    kv = kv < 0 ? 0 : most;
  }
}

// Key tiles of block k of a request of n tokens: fills the item's list.
__device__ __forceinline__ int block_tiles(const Params& p, int n, int kv, int k, Item& it) {
  const int tok = k * 2 * p.tile_tok;
  it.n_tok = min(2 * p.tile_tok, n - tok);
  it.pos = kv - n + tok;
  it.hi = max(0, min(it.pos + it.n_tok, kv));
  it.lo = p.a.window ? max(0, it.pos + 1 - p.a.window) : 0;
  it.sink_hi = min(min(p.a.sinks, it.lo), it.hi);
  it.t_lo = it.lo / KT;
  it.n_sink = min((it.sink_hi + KT - 1) / KT, it.t_lo);
  return it.n_sink + (it.hi > it.lo ? (it.hi + KT - 1) / KT - it.t_lo : 0);
}
// Its length on the line: the key tiles, and before them what a block costs by
// itself (queries, pipeline fill, results), in key tiles.
__device__ __forceinline__ int block_lead(const Params& p, const Item& it) { return it.n_tok > p.tile_tok ? LEAD_TWO : LEAD_ONE; }
__device__ __forceinline__ int block_cost(const Params& p, int n, int kv, int k) {
  Item it;
  const int tiles = max(1, block_tiles(p, n, kv, k, it));
  return tiles + block_lead(p, it);
}
__device__ __forceinline__ int n_blocks(const Params& p, int n) { return (n + 2 * p.tile_tok - 1) / (2 * p.tile_tok); }

// Sum of the costs of a request's blocks; the lanes of a warp share long ones.
__device__ __forceinline__ long long request_cost(const Params& p, int b, bool valid, bool report) {
  const int lane = threadIdx.x & 31;
  int t0 = 0, n = 0, kv = 0;
  if (valid) request(p.a, b, t0, n, kv, report);
  const int blocks = n_blocks(p, n);
  long long cost = 0;
  if (blocks <= 4)
    for (int k = 0; k < blocks; ++k) cost += block_cost(p, n, kv, k);
  unsigned big = __ballot_sync(0xffffffffu, blocks > 4);
  while (big) {
    const int src = __ffs(big) - 1;
    big &= big - 1;
    const int n_s = __shfl_sync(0xffffffffu, n, src), kv_s = __shfl_sync(0xffffffffu, kv, src);
    const int blocks_s = __shfl_sync(0xffffffffu, blocks, src);
    long long sum = 0;
    for (int k = lane; k < blocks_s; k += 32) sum += block_cost(p, n_s, kv_s, k);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (lane == src) cost = sum;
  }
  return cost;
}

// --- the copying warp ------------------------------------------------------------------
// joined copies: k and v of five dimensions, else of four
struct Maps {
  CUtensorMap k, v, q, q1;  // q: a tile's tokens in a box, q1: one token
};

__device__ __forceinline__ int list_tile(const Item& it, int i) { return i < it.n_sink ? i : it.t_lo + i - it.n_sink; }

// The list entries that query tile s of a block sees: sink tiles, then a range.
__device__ __forceinline__ void tile_range(const Params& p, Item& it, int s) {
  const int first = it.pos + s * p.tile_tok, last = min(it.pos + it.n_tok, first + p.tile_tok);
  const int hi = max(0, min(last, it.kv)), lo = p.a.window ? max(0, first + 1 - p.a.window) : 0;
  it.act[s][0] = (min(p.a.sinks, hi) + KT - 1) / KT;  // past n_sink the list runs on without a gap
  it.act[s][1] = it.n_sink + max(0, lo / KT - it.t_lo);
  it.act[s][2] = hi > lo ? it.n_sink + (hi + KT - 1) / KT - it.t_lo : 0;
}
__device__ __forceinline__ bool active(const int (&act)[3], int i) { return i < act[0] || (i >= act[1] && i < act[2]); }

__device__ __forceinline__ void load_role(const Params& p, const Maps& maps, Smem& sm, unsigned char* q_smem, unsigned char* kv_smem) {
  const int lane = threadIdx.x & 31;
  unsigned* err = p.a.err;
  uint32_t fills = 0, tiles = 0, q_count = 0;
  int merges = 0;       // joined results before this item
  int rows_before = 0;  // rows of the last block whose results are joined
  for (uint32_t items = 0;; ++items) {
    const uint32_t slot = items % RING;
    wait(&sm.ring_full[slot], (items / RING) & 1, sm, err);
    if (__any_sync(0xffffffffu, is_dead(sm))) break;
    const Item it = sm.ring[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.ring_empty[slot]);
    if (it.b < 0) break;
    if (it.i1 == it.i0) continue;
    const int32_t* table = p.a.table + (int64_t)it.b * p.a.table_stride;
    const int page = 1 << p.a.page_shift, box = min(page, KT);
    // Page of lane's box of list entry i; -1 for one that no row sees (the copy
    // then asks for a page past the cache, which reads nothing and fills with
    // zeros): a hidden one, or one outside the window in a tile at its edge.
    auto page_of = [&](int i) {
      if (lane >= p.boxes || i >= it.i1) return -1;
      const int key = list_tile(it, i) * KT + lane * box;
      if (!((key < it.hi && key + box > it.lo) || key < it.sink_hi)) return -1;
      const int pg = table[key >> p.a.page_shift];
      if (pg >= p.a.n_pages) set_error(err, ERR_INDEX);
      return pg < 0 || pg >= p.a.n_pages ? -1 : pg;
    };
    int pg = page_of(it.i0);
    // Queries: their buffer is free only when the item before is through, so the
    // first keys and values go ahead of them while there is room.
    bool asked = false;
    auto queries = [&]() {
      asked = true;
      const bool two = it.n_tok > p.tile_tok;
      warp_wait(&sm.q_empty, (q_count & 1) ^ 1, sm, err);
      // Blocks of one tile join their results in the second tile's place, or in
      // all of the buffer: the last such joining has to be over if it is in the
      // way.  (A count and no barrier: this warp does not see every joining.)
      if (two || rows_before > MERGE_ROWS) wait_joined(sm, merges, err);
      if (__any_sync(0xffffffffu, is_dead(sm))) return;
      const bool joins = !two && it.i1 - it.i0 > 1;
      merges += joins;
      if (joins) rows_before = it.n_tok * p.group;
      ++q_count;
      const bool single = it.n_tok <= 8;
      const uint32_t box_bytes = (uint32_t)p.group * 128u;
      if (lane == 0)
        mbar_arrive_expect_tx(&sm.q_full, single ? 2u * it.n_tok * box_bytes : (two ? 4u : 2u) * p.tile_tok * box_bytes);
      __syncwarp();
      if (single) {
        // the swizzle goes by the shared-memory address, so a box may begin at any row of an 8-row group
        if (lane < 2 * it.n_tok) {
          const int i = lane >> 1, half = lane & 1, s = i / p.tile_tok, r = (i % p.tile_tok) * p.group;
          tma_load4(q_smem + s * TILE_BYTES + half * HALF_BYTES + r * 128, &maps.q1, half * 64, 0, it.kvh, it.tok + i, &sm.q_full);
        }
      } else if (lane < (two ? 4 : 2)) {
        const int s = lane >> 1, half = lane & 1;
        tma_load4(q_smem + s * TILE_BYTES + half * HALF_BYTES, &maps.q, half * 64, 0, it.kvh, it.tok + s * p.tile_tok, &sm.q_full);
      }
      __syncwarp();
    };
    // keys and values
    for (int i = it.i0; i < it.i1; ++i, ++tiles) {
      const int row = (list_tile(it, i) * KT) & (page - 1) & ~(box - 1);
      const int c_page = __shfl_sync(0xffffffffu, pg < 0 ? p.a.n_pages : pg, p.joined ? lane : lane >> 1);
      const unsigned held = __ballot_sync(0xffffffffu, pg >= 0);
      pg = page_of(i + 1);
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++fills) {
        const uint32_t st = fills % STAGES;
        const uint32_t parity = ((fills / STAGES) & 1) ^ 1;
        if (!asked && __any_sync(0xffffffffu, mbar_test_wait(&sm.q_empty, (q_count & 1) ^ 1) ||
                                                  !mbar_test_wait(&sm.kv_empty[st], parity)))
          queries();
        if (!__all_sync(0xffffffffu, wait_or_stop(&sm.kv_empty[st], parity, sm, err))) goto out;
        if (lane == 0) {
          if (kv == 0) *(volatile int*)&sm.page_mask[tiles % MASKS] = (int)held;
          mbar_arrive_expect_tx(&sm.kv_full[st], TILE_BYTES);
        }
        __syncwarp();
        if (p.joined) {  // a lane a box
          if (lane < p.boxes)
            tma_load5(kv_smem + st * TILE_BYTES + lane * box * 256, kv == 0 ? &maps.k : &maps.v,
                      c_page * p.page_groups + (row >> 3), c_page * p.page_outer + it.kvh, &sm.kv_full[st]);
        } else if (lane < 2 * p.boxes)  // page, half
          tma_load4(kv_smem + st * TILE_BYTES + (lane & 1) * HALF_BYTES + (lane >> 1) * box * 128, kv == 0 ? &maps.k : &maps.v,
                    (lane & 1) * 64, row, it.kvh, c_page, &sm.kv_full[st]);
      }
    }
    if (!asked) queries();
  }
out:
  if (is_dead(sm) && lane == 0) {
    // copies in flight land before the CTA ends
    for (uint32_t f = fills > STAGES ? fills - STAGES : 0; f < fills; ++f)
      mbar_wait_bounded(&sm.kv_full[f % STAGES], (f / STAGES) & 1, err);
    if (q_count > 0) mbar_wait_bounded(&sm.q_full, (q_count - 1) & 1, err);
  }
}

// --- the issuing warps -------------------------------------------------------------------
// One warp a stream, so that neither waits for the other's softmax.  Every lane runs the role, so
// that its values are uniform and live in the registers that the tensor
// instructions read; one elected lane issues.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// A place in the ring of K and V tiles and the parity of its fill.
struct Stage {
  uint32_t at = 0, parity = 0;
  __device__ __forceinline__ void skip(uint32_t n) {
    at += n;
    if (at >= STAGES) {
      at -= STAGES;
      parity ^= 1;
    }
  }
};

__device__ __forceinline__ void mma_role(const Params& p, Smem& sm, int s, uint32_t q_addr, uint32_t kv_addr, uint32_t tmem,
                                         uint32_t bf16) {
  unsigned* err = p.a.err;
  const uint32_t id_qk = tc::idesc_f16(ROWS, KT, bf16), id_pv = tc::idesc_f16(ROWS, D, bf16) | (1u << 16);
  const uint32_t t_s = tmem + s * 128, t_o = tmem + 256 + s * 128;
  Stage next;  // of list index i0 of the next item
  uint32_t q_parity = 0, p_parity = 0, o_parity = 1;
  const uint64_t k_desc = smem_desc_rows(kv_addr, p.group_bytes, p.half_bytes, false);
  const uint64_t v_desc = smem_desc_rows(kv_addr, p.group_bytes, p.half_bytes, true);
  const uint32_t k_half = (uint32_t)p.half_bytes >> 4, v_step = (uint32_t)p.group_bytes >> 3;  // 16 keys: two groups
  auto await = [&](uint64_t* bar, uint32_t parity) { warp_wait(bar, parity, sm, err); };
  // In blocks of two tiles the streams take turns at the tensor cores, key tile
  // by key tile: a product of one and its next scores go in a row.  Left to mix,
  // both streams' products finish late together, and both softmaxes run while
  // the tensor cores idle.  (The turn passes through barriers: a lock in shared
  // memory, spun on or slept on, halved the rate of the products themselves.)
  uint32_t turn = s == 0 ? 1 : 0;  // parity: the first stream's first turn needs no pass
  auto pass = [&]() {
    if (elect_one()) mbar_arrive(&sm.turn[s ^ 1]);
    __syncwarp();
  };
  for (uint32_t items = 0;; ++items) {
    const uint32_t slot = items % RING;
    await(&sm.ring_full[slot], (items / RING) & 1);
    if (__any_sync(0xffffffffu, is_dead(sm))) break;
    const Item& from = sm.ring[slot];
    Item it;
    it.b = uniform(from.b);
    it.n_tok = uniform(from.n_tok);
    it.i0 = uniform(from.i0);
    it.i1 = uniform(from.i1);
    const int act[3] = {uniform(from.act[s][0]), uniform(from.act[s][1]), uniform(from.act[s][2])};
    const int odd = uniform(from.lead) ^ s;  // block of one tile: this stream takes every other key tile
    if (elect_one()) mbar_arrive(&sm.ring_empty[slot]);
    __syncwarp();
    if (it.b < 0) break;
    if (it.i1 == it.i0) continue;
    const bool two = it.n_tok > p.tile_tok;
    await(&sm.q_full, q_parity);
    q_parity ^= 1;
    const uint64_t qd = tc::smem_desc_sw128(q_addr + (two ? s * TILE_BYTES : 0));
    int last = it.i1 - 1;  // this stream's last tile
    if (two) {
      while (last >= it.i0 && !active(act, last)) --last;
    } else {
      last -= (last - it.i0 - odd) & 1;
    }
    bool first = true;
    Stage st = next;
    bool scored = false;  // this tile's scores have been issued behind the last tile's product
    auto scores = [&](int i, const Stage& at) {
      const uint64_t kd = k_desc + at.at * (TILE_BYTES >> 4);
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint32_t in = (j & 3) * 2;  // 32 bytes
          tc::mma_f16(t_s, qd + (j >> 2) * (HALF_BYTES >> 4) + in, kd + (j >> 2) * k_half + in, id_qk, j > 0 ? 1u : 0u);
        }
        tc::mma_commit(&sm.s_full[s]);
        tc::mma_commit(&sm.kv_empty[at.at]);
        if (i == last) {
          tc::mma_commit(&sm.q_empty);  // this stream's products have read the queries
          // .. and the other stream's result may take their place, where it does
          if (!two && !odd && it.i1 - it.i0 > 1 && it.n_tok * p.group > MERGE_ROWS) tc::mma_commit(&sm.q_read);
        }
      }
      __syncwarp();
    };
    for (int i = it.i0; i < it.i1; ++i, st.skip(2)) {
      Stage sv = st;
      sv.skip(1);
      if (two ? !active(act, i) : ((i - it.i0) & 1) != odd) {
        // hidden from every row, or the other stream's: both streams see every
        // fill, so that none is two fills behind (a wait tells odd from even)
        await(&sm.kv_full[st.at], st.parity);
        await(&sm.kv_full[sv.at], sv.parity);
        if (elect_one()) {
          mbar_arrive(&sm.kv_empty[st.at]);
          mbar_arrive(&sm.kv_empty[sv.at]);
        }
        __syncwarp();
        if (two) {
          await(&sm.turn[s], turn);
          turn ^= 1;
          pass();
        }
        continue;
      }
      if (!scored) {
        await(&sm.kv_full[st.at], st.parity);
        tc::fence_after_sync();
        scores(i, st);
      }
      scored = false;
      // off the path from the weights to the next scores
      const bool more = two && i + 1 < it.i1 && active(act, i + 1);
      Stage sk = sv;
      sk.skip(1);
      await(&sm.kv_full[sv.at], sv.parity);
      if (first) {
        await(&sm.o_free[s], o_parity);
        o_parity ^= 1;
      }
      const uint64_t vd = v_desc + sv.at * (TILE_BYTES >> 4);
      if (two) {
        await(&sm.turn[s], turn);
        turn ^= 1;
      }
      await(&sm.p_full[s], p_parity);
      p_parity ^= 1;
      tc::fence_after_sync();
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < KT / 16; ++j)  // 16 keys: two 8-row groups of V
          mma_f16_ts(t_o, t_s + (j >> 2) * 64 + (j & 3) * 8, vd + j * v_step, id_pv, (j > 0 || !first) ? 1u : 0u);
        tc::mma_commit(&sm.kv_empty[sv.at]);
      }
      __syncwarp();
      if (more) {
        scored = __all_sync(0xffffffffu, mbar_test_wait(&sm.kv_full[sk.at], sk.parity));
        if (scored) {
          tc::fence_after_sync();
          scores(i + 1, sk);
        }
      }
      if (two) pass();
      first = false;
    }
    next = st;
    if (elect_one()) {
      if (!first) tc::mma_commit(&sm.o_full[s]);
      else mbar_arrive(&sm.q_empty);  // nothing for this stream here
    }
    __syncwarp();
  }
  // every product has ended before tensor memory is freed
  if (elect_one()) tc::mma_commit(&sm.drained[s]);
  __syncwarp();
  mbar_wait_bounded(&sm.drained[s], 0, err);
}

// --- the planning warp -----------------------------------------------------------------
__device__ __forceinline__ void plan_role(const Params& p, Smem& sm, int cta, long long piece) {
  const int lane = threadIdx.x & 31;
  unsigned* err = p.a.err;
  const long long total = sm.total, all = total * p.a.hkv;
  const long long u0 = cta * piece, u1 = min(all, u0 + piece);
  uint32_t items = 0;
  int turn = 0;
  bool ok = true;
  auto post = [&](const Item& it) {
    const uint32_t slot = items % RING;
    if (lane == 0) {
      wait(&sm.ring_empty[slot], ((items / RING) & 1) ^ 1, sm, err);
      ok = !is_dead(sm);
      if (ok) {
        sm.ring[slot] = it;
        mbar_arrive(&sm.ring_full[slot]);
      }
    }
    ++items;
    ok = __shfl_sync(0xffffffffu, ok, 0);
  };
  if (u0 < u1) {
    int h = (int)quotient(u0, total), b = sm.start_b;
    long long at = h * total + sm.start_before;  // of request b's first block
    while (ok && at < u1) {
      int t0, n, kv;
      request(p.a, b, t0, n, kv, false);
      const int blocks = n_blocks(p, n);
      // block k, which begins at s on the line; pieces divide its key tiles
      auto emit = [&](int k, long long s) {
        Item it;
        const int tiles = block_tiles(p, n, kv, k, it);
        s += block_lead(p, it);
        const long long e = s + max(1, tiles);
        if (s >= u1 || e <= u0) return;
        it.b = b;
        it.kvh = h;
        it.tok = t0 + k * 2 * p.tile_tok;
        it.kv = kv;
        it.i0 = (int)max(0LL, u0 - s);
        it.i1 = (int)min((long long)tiles, u1 - s);
        it.first = (int)quotient(s, piece);
        it.parts = (int)quotient(e - 1, piece) - it.first + 1;
        it.part = cta - it.first;
        it.lead = turn;
        turn ^= 1;
        tile_range(p, it, 0);
        tile_range(p, it, 1);
        post(it);
      };
      for (int k0 = 0; ok && k0 < blocks && at < u1; k0 += 32) {
        // 32 blocks at once, unless the request has but one
        long long upto = k0 + lane < blocks ? block_cost(p, n, kv, k0 + lane) : 0;
        const long long mine = upto;
        if (blocks > 1) {
#pragma unroll 1
          for (int m = 1; m < 32; m <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += x;
          }
        }
        const long long begin = at + upto - mine;
        unsigned todo = __ballot_sync(0xffffffffu, mine > 0 && begin < u1 && begin + mine > u0);
        while (ok && todo) {
          const int src = __ffs(todo) - 1;
          todo &= todo - 1;
          emit(k0 + src, __shfl_sync(0xffffffffu, begin, src));
        }
        at += __shfl_sync(0xffffffffu, upto, min(31, blocks - 1 - k0));
      }
      if (++b == p.a.n_req) {
        b = 0;
        ++h;
      }
    }
  }
  Item end;
  end.b = -1;
  if (ok) post(end);
}

// Costs of all requests: the line's length, and the request in which this CTA's
// piece begins.  By the softmax warps, while the others set the CTA up; all
// meet at the barrier inside.
__device__ __forceinline__ long long measure_line(const Params& p, Smem& sm, int cta) {
  constexpr int COUNTERS = SOFTMAX_WARPS * 32;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const bool counts = warp < SOFTMAX_WARPS;
  const int each = (p.a.n_req + COUNTERS - 1) / COUNTERS;
  long long cost = 0, upto = 0;
  if (counts) {
    for (int j = 0; j < each; ++j) cost += request_cost(p, t * each + j, t * each + j < p.a.n_req, cta == 0);
    upto = cost;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, m);
      if (lane >= m) upto += x;
    }
    if (lane == 31) sm.sums[warp] = upto;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < SOFTMAX_WARPS; ++w) {
    if (w < warp) upto += sm.sums[w];
    total += sm.sums[w];
  }
  const long long all = total * p.a.hkv;
  const long long piece = max(quotient(all + p.n_cta - 1, p.n_cta), (long long)p.min_piece);
  const long long u0 = cta * piece;
  if (counts && u0 < all) {
    const long long w0 = u0 - quotient(u0, total) * total;
    long long before = upto - cost;
    const bool mine = before <= w0 && w0 < upto;
    if (each == 1) {
      if (mine) {
        sm.start_b = t;
        sm.start_before = before;
      }
    } else if (__any_sync(0xffffffffu, mine)) {
      bool found = false;
      for (int j = 0; j < each; ++j) {
        const long long c = request_cost(p, t * each + j, t * each + j < p.a.n_req, false);
        if (mine && !found && w0 < before + c) {
          found = true;
          sm.start_b = t * each + j;
          sm.start_before = before;
        }
        before += c;
      }
    }
  }
  if (t == 0) sm.total = total;
  return piece;
}

// --- a softmax warpgroup -----------------------------------------------------------------
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// Where 16-byte piece c of a partial row lies: pieces of 8 rows fill a line, so
// that threads of neighbouring rows write, and lanes of 8 rows and 4 pieces
// read, whole lines.
__device__ __forceinline__ size_t part_piece(size_t row, int c) { return ((row >> 3) * 32 + c) * 8 + (row & 7); }

// Joins rows of a tile's parts: a unit is 8 rows by 4 PIECES pieces, a lane one
// row and PIECES pieces.
template <bool FP16, int PIECES>
__device__ __forceinline__ void join_rows(const Params& p, Smem& sm, int s, const Item& it, int tile, int n_rows) {
  constexpr int UNITS = 8 / PIECES;  // of 8 rows
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 7;
  const int parts = it.parts, first = it.first;
  for (int u = warp; u < (n_rows + 7) / 8 * UNITS; u += 8) {
    const bool real = u / UNITS * 8 + (lane & 7) < n_rows;
    const int row = min(u / UNITS * 8 + (lane & 7), n_rows - 1), c = u % UNITS * 4 * PIECES + (lane >> 3);
    float top = -CUDART_INF_F, l = 0.f, o[4 * PIECES];
#pragma unroll
    for (int j = 0; j < 4 * PIECES; ++j) o[j] = 0.f;
#pragma unroll(PIECES > 2 ? 1 : 4)
    for (int k = 0; k < parts; ++k) {
      const size_t at = (((size_t)(first + k) * 2 + (k == 0 ? 1 : 0)) * 2 + tile) * ROWS + row;
      const float2 ml = __ldcg(&p.part_ml[at]);
      float4 z[PIECES];
#pragma unroll
      for (int i = 0; i < PIECES; ++i) z[i] = __ldcg(p.part_o + part_piece(at, c) + i * 32);  // 4 pieces on
      // a part that has seen nothing has a weight of 0 (and zeros, unless the
      // values of keys without weight were not finite: the row is then looked at again)
      const float reach = fmaxf(top, ml.x);
      const float corr = top == reach ? 1.f : ex2(top - reach), w = ml.x == -CUDART_INF_F ? 0.f : ex2(ml.x - reach);
      l = l * corr + w * ml.y;
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const float v[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) o[4 * i + j] = o[4 * i + j] * corr + w * v[j];
      }
      top = reach;
    }
    if (!real) continue;
    const float inv = 1.f / l;
    float poison = 0.f;
#pragma unroll
    for (int j = 0; j < 4 * PIECES; ++j) {
      o[j] = l == 0.f ? 0.f : o[j] * inv;
      poison += o[j] * 0.f;  // NaN from then on when one is not finite
    }
    if (poison != 0.f && l == l) atomicOr(&sm.poisoned[s][0][row >> 5], 1u << (row & 31));
    const int tok = it.tok + tile * p.tile_tok + row / p.group, head = it.kvh * p.group + row % p.group;
    __nv_bfloat16* out = p.a.out + ((int64_t)tok * p.a.hq + head) * D + c * 4;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      *reinterpret_cast<uint2*>(out + i * 16) =
          make_uint2(act_pack2<FP16>(o[4 * i], o[4 * i + 1]), act_pack2<FP16>(o[4 * i + 2], o[4 * i + 3]));
    if (p.a.lse && c == 0)
      p.a.lse[(int64_t)tok * p.a.hq + head] = l == 0.f ? -CUDART_INF_F : (top + log2f(l) - WEIGHT_EXP<FP16>) * LN2;
  }
}

// Joins a tile's parts, by the stream's warpgroups that finished the last of
// them.  Many rows: a lane takes a quarter of its row, so that each part's loads
// are many.  Few: a sixteenth, so that all warps have some, and several parts'
// loads at once.
template <bool FP16>
__device__ __forceinline__ void join_parts(const Params& p, Smem& sm, int s, const Item& it, int tile, int n_rows) {
  const int warp = (threadIdx.x >> 5) & 7, bar = STREAM_BAR + s;
  if ((threadIdx.x & 255) < 4) sm.poisoned[s][0][threadIdx.x & 3] = 0;
  named_bar_sync(bar, 256);
  if (n_rows > 32) join_rows<FP16, 8>(p, sm, s, it, tile, n_rows);
  else join_rows<FP16, 2>(p, sm, s, it, tile, n_rows);
  __syncwarp();
  named_bar_sync(bar, 256);
  const int quarter = warp & 3;
  const unsigned bad = sm.poisoned[s][0][quarter];
  if (bad) mend_rows<FP16>(p, sm, s, warp >> 2, quarter, PAIR_BAR + s * 4 + quarter, it, tile, bad);
}

template <bool FP16>
__device__ __forceinline__ void softmax_role(const Params& p, Smem& sm, unsigned char* q_smem, unsigned char* kv_smem,
                                             uint32_t tmem) {
  unsigned* err = p.a.err;
  const int s = threadIdx.x >> 8, half = (threadIdx.x >> 7) & 1;  // stream; half of the tile's keys, and of the dimensions
  const int r = threadIdx.x & 127, lane = r & 31, quarter = r >> 5;
  const int bar = STREAM_BAR + s, pair = PAIR_BAR + s * 4 + quarter;
  const uint32_t lane_base = tmem + ((uint32_t)(r & 96) << 16);
  const uint32_t t_s = lane_base + s * 128 + half * 64, t_o = lane_base + 256 + s * 128 + half * 64;
  const int row_tok = r / p.group, row_head = r % p.group;
  const float sl = p.a.scale * LOG2E;
  const int all_held = (1 << p.boxes) - 1;
  const int box_shift = p.a.page_shift < 7 ? p.a.page_shift : 7;
  uint32_t fills = 0, tiles = 0, s_count = 0, o_count = 0, merges = 0, q_reads = 0;
  for (uint32_t items = 0;; ++items) {
    const uint32_t slot = items % RING;
    wait(&sm.ring_full[slot], (items / RING) & 1, sm, err);
    if (named_bar_or(bar, 256, is_dead(sm))) break;
    const Item& it = sm.ring[slot];
    if (it.b < 0) break;
    const bool two = it.n_tok > p.tile_tok;
    const int tile = two ? s : 0, i0 = it.i0, i1 = it.i1, kv = it.kv, odd = it.lead ^ s;
    const int tb = tile * p.tile_tok + row_tok;
    const bool valid = row_tok < p.tile_tok && tb < it.n_tok;
    const int pos = it.pos + tb;
    const int hi = valid ? max(0, min(pos + 1, kv)) : 0, lo = p.a.window ? max(0, pos + 1 - p.a.window) : 0;
    const int sink = min(p.a.sinks, hi);
    const bool any_row = __any_sync(0xffffffffu, valid);
    const int hi_min = __reduce_min_sync(0xffffffffu, valid ? hi : 0x7fffffff);
    const int lo_max = __reduce_max_sync(0xffffffffu, valid ? lo : 0);
    const int sink_min = __reduce_min_sync(0xffffffffu, valid ? sink : 0x7fffffff);
    // key tiles that every row of the warp sees whole: up to clear_hi, from
    // clear_lo on or below clear_sink
    const int clear_hi = hi_min - 64 - half * 64, clear_lo = lo_max - half * 64, clear_sink = sink_min - 64 - half * 64;
    float m = -CUDART_INF_F, l = 0.f;  // m is the row's, l this half's
    bool stepped = false;
    // the last joined results have been read (where they are, and what was told
    // with them, is written anew)
    warp_wait(&sm.merge_free, (merges & 1) ^ 1, sm, err);
    for (int i = two ? i0 : i0 + odd; i < i1; i += two ? 1 : 2) {
      if (two && !active(it.act[s], i)) continue;
      const int first_key = list_tile(it, i) * KT, key = first_key + half * 64;
      const bool clear = first_key <= clear_hi && (first_key >= clear_lo || first_key <= clear_sink);
      warp_wait(&sm.s_full[s], s_count & 1, sm, err);
      ++s_count;
      tc::fence_after_sync();
      if (key + 64 > kv) {
        // the rows past the cached tokens hold whatever was there: zeros there
        // keep the products finite
        const uint32_t f = fills + 2 * (i - i0) + 1;
        wait(&sm.kv_full[f % STAGES], (f / STAGES) & 1, sm, err);
        const int from = max(0, kv - key);
        unsigned char* v = kv_smem + (f % STAGES) * TILE_BYTES;
        for (int c = r; c < (64 - from) * 16; c += 128) {
          const int row = half * 64 + from + (c >> 4);
          *reinterpret_cast<int4*>(v + (row >> 3) * p.group_bytes + ((c >> 3) & 1) * p.half_bytes + (row & 7) * 128 + (c & 7) * 16) =
              make_int4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (any_row) {
        const int held = *(volatile int*)&sm.page_mask[(tiles + i - i0) % MASKS];
        if (!clear || held != all_held) {
          // hidden scores become -inf where they are
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
            tc::tmem_ld32_async(t_s + c * 32, x);
            const int k0 = key + c * 32, box = half * 2 + c;
            uint32_t seen = bits_below(hi - k0) & (~bits_below(lo - k0) | bits_below(sink - k0));
            if (box_shift == 4)
              seen &= ((held >> (2 * box)) & 1 ? 0xffffu : 0u) | ((held >> (2 * box + 1)) & 1 ? 0xffff0000u : 0u);
            else if (!((held >> ((box * 32) >> box_shift)) & 1))
              seen = 0;
            tc::tmem_wait_ld();
            tc::tmem_regs(x);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = (seen >> j) & 1 ? x[j] : 0xff800000u;
            tmem_st32(t_s + c * 32, x);
          }
          tmem_wait_st();
        }
        // Weights 2^(s sl - m sl + e), one fma and one ex2 each, against the
        // reference as it stands: no maximum is looked for while their sum
        // stays below LIMIT.  Where it does not (or the row has no reference
        // yet), the reference moves to the row's maximum so far, and the weights
        // are formed once more.
        uint32_t x[32], w[2][16];
        auto load = [&](int c) {
          tc::tmem_ld32_async(t_s + c * 32, x);
          tc::tmem_wait_ld();
          tc::tmem_regs(x);
        };
        float2 sum[2];
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          if (stepped || pass > 0) {
            const float ref = WEIGHT_EXP<FP16> - (m == -CUDART_INF_F ? 0.f : m * sl);
            const float2 sl2 = make_float2(sl, sl), ref2 = make_float2(ref, ref);
            sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              load(c);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 e = ffma2(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), sl2, ref2);
                const float2 y = make_float2(ex2(e.x), ex2(e.y));
                sum[j & 1] = fadd2(sum[j & 1], y);
                w[c][j] = act_pack2<FP16>(y.x, y.y);
              }
            }
            sum[0] = fadd2(sum[0], sum[1]);
            sum[0].x += sum[0].y;
            // rows past the block hold anything and have no say
            if (pass > 0 || !named_bar_or(pair, 64, valid && (m == -CUDART_INF_F || !(sum[0].x <= LIMIT)))) break;
          }
          float m_new = m;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            load(c);
            float top[2] = {m_new, m_new};
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              top[0] = max3(top[0], __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
              top[1] = max3(top[1], __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
            }
            m_new = fmaxf(top[0], top[1]);
          }
          sm.share[s][half][r] = m_new;
          named_bar_sync(pair, 64);
          m_new = fmaxf(m_new, sm.share[s][half ^ 1][r]);
          const float corr = m_new == -CUDART_INF_F ? 1.f : ex2((m - m_new) * sl);
          m = m_new;
          l *= corr;
          if (stepped) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t y[16];
              tc::tmem_ld16_async(t_o + c * 16, y);
              tc::tmem_wait_ld();
              tc::tmem_regs(y);
#pragma unroll
              for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * corr);
              tmem_st16(t_o + c * 16, y);
            }
          }
        }
        l += sum[0].x;
        // they take the place of the first 32 of this half's columns of S
        tmem_st16(t_s, w[0]);
        tmem_st16(t_s + 16, w[1]);
        tmem_wait_st();
      }
      stepped = true;
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[s]);
    }
    fills += 2 * (i1 - i0);
    tiles += i1 - i0;
    if (stepped) {
      // The row's sum goes where the maximum was: the other half may have yet to
      // read that when the last tile moved the reference.  (No room for a second
      // array; the last product is still under way.)
      named_bar_sync(pair, 64);
      sm.share[s][half][r] = l;
      named_bar_sync(pair, 64);
      l += sm.share[s][half ^ 1][r];
      warp_wait(&sm.o_full[s], o_count & 1, sm, err);
      ++o_count;
      tc::fence_after_sync();
    }
    // m2: the reference in powers of two, -inf where the row has seen nothing, and
    // there alone: scores that are all NaN leave no maximum, but a sum, which has
    // to reach the parts' joining.
    float m2 = l == 0.f ? -CUDART_INF_F : m == -CUDART_INF_F ? 0.f : m * sl;
    const bool merged = !two && i1 - i0 > 1;
    unsigned char* merge = q_smem + (it.n_tok * p.group <= MERGE_ROWS ? TILE_BYTES : 0);
    if (!two && odd) {
      if (merged) {
        if (merge == q_smem) {
          warp_wait(&sm.q_read, q_reads & 1, sm, err);
          ++q_reads;
        }
        ++merges;
        // rows of 512 bytes, their 16-byte pieces rotated by the row: no bank conflicts
#pragma unroll 1
        for (int c = 0; c < 4 && any_row; ++c) {
          float v[16];
          tc::tmem_ld16(t_o + c * 16, v);
          if (valid) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<float4*>(merge + r * 512 + (((half * 16 + c * 4 + j) ^ lane) << 4)) =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
          __syncwarp();
        }
        named_bar_sync(pair, 64);  // both halves have read their sums
        if (half == 0) {
          sm.share[s][0][r] = m2;
          sm.share[s][1][r] = l;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.o_free[s]);
          mbar_arrive(&sm.merge_full);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ring_empty[slot]);
      continue;
    }
    float w0 = 1.f, w1 = 0.f;
    if (merged) {
      warp_wait(&sm.merge_full, merges & 1, sm, err);
      ++merges;
      if (merge == q_smem) ++q_reads;  // over: the other stream has waited for it
      const float2 other = make_float2(sm.share[s ^ 1][0][r], sm.share[s ^ 1][1][r]);
      const float top = fmaxf(m2, other.x);
      if (top == -CUDART_INF_F) {
        l = 0.f;
      } else {
        w0 = m2 == -CUDART_INF_F ? 0.f : ex2(m2 - top);
        w1 = other.x == -CUDART_INF_F ? 0.f : ex2(other.x - top);
        l = l * w0 + other.y * w1;
        m2 = top;
      }
    }
    const bool whole_pair = it.parts == 1;
    const int tok = it.tok + tb, head = it.kvh * p.group + row_head;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const size_t part_row = (((size_t)blockIdx.x * 2 + (it.part == 0 ? 1 : 0)) * 2 + tile) * ROWS + r;
    float poison = 0.f;
#pragma unroll 1
    for (int c = 0; c < 4 && any_row; ++c) {
      float v[16];
      if (stepped) {
        tc::tmem_ld16(t_o + c * 16, v);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.f;
      }
      if (merged && valid) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 y = *reinterpret_cast<const float4*>(merge + r * 512 + (((half * 16 + c * 4 + j) ^ lane) << 4));
          v[4 * j] = v[4 * j] * w0 + y.x * w1;
          v[4 * j + 1] = v[4 * j + 1] * w0 + y.y * w1;
          v[4 * j + 2] = v[4 * j + 2] * w0 + y.z * w1;
          v[4 * j + 3] = v[4 * j + 3] * w0 + y.w * w1;
        }
      }
      if (valid && whole_pair) {
        __nv_bfloat16* out = p.a.out + ((int64_t)tok * p.a.hq + head) * D + half * 64 + c * 16;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          v[j] *= inv;
          poison += v[j] * 0.f;  // NaN from then on when one is not finite
        }
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = act_pack2<FP16>(v[2 * j], v[2 * j + 1]);
        store32(out, w);
      } else if (valid) {
#pragma unroll
        for (int j = 0; j < 4; ++j)  // pieces are 8 apart
          __stcg(p.part_o + part_piece(part_row, 0) + (half * 16 + c * 4 + j) * 8,
                 make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
      }
      __syncwarp();
    }
    if (stepped) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_free[s]);
    }
    if (merged) {
      // queries may land where the other stream's result was
      fence_proxy_async_smem();
      named_bar_sync(bar, 256);
      if ((threadIdx.x & 255) == 0) {
        mbar_arrive(&sm.merge_free);
        asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(smem_u32(&sm.joined)), "r"((int)merges) : "memory");
      }
    }
    if (whole_pair) {
      if (valid && l == 0.f && poison != 0.f) {
        // 0 where the sum is 0, whatever the values were
        __nv_bfloat16* out = p.a.out + ((int64_t)tok * p.a.hq + head) * D + half * 64;
        const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
        for (int c = 0; c < 4; ++c) store32(out + c * 16, zero);
        poison = 0.f;
      }
      if (half == 0 && valid && p.a.lse)
        p.a.lse[(int64_t)tok * p.a.hq + head] = l == 0.f ? -CUDART_INF_F : (m2 + log2f(l) - WEIGHT_EXP<FP16>) * LN2;
      const unsigned mine = __ballot_sync(0xffffffffu, valid && poison != 0.f && l == l);
      if (lane == 0) sm.poisoned[s][half][quarter] = mine;
      named_bar_sync(pair, 64);  // the row's own stores come before what is read of them
      const unsigned bad = mine | sm.poisoned[s][half ^ 1][quarter];
      if (bad) mend_rows<FP16>(p, sm, s, half, quarter, pair, it, tile, bad);
    } else {
      if (half == 0 && valid) __stcg(&p.part_ml[part_row], make_float2(m2, l));
      named_bar_sync(bar, 256);
      if ((threadIdx.x & 255) == 0) {
        __threadfence();  // for all of the stream's stores, which the barrier put before it
        unsigned* counter = &p.counters[it.first * 2 + tile];
        const bool last = atomicAdd(counter, 1u) + 1 == (unsigned)it.parts;
        if (last) {
          *counter = 0;
          __threadfence();
        }
        sm.last[s] = last;
      }
      named_bar_sync(bar, 256);
      if (sm.last[s]) {
        join_parts<FP16>(p, sm, s, it, tile, min(p.tile_tok, it.n_tok - tile * p.tile_tok) * p.group);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.ring_empty[slot]);
  }
}

template <bool FP16>
__global__ void __launch_bounds__(THREADS, 1)
    attention_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) unsigned char q_smem[];  // the swizzle repeats every 1024 bytes
  unsigned char* kv_smem = q_smem + 2 * TILE_BYTES;
  Smem& sm = *reinterpret_cast<Smem*>(kv_smem + STAGES * TILE_BYTES);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  if (threadIdx.x == PLAN_WARP * 32) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&sm.kv_full[i], 1);
      mbar_init(&sm.kv_empty[i], 2);  // both streams
    }
    for (int i = 0; i < RING; ++i) {
      mbar_init(&sm.ring_full[i], 1);
      mbar_init(&sm.ring_empty[i], 3 + SOFTMAX_WARPS);  // copying lane, two issuing lanes, softmax warps
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 2);
    mbar_init(&sm.q_read, 1);
    mbar_init(&sm.merge_full, 8);
    mbar_init(&sm.merge_free, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], 8);
      mbar_init(&sm.turn[s], 1);
      mbar_init(&sm.drained[s], 1);
      mbar_init(&sm.o_full[s], 1);
      mbar_init(&sm.o_free[s], 8);
    }
    sm.dead = sm.beat = 0;
    sm.joined = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  // the set-up above overlaps the end of the kernel before; what it wrote is read below
  griddep_launch_dependents();
  griddep_wait();
  const long long piece = measure_line(p, sm, blockIdx.x);
  __syncthreads();
  const uint32_t tmem = sm.tmem;
  if (warp < SOFTMAX_WARPS) {
    softmax_role<FP16>(p, sm, q_smem, kv_smem, tmem);
  } else if (warp == LOAD_WARP) {
    load_role(p, maps, sm, q_smem, kv_smem);
  } else if (warp >= MMA_WARP) {
    mma_role(p, sm, warp - MMA_WARP, smem_u32(q_smem), smem_u32(kv_smem), tmem, FP16 ? 0u : 1u);
  } else if (warp == PLAN_WARP) {
    plan_role(p, sm, blockIdx.x, piece);
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == MMA_WARP) tc::tmem_dealloc(tmem, 512);
}

constexpr size_t SMEM_BYTES = (2 + STAGES) * TILE_BYTES + sizeof(Smem);
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");

int sm_count() {
  static int counts[64] = {0};
  static uint64_t done = 0;
  int dev = 0;
  const bool have = once_per_device(done, [&](int d) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) == cudaSuccess) counts[d] = n;
    cudaFuncSetAttribute(attention_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    cudaFuncSetAttribute(attention_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  });
  if (!have || cudaGetDevice(&dev) != cudaSuccess || counts[dev] <= 0) {
    cudaGetLastError();  // no device here: size for a full GB300
    return 152;
  }
  return counts[dev] < 512 ? counts[dev] : 512;
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::lock_guard<std::mutex> lk(host_mutex());
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// [n3, n2, n1, 128] elements, strides s3, s2, s1 (elements); boxes of 64 x b1 x b2 x b3
bool encode(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, bool fp16, const void* base, int64_t n1, int64_t s1,
            int64_t n2, int64_t s2, int64_t n3, int64_t s3, uint32_t b1, uint32_t b2, uint32_t b3) {
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)n1, (cuuint64_t)n2, (cuuint64_t)n3};
  // the stride of a dimension of size 1 is free, but not 0
  const cuuint64_t strides[3] = {(cuuint64_t)(n1 > 1 ? s1 : D) * 2, (cuuint64_t)(n2 > 1 ? s2 : D) * 2,
                                 (cuuint64_t)(n3 > 1 ? s3 : D) * 2};
  const cuuint32_t box[4] = {64, b1, b2, b3}, step[4] = {1, 1, 1, 1};
  return enc(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
             dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same rows for joined copies: boxes of 64 x 8 rows x both halves x groups,
// from n_groups groups of 8 rows (stride 8 s1) and an outer dimension.
bool encode_joined(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, bool fp16, const void* base, int64_t s1,
                   int64_t n_groups, int64_t n_outer, int64_t s_outer, uint32_t groups) {
  const cuuint64_t dims[5] = {64, 8, 2, (cuuint64_t)n_groups, (cuuint64_t)n_outer};
  const cuuint64_t strides[4] = {(cuuint64_t)s1 * 2, 128, (cuuint64_t)s1 * 16, (cuuint64_t)(n_outer > 1 ? s_outer : D) * 2};
  const cuuint32_t box[5] = {64, 8, 2, groups, 1}, step[5] = {1, 1, 1, 1, 1};
  return enc(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base),
             dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t attention_workspace_bytes() {
  return KDA_ATTENTION_ZEROED_BYTES + (size_t)sm_count() * 4 * ROWS * (sizeof(float2) + 32 * sizeof(float4));
}

int launch_attention(const AttentionParams& a, bool fp16, void* workspace, cudaStream_t stream) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
  if (!enc) return -1;
  Params p;
  p.a = a;
  p.group = a.hq / a.hkv;
  p.tile_tok = ROWS / p.group;
  p.n_cta = sm_count();
  const int page = 1 << a.page_shift;
  p.boxes = page < KT ? KT / page : 1;
  // No piece below two key tiles, one a stream: one token over 4096 cached takes
  // 14.5 us with 2, 18 with 8.  Where most blocks are full tiles, joining them
  // costs more: a prompt of 512 tokens takes 20.9 us with 2, 19.2 with 4 and 23.8
  // with 6, one of 299 with 8 heads 17.4, 12.7 and 21.3.
  p.min_piece = (int64_t)a.t_total * p.group > (int64_t)ROWS * a.n_req ? 4 : 2;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.counters = reinterpret_cast<unsigned*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + KDA_ATTENTION_ZEROED_BYTES);
  p.part_o = reinterpret_cast<float4*>(p.part_ml + (size_t)p.n_cta * 4 * ROWS);
  Maps maps;
  const int box = page < KT ? page : KT;
  // Joined copies where page and row group, or page and head, are one dimension
  // (pages of whole token-major or head-major rows without gaps).
  const bool by_rows = a.kc_sp == page * a.kc_st && a.vc_sp == page * a.vc_st;
  const bool by_heads = a.kc_sp == a.hkv * a.kc_sh && a.vc_sp == a.hkv * a.vc_sh;
  p.joined = by_rows || by_heads;
  p.group_bytes = p.joined ? 2048 : 1024;
  p.half_bytes = p.joined ? 1024 : HALF_BYTES;
  p.page_groups = by_rows ? page / 8 : 0;
  p.page_outer = by_rows ? 0 : a.hkv;
  const int64_t groups = by_rows ? (int64_t)a.n_pages * (page / 8) : page / 8, outer = by_rows ? a.hkv : (int64_t)a.n_pages * a.hkv;
  const bool ok =
      p.joined ? encode_joined(enc, &maps.k, fp16, a.kc, a.kc_st, groups, outer, a.kc_sh, box / 8) &&
                     encode_joined(enc, &maps.v, fp16, a.vc, a.vc_st, groups, outer, a.vc_sh, box / 8)
               : encode(enc, &maps.k, fp16, a.kc, page, a.kc_st, a.hkv, a.kc_sh, a.n_pages, a.kc_sp, box, 1, 1) &&
                     encode(enc, &maps.v, fp16, a.vc, page, a.vc_st, a.hkv, a.vc_sh, a.n_pages, a.vc_sp, box, 1, 1);
  if (!ok || !encode(enc, &maps.q, fp16, a.q, p.group, a.q_sh, a.hkv, a.q_sh * p.group, a.t_total, a.q_st, p.group, 1, p.tile_tok) ||
      !encode(enc, &maps.q1, fp16, a.q, p.group, a.q_sh, a.hkv, a.q_sh * p.group, a.t_total, a.q_st, p.group, 1, 1))
    return -1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.n_cta);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_begin("attention", stream);
  if (fp16) cudaLaunchKernelEx(&cfg, attention_kernel<true>, p, maps);
  else cudaLaunchKernelEx(&cfg, attention_kernel<false>, p, maps);
  trace_end(stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace kda
