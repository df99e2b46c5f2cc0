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
//
// The cache in 8 bits.  k_j = 2^e q_j with e4m3 numbers q_j and a scale for each 16
// keys of a head, v_j likewise; tiles of 16 KB.
// - The keys go to the tensor cores as they are, as operands of 8 bits, twice as many
//   of which are multiplied at once; a query row is a power of two times the sum of
//   two e4m3 numbers (bf16) or three (fp16), by a kernel of its own,
//   split_queries_kernel: exact, but for elements below 2^-10 of the row's largest,
//   which are off by at most 2^-17 of it.
// - The keys' scale and the row's are a factor of the score.  The values' is part
//   of it: p_j = 2^(a s_j + log2 v_scale - m) is what the tensor cores take, and
//   p_j / v_scale what the row's sum takes.
// - The weights are fp16, and so are the values once the softmax warps have widened
//   them (exactly), a sixteenth of a tile each, while they wait for its scores: 30
//   instructions a thread.  The values as they are, with weights as sums of two or
//   three 8-bit numbers, took 160 and more of them, between the scores and
//   the product (8192 tokens over 16384 2.06 -> 1.95 ms); widened by the issuing warps,
//   2.65 ms.
// - In narrow blocks (see NARROW_ROWS) weights are few and the values many: there the
//   values stay in 8 bits and a weight, formed in fp16 as well, is the sum of three e5m2
//   numbers (see next_part), all of it: e5m2 has fp16's exponents.
// Outputs are off 64 bits by 1.62e-3 to 1.65e-3 of their norm in bf16, their own rounding,
// and by 2.1e-4 to 2.3e-4 in fp16, where their own is 2.0e-4: the weights' rounding to fp16
// is the rest, in blocks of all sizes.
// So prompt chunks take as many tensor cycles as over 16 bits (fp16: a quarter more),
// and are bound by the same chain of scores, weights and product, with the values' part
// in it: of a key tile's 3,300 cycles a stream spends 1,400 on weights, 200 on their
// store and the rest on the next scores, during which it widens values.  8192 tokens over
// 16384 of 32 heads 1.93 to 2.01 ms (1425 to 1370 TFLOP/s), in fp16 2.28 ms.
// Single tokens read half the bytes: see NARROW_ROWS.  256 requests over 2.2 GB
// 372 to 378 us, 5.9 TB/s; copies alone take 350 to 377 us by the chip (rows of 128 bytes, 1 KB
// apart; 256-byte rows run at 6.9 TB/s in the same ring).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <type_traits>

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
// Over an 8-bit cache, where blocks differ more: what a key tile and the lead count
// (COST_TWO8: a key tile of a block of two tiles).  A mixed batch of 64 requests took
// 221 us with 1 for all tiles, 158 with such counts; a third more or less of any moves
// it, or prompts of 97 to 4096 tokens (322 us), by 2 %.
constexpr int COST_TWO8 = 6, COST_NARROW8 = 2, COST_ONE8 = 3, LEAD_NARROW8 = 6, LEAD_ONE8 = 5, LEAD_TWO8 = 12;
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

// Over an 8-bit cache: tiles of 16 KB, and the scales of the key tiles in flight.
// A query tile takes two places of 16 KB (bf16) or three (fp16).
constexpr int TILE8_BYTES = KT * D, BLOCKS8 = KT / KDA_KV_BLOCK;
constexpr int SCALES = 32;  // key tiles whose scales fit
// When a tile's copy begins, the fifth before it is done with: its first place was the
// values' of that one, where tiles take two of nine places each (of seven: of the
// fourth), and a later one's where they take three.
constexpr int IN_FLIGHT = 5;
template <bool FP16>
constexpr int Q_PARTS = FP16 ? 3 : 2;
constexpr int W_PARTS = 3;  // of a weight in narrow blocks
template <bool FP16>
constexpr int STAGES8 = FP16 ? 7 : 9;
// Narrow blocks: few rows (single tokens, short windows) over an 8-bit cache.  A
// row a lane would leave all but one of the SM's four schedulers idle, because a
// warp reaches 32 lanes of tensor memory only.  So the keys are the lanes here:
// S^T = K Q^T (128 keys x rows) and O^T = V^T P^T (128 dimensions x rows), with the
// parts of the queries and of the weights side by side in the columns, and a
// thread has one key and all rows.  The streams take such blocks in turn, so that
// one begins while the other ends; a stream's two warpgroups take its key tiles in
// turn, each with a reference, sums and an O^T of its own, and their results are
// joined in shared memory.  256 single tokens of four heads a key head: 530 us with
// a row a lane, 372 so, the tensor cores 6 % busy.
// With 9 to 16 rows, which no longer wait in registers, it still is where caches are
// long: 64 requests of four tokens by four heads over 512 to 8191 cached 163 us with a
// row a lane and 121 so (fp16 192 and 124), 128 of 16 heads 166 and 123 (199 and 127); 200
// requests of up to 64 cached 80 and 83, one of 4096 19.4 and 21.1.
constexpr int NARROW_ROWS = 16;
// In the queries' buffer: those of two narrow blocks, so that the next one's are
// there when it begins, and behind them the weights.
constexpr int NARROW_ROW_BYTES = NARROW_ROWS * D;  // a part of the queries
template <bool FP16>
constexpr int NARROW_Q = Q_PARTS<FP16> * NARROW_ROW_BYTES;
template <bool FP16>
constexpr int NARROW_P = 2 * NARROW_Q<FP16>;
__device__ __forceinline__ bool is_narrow(int n_tok, int group) { return n_tok * group <= NARROW_ROWS; }
__device__ __forceinline__ int octets(int n_tok, int group) { return n_tok * group <= 8 ? 1 : 2; }  // of rows
__host__ __device__ constexpr int columns(int octets, int parts) { return (octets * parts + 1) / 2 * 16; }
constexpr int NARROW_W = columns(NARROW_ROWS / 8, W_PARTS) * KT;  // bytes of a group's weights
struct QuantSmem : Smem {
  uint64_t full8[STAGES8<false>], empty8[STAGES8<false>];
  uint64_t wide_full[STAGES8<false>];  // the values copied to this place are there in fp16
  // The scales of the key tiles to come, by the planning warp: a scale comes from
  // memory behind a page number, and where the copies keep memory busy that takes
  // 3 us and more, several tiles.
  uint64_t scales_full[SCALES];
  int4 clear[SOFTMAX_WARPS];              // bounds of the key tiles that a warp's rows see whole: no registers left for them
  float4 k_scale[SCALES][BLOCKS8 / 4];    // of each block of 16 keys
  float4 v_log[SCALES][BLOCKS8 / 4];      // the scale of its values in powers of two,
  float4 v_inverse[SCALES][BLOCKS8 / 4];  // and what takes it out of their weights' sum
  int held[SCALES];                       // the blocks that some row may see, a bit each
  int copied;                             // the key tile that the copies have come to
  // narrow blocks, by group
  uint64_t narrow_s[4], narrow_p[4], narrow_q_full[2], narrow_q_empty[2];
  float4 narrow_factor[4][NARROW_ROWS / 4], narrow_m[4][NARROW_ROWS / 4];
  float narrow_top[4][4 * NARROW_ROWS];  // of each warp's keys
  int narrow_done[2];                    // blocks of each stream
};
// What differs between the two caches.
template <bool FP16, bool QUANT>
struct Kind {
  static constexpr int stages = QUANT ? STAGES8<FP16> : STAGES;
  static constexpr int tile = QUANT ? TILE8_BYTES : TILE_BYTES;             // bytes of a K or V tile
  static constexpr int q_tile = QUANT ? Q_PARTS<FP16> * TILE8_BYTES : TILE_BYTES;
  static constexpr float weight_exp = WEIGHT_EXP<FP16 || QUANT>;
  static __device__ __forceinline__ uint64_t* full(Smem& sm, uint32_t i) {
    if constexpr (QUANT) return &static_cast<QuantSmem&>(sm).full8[i];
    else return &sm.kv_full[i];
  }
  static __device__ __forceinline__ uint64_t* empty(Smem& sm, uint32_t i) {
    if constexpr (QUANT) return &static_cast<QuantSmem&>(sm).empty8[i];
    else return &sm.kv_empty[i];
  }
};

struct Params {
  AttentionParams a;
  KvQuantCache c;          // the 8-bit cache
  const float* q_scale;    // of the rows of its queries' parts, [t_total, hq], with scale and log2 e
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

// hardware barriers: a pair of warps that share rows (stream, quarter), a stream's eight warps, a warpgroup
constexpr int PAIR_BAR = 1, STREAM_BAR = 9, GROUP_BAR = 11;

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
__device__ __forceinline__ void store_release(int* at, int x) {
  asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(smem_u32(at)), "r"(x) : "memory");
}
// until a counter in shared memory has come to ``count``
__device__ __forceinline__ void wait_count(const int* counter, int count, Smem& sm, unsigned* err) {
  Patience patience;
  for (uint32_t i = 0;; ++i) {
    int now;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(now) : "r"(smem_u32(counter)) : "memory");
    if (now >= count || is_dead(sm)) break;
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
// of what no one reads again
__device__ __forceinline__ void tma_load4_once(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar,
                                               uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], "
      "[%6], %7;" ::"r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)), "l"(policy) : "memory");
}
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
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
// the same products of 8-bit operands, 32 of the summed dimension at once
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// Instruction descriptor of kind::f8f6f4 with fp32 accumulation.
constexpr uint32_t E4M3 = 0, E5M2 = 1, A_MN_MAJOR = 1u << 15, B_MN_MAJOR = 1u << 16;
__host__ __device__ constexpr uint32_t idesc_f8(uint32_t M, uint32_t N, uint32_t a, uint32_t b) {
  return (1u << 4) | (a << 7) | (b << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void tma_load5(void* dst, const CUtensorMap* map, int c1, int c2, int c3, int c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      ::"r"(smem_u32(dst)), "l"(map), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar)) : "memory");
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

// Four numbers of 8 bits.
__device__ __forceinline__ void widen4(uint32_t w, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w >> 16 * i)));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * i] = x.x;
    v[2 * i + 1] = x.y;
  }
}
// A scale as the calls take it: within the range that they ask for.
constexpr float SCALE_MIN = 0x1p-48f, SCALE_MAX = 0x1p48f;
__device__ __forceinline__ float in_range(float s) { return s != s ? 1.f : fminf(fmaxf(s, SCALE_MIN), SCALE_MAX); }
// Four dimensions a lane of a key's or value's row, as they are in the cache.
template <bool QUANT>
using Raw4 = typename std::conditional<QUANT, uint32_t, uint2>::type;
template <bool FP16, bool QUANT>
__device__ __forceinline__ Raw4<QUANT> load_row4(const Params& p, bool values, int kvh, int pg, int row) {
  const int lane = threadIdx.x & 31;
  if constexpr (QUANT) {
    const uint8_t* x = values ? p.c.v + pg * p.c.v_sp + row * p.c.v_st + kvh * p.c.v_sh : p.c.k + pg * p.c.k_sp + row * p.c.k_st + kvh * p.c.k_sh;
    return *reinterpret_cast<const uint32_t*>(x + lane * 4);
  } else {
    const AttentionParams& a = p.a;
    const __nv_bfloat16* x = (values ? a.vc + (int64_t)kvh * a.vc_sh : a.kc + (int64_t)kvh * a.kc_sh) + lane * 4;
    return *reinterpret_cast<const uint2*>(values ? x + pg * a.vc_sp + row * a.vc_st : x + pg * a.kc_sp + row * a.kc_st);
  }
}
template <bool FP16>
__device__ __forceinline__ void widen_row4(const uint2& raw, float (&v)[4]) {
  load_act4<FP16>(reinterpret_cast<const __nv_bfloat16*>(&raw), v);
}
template <bool FP16>
__device__ __forceinline__ void widen_row4(uint32_t raw, float (&v)[4]) { widen4(raw, v); }

// What the values of keys [from, to) hold (none where from >= to: rows of a narrow
// window may share no key), by a warp that takes every other group of them; ends early where every dimension has a NaN.
template <bool FP16, bool QUANT>
__device__ __forceinline__ unsigned scan_values(const Params& q, Smem& sm, const int32_t* table, int kvh, int from, int to,
                                                int half, unsigned f) {
  if (from >= to) return f;
  const AttentionParams& p = q.a;
  const int lane = threadIdx.x & 31, page = 1 << p.page_shift;
#pragma unroll 1
  for (int g = from / GROUP + ((from / GROUP ^ half) & 1); g * GROUP < to; g += 2) {
    if (__all_sync(0xffffffffu, (f & 15) == 15)) break;
    if (lane == 0) *(volatile int*)&sm.beat = (int)clock();
    const int pg = table[(g * GROUP) >> p.page_shift];  // pages hold whole groups
    if (pg < 0 || pg >= p.n_pages) continue;
    float poison = 0.f;
    Raw4<QUANT> raw[GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      const int row = min(max(g * GROUP + i, from), to - 1) & (page - 1);
      raw[i] = load_row4<FP16, QUANT>(q, true, kvh, pg, row);
    }
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      float v[4];
      widen_row4<FP16>(raw[i], v);
      poison += v[0] * 0.f + v[1] * 0.f + v[2] * 0.f + v[3] * 0.f;
    }
    if (poison != 0.f) {
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        float v[4];
        widen_row4<FP16>(raw[i], v);
        f |= classify(v);
      }
    }
  }
  return f;
}

// The definition row by row, by one warp, four of the 128 dimensions a lane.
template <bool FP16, bool QUANT>
__device__ __forceinline__ void attend_row(const Params& all, Smem& sm, int b, int tok, int head, int pos, int kv) {
  const AttentionParams& p = all.a;
  const int lane = threadIdx.x & 31;
  const int kvh = head / (p.hq / p.hkv), page = 1 << p.page_shift;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -CUDART_INF_F, l = 0.f;
  load_act4<FP16>(p.q + (int64_t)tok * p.q_st + (int64_t)head * p.q_sh + lane * 4, q);
  const int hi = min(pos + 1, kv), lo = p.window ? max(0, pos + 1 - p.window) : 0;
  const int32_t* table = p.table + (int64_t)b * p.table_stride;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int from = part == 0 ? 0 : lo, to = part == 0 ? min(min(p.sinks, lo), hi) : hi;
#pragma unroll 1
    for (int g = from / GROUP; g * GROUP < to; ++g) {
      if (lane == 0) *(volatile int*)&sm.beat = (int)clock();
      const int pg = table[(g * GROUP) >> p.page_shift];
      if (pg < 0 || pg >= p.n_pages) continue;
      Raw4<QUANT> raw[GROUP];
      float s[GROUP], top = m, scale = p.scale, v_scale = 1.f;
      if constexpr (QUANT) {  // a group lies in one block
        const int64_t at = (((int64_t)pg * p.hkv + kvh) << (p.page_shift - 4)) + ((g * GROUP) & (page - 1)) / KDA_KV_BLOCK;
        scale *= in_range(all.c.k_scale[at]);
        v_scale = in_range(all.c.v_scale[at]);
      }
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        const int row = min(max(g * GROUP + i, from), to - 1) & (page - 1);
        float k[4];
        widen_row4<FP16>(load_row4<FP16, QUANT>(all, false, kvh, pg, row), k);
        raw[i] = load_row4<FP16, QUANT>(all, true, kvh, pg, row);
        s[i] = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
      }
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        s[i] = scale * warp_sum(s[i]);
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
        widen_row4<FP16>(raw[i], v);
        l += w;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += w * (QUANT ? v[j] * v_scale : v[j]);
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
template <bool FP16, bool QUANT>
__device__ __forceinline__ void mend_rows(const Params& p, Smem& sm, int s, int half, int quarter, int bar, const Item& it, int tile,
                                          unsigned bad) {
  const int lane = threadIdx.x & 31, r = quarter * 32 + lane;
  const bool mine = (bad >> lane) & 1;
  const int tb = tile * p.tile_tok + r / p.group, pos = it.pos + tb;
  const int hi = __reduce_min_sync(0xffffffffu, mine ? min(pos + 1, it.kv) : 0x7fffffff);
  const int lo = __reduce_max_sync(0xffffffffu, mine && p.a.window ? max(0, pos + 1 - p.a.window) : 0);
  const int32_t* table = p.a.table + (int64_t)it.b * p.a.table_stride;
  unsigned f = 0;
  f = scan_values<FP16, QUANT>(p, sm, table, it.kvh, 0, min(min(p.a.sinks, lo), hi), half, f);
  f = scan_values<FP16, QUANT>(p, sm, table, it.kvh, lo, hi, half, f);
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
    if (!__all_sync(0xffffffffu, stands)) attend_row<FP16, QUANT>(p, sm, it.b, tok, head, it.pos + i, it.kv);
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
template <bool QUANT>
__device__ __forceinline__ int block_lead(const Params& p, const Item& it) {
  if constexpr (QUANT) return it.n_tok > p.tile_tok ? LEAD_TWO8 : is_narrow(it.n_tok, p.group) ? LEAD_NARROW8 : LEAD_ONE8;
  return it.n_tok > p.tile_tok ? LEAD_TWO : LEAD_ONE;
}
// What a key tile of it counts.
template <bool QUANT>
__device__ __forceinline__ int tile_cost(const Params& p, const Item& it) {
  if constexpr (QUANT) return it.n_tok > p.tile_tok ? COST_TWO8 : is_narrow(it.n_tok, p.group) ? COST_NARROW8 : COST_ONE8;
  return 1;
}
template <bool QUANT>
__device__ __forceinline__ int block_cost(const Params& p, int n, int kv, int k) {
  Item it;
  const int tiles = max(1, block_tiles(p, n, kv, k, it));
  return tiles * tile_cost<QUANT>(p, it) + block_lead<QUANT>(p, it);
}
__device__ __forceinline__ int n_blocks(const Params& p, int n) { return (n + 2 * p.tile_tok - 1) / (2 * p.tile_tok); }

// Sum of the costs of a request's blocks; the lanes of a warp share long ones.
template <bool QUANT>
__device__ __forceinline__ long long request_cost(const Params& p, int b, bool valid, bool report) {
  const int lane = threadIdx.x & 31;
  int t0 = 0, n = 0, kv = 0;
  if (valid) request(p.a, b, t0, n, kv, report);
  const int blocks = n_blocks(p, n);
  long long cost = 0;
  if (blocks <= 4)
    for (int k = 0; k < blocks; ++k) cost += block_cost<QUANT>(p, n, kv, k);
  unsigned big = __ballot_sync(0xffffffffu, blocks > 4);
  while (big) {
    const int src = __ffs(big) - 1;
    big &= big - 1;
    const int n_s = __shfl_sync(0xffffffffu, n, src), kv_s = __shfl_sync(0xffffffffu, kv, src);
    const int blocks_s = __shfl_sync(0xffffffffu, blocks, src);
    long long sum = 0;
    for (int k = lane; k < blocks_s; k += 32) sum += block_cost<QUANT>(p, n_s, kv_s, k);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (lane == src) cost = sum;
  }
  return cost;
}

// --- the copying warp ------------------------------------------------------------------
// joined copies: k and v of five dimensions, else of four; q of four, in 8 bits
// (its parts) of five
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

template <bool FP16, bool QUANT>
__device__ __forceinline__ void load_role(const Params& p, const Maps& maps, Smem& sm, unsigned char* q_smem, unsigned char* kv_smem) {
  using K = Kind<FP16, QUANT>;
  const int lane = threadIdx.x & 31;
  unsigned* err = p.a.err;
  uint32_t fills = 0, tiles = 0, q_count = 0;
  uint32_t place = 0, parity = 0;  // in 8 bits: of the next fill
  int merges = 0;       // joined results before this item
  int rows_before = 0;  // rows of the last block whose results are joined
  uint32_t narrow_count = 0;
  int narrow_of[2] = {0, 0};  // by stream
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
    int pg = QUANT ? -1 : page_of(it.i0);
    // Queries: their buffer is free only when the item before is through, so the
    // first keys and values go ahead of them while there is room.  (Not those of the
    // CTA's first item: its buffer is free, and in 8 bits they wait for the split.)
    bool asked = false;
    const bool narrow = QUANT && is_narrow(it.n_tok, p.group);
    auto queries_free = [&]() {
      const bool last = mbar_test_wait(&sm.q_empty, (q_count & 1) ^ 1);
      if constexpr (QUANT) {
        if (narrow) return last && mbar_test_wait(&static_cast<QuantSmem&>(sm).narrow_q_empty[narrow_count & 1], ((narrow_count >> 1) & 1) ^ 1);
      }
      return last;
    };
    auto queries = [&]() {
      asked = true;
      if constexpr (QUANT) griddep_wait();  // at once after the first time
      const bool two = it.n_tok > p.tile_tok;
      warp_wait(&sm.q_empty, (q_count & 1) ^ 1, sm, err);
      if constexpr (QUANT) {
        if (narrow) {
          QuantSmem& qs = static_cast<QuantSmem&>(sm);
          const uint32_t place = narrow_count & 1;
          warp_wait(&qs.narrow_q_empty[place], ((narrow_count >> 1) & 1) ^ 1, sm, err);
          if (rows_before > MERGE_ROWS) wait_count(&sm.joined, merges, sm, err);
          if (__any_sync(0xffffffffu, is_dead(sm))) return;
          rows_before = 0;
          ++narrow_count;
          ++narrow_of[it.lead];
          constexpr int PARTS = Q_PARTS<FP16>;
          const int rows = 8 * octets(it.n_tok, p.group);
          if (lane == 0) mbar_arrive_expect_tx(&qs.narrow_q_full[place], PARTS * it.n_tok * p.group * 128u);
          __syncwarp();
          for (int x = lane; x < PARTS * it.n_tok; x += 32) {
            const int i = x / PARTS, part = x % PARTS;
            tma_load5(q_smem + place * NARROW_Q<FP16> + (part * rows + i * p.group) * 128, &maps.q1, 0, it.kvh, it.tok + i, part,
                      &qs.narrow_q_full[place]);
          }
          __syncwarp();
          return;
        }
      }
      // Blocks of one tile join their results in the second tile's place, or in
      // all of the buffer: the last such joining has to be over if it is in the
      // way.  (A count and no barrier: this warp does not see every joining.)
      if (two || rows_before > MERGE_ROWS) wait_count(&sm.joined, merges, sm, err);
      if constexpr (QUANT) {  // narrow blocks' weights and results lie in the way as well
        wait_count(&static_cast<QuantSmem&>(sm).narrow_done[0], narrow_of[0], sm, err);
        wait_count(&static_cast<QuantSmem&>(sm).narrow_done[1], narrow_of[1], sm, err);
      }
      if (__any_sync(0xffffffffu, is_dead(sm))) return;
      const bool joins = !two && it.i1 - it.i0 > 1;
      merges += joins;
      if (joins) rows_before = it.n_tok * p.group;
      ++q_count;
      const bool single = it.n_tok <= 8;
      const uint32_t box_bytes = (uint32_t)p.group * 128u;
      if constexpr (QUANT) {
        constexpr int PARTS = Q_PARTS<FP16>;
        if (lane == 0)
          mbar_arrive_expect_tx(&sm.q_full, PARTS * (single ? it.n_tok : (two ? 2u : 1u) * p.tile_tok) * box_bytes);
        __syncwarp();
        if (single) {
          if (lane < PARTS * it.n_tok) {
            const int i = lane / PARTS, part = lane % PARTS, s = i / p.tile_tok, r = (i % p.tile_tok) * p.group;
            tma_load5(q_smem + s * K::q_tile + part * TILE8_BYTES + r * 128, &maps.q1, 0, it.kvh, it.tok + i, part, &sm.q_full);
          }
        } else if (lane < (two ? 2 : 1) * PARTS) {
          const int s = lane / PARTS, part = lane % PARTS;
          tma_load5(q_smem + s * K::q_tile + part * TILE8_BYTES, &maps.q, 0, it.kvh, it.tok + s * p.tile_tok, part, &sm.q_full);
        }
        __syncwarp();
        return;
      }
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
    if constexpr (QUANT) {
      // Places of the ring: a narrow block's tile takes one for the keys and one for the
      // values; another's, whose values are widened to two places, one for the keys
      // and two, the second of which their copy goes to.
      // A tile's keys and values in one step, a lane a box of either: at half the
      // bytes a tile, two steps took longer than the memory (1600 cycles a tile
      // against 700 with pages of 64).  The page number is not looked at before the step
      // that needs it.
      QuantSmem& qs = static_cast<QuantSmem&>(sm);
      const bool values = lane >= p.boxes, copies = lane < 2 * p.boxes;
      const int my_box = values ? lane - p.boxes : lane;
      const CUtensorMap* map = values ? &maps.v : &maps.k;
      unsigned char* to = kv_smem + my_box * box * 128;
      const uint64_t policy = evict_first();  // a narrow block is all who read its keys: 391 -> 375 us on 256 requests
      auto entry = [&](int i) {  // of the table; -1 for a box that no row sees
        if (!copies || i >= it.i1) return -1;
        const int key = list_tile(it, i) * KT + my_box * box;
        return (key < it.hi && key + box > it.lo) || key < it.sink_hi ? table[key >> p.a.page_shift] : -1;
      };
      auto copy = [&](auto wide) {  // false: the CTA is marked
        int next = entry(it.i0);
        for (int i = it.i0; i < it.i1; ++i, ++tiles, fills += wide ? 3 : 2) {
          const int now = next;
          next = entry(i + 1);
          if (!asked && __any_sync(0xffffffffu, queries_free() || !mbar_test_wait(K::empty(sm, place), parity ^ 1))) queries();
          const uint32_t middle = place + 1 == K::stages ? 0 : place + 1, middle_parity = middle == 0 ? parity ^ 1 : parity;
          const uint32_t second = !wide ? middle : middle + 1 == K::stages ? 0 : middle + 1;
          const uint32_t second_parity = wide && second == 0 ? middle_parity ^ 1 : middle_parity;
          if (!__all_sync(0xffffffffu, wait_or_stop(K::empty(sm, place), parity ^ 1, sm, err) &&
                                           (!wide || wait_or_stop(K::empty(sm, middle), middle_parity ^ 1, sm, err)) &&
                                           wait_or_stop(K::empty(sm, second), second_parity ^ 1, sm, err)))
            return false;
          if (lane == 0) {
            store_release(&qs.copied, (int)tiles);
            mbar_arrive_expect_tx(K::full(sm, place), K::tile);
            if (wide) mbar_arrive(K::full(sm, middle));  // a fill without a copy, before the one that is waited for
            mbar_arrive_expect_tx(K::full(sm, second), K::tile);
          }
          if (now >= p.a.n_pages) set_error(err, ERR_INDEX);
          __syncwarp();
          if (copies) {
            const int row = (list_tile(it, i) * KT) & (page - 1) & ~(box - 1);
            const uint32_t st = values ? second : place;
            const int pg = now < 0 || now > p.a.n_pages ? p.a.n_pages : now;
            if (wide) tma_load4(to + st * K::tile, map, 0, row, it.kvh, pg, K::full(sm, st));
            else tma_load4_once(to + st * K::tile, map, 0, row, it.kvh, pg, K::full(sm, st), policy);
          }
          place = second + 1 == K::stages ? 0 : second + 1;
          parity = place == 0 ? second_parity ^ 1 : second_parity;
        }
        return true;
      };
      if (!(narrow ? copy(std::false_type()) : copy(std::true_type()))) goto out;
    } else {
      // keys and values
      for (int i = it.i0; i < it.i1; ++i, ++tiles) {
        const int row = (list_tile(it, i) * KT) & (page - 1) & ~(box - 1);
        const int c_page = __shfl_sync(0xffffffffu, pg < 0 ? p.a.n_pages : pg, p.joined ? lane : lane >> 1);
        const unsigned held = __ballot_sync(0xffffffffu, pg >= 0);
        pg = page_of(i + 1);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++fills) {
          const uint32_t st = fills % K::stages;
          const uint32_t parity = ((fills / K::stages) & 1) ^ 1;
          if (!asked && __any_sync(0xffffffffu, queries_free() || !mbar_test_wait(K::empty(sm, st), parity))) queries();
          if (!__all_sync(0xffffffffu, wait_or_stop(K::empty(sm, st), parity, sm, err))) goto out;
          if (lane == 0) {
            if (kv == 0) *(volatile int*)&sm.page_mask[tiles % MASKS] = (int)held;
            mbar_arrive_expect_tx(K::full(sm, st), K::tile);
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
    }
    if (!asked) queries();
  }
out:
  if (is_dead(sm) && lane == 0) {
    // copies in flight land before the CTA ends
    for (uint32_t f = fills > K::stages ? fills - K::stages : 0; f < fills; ++f)
      mbar_wait_bounded(K::full(sm, f % K::stages), (f / K::stages) & 1, err);
    if (q_count > 0) mbar_wait_bounded(&sm.q_full, (q_count - 1) & 1, err);
    if constexpr (QUANT) {
      for (uint32_t c = narrow_count > 2 ? narrow_count - 2 : 0; c < narrow_count; ++c)
        mbar_wait_bounded(&static_cast<QuantSmem&>(sm).narrow_q_full[c & 1], (c >> 1) & 1, err);
    }
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
template <int N>
struct Stage {
  uint32_t at = 0, parity = 0;
  __device__ __forceinline__ void skip(uint32_t n) {
    at += n;
    if (at >= N) {
      at -= N;
      parity ^= 1;
    }
  }
};

template <bool FP16, bool QUANT>
__device__ __forceinline__ void mma_role(const Params& p, Smem& sm, int s, uint32_t q_addr, unsigned char* kv_smem, uint32_t tmem,
                                         uint32_t bf16) {
  using K = Kind<FP16, QUANT>;
  using Stage = Stage<K::stages>;
  unsigned* err = p.a.err;
  const uint32_t id_qk = QUANT ? idesc_f8(ROWS, KT, E4M3, E4M3) : tc::idesc_f16(ROWS, KT, bf16);
  const uint32_t id_pv = tc::idesc_f16(ROWS, D, QUANT ? 0u : bf16) | B_MN_MAJOR;
  const uint32_t t_s = tmem + s * 128, t_o = tmem + 256 + s * 128, kv_addr = smem_u32(kv_smem);
  Stage next;  // of list index i0 of the next item
  uint32_t q_parity = 0, p_parity = 0, o_parity = 1;
  uint32_t narrow_parity = 0;  // of the two warpgroups' weights, a bit each
  uint32_t narrow_blocks = 0;
  const uint64_t k_desc = smem_desc_rows(kv_addr, p.group_bytes, p.half_bytes, false);
  const uint64_t v_desc = smem_desc_rows(kv_addr, p.group_bytes, p.half_bytes, true);
  const uint32_t k_half = (uint32_t)p.half_bytes >> 4, v_step = (uint32_t)p.group_bytes >> 3;  // 16 keys: two groups
  constexpr int PLACES = QUANT ? 3 : 2;  // of a key tile in the ring
  const uint64_t wide_desc = smem_desc_rows(kv_addr, 1024, TILE8_BYTES, true);
  uint32_t wide_parity = 0;  // a bit a place
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
    const bool narrow = QUANT && is_narrow(it.n_tok, p.group);
    if (!narrow) {
      await(&sm.q_full, q_parity);
      q_parity ^= 1;
    }
    const uint64_t qd = tc::smem_desc_sw128(q_addr + (two ? s * K::q_tile : 0));
    if constexpr (QUANT) {
      if (narrow) {
        // The key tiles go to the two warpgroups of the block's stream in turn; the
        // other stream sees their copies alone.  Scores are issued up to two tiles
        // ahead of the weights' product, whichever is ready.
        QuantSmem& qs = static_cast<QuantSmem&>(sm);
        const int oct = octets(it.n_tok, p.group), n_tiles = it.i1 - it.i0;
        const int mine = odd ? 0 : n_tiles;
        const uint32_t n_qk = columns(oct, Q_PARTS<FP16>), n_pv = columns(oct, W_PARTS);
        const uint32_t id_s = idesc_f8(KT, n_qk, E4M3, E4M3), id_o = idesc_f8(D, n_pv, E4M3, E5M2) | A_MN_MAJOR | B_MN_MAJOR;
        const uint32_t place = narrow_blocks & 1, q_full_parity = (narrow_blocks >> 1) & 1;
        if (!odd) await(&qs.narrow_q_full[place], q_full_parity);
        ++narrow_blocks;
        const uint64_t q_desc = tc::smem_desc_sw128(q_addr + place * NARROW_Q<FP16>);
        const uint64_t w_desc = tc::smem_desc(q_addr + NARROW_P<FP16> + s * 2 * NARROW_W, 128, 2048);
        int tile = 0, scored_n = 0, done = 0;  // key tiles passed, scored, finished
        Stage at = next, v_at = next;
        v_at.skip(1);
        Patience patience;
        while (done < mine || tile < n_tiles) {
          bool moved = false;
          if (done < scored_n && __all_sync(0xffffffffu, mbar_test_wait(&qs.narrow_p[s * 2 + (done & 1)], narrow_parity >> (done & 1) & 1))) {
            const int g = done & 1;
            narrow_parity ^= 1u << g;
            if (done == 0) {
              await(&sm.o_free[s], o_parity);
              o_parity ^= 1;
            }
            await(K::full(sm, v_at.at), v_at.parity);
            tc::fence_after_sync();
            if (elect_one()) {
              const uint64_t vd = v_desc + v_at.at * (K::tile >> 4);
#pragma unroll
              for (int j = 0; j < KT / 32; ++j)
                mma_f8(t_o + g * 64, vd + j * 2 * v_step, w_desc + g * (NARROW_W >> 4) + j * (512 >> 4), id_o,
                       (j > 0 || done > 1) ? 1u : 0u);
              tc::mma_commit(K::empty(sm, v_at.at));
            }
            __syncwarp();
            v_at.skip(2);
            ++done;
            moved = true;
          }
          if (tile < n_tiles && scored_n < done + 2 && __all_sync(0xffffffffu, mbar_test_wait(K::full(sm, at.at), at.parity))) {
            Stage v = at;
            v.skip(1);
            if (!odd) {
              tc::fence_after_sync();
              const int g = scored_n & 1;
              if (elect_one()) {
                const uint64_t kd = k_desc + at.at * (K::tile >> 4);
#pragma unroll
                for (int j = 0; j < D / 32; ++j) mma_f8(t_s + g * 64, kd + j * 2, q_desc + j * 2, id_s, j > 0 ? 1u : 0u);
                tc::mma_commit(&qs.narrow_s[s * 2 + g]);
                tc::mma_commit(K::empty(sm, at.at));
                if (scored_n + 1 == mine) tc::mma_commit(&qs.narrow_q_empty[place]);
              }
              ++scored_n;
            } else {
              await(K::full(sm, v.at), v.parity);
              if (elect_one()) {
                mbar_arrive(K::empty(sm, at.at));
                mbar_arrive(K::empty(sm, v.at));
              }
            }
            __syncwarp();
            at.skip(2);
            ++tile;
            moved = true;
          }
          if (moved) {
            patience.t0 = 0;
          } else if (__any_sync(0xffffffffu, is_dead(sm) || patience.over(sm))) {
            *(volatile int*)&sm.dead = 1;
            set_error(err, ERR_TIMEOUT);
            break;
          }
        }
        // The other stream sees these queries land as well: a wait tells odd fills from
        // even, and this place's next block may be its own (blocks without keys count in
        // the streams' turn, so that one stream may lead several in a row).
        if (odd) await(&qs.narrow_q_full[place], q_full_parity);
        if (elect_one()) {
          if (mine > 0) tc::mma_commit(&sm.o_full[s]);
          else mbar_arrive(&qs.narrow_q_empty[place]);
        }
        __syncwarp();
        next.skip((2 * n_tiles) % K::stages);
        next.parity ^= (2 * n_tiles / K::stages) & 1;
        continue;
      }
    }
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
      const uint64_t kd = k_desc + at.at * (K::tile >> 4);
      if (elect_one()) {
        if constexpr (QUANT) {
#pragma unroll
          for (int j = 0; j < Q_PARTS<FP16> * (D / 32); ++j)  // the queries' parts one after another
            mma_f8(t_s, qd + (j >> 2) * (TILE8_BYTES >> 4) + (j & 3) * 2, kd + (j & 3) * 2, id_qk, j > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t in = (j & 3) * 2;  // 32 bytes
            tc::mma_f16(t_s, qd + (j >> 2) * (HALF_BYTES >> 4) + in, kd + (j >> 2) * k_half + in, id_qk, j > 0 ? 1u : 0u);
          }
        }
        tc::mma_commit(&sm.s_full[s]);
        tc::mma_commit(K::empty(sm, at.at));
        if (i == last) {
          tc::mma_commit(&sm.q_empty);  // this stream's products have read the queries
          // .. and the other stream's result may take their place, where it does
          if (!two && !odd && it.i1 - it.i0 > 1 && it.n_tok * p.group > MERGE_ROWS) tc::mma_commit(&sm.q_read);
        }
      }
      __syncwarp();
    };
    for (int i = it.i0; i < it.i1; ++i, st.skip(PLACES)) {
      Stage sv = st;
      sv.skip(PLACES - 1);
      const uint32_t middle = st.at + 1 == K::stages ? 0 : st.at + 1;  // in 8 bits, for half of the wide values
      if (two ? !active(act, i) : ((i - it.i0) & 1) != odd) {
        // hidden from every row, or the other stream's: both streams see every
        // fill, so that none is two fills behind (a wait tells odd from even)
        await(K::full(sm, st.at), st.parity);
        await(K::full(sm, sv.at), sv.parity);
        if constexpr (QUANT) {
          await(&static_cast<QuantSmem&>(sm).wide_full[sv.at], (wide_parity >> sv.at) & 1);
          wide_parity ^= 1u << sv.at;
        }
        if (elect_one()) {
          mbar_arrive(K::empty(sm, st.at));
          if constexpr (QUANT) mbar_arrive(K::empty(sm, middle));
          mbar_arrive(K::empty(sm, sv.at));
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
        await(K::full(sm, st.at), st.parity);
        tc::fence_after_sync();
        scores(i, st);
      }
      scored = false;
      // off the path from the weights to the next scores
      const bool more = two && i + 1 < it.i1 && active(act, i + 1);
      Stage sk = sv;
      sk.skip(1);
      await(K::full(sm, sv.at), sv.parity);
      if (first) {
        await(&sm.o_free[s], o_parity);
        o_parity ^= 1;
      }
      if (two) {
        await(&sm.turn[s], turn);
        turn ^= 1;
      }
      await(&sm.p_full[s], p_parity);
      p_parity ^= 1;
      if constexpr (QUANT) {
        await(&static_cast<QuantSmem&>(sm).wide_full[sv.at], (wide_parity >> sv.at) & 1);
        wide_parity ^= 1u << sv.at;
      }
      tc::fence_after_sync();
      if (elect_one()) {
        // 16 keys: two 8-row groups of V
        if (!QUANT || sv.at > 0) {
          const uint64_t vd = QUANT ? wide_desc + middle * (K::tile >> 4) : v_desc + sv.at * (K::tile >> 4);
          const uint32_t step = QUANT ? 2 * 1024 >> 4 : v_step;
#pragma unroll
          for (int j = 0; j < KT / 16; ++j)
            mma_f16_ts(t_o, t_s + (j >> 2) * 64 + (j & 3) * 8, vd + j * step, id_pv, (j > 0 || !first) ? 1u : 0u);
        } else {  // the halves at the ring's two ends
#pragma unroll
          for (int j = 0; j < 2 * (KT / 16); ++j)
            mma_f16_ts(t_o + (j & 1) * 64, t_s + (j >> 3) * 64 + (j >> 1 & 3) * 8,
                       wide_desc + (j & 1 ? 0 : middle) * (K::tile >> 4) + (j >> 1) * (2 * 1024 >> 4),
                       tc::idesc_f16(ROWS, D / 2, 0) | B_MN_MAJOR, (j > 1 || !first) ? 1u : 0u);
        }
        if constexpr (QUANT) tc::mma_commit(K::empty(sm, middle));
        tc::mma_commit(K::empty(sm, sv.at));
      }
      __syncwarp();
      if (more) {
        scored = __all_sync(0xffffffffu, mbar_test_wait(K::full(sm, sk.at), sk.parity));
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
// The scales of an item's key tiles, four tiles at once, a lane a block of 16 keys;
// the pages of the next four and then their scales are under way meanwhile.
// ``tiles``: key tiles before the item's.
__device__ __forceinline__ void fetch_scales(const Params& p, QuantSmem& sm, const Item& it, uint32_t tiles) {
  const int lane = threadIdx.x & 31, b = lane & 7;
  unsigned* err = p.a.err;
  const int32_t* table = p.a.table + (int64_t)it.b * p.a.table_stride;
  auto page_of = [&](int i) {  // -1 for a block that no row sees
    if (i >= it.i1) return -1;
    const int key = list_tile(it, i) * KT + b * KDA_KV_BLOCK;
    if (!((key < it.hi && key + KDA_KV_BLOCK > it.lo) || key < it.sink_hi)) return -1;
    const int pg = table[key >> p.a.page_shift];
    return pg >= p.a.n_pages ? -1 : pg;  // reported by the copies
  };
  auto scales_of = [&](int i, int pg) {
    if (pg < 0) return make_float2(1.f, 1.f);
    const int row = (list_tile(it, i) * KT + b * KDA_KV_BLOCK) & ((1 << p.a.page_shift) - 1);
    const int64_t at = (((int64_t)pg * p.a.hkv + it.kvh) << (p.a.page_shift - 4)) + row / KDA_KV_BLOCK;
    return make_float2(p.c.k_scale[at], p.c.v_scale[at]);
  };
  // pages of the four tiles from i on, of the next four and of those after; scales of the first and second
  int i = it.i0 + (lane >> 3);
  int pg[3] = {page_of(i), page_of(i + 4), page_of(i + 8)};
  float2 x[2] = {scales_of(i, pg[0]), scales_of(i + 4, pg[1])};
  for (int from = it.i0; from < it.i1; from += 4, i += 4) {
    const int n = min(4, it.i1 - from);  // tiles of these four
    const uint32_t first = tiles + (from - it.i0);
    const float2 after = scales_of(i + 8, pg[2]);
    const int pages = pg[0];
    pg[0] = pg[1];
    pg[1] = pg[2];
    pg[2] = page_of(i + 12);
    wait_count(&sm.copied, (int)(first + n - 1) - (SCALES - IN_FLIGHT), sm, err);
    const float ks = in_range(x[0].x), vs = in_range(x[0].y);
    if (ks != x[0].x || vs != x[0].y) set_error(err, ERR_RANGE);
    const unsigned held = __ballot_sync(0xffffffffu, pages >= 0);
    if ((lane >> 3) < n) {
      const uint32_t place = (first + (lane >> 3)) % SCALES;
      reinterpret_cast<float*>(sm.k_scale[place])[b] = ks;
      reinterpret_cast<float*>(sm.v_log[place])[b] = log2f(vs);
      reinterpret_cast<float*>(sm.v_inverse[place])[b] = 1.f / vs;
      if (b == 0) sm.held[place] = (held >> (lane & 24)) & 0xff;
    }
    __syncwarp();
    if (lane < n) mbar_arrive(&sm.scales_full[(first + lane) % SCALES]);
    x[0] = x[1];
    x[1] = after;
  }
}

template <bool QUANT>
__device__ __forceinline__ void plan_role(const Params& p, Smem& sm, int cta, long long piece) {
  const int lane = threadIdx.x & 31;
  unsigned* err = p.a.err;
  const long long total = sm.total, all = total * p.a.hkv;
  const long long u0 = cta * piece, u1 = min(all, u0 + piece);
  uint32_t items = 0, key_tiles = 0;
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
        const int each = tile_cost<QUANT>(p, it);
        s += block_lead<QUANT>(p, it);
        const long long e = s + (long long)max(1, tiles) * each;
        if (s >= u1 || e <= u0) return;
        it.b = b;
        it.kvh = h;
        it.tok = t0 + k * 2 * p.tile_tok;
        it.kv = kv;
        // a tile belongs to the piece in which it begins (a block without tiles has
        // the length of one)
        it.i0 = u0 <= s ? 0 : min(tiles, (int)quotient(u0 - s + each - 1, each));
        it.i1 = u1 >= e ? tiles : min(tiles, (int)quotient(u1 - s + each - 1, each));
        it.first = (int)quotient(s, piece);
        it.parts = (int)quotient(e - 1, piece) - it.first + 1;
        it.part = cta - it.first;
        it.lead = turn;
        turn ^= 1;
        tile_range(p, it, 0);
        tile_range(p, it, 1);
        post(it);
        if constexpr (QUANT) {
          if (ok) fetch_scales(p, static_cast<QuantSmem&>(sm), it, key_tiles);
          key_tiles += it.i1 - it.i0;
        }
      };
      for (int k0 = 0; ok && k0 < blocks && at < u1; k0 += 32) {
        // 32 blocks at once, unless the request has but one
        long long upto = k0 + lane < blocks ? block_cost<QUANT>(p, n, kv, k0 + lane) : 0;
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
template <bool QUANT>
__device__ __forceinline__ long long measure_line(const Params& p, Smem& sm, int cta) {
  constexpr int COUNTERS = SOFTMAX_WARPS * 32;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const bool counts = warp < SOFTMAX_WARPS;
  const int each = (p.a.n_req + COUNTERS - 1) / COUNTERS;
  long long cost = 0, upto = 0;
  if (counts) {
    for (int j = 0; j < each; ++j) cost += request_cost<QUANT>(p, t * each + j, t * each + j < p.a.n_req, cta == 0);
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
        const long long c = request_cost<QUANT>(p, t * each + j, t * each + j < p.a.n_req, false);
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

// --- weights in 8 bits ---------------------------------------------------------------------
// A score's factor of its row and its key's block, not 0 (hidden scores are -inf).
__device__ __forceinline__ float row_factor(float sl, float ks) { return fmaxf(sl * ks, 1e-37f); }

// Weights as sums of W_PARTS e5m2 numbers, from the largest on: e5m2 is the upper
// half of fp16 with its exponents.  Each part takes what is left to its nearest 3
// significant bits (half up, in fp16's bits), and what is left then is taken PART_STEP
// times larger, which the results' joining takes back: 11 bits are 3 + 4 + 4 with the
// signs, and at fp16's lower end, where e5m2 ends 8 bits earlier, the steps make up for
// them.  So three parts are the weight exactly, whatever its size up to LIMIT.  Two parts
// left up to 2^-7 of it, with the same sign for equal weights (outputs of 256 single
// tokens in bf16 off by 2.0e-3 of their norm, with three by 1.62e-3), and saved next to
// nothing: 378 us either way, a mixed batch 149 us instead of 150.
constexpr float PART_STEP = 16.f;
// The next part of four weights, two by two in h, which keeps what is left of them
// where more parts follow.
template <bool MORE>
__device__ __forceinline__ uint32_t next_part(uint32_t (&h)[2]) {
  uint32_t r[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    r[k] = h[k];
    if constexpr (MORE) {
      r[k] += 0x00800080u;
      const uint32_t top = r[k] & 0xff00ff00u;
      const __half2 rest = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&h[k]), *reinterpret_cast<const __half2*>(&top)),
                                   __float2half2_rn(PART_STEP));
      h[k] = *reinterpret_cast<const uint32_t*>(&rest);
    }
  }
  return __byte_perm(r[0], r[1], 0x7531);
}

// Eight rows of an 8-bit values' tile, from row ``from`` on, to fp16, zeros from row
// ``end`` on: dimensions 0 - 63 of a row to the place before, 64 - 127 to where the
// row was (each 128 bytes, swizzled alike).  By one warp, 4 lanes a row; 8 lanes side
// by side have the same piece of all rows, which the swizzle spreads over the banks.
__device__ __forceinline__ void widen_values(unsigned char* kv_smem, uint32_t at, uint32_t places, int from, int end) {
  const int lane = threadIdx.x & 31, row = lane & 7, j = lane >> 3;
  const uint32_t first = from * 128 + row * 128, c = (j ^ row) << 4, to = (2 * j ^ row) << 4;
  unsigned char* upper = kv_smem + at * TILE8_BYTES + first;
  unsigned char* lower = kv_smem + (at == 0 ? places - 1 : at - 1) * TILE8_BYTES + first;
  uint4 x[2] = {*reinterpret_cast<const uint4*>(upper + c), *reinterpret_cast<const uint4*>(upper + (c ^ 64))};
  if (from + row >= end) x[0] = x[1] = make_uint4(0, 0, 0, 0);
  __syncwarp();  // a row's lanes have read it
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[k]) : "h"((uint16_t)(w[k >> 1] >> (k & 1) * 16)));
    unsigned char* row_at = i == 0 ? lower : upper;
    *reinterpret_cast<uint4*>(row_at + to) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(row_at + (to ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// --- a softmax warpgroup -----------------------------------------------------------------
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// Where 16-byte piece c of a partial row lies: pieces of 8 rows fill a line, so
// that threads of neighbouring rows write, and lanes of 8 rows and 4 pieces
// read, whole lines.
__device__ __forceinline__ size_t part_piece(size_t row, int c) { return ((row >> 3) * 32 + c) * 8 + (row & 7); }

// Joins rows of a tile's parts: a unit is 8 rows by 4 PIECES pieces, a lane one
// row and PIECES pieces.
template <bool FP16, bool QUANT, int PIECES>
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
      p.a.lse[(int64_t)tok * p.a.hq + head] = l == 0.f ? -CUDART_INF_F : (top + log2f(l) - Kind<FP16, QUANT>::weight_exp) * LN2;
  }
}

// Counts a tile's part, whose results the stream has stored; true with the last one.
__device__ __forceinline__ bool last_part(const Params& p, Smem& sm, int s, const Item& it, int tile, int bar) {
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
  return sm.last[s];
}

// Joins a tile's parts, by the stream's warpgroups that finished the last of
// them.  Many rows: a lane takes a quarter of its row, so that each part's loads
// are many.  Few: a sixteenth, so that all warps have some, and several parts'
// loads at once.
template <bool FP16, bool QUANT>
__device__ __forceinline__ void join_parts(const Params& p, Smem& sm, int s, const Item& it, int tile, int n_rows) {
  const int warp = (threadIdx.x >> 5) & 7, bar = STREAM_BAR + s;
  if ((threadIdx.x & 255) < 4) sm.poisoned[s][0][threadIdx.x & 3] = 0;
  named_bar_sync(bar, 256);
  if (n_rows > 32) join_rows<FP16, QUANT, 8>(p, sm, s, it, tile, n_rows);
  else join_rows<FP16, QUANT, 2>(p, sm, s, it, tile, n_rows);
  __syncwarp();
  named_bar_sync(bar, 256);
  const int quarter = warp & 3;
  const unsigned bad = sm.poisoned[s][0][quarter];
  if (bad) mend_rows<FP16, QUANT>(p, sm, s, warp >> 2, quarter, PAIR_BAR + s * 4 + quarter, it, tile, bad);
}

__device__ __forceinline__ void tmem_ld8_async(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_regs8(uint32_t (&r)[8]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}

// A narrow block by one of the stream's warpgroups: thread r has key r of its tiles
// and dimension r of the results, which go to shared memory; the leading stream
// joins them.  The counters are those of the softmax role.
template <bool FP16, int OCT>
__device__ __forceinline__ void narrow_block(const Params& p, QuantSmem& sm, const Item& it, unsigned char* q_smem,
                                          unsigned char* kv_smem, uint32_t tmem, uint32_t tiles, uint32_t fills,
                                          uint32_t s_count, uint32_t o_count, uint32_t merges) {
  using K = Kind<FP16, true>;
  constexpr int RP = OCT * 8;
  unsigned* err = p.a.err;
  const int s = threadIdx.x >> 8, half = (threadIdx.x >> 7) & 1, g = s * 2 + half;
  const int r = threadIdx.x & 127, lane = r & 31, quarter = r >> 5, bar = GROUP_BAR + g;
  const uint32_t lane_base = tmem + ((uint32_t)(r & 96) << 16);
  const uint32_t t_s = lane_base + s * 128 + half * 64, t_o = lane_base + 256 + s * 128 + half * 64;
  const int i0 = it.i0, i1 = it.i1, kv = it.kv, n_rows = it.n_tok * p.group;
  float* factor = reinterpret_cast<float*>(sm.narrow_factor[g]);
  float* ref = reinterpret_cast<float*>(sm.narrow_m[g]);  // the rows' references, in powers of two
  unsigned char* weights = q_smem + NARROW_P<FP16> + g * NARROW_W + r * 16;
  // what row ``lane`` sees
  const int pos = it.pos + (lane < n_rows ? lane / p.group : 0);
  const int row_hi = max(0, min(pos + 1, kv)), row_lo = p.a.window ? max(0, pos + 1 - p.a.window) : 0;
  const int row_sink = min(p.a.sinks, row_hi);
  const bool real = lane < n_rows;
  const int hi_min = __reduce_min_sync(0xffffffffu, real ? row_hi : 0x7fffffff);
  const int lo_max = __reduce_max_sync(0xffffffffu, real ? row_lo : 0);
  const int sink_min = __reduce_min_sync(0xffffffffu, real ? row_sink : 0x7fffffff);
  if (r < RP) {
    factor[r] = real ? p.q_scale[(int64_t)(it.tok + r / p.group) * p.a.hq + it.kvh * p.group + r % p.group] : 1.f;
    ref[r] = -CUDART_INF_F;
  }
  named_bar_sync(bar, 128);
  float l[RP];
#pragma unroll
  for (int k = 0; k < RP; ++k) l[k] = 0.f;
  bool stepped = false;
#pragma unroll 1
  for (int i = i0 + half; i < i1; i += 2) {
    const int first_key = list_tile(it, i) * KT, key = first_key + r, place = (tiles + i - i0) % SCALES;
    // what the key brings, before the scores are there
    warp_wait(&sm.scales_full[place], ((tiles + i - i0) / SCALES) & 1, sm, err);
    const float ks = reinterpret_cast<const float*>(sm.k_scale[place])[r >> 4];
    const float lv = reinterpret_cast<const float*>(sm.v_log[place])[r >> 4];
    const float iv = reinterpret_cast<const float*>(sm.v_inverse[place])[r >> 4];
    const int held = sm.held[place];
    const bool clear = held == (1 << BLOCKS8) - 1 && first_key + KT <= hi_min && (first_key >= lo_max || first_key + KT <= sink_min);
    // Weights are 2^(a score + b).  Of 8 rows a and b wait in registers, of 16 (no
    // room) they are formed where they are used.
    bool begun = true;  // every row has a reference
    auto terms = [&](int k, float2& a, float2& b) {
      const float2 f = *reinterpret_cast<const float2*>(factor + k), m = *reinterpret_cast<const float2*>(ref + k);
      a = make_float2(row_factor(f.x, ks), row_factor(f.y, ks));
      b = make_float2(K::weight_exp - (m.x == -CUDART_INF_F ? 0.f : m.x) + lv,
                      K::weight_exp - (m.y == -CUDART_INF_F ? 0.f : m.y) + lv);
      begun = begun && (k >= n_rows || m.x != -CUDART_INF_F) && (k + 1 >= n_rows || m.y != -CUDART_INF_F);
    };
    float2 a8[4], b8[4];
    if constexpr (OCT == 1) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) terms(k, a8[k / 2], b8[k / 2]);
    }
    warp_wait(&sm.narrow_s[g], s_count & 1, sm, err);
    ++s_count;
    tc::fence_after_sync();
    float x[RP];
#pragma unroll
    for (int o = 0; o < OCT; ++o) {
      uint32_t y[Q_PARTS<FP16>][8];
#pragma unroll
      for (int part = 0; part < Q_PARTS<FP16>; ++part) tmem_ld8_async(t_s + part * RP + o * 8, y[part]);
      tc::tmem_wait_ld();
#pragma unroll
      for (int part = 0; part < Q_PARTS<FP16>; ++part) tmem_regs8(y[part]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[o * 8 + k] = __uint_as_float(y[0][k]);
#pragma unroll
        for (int part = 1; part < Q_PARTS<FP16>; ++part) x[o * 8 + k] += __uint_as_float(y[part][k]);
      }
    }
    if (!clear) {
      const bool there = (held >> (r >> 4)) & 1;
#pragma unroll
      for (int k = 0; k < RP; ++k) {
        const int hi = __shfl_sync(0xffffffffu, row_hi, k), lo = __shfl_sync(0xffffffffu, row_lo, k);
        const int sink = __shfl_sync(0xffffffffu, row_sink, k);
        if (!there || key >= hi || (key < lo && key >= sink)) x[k] = -CUDART_INF_F;
      }
      if (first_key + KT > kv) {
        // the rows past the cached tokens hold whatever was there
        const uint32_t f = fills + 2 * (i - i0) + 1;
        wait(K::full(sm, f % K::stages), (f / K::stages) & 1, sm, err);
        if (key >= kv) {
          int4* v = reinterpret_cast<int4*>(kv_smem + (f % K::stages) * K::tile + r * 128);
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = make_int4(0, 0, 0, 0);
        }
        __syncwarp();
      }
    }
    uint32_t w[RP / 2];
    float sum[RP];
    auto weigh = [&]() {
      bool fits = true;
#pragma unroll
      for (int k = 0; k < RP; k += 2) {
        float2 a, b;
        if constexpr (OCT == 1) {
          a = a8[k / 2];
          b = b8[k / 2];
        } else {
          terms(k, a, b);
        }
        const float2 e = ffma2(make_float2(x[k], x[k + 1]), a, b);
        // rows past the block hold anything: no weight
        sum[k] = k < n_rows ? ex2(e.x) : 0.f;
        sum[k + 1] = k + 1 < n_rows ? ex2(e.y) : 0.f;
        fits = fits && sum[k] <= LIMIT && sum[k + 1] <= LIMIT;
        w[k / 2] = act_pack2<true>(sum[k], sum[k + 1]);
      }
      return fits;
    };
    const bool fits = weigh();
    if (named_bar_or(bar, 128, !begun || !fits)) {
      // the reference moves to each row's largest score so far
      float* share = sm.narrow_top[g];
#pragma unroll
      for (int k = 0; k < RP; ++k) {
        const float y = fmaf(x[k], row_factor(factor[k], ks), lv);
        // in the order of whole numbers; NaN has no say
        const int bits = __float_as_int(y == y ? y : -CUDART_INF_F), top = __reduce_max_sync(0xffffffffu, bits ^ ((bits >> 31) & 0x7fffffff));
        if (lane == 0) share[quarter * NARROW_ROWS + k] = __int_as_float(top ^ ((top >> 31) & 0x7fffffff));
      }
      named_bar_sync(bar, 128);
      float corr[RP], m_mine = -CUDART_INF_F;
#pragma unroll
      for (int k = 0; k < RP; ++k) {
        const float m = ref[k];
        float m_new = m;
#pragma unroll
        for (int q = 0; q < 4; ++q) m_new = fmaxf(m_new, share[q * NARROW_ROWS + k]);
        corr[k] = m_new == -CUDART_INF_F ? 1.f : ex2(m - m_new);
        l[k] *= corr[k];
        if (r == k) m_mine = m_new;
      }
      if (stepped) {
#pragma unroll 1
        for (int part = 0; part < W_PARTS; ++part) {
#pragma unroll
          for (int o = 0; o < OCT; ++o) {
            uint32_t y[8];
            tmem_ld8_async(t_o + part * RP + o * 8, y);
            tc::tmem_wait_ld();
            tmem_regs8(y);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * corr[o * 8 + k]);
            tmem_st8(t_o + part * RP + o * 8, y);
          }
        }
        tmem_wait_st();
      }
      named_bar_sync(bar, 128);  // all have read the references
      if (r < RP) ref[r] = m_mine;
      named_bar_sync(bar, 128);
      if constexpr (OCT == 1) {
#pragma unroll
        for (int k = 0; k < 8; k += 2) terms(k, a8[k / 2], b8[k / 2]);
      }
      weigh();
    }
#pragma unroll
    for (int k = 0; k < RP; ++k) l[k] += sum[k] * iv;
    // key r's weights of all rows, part after part: 16 bytes a line, 128 lines to 16 columns
#pragma unroll
    for (int part = 0; part < W_PARTS; ++part) {
#pragma unroll
      for (int o = 0; o < OCT; ++o) {
        uint32_t y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t h[2] = {w[o * 4 + j * 2], w[o * 4 + j * 2 + 1]};
          y[j] = part + 1 < W_PARTS ? next_part<true>(h) : next_part<false>(h);
          w[o * 4 + j * 2] = h[0];
          w[o * 4 + j * 2 + 1] = h[1];
        }
        const int column = part * RP + o * 8;
        *reinterpret_cast<uint2*>(weights + (column >> 4) * 2048 + (column & 8)) = make_uint2(y[0], y[1]);
      }
    }
    fence_proxy_async_smem();
    stepped = true;
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.narrow_p[g]);
  }
  // results: O^T and the sums of each warp's keys
  float* merge = reinterpret_cast<float*>(q_smem + K::q_tile) + g * NARROW_ROWS * D;
  float* share = sm.share[s][half];
  warp_wait(&sm.merge_free, (merges & 1) ^ 1, sm, err);  // the last joined results have been read
  warp_wait(&sm.o_full[s], o_count & 1, sm, err);
  tc::fence_after_sync();
  if (stepped) {
#pragma unroll
    for (int o = 0; o < OCT; ++o) {
      uint32_t y[W_PARTS][8];
#pragma unroll
      for (int part = 0; part < W_PARTS; ++part) tmem_ld8_async(t_o + part * RP + o * 8, y[part]);
      tc::tmem_wait_ld();
#pragma unroll
      for (int part = 0; part < W_PARTS; ++part) tmem_regs8(y[part]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float sum = __uint_as_float(y[W_PARTS - 1][k]);
#pragma unroll
        for (int part = W_PARTS - 2; part >= 0; --part) sum = fmaf(sum, 1.f / PART_STEP, __uint_as_float(y[part][k]));
        merge[(o * 8 + k) * D + r] = sum;
      }
    }
  }
  tc::fence_before_sync();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm.o_free[s]);
#pragma unroll
  for (int k = 0; k < RP; ++k) {
    const float sum = warp_sum(l[k]);
    if (lane == 0) share[quarter * NARROW_ROWS + k] = sum;
  }
  if (r < RP) share[4 * NARROW_ROWS + r] = ref[r];
  __syncwarp();
}

// A stream's eight warps join its two warpgroups' results of a narrow block.
template <bool FP16>
__device__ __forceinline__ void join_groups(const Params& p, QuantSmem& sm, const Item& it, unsigned char* q_smem) {
  using K = Kind<FP16, true>;
  const int s = threadIdx.x >> 8, t = threadIdx.x & 255, n_rows = it.n_tok * p.group;
  const float* merge = reinterpret_cast<const float*>(q_smem + K::q_tile);
  if (t < 4) sm.poisoned[s][0][t] = 0;
  named_bar_sync(STREAM_BAR + s, 256);
  const int c = t & 31;  // 4 dimensions
#pragma unroll 1
  for (int row = t >> 5; row < n_rows; row += 8) {
    float m[2], l[2], top = -CUDART_INF_F;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      l[g] = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) l[g] += sm.share[s][g][q * NARROW_ROWS + row];
      const float ref = sm.share[s][g][4 * NARROW_ROWS + row];
      m[g] = l[g] == 0.f ? -CUDART_INF_F : ref == -CUDART_INF_F ? 0.f : ref;
      top = fmaxf(top, m[g]);
    }
    float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (m[g] == -CUDART_INF_F) continue;
      const float w = ex2(m[g] - top);
      const float4 x = *reinterpret_cast<const float4*>(merge + ((s * 2 + g) * NARROW_ROWS + row) * D + c * 4);
      sum += l[g] * w;
      o[0] += x.x * w;
      o[1] += x.y * w;
      o[2] += x.z * w;
      o[3] += x.w * w;
    }
    const int tok = it.tok + row / p.group, head = it.kvh * p.group + row % p.group;
    if (it.parts == 1) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      float poison = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j] *= inv;
        poison += o[j] * 0.f;
      }
      *reinterpret_cast<uint2*>(p.a.out + ((int64_t)tok * p.a.hq + head) * D + c * 4) =
          make_uint2(act_pack2<FP16>(o[0], o[1]), act_pack2<FP16>(o[2], o[3]));
      if (p.a.lse && c == 0)
        p.a.lse[(int64_t)tok * p.a.hq + head] = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum) - K::weight_exp) * LN2;
      if (poison != 0.f && sum == sum) atomicOr(&sm.poisoned[s][0][0], 1u << row);
    } else {
      const size_t part_row = (((size_t)blockIdx.x * 2 + (it.part == 0 ? 1 : 0)) * 2) * ROWS + row;
      __stcg(p.part_o + part_piece(part_row, c), make_float4(o[0], o[1], o[2], o[3]));
      if (c == 0) __stcg(&p.part_ml[part_row], make_float2(top, sum));
    }
  }
  __syncwarp();
}

// What the softmax warps count.
struct Counts {
  uint32_t items = 0, fills = 0, tiles = 0;
  // In one register, as there are none to spare (prompts over 8 bits 330 -> 325 us):
  // parities of the scores, outputs, readings of the queries and narrow tiles seen, and
  // the number of joined results.
  uint32_t seen = 0;
  static constexpr uint32_t S = 1, O = 2, Q = 4, NARROW = 8, MERGE = 16;
  __device__ __forceinline__ uint32_t parity(uint32_t of) const { return (seen & of) != 0; }
};

// Items up to the end, or (true) up to a narrow one.
template <bool FP16, bool QUANT>
__device__ __forceinline__ bool softmax_items(const Params& p, Smem& sm, unsigned char* q_smem, unsigned char* kv_smem,
                                              uint32_t tmem, Counts& n) {
  using K = Kind<FP16, QUANT>;
  unsigned* err = p.a.err;
  const int s = threadIdx.x >> 8, half = (threadIdx.x >> 7) & 1;  // stream; half of the tile's keys, and of the dimensions
  const int r = threadIdx.x & 127, lane = r & 31, quarter = r >> 5;
  const int bar = STREAM_BAR + s, pair = PAIR_BAR + s * 4 + quarter;
  const uint32_t lane_base = tmem + ((uint32_t)(r & 96) << 16);
  const uint32_t t_s = lane_base + s * 128 + half * 64, t_o = lane_base + 256 + s * 128 + half * 64;
  const int row_tok = r / p.group, row_head = r % p.group;
  float sl = p.a.scale * LOG2E;
  const int all_held = QUANT ? (1 << BLOCKS8) - 1 : (1 << p.boxes) - 1;
  const int box_shift = p.a.page_shift < 7 ? p.a.page_shift : 7;
  uint32_t &fills = n.fills, &tiles = n.tiles;
  for (uint32_t& items = n.items;; ++items) {
    const uint32_t slot = items % RING;
    wait(&sm.ring_full[slot], (items / RING) & 1, sm, err);
    if (named_bar_or(bar, 256, is_dead(sm))) break;
    const Item& it = sm.ring[slot];
    if (it.b < 0) break;
    if constexpr (QUANT) {
      if (is_narrow(it.n_tok, p.group) && it.i1 > it.i0) return true;
    }
    const bool two = it.n_tok > p.tile_tok;
    const int tile = two ? s : 0, i0 = it.i0, i1 = it.i1, kv = it.kv, odd = it.lead ^ s;
    const int tb = tile * p.tile_tok + row_tok;
    const bool valid = row_tok < p.tile_tok && tb < it.n_tok;
    const int pos = it.pos + tb;
    const int hi = valid ? max(0, min(pos + 1, kv)) : 0, lo = p.a.window ? max(0, pos + 1 - p.a.window) : 0;
    const int sink = min(p.a.sinks, hi);
    if constexpr (QUANT) sl = valid ? p.q_scale[(int64_t)(it.tok + tb) * p.a.hq + it.kvh * p.group + row_head] : 1.f;
    const bool any_row = __any_sync(0xffffffffu, valid);
    const int hi_min = __reduce_min_sync(0xffffffffu, valid ? hi : 0x7fffffff);
    const int lo_max = __reduce_max_sync(0xffffffffu, valid ? lo : 0);
    const int sink_min = __reduce_min_sync(0xffffffffu, valid ? sink : 0x7fffffff);
    // key tiles that every row of the warp sees whole: up to clear_hi, from
    // clear_lo on or below clear_sink
    const int clear_hi = hi_min - 64 - half * 64, clear_lo = lo_max - half * 64, clear_sink = sink_min - 64 - half * 64;
    if constexpr (QUANT) {
      if (lane == 0) static_cast<QuantSmem&>(sm).clear[threadIdx.x >> 5] = make_int4(clear_hi, clear_lo, clear_sink, 0);
      __syncwarp();
    }
    float m = -CUDART_INF_F, l = 0.f;  // m is the row's (in 8 bits: in powers of two), l this half's
    bool stepped = false;
    // the last joined results have been read (where they are, and what was told
    // with them, is written anew)
    warp_wait(&sm.merge_free, n.parity(Counts::MERGE) ^ 1, sm, err);
    // over 8 bits the streams' warps share every tile's values
    for (int i = QUANT || two ? i0 : i0 + odd; i < i1; i += QUANT || two ? 1 : 2) {
      const int first_key = list_tile(it, i) * KT, key = first_key + half * 64;
      if constexpr (QUANT) {
        // Each takes eight rows to fp16 (a tile's places: keys, half of the wide
        // values, values), while its scores are on their way.
        const uint32_t f = fills + 3 * (i - i0) + 2, at = f % K::stages;
        // These warps do not see narrow blocks' copies, and a wait tells odd fills from
        // even: until the ring has gone round, the copy has to have begun.
        if (i - i0 < 3) wait_count(&static_cast<QuantSmem&>(sm).copied, (int)(tiles + i - i0), sm, err);
        warp_wait(K::full(sm, at), (f / K::stages) & 1, sm, err);
        widen_values(kv_smem, at, K::stages, (threadIdx.x >> 5) * 8, kv - first_key);
        if (lane == 0) mbar_arrive(&static_cast<QuantSmem&>(sm).wide_full[at]);
      }
      if (two ? !active(it.act[s], i) : QUANT && ((i - i0) & 1) != odd) continue;
      bool clear;
      if constexpr (QUANT) {
        const int4 c = static_cast<QuantSmem&>(sm).clear[threadIdx.x >> 5];
        clear = first_key <= c.x && (first_key >= c.y || first_key <= c.z);
      } else {
        clear = first_key <= clear_hi && (first_key >= clear_lo || first_key <= clear_sink);
      }
      int held = 0;
      const uint32_t scales = QUANT ? (tiles + i - i0) % SCALES : 0;
      if constexpr (QUANT) {
        if (any_row) {
          QuantSmem& qs = static_cast<QuantSmem&>(sm);
          warp_wait(&qs.scales_full[scales], ((tiles + i - i0) / SCALES) & 1, sm, err);
          held = *(volatile int*)&qs.held[scales];
        }
      }
      auto scale_of = [&](const float4 (&of)[SCALES][BLOCKS8 / 4], int b) { return reinterpret_cast<const float*>(&of[scales][half])[b]; };
      warp_wait(&sm.s_full[s], n.parity(Counts::S), sm, err);
      n.seen ^= Counts::S;
      tc::fence_after_sync();
      if (!QUANT && key + 64 > kv) {
        // the rows past the cached tokens hold whatever was there: zeros there
        // keep the products finite
        const uint32_t f = fills + 2 * (i - i0) + 1;
        wait(K::full(sm, f % K::stages), (f / K::stages) & 1, sm, err);
        const int from = max(0, kv - key);
        unsigned char* v = kv_smem + (f % K::stages) * K::tile;
        for (int c = r; c < (64 - from) * 16; c += 128) {
          const int row = half * 64 + from + (c >> 4);
          *reinterpret_cast<int4*>(v + (row >> 3) * p.group_bytes + ((c >> 3) & 1) * p.half_bytes + (row & 7) * 128 + (c & 7) * 16) =
              make_int4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (any_row) {
        if constexpr (!QUANT) held = *(volatile int*)&sm.page_mask[(tiles + i - i0) % MASKS];
        if (!clear || held != all_held) {
          // hidden scores become -inf where they are
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
            tc::tmem_ld32_async(t_s + c * 32, x);
            const int k0 = key + c * 32, box = half * 2 + c;
            uint32_t seen = bits_below(hi - k0) & (~bits_below(lo - k0) | bits_below(sink - k0));
            if (QUANT || box_shift == 4)
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
            float total;  // of the weights, which has to stay below LIMIT
            if constexpr (QUANT) {
              // The values' scale is part of the score here, so that a weight is what
              // their number is multiplied by, and is taken out of the row's sum.
              const QuantSmem& qs = static_cast<const QuantSmem&>(sm);
              const float ref = K::weight_exp - (m == -CUDART_INF_F ? 0.f : m);
              total = 0.f;
              sum[0].x = 0.f;
              uint32_t z[2][16];  // a block's scores, and the next one's on their way
              tc::tmem_ld16_async(t_s, z[0]);
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                const float a = row_factor(sl, scale_of(qs.k_scale, b)), r0 = ref + scale_of(qs.v_log, b);
                const float2 a2 = make_float2(a, a), r2 = make_float2(r0, r0);
                float2 block = make_float2(0.f, 0.f);
                tc::tmem_wait_ld();
                tc::tmem_regs(z[b & 1]);
                if (b < 3) tc::tmem_ld16_async(t_s + (b + 1) * 16, z[(b + 1) & 1]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float2 e = ffma2(make_float2(__uint_as_float(z[b & 1][2 * j]), __uint_as_float(z[b & 1][2 * j + 1])), a2, r2);
                  const float2 y = make_float2(ex2(e.x), ex2(e.y));
                  block = fadd2(block, y);
                  w[b >> 1][(b & 1) * 8 + j] = act_pack2<true>(y.x, y.y);
                }
                const float t = block.x + block.y;
                total += t;
                sum[0].x += t * scale_of(qs.v_inverse, b);
              }
            } else {
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
              total = sum[0].x;
            }
            // rows past the block hold anything and have no say
            if (pass > 0 || !named_bar_or(pair, 64, valid && (m == -CUDART_INF_F || !(total <= LIMIT)))) break;
          }
          float m_new = m;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            load(c);
            if constexpr (QUANT) {
              const QuantSmem& qs = static_cast<const QuantSmem&>(sm);
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                float top = -CUDART_INF_F;
#pragma unroll
                for (int j = b * 16; j < b * 16 + 16; j += 2)
                  top = max3(top, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                m_new = fmaxf(m_new, fmaf(top, row_factor(sl, scale_of(qs.k_scale, c * 2 + b)), scale_of(qs.v_log, c * 2 + b)));
              }
            } else {
              float top[2] = {m_new, m_new};
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                top[0] = max3(top[0], __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                top[1] = max3(top[1], __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
              }
              m_new = fmaxf(top[0], top[1]);
            }
          }
          sm.share[s][half][r] = m_new;
          named_bar_sync(pair, 64);
          m_new = fmaxf(m_new, sm.share[s][half ^ 1][r]);
          const float corr = m_new == -CUDART_INF_F ? 1.f : ex2(QUANT ? m - m_new : (m - m_new) * sl);
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
    fills += (QUANT ? 3 : 2) * (i1 - i0);
    tiles += i1 - i0;
    if (stepped) {
      // The row's sum goes where the maximum was: the other half may have yet to
      // read that when the last tile moved the reference.  (No room for a second
      // array; the last product is still under way.)
      named_bar_sync(pair, 64);
      sm.share[s][half][r] = l;
      named_bar_sync(pair, 64);
      l += sm.share[s][half ^ 1][r];
      warp_wait(&sm.o_full[s], n.parity(Counts::O), sm, err);
      n.seen ^= Counts::O;
      tc::fence_after_sync();
    }
    // m2: the reference in powers of two, -inf where the row has seen nothing, and
    // there alone: scores that are all NaN leave no maximum, but a sum, which has
    // to reach the parts' joining.
    float m2 = l == 0.f ? -CUDART_INF_F : m == -CUDART_INF_F ? 0.f : QUANT ? m : m * sl;
    const bool merged = !two && i1 - i0 > 1;
    unsigned char* merge = q_smem + (it.n_tok * p.group <= MERGE_ROWS ? K::q_tile : 0);
    if (!two && odd) {
      if (merged) {
        if (merge == q_smem) {
          warp_wait(&sm.q_read, n.parity(Counts::Q), sm, err);
          n.seen ^= Counts::Q;
        }
        n.seen += Counts::MERGE;
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
      warp_wait(&sm.merge_full, n.parity(Counts::MERGE), sm, err);
      n.seen += Counts::MERGE;
      if (merge == q_smem) n.seen ^= Counts::Q;  // over: the other stream has waited for it
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
        store_release(&sm.joined, (int)(n.seen / Counts::MERGE));
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
        p.a.lse[(int64_t)tok * p.a.hq + head] = l == 0.f ? -CUDART_INF_F : (m2 + log2f(l) - K::weight_exp) * LN2;
      const unsigned mine = __ballot_sync(0xffffffffu, valid && poison != 0.f && l == l);
      if (lane == 0) sm.poisoned[s][half][quarter] = mine;
      named_bar_sync(pair, 64);  // the row's own stores come before what is read of them
      const unsigned bad = mine | sm.poisoned[s][half ^ 1][quarter];
      if (bad) mend_rows<FP16, QUANT>(p, sm, s, half, quarter, pair, it, tile, bad);
    } else {
      if (half == 0 && valid) __stcg(&p.part_ml[part_row], make_float2(m2, l));
      if (last_part(p, sm, s, it, tile, bar)) {
        join_parts<FP16, QUANT>(p, sm, s, it, tile, min(p.tile_tok, it.n_tok - tile * p.tile_tok) * p.group);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.ring_empty[slot]);
  }
  return false;
}

// With a copy of the counts, so that the narrow blocks' calls cost the loop above no registers.
template <bool FP16>
__device__ __forceinline__ bool wide_items(const Params& p, QuantSmem& sm, unsigned char* q_smem, unsigned char* kv_smem, uint32_t tmem,
                                        Counts& n) {
  Counts c = n;  // in registers
  const bool narrow = softmax_items<FP16, true>(p, sm, q_smem, kv_smem, tmem, c);
  n = c;
  return narrow;
}

// A narrow block: by its stream's warps, the others pass it.
template <bool FP16>
__device__ __forceinline__ void narrow_item(const Params& p, QuantSmem& sm, const Item& it, unsigned char* q_smem,
                                            unsigned char* kv_smem, uint32_t tmem, Counts& n) {
  const int s = threadIdx.x >> 8, half = (threadIdx.x >> 7) & 1, quarter = (threadIdx.x >> 5) & 3;
  const int bar = STREAM_BAR + s, n_tiles = it.i1 - it.i0;
  if (it.lead == s) {
    if (octets(it.n_tok, p.group) == 1)
      narrow_block<FP16, 1>(p, sm, it, q_smem, kv_smem, tmem, n.tiles, n.fills, n.parity(Counts::NARROW), n.parity(Counts::O),
                            n.parity(Counts::MERGE));
    else
      narrow_block<FP16, 2>(p, sm, it, q_smem, kv_smem, tmem, n.tiles, n.fills, n.parity(Counts::NARROW), n.parity(Counts::O),
                            n.parity(Counts::MERGE));
    if ((n_tiles - half + 1) >> 1 & 1) n.seen ^= Counts::NARROW;
    n.seen ^= Counts::O;
    join_groups<FP16>(p, sm, it, q_smem);
    // queries may land where the results were
    fence_proxy_async_smem();
    named_bar_sync(bar, 256);
    if ((threadIdx.x & 255) == 0) store_release(&sm.narrow_done[s], sm.narrow_done[s] + 1);
    if (it.parts == 1) {
      const unsigned bad = sm.poisoned[s][0][0];
      if (bad && quarter == 0) mend_rows<FP16, true>(p, sm, s, half, quarter, PAIR_BAR + s * 4, it, 0, bad);
    } else if (last_part(p, sm, s, it, 0, bar)) {
      join_parts<FP16, true>(p, sm, s, it, 0, it.n_tok * p.group);
    }
  }
  n.fills += 2 * n_tiles;
  n.tiles += n_tiles;
}

template <bool FP16, bool QUANT>
__device__ __forceinline__ void softmax_role(const Params& p, Smem& sm, unsigned char* q_smem, unsigned char* kv_smem,
                                             uint32_t tmem) {
  Counts n;
  if constexpr (QUANT) griddep_wait();  // the rows' factors
  if constexpr (QUANT) {
    QuantSmem& qs = static_cast<QuantSmem&>(sm);
    const int lane = threadIdx.x & 31;
    while (wide_items<FP16>(p, qs, q_smem, kv_smem, tmem, n)) {
      narrow_item<FP16>(p, qs, sm.ring[n.items % RING], q_smem, kv_smem, tmem, n);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ring_empty[n.items % RING]);
      ++n.items;
    }
  } else {
    softmax_items<FP16, QUANT>(p, sm, q_smem, kv_smem, tmem, n);
  }
}

template <bool FP16, bool QUANT>
__global__ void __launch_bounds__(THREADS, 1)
    attention_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) unsigned char q_smem[];  // the swizzle repeats every 1024 bytes
  using K = Kind<FP16, QUANT>;
  unsigned char* kv_smem = q_smem + 2 * K::q_tile;
  using Shared = typename std::conditional<QUANT, QuantSmem, Smem>::type;
  Shared& sm = *reinterpret_cast<Shared*>(kv_smem + K::stages * K::tile);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  if (threadIdx.x == PLAN_WARP * 32) {
    for (int i = 0; i < K::stages; ++i) {
      mbar_init(K::full(sm, i), 1);
      mbar_init(K::empty(sm, i), 2);  // both streams
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
    if constexpr (QUANT) {
      for (int g = 0; g < 4; ++g) {
        mbar_init(&sm.narrow_s[g], 1);
        mbar_init(&sm.narrow_p[g], 4);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.narrow_q_full[i], 1);
        mbar_init(&sm.narrow_q_empty[i], 2);  // both streams
      }
      for (int i = 0; i < SCALES; ++i) mbar_init(&sm.scales_full[i], 1);
      for (int i = 0; i < K::stages; ++i) mbar_init(&sm.wide_full[i], SOFTMAX_WARPS);
      sm.copied = sm.narrow_done[0] = sm.narrow_done[1] = 0;
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
  // In 8 bits the kernel before is the queries' split, which lets this one begin
  // when what came before it is done: only those who take its results wait for it.
  if constexpr (!QUANT) griddep_wait();
  const long long piece = measure_line<QUANT>(p, sm, blockIdx.x);
  __syncthreads();
  const uint32_t tmem = sm.tmem;
  if (warp < SOFTMAX_WARPS) {
    softmax_role<FP16, QUANT>(p, sm, q_smem, kv_smem, tmem);
  } else if (warp == LOAD_WARP) {
    load_role<FP16, QUANT>(p, maps, sm, q_smem, kv_smem);
  } else if (warp >= MMA_WARP) {
    mma_role<FP16, QUANT>(p, sm, warp - MMA_WARP, smem_u32(q_smem), kv_smem, tmem, FP16 ? 0u : 1u);
  } else if (warp == PLAN_WARP) {
    plan_role<QUANT>(p, sm, blockIdx.x, piece);
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == MMA_WARP) tc::tmem_dealloc(tmem, 512);
}

constexpr size_t SMEM_BYTES = (2 + STAGES) * TILE_BYTES + sizeof(Smem);
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");
template <bool FP16>
constexpr size_t SMEM_BYTES8 = 2 * Kind<FP16, true>::q_tile + STAGES8<FP16> * TILE8_BYTES + sizeof(QuantSmem);
static_assert(SMEM_BYTES8<false> <= 232448 && SMEM_BYTES8<true> <= 232448, "shared memory of one CTA");
static_assert(NARROW_P<false> + 4 * NARROW_W <= Kind<false, true>::q_tile &&
                  NARROW_P<true> + 4 * NARROW_W <= Kind<true, true>::q_tile,
              "narrow blocks' queries and weights in the first tile's place");
static_assert(4 * NARROW_ROWS * D * 4 <= Kind<false, true>::q_tile, "their results in the second one's");

// The queries of a call in 8-bit parts, [part][token][head][128], and each row's
// factor: a row is taken to [2^7, 2^8) by a power of two, and every part what is
// left to the nearest e4m3 (4 significant bits).  Two parts are a bf16 number,
// three an fp16 one, down to 2^-17 of the row's largest.  16 lanes a row.  Bound by
// memory (256 bytes in, 256 or 384 out a row): 11,000 tokens of 32 heads 27 us.
constexpr int SPLIT_ROWS = 4;  // that a thread has under way
template <bool FP16>
__global__ void __launch_bounds__(256) split_queries_kernel(AttentionParams p, uint8_t* parts, float* factors) {
  // In this order: the attention kernel may begin once all of this grid is past the
  // wait, and so after everything before this call.
  griddep_wait();
  griddep_launch_dependents();
  const int64_t rows = (int64_t)p.t_total * p.hq, first = blockIdx.x * (16ll * SPLIT_ROWS) + (threadIdx.x >> 4);
  const int c = (threadIdx.x & 15) * 8;
  const unsigned group = 0xffffu << (threadIdx.x & 16);
  uint4 raw[SPLIT_ROWS];
#pragma unroll
  for (int i = 0; i < SPLIT_ROWS; ++i) {
    const int64_t row = first + i * 16, tok = row / p.hq;
    if (row < rows) raw[i] = *reinterpret_cast<const uint4*>(p.q + tok * p.q_st + (row - tok * p.hq) * p.q_sh + c);
  }
#pragma unroll
  for (int i = 0; i < SPLIT_ROWS; ++i) {
    const int64_t row = first + i * 16;
    if (row >= rows) return;  // 16 lanes alike
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    float x[8], top = 0.f;
    bool finite = true;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = act_f2<FP16>(reinterpret_cast<const __nv_bfloat16*>(&w[k]));
      x[2 * k] = v.x;
      x[2 * k + 1] = v.y;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      top = fmaxf(top, fabsf(x[k]));
      finite = finite && fabsf(x[k]) < CUDART_INF_F;
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(group, top, d));
    finite = __all_sync(group, finite);
    const int e = max(-110, (__float_as_int(top) >> 23) - 127 - 7);  // of the row's power of two (0 and what is not finite: any)
    const float down = __int_as_float((127 - (finite ? e : 0)) << 23);
#pragma unroll
    for (int part = 0; part < Q_PARTS<FP16>; ++part) {
      uint32_t y[2];
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float a = part == 0 ? x[k] * down : x[k], b = part == 0 ? x[k + 1] * down : x[k + 1];
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(b), "f"(a));
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        const float2 taken = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x[k] = a - taken.x;
        x[k + 1] = b - taken.y;
        if (!finite) two = 0x7f7f;
        if (k & 2) y[k >> 2] |= (uint32_t)two << 16;
        else y[k >> 2] = two;
      }
      *reinterpret_cast<uint2*>(parts + ((int64_t)part * rows + row) * D + c) = make_uint2(y[0], y[1]);
    }
    if (c == 0) factors[row] = p.scale * LOG2E * __int_as_float((127 + (finite ? e : 0)) << 23);
  }
}

int sm_count() {
  static int counts[64] = {0};
  static uint64_t done = 0;
  int dev = 0;
  const bool have = once_per_device(done, [&](int d) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) == cudaSuccess) counts[d] = n;
    cudaFuncSetAttribute(attention_kernel<false, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    cudaFuncSetAttribute(attention_kernel<true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    cudaFuncSetAttribute(attention_kernel<false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES8<false>);
    cudaFuncSetAttribute(attention_kernel<true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES8<true>);
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

// Bytes: [n4, n3, n2, n1, 128], strides s4 .. s1; boxes of whole rows, b1 x b2 x b3 of them.
bool encode8(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, int rank, const void* base, int64_t n1, int64_t s1, int64_t n2,
             int64_t s2, int64_t n3, int64_t s3, int64_t n4, int64_t s4, uint32_t b1, uint32_t b2, uint32_t b3) {
  const cuuint64_t dims[5] = {(cuuint64_t)D, (cuuint64_t)n1, (cuuint64_t)n2, (cuuint64_t)n3, (cuuint64_t)n4};
  const cuuint64_t strides[4] = {(cuuint64_t)(n1 > 1 ? s1 : D), (cuuint64_t)(n2 > 1 ? s2 : D), (cuuint64_t)(n3 > 1 ? s3 : D),
                                 (cuuint64_t)(n4 > 1 ? s4 : D)};
  const cuuint32_t box[5] = {D, b1, b2, b3, 1}, step[5] = {1, 1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Work and workspace of a call, whatever the cache.
void plan_call(Params& p, const AttentionParams& a, void* workspace) {
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
}

void launch_kernel(void (*kernel)(const Params, const Maps), const Params& p, const Maps& maps, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.n_cta);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, p, maps);
}

}  // namespace

size_t attention_workspace_bytes() {
  return KDA_ATTENTION_ZEROED_BYTES + (size_t)sm_count() * 4 * ROWS * (sizeof(float2) + 32 * sizeof(float4));
}

int launch_attention(const AttentionParams& a, bool fp16, void* workspace, cudaStream_t stream) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
  if (!enc) return -1;
  Params p = {};
  plan_call(p, a, workspace);
  const int page = 1 << a.page_shift;
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
  trace_begin("attention", stream);
  launch_kernel(fp16 ? attention_kernel<true, false> : attention_kernel<false, false>, p, maps, SMEM_BYTES, stream);
  trace_end(stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

size_t attention_quant_workspace_bytes(int t_total, int hq) {
  return attention_workspace_bytes() + (size_t)t_total * hq * (3 * D + sizeof(float));
}

int launch_attention_quant(const AttentionParams& a, const KvQuantCache& c, bool fp16, void* workspace, cudaStream_t stream) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
  if (!enc) return -1;
  Params p = {};
  plan_call(p, a, workspace);
  p.c = c;
  p.min_piece *= COST_NARROW8;
  const int page = 1 << a.page_shift, box = page < KT ? page : KT, parts = fp16 ? Q_PARTS<true> : Q_PARTS<false>;
  p.group_bytes = 1024;
  p.half_bytes = 16;  // a row is whole: not used
  const int64_t rows = (int64_t)a.t_total * a.hq;
  uint8_t* q_parts = static_cast<uint8_t*>(workspace) + attention_workspace_bytes();
  float* factors = reinterpret_cast<float*>(q_parts + 3 * rows * D);
  p.q_scale = factors;
  Maps maps;
  const int64_t head = D, kv_head = (int64_t)p.group * D, tok = (int64_t)a.hq * D;
  if (!encode8(enc, &maps.k, 4, c.k, page, c.k_st, a.hkv, c.k_sh, a.n_pages, c.k_sp, 1, D, box, 1, 1) ||
      !encode8(enc, &maps.v, 4, c.v, page, c.v_st, a.hkv, c.v_sh, a.n_pages, c.v_sp, 1, D, box, 1, 1) ||
      !encode8(enc, &maps.q, 5, q_parts, p.group, head, a.hkv, kv_head, a.t_total, tok, parts, rows * D, p.group, 1, p.tile_tok) ||
      !encode8(enc, &maps.q1, 5, q_parts, p.group, head, a.hkv, kv_head, a.t_total, tok, parts, rows * D, p.group, 1, 1))
    return -1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((rows + 16 * SPLIT_ROWS - 1) / (16 * SPLIT_ROWS)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_begin("split_queries", stream);
  cudaLaunchKernelEx(&cfg, fp16 ? split_queries_kernel<true> : split_queries_kernel<false>, a, q_parts, factors);
  trace_end(stream);
  trace_begin("attention_quant", stream);
  if (fp16) launch_kernel(attention_kernel<true, true>, p, maps, SMEM_BYTES8<true>, stream);
  else launch_kernel(attention_kernel<false, true>, p, maps, SMEM_BYTES8<false>, stream);
  trace_end(stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace kda
