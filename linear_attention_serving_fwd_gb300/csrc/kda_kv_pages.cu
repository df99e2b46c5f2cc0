// Pages for a step's tokens (extend), their return (truncate) and the write
// of keys and values to their slots (append).
//
// extend and truncate are sums over the requests (pages wanted, tokens) and
// writes found by a search in them.  A few hundred bytes to a few hundred
// kilobytes move, so the time is latency: launch, length loads, the block's
// sums, the search, a table or free-list load.  Measured on the device, extend
// and truncate together: 6.8 us for one token each of 16 requests, 8.3 for 256,
// 17.8 for four each of 2048 (two rounds of 1024), 17.1 for 98,000 tokens of 48.
// append moves 256 bytes per token and head of keys and of values: 1.8 us for
// 256 tokens of 8 heads, 40.9 us for 32768 (268 MB, 6.6 TB/s, a copy's rate).
#include "kda_kv.cuh"

namespace kda {
namespace {

constexpr int PT = 1024;  // threads: one request each per round
// One CTA writes up to EXTEND_ONE slots, a thread each, a cluster of EXTEND_CTAS
// more (extend and truncate together, one CTA against eight): 16 slots 6.8 us
// against 7.0, 1000 slots 9.4 against 9.8, 1200 slots 10.8 against 10.2, 4096
// slots 12.9 against 10.3, 98,000 slots 60 against 17.1.
constexpr int EXTEND_CTAS = 8, EXTEND_ONE = PT;

// Inclusive sums of two values over the block, and both totals.
struct Scan2 {
  long long a, b, total_a, total_b;
};
__device__ __forceinline__ Scan2 block_scan2(long long a, long long b, long long (*sums)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, s), y = __shfl_up_sync(0xffffffffu, b, s);
    if (lane >= s) {
      a += x;
      b += y;
    }
  }
  __syncthreads();  // the previous call's sums have been read
  if (lane == 31) {
    sums[warp][0] = a;
    sums[warp][1] = b;
  }
  __syncthreads();
  if (warp == 0) {
    long long x = sums[lane][0], y = sums[lane][1];
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, s), v = __shfl_up_sync(0xffffffffu, y, s);
      if (lane >= s) {
        x += u;
        y += v;
      }
    }
    sums[lane][0] = x;
    sums[lane][1] = y;
  }
  __syncthreads();
  if (warp > 0) {
    a += sums[warp - 1][0];
    b += sums[warp - 1][1];
  }
  return {a, b, sums[31][0], sums[31][1]};
}

// Last i in [0, n) with off[i] <= x (off non-decreasing, off[0] <= x): the
// owner of element x when off holds exclusive sums.
template <typename T>
__device__ __forceinline__ int owner(const T* off, int n, T x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

__device__ __forceinline__ int clamped_count(const KvPagesParams& p, bool report) {
  const int c = *p.free_count;
  if (c < 0 || c > p.n_pages) {
    if (report) set_error(p.err, ERR_INDEX);
    return c < 0 ? 0 : p.n_pages;
  }
  return c;
}

// One thread per request and round: page counts and token counts are summed
// over the block, then the round's tokens and pages are spread over all
// threads, each finding its request in the sums.  The CTAs of the cluster
// each form the same sums, share out tokens and pages, and only the first
// updates the lengths and the free count, once all have read them.
__global__ void __launch_bounds__(PT) kv_extend_kernel(KvPagesParams p) {
  __shared__ long long sums[32][2];
  __shared__ long long page_off[PT];  // what a round asks for can pass 32 bits, though no free list does
  __shared__ int tok_off[PT], r_len[PT], r_have[PT];  // r_have < 0: not admitted
  const int t = threadIdx.x, page = 1 << p.page_shift;
  const int rank = cluster_rank(), stride = PT * (int)gridDim.x, first = rank * PT + t;
  const int count = clamped_count(p, first == 0);
  long long tok_base = 0, page_base = 0, taken = 0;
  for (int r0 = 0; r0 < p.n_req; r0 += PT) {
    const int b = r0 + t, n_round = min(PT, p.n_req - r0);
    long long n_new = 0, add = 0;
    int len = 0, have = 0;
    bool valid = false;
    if (b < p.n_req) {
      len = p.kv_lens[b];
      n_new = p.lens[b];
      valid = n_new >= 0 && len >= 0 && len <= (p.table_cols << p.page_shift);
      if (n_new < 0) n_new = 0;
      if (valid) {
        have = (len + page - 1) >> p.page_shift;
        const long long need = (len + n_new + page - 1) >> p.page_shift;
        valid = need <= p.table_cols;
        add = valid ? need - have : 0;
      }
      if (!valid && rank == 0) set_error(p.err, ERR_INDEX);
    }
    if (gridDim.x > 1) cluster_arrive();  // lengths (and the count) have been read
    const Scan2 s = block_scan2(n_new, add, sums);
    const bool fits = valid && (add == 0 || page_base + s.b <= count);
    tok_off[t] = (int)min(tok_base + s.a - n_new, 0x7fffffffLL);
    page_off[t] = s.b - add;
    r_len[t] = len;
    r_have[t] = fits ? have : -1;
    // admitted pages are a prefix of the sums: the first refusal ends it
    long long top = fits && add > 0 ? page_base + s.b : 0;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
    __syncthreads();
    if ((t & 31) == 0) sums[t >> 5][0] = top;
    if (gridDim.x > 1) cluster_wait();
    if (rank == 0 && b < p.n_req) {
      // sums past int32 are out of max_tokens' range as well
      p.cu_seqlens[b + 1] = (int)min(tok_base + s.a, 0x7fffffffLL);
      p.step_lens[b] = fits ? (int)(len + n_new) : 0;
      if (fits && n_new > 0) p.kv_lens[b] = (int)(len + n_new);
      if (tok_base + s.a > p.max_tokens && n_new > 0) set_error(p.err, ERR_INDEX);
    }
    const long long tok_end = min(tok_base + s.total_a, (long long)p.max_tokens);
    const int pages_end = (int)min(s.total_b, max(0LL, count - page_base));
    for (int i = first; i < pages_end; i += stride) {
      const int r = owner(page_off, n_round, (long long)i);
      if (r_have[r] < 0) continue;
      const int col = r_have[r] + (int)(i - page_off[r]);
      p.table[(int64_t)(r0 + r) * p.table_stride + col] = p.free_pages[count - 1 - (page_base + i)];
    }
#pragma unroll 4
    for (long long i = tok_base + first; i < tok_end; i += stride) {
      const int r = owner(tok_off, n_round, (int)i);
      int slot = -1;
      if (r_have[r] >= 0) {
        const int pos = r_len[r] + (int)i - tok_off[r], col = pos >> p.page_shift;
        const int32_t* from = col < r_have[r] ? p.table + (int64_t)(r0 + r) * p.table_stride + col
                                              : p.free_pages + (count - 1 - (page_base + page_off[r] + col - r_have[r]));
        const int pg = *from;
        slot = (pg << p.page_shift) + (pos & (page - 1));
        if (pg < 0 || pg >= p.n_pages) {
          set_error(p.err, ERR_INDEX);
          slot = -1;
        }
      }
      p.slot_map[i] = slot;
    }
    __syncthreads();
    for (int i = 0; i < 32; ++i) taken = max(taken, sums[i][0]);
    tok_base += s.total_a;
    page_base += s.total_b;
  }
  for (long long i = tok_base + first; i < p.max_tokens; i += stride) p.slot_map[i] = -1;
  if (first == 0) {
    p.cu_seqlens[0] = 0;
    *p.free_count = count - (int)taken;
  }
}

// Requests from the last to the first, one per thread and round.  The columns
// they give up are read in the stack's order, a thread each, and those that hold
// a page move together: a page that left a window has been handed back by
// whoever put a negative entry in its place.
__global__ void __launch_bounds__(PT) kv_truncate_kernel(KvPagesParams p) {
  __shared__ long long sums[32][2];
  __shared__ long long page_off[PT];
  __shared__ int r_have[PT], held[2][32];  // held: pages of each warp, by parity of the step
  const int t = threadIdx.x, lane = t & 31, page = 1 << p.page_shift;
  const int count = clamped_count(p, t == 0);
  long long base = 0;
  int step = 0;
  for (int r0 = 0; r0 < p.n_req; r0 += PT) {
    const int b = p.n_req - 1 - (r0 + t), n_round = min(PT, p.n_req - r0);
    long long drop = 0;
    int have = 0;
    if (b >= 0) {
      const int len = p.kv_lens[b], keep = p.lens[b];
      if (keep < 0 || len < 0 || len > (p.table_cols << p.page_shift)) {
        set_error(p.err, ERR_INDEX);
      } else if (keep < len) {
        have = (len + page - 1) >> p.page_shift;
        drop = have - ((keep + page - 1) >> p.page_shift);
        p.kv_lens[b] = keep;
      }
    }
    const Scan2 s = block_scan2(0, drop, sums);
    page_off[t] = s.b - drop;
    r_have[t] = have;
    __syncthreads();
    for (long long i0 = 0; i0 < s.total_b; i0 += PT, step ^= 1) {
      const long long i = i0 + t;
      int32_t* entry = nullptr;
      int pg = -1;
      if (i < s.total_b) {
        const int r = owner(page_off, n_round, i);
        const int col = r_have[r] - 1 - (int)(i - page_off[r]);
        entry = p.table + (int64_t)(p.n_req - 1 - (r0 + r)) * p.table_stride + col;
        pg = *entry;
        if (pg >= p.n_pages) {
          set_error(p.err, ERR_INDEX);
          pg = -1;
        }
      }
      const unsigned pages = __ballot_sync(0xffffffffu, pg >= 0);
      if (lane == 0) held[step][t >> 5] = __popc(pages);
      __syncthreads();
      const int n = held[step][lane];
      const int before = __reduce_add_sync(0xffffffffu, lane < (t >> 5) ? n : 0) + __popc(pages & ((1u << lane) - 1));
      const long long at = count + base + before;
      if (pg >= 0 && at >= p.n_pages) {
        set_error(p.err, ERR_INDEX);
      } else if (entry) {
        if (pg >= 0) p.free_pages[at] = pg;
        *entry = -1;
      }
      base += __reduce_add_sync(0xffffffffu, n);
    }
    __syncthreads();
  }
  if (t == 0) *p.free_count = (int)min(count + base, (long long)p.n_pages);
}

// One 16-byte piece of a key and of a value row per thread and step.
__global__ void __launch_bounds__(256) kv_append_kernel(KvAppendParams p) {
  const int64_t pieces = (int64_t)p.t_total * p.hkv * (D / 8);
  const int64_t rows = (int64_t)p.n_pages << p.page_shift;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < pieces; i += gridDim.x * 256ll) {
    const int c = (int)(i % (D / 8)) * 8;
    const int64_t th = i / (D / 8);
    const int h = (int)(th % p.hkv), t = (int)(th / p.hkv);
    const int slot = p.slot_map[t];
    if (slot < 0) continue;
    if (slot >= rows) {
      set_error(p.err, ERR_INDEX);
      continue;
    }
    const int64_t pg = slot >> p.page_shift, row = slot & ((1 << p.page_shift) - 1);
    const int4 kx = *reinterpret_cast<const int4*>(p.k + t * p.k_st + h * p.k_sh + c);
    const int4 vx = *reinterpret_cast<const int4*>(p.v + t * p.v_st + h * p.v_sh + c);
    *reinterpret_cast<int4*>(p.kc + pg * p.kc_sp + row * p.kc_st + h * p.kc_sh + c) = kx;
    *reinterpret_cast<int4*>(p.vc + pg * p.vc_sp + row * p.vc_st + h * p.vc_sh + c) = vx;
  }
}

}  // namespace

int launch_kv_extend(const KvPagesParams& p, cudaStream_t stream) {
  trace_begin("kv_extend", stream);
  // One cluster: the lengths are updated in place, so the CTAs that share the
  // tokens out have to agree on when they have been read.
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  const unsigned ctas = p.max_tokens > EXTEND_ONE ? EXTEND_CTAS : 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(PT);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kv_extend_kernel, p);
  trace_end(stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_kv_truncate(const KvPagesParams& p, cudaStream_t stream) {
  trace_begin("kv_truncate", stream);
  kv_truncate_kernel<<<1, PT, 0, stream>>>(p);
  trace_end(stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_kv_append(const KvAppendParams& p, cudaStream_t stream) {
  const int64_t pieces = (int64_t)p.t_total * p.hkv * (D / 8);
  const int64_t blocks = (pieces + 255) / 256;
  trace_begin("kv_append", stream);
  kv_append_kernel<<<(unsigned)(blocks < 152 * 32 ? blocks : 152 * 32), 256, 0, stream>>>(p);
  trace_end(stream);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace kda
