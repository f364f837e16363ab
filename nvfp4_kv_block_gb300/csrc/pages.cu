// Pages of a cache that several sequences share: pages for new tokens, forks of a
// sequence, their release, page copies, and the accepted drafts of a tree moved
// together behind their sequence's context.
//
// A pool's pages are counted: refs[p] block-table entries hold page p, and bit p of
// the free mask is set while that is none.  A sequence holds the entries of its row that
// are not negative, those behind its length (kept for later tokens) too.  Pages are dealt
// lowest number first, in the order of the call's sequences, so that the same calls on the
// same state give the same pages whatever the launch.
//
// Bookkeeping is a few kilobytes and a chain of latencies: one CTA reads lengths and
// the mask (a bit a page: 61,440 pages are 7.5 KB, where their counts are 240 KB), finds the
// first free pages by a scan over the words' bit counts and writes tables and slots.  Bytes
// of tokens move in a second, wide launch, the bytes of the tokens that exist only.
//
// Every kernel is a programmatic dependent of the one before it and lets the next begin
// launching at once; it touches memory behind pdl_wait only (release, fork and extension of
// 256 rows, 45.4 us a pass; before targets' rows were looked at as a whole 43.8, and 49.8 with plain launches).  On the
// GPU the pass takes 3.4 for the release, 1.3 for the look at the targets' rows, 8 for the plan, 28 for the copies (12 layers, 246 MB read and written, 8.8 TB/s: partly
// from L2) and 7.5 for the extension: three chains of a few dependent loads and one launch bound
// by memory.  A commit of 8 x 8 drafts takes 2.4 us, of 64 x 64 in 12 layers 6 to 7.5 (9.8 MB).
#include "common.cuh"

namespace msa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kOwnSeqs = kMaxSeqs / kPlanThreads;  // sequences or pairs of a planning thread
constexpr int kCopyThreads = 128;
constexpr int kParts = kKvHeads + 1;  // of a page: its heads, and its index keys

struct LayerPools {
  uint8_t* kv[kMaxLayers];
  uint8_t* idx[kMaxLayers];
  int n_layers;
  int64_t n_pages;  // of the smallest pool
};

struct Pool {
  int* refs;
  uint32_t* free_mask;
  int n_pages;
  int* status;
};

// Exclusive prefix of x over the CTA's threads and its sum; s_warp: 32 words.
__device__ __forceinline__ int block_scan(int x, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  __syncthreads();  // (the words' last readers)
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  const int w = lane < kPlanThreads / 32 ? s_warp[lane] : 0;
  int sums = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += v;
  }
  total = __shfl_sync(0xffffffffu, sums, 31);
  const int before = __shfl_sync(0xffffffffu, sums - w, warp);
  return before + incl - x;
}

// The first `want` free pages, ascending, into list; returns how many there are (up to want).
// Nothing is taken yet.
__device__ int find_free(const Pool& p, int want, int* list, int* s_warp) {
  int found = 0;
  const int words = (p.n_pages + 31) / 32;
  for (int w0 = 0; w0 < words && found < want; w0 += 4 * kPlanThreads) {
    uint32_t m[4];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = w0 + 4 * threadIdx.x + i;
      m[i] = w < words ? p.free_mask[w] : 0u;
      if (w == words - 1 && p.n_pages % 32) m[i] &= (1u << p.n_pages % 32) - 1;
      mine += __popc(m[i]);
    }
    int total;
    int at = found + block_scan(mine, s_warp, total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      for (uint32_t x = m[i]; x && at < want; x &= x - 1, ++at)
        list[at] = 32 * (w0 + 4 * (int)threadIdx.x + i) + __ffs(x) - 1;
    found += total;
  }
  __syncthreads();
  return min(found, want);
}
__device__ __forceinline__ void take(const Pool& p, int page) {
  p.refs[page] = 1;
  atomicAnd(p.free_mask + page / 32, ~(1u << page % 32));
}

// ---- pages and slots of new tokens ------------------------------------------------
struct ExtendParams {
  Pool pool;
  int* block_table;
  int max_pages;
  int* seq_lens;
  const int* q_start_loc;
  int n_seqs;
  int n_tokens;
  int64_t* slots;
  int wide;  // the slots behind each sequence's first are left to slots_kernel
};
// Pages that one call can deal: a sequence touches at most n / 128 + 2 blocks.
constexpr int kMaxExtendTokens = 262144;
constexpr int kMaxDealt = kMaxExtendTokens / kPageTokens + 2 * kMaxSeqs;
constexpr int kExtendSmem = (kMaxDealt + 2 * (kMaxSeqs + 1) + 32) * sizeof(int);
// Entries of a sequence that one thread looks at and deals; a warp takes more of them (with the release behind
// it, 16 rows of 2,048 tokens: 13 us, 18 where a warp takes 9 entries and more; one of 8,192: 9.5, 16 without warps).
constexpr int kOwnEntries = 20;
// Tokens whose slots the planning CTA writes, 1,024 at a time; a wide launch behind it those of more
// (with the release, 4,096 tokens: 6.3 to 7.8 us, 8.5 by a wide launch; 262,144: 324 and 37 to 39).
constexpr int kPlanTokens = 4096;

__device__ __forceinline__ int64_t slot_at(const int* row, int pos) {
  return (int64_t)row[pos / kPageTokens] * kPageTokens + pos % kPageTokens;
}

__global__ void __launch_bounds__(kPlanThreads) extend_kernel(const __grid_constant__ ExtendParams p) {
  extern __shared__ int smem[];
  int* list = smem;                         // [kMaxDealt]
  int* s_start = list + kMaxDealt;          // [n_seqs + 1] first token
  int* s_len = s_start + kMaxSeqs + 1;      // [n_seqs] tokens before, or -1: no page was left or no sequence
  int* s_warp = s_len + kMaxSeqs + 1;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  // sequences per * tid ..: the entries from first to last get pages; what each is short of (-1: left out)
  const int per = (p.n_seqs + kPlanThreads - 1) / kPlanThreads;
  int need[kOwnSeqs], first[kOwnSeqs], last[kOwnSeqs], mine = 0;
  bool back = false;
#pragma unroll
  for (int i = 0; i < kOwnSeqs; ++i) {
    const int b = per * tid + i;
    need[i] = -1;
    first[i] = 0;
    last[i] = -1;
    if (i < per && b < p.n_seqs) {
      const int start = p.q_start_loc[b], n = p.q_start_loc[b + 1] - start, len = p.seq_lens[b];
      s_start[b] = start;
      back |= n < 0;
      if (b == p.n_seqs - 1) s_start[b + 1] = start + n;
      bool ok = n >= 0 && start >= 0 && n <= p.n_tokens - start && len >= 0 && (long long)len + n <= (long long)p.max_pages * kPageTokens;
      const int* row = p.block_table + (size_t)b * p.max_pages;
      if (!ok) {
        set_status(p.pool.status, MSA_STATUS_BAD_SEQ);
      } else if (n > 0 && len % kPageTokens && row[len / kPageTokens] < 0) {  // tokens without a page
        set_status(p.pool.status, MSA_STATUS_BAD_PAGE);
        ok = false;
      }
      s_len[b] = ok ? len : -1;
      if (ok) {
        need[i] = 0;
        first[i] = (len + kPageTokens - 1) / kPageTokens;
        last[i] = n > 0 ? (len + n - 1) / kPageTokens : -1;
        if (last[i] - first[i] < kOwnEntries)
#pragma unroll
          for (int u = 0; u < kOwnEntries; ++u) need[i] += first[i] + u <= last[i] && row[first[i] + u] < 0;
      }
    }
    for (uint32_t m = __ballot_sync(0xffffffffu, last[i] - first[i] >= kOwnEntries); m; m &= m - 1) {
      const int who = __ffs(m) - 1, x1 = __shfl_sync(0xffffffffu, last[i], who);
      const int* row = p.block_table + (size_t)(per * (tid - lane + who) + i) * p.max_pages;
      int count = 0;
#pragma unroll 4
      for (int x = __shfl_sync(0xffffffffu, first[i], who) + lane; x <= x1; x += 32) count += row[x] < 0;
      count = __reduce_add_sync(0xffffffffu, count);
      if (lane == who) need[i] = count;
    }
    mine += max(need[i], 0);
  }
  // Where q_start_loc goes back some tokens are of several sequences, and which slots they and the tokens behind
  // them had would depend on the threads' order: none grows then.
  if (__syncthreads_or(back)) {
    mine = 0;
#pragma unroll
    for (int i = 0; i < kOwnSeqs; ++i)
      if (need[i] >= 0) {
        need[i] = -1;
        s_len[per * tid + i] = -1;
      }
  }
  int want;
  int at = block_scan(mine, s_warp, want);
  const int have = want > 0 ? find_free(p.pool, min(want, kMaxDealt), list, s_warp) : 0;
  // from the first sequence that does not fit on, none gets a page
#pragma unroll
  for (int i = 0; i < kOwnSeqs; ++i) {
    const int b = per * tid + i;
    bool dealt = false;
    if (need[i] >= 0) {
      const int n = p.q_start_loc[b + 1] - p.q_start_loc[b], len = s_len[b];
      dealt = need[i] == 0 || at + need[i] <= have;
      if (!dealt) {
        set_status(p.pool.status, MSA_STATUS_NO_PAGES);
        s_len[b] = -1;
      } else if (n > 0) {
        p.seq_lens[b] = len + n;
      }
      if (dealt && last[i] - first[i] < kOwnEntries) {
        int* row = p.block_table + (size_t)b * p.max_pages;
        for (int x = first[i], k = at; k < at + need[i]; ++x)
          if (row[x] < 0) {
            const int page = list[k++];
            take(p.pool, page);
            row[x] = page;
          }
      }
    }
    for (uint32_t m = __ballot_sync(0xffffffffu, dealt && need[i] > 0 && last[i] - first[i] >= kOwnEntries); m; m &= m - 1) {
      const int who = __ffs(m) - 1, x1 = __shfl_sync(0xffffffffu, last[i], who);
      int* row = p.block_table + (size_t)(per * (tid - lane + who) + i) * p.max_pages;
      int k = __shfl_sync(0xffffffffu, at, who);
      for (int x0 = __shfl_sync(0xffffffffu, first[i], who); x0 <= x1; x0 += 32) {
        const int x = x0 + lane;
        const bool empty = x <= x1 && row[x] < 0;
        const uint32_t all = __ballot_sync(0xffffffffu, empty);
        if (empty) {
          const int page = list[k + __popc(all & ((1u << lane) - 1))];
          take(p.pool, page);
          row[x] = page;
        }
        k += __popc(all);
      }
    }
    at += max(need[i], 0);
  }
  __syncthreads();
  if (p.wide) {
    for (int b = tid; b < p.n_seqs; b += kPlanThreads) {
      const int t = s_start[b];
      if (t >= 0 && t < p.n_tokens && s_start[b + 1] > t)
        p.slots[t] = s_len[b] >= 0 ? slot_at(p.block_table + (size_t)b * p.max_pages, s_len[b]) : -1;
    }
    return;
  }
  for (int t = tid; t < p.n_tokens; t += kPlanThreads) {
    int lo = 0, hi = p.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_start[mid] <= t) lo = mid; else hi = mid - 1;
    }
    int64_t slot = -1;
    if (t >= s_start[lo] && t < s_start[lo + 1] && s_len[lo] >= 0)
      slot = slot_at(p.block_table + (size_t)lo * p.max_pages, s_len[lo] + t - s_start[lo]);
    p.slots[t] = slot;
  }
}
// The slots behind a sequence's first one, whose sign says whether the sequence grew.
__global__ void __launch_bounds__(kCopyThreads) slots_kernel(const __grid_constant__ ExtendParams p) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x * kCopyThreads + threadIdx.x;
  if (t >= p.n_tokens) return;
  int lo = 0, hi = p.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.q_start_loc[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int start = p.q_start_loc[lo], n = p.q_start_loc[lo + 1] - start;
  int64_t slot = -1;
  if (t >= start && t - start < n) {
    if (t == start) return;
    const long long pos = (long long)p.seq_lens[lo] - n + (t - start);
    if (start >= 0 && p.slots[start] >= 0 && pos >= 0 && pos < (long long)p.max_pages * kPageTokens)
      slot = slot_at(p.block_table + (size_t)lo * p.max_pages, (int)pos);
  }
  p.slots[t] = slot;
}

// ---- forks ------------------------------------------------------------------------
struct ForkParams {
  Pool pool;
  int* block_table;
  int max_pages;
  int* seq_lens;
  int n_seqs;
  const int* src;
  const int* dst;
  int n;
  int4* plan;  // [n] workspace: tokens (-1: no fork), page to copy from and to (-1: none), 0
  int wide;    // the targets' rows were looked at by fork_rows_kernel (plan[x].x: a page is held)
  LayerPools layers;
};
// A target is empty if no entry of its row holds a page; a caller may keep one anywhere in it.  Up to one entry a
// thread of the planning CTA it looks at them itself (with the release behind it, 16 rows of 34 entries: 8.0 us; a wide
// launch takes the host another 3.5), a wide launch before it at more (256 rows of 34: 13.4 us, 19 by the planning
// CTA; 128 of 1,024: 15.2 and 85).
constexpr int kPlanEntries = kPlanThreads;
__global__ void __launch_bounds__(kCopyThreads) fork_rows_kernel(const __grid_constant__ ForkParams p) {
  const int x = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int dst = p.dst[x];
  int holds = 0;
  if (dst >= 0 && dst < p.n_seqs)
    for (int i = threadIdx.x; i < p.max_pages; i += kCopyThreads) holds |= p.block_table[(size_t)dst * p.max_pages + i] >= 0;
  holds = __syncthreads_or(holds);
  if (threadIdx.x == 0) p.plan[x] = make_int4(holds, 0, 0, 0);
}
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const __grid_constant__ ForkParams p) {
  __shared__ int list[kMaxSeqs], claim[kMaxSeqs], s_warp[32];
  __shared__ uint32_t held[kPlanEntries / 32];  // pairs whose target's row holds a page
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  for (int i = tid; i < p.n_seqs; i += kPlanThreads) claim[i] = 0x7FFFFFFF;
  if (tid < kPlanEntries / 32) held[tid] = 0;
  __syncthreads();
  if (!p.wide && tid < p.n * p.max_pages) {
    const int x = tid / p.max_pages, row = p.dst[x];
    if (row >= 0 && row < p.n_seqs && p.block_table[(size_t)row * p.max_pages + tid % p.max_pages] >= 0) atomicOr(held + x / 32, 1u << x % 32);
  }
  __syncthreads();
  const int per = (p.n + kPlanThreads - 1) / kPlanThreads;  // pairs per * tid .. of a thread
  int src[kOwnSeqs], dst[kOwnSeqs], len[kOwnSeqs], last[kOwnSeqs], need = 0;
#pragma unroll
  for (int i = 0; i < kOwnSeqs; ++i) {
    const int x = per * tid + i;
    len[i] = -1;
    if (i >= per || x >= p.n) continue;
    src[i] = p.src[x];
    dst[i] = p.dst[x];
    if (src[i] >= 0 && src[i] < p.n_seqs && dst[i] >= 0 && dst[i] < p.n_seqs) {
      len[i] = p.seq_lens[src[i]];
      // the target has to be empty: neither tokens nor pages
      if (len[i] < 0 || len[i] > (long long)p.max_pages * kPageTokens || p.seq_lens[dst[i]] != 0 ||
          (p.wide ? p.plan[x].x != 0 : (held[x / 32] >> x % 32 & 1) != 0))
        len[i] = -1;
      else
        atomicMin(claim + dst[i], x);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOwnSeqs; ++i) {
    const int x = per * tid + i;
    if (i >= per || x >= p.n) continue;
    // (the first of two forks into one row; a source without tokens may be another's target)
    if (len[i] >= 0 && claim[dst[i]] != x) len[i] = -1;
    last[i] = -1;
    if (len[i] >= 0 && len[i] % kPageTokens) {
      last[i] = p.block_table[(size_t)src[i] * p.max_pages + len[i] / kPageTokens];
      if (last[i] < 0 || last[i] >= p.pool.n_pages || last[i] >= p.layers.n_pages) {
        set_status(p.pool.status, MSA_STATUS_BAD_PAGE);
        len[i] = -2;
      }
    }
    if (len[i] == -1) set_status(p.pool.status, MSA_STATUS_BAD_SEQ);
    need += len[i] >= 0 && len[i] % kPageTokens != 0;
  }
  int want;
  int at = block_scan(need, s_warp, want);
  const int have = want > 0 ? find_free(p.pool, want, list, s_warp) : 0;
#pragma unroll
  for (int i = 0; i < kOwnSeqs; ++i) {
    const int x = per * tid + i;
    if (i >= per || x >= p.n) continue;
    int page = -1;
    if (len[i] >= 0 && len[i] % kPageTokens) {
      if (at < have) {
        page = list[at];
        take(p.pool, page);
      } else {
        set_status(p.pool.status, MSA_STATUS_NO_PAGES);
        len[i] = -1;
      }
      ++at;
    }
    p.plan[x] = make_int4(max(len[i], -1), last[i], page, 0);
    if (len[i] > 0) p.seq_lens[dst[i]] = len[i];
  }
}

// The first `tokens` tokens' bytes of part `part` of page `from` to page `to`, whose other bytes
// stay as they are; one CTA, every 16 bytes a load of their own, all of a thread's loads first.
__device__ __forceinline__ void copy_page_part(const LayerPools& l, int layer, int part, int64_t from, int64_t to, int tokens) {
  const int tid = threadIdx.x;
  if (part == kKvHeads) {
    const uint4* a = reinterpret_cast<const uint4*>(l.idx[layer] + from * kIdxPageBytes);
    uint4* b = reinterpret_cast<uint4*>(l.idx[layer] + to * kIdxPageBytes);
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (tid + i * kCopyThreads < 8 * tokens) v[i] = a[tid + i * kCopyThreads];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (tid + i * kCopyThreads < 8 * tokens) b[tid + i * kCopyThreads] = v[i];
    return;
  }
  const uint8_t* a = l.kv[layer] + from * kKvPageBytes + part * kHeadBytes;
  uint8_t* b = l.kv[layer] + to * kKvPageBytes + part * kHeadBytes;
  uint4 v[8], s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = tid + (i & 3) * kCopyThreads;
    if (at < 4 * tokens) v[i] = *reinterpret_cast<const uint4*>(a + (i < 4 ? kOffKc : kOffVc) + 16 * at);
  }
  // scales: thread = (K or V, group, 16 tokens)
  const int first = 16 * (tid & 7), off = (tid < 64 ? kOffKs : kOffVs) + (tid >> 3 & 7) * kPageTokens + first;
  const int live = min(tokens - first, 16);
  if (live > 0) {
    s = *reinterpret_cast<const uint4*>(a + off);
    if (live < 16) {  // bytes of tokens that are not copied
      const uint4 o = *reinterpret_cast<const uint4*>(b + off);
      auto mix = [&](uint32_t x, uint32_t y, int i) {
        const int k = live - 4 * i;
        const uint32_t m = k >= 4 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << 8 * k) - 1;
        return (x & m) | (y & ~m);
      };
      s = make_uint4(mix(s.x, o.x, 0), mix(s.y, o.y, 1), mix(s.z, o.z, 2), mix(s.w, o.w, 3));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = tid + (i & 3) * kCopyThreads;
    if (at < 4 * tokens) *reinterpret_cast<uint4*>(b + (i < 4 ? kOffKc : kOffVc) + 16 * at) = v[i];
  }
  if (live > 0) *reinterpret_cast<uint4*>(b + off) = s;
}

// Grid: (pair, 1 + layer and part); y = 0: the target's row of the table and the counts of the pages it shares.
__global__ void __launch_bounds__(kCopyThreads) fork_copy_kernel(const __grid_constant__ ForkParams p) {
  const int x = blockIdx.x, y = (int)blockIdx.y - 1;
  pdl_wait();
  pdl_trigger();
  const int src = p.src[x], dst = p.dst[x];
  const int4 plan = p.plan[x];
  if (plan.x < 0) return;
  if (y >= 0) {
    if (plan.z >= 0) copy_page_part(p.layers, y / kParts, y % kParts, plan.y, plan.z, plan.x % kPageTokens);
    return;
  }
  const int full = plan.x / kPageTokens;
  const int* from = p.block_table + (size_t)src * p.max_pages;
  int* to = p.block_table + (size_t)dst * p.max_pages;
  for (int i = threadIdx.x; i < p.max_pages; i += kCopyThreads) {
    int page = i == full ? plan.z : -1;
    if (i < full) {
      page = from[i];
      if (page >= 0 && page < p.pool.n_pages) {
        atomicAdd(p.pool.refs + page, 1);
      } else {
        set_status(p.pool.status, MSA_STATUS_BAD_PAGE);
      }
    }
    to[i] = page;
  }
}

// ---- release ------------------------------------------------------------------------
struct ReleaseParams {
  Pool pool;
  int* block_table;
  int max_pages;
  int* seq_lens;
  int n_seqs;
  const int* rows;
};
__global__ void __launch_bounds__(kCopyThreads) release_kernel(const __grid_constant__ ReleaseParams p) {
  pdl_wait();
  pdl_trigger();
  const int b = p.rows[blockIdx.x];
  if (b < 0 || b >= p.n_seqs) {
    if (threadIdx.x == 0) set_status(p.pool.status, MSA_STATUS_BAD_SEQ);
    return;
  }
  int* row = p.block_table + (size_t)b * p.max_pages;
  if (threadIdx.x == 0) p.seq_lens[b] = 0;
  for (int i = threadIdx.x; i < p.max_pages; i += kCopyThreads) {
    if (row[i] < 0) continue;
    const int page = atomicExch(row + i, -1);  // (a row that is listed twice gives each page back once)
    if (page < 0) continue;
    if (page >= p.pool.n_pages) {
      set_status(p.pool.status, MSA_STATUS_BAD_PAGE);
      continue;
    }
    const int before = atomicSub(p.pool.refs + page, 1);
    if (before == 1) atomicOr(p.pool.free_mask + page / 32, 1u << page % 32);
    if (before <= 0) {  // nobody held it
      atomicAdd(p.pool.refs + page, 1);
      set_status(p.pool.status, MSA_STATUS_BAD_PAGE);
    }
  }
}

// ---- page copies --------------------------------------------------------------------
struct CopyParams {
  LayerPools layers;
  const int* src;
  const int* dst;
  const int* tokens;  // or null: whole pages
  int* status;
};
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  pdl_wait();
  pdl_trigger();
  const int from = p.src[blockIdx.x], to = p.dst[blockIdx.x];
  if (from < 0 || to < 0 || from == to) return;
  const int tokens = p.tokens ? p.tokens[blockIdx.x] : kPageTokens;
  if (from >= p.layers.n_pages || to >= p.layers.n_pages) {
    if (threadIdx.x == 0 && blockIdx.y == 0) set_status(p.status, MSA_STATUS_BAD_PAGE);
    return;
  }
  if (tokens <= 0) return;
  copy_page_part(p.layers, blockIdx.y / kParts, blockIdx.y % kParts, from, to, min(tokens, kPageTokens));
}

// ---- accepted drafts ------------------------------------------------------------------
struct CommitParams {
  LayerPools layers;
  const int* block_table;
  int max_pages;
  const int* seq_lens;
  const int* q_start_loc;
  const unsigned long long* accepted;
  int* new_lens;
  int* status;
};
// Grid: (sequence, layer and part).  The k-th accepted draft moves from position ctx + j to ctx + k,
// k <= j: a CTA loads its part of every token that moves (up to 64 x 144 bytes in registers), then
// stores, so that a token whose place another one takes is read before.
__global__ void __launch_bounds__(kCopyThreads) commit_kernel(const __grid_constant__ CommitParams p) {
  __shared__ int s_from[64], s_to[64];  // slots of the tokens that move: page * 128 + offset
  __shared__ int64_t s_page[2][64];
  const int b = blockIdx.x, part = blockIdx.y % kParts, layer = blockIdx.y / kParts, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const SeqInfo s = load_seq(b, p.seq_lens, p.q_start_loc, p.max_pages, 0x7FFFFFFF);
  const bool lead = blockIdx.y == 0;
  if (!s.ok || s.n_q > MSA_TREE_MAX_DRAFTS) {
    if (tid == 0 && lead) {
      set_status(p.status, MSA_STATUS_BAD_SEQ);
      p.new_lens[b] = s.seq_len;
    }
    return;
  }
  const unsigned long long word = s.n_q == 0 ? 0ull : p.accepted[b] & (~0ull >> (64 - s.n_q));
  const int ctx = s.seq_len - s.n_q, kept = __popcll(word);
  if (tid == 0 && lead) p.new_lens[b] = ctx + kept;
  const int still = __ffsll(~word) - 1;  // drafts 0 .. still - 1 stay where they are (-1: all 64)
  const int moves = still < 0 ? 0 : kept - still;
  if (moves == 0) return;
  if (tid < 64 && (word >> tid & 1)) {
    const int k = __popcll(word & ((1ull << tid) - 1));
    if (k < tid) {
      const int* row = p.block_table + (size_t)b * p.max_pages;
      const int i = k - still, from = ctx + tid, to = ctx + k;
      int64_t pf = row[from / kPageTokens], pt = row[to / kPageTokens];
      if (pf < 0 || pt < 0 || pf >= p.layers.n_pages || pt >= p.layers.n_pages) {
        if (lead) set_status(p.status, MSA_STATUS_BAD_PAGE);
        pf = -1;
      }
      s_page[0][i] = pf;
      s_page[1][i] = pt;
      s_from[i] = from % kPageTokens;
      s_to[i] = to % kPageTokens;
    }
  }
  __syncthreads();
  // 16-byte chunks: 8 of a token and part (K's four and V's, or the index key's); thread = chunk tid % 8
  // of tokens tid / 8, + 16, ...
  const int c = tid & 7;
  uint4 v[4];
  uint32_t sc[4] = {0, 0, 0, 0};  // a head's scale bytes of K and V, group c
  if (part == kKvHeads) {
    uint8_t* pool = p.layers.idx[layer];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = (tid >> 3) + 16 * u;
      if (i < moves && s_page[0][i] >= 0)
        v[u] = *reinterpret_cast<const uint4*>(pool + s_page[0][i] * kIdxPageBytes + s_from[i] * kIdxDim + ((c ^ (s_from[i] & 7)) << 4));
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = (tid >> 3) + 16 * u;
      if (i < moves && s_page[0][i] >= 0)
        *reinterpret_cast<uint4*>(pool + s_page[1][i] * kIdxPageBytes + s_to[i] * kIdxDim + ((c ^ (s_to[i] & 7)) << 4)) = v[u];
    }
    return;
  }
  uint8_t* pool = p.layers.kv[layer] + part * kHeadBytes;
  const int half = c < 4 ? kOffKc : kOffVc;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = (tid >> 3) + 16 * u;
    if (i < moves && s_page[0][i] >= 0) {
      const uint8_t* page = pool + s_page[0][i] * kKvPageBytes;
      v[u] = *reinterpret_cast<const uint4*>(page + half + s_from[i] * 64 + (code_chunk_pos(c & 3, s_from[i]) << 4));
      sc[u] = page[kOffKs + c * kPageTokens + s_from[i]] | page[kOffVs + c * kPageTokens + s_from[i]] << 8;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = (tid >> 3) + 16 * u;
    if (i < moves && s_page[0][i] >= 0) {
      uint8_t* page = pool + s_page[1][i] * kKvPageBytes;
      *reinterpret_cast<uint4*>(page + half + s_to[i] * 64 + (code_chunk_pos(c & 3, s_to[i]) << 4)) = v[u];
      page[kOffKs + c * kPageTokens + s_to[i]] = (uint8_t)sc[u];
      page[kOffVs + c * kPageTokens + s_to[i]] = (uint8_t)(sc[u] >> 8);
    }
  }
}

LayerPools layer_pools(const msa_cache* layers, int n_layers) {
  LayerPools l{};
  l.n_layers = n_layers;
  for (int i = 0; i < n_layers; ++i) {
    l.kv[i] = static_cast<uint8_t*>(layers[i].kv_pool);
    l.idx[i] = static_cast<uint8_t*>(layers[i].idx_pool);
    if (i == 0 || layers[i].n_pages < l.n_pages) l.n_pages = layers[i].n_pages;
  }
  return l;
}
Pool pool_of(const msa_page_pool* p) { return Pool{p->refs, p->free_mask, p->n_pages, p->status}; }

}  // namespace

int max_extend_tokens() { return kMaxExtendTokens; }
size_t fork_workspace_bytes(int n) { return (size_t)n * sizeof(int4); }

cudaError_t launch_extend(const msa_page_pool* pool, int* block_table, int max_pages, int* seq_lens,
                          const int* q_start_loc, int n_seqs, int n_tokens, int64_t* slots, cudaStream_t stream) {
  if (n_seqs == 0 || n_tokens == 0) return cudaSuccess;
  static DeviceSetup setup;
  int dev = 0, n_sm = 0;
  const cudaError_t e = setup.get(&dev, &n_sm, [](int) {
    return cudaFuncSetAttribute(extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kExtendSmem);
  });
  if (e != cudaSuccess) return e;
  const ExtendParams p{pool_of(pool), block_table, max_pages, seq_lens, q_start_loc, n_seqs, n_tokens, slots, n_tokens > kPlanTokens};
  if (const cudaError_t r = launch_pdl(extend_kernel, dim3(1), dim3(kPlanThreads), kExtendSmem, stream, p); r != cudaSuccess || !p.wide) return r;
  return launch_pdl(slots_kernel, dim3((n_tokens + kCopyThreads - 1) / kCopyThreads), dim3(kCopyThreads), 0, stream, p);
}

cudaError_t launch_fork(const msa_cache* layers, int n_layers, const msa_page_pool* pool, int* block_table,
                        int max_pages, int* seq_lens, int n_seqs, const int* src, const int* dst, int n, void* ws,
                        cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  const ForkParams p{pool_of(pool), block_table, max_pages, seq_lens, n_seqs, src, dst, n, static_cast<int4*>(ws),
                     (long long)n * max_pages > kPlanEntries, layer_pools(layers, n_layers)};
  if (p.wide)
    if (const cudaError_t e = launch_pdl(fork_rows_kernel, dim3(n), dim3(kCopyThreads), 0, stream, p); e != cudaSuccess) return e;
  const cudaError_t e = launch_pdl(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(fork_copy_kernel, dim3(n, 1 + n_layers * kParts), dim3(kCopyThreads), 0, stream, p);
}

cudaError_t launch_release(const msa_page_pool* pool, int* block_table, int max_pages, int* seq_lens, int n_seqs,
                           const int* rows, int n, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  const ReleaseParams p{pool_of(pool), block_table, max_pages, seq_lens, n_seqs, rows};
  return launch_pdl(release_kernel, dim3(n), dim3(kCopyThreads), 0, stream, p);
}

cudaError_t launch_copy_pages(const msa_cache* layers, int n_layers, const int* src, const int* dst, const int* tokens,
                              int n, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  const CopyParams p{layer_pools(layers, n_layers), src, dst, tokens, layers[0].status};
  return launch_pdl(copy_pages_kernel, dim3(n, n_layers * kParts), dim3(kCopyThreads), 0, stream, p);
}

cudaError_t launch_commit(const msa_cache* layers, int n_layers, const int* block_table, int max_pages,
                          const int* seq_lens, const int* q_start_loc, int n_seqs, const uint64_t* accepted,
                          int* new_lens, cudaStream_t stream) {
  if (n_seqs == 0) return cudaSuccess;
  const CommitParams p{layer_pools(layers, n_layers), block_table, max_pages, seq_lens, q_start_loc,
                       reinterpret_cast<const unsigned long long*>(accepted), new_lens, layers[0].status};
  return launch_pdl(commit_kernel, dim3(n_seqs, n_layers * kParts), dim3(kCopyThreads), 0, stream, p);
}

}  // namespace msa
