// Attention of drafted tokens over a paged NVFP4 cache: every draft sees its
// sequence's committed context (all of it, or one block selection shared by the
// sequence's drafts) and the drafts that its mask names (its ancestors in a tree
// of drafts and itself).
//
// Mathematics.  For a row (draft, query head) with FP8 query q and keys k8_t, the
// NVFP4 operands dequantised to FP8 as in the sparse decode path,
//   x_t = (q . k8_t) scale / s_enc_k log2(e),  out = sum_t 2^x_t v8_t / sum_t 2^x_t / s_enc_v
// over the visible t, in one pass with a reference m per row that follows the
// running maximum: weights 2^(x_t - m + 8) are summed in fp32 (l) and multiply V
// in f16.  m moves only when 32 weights sum to more than 49,152, so that they stay
// below f16's end and the accumulator is rescaled a few times per row;
// they keep full f16 precision down to 2^-22 of the reference's (an E4M3 weight, with
// its 17 binades, would lose the bulk of a long context behind one large key).  A move
// multiplies by less than 1/6 (its largest weight was above 1,536 = 6 2^8): l and the
// accumulator in fp32, the weights of the page's earlier chunks with a second rounding to f16.
// V8 is an f16 value by moving its seven magnitude bits: E4M3 bits << 7 is
// v8 2^-8 exactly, subnormals included.
//
// One persistent CTA per SM; rows of one (sequence, KV head) are row 4 i + h of
// one tile of 128 (up to 32 drafts) or two, so K and V are converted once for all
// drafts.  The (sequence, KV head, page) units are cut into equal weighted ranges,
// one per CTA; a (sequence, KV head) cut across CTAs leaves fp32 partial rows in
// the workspace, merged by a second kernel.  Roles, all hand-offs mbarriers with
// bounded waits:
//   warp 0        segment records and one 18,432-byte bulk copy per page;
//   warp 1        MMA issuer: S = Q K8^T (kind::f8f6f4, 128 x 128 x 128), then
//                 O += P V (kind::f16, P from tensor memory over S's own columns,
//                 V MN-major), the set's next QK behind it;
//   warp 2        query rows of the next segment (cp.async);
//   warps 4-11    two softmax sets, thread = row: with one row tile a set takes
//                 every other page (its own reference, sum and accumulator, joined
//                 at the segment's end), with two tiles a set takes a tile;
//   warps 12-23   K conversion (four warps, thread = token) and V conversion (eight,
//                 thread = token and half of the channels).
//
// What bounds it.  A page of 18,432 bytes takes a CTA 0.76 us with up to 8 drafts, 0.91 us up
// to 16, 0.98 us up to 32 and 1.74 us with two tiles; its products take the tensor pipe 0.39 us
// per tile.  The rest is instruction issue and hand-offs: 1,958 warp instructions of
// conversion a page (K 763, V 1,195), 911 (one draft) to 2,550 (32) of softmax, about 1,100
// of waits.  32 sequences of 32,768 tokens, one draft each: 183 us, 3.3 TB/s; 8 of 131,072
// with 64 drafts: 385 us, 1.35 PFLOP/s; one of 4,096: 14.8 us, a chain of latencies
// (lengths and ranges 2.6, first page 2.4, its scores 1.4, joining the row copies 1.7, the
// merge kernel 4).
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "attn_ops.cuh"

namespace msa {
namespace {

constexpr int kTreeThreads = 768;
constexpr int kTreeMaxDrafts = 64;  // per sequence: one 64-bit mask word, two row tiles
constexpr int kTreeCtas = 152;      // most CTAs of a launch (the workspace is sized for them)
constexpr int kRaw = 4;             // raw page stages
constexpr int kSlot = 2;            // converted pages in flight (page e in slot e & 1)
constexpr int kRecs = 4;
constexpr int kInfo = 16;
constexpr int kKTabCopies = 4, kVTabCopies = 8;

constexpr int kOffQ = 0;                                      // 2 tiles [128 rows][128 B]
constexpr int kOffK8 = kOffQ + 2 * 16384;                     // kSlot x [8 groups of 16 channels][128 tokens][16 B]
constexpr int kOffV16 = kOffK8 + kSlot * 16384;               // kSlot x [16 groups of 8 channels][128 tokens][16 B]
constexpr int kOffRaw = kOffV16 + kSlot * 32768;              // kRaw x 18,432
constexpr int kOffKTab = kOffRaw + kRaw * kHeadBytes;         // uint2 [128][copies]
constexpr int kOffVTab = kOffKTab + 128 * 8 * kKTabCopies;    // uint4 [128][copies]
constexpr int kOffMl = kOffVTab + 128 * 16 * kVTabCopies;     // float2 [2 parities][2 sets][128]
constexpr int kOffRecs = kOffMl + 2 * 2 * 128 * 8;            // kRecs x 64 B
constexpr int kOffInfo = kOffRecs + kRecs * 64;               // int2 [kInfo]: first position, valid tokens
constexpr int kOffRow = kOffInfo + kInfo * 8;                 // float2 [2 sets][64]: a row's reference and sum
constexpr int kOffScan = kOffRow + 2 * 64 * 8;                // long long [32] and the start
constexpr int kOffTreeBars = kOffScan + 32 * 8 + 64;
constexpr int kBRawFull = 0, kBRawEmpty = kBRawFull + kRaw, kBKFull = kBRawEmpty + kRaw, kBKEmpty = kBKFull + kSlot,
              kBVEmpty = kBKEmpty + kSlot, kBSFull = kBVEmpty + kSlot, kBPFull = kBSFull + 2,  // P: [set][slot]
              kBPvDone = kBPFull + 2 * kSlot, kBOFree = kBPvDone + 2, kBMl = kBOFree + 1, kBQFull = kBMl + 1,
              kBQEmpty = kBQFull + 1, kBRecFull = kBQEmpty + 1, kBRecEmpty = kBRecFull + kRecs,
              kBDone = kBRecEmpty + kRecs, kTreeBars = kBDone + 1;
constexpr int kOffTreeMisc = kOffTreeBars + 8 * ((kTreeBars + 1) & ~1);  // tmem, abort, copies issued
constexpr int kTreeSmem = 1024 + kOffTreeMisc + 16;
static_assert(kTreeSmem <= 232448, "shared memory of one CTA");
static_assert(kOffRaw % 16 == 0 && kOffVTab % 16 == 0 && kOffTreeBars % 8 == 0, "alignment");
constexpr uint32_t kTmemS = 0, kTmemO = 256;  // S of set s at 128 s, O of set s at 256 + 128 s
constexpr float kTreeBias = 8.0f;
constexpr float kTreeMost = 49152.0f;  // largest sum of a chunk's weights, and so largest weight (f16 ends at 65,504)
constexpr float kTreeUnset = 3e38f;    // shift of a row without a reference: a visible token's weight is infinite
constexpr float kTreeLog2e = 1.4426950408889634f, kTreeLn2 = 0.6931471805599453f;

// Weights of the partition, in units of about 0.19 us: a page of a sequence with up to 8, 16,
// 32 and 64 drafts (0.76, 0.91, 1.02 and 1.82 us per page of a CTA, from 24 sequences of 16,384
// and of 49,152 tokens; in the kernel without row copies 0.98 and 1.74 us up to 32 and 64),
// and the fixed part of a (sequence, KV head).
// The least share of a CTA is a page's weight, so that every CTA between a sequence's
// first and last has pages of it.
template <bool kCopies>
__device__ __forceinline__ int tree_page_weight(int n_q) {
  if (!kCopies) return n_q <= 32 ? 5 : 9;
  return n_q <= 8 ? 4 : n_q <= 16 ? 5 : n_q <= 32 ? 6 : 10;
}
constexpr int kFixedWeight = 10, kLeastShare1 = 6, kLeastShare2 = 10;

// Copies of the query rows in a one-tile segment's 128 rows: with few rows every
// warp quad (32 lanes of tensor memory) gets the same rows and its own share of a
// page's tokens, so that no softmax warp is idle (32 sequences of 32,768 tokens, one draft
// each: 184 us, with two copies 211, with one 224).
__host__ __device__ __forceinline__ int tree_copies(int n_q) { return n_q <= 8 ? 4 : n_q <= 16 ? 2 : 1; }

struct SegRec {
  int n_pg;      // pages of the segment; -1: no more segments
  int g, q0, n_q;
  int ctx;       // tokens before the drafts
  int slot;      // partial slot, or -1: the segment is the whole (sequence, KV head)
};
static_assert(sizeof(SegRec) <= 64, "record slot");

struct TreeParams {
  const uint8_t* kv_pool;
  int64_t n_pages;
  const uint8_t* q;  // [T][16][128]
  const int* block_table;
  int max_pages;
  const int* seq_lens;
  const int* q_start_loc;
  int n_seqs;
  int n_q_total;
  const unsigned long long* tree_mask;  // [T] or null (draft j sees drafts 0 .. j)
  const int* sel;                       // [n_seqs][17] or null (all blocks)
  const int* n_sel;
  float scale_log2;
  float out_scale;  // 2^8 / s_enc_v
  int out_f16;
  uint16_t* out;    // [T][16][128] bf16 or f16
  float* lse;       // [T][16] or null
  int* row_desc;    // [T][4] workspace: first CTA | parts << 8 | draft << 20, 0 = nothing to merge
  float* part_o;    // [2 kTreeCtas][rows][128]
  float2* part_ml;  // [2 kTreeCtas][rows]
  int part_rows;
  int* status;
  unsigned long long wait_ns;
  int inject;  // test only: a CTA's first page is not copied, so that the waits for it run out
};

// Blocks a sequence's drafts visit: `chosen` of the selection, then those that can
// hold drafts; and the units' weight.
struct SeqWork {
  SeqInfo s;
  int ctx, first, chosen, n_vis, pw;
};
template <bool kCopies>
__device__ __forceinline__ SeqWork seq_work(const TreeParams& p, int b) {
  SeqWork w;
  // (all loads at once: a sequence's start is a chain of them)
  int id[kSelStride], n = 0;
  if (p.sel) {
    n = p.n_sel[b];
#pragma unroll
    for (int i = 0; i < kSelStride; ++i) id[i] = p.sel[(size_t)b * kSelStride + i];
  }
  w.s = load_seq(b, p.seq_lens, p.q_start_loc, p.max_pages, p.n_q_total);
  if (w.s.n_q > kTreeMaxDrafts) w.s.ok = false;
  w.ctx = w.s.seq_len - w.s.n_q;
  w.first = w.ctx / kPageTokens;
  w.chosen = w.first;
  w.n_vis = 0;
  w.pw = tree_page_weight<kCopies>(w.s.n_q);
  if (!w.s.ok || w.s.n_q == 0) return w;
  if (p.sel) {
    int top = -1;
    w.chosen = 0;
#pragma unroll
    for (int i = 0; i < kSelStride; ++i)
      if (i < n) {
        w.chosen += id[i] > top && id[i] < w.first;
        top = max(top, id[i]);
      }
  }
  w.n_vis = w.chosen + (w.s.seq_len - 1) / kPageTokens - w.first + 1;
  return w;
}

static_assert(sizeof(SeqWork) <= 64, "beside the scan");
// Start of CTA c's range of total = G quota + extra units.
__device__ __forceinline__ long long range_start(long long quota, int extra, int c) { return c * quota + min(c, extra); }

// The 32 drafts' bits of the positions pos .. pos + 31 for a row with mask word tm
// (bits of drafts that exist only): context tokens are visible.
__device__ __forceinline__ uint32_t visible_bits(unsigned long long tm, int pos, int ctx) {
  const int sh = pos - ctx;
  if (sh >= 64) return 0u;
  if (sh >= 0) return (uint32_t)(tm >> sh);
  if (sh <= -32) return 0xFFFFFFFFu;
  return ((uint32_t)tm << -sh) | ((1u << -sh) - 1u);
}

// kCopies false: one copy of the rows whatever their number.
template <bool kCopies>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_attn_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ uint8_t smem_raw[];
  // (pointer arithmetic, no integer cast: the accesses stay shared-memory instructions)
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + kOffTreeBars + 8 * i; };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffTreeMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffTreeMisc + 4);
  int* s_issued = reinterpret_cast<int*>(smem + kOffTreeMisc + 8);
  const WaitCtl wc{s_abort, p.wait_ns};
  auto rec = [&](int k) { return reinterpret_cast<SegRec*>(smem + kOffRecs + 64 * (k % kRecs)); };
  int2* s_info = reinterpret_cast<int2*>(smem + kOffInfo);
  long long* s_scan = reinterpret_cast<long long*>(smem + kOffScan);  // [24] warp sums, then total, start b, its offset
  SeqWork* s_first = reinterpret_cast<SeqWork*>(smem + kOffScan + 32 * 8);  // the first sequence of the range
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- prologue ------------------------------------------------------------------
  {
    uint2* kt = reinterpret_cast<uint2*>(smem + kOffKTab);
    uint4* vt = reinterpret_cast<uint4*>(smem + kOffVTab);
    if (tid < 128) convert_tables<kKTabCopies, kVTabCopies>(tid, kt, vt);
  }
  if (tid == 0) {
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(bar(kBRawFull + i), 1);
      mbar_init(bar(kBRawEmpty + i), 12);
    }
    for (int i = 0; i < kSlot; ++i) {
      mbar_init(bar(kBKFull + i), 4);
      mbar_init(bar(kBKEmpty + i), 1);
      mbar_init(bar(kBVEmpty + i), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kBSFull + s), 1);
      mbar_init(bar(kBPFull + 2 * s), 4 + 8);  // the set's softmax warps and the V conversion
      mbar_init(bar(kBPFull + 2 * s + 1), 4 + 8);
      mbar_init(bar(kBPvDone + s), 1);
    }
    mbar_init(bar(kBOFree), 8);
    mbar_init(bar(kBMl), 8);
    mbar_init(bar(kBQFull), 1);
    mbar_init(bar(kBQEmpty), 1);
    for (int i = 0; i < kRecs; ++i) {
      mbar_init(bar(kBRecFull + i), 1);
      mbar_init(bar(kBRecEmpty + i), 1 + 1 + 8 + 4 + 8);  // MMA, queries, softmax, K and V conversion
    }
    mbar_init(bar(kBDone), 1);
    *s_abort = 0;
    *s_issued = 0;
    fence_barrier_init();
  }
  if (warp == 3) tmem_alloc(smem_u32(s_tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_wait();  // everything below may come from the previous kernel
  pdl_trigger();

  // ---- this CTA's range of the weighted units ------------------------------------------
  // thread i sums the sequences i * per .. of its share, then a scan over the CTA
  const int per = (p.n_seqs + kTreeThreads - 1) / kTreeThreads;
  bool wide = false;  // some sequence has two row tiles
  {
    long long mine = 0;
    SeqWork last{};
    const int b0 = min(tid * per, p.n_seqs), b1 = min(b0 + per, p.n_seqs);
    for (int b = b0; b < b1; ++b) {
      const SeqWork w = seq_work<kCopies>(p, b);
      last = w;
      if (!w.s.ok && blockIdx.x == 0) set_status(p.status, MSA_STATUS_BAD_SEQ);
      if (w.n_vis > 0) mine += (long long)kKvHeads * (w.pw * w.n_vis + kFixedWeight);
      wide |= w.n_vis > 0 && w.s.n_q > 32;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    wide = __syncthreads_or(wide);
    long long before = 0, total = 0;
    for (int i = 0; i < kTreeThreads / 32; ++i) {
      if (i < warp) before += s_scan[i];
      total += s_scan[i];
    }
    const int G = (int)min((long long)gridDim.x, max(1ll, total / (wide ? kLeastShare2 : kLeastShare1)));
    const long long lo = (int)blockIdx.x < G ? range_start(total / G, (int)(total % G), blockIdx.x) : total;
    const long long mine0 = before + incl - mine;
    if (mine > 0 && lo >= mine0 && lo < mine0 + mine) {  // the first sequence of the range is in this share
      s_scan[25] = b0;
      s_scan[26] = mine0;
      *s_first = last;  // (of use if the share is this sequence alone)
    }
    if (tid == 0) s_scan[24] = total;
    __syncthreads();
  }
  const long long total = s_scan[24];
  const int G = (int)min((long long)gridDim.x, max(1ll, total / (wide ? kLeastShare2 : kLeastShare1)));
  const bool idle = (int)blockIdx.x >= G || total == 0;

  // registers: 128 threads x 80 (as launched) + 256 x 112 + 384 x 56 of the launch's 768 x 80
  // (64, 120 and 56 cost the issuer and the page walk spills: 2 % on every case)
  if (warp < 4) {
    if (warp == 0) {
      // ---------------- segment records and page copies -------------------------------------
      int e = 0, k = 0;
      bool ok = true;
      if (!idle) {
        const long long quota = total / G;
        const int extra = (int)(total - quota * G);
        const long long lo = range_start(quota, extra, blockIdx.x), hi = range_start(quota, extra, blockIdx.x + 1);
        long long off = s_scan[26];
        for (int b = (int)s_scan[25]; ok && b < p.n_seqs && off < hi; ++b) {
          const SeqWork w = per == 1 && b == (int)s_scan[25] ? *s_first : seq_work<kCopies>(p, b);
          if (w.n_vis == 0) continue;
          const long long wg = (long long)w.pw * w.n_vis + kFixedWeight;
          // the selection, one entry per lane: its place among the chosen ones
          int my_blk = -1;
          if (p.sel && off + kKvHeads * wg > lo) {
            const int n = min(max(p.n_sel[b], 0), kSelStride);
            const int id = lane < n ? p.sel[(size_t)b * kSelStride + lane] : -1;
            int top = id;  // the largest entry so far, this one included
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int v = __shfl_up_sync(0xffffffffu, top, o);
              if (lane >= o) top = max(top, v);
            }
            const int prev = __shfl_up_sync(0xffffffffu, top, 1);
            const bool up = lane < n && id > (lane ? max(prev, -1) : -1);
            if (lane < n && (!up || id > (w.s.seq_len - 1) / kPageTokens)) set_status(p.status, MSA_STATUS_BAD_SELECTION);
            const unsigned chosen = __ballot_sync(0xffffffffu, up && id < w.first);
            // lane i takes the i-th chosen entry
            int src = 0;
            for (int i = 0, c = 0; i < kSelStride; ++i)
              if (chosen >> i & 1) {
                if (c == lane) src = i;
                ++c;
              }
            my_blk = __shfl_sync(0xffffffffu, id, src);
          }
          for (int g = 0; ok && g < kKvHeads; ++g, off += wg) {
            // page i starts at weight off + kFixedWeight + i pw; it belongs to the range that holds its start
            const long long base = off + kFixedWeight;
            auto page_at = [&](long long x) {  // the first page that starts at weight x or behind it
              if (x <= base) return 0;
              return x - base > (long long)w.n_vis * w.pw ? w.n_vis : ((int)(x - base) + w.pw - 1) / w.pw;
            };
            const int a = page_at(lo), z = page_at(hi);
            if (a >= z) continue;
            if (!twait(bar(kBRecEmpty + k % kRecs), ((k / kRecs) & 1) ^ 1, wc)) {
              ok = false;
              break;
            }
            const bool whole = a == 0 && z == w.n_vis;
            if (lane == 0) {
              SegRec* r = rec(k);
              r->n_pg = z - a;
              r->g = g;
              r->q0 = w.s.q0;
              r->n_q = w.s.n_q;
              r->ctx = w.ctx;
              r->slot = whole ? -1 : 2 * (int)blockIdx.x + (a > 0 ? 0 : 1);
            }
            if (!whole && a == 0) {
              // the first part tells the merge who has the others
              const long long last = base + (long long)(w.n_vis - 1) * w.pw;
              const long long big = extra * (quota + 1);  // the first `extra` CTAs have one unit more
              const int c_last = last < big ? (int)(last / (quota + 1)) : extra + (int)((last - big) / quota);
              const int parts = c_last - (int)blockIdx.x + 1;
              for (int i = lane; i < w.s.n_q; i += 32)
                p.row_desc[(size_t)(w.s.q0 + i) * kKvHeads + g] = (int)blockIdx.x | parts << 8 | i << 20;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBRecFull + k % kRecs));
            ++k;
            const uint8_t* head = p.kv_pool + (size_t)g * kHeadBytes;
            for (int i0 = a; ok && i0 < z; i0 += 32) {
              const int i = i0 + lane, cnt = min(32, z - i0);
              int blk = i;
              if (p.sel) {
                const int from = __shfl_sync(0xffffffffu, my_blk, i & 31);
                blk = i < w.chosen ? from : w.first + i - w.chosen;
              }
              int phys = -1;
              if (lane < cnt) {
                phys = p.block_table[(size_t)b * p.max_pages + blk];
                if (phys < 0 || phys >= p.n_pages) {
                  set_status(p.status, MSA_STATUS_BAD_PAGE);
                  phys = -1;
                }
              }
              for (int j = 0; j < cnt; ++j, ++e) {
                const int ph = __shfl_sync(0xffffffffu, phys, j), bl = __shfl_sync(0xffffffffu, blk, j);
                const int st = e % kRaw;
                if (!twait(bar(kBRawEmpty + st), ((e / kRaw) & 1) ^ 1, wc)) {
                  ok = false;
                  break;
                }
                if (lane == 0) {
                  const int pos = bl * kPageTokens;
                  s_info[e % kInfo] = make_int2(pos, ph < 0 ? 0 : min(kPageTokens, w.s.seq_len - pos));
                  if (p.inject && e == 0) {
                  } else if (ph < 0) {
                    mbar_arrive(bar(kBRawFull + st));  // nothing to copy: no token of the page is valid
                  } else {
                    mbar_arrive_expect_tx(bar(kBRawFull + st), kHeadBytes);
                    bulk_g2s(sbase + kOffRaw + st * kHeadBytes, head + (size_t)ph * kKvPageBytes, kHeadBytes,
                             bar(kBRawFull + st));
                  }
                  *s_issued = e + 1;
                }
                __syncwarp();
              }
            }
          }
        }
      }
      // no more segments
      if (ok && twait(bar(kBRecEmpty + k % kRecs), ((k / kRecs) & 1) ^ 1, wc) && lane == 0) {
        rec(k)->n_pg = -1;
        mbar_arrive(bar(kBRecFull + k % kRecs));
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer ---------------------------------------------------------------------
      // Job j of a segment belongs to set j & 1: page j with one row tile, tile j & 1 of page j / 2
      // with two.  In turn: PV(j), then QK(j + 2) into the same columns.  The two sets' jobs
      // alternate on one issuer, so that one set's products run under the other's softmax (an
      // issuer per set lets two tiles fall into step: 603 against 482 us on 8 x 128K x 64 drafts).
      // The warp stays together and elects a lane for the MMAs only: in a loop that one lane runs
      // alone nothing is warp-uniform, and an MMA then takes three times as long to issue.
      const uint32_t idesc_qk = umma_idesc_e4m3(128, 128);
      // D fp32, A and B f16, A K-major, B MN-major
      const uint32_t idesc_pv = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
      int e0 = 0;
      uint32_t phases = 0;  // of the four P barriers
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!twait(bar(kBRecFull + k % kRecs), (k / kRecs) & 1, wc)) break;
        const int n_pg = __shfl_sync(0xffffffffu, rec(k)->n_pg, 0);
        if (n_pg < 0) break;
        const bool two = __shfl_sync(0xffffffffu, rec(k)->n_q, 0) > 32;
        if (lane == 0) mbar_arrive(bar(kBRecEmpty + k % kRecs));
        const int n_jobs = two ? 2 * n_pg : n_pg;
        if (!twait(bar(kBQFull), k & 1, wc)) break;
        auto k_ready = [&](int e) { return twait(bar(kBKFull + (e & 1)), (e >> 1) & 1, wc); };
        // QK of page e for a set (inside an elected lane); free_k: the last reader of the K tile.
        // (The loops stay short: straight-line MMAs are long, and a long way round the warp's
        // code misses the instruction cache.)
        auto issue_qk = [&](int set, int e, bool free_k, bool free_q) {
          const uint64_t qdesc = umma_desc_sw128(sbase + kOffQ + (two ? set : 0) * 16384);
          // K-major without swizzle: 8 tokens x 16 channels are 128 contiguous bytes, the next 16
          // channels 2,048 further (so that a converting thread's stores are at fixed offsets)
          const uint64_t kdesc = umma_desc_noswz_lbo_sbo(sbase + kOffK8 + (e & 1) * 16384, 2048, 128);
#pragma unroll 2
          for (int kk = 0; kk < 4; ++kk)  // 32 channels each
            umma_e4m3(tmem + kTmemS + 128 * set, qdesc + 2 * kk, kdesc + kk * (4096 >> 4), idesc_qk, kk > 0);
          umma_commit(bar(kBSFull + set));
          if (free_k) umma_commit(bar(kBKEmpty + (e & 1)));
          if (free_q) umma_commit(bar(kBQEmpty));
        };
        // first QKs of both sets, then job after job
        for (int j = -2; ok && j < n_jobs; ++j) {
          const int set = j & 1;
          const int e = e0 + (two ? j >> 1 : j), en = e + (two ? 1 : 2);
          const bool next = j + 2 < n_jobs;
          if (next && !(two && set) && !k_ready(en)) {
            ok = false;
            break;
          }
          if (j == 0 && k > 0 && !twait(bar(kBOFree), (k - 1) & 1, wc)) {  // both accumulators are read
            ok = false;
            break;
          }
          const int pb = kSlot * set + (e & 1);
          if (j >= 0) {
            if (!twait(bar(kBPFull + pb), phases >> pb & 1, wc)) {
              ok = false;
              break;
            }
            phases ^= 1u << pb;
          }
          tc_fence_after();
          // MN-major without swizzle: 8 tokens x 8 channels are 128 contiguous bytes, the next 8 tokens
          // follow, the next 8 channels are 2,048 further
          const uint64_t vdesc = umma_desc_noswz_lbo_sbo(sbase + kOffV16 + (e & 1) * 32768, 128, 2048);
          if (elect_one()) {
            if (j >= 0) {
#pragma unroll 4
              for (int kk = 0; kk < 8; ++kk)  // 16 tokens each: 8 columns of P inside S's 32-column chunks
                umma_f16_ts(tmem + kTmemO + 128 * set, tmem + kTmemS + 128 * set + 32 * (kk >> 1) + 8 * (kk & 1),
                            vdesc + kk * (256 >> 4), idesc_pv, (j >= 2 || kk > 0) ? 1u : 0u);
              if (!(two && set == 0)) umma_commit(bar(kBVEmpty + (e & 1)));
            }
            if (next) issue_qk(set, en, !(two && set == 0), j + 3 == n_jobs);
            else if (j >= 0) umma_commit(bar(kBPvDone + set));  // the set's accumulator is final
            // (a set without a job: behind the wait for the last segment's readers, who would miss a phase)
            if (n_jobs == 1 && j == 0) umma_commit(bar(kBPvDone + 1));
          }
          __syncwarp();
        }
        e0 += n_pg;
      }
      __syncwarp();
      if (elect_one()) umma_commit(bar(kBDone));
      __syncwarp();
    } else if (warp == 2) {
      // ---------------- query rows of a segment: row 4 i + h of draft i, head 4 g + h -----------------
      for (int k = 0;; ++k) {
        if (!twait(bar(kBRecFull + k % kRecs), (k / kRecs) & 1, wc)) break;
        const SegRec r = *rec(k);
        __syncwarp();
        if (r.n_pg < 0) break;
        if (lane == 0) mbar_arrive(bar(kBRecEmpty + k % kRecs));
        if (k > 0 && !twait(bar(kBQEmpty), (k - 1) & 1, wc)) break;
        // the second tile is also the exchange buffer of a segment with row copies (all segments or
        // none wait: a parity does not tell phase k - 1 from k - 3, so every phase is seen in turn)
        if (wide && k > 0 && !twait(bar(kBOFree), (k - 1) & 1, wc)) break;
        const int copies = kCopies ? tree_copies(r.n_q) : 1, gap = 128 / copies;
        for (int x = lane; x < r.n_q * 32; x += 32) {
          const int row = x >> 3, c = x & 7;
          const uint8_t* src = p.q + ((size_t)(r.q0 + (row >> 2)) * kQHeads + kGqa * r.g + (row & 3)) * kHeadDim + 16 * c;
          for (int i = 0; i < copies; ++i)
            cp_async16(sbase + kOffQ + (row + i * gap) * 128 + ((c ^ (row & 7)) << 4), src);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBQFull));
      }
    }
  } else if (warp < 12) {
    regs_inc<112>();
    // ---------------- softmax: set = (warp - 4) / 4, row = TMEM lane ------------------------------------
    const int set = (warp - 4) >> 2, quad = warp & 3, lrow = 32 * quad + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t t_s = tl + kTmemS + 128 * set;
    const uint64_t scale2 = pair64(__float_as_uint(p.scale_log2), __float_as_uint(p.scale_log2));
    int e0 = 0, jobs = 0;  // pages so far, jobs of this set so far
    bool ok = true;
    // One segment; false: the set leaves.  A copy of the code per mode (0: one row tile with row
    // copies, 1: one tile, 2: two tiles): with the counts known the page loop is shorter and needs
    // fewer registers (8 sequences of 131,072 with 64 drafts: 414 us, 444 with one code for all).
    auto segment = [&](const SegRec& r, int k, auto mode) -> bool {
      constexpr int kMode = decltype(mode)::value, two = kMode == 2;
      const int n_jobs = r.n_pg << two;
      const int n_rows = kGqa * r.n_q;
      const int copies = kMode == 0 ? tree_copies(r.n_q) : 1, gap = 128 / copies;
      const int row = two ? 128 * set + lrow : lrow & (gap - 1);
      const int copy = lrow / gap;
      const bool busy = row - lane < n_rows;  // some lane of the warp has a row
      const bool mine = row < n_rows;
      const int draft = row >> 2;
      // this warp's token chunks of a page: 32-column chunks c0 .. c1 - 1
      const int c0 = copy * 4 / copies, c1 = c0 + 4 / copies;
      unsigned long long tm = 0;
      if (mine) {
        tm = p.tree_mask ? p.tree_mask[r.q0 + draft] : (2ull << draft) - 1;
        if (r.n_q < 64) tm &= (1ull << r.n_q) - 1;
      }
      float shift = kTreeUnset, l = 0.f;  // kTreeBias less the reference, and the sum of weights
      // Multiplies what the row has so far by f: the earlier pages' sums (the PVs before this S
      // are done) and this page's weights of the chunks before c.
      auto rescale = [&](int c, bool sums, float f) {
        if (sums)
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            uint32_t u[32];
            const uint32_t t_o = tl + kTmemO + 128 * set + 32 * i;
            tmem_ld32x32b_x32(t_o, u);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) u[x] = __float_as_uint(__uint_as_float(u[x]) * f);
            tmem_st32(t_o, u);
          }
        tmem_wait_st();
#pragma unroll 1
        for (int i = c0; i < c; ++i) {
          uint32_t u[16];
          tmem_ld32x32b_x16(t_s + 32 * i, u);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&u[x]));
            u[x] = cvt_f16x2_f32(w.y * f, w.x * f);
          }
          tmem_st_x16(t_s + 32 * i, u);
        }
      };
      for (int j = set; j < n_jobs; j += 2) {
        if (!twait(bar(kBSFull + set), jobs & 1, wc)) {
          ok = false;
          break;
        }
        ++jobs;
        if (busy) {
          const int2 info = s_info[(e0 + (j >> two)) % kInfo];
          const bool edge = info.y < kPageTokens || info.x + kPageTokens > r.ctx;  // warp-uniform
          tc_fence_after();
          // One chunk of 32 tokens at a time, in a loop that stays rolled (as the issuer's): weights
          // relative to the row's reference as f16 pairs over the first half of the chunk's own
          // columns.  There is no pass for the maximum: a chunk whose weights sum to kTreeMost
          // or less has no weight above it, and any other (a row's first one: its shift is
          // kTreeUnset) moves the reference to its maximum and is weighed again.
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            uint32_t v[32], o[16];
            tmem_ld32x32b_x32(t_s + 32 * c, v);
            tmem_wait_ld();
            if (edge) {  // -inf where the row does not see the token
              const uint32_t vis = info.y > 0 ? visible_bits(tm, info.x + 32 * c, r.ctx) : 0u;
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = vis >> i & 1 ? v[i] : 0xFF800000u;
            }
            float sh = shift;
            for (;;) {
              const uint64_t shift2 = pair64(__float_as_uint(sh), __float_as_uint(sh));
              uint64_t sums[2] = {0, 0};
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint2 x = split64(fma_f32x2(pair64(v[2 * i], v[2 * i + 1]), scale2, shift2));
                const float a = fast_exp2(__uint_as_float(x.x)), b = fast_exp2(__uint_as_float(x.y));
                sums[i & 1] = add_f32x2(sums[i & 1], pair64(__float_as_uint(a), __float_as_uint(b)));
                o[i] = cvt_f16x2_f32(b, a);
              }
              const uint2 sum2 = split64(add_f32x2(sums[0], sums[1]));
              const float sum = __uint_as_float(sum2.x) + __uint_as_float(sum2.y);
              const bool over = mine && sum > kTreeMost;
              if (!__any_sync(0xffffffffu, over)) {
                l += sum;
                break;
              }
              float f = 1.f;
              if (over) {
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 32; ++i) top = fmaxf(top, __uint_as_float(v[i]));
                const float next = kTreeBias - top * p.scale_log2;
                f = fast_exp2(next - shift);  // (0 for the first: shift is kTreeUnset)
                shift = next;
                l *= f;
                // weighed again as differences from the maximum: no weight above 2^kTreeBias
                // whatever the product's rounding, so that a chunk is weighed twice at most
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) - top);
                sh = kTreeBias;
              }
              __syncwarp();  // (tensor memory is read, written and waited for by whole warps)
              rescale(c, j >= 2, f);
            }
            tmem_st_x16(t_s + 32 * c, o);
          }
          if (copies > 1) {  // the other copies' tokens
            const uint32_t zero[16] = {};
#pragma unroll 1
            for (int c = 0; c < 4; ++c)
              if (c < c0 || c >= c1) tmem_st_x16(t_s + 32 * c, zero);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBPFull + 2 * set + ((e0 + (j >> two)) & 1)));
      }
      // ---- end of the segment: both accumulators are final ---------------------------------------------
      const bool any1 = n_jobs > 1;
      if (ok) {
        ok = twait(bar(kBPvDone + set), k & 1, wc);
      }
      tc_fence_before();  // (a set's accumulator is read by both sets, behind kBMl)
      float2* ml = reinterpret_cast<float2*>(smem + kOffMl) + (k & 1) * 256;
      const float m_ref = kTreeBias - shift;
      ml[128 * set + lrow] = make_float2(m_ref, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBMl));
      ok = ok && twait(bar(kBMl), k & 1, wc);
      if (barrier_or(1 + set, 128, !ok)) return false;
      // the row's parts (one per set and copy): the joint reference and sum, the weights of this lane's
      float w0 = 1.f, w1 = 0.f, m = m_ref, L = l;
      if (!two) {
        m = -INFINITY;
        for (int i = 0; i < copies; ++i) m = fmaxf(m, fmaxf(ml[row + i * gap].x, ml[128 + row + i * gap].x));
        L = 0.f;
        for (int i = 0; i < copies; ++i) {
          const float2 a = ml[row + i * gap], b = ml[128 + row + i * gap];
          const float wa = a.y != 0.f ? fast_exp2(a.x - m) : 0.f, wb = b.y != 0.f ? fast_exp2(b.x - m) : 0.f;
          L = fmaf(a.y, wa, fmaf(b.y, wb, L));
          if (i == copy) {
            w0 = wa;
            w1 = wb;
          }
        }
      }
      const size_t at0 = (size_t)r.q0 * kQHeads + kGqa * r.g;  // row i of the segment: + 16 (i / 4) + i % 4
      auto store4 = [&](int i, int ch, float Li, float a, float b, float c, float d) {
        if (r.slot < 0) {
          const float inv = p.out_scale / Li;  // (a NaN of the query stays one)
          uint2 x = make_uint2(pack16(a * inv, b * inv, p.out_f16), pack16(c * inv, d * inv, p.out_f16));
          if (Li == 0.f) x = make_uint2(0u, 0u);
          *reinterpret_cast<uint2*>(p.out + (at0 + (size_t)(i >> 2) * kQHeads + (i & 3)) * kHeadDim + ch) = x;
        } else {
          *reinterpret_cast<float4*>(p.part_o + ((size_t)r.slot * p.part_rows + i) * kHeadDim + ch) =
              Li != 0.f ? make_float4(a, b, c, d) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      };
      tc_fence_after();
      if (copies > 1) {
        // set s joins channels 64 s .. of both accumulators across the warps' copies: as many groups
        // of 16 channels at a time as the set's 8 KB hold (all four up to two drafts)
        const int parts = n_rows * copies, ush = parts <= 32 ? 2 : parts <= 64 ? 1 : 0, units = 1 << ush;
        const int me = copy * n_rows + row;  // (with a row)
        float* xb = reinterpret_cast<float*>(smem + kOffQ + 16384 + 8192 * set);  // [units][parts][16], chunks swizzled
        float2* rows = reinterpret_cast<float2*>(smem + kOffRow) + 64 * set;
        if (copy == 0 && mine) rows[row] = make_float2(m, L);
#pragma unroll 1
        for (int q = 0; q < 4; q += units) {
          __syncwarp();
          if (q > 0) named_barrier_sync(1 + set, 128);
          if (busy)
#pragma unroll 1
            for (int un = 0; un < units; ++un) {
              uint32_t u[16], v[16];
              tmem_ld32x32b_x16(tl + kTmemO + 64 * set + 16 * (q + un), u);
              if (any1) tmem_ld32x32b_x16(tl + kTmemO + 128 + 64 * set + 16 * (q + un), v);
              tmem_wait_ld();
              if (mine) {
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  x[i] = w0 > 0.f ? __uint_as_float(u[i]) * w0 : 0.f;
                  if (any1 && w1 > 0.f) x[i] = fmaf(__uint_as_float(v[i]), w1, x[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  *reinterpret_cast<float4*>(xb + 16 * (un * parts + me) + 4 * (i ^ (row >> 1 & 3))) =
                      make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
              }
              __syncwarp();
            }
          __syncwarp();
          named_barrier_sync(1 + set, 128);
          for (int i = lrow; i < 4 * units * n_rows; i += 128) {  // (row, unit, chunk)
            const int c = i & (4 * units - 1), ri = i >> (2 + ush), un = c >> 2;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            const float* part = xb + 16 * (un * parts + ri) + 4 * ((c & 3) ^ (ri >> 1 & 3));
#pragma unroll 2
            for (int cp = 0; cp < copies; ++cp, part += 16 * n_rows) {
              const float4 z = *reinterpret_cast<const float4*>(part);
              y.x += z.x;
              y.y += z.y;
              y.z += z.z;
              y.w += z.w;
            }
            store4(ri, 64 * set + 16 * q + 4 * c, rows[ri].y, y.x, y.y, y.z, y.w);
          }
        }
      } else if (busy) {
        // one tile: set s writes channels 64 s .. of both accumulators' sum; two tiles: all of its own
        const int ca = two ? 0 : 2 * set, cz = two ? 4 : 2 * set + 2;
#pragma unroll 1
        for (int c = ca; c < cz; ++c) {
          __syncwarp();
          uint32_t v[32];
          tmem_ld32x32b_x32(tl + kTmemO + (two ? 128 * set : 0) + 32 * c, v);
          if (!two && any1) {
            uint32_t u[32];
            tmem_ld32x32b_x32(tl + kTmemO + 128 + 32 * c, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[i] = __float_as_uint((w0 > 0.f ? __uint_as_float(v[i]) * w0 : 0.f) +
                                     (w1 > 0.f ? __uint_as_float(u[i]) * w1 : 0.f));
          } else {
            tmem_wait_ld();
          }
          if (mine)
#pragma unroll
            for (int u = 0; u < 8; ++u)
              store4(row, 32 * c + 4 * u, L, __uint_as_float(v[4 * u]), __uint_as_float(v[4 * u + 1]),
                     __uint_as_float(v[4 * u + 2]), __uint_as_float(v[4 * u + 3]));
        }
      }
      if (mine && copy == 0 && (two || set == 0)) {
        if (r.slot >= 0) p.part_ml[(size_t)r.slot * p.part_rows + row] = make_float2(m, L);
        else if (p.lse)
          p.lse[at0 + (size_t)(row >> 2) * kQHeads + (row & 3)] = L != 0.f ? (m - kTreeBias + log2f(L)) * kTreeLn2 : -INFINITY;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBOFree));
      return true;
    };
    for (int k = 0;; ++k) {
      // (the set's warps leave together: they meet at named barriers below)
      if (barrier_or(1 + set, 128, !twait(bar(kBRecFull + k % kRecs), (k / kRecs) & 1, wc))) break;
      const SegRec r = *rec(k);
      __syncwarp();
      if (r.n_pg < 0) break;
      if (lane == 0) mbar_arrive(bar(kBRecEmpty + k % kRecs));
      bool go;
      if constexpr (kCopies) {
        go = tree_copies(r.n_q) > 1 ? segment(r, k, std::integral_constant<int, 0>{})
             : r.n_q <= 32          ? segment(r, k, std::integral_constant<int, 1>{})
                                    : segment(r, k, std::integral_constant<int, 2>{});
      } else {
        go = r.n_q <= 32 ? segment(r, k, std::integral_constant<int, 1>{}) : segment(r, k, std::integral_constant<int, 2>{});
      }
      if (!go) break;
      e0 += r.n_pg;
    }
  } else {
    regs_dec<56>();
    // A scheduler (warp % 4) runs one of the two conversions, as far as the counts allow: the
    // fewer roles it has, the less its instruction cache is fought over.  V: warps 12, 16, 20,
    // 13, 17, 21, 14, 18; K: warps 15, 19, 23, 22.
    const int sched = warp & 3, turn = (warp - 12) >> 2;
    const bool is_v = sched < 2 || (sched == 2 && turn < 2);
    const int part = is_v ? 3 * sched + turn : sched == 3 ? turn : 3;
    if (is_v) {
      // ---------------- V conversion: token tok, channels 64 half .. 64 half + 63 ----------------------
      const int half = part >> 2, tok = 32 * (part & 3) + lane;
      const uint32_t tab = sbase + kOffVTab + 16 * (lane & (kVTabCopies - 1));
      const uint32_t raw0 = sbase + kOffRaw + kOffVc, out0 = sbase + kOffV16 + half * 16384 + tok * 16;
      const uint32_t code0 = tok * 64 + 16 * code_chunk_pos(2 * half, tok);
      const uint32_t code1 = tok * 64 + 16 * code_chunk_pos(2 * half + 1, tok);
      const uint32_t scale0 = (kOffKs - kOffKc) + 4 * half * kPageTokens + tok;
      int e = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!twait(bar(kBRecFull + k % kRecs), (k / kRecs) & 1, wc)) break;
        const int n_pg = rec(k)->n_pg;
        const bool two = rec(k)->n_q > 32;
        __syncwarp();
        if (n_pg < 0) break;
        if (lane == 0) mbar_arrive(bar(kBRecEmpty + k % kRecs));
        for (int i = 0; i < n_pg; ++i, ++e) {
          const int st = e % kRaw, sl = e % kSlot;
          if (!twait(bar(kBRawFull + st), (e / kRaw) & 1, wc)) {
            ok = false;
            break;
          }
          const uint32_t raw = raw0 + st * kHeadBytes, dst = out0 + sl * 32768;
          const int valid = s_info[e % kInfo].y;
          uint4 w[2] = {lds128(raw + code0), lds128(raw + code1)}, t[4];
          uint32_t sb[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) sb[u] = lds_u8(raw + scale0 + u * kPageTokens) & 127;
#pragma unroll
          for (int u = 0; u < 4; ++u) t[u] = lds128(tab + sb[u] * (16 * kVTabCopies));
          if (valid < kPageTokens && tok >= valid) {  // rows behind the sequence become zeros: a scale of zero
#pragma unroll
            for (int u = 0; u < 4; ++u) t[u] = make_uint4(0, 0, 0, 0);
            w[0] = w[1] = make_uint4(0, 0, 0, 0);
          }
          // (the loads are under way while the slot's last PV ends)
          if (!twait(bar(kBVEmpty + sl), ((e / kSlot) & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          // 8 channels of 128 tokens are 2,048 contiguous bytes
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            sts128(dst + (4 * cc) * 2048, dequant8_f16(w[cc].x, t[2 * cc]));
            sts128(dst + (4 * cc + 1) * 2048, dequant8_f16(w[cc].y, t[2 * cc]));
            sts128(dst + (4 * cc + 2) * 2048, dequant8_f16(w[cc].z, t[2 * cc + 1]));
            sts128(dst + (4 * cc + 3) * 2048, dequant8_f16(w[cc].w, t[2 * cc + 1]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (two || (i & 1) == 0) mbar_arrive(bar(kBPFull + sl));
            if (two || (i & 1) == 1) mbar_arrive(bar(kBPFull + 2 + sl));
            mbar_arrive(bar(kBRawEmpty + st));
          }
        }
      }
    } else {
      // ---------------- K conversion: token tok ----------------------------------------------------------
      const int tok = 32 * part + lane;
      const uint32_t tab = sbase + kOffKTab + 8 * (lane & (kKTabCopies - 1));
      const uint32_t raw0 = sbase + kOffRaw + kOffKc, out0 = sbase + kOffK8 + tok * 16;
      const uint32_t code0 = tok * 64 + 16 * code_chunk_pos(0, tok), scale0 = (kOffKs - kOffKc) + tok;
      int e = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!twait(bar(kBRecFull + k % kRecs), (k / kRecs) & 1, wc)) break;
        const int n_pg = rec(k)->n_pg;
        __syncwarp();
        if (n_pg < 0) break;
        if (lane == 0) mbar_arrive(bar(kBRecEmpty + k % kRecs));
        for (int i = 0; i < n_pg; ++i, ++e) {
          const int st = e % kRaw, sl = e % kSlot;
          if (!twait(bar(kBRawFull + st), (e / kRaw) & 1, wc) || !twait(bar(kBKEmpty + sl), ((e / kSlot) & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          const uint32_t raw = raw0 + st * kHeadBytes, dst = out0 + sl * 16384;
          // half of the channels at a time; 16 channels of 128 tokens are 2,048 contiguous bytes
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            // (code chunk c is at chunk c ^ x of the row: (code0 ^ 16 c) for the offset of chunk 0)
            const uint32_t ch = raw + (code0 ^ (32 * h)), ch1 = raw + (code0 ^ (32 * h + 16));
            const uint4 w[2] = {lds128(ch), lds128(ch1)};
            uint32_t sb[4];
            uint2 t[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) sb[u] = lds_u8(raw + scale0 + (4 * h + u) * kPageTokens) & 127;
#pragma unroll
            for (int u = 0; u < 4; ++u) t[u] = lds64(tab + sb[u] * (8 * kKTabCopies));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint2 a = dequant8(w[c].x, t[2 * c]), b = dequant8(w[c].y, t[2 * c]);
              const uint2 d = dequant8(w[c].z, t[2 * c + 1]), f = dequant8(w[c].w, t[2 * c + 1]);
              sts128(dst + (4 * h + 2 * c) * 2048, make_uint4(a.x, a.y, b.x, b.y));
              sts128(dst + (4 * h + 2 * c + 1) * 2048, make_uint4(d.x, d.y, f.x, f.y));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(kBKFull + sl));
            mbar_arrive(bar(kBRawEmpty + st));
          }
        }
      }
    }
  }

  // ---- teardown -------------------------------------------------------------------------
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    mbar_wait_drain(bar(kBDone), 0, drain_ns(p.wait_ns));  // every tcgen05.mma is done
    if (*s_abort) {
      set_status(p.status, MSA_STATUS_TIMEOUT);
      for (int e = max(p.inject ? 1 : 0, *s_issued - kRaw); e < *s_issued; ++e)  // copies that may still be landing
        mbar_wait_drain(bar(kBRawFull + e % kRaw), (e / kRaw) & 1, drain_ns(p.wait_ns));
    }
  }
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Rows whose pages were cut across CTAs: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
// One CTA per (draft, KV head): two warps per query head, each with every other part, lane =
// 4 channels.  A latency chain: a descriptor, then up to 12 parts' loads of a warp at once
// (relative to their own maximum; the two warps' halves join in shared memory).
constexpr int kMergeParts = 12;
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float4 s_o[4][32];
  __shared__ float2 s_ml[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = warp & 3, half = warp >> 2;
  const int tg = blockIdx.x;  // (token, KV head)
  pdl_wait();
  const int desc = p.row_desc[tg];
  __syncthreads();
  if (desc == 0) return;
  if (threadIdx.x == 0) p.row_desc[tg] = 0;  // at rest for the next call
  const int c0 = desc & 255, parts = (desc >> 8) & 4095, row = 4 * (desc >> 20) + h;
  float M = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = half; i0 < parts; i0 += 2 * kMergeParts) {
    float4 x[kMergeParts];
    float2 ml = make_float2(-INFINITY, 0.f);  // lane u: part i0 + 2 u
    auto slot = [&](int u) { return (size_t)(2 * (c0 + i0 + 2 * u) + (i0 + 2 * u == 0)) * p.part_rows + row; };
    if (lane < kMergeParts && i0 + 2 * lane < parts) ml = p.part_ml[slot(lane)];
#pragma unroll
    for (int u = 0; u < kMergeParts; ++u) {
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + 2 * u < parts) x[u] = reinterpret_cast<const float4*>(p.part_o + slot(u) * kHeadDim)[lane];
    }
    const float top = fmaxf(M, warp_max_f32(ml.y != 0.f ? ml.x : -INFINITY));
    const float f = M > -INFINITY ? fast_exp2(M - top) : 0.f, w = ml.y != 0.f ? fast_exp2(ml.x - top) : 0.f;
    M = top;
    L *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int u = 0; u < kMergeParts; ++u) {
      const float wu = __shfl_sync(0xffffffffu, w, u);
      L = fmaf(__shfl_sync(0xffffffffu, ml.y, u), wu, L);
      o.x = fmaf(x[u].x, wu, o.x);
      o.y = fmaf(x[u].y, wu, o.y);
      o.z = fmaf(x[u].z, wu, o.z);
      o.w = fmaf(x[u].w, wu, o.w);
    }
  }
  if (half == 1) {
    s_o[h][lane] = o;
    if (lane == 0) s_ml[h] = make_float2(M, L);
  }
  __syncthreads();
  if (half == 1) return;
  const float2 b = s_ml[h];
  const float4 y = s_o[h][lane];
  const float top = fmaxf(M, b.x);
  const float wa = L != 0.f ? fast_exp2(M - top) : 0.f, wb = b.y != 0.f ? fast_exp2(b.x - top) : 0.f;
  L = L * wa + b.y * wb;
  o = make_float4(o.x * wa + y.x * wb, o.y * wa + y.y * wb, o.z * wa + y.z * wb, o.w * wa + y.w * wb);
  const float inv = L != 0.f ? p.out_scale / L : 0.f;  // (a NaN of the query stays one)
  const size_t at = (size_t)(tg >> 2) * kQHeads + kGqa * (tg & 3) + h;
  *reinterpret_cast<uint2*>(p.out + at * kHeadDim + 4 * lane) =
      make_uint2(pack16(o.x * inv, o.y * inv, p.out_f16), pack16(o.z * inv, o.w * inv, p.out_f16));
  if (p.lse && lane == 0) p.lse[at] = L != 0.f ? (top - kTreeBias + log2f(L)) * kTreeLn2 : -INFINITY;
}

int tree_rows(int n_q_total) { return n_q_total < kTreeMaxDrafts ? kGqa * n_q_total : kGqa * kTreeMaxDrafts; }
// The descriptors first, at a size of their own: the words that have to be zero between
// calls are in one place whatever the sizes of the calls that share a workspace.
constexpr size_t kDescBytes = (size_t)65536 * kKvHeads * sizeof(int);
size_t ml_bytes(size_t rows) { return (2 * kTreeCtas * rows * sizeof(float2) + 255) / 256 * 256; }

}  // namespace

size_t tree_attn_workspace_bytes(int n_q_total) {
  const size_t rows = tree_rows(n_q_total);
  return kDescBytes + ml_bytes(rows) + 2 * kTreeCtas * rows * kHeadDim * sizeof(float);
}

cudaError_t launch_tree_attn(const msa_cache* c, const uint8_t* q, float softmax_scale, const int* block_table,
                             int max_pages, const int* seq_lens, const int* q_start_loc, int n_seqs, int n_q_total,
                             const uint64_t* tree_mask, const int* sel, const int* n_sel, int dtype, void* out,
                             float* lse, void* ws, cudaStream_t stream) {
  if (n_q_total == 0 || n_seqs == 0) return cudaSuccess;
  static DeviceSetup setup;
  int dev = 0, n_sm = 0;
  cudaError_t e = setup.get(&dev, &n_sm, [](int) {
    constexpr auto kMax = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<true>, kMax, kTreeSmem);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(tree_attn_kernel<false>, kMax, kTreeSmem);
  });
  if (e != cudaSuccess) return e;
  TreeParams tp{};
  tp.kv_pool = static_cast<const uint8_t*>(c->kv_pool);
  tp.n_pages = c->n_pages;
  tp.q = q;
  tp.block_table = block_table;
  tp.max_pages = max_pages;
  tp.seq_lens = seq_lens;
  tp.q_start_loc = q_start_loc;
  tp.n_seqs = n_seqs;
  tp.n_q_total = n_q_total;
  tp.tree_mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  tp.sel = sel;
  tp.n_sel = n_sel;
  // (a quotient below fp32's normal numbers is as good as the smallest: the scores, below 2^25 times
  // it, leave every weight alike; zero would make a hidden token's -inf a NaN)
  tp.scale_log2 = std::max(softmax_scale / c->s_enc_k * kTreeLog2e, FLT_MIN);
  tp.out_scale = 256.0f / c->s_enc_v;
  tp.out_f16 = dtype == MSA_DTYPE_F16;
  tp.out = static_cast<uint16_t*>(out);
  tp.lse = lse;
  tp.part_rows = tree_rows(n_q_total);
  uint8_t* w = static_cast<uint8_t*>(ws);
  tp.row_desc = reinterpret_cast<int*>(w);
  w += kDescBytes;
  tp.part_ml = reinterpret_cast<float2*>(w);
  w += ml_bytes(tp.part_rows);
  tp.part_o = reinterpret_cast<float*>(w);
  tp.status = c->status;
  tp.wait_ns = launch_settings().wait_ns;
  tp.inject = (launch_settings().inject & MSA_INJECT_ATTENTION_TIMEOUT) != 0;
  const int most = n_sm < kTreeCtas ? n_sm : kTreeCtas;
  // Without the row copies' code two tiles run faster (8 sequences of 131,072 with 64 drafts: 386 us,
  // 417 with it; 24 of 30,720 with 17 to 32 drafts 177 us, 187), few drafts slower (8 to 16 drafts:
  // 170 us, 161 with it): by the mean, mixtures included (4 to 24 drafts, mean 14: 171 us both; 2 to
  // 40, mean 21: 196 and 202; 1 to 64, mean 38: 263 and 278).  The lengths are on the device, so
  // the mean is of the rows that the call passes: padding rows and empty sequences count.
  e = launch_pdl(n_q_total > 16ll * n_seqs ? tree_attn_kernel<false> : tree_attn_kernel<true>, dim3(most),
                 dim3(kTreeThreads), kTreeSmem, stream, tp);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_merge_kernel, dim3((unsigned)(n_q_total * kKvHeads)), dim3(256), 0, stream, tp);
}

}  // namespace msa
