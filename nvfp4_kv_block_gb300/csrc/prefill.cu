// Attention of a prompt's tokens, any number a sequence, over the sequence's pages of the
// NVFP4 cache: causal, within a window, or up to an end that each token brings along.
//
// Mathematics.  For a row (token, query head) with FP8 query q, the keys k8_t and values v8_t
// dequantised to FP8 as in the other attention kernels, over start <= t < end,
//   x_t = (q . k8_t) scale / s_enc_k log2(e),  out = sum_t 2^x_t v8_t / sum_t 2^x_t / s_enc_v,
// in one pass over the pages with a reference m per row: weights 2^(x_t - m + 8), summed in
// fp32, multiply V in f16 (a relative 2^-11; an E4M3 weight would lose the bulk of a long
// context behind one large key).  m moves only when the weights of 64 tokens, half a page, would sum to more
// than 49,152 (f16 ends at 65,504), and to the maximum of those 64: 1.1 (all alike) to 5.3 (one alone) natural units above m and more.  A row's
// first 64 tokens do it always, later ones where scores spread: then the half's scores are read twice more and the
// accumulator is rescaled, for 32 rows when one of them needs it.  Scores that deviate by 0.5: 8,192 tokens 161 us,
// 2,048 over 131,072 1,113; by 1.6: 164 and 1,132; by 3.2: 257 and 1,293, and 255 and 1,504 where keys grow eightfold along
// the context; by 6.3: 287 and 1,371.
//
// Three kernels.  (1) Every page that a sequence visits is converted once per KV head into the
// operand tiles of the products, 16 KB of E4M3 keys and 32 KB of f16 values, by a kernel bound
// by memory (a page that several sequences of the call share, once for each of them); it also writes down the tiles of
// 64 tokens and their pages.  (2) The attention: a job
// is a tile (256 rows, 4 i + h for token i and head h of the group) and a KV head; the jobs'
// pages in a row are cut into equal weighted ranges, one per persistent CTA, or, where that is nearly as even, jobs are
// taken whole from a queue.  A job that was cut
// leaves fp32 rows, which the last of its parts joins in the order of the parts (each warp for
// its rows, behind a counter).  (3) Jobs in more parts, and those of calls without whole jobs, are joined by a
// kernel of their own.
//
// Roles of the attention's warps, all hand-offs mbarriers with bounded waits:
//   warp 0      segment records, a bulk copy of 48 KB per page;
//   warp 1      MMA issuer: S = Q K8^T (kind::f8f6f4, 128 x 128 x 128), then O += P V
//               (kind::f16, P from tensor memory over S's own columns);
//   warp 2      query rows of the next segment;
//   warps 4-11  softmax, thread = row: a set of four warps for each 128 rows;
//   warps 12-15 rows of finished segments on their way out.
//
// What bounds it.  A page of two row tiles is 1,536 cycles of the tensor pipe (PV 512 and QK 256 each) and
// takes about 2,330: a set's chain is its softmax (850 cycles for 128 keys), the hand-over of the weights
// (290), PV and the next QK into the same columns (820), the hand-over of the scores (400), and the two
// sets run half a period apart.  Two tiles of scores and two accumulators are all of tensor memory, so there is no
// third one to fill the gaps.  From card to card, 2,048 tokens over 131,072: 1,113 to 1,136 us, 1.95 to 1.99 PFLOP/s (1.90
// is the measured bf16 rate; at that rate for PV and twice it for QK the products alone take 877); 8,192 from the
// beginning: 161 to 163 us, the products 109; 4,096 with a window of 4,096: 97 to 98, 55.  Tiles of 64 tokens x 4 heads: a page's 48 KB then feed two products
// of 128 rows, 21 bytes a cycle and SM from L2.  100 tokens: 18 us, two launches and a chain of some
// thirty latencies.
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>

#include "attn_ops.cuh"
#include "tensor_map.cuh"

namespace msa {
namespace {

constexpr int kPrefillThreads = 512;
constexpr int kTileTokens = 64;       // two row tiles of 32 tokens x 4 heads
constexpr int kPrefillCtas = 152;     // most CTAs of a launch (the workspace is sized for them)
constexpr int kStages = 3;            // pages in flight
constexpr int kRecs = 4;
constexpr int kInfo = 16;
constexpr int kImageK = 16384, kImage = kImageK + 32768;  // bytes of a converted (page, KV head)

constexpr int kOffQ = 0;                                  // 2 segments x 2 tiles [128 rows][128 B]
// kStages x (K [8 groups of 16 channels][128 tokens][16 B], V [16 groups of 8 channels][128 tokens][16 B])
constexpr int kOffK = kOffQ + 4 * 16384;
constexpr int kOffRecs = kOffK + kStages * kImage;        // kRecs x 64 B
constexpr int kOffInfo = kOffRecs + kRecs * 64;           // int [kInfo]: page inside the pool
constexpr int kOffScan = kOffInfo + kInfo * 4;            // long long [32]
constexpr int kOffRange = kOffScan + 32 * 8;              // long long [kPrefillCtas + 1]
constexpr int kOffMl = kOffRange + 160 * 8;                 // float2 [2 sets][2 parities][128]: a row's reference and sum
constexpr int kOffJoin = (kOffMl + 2 * 2 * 128 * 8 + 1023) / 1024 * 1024;  // 4 output warps x [32 rows][64 B]
constexpr int kOffBars = kOffJoin + 4 * 2048;
constexpr int kBFull = 0, kBEmpty = kBFull + kStages, kBQFull = kBEmpty + kStages, kBQEmpty = kBQFull + 2,
              kBSFull = kBQEmpty + 2, kBPFull = kBSFull + 2, kBPvDone = kBPFull + 2, kBOFree = kBPvDone + 2, kBMl = kBOFree + 2, kBRecFull = kBMl + 4,  // kBMl: [set][parity]
              kBRecEmpty = kBRecFull + kRecs,
              kBDone = kBRecEmpty + kRecs, kBars = kBDone + 1;
constexpr int kOffMisc = kOffBars + 8 * ((kBars + 1) & ~1);  // tmem, abort, pages issued
constexpr int kSorted = 256;  // tiles that a queue has in order of their weights
constexpr int kOffOrder = kOffMisc + 16;                     // uint16_t [kSorted]
constexpr int kPrefillSmem = 1024 + kOffOrder + 2 * kSorted;
static_assert(kPrefillSmem <= 232448, "shared memory of one CTA");
static_assert(kOffBars % 8 == 0, "barriers");
constexpr uint32_t kTmemS = 0, kTmemO = 256;  // S of set s at 128 s, O of set s at 256 + 128 s
constexpr float kBias = 8.0f;
constexpr float kMost = 49152.0f;  // largest sum of 64 weights, and so largest weight
constexpr float kUnset = 3e38f;           // shift of a row without a reference
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Weights of the partition: a page, whether a tile has up to 32 tokens or up to 64 (one set's chain
// takes as long as two sets': 2,330 cycles); the fixed part of a job, records, queries and the rows' way out
// (16: 8,192 tokens 170 us, 159 with 24, 165 with 40; 14 other calls, geometric mean, 62.3, 59.7, and 20 to 32 alike);
// the least weight of a job (one of a page or two takes as long as five: the chain of its first scores and of its rows'
// way out); and the least share of a CTA (a page's weight at least, so that every CTA between a job's first and
// last has pages of it).
constexpr int kPageWeight = 9, kFixed = 24, kSmall = 45, kLeast = 10;

// Jobs stay whole if the CTA with most then has no more than an equal share and kCut: parts cost their rows'
// way to memory and back, some 16,000 cycles, with nothing under it at a call's end.  The same 14 calls: 59.0 us where
// all is cut, 54.7 with 30, 51.8 with 100, 52.6 with 150 (sequences of 69 to 126 tokens: 36.8 and 24.4).  They are
// taken from a queue, the heaviest first (of up to 256 tiles, each ranked by one thread; the last tile of all, which
// sees most of its sequence, where there are more): 8,192 tokens 163 us with cut jobs, 160; 15 chunks of up to 249
// tokens at places up to 2,111, last tile first 56.5, heaviest first 48.0.  Which CTA takes a job changes no row of it.
constexpr int kCut = 100;

// Parts of a job that its last one joins: under other jobs' pages where CTAs have whole jobs behind the cut ones
// (up to 6; with a window of 4,096 97 us, 100 with 2 parts at most and the third kernel for the others), none where
// they have not: the third kernel's many CTAs read the parts at once (45 us against 31 for sequences of 5 to
// 110 tokens over 1,943).
constexpr int kInline = 6, kAlone = 1;

struct TileRec {
  int q0, n_tok;  // rows of the call
  int pos;        // position of the first token
  int len;        // tokens of the sequence
  int page0;      // first page (block of the sequence), and how many (0: nothing to do)
  int n_pg;
  int ws_page;    // its place among the converted pages
  int pad;
};
static_assert(sizeof(TileRec) == 32, "loaded by eight lanes");

struct SegRec {
  int n_pg;  // pages of the segment; -1: no more segments
  int g, q0, n_tok, pos, len;
  int page0;
  int part, parts;  // which part of the job the segment is, and of how many
  int c0;           // CTA of part 0
  int job;
  int join;  // the last part joins them
};
// Place of part i of a job whose first part is CTA c0's: a CTA's last segment, then first ones.
__device__ __forceinline__ size_t part_slot(int c0, int i) { return 2 * (c0 + i) + (i == 0); }
static_assert(sizeof(SegRec) <= 64, "record slot");

struct PrefillParams {
  CUtensorMap out_map, out_map32;  // out as [T][16][128], boxes of 8 tokens x 4 heads x 64 and 32 channels
  const uint8_t* kv_pool;
  int64_t n_pages;
  const uint8_t* q;  // [T][16][128]
  const int* block_table;
  int max_pages;
  const int* seq_lens;
  const int* q_start_loc;
  int n_seqs;
  int n_q_total;
  int window;       // 0: none
  const int* ends;  // [T] or null
  float scale_log2;
  float out_scale;  // 2^8 / s_enc_v
  int out_f16;
  uint16_t* out;  // [T][16][128]
  float* lse;     // [T][16] or null
  int* n_tiles;   // workspace from here on
  TileRec* tiles;
  int max_tiles;
  int* next;         // whole jobs that were taken from the queue
  int* n_big;        // jobs of the third kernel, and which: job, first CTA | parts << 8
  int2* big;         // [4 max_tiles]
  int* tickets;      // [max_tiles][4][8]: parts that a warp's rows are there of
  int* page_ok;      // [cap]
  int cap;           // converted pages that fit
  // a part's rows, 32 (a softmax warp's) at a time: [2 kPrefillCtas][part_quads]
  float4* part_o;    // ... [32 of 4 channels][32 rows]
  float2* part_ml;   // ... [32 rows]: reference and sum
  int part_quads;
  uint8_t* images;   // [cap][4][kImage]
  int* status;
  unsigned long long wait_ns;
  int inject;  // test only: a CTA's first page is not copied, so that the waits for it run out
};

// ---- (1) conversion and tiles -------------------------------------------------------
// Once a call and not in every tile's CTA: a page of 8,192 tokens' prompt is seen by up to 128 tiles, and converting
// it costs 2,000 warp instructions a head each time.  18 KB in, 48 KB out per page and head; a call more of it
// takes 6 us for 64 pages, 47 for 1,040 (6.0 TB/s of those bytes, a part of which stays in L2 for the attention).
constexpr int kConvThreads = 256;
constexpr int kConvKCopies = 4, kConvVCopies = 8;
constexpr int kConvTables = 128 * (8 * kConvKCopies + 16 * kConvVCopies);

// First page that a sequence's rows can see, and pages from there to its end.
__device__ __forceinline__ int first_page(const PrefillParams& p, int pos) {
  return p.window ? max(0, pos + 1 - p.window) / kPageTokens : 0;
}

__global__ void __launch_bounds__(kConvThreads) prefill_convert_kernel(const __grid_constant__ PrefillParams p) {
  extern __shared__ __align__(16) uint8_t conv_smem[];
  __shared__ int2 s_warp[kConvThreads / 32];
  uint2* kt = reinterpret_cast<uint2*>(conv_smem);
  uint4* vt = reinterpret_cast<uint4*>(conv_smem + 128 * 8 * kConvKCopies);
  int* s_page = reinterpret_cast<int*>(conv_smem + kConvTables);  // [n_seqs + 1] pages before sequence b
  int* s_tile = s_page + p.n_seqs + 1;                            // tiles before it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 128) convert_tables<kConvKCopies, kConvVCopies>(tid, kt, vt);
  pdl_wait();
  pdl_trigger();
  const int per = (p.n_seqs + kConvThreads - 1) / kConvThreads;
  int2 mine = make_int2(0, 0);
  auto work = [&](int b) {  // pages and tiles of a sequence
    const SeqInfo s = load_seq(b, p.seq_lens, p.q_start_loc, p.max_pages, p.n_q_total);
    if (!s.ok) {
      if (blockIdx.x == 0) set_status(p.status, MSA_STATUS_BAD_SEQ);
      return make_int2(0, 0);
    }
    if (s.n_q == 0) return make_int2(0, 0);
    return make_int2((s.seq_len + kPageTokens - 1) / kPageTokens - first_page(p, s.seq_len - s.n_q),
                     (s.n_q + kTileTokens - 1) / kTileTokens);
  };
  const int b0 = min(tid * per, p.n_seqs), b1 = min(b0 + per, p.n_seqs);
  for (int b = b0; b < b1; ++b) {
    const int2 w = work(b);
    s_page[b + 1] = w.x;
    s_tile[b + 1] = w.y;
    mine.x += w.x;
    mine.y += w.y;
  }
  int2 incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) {
      incl.x += x;
      incl.y += y;
    }
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int2 at = make_int2(incl.x - mine.x, incl.y - mine.y);
  for (int i = 0; i < warp; ++i) {
    at.x += s_warp[i].x;
    at.y += s_warp[i].y;
  }
  if (tid == 0) s_page[0] = s_tile[0] = 0;
  for (int b = b0; b < b1; ++b) {
    at.x += s_page[b + 1];
    at.y += s_tile[b + 1];
    s_page[b + 1] = at.x;
    s_tile[b + 1] = at.y;
  }
  __syncthreads();
  // (what does not fit the workspace is left out: more pages than it is for, or rows that several
  // sequences claim)
  auto fits = [&](int b) { return s_page[b + 1] <= p.cap && s_tile[b + 1] <= p.max_tiles; };
  auto find = [&](const int* prefix, int x) {  // the last b with prefix[b] <= x
    int lo = 0, hi = p.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  const int n_tiles = min(s_tile[p.n_seqs], p.max_tiles);
  if (blockIdx.x == 0) {
    if (tid == 0) {
      *p.n_tiles = n_tiles;
      *p.n_big = 0;
      *p.next = 0;
    }
    for (int b = tid; b < p.n_seqs; b += kConvThreads)
      if (s_page[b + 1] > s_page[b] && !fits(b)) set_status(p.status, MSA_STATUS_BAD_SEQ);
  }
  // a warp per tile
  for (int t = (int)blockIdx.x * (kConvThreads / 32) + warp; t < n_tiles; t += (int)gridDim.x * (kConvThreads / 32)) {
    const int b = find(s_tile, t);
    const SeqInfo s = load_seq(b, p.seq_lens, p.q_start_loc, p.max_pages, p.n_q_total);
    TileRec r{};
    const int i0 = kTileTokens * (t - s_tile[b]);
    r.q0 = s.q0 + i0;
    r.n_tok = min(kTileTokens, s.n_q - i0);
    r.pos = s.seq_len - s.n_q + i0;
    r.len = s.seq_len;
    int top = r.pos + r.n_tok;  // behind the last key that some row sees
    if (p.ends) {
      top = max(lane < r.n_tok ? p.ends[r.q0 + lane] : 0, lane + 32 < r.n_tok ? p.ends[r.q0 + lane + 32] : 0);
      top = min(__reduce_max_sync(0xffffffffu, top), r.len);
    }
    const int seq0 = first_page(p, s.seq_len - s.n_q);
    r.page0 = first_page(p, r.pos);
    r.n_pg = fits(b) ? max(1, (top + kPageTokens - 1) / kPageTokens - r.page0) : 0;
    r.ws_page = s_page[b] + r.page0 - seq0;
    if (lane == 0) p.tiles[t] = r;
    p.tickets[t * 32 + lane] = 0;
  }
  // (page, head) units: thread = token and half of the channels
  const int tok = tid & 127, half = tid >> 7;
  const uint2* my_kt = kt + (lane & (kConvKCopies - 1));
  const uint4* my_vt = vt + (lane & (kConvVCopies - 1));
  const int units = min(s_page[p.n_seqs], p.cap) * kKvHeads;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int page = u / kKvHeads, g = u % kKvHeads;
    const int b = find(s_page, page);
    if (!fits(b)) continue;
    const int n_q = p.q_start_loc[b + 1] - p.q_start_loc[b];
    const int blk = first_page(p, p.seq_lens[b] - n_q) + page - s_page[b];
    const int phys = p.block_table[(size_t)b * p.max_pages + blk];
    const bool ok = phys >= 0 && phys < p.n_pages;
    if (tid == 0 && g == 0) {
      if (!ok) set_status(p.status, MSA_STATUS_BAD_PAGE);
      p.page_ok[page] = ok;
    }
    uint8_t* out = p.images + ((size_t)page * kKvHeads + g) * kImage;
    uint4* ko = reinterpret_cast<uint4*>(out) + 4 * half * kPageTokens + tok;            // group 4 half + i: + 128 i
    uint4* vo = reinterpret_cast<uint4*>(out + kImageK) + 8 * half * kPageTokens + tok;  // group 8 half + i
    if (!ok) {  // zeros: the values meet weights of zero
#pragma unroll
      for (int i = 0; i < 4; ++i) ko[i * kPageTokens] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) vo[i * kPageTokens] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint8_t* head = p.kv_pool + (size_t)phys * kKvPageBytes + (size_t)g * kHeadBytes;
    uint4 kc[2], vc[2];
    uint32_t ks[4], vs[4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int off = tok * 64 + 16 * code_chunk_pos(2 * half + c, tok);
      kc[c] = ld_stream_v4(head + kOffKc + off);
      vc[c] = ld_stream_v4(head + kOffVc + off);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ks[i] = __ldg(head + kOffKs + (4 * half + i) * kPageTokens + tok) & 127;
      vs[i] = __ldg(head + kOffVs + (4 * half + i) * kPageTokens + tok) & 127;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint2 t0 = my_kt[ks[2 * c] * kConvKCopies], t1 = my_kt[ks[2 * c + 1] * kConvKCopies];
      const uint2 a = dequant8(kc[c].x, t0), d = dequant8(kc[c].y, t0), e = dequant8(kc[c].z, t1), f = dequant8(kc[c].w, t1);
      ko[(2 * c) * kPageTokens] = make_uint4(a.x, a.y, d.x, d.y);
      ko[(2 * c + 1) * kPageTokens] = make_uint4(e.x, e.y, f.x, f.y);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 t0 = my_vt[vs[2 * c] * kConvVCopies], t1 = my_vt[vs[2 * c + 1] * kConvVCopies];
      vo[(4 * c) * kPageTokens] = dequant8_f16(vc[c].x, t0);
      vo[(4 * c + 1) * kPageTokens] = dequant8_f16(vc[c].y, t0);
      vo[(4 * c + 2) * kPageTokens] = dequant8_f16(vc[c].z, t1);
      vo[(4 * c + 3) * kPageTokens] = dequant8_f16(vc[c].w, t1);
    }
  }
}

// ---- (2) attention --------------------------------------------------------------------
// a / b of weights: in 32 bits where they fit (nearly always; a 64-bit division is a subroutine, and ten of
// them took 1.3 us of a call's start).
__device__ __forceinline__ long long quot(long long a, long long b) {
  return (a | b) >> 31 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}
__device__ __forceinline__ int job_weight(int n_pg) { return n_pg > 0 ? max(kFixed + n_pg * kPageWeight, kSmall) : 0; }

// Bits 0 .. n - 1 (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1; }

// 32 bytes at once (aligned).
__device__ __forceinline__ void st32(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f, uint32_t g, uint32_t h) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
               : "memory");
}

// Waits for tensor memory loads; the 32 values (one of them) are not touched before.
__device__ __forceinline__ void wait_ld32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}
// Weights of 32 scores as f16 pairs, and their sums.
__device__ __forceinline__ void weigh32(const uint32_t (&v)[32], uint64_t scale2, uint64_t shift2, uint64_t (&sums)[2], uint32_t* o) {
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    const uint2 y = split64(fma_f32x2(pair64(v[2 * x], v[2 * x + 1]), scale2, shift2));
    const float a = fast_exp2(__uint_as_float(y.x)), b = fast_exp2(__uint_as_float(y.y));
    sums[x & 1] = add_f32x2(sums[x & 1], pair64(__float_as_uint(a), __float_as_uint(b)));
    o[x] = cvt_f16x2_f32(b, a);
  }
}
// A row's accumulator, and its weights of a page's first half, times f.
__device__ __forceinline__ void scale_acc(uint32_t t_o, float f) {
#pragma unroll 1
  for (int c = 0; c < kHeadDim; c += 16) {
    uint32_t u[16];
    tmem_ld32x32b_x16(t_o + c, u);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 16; ++x) u[x] = __float_as_uint(__uint_as_float(u[x]) * f);
    tmem_st_x16(t_o + c, u);
  }
}
__device__ __forceinline__ void scale_p(uint32_t t_p, float f) {
  tmem_wait_st();
#pragma unroll 1
  for (int c = 0; c < 64; c += 32) {
    uint32_t u[16];
    tmem_ld32x32b_x16(t_p + c, u);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&u[x]));
      u[x] = cvt_f16x2_f32(w.y * f, w.x * f);
    }
    tmem_st_x16(t_p + c, u);
  }
}

// Bulk copies from shared memory, and waits for a thread's own: read, or done.
__device__ __forceinline__ void bulk_s2g(void* to, uint32_t from, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tensor_s2g(const CUtensorMap* map, int x, int y, int z, uint32_t from) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y), "r"(z),
               "r"(from)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_read_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 32 channels (the c-th of four) of 32 rows, lane = row, on their way out: into a box of 64 channels x 4
// heads x 8 tokens in shared memory (rows of 128 bytes, swizzled), which leaves with its second half, or
// (kNarrow) into one of 32 channels.
template <bool kNarrow>
__device__ __forceinline__ void put32(const PrefillParams& p, const SegRec& r, const float (&o)[32], float inv, int c, int tok0,
                                      int lane, uint32_t stage) {
  uint32_t y[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) y[x] = pack16(o[2 * x] * inv, o[2 * x + 1] * inv, p.out_f16);
  if (tok0 + 8 <= r.n_tok) {
    const uint32_t box = kNarrow ? stage : stage + (c >> 1) * 4096;
    if (kNarrow) {
      if (lane == 0) bulk_read_wait();
      __syncwarp();
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      sts128(kNarrow ? box + lane * 64 + ((x ^ (lane >> 1 & 3)) << 4) : box + lane * 128 + (((4 * (c & 1) + x) ^ (lane & 7)) << 4),
             make_uint4(y[4 * x], y[4 * x + 1], y[4 * x + 2], y[4 * x + 3]));
    if (kNarrow || (c & 1)) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tensor_s2g(kNarrow ? &p.out_map32 : &p.out_map, kNarrow ? 32 * c : 32 * (c - 1), kGqa * r.g, r.q0 + tok0, box);
        bulk_commit();
      }
    }
  } else if (tok0 + (lane >> 2) < r.n_tok) {  // the last tokens of a sequence: a box would go on into the next one's rows
    uint16_t* to = p.out + ((size_t)(r.q0 + tok0 + (lane >> 2)) * kQHeads + kGqa * r.g + (lane & 3)) * kHeadDim + 32 * c;
    st32(to, y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]);
    st32(to + 16, y[8], y[9], y[10], y[11], y[12], y[13], y[14], y[15]);
  }
}
__device__ __forceinline__ void put_lse(const PrefillParams& p, const SegRec& r, float m, float l, int tok0, int lane) {
  const int token = tok0 + (lane >> 2);
  if (p.lse && token < r.n_tok)
    p.lse[(size_t)(r.q0 + token) * kQHeads + kGqa * r.g + (lane & 3)] = l != 0.f ? (m - kBias + log2f(l)) * kLn2 : -INFINITY;
}

// A segment's part of a cut job (a warp's 32 rows from token tok0 on; own: a row's reference and sum): its
// rows on their way to the part's place (zeros where a row saw nothing).  freed: called when the accumulator
// is read.
template <typename F>
__device__ __forceinline__ void put_part(const PrefillParams& p, const SegRec& r, float2 own, int tok0, int lane, uint32_t t_o,
                                         uint32_t stage, F&& freed) {
  auto rows_of = [&](int i) { return (part_slot(r.c0, i) * p.part_quads + (tok0 >> 3)) * 32; };
  p.part_ml[rows_of(r.part) + lane] = own;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {  // 64 channels of 32 rows: [16 of 4 channels][32 rows]
    uint32_t v[64];
    __syncwarp();  // (lane 0 was apart: tensor memory is read by whole warps)
    tmem_ld32x32b_x64(t_o + 64 * c, v);
    tmem_wait_ld();
    if (c) freed();
    if (own.y == 0.f)
#pragma unroll
      for (int x = 0; x < 64; ++x) v[x] = 0;
    if (lane == 0) bulk_read_wait();
    __syncwarp();
#pragma unroll
    for (int x = 0; x < 16; ++x)
      sts128(stage + (x * 32 + lane) * 16, make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      bulk_s2g(p.part_o + (rows_of(r.part) + 16 * c) * 32, stage, 8192);
      bulk_commit();
    }
  }
}
// Behind it, when the rows are there: if those of all parts are now, the parts' sum to the output.
__device__ __forceinline__ void join_parts(const PrefillParams& p, const SegRec& r, int tok0, int lane, uint32_t stage) {
  auto rows_of = [&](int i) { return (part_slot(r.c0, i) * p.part_quads + (tok0 >> 3)) * 32; };
  __threadfence();
  __syncwarp();
  int before = 0;
  if (lane == 0) {
    bulk_wait();
    __threadfence();
    before = atomicAdd(p.tickets + (r.job * 8 + (tok0 >> 3)), 1);
  }
  if (__shfl_sync(0xffffffffu, before, 0) != r.parts - 1) return;
  __threadfence();
  float2 ml[kInline];
  float top = -INFINITY, sum = 0.f, w[kInline];
#pragma unroll
  for (int i = 0; i < kInline; ++i) ml[i] = i < r.parts ? __ldcg(p.part_ml + rows_of(i) + lane) : make_float2(-INFINITY, 0.f);
#pragma unroll
  for (int i = 0; i < kInline; ++i)
    if (ml[i].y != 0.f) top = fmaxf(top, ml[i].x);
#pragma unroll
  for (int i = 0; i < kInline; ++i) {
    w[i] = ml[i].y != 0.f ? fast_exp2(ml[i].x - top) : 0.f;
    sum = fmaf(ml[i].y, w[i], sum);
  }
  put_lse(p, r, top, sum, tok0, lane);
  const float inv = sum != 0.f ? p.out_scale / sum : 0.f;  // (a NaN of the query stays one)
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float s[32] = {};
#pragma unroll 1
    for (int i = 0; i < r.parts; i += 2) {  // two parts' loads at once
      float4 z[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < 8; ++x)
          z[h][x] = i + h < r.parts ? __ldcg(p.part_o + (rows_of(i + h) + 8 * c + x) * 32 + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float f = i + h < r.parts ? w[i + h] : 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          s[4 * x] = fmaf(z[h][x].x, f, s[4 * x]);
          s[4 * x + 1] = fmaf(z[h][x].y, f, s[4 * x + 1]);
          s[4 * x + 2] = fmaf(z[h][x].z, f, s[4 * x + 2]);
          s[4 * x + 3] = fmaf(z[h][x].w, f, s[4 * x + 3]);
        }
      }
    }
    put32<true>(p, r, s, inv, c, tok0, lane, stage);
  }
}

__global__ void __launch_bounds__(kPrefillThreads, 1) prefill_attn_kernel(const __grid_constant__ PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + kOffBars + 8 * i; };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int* s_issued = reinterpret_cast<int*>(smem + kOffMisc + 8);  // pages
  const WaitCtl wc{s_abort, p.wait_ns};
  auto rec = [&](int k) { return reinterpret_cast<SegRec*>(smem + kOffRecs + 64 * (k % kRecs)); };
  int* s_info = reinterpret_cast<int*>(smem + kOffInfo);
  // [24] warp sums; 24: start of the cut jobs, CTAs, whole jobs of each (-1: all), first cut job, its start, last one, its start
  long long* s_scan = reinterpret_cast<long long*>(smem + kOffScan);
  uint16_t* s_order = reinterpret_cast<uint16_t*>(smem + kOffOrder);
  int* s_weight = reinterpret_cast<int*>(smem + kOffJoin);  // of the first kSorted tiles, here only
  long long* s_range = reinterpret_cast<long long*>(smem + kOffRange);  // [CTAs + 1] starts of the CTAs' ranges of the cut jobs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- prologue ------------------------------------------------------------------
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(kBFull + i), 1);
      mbar_init(bar(kBEmpty + i), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kBQFull + s), 1);
      mbar_init(bar(kBQEmpty + s), 1 + 4);  // the products, and the outputs that leave through the tiles
      mbar_init(bar(kBSFull + s), 1);
      mbar_init(bar(kBPFull + s), 4);
      mbar_init(bar(kBPvDone + s), 1);
      mbar_init(bar(kBOFree + s), 4);
      mbar_init(bar(kBMl + 2 * s), 4);
      mbar_init(bar(kBMl + 2 * s + 1), 4);
    }
    for (int i = 0; i < kRecs; ++i) {
      mbar_init(bar(kBRecFull + i), 1);
      mbar_init(bar(kBRecEmpty + i), 1 + 1 + 8 + 4);  // MMA, queries, softmax, outputs
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
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's range of the weighted jobs: (KV head, tile), tile fastest ------------------
  const int n_tiles = *p.n_tiles;
  {
    const int per = (n_tiles + kPrefillThreads - 1) / kPrefillThreads;
    const int t0 = min(tid * per, n_tiles), t1 = min(t0 + per, n_tiles);
    long long mine = 0;
    for (int t = t0; t < t1; ++t) mine += job_weight(p.tiles[t].n_pg);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    if (tid < kSorted) s_weight[tid] = (int)mine;
    __syncthreads();
    long long before = 0, one = 0;
    for (int i = 0; i < kPrefillThreads / 32; ++i) {
      if (i < warp) before += s_scan[i];
      one += s_scan[i];
    }
    const long long total = kKvHeads * one;
    const int n_jobs = kKvHeads * n_tiles, G = (int)min((long long)gridDim.x, max(1ll, quot(total, kLeast)));
    const long long quota = quot(total, G);
    auto weight = [&](int job) { return job_weight(p.tiles[job % n_tiles].n_pg); };
    // Whole jobs c, c + G, ... of CTA c: as many rounds as leave every CTA a share of the cut ones
    int whole = total > 0 ? n_jobs / G : 0;
    long long w = 0;
    if (tid < G)
      for (int i = 0; i < whole; ++i) w += weight(tid + i * G);
    const int rest = tid < G && tid + whole * G < n_jobs ? weight(tid + whole * G) : 0;
    // None is cut if all of them, dealt like that, leave no CTA with more than an equal share and kCut, or if a
    // queue of them, heaviest first (or last tile first), does: a job begins when those before it, S in all, are
    // out of the queue, at S / G or earlier
    bool late = false;
    auto begins_late = [&](long long ahead, int w) { return kKvHeads * ahead + (kKvHeads - 1 + G) * (long long)w > G * (quota + kCut); };
    if (n_jobs > G && n_tiles <= kSorted) {
      if (tid < n_tiles) {
        const int own = (int)mine;
        int rank = 0, ahead = 0;
        for (int i = 0; i < n_tiles; i += 4) {
          const int4 v = *reinterpret_cast<const int4*>(s_weight + i);
          const int u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i + j < n_tiles && (u[j] > own || (u[j] == own && i + j > tid))) {
              ++rank;
              ahead += u[j];
            }
        }
        s_order[rank] = (uint16_t)tid;
        late = begins_late(ahead, own);
      }
    } else {
      long long upto_t = before + incl - mine;
      for (int t = t0; t < t1; ++t) {
        const int w = job_weight(p.tiles[t].n_pg);
        upto_t += w;
        late |= begins_late(one - upto_t, w);
      }
    }
    const bool dealt = __syncthreads_or(w + rest > quota + kCut), cut = __syncthreads_or(late) && dealt;
    while (__syncthreads_or(whole > 0 && tid < G && w + kLeast > quota)) {
      --whole;
      if (tid < G) w -= weight(tid + whole * G);
    }
    // and what is left to each, of the jobs behind them
    long long left = total > 0 && tid < G ? quota + (tid < (int)(total - quota * G)) - w : 0, upto = left;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31 && warp < 8) s_scan[16 + warp] = upto;
    const int first_g = total > 0 ? whole * G / n_tiles : 0, first_t = total > 0 ? whole * G % n_tiles : 0;
    if (t0 <= first_t && first_t < t1) {
      long long x = first_g * one + before + incl - mine;
      for (int t = t0; t < first_t; ++t) x += job_weight(p.tiles[t].n_pg);
      s_scan[24] = x;
    }
    __syncthreads();
    for (int i = 0; i < warp && i < 8; ++i) upto += s_scan[16 + i];
    if (tid <= G && tid <= kPrefillCtas) s_range[tid] = s_scan[24] + upto - left;
    if (tid == 0) {
      s_scan[25] = total == 0 ? 0 : cut ? G : min(G, n_jobs);
      s_scan[26] = cut ? whole : -1;
    }
    __syncthreads();
    if (total > 0 && cut && (int)blockIdx.x < G) {
      // the jobs that hold the first and the last weight of the CTA's range, if they are among this thread's tiles
#pragma unroll 1
      for (int end = 0; end < 2; ++end) {
        const long long at = s_range[blockIdx.x + end] - end;
        const int g = (int)quot(at, one);
        const long long in = at - g * one;
        long long x = before + incl - mine;
        if (mine > 0 && in >= x && in < x + mine) {
          int t = t0;
          for (;; ++t) {
            const int w = job_weight(p.tiles[t].n_pg);
            if (in < x + w) break;
            x += w;
          }
          s_scan[27 + 2 * end] = (long long)g << 32 | t;
          s_scan[28 + 2 * end] = at - in + x;
        }
      }
    }
    __syncthreads();
  }
  const int G = (int)s_scan[25], whole = (int)s_scan[26];
  const bool idle = (int)blockIdx.x >= G;

  // registers: 128 threads x 64 + 256 x 160 + 128 x 128 of the launch's 512 x 128
  // (the longest loop's code first: 100 tokens 17 us, 18 behind the others')
  if (warp >= 4 && warp < 12) {
    regs_inc<160>();
    // ---------------- softmax: set = (warp - 4) / 4, row = TMEM lane ------------------------------------
    const int set = (warp - 4) >> 2, quad = warp & 3, lrow = 32 * quad + lane;
    const uint32_t t_s = tmem + ((uint32_t)(32 * quad) << 16) + kTmemS + 128 * set, t_o = t_s + kTmemO - kTmemS;
    const uint64_t scale2 = pair64(__float_as_uint(p.scale_log2), __float_as_uint(p.scale_log2));
    uint32_t e = 0, par = 0, segs = 0;  // pages so far, parity of this set's jobs, its segments
    for (int k = 0;; ++k) {
      if (!swait(bar(kBRecFull + k % kRecs), (k / kRecs) & 1, wc)) break;
      const SegRec r = *rec(k);
      __syncwarp();
      if (r.n_pg < 0) break;
      if (lane == 0) mbar_arrive(bar(kBRecEmpty + k % kRecs));
      if (set == 1 && r.n_tok <= 32) {
        e += r.n_pg;
        continue;
      }
      const int token = 32 * set + (lrow >> 2);
      const bool busy = 32 * set + 8 * quad < r.n_tok, mine = token < r.n_tok;
      // keys that the row sees, counted from the first one of the page
      int start = 0, end = 0x7FFFFFFF;
      if (mine) {
        const int pos = r.pos + token;
        start = (p.window ? max(0, pos + 1 - p.window) : 0) - r.page0 * kPageTokens;
        end = (p.ends ? min(max(p.ends[r.q0 + token], 0), r.len) : pos + 1) - r.page0 * kPageTokens;
      }
      // (a row that sees nothing is weighed as if it saw all, so that its warp's pages need no masks; its sum is 0)
      const bool none = end <= start;
      if (none) {
        start = 0;
        end = 0x7FFFFFFF;
      }
      float shift = kUnset, l = 0.f;  // kBias less the reference, and the sum of weights
      bool ok = true;
      for (const uint32_t e0 = e; e - e0 < (uint32_t)r.n_pg; ++e) {
        if (!swait(bar(kBSFull + set), par, wc)) {
          ok = false;
          break;
        }
        par ^= 1;
        if (busy) {
          tc_fence_after();
          const int hi = s_info[e % kInfo] ? end : 0;
          if (__any_sync(0xffffffffu, start > 0 || hi < kPageTokens)) {  // -inf where the row does not see the token
#pragma unroll 1
            for (int c = 0; c < kPageTokens; c += 32) {
              uint32_t v[32];
              const uint32_t vis = low_bits(hi - c) & ~low_bits(start - c);
              if (__all_sync(0xffffffffu, vis == 0xFFFFFFFFu)) continue;
              tmem_ld32x32b_x32(t_s + c, v);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 32; ++x) v[x] = vis >> x & 1 ? v[x] : 0xFF800000u;
              tmem_st32(t_s + c, v);
            }
            tmem_wait_st();
          }
          // Half a page at a time, the next 32 scores loaded under the exponentials of 32.  There is no pass
          // for the maximum: 64 weights that sum to 49,152 or less have none above it, and others (a
          // row's first ones: its shift is kUnset) move the reference and are weighed again.
          uint32_t v[2][32];
          tmem_ld32x32b_x32(t_s, v[0]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t shift2 = pair64(__float_as_uint(shift), __float_as_uint(shift));
            uint64_t sums[2] = {0, 0};
            uint32_t o[32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              wait_ld32(v[c]);
              if (h + c < 2) tmem_ld32x32b_x32(t_s + 64 * h + 32 * c + 32, v[(c + 1) & 1]);
              weigh32(v[c], scale2, shift2, sums, o + 16 * c);
            }
            const uint2 sum2 = split64(add_f32x2(sums[0], sums[1]));
            float sum = __uint_as_float(sum2.x) + __uint_as_float(sum2.y);
            const bool over = mine && sum > kMost;
            if (__any_sync(0xffffffffu, over)) {
              // (S of this half is as it was; the other half's load may be under way)
              wait_ld32(v[0]);
              float top = -INFINITY;
#pragma unroll 1
              for (int c = 0; c < 64; c += 16) {
                uint32_t u[16];
                tmem_ld32x32b_x16(t_s + 64 * h + c, u);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 16; ++x) top = fmaxf(top, __uint_as_float(u[x]));
              }
              float f = 1.f;
              if (over) {
                const float next = kBias - top * p.scale_log2;
                f = fast_exp2(next - shift);  // (0 for the first: shift is kUnset)
                shift = next;
                l *= f;
              }
              __syncwarp();
              if (e != e0) scale_acc(t_o, f);  // (the PVs before this S are done)
              if (h) scale_p(t_s, f);
              const uint64_t again2 = pair64(__float_as_uint(shift), __float_as_uint(shift));
              sums[0] = sums[1] = 0;
#pragma unroll 1
              for (int c = 0; c < 64; c += 32) {
                uint32_t u[32], y[16];
                tmem_ld32x32b_x32(t_s + 64 * h + c, u);
                tmem_wait_ld();
                weigh32(u, scale2, again2, sums, y);
                tmem_st_x16(t_s + 64 * h + c, y);
              }
              const uint2 again = split64(add_f32x2(sums[0], sums[1]));
              sum = __uint_as_float(again.x) + __uint_as_float(again.y);
            } else {
              tmem_st_x16(t_s + 64 * h, o);
              tmem_st_x16(t_s + 64 * h + 32, o + 16);
            }
            l += sum;
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBPFull + set));
        start -= kPageTokens;
        if (mine && !none) end -= kPageTokens;
      }
      if (!ok) break;
      reinterpret_cast<float2*>(smem + kOffMl)[256 * set + 128 * (segs & 1) + lrow] = make_float2(kBias - shift, none ? 0.f : l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBMl + 2 * set + (segs & 1)));
      ++segs;
    }
  } else if (warp < 4) {
    regs_dec<64>();
    if (warp == 0) {
      // ---------------- segment records and page copies -------------------------------------
      int e = 0, k = 0;
      bool ok = true;
      if (!idle) {
        const long long lo = s_range[blockIdx.x], hi = s_range[blockIdx.x + 1];
        auto tile = [&](int t) {
          const int word = lane < 8 ? reinterpret_cast<const int*>(p.tiles + t)[lane] : 0;
          TileRec r;
          r.q0 = __shfl_sync(0xffffffffu, word, 0);
          r.n_tok = __shfl_sync(0xffffffffu, word, 1);
          r.pos = __shfl_sync(0xffffffffu, word, 2);
          r.len = __shfl_sync(0xffffffffu, word, 3);
          r.page0 = __shfl_sync(0xffffffffu, word, 4);
          r.n_pg = __shfl_sync(0xffffffffu, word, 5);
          r.ws_page = __shfl_sync(0xffffffffu, word, 6);
          return r;
        };
        // the pages a .. z - 1 of a tile and KV head
        auto segment = [&](const TileRec& r, int t, int g, int a, int z, int c0, int parts) {
          if (!twait(bar(kBRecEmpty + k % kRecs), ((k / kRecs) & 1) ^ 1, wc)) return false;
          if (lane == 0) {
            SegRec* s = rec(k);
            s->n_pg = z - a;
            s->g = g;
            s->q0 = r.q0;
            s->n_tok = r.n_tok;
            s->pos = r.pos;
            s->len = r.len;
            s->page0 = r.page0 + a;
            s->part = (int)blockIdx.x - c0;
            s->parts = parts;
            s->c0 = c0;
            s->job = t * kKvHeads + g;
            const int most = whole > 0 ? kInline : kAlone;
            s->join = parts > 1 && parts <= most;
            if (parts > most && a == 0) p.big[atomicAdd(p.n_big, 1)] = make_int2(s->job, c0 | parts << 8);
            mbar_arrive(bar(kBRecFull + k % kRecs));
          }
          __syncwarp();
          ++k;
          const uint8_t* image = p.images + ((size_t)(r.ws_page + a) * kKvHeads + g) * kImage;
          for (int i0 = a; i0 < z; i0 += 32) {
            const int cnt = min(32, z - i0);
            const int there = lane < cnt ? p.page_ok[r.ws_page + i0 + lane] : 0;
            for (int j = 0; j < cnt; ++j, ++e, image += kKvHeads * kImage) {
              const int st = e % kStages, ph = ((e / kStages) & 1) ^ 1, good = __shfl_sync(0xffffffffu, there, j);
              if (!twait(bar(kBEmpty + st), ph, wc)) return false;
              if (lane == 0) {
                s_info[e % kInfo] = good;
                if (!(p.inject && e == 0)) {
                  mbar_arrive_expect_tx(bar(kBFull + st), kImage);
                  bulk_g2s(sbase + kOffK + st * kImage, image, kImage, bar(kBFull + st));
                }
                *s_issued = e + 1;
              }
              __syncwarp();
            }
          }
          return true;
        };
        auto owner = [&](long long x) {  // the CTA whose range holds a weight
          int c = 0;
          for (int step = 128; step; step >>= 1)
            if (c + step < G && s_range[c + step] <= x) c += step;
          return c;
        };
        // The range of jobs that are cut comes first, and of these the one that goes on in the next CTA's
        // range: the parts' rows are then written and joined under whole jobs.
        long long early = -1;
#pragma unroll 1
        for (int pass = whole < 0 ? 2 : 0; pass < 3; ++pass) {
          const bool cut = pass < 2;
          int x = (int)blockIdx.x;  // place in the queue
          long long off = cut ? s_scan[pass ? 28 : 30] : 0;
          int g = (int)(s_scan[pass ? 27 : 29] >> 32), t = (int)s_scan[pass ? 27 : 29];
          for (int i = 0; ok && (cut ? off < hi && g < kKvHeads : whole < 0 ? x < kKvHeads * n_tiles : i < whole); ++i) {
            if (!cut) {
              const int job = (int)blockIdx.x + i * G;
              g = whole < 0 ? x % kKvHeads : job / n_tiles;
              t = whole >= 0 ? job % n_tiles : kKvHeads * n_tiles > G && n_tiles <= kSorted ? s_order[x / kKvHeads] : n_tiles - 1 - x / kKvHeads;
            }
            const TileRec r = tile(t);
            // page i starts at weight base + i kPageWeight; it belongs to the range that holds its start
            const long long base = off + kFixed;
            auto page_at = [&](long long x) {  // the first page that starts at weight x or behind it
              if (x <= base) return 0;
              return x - base > (long long)r.n_pg * kPageWeight ? r.n_pg : ((int)(x - base) + kPageWeight - 1) / kPageWeight;
            };
            const int a = cut && r.n_pg > 0 ? page_at(lo) : 0, z = cut && r.n_pg > 0 ? page_at(hi) : r.n_pg;
            const bool take = a < z && (pass ? !cut || off != early : z < r.n_pg);
            if (take) {
              if (pass == 0) early = off;
              const int c0 = cut ? owner(base) : (int)blockIdx.x;
              ok = segment(r, t, g, a, z, c0, cut ? owner(base + (long long)(r.n_pg - 1) * kPageWeight) - c0 + 1 : 1);
            }
            if (whole < 0) x = G + __shfl_sync(0xffffffffu, lane == 0 ? atomicAdd(p.next, 1) : 0, 0);
            off += job_weight(r.n_pg);
            if (++t == n_tiles) {
              t = 0;
              ++g;
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
      // For each page and row tile PV, then the tile's next QK into the same columns (the next segment's
      // first one behind the last); so one tile's products run under the other's softmax.  The warp stays
      // together and elects a lane for the MMAs only (in a loop that one lane runs alone nothing is
      // warp-uniform, and an MMA takes three times as long to issue).
      const uint32_t idesc_qk = umma_idesc_e4m3(128, 128);
      // D fp32, A and B f16, A K-major, B MN-major
      const uint32_t idesc_pv = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
      // K-major without swizzle: 8 tokens x 16 channels are 128 contiguous bytes, the next 16 channels
      // 2,048 further.  MN-major without swizzle: 8 tokens x 8 channels are 128 contiguous bytes, the
      // next 8 tokens follow, the next 8 channels are 2,048 further
      const uint64_t kdesc0 = umma_desc_noswz_lbo_sbo(sbase + kOffK, 2048, 128);
      const uint64_t vdesc0 = umma_desc_noswz_lbo_sbo(sbase + kOffK + kImageK, 128, 2048);
      const uint64_t qdesc0 = umma_desc_sw128(sbase + kOffQ);
      // (inside an elected lane)
      auto pv = [&](int set, int stage, uint32_t acc) {
        const uint32_t s = tmem + kTmemS + 128 * set;
        const uint64_t vdesc = vdesc0 + stage * (kImage >> 4);
#pragma unroll 4
        for (int kk = 0; kk < 8; ++kk, acc = 1)  // 16 tokens each: 8 columns of P inside S's 32-column chunks
          umma_f16_ts(s + kTmemO - kTmemS, s + 32 * (kk >> 1) + 8 * (kk & 1), vdesc + kk * (256 >> 4), idesc_pv, acc);
      };
      auto qk = [&](int set, int stage, int k) {
        const uint32_t s = tmem + kTmemS + 128 * set;
        const uint64_t qdesc = qdesc0 + (2 * (k & 1) + set) * (16384 >> 4), kdesc = kdesc0 + stage * (kImage >> 4);
#pragma unroll 2
        for (int kk = 0; kk < 4; ++kk)  // 32 channels each
          umma_e4m3(s, qdesc + 2 * kk, kdesc + kk * (4096 >> 4), idesc_qk, kk > 0);
        umma_commit(bar(kBSFull + set));
      };
      uint32_t p_par = 0, o_par = 0, o_any = 0;  // bit per set: parity of its next P, of its segments, whether it had one
      int st = kStages - 1, full = 0;            // stage of the page whose P is awaited; parity of the next one's stage
      int n_pg = 0, sets = 0;                    // the segment
      bool ok = true;
      for (int k = -1; ok;) {
        // all pages but the last (a short loop: a long way round the warp's code misses the instruction cache,
        // which the softmax's code fills: 2,420 cycles a page, 2,800 with the segment's end in the loop)
        uint32_t acc = 0;
        for (int i = 1; i < n_pg; ++i, acc = 1) {
          const int next = st == kStages - 1 ? 0 : st + 1;
          if (!swait(bar(kBFull + next), full, wc)) {
            ok = false;
            break;
          }
          for (int set = 0; set < sets; ++set) {
            if (!swait(bar(kBPFull + set), p_par >> set & 1, wc)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (elect_one()) {
              pv(set, st, acc);
              if (set == sets - 1) umma_commit(bar(kBEmpty + st));
              qk(set, next, k);
            }
            __syncwarp();
          }
          if (!ok) break;
          p_par ^= sets == 2 ? 3u : 1u;
          st = next;
          full ^= next == kStages - 1;
        }
        if (!ok) break;
        // the last one, and the next segment's first
        if (!swait(bar(kBRecFull + (k + 1) % kRecs), ((k + 1) / kRecs) & 1, wc)) break;
        const int next_pg = __shfl_sync(0xffffffffu, rec(k + 1)->n_pg, 0);
        const int next_sets = next_pg < 0 ? 0 : __shfl_sync(0xffffffffu, rec(k + 1)->n_tok, 0) > 32 ? 2 : 1;
        const int next = st == kStages - 1 ? 0 : st + 1;
        if (next_sets) {
          if (lane == 0) mbar_arrive(bar(kBRecEmpty + (k + 1) % kRecs));
          if (!swait(bar(kBQFull + ((k + 1) & 1)), ((k + 1) >> 1) & 1, wc) || !swait(bar(kBFull + next), full, wc)) break;
        }
#pragma unroll 1
        for (int set = 0; set < max(sets, next_sets); ++set) {
          if (set < sets && !swait(bar(kBPFull + set), p_par >> set & 1, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            if (set < sets) {
              pv(set, st, acc);
              umma_commit(bar(kBPvDone + set));
              if (set == sets - 1) {
                umma_commit(bar(kBEmpty + st));
                umma_commit(bar(kBQEmpty + (k & 1)));
              }
            }
            if (set < next_sets) qk(set, next, k + 1);
          }
          __syncwarp();
        }
        if (!ok || !next_sets) break;
        const uint32_t had = sets == 2 ? 3u : (uint32_t)sets, has = next_sets == 2 ? 3u : 1u;
        p_par ^= had;
        o_par ^= had;
        o_any |= had;
        ++k;
        n_pg = next_pg;
        sets = next_sets;
        st = next;
        full ^= next == kStages - 1;
        // (the first PVs write over accumulators that have to be read)
        for (int set = 0; set < 2 && ok; ++set)
          if ((has & o_any) >> set & 1) ok = swait(bar(kBOFree + set), (o_par >> set & 1) ^ 1, wc);
      }
      __syncwarp();
      if (elect_one()) umma_commit(bar(kBDone));
      __syncwarp();
    } else if (warp == 2) {
      // ---------------- query rows of a segment: row 4 i + h of token i, head 4 g + h -----------------
      for (int k = 0;; ++k) {
        if (!twait(bar(kBRecFull + k % kRecs), (k / kRecs) & 1, wc)) break;
        const SegRec r = *rec(k);
        __syncwarp();
        if (r.n_pg < 0) break;
        if (lane == 0) mbar_arrive(bar(kBRecEmpty + k % kRecs));
        if (k > 1 && !twait(bar(kBQEmpty + (k & 1)), ((k >> 1) - 1) & 1, wc)) break;
        for (int x = lane; x < r.n_tok * 32; x += 32) {
          const int row = x >> 3, c = x & 7;
          const uint8_t* src = p.q + ((size_t)(r.q0 + (row >> 2)) * kQHeads + kGqa * r.g + (row & 3)) * kHeadDim + 16 * c;
          cp_async16(sbase + kOffQ + (k & 1) * 32768 + row * 128 + ((c ^ (row & 7)) << 4), src);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBQFull + (k & 1)));
      }
    }
  } else {
    // ---------------- outputs: the rows of a finished segment, one set after the other, while the softmax
    // warps are at the next.  They leave through shared memory (the segment's query tiles, which are of no
    // use any more) by bulk copies: stores of the threads themselves take an SM 4,000 cycles for a tile,
    // and hold up every other access to shared memory, barriers among them. -------------------------------
    const int quad = warp & 3, lrow = 32 * quad + lane;
    uint32_t seg[2] = {0, 0};  // segments of each set
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!swait(bar(kBRecFull + k % kRecs), (k / kRecs) & 1, wc)) break;
      const SegRec r = *rec(k);
      __syncwarp();
      if (r.n_pg < 0) break;
      if (lane == 0) mbar_arrive(bar(kBRecEmpty + k % kRecs));
      const uint32_t stage = sbase + kOffQ + (k & 1) * 32768 + quad * 8192;
#pragma unroll
      for (int set = 0; set < 2; ++set) {
        if (set == 1 && r.n_tok <= 32) continue;
        const uint32_t n = seg[set]++;
        if (!ok || !swait(bar(kBMl + 2 * set + (n & 1)), n >> 1 & 1, wc) || !swait(bar(kBPvDone + set), n & 1, wc)) {
          ok = false;
          continue;
        }
        const uint32_t t_o = tmem + ((uint32_t)(32 * quad) << 16) + kTmemO + 128 * set;
        const int tok0 = 32 * set + 8 * quad;  // the warp's first token
        const float2 own = reinterpret_cast<const float2*>(smem + kOffMl)[256 * set + 128 * (n & 1) + lrow];
        auto freed = [&] {  // the accumulator is read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBOFree + set));
        };
        tc_fence_after();
        if (tok0 >= r.n_tok) {
          freed();
        } else if (r.parts > 1) {
          put_part(p, r, own, tok0, lane, t_o, stage, freed);
        } else {
          const float inv = own.y != 0.f ? p.out_scale / own.y : 0.f;  // (a NaN of the query stays one)
          if (lane == 0) bulk_read_wait();
          __syncwarp();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            __syncwarp();  // (lanes part ways in put32: tensor memory is read by whole warps)
            tmem_ld32x32b_x32(t_o + 32 * c, v);
            wait_ld32(v);
            if (c == 3) freed();
            float o[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = own.y != 0.f ? __uint_as_float(v[x]) : 0.f;
            put32<false>(p, r, o, inv, c, tok0, lane, stage);
          }
          put_lse(p, r, own.x, own.y, tok0, lane);
        }
      }
      // (the tiles may be written again)
      if (lane == 0) {
        bulk_read_wait();
        mbar_arrive(bar(kBQEmpty + (k & 1)));
      }
      __syncwarp();
      if (ok && r.join)
#pragma unroll 1
        for (int set = 0; set < 2; ++set)
          if (32 * set + 8 * quad < r.n_tok) join_parts(p, r, 32 * set + 8 * quad, lane, sbase + kOffJoin + quad * 2048);
    }
    if (lane == 0) bulk_wait();
    __syncwarp();
  }

  // ---- teardown -------------------------------------------------------------------------
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    mbar_wait_drain(bar(kBDone), 0, drain_ns(p.wait_ns));  // every tcgen05.mma is done
    if (*s_abort) {
      set_status(p.status, MSA_STATUS_TIMEOUT);
      for (int e = max(p.inject ? 1 : 0, *s_issued - kStages); e < *s_issued; ++e)  // copies that may still be landing
        mbar_wait_drain(bar(kBFull + e % kStages), (e / kStages) & 1, drain_ns(p.wait_ns));
    }
  }
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- (3) jobs that were cut ---------------------------------------------------------------
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.  A unit is 32 rows of a job, lane = row; a warp takes
// 4 kChunks of its channels, kParts parts' loads at once.  Eight warps a unit with four parts at once keep more units
// going; where there are fewer units than CTAs (few tokens over a long context: many parts) sixteen warps
// with eight halve the chain of loads (two sequences of up to 64 tokens over 6,034: 34.7 us, 31.7).
constexpr int kMergeThreads = 512, kQuads = kGqa * kTileTokens / 32;
template <int kParts, int kChunks>
__device__ __forceinline__ void merge_unit(const PrefillParams& p, int u, int chunk0, int lane) {
  const int2 big = p.big[u / kQuads];
  const int t = big.x / kKvHeads, g = big.x % kKvHeads, quad = u % kQuads, c0 = big.y & 255, parts = big.y >> 8;
  const int q0 = p.tiles[t].q0, n_rows = kGqa * p.tiles[t].n_tok, row = 32 * quad + lane;
  if (32 * quad >= n_rows) return;
  float M = -INFINITY, L = 0.f, o[4 * kChunks] = {};
  for (int i0 = 0; i0 < parts; i0 += kParts) {
    float4 x[kParts][kChunks];
    float2 ml[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (i0 + i < parts) {
        const size_t at = (part_slot(c0, i0 + i) * p.part_quads + quad) * 32;
        ml[i] = p.part_ml[at + lane];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) x[i][c] = p.part_o[(at + chunk0 + c) * 32 + lane];
      }
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      if (ml[i].y != 0.f) top = fmaxf(top, ml[i].x);
    const float f = M > -INFINITY ? fast_exp2(M - top) : 0.f;
    M = top;
    L *= f;
#pragma unroll
    for (int c = 0; c < 4 * kChunks; ++c) o[c] *= f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      if (i0 + i >= parts) break;
      const float w = ml[i].y != 0.f ? fast_exp2(ml[i].x - top) : 0.f;
      L = fmaf(ml[i].y, w, L);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        o[4 * c] = fmaf(x[i][c].x, w, o[4 * c]);
        o[4 * c + 1] = fmaf(x[i][c].y, w, o[4 * c + 1]);
        o[4 * c + 2] = fmaf(x[i][c].z, w, o[4 * c + 2]);
        o[4 * c + 3] = fmaf(x[i][c].w, w, o[4 * c + 3]);
      }
    }
  }
  if (row >= n_rows) return;
  const float inv = L != 0.f ? p.out_scale / L : 0.f;  // (a NaN of the query stays one)
  const size_t at = (size_t)(q0 + (row >> 2)) * kQHeads + kGqa * g + (row & 3);
#pragma unroll
  for (int h = 0; h < kChunks / 2; ++h) {
    uint32_t y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = pack16(o[8 * h + 2 * c] * inv, o[8 * h + 2 * c + 1] * inv, p.out_f16);
    *reinterpret_cast<uint4*>(p.out + at * kHeadDim + 4 * chunk0 + 8 * h) = make_uint4(y[0], y[1], y[2], y[3]);
  }
  if (p.lse && chunk0 == 0) p.lse[at] = L != 0.f ? (M - kBias + log2f(L)) * kLn2 : -INFINITY;
}
__global__ void __launch_bounds__(kMergeThreads) prefill_merge_kernel(const __grid_constant__ PrefillParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  const int units = *p.n_big * kQuads;
  if (units <= (int)gridDim.x) {
    if ((int)blockIdx.x < units) merge_unit<8, 2>(p, blockIdx.x, 2 * warp, lane);
  } else {
    for (int u = 2 * blockIdx.x + (warp >> 3); u < units; u += 2 * gridDim.x) merge_unit<4, 4>(p, u, 4 * (warp & 7), lane);
  }
}

int prefill_quads(int n_q_total) { return (kGqa * std::min(n_q_total, kTileTokens) + 31) / 32; }
int prefill_tiles(int n_q_total, int n_seqs) { return n_q_total / kTileTokens + std::min(n_q_total, n_seqs); }
bool make_out_map(CUtensorMap* m, void* out, int n_q_total, cuuint32_t channels) {
  const auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {kHeadDim, kQHeads, (cuuint64_t)n_q_total};
  const cuuint64_t strides[2] = {kHeadDim * 2, kQHeads * kHeadDim * 2};
  const cuuint32_t box[3] = {channels, kGqa, 8}, steps[3] = {1, 1, 1};
  // (16-bit words whatever their type)
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, out, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
            channels == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
size_t padded(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t prefill_workspace_bytes(int n_q_total, int n_seqs, int n_pages) {
  const size_t quads = prefill_quads(n_q_total), tiles = prefill_tiles(n_q_total, n_seqs);
  return 256 + padded(tiles * sizeof(TileRec)) + padded(tiles * kKvHeads * sizeof(int2)) + padded(tiles * 32 * sizeof(int)) + padded((size_t)n_pages * sizeof(int)) +
         padded(2 * kPrefillCtas * quads * 32 * sizeof(float2)) + 2 * kPrefillCtas * quads * 32 * kHeadDim * sizeof(float) +
         (size_t)n_pages * kKvHeads * kImage;
}

cudaError_t launch_prefill_attn(const msa_cache* c, const uint8_t* q, float softmax_scale, const int* block_table,
                                int max_pages, const int* seq_lens, const int* q_start_loc, int n_seqs, int n_q_total,
                                int window, const int* ends, int n_visited, int dtype, void* out, float* lse, void* ws,
                                cudaStream_t stream) {
  if (n_q_total == 0 || n_seqs == 0) return cudaSuccess;
  static DeviceSetup setup;
  int dev = 0, n_sm = 0;
  const int conv_smem = kConvTables + 2 * (n_seqs + 1) * (int)sizeof(int);
  cudaError_t e = setup.get(&dev, &n_sm, [](int) {
    constexpr auto kMax = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const cudaError_t e = cudaFuncSetAttribute(prefill_attn_kernel, kMax, kPrefillSmem);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(prefill_convert_kernel, kMax, kConvTables + 2 * (kMaxSeqs + 1) * (int)sizeof(int));
  });
  if (e != cudaSuccess) return e;
  PrefillParams pp{};
  pp.kv_pool = static_cast<const uint8_t*>(c->kv_pool);
  pp.n_pages = c->n_pages;
  pp.q = q;
  pp.block_table = block_table;
  pp.max_pages = max_pages;
  pp.seq_lens = seq_lens;
  pp.q_start_loc = q_start_loc;
  pp.n_seqs = n_seqs;
  pp.n_q_total = n_q_total;
  pp.window = window;
  pp.ends = ends;
  // (a quotient below fp32's normal numbers is as good as the smallest: every score is zero then)
  pp.scale_log2 = std::max(softmax_scale / c->s_enc_k * kLog2e, FLT_MIN);
  pp.out_scale = 256.0f / c->s_enc_v;
  pp.out_f16 = dtype == MSA_DTYPE_F16;
  pp.out = static_cast<uint16_t*>(out);
  if (!make_out_map(&pp.out_map, out, n_q_total, 64) || !make_out_map(&pp.out_map32, out, n_q_total, 32)) return cudaErrorInvalidValue;
  pp.lse = lse;
  pp.part_quads = prefill_quads(n_q_total);
  pp.max_tiles = prefill_tiles(n_q_total, n_seqs);
  pp.cap = n_visited;
  uint8_t* w = static_cast<uint8_t*>(ws);
  auto piece = [&](size_t bytes) {
    uint8_t* at = w;
    w += padded(bytes);
    return at;
  };
  pp.n_tiles = reinterpret_cast<int*>(piece(256));
  pp.n_big = pp.n_tiles + 1;
  pp.next = pp.n_tiles + 2;
  pp.tiles = reinterpret_cast<TileRec*>(piece(pp.max_tiles * sizeof(TileRec)));
  pp.big = reinterpret_cast<int2*>(piece((size_t)pp.max_tiles * kKvHeads * sizeof(int2)));
  pp.tickets = reinterpret_cast<int*>(piece((size_t)pp.max_tiles * 32 * sizeof(int)));
  pp.page_ok = reinterpret_cast<int*>(piece((size_t)pp.cap * sizeof(int)));
  pp.part_ml = reinterpret_cast<float2*>(piece(2 * kPrefillCtas * (size_t)pp.part_quads * 32 * sizeof(float2)));
  pp.part_o = reinterpret_cast<float4*>(piece(2 * kPrefillCtas * (size_t)pp.part_quads * 32 * kHeadDim * sizeof(float)));
  pp.images = w;
  pp.status = c->status;
  pp.wait_ns = launch_settings().wait_ns;
  pp.inject = (launch_settings().inject & MSA_INJECT_ATTENTION_TIMEOUT) != 0;
  const long long units = (long long)n_visited * kKvHeads;
  const int conv_grid = (int)std::max(1ll, std::min(units, 5ll * n_sm));
  e = launch_pdl(prefill_convert_kernel, dim3(conv_grid), dim3(kConvThreads), conv_smem, stream, pp);
  if (e != cudaSuccess) return e;
  e = launch_pdl(prefill_attn_kernel, dim3(std::min(n_sm, kPrefillCtas)), dim3(kPrefillThreads), kPrefillSmem, stream, pp);
  if (e != cudaSuccess) return e;
  // (a job has no more parts than pages)
  if (n_visited <= kAlone) return cudaSuccess;
  return launch_pdl(prefill_merge_kernel, dim3(2 * std::min(n_sm, kPrefillCtas)), dim3(kMergeThreads), 0, stream, pp);
}

}  // namespace msa
