/*
 * msa.h -- C ABI of the block-sparse attention decode path over an NVFP4 KV cache
 * (library libmsa.so, built for sm_103a).
 *
 * What the path computes (sources: "vLLM Delivers Day-0 Support for
 * MiniMax-M3.1-Flash", yuxiaoba.github.io, sections "Sparse attention still
 * scans an index" and "Capacity savings must pay for conversion"; ai4snews
 * article on MiniMax-M3.1-Flash in vLLM, first and third paragraphs;
 * kongchang.com article, "NVFP4 KV Cache and MoE Weights"):
 *   - the KV cache lives in 128-token blocks (pages), K and V stored as NVFP4:
 *     E2M1 values with one E4M3 scale per 16 channels and an fp32 per-tensor
 *     encode scale;
 *   - a lightweight indexer scores every cached token from FP8 index keys
 *     (128 bytes per token), score(t) = sum_h w_h * ReLU(q_h . k_idx(t)),
 *     takes the max per block, keeps the top-16 blocks (ties to the lower block
 *     index) and always the most recent block;
 *   - exact GQA attention (16 query heads over 4 KV heads, head dim 128) runs
 *     over the selected tokens only, FP8 E4M3 queries against K/V dequantised
 *     from NVFP4 to FP8, with an fp32 online softmax split over the context and
 *     merged by log-sum-exp.
 *
 * Conventions shared by every entry point:
 *   - Pointers are DEVICE pointers unless a parameter says "host".  The library
 *     never allocates, frees or synchronises (msa_read_status excepted); all
 *     work is enqueued on `stream` (a cudaStream_t; NULL = legacy stream).
 *   - Return value: MSA_OK (0) when the work was enqueued, or a negative
 *     MSA_ERR_* code when host-side validation failed (nothing is enqueued).
 *   - Data errors that only the device can see (a physical page id outside the
 *     pool, a sequence with more query tokens than cached tokens, ...) OR a
 *     MSA_STATUS_* bit into the cache's device status word; the offending item
 *     is skipped.  No kernel traps, asserts or waits without a bound.
 *   - Supported shape: 128-token pages, 4 KV heads, head dim 128, index dim
 *     128, 8 indexer heads, 16 query heads (GQA group 4).  Anything else is
 *     MSA_ERR_UNSUPPORTED_SHAPE.
 *
 * Page formats (one physical page id p addresses both pools):
 *   KV page p at kv_pool + p * 73,728 bytes = 4 heads x 18,432 bytes; head g
 *   at offset g * 18,432:
 *     +0       K codes  [128 tokens][64 B]: little-endian 32-bit word i of a
 *              row holds channels 8i..8i+7 as E2M1 codes (sign s, magnitude m):
 *              m of channel 8i+n at bits 4n..4n+2 (n = 0..7), s of channel 8i+n
 *              at bit 8n+7 and s of channel 8i+4+n at bit 8n+3 (n = 0..3); the
 *              16-byte chunk c (channels 32c..32c+31) of token t is stored at
 *              chunk position c XOR ((t >> 1) mod 4) of its row
 *     +8,192   K scales [8 groups][128 tokens]: E4M3 scale of channels 16k..16k+15
 *     +9,216   V codes  [128 tokens][64 B], chunks placed like the K codes
 *     +17,408  V scales [8 groups][128 tokens]
 *   (576 bytes per token and layer: the 34,560 bytes/token of the ai4snews
 *   article over the model's layers.)
 *   Index page p at idx_pool + p * 16,384 bytes = [128 tokens][128 B] E4M3
 *   index keys; the 16-byte chunk c of token t's row (dims 16c..16c+15) is
 *   stored at chunk position c XOR (t mod 8).
 *
 * Sequences and query tokens: sequence b has seq_lens[b] cached tokens (the
 * new query tokens already inserted) and q_start_loc[b+1] - q_start_loc[b]
 * query tokens; query token j of b sits at position
 * pos_j = seq_lens[b] - n_q + j, sees keys at positions <= pos_j, and its
 * recent block is r_j = pos_j / 128.  block_table[b * max_pages + i] is the
 * physical page of logical block i of sequence b.
 */
#ifndef MSA_H
#define MSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* msa_stream_t; /* same type as cudaStream_t */

/* Host-side return codes. */
#define MSA_OK 0
#define MSA_ERR_INVALID_ARG (-1)      /* null pointer, negative size, ... */
#define MSA_ERR_UNSUPPORTED_SHAPE (-2)
#define MSA_ERR_WORKSPACE_TOO_SMALL (-3)
#define MSA_ERR_LAUNCH_FAILED (-4)    /* a kernel launch returned an error */
#define MSA_ERR_SCRATCH_CAPACITY (-5) /* msa_indexer_topk_noalloc: shape beyond its static scratch */

/* Bytes of the static scratch behind msa_indexer_topk_noalloc. */
#define MSA_INDEXER_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)

/* Sticky device status bits (OR-ed into *msa_cache.status). */
#define MSA_STATUS_BAD_SLOT 0x1       /* slot_mapping points outside the pool */
#define MSA_STATUS_BAD_PAGE 0x2       /* block_table entry outside the pool */
#define MSA_STATUS_BAD_SEQ 0x4        /* n_q < 0, n_q > seq_len or seq_len > max_pages*128 */
#define MSA_STATUS_BAD_SELECTION 0x8  /* a selected block id outside 0..r_j */
#define MSA_STATUS_TIMEOUT 0x10       /* a bounded on-chip wait gave up (results invalid) */
#define MSA_STATUS_NO_PAGES 0x20      /* a page pool ran out of free pages */
/* Every on-chip wait is bounded (2 s by default): a wait that runs out sets
 * MSA_STATUS_TIMEOUT, the kernel abandons its work, waits (bounded) for its own
 * copies and tensor-core operations in flight, releases tensor memory and
 * returns.  The context stays usable. */

/* The KV cache and its metadata.  Caller-owned; the library only reads it.  Both
 * pools begin on 16-byte boundaries: a call whose kernels would meet a misaligned
 * address returns MSA_ERR_INVALID_ARG. */
typedef struct msa_cache {
  void* kv_pool;        /* device, n_pages * 73,728 bytes (format above), 16-byte aligned */
  void* idx_pool;       /* device, n_pages * 16,384 bytes (format above), 16-byte aligned */
  int64_t n_pages;      /* physical pages in both pools */
  int32_t page_tokens;  /* must be 128 */
  int32_t n_kv_heads;   /* must be 4 */
  int32_t head_dim;     /* must be 128 */
  int32_t idx_dim;      /* must be 128 */
  float s_enc_k;        /* host value: fp32 per-tensor encode scale of K, > 0 */
  float s_enc_v;        /* host value: fp32 per-tensor encode scale of V, > 0 */
  int32_t* status;      /* device int32, sticky MSA_STATUS_* bits; may be NULL */
} msa_cache;

/*
 * Quantise new tokens to NVFP4 / FP8 and write them into their cache slots.
 * (NVFP4 KV cache: ai4snews article, first and third paragraphs; index keys of
 * 128 FP8 bytes per token: blog, "Sparse attention still scans an index".)
 *
 *   k, v         fp32 [n_tokens][4][128], row-major, contiguous.
 *   idx_k        fp32 [n_tokens][128] index keys.
 *   slot_mapping int64 [n_tokens]: page * 128 + offset; a negative entry skips
 *                the token.  A page >= n_pages sets MSA_STATUS_BAD_SLOT.
 * Per (token, head, 16-channel group) with s = s_enc_k (K) or s_enc_v (V):
 *   a = max|x|, sb = E4M3_RNE_satfinite(fp32(fp32(a / 6) * s)),
 *   code = E2M1 round-to-nearest-even (ties to the even code, saturating at 6)
 *          of fp32(|x| * s) / sb evaluated exactly, sign on non-zero codes only,
 *          all codes 0 when sb == 0.
 * Index keys: E4M3_RNE_satfinite(x); a zero result is stored as 0x00.
 * Slots written by one call must be distinct.
 */
int msa_quantize_kv_insert(const msa_cache* cache, const float* k, const float* v,
                           const float* idx_k, const int64_t* slot_mapping,
                           int32_t n_tokens, msa_stream_t stream);

/*
 * Indexer scan and top-k selection (blog, "Sparse attention still scans an
 * index": 16 blocks plus the most recent one; "Parallelize index work across
 * context": the split scan keeps the selection exact).
 *
 *   q_idx       E4M3 [n_q_total][n_idx_heads = 8][128] index queries.
 *   w           fp32 [n_q_total][8] head weights (>= 0 for the ReLU reading).
 *   block_table int32 [n_seqs][max_pages]; seq_lens int32 [n_seqs];
 *   q_start_loc int32 [n_seqs + 1], non-decreasing, q_start_loc[0] = 0,
 *               q_start_loc[n_seqs] = n_q_total.
 *   topk        must be 16.
 *   sel         int32 [n_q_total][topk + 1] out: min(topk, r_j) selected block
 *               ids of blocks 0..r_j-1 (highest block score first wins, ties to
 *               the lower id) in ascending order, then r_j; padded with -1.
 *   n_sel       int32 [n_q_total] out: min(topk, r_j) + 1.
 *   ws, ws_bytes scratch of at least msa_indexer_workspace_bytes(...) bytes,
 *               16-byte aligned, ZEROED before its first use.  Its first 256
 *               bytes hold grid-barrier words; every call, also one whose
 *               barrier timed out, leaves them at rest (a generation count
 *               apart), so later calls need no clearing.  From
 *               byte 256, after the stream reaches the end of this call, it holds
 *               for every query token j and block i < r_j four fp32 partial
 *               maxima P[j][i][0..3] (row stride 4 * max_pages floats): the maxima
 *               over the block's token quarters; the block score is their max.
 *               Other entries are unspecified.  Calls sharing a workspace must
 *               not overlap on the GPU.
 * Block score S[j][i] = max over the 128 tokens t of block i of
 *   sum_h w[j][h] * max(0, q_idx[j][h] . key(t)), computed with fp32 sums of
 *   exact FP8 products.
 * n_seqs <= 4096.
 */
int msa_indexer_topk(const msa_cache* cache, const uint8_t* q_idx, const float* w,
                     int32_t n_idx_heads, const int32_t* block_table, int32_t max_pages,
                     const int32_t* seq_lens, const int32_t* q_start_loc, int32_t n_seqs,
                     int32_t n_q_total, int32_t topk, int32_t* sel, int32_t* n_sel,
                     void* ws, size_t ws_bytes, msa_stream_t stream);

/*
 * Context-split indexer (blog, "Parallelize index work across context": each
 * GPU scans a part of the context, the local candidates are exchanged, and
 * merging them gives the final top-16 exactly: every block competes once,
 * with the same score, in one part).  The two calls below let a caller run
 * each part where its index pages live and merge anywhere.
 *
 * msa_indexer_topk_range: msa_indexer_topk restricted to the logical blocks
 * [blk_lo, blk_hi) (0 <= blk_lo <= blk_hi) of every sequence: for query token
 * j, only blocks i with blk_lo <= i < min(blk_hi, r_j) are scanned and
 * compete; instead of sel / n_sel it writes
 *   cand  uint64 [n_q_total][16] out: the local top-16 as keys, best first,
 *         zero-padded (fewer than 16 blocks in the range: all of them).
 *         key = (ordered(S) << 32) | (0xFFFFFFFF - block), where ordered(x)
 *         is the fp32 bit pattern of x with the sign bit set for x >= +0 and
 *         all bits inverted for x < 0; a larger key is a higher score, then
 *         a lower block; 0 = no block.
 * Only the block-table entries of the range are read.  Workspace and every
 * other argument as msa_indexer_topk (its scores are written for the blocks
 * of the range only).
 *
 * msa_indexer_merge_candidates: cand holds n_shards (1..64) such arrays,
 * [n_shards][n_q_total][16], whose block ranges are disjoint; per query token
 * the 16 largest non-zero keys win and sel / n_sel are written exactly as
 * msa_indexer_topk writes them (winners ascending, then r_j, -1 padding;
 * n_sel = winners + 1).  When the ranges tile [0, r_j) of every token, the
 * result equals msa_indexer_topk's.  Status bits go to cache->status (the
 * cache's pools are not read): MSA_STATUS_BAD_SEQ for an inconsistent
 * sequence, MSA_STATUS_BAD_SELECTION for a key whose block is not below r_j.
 * Launched as a programmatic dependent of the previous kernel in the stream.
 */
int msa_indexer_topk_range(const msa_cache* cache, const uint8_t* q_idx, const float* w,
                           int32_t n_idx_heads, const int32_t* block_table, int32_t max_pages,
                           const int32_t* seq_lens, const int32_t* q_start_loc, int32_t n_seqs,
                           int32_t n_q_total, int32_t topk, int32_t blk_lo, int32_t blk_hi,
                           uint64_t* cand, void* ws, size_t ws_bytes, msa_stream_t stream);
int msa_indexer_merge_candidates(const msa_cache* cache, const uint64_t* cand, int32_t n_shards,
                                 const int32_t* seq_lens, const int32_t* q_start_loc,
                                 int32_t n_seqs, int32_t max_pages, int32_t n_q_total,
                                 int32_t topk, int32_t* sel, int32_t* n_sel, msa_stream_t stream);

/* Bytes of scratch msa_indexer_topk needs (a multiple of 256). */
size_t msa_indexer_workspace_bytes(int32_t n_q_total, int32_t max_pages);

/*
 * msa_indexer_topk without a workspace argument, for callers that cannot
 * allocate device memory: code that runs inside a host framework which owns
 * every device allocation, real-time decode loops where a cudaMalloc (which
 * may synchronise the device) is not allowed between steps, or plug-ins that
 * receive only their input and output buffers.  The pages have no counterpart
 * of this call; it is a deployment convenience.
 *
 * Same arguments, results and errors as msa_indexer_topk minus ws/ws_bytes.
 * The scratch is a file-scope device array of MSA_INDEXER_NOALLOC_SCRATCH_BYTES
 * (8 MiB) inside the library; every GPU that loads the library keeps it until
 * the process exits.  Shapes that need more, i.e.
 * msa_indexer_workspace_bytes(n_q_total, max_pages) > that capacity, return
 * MSA_ERR_SCRATCH_CAPACITY and enqueue nothing.  Nothing in the array needs
 * clearing by the caller: every score entry a call reads was written earlier
 * by that same call.
 * The array is shared by all calls on a device and keeps the last call's
 * contents, so calls whose kernels overlap on the GPU (e.g. on two streams
 * without ordering) race and must not be issued.  The first call on each
 * device looks up the array's device address (with that device current);
 * make that first call before any stream capture.  No cudaMalloc, cudaFree
 * or allocating routine is called.  (The array starts zeroed when the library
 * is loaded; its grid-barrier words return to rest after every call, also
 * after one that timed out.)
 */
int msa_indexer_topk_noalloc(const msa_cache* cache, const uint8_t* q_idx, const float* w,
                             int32_t n_idx_heads, const int32_t* block_table, int32_t max_pages,
                             const int32_t* seq_lens, const int32_t* q_start_loc, int32_t n_seqs,
                             int32_t n_q_total, int32_t topk, int32_t* sel, int32_t* n_sel,
                             msa_stream_t stream);


/*
 * Split-context sparse GQA attention over the selected blocks (blog, "Sparse
 * attention still scans an index": exact attention over the selected blocks;
 * ai4snews article, third paragraph: FP8 queries, NVFP4 K/V dequantised to FP8
 * before the matmul).
 *
 *   q           E4M3 [n_q_total][n_q_heads = 16][128] queries.
 *   sel, n_sel  as written by msa_indexer_topk (any ascending or unordered
 *               list of distinct block ids <= r_j is accepted).
 *   n_splits    1..64: the selected blocks of each query token are dealt
 *               round-robin to n_splits partial attentions.
 *   o_part      fp32 [n_q_total][n_splits][16][128] out: each split's
 *               normalised output (zero for an empty split).
 *   lse_part    fp32 [n_q_total][n_splits][16] out: natural-log sum of exp of
 *               the split's logits (-inf for an empty split).
 * Per element the FP8 operand is sign(code) | E4M3_RNE(|e2m1(code)| * sb);
 * logits = (q . k8) * softmax_scale / s_enc_k; the value contraction is
 * divided by s_enc_v.  Keys after pos_j are masked.  Limits: n_seqs <= 4096,
 * n_q_total <= 65535 (else MSA_ERR_UNSUPPORTED_SHAPE).
 * Launched as a programmatic dependent of the previous kernel in the stream
 * (msa_indexer_topk lets it start early): it waits for that kernel before it
 * reads sel and n_sel, but copies q_start_loc before the wait, so the kernel
 * just before it must not write q_start_loc.
 */
int msa_sparse_attn_decode(const msa_cache* cache, const uint8_t* q, int32_t n_q_heads,
                           float softmax_scale, const int32_t* sel, const int32_t* n_sel,
                           const int32_t* block_table, int32_t max_pages,
                           const int32_t* seq_lens, const int32_t* q_start_loc,
                           int32_t n_seqs, int32_t n_q_total, int32_t n_splits,
                           float* o_part, float* lse_part, msa_stream_t stream);

/*
 * Log-sum-exp merge of the split partials (blog, "Sparse attention still scans
 * an index": attention over the selected blocks is exact; a split computes it
 * over part of them, and the parts combine by their softmax normalisers):
 *   out[j][h] = sum_s exp(lse[j][s][h] - L) * o_part[j][s][h],
 *   L = log sum_s exp(lse[j][s][h]).
 *   out  fp32 [n_q_total][n_q_heads][128].  A row whose splits are all empty
 *        is written as zeros.
 *   lse  fp32 [n_q_total][n_q_heads] out, or NULL: the merged L (-inf for a
 *        row whose splits are all empty), so that merged results can be merged
 *        again.
 * Limits: n_q_heads <= 1024, n_q_total <= 65535 (else MSA_ERR_UNSUPPORTED_SHAPE).
 */
int msa_merge_splits(const float* o_part, const float* lse_part, int32_t n_q_total,
                     int32_t n_q_heads, int32_t n_splits, float* out, float* lse,
                     msa_stream_t stream);

/*
 * The whole decode step in ONE launch, for low concurrency (blog, "AMD uses
 * different conversion and communication mechanisms": a separate
 * single-kernel strategy reduces launches at low concurrency; "Keep capacity,
 * layer, and system results separate": that advantage need not hold at high
 * concurrency, where msa_indexer_topk + msa_sparse_attn_decode +
 * msa_merge_splits stay the faster path).  Computes exactly what those three
 * calls compute, with the same rounding: the selection into sel / n_sel (as
 * msa_indexer_topk) and the merged output
 *   out fp32 [n_q_total][16][128].
 * One cooperative launch of at most one CTA per SM runs the scan, the top-k,
 * the attention (one page per work item, each selected block a split) and the
 * merge, with a bounded grid barrier between phases.
 *   ws, ws_bytes  scratch of at least msa_decode_fused_workspace_bytes(n_q_total,
 *                 max_pages) bytes, 16-byte aligned, ZEROED before its first use
 *                 (its first 256 bytes hold grid-barrier words that every call,
 *                 also one that timed out, leaves at rest).  Calls sharing a
 *                 workspace must not overlap on the GPU.
 * Other arguments as msa_indexer_topk and msa_sparse_attn_decode.  Limits:
 * n_seqs <= 64, n_q_total <= 64 (else MSA_ERR_UNSUPPORTED_SHAPE).
 */
int msa_decode_fused(const msa_cache* cache, const uint8_t* q, const uint8_t* q_idx, const float* w,
                     int32_t n_q_heads, int32_t n_idx_heads, float softmax_scale,
                     const int32_t* block_table, int32_t max_pages, const int32_t* seq_lens,
                     const int32_t* q_start_loc, int32_t n_seqs, int32_t n_q_total, int32_t topk,
                     int32_t* sel, int32_t* n_sel, float* out, void* ws, size_t ws_bytes,
                     msa_stream_t stream);
size_t msa_decode_fused_workspace_bytes(int32_t n_q_total, int32_t max_pages);

/*
 * Fused QKV projection -> RMS norm -> RoPE -> FP8 queries and cache insertion
 * (blog, "Reduce both data movement and resource waits": fusing the projection
 * with normalisation, RoPE and cache insertion avoids writing the intermediate
 * tensor to HBM and reading it back).  The projection's accumulators stay on
 * the SM; nothing but the outputs below is written.
 *
 *   x          bf16 [n_tokens][d_model] hidden states, row-major, 16-byte aligned;
 *              d_model a multiple of 64 (64 .. 65,536).
 *   w          bf16 [25 * 128][d_model] projection (row = output channel),
 *              16-byte aligned: heads 0-15 queries, 16-19 keys, 20-23 values,
 *              24 the index key (MSA_QKV_HEADS = 25 heads of 128).
 *   gamma_q, gamma_k, gamma_idx  fp32 [128] RMS-norm gains of each head kind.
 *   cos_sin    fp32 [max_pos][128]: cos of the 64 pair angles, then their sin
 *              (msa_rope_table writes it); positions int32 [n_tokens] index it
 *              (a position outside [0, max_pos) leaves the head unrotated and
 *              sets MSA_STATUS_BAD_SEQ).
 *   slot_mapping int64 [n_tokens] as msa_quantize_kv_insert (negative: skip).
 *   q8         uint8 [n_tokens][16][128] out: E4M3 queries (RNE, satfinite).
 *   y_out      fp32 [n_tokens][25][128] out, or NULL: every head's row just
 *              before rounding (diagnostic).
 * Per token: z = W x (fp32 accumulation of bf16 products); query, key and
 * index-key heads y = RoPE(z / sqrt(mean(z^2) + eps) * gamma), channel pairs
 * (i, i + 64) turned by the table's angle i: (a, b) -> (a cos - b sin,
 * b cos + a sin); value heads y = z.  Queries -> q8; keys and values -> NVFP4
 * in the slot, exactly the quantiser of msa_quantize_kv_insert with the
 * cache's s_enc_k / s_enc_v; index keys -> E4M3 in the index page.
 */
#define MSA_QKV_HEADS 25
int msa_qkv_project_insert(const msa_cache* cache, const void* x, const void* w, int32_t n_tokens,
                           int32_t d_model, const float* gamma_q, const float* gamma_k,
                           const float* gamma_idx, const float* cos_sin, int32_t max_pos,
                           const int32_t* positions, const int64_t* slot_mapping, float eps,
                           uint8_t* q8, float* y_out, msa_stream_t stream);
/* RoPE table for msa_qkv_project_insert: cos_sin[pos][i] = cos(pos * base^(-2i/128))
 * and cos_sin[pos][64 + i] = the sin, i < 64, computed in double precision and
 * rounded to fp32 (base > 1, e.g. 10,000). */
int msa_rope_table(float* cos_sin, int32_t max_pos, double base, msa_stream_t stream);

/* Element types of rows that the calls below take or return. */
#define MSA_DTYPE_F32 0
#define MSA_DTYPE_BF16 1
#define MSA_DTYPE_F16 2

/* Projected rows of new tokens, in one element type: channels and heads
 * contiguous (head h of token t at pointer + t * stride + 128 h, strides in
 * elements), so that slices of one projection's output can be passed as they
 * are.  Pointers and strides * element size are multiples of 16 bytes. */
typedef struct msa_rows {
  const void* q;      /* [n_tokens][16][128] */
  const void* k;      /* [n_tokens][4][128] */
  const void* v;      /* [n_tokens][4][128] */
  const void* idx_k;  /* [n_tokens][128] */
  const void* q_idx;  /* [n_tokens][8][128], or NULL: no index queries */
  int64_t q_stride, k_stride, v_stride, idx_k_stride, q_idx_stride;
  int32_t dtype;      /* MSA_DTYPE_* */
} msa_rows;

/*
 * Rotary positions on projected rows, FP8 queries and index queries, and cache
 * insertion (the part of msa_qkv_project_insert behind its projection and norm,
 * for models that turn their heads in another way or project elsewhere).
 *
 *   rot_dim      channels 0 .. rot_dim - 1 of every query, key, index-key and
 *                index-query head are turned; a multiple of 16, 0 .. 128 (0:
 *                nothing is turned, cos_sin may be NULL).
 *   interleaved  0: pairs (i, i + rot_dim / 2); 1: pairs (2 i, 2 i + 1).
 *   cos_sin      fp32 [max_pos][rot_dim]: cos of the rot_dim / 2 pairs, then
 *                their sin (msa_rope_table for rot_dim 128, msa_rope_table_freqs
 *                for any), 16-byte aligned; positions int32 [n_tokens] index it
 *                (a position outside [0, max_pos) leaves the token unturned and
 *                sets MSA_STATUS_BAD_SEQ).
 *   slot_mapping int64 [n_tokens] as msa_quantize_kv_insert (negative: the
 *                token's cache entry is not written, its queries are).
 *   q8, q_idx8   uint8 [n_tokens][16][128] and [n_tokens][8][128] out: E4M3
 *                (RNE, satfinite, zeros as 0x00), 16-byte aligned; q_idx8 is
 *                used with rows->q_idx only.
 * A pair (a, b) becomes (fl(fl(a c) - fl(b s)), fl(fl(b c) + fl(a s))) in fp32,
 * every product and sum rounded on its own.  Keys and values -> NVFP4 and index
 * keys -> E4M3 in the slot, exactly as msa_quantize_kv_insert writes them.
 * Slots written by one call must be distinct.
 */
int msa_rotary_insert(const msa_cache* cache, const msa_rows* rows, int32_t n_tokens, const float* cos_sin,
                      int32_t max_pos, int32_t rot_dim, int32_t interleaved, const int32_t* positions,
                      const int64_t* slot_mapping, uint8_t* q8, uint8_t* q_idx8, msa_stream_t stream);
/*
 * The same with positions on several axes (time, height and width of images and
 * video, text alike on all of them): pair i turns by its axis's position,
 *   positions     int32 [n_axes][n_tokens], n_axes 1 .. MSA_MAX_AXES;
 *   axis_of_pair  HOST array of rot_dim / 2 bytes: axis of pair i, below n_axes
 *                 (not read for one axis, where every pair is of axis 0);
 * and uses the cos and sin of table row positions[axis_of_pair[i]][t].  A token with
 * a position outside [0, max_pos) on any axis is left unturned and sets
 * MSA_STATUS_BAD_SEQ.
 */
#define MSA_MAX_AXES 4
int msa_rotary_insert_axes(const msa_cache* cache, const msa_rows* rows, int32_t n_tokens, const float* cos_sin,
                           int32_t max_pos, int32_t rot_dim, int32_t interleaved, const int32_t* positions,
                           int32_t n_axes, const uint8_t* axis_of_pair, const int64_t* slot_mapping, uint8_t* q8,
                           uint8_t* q_idx8, msa_stream_t stream);
/* RoPE table of given frequencies: cos_sin[pos][i] = amplitude * cos(pos * freq[i])
 * and cos_sin[pos][rot_dim / 2 + i] = amplitude * sin(pos * freq[i]), computed in
 * double precision and rounded to fp32.  freq is a HOST array of rot_dim / 2
 * finite doubles (rot_dim a multiple of 16, 0 .. 128); amplitude is finite. */
int msa_rope_table_freqs(float* cos_sin, int32_t max_pos, const double* freq, int32_t rot_dim, double amplitude,
                         msa_stream_t stream);

/*
 * Read-back of cache slots (a prefill that goes on with the values later steps
 * will see; hand-over to an engine with a 16-bit cache).
 *
 *   slot_mapping int64 [n_tokens]: page * 128 + offset; a negative entry leaves
 *                the token's rows as they are, a page >= n_pages too and sets
 *                MSA_STATUS_BAD_SLOT.  A slot may be listed more than once.
 *   k, v         [n_tokens][4][128] out, idx_k [n_tokens][128] out, in the type
 *                `dtype` (MSA_DTYPE_*), 16-byte aligned; NULL: not wanted.
 * K and V elements are e2m1(code) * fl(sb * fl(1 / s_enc)), the product rounded
 * to fp32 and then to the output type; index keys are their E4M3 values.
 */
int msa_read_kv(const msa_cache* cache, const int64_t* slot_mapping, int32_t n_tokens, int32_t dtype, void* k,
                void* v, void* idx_k, msa_stream_t stream);

/*
 * Attention of drafted tokens over the whole cached context: a tree of drafts
 * per sequence (speculative verification), a plain causal run of up to 64 new
 * tokens, or one token of a layer without block selection.
 *
 *   q           E4M3 [n_q_total][n_q_heads = 16][128] queries; the drafts' keys and
 *               values are in the cache already (draft i of a sequence at position
 *               ctx + i, ctx = seq_lens[b] - n_q; its rotary position is its depth's,
 *               msa_rotary_insert).
 *   block_table, max_pages, seq_lens, q_start_loc, n_seqs, n_q_total as
 *               msa_sparse_attn_decode; a sequence has at most MSA_TREE_MAX_DRAFTS
 *               query tokens (more, like any inconsistent sequence, sets
 *               MSA_STATUS_BAD_SEQ and leaves the sequence's rows as they were).
 *   tree_mask   uint64 [n_q_total] or NULL: bit i of a draft's word = it sees draft
 *               i of its sequence (its own bit included only if set; bits of drafts
 *               that do not exist are ignored).  NULL: draft j sees drafts 0 .. j.
 *               The ctx tokens before the drafts are visible to every draft.
 *   sel, n_sel  int32 [n_seqs][17] and [n_seqs], or both NULL (every block): one list
 *               of block ids per sequence, strictly ascending, shared by its drafts,
 *               as msa_indexer_topk writes it for one query token.  Visited are the
 *               listed blocks below ctx / 128 and the blocks from ctx / 128 on (those
 *               that can hold drafts).  An entry that is not above the ones before
 *               it, or behind the sequence, is left out and sets
 *               MSA_STATUS_BAD_SELECTION.
 *   dtype       MSA_DTYPE_BF16 or MSA_DTYPE_F16: type of out.
 *   out         [n_q_total][16][128], 16-byte aligned; zeros where a row sees nothing.
 *   lse         fp32 [n_q_total][16] out or NULL: natural-log sum of exp of the row's
 *               logits (-inf where it sees nothing).
 *   ws, ws_bytes scratch of at least msa_tree_attn_workspace_bytes(n_q_total) bytes,
 *               16-byte aligned, ZEROED before its first use (every call leaves the
 *               words that have to be zero so; calls of different sizes may share
 *               one).  Calls sharing a workspace must not overlap on the GPU.
 * Rows behind the last sequence (q_start_loc[n_seqs] .. n_q_total - 1) are left as
 * they were; they count among n_q_total, which with n_seqs chooses the kernel (more than
 * 16 rows a sequence: the one for many drafts, 224 us against 184 if 32 sequences of 32,768
 * tokens have one draft each and the rest is padding).
 * Operands as msa_sparse_attn_decode.  The weights are rounded to f16 before they meet
 * the values (2^-11 relative, or 2^-33 of the weight at the row's reference, whichever
 * is more), and those of the same page's earlier tokens are multiplied and rounded again
 * when the reference moves to a larger score inside the page (at most three times); sums,
 * references and accumulators are fp32.  Rows are summed in an order that depends on the
 * call's sizes only.  A physical page outside
 * the pool sets MSA_STATUS_BAD_PAGE and its tokens are not seen.  A cache scale byte
 * of 0x7F or 0xFF (no number, never written by the library) counts as zero.
 * A query byte of 0x7F or 0xFF makes its row's out and lse NaN (zeros and -inf where the
 * row sees nothing).  Rows that two
 * sequences claim (q_start_loc not ascending) hold numbers of no meaning.
 * softmax_scale > 0, and softmax_scale / s_enc_k times 2^26 finite (where the quotient
 * is below 2^-126, or underflows, every score is zero to fp32 and a row's out is the mean of
 * the values that it sees).
 * s_enc_v above 2^-120 and at most 2^100.
 * Limits: n_seqs <= 4096, n_q_total <= 65535.  Two launches, both programmatic
 * dependents of the kernel before them.
 */
#define MSA_TREE_MAX_DRAFTS 64
int msa_tree_attn(const msa_cache* cache, const uint8_t* q, int32_t n_q_heads, float softmax_scale,
                  const int32_t* block_table, int32_t max_pages, const int32_t* seq_lens,
                  const int32_t* q_start_loc, int32_t n_seqs, int32_t n_q_total, const uint64_t* tree_mask,
                  const int32_t* sel, const int32_t* n_sel, int32_t dtype, void* out, float* lse, void* ws,
                  size_t ws_bytes, msa_stream_t stream);
size_t msa_tree_attn_workspace_bytes(int32_t n_q_total);

/*
 * Attention of a prompt's tokens over the cached context: any number of query tokens a
 * sequence (a whole prompt, a chunk of one, chunks of several prompts in one call), whose
 * keys and values are in the cache already.
 *
 *   q, block_table, max_pages, seq_lens, q_start_loc, n_seqs, n_q_total as msa_tree_attn,
 *               with any number of tokens a sequence.  Token i of a sequence is at position
 *               pos = seq_lens[b] - n_q + i.
 *   window      0, or the number of positions that a token sees, its own the last of them:
 *               start = max(0, pos + 1 - window) (0: start = 0).
 *   ends        int32 [n_q_total] or NULL: the tokens of its sequence that a token sees
 *               end before position ends[j] (clamped to 0 .. seq_lens[b]), so that, for
 *               instance, the tokens of an image see all of it.  NULL: ends[j] = pos + 1.
 *               A token sees the positions start <= t < end; none where end <= start.
 *   n_visited   pages that ws has room for: the sequences' pages from the first that
 *               their first token sees to their last, summed over the call, at most (the
 *               sum of ceil(seq_lens[b] / 128) always will do; a page that several
 *               sequences of the call share counts, and is converted, once for each).
 *               A sequence behind that many sets MSA_STATUS_BAD_SEQ and keeps its rows.
 *   dtype, out, lse as msa_tree_attn; out on a 32-byte boundary.
 *   ws, ws_bytes scratch of at least msa_prefill_workspace_bytes(n_q_total, n_seqs,
 *               n_visited) bytes, 16-byte aligned, nothing of which is kept between calls.
 *               Calls sharing a workspace must not overlap on the GPU.
 * Rows behind the last sequence, and those of an inconsistent one (MSA_STATUS_BAD_SEQ),
 * are left as they were; rows that several sequences claim (q_start_loc goes back) hold
 * any of their results.  Operands, sums and special values as msa_tree_attn; the weights
 * are rounded to f16 (2^-11 relative, or 2^-33 of the weight at the row's reference) once,
 * those of the first 64 tokens of a page once more where the page's others move the row's
 * reference.  Rows are summed in an order that depends on the call's sizes and the device's
 * SMs only.
 * softmax_scale > 0 and at most 2^26 s_enc_k / (448 * 448 * 128 log2(e)); s_enc_v above
 * 2^-120 and at most 2^100.  Limits: n_seqs <= 4096, n_q_total <= 262,144, n_visited <=
 * 1,048,576.  Three launches (two, when n_visited is small), programmatic dependents of
 * the kernel before them.
 */
int msa_prefill_attn(const msa_cache* cache, const uint8_t* q, int32_t n_q_heads, float softmax_scale,
                     const int32_t* block_table, int32_t max_pages, const int32_t* seq_lens,
                     const int32_t* q_start_loc, int32_t n_seqs, int32_t n_q_total, int32_t window,
                     const int32_t* ends, int32_t n_visited, int32_t dtype, void* out, float* lse, void* ws,
                     size_t ws_bytes, msa_stream_t stream);
size_t msa_prefill_workspace_bytes(int32_t n_q_total, int32_t n_seqs, int32_t n_visited);

/*
 * Block-outer transfer rows (blog, "AMD uses different conversion and
 * communication mechanisms": a KV block kept as one contiguous row is moved in
 * one read instead of one read per page).  The row of a block holds, for every
 * layer l = 0 .. n_layers-1 in order, that layer's KV page (73,728 bytes, the
 * format above) followed by its index page (16,384 bytes): 90,112 bytes per
 * layer, msa_block_row_bytes(n_layers) per row.
 *
 *   layers   HOST array of n_layers caches (1 <= n_layers <= 128), one per
 *            model layer; block i lives at the same physical page pages[i] in
 *            every layer's pools.
 *   pages    int32 [n_blocks] physical page of each block.  A page outside a
 *            layer's pool sets MSA_STATUS_BAD_PAGE in layers[0].status and that
 *            (block, layer) part of the row is left untouched.
 *   rows     uint8 [n_blocks][msa_block_row_bytes(n_layers)], 16-byte aligned.
 * msa_pack_blocks copies pages -> rows; msa_unpack_blocks copies rows -> pages
 * (so a receiver may place a block at different page ids).  Rows and pages
 * must not overlap; the pages listed in one unpack call must be distinct.
 */
int msa_pack_blocks(const msa_cache* layers, int32_t n_layers, const int32_t* pages,
                    int32_t n_blocks, uint8_t* rows, msa_stream_t stream);
int msa_unpack_blocks(const msa_cache* layers, int32_t n_layers, const uint8_t* rows,
                      const int32_t* pages, int32_t n_blocks, msa_stream_t stream);
/* Bytes of one block-outer row: n_layers * 90,112 (0 for n_layers <= 0). */
size_t msa_block_row_bytes(int32_t n_layers);

/*
 * Pages that sequences share.  A pool counts, for each page id below n_pages, the
 * block-table entries that hold it, and keeps a mask of those that none holds (bit
 * p % 32 of word p / 32).  A sequence is a row of block_table and its entry of
 * seq_lens; it holds the row's entries that are not negative, also those behind its
 * length.  Page p is the same page in every layer's pools, as in the block-outer rows.
 * Every call below changes tables, lengths, counts and mask on the device, in stream
 * order; calls on one pool must not overlap on the GPU.  Pages are dealt lowest number
 * first in the order of the call's sequences; from the first sequence that finds too few
 * of them on, none that needs a page gets one (MSA_STATUS_NO_PAGES).  Status bits go to
 * pool->status.  n_seqs <= 4096, max_pages <= 65,536.
 */
typedef struct msa_page_pool {
  int32_t* refs;        /* device, [n_pages] */
  uint32_t* free_mask;  /* device, [(n_pages + 31) / 32] */
  int32_t n_pages;
  int32_t* status;      /* device int32, sticky MSA_STATUS_* bits; may be NULL */
} msa_page_pool;

/*
 * Pages and slots for new tokens: sequence b gets room for n = q_start_loc[b + 1] -
 * q_start_loc[b] tokens behind its length (entries of its row that hold a page already
 * are used as they are) and grows by n.
 *   slots  int64 [n_tokens] out: slot (page * 128 + offset) of every new token, in the
 *          sequences' order, for msa_rotary_insert and its like; -1 for the tokens of a
 *          sequence that could not grow and for rows behind the last sequence.
 * A sequence that could not grow keeps its length and row: one without enough free
 * pages, one with tokens outside [0, n_tokens) or more than max_pages * 128 of them
 * (MSA_STATUS_BAD_SEQ), one whose last tokens have no page (MSA_STATUS_BAD_PAGE).  Where
 * n < 0 for some sequence, tokens belong to several of them and none grows
 * (MSA_STATUS_BAD_SEQ).
 * n_tokens <= 262,144.
 */
int msa_extend_sequences(const msa_page_pool* pool, int32_t* block_table, int32_t max_pages, int32_t* seq_lens,
                         const int32_t* q_start_loc, int32_t n_seqs, int32_t n_tokens, int64_t* slots,
                         msa_stream_t stream);

/*
 * Forks: for each of n pairs, row dst[i], which has to be empty, becomes a second copy
 * of row src[i]: its full pages are shared, the tokens of its last page (if that is not
 * full) are copied to a page of dst's own, in every layer.  Pages that src holds behind
 * its length are not shared.
 *   layers    HOST array of n_layers caches (1 .. 128), each with pool->n_pages pages
 *             or more.
 *   ws        device scratch of msa_fork_workspace_bytes(n) bytes, 16-byte aligned.
 * A pair outside the table, with a target that has tokens or holds a page in any entry of
 * its row, or that an earlier pair which is not left out for these reasons names, is left
 * out (MSA_STATUS_BAD_SEQ), so a row that is another pair's target counts as empty; so is
 * one whose last page is outside the pool, and an entry outside it is taken over and
 * flagged (MSA_STATUS_BAD_PAGE).  n <= 4096.
 */
int msa_fork_sequences(const msa_cache* layers, int32_t n_layers, const msa_page_pool* pool, int32_t* block_table,
                       int32_t max_pages, int32_t* seq_lens, int32_t n_seqs, const int32_t* src, const int32_t* dst,
                       int32_t n, void* ws, size_t ws_bytes, msa_stream_t stream);
size_t msa_fork_workspace_bytes(int32_t n);

/*
 * Release of the rows listed in rows (int32 [n]; the same row twice counts once): every
 * page they hold loses one count and is free when that was the last, the rows' entries
 * become -1 and their lengths 0.  A page that nobody was counted for or outside the
 * pool sets MSA_STATUS_BAD_PAGE, a row outside the table MSA_STATUS_BAD_SEQ.
 */
int msa_release_sequences(const msa_page_pool* pool, int32_t* block_table, int32_t max_pages, int32_t* seq_lens,
                          int32_t n_seqs, const int32_t* rows, int32_t n, msa_stream_t stream);

/*
 * Page copies in every layer: page src[i] to page dst[i] (negative, or src[i] = dst[i]:
 * none), the first tokens[i] tokens (NULL: all 128; the bytes of the others stay).  The
 * targets must be distinct, and no target may be another pair's source.  A page outside
 * a pool leaves the pair out and sets MSA_STATUS_BAD_PAGE in layers[0].status.
 */
int msa_copy_pages(const msa_cache* layers, int32_t n_layers, const int32_t* src, const int32_t* dst,
                   const int32_t* tokens, int32_t n, msa_stream_t stream);

/*
 * Accepted drafts: of each sequence's n = q_start_loc[b + 1] - q_start_loc[b] last tokens
 * (drafts that msa_tree_attn verified, at most MSA_TREE_MAX_DRAFTS) those stay whose bits
 * accepted[b] has; the k-th of them moves to position ctx + k, ctx = seq_lens[b] - n, in
 * every layer's K/V and index pages.  Keys keep the rotary position they were written
 * with: a draft's is its depth's, which is k for a path from the root.
 *   accepted  uint64 [n_seqs]; bits of drafts that do not exist are ignored.
 *   new_lens  int32 [n_seqs] out, apart from seq_lens: ctx + the number of accepted drafts.
 * Pages behind the new length stay in the row, for later tokens.  An inconsistent
 * sequence keeps its length (MSA_STATUS_BAD_SEQ); a token whose page or whose new
 * place's page is outside the pool is not moved (MSA_STATUS_BAD_PAGE).  Status bits go to
 * layers[0].status.  The pages of drafts must not be shared: a fork comes before the drafts
 * or behind their commit (one made between shares the full pages among them).
 */
int msa_commit_drafts(const msa_cache* layers, int32_t n_layers, const int32_t* block_table, int32_t max_pages,
                      const int32_t* seq_lens, const int32_t* q_start_loc, int32_t n_seqs, const uint64_t* accepted,
                      int32_t* new_lens, msa_stream_t stream);

/*
 * Helpers for the per-tensor scale.  msa_absmax folds max|x[i]| over n fp32
 * values into *amax (device float, caller-initialised to 0): call it on every
 * chunk of a tensor, then msa_encode_scale(amax) returns the fp32 encode scale
 * 448 / amax (1 for amax == 0).
 */
int msa_absmax(const float* x, int64_t n, float* amax, msa_stream_t stream);
float msa_encode_scale(float amax);

/*
 * Diagnostic: the FP8 operands the attention kernel multiplies, for one page.
 * k8, v8: uint8 [4 heads][128 tokens][128 channels] out, E4M3 bytes in
 * logical channel order, produced by the same device dequantiser as
 * msa_sparse_attn_decode.
 */
int msa_debug_fp8_page(const msa_cache* cache, int64_t page, uint8_t* k8, uint8_t* v8,
                       msa_stream_t stream);

/*
 * Test hook for the failure paths (the pages have no counterpart).  Sets, for
 * every later launch of the library in this process, the time limit of one
 * bounded on-chip wait (wait_limit_ns; 0 restores the default of 2 s) and the
 * fault-injection flags (0 = none):
 *   MSA_INJECT_BARRIER_TIMEOUT  the indexer's grid barrier waits for one CTA
 *                               more than the launch has, so every CTA's wait
 *                               runs out after wait_limit_ns: the call sets
 *                               MSA_STATUS_TIMEOUT, leaves sel/n_sel unwritten
 *                               and its workspace barrier word at rest;
 *   MSA_INJECT_ATTENTION_TIMEOUT  every CTA of an attention kernel (sparse
 *                               decode, tree or prefill) leaves out the copy of its first page, so the waits for it
 *                               run out after wait_limit_ns: the call sets
 *                               MSA_STATUS_TIMEOUT, its CTAs release tensor
 *                               memory only after their copies and tensor-core
 *                               products in flight are done, and return.
 * Launches already captured into a CUDA graph keep the settings they were
 * captured with.  Unknown flags return MSA_ERR_INVALID_ARG.
 */
#define MSA_INJECT_BARRIER_TIMEOUT 0x1
#define MSA_INJECT_ATTENTION_TIMEOUT 0x2
int msa_debug_set_fault_injection(int32_t flags, uint64_t wait_limit_ns);

/* Copies the device status word to *host_out (synchronous on the stream). */
int msa_read_status(const msa_cache* cache, int32_t* host_out, msa_stream_t stream);

/* Static description of a return code or status bit set. */
const char* msa_status_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H */
