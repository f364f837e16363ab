// Rotary positions on projected rows, FP8 queries and index queries, and the
// NVFP4 / FP8 cache insertion, for projections that run elsewhere (the fused
// projection of qkv.cu turns whole heads by half pairs; this is the general
// form: half or interleaved pairs, any first part of the head, any table).
//
// Per token: the first rot channels of the query, key, index-key and
// index-query heads are turned pair by pair,
//   (a, b) -> (fl(fl(a c) - fl(b s)), fl(fl(b c) + fl(a s))),
// every product and sum rounded to fp32 on its own (no contraction), so that
// the bytes written are those of the same formula evaluated step by step
// anywhere else; then queries -> E4M3, keys and values -> NVFP4 (the quantiser
// of msa_quantize_kv_insert), index keys -> E4M3.
//
// Bound by memory: a bf16 token of 33 heads reads 8,448 bytes and writes 3,776.
// One half-warp takes one head row, lane l its channels 8l .. 8l + 7: one or two
// 16-byte loads, one 8-byte FP8 store or one 32-bit code word, a 16-channel
// group is two lanes, and the partner channels of a half pair sit in one lane
// a fixed distance away.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace msa {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  const void* rows[5];     // q, k, v, idx_k, q_idx (may be null)
  long long stride[5];     // elements from one token's rows to the next
  int n_tokens;
  int n_pairs;             // half-warp jobs come in pairs: 17 per token, 13 without index queries
  const float* cos_sin;    // [max_pos][rot]: cos of the rot / 2 pairs, then their sin
  int max_pos;
  int rot;
  int interleaved;
  const int* positions;
  const int64_t* slot_mapping;
  uint8_t* kv_pool;
  uint8_t* idx_pool;
  int64_t n_pages;
  float s_enc_k, s_enc_v;
  uint8_t* q8;   // [n_tokens][16][128]
  uint8_t* qi8;  // [n_tokens][8][128]
  int* status;
};

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = ld_stream_v4(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
  const uint4 v = ld_stream_v4(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Eight E4M3 bytes (RNE, satfinite, zeros as 0x00), channel order.
__device__ __forceinline__ uint2 to_fp8x8(const float (&x)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = f32x2_to_e4m3x2(x[4 * h], x[4 * h + 1]), hi = f32x2_to_e4m3x2(x[4 * h + 2], x[4 * h + 3]);
    w[h] = canon_zero(lo & 0xFF) | (canon_zero(lo >> 8) << 8) | (canon_zero(hi & 0xFF) << 16) | (canon_zero(hi >> 8) << 24);
  }
  return make_uint2(w[0], w[1]);
}

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rotary_insert_kernel(RopeParams p) {
  const int lane = threadIdx.x & 31, l = lane & 15;
  const long long n_jobs = (long long)p.n_tokens * p.n_pairs;
  const long long warp0 = ((long long)blockIdx.x * kRopeThreads + threadIdx.x) >> 5;
  const long long n_warps = ((long long)gridDim.x * kRopeThreads) >> 5;
  for (long long job = warp0; job < n_jobs; job += n_warps) {
    const int t = (int)(job / p.n_pairs);
    // rows of a token in job order: 16 q, 4 k, 4 v, 8 q_idx, idx_k (and one idle half)
    int row = 2 * (int)(job % p.n_pairs) + (lane >> 4);
    if (p.n_pairs == 13 && row >= 24) row += 8;
    const int kind = row < 16 ? 0 : row < 20 ? 1 : row < 24 ? 2 : row < 32 ? 4 : 3;
    const int head = kind == 0 ? row : kind == 1 ? row - 16 : kind == 2 ? row - 20 : kind == 4 ? row - 24 : 0;
    const bool live = row <= 32;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live)
      load8(static_cast<const T*>(p.rows[kind]) + (size_t)t * p.stride[kind] + head * kHeadDim + 8 * l, x);
    // rotation (values stay as they are)
    const int pos = p.positions[t];
    const bool turn = pos >= 0 && pos < p.max_pos;
    if (p.rot > 0 && !turn && lane == 0 && row == 0) set_status(p.status, MSA_STATUS_BAD_SEQ);
    if (turn && p.rot > 0) {
      const float* cs = p.cos_sin + (size_t)pos * p.rot;
      const int half = p.rot >> 1;
      const bool mine = kind != 2 && 8 * l < p.rot;
      if (p.interleaved) {
        if (mine) {
          const float4 c = __ldg(reinterpret_cast<const float4*>(cs + 4 * l));
          const float4 s = __ldg(reinterpret_cast<const float4*>(cs + half + 4 * l));
          const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(a, cc[i]), __fmul_rn(b, ss[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(b, cc[i]), __fmul_rn(a, ss[i]));
          }
        }
      } else {
        // channel c < half pairs with c + half: half / 8 lanes further on
        const int step = half >> 3;
        const bool first = l < step;
        const int src = (lane & 16) | ((first ? l + step : l - step) & 15);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], src);
        if (mine) {
          const int at = 8 * (first ? l : l - step);
          float c[8], s[8];
          load8(cs + at, c);
          load8(cs + half + at, s);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float u = __fmul_rn(x[i], c[i]), w = __fmul_rn(o[i], s[i]);
            x[i] = first ? __fsub_rn(u, w) : __fadd_rn(u, w);
          }
        }
      }
    }
    if (kind == 0 || kind == 4) {
      uint8_t* dst = kind == 0 ? p.q8 + ((size_t)t * kQHeads + head) * kHeadDim
                               : p.qi8 + ((size_t)t * kIdxHeads + head) * kIdxDim;
      *reinterpret_cast<uint2*>(dst + 8 * l) = to_fp8x8(x);
    }
    // NVFP4 scale of the 16-channel group: this lane and its neighbour
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    const int64_t slot = p.slot_mapping[t];
    const int64_t page = slot >> 7;
    const int off = (int)(slot & 127);
    if (!live || slot < 0 || kind == 0 || kind == 4) continue;
    if (page >= p.n_pages) {
      if (l == 0) set_status(p.status, MSA_STATUS_BAD_SLOT);
      continue;
    }
    if (kind == 3) {
      uint8_t* dst = p.idx_pool + (size_t)page * kIdxPageBytes + off * kIdxDim;
      *reinterpret_cast<uint2*>(dst + (((l >> 1) ^ (off & 7)) << 4) + 8 * (l & 1)) = to_fp8x8(x);
      continue;
    }
    const float s_enc = kind == 1 ? p.s_enc_k : p.s_enc_v;
    const uint32_t sb_byte = f32_to_e4m3(__fmul_rn(__fdiv_rn(a, 6.0f), s_enc));
    const float sb = e4m3_to_f32(sb_byte);
    uint32_t word = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = x[4 * h + i];
        c[i] = e2m1_code(__fmul_rn(fabsf(v), s_enc), sb);
        c[i] |= (v < 0.f && c[i]) ? 8u : 0u;
      }
      word |= code_word_part(c, h);
    }
    uint8_t* hb = p.kv_pool + (size_t)page * kKvPageBytes + head * kHeadBytes;
    const int off_c = kind == 1 ? kOffKc : kOffVc, off_s = kind == 1 ? kOffKs : kOffVs;
    *reinterpret_cast<uint32_t*>(hb + off_c + off * 64 + (code_chunk_pos(l >> 2, off) << 4) + 4 * (l & 3)) = word;
    if ((l & 1) == 0) hb[off_s + (l >> 1) * kPageTokens + off] = (uint8_t)sb_byte;
  }
}

// cos / sin of pos * freq[i] in double precision, times the amplitude, rounded to fp32.
struct FreqParams {
  double freq[kHeadDim / 2];
};
__global__ void rope_table_freqs_kernel(float* table, int max_pos, int half, FreqParams f, double amplitude) {
  const long long id = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= (long long)max_pos * half) return;
  const int pos = (int)(id / half), i = (int)(id % half);
  double s, c;
  sincos((double)pos * f.freq[i], &s, &c);
  table[(size_t)pos * 2 * half + i] = (float)(c * amplitude);
  table[(size_t)pos * 2 * half + half + i] = (float)(s * amplitude);
}

}  // namespace

cudaError_t launch_rotary_insert(const msa_cache* c, const msa_rows* r, int n_tokens, const float* cos_sin,
                                 int max_pos, int rot, int interleaved, const int* positions,
                                 const int64_t* slot_mapping, uint8_t* q8, uint8_t* qi8, cudaStream_t stream) {
  if (n_tokens == 0) return cudaSuccess;
  static DeviceSetup setup;
  int dev = 0, n_sm = 0;
  cudaError_t e = setup.get(&dev, &n_sm, [](int) { return cudaSuccess; });
  if (e != cudaSuccess) return e;
  RopeParams rp{};
  const void* rows[5] = {r->q, r->k, r->v, r->idx_k, r->q_idx};
  const int64_t strides[5] = {r->q_stride, r->k_stride, r->v_stride, r->idx_k_stride, r->q_idx_stride};
  for (int i = 0; i < 5; ++i) {
    rp.rows[i] = rows[i];
    rp.stride[i] = strides[i];
  }
  rp.n_tokens = n_tokens;
  rp.n_pairs = r->q_idx ? 17 : 13;
  rp.cos_sin = cos_sin;
  rp.max_pos = max_pos;
  rp.rot = rot;
  rp.interleaved = interleaved;
  rp.positions = positions;
  rp.slot_mapping = slot_mapping;
  rp.kv_pool = static_cast<uint8_t*>(c->kv_pool);
  rp.idx_pool = static_cast<uint8_t*>(c->idx_pool);
  rp.n_pages = c->n_pages;
  rp.s_enc_k = c->s_enc_k;
  rp.s_enc_v = c->s_enc_v;
  rp.q8 = q8;
  rp.qi8 = qi8;
  rp.status = c->status;
  const long long warps = (long long)n_tokens * rp.n_pairs;
  long long blocks = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (blocks > 8ll * n_sm) blocks = 8ll * n_sm;
  const dim3 grid((unsigned)blocks), block(kRopeThreads);
  if (r->dtype == MSA_DTYPE_F32) rotary_insert_kernel<float><<<grid, block, 0, stream>>>(rp);
  else if (r->dtype == MSA_DTYPE_BF16) rotary_insert_kernel<__nv_bfloat16><<<grid, block, 0, stream>>>(rp);
  else rotary_insert_kernel<__half><<<grid, block, 0, stream>>>(rp);
  return cudaGetLastError();
}

cudaError_t launch_rope_table_freqs(float* table, int max_pos, const double* freq, int rot, double amplitude,
                                    cudaStream_t stream) {
  if (max_pos == 0 || rot == 0) return cudaSuccess;
  FreqParams f{};
  for (int i = 0; i < rot / 2; ++i) f.freq[i] = freq[i];
  const long long n = (long long)max_pos * (rot / 2);
  rope_table_freqs_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(table, max_pos, rot / 2, f, amplitude);
  return cudaGetLastError();
}

}  // namespace msa
