// Read-back of cache slots: the K, V and index-key values that the cache holds,
// in 32 or 16 bits, one row per slot.
//
// An NVFP4 element is x = e2m1(code) * d with d = fl(sb * r), sb the E4M3 scale
// of its 16 channels and r = fl(1 / s_enc) the tensor's decode factor; the
// product is rounded to fp32 and then to the output type.  Index keys are E4M3
// values.  Memory-bound: 704 bytes in and 1,152 values out per token.
//
// One half-warp takes one row (a KV head's K or V, or the index key), lane l
// its channels 8l .. 8l + 7: one 32-bit code word, one scale byte (shared by
// two lanes), one or two 16-byte stores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace msa {
namespace {

constexpr int kReadThreads = 256;

struct ReadParams {
  const uint8_t* kv_pool;
  const uint8_t* idx_pool;
  int64_t n_pages;
  const int64_t* slot_mapping;
  int n_tokens;
  float dec_k, dec_v;
  void* k;    // [n_tokens][4][128] or null
  void* v;    // [n_tokens][4][128] or null
  void* idx;  // [n_tokens][128] or null
  int* status;
};

__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 b = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Values of the eight E2M1 codes of a code word, times d.  An E2M1 magnitude as
// f16 has a zero low byte, so a byte permute of eight constants by the
// magnitudes gives four high bytes at a time; the signs are merged in place.
__device__ __forceinline__ void decode_word(uint32_t w, float d, float (&x)[8]) {
  const uint32_t m = w & 0x77777777u;
  const uint32_t h0 = prmt(0x3E3C3800u, 0x46444240u, m) | (w & 0x80808080u);
  const uint32_t h1 = prmt(0x3E3C3800u, 0x46444240u, m >> 16) | ((w << 4) & 0x80808080u);
  const uint32_t pairs[4] = {prmt(h0, 0, 0x1404u), prmt(h0, 0, 0x3424u), prmt(h1, 0, 0x1404u), prmt(h1, 0, 0x3424u)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&pairs[i]));
    x[2 * i] = __fmul_rn(f.x, d);
    x[2 * i + 1] = __fmul_rn(f.y, d);
  }
}

template <typename T>
__global__ void __launch_bounds__(kReadThreads) read_kv_kernel(ReadParams p) {
  const int l = threadIdx.x & 15;
  const long long n_jobs = (long long)p.n_tokens * 9;
  const long long job0 = ((long long)blockIdx.x * kReadThreads + threadIdx.x) >> 4;
  const long long step = ((long long)gridDim.x * kReadThreads) >> 4;
  for (long long job = job0; job < n_jobs; job += step) {
    const int t = (int)(job / 9), row = (int)(job % 9);
    const int64_t slot = p.slot_mapping[t];
    if (slot < 0) continue;
    const int64_t page = slot >> 7;
    const int off = (int)(slot & 127);
    if (page >= p.n_pages) {
      if (l == 0) set_status(p.status, MSA_STATUS_BAD_SLOT);
      continue;
    }
    float x[8];
    T* dst;
    if (row == 8) {
      if (!p.idx) continue;
      const uint8_t* src = p.idx_pool + (size_t)page * kIdxPageBytes + off * kIdxDim;
      const uint2 b = ld_stream_v2(src + (((l >> 1) ^ (off & 7)) << 4) + 8 * (l & 1));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = e4m3_to_f32(b.x >> (8 * i));
        x[4 + i] = e4m3_to_f32(b.y >> (8 * i));
      }
      dst = static_cast<T*>(p.idx) + (size_t)t * kIdxDim;
    } else {
      const bool is_v = row >= 4;
      void* out = is_v ? p.v : p.k;
      if (!out) continue;
      const int head = row & 3;
      const uint8_t* hb = p.kv_pool + (size_t)page * kKvPageBytes + head * kHeadBytes;
      const uint32_t w = ld_stream_u32(hb + (is_v ? kOffVc : kOffKc) + off * 64 + (code_chunk_pos(l >> 2, off) << 4) + 4 * (l & 3));
      const uint8_t sb = __ldg(hb + (is_v ? kOffVs : kOffKs) + (l >> 1) * kPageTokens + off);
      decode_word(w, __fmul_rn(e4m3_to_f32(sb), is_v ? p.dec_v : p.dec_k), x);
      dst = static_cast<T*>(out) + ((size_t)t * kKvHeads + head) * kHeadDim;
    }
    store8(dst + 8 * l, x);
  }
}

}  // namespace

cudaError_t launch_read_kv(const msa_cache* c, const int64_t* slot_mapping, int n_tokens, int dtype, void* k, void* v,
                           void* idx, cudaStream_t stream) {
  if (n_tokens == 0 || (!k && !v && !idx)) return cudaSuccess;
  static DeviceSetup setup;
  int dev = 0, n_sm = 0;
  cudaError_t e = setup.get(&dev, &n_sm, [](int) { return cudaSuccess; });
  if (e != cudaSuccess) return e;
  const ReadParams rp{static_cast<const uint8_t*>(c->kv_pool), static_cast<const uint8_t*>(c->idx_pool), c->n_pages,
                      slot_mapping, n_tokens, 1.0f / c->s_enc_k, 1.0f / c->s_enc_v, k, v, idx, c->status};
  long long blocks = ((long long)n_tokens * 9 + kReadThreads / 16 - 1) / (kReadThreads / 16);
  if (blocks > 8ll * n_sm) blocks = 8ll * n_sm;
  const dim3 grid((unsigned)blocks), block(kReadThreads);
  if (dtype == MSA_DTYPE_F32) read_kv_kernel<float><<<grid, block, 0, stream>>>(rp);
  else if (dtype == MSA_DTYPE_BF16) read_kv_kernel<__nv_bfloat16><<<grid, block, 0, stream>>>(rp);
  else read_kv_kernel<__half><<<grid, block, 0, stream>>>(rp);
  return cudaGetLastError();
}

}  // namespace msa
