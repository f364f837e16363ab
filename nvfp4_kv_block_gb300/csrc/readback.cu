// Read-back of cache slots: the K, V and index-key values that the cache holds,
// in 32 or 16 bits, one row per slot.
//
// An NVFP4 element is x = e2m1(code) * d with d = fl(sb * r), sb the E4M3 scale
// of its 16 channels and r = fl(1 / s_enc) the tensor's decode factor; the
// product is rounded to fp32 and then to the output type.  Index keys are E4M3
// values.  704 bytes in and 1,152 values out per token.  Whole pages are bound by memory
// (131,072 tokens in bf16: 74 us, 5.3 TB/s of those bytes), scattered slots by latency, a
// chain of slot, scales, codes and store with no rate near its end (20,011 tokens in fp32:
// 23 us, 4.6 TB/s, DRAM at 25 % and issue slots at 29 %; 16,384 in bf16: 18 us, 2.7 TB/s).
// A programmatic dependent, as the rotary insert (2 us less a call, one after the other).
//
// A warp takes one KV head's K or V (or the index key) of a tile of tokens, four
// tokens at a time: eight lanes a row, lane l its channels 16l .. 16l + 15: two
// code words, one scale, two or four 16-byte stores.  The tile's scale bytes are
// loaded first, lane = token (a group's scales of consecutive tokens are
// consecutive bytes of the page), and handed out by shuffles.
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
  int wide;  // outputs on 32-byte boundaries: 32-byte stores
  int tile;  // tokens of a warp's tile (a multiple of 4, at most 32)
  float dec_k, dec_v;
  void* k;    // [n_tokens][4][128] or null
  void* v;    // [n_tokens][4][128] or null
  void* idx;  // [n_tokens][128] or null
  int* status;
};

// 32 bytes as one store (a whole sector per lane) or two (20,011 tokens in fp32: 25 us, 31 in two).
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void store16(float* p, const float (&x)[16], bool wide) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[8 * h + i]);
    store32(p + 8 * h, w, wide);
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  store32(p, w, wide);
}
__device__ __forceinline__ void store16(__half* p, const float (&x)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 b = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  store32(p, w, wide);
}

// Values of the eight E2M1 codes of a code word, times d.  An E2M1 magnitude as
// f16 has a zero low byte, so a byte permute of eight constants by the
// magnitudes gives four high bytes at a time; the signs are merged in place.
__device__ __forceinline__ void decode_word(uint32_t w, float d, float* x) {
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
__global__ void __launch_bounds__(kReadThreads) read_kv_kernel(const __grid_constant__ ReadParams p) {
  const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3;
  pdl_wait();
  pdl_trigger();
  const long long n_jobs = (long long)((p.n_tokens + p.tile - 1) / p.tile) * 9;
  const long long job0 = ((long long)blockIdx.x * kReadThreads + threadIdx.x) >> 5;
  const long long step = ((long long)gridDim.x * kReadThreads) >> 5;
  for (long long job = job0; job < n_jobs; job += step) {
    const int t0 = (int)(job / 9) * p.tile, cnt = min(p.tile, p.n_tokens - t0), row = (int)(job % 9);
    int64_t my_slot = lane < cnt ? p.slot_mapping[t0 + lane] : -1;
    if (my_slot >= 0 && (my_slot >> 7) >= p.n_pages) {
      set_status(p.status, MSA_STATUS_BAD_SLOT);
      my_slot = -1;
    }
    if (row == 8) {
      if (!p.idx) continue;
      T* dst = static_cast<T*>(p.idx) + (size_t)t0 * kIdxDim + 16 * l;
#pragma unroll 4
      for (int i0 = 0; i0 < cnt; i0 += 4) {
        const int i = i0 + sub;
        const int64_t slot = __shfl_sync(0xffffffffu, my_slot, i & 31);
        const int off = (int)(slot & 127);
        if (i >= cnt || slot < 0) continue;
        const uint4 b = ld_stream_v4(p.idx_pool + (size_t)(slot >> 7) * kIdxPageBytes + off * kIdxDim + ((l ^ (off & 7)) << 4));
        const uint32_t w[4] = {b.x, b.y, b.z, b.w};
        float x[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = e4m3_to_f32(w[c >> 2] >> (8 * (c & 3)));
        store16(dst + (size_t)i * kIdxDim, x, p.wide);
      }
      continue;
    }
    const bool is_v = row >= 4;
    void* out = is_v ? p.v : p.k;
    if (!out) continue;
    const int head = row & 3;
    const float dec = is_v ? p.dec_v : p.dec_k;
    const uint8_t* hb = p.kv_pool + head * kHeadBytes + (is_v ? kOffVc : kOffKc);
    uint32_t sc[2] = {0, 0};  // lane = token: its eight scale bytes
    if (my_slot >= 0) {
      const uint8_t* s = hb + (size_t)(my_slot >> 7) * kKvPageBytes + (kOffKs - kOffKc) + (my_slot & 127);
#pragma unroll
      for (int g = 0; g < 8; ++g) sc[g >> 2] |= (uint32_t)__ldg(s + g * kPageTokens) << (8 * (g & 3));
    }
    T* dst = static_cast<T*>(out) + ((size_t)t0 * kKvHeads + head) * kHeadDim + 16 * l;
#pragma unroll 4
    for (int i0 = 0; i0 < cnt; i0 += 4) {
      const int i = i0 + sub;
      const int64_t slot = __shfl_sync(0xffffffffu, my_slot, i & 31);
      const uint32_t s0 = __shfl_sync(0xffffffffu, sc[0], i & 31), s1 = __shfl_sync(0xffffffffu, sc[1], i & 31);
      const int off = (int)(slot & 127);
      if (i >= cnt || slot < 0) continue;
      const uint2 w = ld_stream_v2(hb + (size_t)(slot >> 7) * kKvPageBytes + off * 64 + (code_chunk_pos(l >> 1, off) << 4) + 8 * (l & 1));
      const float d = __fmul_rn(e4m3_to_f32(((l & 4) ? s1 : s0) >> (8 * (l & 3))), dec);
      float x[16];
      decode_word(w.x, d, x);
      decode_word(w.y, d, x + 8);
      store16(dst + (size_t)i * kKvHeads * kHeadDim, x, p.wide);
    }
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
  // the largest tile that still makes 48 warps per SM: longer tiles share the loads of their
  // scales, short ones fill the SMs (single calls on a cold L2: 131,072 tokens in pages 78 us with
  // 32, 82 with 16, 86 with 8, 100 with 4; 300 tokens 8 us with 4, 12 with 32)
  int tile = 32;
  while (tile > 4 && (long long)n_tokens / tile * 9 < 48ll * n_sm) tile >>= 1;
  const int wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(idx)) & 31) == 0;
  const ReadParams rp{static_cast<const uint8_t*>(c->kv_pool), static_cast<const uint8_t*>(c->idx_pool), c->n_pages,
                      slot_mapping, n_tokens, wide, tile, 1.0f / c->s_enc_k, 1.0f / c->s_enc_v, k, v, idx, c->status};
  const long long warps = ((long long)n_tokens + tile - 1) / tile * 9;
  long long blocks = (warps + kReadThreads / 32 - 1) / (kReadThreads / 32);
  if (blocks > 64ll * n_sm) blocks = 64ll * n_sm;
  const dim3 grid((unsigned)blocks), block(kReadThreads);
  return launch_pdl(dtype == MSA_DTYPE_F32 ? read_kv_kernel<float> : dtype == MSA_DTYPE_BF16 ? read_kv_kernel<__nv_bfloat16> : read_kv_kernel<__half>,
                    grid, block, 0, stream, rp);
}

}  // namespace msa
