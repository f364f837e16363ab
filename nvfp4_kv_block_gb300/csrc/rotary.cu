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
// Eight lanes take one head row, each two chunks of 8 channels: with half pairs
// lane l < rot / 16 the chunks l and l + rot / 16, partners of each other, with
// interleaved pairs and unturned channels the chunks 2 l and 2 l + 1; so a
// rotation needs no other lane and each cos and sin is loaded once for both
// chunks.  A warp takes one head of a tile of tokens, four at a time, and keeps
// the tile's scale bytes in shared memory: a group's scales of consecutive tokens
// are consecutive bytes of the page, so a tile of tokens in page order leaves as
// whole sectors and not byte by byte.
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
  int n_rows;              // head rows of a token: 33, 25 without index queries
  int tile;                // tokens of a warp's tile (a multiple of 4, at most 32)
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
// Eight channels as they lie in memory (loaded ahead of their turn) and as floats.
template <typename T>
struct Chunk {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = ld_stream_v4(reinterpret_cast<const uint4*>(p) + i);
  }
};
__device__ __forceinline__ void to_floats(const Chunk<float>& c, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(c.v[i].x);
    x[4 * i + 1] = __uint_as_float(c.v[i].y);
    x[4 * i + 2] = __uint_as_float(c.v[i].z);
    x[4 * i + 3] = __uint_as_float(c.v[i].w);
  }
}
__device__ __forceinline__ void to_floats(const Chunk<__nv_bfloat16>& c, float (&x)[8]) {
  const uint32_t w[4] = {c.v[0].x, c.v[0].y, c.v[0].z, c.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void to_floats(const Chunk<__half>& c, float (&x)[8]) {
  const uint32_t w[4] = {c.v[0].x, c.v[0].y, c.v[0].z, c.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Eight E4M3 bytes (RNE, satfinite, zeros as 0x00: a byte's sign stays where its
// seven magnitude bits carry into bit 7), channel order.
__device__ __forceinline__ uint2 to_fp8x8(const float (&x)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t b = f32x2_to_e4m3x2(x[4 * h], x[4 * h + 1]) | (f32x2_to_e4m3x2(x[4 * h + 2], x[4 * h + 3]) << 16);
    w[h] = b & (((b & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | 0x7F7F7F7Fu);
  }
  return make_uint2(w[0], w[1]);
}

// Code word (8 channels) of finite x under the scale sb.  A code is the E2M1
// rounding (to nearest even, saturating) of y / sb, y = fl(x s_enc), and the
// hardware rounds an fp32 quotient.  The quotient must only not move onto or off a
// midpoint: y = mid sb (exact in fp32) has to give mid, and any other y lies at
// least an ulp of y away, more than half an ulp of mid, so the correctly rounded
// quotient is on the same side.  It is q + r (y - q sb) with q = y r, r the rounded
// reciprocal of sb (P. Markstein, 1990); a remainder that underflows belongs to a
// quotient far below the first midpoint.  inv: r, 0 for sb = 0.  The insert kernel
// compares y with every midpoint: five times the instructions.
__device__ __forceinline__ uint32_t code_word(const float (&x)[8], float s_enc, float sb, float inv) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __fmul_rn(x[i], s_enc), q0 = __fmul_rn(y, inv);
    q[i] = __fmaf_rn(__fmaf_rn(-q0, sb, y), inv, q0);
  }
  uint32_t n;  // nibble i: code of channel i
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(n)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  const uint32_t m = n & 0x77777777u;
  const uint32_t sg = (n & (m + 0x77777777u) & 0x88888888u) >> 3;  // signs of codes that are not zero, at bit 4 i
  // sign of channel i < 4 to bit 8 i + 7, of channel 4 + i to bit 8 i + 3
  uint32_t lo = sg & 0x1111u, hi = sg >> 16;
  lo = (lo | (lo << 8)) & 0x00110011u;
  lo = (lo | (lo << 4)) & 0x01010101u;
  hi = (hi | (hi << 8)) & 0x00110011u;
  hi = (hi | (hi << 4)) & 0x01010101u;
  return m | (lo << 7) | (hi << 3);
}
// Values that are none, for code_word: NaN has the code 0, what is beyond `most` the largest.
__device__ __forceinline__ void make_finite(float (&x)[8], float most) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -most), most) : 0.f;
}
// Largest magnitude (fmaxf drops NaN, as the insert kernel's does); `all` keeps NaN.
__device__ __forceinline__ float max_abs(const float (&x)[8], float& all) {
  float a = 0.f, n = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a = fmaxf(a, fabsf(x[i]));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(n) : "f"(fabsf(x[i])));
  }
  all = n;
  return a;
}
// (a, b) turned by c and s: two products and a sum, each rounded on its own.  (Not as packed
// pairs: the compiler joins a packed product and sum to one rounding.)
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

template <typename T>
__global__ void __launch_bounds__(kRopeThreads, 3) rotary_insert_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(8) uint8_t s_scales[kRopeThreads / 32][32 * 8];  // [warp][token][group]
  const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3;
  uint8_t* scales = s_scales[threadIdx.x >> 5];
  const long long n_jobs = (long long)((p.n_tokens + p.tile - 1) / p.tile) * p.n_rows;
  const long long warp0 = ((long long)blockIdx.x * kRopeThreads + threadIdx.x) >> 5;
  const long long n_warps = ((long long)gridDim.x * kRopeThreads) >> 5;
  const int half = p.rot >> 1;
  for (long long job = warp0; job < n_jobs; job += n_warps) {
    // rows of a token in job order: 16 q, 4 k, 4 v, idx_k, 8 q_idx
    const int t0 = (int)(job / p.n_rows) * p.tile, cnt = min(p.tile, p.n_tokens - t0), row = (int)(job % p.n_rows);
    const int kind = row < 16 ? 0 : row < 20 ? 1 : row < 24 ? 2 : row == 24 ? 3 : 4;
    const int head = kind == 0 ? row : kind == 1 ? row - 16 : kind == 2 ? row - 20 : kind == 4 ? row - 25 : 0;
    const bool cached = kind >= 1 && kind <= 3;
    const int my_pos = lane < cnt && p.rot > 0 ? p.positions[t0 + lane] : 0;
    int64_t my_slot = lane < cnt && cached ? p.slot_mapping[t0 + lane] : -1;
    if (my_slot >= 0 && (my_slot >> 7) >= p.n_pages) {
      set_status(p.status, MSA_STATUS_BAD_SLOT);
      my_slot = -1;
    }
    if (row == 0 && p.rot > 0 && (my_pos < 0 || my_pos >= p.max_pos)) set_status(p.status, MSA_STATUS_BAD_SEQ);
    // half pairs: lanes below h have partner chunks h apart (values are not turned)
    const int h = p.interleaved || kind == 2 ? 0 : p.rot >> 4;
    const int ca = l < h ? l : 2 * l, cb = l < h ? l + h : 2 * l + 1;
    const bool turns = kind != 2 && (p.interleaved ? 16 * l < p.rot : l < h);
    const T* src = static_cast<const T*>(p.rows[kind]) + (size_t)t0 * p.stride[kind] + head * kHeadDim;
    const size_t stride = p.stride[kind];
    Chunk<T> na = {}, nb = {};  // of the next four tokens
    if (sub < cnt) {
      na.load(src + sub * stride + 8 * ca);
      nb.load(src + sub * stride + 8 * cb);
    }
    for (int i0 = 0; i0 < cnt; i0 += 4) {
      const int i = i0 + sub, t = t0 + i;
      const int pos = __shfl_sync(0xffffffffu, my_pos, i & 31);
      const int64_t slot = __shfl_sync(0xffffffffu, my_slot, i & 31);
      const bool live = i < cnt;
      float a[8], b[8];
      to_floats(na, a);
      to_floats(nb, b);
      if (i + 4 < cnt) {
        na.load(src + (i + 4) * stride + 8 * ca);
        nb.load(src + (i + 4) * stride + 8 * cb);
      }
      if (live && turns && pos >= 0 && pos < p.max_pos) {
        const float* cs = p.cos_sin + (size_t)pos * p.rot + 8 * l;
        float c[8], s[8];
        load8(cs, c);
        load8(cs + half, s);
        if (h) {
#pragma unroll
          for (int u = 0; u < 8; ++u) turn(a[u], b[u], c[u], s[u]);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            turn(a[2 * u], a[2 * u + 1], c[u], s[u]);
            turn(b[2 * u], b[2 * u + 1], c[4 + u], s[4 + u]);
          }
        }
      }
      if (!cached) {
        if (live) {
          uint8_t* dst = kind == 0 ? p.q8 + ((size_t)t * kQHeads + head) * kHeadDim
                                   : p.qi8 + ((size_t)t * kIdxHeads + head) * kIdxDim;
          *reinterpret_cast<uint2*>(dst + 8 * ca) = to_fp8x8(a);
          *reinterpret_cast<uint2*>(dst + 8 * cb) = to_fp8x8(b);
        }
        continue;
      }
      // maxima of the two 16-channel groups: the other chunk of group c / 2 is c ^ 1
      float all_a, all_b;
      const float ma = max_abs(a, all_a), mb = max_abs(b, all_b);
      float ga = fmaxf(ma, mb), gb = ga;
      if (h) {
        const int xa = ca ^ 1, xb = cb ^ 1;  // (of lanes below h: held by lane c or c - h)
        const int la = l < h ? (lane & 24) | (xa < h ? xa : xa - h) : lane, lb = l < h ? (lane & 24) | (xb < h ? xb : xb - h) : lane;
        const float a1 = __shfl_sync(0xffffffffu, ma, la), a2 = __shfl_sync(0xffffffffu, mb, la);
        const float b1 = __shfl_sync(0xffffffffu, ma, lb), b2 = __shfl_sync(0xffffffffu, mb, lb);
        if (l < h) {
          ga = fmaxf(ma, xa < h ? a1 : a2);
          gb = fmaxf(mb, xb < h ? b1 : b2);
        }
      }
      if (!live || slot < 0) continue;
      const int off = (int)(slot & 127);
      if (kind == 3) {
        uint8_t* dst = p.idx_pool + (size_t)(slot >> 7) * kIdxPageBytes + off * kIdxDim;
        *reinterpret_cast<uint2*>(dst + (((ca >> 1) ^ (off & 7)) << 4) + 8 * (ca & 1)) = to_fp8x8(a);
        *reinterpret_cast<uint2*>(dst + (((cb >> 1) ^ (off & 7)) << 4) + 8 * (cb & 1)) = to_fp8x8(b);
        continue;
      }
      const float s_enc = kind == 1 ? p.s_enc_k : p.s_enc_v;
      const uint32_t sa = f32_to_e4m3(__fmul_rn(__fdiv_rn(ga, 6.0f), s_enc));
      const uint32_t sb = f32_to_e4m3(__fmul_rn(__fdiv_rn(gb, 6.0f), s_enc));
      uint8_t* codes = p.kv_pool + (size_t)(slot >> 7) * kKvPageBytes + head * kHeadBytes + (kind == 1 ? kOffKc : kOffVc) + off * 64;
      const float fa = e4m3_to_f32(sa), fb = e4m3_to_f32(sb);
      if (!(fmaxf(all_a, all_b) * s_enc < 1e30f) || all_a != all_a || all_b != all_b) {
        const float most = fminf(1e30f / s_enc, 3e38f);
        make_finite(a, most);
        make_finite(b, most);
      }
      const uint32_t wa = code_word(a, s_enc, fa, fa > 0.f ? __frcp_rn(fa) : 0.f);
      const uint32_t wb = code_word(b, s_enc, fb, fb > 0.f ? __frcp_rn(fb) : 0.f);
      *reinterpret_cast<uint32_t*>(codes + (code_chunk_pos(ca >> 2, off) << 4) + 4 * (ca & 3)) = wa;
      *reinterpret_cast<uint32_t*>(codes + (code_chunk_pos(cb >> 2, off) << 4) + 4 * (cb & 3)) = wb;
      if ((ca & 1) == 0) scales[i * 8 + (ca >> 1)] = (uint8_t)sa;
      if ((cb & 1) == 0) scales[i * 8 + (cb >> 1)] = (uint8_t)sb;
    }
    if (kind == 1 || kind == 2) {  // lane = token: its eight scale bytes
      __syncwarp();
      if (my_slot >= 0) {
        const uint2 sc = *reinterpret_cast<const uint2*>(scales + 8 * lane);
        uint8_t* dst = p.kv_pool + (size_t)(my_slot >> 7) * kKvPageBytes + head * kHeadBytes +
                       (kind == 1 ? kOffKs : kOffVs) + (my_slot & 127);
#pragma unroll
        for (int g = 0; g < 8; ++g) dst[g * kPageTokens] = (uint8_t)((g < 4 ? sc.x : sc.y) >> (8 * (g & 3)));
      }
      __syncwarp();
    }
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
  rp.n_rows = r->q_idx ? 33 : 25;
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
  // the largest tile that still makes 48 warps per SM
  rp.tile = 32;
  while (rp.tile > 4 && (long long)n_tokens / rp.tile * rp.n_rows < 48ll * n_sm) rp.tile >>= 1;
  const long long warps = ((long long)n_tokens + rp.tile - 1) / rp.tile * rp.n_rows;
  long long blocks = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (blocks > 64ll * n_sm) blocks = 64ll * n_sm;
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
