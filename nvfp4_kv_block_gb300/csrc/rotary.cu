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
// A warp takes a part (four heads, or the index key) of four tokens: one bulk copy
// per token brings its 1,024 bytes to shared memory, so that 4 KB per warp are on
// their way without a register for them.  Eight lanes take one head row, each two
// chunks of 8 channels: with half pairs lane l < rot / 16 the chunks l and l + rot / 16,
// partners of each other, with interleaved pairs and unturned channels the chunks 2 l
// and 2 l + 1; so a rotation needs no other lane, and a token's cos and sin are
// loaded once for the part's heads.  The scale bytes of the four tokens wait in
// shared memory: a group's scales of consecutive tokens are consecutive bytes of the
// page, and leave together.  8,192 bf16 tokens: 25 us, 4.1 TB/s of the bytes above; 16,384
// fp32 tokens at scattered slots: 62 us, 5.5 TB/s.  As a programmatic dependent of the kernel before
// it, which lets the next one begin launching (memory is touched behind pdl_wait only): with the
// read-back behind it 29.8 us a pass, 33.3 with plain launches.  Positions on several axes cost an
// int32 a token and axis more, and table rows of which a pair reads its own: 8,185 fp16 tokens (slices) on three
// axes, dealt pair by pair, and the read-back 31.9 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"

namespace msa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kPartHeads = 4;  // heads of a warp's part
constexpr int kTile = 4;       // its tokens
static_assert(kPartHeads == kKvHeads && kTile == 4, "the parts of a token, and a lane per (head, group)");

struct RopeParams {
  const void* rows[5];     // q, k, v, idx_k, q_idx (may be null)
  long long stride[5];     // elements from one token's rows to the next
  int n_tokens;
  unsigned long long wait_ns;
  const float* cos_sin;    // [max_pos][rot]: cos of the rot / 2 pairs, then their sin
  int max_pos;
  int rot;
  int interleaved;
  const int* positions;  // [n_axes][n_tokens]
  int n_axes;
  uint32_t axes[4];      // axis of pair i: bits 2 (i % 16) and up of word i / 16
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
// Eight channels as they lie in memory and as floats.
template <typename T>
struct Chunk {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ Chunk(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
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
// Largest magnitude without NaN, as the insert kernel takes it; `fine` if all values
// are finite and their products with s_enc far from overflow.
__device__ __forceinline__ float max_abs(const float (&x)[8], float s_enc, bool& fine) {
  float n = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(n) : "f"(fabsf(x[i])));
  fine = n * s_enc < 1e30f;
  if (fine) return n;
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
  return a;
}
// fl(a / 6): q + r (a - 6 q), q = a r, r = fl(1 / 6) (P. Markstein, 1990), away from the
// ends of the range.
__device__ __forceinline__ float sixth(float a) {
  if (!(a > 1e-30f && a < 1e36f)) return __fdiv_rn(a, 6.0f);
  constexpr float r = 1.0f / 6.0f;
  const float q = __fmul_rn(a, r);
  return __fmaf_rn(__fmaf_rn(-q, 6.0f, a), r, q);
}
// (a, b) turned by c and s: two products and a sum, each rounded on its own.  (Not as packed
// pairs: the compiler joins a packed product and sum to one rounding.)
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// kAxes: a pair turns by the table row of its own axis's position (axis 0 for every pair otherwise).
// A lane's eight pairs mostly share an axis (sections of 8 pairs and more): one row's loads; where
// they do not, it takes the pairs from each axis's row.
template <typename T, bool kAxes>
__global__ void __launch_bounds__(kRopeThreads, 6) rotary_insert_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPart = kPartHeads * kHeadDim * sizeof(T);  // bytes of a token's part
  constexpr int kWarps = kRopeThreads / 32;
  __shared__ __align__(128) uint8_t s_rows[kWarps][kTile * kPart];
  __shared__ __align__(4) uint8_t s_scales[kWarps][kPartHeads * 8 * kTile];  // [warp][head][group][token]
  __shared__ float s_inv[128];  // fl(1 / sb) of a scale byte, 0 for the scale 0
  __shared__ __align__(8) uint64_t s_bar[kWarps];
  __shared__ int s_abort;
  const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3, warp = threadIdx.x >> 5;
  const uint32_t bar = smem_u32(&s_bar[warp]);
  // part: 0 keys, 1 values, 2-5 queries, 6 index key, 7-8 index queries (the longest first)
  const int part = blockIdx.y, kind = part == 0 ? 1 : part == 1 ? 2 : part < 6 ? 0 : part == 6 ? 3 : 4;
  const bool cached = kind >= 1 && kind <= 3;
  if (threadIdx.x < 128) s_inv[threadIdx.x] = threadIdx.x ? __frcp_rn(e4m3_to_f32(threadIdx.x)) : 0.f;
  if (lane == 0) {
    mbar_init(bar, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int head0 = kind == 0 ? 4 * (part - 2) : kind == 4 ? 4 * (part - 7) : 0, heads = kind == 3 ? 1 : kPartHeads;
  const uint32_t bytes = heads * kHeadDim * sizeof(T);
  int phase = 0;
  for (int t0 = ((int)blockIdx.x * kWarps + warp) * kTile, more = 1; t0 < p.n_tokens && more;
       t0 += (int)gridDim.x * kWarps * kTile, phase ^= 1, more = sizeof(T) == 4) {
    const int cnt = min(kTile, p.n_tokens - t0);
    __syncwarp();  // the last tile is read
    if (lane == 0) mbar_arrive_expect_tx(bar, cnt * bytes);
    __syncwarp();
    if (lane < cnt)
      bulk_g2s(smem_u32(s_rows[warp]) + lane * kPart,
               static_cast<const T*>(p.rows[kind]) + (size_t)(t0 + lane) * p.stride[kind] + head0 * kHeadDim, bytes, bar);
    // lane = (token sub, part l of its rows)
    const bool live = sub < cnt;
    const int t = t0 + sub;
    int pos[kAxes ? 4 : 1];
    bool known = true;
#pragma unroll
    for (int a = 0; a < (kAxes ? 4 : 1); ++a) {
      pos[a] = live && p.rot > 0 && (!kAxes || a < p.n_axes) ? p.positions[(size_t)a * p.n_tokens + t] : 0;
      known &= pos[a] >= 0 && pos[a] < p.max_pos;
    }
    int64_t slot = live && cached ? p.slot_mapping[t] : -1;
    if (slot >= 0 && (slot >> 7) >= p.n_pages) {
      set_status(p.status, MSA_STATUS_BAD_SLOT);
      slot = -1;
    }
    if (part == 2 && p.rot > 0 && live && !known) set_status(p.status, MSA_STATUS_BAD_SEQ);
    // half pairs: lanes below h have partner chunks h apart (values are not turned)
    const int h = p.interleaved || kind == 2 ? 0 : p.rot >> 4;
    const int ca = l < h ? l : 2 * l, cb = l < h ? l + h : 2 * l + 1;
    const bool turned = live && known && kind != 2 && (p.interleaved ? 16 * l < p.rot : l < h);
    float c[8], s[8];
    if (turned) {
      if constexpr (kAxes) {
        const uint32_t mine = p.axes[l >> 1] >> (16 * (l & 1)) & 0xFFFFu, first = mine & 3;
        const float* cs = p.cos_sin + (size_t)(first < 2 ? (first ? pos[1] : pos[0]) : first == 2 ? pos[2] : pos[3]) * p.rot + 8 * l;
        load8(cs, c);
        load8(cs + (p.rot >> 1), s);
        if (mine != first * 0x5555u) {
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const uint32_t no = mine ^ (a * 0x5555u), is = ~(no | no >> 1) & 0x5555u;  // bit 2 u: pair u is of axis a
            if (is == 0 || a == (int)first) continue;
            float c1[8], s1[8];
            cs = p.cos_sin + (size_t)pos[a] * p.rot + 8 * l;
            load8(cs, c1);
            load8(cs + (p.rot >> 1), s1);
#pragma unroll
            for (int u = 0; u < 8; ++u)
              if (is >> (2 * u) & 1) {
                c[u] = c1[u];
                s[u] = s1[u];
              }
          }
        }
      } else {
        const float* cs = p.cos_sin + (size_t)pos[0] * p.rot + 8 * l;
        load8(cs, c);
        load8(cs + (p.rot >> 1), s);
      }
    }
    if (!__all_sync(0xffffffffu, mbar_wait(bar, phase, WaitCtl{&s_abort, p.wait_ns}))) {
      // nothing of the tile is written, and the copies in flight are waited for
      if (lane == 0) set_status(p.status, MSA_STATUS_TIMEOUT);
      mbar_wait_drain(bar, phase, drain_ns(p.wait_ns));
      return;
    }
    const uint8_t* ra = s_rows[warp] + sub * kPart + 8 * ca * sizeof(T);
    const uint8_t* rb = s_rows[warp] + sub * kPart + 8 * cb * sizeof(T);
    auto rows = [&](int hd, float (&a)[8], float (&b)[8]) {
      to_floats(Chunk<T>(ra + hd * kHeadDim * sizeof(T)), a);
      to_floats(Chunk<T>(rb + hd * kHeadDim * sizeof(T)), b);
      if (!turned) return;
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
    };
    if (!cached) {
      uint8_t* dst = (kind == 0 ? p.q8 + (size_t)t * kQHeads * kHeadDim : p.qi8 + (size_t)t * kIdxHeads * kIdxDim) + head0 * kHeadDim;
#pragma unroll 1
      for (int hd = 0; hd < kPartHeads; ++hd, dst += kHeadDim) {
        float a[8], b[8];
        rows(hd, a, b);
        if (live) {
          *reinterpret_cast<uint2*>(dst + 8 * ca) = to_fp8x8(a);
          *reinterpret_cast<uint2*>(dst + 8 * cb) = to_fp8x8(b);
        }
      }
      continue;
    }
    const int off = (int)(slot & 127);
    if (kind == 3) {
      float a[8], b[8];
      rows(0, a, b);
      if (slot >= 0) {
        uint8_t* dst = p.idx_pool + (size_t)(slot >> 7) * kIdxPageBytes + off * kIdxDim;
        *reinterpret_cast<uint2*>(dst + (((ca >> 1) ^ (off & 7)) << 4) + 8 * (ca & 1)) = to_fp8x8(a);
        *reinterpret_cast<uint2*>(dst + (((cb >> 1) ^ (off & 7)) << 4) + 8 * (cb & 1)) = to_fp8x8(b);
      }
      continue;
    }
    const float s_enc = kind == 1 ? p.s_enc_k : p.s_enc_v;
    uint8_t* head = p.kv_pool + (size_t)(slot >= 0 ? slot >> 7 : 0) * kKvPageBytes + (kind == 1 ? kOffKc : kOffVc);
    const int wa = off * 64 + (code_chunk_pos(ca >> 2, off) << 4) + 4 * (ca & 3);
    const int wb = off * 64 + (code_chunk_pos(cb >> 2, off) << 4) + 4 * (cb & 3);
    // the other chunk of a 16-channel group is c ^ 1; of lanes below h lane c or c - h has it
    const int xa = ca ^ 1, xb = cb ^ 1;
    const int la = (lane & 24) | (l >= h ? l : xa < h ? xa : xa - h), lb = (lane & 24) | (l >= h ? l : xb < h ? xb : xb - h);
    uint8_t* scales = s_scales[warp] + sub;
#pragma unroll 1
    for (int hd = 0; hd < kPartHeads; ++hd, head += kHeadBytes) {
      float a[8], b[8];
      rows(hd, a, b);
      bool fine_a, fine_b;
      const float ma = max_abs(a, s_enc, fine_a), mb = max_abs(b, s_enc, fine_b);
      float ga = fmaxf(ma, mb), gb = ga;
      if (h) {
        const float a1 = __shfl_sync(0xffffffffu, ma, la), a2 = __shfl_sync(0xffffffffu, mb, la);
        const float b1 = __shfl_sync(0xffffffffu, ma, lb), b2 = __shfl_sync(0xffffffffu, mb, lb);
        if (l < h) {
          ga = fmaxf(ma, xa < h ? a1 : a2);
          gb = fmaxf(mb, xb < h ? b1 : b2);
        }
      }
      if (!(fine_a && fine_b)) {
        const float most = fminf(1e30f / s_enc, 3e38f);
        make_finite(a, most);
        make_finite(b, most);
      }
      const uint32_t sa = f32_to_e4m3(__fmul_rn(sixth(ga), s_enc)), sb = f32_to_e4m3(__fmul_rn(sixth(gb), s_enc));
      const uint32_t va = code_word(a, s_enc, e4m3_to_f32(sa), s_inv[sa]), vb = code_word(b, s_enc, e4m3_to_f32(sb), s_inv[sb]);
      if (slot >= 0) {
        *reinterpret_cast<uint32_t*>(head + wa) = va;
        *reinterpret_cast<uint32_t*>(head + wb) = vb;
      }
      if ((ca & 1) == 0) scales[(hd * 8 + (ca >> 1)) * kTile] = (uint8_t)sa;
      if ((cb & 1) == 0) scales[(hd * 8 + (cb >> 1)) * kTile] = (uint8_t)sb;
    }
    // the scale bytes: lane = (head, group) of the four tokens, as one word where they are consecutive
    __syncwarp();
    const uint32_t word = reinterpret_cast<const uint32_t*>(s_scales[warp])[lane];
    const int64_t slot0 = __shfl_sync(0xffffffffu, slot, 0);
    const bool run = __all_sync(0xffffffffu, slot == slot0 + sub && (slot0 & 3) == 0);
    const size_t place = (size_t)(lane >> 3) * kHeadBytes + (kind == 1 ? kOffKs : kOffVs) + (lane & 7) * kPageTokens;
    if (run) {
      if (slot0 >= 0) *reinterpret_cast<uint32_t*>(p.kv_pool + (size_t)(slot0 >> 7) * kKvPageBytes + place + (slot0 & 127)) = word;
    } else {
#pragma unroll
      for (int i = 0; i < kTile; ++i) {
        const int64_t si = __shfl_sync(0xffffffffu, slot, 8 * i);
        if (si >= 0) p.kv_pool[(size_t)(si >> 7) * kKvPageBytes + place + (si & 127)] = (uint8_t)(word >> (8 * i));
      }
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
                                 int max_pos, int rot, int interleaved, const int* positions, int n_axes,
                                 const uint8_t* axis_of_pair, const int64_t* slot_mapping, uint8_t* q8, uint8_t* qi8, cudaStream_t stream) {
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
  rp.cos_sin = cos_sin;
  rp.max_pos = max_pos;
  rp.rot = rot;
  rp.interleaved = interleaved;
  rp.positions = positions;
  rp.n_axes = n_axes;
  for (int i = 0; axis_of_pair && i < rot / 2; ++i) rp.axes[i / 16] |= (uint32_t)axis_of_pair[i] << (2 * (i % 16));
  rp.slot_mapping = slot_mapping;
  rp.kv_pool = static_cast<uint8_t*>(c->kv_pool);
  rp.idx_pool = static_cast<uint8_t*>(c->idx_pool);
  rp.n_pages = c->n_pages;
  rp.s_enc_k = c->s_enc_k;
  rp.s_enc_v = c->s_enc_v;
  rp.q8 = q8;
  rp.qi8 = qi8;
  rp.status = c->status;
  rp.wait_ns = launch_settings().wait_ns;
  // tiles of a warp of fp32 rows: up to three while the grid still fills six CTAs per SM twice (16,384
  // tokens at scattered slots: 62 us, 66 with one).  One of 16-bit rows (16,384 tokens: 41.6 us, 42.7
  // with three).
  const int per_block = kRopeThreads / 32 * kTile, parts = r->q_idx ? 9 : 7;
  const long long blocks = ((long long)n_tokens + per_block - 1) / per_block;
  const long long tiles = r->dtype == MSA_DTYPE_F32 ? std::min(3ll, std::max(1ll, blocks * parts / (12ll * n_sm))) : 1;
  const dim3 grid((unsigned)((blocks + tiles - 1) / tiles), parts), block(kRopeThreads);
  const bool axes = n_axes > 1;
  auto launch = [&](auto zero) {
    using T = decltype(zero);
    return launch_pdl(axes ? rotary_insert_kernel<T, true> : rotary_insert_kernel<T, false>, grid, block, 0, stream, rp);
  };
  return r->dtype == MSA_DTYPE_F32 ? launch(0.f) : r->dtype == MSA_DTYPE_BF16 ? launch(__nv_bfloat16{}) : launch(__half{});
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
